import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line(
        "markers", "gpu: needs a CUDA GPU (sm_103a) and the built library")


def pytest_collection_modifyitems(items):
    # the cost model's tests compare times, which another process can disturb:
    # they come behind the tests of results, so that under -x they hide none
    # (test_zz_no_alloc wants to be last)
    order = {"test_gpu_costmodel": 1, "test_zz_no_alloc": 2}
    items.sort(key=lambda i: order.get(i.path.stem, 0))


@pytest.fixture(scope="session")
def golden():
    import json
    with open(os.path.join(ROOT, "tests", "golden", "closed_forms.json")) as f:
        return json.load(f)
