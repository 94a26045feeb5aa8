"""The head's cross entropy and the clipping of gradients where something goes wrong or
stands close: waits that run out, guards around outputs and workspaces, the checked
build."""
import time

import pytest
import torch

import dsmem_thread_block_gb300 as credit
from dsmem_thread_block_gb300 import _credit as C
from test_gpu_linear_ce import make

pytestmark = pytest.mark.gpu


def test_a_tile_that_gives_up_waits_for_its_copies_and_no_longer():
    # Two tiles, each with one wait that runs out after a second.  The copies that were
    # issued are there long before, so waiting for them takes no time: a second limit
    # spent on a stage whose other operand never comes would make four seconds.
    dev = torch.cuda.current_device()
    h, w, target = make(300, 64, 500, torch.bfloat16)
    want = credit.linear_cross_entropy_forward(h, w, target)
    assert C.credit_get_device_error(dev) == C.OK
    t0 = time.perf_counter()
    assert C.credit_selftest_tile_timeout(dev) == C.ERR_DEVICE_TIMEOUT
    took = time.perf_counter() - t0
    assert 2.0 <= took < 3.5, took
    assert C.credit_get_device_error(dev) == C.OK
    got = credit.linear_cross_entropy_forward(h, w, target)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
