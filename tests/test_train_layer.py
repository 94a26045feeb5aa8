"""The training operators' Python layer without a GPU: importing the package,
`Dropout` objects, the build of the torch layer, and refusals on the host."""
import os
import subprocess
import sys

import pytest
import torch

import dsmem_thread_block_gb300 as credit
from dsmem_thread_block_gb300 import build as B
from dsmem_thread_block_gb300 import train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    B.build_torch()


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_star_import_needs_neither_torch_nor_its_layer():
    # the names are there before anything is built; the first call asks for it
    r = python("""
import sys
sys.modules["torch"] = None  # not installed
from dsmem_thread_block_gb300 import build
build.TORCH_LIB = "/nowhere/credit_train_torch.so"
from dsmem_thread_block_gb300 import *
print(callable(layernorm_forward), Dropout(0.1, 1).p)
""")
    assert r.returncode == 0 and r.stdout.split() == ["True", "0.1"], r.stderr


def test_a_missing_torch_layer_raises_at_the_first_call():
    r = python("""
from dsmem_thread_block_gb300 import build
build.TORCH_LIB = "/nowhere/credit_train_torch.so"
import torch
import dsmem_thread_block_gb300 as credit
try:
    credit.rmsnorm_forward(torch.zeros(2, 8))
except RuntimeError as e:
    print("refused:", e)
""")
    assert r.returncode == 0 and "torch layer is not built" in r.stdout, r.stderr
