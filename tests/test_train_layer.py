"""The training operators' Python layer without a GPU: importing the package,
`Dropout` objects, the build of the torch layer, and refusals on the host."""
import copy
import dataclasses
import os
import pickle
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


class Word:
    """Stands for a one-element int64 CUDA tensor."""
    dtype, is_cuda, device = torch.int64, True, "cuda:0"

    def __init__(self, address):
        self.address = address

    def numel(self):
        return 1

    def data_ptr(self):
        return self.address


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, dataclasses.replace,
                                   lambda d: pickle.loads(pickle.dumps(d))])
def test_dropout_objects_are_copied_and_pickled(again):
    for word in (None, Word(4096)):
        d = credit.Dropout(0.25, (1 << 63) + 5, (1 << 40) + 3, word)
        e = again(d)
        assert (e.p, e.seed, e.offset) == (d.p, d.seed, d.offset)
        # the C struct is the copy's own and says the same
        assert e._fields is not d._fields and e._address != d._address
        assert (e._fields.p, e._fields.seed, e._fields.offset, e._fields.device_offset) == \
            (0.25, (1 << 63) + 5, (1 << 40) + 3, 4096 if word else None)
        if word is None:
            assert e == d and hash(e) == hash(d)


def test_the_device_word_is_found_at_every_call():
    # the tensor may be given other storage between two calls (`t.data = u`)
    word = Word(4096)
    d = credit.Dropout(0.25, 1, 2, word)
    word.address = 8192
    assert train._drop(d, word) == d._address and d._fields.device_offset == 8192
    word.dtype = torch.int32
    with pytest.raises(ValueError):
        train._drop(d, word)


@pytest.fixture
def built(monkeypatch):
    """What build_all builds, recorded instead of compiled."""
    calls = []
    monkeypatch.setattr(B, "build", lambda force=False, verbose=False, extra=None, checked=False:
                        calls.append("checked" if checked else "regular") or calls[-1])
    monkeypatch.setattr(B, "build_torch", lambda force=False: calls.append("torch"))
    return calls


def test_the_libraries_build_without_torch(built, monkeypatch):
    assert B.build_all() == ("regular", "checked") and sorted(built) == ["checked", "regular",
                                                                        "torch"]
    built.clear()
    monkeypatch.setitem(sys.modules, "torch", None)  # not installed
    assert B.build_all() == ("regular", "checked") and sorted(built) == ["checked", "regular"]


def test_a_torch_layer_that_does_not_compile_raises(built, monkeypatch):
    def fails(force=False):
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(B, "build_torch", fails)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        B.build_all()
    assert sorted(built) == ["checked", "regular"]


def test_the_torch_layer_follows_the_installed_torch(tmp_path, monkeypatch):
    import types
    runs, version = [], tmp_path / "torch" / "version.py"
    version.parent.mkdir()
    version.write_text("1.0")

    def run(cmd, **kw):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(version.read_text())
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "TORCH_LIB", str(tmp_path / "credit_train_torch.so"))
    monkeypatch.setattr(B, "_torch_root", lambda: str(version.parent))
    monkeypatch.setattr(B.subprocess, "run", run)
    B.build_torch()
    B.build_torch()
    assert len(runs) == 1  # up to date
    version.write_text("2.0")
    B.build_torch()
    B.build_torch()
    assert len(runs) == 2
    with open(B.TORCH_LIB) as f:
        assert f.read() == "2.0"
    os.remove(B.TORCH_LIB)
    B.build_torch()
    assert len(runs) == 3


def test_tensors_that_require_a_gradient_are_refused_under_grad_mode():
    # every tensor argument of every call; the refusal comes before any look at
    # the tensors themselves, which is all that a machine without a GPU can see
    x, v = torch.zeros(4, 8), torch.zeros(8)
    m = torch.zeros(4)
    calls = [(lambda x, r, o: credit.dropout(x, None, residual=r, out=o), (x, x, x)),
             (lambda x, g, b, r, o, h: credit.layernorm_forward(x, g, b, residual=r, out=o, h_out=h),
              (x, v, v, x, x, x)),
             (lambda x, w, r: credit.rmsnorm_forward(x, w, residual=r), (x, v, x)),
             (lambda dy, h, mu, s, g, dh, dx, dr, b: credit.layernorm_backward(
                 dy, h, mu, s, g, dh=dh, dx=dx, dresidual=dr, beta=b), (x, x, m, m, v, x, x, x, v)),
             (lambda dy, h, s, w, dh: credit.rmsnorm_backward(dy, h, s, w, dh=dh), (x, x, m, v, x))]
    for call, args in calls:
        for i in range(len(args)):
            bad = [a.clone() for a in args]
            bad[i].requires_grad_()
            with pytest.raises(RuntimeError, match="record no autograd graph"):
                call(*bad)
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
                call(*bad)
        with pytest.raises(ValueError, match="CUDA"):
            call(*args)

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return credit.rmsnorm_forward(x)[0]

    with pytest.raises(ValueError, match="CUDA"):  # not refused for its gradient
        Norm.apply(x.clone().requires_grad_())
