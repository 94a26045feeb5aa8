"""Host-side checks of the head's cross entropy and of gradient clipping: no GPU
is touched, every refusal comes before the first CUDA call."""
import ctypes
import os
import subprocess

import pytest

from dsmem_thread_block_gb300 import _credit as C
from dsmem_thread_block_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
H, W, T, L, S, D = (i << 32 for i in range(1, 7))  # addresses that nothing follows
WS = 1 << 36


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()


def forward(h=H, w=W, t=T, loss=L, lse=S, tokens=4, hidden=64, vocab=100, dtype=C.BF16, ws=WS, wb=1 << 30):
    return C.credit_linear_ce_forward(h, w, t, -100, loss, lse, tokens, hidden, vocab, dtype, ws, wb)


def backward(dloss=D, dlse=0, h=H, w=W, t=T, lse=S, dh=7 << 32, dw=8 << 32, tokens=4, hidden=64, vocab=100,
             dtype=C.BF16, ws=WS, wb=1 << 30):
    return C.credit_linear_ce_backward(dloss, dlse, h, w, t, -100, lse, dh, dw, tokens, hidden, vocab, dtype,
                                       ws, wb)


@pytest.mark.parametrize("bad", [
    dict(h=0), dict(w=0), dict(t=0), dict(loss=0), dict(lse=0), dict(tokens=-1), dict(hidden=0),
    dict(vocab=0), dict(h=H + 1), dict(w=W + 1), dict(t=T + 4), dict(loss=L + 2), dict(lse=S + 1),
    dict(loss=H), dict(lse=W + 8), dict(lse=L + 4), dict(loss=T + 8), dict(ws=0), dict(ws=WS + 8),
    dict(ws=H), dict(tokens=1 << 31), dict(vocab=1 << 31), dict(hidden=(1 << 24) + 1),
    dict(tokens=1 << 30, vocab=1 << 30)])
def test_forward_refuses(bad):
    assert forward(**bad) == C.ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(dloss=0), dict(h=0), dict(w=0), dict(t=0), dict(lse=0), dict(tokens=-1), dict(hidden=0),
    dict(vocab=0), dict(dloss=D + 2), dict(dlse=D + 1), dict(dh=(7 << 32) + 1), dict(dw=(8 << 32) + 1),
    dict(dh=H), dict(dw=W), dict(dh=W + 64), dict(dw=7 << 32), dict(dh=S), dict(ws=W)])
def test_backward_refuses(bad):
    assert backward(**bad) == C.ERR_INVALID_ARG


def test_types_and_empty_calls():
    assert forward(dtype=7) == C.ERR_UNSUPPORTED and backward(dtype=7) == C.ERR_UNSUPPORTED
    assert forward(tokens=0) == C.OK
    assert backward(dh=0, dw=0) == C.OK and backward(tokens=0, dw=0) == C.OK


def test_workspace_refuses():
    for bad in (dict(h=H + 1), dict(hidden=0), dict(vocab=0), dict(tokens=-1)):
        a = dict(dict(h=H, tokens=100, hidden=64, vocab=1000), **bad)
        with pytest.raises(C.CreditError):
            C.credit_linear_ce_workspace(False, a["h"], W, a["tokens"], a["hidden"], a["vocab"], C.BF16)
    assert C.credit_linear_ce_workspace(True, H, W, 0, 64, 1000, C.F32) == 0


def clip(entries, max_norm=1.0, eps=1e-6, norm=L, ws=WS, wb=1 << 20):
    return C.credit_grad_clip(C.tensors(entries), max_norm, eps, norm, ws, wb)


G = (H, H, 100, C.F32)


@pytest.mark.parametrize("entries", [
    [(0, H, 4, C.F32)], [(H + 2, H + 2, 4, C.F32)], [(H + 1, H + 1, 4, C.BF16)], [(H, H, -1, C.F32)],
    [(H, 0, 4, C.F32)], [(H, H + 4, 4, C.F32)], [G, G], [G, (H + 396, H + 396, 4, C.F32)],
    [(H, W, 4, C.F32), (T, W + 12, 4, C.F32)], [(H, W, 4, C.F32), (W + 8, T, 4, C.F32)],
    [(H, L, 4, C.F32)], [(H, WS + 8, 4, C.F32)], [(H, H, 1 << 62, C.F32)]])
def test_clipping_refuses(entries):
    assert clip(entries) == C.ERR_INVALID_ARG


def test_clipping_refuses_its_numbers():
    for bad in (-1.0, float("nan")):
        assert clip([G], max_norm=bad) == C.ERR_INVALID_ARG
        assert clip([G], eps=bad) == C.ERR_INVALID_ARG
    assert clip([G], norm=0) == C.ERR_INVALID_ARG and clip([G], norm=L + 2) == C.ERR_INVALID_ARG
    assert clip([(H, H, 4, 7)]) == C.ERR_UNSUPPORTED
    # the norm alone reads: the same tensor may come twice, its outputs are not looked at
    assert C.credit_grad_norm(C.tensors([(H, 0, 4, 7)]), L, WS, 64) == C.ERR_UNSUPPORTED
    assert C.credit_grad_norm(C.tensors([(L, 0, 4, C.F32)]), L, WS, 64) == C.ERR_INVALID_ARG


def test_the_tensor_struct_matches_the_header(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text("""
#include <stddef.h>
#include <stdio.h>
#include "credit.h"
int main(void) {
    printf("%zu %zu %zu\\n", sizeof(credit_tensor_t), offsetof(credit_tensor_t, count),
           offsetof(credit_tensor_t, dtype));
    return 0;
}
""")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include", str(src),
                    "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [ctypes.sizeof(C.Tensor), C.Tensor.count.offset, C.Tensor.dtype.offset]


def test_the_precise_gradient_refuses_as_the_other():
    def precise(dloss=D, h=H, w=W, tokens=100, vocab=1000, dtype=C.BF16, dh=7 << 32):
        return C.credit_linear_ce_backward_precise(dloss, 0, h, w, T, -100, S, dh, 8 << 32, tokens, 64, vocab,
                                                   dtype, WS, 1 << 30)

    for bad in (dict(dloss=0), dict(h=H + 1), dict(w=0), dict(vocab=0), dict(dh=W + 64), dict(tokens=-1),
                dict(tokens=1 << 30, vocab=64)):  # (the last: two rows a token pass 31 bits)
        assert precise(**bad) == C.ERR_INVALID_ARG
    assert precise(dtype=7) == C.ERR_UNSUPPORTED
    for backward in (-1, 3):
        with pytest.raises(C.CreditError):
            C.credit_linear_ce_workspace(backward, H, W, 100, 64, 1000, C.BF16)
