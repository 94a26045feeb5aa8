"""The training operators without a GPU: the mask generator's published
vectors, the 64-bit definition against differences, the ABI's struct and the
refusals, which all come before any CUDA call."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import dsmem_thread_block_gb300 as credit
from dsmem_thread_block_gb300 import _credit as C
from dsmem_thread_block_gb300 import build as B

import train_helpers as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    B.build_torch()
    return C.load()


@pytest.mark.parametrize("counter, seed, want", [
    ((0, 0, 0, 0), 0, (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, 0xFFFFFFFFFFFFFFFF, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), 0x299F31D0A4093822,
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator_known_answers(counter, seed, want):
    # the known-answer vectors published with the generator
    got = R.philox([np.array([c]) for c in counter], seed)
    assert tuple(int(v[0]) for v in got) == want


def test_mask_rate_and_independence():
    a = R.keep_mask(256, 4096, 0.25, 11, 0).double()
    n = a.numel()
    assert abs(float(a.mean()) - 0.75) < 5 * (0.25 * 0.75 / n) ** 0.5
    for other in (R.keep_mask(256, 4096, 0.25, 12, 0), R.keep_mask(256, 4096, 0.25, 11, 1),
                  R.keep_mask(256, 4096, 0.25, 11, 1 << 32)):
        assert abs(float((a * other).mean()) - 0.75 ** 2) < 5 * (0.25 / n) ** 0.5


@pytest.mark.parametrize("norm", ["layernorm", "rmsnorm"])
def test_reference_gradient_against_differences(norm):
    g = torch.Generator().manual_seed(5)
    rows, cols, p, eps, step = 3, 10, 0.3, 1e-5, 1e-6
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, res, gamma, dy, dh = r(rows, cols), r(rows, cols), r(cols), r(rows, cols), r(rows, cols)
    beta = r(cols) if norm == "layernorm" else None
    mask = R.keep_mask(rows, cols, p, 3, 9)

    def loss(x, res, gamma, beta):
        h, _ = R.ref_h(x, res, p, mask)
        y = R.ref_forward(norm, h, gamma, beta, eps)[0]
        return float((y * dy).sum() + (h * dh).sum())

    h, _ = R.ref_h(x, res, p, mask)
    _, _, mean, rstd = R.ref_forward(norm, h, gamma, beta, eps)
    dtot, dx, dgamma, dbeta = R.ref_backward(norm, dy, dh, h, mean, rstd, gamma, p, mask)[:4]
    args = [x, res, gamma] + ([beta] if beta is not None else [])
    for a, want in zip(args, [dx, dtot, dgamma, dbeta]):
        for i in range(a.numel()):
            up, down = [v.clone() if v is a else v for v in args], \
                [v.clone() if v is a else v for v in args]
            k = next(n for n, v in enumerate(args) if v is a)
            up[k].view(-1)[i] += step
            down[k].view(-1)[i] -= step
            pad = [] if beta is not None else [None]
            d = (loss(*up, *pad) - loss(*down, *pad)) / (2 * step)
            # central differences: O(step^2) and 2^-53 |loss| / step
            assert abs(d - float(want.view(-1)[i])) < 1e-6 * (1 + abs(d))


def test_dropout_struct_matches_the_header(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text("""
#include <stddef.h>
#include <stdio.h>
#include "credit.h"
int main(void) {
    printf("%zu %zu %zu\\n", sizeof(credit_dropout_t), offsetof(credit_dropout_t, offset),
           offsetof(credit_dropout_t, device_offset));
    return 0;
}
""")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [ctypes.sizeof(C.DropoutFields), C.DropoutFields.offset.offset,
                   C.DropoutFields.device_offset.offset]


BAD, UNSUP = C.ERR_INVALID_ARG, C.ERR_UNSUPPORTED
X, Y, RES, H = 1 << 20, 2 << 20, 3 << 20, 4 << 20
MEAN, RSTD, G, BT, WS = 5 << 20, 6 << 20, 7 << 20, 8 << 20, 9 << 20


def drop(p=0.1, device_offset=0):
    return C.dropout_fields(p, 1, 2, device_offset)


def test_dropout_refusals():
    def call(x=X, res=RES, y=Y, rows=4, cols=64, dtype=C.F32, d=None):
        return C.credit_dropout(x, res, y, rows, cols, dtype, d if d is not None else drop())

    assert call(x=0) == BAD and call(y=0) == BAD
    assert call(rows=-1) == BAD and call(cols=0) == BAD and call(cols=-4) == BAD
    assert call(dtype=7) == UNSUP
    assert call(rows=1 << 40, cols=1 << 40) == BAD
    for p in (-0.1, 1.0, 1.5, float("nan"), float("inf")):
        assert call(d=drop(p)) == BAD
    assert call(d=drop(device_offset=12)) == BAD          # not 8-byte aligned
    assert call(d=drop(device_offset=Y + 8)) == BAD       # inside the output
    assert call(x=X + 2) == BAD and call(y=Y + 1) == BAD and call(res=RES + 2) == BAD
    assert call(y=X + 4) == BAD and call(y=RES + 16) == BAD   # partial overlap
    assert call(cols=(1 << 30) + 1, rows=1) == BAD
    assert call(rows=(1 << 32) + 1, cols=1) == BAD        # the mask's row counter
    assert call(x=0, res=0, y=0, rows=0) == C.OK          # an empty batch


def test_forward_refusals():
    def call(op=C.LAYERNORM, x=X, res=RES, d=None, y=Y, h=H, mean=MEAN, rstd=RSTD, rows=4, cols=64,
             dtype=C.BF16, g=G, b=BT, pdtype=C.F32, eps=1e-5, ws=WS, wb=1 << 20):
        return C.credit_norm_forward(op, x, res, d, y, h, mean, rstd, rows, cols, dtype, g, b,
                                     pdtype, eps, ws, wb)

    assert call(op=C.SOFTMAX) == UNSUP and call(op=C.QUANTIZE) == UNSUP
    assert call(dtype=2) == UNSUP and call(pdtype=2) == UNSUP
    assert call(x=0) == BAD and call(y=0) == BAD and call(rows=-1) == BAD and call(cols=0) == BAD
    assert call(eps=-1.0) == BAD and call(eps=float("nan")) == BAD
    assert call(op=C.RMSNORM) == BAD                      # beta and mean are LayerNorm's
    assert call(op=C.RMSNORM, mean=0) == BAD and call(op=C.RMSNORM, b=0) == BAD
    assert call(d=drop(1.0)) == BAD
    assert call(x=X + 1) == BAD and call(g=G + 2) == BAD and call(mean=MEAN + 2) == BAD
    assert call(y=H) == BAD                               # the outputs are two buffers
    assert call(y=X + 16) == BAD and call(h=RES + 2) == BAD
    assert call(mean=RSTD) == BAD and call(rstd=X) == BAD and call(y=G) == BAD
    assert call(ws=X) == BAD                              # workspace over an input
    assert call(rows=0, x=0, y=0, ws=0, wb=0) == C.OK


def test_backward_refusals():
    DX, DR, DG, DB = 10 << 20, 11 << 20, 12 << 20, 13 << 20

    def call(op=C.LAYERNORM, dy=X, dh=RES, h=H, mean=MEAN, rstd=RSTD, g=G, pdtype=C.F32, d=None,
             dx=DX, dr=DR, dg=DG, db=DB, rows=4, cols=64, dtype=C.BF16, ws=WS, wb=1 << 20):
        return C.credit_norm_backward(op, dy, dh, h, mean, rstd, g, pdtype, d, dx, dr, dg, db,
                                      rows, cols, dtype, ws, wb)

    assert call(op=C.PEARSON) == UNSUP and call(dtype=5) == UNSUP and call(pdtype=5) == UNSUP
    assert call(dy=0) == BAD and call(h=0) == BAD and call(dx=0) == BAD
    assert call(mean=0) == BAD and call(rstd=0) == BAD
    assert call(op=C.RMSNORM) == BAD                      # mean and dbeta are LayerNorm's
    assert call(op=C.RMSNORM, mean=0) == BAD and call(op=C.RMSNORM, db=0) == BAD
    assert call(d=drop(-1.0)) == BAD
    assert call(dx=DR) == BAD and call(dx=X + 2) == BAD and call(dr=H + 16) == BAD
    assert call(dg=G) == BAD and call(dg=DB) == BAD and call(dx=RSTD) == BAD
    assert call(dg=DG + 2) == BAD and call(dy=X + 1) == BAD
    assert call(ws=DX) == BAD
    assert call(rows=-1) == BAD and call(cols=0) == BAD
    assert call(rows=0, dg=0, db=0, dy=0, h=0, dx=0, mean=0, rstd=0) == C.OK


def test_workspace_refusals(lib):
    n = ctypes.c_size_t()
    assert lib.credit_norm_workspace(C.LAYERNORM, 0, 4, 4, C.F32, 0, None) == BAD
    assert lib.credit_norm_workspace(C.SOFTMAX, 0, 4, 4, C.F32, 0, ctypes.byref(n)) == UNSUP
    assert lib.credit_norm_workspace(C.LAYERNORM, 0, -1, 4, C.F32, 0, ctypes.byref(n)) == BAD
    assert lib.credit_norm_workspace(C.LAYERNORM, 1, 4, 0, C.F32, 0, ctypes.byref(n)) == BAD
    assert lib.credit_norm_workspace(C.RMSNORM, 1, 4, 4, 9, 0, ctypes.byref(n)) == UNSUP


def test_torch_layer_refuses_on_the_host():
    for p in (-0.5, 1.0, float("nan")):
        with pytest.raises(ValueError):
            credit.Dropout(p, 1)
    for seed, offset in ((-1, 0), (1 << 64, 0), (0, -1), (0, 1 << 64)):
        with pytest.raises(ValueError):
            credit.Dropout(0.1, seed, offset)
    with pytest.raises(ValueError):
        credit.Dropout(0.1, 1, device_offset=torch.zeros(1, dtype=torch.int64))  # a CPU tensor
    with pytest.raises(ValueError):
        credit.dropout(torch.zeros(4, 8), credit.Dropout(0.1, 1))
    with pytest.raises(ValueError):
        credit.layernorm_forward(torch.zeros(4, 8))
    with pytest.raises(ValueError):
        credit.rmsnorm_backward(torch.zeros(4, 8), torch.zeros(4, 8), torch.zeros(4))
