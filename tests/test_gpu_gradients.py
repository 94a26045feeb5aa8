"""The norm of many gradients together, and clipping, against 64 bits.

Bounds count roundings, u = 2^-24: a chunk's squares and their sum pass at most 33
roundings in a thread (32 additions and a square), the sums of threads and chunks
are in 64 bits; the norm is off by half of that and one rounding, 18 u.  The factor
adds two, its product one, and the output's type its own.
"""
import math

import pytest
import torch

import dsmem_thread_block_gb300 as credit
from dsmem_thread_block_gb300 import _credit as C
from train_helpers import DT, U, U_OUT

pytestmark = pytest.mark.gpu


def make(lengths, dtypes, seed=0, std=1.0, shift=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = []
    for i, n in enumerate(lengths):
        room = torch.randn(n + shift, generator=g, device="cuda") * std
        out.append(room.to(DT[dtypes[i % len(dtypes)]])[shift:])
    return out


def norm_of(grads):
    return math.sqrt(math.fsum(float(t.double().pow(2).sum()) for t in grads))


def check_norm(got, grads):
    want = norm_of(grads)
    assert abs(float(got) - want) <= 18 * U * want, (float(got), want)
    return want


def check_clipped(out, grads, want, max_norm, eps=1e-6):
    factor = min(1.0, max_norm / (want + eps))
    for o, g in zip(out, grads):
        exact = g.double() * factor
        bound = (22 * U + U_OUT[g.dtype]) * exact.abs() + torch.finfo(g.dtype).tiny * U_OUT[g.dtype] * 2
        assert bool(((o.double() - exact).abs() <= bound).all())


SETS = [[1], [2, 0, 3], [8191, 8192, 8193], [16383, 16384, 16385, 7], [1000003], [5] * 63, [33] * 64,
        [1 + i % 50 for i in range(65)], [i % 7 for i in range(1200)], [40000] * 961, [1 << 22, 5, 1 << 20]]


@pytest.mark.parametrize("dtypes", [("f32",), ("bf16",), ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("lengths", SETS, ids=lambda s: f"{len(s)}x{s[0]}")
def test_norm_and_clipping(lengths, dtypes):
    grads = make(lengths, dtypes, seed=len(lengths))
    norm = credit.gradient_norm(grads)
    assert norm.shape == () and norm.dtype == torch.float32
    want = check_norm(norm, grads)
    out = [torch.empty_like(g) for g in grads]
    for max_norm in (0.3 * want, 2 * want + 1):
        got = credit.clip_gradients(grads, max_norm, out=out)
        assert float(got) == float(norm)
        check_clipped(out, grads, want, max_norm)
    kept = [g.clone() for g in grads]
    assert float(credit.clip_gradients(grads, 2 * want + 1)) == float(norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))
    assert float(credit.clip_gradients(grads, 0.3 * want)) == float(norm)
    check_clipped(grads, kept, want, 0.3 * want)


@pytest.mark.parametrize("out_shift", [0, 1, 5])
@pytest.mark.parametrize("shift", [0, 1, 3, 7])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_any_alignment_and_nothing_beside(dtype, shift, out_shift):
    lengths = [1, 9, 8190, 20000]
    grads = make(lengths, (dtype,), seed=3, shift=shift)
    want = check_norm(credit.gradient_norm(grads), grads)
    rooms = [torch.full((n + out_shift + 16,), 7.0, dtype=DT[dtype], device="cuda") for n in lengths]
    out = [r[out_shift:out_shift + n] for r, n in zip(rooms, lengths)]
    credit.clip_gradients(grads, 0.5 * want, out=out)
    check_clipped(out, grads, want, 0.5 * want)
    for r, n in zip(rooms, lengths):
        assert bool((r[:out_shift] == 7).all()) and bool((r[out_shift + n:] == 7).all())
    room = torch.full((20032,), 7.0, dtype=DT[dtype], device="cuda")  # in place
    room[shift + 1:shift + 20001] = grads[3]
    credit.clip_gradients([room[shift + 1:shift + 20001]], 0.5)
    assert bool((room[:shift + 1] == 7).all()) and bool((room[shift + 20001:] == 7).all())


@pytest.mark.parametrize("std", [1e-38, 1e-30, 1e-20, 1e-12, 1e10, 1e19, 1e25, 1e34])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_squares_outside_the_type(dtype, std):
    grads = make([3000, 17], (dtype,), std=std)
    got = credit.gradient_norm(grads)
    want = norm_of(grads)
    assert abs(float(got) - want) <= 18 * U * want
    # large ones among small ones
    grads.append(torch.full((3,), 1.0, device="cuda", dtype=DT[dtype]))
    check_norm(credit.gradient_norm(grads), grads)


def test_zeros_infinities_and_nans():
    z = torch.zeros(5000, device="cuda")
    assert float(credit.gradient_norm([z])) == 0.0
    assert float(credit.clip_gradients([z], 1.0)) == 0.0 and bool((z == 0).all())
    g = torch.ones(5000, device="cuda")
    g[7] = float("inf")
    assert float(credit.clip_gradients([g], 1.0)) == math.inf
    assert math.isnan(float(g[7])) and bool((g[:7] == 0).all()) and bool((g[8:] == 0).all())
    g = torch.ones(5000, device="cuda")
    g[4999] = float("nan")
    assert math.isnan(float(credit.clip_gradients([g], 1.0))) and bool(torch.isnan(g).all())
    g = torch.ones(16, device="cuda")
    assert float(credit.clip_gradients([g], 0.0)) == 4.0 and bool((g == 0).all())


def test_dense_strides():
    t = torch.randn(40, 60, device="cuda")
    grads = [t.t(), torch.randn(2, 3, 4, 5, device="cuda").to(memory_format=torch.channels_last)]
    out = [torch.empty_like(g) for g in grads]
    want = check_norm(credit.clip_gradients(grads, 1.0, out=out), grads)
    check_clipped(out, grads, want, 1.0)
    with pytest.raises(ValueError):  # other strides
        credit.clip_gradients([t.t()], 1.0, out=[torch.empty(60, 40, device="cuda")])
    with pytest.raises(ValueError):  # holes
        credit.gradient_norm([t[:, :30]])


def test_repeats_streams_and_graphs():
    grads = make([100001, 5, 77777, 1 << 20], ("f32", "bf16"), seed=4)
    first = float(credit.gradient_norm(grads))
    out = [torch.empty_like(g) for g in grads]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        assert float(credit.gradient_norm(grads)) == first
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = credit.clip_gradients(grads, 1.0, out=out, workspace=ws)
    for scale in (1.0, 3.0):
        for g in grads:
            g.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        want = check_norm(norm, grads)
        check_clipped(out, grads, want, 1.0)


def test_the_same_tensor_twice():
    g = torch.ones(100, device="cuda")
    assert float(credit.gradient_norm([g, g])) == float(torch.tensor(200.0).sqrt())
    with pytest.raises(credit.CreditError):
        credit.clip_gradients([g, g], 1.0)
    with pytest.raises(credit.CreditError):  # one output for two
        credit.clip_gradients([g, g.clone()], 1.0, out=[torch.empty_like(g)] * 2)
    with pytest.raises(credit.CreditError):  # an output that holds another's input
        b = torch.ones(200, device="cuda")
        credit.clip_gradients([b[:100], b[100:]], 1.0, out=[b[50:150], torch.empty_like(g)])
    assert bool((g == 1).all())


@pytest.mark.parametrize("what", ["empty", "cpu", "half", "graph", "lengths", "negative", "nan", "number",
                                  "none", "workspace"])
def test_refusals(what):
    g = torch.ones(10, device="cuda")
    with pytest.raises((ValueError, TypeError, RuntimeError, credit.CreditError)):
        if what == "empty":
            credit.gradient_norm([])
        elif what == "cpu":
            credit.gradient_norm([g, torch.ones(10)])
        elif what == "half":
            credit.gradient_norm([g.half()])
        elif what == "graph":
            credit.clip_gradients([g.clone().requires_grad_()], 1.0)
        elif what == "lengths":
            credit.clip_gradients([g], 1.0, out=[])
        elif what == "negative":
            credit.clip_gradients([g], -1.0)
        elif what == "nan":
            credit.clip_gradients([g], float("nan"))
        elif what == "number":
            credit.gradient_norm(3)
        elif what == "none":
            credit.gradient_norm([g, None])
        elif what == "workspace":
            credit.gradient_norm([g], workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))


def test_iterators_and_tuples():
    grads = make([100, 7, 3000], ("f32", "bf16"), seed=9)
    want = float(credit.gradient_norm(grads))
    assert float(credit.gradient_norm(tuple(grads))) == want
    assert float(credit.gradient_norm(g for g in grads)) == want
    out = [torch.empty_like(g) for g in grads]
    assert float(credit.clip_gradients((g for g in grads), 0.5, out=(o for o in out))) == want
    copy = [g.clone() for g in grads]
    assert float(credit.clip_gradients((g for g in copy), 0.5)) == want
    assert all(torch.equal(a, b) for a, b in zip(copy, out))


def test_more_elements_than_32_bits_count():
    n = (1 << 32) + 12345
    g = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    g[0], g[1 << 31], g[n - 1] = 3.0, 4.0, 12.0
    assert float(credit.clip_gradients([g], 6.5, eps=0.0)) == 13.0
    assert (float(g[0]), float(g[1 << 31]), float(g[n - 1])) == (1.5, 2.0, 6.0)
    assert int(torch.count_nonzero(g[: 1 << 31])) + int(torch.count_nonzero(g[1 << 31:])) == 3


def test_versions_of_what_is_written():
    g = torch.ones(10, device="cuda")
    o, v = torch.empty_like(g), g._version
    credit.clip_gradients([g], 1.0, out=[o])
    assert g._version == v and o._version == 1
    credit.clip_gradients([g], 1.0)
    assert g._version == v + 1
