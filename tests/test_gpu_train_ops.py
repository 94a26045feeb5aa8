"""The training operators on the GPU against their 64-bit definition: shapes
from one element to the widest rows, aligned and ragged, both types, every
optional part present and absent, in place, misaligned, on other streams,
captured and replayed, and chained as a training step uses them."""
import pytest
import torch

import dsmem_thread_block_gb300 as credit
from dsmem_thread_block_gb300 import _credit as C

import train_helpers as R

pytestmark = pytest.mark.gpu

EPS = {"layernorm": 1e-5, "rmsnorm": 1e-6}
SHAPES = [(1, 1), (3, 2), (2, 7), (5, 8), (9, 64), (300, 100), (7, 257), (33, 256), (64, 1000),
          (160, 1024), (37, 1025), (19, 2056), (700, 512), (5, 4096), (301, 4096), (9, 5000),
          (157, 8192), (6, 10001), (3, 16384), (2, 16392), (3, 40000), (2, 70001), (3, 65536),
          (2, 262144), (1, 524296), (2, 786432)]


def make(shape, dtype, seed, mean=0.0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def problem(rows, cols, dtype, norm, residual, p, pdtype, seed=1):
    t, pt = R.DT[dtype], R.DT[pdtype]
    return {
        "x": make((rows, cols), t, seed), "eps": EPS[norm],
        "residual": make((rows, cols), t, seed + 1, 0.25, 1.5) if residual else None,
        "gamma": make((cols,), pt, seed + 2, 1.0, 0.1),
        "beta": make((cols,), pt, seed + 3, 0.0, 0.1) if norm == "layernorm" else None,
        "drop": credit.Dropout(p, 0xABCDEF0123456789 ^ seed, (seed << 33) | 5) if p else None,
        "mask": R.keep_mask(rows, cols, p, 0xABCDEF0123456789 ^ seed, (seed << 33) | 5).cuda()
        if p else None, "p": p}


def forward(norm, q, **kw):
    if norm == "layernorm":
        return credit.layernorm_forward(q["x"], q["gamma"], q["beta"], eps=q["eps"],
                                        residual=q["residual"], dropout=q["drop"], **kw)
    y, h, rstd = credit.rmsnorm_forward(q["x"], q["gamma"], eps=q["eps"], residual=q["residual"],
                                        dropout=q["drop"], **kw)
    return y, h, None, rstd


def backward(norm, q, dy, h, mean, rstd, dh, **kw):
    if norm == "layernorm":
        return credit.layernorm_backward(dy, h, mean, rstd, q["gamma"], dh=dh, dropout=q["drop"],
                                         **kw)
    return (*credit.rmsnorm_backward(dy, h, rstd, q["gamma"], dh=dh, dropout=q["drop"], **kw), None)


def check_forward(norm, q, out):
    y, h, mean, rstd = out
    x = q["x"]
    rh, mag = R.ref_h(x, q["residual"], q["p"], q["mask"])
    ry, z, rm, rr = R.ref_forward(norm, rh, q["gamma"], q["beta"], q["eps"])
    bh, by, bm, br = R.forward_bounds(norm, rh, mag, ry, z, rm, rr, q["gamma"], q["beta"],
                                      q["eps"], x.dtype)
    R.assert_close(h, rh, bh, "h")
    R.assert_close(y, ry, by, "y")
    if mean is not None:
        R.assert_close(mean, rm, bm, "mean")
    R.assert_close(rstd, rr, br, "rstd")


def check_backward(norm, q, dy, h, mean, rstd, dh, out):
    dx, dres, dgamma, dbeta = out
    d, rx, rg, rb, ed, ex, eg, eb = R.ref_backward(norm, dy, dh, h, mean, rstd, q["gamma"],
                                                   q["p"], q["mask"])
    uo = R.U_OUT[dy.dtype]
    R.assert_close(dx, rx, uo * rx.abs() + R.U * ex, "dx")
    if dres is not None:
        R.assert_close(dres, d, uo * d.abs() + R.U * ed, "dresidual")
    if dgamma is not None:
        po = R.U_OUT[dgamma.dtype]
        R.assert_close(dgamma, rg, po * rg.abs() + R.U * eg, "dgamma")
        if dbeta is not None:
            R.assert_close(dbeta, rb, po * rb.abs() + R.U * eb, "dbeta")


def grads(rows, cols, dtype, seed=50):
    return make((rows, cols), R.DT[dtype], seed), make((rows, cols), R.DT[dtype], seed + 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_dropout(rows, cols, dtype):
    for residual in (False, True):
        q = problem(rows, cols, dtype, "rmsnorm", residual, 0.3, "f32")
        got = credit.dropout(q["x"], q["drop"], residual=q["residual"])
        want, mag = R.ref_h(q["x"], q["residual"], 0.3, q["mask"])
        R.assert_close(got, want, R.U_OUT[q["x"].dtype] * want.abs() + 4 * R.U * mag, "y")
        if not residual:
            assert torch.equal(got != 0, q["mask"] & (q["x"] != 0))
    assert torch.equal(credit.dropout(q["x"], None), q["x"])


@pytest.mark.parametrize("norm", ["layernorm", "rmsnorm"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_forward(rows, cols, dtype, norm):
    for residual, p, pdtype in ((True, 0.2, "f32"), (False, 0.0, "bf16"), (True, 0.0, "bf16"),
                                (False, 0.5, "f32")):
        q = problem(rows, cols, dtype, norm, residual, p, pdtype)
        check_forward(norm, q, forward(norm, q))
    assert credit.device_error() == 0


@pytest.mark.parametrize("norm", ["layernorm", "rmsnorm"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_backward(rows, cols, dtype, norm):
    for residual, p, pdtype in ((True, 0.2, "f32"), (False, 0.0, "bf16"), (True, 0.0, "bf16"),
                                (False, 0.5, "f32")):
        q = problem(rows, cols, dtype, norm, residual, p, pdtype)
        _, h, mean, rstd = forward(norm, q)
        dy, dh = grads(rows, cols, dtype)
        dh = dh if residual else None
        out = backward(norm, q, dy, h, mean, rstd, dh, need_dresidual=residual)
        check_backward(norm, q, dy, h, mean, rstd, dh, out)
        again = backward(norm, q, dy, h, mean, rstd, dh, need_dresidual=residual)
        for a, b in zip(out, again):  # a fixed order of every sum: bit for bit
            assert a is b is None or torch.equal(a, b)
    assert credit.device_error() == 0


@pytest.mark.parametrize("norm", ["layernorm", "rmsnorm"])
@pytest.mark.parametrize("rows, cols, dtype", [(5003, 768, "bf16"), (9000, 64, "f32"),
                                               (2000, 1111, "bf16"), (70000, 40, "bf16")])
def test_many_rows(rows, cols, dtype, norm):
    q = problem(rows, cols, dtype, norm, True, 0.1, "f32", seed=7)
    out = forward(norm, q)
    check_forward(norm, q, out)
    _, h, mean, rstd = out
    dy, dh = grads(rows, cols, dtype)
    check_backward(norm, q, dy, h, mean, rstd, dh,
                   backward(norm, q, dy, h, mean, rstd, dh, need_dresidual=True))


# rows shared by CTAs across the GPU (more rows than a team has in flight, odd
# counts, more teams than one), and rows beyond them, swept in two passes
WIDE = [(13, 300008, "bf16"), (27, 300001, "bf16"), (41, 300000, "f32"), (6, 600008, "f32"),
        (40, 131080, "bf16"), (90, 60000, "f32"), (75, 70001, "bf16"), (3, 1300000, "bf16"),
        (2, 1200001, "f32")]


@pytest.mark.parametrize("norm", ["layernorm", "rmsnorm"])
@pytest.mark.parametrize("rows, cols, dtype", WIDE)
def test_wide_rows(rows, cols, dtype, norm):
    for residual, p in ((True, 0.1), (False, 0.0)):
        q = problem(rows, cols, dtype, norm, residual, p, "f32", seed=17)
        out = forward(norm, q)
        check_forward(norm, q, out)
        _, h, mean, rstd = out
        dy, dh = grads(rows, cols, dtype)
        dh = dh if residual else None
        back = backward(norm, q, dy, h, mean, rstd, dh, need_dresidual=residual)
        check_backward(norm, q, dy, h, mean, rstd, dh, back)
        again = backward(norm, q, dy, h, mean, rstd, dh, need_dresidual=residual)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(back, again))
    assert credit.device_error() == 0


@pytest.mark.parametrize("norm", ["layernorm", "rmsnorm"])
@pytest.mark.parametrize("rows, cols, dtype", [(250, 300008, "bf16"), (150, 300001, "f32")])
def test_wide_rows_again_and_again(rows, cols, dtype, norm):
    # two teams of 54 CTAs or more: 125 and 75 turns, so every stage and every
    # slot of the exchange is used again and every CTA leads more than one turn
    q = problem(rows, cols, dtype, norm, True, 0.0, "f32", seed=19)
    out = forward(norm, q)
    check_forward(norm, q, out)
    _, h, mean, rstd = out
    dy, dh = grads(rows, cols, dtype)
    back = backward(norm, q, dy, h, mean, rstd, dh)
    check_backward(norm, q, dy, h, mean, rstd, dh, back)
    # in place, with rows still to come in flight
    x, res = q["x"].clone(), q["residual"].clone()
    again = forward(norm, dict(q, x=x, residual=res), out=x, h_out=res)
    assert again[0] is x and all(a is b is None or torch.equal(a, b) for a, b in zip(again, out))
    dy2 = dy.clone()
    again = backward(norm, q, dy2, h, mean, rstd, dh, dx=dy2)
    assert again[0] is dy2 and all(a is b is None or torch.equal(a, b) for a, b in zip(again, back))
    assert credit.device_error() == 0


def test_wide_rows_on_two_streams_at_once():
    # both calls want every SM: one runs after the other, neither waits in vain
    qs = [problem(20, 300008 + 8 * i, "bf16", "layernorm", False, 0.0, "f32", seed=80 + i)
          for i in range(2)]
    dys = [grads(20, 300008 + 8 * i, "bf16")[0] for i in range(2)]

    def step(q, dy):
        f = forward("layernorm", q)
        return f, backward("layernorm", q, dy, *f[1:], None)

    want = [step(q, dy) for q, dy in zip(qs, dys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(4):
        got = []
        for s, q, dy in zip(streams, qs, dys):
            with torch.cuda.stream(s):
                got.append(step(q, dy))
        torch.cuda.synchronize()
        for (f, b), (wf, wb) in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(f, wf))
            assert all(u is v is None or torch.equal(u, v) for u, v in zip(b, wb))
    assert credit.device_error() == 0


def test_a_training_step_of_two_blocks():
    # two residual steps forward and back; the second's input gradient is the
    # first's incoming one, and every gradient is autograd's in 64 bits on the
    # values that were stored
    rows, cols, p = 48, 1536, 0.1
    q1 = problem(rows, cols, "bf16", "layernorm", True, p, "f32", seed=21)
    q2 = problem(rows, cols, "bf16", "rmsnorm", True, p, "f32", seed=31)
    y1, h1, m1, r1 = forward("layernorm", q1)
    q2["x"], q2["residual"] = y1, h1
    y2, h2, _, r2 = forward("rmsnorm", q2)
    check_forward("layernorm", q1, (y1, h1, m1, r1))
    check_forward("rmsnorm", q2, (y2, h2, None, r2))
    dy = make((rows, cols), torch.bfloat16, 41)
    dx2, dres2, dg2, _ = backward("rmsnorm", q2, dy, h2, None, r2, None, need_dresidual=True)
    out1 = backward("layernorm", q1, dx2, h1, m1, r1, dres2, need_dresidual=True)
    check_backward("rmsnorm", q2, dy, h2, None, r2, None, (dx2, dres2, dg2, None))
    check_backward("layernorm", q1, dx2, h1, m1, r1, dres2, out1)
    # dropout's own backward pass is the same call on the gradient
    assert torch.equal(credit.dropout(out1[1], q1["drop"]) != 0, q1["mask"] & (out1[1] != 0))


def test_fused_and_separate_dropout_draw_one_mask():
    for cols in (1024, 1001, 40000):
        q = problem(6, cols, "f32", "rmsnorm", False, 0.4, "f32", seed=3)
        _, h, _, rstd = forward("rmsnorm", q)
        assert torch.equal(h, credit.dropout(q["x"], q["drop"]))
        dy, _ = grads(6, cols, "f32")
        dx = backward("rmsnorm", q, dy, h, None, rstd, None)[0]
        assert torch.equal(dx != 0, q["mask"])


@pytest.mark.parametrize("cols", [512, 1001, 8192, 40000, 300000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(cols, dtype):
    for norm in ("layernorm", "rmsnorm"):
        q = problem(5, cols, dtype, norm, True, 0.2, "f32")
        want = forward(norm, q)
        x, res = q["x"].clone(), q["residual"].clone()
        q2 = dict(q, x=x, residual=res)
        got = forward(norm, q2, out=x, h_out=res)
        assert got[0] is x and got[1] is res
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))
        _, h, mean, rstd = want
        dy, dh = grads(5, cols, dtype)
        wb = backward(norm, q, dy, h, mean, rstd, dh, need_dresidual=True)
        dy2, dh2 = dy.clone(), dh.clone()
        gb = backward(norm, q, dy2, h, mean, rstd, dh2, need_dresidual=True, dx=dy2, dresidual=dh2)
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(gb, wb))
        z = q["x"].clone()
        assert torch.equal(credit.dropout(z, q["drop"], residual=q["residual"], out=z),
                           credit.dropout(q["x"], q["drop"], residual=q["residual"]))


def offset_by(t, n):
    """The same values at an address n elements past an allocation's start."""
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    v = buf[n:].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("cols", [64, 1024, 4096, 20000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_misaligned_pointers(cols, dtype):
    q = problem(6, cols, dtype, "layernorm", True, 0.2, "bf16")
    dy, dh = grads(6, cols, dtype)
    for name, n in (("x", 1), ("residual", 3), ("gamma", 1), ("beta", 2)):
        q2 = dict(q)
        q2[name] = offset_by(q[name], n)
        out = forward("layernorm", q2)
        check_forward("layernorm", q2, out)
        _, h, mean, rstd = out
        check_backward("layernorm", q2, offset_by(dy, 1), h, mean, rstd, dh,
                       backward("layernorm", q2, offset_by(dy, 1), h, mean, rstd, dh,
                                need_dresidual=True))
        check_backward("layernorm", q2, dy, offset_by(h, 1), mean, rstd, offset_by(dh, 1),
                       backward("layernorm", q2, dy, offset_by(h, 1), mean, rstd,
                                offset_by(dh, 1), need_dresidual=True))
    assert torch.equal(credit.dropout(offset_by(q["x"], 1), q["drop"]),
                       credit.dropout(q["x"], q["drop"]))


def test_outputs_stay_inside_their_buffers():
    # a guard of untouched values before and behind every output
    for rows, cols in ((3, 1001), (2, 4096), (1, 30001)):
        q = problem(rows, cols, "bf16", "layernorm", True, 0.2, "bf16")
        dy, dh = grads(rows, cols, "bf16")

        def guarded():
            buf = torch.full((rows * cols + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
            return buf, buf[32:32 + rows * cols].view(rows, cols)

        bufs = [guarded() for _ in range(4)]
        _, h, mean, rstd = forward("layernorm", q, out=bufs[0][1], h_out=bufs[1][1])
        backward("layernorm", q, dy, h, mean, rstd, dh, need_dresidual=True, dx=bufs[2][1],
                 dresidual=bufs[3][1])
        for buf, _ in bufs:
            assert bool((buf[:32] == 7).all()) and bool((buf[32 + rows * cols:] == 7).all())


def test_dropped_elements_ignore_nan_and_infinity():
    for cols in (256, 1001):
        q = problem(4, cols, "f32", "layernorm", True, 0.5, "f32")
        x = q["x"].clone()
        x[~q["mask"]] = float("nan")
        x[0][~q["mask"][0]] = float("inf")
        for a, b in zip(forward("layernorm", dict(q, x=x)), forward("layernorm", q)):
            assert torch.equal(a, b)
        assert torch.equal(credit.dropout(x, q["drop"]), credit.dropout(q["x"], q["drop"]))


def test_nan_stays_in_its_row():
    q = problem(5, 4096, "bf16", "layernorm", False, 0.0, "f32")
    clean = forward("layernorm", q)
    x = q["x"].clone()
    x[2, 17] = float("nan")
    y, _, mean, rstd = forward("layernorm", dict(q, x=x))
    rows = [0, 1, 3, 4]
    assert bool(y[2].isnan().all()) and bool(mean[2].isnan()) and bool(rstd[2].isnan())
    assert torch.equal(y[rows], clean[0][rows])


def test_constant_rows_and_large_means():
    q = problem(4, 2048, "f32", "layernorm", False, 0.0, "f32")
    q["x"] = torch.full((4, 2048), 3.0, device="cuda")
    y, _, mean, rstd = forward("layernorm", q)
    assert torch.equal(y, q["beta"].expand(4, -1)) and bool((mean == 3.0).all())
    assert bool(((rstd - 1e-5 ** -0.5).abs() <= 4 * R.U * 1e-5 ** -0.5).all())
    q["x"] = make((4, 2048), torch.float32, 9, 1000.0, 1.0)
    check_forward("layernorm", q, forward("layernorm", q))


def test_absent_parameters_and_outputs():
    q = problem(6, 1024, "bf16", "layernorm", True, 0.2, "f32")
    q["gamma"] = q["beta"] = None
    out = forward("layernorm", q)
    check_forward("layernorm", q, out)
    dy, dh = grads(6, 1024, "bf16")
    back = backward("layernorm", q, dy, *out[1:], dh)
    assert back[1] is back[2] is back[3] is None
    check_backward("layernorm", q, dy, *out[1:], dh, back)
    # no statistics and no h wanted, through the C ABI
    x, res = q["x"], q["residual"]
    y = torch.empty_like(x)
    need = C.credit_norm_workspace(C.LAYERNORM, False, 6, 1024, C.BF16, 0)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert C.credit_norm_forward(C.LAYERNORM, x.data_ptr(), res.data_ptr(), q["drop"]._fields,
                                 y.data_ptr(), 0, 0, 0, 6, 1024, C.BF16, 0, 0, C.F32, q["eps"],
                                 ws.data_ptr(), need, s) == C.OK
    assert torch.equal(y, out[0])
    if need:
        assert C.credit_norm_forward(C.LAYERNORM, x.data_ptr(), 0, None, y.data_ptr(), 0, 0, 0, 6,
                                     1024, C.BF16, 0, 0, C.F32, q["eps"], ws.data_ptr(), need - 1,
                                     s) == C.ERR_INVALID_ARG


def test_empty_batch():
    q = problem(1, 96, "bf16", "layernorm", True, 0.2, "bf16")
    q = dict(q, x=q["x"][:0], residual=q["residual"][:0])
    y, h, mean, rstd = forward("layernorm", q)
    assert y.shape == (0, 96) and h.shape == (0, 96) and mean.numel() == rstd.numel() == 0
    dx, dres, dgamma, dbeta = backward("layernorm", q, q["x"], h, mean, rstd, None,
                                       need_dresidual=True)
    assert dx.shape == (0, 96) and bool((dgamma == 0).all()) and bool((dbeta == 0).all())
    assert credit.dropout(q["x"], q["drop"]).shape == (0, 96)


def test_leading_dimensions_and_other_stream():
    q = problem(6, 512, "bf16", "layernorm", True, 0.2, "f32")
    want = forward("layernorm", q)
    q3 = dict(q, x=q["x"].view(2, 3, 512), residual=q["residual"].view(2, 3, 512))
    got = forward("layernorm", q3)
    assert got[0].shape == (2, 3, 512) and got[2].shape == (2, 3)
    assert all(torch.equal(a.view(-1), b.view(-1)) for a, b in zip(got, want))
    dy, dh = grads(6, 512, "bf16")
    wb = backward("layernorm", q, dy, *want[1:], dh, need_dresidual=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = forward("layernorm", q)
        b = backward("layernorm", q, dy, *a[1:], dh, need_dresidual=True)
    s.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, want))
    assert all(torch.equal(u, v) for u, v in zip(b, wb))


def test_two_streams_at_once():
    qs = [problem(200, 1024 + 8 * i, "bf16", "layernorm", True, 0.1, "f32", seed=60 + i)
          for i in range(2)]
    dys = [grads(200, 1024 + 8 * i, "bf16") for i in range(2)]
    want = []
    for q, (dy, dh) in zip(qs, dys):
        f = forward("layernorm", q)
        want.append((f, backward("layernorm", q, dy, *f[1:], dh, need_dresidual=True)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        got = []
        for s, q, (dy, dh) in zip(streams, qs, dys):
            with torch.cuda.stream(s):
                f = forward("layernorm", q)
                got.append((f, backward("layernorm", q, dy, *f[1:], dh, need_dresidual=True)))
        torch.cuda.synchronize()
        for (f, b), (wf, wb) in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(f, wf))
            assert all(torch.equal(u, v) for u, v in zip(b, wb))


@pytest.mark.parametrize("rows, cols", [(40, 1024), (3, 40000), (2, 600008), (12, 1001)])
def test_captured_step_draws_new_masks(rows, cols):
    q = problem(rows, cols, "f32", "rmsnorm", True, 0.25, "f32", seed=70)
    word = torch.zeros(1, dtype=torch.int64, device="cuda")
    base = (1 << 32) - 1  # the device word carries into the offset's high half
    q["drop"] = credit.Dropout(0.25, 77, base, device_offset=word)
    dy, dh = grads(rows, cols, "f32")

    def step():
        y, h, _, rstd = forward("rmsnorm", q)
        dx, dres, dg, _ = backward("rmsnorm", q, dy, h, None, rstd, dh, need_dresidual=True)
        return y, h, rstd, dx, dres, dg

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for k in (0, 1, 5):
        word.fill_(k)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        q2 = dict(q, mask=R.keep_mask(rows, cols, 0.25, 77, base + k).cuda())
        check_forward("rmsnorm", q2, (got[0], got[1], None, got[2]))
        check_backward("rmsnorm", q2, dy, got[1], None, got[2], dh, (got[3], got[4], got[5], None))
        eager = step()
        assert all(torch.equal(a, b) for a, b in zip(got, eager))


def test_checked_build_runs_every_form():
    # the checked build's kernels, reached through the same calls: no index
    # check fires, and the results are the regular build's
    cases = [(5, 300, "bf16"), (40, 4096, "bf16"), (7, 10001, "f32"), (6, 40000, "bf16"),
             (64, 70000, "bf16"), (9, 300008, "f32"), (2, 1300000, "bf16")]
    for rows, cols, dtype in cases:
        q = problem(rows, cols, dtype, "layernorm", True, 0.1, "f32", seed=90)
        dy, dh = grads(rows, cols, dtype)

        def step():
            f = forward("layernorm", q)
            return (*f, *backward("layernorm", q, dy, *f[1:], dh, need_dresidual=True),
                    credit.dropout(q["x"], q["drop"]))

        want = step()
        torch.cuda.synchronize()
        with C.use_checked_build():
            got = step()
            assert C.credit_get_device_error(torch.cuda.current_device()) == C.OK
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    credit.dropout(q["x"], q["drop"])  # back on the regular build
    assert credit.device_error() == 0


def test_torch_layer_rejects_bad_tensors():
    q = problem(4, 64, "f32", "layernorm", True, 0.2, "f32")
    x, res, g, b = q["x"], q["residual"], q["gamma"], q["beta"]
    dy = make((4, 64), torch.float32, 3)
    y, h, mean, rstd = forward("layernorm", q)
    with pytest.raises(ValueError):
        credit.dropout(x.t(), q["drop"])                      # not contiguous
    with pytest.raises(ValueError):
        credit.dropout(x, q["drop"], residual=res[:2])
    with pytest.raises(ValueError):
        credit.layernorm_forward(x, g[:63], b)
    with pytest.raises(ValueError):
        credit.layernorm_forward(x, g, b.bfloat16())          # one parameter dtype
    with pytest.raises(ValueError):
        credit.layernorm_forward(x, g, b, residual=res.bfloat16())
    with pytest.raises(ValueError):
        credit.layernorm_forward(x, g, b, out=torch.empty(4, 32, device="cuda"))
    with pytest.raises(TypeError):
        credit.rmsnorm_forward(x.half(), g)
    with pytest.raises(ValueError):
        credit.layernorm_backward(dy, h, mean[:3], rstd, g)
    with pytest.raises(ValueError):
        credit.layernorm_backward(dy, h, None, rstd, g)
    with pytest.raises(ValueError):
        credit.layernorm_backward(dy, h, mean, rstd.double(), g)
    with pytest.raises(ValueError):
        credit.rmsnorm_backward(dy, None, rstd, g)
    with pytest.raises(credit.CreditError):
        credit.layernorm_backward(dy, h, mean, rstd, g, dropout=q["drop"], dx=dy, dresidual=dy)
    with pytest.raises(credit.CreditError):
        credit.layernorm_forward(x, g, b, eps=-1.0)
    with pytest.raises(ValueError):
        credit.dropout(torch.zeros(4, 0, device="cuda"), q["drop"])
    assert credit.device_error() == 0
