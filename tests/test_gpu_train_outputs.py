"""What the training operators hand back beside y: h where a caller asks for
it, and gradients formed from what the forward pass returned, in every form
(a warp, a ring, a team, a sweep a row), aligned and odd."""
import time

import pytest
import torch

import dsmem_thread_block_gb300 as credit
from dsmem_thread_block_gb300 import _credit as C

import test_gpu_train_ops as T

pytestmark = pytest.mark.gpu

# a warp a row; rings of one CTA (two rows a turn where there are many) and of
# several; a team; a sweep
FORMS = [(5, 512), (700, 4096), (9, 5000), (6, 10001), (3, 40000), (5, 300008), (4, 300001),
         (2, 1300000), (2, 1200001)]


def same(got, want):
    return all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("norm", ["layernorm", "rmsnorm"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows, cols", FORMS)
def test_h_out_without_residual_and_dropout(rows, cols, dtype, norm):
    # h is x then, and a buffer given for it holds a copy
    q = T.problem(rows, cols, dtype, norm, False, 0.0, "f32", seed=23)
    want = T.forward(norm, q)
    T.check_forward(norm, q, want)
    for drop in (None, credit.Dropout(0.0, 1)):
        buf = torch.full_like(q["x"], 7.0)
        got = T.forward(norm, dict(q, drop=drop), h_out=buf)
        assert got[1] is buf and same(got, want)
    x = q["x"].clone()  # x itself as h's buffer
    got = T.forward(norm, dict(q, x=x), h_out=x)
    assert got[1] is x and same(got, want)
    assert credit.device_error() == 0


@pytest.mark.parametrize("norm", ["layernorm", "rmsnorm"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows, cols", FORMS)
def test_y_in_place_of_x_leaves_h(rows, cols, dtype, norm):
    # y overwrites x: the h handed back is what x held, and a backward pass on
    # it is the one on untouched buffers
    q = T.problem(rows, cols, dtype, norm, False, 0.0, "f32", seed=29)
    want = T.forward(norm, q)
    dy, _ = T.grads(rows, cols, dtype)
    back = T.backward(norm, q, dy, *want[1:], None)
    for drop, given in ((None, False), (credit.Dropout(0.0, 1), False), (None, True)):
        x = q["x"].clone()
        kw = {"h_out": torch.full_like(x, 7.0)} if given else {}
        got = T.forward(norm, dict(q, x=x, drop=drop), out=x, **kw)
        assert got[0] is x and got[1] is not x and same(got, want)
        assert same(T.backward(norm, q, dy, *got[1:], None), back)
    assert credit.device_error() == 0


def test_y_in_place_of_an_empty_x():
    x = torch.empty(0, 64, device="cuda")
    y, h, mean, rstd = credit.layernorm_forward(x, out=x)
    assert y is x and h.shape == (0, 64) and mean.numel() == rstd.numel() == 0


@pytest.mark.parametrize("rows, cols, dtype", [(16000, 1024, "bf16"), (2500, 4096, "f32"),
                                               (420, 20000, "bf16"), (180, 70001, "f32"),
                                               (70, 300008, "bf16")])
def test_stages_filled_again_after_a_cut_line(rows, cols, dtype):
    # matrices that start inside a 16-byte line: the first row's stage holds
    # elements that were copied one by one, and whole lines of later rows after
    # that; every output repeats and is the definition's
    for norm in ("layernorm", "rmsnorm"):
        q = T.problem(rows, cols, dtype, norm, True, 0.0, "f32", seed=37)
        for n in (1, 3):
            q2 = dict(q, x=T.offset_by(q["x"], n), residual=T.offset_by(q["residual"], n + 1))
            out = T.forward(norm, q2)
            T.check_forward(norm, q2, out)
            assert same(T.forward(norm, q2), out)
            dy, dh = T.grads(rows, cols, dtype)
            dy, dh, h = T.offset_by(dy, n), T.offset_by(dh, n + 1), T.offset_by(out[1], n)
            back = T.backward(norm, q2, dy, h, *out[2:], dh)
            T.check_backward(norm, q2, dy, h, *out[2:], dh, back)
            assert same(T.backward(norm, q2, dy, h, *out[2:], dh), back)
    assert credit.device_error() == 0


@pytest.mark.parametrize("norm", ["layernorm", "rmsnorm"])
@pytest.mark.parametrize("rows, cols, dtype", [(37, 1300000, "bf16"), (45, 900000, "bf16"),
                                               (43, 900001, "bf16"), (23, 1300000, "f32"),
                                               (21, 1000003, "f32")])
def test_sweep_of_several_batches(rows, cols, dtype, norm):
    # rows beyond the teams', in several batches with an uneven last one: a
    # launch sums one batch while it writes the one before, and the parameters'
    # sums go on from batch to batch
    for residual, p in ((True, 0.1), (False, 0.0)):
        q = T.problem(rows, cols, dtype, norm, residual, p, "f32", seed=43)
        out = T.forward(norm, q)
        T.check_forward(norm, q, out)
        dy, dh = T.grads(rows, cols, dtype)
        dh = dh if residual else None
        back = T.backward(norm, q, dy, *out[1:], dh, need_dresidual=residual)
        T.check_backward(norm, q, dy, *out[1:], dh, back)
        # in place: a batch is written while the next one's rows are summed
        x = q["x"].clone()
        res = q["residual"].clone() if residual else None
        got = T.forward(norm, dict(q, x=x, residual=res), out=x, h_out=res)
        assert got[0] is x and same(got, out)
        dy2, h2 = dy.clone(), out[1].clone()
        got = T.backward(norm, q, dy2, h2, *out[2:], dh, need_dresidual=residual, dx=dy2,
                         dresidual=h2 if p else None)
        assert got[0] is dy2 and same(got, back)
    assert credit.device_error() == 0


def test_sweep_of_several_batches_captured():
    rows, cols = 21, 1300000
    q = T.problem(rows, cols, "bf16", "layernorm", True, 0.1, "f32", seed=47)
    dy, dh = T.grads(rows, cols, "bf16")

    def step():
        f = T.forward("layernorm", q)
        return (*f, *T.backward("layernorm", q, dy, *f[1:], dh, need_dresidual=True))

    want = step()
    T.check_forward("layernorm", q, want[:4])
    T.check_backward("layernorm", q, dy, *want[1:4], dh, want[4:])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same(out, want)
    assert credit.device_error() == 0


@pytest.mark.parametrize("cols", [256, 1001, 4096, 40000, 300008])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinity_in_a_kept_element(cols, dtype):
    q = T.problem(5, cols, dtype, "layernorm", True, 0.5, "f32", seed=53)
    j = int(q["mask"][2].nonzero()[-1])  # the row's last kept column
    x = q["x"].clone()
    x[2, j] = float("inf")
    rows = [0, 1, 3, 4]
    clean = T.forward("layernorm", q)
    y, h, mean, rstd = T.forward("layernorm", dict(q, x=x))
    # h - mean is -inf, and NaN at the infinity: so is the variance
    assert bool(y[2].isnan().all()) and bool(rstd[2].isnan()) and float(mean[2]) == float("inf")
    assert float(h[2, j]) == float("inf") and bool(h[2].isinf().sum() == 1)
    assert all(torch.equal(a[rows], b[rows]) for a, b in zip((y, h, mean, rstd), clean))
    # the mean square is infinite, 1 / sqrt of it zero
    clean = T.forward("rmsnorm", q)
    y, h, _, rstd = T.forward("rmsnorm", dict(q, x=x))
    assert float(rstd[2]) == 0.0 and bool(y[2, j].isnan()) and int((y[2] != 0).sum()) == 1
    assert all(torch.equal(a[rows], b[rows]) for a, b in zip((y, h, rstd), (clean[0], clean[1],
                                                                           clean[3])))


@pytest.mark.parametrize("cols", [256, 512, 4096, 8192])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_variance_without_eps(cols, dtype):
    # widths whose reciprocal is exact, so that the mean is: 0 / 0 in the
    # definition, NaN, and the statistics as they are (1 / sqrt within 2 units
    # in the last place, 4 u)
    x = torch.full((3, cols), 2.0, device="cuda", dtype=T.R.DT[dtype])
    y, h, mean, rstd = credit.layernorm_forward(x, eps=0.0)
    assert bool(y.isnan().all()) and bool((mean == 2.0).all()) and bool(rstd.isposinf().all())
    y, _, rstd = credit.rmsnorm_forward(x, eps=0.0)
    assert bool(((rstd - 0.5).abs() <= 4 * T.R.U * 0.5).all())
    assert bool(((y.double() - 1.0).abs() <= 6 * T.R.U + T.R.U_OUT[x.dtype]).all())
    y, _, rstd = credit.rmsnorm_forward(torch.zeros_like(x), eps=0.0)
    assert bool(y.isnan().all()) and bool(rstd.isposinf().all())


def test_dropout_overflow_and_signed_zero():
    big = torch.finfo(torch.float32).max
    for cols in (64, 1001):
        x = torch.full((2, cols), big, device="cuda")
        x[1] = -0.0
        drop = credit.Dropout(0.5, 9, 4)
        keep = T.R.keep_mask(2, cols, 0.5, 9, 4).cuda()
        y = credit.dropout(x, drop)
        assert bool(y[0][keep[0]].isposinf().all()) and bool((y[0][~keep[0]] == 0).all())
        assert torch.equal(y[1].signbit(), keep[1]) and bool((y[1] == 0).all())


def test_device_word_with_new_storage():
    x = T.make((4, 4096), torch.float32, 5)
    word = torch.zeros(1, dtype=torch.int64, device="cuda")
    drop = credit.Dropout(0.5, 21, 3, word)
    assert torch.equal(credit.dropout(x, drop), credit.dropout(x, credit.Dropout(0.5, 21, 3)))
    word.data = torch.full((1,), 6, dtype=torch.int64, device="cuda")
    assert torch.equal(credit.dropout(x, drop), credit.dropout(x, credit.Dropout(0.5, 21, 9)))


@pytest.mark.parametrize("rows, cols, dtype, pdtype", [
    (40, 512, "bf16", "bf16"), (9, 5000, "f32", "f32"), (64, 8192, "bf16", "f32"),
    (5, 300008, "bf16", "bf16"), (9, 1300000, "bf16", "f32")])
def test_gradient_of_beta_without_gamma(rows, cols, dtype, pdtype):
    # the forward pass takes beta alone, so the backward pass gives its gradient
    q = T.problem(rows, cols, dtype, "layernorm", False, 0.0, pdtype, seed=59)
    beta, q["gamma"] = q["beta"].view(1, cols), None
    out = T.forward("layernorm", dict(q, beta=beta))
    T.check_forward("layernorm", q, out)
    dy, _ = T.grads(rows, cols, dtype)
    back = T.backward("layernorm", q, dy, *out[1:], None, beta=beta)
    assert back[2] is None and back[3].shape == beta.shape and back[3].dtype == beta.dtype
    _, rx, _, rb, _, ex, _, eb = T.R.ref_backward("layernorm", dy, None, *out[1:], None, 0.0, None)
    T.R.assert_close(back[0], rx, T.R.U_OUT[dy.dtype] * rx.abs() + T.R.U * ex, "dx")
    T.R.assert_close(back[3].view(-1), rb, T.R.U_OUT[beta.dtype] * rb.abs() + T.R.U * eb, "dbeta")
    # beside gamma the same call takes beta's shape, and without either gives none
    gamma = torch.ones_like(beta).view(-1)
    both = credit.layernorm_backward(dy, *out[1:], gamma, beta=beta)
    assert both[2].shape == gamma.shape and both[3].shape == beta.shape
    assert torch.equal(both[3], back[3]) and torch.equal(both[0], back[0])
    assert T.backward("layernorm", q, dy, *out[1:], None)[2:] == (None, None)
    with pytest.raises(ValueError):
        credit.layernorm_backward(dy, *out[1:], beta=beta[:, :-1].contiguous())
    with pytest.raises(ValueError):
        credit.layernorm_backward(dy, *out[1:], gamma, beta=beta.to(
            torch.float32 if pdtype == "bf16" else torch.bfloat16))
    assert credit.device_error() == 0


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta):
        y, h, mean, rstd = credit.layernorm_forward(x, gamma, beta)
        ctx.save_for_backward(h, mean, rstd, gamma)
        return y

    @staticmethod
    def backward(ctx, dy):
        dx, _, dgamma, dbeta = credit.layernorm_backward(dy.contiguous(), *ctx.saved_tensors)
        return dx, dgamma, dbeta


def test_the_pair_inside_an_autograd_function():
    q = T.problem(33, 1500, "f32", "layernorm", False, 0.0, "f32", seed=61)
    leaves = [q[k].clone().requires_grad_() for k in ("x", "gamma", "beta")]
    with pytest.raises(RuntimeError, match="record no autograd graph"):
        credit.layernorm_forward(*leaves)
    y = LayerNorm.apply(*leaves)
    dy, _ = T.grads(33, 1500, "f32")
    y.backward(dy)
    with torch.no_grad():
        out = credit.layernorm_forward(*leaves)  # a step written out by hand
        assert torch.equal(y, out[0])
        T.check_backward("layernorm", q, dy, *out[1:], None,
                         (leaves[0].grad, None, leaves[1].grad, leaves[2].grad))


def test_tensors_written_in_place_are_known_to_autograd():
    # a tensor that an earlier product saved is overwritten: its backward pass
    # is refused, as after torch's own in-place operators
    def saved():
        x = T.make((4, 512), torch.float32, 5)
        w = torch.ones(512, device="cuda", requires_grad=True)
        return x, (x * w).sum()

    dy, _ = T.grads(4, 512, "f32")
    h = T.make((4, 512), torch.float32, 6)
    s = torch.ones(4, device="cuda")
    drop = credit.Dropout(0.5, 3)
    writes = [lambda x: credit.dropout(x, drop, out=x),
              lambda x: credit.layernorm_forward(x, out=x),
              lambda x: credit.rmsnorm_forward(h, residual=x, h_out=x),
              lambda x: credit.layernorm_backward(x, h, s, s, dx=x),
              lambda x: credit.rmsnorm_backward(dy, x, s, dropout=drop, dresidual=x)]
    for write in writes:
        x, loss = saved()
        write(x)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    x, loss = saved()
    credit.layernorm_forward(x)  # reading leaves it as it is
    loss.backward()
    with torch.inference_mode():
        x = T.make((4, 512), torch.float32, 5)
    credit.layernorm_forward(x, out=x)  # a tensor without a version


def test_a_team_whose_wait_gives_up_ends():
    # a CTA whose peer never deposits: it gives up after a second, and its other
    # 39 turns and the waits of its other warps cost no second each
    dev = torch.cuda.current_device()
    assert credit.device_error(dev) == 0
    for load in (C.load(), None):
        t0 = time.monotonic()
        if load is not None:
            assert C.credit_selftest_team_timeout(dev) == C.ERR_DEVICE_TIMEOUT
        else:
            with C.use_checked_build():
                assert C.credit_selftest_team_timeout(dev) == C.ERR_DEVICE_TIMEOUT
        assert time.monotonic() - t0 < 5.0
    assert credit.device_error(dev) == 0  # read and cleared
    q = T.problem(13, 300008, "bf16", "layernorm", True, 0.1, "f32", seed=67)
    T.check_forward("layernorm", q, T.forward("layernorm", q))
    assert credit.device_error(dev) == 0
