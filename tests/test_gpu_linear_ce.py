"""The linear head's cross entropy and its gradient against their definition in
64 bits.

Bounds count roundings, u = 2^-24.  A logit is a sum of D products that are exact
in fp32 (bf16 operands), added sixteen at a time; the tensor cores do not say how
they round, so an addition may drop up to a whole last digit, 2 u of the sum of
magnitudes: ez = 2 u (D / 16 + 17) sum |h w|.  fp32 operands take six such sums
and leave out 3 u sum |h w|.  lse moves by no more than the worst logit does; its
exponentials err by their argument's roundings, 4 u (max - min), and by 4 u, its
sum by 100 additions, the logarithm and the sum with the maximum by 4 u |lse|.
g errs by its logit's and lse's argument, and is rounded to bf16 (2^-8) for the
products of more than 32 tokens; fewer keep two terms, or fp32, fp32 operands three
(u).  dhidden and dweight sum over V and D terms
as the logits do over D, in fp32 parts that are added in order, and are rounded
once.  Where operands are small whole numbers every product and sum is exact, and
so is the comparison.
"""
import pytest
import torch

import dsmem_thread_block_gb300 as credit
from dsmem_thread_block_gb300 import _credit as C
from train_helpers import DT, U, U_OUT, assert_close

pytestmark = pytest.mark.gpu
IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def no_device_error():
    yield
    assert C.credit_get_device_error(torch.cuda.current_device()) == C.OK


def make(tokens, hidden, vocab, dtype, seed=0, spread=2.5, ignored=0.2):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.randn((tokens, hidden), generator=g, device="cuda").to(dtype)
    w = (torch.randn((vocab, hidden), generator=g, device="cuda") * (spread / hidden ** 0.5)).to(dtype)
    target = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    skip = torch.rand((tokens,), generator=g, device="cuda") < ignored
    return h, w, torch.where(skip, torch.full_like(target, IGNORE), target)


def sums_err(n, dtype, mag):
    """Of n products added up, `mag` the sum of their magnitudes."""
    one = 2 * U * (n / 16 + 17) * mag
    return one if dtype == torch.bfloat16 else 6 * one + 3 * U * mag


def ref_logits(h, w):
    z = h.double() @ w.double().t()
    return z, sums_err(h.shape[1], h.dtype, h.double().abs() @ w.double().abs().t())


def ref_forward(h, w, target, ignore=IGNORE):
    z, ez = ref_logits(h, w)
    lse = torch.logsumexp(z, 1)
    span = (z.amax(1) - z.amin(1)).abs()
    e = ez.amax(1) + U * (104 + 4 * span + 4 * lse.abs() + 4 * z.amax(1).abs())
    kept = target != ignore
    at = torch.where(kept, target, torch.zeros_like(target))[:, None]
    loss = torch.where(kept, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    el = torch.where(kept, e + ez.gather(1, at)[:, 0] + U * loss.abs(), torch.zeros_like(e))
    return loss, lse, el, e


def ref_backward(dloss, dlse, h, w, target, lse, ignore=IGNORE):
    z, ez = ref_logits(h, w)
    kept = target != ignore
    scale = torch.where(kept, dloss.double(), torch.zeros_like(dloss.double()))
    both = scale + (dlse.double() if dlse is not None else 0.0)
    x = z - lse.double()[:, None]
    p = x.exp()
    g = both[:, None] * p
    eg = (both.abs() + 2 * U * scale.abs())[:, None] * p * (ez + U * (6 * x.abs() + 2 * z.abs() + 10))
    at = torch.where(kept, target, torch.zeros_like(target))[:, None]
    g.scatter_add_(1, at, -scale[:, None])
    del z, ez, x, p
    eg += (U_OUT[h.dtype] + 2 * U) * (g.abs() + eg)
    hd, wd = h.double(), w.double()
    dh, dw = g @ wd, g.t() @ hd
    # (up to 64 parts of a sum over the vocabulary)
    bh = eg @ wd.abs() + sums_err(w.shape[0] + 1024, h.dtype, g.abs() @ wd.abs())
    bw = eg.t() @ hd.abs() + sums_err(h.shape[0], h.dtype, g.abs().t() @ hd.abs())
    uo = U_OUT[h.dtype]
    return dh, dw, bh * (1 + uo) + uo * dh.abs(), bw * (1 + uo) + uo * dw.abs()


SHAPES = [(1, 8, 1), (1, 64, 2), (2, 1, 3), (3, 7, 255), (31, 64, 256), (33, 100, 257), (128, 65, 1000),
          (129, 512, 513), (300, 1001, 5003), (64, 1024, 4096), (1, 4096, 20000), (1000, 16, 40),
          (257, 192, 1), (5, 2056, 777), (8, 264, 1000), (9, 264, 1000), (4, 1001, 3001), (8, 4096, 600),
          (6, 33, 130), (1, 20000, 37), (1, 30000, 40), (38, 4864, 246), (124, 2415, 128),
          (3000, 40, 100), (40, 8192, 1), (2100, 136, 300), (9, 256, 65536), (13, 1001, 17000),
          (16, 264, 63551), (17, 260, 65003), (16, 256, 65535), (8, 6400, 300), (8, 6401, 300)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,hidden,vocab", SHAPES)
def test_forward(tokens, hidden, vocab, dtype):
    h, w, target = make(tokens, hidden, vocab, DT[dtype], seed=tokens + vocab)
    loss, lse = credit.linear_cross_entropy_forward(h, w, target)
    assert loss.dtype == lse.dtype == torch.float32 and loss.shape == lse.shape == target.shape
    want, want_lse, bound, bound_lse = ref_forward(h, w, target)
    assert_close(lse, want_lse, bound_lse, "lse")
    assert_close(loss, want, bound, "loss")
    assert bool((loss[target == IGNORE] == 0).all())


@pytest.mark.parametrize("zloss", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,hidden,vocab", SHAPES)
def test_backward(tokens, hidden, vocab, dtype, zloss):
    h, w, target = make(tokens, hidden, vocab, DT[dtype], seed=2 * tokens + vocab)
    lse = torch.logsumexp(h.double() @ w.double().t(), 1).float()
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    dloss = torch.randn((tokens,), generator=g, device="cuda")
    dlse = 0.1 * torch.randn((tokens,), generator=g, device="cuda") if zloss else None
    dh, dw = credit.linear_cross_entropy_backward(dloss, h, w, target, lse, dlse=dlse)
    want_h, want_w, bound_h, bound_w = ref_backward(dloss, dlse, h, w, target, lse)
    assert dh.dtype == dw.dtype == h.dtype and dh.shape == h.shape and dw.shape == w.shape
    assert_close(dh, want_h, bound_h, "dhidden")
    assert_close(dw, want_w, bound_w, "dweight")


def whole_numbers(shape, top, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(dtype)


# (8192 tokens: the vocabulary in two pieces; few tokens: parts of a sum over it)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,hidden,vocab", [(1, 8, 5), (7, 72, 300), (4, 1001, 2000), (11, 72, 300), (130, 264, 700), (300, 1001, 1000),
                                                 (200, 24, 20011), (5000, 72, 130), (130, 3000, 200), (20, 5000, 333), (8192, 40, 20000), (4099, 72, 33333)])
def test_gradients_of_whole_numbers_are_exact(tokens, hidden, vocab, dtype):
    # with w = 0 (or h = 0) every logit is 0, and with lse = 0 every p is 1:
    # g = dloss (1 - [target]) + dlse, whole numbers
    dt = DT[dtype]
    _, _, target = make(tokens, 1, vocab, dt, seed=vocab)
    dloss, dlse = (whole_numbers((tokens,), 1, torch.float32, s) for s in (1, 2))
    lse = torch.zeros((tokens,), device="cuda")
    g = (torch.where(target == IGNORE, torch.zeros_like(dloss), dloss) + dlse)[:, None].double().expand(
        tokens, vocab).clone()
    rows = (target != IGNORE).nonzero()[:, 0]
    g[rows, target[rows]] -= dloss[rows].double()
    h, w = whole_numbers((tokens, hidden), 1, dt, 3), torch.zeros((vocab, hidden), device="cuda", dtype=dt)
    dh, dw = credit.linear_cross_entropy_backward(dloss, h, w, target, lse, dlse=dlse)
    assert bool((dh == 0).all())
    assert torch.equal(dw, (g.t() @ h.double()).float().to(dt))
    h, w = torch.zeros_like(h), whole_numbers((vocab, hidden), 1, dt, 4)
    dh, dw = credit.linear_cross_entropy_backward(dloss, h, w, target, lse, dlse=dlse)
    assert bool((dw == 0).all())
    assert torch.equal(dh, (g @ w.double()).float().to(dt))


@pytest.mark.parametrize("tokens", [1, 3, 70])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_logits_neither_overflow_nor_vanish(dtype, tokens):
    h, w, target = make(tokens, 128, 900, DT[dtype], seed=3, spread=2000.0, ignored=0.0)
    loss, lse = credit.linear_cross_entropy_forward(h, w, target)
    want, want_lse, bound, bound_lse = ref_forward(h, w, target)
    assert bool(torch.isfinite(loss).all()) and float(want_lse.max()) > 500
    assert_close(lse, want_lse, bound_lse, "lse")
    assert_close(loss, want, bound, "loss")


@pytest.mark.parametrize("tokens,hidden", [(1, 64), (4, 65), (4, 64), (50, 64)])
def test_what_a_forward_pass_leaves_makes_a_gradient_without_a_sum(tokens, hidden):
    # sum_v g_tv = dloss (sum_v p_tv - 1) = 0: with a weight of ones dhidden is 0, but
    # for the roundings of p, and a wrong lse shows
    h, w, target = make(tokens, hidden, 700, torch.bfloat16, seed=21, ignored=0.0)
    w[:, 0] = 1
    loss, lse = credit.linear_cross_entropy_forward(h, w, target)
    dh, _ = credit.linear_cross_entropy_backward(torch.ones(tokens, device="cuda"), h, w, target, lse)
    # g: 2^-8 of each p, which add up to 1, and of p - 1
    assert float(dh[:, 0].abs().max()) <= 2 * 2.0 ** -8 + 1e-4


@pytest.mark.parametrize("hidden", [72, 4104])
def test_targets_at_every_place_of_a_tile_and_outside(hidden):
    vocab, tokens = 600, 600
    h, w, _ = make(tokens, hidden, vocab, torch.bfloat16, seed=9)
    target = torch.arange(tokens, device="cuda")
    loss, _ = credit.linear_cross_entropy_forward(h, w, target)
    want, _, bound, _ = ref_forward(h, w, target)
    assert_close(loss, want, bound, "loss")
    lse = torch.logsumexp(h.double() @ w.double().t(), 1).float()
    dloss = torch.ones(tokens, device="cuda")
    bad = target.clone()
    bad[5], bad[130], bad[7], bad[8] = -1, vocab, 1 << 62, -(1 << 62)
    loss, lse2 = credit.linear_cross_entropy_forward(h, w, bad)
    out = torch.zeros(tokens, dtype=torch.bool, device="cuda")
    out[[5, 130, 7, 8]] = True
    assert bool(torch.isnan(loss[out]).all()) and bool(torch.isfinite(loss[~out]).all())
    assert bool(torch.isfinite(lse2).all())
    for n in (1, 8):  # a few tokens, of whole lines and not
        one, _ = credit.linear_cross_entropy_forward(h[4:4 + n].float(), w.float(), bad[4:4 + n])
        assert bool((torch.isnan(one) == out[4:4 + n]).all())
        dh, _ = credit.linear_cross_entropy_backward(dloss[:n], h[4:4 + n].float(), w.float(), bad[4:4 + n],
                                                     lse[4:4 + n])
        assert bool((torch.isnan(dh).any(1) == out[4:4 + n]).all())
    dh, dw = credit.linear_cross_entropy_backward(dloss, h, w, bad, lse)
    assert bool(torch.isnan(dh[out]).all()) and bool(torch.isfinite(dh[~out]).all())
    # ignore_index may be any number, one of the vocabulary's too
    loss, _ = credit.linear_cross_entropy_forward(h, w, target, ignore_index=17)
    assert float(loss[17]) == 0 and bool((loss[:17] > 0).all())


@pytest.mark.parametrize("tokens,hidden", [(1, 64), (3, 65), (2, 64), (140, 64)])
def test_every_target_ignored(tokens, hidden):
    h, w, target = make(tokens, hidden, 300, torch.bfloat16, ignored=2.0)
    dloss = torch.full((tokens,), float("nan"), device="cuda")  # of ignored tokens: not looked at
    loss, lse = credit.linear_cross_entropy_forward(h, w, target)
    assert bool((loss == 0).all())
    dh, dw = credit.linear_cross_entropy_backward(dloss, h, w, target, lse)
    assert bool((dh == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,hidden", [(5, 64), (40, 64), (40, 4096)])
def test_one_token_that_is_not_finite_leaves_the_others(dtype, tokens, hidden):
    h, w, target = make(tokens, hidden, 500, DT[dtype], seed=4, ignored=0.0)
    loss, lse = credit.linear_cross_entropy_forward(h, w, target)
    for value in (float("nan"), float("inf")):
        hb = h.clone()
        hb[3, 5] = value
        lb, sb = credit.linear_cross_entropy_forward(hb, w, target)
        rest = torch.arange(tokens, device="cuda") != 3
        assert torch.equal(lb[rest], loss[rest]) and torch.equal(sb[rest], lse[rest])
        assert not bool(torch.isfinite(sb[3]))
    # a padded token's infinite exponentials give no gradient to the hidden states
    tb = target.clone()
    tb[3] = IGNORE
    big = lse.clone()
    big[3] = -1e30
    dh, _ = credit.linear_cross_entropy_backward(torch.ones(tokens, device="cuda"), h, w, tb, big)
    assert bool((dh[3] == 0).all())


def guarded(shape, dtype):
    """A tensor between two guards, and the whole of them."""
    n = 1
    for s in shape:
        n *= s
    whole = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
    return whole[32:32 + n].view(shape), whole


@pytest.mark.parametrize("tokens", [3, 150])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_addresses_and_given_outputs(dtype, shift, tokens):
    hidden, vocab = 72, 410
    dt = DT[dtype]
    h, w, target = make(tokens, hidden, vocab, dt, seed=6)
    dloss = torch.rand(tokens, device="cuda")
    loss, lse = credit.linear_cross_entropy_forward(h, w, target)
    dh, dw = credit.linear_cross_entropy_backward(dloss, h, w, target, lse)

    def moved(t):
        room = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        room[shift:] = t.reshape(-1)
        return room[shift:].view(t.shape)

    hm, wm = moved(h), moved(w)
    loss2, lse2 = credit.linear_cross_entropy_forward(hm, wm, target)
    if tokens > 8:  # (a few tokens' dot products are added in another order at other addresses)
        assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    want, want_lse, bound, bound_lse = ref_forward(h, w, target)
    assert_close(lse2, want_lse, bound_lse, "lse")
    assert_close(loss2, want, bound, "loss")
    oh, all_h = guarded(h.shape, dt)
    ow, all_w = guarded((vocab * hidden + 1,), dt)
    ow = ow[1:].view(vocab, hidden) if shift else guarded(w.shape, dt)[0]
    rh, rw = credit.linear_cross_entropy_backward(dloss, hm, wm, target, lse, dhidden=oh, dweight=ow)
    assert rh is oh or rh.data_ptr() == oh.data_ptr()
    if tokens > 8:
        assert torch.equal(oh, dh) and torch.equal(ow, dw)
    want_h, want_w, bound_h, bound_w = ref_backward(dloss, None, h, w, target, lse)
    assert_close(oh, want_h, bound_h, "dhidden")
    assert_close(ow, want_w, bound_w, "dweight")
    assert bool((all_h[:32] == 7).all()) and bool((all_h[-32:] == 7).all())
    if shift:
        assert bool((all_w[:33] == 7).all()) and bool((all_w[-32:] == 7).all())


@pytest.mark.parametrize("need_h,need_w", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("tokens,hidden", [(1, 136), (7, 133), (7, 136), (200, 136)])
def test_gradients_that_are_not_needed(need_h, need_w, tokens, hidden):
    h, w, target = make(tokens, hidden, 3000, torch.bfloat16, seed=8)
    dloss = torch.rand(tokens, device="cuda")
    _, lse = credit.linear_cross_entropy_forward(h, w, target)
    want = ref_backward(dloss, None, h, w, target, lse)
    dh, dw = credit.linear_cross_entropy_backward(dloss, h, w, target, lse, need_dhidden=need_h,
                                                  need_dweight=need_w)
    if need_h:
        assert_close(dh, want[0], want[2], "dhidden")
    else:
        assert dh is None
    if need_w:
        assert_close(dw, want[1], want[3], "dweight")
    else:
        assert dw is None


@pytest.mark.parametrize("tokens", [1, 20])
def test_a_weight_of_more_elements_than_31_bits_count(tokens):
    hidden, vocab = 8192, 270000
    h, _, target = make(tokens, hidden, 8, torch.bfloat16, seed=15, ignored=0.0)
    w = torch.zeros((vocab, hidden), dtype=torch.bfloat16, device="cuda")
    # a few words of all zeros' company, the last one among them
    words = torch.tensor([0, 5, 131071, 262143, 262144, vocab - 1], device="cuda")
    w[words] = make(1, hidden, 6, torch.bfloat16, seed=16)[1] * 4
    target = words[torch.arange(tokens, device="cuda") % 6]
    loss, lse = credit.linear_cross_entropy_forward(h, w, target)
    z, ez = ref_logits(h, w[words])
    want = torch.logsumexp(torch.cat([z, torch.full((tokens, 1), (vocab - 6.0), device="cuda").double().log()], 1), 1)
    e = ez.amax(1) + U * (104 + 8 * z.abs().amax(1) + 4 * want)
    picked = z[torch.arange(tokens, device="cuda"), torch.arange(tokens, device="cuda") % 6]
    assert_close(lse, want, e, "lse")
    assert_close(loss, want - picked, e + ez.amax(1), "loss")
    dloss = torch.ones(tokens, device="cuda")
    dh, dw = credit.linear_cross_entropy_backward(dloss, h, w, target, lse)
    # Of the words: the others' logits are 0.  g = p - [target] errs as p does, whose
    # argument errs by its logit's and lse's roundings, and by its own rounding to
    # bf16; the products add their sums' and outputs' roundings (ref_backward's bounds).
    x = z - lse.double()[:, None]
    p = x.exp()
    g, eg = p.clone(), p * (ez + U * (6 * x.abs() + 2 * z.abs() + 10))
    g[torch.arange(tokens), torch.arange(tokens) % 6] -= 1
    eg = eg + (2.0 ** -8 + 2 * U) * (g.abs() + eg)
    hd, wd = h.double(), w[words].double()

    def bound(e, a, b, n):
        mag = a.abs() @ b.abs()
        return (e @ b.abs() + sums_err(n, h.dtype, mag)) * 1.01 + 2.0 ** -8 * (a @ b).abs()

    assert_close(dw[words], g.t() @ hd, bound(eg.t(), g.t(), hd, tokens), "dweight")
    assert_close(dh, g @ wd, bound(eg, g, wd, vocab), "dhidden")
    # a word that is all zeros, anywhere: its logit is exactly 0
    rest = (-lse.double()).exp()[:, None]
    er = rest * U * (6 * lse.double().abs()[:, None] + 10) + (2.0 ** -8 + 2 * U) * rest
    for v in (1, 131072, 262145, vocab - 2):
        assert_close(dw[v], (rest.t() @ hd)[0], bound(er.t(), rest.t(), hd, tokens)[0], "dweight")


def test_more_logits_than_32_bits_count():
    # the first 1000 tokens over and over: every copy gets the same bits
    hidden, vocab, copies = 24, 61000, 72
    h, w, target = make(1000, hidden, vocab, torch.bfloat16, seed=17)
    dloss = torch.rand(1000, device="cuda")
    many = [t.repeat((copies,) + (1,) * (t.dim() - 1)) for t in (h, target, dloss)]
    loss, lse = credit.linear_cross_entropy_forward(many[0], w, many[1])
    want, want_lse, bound, bound_lse = ref_forward(h, w, target)
    assert_close(lse[:1000], want_lse, bound_lse, "lse")
    assert_close(loss[:1000], want, bound, "loss")
    for t in (loss, lse):
        assert bool((t.view(copies, 1000) == t[:1000]).all())
    dh, dw = credit.linear_cross_entropy_backward(many[2], many[0], w, many[1], lse)
    want_h, want_w, bound_h, bound_w = ref_backward(dloss, None, h, w, target, lse[:1000])
    assert_close(dh[:1000], want_h, bound_h, "dhidden")
    assert bool((dh.view(copies, 1000, hidden) == dh[:1000]).all())
    # (the sum over 72 times the tokens errs 72 times over 72 times the magnitude)
    assert_close(dw, copies * want_w, copies * copies * bound_w, "dweight")


def test_no_tokens():
    w = torch.ones((20, 16), device="cuda", dtype=torch.bfloat16)
    h = torch.empty((0, 16), device="cuda", dtype=torch.bfloat16)
    target, none = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    loss, lse = credit.linear_cross_entropy_forward(h, w, target)
    assert loss.shape == lse.shape == (0,)
    dh, dw = credit.linear_cross_entropy_backward(none, h, w, target, lse)
    assert dh.shape == (0, 16) and bool((dw == 0).all())


def test_batches_of_sequences_keep_their_shape():
    h, w, target = make(60, 64, 100, torch.bfloat16)
    loss, lse = credit.linear_cross_entropy_forward(h, w, target)
    h3, t2 = h.view(3, 20, 64), target.view(3, 20)
    loss3, lse3 = credit.linear_cross_entropy_forward(h3, w, t2)
    assert loss3.shape == (3, 20) and torch.equal(loss3.view(-1), loss)
    dh, _ = credit.linear_cross_entropy_backward(loss3, h3, w, t2, lse3)
    assert dh.shape == h3.shape


@pytest.mark.parametrize("tokens,hidden", [(1, 264), (4, 263), (4, 264), (500, 264)])
def test_results_repeat_bit_for_bit_on_any_stream(tokens, hidden):
    h, w, target = make(tokens, hidden, 9000, torch.bfloat16, seed=12)
    dloss = torch.rand(tokens, device="cuda")

    def both():
        loss, lse = credit.linear_cross_entropy_forward(h, w, target)
        return (loss, lse) + credit.linear_cross_entropy_backward(dloss, h, w, target, lse)

    first = both()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    results = []
    for s in streams:  # side by side
        with torch.cuda.stream(s):
            results.append(both())
    torch.cuda.synchronize()
    for r in results:
        assert all(torch.equal(a, b) for a, b in zip(first, r))


@pytest.mark.parametrize("hidden", [264, 263])
@pytest.mark.parametrize("tokens", [9, 13, 16])
def test_fp32_tokens_eight_at_a_time(tokens, hidden):
    """A weight that takes that form: targets outside, ignored and at the ends in each
    eight, a token that is not finite, streams side by side and a graph."""
    vocab = 64007  # (x 263: 2^24 and some)
    h, w, target = make(tokens, hidden, vocab, torch.float32, seed=15, ignored=0.0)
    target[1], target[2], target[3], target[8] = IGNORE, vocab - 1, 0, vocab - 1
    want, want_lse, bound, bound_lse = ref_forward(h, w, target)
    loss, lse = credit.linear_cross_entropy_forward(h, w, target)
    assert_close(lse, want_lse, bound_lse, "lse")
    assert_close(loss, want, bound, "loss")
    rest = torch.ones(tokens, dtype=torch.bool, device="cuda")
    rest[[0, tokens - 1]] = False
    bad, hb = target.clone(), h.clone()
    bad[0], bad[tokens - 1] = vocab, -1
    hb[0, 7] = float("inf")
    lb, sb = credit.linear_cross_entropy_forward(hb, w, bad)
    assert torch.equal(lb[rest], loss[rest]) and torch.equal(sb[rest], lse[rest])
    assert bool(torch.isnan(lb[~rest]).all()) and torch.equal(sb[-1], lse[-1])
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    results = []
    for s in streams:
        with torch.cuda.stream(s):
            results.append(credit.linear_cross_entropy_forward(h, w, target))
    torch.cuda.synchronize()
    assert all(torch.equal(a, loss) and torch.equal(b, lse) for a, b in results)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cl, cs = credit.linear_cross_entropy_forward(h, w, target)
    h.copy_(h.roll(1, 0))
    target.copy_(target.roll(1, 0))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cl, loss.roll(1, 0)) and torch.equal(cs, lse.roll(1, 0))


@pytest.mark.parametrize("tokens", [1, 2, 200])
def test_captured_calls_take_new_inputs(tokens):
    h, w, target = make(tokens, 128, 2100, torch.bfloat16, seed=13)
    dloss = torch.rand(tokens, device="cuda")
    ws = [torch.empty(C.credit_linear_ce_workspace(b, h.data_ptr(), w.data_ptr(), tokens, 128, 2100, C.BF16,
                                                   h.device.index), dtype=torch.uint8, device="cuda")
          for b in (0, 1)]

    def both():
        loss, lse = credit.linear_cross_entropy_forward(h, w, target, workspace=ws[0])
        return (loss, lse) + tuple(credit.linear_cross_entropy_backward(dloss, h, w, target, lse,
                                                                        workspace=ws[1]))

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for seed in (20, 21):
        h2, w2, t2 = make(tokens, 128, 2100, torch.bfloat16, seed=seed)
        h.copy_(h2), w.copy_(w2), target.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, both()))


def test_against_differences():
    # the loss's own change along a direction, in fp32 operands
    h, w, target = make(20, 48, 90, torch.float32, seed=14)
    weight = torch.rand(20, device="cuda").double()
    _, lse = credit.linear_cross_entropy_forward(h, w, target)
    dh, dw = credit.linear_cross_entropy_backward(weight.float(), h, w, target, lse)
    eps = 2.0 ** -12
    for x, d in ((h, dh), (w, dw)):
        v = torch.randn_like(x)
        up = credit.linear_cross_entropy_forward(*((x + eps * v, w) if x is h else (h, x + eps * v)), target)[0]
        dn = credit.linear_cross_entropy_forward(*((x - eps * v, w) if x is h else (h, x - eps * v)), target)[0]
        change = float(((up.double() - dn.double()) * weight).sum()) / (2 * eps)
        # 20 losses of 1e-6 each over 2 eps, and the third derivative's eps^2
        assert abs(change - float((d.double() * v.double()).sum())) < 20 * 4e-6 / (2 * eps) + 0.01


@pytest.mark.parametrize("what", ["dtype", "weight dtype", "strided", "target type", "target shape", "cpu",
                                  "lse shape", "dloss type", "graph", "workspace", "weight shape",
                                  "overlap"])
def test_refusals(what):
    h, w, target = make(12, 64, 100, torch.bfloat16)
    one = torch.ones(12, device="cuda")
    with pytest.raises((ValueError, TypeError, RuntimeError, credit.CreditError)):
        if what == "dtype":
            credit.linear_cross_entropy_forward(h.half(), w.half(), target)
        elif what == "weight dtype":
            credit.linear_cross_entropy_forward(h, w.float(), target)
        elif what == "strided":
            credit.linear_cross_entropy_forward(h, w.t().contiguous().t(), target)
        elif what == "target type":
            credit.linear_cross_entropy_forward(h, w, target.int())
        elif what == "target shape":
            credit.linear_cross_entropy_forward(h, w, target[:-1])
        elif what == "cpu":
            credit.linear_cross_entropy_forward(h, w, target.cpu())
        elif what == "weight shape":
            credit.linear_cross_entropy_forward(h, w[:, :32].contiguous(), target)
        elif what == "lse shape":
            credit.linear_cross_entropy_backward(one, h, w, target, one[:-1])
        elif what == "dloss type":
            credit.linear_cross_entropy_backward(one.double(), h, w, target, one)
        elif what == "graph":
            credit.linear_cross_entropy_forward(h.requires_grad_(), w, target)
        elif what == "workspace":
            credit.linear_cross_entropy_forward(h, w, target, workspace=torch.empty(16, device="cuda"))
        elif what == "overlap":
            credit.linear_cross_entropy_backward(one, h, w, target, one, dhidden=h)
