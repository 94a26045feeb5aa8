"""What the roundings inside the head's cross entropy may cost: the logits' gradient's,
the exponentials' and the long sums'.  u = 2^-24; a rounding to bf16 is off by 2^-8 of
the value at most."""
import pytest
import torch

import dsmem_thread_block_gb300 as credit
from dsmem_thread_block_gb300 import _credit as C
from test_gpu_linear_ce import IGNORE, make
from train_helpers import U, assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def no_device_error():
    yield
    assert C.credit_get_device_error(torch.cuda.current_device()) == C.OK


@pytest.mark.parametrize("n", [3686, 30000, 777, 300])
@pytest.mark.parametrize("tokens,hidden,vocab", [(300, 64, 700), (130, 264, 20011), (150, 4096, 333),
                                                 (3000, 40, 100)])
def test_a_means_dloss_is_not_rounded(tokens, hidden, vocab, n):
    # With an lse of 300 every exponential is 0: g = -dloss of the target, the same number
    # for every token.  dhidden is one product, dloss w, rounded once; dweight a sum of
    # the hidden states of each word's tokens (whole numbers: exact) times dloss.
    h, w, target = make(tokens, hidden, vocab, torch.bfloat16, seed=n)
    h = (3 * h.float()).round().bfloat16()
    lse = torch.full((tokens,), 300.0, device="cuda")
    dloss = torch.full((tokens,), 1.0 / n, device="cuda")
    dloss[::3] = torch.where(target[::3] == IGNORE, float("nan"), dloss[::3])  # (not looked at)
    dh, dw = credit.linear_cross_entropy_backward(dloss, h, w, target, lse)
    kept = target != IGNORE
    one = torch.full((), 1.0 / n, dtype=torch.float32).double().cuda()
    g = torch.zeros((tokens, vocab), dtype=torch.float64, device="cuda")
    g[kept, target[kept]] = -one
    for got, want in ((dh, g @ w.double()), (dw, g.t() @ h.double())):
        # (one rounding to bf16, and fp32's of the factor taken out and put back)
        assert_close(got, want, (2.0 ** -8 + 4 * U) * want.abs(), "gradient")
    # to be sure that it is this that the bound shows: rounded to bf16 first, n's dloss
    # and the output's rounding would pass it
    if n == 777:
        first = (-one).float().bfloat16().double() * w.double()[target[kept]]
        off = (first.float().bfloat16().double() - (g @ w.double())[kept]).abs()
        assert bool((off > (2.0 ** -8 + 4 * U) * (g @ w.double())[kept].abs()).any())


def test_dloss_of_every_size_and_none():
    h, w, target = make(200, 64, 300, torch.bfloat16, seed=2, ignored=0.0)
    lse = torch.logsumexp(h.double() @ w.double().t(), 1).float()
    one = torch.ones(200, device="cuda")
    base = credit.linear_cross_entropy_backward(one, h, w, target, lse)
    for k in (-100, -3, 60):  # a power of two changes the exponents alone
        got = credit.linear_cross_entropy_backward(one * 2.0 ** k, h, w, target, lse)
        assert all(torch.equal(a.double(), b.double() * 2.0 ** k) for a, b in zip(got, base))
    got = credit.linear_cross_entropy_backward(0 * one, h, w, target, lse, dlse=one)
    p = (h.double() @ w.double().t() - lse.double()[:, None]).exp()
    assert float((got[0].double() - p @ w.double()).norm()) < 0.01 * float((p @ w.double()).norm())
    spoilt = one.clone()
    spoilt[7], spoilt[9] = float("inf"), float("nan")
    dh, _ = credit.linear_cross_entropy_backward(spoilt, h, w, target, lse)
    rest = torch.ones(200, dtype=torch.bool, device="cuda")
    rest[[7, 9]] = False
    assert torch.equal(dh[rest], base[0][rest]) and not bool(torch.isfinite(dh[~rest]).any())


def exact_ones(tokens, vocab, seed):
    """With w = 0 (or h = 0) every logit is 0, and with lse = 0 every p is 1: g = dloss (1 -
    [target]) + dlse, of whole numbers, 0, 1, 256 or 257 in magnitude: the last takes two
    bf16 terms."""
    _, _, target = make(tokens, 1, vocab, torch.bfloat16, seed=seed, ignored=0.1)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dloss = torch.randint(0, 2, (tokens,), generator=g, device="cuda").float()
    dlse = (256 * (2 * torch.randint(0, 2, (tokens,), generator=g, device="cuda") - 1)).float()
    counted = torch.where(target == IGNORE, torch.zeros_like(dloss), dloss)
    grad = (counted + dlse)[:, None].double().expand(tokens, vocab).clone()
    rows = (target != IGNORE).nonzero()[:, 0]
    grad[rows, target[rows]] -= dloss[rows].double()
    return target, dloss, dlse, grad


# few tokens' form (fp32 g), whole and split products, several pieces, splits of both sums
@pytest.mark.parametrize("tokens,hidden,vocab,precise", [
    (1, 72, 300, False), (4, 65, 300, False), (9, 72, 300, False), (20, 5000, 333, False),
    (32, 64, 4000, False), (33, 64, 4000, False), (64, 136, 1000, False), (64, 4104, 300, False),
    (64, 72, 1100000, False), (65, 72, 700, True), (300, 136, 1000, True), (300, 1001, 2000, True),
    (4099, 72, 33333, True), (200, 4104, 200, True), (3000, 40, 100, True)])
def test_a_gradient_of_two_terms_keeps_them(tokens, hidden, vocab, precise):
    target, dloss, dlse, g = exact_ones(tokens, vocab, tokens)
    lse = torch.zeros(tokens, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)

    def ones(shape):
        return (2 * torch.randint(0, 2, shape, generator=gen, device="cuda") - 1).bfloat16()

    h, w = ones((tokens, hidden)), torch.zeros((vocab, hidden), device="cuda", dtype=torch.bfloat16)
    dh, dw = credit.linear_cross_entropy_backward(dloss, h, w, target, lse, dlse=dlse, precise=precise)
    assert bool((dh == 0).all())
    # (sums below 2^24: exact in fp32, and rounded once)
    assert torch.equal(dw, (g.t() @ h.double()).float().bfloat16())
    # pairs of rows that cancel but for the small term: what one term would drop is all there is
    w = ones((vocab // 2, hidden)).repeat_interleave(2, 0)
    w[1::2] *= -1
    w = torch.cat([w, torch.zeros((vocab - len(w), hidden), device="cuda").bfloat16()])
    dh, dw = credit.linear_cross_entropy_backward(dloss, 0 * h, w, target, lse, dlse=dlse, precise=precise)
    assert bool((dw == 0).all())
    assert torch.equal(dh, (g @ w.double()).float().bfloat16())
    assert tokens < 9 or float(dh.abs().max()) == 1


@pytest.mark.parametrize("tokens,hidden,vocab,precise", [
    (20, 64, 700, False), (64, 264, 1003, False), (50, 4104, 300, False), (40, 33, 700, False),
    (65, 264, 1003, True), (333, 128, 5000, True), (2100, 136, 300, True)])
def test_two_terms_leave_the_outputs_rounding(tokens, hidden, vocab, precise):
    # ones in a column of w: dhidden there is dloss (sum p - 1) = 0 but for g's roundings,
    # 2^-16 of each |g| for two terms, which add up to 2, and p's and lse's, 2^-24 of
    # their arguments (logits up to some 20, 1000 of k at most)
    h, w, target = make(tokens, hidden, vocab, torch.bfloat16, seed=21, ignored=0.0)
    w[:, 0] = 1
    _, lse = credit.linear_cross_entropy_forward(h, w, target)
    one = torch.ones(tokens, device="cuda")
    dh, dw = credit.linear_cross_entropy_backward(one, h, w, target, lse, precise=precise)
    assert float(dh[:, 0].abs().max()) <= 2 * 2.0 ** -16 + 1e-4
    g = (h.double() @ w.double().t() - lse.double()[:, None]).exp()
    g[torch.arange(tokens), target] -= 1
    for got, want in ((dh[:, 1:], (g @ w.double())[:, 1:]), (dw, g.t() @ h.double())):
        own = (want.bfloat16().double() - want).norm() / want.norm()
        off = (got.double() - want).norm() / want.norm()
        # (sums of two terms err by 2^-16 of |g| against 2^-9 of the output's own rounding)
        assert float(off) <= float(own) * 1.02 + 2.0 ** -16


def test_precise_changes_nothing_else():
    for tokens, dtype in ((5, torch.bfloat16), (30, torch.bfloat16), (300, torch.float32)):
        h, w, target = make(tokens, 64, 500, dtype, seed=4)
        loss, lse = credit.linear_cross_entropy_forward(h, w, target)
        a = credit.linear_cross_entropy_backward(loss, h, w, target, lse)
        b = credit.linear_cross_entropy_backward(loss, h, w, target, lse, precise=True)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_precise_with_given_outputs_a_workspace_and_a_graph():
    h, w, target = make(300, 128, 2100, torch.bfloat16, seed=13)
    _, lse = credit.linear_cross_entropy_forward(h, w, target)
    dloss = torch.rand(300, device="cuda")
    want = credit.linear_cross_entropy_backward(dloss, h, w, target, lse, precise=True)
    ws = torch.empty(C.credit_linear_ce_workspace(2, h.data_ptr(), w.data_ptr(), 300, 128, 2100, C.BF16,
                                                  h.device.index), dtype=torch.uint8, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty_like(w)

    def call():
        return credit.linear_cross_entropy_backward(dloss, h, w, target, lse, dhidden=dh, dweight=dw,
                                                    workspace=ws, precise=True)

    call()
    assert torch.equal(dh, want[0]) and torch.equal(dw, want[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    h.copy_(h.roll(1, 0)), target.copy_(target.roll(1, 0))
    lse.copy_(lse.roll(1, 0)), dloss.copy_(dloss.roll(1, 0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dh, want[0].roll(1, 0))
    only = credit.linear_cross_entropy_backward(dloss, h, w, target, lse, need_dweight=False, precise=True)
    # (its sums may be split at other places: another rounding of some elements)
    assert only[1] is None and float((only[0] - dh).float().norm()) <= 2.0 ** -8 * float(dh.float().norm())
    with pytest.raises(credit.CreditError):
        credit.linear_cross_entropy_backward(dloss, h, w, target, lse, workspace=ws[:256], precise=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spread", [20.0, 100.0, 1000.0])
@pytest.mark.parametrize("tokens,hidden,vocab", [(1, 128, 1000), (40, 128, 1000), (300, 1001, 777), (130, 128, 70000),
                                                 (4096, 128, 1000), (40, 4096, 500)])
def test_no_loss_is_below_zero(tokens, hidden, vocab, spread, dtype):
    # the target's logit is among those whose exponentials are summed: the sum is 1 or
    # more times the largest's, which is the target's or above it
    h, w, _ = make(tokens, hidden, vocab, dtype, seed=7, spread=spread)
    z = h.double() @ w.double().t()
    loss, _ = credit.linear_cross_entropy_forward(h, w, z.argmax(1))
    assert bool((loss >= 0).all())


@pytest.mark.parametrize("tokens", [1, 8, 40, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1e4, 1e6, 1e8, 1e10, 1e20, 1e30, 1e38, 2e38])
def test_logits_of_any_finite_size(scale, dtype, tokens):
    # one product a logit, so every logit is exact; the largest stands far above the others
    vocab = 500
    h = torch.zeros((tokens, 64), device="cuda", dtype=dtype)
    w = torch.zeros((vocab, 64), device="cuda", dtype=dtype)
    h[:, 0] = 1
    for sign in (1, -1):
        w[:, 0] = (torch.linspace(0.2, 1, vocab, device="cuda") * scale * sign).to(dtype)
        w[13, 0] = 1.5 * scale if sign > 0 else 0.1 * scale * -1
        z = w[:, 0].double()
        target = torch.full((tokens,), 13, device="cuda")
        loss, lse = credit.linear_cross_entropy_forward(h, w, target)
        assert bool((lse.double() == z[13]).all()) and bool((loss == 0).all())
        loss, _ = credit.linear_cross_entropy_forward(h, w, target + 1)
        assert_close(loss, (z[13] - z[14]).expand(tokens), (2 * U * (z[13] - z[14]).abs()).expand(tokens), "loss")
        # p is 1 for the largest and 0 for the others
        one = torch.ones(tokens, device="cuda")
        dh, dw = credit.linear_cross_entropy_backward(one, h, w, target + 1, lse)
        assert bool((dw[13, 0] == tokens).all()) and bool((dw[14, 0] == -tokens).all())
        dw[13:15, 0] = 0
        assert bool((dw == 0).all())
        want = (z[13] - z[14]).expand(tokens)
        assert_close(dh[:, 0], want, (2.0 ** -8 if dtype == torch.bfloat16 else 8 * U) * want.abs() + 8 * U * 1.5 * scale,
                     "dhidden")
        assert bool((dh[:, 1:] == 0).all())


def bias(got, want):
    return float(((got.double() - want) / want).mean())


@pytest.mark.parametrize("precise", [False, True])
def test_a_long_sum_of_one_sign_does_not_sink(precise):
    # Sums over a million tokens, or words, of products in 1 to 4.  The accumulator drops
    # less than its last digit, 2^-23 of the sum so far, at each addition of sixteen
    # products; 8192 additions to a part whose sum grows evenly make 2^-11.  The sums of a
    # million numbers are nearly alike, so the outputs' own rounding is too: the rounded
    # sums are compared.  Those that lie within 2^-11 of a rounding's border may fall on
    # either side: of dweight's, 2346614 to 2347710 beside a border at 2334720, none; of
    # dhidden's, a hundred different ones, an eighth, which is another 2^-11 of the mean.
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def ones_to_twos(shape):
        return (1 + torch.randint(0, 128, shape, generator=g, device="cuda") / 128).bfloat16()

    tokens, hidden, vocab = 1 << 20, 5120, 256
    h = torch.empty((tokens, hidden), dtype=torch.bfloat16, device="cuda")
    for i in range(0, tokens, 1 << 16):
        h[i:i + (1 << 16)] = ones_to_twos((1 << 16, hidden))
    w = torch.zeros((vocab, hidden), dtype=torch.bfloat16, device="cuda")
    none, zero = torch.full((tokens,), IGNORE, device="cuda"), torch.zeros(tokens, device="cuda")
    dlse = ones_to_twos((tokens,)).float()  # (with w = 0 and lse = 0 every p is 1: g = dlse)
    _, dw = credit.linear_cross_entropy_backward(zero, h, w, none, zero, dlse=dlse, need_dhidden=False,
                                                 precise=precise)
    want = torch.zeros(hidden, dtype=torch.float64, device="cuda")
    for i in range(0, tokens, 1 << 14):
        want += dlse[i:i + (1 << 14)].double() @ h[i:i + (1 << 14)].double()
    assert abs(bias(dw, want.bfloat16().double().expand(vocab, hidden))) <= 2.0 ** -11
    del h, dw
    tokens, hidden, vocab = 100, 136, 1300000
    h = torch.zeros((tokens, hidden), dtype=torch.bfloat16, device="cuda")
    w, dlse = ones_to_twos((vocab, hidden)), ones_to_twos((tokens,)).float()
    for need_w in (True, False):
        dh, _ = credit.linear_cross_entropy_backward(zero[:tokens], h, w, none[:tokens], zero[:tokens], dlse=dlse,
                                                     need_dweight=need_w, precise=precise)
        want = dlse.double()[:, None] * w.double().sum(0)
        assert abs(bias(dh, want.bfloat16().double())) <= 2 * 2.0 ** -11


@pytest.mark.parametrize("tokens", [4096, 20000])  # (few tiles: k is split)
def test_a_logits_sum_sinks_no_more_than_its_parts_do(tokens):
    # One word: lse is its logit, a sum of 4096 products in 1 to 4, multiples of 2^-14.  The
    # accumulator holds 256 of k, below 1024, so 24 bits and exact; of more it would drop
    # digits towards zero.  The sixteen parts are added to nearest, u of the sum each at most
    # in either direction: 16 u / sqrt(3) / sqrt(4096) = 0.14 u on average over the tokens.
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    h = (1 + torch.randint(0, 128, (tokens, 4096), generator=g, device="cuda") / 128).bfloat16()
    w = (1 + torch.randint(0, 128, (1, 4096), generator=g, device="cuda") / 128).bfloat16()
    target = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    loss, lse = credit.linear_cross_entropy_forward(h, w, target)
    assert bool((loss == 0).all())
    want = torch.cat([h[i:i + 4096].double() @ w[0].double() for i in range(0, tokens, 4096)])
    assert abs(bias(lse, want)) <= 0.5 * U
