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
