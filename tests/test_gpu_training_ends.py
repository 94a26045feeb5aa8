"""A training step's row work from the last block to the optimizer: the final
norm, the head's loss and its gradient, the norm's gradient, and the clipping of
all of them, against the same step in 64 bits by autograd."""
import pytest
import torch

import dsmem_thread_block_gb300 as credit
from dsmem_thread_block_gb300 import _credit as C

pytestmark = pytest.mark.gpu


class HeadLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, target):
        loss, lse = credit.linear_cross_entropy_forward(hidden, weight, target)
        ctx.save_for_backward(hidden, weight, target, lse)
        return loss, lse

    @staticmethod
    def backward(ctx, dloss, dlse):
        hidden, weight, target, lse = ctx.saved_tensors
        dh, dw = credit.linear_cross_entropy_backward(dloss.contiguous(), hidden, weight, target, lse,
                                                      dlse=dlse.contiguous())
        return dh, dw, None


def step(x, gamma, w, target, dtype):
    """The step by the package's calls: gradients of x, gamma and w, clipped."""
    y, h, rstd = credit.rmsnorm_forward(x, gamma)
    loss, lse = credit.linear_cross_entropy_forward(y, w, target)
    n = (target != -100).sum().clamp(min=1).float()
    total = loss.sum() / n + 1e-2 * lse.square().mean()
    dloss = (torch.ones_like(loss) / n).contiguous()
    dy, dw = credit.linear_cross_entropy_backward(dloss, y, w, target, lse,
                                                  dlse=2e-2 * lse / lse.numel())
    dx, _, dgamma = credit.rmsnorm_backward(dy, h, rstd, gamma)
    grads = [dx, dgamma, dw]
    norm = credit.clip_gradients(grads, 0.05)
    return total, norm, grads


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_step(dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    tokens, hidden, vocab = 300, 256, 1500
    x = torch.randn((tokens, hidden), generator=g, device="cuda").to(dtype)
    gamma = (1 + 0.1 * torch.randn((hidden,), generator=g, device="cuda")).to(dtype)
    w = (torch.randn((vocab, hidden), generator=g, device="cuda") * 0.15).to(dtype)
    target = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    target[::7] = -100
    total, norm, grads = step(x, gamma, w, target, dtype)

    xd, gd, wd = (t.double().requires_grad_() for t in (x, gamma, w))
    y = xd * torch.rsqrt(xd.square().mean(1, keepdim=True) + 1e-6) * gd
    z = y @ wd.t()
    lse = torch.logsumexp(z, 1)
    kept = target != -100
    loss = (lse - z.gather(1, target.clamp(min=0)[:, None])[:, 0])[kept].mean() + 1e-2 * lse.square().mean()
    loss.backward()
    want = torch.cat([t.grad.reshape(-1) for t in (xd, gd, wd)]).norm()
    # bf16: y, dy and every gradient are rounded, 2^-8 each, and g once more
    tol = 2e-5 if dtype == torch.float32 else 4 * 2.0 ** -8
    loss = loss.detach()
    assert abs(float(total) - float(loss)) <= tol * abs(float(loss))
    assert abs(float(norm) - float(want)) <= tol * float(want)
    factor = min(1.0, 0.05 / (float(want) + 1e-6))
    assert factor < 1
    for got, t in zip(grads, (xd, gd, wd)):
        exact = t.grad * factor
        assert float((got.double() - exact).norm()) <= 2 * tol * float(exact.norm())


def test_inside_an_autograd_function():
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    h = torch.randn((50, 64), generator=g, device="cuda").requires_grad_()
    w = (0.3 * torch.randn((200, 64), generator=g, device="cuda")).requires_grad_()
    target = torch.randint(0, 200, (50,), generator=g, device="cuda")
    loss, lse = HeadLoss.apply(h, w, target)
    (loss.mean() + 0.1 * lse.square().mean()).backward()
    hd, wd = h.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    z = hd @ wd.t()
    l = torch.logsumexp(z, 1)
    ((l - z.gather(1, target[:, None])[:, 0]).mean() + 0.1 * l.square().mean()).backward()
    for a, b in ((h, hd), (w, wd)):
        assert float((a.grad.double() - b.grad).norm()) <= 2e-5 * float(b.grad.norm())


def test_a_captured_step():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn((128, 128), generator=g, device="cuda").bfloat16()
    gamma = torch.ones(128, device="cuda").bfloat16()
    w = (0.2 * torch.randn((700, 128), generator=g, device="cuda")).bfloat16()
    target = torch.randint(0, 700, (128,), generator=g, device="cuda")
    eager = step(x, gamma, w, target, torch.bfloat16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, gamma, w, target, torch.bfloat16)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])
    assert all(torch.equal(a, b) for a, b in zip(out[2], eager[2]))


def test_a_checked_build_runs_the_same_step():
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn((300, 192), generator=g, device="cuda").bfloat16()
    gamma = torch.ones(192, device="cuda").bfloat16()
    w = (0.2 * torch.randn((1100, 192), generator=g, device="cuda")).bfloat16()
    target = torch.randint(0, 1100, (300,), generator=g, device="cuda")
    want = step(x, gamma, w, target, torch.bfloat16)
    with C.use_checked_build():
        assert C.credit_debug_build() == 1
        got = step(x, gamma, w, target, torch.bfloat16)
        assert C.credit_get_device_error(torch.cuda.current_device()) == C.OK
    assert torch.equal(got[1], want[1]) and all(torch.equal(a, b) for a, b in zip(got[2], want[2]))


def test_waits_that_run_out_end_the_tiles_and_leave_the_context():
    dev = torch.cuda.current_device()
    assert C.credit_get_device_error(dev) == C.OK
    assert C.credit_selftest_tile_timeout(dev) == C.ERR_DEVICE_TIMEOUT
    assert C.credit_get_device_error(dev) == C.OK  # read and cleared
    # tensor memory is free and the kernels work
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    h = torch.randn((400, 128), generator=g, device="cuda").bfloat16()
    w = (0.2 * torch.randn((1000, 128), generator=g, device="cuda")).bfloat16()
    target = torch.randint(0, 1000, (400,), generator=g, device="cuda")
    _, lse = credit.linear_cross_entropy_forward(h, w, target)
    want = torch.logsumexp(h.double() @ w.double().t(), 1)
    assert float((lse.double() - want).abs().max()) < 1e-4
