"""Forward-mode tangents: the training operators have no such derivative, and refuse a
tensor that carries one before they look at anything else."""
import pytest

torch = pytest.importorskip("torch")
fwAD = torch.autograd.forward_ad

import dsmem_thread_block_gb300 as credit
from dsmem_thread_block_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    B.build_torch()


def dual(t):
    return fwAD.make_dual(t, torch.ones_like(t))


def calls():
    """Each operator, of tensors of which `f` makes those that are differentiated."""
    h, w, g = torch.ones(4, 8), torch.ones(5, 8), torch.ones(8)
    one, target = torch.ones(4), torch.zeros(4, dtype=torch.int64)
    return {
        "dropout": lambda f: credit.dropout(f(h), credit.Dropout(0.5, 1)),
        "rmsnorm forward": lambda f: credit.rmsnorm_forward(h, f(g)),
        "rmsnorm backward": lambda f: credit.rmsnorm_backward(f(h), h, one, g),
        "layernorm forward": lambda f: credit.layernorm_forward(f(h), g),
        "loss of hidden": lambda f: credit.linear_cross_entropy_forward(f(h), w, target),
        "loss of weight": lambda f: credit.linear_cross_entropy_forward(h, f(w), target),
        "loss's gradient of dloss": lambda f: credit.linear_cross_entropy_backward(f(one), h, w, target, one),
        "loss's gradient of lse": lambda f: credit.linear_cross_entropy_backward(one, h, w, target, f(one)),
        "loss's gradient of dlse": lambda f: credit.linear_cross_entropy_backward(one, h, w, target, one, dlse=f(one)),
        "gradient norm": lambda f: credit.gradient_norm([h, f(w)]),
        "clipping": lambda f: credit.clip_gradients([f(h)], 1.0),
        "clipping into": lambda f: credit.clip_gradients([h], 1.0, out=[f(h)]),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_a_tangent_is_refused(name):
    call = calls()[name]
    with fwAD.dual_level():
        for grad in (True, False):
            with torch.set_grad_enabled(grad), pytest.raises(RuntimeError, match="tangent"):
                call(dual)
        # where forward mode is off, or a tensor has none, the next check speaks: no GPU here
        with fwAD._set_fwd_grad_enabled(False), pytest.raises(ValueError):
            call(dual)
        with pytest.raises(ValueError):
            call(lambda t: t)


@pytest.mark.parametrize("name", list(calls()))
def test_a_gradient_is_refused_as_before(name):
    call = calls()[name]
    with pytest.raises(RuntimeError, match="requires a gradient"):
        call(lambda t: t.clone().requires_grad_())
    with torch.no_grad(), pytest.raises(ValueError):
        call(lambda t: t.clone().requires_grad_())
