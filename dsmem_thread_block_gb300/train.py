"""The training operators on torch tensors: dropout, the norms' forward pass
with residual add, dropout and saved statistics, and its gradient; the linear
head's cross entropy, and its gradient; the norm of all gradients, and clipping.

The functions here carry the arguments' meaning; a small extension
(csrc/train_torch.cpp) checks the tensors, allocates outputs and workspace from
torch's allocator, and calls the C ABI on the input's device and its current
stream.  The extension is loaded by the first call; a missing one raises there,
as a missing library does.

The calls record no autograd graph: they are the two halves of a
torch.autograd.Function, or of a step written out by hand.  Under grad mode they
refuse tensors that require a gradient, whose gradient would be lost.
"""
from __future__ import annotations

import ctypes
import dataclasses
import importlib.machinery
import importlib.util
import os

from . import _credit as C
from . import build as _build
from ._credit import CreditError


def _load():
    import torch  # noqa: F401  (the extension's libraries)
    path = _build.TORCH_LIB
    if not os.path.exists(path):
        raise RuntimeError(f"the training operators' torch layer is not built ({path}); run "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    loader = importlib.machinery.ExtensionFileLoader("credit_train_torch", path)
    spec = importlib.util.spec_from_loader("credit_train_torch", loader)
    module = importlib.util.module_from_spec(spec)
    loader.exec_module(module)
    return module


_ext = None    # the extension
_bound = None  # the library whose functions it calls


def _bind():
    """Hand the extension the current library's functions (the regular build's,
    or the checked build's inside `use_checked_build`)."""
    global _ext, _bound
    lib = C.load()
    if _ext is None:
        _ext = _load()
    _ext.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value
                for f in ("credit_dropout", "credit_norm_workspace", "credit_norm_forward",
                          "credit_norm_backward", "credit_linear_ce_workspace",
                          "credit_linear_ce_forward", "credit_linear_ce_backward",
                          "credit_grad_workspace", "credit_grad_norm", "credit_grad_clip",
                          "credit_linear_ce_backward_precise")))
    _bound = lib


def _word(d):
    """The address of a device_offset tensor (0: none)."""
    if d is None:
        return 0
    import torch
    if d.dtype != torch.int64 or d.numel() != 1 or not d.is_cuda:
        raise ValueError("credit: device_offset must be an int64 CUDA tensor of one element")
    return d.data_ptr()


@dataclasses.dataclass(frozen=True)
class Dropout:
    """A dropout stream: drop probability 0 <= p < 1, a 64-bit seed and a
    64-bit offset (calls that must not share a mask differ in one of them).
    `device_offset`, an int64 CUDA tensor of one element, is added to the
    offset when the kernel runs, so a captured graph draws a new mask at each
    replay once the tensor has changed.  The backward call takes the forward
    call's object."""
    p: float
    seed: int
    offset: int = 0
    device_offset: object = None

    def __post_init__(self):
        if not 0.0 <= self.p < 1.0:
            raise ValueError("credit: dropout needs 0 <= p < 1")
        if not (0 <= self.seed < 1 << 64 and 0 <= self.offset < 1 << 64):
            raise ValueError("credit: dropout seed and offset are unsigned 64-bit integers")
        fields = C.dropout_fields(self.p, self.seed, self.offset, _word(self.device_offset))
        object.__setattr__(self, "_fields", fields)
        object.__setattr__(self, "_address", ctypes.addressof(fields))

    def __reduce__(self):
        # a copy has a C struct of its own
        return type(self), (self.p, self.seed, self.offset, self.device_offset)


def _drop(d, x):
    if d is None:
        return None
    if d.device_offset is not None:
        if d.device_offset.device != x.device:
            raise ValueError("credit: device_offset must be on the input's device")
        # the tensor may have been given other storage since the last call
        d._fields.device_offset = _word(d.device_offset)
    return d._address


def dropout(x, drop: Dropout, residual=None, out=None):
    """residual + dropout(x) with a mask drawn from the counter-based
    generator and never stored.  On the incoming gradient, without residual,
    it is its own backward pass.  `out` may be x or residual (in place)."""
    if C._lib is not _bound or _bound is None:
        _bind()
    r = _ext.dropout(x, _drop(drop, x), residual, out)
    if type(r) is int:
        raise CreditError(r, "credit_dropout")
    return out if out is not None else r[0]


def _norm_forward(op, x, gamma, beta, eps, residual, drop, out, h_out, workspace):
    if C._lib is not _bound or _bound is None:
        _bind()
    r = _ext.norm_forward(op, x, gamma, beta, eps, residual, _drop(drop, x), out, h_out, workspace)
    if type(r) is int:
        raise CreditError(r, "credit_norm_forward")
    return r


def layernorm_forward(x, gamma=None, beta=None, eps: float = 1e-5, residual=None,
                      dropout: Dropout | None = None, out=None, h_out=None, workspace=None):
    """h = residual + dropout(x), y = LayerNorm(h) over the last dimension;
    returns (y, h, mean, rstd): what layernorm_backward needs, mean and rstd
    fp32, one per row.  Without residual and dropout h is x itself, or a copy
    of it in `h_out` or where `out` is x.  `out` and `h_out` may each be x or
    residual (in place)."""
    return _norm_forward(C.LAYERNORM, x, gamma, beta, eps, residual, dropout, out, h_out,
                         workspace)


def rmsnorm_forward(x, weight=None, eps: float = 1e-6, residual=None,
                    dropout: Dropout | None = None, out=None, h_out=None, workspace=None):
    """As layernorm_forward for RMSNorm; returns (y, h, rstd)."""
    y, h, _, rstd = _norm_forward(C.RMSNORM, x, weight, None, eps, residual, dropout, out, h_out,
                                  workspace)
    return y, h, rstd


def _norm_backward(op, dy, h, mean, rstd, gamma, dh, drop, need_dresidual, dx, dresidual,
                   workspace, beta=None):
    if C._lib is not _bound or _bound is None:
        _bind()
    r = _ext.norm_backward(op, dy, h, mean, rstd, gamma, dh, _drop(drop, dy), need_dresidual, dx,
                           dresidual, workspace, beta)
    if type(r) is int:
        raise CreditError(r, "credit_norm_backward")
    return r


def layernorm_backward(dy, h, mean, rstd, gamma=None, dh=None, dropout: Dropout | None = None,
                       need_dresidual: bool = False, dx=None, dresidual=None, workspace=None,
                       beta=None):
    """The gradient of layernorm_forward: from dy (of y) and dh (the gradient
    that reaches h past the norm, or None), returns (dx, dresidual, dgamma,
    dbeta).  dresidual is None unless asked for, and dx itself where there is
    no dropout.  dgamma is None without gamma; dbeta is None without gamma
    and without `beta`, of which only the shape and type count (those of
    gamma where it is not given).  `dx` and `dresidual` may each be dy, dh or h
    (in place)."""
    return _norm_backward(C.LAYERNORM, dy, h, mean, rstd, gamma, dh, dropout, need_dresidual, dx,
                          dresidual, workspace, beta)


def rmsnorm_backward(dy, h, rstd, weight=None, dh=None, dropout: Dropout | None = None,
                     need_dresidual: bool = False, dx=None, dresidual=None, workspace=None):
    """As layernorm_backward for rmsnorm_forward; returns (dx, dresidual,
    dweight)."""
    return _norm_backward(C.RMSNORM, dy, h, None, rstd, weight, dh, dropout, need_dresidual, dx,
                          dresidual, workspace)[:3]


def linear_cross_entropy_forward(hidden, weight, target, ignore_index: int = -100, workspace=None):
    """Softmax cross entropy of the logits hidden @ weight.T, which are never
    stored: returns (loss, lse), fp32, one per token.  lse is the logarithm of the
    sum of the logits' exponentials, loss is lse less the target's logit, and 0
    where the target is `ignore_index`.  hidden is (..., hidden size), weight
    (vocabulary, hidden size), target int64 (...); the caller takes the mean, or a
    sum of its own weights.  A target outside the vocabulary that is not
    ignore_index gives NaN.

    fp32 losses of 17 to some 60 tokens and a large weight are slower than the logits
    themselves from a library's fp32 product (17 of 32768 x 4096: 387 and 237 us): all of
    the weight is taken apart for the tensor cores first."""
    if C._lib is not _bound or _bound is None:
        _bind()
    r = _ext.linear_ce_forward(hidden, weight, target, ignore_index, workspace)
    if type(r) is int:
        raise CreditError(r, "credit_linear_ce_forward")
    return r


def linear_cross_entropy_backward(dloss, hidden, weight, target, lse, dlse=None,
                                  ignore_index: int = -100, need_dhidden: bool = True,
                                  need_dweight: bool = True, dhidden=None, dweight=None,
                                  workspace=None, precise: bool = False):
    """The gradient of linear_cross_entropy_forward: from dloss (of each token's
    loss; of an ignored one it does not count) and dlse (of its lse, or None), both
    fp32 and contiguous (what autograd hands a mean's backward is expanded:
    `.contiguous()`), returns (dhidden, dweight).  One that is not needed is None, unless a tensor
    for it is given in `dhidden` or `dweight`.

    Of more than 64 bf16 tokens the logits' gradient is rounded to bf16 for the two
    products, which takes 2.2e-3 of the 2-norm where dloss differs from token to token
    (1.7e-3, the outputs' own rounding, where it is a mean's).  `precise` keeps it in two
    bf16 terms, for about twice the time of the products; other calls do not change."""
    if C._lib is not _bound or _bound is None:
        _bind()
    r = _ext.linear_ce_backward(dloss, hidden, weight, target, lse, dlse, ignore_index,
                                need_dhidden, need_dweight, dhidden, dweight, workspace, precise)
    if type(r) is int:
        raise CreditError(r, "credit_linear_ce_backward")
    return r


def gradient_norm(gradients, workspace=None):
    """The 2-norm of all elements of a list of tensors (fp32 and bf16, any dense
    strides, one device), a fp32 tensor of no dimensions on their device."""
    if C._lib is not _bound or _bound is None:
        _bind()
    r = _ext.gradients(gradients, None, False, 0.0, 0.0, workspace)
    if type(r) is int:
        raise CreditError(r, "credit_grad_norm")
    return r[0]


def clip_gradients(gradients, max_norm: float, eps: float = 1e-6, out=None, workspace=None):
    """Scale a list of tensors by min(1, max_norm / (norm + eps)), in place or into
    the tensors of `out`, and return their norm before that, as gradient_norm does.
    Nothing waits for the GPU.  A norm that is not finite is the caller's to look
    at: an infinite one makes the factor 0, a NaN makes it NaN."""
    if C._lib is not _bound or _bound is None:
        _bind()
    r = _ext.gradients(gradients, out, True, max_norm, eps, workspace)
    if type(r) is int:
        raise CreditError(r, "credit_grad_clip")
    return r[0]
