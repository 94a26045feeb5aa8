"""The training operators on torch tensors: dropout, the norms' forward pass
with residual add, dropout and saved statistics, and its gradient.

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
                          "credit_norm_backward")))
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
