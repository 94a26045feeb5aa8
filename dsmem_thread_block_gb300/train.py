"""The training operators on torch tensors: dropout, the norms' forward pass
with residual add, dropout and saved statistics, and its gradient.

Thin calls of the C ABI, like the package's other functions: they check the
tensors, allocate outputs and workspace from torch's allocator and launch on
the input's device and its current stream.  Small calls are bound by what
happens here, so each check is made once and nothing is looked up twice.
"""
from __future__ import annotations

import dataclasses

import torch

from . import _credit as C
from ._credit import CreditError

_DTYPES = {torch.float32: C.F32, torch.bfloat16: C.BF16}
_raw_stream = torch._C._cuda_getCurrentRawStream  # torch.cuda.current_stream, without its object
_ws_cache: dict = {}


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
        d = self.device_offset
        if d is not None and (d.dtype != torch.int64 or d.numel() != 1 or not d.is_cuda):
            raise ValueError("credit: device_offset must be an int64 CUDA tensor of one element")
        object.__setattr__(self, "_fields", C.dropout_fields(
            self.p, self.seed, self.offset, d.data_ptr() if d is not None else 0))


def _launch(dev, call, *args):
    """call(*args, stream) on device `dev`, whatever the current one is."""
    if torch.cuda.current_device() == dev:
        return call(*args, _raw_stream(dev))
    with torch.cuda.device(dev):
        return call(*args, _raw_stream(dev))


def _input(x):
    """(rows, cols, dtype code, device index) of a call's first matrix."""
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("credit: inputs must be contiguous CUDA tensors")
    shape = x.shape
    if not shape or shape[-1] < 1:
        raise ValueError("credit: the last dimension must hold at least one element")
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"credit: unsupported dtype {x.dtype} (fp32 and bf16 only)")
    return x.numel() // shape[-1], shape[-1], code, x.get_device()


def _matrix(t, x, name):
    if t is None:
        return 0
    if t.shape != x.shape or t.dtype != x.dtype or t.device != x.device or not t.is_contiguous():
        raise ValueError(f"credit: {name} must be a contiguous tensor shaped like the input, "
                         "of its dtype and on its device")
    return t.data_ptr()


def _rowvec(t, x, rows, name):
    if t is None:
        raise ValueError(f"credit: {name} is required")
    if t.dtype != torch.float32 or t.numel() != rows or t.device != x.device or \
            not t.is_contiguous():
        raise ValueError(f"credit: {name} must be a contiguous fp32 tensor on the input's device, "
                         "one element per row")
    return t.data_ptr()


def _params(gamma, beta, x, cols):
    """(gamma pointer, beta pointer, dtype code) of a call's parameters."""
    code = None
    for t in (gamma, beta):
        if t is None:
            continue
        if t.numel() != cols or t.device != x.device or not t.is_contiguous():
            raise ValueError("credit: parameters must be contiguous tensors of cols elements on "
                             "the input's device")
        c = _DTYPES.get(t.dtype)
        if c is None:
            raise TypeError(f"credit: unsupported dtype {t.dtype} (fp32 and bf16 only)")
        if code is not None and c != code:
            raise ValueError("credit: parameters must have one dtype")
        code = c
    return (gamma.data_ptr() if gamma is not None else 0,
            beta.data_ptr() if beta is not None else 0, C.F32 if code is None else code)


def _drop(d, x):
    if d is None:
        return None
    if d.device_offset is not None and d.device_offset.device != x.device:
        raise ValueError("credit: device_offset must be on the input's device")
    return d._fields


def _workspace(op, backward, rows, cols, code, dev, x, workspace):
    key = (op, backward, rows, cols, code, dev)
    need = _ws_cache.get(key)
    if need is None:
        need = C.credit_norm_workspace(op, backward, rows, cols, code, dev)
        if len(_ws_cache) >= 4096:
            _ws_cache.clear()
        _ws_cache[key] = need
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
    if workspace.device != x.device or not workspace.is_contiguous():
        raise ValueError("credit: workspace must be a contiguous tensor on the input's device")
    return workspace


def _bytes(t):
    return (0, 0) if t is None else (t.data_ptr(), t.numel() * t.element_size())


def dropout(x, drop: Dropout, residual=None, out=None):
    """residual + dropout(x) with a mask drawn from the counter-based
    generator and never stored.  On the incoming gradient, without residual,
    it is its own backward pass.  `out` may be x or residual (in place)."""
    rows, cols, code, dev = _input(x)
    rp = _matrix(residual, x, "residual")
    if out is None:
        out = torch.empty_like(x)
        op = out.data_ptr()
    else:
        op = _matrix(out, x, "out")
    st = _launch(dev, C.credit_dropout, x.data_ptr(), rp, op, rows, cols, code, _drop(drop, x))
    if st != C.OK:
        raise CreditError(st, "credit_dropout")
    return out


def _norm_forward(op, x, gamma, beta, eps, residual, drop, out, h_out, workspace):
    rows, cols, code, dev = _input(x)
    gp, bp, pcode = _params(gamma, beta, x, cols)
    rp = _matrix(residual, x, "residual")
    fields = _drop(drop, x)
    if out is None:
        out = torch.empty_like(x)
        yp = out.data_ptr()
    else:
        yp = _matrix(out, x, "out")
    h = h_out
    if h_out is not None:
        hp = _matrix(h_out, x, "h_out")
    elif residual is None and (drop is None or drop.p == 0.0):
        h, hp = x, 0
    else:
        h = torch.empty_like(x)
        hp = h.data_ptr()
    per_row = x.shape[:-1]
    rstd = torch.empty(per_row, dtype=torch.float32, device=x.device)
    mean = torch.empty_like(rstd) if op == C.LAYERNORM else None
    ws = _workspace(op, False, rows, cols, code, dev, x, workspace)
    wp, wb = _bytes(ws)
    st = _launch(dev, C.credit_norm_forward, op, x.data_ptr(), rp, fields, yp, hp,
                 mean.data_ptr() if mean is not None else 0, rstd.data_ptr(), rows, cols, code, gp,
                 bp, pcode, eps, wp, wb)
    if st != C.OK:
        raise CreditError(st, "credit_norm_forward")
    return out, h, mean, rstd


def layernorm_forward(x, gamma=None, beta=None, eps: float = 1e-5, residual=None,
                      dropout: Dropout | None = None, out=None, h_out=None, workspace=None):
    """h = residual + dropout(x), y = LayerNorm(h) over the last dimension;
    returns (y, h, mean, rstd): what layernorm_backward needs, mean and rstd
    fp32, one per row.  Without residual and dropout h is x itself.  `out` and
    `h_out` may each be x or residual (in place)."""
    return _norm_forward(C.LAYERNORM, x, gamma, beta, eps, residual, dropout, out, h_out,
                         workspace)


def rmsnorm_forward(x, weight=None, eps: float = 1e-6, residual=None,
                    dropout: Dropout | None = None, out=None, h_out=None, workspace=None):
    """As layernorm_forward for RMSNorm; returns (y, h, rstd)."""
    y, h, _, rstd = _norm_forward(C.RMSNORM, x, weight, None, eps, residual, dropout, out, h_out,
                                  workspace)
    return y, h, rstd


def _norm_backward(op, dy, h, mean, rstd, gamma, dh, drop, need_dresidual, dx, dresidual,
                   workspace):
    rows, cols, code, dev = _input(dy)
    if h is None:
        raise ValueError("credit: h is required")
    hp, dhp = _matrix(h, dy, "h"), _matrix(dh, dy, "dh")
    mp = _rowvec(mean, dy, rows, "mean") if op == C.LAYERNORM else 0
    sp = _rowvec(rstd, dy, rows, "rstd")
    gp, _, pcode = _params(gamma, None, dy, cols)
    fields = _drop(drop, dy)
    if dx is None:
        dx = torch.empty_like(dy)
        dxp = dx.data_ptr()
    else:
        dxp = _matrix(dx, dy, "dx")
    if dresidual is None and need_dresidual and drop is not None and drop.p > 0.0:
        dresidual = torch.empty_like(dy)
    drp = _matrix(dresidual, dy, "dresidual")
    dgamma = torch.empty_like(gamma) if gamma is not None else None
    dbeta = torch.empty_like(gamma) if gamma is not None and op == C.LAYERNORM else None
    ws = _workspace(op, True, rows, cols, code, dev, dy, workspace)
    wp, wb = _bytes(ws)
    st = _launch(dev, C.credit_norm_backward, op, dy.data_ptr(), dhp, hp, mp, sp, gp, pcode, fields,
                 dxp, drp, dgamma.data_ptr() if dgamma is not None else 0,
                 dbeta.data_ptr() if dbeta is not None else 0, rows, cols, code, wp, wb)
    if st != C.OK:
        raise CreditError(st, "credit_norm_backward")
    if dresidual is None and need_dresidual:
        dresidual = dx  # without dropout the two gradients are one
    return dx, dresidual, dgamma, dbeta


def layernorm_backward(dy, h, mean, rstd, gamma=None, dh=None, dropout: Dropout | None = None,
                       need_dresidual: bool = False, dx=None, dresidual=None, workspace=None):
    """The gradient of layernorm_forward: from dy (of y) and dh (the gradient
    that reaches h past the norm, or None), returns (dx, dresidual, dgamma,
    dbeta).  dresidual is None unless asked for, and dx itself where there is
    no dropout; dgamma and dbeta are None without gamma.  `dx` and `dresidual`
    may each be dy, dh or h (in place)."""
    return _norm_backward(C.LAYERNORM, dy, h, mean, rstd, gamma, dh, dropout, need_dresidual, dx,
                          dresidual, workspace)


def rmsnorm_backward(dy, h, rstd, weight=None, dh=None, dropout: Dropout | None = None,
                     need_dresidual: bool = False, dx=None, dresidual=None, workspace=None):
    """As layernorm_backward for rmsnorm_forward; returns (dx, dresidual,
    dweight)."""
    dx, dresidual, dweight, _ = _norm_backward(C.RMSNORM, dy, h, None, rstd, weight, dh, dropout,
                                               need_dresidual, dx, dresidual, workspace)
    return dx, dresidual, dweight
