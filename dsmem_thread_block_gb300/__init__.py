"""GB300-native CREDIT reduce-reuse library.

Clustered DSMEM row softmax, LayerNorm, RMSNorm, int8 quantization, weighted
standardization and Pearson correlation, and the row norms' training step
(dropout, residual add and norm with saved statistics, and its gradient),
behind a C ABI
(``libcredit.so``, declared in ``include/credit.h``), with this thin torch
binding on top.  The binding only marshals arguments (device pointers, sizes,
the current CUDA stream, a workspace from torch's allocator); every step of
the computation runs in the library's CUDA kernels, and a missing library
raises instead of falling back to anything else.

    import torch, dsmem_thread_block_gb300 as credit
    y = credit.layernorm(x, gamma, beta, eps=1e-5)       # plans automatically
    p = credit.plan("softmax", rows, cols, torch.float32, cluster_size=4)
    y = credit.softmax(x, plan=p)                         # forced cluster size
"""
from __future__ import annotations

import contextlib
import dataclasses

from . import _credit as C
from ._credit import CreditError, Plan  # noqa: F401

__all__ = ["softmax", "layernorm", "rmsnorm", "quantize", "weighted_std", "pearson", "plan",
           "Dropout", "dropout", "layernorm_forward", "layernorm_backward", "rmsnorm_forward",
           "rmsnorm_backward", "CreditError", "Plan", "device_error", "load_library"]

_OPS = {"softmax": C.SOFTMAX, "layernorm": C.LAYERNORM, "rmsnorm": C.RMSNORM,
        "quantize": C.QUANTIZE, "weighted_std": C.WEIGHTED_STD, "pearson": C.PEARSON}
_plan_cache: dict = {}


def load_library():
    """Load libcredit.so (raises if it has not been built)."""
    return C.load()


def _dtype(t):
    import torch
    if t == torch.float32:
        return C.F32
    if t == torch.bfloat16:
        return C.BF16
    raise TypeError(f"credit: unsupported dtype {t} (fp32 and bf16 only)")


def plan(op: str, rows: int, cols: int, dtype, device: int | None = None,
         variant: str | None = None, cluster_size: int = 1, rows_per_cluster: int = 0,
         exchange: str | None = None, staged_elems: int = 0) -> Plan:
    """Plan a call: automatically (variant None) or for a forced variant
    ("cluster" with `cluster_size` and optionally `rows_per_cluster` or
    `staged_elems` (an L2-tail plan staging that many elements of each
    slice), "persistent" or "pipelined" with `cluster_size`, "warp_rows" or
    "two_pass"); `exchange` ("async" or "barrier") picks how a clustered plan
    exchanges its partials."""
    import torch
    dev = torch.cuda.current_device() if device is None else int(device)
    code = _OPS[op]
    if variant is None:
        return C.credit_plan(code, rows, cols, _dtype(dtype), dev)
    v = {"cluster": C.CLUSTER, "persistent": C.CLUSTER_PERSISTENT,
         "pipelined": C.CLUSTER_PIPELINED, "warp_rows": C.WARP_ROWS,
         "two_pass": C.TWO_PASS}[variant]
    x = {None: C.EXCHANGE_DEFAULT, "async": C.EXCHANGE_ASYNC,
         "barrier": C.EXCHANGE_BARRIER}[exchange]
    return C.credit_plan_with(code, rows, cols, _dtype(dtype), dev, v, cluster_size,
                              rows_per_cluster=rows_per_cluster, exchange=x,
                              staged_elems=staged_elems)


def _prep(x, out):
    import torch
    if not x.is_cuda:
        raise ValueError("credit: x must be a CUDA tensor")
    if not x.is_contiguous():
        raise ValueError("credit: x must be contiguous")
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    if out is None:
        out = torch.empty_like(x)
    elif out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous():
        raise ValueError("credit: out must be a contiguous tensor shaped like x")
    return rows, cols, out


def _plan_and_ws(op, rows, cols, x, p, workspace):
    import torch
    if p is None:
        key = (op, rows, cols, x.dtype, x.device.index)
        p = _plan_cache.get(key)
        if p is None:
            p = C.credit_plan(_OPS[op], rows, cols, _dtype(x.dtype), x.device.index)
            _plan_cache[key] = p
    need = int(p.workspace_bytes)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    wptr = workspace.data_ptr() if workspace is not None else 0
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return p, wptr, wbytes


def _stream(x):
    import torch
    return torch.cuda.current_stream(x.device).cuda_stream


def _ptr(t):
    return t.data_ptr() if t is not None else 0


def _pdtype(*ts):
    ts = [t for t in ts if t is not None]
    if not ts:
        return C.F32
    d = ts[0].dtype
    for t in ts:
        if t.dtype != d or not t.is_cuda or not t.is_contiguous():
            raise ValueError("credit: parameters must be contiguous CUDA tensors of one dtype")
    return _dtype(d)


def softmax(x, out=None, plan: Plan | None = None, workspace=None):
    """Row softmax over the last dimension."""
    rows, cols, out = _prep(x, out)
    p, w, wb = _plan_and_ws("softmax", rows, cols, x, plan, workspace)
    st = C.credit_softmax(x.data_ptr(), out.data_ptr(), rows, cols, _dtype(x.dtype), p, w, wb,
                          _stream(x))
    if st != C.OK:
        raise CreditError(st, "credit_softmax")
    return out


def layernorm(x, gamma=None, beta=None, eps: float = 1e-5, out=None, plan: Plan | None = None,
              workspace=None):
    """LayerNorm over the last dimension (biased variance, eps inside the sqrt)."""
    rows, cols, out = _prep(x, out)
    for t in (gamma, beta):
        if t is not None and t.numel() != cols:
            raise ValueError("credit: gamma/beta must have cols elements")
    p, w, wb = _plan_and_ws("layernorm", rows, cols, x, plan, workspace)
    st = C.credit_layernorm(x.data_ptr(), out.data_ptr(), rows, cols, _dtype(x.dtype),
                            _ptr(gamma), _ptr(beta), _pdtype(gamma, beta), float(eps), p, w, wb,
                            _stream(x))
    if st != C.OK:
        raise CreditError(st, "credit_layernorm")
    return out


def rmsnorm(x, weight=None, eps: float = 1e-6, out=None, plan: Plan | None = None,
            workspace=None):
    """RMSNorm over the last dimension."""
    rows, cols, out = _prep(x, out)
    if weight is not None and weight.numel() != cols:
        raise ValueError("credit: weight must have cols elements")
    p, w, wb = _plan_and_ws("rmsnorm", rows, cols, x, plan, workspace)
    st = C.credit_rmsnorm(x.data_ptr(), out.data_ptr(), rows, cols, _dtype(x.dtype),
                          _ptr(weight), _pdtype(weight), float(eps), p, w, wb, _stream(x))
    if st != C.OK:
        raise CreditError(st, "credit_rmsnorm")
    return out


def quantize(x, out=None, scales=None, plan: Plan | None = None, workspace=None):
    """Row-wise symmetric int8 quantization over the last dimension; returns
    (codes int8 shaped like x, fp32 scales, one per row)."""
    import torch
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("credit: x must be a contiguous CUDA tensor")
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    if out is None:
        out = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    if scales is None:
        scales = torch.empty(rows, dtype=torch.float32, device=x.device)
    p, w, wb = _plan_and_ws("quantize", rows, cols, x, plan, workspace)
    st = C.credit_quantize(x.data_ptr(), out.data_ptr(), scales.data_ptr(), rows, cols,
                           _dtype(x.dtype), p, w, wb, _stream(x))
    if st != C.OK:
        raise CreditError(st, "credit_quantize")
    return out, scales


def weighted_std(x, weights, eps: float = 1e-5, out=None, plan: Plan | None = None,
                 workspace=None):
    """Weighted standardization over the last dimension with per-column
    weights: (x - mean_w) / sqrt(var_w + eps)."""
    rows, cols, out = _prep(x, out)
    if weights is None or weights.numel() != cols:
        raise ValueError("credit: weights must have cols elements")
    p, w, wb = _plan_and_ws("weighted_std", rows, cols, x, plan, workspace)
    st = C.credit_weighted_std(x.data_ptr(), out.data_ptr(), rows, cols, _dtype(x.dtype),
                               weights.data_ptr(), _pdtype(weights), float(eps), p, w, wb,
                               _stream(x))
    if st != C.OK:
        raise CreditError(st, "credit_weighted_std")
    return out


def pearson(x, u, eps: float = 0.0, out=None, r=None, plan: Plan | None = None, workspace=None):
    """Row-wise Pearson correlation of x and u over the last dimension;
    returns (standardized co-deviations shaped like x, fp32 r per row)."""
    import torch
    rows, cols, out = _prep(x, out)
    if u is None or u.shape != x.shape or u.dtype != x.dtype or not u.is_cuda or \
            not u.is_contiguous():
        raise ValueError("credit: u must be a contiguous CUDA tensor shaped like x")
    if r is None:
        r = torch.empty(rows, dtype=torch.float32, device=x.device)
    p, w, wb = _plan_and_ws("pearson", rows, cols, x, plan, workspace)
    st = C.credit_pearson(x.data_ptr(), u.data_ptr(), out.data_ptr(), r.data_ptr(), rows, cols,
                          _dtype(x.dtype), float(eps), p, w, wb, _stream(x))
    if st != C.OK:
        raise CreditError(st, "credit_pearson")
    return out, r


# ------------------------------------------------------- training operators
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
        import torch
        if not 0.0 <= self.p < 1.0:
            raise ValueError("credit: dropout needs 0 <= p < 1")
        for v in (self.seed, self.offset):
            if not 0 <= v < 1 << 64:
                raise ValueError("credit: dropout seed and offset are unsigned 64-bit integers")
        d = self.device_offset
        if d is not None and (d.dtype != torch.int64 or d.numel() != 1 or not d.is_cuda):
            raise ValueError("credit: device_offset must be an int64 CUDA tensor of one element")
        object.__setattr__(self, "_fields", C.dropout_fields(
            self.p, self.seed, self.offset, d.data_ptr() if d is not None else 0))


_ws_cache: dict = {}


def _on(x):
    """Launch on x's device, whatever the current one is."""
    import torch
    if torch.cuda.current_device() == x.device.index:
        return contextlib.nullcontext()
    return torch.cuda.device(x.device)


def _matrix(t, x, name):
    if t is None:
        return 0
    if t.shape != x.shape or t.dtype != x.dtype or t.device != x.device or not t.is_contiguous():
        raise ValueError(f"credit: {name} must be a contiguous tensor shaped like the input, "
                         "of its dtype and on its device")
    return t.data_ptr()


def _rowvec(t, x, rows, name):
    import torch
    if t is None:
        raise ValueError(f"credit: {name} is required")
    if t.dtype != torch.float32 or t.numel() != rows or t.device != x.device or \
            not t.is_contiguous():
        raise ValueError(f"credit: {name} must be a contiguous fp32 tensor on the input's device, "
                         "one element per row")
    return t.data_ptr()


def _colvec(t, x, cols, name):
    if t is None:
        return 0
    if t.numel() != cols or t.device != x.device:
        raise ValueError(f"credit: {name} must have cols elements on the input's device")
    return t.data_ptr()


def _shape(x):
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("credit: inputs must be contiguous CUDA tensors")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("credit: the last dimension must hold at least one element")
    cols = x.shape[-1]
    return x.numel() // cols, cols


def _drop(d, x):
    if d is None:
        return None
    if d.device_offset is not None and d.device_offset.device != x.device:
        raise ValueError("credit: device_offset must be on the input's device")
    return d._fields


def _norm_ws(op, backward, rows, cols, x, workspace):
    import torch
    key = (op, backward, rows, cols, x.dtype, x.device.index)
    need = _ws_cache.get(key)
    if need is None:
        need = C.credit_norm_workspace(op, backward, rows, cols, _dtype(x.dtype), x.device.index)
        if len(_ws_cache) >= 4096:
            _ws_cache.clear()
        _ws_cache[key] = need
    if workspace is None:
        if not need:
            return None, 0, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    elif workspace.device != x.device or not workspace.is_contiguous():
        raise ValueError("credit: workspace must be a contiguous tensor on the input's device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def dropout(x, drop: Dropout, residual=None, out=None):
    """residual + dropout(x) with a mask drawn from the counter-based
    generator and never stored.  On the incoming gradient, without residual,
    it is its own backward pass."""
    import torch
    rows, cols = _shape(x)
    rp = _matrix(residual, x, "residual")
    if out is None:
        out = torch.empty_like(x)
    op = _matrix(out, x, "out")
    with _on(x):
        st = C.credit_dropout(x.data_ptr(), rp, op, rows, cols, _dtype(x.dtype), _drop(drop, x),
                              _stream(x))
    if st != C.OK:
        raise CreditError(st, "credit_dropout")
    return out


def _norm_forward(op, x, gamma, beta, eps, residual, drop, out, h_out, workspace):
    import torch
    rows, cols = _shape(x)
    gp, bp = _colvec(gamma, x, cols, "gamma"), _colvec(beta, x, cols, "beta")
    rp = _matrix(residual, x, "residual")
    pdtype = _pdtype(gamma, beta)
    fields = _drop(drop, x)
    if out is None:
        out = torch.empty_like(x)
    same = residual is None and (drop is None or drop.p == 0.0)
    if h_out is None and not same:
        h_out = torch.empty_like(x)
    hp = _matrix(h_out, x, "h_out")
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) \
        if op == C.LAYERNORM else None
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    ws, wp, wb = _norm_ws(op, False, rows, cols, x, workspace)
    with _on(x):
        st = C.credit_norm_forward(op, x.data_ptr(), rp, fields, _matrix(out, x, "out"), hp,
                                   _ptr(mean), rstd.data_ptr(), rows, cols, _dtype(x.dtype), gp,
                                   bp, pdtype, float(eps), wp, wb, _stream(x))
    if st != C.OK:
        raise CreditError(st, "credit_norm_forward")
    return out, h_out if h_out is not None else x, mean, rstd


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
    import torch
    rows, cols = _shape(dy)
    hp, dhp = _matrix(h, dy, "h"), _matrix(dh, dy, "dh")
    if h is None:
        raise ValueError("credit: h is required")
    mp = _rowvec(mean, dy, rows, "mean") if op == C.LAYERNORM else 0
    sp = _rowvec(rstd, dy, rows, "rstd")
    gp = _colvec(gamma, dy, cols, "gamma")
    pdtype = _pdtype(gamma)
    fields = _drop(drop, dy)
    drops = drop is not None and drop.p > 0.0
    if dx is None:
        dx = torch.empty_like(dy)
    if dresidual is None and need_dresidual and drops:
        dresidual = torch.empty_like(dy)
    dgamma = torch.empty_like(gamma) if gamma is not None else None
    dbeta = torch.empty_like(gamma) if gamma is not None and op == C.LAYERNORM else None
    ws, wp, wb = _norm_ws(op, True, rows, cols, dy, workspace)
    with _on(dy):
        st = C.credit_norm_backward(op, dy.data_ptr(), dhp, hp, mp, sp, gp, pdtype, fields,
                                    _matrix(dx, dy, "dx"), _matrix(dresidual, dy, "dresidual"),
                                    _ptr(dgamma), _ptr(dbeta), rows, cols, _dtype(dy.dtype), wp,
                                    wb, _stream(dy))
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


def device_error(device: int = 0) -> int:
    """Read and clear the device error word (CREDIT_ERR_DEVICE_TIMEOUT if a
    bounded device wait gave up)."""
    return C.credit_get_device_error(device)
