"""The training operators' definition in 64 bits, and the tolerances their
fp32 evaluation is held to.

Tolerances count roundings (u = 2^-24, half a step of fp32 relative to the
value; an output's own rounding is u_out = 2^-8 for bf16).  A fixed-order sum
of positive terms that no term enters through more than D additions is off by
at most D u times the sum of the terms' magnitudes; a row's sums go through at
most 32 additions in a thread, 5 + 5 in shuffles, 16 over warps, 16 over
cluster ranks and 25 over chunks (the widest row here), so D = 100.  A
column's sum over R rows goes through at most R additions.
"""
import numpy as np
import torch

U = 2.0 ** -24
D = 100.0
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U_OUT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def philox(counter, seed):
    """Philox4x32-10 of uint32 counter arrays (4 of them) and a 64-bit seed."""
    m = np.uint64(0xFFFFFFFF)
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        s32 = np.uint64(32)
        c = [(p1 >> s32) ^ c[1] ^ np.uint64(k[0]), p1 & m,
             (p0 >> s32) ^ c[3] ^ np.uint64(k[1]), p0 & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep_mask(rows, cols, p, seed, offset):
    """True where element (r, c) is kept."""
    g, r = np.meshgrid(np.arange((cols + 3) // 4), np.arange(rows))
    z = np.zeros_like(g)
    w = philox([g, r, z + (offset & 0xFFFFFFFF), z + (offset >> 32)], seed)
    words = np.stack(w, axis=-1).reshape(rows, -1)[:, :cols]
    return torch.from_numpy(words >= np.uint64(int(np.floor(p * 2.0 ** 32))))


def ref_h(x, residual, p, mask):
    """(h, the magnitude its evaluation carries) in 64 bits."""
    h = x.double()
    if p:
        h = torch.where(mask.to(x.device), h / (1.0 - p), torch.zeros_like(h))
    mag = h.abs()
    if residual is not None:
        h, mag = h + residual.double(), mag + residual.double().abs()
    return h, mag


def ref_forward(norm, h, gamma, beta, eps):
    mean = h.mean(1, keepdim=True) if norm == "layernorm" else torch.zeros_like(h[:, :1])
    z = h - mean
    rstd = 1.0 / torch.sqrt((z * z).mean(1, keepdim=True) + eps)
    z = z * rstd
    y = z * gamma.double() if gamma is not None else z
    if beta is not None:
        y = y + beta.double()
    return y, z, mean, rstd


def forward_bounds(norm, h, mag, y, z, mean, rstd, gamma, beta, eps, dtype):
    """Bounds on |error| of (h, y, mean, rstd).  h: three roundings of its
    terms, then its own.  mean: D additions and h's error.  rstd: the sum of
    squares D u, h's error 4 u mag moves it by 2 rms(4 u mag) / rms(h - mean),
    a handful of roundings after."""
    uo = U_OUT[dtype]
    bh = uo * h.abs() + 4 * U * mag
    m = mag.mean(1, keepdim=True)
    bmean = (D + 4) * U * m
    rms = mag.square().mean(1, keepdim=True).sqrt()
    rel = U * (D + 8 + 8 * rms * rstd)
    g = gamma.double().abs() if gamma is not None else 1.0
    b = beta.double().abs() if beta is not None else 0.0
    by = uo * y.abs() + g * rstd * (6 * U * mag + bmean) + g * z.abs() * (rel + 8 * U) + 4 * U * b
    return bh, by, bmean, rel * rstd


def ref_backward(norm, dy, dh, h, mean, rstd, gamma, p, mask):
    """(dtot, dx, dgamma, dbeta) in 64 bits, with the magnitudes (of dtot, dx,
    dgamma, dbeta) their fp32 evaluation errs by, in units of u."""
    dy, h, rstd = dy.double(), h.double(), rstd.double().view(-1, 1)
    mu = mean.double().view(-1, 1) if norm == "layernorm" else torch.zeros_like(rstd)
    xh = (h - mu) * rstd
    w = dy * gamma.double() if gamma is not None else dy
    c1 = (w * xh).mean(1, keepdim=True)
    c2 = w.mean(1, keepdim=True) if norm == "layernorm" else torch.zeros_like(c1)
    d = rstd * (w - c2 - xh * c1)
    # h - mu, its product with rstd and w: a rounding each
    e1 = (D + 5) * (w * xh).abs().mean(1, keepdim=True)
    e2 = (D + 5) * w.abs().mean(1, keepdim=True) if norm == "layernorm" else 0.0
    e = rstd * (8 * w.abs() + xh.abs() * (8 * c1.abs() + e1) + 8 * c2.abs() + e2)
    if dh is not None:
        d, e = d + dh.double(), e + 4 * (d.abs() + dh.double().abs())
    dx, ex = d, e
    if p:
        k = mask.to(d.device)
        dx = torch.where(k, d / (1.0 - p), torch.zeros_like(d))
        ex = torch.where(k, (e + 3 * d.abs()) / (1.0 - p), torch.zeros_like(d))
    rows = dy.shape[0] + 8.0
    return (d, dx, (dy * xh).sum(0), dy.sum(0),
            e, ex, rows * (dy * xh).abs().sum(0), rows * dy.abs().sum(0))


def assert_close(got, want, bound, what):
    got = got.double().view(want.shape)
    bad = ~((got - want).abs() <= bound)
    if bool(bad.any()):
        i = int(torch.where(bad.view(-1))[0][0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} elements off, first at {i}: "
                             f"{float(got.view(-1)[i])} for {float(want.view(-1)[i])}, bound "
                             f"{float(bound.expand_as(want).reshape(-1)[i])}")
