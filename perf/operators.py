"""The training operators of the row norms, measured as a user calls them.

Three operators stand beside the library's row-wise forward kernels:

  norm_forward   h = residual + dropout(x), y = norm(h), with the row
                 statistics the backward pass needs (LayerNorm or RMSNorm;
                 residual and dropout optional)
  norm_backward  the gradient of that step: of x, of the residual, and of the
                 norm's parameters (reduced over every row)
  dropout        y = residual + dropout(x) on its own; with the incoming
                 gradient as x it is its own backward pass

Dropout draws its mask from a counter-based generator and never stores it:
Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
numbers: as easy as 1, 2, 3", 2011).  The element in row r and column c of a
call reads word c % 4 of the block with counter (c / 4, r, offset low, offset
high) and key (seed low, seed high), and is kept when that word is at least
floor(p 2^32).

``own`` False computes the operators in their plain form, elementary torch
operations in 32 bits; ``own`` True makes the package's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = {"layernorm": 1e-5, "rmsnorm": 1e-6}
MASK32 = 0xFFFFFFFF
MOST_ELEMENTS = 1 << 27   # of a drawn case: half of the largest listed one


def _case(name, op, rows, cols, dtype, norm="layernorm", pdtype="f32", residual=False, p=0.0):
    return {"name": name, "op": op, "norm": norm, "rows": rows, "cols": cols, "dtype": dtype,
            "pdtype": pdtype, "residual": residual, "p": p}


def listed():
    return [
        # one token of a generation step: the residual add and the next norm
        _case("fwd_rms_token", "norm_forward", 1, 4096, "bf16", "rmsnorm", "bf16", residual=True),
        # a generation step of 64 sequences
        _case("fwd_ln_decode", "norm_forward", 64, 8192, "bf16", residual=True),
        # a training step's block: dropout, residual add and norm of 16384 tokens
        _case("fwd_ln_train", "norm_forward", 16384, 4096, "bf16", residual=True, p=0.1),
        # rows of an odd width, none of which starts on a vector boundary
        _case("fwd_ln_ragged", "norm_forward", 2048, 10001, "bf16", residual=True, p=0.1),
        # the wide LayerNorm workload of the benchmarks, with statistics kept
        _case("fwd_ln_wide", "norm_forward", 1024, 262144, "bf16"),
        # the backward pass of a few short fp32 rows: launch latency counts
        _case("bwd_ln_small", "norm_backward", 32, 1024, "f32"),
        # the backward pass of the training block above
        _case("bwd_ln_train", "norm_backward", 16384, 4096, "bf16", residual=True, p=0.1),
        # RMSNorm's backward pass at a larger hidden size, no dropout
        _case("bwd_rms_train", "norm_backward", 8192, 8192, "bf16", "rmsnorm", "bf16",
              residual=True),
        # fp32 rows of an odd width
        _case("bwd_ln_ragged", "norm_backward", 2048, 10001, "f32"),
        # few rows of the widest RMSNorm workload of the benchmarks
        _case("bwd_rms_wide", "norm_backward", 256, 786432, "bf16", "rmsnorm", "bf16"),
        # dropout of a small activation
        _case("drop_small", "dropout", 64, 4096, "bf16", p=0.1),
        # dropout and residual add of a training step's activations
        _case("drop_add_train", "dropout", 16384, 8192, "bf16", residual=True, p=0.1),
    ]


def draw(rng):
    """One more case: a decode, training or wide shape of any of the operators."""
    op = rng.choice(["norm_forward", "norm_backward", "norm_forward", "norm_backward", "dropout"])
    norm = rng.choice(["layernorm", "rmsnorm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    while True:
        rows = int(round(2.0 ** rng.uniform(0.0, 16.0)))
        cols = int(round(2.0 ** rng.uniform(6.0, math.log2(786432))))
        if rng.random() < 0.6:  # hidden sizes are mostly multiples of 64; the others stay odd
            cols = max(64, cols // 64 * 64)
        if 1024 <= rows * cols <= MOST_ELEMENTS:
            break
    p = rng.choice([0.05, 0.1, 0.25, 0.5]) if op == "dropout" or rng.random() < 0.5 else 0.0
    return {"op": op, "norm": norm, "rows": rows, "cols": cols, "dtype": dtype,
            "pdtype": dtype if rng.random() < 0.5 else "f32", "residual": rng.random() < 0.6,
            "p": p}


def prepare(case, seed):
    """Activations with a few large channels, as residual streams have, the
    parameters, the row statistics a forward pass left and the dropout's seed."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rows, cols, dt, pdt = case["rows"], case["cols"], DTYPES[case["dtype"]], DTYPES[case["pdtype"]]

    def normal(shape, mean, std, dtype):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(std) \
            .add_(mean).to(dtype)

    state = {"case": dict(case), "eps": EPS[case["norm"]], "p": case["p"],
             "seed": (seed * 0x9E3779B97F4A7C15 + 0x1234567) & 0xFFFFFFFFFFFFFFFF,
             "offset": (seed * 40503 + 7) & 0xFFFFFFFFFF, "residual": None}
    channel = torch.ones(cols, device=dev)
    channel[:: max(1, cols // 4)] = 12.0

    def stream(std, mean):  # a residual stream's rows
        return (torch.randn((rows, cols), generator=g, device=dev).mul_(std).mul_(channel)
                .add_(mean)).to(dt)

    if case["op"] in ("norm_forward", "dropout"):
        state["x"] = normal((rows, cols), 0.1, 1.0, dt)
        if case["residual"]:
            state["residual"] = stream(1.5, 0.25)
    if case["op"] != "dropout":
        state["gamma"] = normal((cols,), 1.0, 0.1, pdt)
        state["beta"] = normal((cols,), 0.0, 0.1, pdt) if case["norm"] == "layernorm" else None
    if case["op"] == "norm_backward":
        state["h"] = stream(1.5, 0.25)
        state["dy"] = normal((rows, cols), 0.0, 1.0, dt)
        # the gradient that reaches h past the norm, along the residual stream
        state["dh"] = normal((rows, cols), 0.0, 1.0, dt) if case["residual"] else None
        h = state["h"].float()
        mean = h.mean(1, keepdim=True) if case["norm"] == "layernorm" else None
        if mean is not None:
            h = h - mean
        state["mean"] = mean.view(-1).contiguous() if mean is not None else None
        state["rstd"] = torch.rsqrt(h.square().mean(1) + state["eps"])
    return state


def run(state):
    case = state["case"]
    if own:
        import dsmem_thread_block_gb300 as credit
        drop = credit.Dropout(state["p"], state["seed"], state["offset"]) if state["p"] else None
        if case["op"] == "dropout":
            return {"y": credit.dropout(state["x"], drop, residual=state["residual"])}
        if case["op"] == "norm_forward":
            if case["norm"] == "layernorm":
                y, h, mean, rstd = credit.layernorm_forward(
                    state["x"], state["gamma"], state["beta"], eps=state["eps"],
                    residual=state["residual"], dropout=drop)
            else:
                mean = None
                y, h, rstd = credit.rmsnorm_forward(
                    state["x"], state["gamma"], eps=state["eps"], residual=state["residual"],
                    dropout=drop)
            return _forward_outputs(case, y, h, mean, rstd)
        if case["norm"] == "layernorm":
            dx, dres, dgamma, dbeta = credit.layernorm_backward(
                state["dy"], state["h"], state["mean"], state["rstd"], state["gamma"],
                dh=state["dh"], dropout=drop, need_dresidual=case["residual"])
        else:
            dbeta = None
            dx, dres, dgamma = credit.rmsnorm_backward(
                state["dy"], state["h"], state["rstd"], state["gamma"], dh=state["dh"],
                dropout=drop, need_dresidual=case["residual"])
        return _backward_outputs(case, dx, dres, dgamma, dbeta)
    return _plain(state)


def _forward_outputs(case, y, h, mean, rstd):
    out = {"y": y, "rstd": rstd}
    if case["norm"] == "layernorm":
        out["mean"] = mean
    if case["residual"] or case["p"]:
        out["h"] = h  # without either, h is x
    return out


def _backward_outputs(case, dx, dres, dgamma, dbeta):
    out = {"dx": dx, "dgamma": dgamma}
    if case["norm"] == "layernorm":
        out["dbeta"] = dbeta
    if case["residual"] and case["p"]:
        out["dresidual"] = dres  # without dropout it equals dx
    return out


# ------------------------------------------------------------ the plain form
def _keep(state, rows, cols, device):
    """The dropout mask of a rows x cols call: Philox4x32-10 on int64 tensors,
    whose products wrap modulo 2^64."""
    c0 = torch.arange((cols + 3) // 4, device=device)[None, :].expand(rows, -1)
    c1 = torch.arange(rows, device=device)[:, None].expand(-1, c0.shape[1])
    c2 = torch.full_like(c0, state["offset"] & MASK32)
    c3 = torch.full_like(c0, state["offset"] >> 32)
    k0, k1 = state["seed"] & MASK32, state["seed"] >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((p1 >> 32) & MASK32) ^ c1 ^ k0, p1 & MASK32,
                          ((p0 >> 32) & MASK32) ^ c3 ^ k1, p0 & MASK32)
        k0, k1 = (k0 + 0x9E3779B9) & MASK32, (k1 + 0xBB67AE85) & MASK32
    words = torch.stack([c0, c1, c2, c3], dim=2).view(rows, -1)[:, :cols]
    return words >= int(state["p"] * 4294967296.0)


def _plain(state):
    case = state["case"]
    rows, cols, dt, pdt = case["rows"], case["cols"], DTYPES[case["dtype"]], DTYPES[case["pdtype"]]
    p = state["p"]
    if case["op"] in ("dropout", "norm_forward"):
        h = state["x"].float()
        if p:
            keep = _keep(state, rows, cols, h.device)
            h = torch.where(keep, h * (1.0 / (1.0 - p)), torch.zeros_like(h))
        if state["residual"] is not None:
            h = h + state["residual"].float()
        if case["op"] == "dropout":
            return {"y": h.to(dt)}
        mean, z = None, h
        if case["norm"] == "layernorm":
            mean = h.sum(1, keepdim=True) / cols
            z = h - mean
        rstd = 1.0 / torch.sqrt((z * z).sum(1, keepdim=True) / cols + state["eps"])
        y = z * rstd * state["gamma"].float()
        if state["beta"] is not None:
            y = y + state["beta"].float()
        return _forward_outputs(case, y.to(dt), h.to(dt), None if mean is None else mean.view(-1),
                                rstd.view(-1))
    dy, h, rstd = state["dy"].float(), state["h"].float(), state["rstd"][:, None]
    z = (h - state["mean"][:, None] if state["mean"] is not None else h) * rstd
    wdy = dy * state["gamma"].float()
    g = wdy - z * ((wdy * z).sum(1, keepdim=True) / cols)
    if state["mean"] is not None:
        g = g - wdy.sum(1, keepdim=True) / cols
    g = g * rstd
    if state["dh"] is not None:
        g = g + state["dh"].float()
    dx = g
    if p:
        keep = _keep(state, rows, cols, g.device)
        dx = torch.where(keep, g * (1.0 / (1.0 - p)), torch.zeros_like(g))
    return _backward_outputs(case, dx.to(dt), g.to(dt), (dy * z).sum(0).to(pdt),
                             dy.sum(0).to(pdt))


def work(case):
    """Each input read once, each output written once."""
    n, cols = case["rows"] * case["cols"], case["cols"]
    es = 4 if case["dtype"] == "f32" else 2
    ps = 4 if case["pdtype"] == "f32" else 2
    ln = case["norm"] == "layernorm"
    both = case["residual"] or case["p"]
    if case["op"] == "dropout":
        return {"bytes": n * es * (3 if case["residual"] else 2),
                "flops": n * (2 if case["residual"] else 1)}
    stats = 4 * case["rows"] * (2 if ln else 1)
    if case["op"] == "norm_forward":
        moved = 2 + (1 if case["residual"] else 0) + (1 if both else 0)
        flops = (8 if ln else 5) + (1 if case["residual"] else 0) + (1 if case["p"] else 0)
        return {"bytes": n * es * moved + cols * ps * (2 if ln else 1) + stats, "flops": n * flops}
    moved = 3 + (1 if case["residual"] else 0) + (1 if case["residual"] and case["p"] else 0)
    flops = (13 if ln else 10) + (1 if case["residual"] else 0) + (1 if case["p"] else 0)
    return {"bytes": n * es * moved + cols * ps * (3 if ln else 2) + stats, "flops": n * flops}


# ------------------------------------------------- the definition in 64 bits
def _mul_halves(a, m):
    """High and low 32 bits of a * m for a tensor of 32-bit values and a 32-bit
    constant, from 16-bit digits so that no product passes 2^49."""
    lo, hi = a * (m & 0xFFFF), a * (m >> 16)
    mid = (hi & 0xFFFF) * 65536 + lo
    return (hi >> 16) + (mid >> 32), mid & MASK32


def _exact_kept(state, shape, device):
    rows, cols = shape
    groups = torch.arange(-(-cols // 4), device=device).repeat(rows, 1)
    ctr = [groups, torch.zeros_like(groups) + torch.arange(rows, device=device).unsqueeze(1),
           torch.zeros_like(groups) + state["offset"] % 4294967296,
           torch.zeros_like(groups) + state["offset"] // 4294967296]
    key = [state["seed"] % 4294967296, state["seed"] // 4294967296]
    for _ in range(10):
        hi0, lo0 = _mul_halves(ctr[0], 0xD2511F53)
        hi1, lo1 = _mul_halves(ctr[2], 0xCD9E8D57)
        ctr = [hi1.bitwise_xor(ctr[1]).bitwise_xor(key[0]), lo1,
               hi0.bitwise_xor(ctr[3]).bitwise_xor(key[1]), lo0]
        key = [(key[0] + 0x9E3779B9) % 4294967296, (key[1] + 0xBB67AE85) % 4294967296]
    threshold = math.floor(state["p"] * 2.0 ** 32)
    kept = torch.empty((rows, groups.shape[1] * 4), dtype=torch.bool, device=device)
    for w in range(4):
        kept[:, w::4] = ctr[w] >= threshold
    return kept[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    norm_ln, n = case["norm"] == "layernorm", case["cols"]

    def dropped(t):
        if not s["p"]:
            return t
        return (t / (1.0 - s["p"])).masked_fill_(~_exact_kept(s, t.shape, t.device), 0.0)

    if case["op"] != "norm_backward":
        total = dropped(s["x"].double())
        if s["residual"] is not None:
            total = total + s["residual"].double()
        if case["op"] == "dropout":
            return {"y": total}
        mu = total.mean(dim=1) if norm_ln else None
        dev2 = (total - mu.unsqueeze(1)).pow(2) if norm_ln else total.pow(2)
        inv = (dev2.mean(dim=1) + s["eps"]).pow(-0.5)
        y = total.sub(mu.unsqueeze(1)) if norm_ln else total.clone()
        y = y.mul_(inv.unsqueeze(1)).mul_(s["gamma"].double())
        if norm_ln:
            y = y.add_(s["beta"].double())
        return _forward_outputs(case, y, total, mu, inv)
    inv = s["rstd"].double().unsqueeze(1)
    xhat = s["h"].double()
    if norm_ln:
        xhat = xhat - s["mean"].double().unsqueeze(1)
    xhat = xhat * inv
    dy = s["dy"].double()
    dgamma, dbeta = (dy * xhat).sum(dim=0), dy.sum(dim=0)
    up = dy * s["gamma"].double()
    # the normalised row's gradient without its parts along the row itself
    # and, for LayerNorm, along the constant row
    along = (up * xhat).sum(dim=1, keepdim=True) / n
    total = up.sub(xhat.mul_(along))
    if norm_ln:
        total = total.sub_(up.sum(dim=1, keepdim=True) / n)
    total = total.mul_(inv)
    if s["dh"] is not None:
        total = total.add_(s["dh"].double())
    return _backward_outputs(case, dropped(total), total, dgamma, dbeta)
