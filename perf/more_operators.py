"""The two ends of a training step, measured as a user calls them.

  ce_forward     the loss of a linear head over a large vocabulary, from the
                 last hidden states and the head's weight, the logits never
                 stored: lse_t = log sum_v exp(h_t . w_v), loss_t = lse_t -
                 h_t . w_target (0 for an ignored target)
  ce_backward    its gradient, of the hidden states and of the weight:
                 g_tv = dloss_t (p_tv - [v = target_t]) + dlse_t p_tv with
                 p_tv = exp(h_t . w_v - lse_t), dhidden = g w, dweight = g^T h
  gradient_norm  the 2-norm of all gradients together, and their clipping to a
                 largest norm: g min(1, max_norm / (norm + eps))

``own`` False computes the operators in their plain form, elementary torch
operations in 32 bits; ``own`` True makes the package's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
IGNORE = -100
CLIP_EPS = 1e-6
MOST_FLOPS = 2.2e12      # of a drawn loss: half of the largest listed one's
MOST_LOGITS = 1 << 29    # which the plain form holds
MOST_GRADS = 1 << 28     # elements of a drawn set of gradients


def _ce(name, op, tokens, hidden, vocab, dtype, ignored=0.0, zloss=False):
    return {"name": name, "op": op, "tokens": tokens, "hidden": hidden, "vocab": vocab,
            "dtype": dtype, "ignored": ignored, "zloss": zloss}


def _clip(name, sizes, dtype, clip=True, repeat=1, vectors=0, mixed=False):
    # `repeat` times matrices of the elements in `sizes` (a text) and `vectors` small ones
    return {"name": name, "op": "gradient_norm", "sizes": sizes, "dtype": dtype, "clip": clip,
            "repeat": repeat, "vectors": vectors, "mixed": mixed}


def listed():
    return [
        # the log-probability of one token of a generation step
        _ce("ce_fwd_token", "ce_forward", 1, 4096, 131072, "bf16"),
        # a few tokens of a small model: launch latency counts
        _ce("ce_fwd_small", "ce_forward", 32, 1024, 4096, "bf16"),
        # the loss of a training step's tokens, padding ignored
        _ce("ce_fwd_train", "ce_forward", 4096, 4096, 131072, "bf16", ignored=0.1),
        # odd sizes throughout: no row starts on a 16-byte boundary
        _ce("ce_fwd_ragged", "ce_forward", 777, 1001, 10001, "bf16", ignored=0.1),
        # fp32 hidden states and weight
        _ce("ce_fwd_f32", "ce_forward", 512, 2048, 16384, "f32"),
        # the gradient of a few tokens
        _ce("ce_bwd_small", "ce_backward", 64, 1024, 4096, "bf16"),
        # the gradient of a training step, with a penalty on lse
        _ce("ce_bwd_train", "ce_backward", 4096, 4096, 65536, "bf16", ignored=0.1, zloss=True),
        # fp32 at odd sizes
        _ce("ce_bwd_ragged", "ce_backward", 333, 1001, 10001, "f32", ignored=0.1),
        # clipping a small model's gradients: launch latency counts
        _clip("clip_small", "65536,4096,262144,1024", "f32", repeat=2, vectors=4),
        # clipping the bf16 gradients of two blocks of hidden size 4096
        _clip("clip_blocks", "50331648,16777216,67108864,67108864", "bf16", repeat=2, vectors=8),
        # the norm alone of many ragged gradients, both types among them
        _clip("norm_many", "1048577,524287,99991,10001", "f32", clip=False, repeat=64, vectors=200,
              mixed=True),
        # clipping fp32 gradients that pass the L2 several times
        _clip("clip_f32", "134217728,16777216", "f32", repeat=2),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(2.0 ** rng.uniform(math.log2(lo), math.log2(hi))))


def draw(rng):
    """One more case: tokens from one to a large batch, hidden sizes and
    vocabularies from small to wide, odd ones among them; sets of a few or many
    gradients."""
    op = rng.choice(["ce_forward", "ce_backward", "gradient_norm"])
    if op == "gradient_norm":
        while True:
            sizes = [_log_uniform(rng, 1, 1 << 26) for _ in range(rng.randint(1, 6))]
            repeat = _log_uniform(rng, 1, 128)
            if sum(sizes) * repeat <= MOST_GRADS:
                break
        return {"op": op, "sizes": ",".join(str(s) for s in sizes),
                "dtype": rng.choice(["bf16", "f32"]), "clip": rng.random() < 0.7, "repeat": repeat,
                "vectors": rng.randint(0, 300), "mixed": rng.random() < 0.4}
    dtype = rng.choice(["bf16", "bf16", "f32"])
    while True:
        tokens = _log_uniform(rng, 1, 8192)
        hidden = _log_uniform(rng, 32, 8192)
        vocab = _log_uniform(rng, 64, 262144)
        if rng.random() < 0.6:  # hidden sizes are mostly multiples of 64; the others stay odd
            hidden = max(64, hidden // 64 * 64)
        if rng.random() < 0.5:
            vocab = max(128, vocab // 128 * 128)
        products = (6 if op == "ce_backward" else 2) * float(tokens) * hidden * vocab
        if products <= MOST_FLOPS and tokens * vocab <= MOST_LOGITS and vocab * hidden <= 1 << 30:
            break
    return {"op": op, "tokens": tokens, "hidden": hidden, "vocab": vocab, "dtype": dtype,
            "ignored": rng.choice([0.0, 0.1, 0.5]), "zloss": rng.random() < 0.4}


def _lengths(case):
    """Elements of each gradient of a set, and whether it has the other type."""
    sizes = [int(s) for s in case["sizes"].split(",")] * case["repeat"]
    sizes += [1024 + 37 * (i % 5) for i in range(case["vectors"])]
    return [(n, case["mixed"] and i % 3 == 1) for i, n in enumerate(sizes)]


def prepare(case, seed):
    """Hidden states behind a final norm, a weight whose logits spread over a few
    units, targets of which some are padding, and what a forward pass left;
    or a step's gradients, each tensor on its own scale."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    state = {"case": dict(case)}
    if case["op"] == "gradient_norm":
        other = torch.bfloat16 if dt == torch.float32 else torch.float32
        grads, square = [], 0.0
        for i, (n, mixed) in enumerate(_lengths(case)):
            std = 10.0 ** (-1.0 - (i % 5))
            square += std * std * n
            grads.append(torch.randn(n, generator=g, device=dev).mul_(std).to(other if mixed else dt))
        state["grads"] = grads
        # most steps of a run that clips are above the limit
        state["max_norm"] = 0.25 * math.sqrt(square)
        if case["clip"]:
            # the clipped gradients lie in one buffer per type, as an optimizer's step takes them
            state["flat"], state["out"] = _flat(grads, lambda t: t.dtype)
        return state
    tokens, hidden, vocab = case["tokens"], case["hidden"], case["vocab"]
    h = torch.randn((tokens, hidden), generator=g, device=dev).to(dt)
    w = torch.empty((vocab, hidden), dtype=dt, device=dev)
    for i in range(0, vocab, 16384):
        n = min(16384, vocab - i)
        w[i:i + n] = torch.randn((n, hidden), generator=g, device=dev).mul_(2.5 / math.sqrt(hidden))
    target = torch.randint(0, vocab, (tokens,), generator=g, device=dev)
    if case["ignored"]:
        pad = torch.rand((tokens,), generator=g, device=dev) < case["ignored"]
        target = torch.where(pad, torch.full_like(target, IGNORE), target)
    state.update(h=h, w=w, target=target)
    if case["op"] == "ce_backward":
        state["lse"] = torch.cat([_pieces_lse(h[i:i + 1024], w) for i in range(0, tokens, 1024)])
        counted = (target != IGNORE).sum().clamp(min=1).float()
        # a mean over the counted tokens, whose weights differ a little
        state["dloss"] = (0.75 + 0.5 * torch.rand((tokens,), generator=g, device=dev)) / counted
        state["dlse"] = 2e-2 * state["lse"] / counted if case["zloss"] else None
    return state


def _flat(tensors, dtype_of):
    """A zeroed buffer per type, and the place of each tensor in them, each at a
    multiple of 64 elements."""
    at, places = {}, []
    for t in tensors:
        first = at.get(t.dtype, 0)
        places.append((t.dtype, first, t.numel()))
        at[t.dtype] = first + (t.numel() + 63) // 64 * 64
    of = {t.dtype: dtype_of(t) for t in tensors}
    flat = {d: torch.zeros(n, dtype=of[d], device=tensors[0].device) for d, n in at.items()}
    return flat, [flat[d][first:first + n] for d, first, n in places]


def _pieces_lse(h, w):
    """lse of some rows, from fp32 logits a piece of the vocabulary at a time."""
    parts = []
    for i in range(0, w.shape[0], 32768):
        parts.append(torch.logsumexp(h.float() @ w[i:i + 32768].float().t(), 1))
    return torch.logsumexp(torch.stack(parts), 0)


def run(state):
    case = state["case"]
    if own:
        import dsmem_thread_block_gb300 as credit
        if case["op"] == "gradient_norm":
            if not case["clip"]:
                return {"norm": credit.gradient_norm(state["grads"])}
            norm = credit.clip_gradients(state["grads"], state["max_norm"], eps=CLIP_EPS,
                                         out=state["out"])
            return _clip_outputs(norm, state["flat"])
        if case["op"] == "ce_forward":
            loss, lse = credit.linear_cross_entropy_forward(
                state["h"], state["w"], state["target"], ignore_index=IGNORE)
            return {"loss": loss, "lse": lse}
        dhidden, dweight = credit.linear_cross_entropy_backward(
            state["dloss"], state["h"], state["w"], state["target"], state["lse"],
            dlse=state["dlse"], ignore_index=IGNORE)
        return {"dhidden": dhidden, "dweight": dweight}
    return _plain(state)


def _clip_outputs(norm, flat):
    out = {"norm": norm}
    for dtype, name in ((torch.float32, "f32"), (torch.bfloat16, "bf16")):
        if dtype in flat:
            out[name] = flat[dtype]
    return out


# ------------------------------------------------------------ the plain form
def _plain(state):
    case = state["case"]
    if case["op"] == "gradient_norm":
        square = torch.zeros((), device=state["grads"][0].device)
        for t in state["grads"]:
            f = t.float()
            square = square + (f * f).sum()
        norm = torch.sqrt(square)
        if not case["clip"]:
            return {"norm": norm}
        factor = torch.clamp(state["max_norm"] / (norm + CLIP_EPS), max=1.0)
        for t, o in zip(state["grads"], state["out"]):
            o.copy_(t.float() * factor)
        return _clip_outputs(norm, state["flat"])
    h, w, target = state["h"].float(), state["w"].float(), state["target"]
    logits = h @ w.t()
    kept = target != IGNORE
    index = torch.where(kept, target, torch.zeros_like(target))[:, None]
    if case["op"] == "ce_forward":
        top = logits.amax(1, keepdim=True)
        lse = (top + torch.log(torch.exp(logits - top).sum(1, keepdim=True)))[:, 0]
        picked = torch.gather(logits, 1, index)[:, 0]
        return {"loss": torch.where(kept, lse - picked, torch.zeros_like(lse)), "lse": lse}
    scale = torch.where(kept, state["dloss"], torch.zeros_like(state["dloss"]))
    both = scale if state["dlse"] is None else scale + state["dlse"]
    grad = torch.exp(logits - state["lse"][:, None]) * both[:, None]
    grad.scatter_add_(1, index, -scale[:, None])
    return {"dhidden": (grad @ w).to(state["h"].dtype), "dweight": (grad.t() @ h).to(state["w"].dtype)}


def work(case):
    """Each input read once, each output written once; the loss's gradient forms
    the logits' products again."""
    if case["op"] == "gradient_norm":
        es = {"f32": 4, "bf16": 2}[case["dtype"]]
        n = sum(c for c, _ in _lengths(case))
        moved = sum(c * (6 - es if mixed else es) for c, mixed in _lengths(case))
        return {"bytes": moved * (2 if case["clip"] else 1) + 4, "flops": n * (3 if case["clip"] else 2)}
    t, d, v = case["tokens"], case["hidden"], case["vocab"]
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "ce_forward":
        return {"bytes": (t + v) * d * es + t * 16, "flops": 2 * t * d * v}
    return {"bytes": 2 * (t + v) * d * es + t * (20 if case["zloss"] else 16), "flops": 6 * t * d * v}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gradient_norm":
        norm = math.sqrt(math.fsum(float(t.double().pow(2).sum()) for t in s["grads"]))
        out = torch.tensor(norm, dtype=torch.float64, device=s["grads"][0].device)
        if not case["clip"]:
            return {"norm": out}
        factor = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
        flat, places = _flat(s["grads"], lambda t: torch.float64)
        for t, o in zip(s["grads"], places):
            torch.mul(t.double(), factor, out=o)
        return _clip_outputs(out, flat)
    h, w, target = s["h"].double(), s["w"], s["target"]
    tokens, vocab, piece = case["tokens"], case["vocab"], 8192
    counted = (target >= 0).double()
    dev = h.device
    if case["op"] == "ce_forward":
        top = torch.full((tokens,), -math.inf, dtype=torch.float64, device=dev)
        total, picked = torch.zeros_like(top), torch.zeros_like(top)
        for v0 in range(0, vocab, piece):
            z = h @ w[v0:v0 + piece].double().t()
            new = torch.maximum(top, z.max(dim=1).values)
            total = total * (top - new).exp() + (z - new[:, None]).exp().sum(dim=1)
            top = new
            here = (target >= v0) & (target < v0 + z.shape[1])
            rows = here.nonzero()[:, 0]
            picked[rows] = z[rows, target[rows] - v0]
        lse = top + total.log()
        return {"loss": (lse - picked) * counted, "lse": lse}
    scale = s["dloss"].double() * counted
    extra = s["dlse"].double() if s["dlse"] is not None else torch.zeros_like(scale)
    dh, dw = torch.zeros_like(h), torch.empty(w.shape, dtype=torch.float64, device=dev)
    for v0 in range(0, vocab, piece):
        wp = w[v0:v0 + piece].double()
        p = (h @ wp.t()).sub_(s["lse"].double()[:, None]).exp_()
        p *= (scale + extra)[:, None]
        rows = ((target >= v0) & (target < v0 + wp.shape[0])).nonzero()[:, 0]
        p[rows, target[rows] - v0] -= scale[rows]
        dh += p @ wp
        dw[v0:v0 + piece] = p.t() @ h
    return {"dhidden": dh, "dweight": dw}
