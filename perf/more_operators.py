"""Measured cases of the operators around the experts' products: the router (top-k, per-expert counts, balance
loss, with gradients), 8-bit integer products with a scale for each token and channel, and the gated activation
kept in 8 bits for the backward pass.

listed() names the cases, draw(rng) gives another of the same ranges, prepare(case, seed) makes what a program
holds before the call, run(state) is one pass through an operator, exact(case, seed) the same outputs in 64 bits,
and work(case) the bytes and operations that a pass cannot do without.  With `own` false run() computes the
operators from elementary torch operations; with `own` true it calls the library.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "f32": 4}


def listed():
    return [
        # One decoding step's tokens on eight experts, no gradients.  Latency.
        {"name": "router-decode", "op": "router", "dtype": "bf16", "tokens": 64, "experts": 8, "k": 2, "normalize": True,
         "train": False, "masked": 0, "closed": 0, "gap": 0},
        # A micro-batch of four sequences in training, a part of the tokens padding.
        {"name": "router-train", "op": "router", "dtype": "bf16", "tokens": 16384, "experts": 64, "k": 6, "normalize": True,
         "train": True, "masked": 700, "closed": 0, "gap": 0},
        # Many small experts with float32 logits, three of them closed (their logits are -inf).
        {"name": "router-train-wide", "op": "router", "dtype": "f32", "tokens": 65536, "experts": 256, "k": 8,
         "normalize": False, "train": True, "masked": 0, "closed": 3, "gap": 0},
        # One token through one projection.
        {"name": "int8-one-token", "op": "int8", "dtype": "bf16", "groups": 1, "tokens": 1, "n": 14336, "k": 4096,
         "skew": "even", "empty": 0, "dead": 0, "gap": 0, "out32": False},
        # One decoding step: 96 routed rows over 64 experts, some without a row.  The weights' bytes.
        {"name": "int8-experts-decode", "op": "int8", "dtype": "bf16", "groups": 64, "tokens": 96, "n": 2048, "k": 7168,
         "skew": "zipf", "empty": 4, "dead": 32, "gap": 0, "out32": False},
        # Prompts through eight large experts.
        {"name": "int8-experts-prompts", "op": "int8", "dtype": "bf16", "groups": 8, "tokens": 16384, "n": 14336,
         "k": 4096, "skew": "dirichlet", "empty": 0, "dead": 0, "gap": 0, "out32": False},
        # Prompts over many small experts with very uneven loads, capacity rows unused.
        {"name": "int8-experts-zipf", "op": "int8", "dtype": "fp16", "groups": 64, "tokens": 32768, "n": 2048, "k": 7168,
         "skew": "zipf", "empty": 4, "dead": 1000, "gap": 0, "out32": False},
        # The weights of eight experts quantized by channel, when a checkpoint is loaded.
        {"name": "int8-quantize-weights", "op": "int8-quantize", "dtype": "bf16", "rows": 114688, "cols": 4096, "gap": 0},
        # A small expert layer's activation.  Latency.
        {"name": "checkpoint-small", "op": "checkpoint", "backward": False, "dtype": "bf16", "groups": 4, "tokens": 128,
         "hidden": 128, "weighted": True, "recompute": False, "dead": 0, "gap": 0},
        # The activation of eight large experts, kept in 8 bits.
        {"name": "checkpoint-forward", "op": "checkpoint", "backward": False, "dtype": "bf16", "groups": 8, "tokens": 16384,
         "hidden": 14336, "weighted": True, "recompute": False, "dead": 0, "gap": 0},
        # Its backward pass: both halves' gradients, the router weight's, and the activation again for the second
        # product's weight gradient.
        {"name": "checkpoint-backward", "op": "checkpoint", "backward": True, "dtype": "bf16", "groups": 8, "tokens": 16384,
         "hidden": 14336, "weighted": True, "recompute": True, "dead": 0, "gap": 0},
        # Many small experts of an odd width, no router weight, capacity rows unused.
        {"name": "checkpoint-backward-odd", "op": "checkpoint", "backward": True, "dtype": "fp16", "groups": 64,
         "tokens": 32000, "hidden": 2080, "weighted": False, "recompute": False, "dead": 768, "gap": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "int8", "int8", "int8-quantize", "checkpoint", "checkpoint"])
    if op == "router":
        experts = _log(rng, 2, 256)
        tokens = _log(rng, 1, 65536)
        return {"op": op, "dtype": rng.choice(["bf16", "fp16", "f32"]), "tokens": tokens, "experts": experts,
                "k": rng.randrange(1, min(experts, 16) + 1), "normalize": rng.random() < 0.5,
                "train": rng.random() < 0.7, "masked": rng.choice([0, tokens // 9]),
                "closed": rng.choice([0, experts // 10]), "gap": rng.choice([0, 0, 3])}
    if op == "int8":
        while True:
            groups = rng.choice([1, _log(rng, 1, 128)])
            case = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "groups": groups, "tokens": _log(rng, 1, 32768),
                    "n": 8 * _log(rng, 8, 1792), "k": 16 * _log(rng, 4, 896),
                    "skew": rng.choice(["even", "dirichlet", "zipf"]), "empty": rng.randrange(groups // 4 + 1),
                    "dead": rng.choice([0, 0, _log(rng, 1, 500)]), "gap": rng.choice([0, 0, 8, 120]),
                    "out32": rng.random() < 0.2}
            if work(case)["flops"] <= 1.9e12 and groups * case["n"] * case["k"] <= 1e9:
                return case
    while True:
        if op == "int8-quantize":
            case = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "rows": _log(rng, 1, 131072),
                    "cols": 16 * _log(rng, 1, 1792), "gap": rng.choice([0, 0, 8])}
            if work(case)["bytes"] <= 1.4e9:
                return case
        else:
            case = {"op": op, "backward": rng.random() < 0.5, "dtype": rng.choice(["bf16", "fp16"]),
                    "groups": _log(rng, 1, 128), "tokens": _log(rng, 1, 65536), "hidden": 32 * _log(rng, 1, 600),
                    "weighted": rng.random() < 0.6, "recompute": rng.random() < 0.5,
                    "dead": rng.choice([0, 0, _log(rng, 1, 500)]), "gap": rng.choice([0, 0, 8])}
            if case["tokens"] * case["hidden"] <= 16384 * 14336:
                return case


# ---------------------------------------------------------------- sizes (of the case alone)


def _case_rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _counts(rng, groups, tokens, skew, empty):
    """Rows of each group: `tokens` drawn over groups - empty live ones."""
    if skew == "zipf":
        p = [(i + 1) ** -1.2 for i in range(groups)]
        rng.shuffle(p)
    elif skew == "dirichlet":
        p = [rng.gammavariate(2.0, 1.0) for _ in range(groups)]
    else:
        p = [1.0] * groups
    for g in rng.sample(range(groups), min(empty, groups - 1)):
        p[g] = 0.0
    counts = [0] * groups
    for g in rng.choices(range(groups), weights=p, k=tokens):
        counts[g] += 1
    return counts


def _row_counts(case):
    return _counts(_case_rng(case), case["groups"], case["tokens"], case.get("skew", "dirichlet"),
                   case.get("empty", 0))


def work(case):
    if case["op"] == "router":
        t, e, k = case["tokens"], case["experts"], case["k"]
        logits = t * e * SIZE[case["dtype"]] + (t if case["masked"] else 0)
        nbytes, flops = logits + 8 * t * k + 8 * e + 8, t * e * (4 + k)
        if case["train"]:  # the backward pass reads the logits again: they may have left the caches
            nbytes += logits + t * e * SIZE[case["dtype"]] + 8 * t * k
            flops += t * e * 8
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "int8":
        counts = _row_counts(case)
        t, n, k = sum(counts), case["n"], case["k"]
        active = sum(c > 0 for c in counts)
        return {"bytes": t * (2 * k + (4 if case["out32"] else 2) * n) + active * n * (k + 4), "flops": 2 * t * n * k}
    if case["op"] == "int8-quantize":
        return {"bytes": case["rows"] * (3 * case["cols"] + 4), "flops": 4 * case["rows"] * case["cols"]}
    t, f = case["tokens"], case["hidden"]
    kept = 2 * f + f // 16  # bytes a row
    if not case["backward"]:
        return {"bytes": t * (4 * f + 2 * f + kept + (4 if case["weighted"] else 0)), "flops": 20 * t * f}
    return {"bytes": t * (kept + 2 * f + 4 * f + (2 * f if case["recompute"] else 0) + (8 if case["weighted"] else 0)),
            "flops": 25 * t * f}


# ---------------------------------------------------------------- inputs


def _normal(gen, shape, dtype, std=1.0, outliers=0.0, gap=0):
    """Normal values rounded to `dtype`, a share of them 20 times as large; with `gap` the first columns of a wider
    buffer."""
    rows, cols = shape
    out = torch.empty((rows, cols + gap), dtype=dtype, device="cuda")[:, :cols]
    step = max(1, (1 << 26) // cols)
    for r in range(0, rows, step):
        m = min(step, rows - r)
        v = torch.randn((m, cols), generator=gen, device="cuda") * std
        if outliers:
            v = torch.where(torch.rand((m, cols), generator=gen, device="cuda") < outliers, v * 20, v)
        out[r:r + m] = v.to(dtype)
    return out


def _offsets(counts):
    ends = [0]
    for c in counts:
        ends.append(ends[-1] + c)
    return ends


def _rows(s, case):
    """The groups' ends, on the host and on the device, and the rows that the buffers hold."""
    s["ends"] = _offsets(_row_counts(case))
    s["offsets"] = torch.tensor(s["ends"], dtype=torch.int64, device="cuda")
    return s["ends"][-1] + case["dead"]


def _int8_weights(gen, groups, n, k):
    """Normal weights in 8 bits, a scale for each channel."""
    w = torch.empty((groups, n, k), dtype=torch.int8, device="cuda")
    scale = torch.empty((groups, n), device="cuda")
    flat, s = w.view(groups * n, k), scale.view(-1)
    step = max(1, (1 << 26) // k)
    for r in range(0, groups * n, step):
        v = torch.randn((min(step, groups * n - r), k), generator=gen, device="cuda") * 0.02
        s[r:r + step] = v.abs().amax(1) / 127
        flat[r:r + step] = (v / s[r:r + step, None]).round_().clamp_(-127, 127).to(torch.int8)
    return w, scale


def _mx_bytes(h):
    """The kept form of h [rows, cols]: E4M3 codes, and a scale byte for each 32 elements of a row.  The scale's
    exponent is that of the block's largest magnitude, less 8; elements are rounded to nearest even and saturate."""
    x = h.float().view(h.shape[0], -1, 32) if h.is_contiguous() else h.float().reshape(h.shape[0], -1, 32)
    amax = x.abs().amax(2)
    byte = torch.where(amax > 0, (torch.frexp(amax).exponent + (126 - 8)).clamp(min=0), 0)
    q = torch.ldexp(x, (127 - byte)[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(h.shape[0], -1).view(torch.uint8), byte.to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if own:
        import block_scaled_grouped_amd as bsg
        s["bsg"] = bsg
    if case["op"] == "router":
        t, e, dt = case["tokens"], case["experts"], DTYPES[case["dtype"]]
        s["logits"] = _normal(gen, (t, e), torch.float32, gap=0)
        s["logits"] += torch.randn(e, generator=gen, device="cuda") * 0.7  # some experts are liked more
        if case["closed"]:
            s["logits"][:, torch.randperm(e, generator=gen, device="cuda")[:case["closed"]]] = -math.inf
        wide = torch.empty((t, e + case["gap"]), dtype=dt, device="cuda")
        wide[:, :e] = s["logits"].to(dt)
        s["logits"] = wide[:, :e]
        s["mask"] = None
        if case["masked"]:
            s["mask"] = torch.ones(t, dtype=torch.bool, device="cuda")
            s["mask"][torch.randperm(t, generator=gen, device="cuda")[:case["masked"]]] = False
        if case["train"]:
            s["d_weights"] = torch.randn((t, case["k"]), generator=gen, device="cuda") / t
            s["d_loss"] = torch.rand(1, generator=gen, device="cuda") * 0.01 + 0.01
        if own:
            s["workspace"] = s["bsg"].moe_router_topk_workspace(t, e)
    elif case["op"] == "int8":
        cap = _rows(s, case)
        s["x"] = _normal(gen, (cap, case["k"]), DTYPES[case["dtype"]], outliers=0.01, gap=case["gap"])
        s["x"][s["ends"][-1]:] = float("nan")  # capacity rows that no group owns
        s["w"], s["w_scales"] = _int8_weights(gen, case["groups"], case["n"], case["k"])
        if own:
            s["workspace"] = s["bsg"].grouped_gemm_int8_dynamic_workspace(cap, case["k"])
    elif case["op"] == "int8-quantize":
        s["x"] = _normal(gen, (case["rows"], case["cols"]), DTYPES[case["dtype"]], std=0.02, gap=case["gap"])
    else:
        cap, f, dt = _rows(s, case), case["hidden"], DTYPES[case["dtype"]]
        h = _normal(gen, (cap, 2 * f), dt, outliers=0.005, gap=0 if case["backward"] else case["gap"])
        s["row_weights"] = torch.rand(cap, generator=gen, device="cuda") if case["weighted"] else None
        if case["backward"]:
            s["data"], s["scales"] = _mx_bytes(h)
            s["dy"] = _normal(gen, (cap, f), dt, std=0.1, gap=case["gap"])
            s["dy"][s["ends"][-1]:] = float("nan")
        else:
            h[s["ends"][-1]:] = float("nan")
            s["h"] = h
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    if own:
        return _run_own(s)
    return {"router": _plain_router, "int8": _plain_int8, "int8-quantize": _plain_quantize,
            "checkpoint": _plain_checkpoint}[s["op"]](s)


def _run_own(s):
    bsg = s["bsg"]
    if s["op"] == "router":
        r = bsg.moe_router_topk(s["logits"], s["k"], mask=s["mask"], normalize=s["normalize"], workspace=s["workspace"])
        out = [r["experts"], r["weights"], r["counts"], r["prob_sums"], r["live"], r["loss"]]
        if s["train"]:
            out.append(bsg.moe_router_topk_backward(
                s["logits"], r["experts"], r["counts"], r["live"], d_weights=s["d_weights"], d_loss=s["d_loss"],
                mask=s["mask"], normalize=s["normalize"]))
        return out
    if s["op"] == "int8":
        y = bsg.grouped_gemm_int8_dynamic(s["x"], s["w"], s["w_scales"], s["offsets"], workspace=s["workspace"],
                                          out_dtype=bsg.BSG_OUT_F32 if s["out32"] else None)
        return y[: s["ends"][-1]]
    if s["op"] == "int8-quantize":
        return bsg.grouped_quantize_int8(s["x"])
    t = s["ends"][-1]
    if not s["backward"]:
        y, data, scales = bsg.grouped_swiglu_checkpoint_mxfp8(s["h"], s["offsets"], row_weights=s["row_weights"])
        return [y[:t], data[:t].view(torch.float8_e4m3fn), scales[:t]]
    dh, dw, y = bsg.grouped_swiglu_checkpoint_mxfp8_backward(
        s["data"], s["scales"], s["dy"], s["offsets"], row_weights=s["row_weights"], recompute=s["recompute"])
    return [dh[:t], dw[:t] if s["weighted"] else None, y[:t] if s["recompute"] else None]


def _plain_router(s):
    l, k = s["logits"].float(), s["k"]
    t, e = l.shape
    live = (l > -math.inf).any(1)
    if s["mask"] is not None:
        live = live & s["mask"]
    ex = torch.exp(l - l.amax(1, keepdim=True))
    p = torch.where(live[:, None], ex / ex.sum(1, keepdim=True), 0.0)
    top, experts = torch.sort(l, dim=1, descending=True, stable=True)  # ties: the lowest index first
    top, experts = top[:, :k], experts[:, :k]
    chosen = live[:, None] & (top > -math.inf)
    w = torch.where(chosen, p.gather(1, experts), 0.0)
    if s["normalize"]:
        w = torch.where(chosen, w / w.sum(1, keepdim=True), 0.0)
    slots = torch.where(chosen, experts, e).reshape(-1)
    counts = torch.zeros(e + 1, dtype=torch.int32, device="cuda").index_add_(
        0, slots, torch.ones_like(slots, dtype=torch.int32))[:e]
    sums, n = p.double().sum(0), live.sum()  # a long sum
    loss = e / (k * n.double() ** 2) * (counts * sums).sum()
    out = [torch.where(chosen, experts, -1).int(), w, counts, sums.float(), n.int().view(1), loss.float().view(1)]
    if not s["train"]:
        return out
    dw = torch.where(chosen, s["d_weights"], 0.0)
    a = (s["d_loss"] * e / (k * n.float() ** 2) * counts).expand(t, e)
    if s["normalize"]:
        dl = p * (a - (p * a).sum(1, keepdim=True))
        dl = dl.scatter_add(1, experts, w * (dw - (w * dw).sum(1, keepdim=True)))
    else:
        a = a.scatter_add(1, experts, dw)
        dl = p * (a - (p * a).sum(1, keepdim=True))
    return out + [torch.where(live[:, None], dl, 0.0).to(s["logits"].dtype)]


def _quantized(x):
    """x = q * scale, row by row.  The quotients in 64 bits: in 32 some round onto the border of two integers."""
    amax = x.abs().amax(1, keepdim=True).float()
    scale = amax / torch.full_like(amax, 127)
    return torch.where(scale > 0, x.double() / scale.double(), 0.0).round_(), scale[:, 0]


def _plain_quantize(s):
    q, scale = _quantized(s["x"])
    return q.to(torch.int8), scale


def _plain_int8(s):
    ends = s["ends"]
    q, scale = _quantized(s["x"][: ends[-1]])
    q = q.float()
    y = torch.empty((ends[-1], s["n"]), dtype=torch.float32 if s["out32"] else s["x"].dtype, device="cuda")
    for g in range(s["groups"]):
        lo, hi = ends[g], ends[g + 1]
        if hi > lo:
            y[lo:hi] = ((q[lo:hi] @ s["w"][g].float().T) * scale[lo:hi, None] * s["w_scales"][g]).to(y.dtype)
    return y


def _plain_checkpoint(s):
    t, f = s["ends"][-1], s["hidden"]
    w = s["row_weights"][:t, None] if s["weighted"] else 1.0
    if not s["backward"]:
        h = s["h"][:t]
        g, u = h[:, :f].float(), h[:, f:].float()
        data, scales = _mx_bytes(h)
        return [(w * (g / (1 + torch.exp(-g))) * u).to(h.dtype), data.view(torch.float8_e4m3fn), scales]
    dy = s["dy"][:t].float()
    elements = s["data"][:t].view(torch.float8_e4m3fn).float().view(t, -1, 32)
    h = torch.ldexp(elements, s["scales"][:t, :, None].int() - 127).view(t, 2 * f)
    g, u = h[:, :f], h[:, f:]
    sig = 1 / (1 + torch.exp(-g))
    act = g * sig
    dh = torch.cat([dy * w * u * sig * (1 + g * (1 - sig)), dy * w * act], 1)
    return [dh.to(s["dy"].dtype), (dy * act * u).sum(1) if s["weighted"] else None,
            (w * act * u).to(s["dy"].dtype) if s["recompute"] else None]


# ---------------------------------------------------------------- in 64 bits


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"router": _exact_router, "int8": _exact_int8, "int8-quantize": _exact_quantize,
            "checkpoint": _exact_checkpoint}[case["op"]](s)


def _exact_router(s):
    l, k = s["logits"].double(), s["k"]
    t, e = l.shape
    live = torch.isfinite(l).any(1)
    if s["mask"] is not None:
        live &= s["mask"]
    n = int(live.sum())
    p = torch.softmax(l, 1)
    p[~live] = 0
    # expert by expert in the order of the logits: how many stand before it
    work = l.clone()
    work[~live] = -math.inf
    rows = torch.arange(t, device="cuda")
    experts = torch.full((t, k), -1, dtype=torch.int64, device="cuda")
    index = torch.arange(e, device="cuda")
    for j in range(k):
        best = work.max(1).values
        first = torch.where(work == best[:, None], index, e).min(1).values
        experts[:, j] = torch.where(best > -math.inf, first, -1)
        work[rows, first] = -math.inf
    chosen = experts >= 0
    at = experts.clamp(min=0)
    raw = torch.where(chosen, p.gather(1, at), 0.0)
    total = raw.sum(1, keepdim=True).clamp(min=1e-300) if s["normalize"] else torch.ones((t, 1), device="cuda").double()
    w = raw / total
    counts = torch.bincount(experts[chosen], minlength=e)
    sums = p.sum(0)
    out = [experts.int(), w, counts.int(), sums, torch.tensor([n], dtype=torch.int32, device="cuda"),
           (counts.double() / (n * k) * (sums / n)).sum().view(1) * e if n else torch.zeros(1, device="cuda").double()]
    if not s["train"]:
        return out
    # through the chain rule: loss and weights to probabilities, probabilities to logits
    dw = torch.where(chosen, s["d_weights"].double(), 0.0)
    draw_ = (dw - (dw * w).sum(1, keepdim=True)) / total if s["normalize"] else dw
    dp = (s["d_loss"].double() * e * counts.double() / max(1, k * n * n)).repeat(t, 1)
    dp.scatter_add_(1, at, torch.where(chosen, draw_, 0.0))
    dl = p * (dp - (p * dp).sum(1, keepdim=True))
    return out + [dl]


def _exact_codes(x):
    """(q, scale) of rows in 8-bit integers; the scale is a float32 number by definition."""
    x = x.double()
    top = x.abs().max(1).values
    scale = (top / torch.full_like(top, 127)).float().double()
    inverse = x / torch.where(scale > 0, scale, 1.0)[:, None]
    low = torch.floor(inverse)
    part = inverse - low
    up = (part > 0.5) | ((part == 0.5) & (low % 2 == 1))
    return low + up, scale


def _exact_quantize(s):
    q, scale = _exact_codes(s["x"])
    return q.to(torch.int8), scale


def _exact_int8(s):
    t = s["ends"][-1]
    q, scale = _exact_codes(s["x"][:t])
    group = torch.bucketize(torch.arange(t, device="cuda"), s["offsets"][1:], right=True)
    y = torch.zeros((t, s["n"]), dtype=torch.float64, device="cuda")
    for g in torch.unique(group).tolist():
        rows = (group == g).nonzero()[:, 0]
        y[rows] = torch.mm(q[rows], s["w"][g].double().t()) * s["w_scales"][g].double()
    return y * scale[:, None]


def _exact_checkpoint(s):
    t, f = s["ends"][-1], s["hidden"]
    w = s["row_weights"][:t].double()[:, None] if s["weighted"] else 1.0
    silu = lambda v: v * torch.sigmoid(v)  # noqa: E731
    if not s["backward"]:
        h = s["h"][:t].double()
        y = silu(h[:, :f]) * h[:, f:] * w
        blocks = h.reshape(t, -1, 32)
        top = blocks.abs().amax(2)
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140)))
        byte = (e - 8 + 127).clamp(min=0)
        v = blocks * torch.exp2(127 - byte)[:, :, None]
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        return [y, (torch.round(v / step) * step).clamp(-448, 448).view(t, 2 * f), byte.to(torch.uint8)]
    scale = torch.exp2(s["scales"][:t].double() - 127)
    h = (s["data"][:t].view(torch.float8_e4m3fn).double().view(t, -1, 32) * scale[:, :, None]).view(t, 2 * f)
    g, u, dy = h[:, :f], h[:, f:], s["dy"][:t].double()
    sig = torch.sigmoid(g)
    dh = torch.empty_like(h)
    dh[:, :f] = dy * w * u * (sig + g * sig * (1 - sig))
    dh[:, f:] = dy * w * silu(g)
    return [dh, (dy * silu(g) * u).sum(1) if s["weighted"] else None, silu(g) * u * w if s["recompute"] else None]
