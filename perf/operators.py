"""Measured cases of the 16-bit operators: products grouped by expert, adapters of many
requests beside a shared projection, and the clipping of gradients by their global norm.

listed() names the cases, draw(rng) gives another of the same ranges, prepare(case, seed)
makes what a program holds before the call, run(state) is one pass through an operator,
exact(case, seed) the same outputs in 64 bits, and work(case) the bytes and operations that
a pass cannot do without.  With `own` false run() computes the operators from elementary
torch operations in 32 bits; with `own` true it calls the library.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "f32": 4}


def listed():
    return [
        # The smallest routed batch: 128 tokens over four small experts, one of them empty.  Latency.
        {"name": "experts-small", "op": "experts", "mode": "fprop", "dtype": "bf16", "groups": 4,
         "tokens": 128, "n": 128, "k": 128, "skew": "even", "empty": 1, "dead": 0, "gap": 0, "main": False},
        # One decoding step: 96 routed rows over 64 experts, some without a row.  The weights' bytes.
        {"name": "experts-decode", "op": "experts", "mode": "fprop", "dtype": "bf16", "groups": 64,
         "tokens": 96, "n": 2048, "k": 7168, "skew": "zipf", "empty": 4, "dead": 32, "gap": 0, "main": False},
        # Forward of eight large experts in training.
        {"name": "experts-forward", "op": "experts", "mode": "fprop", "dtype": "bf16", "groups": 8,
         "tokens": 16384, "n": 14336, "k": 4096, "skew": "dirichlet", "empty": 0, "dead": 0, "gap": 0, "main": False},
        # Forward of many small experts with very uneven loads, odd sizes, capacity rows unused.
        {"name": "experts-forward-zipf", "op": "experts", "mode": "fprop", "dtype": "fp16", "groups": 64,
         "tokens": 32768, "n": 2048, "k": 7168, "skew": "zipf", "empty": 4, "dead": 1000, "gap": 0, "main": False},
        # Data gradient of the eight large experts.
        {"name": "experts-data-gradient", "op": "experts", "mode": "dgrad", "dtype": "bf16", "groups": 8,
         "tokens": 16384, "n": 4096, "k": 14336, "skew": "dirichlet", "empty": 0, "dead": 0, "gap": 0, "main": False},
        # Weight gradients added to 32-bit main gradients, two experts without tokens.
        {"name": "experts-weight-gradient", "op": "experts", "mode": "wgrad", "dtype": "bf16", "groups": 8,
         "tokens": 16384, "n": 4096, "k": 4096, "skew": "dirichlet", "empty": 2, "dead": 0, "gap": 0, "main": True},
        # One request decoding one token through an adapted projection.
        {"name": "adapters-one-token", "op": "adapters", "dtype": "bf16", "requests": 1, "tokens": 1,
         "n": 4096, "k": 4096, "rank": 16, "adapters": 4, "bare": 0, "dead": 0},
        # A decoding step of 48 requests with 16 adapters among them, six requests without one.
        {"name": "adapters-decode", "op": "adapters", "dtype": "fp16", "requests": 48, "tokens": 48,
         "n": 14336, "k": 4096, "rank": 32, "adapters": 16, "bare": 6, "dead": 16},
        # The prompts of 24 requests of different lengths, some without an adapter.
        {"name": "adapters-prompts", "op": "adapters", "dtype": "bf16", "requests": 24, "tokens": 6000,
         "n": 4096, "k": 4096, "rank": 64, "adapters": 12, "bare": 4, "dead": 144},
        # Four hundred small tensors of odd sizes (biases, norms, adapters).  Latency.
        {"name": "clip-many-small", "op": "clip", "dtype": "mixed", "tensors": 400, "elements": 1 << 20,
         "max_norm": 1.0},
        # 16-bit gradients of a model of a few hundred tensors.
        {"name": "clip-bf16", "op": "clip", "dtype": "bf16", "tensors": 300, "elements": 200_000_000,
         "max_norm": 1.0},
        # 32-bit main gradients of a few stacks of experts.
        {"name": "clip-main-gradients", "op": "clip", "dtype": "f32", "tensors": 4, "elements": 1 << 29,
         "max_norm": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["experts", "experts", "adapters", "clip"])
    if op == "experts":
        while True:
            groups = _log(rng, 1, 128)
            case = {"op": op, "mode": rng.choice(["fprop", "dgrad", "wgrad"]), "dtype": rng.choice(["bf16", "fp16"]),
                    "groups": groups, "tokens": _log(rng, 1, 32768), "n": 8 * _log(rng, 8, 1792),
                    "k": 8 * _log(rng, 8, 1792), "skew": rng.choice(["even", "dirichlet", "zipf"]),
                    "empty": rng.randrange(groups // 4 + 1), "dead": rng.choice([0, 0, _log(rng, 1, 500)]),
                    "gap": rng.choice([0, 0, 8, 120]), "main": False}
            case["main"] = case["mode"] == "wgrad" and rng.random() < 0.5
            w = work(case)
            if w["flops"] <= 1.9e12 and w["bytes"] <= 2.0e9 and groups * case["n"] * case["k"] <= 1e9:
                return case
    if op == "adapters":
        while True:
            requests = _log(rng, 1, 200)
            adapters = _log(rng, 1, 64)
            case = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "requests": requests,
                    "tokens": max(requests, _log(rng, 1, 8192)), "n": 8 * _log(rng, 16, 1792),
                    "k": 8 * _log(rng, 16, 1792), "rank": rng.choice([8, 16, 24, 32, 64, 128]),
                    "adapters": adapters, "bare": rng.randrange(requests // 3 + 1),
                    "dead": rng.choice([0, 0, _log(rng, 1, 500)])}
            if work(case)["flops"] <= 1.0e12:
                return case
    return {"op": op, "dtype": rng.choice(["bf16", "fp16", "f32", "mixed"]), "tensors": _log(rng, 1, 600),
            "elements": _log(rng, 1 << 12, 1 << 28), "max_norm": rng.choice([1.0, 0.3, 1e9])}


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


def _request_lengths(rng, requests, tokens):
    """Every request has a row; the rest are drawn with uneven weights."""
    extra = _counts(rng, requests, tokens - requests, "dirichlet", 0)
    return [1 + e for e in extra]


def _request_adapters(rng, requests, adapters, bare):
    ids = [rng.randrange(adapters) for _ in range(requests)]
    for g in rng.sample(range(requests), bare):
        ids[g] = -1
    return ids


def _tensor_sizes(rng, tensors, elements):
    p = [rng.gammavariate(0.5, 1.0) + 1e-3 for _ in range(tensors)]
    total = sum(p)
    return [max(1, int(elements * q / total)) for q in p]


def _expert_shapes(case):
    """(columns of the ragged operand a, shape of b's second operand) of a mode."""
    n, k = case["n"], case["k"]
    return {"fprop": (k, n, k), "dgrad": (k, k, n), "wgrad": (n, k, None)}[case["mode"]]


def work(case):
    rng = _case_rng(case)
    if case["op"] == "experts":
        counts = _counts(rng, case["groups"], case["tokens"], case["skew"], case["empty"])
        t, n, k = sum(counts), case["n"], case["k"]
        active = sum(c > 0 for c in counts)
        if case["mode"] == "wgrad":
            out = case["groups"] * n * k * (8 if case["main"] else 2)  # main gradients are read and written
            return {"bytes": 2 * t * (n + k) + out, "flops": 2 * t * n * k}
        return {"bytes": 2 * (t * (n + k) + active * n * k), "flops": 2 * t * n * k}
    if case["op"] == "adapters":
        lengths = _request_lengths(rng, case["requests"], case["tokens"])
        ids = _request_adapters(rng, case["requests"], case["adapters"], case["bare"])
        n, k, r, t = case["n"], case["k"], case["rank"], case["tokens"]
        used = len({i for i in ids if i >= 0})
        adapted = sum(c for c, i in zip(lengths, ids) if i >= 0)
        return {"bytes": 2 * (t * (n + k) + n * k + used * r * (n + k)),
                "flops": 2 * t * n * k + 2 * adapted * r * (n + k)}
    sizes = _tensor_sizes(rng, case["tensors"], case["elements"])
    total = sum(s * SIZE[d] for s, d in zip(sizes, _clip_dtypes(case, len(sizes))))
    return {"bytes": 2 * total, "flops": 3 * sum(sizes)}


def _clip_dtypes(case, tensors):
    if case["dtype"] != "mixed":
        return [case["dtype"]] * tensors
    return ["f32" if i < tensors // 3 else "bf16" for i in range(tensors)]


# ---------------------------------------------------------------- inputs


def _normal(gen, shape, dtype, std=1.0, outliers=0.0, gap=0):
    """Normal values rounded to `dtype`, a share of them 20 times as large; with `gap` the rows
    of a wider buffer's first columns."""
    out = torch.empty(shape[:-1] + (shape[-1] + gap,), dtype=dtype, device="cuda")[..., : shape[-1]]
    rows = out.reshape(-1, shape[-1]) if not gap else out.view(-1, shape[-1])
    step = max(1, (1 << 26) // shape[-1])
    for r in range(0, rows.shape[0], step):
        m = min(step, rows.shape[0] - r)
        v = torch.randn((m, shape[-1]), generator=gen, device="cuda") * std
        if outliers:
            v = torch.where(torch.rand((m, shape[-1]), generator=gen, device="cuda") < outliers, v * 20, v)
        rows[r:r + m] = v.to(dtype)
    return out


def _offsets(counts):
    ends = [0]
    for c in counts:
        ends.append(ends[-1] + c)
    return ends


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = _case_rng(case)
    s = dict(case)
    if own:
        import block_scaled_grouped_amd as bsg
        s["bsg"] = bsg
    if case["op"] == "experts":
        dt = DTYPES[case["dtype"]]
        counts = _counts(rng, case["groups"], case["tokens"], case["skew"], case["empty"])
        s["ends"] = _offsets(counts)
        s["offsets"] = torch.tensor(s["ends"], dtype=torch.int64, device="cuda")
        cap = s["ends"][-1] + case["dead"]
        acols, brows, bcols = _expert_shapes(case)
        if case["mode"] == "fprop":
            s["a"] = _normal(gen, (cap, acols), dt, outliers=0.01, gap=case["gap"])
        else:
            s["a"] = _normal(gen, (cap, acols), dt, std=0.1, gap=case["gap"])
        if case["mode"] == "wgrad":
            s["b"] = _normal(gen, (cap, brows), dt, outliers=0.01)
            if case["main"]:
                s["c"] = _normal(gen, (case["groups"], case["n"], case["k"]), torch.float32)
        else:
            s["b"] = _normal(gen, (case["groups"], brows, bcols), dt, std=0.02)
        s["a"][s["ends"][-1]:] = float("nan")  # capacity rows that no group owns
        if case["mode"] == "wgrad":
            s["b"][s["ends"][-1]:] = float("nan")
        if own:
            s["workspace"] = s["bsg"].gemm_workspace()
    elif case["op"] == "adapters":
        dt = DTYPES[case["dtype"]]
        n, k, r = case["n"], case["k"], case["rank"]
        lengths = _request_lengths(rng, case["requests"], case["tokens"])
        ids = _request_adapters(rng, case["requests"], case["adapters"], case["bare"])
        s["ends"], s["ids"] = _offsets(lengths), ids
        s["offsets"] = torch.tensor(s["ends"], dtype=torch.int64, device="cuda")
        s["adapter"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
        s["x"] = _normal(gen, (case["tokens"] + case["dead"], k), dt, outliers=0.01)
        s["x"][case["tokens"]:] = float("nan")
        s["w"] = _normal(gen, (n, k), dt, std=0.02)
        s["lora_a"] = _normal(gen, (case["adapters"], r, k), dt, std=k ** -0.5)
        s["lora_b"] = _normal(gen, (case["adapters"], n, r), dt, std=0.02)
        s["scale"] = torch.rand(case["adapters"], generator=gen, device="cuda") * 1.5 + 0.5
        if own:
            s["workspace"] = s["bsg"].grouped_lora_gemm_16bit_workspace(s["x"].shape[0], n, k, r)
    else:
        sizes = _tensor_sizes(rng, case["tensors"], case["elements"])
        kinds = _clip_dtypes(case, len(sizes))
        spread = [10.0 ** rng.uniform(-4, 0) for _ in sizes]  # layers' gradients differ in scale
        s["flat"], s["out"], grads, outs = [], [], [], []
        for kind in sorted(set(kinds)):  # one bucket for each type, as data-parallel training keeps them
            mine = [(n, std) for n, q, std in zip(sizes, kinds, spread) if q == kind]
            flat = torch.empty(sum(n for n, _ in mine), dtype=DTYPES[kind], device="cuda")
            out = torch.empty_like(flat)
            at = 0
            for n, std in mine:
                grads.append(flat[at:at + n])
                outs.append(out[at:at + n])
                at += n
                for p in range(0, n, 1 << 27):
                    q = grads[-1][p:p + (1 << 27)]
                    q.copy_(torch.randn(q.shape, generator=gen, device="cuda") * std)
            s["flat"].append(flat)
            s["out"].append(out)
        if own:
            s["plan"] = s["bsg"].grad_clip_plan(grads, outs)
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    if own:
        return _run_own(s)
    return {"experts": _plain_experts, "adapters": _plain_adapters, "clip": _plain_clip}[s["op"]](s)


def _run_own(s):
    bsg = s["bsg"]
    if s["op"] == "experts":
        mode = {"fprop": bsg.BSG_FPROP_TN, "dgrad": bsg.BSG_DGRAD_NN, "wgrad": bsg.BSG_WGRAD_NT}[s["mode"]]
        y = bsg.grouped_gemm_16bit(mode, s["a"], s["b"], s["offsets"], c=s.get("c"), workspace=s["workspace"])
        return y if s["mode"] == "wgrad" else y[: s["ends"][-1]]
    if s["op"] == "adapters":
        y = bsg.grouped_lora_gemm_16bit(s["x"], s["w"], s["lora_a"], s["lora_b"], s["offsets"], s["adapter"],
                                        s["scale"], workspace=s["workspace"])
        return y[: s["tokens"]]
    return [bsg.clip_grad_norm(s["plan"], s["max_norm"])] + s["out"]


def _plain_experts(s):
    """Each expert's rows times its weights (fprop a b^T, dgrad a b, wgrad a^T b)."""
    a, b, ends, dt = s["a"], s["b"], s["ends"], s["a"].dtype
    if s["mode"] == "wgrad":
        c = s.get("c")
        out = torch.zeros((s["groups"], s["n"], s["k"]), dtype=dt, device="cuda") if c is None else c.clone()
        for g in range(s["groups"]):
            lo, hi = ends[g], ends[g + 1]
            if hi > lo:
                product = a[lo:hi].float().T @ b[lo:hi].float()
                out[g] = product.to(dt) if c is None else c[g] + product
        return out
    out = torch.empty((ends[-1], s["n"]), dtype=dt, device="cuda")
    for g in range(s["groups"]):
        lo, hi = ends[g], ends[g + 1]
        if hi > lo:
            w = b[g].float()
            out[lo:hi] = (a[lo:hi].float() @ (w.T if s["mode"] == "fprop" else w)).to(dt)
    return out


def _plain_adapters(s):
    """x w^T plus, in the columns of each row's own adapter only, scale (x A^T) B^T."""
    t, r, count = s["tokens"], s["rank"], s["adapters"]
    x = s["x"][:t].float()
    rows = torch.arange(t, device="cuda")
    request = (rows[:, None] >= s["offsets"][None, 1:]).sum(1)
    mine = s["adapter"][request][:, None] == torch.arange(count, device="cuda")[None, :]
    low = x @ s["lora_a"].float().reshape(count * r, -1).T
    low = low.view(t, count, r) * (mine * s["scale"][None, :])[:, :, None]
    up = s["lora_b"].float().permute(0, 2, 1).reshape(count * r, -1)
    return (x @ s["w"].float().T + low.view(t, count * r) @ up).to(s["x"].dtype)


def _plain_clip(s):
    """The norm over all tensors (long sums: in 64 bits), and the tensors times min(1, max_norm / (norm + 1e-6))."""
    norm = torch.stack([f.double().square().sum() for f in s["flat"]]).sum().sqrt()
    factor = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    return [norm.float()] + [(f.float() * factor).to(f.dtype) for f in s["flat"]]


# ---------------------------------------------------------------- in 64 bits


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "experts":
        t = s["ends"][-1]
        group = torch.bucketize(torch.arange(t, device="cuda"), s["offsets"][1:], right=True)
        a = s["a"][:t].double()
        if case["mode"] == "wgrad":
            out = s["c"].double() if "c" in s else torch.zeros(
                (case["groups"], case["n"], case["k"]), dtype=torch.float64, device="cuda")
            b = s["b"][:t].double()
            for g in torch.unique(group).tolist():
                rows = (group == g).nonzero()[:, 0]
                out[g].addmm_(a[rows].t().contiguous(), b[rows])
            return out
        out = torch.zeros((t, case["n"]), dtype=torch.float64, device="cuda")
        for g in torch.unique(group).tolist():
            rows = (group == g).nonzero()[:, 0]
            w = s["b"][g].double()
            out[rows] = torch.mm(a[rows], w.t() if case["mode"] == "fprop" else w)
        return out
    if case["op"] == "adapters":
        x = s["x"][: case["tokens"]].double()
        out = torch.mm(x, s["w"].double().t())
        for q, adapter in enumerate(s["ids"]):
            if adapter >= 0:
                rows = slice(s["ends"][q], s["ends"][q + 1])
                low = torch.mm(x[rows], s["lora_a"][adapter].double().t())
                out[rows] += s["scale"][adapter].double() * torch.mm(low, s["lora_b"][adapter].double().t())
        return out
    squares = sum(torch.dot(p, p).item() for f in s["flat"] for q in f.split(1 << 26) for p in [q.double()])
    norm = math.sqrt(squares)
    factor = min(1.0, case["max_norm"] / (norm + 1e-6))
    return [torch.tensor(norm, dtype=torch.float64, device="cuda")] + [f.double() * factor for f in s["flat"]]
