"""moe_router_topk and its backward pass against the formulas in 64 bits.

Tolerances.  A probability is exp(x) / sum with x = l - max rounded once (2^-24 |x| absolute, so that relative
in exp(x)), exp to two steps of 2^-23, a sum of at most 16 + 4 additions, a reciprocal and a product: off by at
most (|x| + 40) 2^-23 of itself, and by 2^-126 where it underflows.  Weights add one sum and one quotient.  Sums
over tokens add at most 4 + 16 + 2 additions in float32 and one rounding.  The gradient's terms are sums and
products of those: 100 + max|x| steps of the sum of their magnitudes, and one rounding to the output's type."""

import math

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device

pytestmark = pytest.mark.gpu

F64 = torch.float64
STEP = 2.0 ** -23
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
SHAPES = [(1, 1, 1), (1, 8, 2), (5, 3, 3), (64, 8, 2), (256, 16, 16), (257, 16, 4), (300, 17, 5), (1000, 64, 6),
          (70, 100, 8), (129, 128, 16), (513, 255, 16), (4097, 256, 8), (2000, 33, 1), (20011, 64, 8)]


def _logits(t, e, dtype, seed, gap=0, std=1.5, ties=False):
    gen = torch.Generator().manual_seed(seed)
    v = torch.randn((t, e), generator=gen) * std
    if ties:
        v = (v * 2).round() / 2
    wide = torch.full((t, e + gap), float("nan"), dtype=dtype)
    wide[:, :e] = v.to(dtype)
    return wide.to(device())[:, :e]


def _reference(logits, k, mask, normalize):
    l = logits.detach().cpu().to(F64)
    t, e = l.shape
    live = (l > -math.inf).any(1) if t else torch.zeros(0, dtype=torch.bool)
    if mask is not None:
        live = live & (mask.cpu() != 0)
    safe = torch.where(live[:, None], l, 0.0)
    x = safe - safe.amax(1, keepdim=True) if t else safe
    p = torch.exp(x) / torch.exp(x).sum(1, keepdim=True) * live[:, None]
    order = torch.sort(l, dim=1, descending=True, stable=True)
    chosen = live[:, None] & (order.values[:, :k] > -math.inf)
    experts = torch.where(chosen, order.indices[:, :k], -1)
    at = experts.clamp(min=0)
    w = torch.where(chosen, p.gather(1, at), 0.0)
    if normalize:
        w = torch.where(chosen, w / w.sum(1, keepdim=True).clamp(min=1e-300), 0.0)
    counts = torch.bincount(experts[chosen], minlength=e)
    n = int(live.sum())
    sums = p.sum(0)
    loss = float((counts * sums).sum()) * e / (k * n * n) if n else 0.0
    return dict(experts=experts, weights=w, counts=counts, prob_sums=sums, live=n, loss=loss, p=p, x=x,
                alive=live, at=at, chosen=chosen)


def _check_forward(r, ref):
    assert torch.equal(r["experts"].cpu().long(), ref["experts"])
    assert torch.equal(r["counts"].cpu().long(), ref["counts"])
    assert int(r["live"]) == ref["live"]
    x = ref["x"].gather(1, ref["at"]).abs() if ref["at"].numel() else ref["weights"]
    tol = (x + 60) * STEP * ref["weights"].abs() + 2.0 ** -126
    assert bool(((r["weights"].cpu().to(F64) - ref["weights"]).abs() <= tol).all())
    big = float(ref["x"].abs().clamp(max=110).max()) if ref["x"].numel() else 0.0
    stol = (min(big, 20) + 80) * STEP * ref["prob_sums"] + 2.0 ** -100
    assert bool(((r["prob_sums"].cpu().to(F64) - ref["prob_sums"]).abs() <= stol).all())
    assert abs(float(r["loss"]) - ref["loss"]) <= (min(big, 20) + 90) * STEP * ref["loss"]


def _reference_backward(ref, e, k, dw, dl, normalize):
    """(gradient, sum of the magnitudes of its terms)"""
    p, at, chosen, n = ref["p"], ref["at"], ref["chosen"], ref["live"]
    b = (dl * e / (k * n * n) * ref["counts"].to(F64)).expand_as(p) if n else torch.zeros_like(p)
    g = torch.where(chosen, dw, 0.0)
    zero = torch.zeros_like(p)
    if normalize:
        w = ref["weights"]
        own = zero.scatter_add(1, at, torch.where(chosen, w * (g - (w * g).sum(1, keepdim=True)), 0.0))
        mag = zero.scatter_add(1, at, torch.where(chosen, w * (g.abs() + (w * g.abs()).sum(1, keepdim=True)), 0.0))
        d = p * (b - (p * b).sum(1, keepdim=True)) + own
        mag = mag + p * (b.abs() + (p * b.abs()).sum(1, keepdim=True))
    else:
        a = b + zero.scatter_add(1, at, g)
        m = b.abs() + zero.scatter_add(1, at, g.abs())
        d = p * (a - (p * a).sum(1, keepdim=True))
        mag = p * (m + (p * m).sum(1, keepdim=True))
    return d * ref["alive"][:, None], mag


def _check_backward(d, ref, e, k, dw, dl, normalize):
    want, mag = _reference_backward(ref, e, k, dw, dl, normalize)
    big = float(ref["x"].abs().clamp(max=110).max()) if ref["x"].numel() else 0.0
    acc = (big + 100) * STEP * mag + 2.0 ** -120
    tiny = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}[d.dtype]
    tol = torch.finfo(d.dtype).eps / 2 * (want.abs() + acc) + acc + tiny
    err = (d.cpu().to(F64) - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,e,k", SHAPES)
def test_router(dtype, t, e, k):
    for seed, (normalize, gap, ties) in enumerate([(True, 0, False), (False, 3, True)]):
        logits = _logits(t, e, dtype, 10 * t + e + seed, gap, ties=ties)
        mask = None
        if seed:
            mask = torch.rand(t, generator=torch.Generator().manual_seed(t)).gt(0.2).to(device())
        r = bsg.moe_router_topk(logits, k, mask=mask, normalize=normalize)
        ref = _reference(logits, k, mask, normalize)
        _check_forward(r, ref)
        gen = torch.Generator().manual_seed(e)
        dw = torch.randn((t, k), generator=gen)
        dl = 0.37
        d = bsg.moe_router_topk_backward(logits, r["experts"], r["counts"], r["live"], d_weights=dw.to(device()),
                                         d_loss=torch.full((1,), dl, device=device()), mask=mask,
                                         normalize=normalize)
        assert d.dtype == dtype
        _check_backward(d, ref, e, k, dw.to(F64), float(torch.tensor(dl)), normalize)


@pytest.mark.parametrize("normalize", [False, True])
def test_closed_experts_and_tokens_without_one(normalize):
    """Experts at -inf, tokens whose logits are all -inf, fewer open experts than slots, and masked tokens that
    hold NaN: the latter are not read."""
    t, e, k = 700, 40, 8
    logits = _logits(t, e, torch.float32, 3)
    logits[:, 5:9] = -math.inf
    logits[::7] = -math.inf
    logits[3::7, 4:] = -math.inf          # four open experts for eight slots
    mask = torch.ones(t, dtype=torch.uint8, device=device())
    mask[5::11] = 0
    clean = logits.clone()
    logits[5::11] = math.nan
    clean[5::11] = 0
    status = torch.zeros(1, dtype=torch.int32, device=device())
    r = bsg.moe_router_topk(logits, k, mask=mask, normalize=normalize, status=status)
    ref = _reference(clean, k, mask, normalize)
    _check_forward(r, ref)
    assert int(status) == 0 and bool((r["experts"] == -1).any())
    dw = torch.randn((t, k), generator=torch.Generator().manual_seed(0))
    dw[ref["experts"] < 0] = math.nan     # of slots without an expert: not read
    d = bsg.moe_router_topk_backward(logits, r["experts"], r["counts"], r["live"], d_weights=dw.to(device()),
                                     d_loss=torch.ones(1, device=device()), mask=mask, normalize=normalize)
    _check_backward(d, ref, e, k, dw.to(F64).nan_to_num(0.0), 1.0, normalize)


def test_nothing_is_live():
    for t in (0, 1, 300):
        logits = torch.full((t, 24), -math.inf, device=device())
        r = bsg.moe_router_topk(logits, 3)
        assert bool((r["experts"] == -1).all()) and bool((r["weights"] == 0).all())
        assert int(r["counts"].sum()) == 0 and int(r["live"]) == 0 and float(r["loss"]) == 0.0
        assert bool((r["prob_sums"] == 0).all())
        d = bsg.moe_router_topk_backward(logits, r["experts"], r["counts"], r["live"],
                                         d_weights=torch.ones((t, 3), device=device()),
                                         d_loss=torch.ones(1, device=device()))
        assert d.shape == (t, 24) and bool((d == 0).all())


@pytest.mark.parametrize("e,k", [(8, 8), (64, 6), (256, 16)])
def test_equal_and_nearly_equal_logits(e, k):
    """float32 logits that differ in their last bits, or not at all, and zeros of both signs: descending order,
    ties to the lowest index."""
    gen = torch.Generator().manual_seed(e)
    base = torch.randint(0, 6, (500, e), generator=gen).float() - 3.0
    near = base + torch.randint(-3, 4, (500, e), generator=gen) * 2.0 ** -22
    signed = torch.where(torch.rand((500, e), generator=gen) < 0.5, -0.0, 0.0)
    for v in (base, near, signed, torch.cat([near[:3], base[:1], near[3:]])):
        logits = v.to(device())
        r = bsg.moe_router_topk(logits, k, normalize=False)
        _check_forward(r, _reference(logits, k, None, False))


def test_values_that_are_not_finite():
    """A NaN or +inf makes its own token's probabilities NaN, as the formula has it, and sets the status bit; a
    NaN is never chosen."""
    for t in (20, 400):
        logits = _logits(t, 12, torch.float32, 1)
        logits[7, 3] = math.nan
        logits[9, 2] = math.inf
        logits[11] = math.nan
        status = torch.zeros(1, dtype=torch.int32, device=device())
        r = bsg.moe_router_topk(logits, 4, status=status)
        assert int(status) == bsg.DEV_NONFINITE
        assert bool((r["experts"][7] != 3).all()) and int(r["experts"][9, 0]) == 2
        assert bool((r["experts"][11] == -1).all())
        w = r["weights"].cpu()
        assert bool(w[7].isnan().all()) and bool(w[9].isnan().all()) and bool((w[11] == 0).all())
        fine = torch.ones(t, dtype=torch.bool)
        fine[[7, 9, 11]] = False
        assert bool(w[fine].isfinite().all()) and bool(r["prob_sums"].isnan().all()) and bool(r["loss"].isnan())
        d = bsg.moe_router_topk_backward(logits, r["experts"], r["counts"], r["live"],
                                         d_weights=torch.ones((t, 4), device=device()))
        assert bool(d.cpu()[fine].isfinite().all()) and bool(d[7].isnan().any())


def test_backward_of_parts():
    """Either gradient alone; counts and live tokens added up over two micro-batches."""
    a, b = _logits(300, 16, torch.float32, 5), _logits(200, 16, torch.float32, 6)
    ra, rb = bsg.moe_router_topk(a, 2), bsg.moe_router_topk(b, 2)
    both = bsg.moe_router_topk(torch.cat([a, b]), 2)
    counts, live = ra["counts"] + rb["counts"], ra["live"] + rb["live"]
    assert torch.equal(counts, both["counts"]) and torch.equal(live, both["live"])
    dl = torch.full((1,), 0.5, device=device())
    got = torch.cat([bsg.moe_router_topk_backward(x, r["experts"], counts, live, d_loss=dl)
                     for x, r in ((a, ra), (b, rb))])
    want = bsg.moe_router_topk_backward(torch.cat([a, b]), both["experts"], both["counts"], both["live"], d_loss=dl)
    assert torch.equal(got, want) and bool((got != 0).any())
    dw = torch.randn((300, 2), device=device())
    only = bsg.moe_router_topk_backward(a, ra["experts"], ra["counts"], ra["live"], d_weights=dw)
    zero = bsg.moe_router_topk_backward(a, ra["experts"], ra["counts"], ra["live"], d_weights=dw,
                                        d_loss=torch.zeros(1, device=device()))
    assert torch.equal(only, zero)
    none = bsg.moe_router_topk_backward(a, ra["experts"], ra["counts"], ra["live"])
    assert bool((none == 0).all())


@pytest.mark.parametrize("normalize", [False, True])
def test_backward_against_differences(normalize):
    """Central differences, step 2^-10, of sum(dw w) + dl loss in 64 bits: their own error is a third derivative
    (at most the sum of the terms' magnitudes) times 2^-20 / 6."""
    t, e, k, h = 12, 9, 3, 2.0 ** -10
    logits = _logits(t, e, torch.float32, 8)
    r = bsg.moe_router_topk(logits, k, normalize=normalize)
    dw, dl = torch.randn((t, k), generator=torch.Generator().manual_seed(1)), 2.0
    d = bsg.moe_router_topk_backward(logits, r["experts"], r["counts"], r["live"], d_weights=dw.to(device()),
                                     d_loss=torch.full((1,), dl, device=device()), normalize=normalize).cpu().to(F64)
    experts, counts = r["experts"].cpu().long(), r["counts"].cpu().to(F64)

    def value(l):
        p = torch.softmax(l, -1)
        w = p.gather(-1, experts.expand(l.shape[:-1] + (k,)))
        if normalize:
            w = w / w.sum(-1, keepdim=True)
        return (w * dw.to(F64)).sum((-1, -2)) + dl * e / (k * t * t) * (p.sum(-2) * counts).sum(-1)

    l = logits.cpu().to(F64)
    eye = torch.eye(t * e, dtype=F64).view(t * e, t, e) * h
    diff = ((value(l + eye) - value(l - eye)) / (2 * h)).view(t, e)
    bound = (dw.abs().sum(1, keepdim=True).to(F64) * 8 + 8 * dl) * h * h + 1e-5 * dw.abs().max()
    assert bool(((d - diff).abs() <= bound).all())


def test_captured_and_on_two_streams():
    logits = [_logits(5000, 64, torch.bfloat16, s) for s in (1, 2)]
    dw = torch.randn((5000, 6), device=device())
    dl = torch.ones(1, device=device())

    def step(x, ws):
        r = bsg.moe_router_topk(x, 6, workspace=ws)
        return r, bsg.moe_router_topk_backward(x, r["experts"], r["counts"], r["live"], d_weights=dw, d_loss=dl)

    ws = [bsg.moe_router_topk_workspace(5000, 64) for _ in range(2)]
    want = [step(x, ws[0]) for x in logits]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for x, w, s in zip(logits, ws, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                out = step(x, w)
            got.append(out)
    torch.cuda.synchronize()
    for (ra, da), (rb, db) in zip(want, got):
        assert all(torch.equal(ra[n], rb[n]) for n in ra) and torch.equal(da, db)

    x = logits[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, d = step(x, ws[0])
    for i in (1, 0, 1):
        x.copy_(logits[i])
        graph.replay()
        step(logits[1 - i], ws[1])
        torch.cuda.synchronize()
        assert all(torch.equal(want[i][0][n], r[n]) for n in r) and torch.equal(want[i][1], d)


def test_outputs_and_refusals():
    logits = _logits(40, 10, torch.float16, 2)
    r = bsg.moe_router_topk(logits, 2)
    wide = torch.full((40, 13), 7.0, dtype=torch.float16, device=device())
    d = bsg.moe_router_topk_backward(logits, r["experts"], r["counts"], r["live"],
                                     d_loss=torch.ones(1, device=device()), out=wide[:, :10])
    assert d.data_ptr() == wide.data_ptr() and bool((wide[:, 10:] == 7).all())
    for bad in (dict(top_k=0), dict(top_k=11), dict(top_k=17)):
        with pytest.raises(bsg.BsgError):
            bsg.moe_router_topk(logits, **bad)
    with pytest.raises(ValueError, match="contiguous"):
        bsg.moe_router_topk(logits.t(), 2)
    with pytest.raises(ValueError, match="mask"):
        bsg.moe_router_topk(logits, 2, mask=torch.ones(40, device=device()))
    with pytest.raises(ValueError, match="mask"):
        bsg.moe_router_topk(logits, 2, mask=torch.ones(39, dtype=torch.bool, device=device()))
    with pytest.raises(bsg.BsgError):
        bsg.moe_router_topk(logits, 2, workspace=torch.empty(64, dtype=torch.uint8, device=device()))
    with pytest.raises(ValueError, match="d_weights"):
        bsg.moe_router_topk_backward(logits, r["experts"], r["counts"], r["live"],
                                     d_weights=torch.ones((40, 3), device=device()))
    with pytest.raises(ValueError, match="counts"):
        bsg.moe_router_topk_backward(logits, r["experts"], r["counts"][:5], r["live"])
