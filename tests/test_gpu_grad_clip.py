"""grad_norm and clip_grad_norm against the formulas in 64 bits.

Tolerances: the squares and their sum are 64-bit, so the norm is off by its rounding to float32 (2^-24) and
a few 2^-53; the factor is rounded to float32 once and each product once to float32 (2^-24 each) and once to
its tensor's type (half a step and half of the smallest subnormal)."""

import math

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device

pytestmark = pytest.mark.gpu

F64 = torch.float64
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
ALL = [torch.bfloat16, torch.float16, torch.float32]


def _tensors(gen, spec, shift=0, std=1.0):
    """Views into one buffer of a type at odd places (shift elements in); spec: (numel, dtype)."""
    dev = device()
    out = []
    for n, dt in spec:
        flat = torch.full((n + shift + 3,), float("nan"), dtype=dt, device=dev)
        flat[shift:shift + n] = (torch.randn(n, generator=gen) * std).to(dt).to(dev)
        out.append(flat[shift:shift + n])
    return out


def _norm(ts):
    return math.sqrt(sum(float((t.cpu().to(F64) ** 2).sum()) for t in ts))


def _clipped_ok(outs, ins, factor):
    for y, x in zip(outs, ins):
        ref = x.cpu().to(F64) * factor
        half = torch.finfo(y.dtype).eps / 2
        tol = (half + 3 * 2.0 ** -24) * ref.abs() + TINY[y.dtype]
        assert bool(((y.cpu().to(F64) - ref).abs() <= tol).all())


SPECS = [
    [(1, torch.float32)],
    [(7, torch.bfloat16)],
    [(0, torch.float32), (5, torch.float16), (0, torch.bfloat16)],
    [(16384, torch.float32), (16385, torch.bfloat16), (16383, torch.float16)],
    [(3 * 16384 + 11, torch.float32), (100003, torch.bfloat16), (1, torch.float16)],
    [(i % 97 + 1, ALL[i % 3]) for i in range(500)],
]


@pytest.mark.parametrize("shift", [0, 1, 5])
@pytest.mark.parametrize("spec", range(len(SPECS)))
def test_norm_and_clip(spec, shift):
    gen = torch.Generator().manual_seed(spec)
    ts = _tensors(gen, SPECS[spec], shift)
    outs = [torch.full((t.numel() + 2,), 9.0, dtype=t.dtype, device=t.device) for t in ts]
    plan = bsg.grad_clip_plan(ts, [o[1:-1] for o in outs])      # aligned otherwise than the inputs
    want = _norm(ts)
    sumsq = torch.zeros(1, dtype=F64, device=device())
    norm = bsg.grad_norm(plan, sumsq=sumsq)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    assert abs(float(sumsq) - want ** 2) <= 1e-12 * want ** 2
    for max_norm in (0.5 * want, 2.0 * want + 1.0, math.inf, 0.0):
        norm = bsg.clip_grad_norm(plan, max_norm)
        assert abs(float(norm) - want) <= 2.0 ** -23 * want
        factor = min(1.0, max_norm / (want + 1e-6))
        _clipped_ok([o[1:-1] for o in outs], ts, factor)
        for o in outs:
            assert float(o[0]) == 9.0 and float(o[-1]) == 9.0
    # the sum of squares from outside (a sharded model's), and the same result twice
    total = sumsq * 4
    bsg.clip_grad_norm(plan, 0.25 * want, sumsq=total)
    _clipped_ok([o[1:-1] for o in outs], ts, min(1.0, 0.25 * want / (2 * want + 1e-6)))
    assert torch.equal(bsg.grad_norm(plan), bsg.grad_norm(plan))


def test_in_place():
    gen = torch.Generator().manual_seed(1)
    ts = _tensors(gen, [(1000, torch.float32), (3001, torch.bfloat16), (17, torch.float16)], 1)
    before = [t.clone() for t in ts]
    plan = bsg.grad_clip_plan(ts)
    want = _norm(ts)
    bsg.clip_grad_norm(plan, want * 1.5)
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    norm = bsg.clip_grad_norm(plan, want / 3)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    _clipped_ok(ts, before, (want / 3) / (want + 1e-6))


@pytest.mark.parametrize("std", [1e-30, 1e25])
def test_squares_outside_of_float32(std):
    gen = torch.Generator().manual_seed(2)
    ts = _tensors(gen, [(5000, torch.float32), (777, torch.bfloat16)], std=std)
    plan = bsg.grad_clip_plan(ts)
    want = _norm(ts)
    assert abs(float(bsg.grad_norm(plan)) - want) <= 2.0 ** -23 * want


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_not_finite(value):
    dev = device()
    t = torch.ones(40000, device=dev)
    t[39999] = value
    other = torch.ones(10, dtype=torch.bfloat16, device=dev)
    plan = bsg.grad_clip_plan([other, t])
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    norm = bsg.clip_grad_norm(plan, 1.0, status=status)
    assert int(status) == bsg.DEV_NONFINITE
    if math.isnan(value):
        assert math.isnan(float(norm)) and bool(torch.isnan(t).all()) and bool(torch.isnan(other).all())
    else:
        assert math.isinf(float(norm)) and bool(torch.isnan(t[39999])) and bool((t[:39999] == 0).all())
        assert bool((other == 0).all())
    status.zero_()
    assert float(bsg.grad_norm(bsg.grad_clip_plan([torch.ones(4, device=dev)]), status=status)) == 2.0
    assert int(status) == 0


def test_no_tensors_and_graph():
    dev = device()
    assert float(bsg.clip_grad_norm(bsg.grad_clip_plan([]), 1.0)) == 0.0
    gen = torch.Generator().manual_seed(3)
    ts = _tensors(gen, [(70000, torch.float32), (33, torch.bfloat16)])
    outs = [torch.zeros_like(t) for t in ts]
    plan = bsg.grad_clip_plan(ts, outs)
    norm = torch.zeros((), device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bsg.clip_grad_norm(plan, 1.0, norm=norm)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsg.clip_grad_norm(plan, 1.0, norm=norm)
    for mul in (1.0, 3.0, 1e-4):
        for t in ts:
            t.mul_(mul)
        graph.replay()
        torch.cuda.synchronize()
        want = _norm(ts)
        assert abs(float(norm) - want) <= 2.0 ** -23 * want
        _clipped_ok(outs, ts, min(1.0, 1.0 / (want + 1e-6)))
        got = [o.clone() for o in outs]
        bsg.clip_grad_norm(plan, 1.0)
        assert all(torch.equal(a, b) for a, b in zip(got, outs))
