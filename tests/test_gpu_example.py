"""examples/adapted_experts.py: its training steps against the same steps in 64 bits, and its serving step
against the formula."""

import importlib.util
import os

import pytest
import torch

from gpu_util import device

pytestmark = pytest.mark.gpu

F64 = torch.float64


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapted_experts.py")
    spec = importlib.util.spec_from_file_location("adapted_experts", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_training_lowers_the_loss():
    device()
    losses, norms = _example().train(steps=12)
    assert losses[-1] < 0.7 * losses[0] and all(n > 0 for n in norms)


def test_gradients_of_a_micro_batch():
    """Main gradients against autograd in 64 bits over the same bf16 weights.  h, dy and dh are rounded to bf16
    (half a step each, 2^-8), which bounds each gradient by a few half steps of the sum of its magnitudes."""
    ex = _example()
    dev = device()
    gen = torch.Generator(device=dev).manual_seed(5)
    model = ex.Experts(4, 64, 128, dev)
    router = torch.randn((64, 4), generator=gen, device=dev)
    x, offsets = ex.route(torch.randn((300, 64), generator=gen, device=dev).to(torch.bfloat16), router, 4)
    target = torch.randn((300, 64), generator=gen, device=dev)
    loss = model.micro_batch(x, target, offsets, 300)
    o = offsets.tolist()
    half = 2.0 ** -8
    total = 0.0
    for g in range(4):
        rows = slice(o[g], o[g + 1])
        w1 = model.master[0][g].to(torch.bfloat16).to(F64).cpu()
        w2 = model.master[1][g].to(torch.bfloat16).to(F64).cpu()
        xs, ts = x[rows].to(F64).cpu(), target[rows].to(F64).cpu()
        pre = xs @ w1.T
        h = pre.relu()
        diff = h @ w2.T - ts
        total += float(diff.square().sum()) / 300
        dy = diff * (2.0 / 300)
        dh = (dy @ w2) * (pre > 0)
        # a value of h is off by half a step; what comes of it in diff is off by the sum over the row, and
        # dy adds a half step of its own
        herr = half * h.abs()
        dyerr = (herr @ w2.abs().T) * (2.0 / 300) + half * dy.abs()
        dherr = dyerr @ w2.abs() + half * (dy @ w2).abs()
        # values next to zero may fall on the other side of the ramp
        edge = (pre.abs() <= half * (xs.abs() @ w1.abs().T)) * (dy.abs() @ w2.abs())
        b2 = dyerr.T @ (h + herr) + dy.abs().T @ herr
        b1 = (dherr + edge).T @ xs.abs()
        for got, want, bound in ((model.main_grads[1][g], dy.T @ h, b2), (model.main_grads[0][g], dh.T @ xs, b1)):
            err = (got.to(F64).cpu() - want).abs()
            assert bool((err <= 1.01 * bound + 1e-6 * want.abs().max()).all()), float((err / bound).max())
    # diff is off by half a step of h's terms: the loss by no more than a few half steps of it
    assert abs(float(loss) - total) <= 5 * half * total


def test_serving_step():
    ex = _example()
    device()
    lengths, ids = (37, 1, 1, 120, 1), (0, 2, -1, 1, 2)
    y, (x, w, A, B, scale) = ex.serve(lengths, ids)
    x, w, A, B, scale = (t.to(F64).cpu() for t in (x, w, A, B, scale))
    at = 0
    for n, a in zip(lengths, ids):
        rows = slice(at, at + n)
        ref, mag = x[rows] @ w.T, x[rows].abs() @ w.abs().T
        if a >= 0:
            ref = ref + scale[a] * (x[rows] @ A[a].T) @ B[a].T
            mag = mag + scale[a] * (x[rows].abs() @ A[a].abs().T) @ B[a].abs().T
        # the output's rounding, and 512 + 16 steps of 2^-23 and the two halves' 2^-16 of the magnitudes
        err = (y[rows].to(F64).cpu() - ref).abs()
        assert bool((err <= 2.0 ** -8 * ref.abs() + 2.0 ** -13 * mag).all())
        at += n
