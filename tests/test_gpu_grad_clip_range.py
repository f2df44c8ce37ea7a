"""Norms and factors outside of float32's normal range.  Tolerances as in test_gpu_grad_clip."""

import math

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device
from test_gpu_grad_clip import _clipped_ok, _norm, _tensors

pytestmark = pytest.mark.gpu


def test_norm_past_float32_is_flagged():
    """The sum of squares is finite in 64 bits, but the norm that a float32 can hold is not."""
    dev = device()
    t = torch.full((100,), 3e38, device=dev)
    other = torch.full((9,), 2.0, dtype=torch.bfloat16, device=dev)
    plan = bsg.grad_clip_plan([t, other], [torch.zeros_like(t), torch.zeros_like(other)])
    for call in (lambda s: bsg.grad_norm(plan, status=s), lambda s: bsg.clip_grad_norm(plan, 1e38, status=s)):
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        assert math.isinf(float(call(status)))
        assert int(status) == bsg.DEV_NONFINITE
    # the factor comes from the 64-bit norm: the clipped gradients are the formula's
    _clipped_ok(plan.outs, plan.tensors, 1e38 / (_norm([t, other]) + 1e-6))


@pytest.mark.parametrize("max_norm", [1.0, 1e-3, 1e-7])
def test_factor_under_float32s_normal_numbers(max_norm):
    gen = torch.Generator().manual_seed(4)
    ts = _tensors(gen, [(5000, torch.float32), (777, torch.bfloat16), (3, torch.float32)], std=1e37)
    outs = [torch.zeros_like(t) for t in ts]
    want = _norm(ts)
    norm = bsg.clip_grad_norm(bsg.grad_clip_plan(ts, outs), max_norm)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want or want > 3.4e38
    _clipped_ok(outs, ts, max_norm / (want + 1e-6))
