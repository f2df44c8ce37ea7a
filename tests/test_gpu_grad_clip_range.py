"""Norms and factors outside of float32's normal range.  Tolerances as in test_gpu_grad_clip."""

import math

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device
from test_gpu_grad_clip import _clipped_ok, _norm

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
