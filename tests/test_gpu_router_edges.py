"""Numbers of experts that are no whole runs of 16 bytes, with masked rows of NaN (the first among them), equal and
nearly equal logits, and tokens of infinities and NaN beside others that a wave takes together."""

import math

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device
from test_gpu_router import DTYPES, F64, _check_backward, _check_forward, _logits, _reference

pytestmark = pytest.mark.gpu

EXPERTS = [1, 2, 7, 16, 17, 30, 32, 63, 64, 65, 126, 127, 128, 129, 250, 252, 255, 256]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("e", EXPERTS)
def test_masked_rows_and_ties(dtype, e):
    k = min(e, 9)
    for t in (1, 3, 65, 300):
        for seed in range(2):
            logits = _logits(t, e, dtype, 31 * e + t + seed, gap=3 * seed, ties=bool(seed))
            if dtype is torch.float32 and seed:  # neighbours in their last bits
                gen = torch.Generator().manual_seed(t)
                logits += (torch.randint(-2, 3, (t, e), generator=gen) * 2.0 ** -22).to(device())
            mask = torch.ones(t, dtype=torch.bool)
            mask[0] = t == 1
            mask[4:9] = False
            mask[::5] &= t < 5
            clean = torch.where(mask[:, None].to(device()), logits, torch.zeros_like(logits))
            logits[~mask.to(device())] = math.nan
            normalize = not seed
            status = torch.zeros(1, dtype=torch.int32, device=device())
            r = bsg.moe_router_topk(logits, k, mask=mask.to(device()), normalize=normalize, status=status)
            ref = _reference(clean, k, mask, normalize)
            _check_forward(r, ref)
            assert int(status) == 0
            dw = torch.randn((t, k), generator=torch.Generator().manual_seed(e))
            d = bsg.moe_router_topk_backward(logits, r["experts"], r["counts"], r["live"],
                                             d_weights=dw.to(device()), d_loss=torch.ones(1, device=device()),
                                             mask=mask.to(device()), normalize=normalize)
            _check_backward(d, ref, e, k, dw.to(F64), 1.0, normalize)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("e", EXPERTS)
def test_not_finite_beside_others(dtype, e):
    """A token of a NaN chooses among the rest, one of +inf the infinity; the tokens beside them are as ever."""
    k, t = min(e, 5), 70
    logits = _logits(t, e, dtype, e)
    fine = torch.ones(t, dtype=torch.bool)
    fine[[1, 6, 64]] = False
    logits[1, e // 2] = math.nan
    logits[6, e - 1] = math.inf
    logits[64] = math.nan
    r = bsg.moe_router_topk(logits, k)
    ref = _reference(torch.where(logits.isnan(), torch.full_like(logits, -math.inf), logits), k, None, True)
    assert torch.equal(r["experts"].cpu().long(), ref["experts"])
    w = r["weights"].cpu().to(F64)
    # the tolerance of the other file's checks, for logits of this spread
    x = ref["x"].gather(1, ref["at"]).abs()
    tol = (x + 60) * 2.0 ** -23 * ref["weights"].abs() + 2.0 ** -126
    assert bool(((w - ref["weights"]).abs() <= tol)[fine].all())
    assert bool(w[6, :1].isnan().all()) and bool((w[64] == 0).all())
    if e > 1:
        assert bool(w[1][ref["experts"][1] >= 0].isnan().all())
