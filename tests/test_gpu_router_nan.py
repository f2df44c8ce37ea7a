"""Tokens whose logits are all NaN, or NaN and -inf: no logit is above -inf, so they are not live, whatever stands
beside them.  Tolerances as in test_gpu_router.py; every other logit is finite."""

import math

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device
from test_gpu_router import DTYPES, F64, _check_backward, _check_forward, _logits, _reference

pytestmark = pytest.mark.gpu

SIGNALLING = [(torch.bfloat16, torch.int16, 0x7f81), (torch.float16, torch.int16, 0x7c01),
              (torch.float32, torch.int32, 0x7f800001)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("e", [1, 2, 7, 16, 17, 32, 64, 65, 100, 128, 129, 250, 256])
def test_tokens_of_nan_are_not_live(dtype, e):
    k = min(e, 10)
    for t in (1, 6, 70, 256, 600):
        for normalize in (False, True):
            logits = _logits(t, e, dtype, 7 * e + t, gap=3 if normalize else 0)
            rows = torch.zeros(t, dtype=torch.bool)
            rows[::9] = True
            rows[t // 2:t // 2 + 5] = True       # a whole wave's four tokens among them
            some = torch.rand((t, e), generator=torch.Generator().manual_seed(t)) < 0.5
            some[:, e // 2] = True               # NaN at least here
            closed = torch.where(some, math.nan, -math.inf).to(dtype)
            closed[::2] = math.nan
            at = rows.to(device())
            logits[at] = closed.to(device())[at]
            status = torch.zeros(1, dtype=torch.int32, device=device())
            r = bsg.moe_router_topk(logits, k, normalize=normalize, status=status)
            ref = _reference(logits, k, None, normalize)
            assert ref["live"] == int((~rows).sum())
            _check_forward(r, ref)
            assert int(status) == bsg.DEV_NONFINITE
            assert bool((r["experts"].cpu()[rows] == -1).all()) and bool((r["weights"].cpu()[rows] == 0).all())
            dw = torch.randn((t, k), generator=torch.Generator().manual_seed(e))
            d = bsg.moe_router_topk_backward(logits, r["experts"], r["counts"], r["live"], d_weights=dw.to(device()),
                                             d_loss=torch.ones(1, device=device()), normalize=normalize)
            assert bool((d.cpu()[rows] == 0).all())
            _check_backward(d, ref, e, k, dw.to(F64), 1.0, normalize)


@pytest.mark.parametrize("dtype,word,bits", SIGNALLING)
def test_tokens_of_signalling_nan_are_not_live(dtype, word, bits):
    for e in (12, 128, 256):
        logits = _logits(70, e, dtype, e)
        logits.view(word)[5] = bits
        r = bsg.moe_router_topk(logits, 4)
        _check_forward(r, _reference(logits, 4, None, True))
        assert int(r["live"]) == 69


def test_every_token_of_nan():
    for t in (3, 300):
        logits = torch.full((t, 24), math.nan, device=device())
        r = bsg.moe_router_topk(logits, 3)
        assert int(r["live"]) == 0 and float(r["loss"]) == 0.0 and int(r["counts"].sum()) == 0
        assert bool((r["prob_sums"] == 0).all()) and bool((r["experts"] == -1).all())
        d = bsg.moe_router_topk_backward(logits, r["experts"], r["counts"], r["live"],
                                         d_weights=torch.ones((t, 3), device=device()),
                                         d_loss=torch.ones(1, device=device()))
        assert bool((d == 0).all())


@pytest.mark.parametrize("dtype,word,bits", SIGNALLING)
@pytest.mark.parametrize("e", [9, 16, 30, 64, 100, 128, 250, 256])
def test_signalling_nan_is_not_chosen(dtype, word, bits, e):
    for t in (70, 300):
        logits = _logits(t, e, dtype, e)
        wrong = torch.rand((t, e), generator=torch.Generator().manual_seed(e)) < 0.3
        wrong[:, 0] = False
        wrong[::3] = False
        held = logits.cpu()
        held.view(word)[wrong] = bits
        logits.copy_(held)
        assert torch.equal(logits.isnan().cpu(), wrong)
        status = torch.zeros(1, dtype=torch.int32, device=logits.device)
        r = bsg.moe_router_topk(logits, 4, status=status)
        ref = _reference(torch.where(logits.isnan(), -math.inf, logits), 4, None, True)
        assert torch.equal(r["experts"].cpu().long(), ref["experts"]) and int(status) == bsg.DEV_NONFINITE
        w, bad = r["weights"].cpu(), wrong.any(1)
        assert bool(w[bad][ref["chosen"][bad]].isnan().all()) and bool(w[~bad].isfinite().all())
