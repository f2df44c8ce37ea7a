"""Logits whose largest are not spread over the experts: sorted, equal, a few open ones, the chosen ones in one run of
experts or at equal distances (an implementation that shares out a token's experts then has to take all of one share),
and float32 logits around the last slot that differ in their last bits alone.  Tolerances as in test_gpu_router.py;
logits are at most 16 apart."""

import math

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device
from test_gpu_router import DTYPES, F64, _check_backward, _check_forward, _reference

pytestmark = pytest.mark.gpu

EXPERTS = [65, 72, 96, 100, 113, 120, 127, 128]


def _shares(e):
    """Sets of experts that 16 shares of a token may be made of."""
    sets = [range(g, g + 8) for g in range(0, e, 8)]
    sets += [range(s, e, 16) for s in range(16)]
    for run in (4, 8):
        sets += [[x for x in range(e) if x // run % 16 == s] for s in range(16)]
    return [torch.tensor([x for x in s if x < e]) for s in sets if any(x < e for x in s)]


def _tokens(e, k, seed):
    """[tokens, e] logits that bfloat16 holds exactly, a few thousand at most."""
    gen = torch.Generator().manual_seed(seed)
    index = torch.arange(e).float() * 2.0 ** -4      # e <= 256: 8 bits
    rows = [torch.zeros(e), index, -index, (index * 16 % 8) * 0.5, torch.full((e,), -1.5)]
    for share in _shares(e):
        noise = torch.randint(-32, 0, (e,), generator=gen).float() * 2.0 ** -4
        closed = torch.full((e,), -math.inf)
        spread = torch.randperm(len(share), generator=gen).float() * 2.0 ** -3
        for below in (noise, closed):
            for top in (spread, torch.zeros(len(share))):   # all different, all equal
                rows.append(below.clone().index_copy_(0, share, top))
        # the share and one expert more, with slots left
        rows.append(rows[-1].clone().index_fill_(0, torch.randint(0, e, (1,), generator=gen), 0.25))
    for n in range(1, 9):                            # n open experts, the first one among them or not
        for first in (True, False):
            row = torch.full((e,), -math.inf)
            pick = torch.randperm(e, generator=gen)[:n]
            if first:
                pick[0] = 0
            rows.append(row.index_copy_(0, pick, torch.randint(-8, 8, (n,), generator=gen).float() / 8))
    rows += list((torch.randn((40, e), generator=gen) * 4).round() / 4)
    return torch.stack(rows)


def _check(logits, k, normalize, mask=None):
    t, e = logits.shape
    r = bsg.moe_router_topk(logits, k, mask=mask, normalize=normalize)
    ref = _reference(logits, k, mask, normalize)
    # x is for the tolerances: (x + 60) STEP times a weight.  Of a slot without an expert the weight is 0 and x is
    # expert 0's, so where that one is closed the product would be inf * 0; open ones are less than 110 apart here
    ref["x"] = ref["x"].clamp(min=-110)
    experts = r["experts"].cpu().long()
    chosen = torch.zeros((t, e + 1), dtype=torch.int64).scatter_add_(1, experts % (e + 1), torch.ones_like(experts))
    assert bool((chosen[:, :e] <= 1).all())          # no expert twice
    _check_forward(r, ref)
    dw = torch.randn((t, k), generator=torch.Generator().manual_seed(k))
    d = bsg.moe_router_topk_backward(logits, r["experts"], r["counts"], r["live"], d_weights=dw.to(device()),
                                     d_loss=torch.ones(1, device=device()), mask=mask, normalize=normalize)
    _check_backward(d, ref, e, k, dw.to(F64), 1.0, normalize)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("e", EXPERTS)
@pytest.mark.parametrize("k", range(8, 17))
def test_one_share_holds_the_largest(dtype, e, k):
    logits = _tokens(e, k, 100 * e + k).to(dtype).to(device())
    _check(logits, k, k % 2 == 0)
    _check(logits[:200], k, k % 2 == 1)              # one launch


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("e,k", [(16, 16), (33, 16), (64, 9), (64, 16), (129, 16), (200, 10), (250, 16), (256, 9),
                                 (256, 16)])
def test_other_numbers_of_experts(dtype, e, k):
    _check(_tokens(e, k, e + k).to(dtype).to(device()), k, True)


@pytest.mark.parametrize("e,k", [(128, 8), (100, 8), (125, 8), (256, 16), (250, 16), (129, 16), (128, 12), (64, 4)])
def test_neighbours_at_the_last_slot(e, k):
    """The k-th and the next share all but their last bits, and the next by value has the higher index; the larger
    ones stand in one share."""
    gen = torch.Generator().manual_seed(e * k)
    rows = []
    for share in _shares(e):
        if len(share) < k:
            continue
        share = share[torch.randperm(len(share), generator=gen)[:k]]
        last = int(share.argmin())
        others = [x for x in range(int(share[last]) + 1, e) if x not in share.tolist()]
        if not others:
            continue
        row = torch.rand(e, generator=gen) - 4.0
        row[share] = torch.rand(k, generator=gen) + 2.0
        row[share[last]] = 1.0
        row[others[int(torch.randint(0, len(others), (1,), generator=gen))]] = 1.0 + 2.0 ** -21
        rows += [row, -2.0 ** -10 * row.flip(0)]
    for n in range(20):                              # without a share: the same two, others anywhere
        row = torch.rand(e, generator=gen) - 4.0
        pick = torch.randperm(e, generator=gen)[:k + 1]
        row[pick] = torch.rand(k + 1, generator=gen) + 2.0
        low, high = sorted(pick[:2].tolist())
        row[low], row[high] = 1.0, 1.0 + 2.0 ** -21
        rows.append(row)
    logits = torch.stack(rows).to(device())
    for normalize in (False, True):
        _check(logits, k, normalize)
