"""Adapters with offsets that decrease, are negative or run past the rows: clamped and flagged, nothing written
outside of what is left."""

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device
from test_gpu_16bit import _rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,k,many", [(136, 72, 1), (136, 1024, 1), (4096, 1024, 6), (8200, 72, 20)])
def test_bad_offsets_stay_in_bounds(n, k, many, dtype):
    dev = device()
    gen = torch.Generator().manual_seed(n + k)
    rows = 100 * many
    x, w = _rand(gen, (rows, k), dtype), _rand(gen, (n, k), dtype, std=0.1)
    A, B = _rand(gen, (2, 24, k), dtype, std=0.2), _rand(gen, (2, n, 24), dtype, std=0.5)
    scale = torch.ones(2, device=dev)
    ids = torch.tensor([0, 1], dtype=torch.int32, device=dev)

    def call(offsets):
        out = torch.full((rows, n), -7.0, dtype=dtype, device=dev)
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        off = torch.tensor([many * o if abs(o) <= 100 else o for o in offsets], device=dev)
        bsg.grouped_lora_gemm_16bit(x, w, A, B, off, ids, scale, out=out, status=status)
        return out, int(status)

    # offsets, the bit that they set, the rows that are left and the offsets that those have
    for bad, bit, left, good in (([0, 50, 1 << 40], bsg.DEV_OVER_CAPACITY, (0, 100), [0, 50, 100]),
                                 ([-9, 50, 100], bsg.DEV_NEGATIVE_SIZE, (0, 100), [0, 50, 100]),
                                 ([-(1 << 50), 50, 100], bsg.DEV_NEGATIVE_SIZE, (0, 100), [0, 50, 100]),
                                 ([0, 90, 30], bsg.DEV_NEGATIVE_SIZE, (0, 30), [0, 30, 30]),
                                 ([60, 20, 10], bsg.DEV_NEGATIVE_SIZE, (0, 0), [0, 0, 0]),
                                 ([100, 100, 0], bsg.DEV_NEGATIVE_SIZE, (0, 0), [0, 0, 0])):
        y, status = call(bad)
        want, clean = call(good)
        assert status == bit and clean == 0, bad
        live = slice(many * left[0], many * left[1])
        assert torch.equal(y[live], want[live]), bad
        assert bool((y[live.stop:] == -7.0).all()), bad
