"""One workspace of the adapters for calls of different sizes: its size never decreases in any argument (host),
and calls of fewer rows, other widths and smaller ranks run in the largest one's (GPU)."""

import pytest
import torch

import block_scaled_grouped_amd as bsg

ROWS = [0, 1, 31, 32, 1000, 1023, 1024, 1025, 1026, 2000, 2047, 2048, 2730, 2731, 4095, 4096, 4097, 100000]
WIDTHS = [8, 64, 1008, 1016, 1024, 1032, 4096, 14336]
RANKS = [8, 16, 24, 56, 64, 72, 128, 136, 256]


def _sizes(rows=4096, n=4096, k=4096, rank=64):
    size = bsg.load_library().grouped_lora_gemm_16bit_workspace_size
    return size(rows, n, k, rank)


@pytest.mark.parametrize("rank", RANKS)
@pytest.mark.parametrize("k", WIDTHS)
def test_size_never_decreases(k, rank):
    for name, values in (("rows", ROWS), ("n", WIDTHS), ("k", WIDTHS), ("rank", RANKS)):
        sizes = [_sizes(**{"k": k, "rank": rank, name: v}) for v in values]
        assert sizes == sorted(sizes) and sizes[0] > 0, (name, sizes)
    sizes = [_sizes(rows=r, k=k, rank=rank) for r in range(900, 5000)]
    assert sizes == sorted(sizes)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_largest_calls_workspace_serves_the_others(dtype):
    from gpu_util import device
    from test_gpu_16bit import F64, TINY, _lora_reference, _offsets, _rand

    device()
    gen = torch.Generator().manual_seed(15)
    work = bsg.grouped_lora_gemm_16bit_workspace(2000, 264, 1016, 72)
    for rows, n, k, r in ((2000, 264, 1016, 72), (1024, 264, 1024, 72), (1000, 520, 1544, 64), (37, 136, 72, 72),
                          (1, 264, 1024, 8)):
        o, off = _offsets([rows - rows // 3, rows // 3])
        x, w = _rand(gen, (rows, k), dtype), _rand(gen, (n, k), dtype, std=0.1)
        A, B = _rand(gen, (2, r, k), dtype, std=0.1), _rand(gen, (2, n, r), dtype, std=0.5)
        scale = (torch.rand(2, generator=gen) + 0.5).to(x.device)
        work.fill_(0xFF)                                      # NaN, whatever it is read as
        y = bsg.grouped_lora_gemm_16bit(x, w, A, B, off, torch.tensor([1, 0], dtype=torch.int32, device=x.device),
                                        scale, out_dtype=bsg.BSG_OUT_F32, workspace=work)
        ref, tol = _lora_reference(x, w, A, B, o, [1, 0], scale, dtype)
        err = (y.cpu().to(F64) - ref).abs()
        bound = tol + 2.0 ** -24 * (ref.abs() + tol) + TINY[torch.float32]
        assert bool((err <= bound).all()), float((err / bound).max())
