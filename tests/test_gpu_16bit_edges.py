"""Edges of the 16-bit operators: subnormal numbers, calls without rows, the most groups."""

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device
from test_gpu_16bit import DTYPES, F64, MODES, _live, _offsets, _operands, _product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype,small,large", [(torch.float16, 2.0 ** -24, 2.0 ** 10),
                                               (torch.bfloat16, 2.0 ** -133, 2.0 ** 120)])
def test_subnormal_operands_count(dtype, small, large, mode):
    """Whole numbers times the type's smallest subnormal, times large ones: exact in float32."""
    gen = torch.Generator().manual_seed(16)
    sizes, n, k = [40, 0, 9], 72, 136
    a, b, _ = _operands(gen, mode, sizes, n, k, dtype)
    a.copy_((torch.randint(-7, 8, a.shape, generator=gen).to(F64) * small).to(dtype))
    b.copy_((torch.randint(-7, 8, b.shape, generator=gen).to(F64) * large).to(dtype))
    o, off = _offsets(sizes)
    y = bsg.grouped_gemm_16bit(mode, a, b, off, out_dtype=bsg.BSG_OUT_F32)
    assert torch.equal(y.cpu().to(F64), _product(mode, a, b, o)[0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_subnormal_outputs_are_rounded_and_not_flushed(dtype):
    """An identity as the second operand: the output is the input, subnormals and all."""
    dev = device()
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    x = (torch.arange(-64, 64, dtype=F64).view(16, 8) * tiny * 3).to(dtype).to(dev)
    eye = torch.eye(8, dtype=dtype, device=dev)[None]
    off = torch.tensor([0, 16], device=dev)
    for mode in MODES[:2]:
        y = bsg.grouped_gemm_16bit(mode, x, eye, off)
        assert torch.equal(y, x)
    assert torch.equal(bsg.grouped_gemm_16bit(bsg.BSG_FPROP_TN, x, torch.zeros_like(eye), off, c=x), x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_clip_of_subnormal_gradients(dtype):
    """Subnormal numbers enter the norm and are scaled: exact for a power of two and whole multiples of it."""
    dev = device()
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    small = (torch.arange(1, 60, dtype=F64) * 2 * tiny).to(dtype).to(dev)
    norm = bsg.grad_norm(bsg.grad_clip_plan([small]))
    want = float(small.cpu().to(F64).square().sum().sqrt())
    assert abs(float(norm) - want) <= 2.0 ** -23 * want + 2.0 ** -150
    # next to a large value that makes the factor 1/2: 1e-6 is far below a half step of 8
    large = torch.full((1,), 8.0, dtype=dtype, device=dev)
    outs = [torch.zeros_like(small), torch.zeros_like(large)]
    bsg.clip_grad_norm(bsg.grad_clip_plan([small, large], outs), 4.0)
    assert bool(((outs[0].cpu().to(F64) - small.cpu().to(F64) / 2).abs() <= tiny / 2).all())
    assert bool((outs[0] != 0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mode", MODES)
def test_no_rows(mode, dtype):
    dev = device()
    n, k = 72, 136
    off = torch.zeros(4, dtype=torch.int64, device=dev)
    a = torch.empty((0, n if mode == bsg.BSG_WGRAD_NT else k), dtype=dtype, device=dev)
    b = torch.empty({bsg.BSG_WGRAD_NT: (0, k), bsg.BSG_FPROP_TN: (3, n, k), bsg.BSG_DGRAD_NN: (3, k, n)}[mode],
                    dtype=dtype, device=dev)
    for work in (None, bsg.gemm_workspace()):
        y = bsg.grouped_gemm_16bit(mode, a, b, off, workspace=work)
        if mode != bsg.BSG_WGRAD_NT:
            assert tuple(y.shape) == (0, n)
            continue
        assert tuple(y.shape) == (3, n, k) and bool((y == 0).all())
        c = torch.full((3, n, k), 5.0, device=dev)
        assert torch.equal(bsg.grouped_gemm_16bit(mode, a, b, off, c=c, workspace=work), c)


@pytest.mark.parametrize("dtype", DTYPES)
def test_adapters_without_rows(dtype):
    dev = device()
    off = torch.zeros(3, dtype=torch.int64, device=dev)
    args = [torch.empty(s, dtype=dtype, device=dev) for s in ((0, 64), (72, 64), (2, 8, 64), (2, 72, 8))]
    ids, scale = torch.tensor([0, 1], dtype=torch.int32, device=dev), torch.ones(2, device=dev)
    assert tuple(bsg.grouped_lora_gemm_16bit(*args, off, ids, scale).shape) == (0, 72)
    # rows that no request owns
    x = torch.full((40, 64), float("nan"), dtype=dtype, device=dev)
    out = torch.full((40, 72), -7.0, dtype=dtype, device=dev)
    bsg.grouped_lora_gemm_16bit(x, *args[1:], off, ids, scale, out=out)
    assert bool((out == -7.0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mode", MODES)
def test_256_groups(mode, dtype):
    gen = torch.Generator().manual_seed(17)
    sizes = [(7 * g) % 5 for g in range(256)]
    n, k = 40, 72
    a, b, _ = _operands(gen, mode, sizes, n, k, dtype)
    a.copy_(torch.randint(-9, 10, a.shape, generator=gen).to(dtype))
    b.copy_(torch.randint(-9, 10, b.shape, generator=gen).to(dtype))
    o, off = _offsets(sizes)
    y = bsg.grouped_gemm_16bit(mode, a, b, off, out_dtype=bsg.BSG_OUT_F32, workspace=bsg.gemm_workspace())
    ref = _product(mode, a, b, o)[0]
    assert torch.equal(_live(mode, y, o).cpu().to(F64), _live(mode, ref, o))
