"""Every form of the int8 products, and the form of few rows where it runs on: tiles of several groups in one
workgroup, tokens that are quantized again for the next group, contractions shorter than a wave's line.  Bit for
bit, as in test_gpu_int8.py."""

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device
from test_gpu_int8 import _case, _product, _quantized, _run

pytestmark = pytest.mark.gpu


def _sizes(groups, rows, seed=0):
    """Group sizes that add up to `rows`, uneven, the second empty."""
    gen = torch.Generator().manual_seed(seed)
    p = torch.rand(groups, generator=gen) + 0.05
    if groups > 1:
        p[1] = 0
    draws = torch.multinomial(p, rows, replacement=True, generator=gen)
    return torch.bincount(draws, minlength=groups).tolist()


@pytest.mark.parametrize("form,groups,rows,n,k", [
    (16, 8, 24, 256, 272), (16, 1, 16, 1032, 4112), (32, 1, 24, 256, 272), (32, 3, 40, 2048, 4096),
    (64, 8, 400, 4104, 272), (128, 1, 1000, 4104, 272), (256, 1, 2048, 4104, 272), (256, 8, 3000, 4104, 2064)])
def test_every_form(form, groups, rows, n, k):
    case = _case(_sizes(groups, rows), n, k, seed=form)
    for ws in (bsg.gemm_workspace(), None):
        if groups != 8 or rows != 3000:
            assert bsg.grouped_gemm_int8_tile_rows(groups, rows, n, k, workspace=ws is not None) == form
        for dtype in (torch.bfloat16, torch.float16, torch.float32):
            _run(case, dtype, ws, gap=8 if dtype == torch.float16 else 0)


@pytest.mark.parametrize("rows,n,k", [(300, 520, 131056), (600, 264, 8208)])
def test_split_contractions(rows, n, k):
    """Long contractions over few tiles: split with a workspace, the same bits without one."""
    a, sa, w, sw, off, ends = _case([rows], n, k, 3)
    whole = bsg.grouped_gemm_int8(a, sa, w, sw, off, out_dtype=bsg.BSG_OUT_F32)
    split = bsg.grouped_gemm_int8(a, sa, w, sw, off, out_dtype=bsg.BSG_OUT_F32, workspace=bsg.gemm_workspace())
    assert torch.equal(whole, split)
    assert torch.equal(whole.cpu(), _product(a, sa, w, sw, ends, torch.float32))


@pytest.mark.parametrize("sizes,n,k", [
    ([16], 16, 16), ([7], 24, 112), ([3], 8, 144), ([2], 40, 400), ([5], 1000, 528),     # waves without a line
    ([1] * 256, 136, 256),                                                              # all groups
    ([4, 0, 30, 1, 17, 0, 0, 12], 4104, 1040),                                          # several blocks of rows
    ([1, 2, 0, 1], 16384, 528), ([16], 20000, 272),                                     # several tiles a workgroup
])
def test_few_rows(sizes, n, k):
    total = sum(sizes)
    assert bsg.grouped_gemm_int8_tile_rows(len(sizes), total, n, k) == 16 or total > 4 * len(sizes)
    for first, gap, low in ((0, 0, -127), (3, 16, -128)):
        case = _case(sizes, n, k, seed=total, first=first, gap=gap, low=low)
        for dtype in (torch.bfloat16, torch.float32):
            _run(case, dtype, gap=8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes,n,k", [
    ([1], 16, 16), ([1], 136, 8192), ([1], 20000, 1024), ([2], 264, 4096), ([8], 520, 1024), ([5], 40, 48),
    ([0, 0, 1], 264, 2048), ([1, 2, 0, 1], 16384, 2048), ([3, 0, 4, 1], 8200, 1008), ([1] * 8, 4096, 512),
    ([0, 0], 64, 128)])
def test_tokens_quantized_in_the_product(dtype, sizes, n, k):
    """At most 8 rows and 8192 integers: one launch."""
    _, _, w, sw, off, ends = _case(sizes, n, k, 7)
    rows = ends[-1]
    gen = torch.Generator().manual_seed(rows + k)
    for gap in (0, 8):
        wide = torch.full((rows, k + gap), float("nan"), dtype=dtype)
        wide[:, :k] = (torch.randn((rows, k), generator=gen) * 10.0 ** torch.randint(-2, 3, (rows, 1), generator=gen)).to(dtype)
        x = wide.to(device())[:, :k]
        for od in (None, bsg.BSG_OUT_F32):
            y = bsg.grouped_gemm_int8_dynamic(x, w, sw, off, out_dtype=od)
            q, s = _quantized(x)
            assert torch.equal(y.cpu(), _product(q, s, w, sw, ends, y.dtype))


@pytest.mark.parametrize("rows,k", [(2, 64), (8, 1024), (1, 8192)])
def test_tokens_in_the_product_not_finite_or_zero(rows, k):
    _, _, w, sw, off, ends = _case([rows], 272, k, 8)
    x = torch.randn((rows, k), device=device()).to(torch.bfloat16)
    x[0] = 0
    status = torch.zeros(1, dtype=torch.int32, device=device())
    y = bsg.grouped_gemm_int8_dynamic(x, w, sw, off, status=status)
    assert bool((y[0] == 0).all()) and int(status) == 0
    x[rows - 1, k - 1] = float("inf")
    y = bsg.grouped_gemm_int8_dynamic(x, w, sw, off, status=status)
    assert int(status) == bsg.DEV_NONFINITE and bool(y[rows - 1].isnan().all())
    assert rows == 1 or bool((y[0] == 0).all())


def test_live_rows_of_a_larger_buffer():
    """Rows outside of the offsets stay as they were, in every form of the tokens' path."""
    for rows, n, k in ((8, 264, 512), (60, 264, 512), (600, 2056, 512)):
        _, _, w, sw, _, _ = _case([1, 1], n, k, 9)
        x = torch.full((rows, k), float("nan"), dtype=torch.bfloat16, device=device())
        lo, mid, hi = rows // 4, rows // 3 + 1, rows - 2
        x[lo:hi] = torch.randn((hi - lo, k), device=device()).to(torch.bfloat16)
        out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device=device())
        status = torch.zeros(1, dtype=torch.int32, device=device())
        bsg.grouped_gemm_int8_dynamic(x, w, sw, torch.tensor([lo, mid, hi], device=device()), out=out, status=status)
        q, s = _quantized(torch.where(x.isnan(), 0, x))
        want = _product(q, s, w, sw, [lo, mid, hi], torch.bfloat16)
        assert int(status) == 0
        assert torch.equal(out[lo:hi].cpu(), want[lo:hi])
        assert bool((out[:lo] == 7).all()) and bool((out[hi:] == 7).all())


@pytest.mark.parametrize("offsets", [[0, -5, 8], [0, 5, 0, 3, 8], [0, 500], [-3, 4], [6, 2], [9, 12]])
def test_bad_offsets_of_few_rows(offsets):
    """Clamped and flagged; what lies outside is not touched."""
    groups = len(offsets) - 1
    _, _, w, sw, _, _ = _case([1] * groups, 72, 256, 10)
    for rows in (8, 12):
        x = torch.randn((rows, 256), device=device()).to(torch.bfloat16)
        guard = torch.full((rows + 8, 72), 7.0, dtype=torch.bfloat16, device=device())
        status = torch.zeros(1, dtype=torch.int32, device=device())
        bsg.grouped_gemm_int8_dynamic(x, w, sw, torch.tensor(offsets, device=device()), out=guard[:rows], status=status)
        assert offsets == [9, 12] and rows == 12 or int(status) != 0
        assert bool((guard[rows:] == 7).all())
