"""The int8 quantizer and products, bit for bit: the quotients are resolved by 64-bit division (an exact quotient
is at least 2^-25 of itself away from the border of two integers, unless it lies on it), the sums are integers,
and a result is the sum rounded to float32, times the row's scale, times the channel's, rounded to its type:
every step of it is repeated here in the same arithmetic."""

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device

pytestmark = pytest.mark.gpu

F64 = torch.float64
OUT = {torch.bfloat16: bsg.BSG_OUT_BF16, torch.float16: bsg.BSG_OUT_F16, torch.float32: bsg.BSG_OUT_F32}


def _quantized(x):
    """(integers, scales) of rows on the host."""
    top = x.cpu().abs().amax(1).float()
    scale = (top / torch.full_like(top, 127.0))
    s = scale.to(F64)
    q = torch.where(s[:, None] > 0, x.cpu().to(F64) / s[:, None].clamp(min=1e-300), 0.0)
    return torch.round(q).to(torch.int8), scale


def _check_quantized(x, got, what=""):
    q, s = _quantized(x)
    assert torch.equal(got[1].cpu().view(torch.int32), s.view(torch.int32)), what
    bad = got[0].cpu() != q
    assert not bool(bad.any()), (what, int(bad.sum()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cols", [16, 48, 512, 528, 1024, 1040, 2048, 2064, 4096, 4112, 8192, 8208, 16384, 16400,
                                  20016])
def test_quantize(dtype, cols):
    gen = torch.Generator().manual_seed(cols)
    for rows, gap in ((1, 0), (9, 8), (70, 0)):
        v = torch.randn((rows, cols), generator=gen) * 10.0 ** torch.randint(-3, 4, (rows, 1), generator=gen)
        v = torch.where(torch.rand((rows, cols), generator=gen) < 0.01, v * 20, v).clamp(-6e4, 6e4)
        wide = torch.full((rows, cols + gap), float("nan"), dtype=dtype)
        wide[:, :cols] = v.to(dtype)
        x = wide.to(device())[:, :cols]
        status = torch.zeros(1, dtype=torch.int32, device=device())
        _check_quantized(x, bsg.grouped_quantize_int8(x, status=status), (rows, gap))
        assert int(status) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_borders(dtype):
    """Values on and next to the borders of two integers, for scales of every kind."""
    gen = torch.Generator().manual_seed(1)
    halves = (torch.arange(-127, 127).to(F64) + 0.5).repeat(8)[:2032]
    tops = [127.0, 254.0, 63.5, 1.0, 3.14159, 100.0, 0.7, 31.75, 2032.0] + torch.rand(300, generator=gen).tolist()
    rows = []
    for top in tops:
        top = torch.tensor(top).to(dtype)
        s = (top.float() / torch.tensor(127.0)).to(F64)
        near = halves * s * (1 + torch.randint(-1, 2, halves.shape, generator=gen) * torch.finfo(dtype).eps)
        rows.append(torch.cat([near.to(dtype).clamp(-top, top), top.view(1), -top.view(1),
                               torch.zeros(14, dtype=dtype)]))
    x = torch.stack(rows).to(device())
    _check_quantized(x, bsg.grouped_quantize_int8(x))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_quantize_extremes(dtype):
    """Rows of zeros, of subnormal numbers, of the type's smallest and largest, and of one value."""
    info = torch.finfo(dtype)
    gen = torch.Generator().manual_seed(2)
    least = info.smallest_normal * info.eps
    rows = [torch.zeros(64), torch.full((64,), -0.0), torch.full((64,), info.max), torch.full((64,), -info.max),
            torch.full((64,), info.smallest_normal), torch.full((64,), least)]
    rows += [(torch.randint(-300, 301, (64,), generator=gen).to(F64) * least * m).float()
             for m in (0.01, 0.1, 1, 2, 5, 100, 1e4)]
    rows += [torch.randn(64, generator=gen) * s for s in (1e-7, 1e-6, 1e-5, 1e-20 if dtype == torch.bfloat16 else 1e-4)]
    x = torch.stack(rows).to(dtype).to(device())
    _check_quantized(x, bsg.grouped_quantize_int8(x))


def test_quantize_not_finite_and_offsets():
    for cols in (64, 3000 // 16 * 16, 20016):
        x = torch.randn((40, cols), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
        x[5, 3], x[7, cols - 1], x[8] = float("nan"), float("-inf"), float("inf")
        x[:2], x[30:] = float("nan"), float("inf")     # rows that no group owns
        off = torch.tensor([2, 11, 11, 30], device=device())
        data = torch.full((40, cols), 99, dtype=torch.int8, device=device())
        scales = torch.full((40,), 5.0, device=device())
        status = torch.zeros(1, dtype=torch.int32, device=device())
        bsg.grouped_quantize_int8(x.to(device()), off, data=data, scales=scales, status=status)
        assert int(status) == bsg.DEV_NONFINITE
        d, s = data.cpu(), scales.cpu()
        assert bool((d[:2] == 99).all()) and bool((d[30:] == 99).all())
        assert bool((s[:2] == 5).all()) and bool((s[30:] == 5).all())
        for r in (5, 7, 8):
            assert bool((d[r] == 0).all()) and bool(s[r].isnan())
        fine = [r for r in range(2, 30) if r not in (5, 7, 8)]
        _check_quantized(x[fine], (d[fine], s[fine]))
    for bad, bit in (([-3, 40], bsg.DEV_NEGATIVE_SIZE), ([0, 41], bsg.DEV_OVER_CAPACITY), ([30, 2], bsg.DEV_NEGATIVE_SIZE)):
        status = torch.zeros(1, dtype=torch.int32, device=device())
        bsg.grouped_quantize_int8(x.to(device()), torch.tensor(bad, device=device()), status=status)
        assert int(status) & bit


def _case(sizes, n, k, seed=0, dead=0, first=0, gap=0, low=-127):
    gen = torch.Generator().manual_seed(seed + n + k)
    ends = [first]
    for s in sizes:
        ends.append(ends[-1] + s)
    rows = ends[-1] + dead
    a = torch.randint(low, 128, (rows, k + gap), generator=gen, dtype=torch.int8)
    w = torch.randint(low, 128, (len(sizes), n, k + gap), generator=gen, dtype=torch.int8)
    sa = torch.rand(rows, generator=gen) * 0.02 + 1e-4
    sw = torch.rand((len(sizes), n), generator=gen) * 0.01
    if dead:
        sa[ends[-1]:] = float("nan")
    sa[:first] = float("nan")
    dev = device()
    return (a.to(dev)[:, :k], sa.to(dev), w.to(dev)[:, :, :k], sw.to(dev), torch.tensor(ends, device=dev), ends)


def _product(a, sa, w, sw, ends, dtype):
    a, sa, w, sw = (t.cpu() for t in (a, sa, w, sw))
    out = torch.zeros((a.shape[0], w.shape[1]), dtype=dtype)
    for g in range(w.shape[0]):
        lo, hi = ends[g], ends[g + 1]
        if hi > lo:
            acc = (a[lo:hi].to(F64) @ w[g].to(F64).t().contiguous()).to(torch.int64).to(torch.float32)
            out[lo:hi] = ((acc * sa[lo:hi, None]) * sw[g]).to(dtype)
    return out


def _run(case, dtype, workspace=None, gap=0):
    a, sa, w, sw, off, ends = case
    wide = torch.full((a.shape[0], w.shape[1] + gap), 7.0, dtype=dtype, device=device())
    y = bsg.grouped_gemm_int8(a, sa, w, sw, off, out=wide[:, :w.shape[1]], workspace=workspace)
    want = _product(a, sa, w, sw, ends, dtype)
    got = wide.cpu()
    assert torch.equal(got[ends[0]:ends[-1], :w.shape[1]], want[ends[0]:ends[-1]])
    assert bool((got[:ends[0]] == 7).all()) and bool((got[ends[-1]:] == 7).all())
    assert bool((got[:, w.shape[1]:] == 7).all())
    return y


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("sizes,n,k", [([1], 8, 16), ([1], 24, 48), ([3, 0, 1], 136, 144), ([17, 0, 0, 40], 264, 528),
                                       ([1] * 9, 120, 1040), ([130, 70], 256, 2048), ([300], 128, 4096),
                                       ([0, 0], 64, 64), ([65, 0, 129], 8, 7168)])
def test_product(dtype, sizes, n, k):
    ws = bsg.gemm_workspace()
    for seed, (dead, first, gap, use) in enumerate([(0, 0, 0, True), (5, 3, 16, True), (0, 2, 0, False)]):
        _run(_case(sizes, n, k, seed, dead, first, gap), dtype, ws if use else None, gap=8 * (seed % 2))


@pytest.mark.parametrize("rows,n,k,bm", [(2048, 4096, 2048, 256), (1500, 4104, 2064, 256), (700, 2056, 1040, 128),
                                         (200, 2048, 4096, 64), (40, 2048, 4096, 32)])
def test_forms(rows, n, k, bm):
    """Every tile form, whole and split, with groups that end inside of tiles."""
    sizes = [rows // 3 + 1, 0, rows - rows // 3 - 1]
    case = _case(sizes, n, k, dead=3)
    forms = set()
    for ws in (bsg.gemm_workspace(), None):
        for dtype in (torch.bfloat16, torch.float32):
            _run(case, dtype, ws)
        forms.add(bsg.grouped_gemm_int8_tile_rows(3, rows + 3, n, k, workspace=ws is not None))
    assert forms


def test_all_forms_are_reached():
    sizes = [(2048, 4096, 2048), (1500, 4104, 2064), (700, 2056, 1040), (200, 2048, 4096), (40, 2048, 4096),
             (16384, 14336, 4096), (1, 4096, 4096)]
    assert {bsg.grouped_gemm_int8_tile_rows(3, r + 3, n, k, workspace=w) for r, n, k in sizes
            for w in (True, False)} >= {32, 256}


def test_largest_sums():
    """The longest contraction, every product at its largest: 128 * 128 * 131056 < 2^31."""
    k = bsg.BSG_MAX_INT8_K
    for value, other in ((-128, -128), (-128, 127), (127, 127)):
        a = torch.full((3, k), value, dtype=torch.int8, device=device())
        w = torch.full((1, 16, k), other, dtype=torch.int8, device=device())
        off = torch.tensor([0, 3], device=device())
        for ws in (None, bsg.gemm_workspace()):
            y = bsg.grouped_gemm_int8(a, torch.ones(3, device=device()), w, torch.ones((1, 16), device=device()), off,
                                      out_dtype=bsg.BSG_OUT_F32, workspace=ws)
            assert bool((y == torch.tensor(float(value * other * k))).all())


def test_scales_that_are_not_finite_stay_in_their_row_and_column():
    case = list(_case([20, 30], 64, 256, 4))
    case[1] = case[1].clone()
    case[1][7] = float("nan")
    case[3] = case[3].clone()
    case[3][1, 5] = float("inf")
    y = bsg.grouped_gemm_int8(*case[:5], out_dtype=bsg.BSG_OUT_F32).cpu()
    bad = torch.zeros((50, 64), dtype=torch.bool)
    bad[7] = True
    bad[20:, 5] = True
    assert bool(y[~bad].isfinite().all()) and bool((~y[bad].isfinite()).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes,n,k", [([1], 2048, 4096), ([1, 0, 2, 1], 264, 1040), ([5], 24, 16), ([9, 0, 30], 512, 528),
                                       ([100, 0, 412], 1032, 2064), ([33], 64, 20016), ([2, 3, 0, 3], 128, 7168)])
def test_dynamic(dtype, sizes, n, k):
    """The tokens quantized on the way: the same bits as in two steps."""
    _, _, w, sw, off, ends = _case(sizes, n, k, 5)
    gen = torch.Generator().manual_seed(7)
    for dead, gap in ((0, 0), (4, 8)):
        rows = ends[-1] + dead
        wide = torch.full((rows, k + gap), float("nan"), dtype=dtype)
        wide[:ends[-1], :k] = (torch.randn((ends[-1], k), generator=gen) * 2).to(dtype)
        x = wide.to(device())[:, :k]
        for od in (None, bsg.BSG_OUT_F32):
            status = torch.zeros(1, dtype=torch.int32, device=device())
            y = bsg.grouped_gemm_int8_dynamic(x, w, sw, off, out_dtype=od, status=status)
            assert y.dtype == (dtype if od is None else torch.float32)
            q, s = _quantized(x[:ends[-1]])
            want = _product(q, s, w, sw, ends, y.dtype)
            assert torch.equal(y[:ends[-1]].cpu(), want[:ends[-1]])
            assert int(status) == 0


def test_dynamic_not_finite():
    """A token that is not finite makes its own row NaN."""
    for rows in (3, 200):
        _, _, w, sw, off, ends = _case([rows], 64, 512, 6)
        x = torch.randn((rows, 512), device=device()).to(torch.bfloat16)
        x[1, 100] = float("inf")
        x[2, 511] = float("nan")
        status = torch.zeros(1, dtype=torch.int32, device=device())
        y = bsg.grouped_gemm_int8_dynamic(x, w, sw, off, status=status).cpu()
        assert int(status) == bsg.DEV_NONFINITE
        assert bool(y[1].isnan().all()) and bool(y[2].isnan().all()) and bool(y[0].isfinite().all())
        assert bool(y[3:].isfinite().all())


def test_bad_offsets_stay_inside():
    _, _, w, sw, _, _ = _case([10, 10], 64, 128, 8)
    x = torch.randn((20, 128), device=device()).to(torch.bfloat16)
    for bad, bit in (([0, -5, 20], bsg.DEV_NEGATIVE_SIZE), ([0, 10, 500], bsg.DEV_OVER_CAPACITY),
                     ([15, 3, 18], bsg.DEV_NEGATIVE_SIZE)):
        status = torch.zeros(1, dtype=torch.int32, device=device())
        bsg.grouped_gemm_int8_dynamic(x, w, sw, torch.tensor(bad, device=device()), status=status)
        assert int(status) & bit


def test_captured_and_on_two_streams():
    _, _, w, sw, off, ends = _case([6, 0, 10, 40], 1024, 2048, 9)
    xs = [torch.randn((ends[-1], 2048), device=device()).to(torch.bfloat16) for _ in range(2)]
    ws = [bsg.grouped_gemm_int8_dynamic_workspace(ends[-1], 2048) for _ in range(2)]
    want = [bsg.grouped_gemm_int8_dynamic(x, w, sw, off, workspace=ws[0]) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for x, b, s in zip(xs, ws, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(5):
                y = bsg.grouped_gemm_int8_dynamic(x, w, sw, off, workspace=b)
            got.append(y)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = bsg.grouped_gemm_int8_dynamic(x, w, sw, off, workspace=ws[0])
    for i in (1, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        bsg.grouped_gemm_int8_dynamic(xs[1 - i], w, sw, off, workspace=ws[1])
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])


def test_binding_refuses_what_does_not_fit():
    a, sa, w, sw, off, _ = _case([4, 4], 64, 128)
    x = torch.zeros((8, 128), dtype=torch.bfloat16, device=device())
    with pytest.raises(ValueError, match="groups"):
        bsg.grouped_gemm_int8(a, sa, w[:1], sw, off)
    with pytest.raises(ValueError, match="a_scales"):
        bsg.grouped_gemm_int8(a, sa[:7], w, sw, off)
    with pytest.raises(ValueError, match="w_scales"):
        bsg.grouped_gemm_int8(a, sa, w, sw[:1], off)
    with pytest.raises(ValueError, match="int8"):
        bsg.grouped_gemm_int8(x, sa, w, sw, off)
    with pytest.raises(ValueError, match="out"):
        bsg.grouped_gemm_int8(a, sa, w, sw, off, out=torch.zeros((8, 72), device=device()))
    with pytest.raises(ValueError, match="out_dtype"):
        bsg.grouped_gemm_int8(a, sa, w, sw, off, out_dtype=9)
    with pytest.raises(bsg.BsgError):
        bsg.grouped_gemm_int8_dynamic(x, w, sw, off, workspace=torch.empty(1024, dtype=torch.uint8, device=device()))
    with pytest.raises(ValueError, match="contiguous"):
        bsg.grouped_quantize_int8(x.t())
    with pytest.raises(ValueError, match="data"):
        bsg.grouped_quantize_int8(x, data=torch.zeros((8, 64), dtype=torch.int8, device=device()))


def test_many_rows():
    """More rows than one launch has workgroups for (2^23), and a capacity far beyond the live ones."""
    rows = (1 << 23) + 5
    for cols, lo in ((16, 0), (2064, rows - 40)):
        x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=device())
        x[-40:] = torch.randn((40, cols), device=device()).to(torch.bfloat16)
        x[:, 3] = 2.0
        off = torch.tensor([lo, rows], device=device())
        data, scales = bsg.grouped_quantize_int8(x, off)
        _check_quantized(x[-40:], (data[-40:], scales[-40:]))
        if lo == 0:
            assert bool((scales[:-40] == torch.tensor(2.0) / torch.tensor(127.0)).all())
            assert bool((data[:-40, 3] == 127).all()) and int(data[:-40].long().sum()) == 127 * (rows - 40)
        del x, data, scales
