"""grouped_gemm_16bit and grouped_lora_gemm_16bit against the formulas in 64 bits.

Tolerances: a product of two 16-bit values is exact in float32 (bf16: 16 bits, fp16: 22 bits), so a
contraction of length L errs by at most L steps of 2^-23 of the sum of the magnitudes (2^-24 rounded to
nearest, twice that where the matrix unit truncates), and the result is rounded once to the output type
(half a step, finfo.eps / 2, and half of the smallest subnormal)."""

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device

pytestmark = pytest.mark.gpu

F64 = torch.float64
DTYPES = [torch.bfloat16, torch.float16]
MODES = [bsg.BSG_FPROP_TN, bsg.BSG_DGRAD_NN, bsg.BSG_WGRAD_NT]
STEP = 2.0 ** -23
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def _offsets(sizes, first=0):
    o = [first]
    for s in sizes:
        o.append(o[-1] + s)
    return o, torch.tensor(o, dtype=torch.int64, device=device())


def _rand(gen, shape, dtype, std=1.0, gap=0, fill=None):
    """Normal values on the device; gap: rows of a wider buffer, whose other columns hold `fill`."""
    wide = torch.full(shape[:-1] + (shape[-1] + gap,), float("nan") if fill is None else fill, dtype=dtype)
    wide[..., :shape[-1]] = (torch.randn(shape, generator=gen) * std).to(dtype)
    return wide.to(device())[..., :shape[-1]]


def _check(y, ref, mag, length, what=""):
    """y against ref; mag: the sum of the magnitudes of the terms; length: how many terms."""
    y, ref = y.detach().cpu().to(F64), ref.cpu()
    assert torch.equal(torch.isfinite(y), torch.isfinite(ref)), what
    fine = torch.isfinite(ref)
    return y[fine], ref[fine], mag.cpu()[fine], length


def _close(y, ref, mag, length, what=""):
    dt = y.dtype
    half = torch.finfo(dt).eps / 2
    yv, r, m, _ = _check(y, ref, mag, length, what)
    if r.numel() == 0:
        return
    acc = (length + 1) * STEP * m
    tol = half * (r.abs() + acc) + acc + TINY[dt]
    bad = (yv - r).abs() > tol
    assert not bool(bad.any()), (what, int(bad.sum()), float(((yv - r).abs() / tol).max()))


def _product(mode, a, b, o, c=None):
    """(reference, sum of magnitudes, longest contraction) in 64 bits on the host."""
    a, b = a.cpu().to(F64), b.cpu().to(F64)
    G = len(o) - 1
    if mode == bsg.BSG_WGRAD_NT:
        ref = torch.zeros((G, a.shape[1], b.shape[1]), dtype=F64)
        mag = ref.clone()
        for g in range(G):
            x, y = a[o[g]:o[g + 1]], b[o[g]:o[g + 1]]
            ref[g], mag[g] = x.T @ y, x.abs().T @ y.abs()
        length = max(o[g + 1] - o[g] for g in range(G))
    else:
        n = b.shape[1] if mode == bsg.BSG_FPROP_TN else b.shape[2]
        ref = torch.zeros((a.shape[0], n), dtype=F64)
        mag = ref.clone()
        for g in range(G):
            w = b[g].T if mode == bsg.BSG_FPROP_TN else b[g]
            x = a[o[g]:o[g + 1]]
            ref[o[g]:o[g + 1]], mag[o[g]:o[g + 1]] = x @ w, x.abs() @ w.abs()
        length = a.shape[1]
    if c is not None:
        ref = ref + c.cpu().to(F64)
        mag = mag + c.cpu().to(F64).abs()
    return ref, mag, length


def _operands(gen, mode, sizes, n, k, dtype, first=0, dead=0, gap=0):
    rows = first + sum(sizes) + dead
    G = len(sizes)
    if mode == bsg.BSG_WGRAD_NT:
        a = _rand(gen, (rows, n), dtype, gap=gap)
        b = _rand(gen, (rows, k), dtype, gap=gap)
        shape = (G, n, k)
    else:
        a = _rand(gen, (rows, k), dtype, gap=gap)
        b = _rand(gen, (G, n, k) if mode == bsg.BSG_FPROP_TN else (G, k, n), dtype, gap=gap)
        shape = (rows, n)
    for t in (a, b) if mode == bsg.BSG_WGRAD_NT else (a,):
        t[:first] = float("nan")
        t[first + sum(sizes):] = float("nan")
    return a, b, shape


def _live(mode, t, o):
    return t if mode == bsg.BSG_WGRAD_NT else t[o[0]:o[-1]]


CASES = [
    # sizes, n, k
    ([1], 8, 8),
    ([0, 0], 64, 40),
    ([0, 1, 0], 136, 72),
    ([5, 0, 130], 264, 104),
    ([32, 0, 64, 32], 128, 128),
    ([300, 0, 257, 1], 520, 328),
    ([17, 33, 64, 65, 127, 2, 3], 1000, 64),
    ([700], 776, 1032),
    ([1, 2, 3, 4, 5, 6, 7, 8, 9, 0, 1, 1], 256, 2056),
    ([16, 16, 31], 24, 4096),
]


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_product(case, mode, dtype, ws):
    sizes, n, k = CASES[case]
    gen = torch.Generator().manual_seed(100 * case + mode)
    a, b, shape = _operands(gen, mode, sizes, n, k, dtype, first=3 * (case % 2), dead=5 * (case % 3))
    o, off = _offsets(sizes, 3 * (case % 2))
    work = bsg.gemm_workspace() if ws else None
    for out_dtype in (None, bsg.BSG_OUT_F32):
        y = bsg.grouped_gemm_16bit(mode, a, b, off, out_dtype=out_dtype, workspace=work)
        assert tuple(y.shape) == shape
        ref, mag, length = _product(mode, a, b, o)
        _close(_live(mode, y, o), _live(mode, ref, o), _live(mode, mag, o), length, (sizes, n, k))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mode", MODES)
def test_addend_strides_and_untouched_memory(mode, dtype, f32):
    sizes, n, k, first = [70, 0, 300, 9], 200, 136, 4
    gen = torch.Generator().manual_seed(7)
    a, b, shape = _operands(gen, mode, sizes, n, k, dtype, first=first, dead=6, gap=24)
    o, off = _offsets(sizes, first)
    odt = torch.float32 if f32 else dtype
    c = _rand(gen, shape, odt, std=10.0, gap=16, fill=3.0)
    ref, mag, length = _product(mode, a, b, o, c)
    work = bsg.gemm_workspace()
    out = _rand(gen, shape, odt, gap=16, fill=5.0)
    out[...] = -77.0
    y = bsg.grouped_gemm_16bit(mode, a, b, off, c=c, out=out, workspace=work,
                               out_dtype=bsg.BSG_OUT_F32 if f32 else None)
    assert y is out
    _close(_live(mode, y, o), _live(mode, ref, o), _live(mode, mag, o), length + 1)
    base = out._base
    assert bool((base[..., shape[-1]:] == 5.0).all())          # the gap between rows
    if mode != bsg.BSG_WGRAD_NT:
        assert bool((out[:first] == -77.0).all()) and bool((out[o[-1]:] == -77.0).all())
    # the same into c itself
    first_y = y.clone()
    bsg.grouped_gemm_16bit(mode, a, b, off, c=c, out=c, workspace=work,
                           out_dtype=bsg.BSG_OUT_F32 if f32 else None)
    assert torch.equal(_live(mode, c, o), _live(mode, first_y, o))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mode", MODES)
def test_infinities_and_nan_stay_in_their_group(mode, dtype):
    sizes, n, k = [40, 300, 31], 264, 200
    gen = torch.Generator().manual_seed(8)
    a, b, _ = _operands(gen, mode, sizes, n, k, dtype)
    o, off = _offsets(sizes)
    a[o[1]:o[2]] = float("inf")                                  # group 1's rows
    if mode == bsg.BSG_WGRAD_NT:
        b[o[1]:o[2]] = float("nan")
    else:
        b[1] = float("nan")
    y = bsg.grouped_gemm_16bit(mode, a, b, off, workspace=bsg.gemm_workspace())
    ref, mag, length = _product(mode, a, b, o)
    if mode == bsg.BSG_WGRAD_NT:
        pick = [(y[g], ref[g], mag[g]) for g in (0, 2)]
        assert bool(torch.isnan(y[1]).all())
    else:
        pick = [(y[o[g]:o[g + 1]], ref[o[g]:o[g + 1]], mag[o[g]:o[g + 1]]) for g in (0, 2)]
        assert bool(torch.isnan(y[o[1]:o[2]]).all())
    for t in pick:
        _close(*t, length)


@pytest.mark.parametrize("dtype", DTYPES)
def test_offsets_past_32_bits(dtype):
    """Rows 2^20 elements apart and groups 2^30 elements apart: both operands span more than 2^32 bytes."""
    dev = device()
    gen = torch.Generator().manual_seed(9)
    n, k, sizes = 72, 64, [2000, 40, 1500]
    o, off = _offsets(sizes)
    a = torch.empty((o[-1], 1 << 20), dtype=dtype, device=dev)[:, :k]
    a.copy_((torch.randn((o[-1], k), generator=gen)).to(dtype))
    b = torch.empty((3, 1 << 30), dtype=dtype, device=dev)[:, :n * k].view(3, n, k)
    b.copy_(torch.randn((3, n, k), generator=gen).to(dtype))
    out = torch.empty((o[-1], 1 << 20), dtype=dtype, device=dev)[:, :n]
    y = bsg.grouped_gemm_16bit(bsg.BSG_FPROP_TN, a, b, off, out=out)
    ref, mag, length = _product(bsg.BSG_FPROP_TN, a, b, o)
    _close(y, ref, mag, length)
    w = bsg.grouped_gemm_16bit(bsg.BSG_WGRAD_NT, y, a, off, workspace=bsg.gemm_workspace())
    ref, mag, length = _product(bsg.BSG_WGRAD_NT, y, a, o)
    _close(w, ref, mag, length)


@pytest.mark.parametrize("mode", MODES)
def test_bad_offsets_stay_in_bounds(mode):
    """Offsets that decrease, are negative or run past the rows are clamped and flagged."""
    dev = device()
    gen = torch.Generator().manual_seed(10)
    a, b, _ = _operands(gen, mode, [50, 50], 64, 64, torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    for bad, bit in (([0, 50, 4000], bsg.DEV_OVER_CAPACITY), ([-9, 50, 100], bsg.DEV_NEGATIVE_SIZE),
                     ([0, 90, 30], bsg.DEV_NEGATIVE_SIZE)):
        status.zero_()
        bsg.grouped_gemm_16bit(mode, a, b, torch.tensor(bad, device=dev), status=status,
                               workspace=bsg.gemm_workspace())
        assert int(status) & bit


@pytest.mark.parametrize("mode", MODES)
def test_graph_replays_and_other_stream(mode):
    """A captured call follows the sizes that its offsets hold at each replay, and equals the eager call."""
    dev = device()
    gen = torch.Generator().manual_seed(11)
    sizes = [[100, 60, 96], [256, 0, 0], [0, 1, 255]]
    a, b, shape = _operands(gen, mode, sizes[0], 264, 712, torch.bfloat16)
    off = _offsets(sizes[0])[1].clone()
    work = bsg.gemm_workspace()
    out = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bsg.grouped_gemm_16bit(mode, a, b, off, out=out, workspace=work)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsg.grouped_gemm_16bit(mode, a, b, off, out=out, workspace=work)
    for s in sizes + sizes:
        off.copy_(_offsets(s)[1])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        eager = bsg.grouped_gemm_16bit(mode, a, b, off, workspace=work)
        o = _offsets(s)[0]
        assert torch.equal(_live(mode, got, o), _live(mode, eager, o))


# ---------------------------------------------------------------- adapters


def _lora_reference(x, w, A, B, o, ids, scale, dtype):
    """(reference, tolerance before the output's rounding) in 64 bits."""
    x, w, A, B, scale = (t.cpu().to(F64) for t in (x, w, A, B, scale))
    k, r = A.shape[2], A.shape[1]
    ref, mag = x @ w.T, x.abs() @ w.abs().T
    tol = (k + 2 * r + 2) * STEP * mag
    # the two 16-bit values of a scaled x A^T miss it by a half step of a half step, or by half of the
    # smallest subnormal
    half = torch.finfo(dtype).eps / 2
    for g, ad in enumerate(ids):
        if not 0 <= ad < A.shape[0]:
            continue
        rows = slice(o[g], o[g + 1])
        low, lmag = x[rows] @ A[ad].T * scale[ad], x[rows].abs() @ A[ad].abs().T * scale[ad].abs()
        lerr = (k + 2) * STEP * lmag + half * half * lmag + TINY[dtype]
        ref[rows] += low @ B[ad].T
        tol[rows] += lerr @ B[ad].abs().T + (k + 2 * r + 4) * STEP * ((lmag + lerr) @ B[ad].abs().T)
    return ref, tol


LORA_CASES = [
    # lengths, adapters of the requests, adapters, rank, n, k
    ([1], [0], 1, 8, 8, 8),
    ([1], [2], 3, 16, 4096, 1032),
    ([1], [-1], 3, 16, 264, 512),
    ([0, 3, 0], [1, 1, 0], 2, 24, 136, 72),
    ([1] * 48, [i % 7 - 1 for i in range(48)], 6, 32, 520, 640),
    ([200, 1, 1, 77, 0, 300], [3, 0, -1, 0, 2, 3], 4, 64, 328, 200),
    ([130, 130], [1, 1], 2, 128, 264, 2048),
    ([9, 500], [0, 1], 2, 256, 776, 128),
    ([1] * 256, [i % 64 for i in range(256)], 64, 16, 128, 264),
    ([40, 2, 30], [0, 1, 0], 2, 40, 1000, 328),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(LORA_CASES)))
def test_lora(case, dtype):
    dev = device()
    lengths, ids, count, r, n, k = LORA_CASES[case]
    gen = torch.Generator().manual_seed(200 + case)
    first, dead = 2 * (case % 2), 3 * (case % 3)
    o, off = _offsets(lengths, first)
    x = _rand(gen, (o[-1] + dead, k), dtype, gap=8 * (case % 2))
    x[:first] = float("nan")
    x[o[-1]:] = float("nan")
    w = _rand(gen, (n, k), dtype, std=0.1, gap=16 * (case % 2))
    A, B = _rand(gen, (count, r, k), dtype, std=0.2), _rand(gen, (count, n, r), dtype, std=0.5)
    scale = (torch.rand(count, generator=gen) * 3 - 1).to(dev)
    adapter = torch.tensor(ids, dtype=torch.int32, device=dev)
    ref, tol = _lora_reference(x, w, A, B, o, ids, scale, dtype)
    live = slice(o[0], o[-1])
    for od, odt in ((None, dtype), (bsg.BSG_OUT_F32, torch.float32)):
        out = torch.full((x.shape[0], n + 8), -7.0, dtype=odt, device=dev)[:, :n]
        y = bsg.grouped_lora_gemm_16bit(x, w, A, B, off, adapter, scale, out=out, out_dtype=od)
        got = y[live].cpu().to(F64)
        bound = tol[live] + torch.finfo(odt).eps / 2 * (ref[live].abs() + tol[live]) + TINY[odt]
        bad = (got - ref[live]).abs() > bound
        assert not bool(bad.any()), float(((got - ref[live]).abs() / bound).max())
        assert bool((out[:first] == -7.0).all()) and bool((out[o[-1]:] == -7.0).all())
        assert bool((out._base[:, n:] == -7.0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths", [[20, 1, 11, 40], [1, 1, 1, 1], [300, 200, 5, 300]])
def test_lora_adapters_do_not_reach_other_requests(lengths, dtype):
    """An adapter of infinities and NaN changes its own requests' rows only, and an index out of range is none."""
    dev = device()
    gen = torch.Generator().manual_seed(12)
    o, off = _offsets(lengths)
    k, n, r = 136, 264, 16
    x, w = _rand(gen, (o[-1], k), dtype), _rand(gen, (n, k), dtype)
    A, B = _rand(gen, (2, r, k), dtype), _rand(gen, (2, n, r), dtype)
    scale = torch.ones(2, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    ids = torch.tensor([0, 1, -1, 9], dtype=torch.int32, device=dev)
    clean = bsg.grouped_lora_gemm_16bit(x, w, A, B, off, ids, scale, status=status)
    assert int(status) == bsg.DEV_BAD_ADAPTER
    A[1], B[1] = float("inf"), float("nan")
    y = bsg.grouped_lora_gemm_16bit(x, w, A, B, off, ids, scale)
    keep = torch.ones(o[-1], dtype=torch.bool, device=dev)
    keep[o[1]:o[2]] = False
    assert torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[~keep]).all())


def test_lora_large_intermediate_fp16():
    """x A^T past fp16's largest value, up to twice of it, is still held by the two parts."""
    dev = device()
    x = torch.full((3, 64), 100.0, dtype=torch.float16, device=dev)
    w = torch.zeros((8, 64), dtype=torch.float16, device=dev)
    A = torch.full((1, 8, 64), 15.0, dtype=torch.float16, device=dev)      # x A^T = 96000
    B = torch.full((1, 8, 8), 2.0 ** -10, dtype=torch.float16, device=dev)
    off = torch.tensor([0, 3], device=dev)
    y = bsg.grouped_lora_gemm_16bit(x, w, A, B, off, torch.zeros(1, dtype=torch.int32, device=dev),
                                    torch.ones(1, device=dev), out_dtype=bsg.BSG_OUT_F32)
    assert torch.equal(y, torch.full_like(y, 96000 * 8 * 2.0 ** -10))


def test_lora_graph_replays():
    dev = device()
    gen = torch.Generator().manual_seed(13)
    o, off = _offsets([1, 1, 60, 2])
    k, n, r = 520, 264, 16
    dt = torch.bfloat16
    x, w = _rand(gen, (64, k), dt), _rand(gen, (n, k), dt)
    A, B = _rand(gen, (3, r, k), dt), _rand(gen, (3, n, r), dt)
    scale = torch.ones(3, device=dev)
    ids = torch.tensor([0, 1, 2, -1], dtype=torch.int32, device=dev)
    ws = bsg.grouped_lora_gemm_16bit_workspace(64, n, k, r)
    out = torch.zeros((64, n), dtype=dt, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bsg.grouped_lora_gemm_16bit(x, w, A, B, off, ids, scale, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsg.grouped_lora_gemm_16bit(x, w, A, B, off, ids, scale, out=out, workspace=ws)
    for lengths, new in (([1, 1, 60, 2], [0, 1, 2, -1]), ([10, 20, 30, 4], [2, 2, 0, 1]),
                         ([64, 0, 0, 0], [1, 0, 0, 0])):
        off.copy_(_offsets(lengths)[1])
        ids.copy_(torch.tensor(new, dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, bsg.grouped_lora_gemm_16bit(x, w, A, B, off, ids, scale))


def test_lora_gradients_are_grouped_products():
    """dX, dA and dB of the adapted projection from grouped_gemm_16bit, against the formulas and against
    differences of the loss in 64 bits."""
    dev = device()
    gen = torch.Generator().manual_seed(14)
    dt = torch.bfloat16
    o, off = _offsets([60, 0, 37])
    k, n, r, T = 136, 72, 16, 97
    x, dy = _rand(gen, (T, k), dt), _rand(gen, (T, n), dt)
    A, B = _rand(gen, (3, r, k), dt), _rand(gen, (3, n, r), dt)
    low = bsg.grouped_gemm_16bit(bsg.BSG_FPROP_TN, x, A, off)                   # x A^T
    dlow = bsg.grouped_gemm_16bit(bsg.BSG_DGRAD_NN, dy, B, off)                 # dy B
    dB = bsg.grouped_gemm_16bit(bsg.BSG_WGRAD_NT, dy, low, off, out_dtype=bsg.BSG_OUT_F32)
    dA = bsg.grouped_gemm_16bit(bsg.BSG_WGRAD_NT, dlow, x, off, out_dtype=bsg.BSG_OUT_F32)
    for got, (p, q) in ((dB, (dy, low)), (dA, (dlow, x))):
        ref, mag, length = _product(bsg.BSG_WGRAD_NT, p, q, o)
        _close(got, ref, mag, length)
    assert bool((dA[1] == 0).all()) and bool((dB[1] == 0).all())
    # the loss sum(dy * (x A^T) B^T) is linear in A and in B: its differences are its derivatives.  The
    # 16-bit roundings of low and dlow are half a step each.
    xd, dyd, Ad, Bd = (t.cpu().to(F64) for t in (x, dy, A, B))
    half = torch.finfo(dt).eps / 2
    for g in (0, 2):
        rows = slice(o[g], o[g + 1])
        low64, dlow64 = xd[rows] @ Ad[g].T, dyd[rows] @ Bd[g]

        def loss(A1, B1):
            return float((dyd[rows] * (xd[rows] @ A1.T @ B1.T)).sum())

        for i, j in ((0, 0), (5, 3), (r - 1, 7)):
            step = torch.zeros_like(Ad[g])
            step[i, j] = 0.5
            diff = loss(Ad[g] + step, Bd[g]) - loss(Ad[g] - step, Bd[g])
            bound = (2 * half) * float((dlow64[:, i].abs() * xd[rows][:, j].abs()).sum()) + \
                (n + T) * STEP * float(((dyd[rows].abs() @ Bd[g].abs())[:, i] * xd[rows][:, j].abs()).sum())
            assert abs(float(dA[g, i, j]) - diff) <= bound
            step = torch.zeros_like(Bd[g])
            step[j, i] = 0.5
            diff = loss(Ad[g], Bd[g] + step) - loss(Ad[g], Bd[g] - step)
            bound = (2 * half) * float((low64[:, i].abs() * dyd[rows][:, j].abs()).sum()) + \
                (k + T) * STEP * float(((xd[rows].abs() @ Ad[g].abs().T)[:, i] * dyd[rows][:, j].abs()).sum())
            assert abs(float(dB[g, j, i]) - diff) <= bound
