"""The 256 x 256 form of the 16-bit products and the edges of its pipeline: sizes at which the calls take it
(thousands of rows and columns), contractions of one stage, of two, of an odd number and of a last stage that
is not whole, several rounds of tiles, split last rounds, groups without rows between others.

Tolerances as in test_gpu_16bit: L + 1 steps of 2^-23 of the sum of the magnitudes, and the output's rounding."""

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device
from test_gpu_16bit import DTYPES, F64, STEP, TINY, _lora_reference, _offsets, _rand

pytestmark = pytest.mark.gpu


def _dev_rand(seed, shape, dtype, std=1.0):
    gen = torch.Generator(device=device()).manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=device()) * std).to(dtype)


def _reference(mode, a, b, o, c=None):
    """(product, sum of magnitudes) in 64 bits on the device."""
    G = len(o) - 1
    if mode == bsg.BSG_WGRAD_NT:
        ref = torch.zeros((G, a.shape[1], b.shape[1]), dtype=F64, device=a.device)
        mag = torch.zeros_like(ref)
        for g in range(G):
            if o[g + 1] > o[g]:
                x, y = a[o[g]:o[g + 1]].to(F64).T.contiguous(), b[o[g]:o[g + 1]].to(F64)
                ref[g], mag[g] = x @ y, x.abs() @ y.abs()
    else:
        n = b.shape[1] if mode == bsg.BSG_FPROP_TN else b.shape[2]
        ref = torch.zeros((a.shape[0], n), dtype=F64, device=a.device)
        mag = torch.zeros_like(ref)
        for g in range(G):
            w = b[g].to(F64)
            w = w.T.contiguous() if mode == bsg.BSG_FPROP_TN else w
            x = a[o[g]:o[g + 1]].to(F64)
            ref[o[g]:o[g + 1]], mag[o[g]:o[g + 1]] = x @ w, x.abs() @ w.abs()
    if c is not None:
        ref, mag = ref + c.to(F64), mag + c.to(F64).abs()
    return ref, mag


def _assert_close(y, ref, mag, length):
    acc = (length + 1) * STEP * mag
    tol = torch.finfo(y.dtype).eps / 2 * (ref.abs() + acc) + acc + TINY[y.dtype]
    err = (y.to(F64) - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


ROWS = [
    # sizes, n, k: enough rows and columns that the tiles fill the chip
    ([4096], 8192, 64),
    ([8000], 4096, 128),
    ([1, 4047, 0, 4050], 4104, 72),
    ([3500, 0, 3, 4600], 4096, 200),
    ([3000, 3000], 8200, 328),
    ([700, 900, 800, 1800, 1200, 999], 6000, 1000),
    ([2304], 7168, 2056),
]


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mode", [bsg.BSG_FPROP_TN, bsg.BSG_DGRAD_NN])
@pytest.mark.parametrize("case", range(len(ROWS)))
def test_rows(case, mode, dtype, ws):
    sizes, n, k = ROWS[case]
    o, off = _offsets(sizes, 5)
    a = _dev_rand(case, (o[-1] + 7, k), dtype)
    a[:5], a[o[-1]:] = float("nan"), float("nan")
    b = _dev_rand(50 + case, (len(sizes), n, k) if mode == bsg.BSG_FPROP_TN else (len(sizes), k, n), dtype)
    ref, mag = _reference(mode, a, b, o)
    live = slice(o[0], o[-1])
    for f32 in (False, True):
        odt = torch.float32 if f32 else dtype
        out = torch.full((a.shape[0], n + 8), -3.0, dtype=odt, device=a.device)[:, :n]
        bsg.grouped_gemm_16bit(mode, a, b, off, out=out, workspace=bsg.gemm_workspace() if ws else None)
        _assert_close(out[live], ref[live], mag[live], k)
        assert bool((out[:5] == -3.0).all()) and bool((out[o[-1]:] == -3.0).all())
        assert bool((out._base[:, n:] == -3.0).all())


GRADS = [
    # sizes, n, k
    ([64], 4096, 4096),
    ([300, 0, 1000, 0], 4096, 2056),
    ([129, 0, 0, 700, 1, 64], 3080, 4096),
    ([0, 2000, 0], 2304, 4096),
]


@pytest.mark.parametrize("addend", [None, "own", "main"])
@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(GRADS)))
def test_weight_gradients(case, dtype, ws, addend):
    sizes, n, k = GRADS[case]
    o, off = _offsets(sizes, 2)
    a, b = _dev_rand(case, (o[-1] + 3, n), dtype), _dev_rand(20 + case, (o[-1] + 3, k), dtype)
    for t in (a, b):
        t[:2], t[o[-1]:] = float("nan"), float("nan")
    c = None
    if addend is not None:
        c = _dev_rand(40 + case, (len(sizes), n, k), torch.float32 if addend == "main" else dtype, 10.0)
    ref, mag = _reference(bsg.BSG_WGRAD_NT, a, b, o, c)
    work = bsg.gemm_workspace() if ws else None
    y = bsg.grouped_gemm_16bit(bsg.BSG_WGRAD_NT, a, b, off, c=c, workspace=work)
    assert y.dtype == (torch.float32 if addend == "main" else dtype)
    _assert_close(y, ref, mag, max(sizes) + 1)
    again = bsg.grouped_gemm_16bit(bsg.BSG_WGRAD_NT, a, b, off, c=c, out=c, workspace=work)
    assert torch.equal(again, y)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [([900, 1, 1100, 300, 0, 800], [0, 1, -1, 2, 0, 1], 64, 4096, 200),
                                   ([40] * 70, [i % 9 - 1 for i in range(70)], 24, 8192, 328),
                                   ([2600, 1500], [1, 0], 136, 8200, 72)])
def test_adapters(shape, dtype):
    lengths, ids, r, n, k = shape
    count = max(ids) + 1
    gen = torch.Generator().manual_seed(n + r)
    o, off = _offsets(lengths, 3)
    x = _rand(gen, (o[-1] + 4, k), dtype)
    x[:3], x[o[-1]:] = float("nan"), float("nan")
    w = _rand(gen, (n, k), dtype, std=0.1)
    A, B = _rand(gen, (count, r, k), dtype, std=0.2), _rand(gen, (count, n, r), dtype, std=0.5)
    scale = (torch.rand(count, generator=gen) * 3 - 1).to(x.device)
    adapter = torch.tensor(ids, dtype=torch.int32, device=x.device)
    ref, tol = _lora_reference(x, w, A, B, o, ids, scale, dtype)
    live = slice(o[0], o[-1])
    for od, odt in ((None, dtype), (bsg.BSG_OUT_F32, torch.float32)):
        y = bsg.grouped_lora_gemm_16bit(x, w, A, B, off, adapter, scale, out_dtype=od)
        err = (y[live].cpu().to(F64) - ref[live]).abs()
        bound = tol[live] + torch.finfo(odt).eps / 2 * (ref[live].abs() + tol[live]) + TINY[odt]
        assert bool((err <= bound).all()), float((err / bound).max())
    if len(lengths) < 10:  # an adapter of infinities and NaN reaches its own requests only
        A[1], B[1] = float("inf"), float("nan")
        bad = bsg.grouped_lora_gemm_16bit(x, w, A, B, off, adapter, scale, out_dtype=bsg.BSG_OUT_F32)
        for g, ad in enumerate(ids):
            rows = slice(o[g], o[g + 1])
            if ad == 1:
                assert bool(torch.isnan(bad[rows]).all())
            else:
                assert torch.equal(bad[rows], y[rows])


@pytest.mark.parametrize("mode", [bsg.BSG_FPROP_TN, bsg.BSG_DGRAD_NN, bsg.BSG_WGRAD_NT])
def test_repeats_bit_for_bit_and_in_a_graph(mode):
    """The same call twice, with a workspace that holds another call's parts, and as a graph whose offsets change."""
    dt = torch.bfloat16
    sizes = [[1000, 0, 2100, 996], [4096, 0, 0, 0], [1, 1, 4000, 94]]
    n, k = 2304, 2056
    a = _dev_rand(1, (4096, n if mode == bsg.BSG_WGRAD_NT else k), dt)
    b = _dev_rand(2, (4096, k) if mode == bsg.BSG_WGRAD_NT else
                  (4, n, k) if mode == bsg.BSG_FPROP_TN else (4, k, n), dt)
    off = _offsets(sizes[0])[1].clone()
    work = bsg.gemm_workspace()
    out = bsg.grouped_gemm_16bit(mode, a, b, off, workspace=work)
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
        work.fill_(0xFF)
        assert torch.equal(got, bsg.grouped_gemm_16bit(mode, a, b, off, workspace=work))
        assert torch.equal(got, bsg.grouped_gemm_16bit(mode, a, b, off, workspace=work))


def test_rows_20_bits_apart():
    """Rows 2^20 elements apart: the large form's offsets within a tile reach 2^29 bytes."""
    dev = device()
    dt = torch.float16
    T, n, k = 3000, 8192, 136
    o, off = _offsets([1800, 1200])
    a = torch.empty((T, 1 << 20), dtype=dt, device=dev)[:, :k]
    a.copy_(_dev_rand(5, (T, k), dt))
    b = _dev_rand(6, (2, n, k), dt)
    out = torch.empty((T, 1 << 20), dtype=dt, device=dev)[:, :n]
    bsg.grouped_gemm_16bit(bsg.BSG_FPROP_TN, a, b, off, out=out)
    ref, mag = _reference(bsg.BSG_FPROP_TN, a, b, o)
    _assert_close(out, ref, mag, k)
    # the columns of a wide buffer as the contraction's rows: dgrad's second operand
    w = torch.empty((2, k, 1 << 20), dtype=dt, device=dev)[:, :, :n]
    w.copy_(_dev_rand(7, (2, k, n), dt))
    bsg.grouped_gemm_16bit(bsg.BSG_DGRAD_NN, a, w, off, out=out)
    ref, mag = _reference(bsg.BSG_DGRAD_NN, a, w, o)
    _assert_close(out, ref, mag, k)


def test_adapters_of_few_rows_with_a_large_intermediate():
    """x A^T past fp16's largest value where its contraction is spread over workgroups (few rows, k >= 1024)."""
    dev = device()
    x = torch.full((3, 1024), 100.0, dtype=torch.float16, device=dev)
    w = torch.zeros((8, 1024), dtype=torch.float16, device=dev)
    A = torch.full((1, 8, 1024), 0.9375, dtype=torch.float16, device=dev)      # x A^T = 96000
    B = torch.full((1, 8, 8), 2.0 ** -10, dtype=torch.float16, device=dev)
    y = bsg.grouped_lora_gemm_16bit(x, w, A, B, torch.tensor([0, 3], device=dev),
                                    torch.zeros(1, dtype=torch.int32, device=dev), torch.ones(1, device=dev),
                                    out_dtype=bsg.BSG_OUT_F32)
    assert torch.equal(y, torch.full_like(y, 96000 * 8 * 2.0 ** -10))


@pytest.mark.parametrize("rows", [1, 16, 33, 64, 100, 1024, 1025])
def test_adapters_from_one_row_to_more_than_a_thousand(rows):
    """The first product's forms meet at 1024 rows and at k = 1024."""
    gen = torch.Generator().manual_seed(rows)
    n, r = 136, 40
    ids = [i % 3 - 1 for i in range(min(rows, 7))]
    cuts = sorted(torch.randperm(rows + 1, generator=gen)[:len(ids) - 1].tolist())
    lengths = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
    o, off = _offsets(lengths)
    for k in (1016, 1024, 1544):
        x, w = _rand(gen, (rows, k), torch.bfloat16), _rand(gen, (n, k), torch.bfloat16, std=0.1)
        A = _rand(gen, (2, r, k), torch.bfloat16, std=0.1)
        B = _rand(gen, (2, n, r), torch.bfloat16, std=0.5)
        scale = (torch.rand(2, generator=gen) + 0.5).to(x.device)
        y = bsg.grouped_lora_gemm_16bit(x, w, A, B, off, torch.tensor(ids, dtype=torch.int32, device=x.device),
                                        scale, out_dtype=bsg.BSG_OUT_F32)
        ref, tol = _lora_reference(x, w, A, B, o, ids, scale, torch.bfloat16)
        err = (y.cpu().to(F64) - ref).abs()
        bound = tol + 2.0 ** -24 * (ref.abs() + tol) + TINY[torch.float32]
        assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("mode", [bsg.BSG_FPROP_TN, bsg.BSG_DGRAD_NN, bsg.BSG_WGRAD_NT])
def test_two_streams_with_a_workspace_each(mode):
    """Calls on two streams at once, each with its own workspace, give what they give alone."""
    dt = torch.bfloat16
    o, off = _offsets([130, 0, 700, 60])
    T, n, k = o[-1], 520, 1544
    ops = []
    for i in range(2):
        a = _dev_rand(60 + i, (T, n if mode == bsg.BSG_WGRAD_NT else k), dt)
        b = _dev_rand(70 + i, (T, k) if mode == bsg.BSG_WGRAD_NT else
                      (4, n, k) if mode == bsg.BSG_FPROP_TN else (4, k, n), dt)
        work = bsg.gemm_workspace()
        ops.append((a, b, work, bsg.grouped_gemm_16bit(mode, a, b, off, workspace=work)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    got = []
    for _ in range(4):
        for s, (a, b, work, _) in zip(streams, ops):
            with torch.cuda.stream(s):
                got.append(bsg.grouped_gemm_16bit(mode, a, b, off, workspace=work))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, ops[i % 2][3])
