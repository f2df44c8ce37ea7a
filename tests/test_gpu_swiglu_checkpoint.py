"""The gated activation with its 8-bit checkpoint, forward and backward, against the formulas in 64 bits.

Tolerances.  sigmoid: exp(-g) from an exponent rounded twice (relative error (|g| + 2) 2^-23), one sum, one
reciprocal to two steps: (|g| + 6) 2^-23 of itself, and by 2^-126 where it underflows.  What follows is at most six
products and sums, so (|g| + 16) 2^-23 of the sum of the terms' magnitudes, and one rounding to the type.  What is
kept is exact."""

import math

import numpy as np
import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device

pytestmark = pytest.mark.gpu

F64 = torch.float64
STEP = 2.0 ** -23
DTYPES = [torch.bfloat16, torch.float16]
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def _kept(h):
    """(E4M3 values, scale bytes) of rows in 64 bits."""
    h = h.cpu().to(F64)
    blocks = h.view(h.shape[0], -1, 32)
    top = blocks.abs().amax(2)
    byte = torch.where(top > 0, (torch.frexp(top).exponent - 1 - 8 + 127).clamp(min=0), 0)
    v = blocks * torch.exp2(127.0 - byte.to(F64))[:, :, None]
    step = torch.exp2((torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent - 1 - 3).to(F64))
    q = (torch.round(v / step) * step).clamp(-448, 448)
    return q.view(h.shape), byte.to(torch.uint8)


def _decoded(data, scales):
    d = data.cpu().view(torch.float8_e4m3fn).to(torch.float32).to(F64)
    s = torch.exp2(scales.cpu().to(F64) - 127)
    return (d.view(d.shape[0], -1, 32) * s[:, :, None]).view(d.shape)


def _close(y, want, mag, g, what=""):
    """mag: the sum of the terms' magnitudes, with 1 for a sigmoid in the place of one that underflows."""
    acc = (g.abs() + 16) * STEP * want.abs() + (g.abs() + 16) * STEP * mag[0] + 2.0 ** -124 * mag[1]
    tol = torch.finfo(y.dtype).eps / 2 * (want.abs() + acc) + acc + TINY[y.dtype]
    err = (y.cpu().to(F64) - want).abs()
    assert bool((err <= tol).all()), (what, float((err / tol).max()))


def _wide(v, gap, fill=float("nan")):
    out = torch.full((v.shape[0], v.shape[1] + gap), fill, dtype=v.dtype)
    out[:, :v.shape[1]] = v
    return out.to(device())[:, :v.shape[1]]


def _h(rows, f, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    v = torch.randn((rows, 2 * f), generator=gen) * 2
    v = torch.where(torch.rand((rows, 2 * f), generator=gen) < 0.01, v * 20, v)
    v[torch.rand((rows, 2 * f), generator=gen) < 0.02] = 0.0
    return v.to(dtype)


SHAPES = [(1, 32), (3, 64), (5, 96), (130, 128), (17, 480), (40, 512), (9, 544), (33, 1024), (20, 1056), (6, 2080),
          (4, 7168), (700, 160)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,f", SHAPES)
def test_forward(dtype, rows, f):
    for weighted, first, dead, gap in ((False, 0, 0, 0), (True, 2, 3, 8)):
        h = _h(rows + first + dead, f, dtype, rows + f)
        h[:first], h[first + rows:] = float("nan"), float("nan")
        w = torch.rand(h.shape[0], generator=torch.Generator().manual_seed(1)).to(device()) if weighted else None
        off = torch.tensor([first, first, first + rows // 2, first + rows], device=device())
        total = h.shape[0]
        out = torch.full((total, f + gap), 7.0, dtype=dtype, device=device())
        data = torch.full((total, 2 * f), 0xAB, dtype=torch.uint8, device=device())
        scales = torch.full((total, f // 16), 0xAB, dtype=torch.uint8, device=device())
        status = torch.zeros(1, dtype=torch.int32, device=device())
        bsg.grouped_swiglu_checkpoint_mxfp8(_wide(h, gap), off, row_weights=w, out=out[:, :f], data=data,
                                            scales=scales, status=status)
        assert int(status) == 0
        live = slice(first, first + rows)
        q, byte = _kept(h[live])
        assert torch.equal(scales[live].cpu(), byte)
        assert torch.equal(data[live].cpu().view(torch.float8_e4m3fn).to(torch.float32).to(F64), q)
        x = h[live].to(F64)
        g, u = x[:, :f], x[:, f:]
        wt = w.cpu().to(F64)[live, None] if weighted else 1.0
        want = wt * g * torch.sigmoid(g) * u
        _close(out[live, :f], want, (0.0, (wt * g * u).abs()), g)
        for t, fill in ((out, 7), (data, 0xAB), (scales, 0xAB)):
            assert bool((t[:first] == fill).all()) and bool((t[first + rows:] == fill).all())
        assert bool((out[:, f:] == 7).all())
        # without a checkpoint: the same activation
        y, d, s = bsg.grouped_swiglu_checkpoint_mxfp8(_wide(h, gap), off, row_weights=w, keep=False)
        assert d is None and s is None and torch.equal(y[live], out[live, :f])


@pytest.mark.parametrize("rows,f", [(64, 128), (33, 1056)])
def test_checkpoint_is_the_rowwise_quantize(rows, f):
    """bf16: the bytes of grouped_quantize_mxfp8."""
    h = _h(rows, f, torch.bfloat16, 3).to(device())
    off = torch.tensor([0, rows], device=device())
    _, data, scales = bsg.grouped_swiglu_checkpoint_mxfp8(h, off)
    q = bsg.grouped_quantize_mxfp8(h, off)
    assert torch.equal(data, q["row_data"].view(torch.uint8).view(rows, 2 * f))
    words = q["row_scales"].view(torch.uint8).reshape(-1)[: (2 * f + 127) // 128 * rows * 4]
    words = words.view(-1, rows, 4)[:, :, [0, 2, 1, 3]]   # a word holds b0, b2, b1, b3
    assert torch.equal(scales, words.permute(1, 0, 2).reshape(rows, -1)[:, : f // 16])


def _reference_backward(data, scales, dy, w, f):
    h = _decoded(data, scales)
    g, u, d = h[:, :f], h[:, f:], dy.cpu().to(F64)
    wt = w.cpu().to(F64)[:, None] if w is not None else torch.ones((h.shape[0], 1), dtype=F64)
    s = torch.sigmoid(g)
    return dict(g=g, u=u, d=d, wt=wt, s=s, dg=d * wt * u * s * (1 + g * (1 - s)), du=d * wt * g * s,
                dw=(d * g * s * u).sum(1), y=wt * g * s * u)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,f", SHAPES)
def test_backward(dtype, rows, f):
    for weighted, recompute, first, dead, gap in ((False, False, 0, 0, 0), (True, True, 2, 3, 8), (True, False, 0, 1, 0),
                                                  (False, True, 1, 0, 0)):
        total = rows + first + dead
        _, data, scales = bsg.grouped_swiglu_checkpoint_mxfp8(
            _h(total, f, dtype, rows + f).to(device()), torch.tensor([0, total], device=device()))
        gen = torch.Generator().manual_seed(2)
        dy = (torch.randn((total, f), generator=gen) * 0.1).to(dtype)
        dy[:first], dy[first + rows:] = float("nan"), float("nan")
        w = torch.rand(total, generator=gen).to(device()) if weighted else None
        off = torch.tensor([first, first + rows // 3, first + rows], device=device())
        dh = torch.full((total, 2 * f + gap), 7.0, dtype=dtype, device=device())
        y = torch.full((total, f + gap), 7.0, dtype=dtype, device=device()) if recompute else None
        dw = torch.full((total,), 7.0, device=device()) if weighted else None
        _, gotw, _ = bsg.grouped_swiglu_checkpoint_mxfp8_backward(
            data, scales, _wide(dy, gap), off, row_weights=w, d_h=dh[:, :2 * f], d_row_weights=dw,
            out=None if y is None else y[:, :f])
        live = slice(first, first + rows)
        r = _reference_backward(data[live], scales[live], dy[live], None if w is None else w[live], f)
        dmag = (r["d"] * r["wt"]).abs()
        _close(dh[live, :f], r["dg"], (dmag * r["u"].abs() * r["s"] * (1 + r["g"].abs()), dmag * r["u"].abs()
                                       * (1 + r["g"].abs())), r["g"], "dg")
        _close(dh[live, f:2 * f], r["du"], (0.0, dmag * r["g"].abs()), r["g"], "du")
        if recompute:
            _close(y[live, :f], r["y"], (0.0, (r["wt"] * r["g"] * r["u"]).abs()), r["g"], "y")
            assert bool((y[:first] == 7).all()) and bool((y[first + rows:] == 7).all()) and bool((y[:, f:] == 7).all())
        if weighted:
            assert gotw is dw
            mag = (r["d"] * r["g"] * r["s"] * r["u"]).abs()
            # a lane adds 8 (f / 512 + 1) terms, then 6 + 4 sums
            tol = ((r["g"].abs() + 30 + f / 64) * STEP * mag).sum(1) + 2.0 ** -120
            assert bool(((dw[live].cpu().to(F64) - r["dw"]).abs() <= tol).all())
            assert bool((dw[:first] == 7).all()) and bool((dw[first + rows:] == 7).all())
        assert bool((dh[:first] == 7).all()) and bool((dh[first + rows:] == 7).all()) and bool((dh[:, 2 * f:] == 7).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_code_and_scale(dtype):
    """Every E4M3 code but NaN at every scale that the forward pass writes comes back exactly: with g = 64 (whose
    sigmoid is 1) and a weight of 1/64 the activation is u itself."""
    codes = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8)
    codes = torch.cat([codes, codes[:2]])                       # 256 columns
    top = 247 if dtype == torch.bfloat16 else 135
    byte = torch.arange(0, top, dtype=torch.uint8)
    rows, f = len(byte), 256
    data = torch.empty((rows, 2 * f), dtype=torch.uint8)
    data[:, :f] = torch.tensor([64.0]).to(torch.float8_e4m3fn).view(torch.uint8)
    data[:, f:] = codes
    scales = torch.empty((rows, f // 16), dtype=torch.uint8)
    scales[:, :f // 32] = 127
    scales[:, f // 32:] = byte[:, None]
    _, _, y = bsg.grouped_swiglu_checkpoint_mxfp8_backward(
        data.to(device()), scales.to(device()), torch.zeros((rows, f), dtype=dtype, device=device()),
        torch.tensor([0, rows], device=device()), row_weights=torch.full((rows,), 1 / 64, device=device()),
        recompute=True)
    want = _decoded(data[:, f:].contiguous(), scales[:, f // 32:].contiguous()).to(dtype)
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_extreme_values(dtype):
    """Gates far out on both sides, subnormal numbers, the type's largest; and values that are not finite, which
    saturate in the checkpoint, set the status bit and reach the activation."""
    big = torch.finfo(dtype).max
    f = 64
    g = torch.tensor([0.0, -0.0, 1e-6, -1e-6, 20.0, -20.0, 88.0, -88.0, -89.0, -104.0, -150.0, 300.0, -3e4, 3e4, big, -big,
                      torch.finfo(dtype).smallest_normal, 1.0]).to(dtype)
    h = torch.zeros((len(g), 2 * f), dtype=dtype)
    h[:, :f] = g[:, None]
    h[:, f:] = torch.tensor([1.0, -0.25], dtype=dtype).repeat(f // 2)
    off = torch.tensor([0, len(g)], device=device())
    status = torch.zeros(1, dtype=torch.int32, device=device())
    y, data, scales = bsg.grouped_swiglu_checkpoint_mxfp8(h.to(device()), off, status=status)
    x = h.to(F64)
    want = x[:, :f] * torch.sigmoid(x[:, :f]) * x[:, f:]
    _close(y, want, (0.0, (x[:, :f] * x[:, f:]).abs()), x[:, :f].clamp(-150, 150))
    assert int(status) == 0
    q, byte = _kept(h)
    assert torch.equal(scales.cpu(), byte) and torch.equal(_decoded(data, scales), q * torch.exp2(
        byte.to(F64) - 127).repeat_interleave(32, 1))
    dy = torch.ones((len(g), f), dtype=dtype, device=device())
    dh, _, _ = bsg.grouped_swiglu_checkpoint_mxfp8_backward(data, scales, dy, off)
    assert bool(dh.isfinite().all())
    for bad in (math.nan, math.inf):
        x = h.clone()
        x[3, 5] = bad
        y, data, scales = bsg.grouped_swiglu_checkpoint_mxfp8(x.to(device()), off, status=status)
        assert int(status) == bsg.DEV_NONFINITE and not bool(y[3, 5].isfinite())
        assert bool(y[4:].isfinite().all())
        status.zero_()


def test_backward_against_differences():
    """Differences, step 2^-8, of sum(dy y) in 64 bits at the kept values; float32's rounding of the bf16 result is
    half a step of 2^-8 of it."""
    rows, f, e = 3, 32, 2.0 ** -8
    h = _h(rows, f, torch.bfloat16, 9).clamp(-8, 8)
    off = torch.tensor([0, rows], device=device())
    w = torch.rand(rows) + 0.5
    _, data, scales = bsg.grouped_swiglu_checkpoint_mxfp8(h.to(device()), off)
    dy = torch.randn((rows, f)).to(torch.bfloat16)
    dh, dw, _ = bsg.grouped_swiglu_checkpoint_mxfp8_backward(data, scales, dy.to(device()), off,
                                                             row_weights=w.to(device()))
    x = _decoded(data, scales)

    def terms(x, w):
        return dy.to(F64) * w.to(F64)[:, None] * x[:, :f] * torch.sigmoid(x[:, :f]) * x[:, f:]

    up, down = x.clone(), x.clone()
    up[:, :f] += e
    down[:, :f] -= e
    dg = (terms(up, w) - terms(down, w)) / (2 * e)
    up, down = x.clone(), x.clone()
    up[:, f:] += e
    down[:, f:] -= e
    du = (terms(up, w) - terms(down, w)) / (2 * e)
    want = torch.cat([dg, du], 1)
    # the third derivative of g s(g) is under 1
    bound = want.abs() * 2.0 ** -8 + e * e * (dy.to(F64).abs() * w.to(F64)[:, None] * x[:, f:].abs()).repeat(1, 2) + 1e-5
    assert bool(((dh.cpu().to(F64) - want).abs() <= bound).all())
    wdiff = (terms(x, w + e) - terms(x, w - e)).sum(1) / (2 * e)
    # w + e in float32
    assert bool(((dw.cpu().to(F64) - wdiff).abs() <= 1e-4 * terms(x, torch.ones(rows)).abs().sum(1) + 1e-6).all())


def test_bad_offsets_stay_inside():
    h = _h(20, 64, torch.bfloat16, 1).to(device())
    for bad, bit in (([-4, 20], bsg.DEV_NEGATIVE_SIZE), ([0, 300], bsg.DEV_OVER_CAPACITY), ([15, 4], bsg.DEV_NEGATIVE_SIZE),
                     ([50, 60], bsg.DEV_OVER_CAPACITY)):
        off = torch.tensor(bad, device=device())
        status = torch.zeros(1, dtype=torch.int32, device=device())
        y, data, scales = bsg.grouped_swiglu_checkpoint_mxfp8(h, off, status=status)
        assert int(status) & bit
        status.zero_()
        bsg.grouped_swiglu_checkpoint_mxfp8_backward(data, scales, y, off, row_weights=torch.ones(20, device=device()),
                                                     status=status)
        assert int(status) & bit


def test_captured():
    hs = [_h(300, 1056, torch.bfloat16, s).to(device()) for s in (1, 2)]
    off = torch.tensor([0, 100, 300], device=device())
    w = torch.rand(300, device=device())
    dy = torch.randn((300, 1056), device=device()).to(torch.bfloat16)

    def step(h):
        y, data, scales = bsg.grouped_swiglu_checkpoint_mxfp8(h, off, row_weights=w)
        return (y, data, scales) + bsg.grouped_swiglu_checkpoint_mxfp8_backward(data, scales, dy, off, row_weights=w,
                                                                               recompute=True)

    want = [step(h) for h in hs]
    h = hs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(h)
    for i in (1, 0, 1):
        h.copy_(hs[i])
        graph.replay()
        step(hs[1 - i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))


def test_binding_refuses_what_does_not_fit():
    h = torch.zeros((8, 128), dtype=torch.bfloat16, device=device())
    off = torch.tensor([0, 8], device=device())
    with pytest.raises(ValueError, match="columns"):
        bsg.grouped_swiglu_checkpoint_mxfp8(h[:, :96], off)
    with pytest.raises(ValueError, match="row_weights"):
        bsg.grouped_swiglu_checkpoint_mxfp8(h, off, row_weights=torch.ones(7, device=device()))
    with pytest.raises(ValueError, match="scales"):
        bsg.grouped_swiglu_checkpoint_mxfp8(h, off, scales=torch.zeros((8, 3), dtype=torch.uint8, device=device()))
    y, data, scales = bsg.grouped_swiglu_checkpoint_mxfp8(h, off)
    with pytest.raises(ValueError, match="data"):
        bsg.grouped_swiglu_checkpoint_mxfp8_backward(data[:4], scales, y, off)
    with pytest.raises(ValueError, match="d_h"):
        bsg.grouped_swiglu_checkpoint_mxfp8_backward(data, scales, y, off, d_h=y)
    assert np.prod(scales.shape) == 8 * 4


def test_many_rows():
    """More rows than one launch has workgroups for: workgroups take several blocks of rows."""
    rows, f = (1 << 24) + 100, 32
    h = torch.zeros((rows, 2 * f), dtype=torch.bfloat16, device=device())
    h[:, 1], h[:, f + 1] = 2.0, 4.0
    h[-9:] = _h(9, f, torch.bfloat16, 5).to(device())
    w = torch.full((rows,), 0.5, device=device())
    off = torch.tensor([0, rows], device=device())
    y, data, scales = bsg.grouped_swiglu_checkpoint_mxfp8(h, off, row_weights=w)
    one = float((0.5 * 2 * torch.sigmoid(torch.tensor(2.0)) * 4).to(torch.bfloat16))
    assert bool((y[:-9, 1] == one).all()) and bool((y[:-9, 2:] == 0).all())
    dy = torch.ones((rows, f), dtype=torch.bfloat16, device=device())
    dh, dw, _ = bsg.grouped_swiglu_checkpoint_mxfp8_backward(data, scales, dy, off, row_weights=w)
    r = _reference_backward(data[-9:], scales[-9:], dy[-9:], w[-9:], f)
    mag = (r["d"] * r["g"] * r["s"] * r["u"]).abs()
    assert bool(((dw[-9:].cpu().to(F64) - r["dw"]).abs() <= ((r["g"].abs() + 31) * STEP * mag).sum(1) + 1e-30).all())
    assert bool((dw[:-9] == dw[0]).all()) and abs(float(dw[0]) - float(8 * torch.sigmoid(torch.tensor(2.0)))) < 1e-5
    assert bool((dh[:-9] == dh[0]).all())
