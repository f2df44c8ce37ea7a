"""Calls whose outputs are large enough for stores past the caches: each gives, bit for bit, what
calls of parts of its rows give (which are small enough for cached stores)."""
import pytest

import block_scaled_grouped_amd as bsg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROWS, PARTS = 26000, 4  # 4096 columns: 102 MiB of bytes, 25 MiB a part


def _tokens(dtype, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(ROWS, cols, generator=g, device="cuda").to(dtype)


def _parts():
    step = ROWS // PARTS
    return [slice(i * step, (i + 1) * step) for i in range(PARTS)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("cols", [4080, 4096, 4112])
def test_quantize_int8(dtype, cols):
    x = _tokens(getattr(torch, dtype), cols, cols)
    data, scales = bsg.grouped_quantize_int8(x)
    for part in _parts():
        d, s = bsg.grouped_quantize_int8(x[part])
        assert torch.equal(data[part], d) and torch.equal(scales[part], s)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("f", [2048, 2080])
def test_swiglu_checkpoint(dtype, f):
    dtype = getattr(torch, dtype)
    h, dy = _tokens(dtype, 2 * f, f), _tokens(dtype, f, f + 1)
    w = torch.rand(ROWS, device="cuda")
    off = torch.tensor([0, ROWS], device="cuda")
    out, data, scales = bsg.grouped_swiglu_checkpoint_mxfp8(h, off, row_weights=w)
    served, _, _ = bsg.grouped_swiglu_checkpoint_mxfp8(h, off, row_weights=w, keep=False)
    dh, dw, again = bsg.grouped_swiglu_checkpoint_mxfp8_backward(data, scales, dy, off, row_weights=w,
                                                                 recompute=True)
    alone, _, _ = bsg.grouped_swiglu_checkpoint_mxfp8_backward(data, scales, dy, off)
    assert torch.equal(out, served)
    for part in _parts():
        o = torch.tensor([0, ROWS // PARTS], device="cuda")
        y, d, s = bsg.grouped_swiglu_checkpoint_mxfp8(h[part], o, row_weights=w[part])
        assert torch.equal(out[part], y) and torch.equal(data[part], d) and torch.equal(scales[part], s)
        g, gw, a = bsg.grouped_swiglu_checkpoint_mxfp8_backward(d, s, dy[part], o, row_weights=w[part],
                                                                recompute=True)
        assert torch.equal(dh[part], g) and torch.equal(again[part], a)
        # a row's sum is taken over its chunks in the same order, whatever rows stand beside it
        assert torch.equal(dw[part], gw)
        g, _, _ = bsg.grouped_swiglu_checkpoint_mxfp8_backward(d, s, dy[part], o)
        assert torch.equal(alone[part], g)
