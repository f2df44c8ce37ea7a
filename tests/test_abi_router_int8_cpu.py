"""Refusals of the router, the int8 products and the 8-bit activation checkpoints: host only, no HIP call."""

import ctypes

import pytest
import torch

import block_scaled_grouped_amd as bsg


@pytest.fixture(scope="module")
def lib():
    return bsg.load_library()


def _buf(n=4096):
    raw = ctypes.create_string_buffer(n + 256)
    return raw, ctypes.c_void_p((ctypes.addressof(raw) + 255) & ~255)


def _off(p, n):
    return ctypes.c_void_p(p.value + n)


def test_router_workspace(lib):
    size = lib.moe_router_topk_workspace_size
    assert size(-1, 8) == 0 and size(1 << 31, 8) == 0 and size(8, 0) == 0 and size(8, 257) == 0
    last = 0
    for experts in range(1, 257):
        need = size(0, experts)
        assert need == size(1 << 20, experts) >= last > -1
        last = need


def test_router_refusals(lib):
    raw, p = _buf()
    need = lib.moe_router_topk_workspace_size(10, 16)
    good = dict(it=0, l=p, ld=16, t=10, E=16, k=4, mask=None, norm=1, ex=p, w=p, c=p, s=p, live=p, loss=p, ws=p,
                wsb=need)

    def call(**kw):
        return lib.moe_router_topk(*dict(good, **kw).values(), None, None)

    for name in ("l", "ex", "w", "c", "s", "live", "loss", "ws"):
        assert call(**{name: None}) == 1, name
    for kw in (dict(it=3), dict(it=-1), dict(norm=2), dict(norm=-1)):
        assert call(**kw) == 4, kw
    for kw in (dict(t=-1), dict(t=1 << 31), dict(E=0), dict(E=257, ld=300), dict(k=0), dict(k=17, E=32, ld=32),
               dict(k=17), dict(k=5, E=4), dict(ld=15), dict(ld=(1 << 20) + 1)):
        assert call(**kw) == 2, kw
    assert call(l=_off(p, 1)) == 3 and call(l=_off(p, 2), it=2) == 3
    for name in ("ex", "w", "c", "s", "live", "loss"):
        assert call(**{name: _off(p, 2)}) == 3, name
    assert call(ws=_off(p, 8)) == 3
    assert call(wsb=need - 1) == 5 and b"workspace" in lib.bsg_last_error()

    good = dict(it=0, l=p, ld=16, t=10, E=16, k=4, mask=None, norm=1, ex=p, dw=p, c=p, live=p, dl=p, out=p, ldo=16)

    def back(**kw):
        return lib.moe_router_topk_backward(*dict(good, **kw).values(), None)

    for name in ("l", "ex", "c", "live", "out"):
        assert back(**{name: None}) == 1, name
    for kw in (dict(it=5), dict(norm=3)):
        assert back(**kw) == 4, kw
    for kw in (dict(t=-1), dict(E=0), dict(E=300), dict(k=0), dict(k=17), dict(ld=8), dict(ldo=15)):
        assert back(**kw) == 2, kw
    for name in ("ex", "dw", "c", "live", "dl"):
        assert back(**{name: _off(p, 2)}) == 3, name
    assert back(out=_off(p, 1)) == 3 and back(it=2, out=_off(p, 2)) == 3


def test_quantize_int8_refusals(lib):
    raw, p = _buf()
    good = dict(it=0, x=p, ldx=64, rows=10, cols=64, G=2, off=p, d=p, s=p)

    def call(**kw):
        return lib.grouped_quantize_int8(*dict(good, **kw).values(), None, None)

    for name in ("x", "d", "s"):
        assert call(**{name: None}) == 1, name
    assert call(it=2) == 4
    for kw in (dict(G=0), dict(G=257), dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=56, ldx=56),
               dict(cols=131072, ldx=131072), dict(ldx=56), dict(ldx=68), dict(ldx=(1 << 20) + 8)):
        assert call(**kw) == 2, kw
    for kw in (dict(x=_off(p, 8)), dict(d=_off(p, 8)), dict(s=_off(p, 2))):
        assert call(**kw) == 3, kw


def test_gemm_int8_refusals(lib):
    raw, p = _buf()
    need = lib.grouped_gemm_int8_workspace_size()
    good = dict(G=2, a=p, lda=64, sa=p, b=p, ldb=64, sb=64 * 24, bs=p, off=p, rows=10, n=24, k=64, out=p, ldo=24,
                od=0, ws=None, wsb=0)

    def call(**kw):
        return lib.grouped_gemm_int8(*dict(good, **kw).values(), None, None)

    for name in ("a", "sa", "b", "bs", "off", "out"):
        assert call(**{name: None}) == 1, name
    assert call(od=3) == 4 and call(od=-1) == 4
    for kw in (dict(G=0), dict(G=257), dict(rows=-1), dict(rows=1 << 31), dict(n=0), dict(n=20), dict(k=0),
               dict(k=40), dict(k=131072, lda=131072, ldb=131072, sb=131072 * 24), dict(lda=48), dict(lda=72),
               dict(ldb=48), dict(ldb=72), dict(ldo=16), dict(ldo=28), dict(sb=64 * 23), dict(sb=64 * 24 + 8),
               dict(lda=(1 << 20) + 16), dict(ldb=(1 << 20) + 16, sb=1 << 26)):
        assert call(**kw) == 2, kw
    for name in ("a", "b", "bs", "out"):
        assert call(**{name: _off(p, 8)}) == 3, name
    assert call(sa=_off(p, 2)) == 3
    assert call(ws=_off(p, 128), wsb=need) == 3
    assert call(ws=p, wsb=need - 1) == 5


def test_gemm_int8_dynamic_refusals(lib):
    raw, p = _buf()
    size = lib.grouped_gemm_int8_dynamic_workspace_size
    need = size(10, 64)
    assert need > lib.grouped_gemm_int8_workspace_size()
    assert size(-1, 64) == 0 and size(10, 131072) == 0 and size(1 << 31, 64) == 0
    good = dict(it=0, G=2, x=p, ldx=64, b=p, ldb=64, sb=64 * 24, bs=p, off=p, rows=10, n=24, k=64, out=p, ldo=24,
                od=0, ws=p, wsb=need)

    def call(**kw):
        return lib.grouped_gemm_int8_dynamic(*dict(good, **kw).values(), None, None)

    for name in ("x", "b", "bs", "off", "out", "ws"):
        assert call(**{name: None}) == 1, name
    assert call(it=2) == 4 and call(od=3) == 4
    for kw in (dict(G=0), dict(G=257), dict(rows=-1), dict(n=20), dict(k=40), dict(ldx=56), dict(ldx=68),
               dict(ldb=48), dict(ldo=16), dict(sb=64)):
        assert call(**kw) == 2, kw
    for name in ("x", "b", "bs", "out", "ws"):
        assert call(**{name: _off(p, 8)}) == 3, name
    assert call(wsb=need - 1) == 5


def test_dynamic_workspace_never_decreases(lib):
    size = lib.grouped_gemm_int8_dynamic_workspace_size
    rows = [0, 1, 7, 8, 9, 31, 32, 33, 64, 100, 256, 1000, 1024, 1025, 5000, 65536]
    cols = [0, 16, 32, 512, 528, 4096, 4112, 8192, 16384, 131056]
    for r0, r1 in zip(rows, rows[1:]):
        assert all(size(r1, k) >= size(r0, k) for k in cols)
    for k0, k1 in zip(cols, cols[1:]):
        assert all(size(r, k1) >= size(r, k0) for r in rows)


def test_int8_tile_rows(lib):
    rows = lib.grouped_gemm_int8_tile_rows
    assert rows(0, 10, 64, 64, 1) == 0 and rows(2, -1, 64, 64, 1) == 0 and rows(2, 10, 60, 64, 1) == 0
    assert rows(2, 10, 64, 40, 1) == 0
    assert rows(8, 16384, 14336, 4096, 1) == 256 and rows(64, 96, 2048, 7168, 1) <= 32


def test_swiglu_refusals(lib):
    raw, p = _buf()
    good = dict(it=0, h=p, ldh=128, w=None, G=2, off=p, rows=10, f=64, out=p, ldo=64, d=p, s=p)

    def call(**kw):
        return lib.grouped_swiglu_checkpoint_mxfp8(*dict(good, **kw).values(), None, None)

    for name in ("h", "off", "out", "d", "s"):
        assert call(**{name: None}) == 1, name
    assert call(it=2) == 4
    for kw in (dict(G=0), dict(G=257), dict(rows=-1), dict(rows=1 << 31), dict(f=0), dict(f=48), dict(ldh=120),
               dict(ldh=132), dict(ldo=56), dict(f=(1 << 19) + 32, ldh=1 << 21, ldo=1 << 20)):
        assert call(**kw) == 2, kw
    for name in ("h", "out", "d"):
        assert call(**{name: _off(p, 8)}) == 3, name
    assert call(w=_off(p, 2)) == 3

    good = dict(it=0, d=p, s=p, w=None, dy=p, ldd=64, G=2, off=p, rows=10, f=64, dh=p, ldh=128, out=p, ldo=64, dw=None)

    def back(**kw):
        return lib.grouped_swiglu_checkpoint_mxfp8_backward(*dict(good, **kw).values(), None, None)

    for name in ("d", "s", "dy", "off", "dh"):
        assert back(**{name: None}) == 1, name
    assert back(it=2) == 4
    for kw in (dict(G=0), dict(G=257), dict(rows=-1), dict(f=0), dict(f=40), dict(ldd=56), dict(ldd=68),
               dict(ldh=120), dict(ldo=56)):
        assert back(**kw) == 2, kw
    for name in ("d", "dy", "dh", "out"):
        assert back(**{name: _off(p, 8)}) == 3, name
    assert back(w=_off(p, 2)) == 3 and back(dw=_off(p, 2)) == 3


def test_binding_refusals():
    """The Python checks come before the library: host tensors, types, shapes."""
    bf = torch.zeros(4, 64, dtype=torch.bfloat16)
    off = torch.tensor([0, 4])
    q = torch.zeros(4, 64, dtype=torch.int8)
    with pytest.raises(ValueError, match="device"):
        bsg.moe_router_topk(bf, 2)
    with pytest.raises(ValueError, match="device"):
        bsg.moe_router_topk_backward(bf, off, off, off)
    with pytest.raises(ValueError, match="device"):
        bsg.grouped_quantize_int8(bf)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        bsg.grouped_quantize_int8(bf.float())
    with pytest.raises(ValueError, match="device"):
        bsg.grouped_gemm_int8(q, off, q.view(1, 4, 64), off, off)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        bsg.grouped_gemm_int8_dynamic(q, q.view(1, 4, 64), off, off)
    with pytest.raises(ValueError, match="device"):
        bsg.grouped_swiglu_checkpoint_mxfp8(bf, off)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        bsg.grouped_swiglu_checkpoint_mxfp8_backward(q, q, bf.float(), off)
    with pytest.raises(ValueError, match="workspace"):
        bsg.moe_router_topk_workspace(10, 300)
    with pytest.raises(ValueError, match="workspace"):
        bsg.grouped_gemm_int8_dynamic_workspace(-1, 64)
