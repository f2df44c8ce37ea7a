"""Refusals of the 16-bit operators, and the chunk table of gradient clipping: host only, no HIP call."""

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


def test_gemm_16bit_refusals(lib):
    raw, p = _buf()
    need = lib.grouped_gemm_16bit_workspace_size()
    assert need > 0
    good = dict(mode=0, it=0, G=2, a=p, lda=64, b=p, ldb=64, sb=64 * 64, off=p, rows=10, n=64, k=64, c=None,
                out=p, ldo=64, so=0, od=0, ws=None, wsb=0)

    def call(**kw):
        v = dict(good, **kw)
        return lib.grouped_gemm_16bit(*v.values(), None, None)

    odd = ctypes.c_void_p(p.value + 8)
    for name in ("a", "b", "off", "out"):
        assert call(**{name: None}) == 1, name
    for mode in (-1, 3, 4):
        assert call(mode=mode) == 4
    assert call(it=2) == 4 and call(od=2) == 4 and call(it=1, od=0) == 4 and call(od=7) == 4
    for G in (0, 257, -1):
        assert call(G=G) == 2
    for kw in (dict(n=0), dict(k=0), dict(n=60), dict(k=36), dict(rows=-1), dict(rows=1 << 31), dict(lda=56),
               dict(lda=68), dict(ldb=56), dict(ldo=56), dict(lda=(1 << 20) + 8), dict(sb=64), dict(sb=4100),
               dict(n=-8), dict(mode=1, so=64), dict(mode=2, sb=8)):
        assert call(**kw) == 2, kw
    for name in ("a", "b", "out", "c"):
        assert call(**{name: odd}) == 3, name
    assert call(ws=odd, wsb=need) == 3
    assert call(ws=p, wsb=need - 1) == 5
    assert b"workspace" in lib.bsg_last_error()


def test_lora_refusals(lib):
    raw, p = _buf()
    need = lib.grouped_lora_gemm_16bit_workspace_size(10, 64, 64, 16)
    assert need > 0
    assert lib.grouped_lora_gemm_16bit_workspace_size(-1, 64, 64, 16) == 0
    good = dict(it=0, G=2, x=p, ldx=64, w=p, ldw=64, A=p, B=p, count=3, r=16, off=p, ad=p, sc=p, rows=10, n=64,
                k=64, out=p, ldo=64, od=0, ws=p, wsb=need)

    def call(**kw):
        v = dict(good, **kw)
        return lib.grouped_lora_gemm_16bit(*v.values(), None, None)

    for name in ("x", "w", "A", "B", "off", "ad", "sc", "out", "ws"):
        assert call(**{name: None}) == 1, name
    assert call(it=5) == 4 and call(od=2) == 4
    for kw in (dict(G=0), dict(G=257), dict(r=0), dict(r=12), dict(r=264), dict(count=0), dict(n=12), dict(k=12),
               dict(ldx=8), dict(ldw=72 + 4), dict(ldo=0), dict(rows=-1)):
        assert call(**kw) == 2, kw
    odd = ctypes.c_void_p(p.value + 2)
    for name in ("x", "w", "A", "B", "out", "ad", "sc", "ws"):
        assert call(**{name: odd}) == 3, name
    assert call(wsb=need - 1) == 5


def test_binding_refusals():
    """The Python checks come before the library: host tensors, types, shapes."""
    a = torch.zeros(4, 8, dtype=torch.bfloat16)
    off = torch.tensor([0, 4])
    with pytest.raises(ValueError, match="device"):
        bsg.grouped_gemm_16bit(bsg.BSG_FPROP_TN, a, a.view(1, 4, 8), off)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        bsg.grouped_gemm_16bit(bsg.BSG_FPROP_TN, a.float(), a, off)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        bsg.grouped_lora_gemm_16bit(a.float(), a, a, a, off, off, off)
    with pytest.raises(ValueError, match="device"):
        bsg.grad_clip_plan([a])
    with pytest.raises(ValueError, match="outputs"):
        bsg.grad_clip_plan([a], [])


def _plan(lib, src, dst, numels, dtypes, room=None):
    n = len(src)
    args = ((ctypes.c_void_p * max(n, 1))(*src), (ctypes.c_void_p * max(n, 1))(*dst),
            (ctypes.c_int64 * max(n, 1))(*numels), (ctypes.c_int32 * max(n, 1))(*dtypes))
    count = ctypes.c_int64(-1)
    rc = lib.grad_clip_plan_fill(n, *args, None, 0, ctypes.byref(count))
    if rc:
        return rc, None
    room = count.value if room is None else room
    buf = ctypes.create_string_buffer(24 * max(room, 1))
    rc = lib.grad_clip_plan_fill(n, *args, buf, 24 * room, ctypes.byref(count))
    if rc:
        return rc, None
    out = []
    for i in range(count.value):
        s, d = (int.from_bytes(buf.raw[24 * i + 8 * j:24 * i + 8 * j + 8], "little") for j in range(2))
        m, t = (int.from_bytes(buf.raw[24 * i + 16 + 4 * j:24 * i + 20 + 4 * j], "little") for j in range(2))
        out.append((s, d, m, t))
    return 0, out


def test_plan_covers_every_element_once(lib):
    src = [1 << 20, (1 << 24) + 2, 5 << 24, 9 << 24]
    dst = [1 << 30, (1 << 30) + (1 << 26) + 6, 5 << 28, 9 << 28]
    numels, dtypes, esz = [1, 100001, 0, 3 * 16384], [2, 0, 1, 2], [4, 2, 2, 4]
    rc, chunks = _plan(lib, src, dst, numels, dtypes)
    assert rc == 0
    at = 0
    for s, d, n, t, e in zip(src, dst, numels, dtypes, esz):
        done = 0
        while done < n:
            cs, cd, cn, ct = chunks[at]
            assert (cs, cd, ct) == (s + done * e, d + done * e, t) and 0 < cn <= 16384
            assert done == 0 or cs % 128 == 0
            done += cn
            at += 1
        assert done == n
    assert at == len(chunks)


def test_plan_and_clip_refusals(lib):
    assert _plan(lib, [64], [64], [10], [3])[0] == 4
    assert _plan(lib, [64], [64], [-1], [0])[0] == 2
    assert _plan(lib, [None], [64], [10], [0])[0] == 1
    assert _plan(lib, [66], [64], [10], [2])[0] == 3
    assert _plan(lib, [64], [64], [100000], [2], room=2)[0] == 5
    assert _plan(lib, [None], [None], [0], [0]) == (0, [])
    assert _plan(lib, [], [], [], []) == (0, [])
    raw, p = _buf()
    need = lib.grad_clip_workspace_size()
    odd = ctypes.c_void_p(p.value + 4)
    assert lib.grad_norm(None, 3, p, need, p, None, None, None) == 1
    assert lib.grad_norm(p, 3, None, need, p, None, None, None) == 1
    assert lib.grad_norm(p, 3, p, need, None, None, None, None) == 1
    assert lib.grad_norm(p, -1, p, need, p, None, None, None) == 2
    assert lib.grad_norm(odd, 3, p, need, p, None, None, None) == 3
    assert lib.grad_norm(p, 3, p, need, p, odd, None, None) == 3
    assert lib.grad_norm(p, 3, p, need - 1, p, None, None, None) == 5
    for bad in (-1.0, float("nan")):
        assert lib.clip_grad_norm(p, 3, bad, None, p, need, None, None, None) == 2
    assert lib.clip_grad_norm(p, 3, 1.0, odd, p, need, None, None, None) == 3
    assert lib.clip_grad_norm(p, 3, 1.0, None, p, 8, None, None, None) == 5
