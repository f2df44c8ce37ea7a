"""What the adapters' second product takes of the first one's sums, at every magnitude of them.

The inputs are whole numbers times powers of two whose sums x A^T hold in 24 bits, in any order, and lora_b has
one power of two in each column, so scale (x A^T) B^T is known exactly and the only error left is what the
16-bit values that carry x A^T leave out."""

import pytest
import torch

import block_scaled_grouped_amd as bsg
from gpu_util import device
from test_gpu_16bit import F64, _offsets

pytestmark = pytest.mark.gpu

# lengths of the requests, their adapters, rank, n, k: tiles of 32, 64, 128 and 256 rows, with the first
# product's contraction whole (k < 1024, or more than 1024 rows) and in parts
SHAPES = [
    ([3, 1, 1], [0, 1, -1], 8, 264, 64),
    ([2, 3], [1, 0], 40, 264, 1024),
    ([390, 1, 9], [1, 0, 1], 136, 8200, 72),
    ([1] * 30 + [570], [i % 3 - 1 for i in range(30)] + [1], 64, 4096, 1024),
    ([700], [0], 24, 8200, 72),
    ([250, 350], [0, 1], 72, 8192, 1024),
    ([900, 0, 1100], [1, 0, 0], 64, 8200, 72),
    ([1400, 1, 99], [1, -1, 0], 32, 6000, 1024),
]
# bits of a factor and terms of a sum: products of b bits each, 2^(24 - 2 b) of them, stay under 2^24
BITS = {torch.float16: (11, 4), torch.bfloat16: (8, 64)}


def _whole(gen, shape, bits):
    """Whole numbers of `bits` bits (the highest one set) and either sign."""
    v = torch.randint(1 << (bits - 1), 1 << bits, shape, generator=gen).to(F64)
    return v * (1 - 2 * torch.randint(0, 2, shape, generator=gen)).to(F64)


def _inputs(dtype, shape, row_exp, col_exp, low_exp, scale_exp, seed):
    """(arguments, scale (x A^T) B^T in 64 bits): row t of x is whole numbers times 2^row_exp(t), column j of
    lora_a's products times 2^col_exp(j), lora_b 2^low_exp, scale 2^scale_exp."""
    lengths, ids, r, n, k = shape
    gen = torch.Generator().manual_seed(seed)
    o, off = _offsets(lengths)
    rows, bits, terms = o[-1], *BITS[dtype]
    x = _whole(gen, (rows, k), bits)
    keep = torch.zeros((rows, k), dtype=torch.bool)
    keep.scatter_(1, torch.rand((rows, k), generator=gen).argsort(1)[:, :terms], True)
    x = torch.where(keep, x, 0.0) * torch.tensor([2.0 ** row_exp(t) for t in range(rows)], dtype=F64)[:, None]
    A = _whole(gen, (2, r, k), bits) * torch.tensor([2.0 ** col_exp(j) for j in range(r)], dtype=F64)[:, None]
    B = torch.zeros((2, n, r), dtype=F64)
    B[:, torch.arange(n), torch.arange(n) % r] = 2.0 ** low_exp
    ref = torch.zeros((rows, n), dtype=F64)
    for g, a in enumerate(ids):
        if a >= 0:
            low = x[o[g]:o[g + 1]] @ A[a].T * 2.0 ** (low_exp + scale_exp)
            ref[o[g]:o[g + 1]] = low[:, torch.arange(n) % r]
    dev = device()
    args = [t.to(dtype).to(dev) for t in (x, torch.zeros((n, k)), A, B)]
    assert all(torch.equal(t.cpu().to(F64), u) for t, u in zip((args[0], args[2], args[3]), (x, A, B)))
    args += [off, torch.tensor(ids, dtype=torch.int32, device=dev), torch.full((2,), 2.0 ** scale_exp, device=dev)]
    return args, ref.to(dev)


# exponents of x, lora_a, lora_b and scale: x A^T of fp16 from 2^-28 (its smallest normal factors) to 2^34
MAGNITUDES = [(-24, -24, 10, 20), (-24, -14, 10, 6), (-14, -14, 0, 0), (-8, -8, 0, -12), (-8, -4, 0, 0),
              (-5, 0, -10, 0), (0, 0, -10, 0), (5, 5, -14, -10)]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("exps", MAGNITUDES)
def test_fp16_keeps_22_bits_at_any_magnitude(exps, shape):
    """Two fp16 values are off by half a step of half a step: 2^-22."""
    xe, ae, be, se = exps
    args, ref = _inputs(torch.float16, SHAPES[shape], lambda t: xe, lambda j: ae, be, se, 10 * shape + 1)
    y = bsg.grouped_lora_gemm_16bit(*args, out_dtype=bsg.BSG_OUT_F32).to(F64)
    err = (y - ref).abs()
    assert bool((err <= 2.0 ** -22 * ref.abs()).all()), float((err / ref.abs()).nan_to_num().max())


@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_fp16_keeps_22_bits_of_values_far_apart(shape):
    """Rows of different magnitudes, and in each row rank columns 2^25 apart."""
    args, ref = _inputs(torch.float16, SHAPES[shape], lambda t: -12 + 17 * (t % 2) - t % 7, lambda j: 5 - j % 26, -3, -6,
                        10 * shape + 2)
    y = bsg.grouped_lora_gemm_16bit(*args, out_dtype=bsg.BSG_OUT_F32).to(F64)
    err = (y - ref).abs()
    assert bool((err <= 2.0 ** -22 * ref.abs()).all()), float((err / ref.abs()).nan_to_num().max())


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shape", [0, 1, 6])
def test_infinities_come_out_as_the_formula_has_them(shape, dtype, value):
    """One rank column of an adapter is infinite or NaN: its sign where lora_b is not zero, NaN where it is."""
    args, ref = _inputs(dtype, SHAPES[shape], lambda t: 0, lambda j: -8, -2, 0, 3)
    x, _, A, B, off, ids, scale = args
    x.copy_(x.abs() + 1)
    A[1, 2] = value
    B[1, 5] = 0
    clean = bsg.grouped_lora_gemm_16bit(x, args[1], A[:1].expand(2, -1, -1).contiguous(), B, off, ids, scale)
    y = bsg.grouped_lora_gemm_16bit(*args)
    lengths, adapters, r = SHAPES[shape][:3]
    o = _offsets(lengths)[0]
    for g, a in enumerate(adapters):
        rows = y[o[g]:o[g + 1]]
        if a != 1:
            assert torch.equal(rows, clean[o[g]:o[g + 1]])
            continue
        # every output takes rank column 2 times its lora_b: 2^-2 in columns 2, r + 2, .., else 0 * value
        want = torch.full((rows.shape[1],), float("nan"), device=x.device)
        want[2::r] = value
        assert torch.equal(rows.float().isnan(), want.isnan().expand(rows.shape[0], -1))
        same = ~want.isnan()
        assert bool((rows.float()[:, same] == want[same]).all())


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("dtype,exps", [(torch.float16, e) for e in MAGNITUDES] +
                         [(torch.bfloat16, e) for e in ((0, 0, 0, 0), (-40, -30, 9, 3), (30, 44, -60, -7))])
def test_all_24_bits_are_kept(dtype, exps, shape):
    """x A^T as float32 holds it: the result is the formula's, bit for bit."""
    xe, ae, be, se = exps
    args, ref = _inputs(dtype, SHAPES[shape], lambda t: xe, lambda j: ae, be, se, 10 * shape + 4)
    assert torch.equal(bsg.grouped_lora_gemm_16bit(*args, out_dtype=bsg.BSG_OUT_F32).to(F64), ref)


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_all_24_bits_are_kept_of_values_far_apart(dtype, shape):
    """Rank columns 2^25 apart (fp16) and 2^50 (bf16) in one row."""
    args, ref = _inputs(dtype, SHAPES[shape], lambda t: -12 + 17 * (t % 2) - t % 7,
                        (lambda j: 5 - j % 26) if dtype == torch.float16 else (lambda j: 20 - j % 51), -3, -6,
                        10 * shape + 5)
    assert torch.equal(bsg.grouped_lora_gemm_16bit(*args, out_dtype=bsg.BSG_OUT_F32).to(F64), ref)
