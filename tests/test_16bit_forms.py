"""Which tile form a 16-bit product takes (host), and every form of every mode against the formulas (GPU).

The form goes by measured times, so each case names the form it is meant for and asks the library for its choice:
a change of those times that moves a case to another form fails here instead of leaving a form untested.
Tolerances as in test_gpu_16bit."""

import pytest
import torch

import block_scaled_grouped_amd as bsg
import test_gpu_16bit as few
import test_gpu_16bit_large as many
from test_gpu_16bit_low_rank import SHAPES

FPROP, DGRAD, WGRAD = bsg.BSG_FPROP_TN, bsg.BSG_DGRAD_NN, bsg.BSG_WGRAD_NT
form = bsg.grouped_gemm_16bit_tile_rows


# ---------------------------------------------------------------- the choice


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("case", range(len(many.ROWS)))
def test_cases_of_the_large_form_take_it(case, ws):
    sizes, n, k = many.ROWS[case]
    for mode in (FPROP, DGRAD):
        assert form(mode, len(sizes), 5 + sum(sizes) + 7, n, k, ws) == 256


@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("case", range(len(many.GRADS)))
def test_weight_gradients_of_the_large_form_take_it(case, ws):
    sizes, n, k = many.GRADS[case]
    assert form(WGRAD, len(sizes), 5 + sum(sizes), n, k, ws) == 256


def test_adapters_of_the_large_form_take_it():
    for lengths, n, k in (([900, 1, 1100, 300, 0, 800], 4096, 200), ([40] * 70, 8192, 328), ([2600, 1500], 8200, 72)):
        assert bsg.grouped_lora_gemm_16bit_tile_rows(sum(lengths) + 7, n, k) == 256


def test_other_cases_of_the_large_form_take_it():
    for mode in (FPROP, DGRAD, WGRAD):
        assert form(mode, 4, 4096, 2304, 2056) == 256          # repeats and graph replays
    for mode in (FPROP, DGRAD):
        assert form(mode, 2, 3000, 8192, 136, False) == 256    # rows 2^20 elements apart


def test_small_cases_take_the_smallest_form():
    for sizes, n, k in few.CASES:
        for ws in (False, True):
            for mode in (FPROP, DGRAD):
                assert form(mode, len(sizes), sum(sizes), n, k, ws) == 32
            assert form(WGRAD, len(sizes), sum(sizes), n, k, ws) == 128


def test_low_rank_shapes_take_each_form():
    got = [bsg.grouped_lora_gemm_16bit_tile_rows(sum(s[0]), s[3], s[4]) for s in SHAPES]
    assert got == [32, 32, 64, 64, 128, 128, 256, 256]


def test_the_choice_goes_by_the_capacity():
    """What the header says: 64 experts' rows in a buffer of 128 and in one of 8192."""
    assert form(FPROP, 64, 128, 2048, 7168) == 32
    assert form(FPROP, 64, 8192, 2048, 7168) == 256


def test_refusals():
    lib = bsg.load_library()
    good = [FPROP, 4, 100, 64, 64, 1]
    assert lib.grouped_gemm_16bit_tile_rows(*good) == 32
    for i, bad in ((0, 3), (0, -1), (1, 0), (1, 257), (2, -1), (2, 1 << 31), (3, 0), (3, 60), (3, (1 << 20) + 8), (4, -8),
                   (4, 12)):
        args = list(good)
        args[i] = bad
        assert lib.grouped_gemm_16bit_tile_rows(*args) == 0, args
        if i > 1:
            assert lib.grouped_lora_gemm_16bit_tile_rows(*args[2:5]) == 0, args
    assert lib.grouped_gemm_16bit_tile_rows(FPROP, 4, (1 << 31) - 1, 1 << 20, 64, 1) == 0   # tiles
    with pytest.raises(ValueError, match="rows_cap"):
        form(FPROP, 4, -1, 64, 64)
    with pytest.raises(ValueError, match="rows_cap"):
        bsg.grouped_lora_gemm_16bit_tile_rows(1, 12, 64)


# ---------------------------------------------------------------- the forms

# form, sizes, n, k: whole and split contractions (one stage, an odd number, a last one that is not whole), groups
# without rows, rows and columns that end inside a tile
FORMS = [
    (64, [300, 0, 257, 1, 94], 8200, 72),
    (64, [200, 1, 0, 191], 6000, 1000),
    (64, [692], 4104, 2056),
    (128, [900, 192], 4104, 72),
    (128, [692], 8200, 64),
    (128, [1, 1200, 0, 799], 8200, 64),
    (128, [500, 0, 100], 8200, 2056),
]


@pytest.mark.gpu
@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("dtype", few.DTYPES)
@pytest.mark.parametrize("mode", [FPROP, DGRAD])
@pytest.mark.parametrize("case", range(len(FORMS)))
def test_middle_forms(case, mode, dtype, ws):
    want, sizes, n, k = FORMS[case]
    o, off = few._offsets(sizes, 3)
    rows = o[-1] + 5
    assert form(mode, len(sizes), rows, n, k, ws) == want
    a = many._dev_rand(case, (rows, k), dtype)
    a[:3], a[o[-1]:] = float("nan"), float("nan")
    b = many._dev_rand(30 + case, (len(sizes), n, k) if mode == FPROP else (len(sizes), k, n), dtype)
    live = slice(o[0], o[-1])
    work = bsg.gemm_workspace() if ws else None
    for f32 in (False, True):
        odt = torch.float32 if f32 else dtype
        for addend in (False, True):
            c = many._dev_rand(60 + case, (rows, n + 8), odt, 10.0)[:, :n] if addend else None
            ref, mag = many._reference(mode, a, b, o, c)
            out = torch.full((rows, n + 8), -3.0, dtype=odt, device=a.device)[:, :n]
            bsg.grouped_gemm_16bit(mode, a, b, off, c=c, out=out, workspace=work)
            many._assert_close(out[live], ref[live], mag[live], k + 1)
            assert bool((out[:3] == -3.0).all()) and bool((out[o[-1]:] == -3.0).all())
            assert bool((out._base[:, n:] == -3.0).all())
