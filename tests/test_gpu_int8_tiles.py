"""Every form of the int8 products with rows in front of the first group and behind the last that have to stay as they
were, groups that end inside of tiles (in their first 16 rows, or one row short of them), and widths of whole tiles and
not.  The form that a case is meant for is asked for, with a workspace and without.  Bit for bit, as in test_gpu_int8.py."""

import pytest
import torch

import block_scaled_grouped_amd as bsg
from test_gpu_int8 import _case, _run

# rows of a tile with a workspace and without, group sizes, n, k, rows in front and behind
CASES = [
    (16, 16, [3, 0, 1, 5, 0, 2, 7, 1], 256, 272, 2, 5),
    (16, 16, [9], 1032, 528, 3, 4),
    (32, 32, [11, 0, 23], 264, 528, 5, 70),
    (32, 32, [33, 1, 62], 512, 1040, 1, 100),
    (64, 32, [40, 0, 7, 65, 1, 2, 63, 3], 2048, 2064, 4, 15),
    (64, 64, [257, 0, 393], 2048, 272, 3, 350),
    (128, 128, [300, 1, 127], 4096, 272, 5, 560),
    (256, 256, [257, 0, 1030], 4096, 272, 5, 700),      # whole tiles of columns; one row and six of the last tiles
    (256, 256, [511, 17, 1], 4096, 272, 3, 1500),
    (256, 256, [530, 0, 1300], 4104, 272, 255, 300),
    (256, 256, [1, 255, 300, 0, 2, 16, 784, 513], 4096, 528, 7, 600),
    (128, 256, [2049, 15, 1200], 4096, 1040, 6, 830),
]


def _forms(case):
    _, _, sizes, n, k, first, dead = case
    rows = first + sum(sizes) + dead
    return tuple(bsg.grouped_gemm_int8_tile_rows(len(sizes), rows, n, k, workspace=w) for w in (True, False))


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "%d-%d-%s-%d-%d" % (c[0], c[1], sum(c[2]), c[3], c[4]))
def test_rows_outside_of_the_groups(case):
    assert _forms(case) == case[:2]
    _, _, sizes, n, k, first, dead = case
    operands = _case(sizes, n, k, seed=first, dead=dead, first=first)
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        for ws in (bsg.gemm_workspace(), None):
            _run(operands, dtype, ws, gap=0 if ws is None else 8)


@pytest.mark.gpu
def test_the_cases_take_every_form():
    assert {f for case in CASES for f in _forms(case)} == {16, 32, 64, 128, 256}


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n,k,with_workspace,without", [
    (2048, 4096, 2048, 256, 256), (1500, 4104, 2064, 128, 128), (700, 2056, 1040, 32, 32), (200, 2048, 4096, 32, 32),
    (40, 2048, 4096, 32, 32)])
def test_forms_of_uneven_groups(rows, n, k, with_workspace, without):
    """Those of test_gpu_int8.test_forms, which runs them."""
    assert [bsg.grouped_gemm_int8_tile_rows(3, rows + 3, n, k, workspace=w) for w in (True, False)] == [
        with_workspace, without]
