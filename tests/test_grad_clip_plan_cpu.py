"""The chunk table of gradient clipping refuses tensors whose outputs workgroups would race for (host only)."""

import random

import pytest

import block_scaled_grouped_amd as bsg
from test_abi_16bit_cpu import _plan

BF16, F16, F32 = bsg.BSG_GRAD_BF16, bsg.BSG_GRAD_F16, bsg.BSG_GRAD_F32


@pytest.fixture(scope="module")
def lib():
    return bsg.load_library()


# (src, dst, numels, dtypes); addresses are never followed
REFUSED = {
    "the same tensor twice, in place": ([4096, 4096], [4096, 4096], [100, 100], [F32, F32]),
    "a tensor and a view of its end": ([4096, 4496], [4096, 4496], [101, 10], [F32, F32]),
    "two outputs in one place": ([4096, 8192], [65536, 65536], [8, 8], [BF16, BF16]),
    "an output in another one's input": ([4096, 8192], [8194, 65536], [8, 8], [BF16, BF16]),
    "an output around another one's input": ([4096, 8192], [8000, 65536], [4000, 1], [F16, F16]),
    "an output one element into its own input": ([4096], [4098], [2], [BF16]),
    "an output one element before its own input": ([4096], [4092], [50000], [F32]),
    "outputs exchanged": ([4096, 8192], [8192, 4096], [8, 8], [F32, F32]),
    "far apart in the list": ([1 << 20, 1 << 24, 1 << 28, (1 << 20) + 4], [1 << 32, 1 << 36, 1 << 40, (1 << 32) + 4],
                              [2, 100, 100, 9], [F32] * 4),
}
TAKEN = {
    "one after the other": ([4096, 4104, 4120], [4096, 4104, 4120], [2, 8, 100], [F32, BF16, F16]),
    "one input twice, two outputs": ([4096, 4096], [8192, 16384], [100, 100], [F32, F32]),
    "overlapping inputs, outputs apart": ([4096, 4100], [8192, 16384], [100, 100], [F32, F32]),
    "an output right after its input": ([4096], [4104], [2], [F32]),
    "no elements in another one's place": ([4096, 4098, 4096], [4096, 4098, 4096], [100, 0, 0], [F32, BF16, F32]),
}


@pytest.mark.parametrize("name", REFUSED)
def test_refused(lib, name):
    assert _plan(lib, *REFUSED[name])[0] == 2
    assert b"shares memory" in lib.bsg_last_error()


@pytest.mark.parametrize("name", TAKEN)
def test_taken(lib, name):
    rc, chunks = _plan(lib, *TAKEN[name])
    assert rc == 0 and sum(c[2] for c in chunks) == sum(TAKEN[name][2])


def test_against_every_pair(lib):
    """Random places: refused exactly where some pair of ranges overlaps, and else the whole table in order."""
    rng = random.Random(1)
    seen = [0, 0]
    for _ in range(400):
        n = rng.randint(1, 6)
        dtypes = [rng.choice([BF16, F16, F32]) for _ in range(n)]
        size = [4 if t == F32 else 2 for t in dtypes]
        numels = [rng.choice([0, 1, 5, 60]) for _ in range(n)]
        src = [4096 + 4 * rng.randrange(400) for _ in range(n)]
        dst = [s if rng.random() < 0.5 else 4096 + 4 * rng.randrange(400) for s in src]

        def meet(i, a, j, b):
            return a < b + numels[j] * size[j] and b < a + numels[i] * size[i] and numels[i] * numels[j] > 0

        bad = any(meet(i, dst[i], j, dst[j]) for i in range(n) for j in range(i)) or any(
            meet(i, dst[i], j, src[j]) and not (i == j and src[i] == dst[i]) for i in range(n) for j in range(n))
        rc, chunks = _plan(lib, src, dst, numels, dtypes)
        assert rc == (2 if bad else 0), (src, dst, numels, dtypes)
        seen[bad] += 1
        if not bad:
            assert chunks == [(s, d, m, t) for s, d, m, t in zip(src, dst, numels, dtypes) if m]
    assert min(seen) > 30
