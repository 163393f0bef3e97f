"""The workspace that the token statistics ask for is bounded by bytes, whatever the vocabulary,
the type and the number of alternatives; the smallest chunk (256 positions, 32 in fp32) is the
only one that may pass the bound. Pure host calls."""
import numpy as np
import pytest

from preference_alignment_b200 import build as B
from preference_alignment_b200 import libdpo

FAKE = 0x100000
BOUND = 1 << 30
SLACK = 1 << 16       # thresholds, target logits, alignment


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return libdpo.load()


def _partials(V, n_top, dtype, n):
    """Partial sums and lists of n positions."""
    K = 0 if n_top == 0 else 1 if n_top == 1 else 8 if n_top <= 8 else 32
    return -(-V // (256 if dtype == "bf16" else 32)) * n * (12 + 8 * K)


@pytest.mark.parametrize("n_top", [0, 1, 8, 32])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1000, 32000, 128256, 151936, 1 << 20, 1 << 24])
def test_rows_size_is_bounded(V, dtype, n_top):
    step = 256 if dtype == "bf16" else 32
    for n in (65, 1000, 8192, 100000, 1 << 30):
        full, least = libdpo.token_stats_rows_size(n, 64, V, n_top, dtype)
        lists = 4 * (1 + 32) * 8192
        assert full <= max(BOUND, _partials(V, n_top, dtype, step)) + lists + SLACK, (n, full)
        assert least <= full
        assert least >= _partials(V, n_top, dtype, min(n, step))


@pytest.mark.parametrize("dtype,n_top", [("bf16", 20), ("f32", 32), ("f32", 8)])
def test_batch_size_is_bounded(dtype, n_top):
    R, L, d, V = 16, 2048, 512, 151936
    b = libdpo.BatchArgs(FAKE, FAKE, FAKE, np.full(R, 4, np.int32), np.full(R, L - 4, np.int32),
                         R=R, L=L, d=d, V=V, dtype=dtype)
    n = R * (L - 4)
    packed = n * (d * 2 if dtype == "bf16" else 0) + 16 * n          # rows, schedule, log-probs
    full, least = libdpo.token_stats_size(b, n_top)
    assert least < full <= BOUND + packed + 4 * 33 * 8192 + SLACK


def test_common_sizes_keep_whole_chunks():
    """8,192 positions at V = 128,256 with up to 8 alternatives stay one launch."""
    for n_top in (0, 1, 8):
        full, _ = libdpo.token_stats_rows_size(8192, 64, 128256, n_top)
        assert full >= _partials(128256, n_top, "bf16", 8192)
