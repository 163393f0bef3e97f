"""Calls on nothing: no rows, or a batch that scores no position, with alternatives asked for. The
outputs then have no elements, and a tensor without elements has no address."""
import ctypes

import numpy as np
import pytest

from preference_alignment_b200 import build as B
from preference_alignment_b200 import libdpo

FAKE = 0x100000     # never dereferenced: nothing is launched
INVALID, WORKSPACE = libdpo.ERR_INVALID_ARG, libdpo.ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    B.build()
    return libdpo.load()


def _rows_call(n, n_top, ids, top, V=100):
    rows = libdpo.TokenRows(n, 64, V, libdpo.BF16, None, 64, FAKE, None)
    out = libdpo.TokenStatsOut(None, None, None, n_top, ids, top)
    fn = libdpo._fn("dpo_token_stats_rows", libdpo._ROWS)
    return fn(ctypes.byref(rows), ctypes.byref(out), None, 0, None)


@pytest.mark.parametrize("n_top", [0, 1, 5, 32])
def test_no_rows_with_alternatives(lib, n_top):
    assert _rows_call(0, n_top, None, None) == libdpo.OK


def test_no_rows_is_checked_as_any_call(lib):
    assert _rows_call(0, 33, None, None) == INVALID
    assert _rows_call(0, -1, None, None) == INVALID
    assert _rows_call(0, 5, None, None, V=0) == INVALID
    assert _rows_call(-1, 5, FAKE, FAKE) == INVALID


def test_a_batch_that_scores_nothing_passes_the_output_check(lib):
    """With missing top pointers the call gets as far as the workspace's check."""
    def call(completion, ids, top):
        b = libdpo.BatchArgs(FAKE, FAKE, FAKE, np.full(4, 4, np.int32), np.full(4, completion, np.int32),
                             R=4, L=32, d=64, V=1000, dtype="bf16")
        out = libdpo.TokenStatsOut(None, None, None, 5, ids, top)
        fn = libdpo._fn("dpo_token_stats", libdpo._STATS)
        return fn(ctypes.byref(b.c), ctypes.byref(out), None, None, 0, None)

    assert call(0, None, None) == WORKSPACE
    assert call(10, None, None) == INVALID
    assert call(10, FAKE, None) == INVALID
    assert call(10, FAKE, FAKE) == WORKSPACE


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tensors_without_rows(dtype):
    import torch
    kind = torch.bfloat16 if dtype == "bf16" else torch.float32
    H = torch.empty(0, 64, device="cuda", dtype=kind)
    W = torch.zeros(100, 64, device="cuda", dtype=kind)
    ids, top = torch.empty(0, 5, device="cuda", dtype=torch.int32), torch.empty(0, 5, device="cuda")
    logp, ent = torch.empty(0, device="cuda"), torch.empty(0, device="cuda")
    tokens = torch.empty(0, device="cuda", dtype=torch.int32)
    need = libdpo.token_stats_rows_size(0, 64, 100, 5, dtype)[0]
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    libdpo.token_stats_rows(H, W, tokens, 5, ws=ws, logp=logp, entropy=ent, top_ids=ids, top_logp=top)
    # and a batch whose rows have no completion: the sums are 0
    Hb = torch.zeros(4, 8, 64, device="cuda", dtype=kind)
    tb = torch.zeros(4, 8, device="cuda", dtype=torch.int32)
    b = libdpo.BatchArgs(Hb, W, tb, np.full(4, 3, np.int32), np.zeros(4, np.int32), dtype=dtype)
    assert b.n_scored == 0
    seq = torch.full((4,), float("nan"), device="cuda")
    ws = torch.empty(libdpo.token_stats_size(b, 5)[0], dtype=torch.uint8, device="cuda")
    libdpo.token_stats(b, 5, ws=ws, logp=logp, seq_logp=seq, top_ids=ids, top_logp=top)
    assert libdpo.check() == libdpo.OK and (seq == 0).all()
