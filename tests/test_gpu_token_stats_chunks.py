"""A position's statistics do not depend on how the call is cut into chunks: the same bits with the
full workspace and with the smallest, also where a call has more positions than one block per
position joins (1,024) and its chunks have fewer."""
import numpy as np
import pytest

from oracle import head_ops_oracle as HO
from preference_alignment_b200 import libdpo
from preference_alignment_b200 import workloads as WL

from dpo_harness import to_device

pytestmark = pytest.mark.gpu


def _run(h, W, tokens, n_top, dtype, ws_bytes):
    import torch
    n = len(h)
    ws = torch.full((ws_bytes,), 0xAB, dtype=torch.uint8, device="cuda")
    out = dict(logp=torch.empty(n, device="cuda"), entropy=torch.empty(n, device="cuda"),
               lse_state=torch.empty(n, device="cuda"))
    if n_top:
        out["top_ids"] = torch.empty(n, n_top, dtype=torch.int32, device="cuda")
        out["top_logp"] = torch.empty(n, n_top, device="cuda")
    libdpo.token_stats_rows(h, W, tokens, n_top, ws=ws, **out)
    assert libdpo.check() == libdpo.OK
    return {k: v.cpu().numpy() for k, v in out.items()}


@pytest.mark.parametrize("n_top", [0, 1, 8, 32])
@pytest.mark.parametrize("dtype,n", [("bf16", 1025), ("bf16", 2500), ("f32", 1025), ("f32", 1300)])
def test_the_smallest_workspace_gives_the_same_bits(dtype, n, n_top):
    import torch
    d, V = 64, 1500
    rng = np.random.default_rng(n + n_top)
    hs = WL.encode(rng.normal(size=(n, d)).astype(np.float32), dtype)
    Ws = WL.encode((rng.normal(size=(V, d)) * 3 / np.sqrt(d)).astype(np.float32), dtype)
    tokens = rng.integers(0, V, n).astype(np.int32)
    h, W, t = to_device(hs, dtype), to_device(Ws, dtype), torch.from_numpy(tokens).cuda()
    full, least = libdpo.token_stats_rows_size(n, d, V, n_top, dtype)
    assert least < full
    a = _run(h, W, t, n_top, dtype, full)
    for size in (least, (least + full) // 2):
        b = _run(h, W, t, n_top, dtype, size)
        for k, v in a.items():
            assert np.array_equal(v, b[k]), (k, size)
    o = HO.token_stats(WL.widen(hs, dtype), WL.widen(Ws, dtype), tokens, n_top)
    # a logit is a sum of 64 products: tz; the sums of e^(z - max) are off by less than 2^-15
    # (exponential 2^-22, its argument 40 * 2^-24, chains of 256 + tiles additions 2^-24 each)
    tz = (np.abs(WL.widen(hs, dtype)) @ np.abs(WL.widen(Ws, dtype)).T).max(axis=1) * d * 2.0 ** -23
    assert np.all(np.abs(a["lse_state"] - o["lse"]) <= tz + 2.0 ** -15 + 2.0 ** -23 * np.abs(o["lse"]))
    assert np.all(np.abs(a["logp"] - o["logp"]) <= 2 * tz + 2.0 ** -15 + 2.0 ** -23 * np.abs(o["logp"]))


@pytest.mark.parametrize("n,d,V", [(300, 1024, 1300), (1500, 200, 2050)])
def test_both_gemm_kernels_give_the_same_bits(n, d, V):
    """A chunk's number of positions decides between the single-CTA kernel and CTA pairs."""
    import torch
    rng = np.random.default_rng(n)
    h = to_device(WL.encode(rng.normal(size=(n, d)).astype(np.float32), "bf16"), "bf16")
    W = to_device(WL.encode((rng.normal(size=(V, d)) * 3 / np.sqrt(d)).astype(np.float32), "bf16"), "bf16")
    t = torch.from_numpy(rng.integers(0, V, n).astype(np.int32)).cuda()
    size = libdpo.token_stats_rows_size(n, d, V, 8)[0]
    got = []
    for mask in (0, 1, 16):
        old = libdpo.set_gemm_variant(mask)
        try:
            got.append(_run(h, W, t, 8, "bf16", size))
        finally:
            libdpo.set_gemm_variant(old)
    for g in got[1:]:
        for k, v in got[0].items():
            assert np.array_equal(v, g[k]), k


def test_default_workspace_cut_by_its_bytes():
    """2,100 fp32 positions with 32 alternatives over 80,000 rows take more than the 1 GB that a
    chunk may: two launches, the ids exact on a grid."""
    import torch
    n, d, V, n_top = 2100, 8, 80000, 32
    rng = np.random.default_rng(9)
    hs = (np.rint(rng.normal(size=(n, d)) * 8) / 8).astype(np.float32)
    Ws = (np.rint(rng.normal(size=(V, d)) * 64) / 64).astype(np.float32)
    tokens = rng.integers(0, V, n).astype(np.int32)
    size = libdpo.token_stats_rows_size(n, d, V, n_top, "f32")[0]
    assert size < (V // 32) * n * 268                  # what one launch of all would take
    got = _run(torch.from_numpy(hs).cuda(), torch.from_numpy(Ws).cuda(),
               torch.from_numpy(tokens).cuda(), n_top, "f32", size)
    for i in (0, 1400, 1980):                          # the oracle in parts: both launches, the last rows
        s = slice(i, i + 120)
        o = HO.token_stats(hs[s], Ws, tokens[s], n_top)
        assert np.array_equal(got["top_ids"][s], o["top_ids"])
        # exact logits; sums as above
        assert np.all(np.abs(got["lse_state"][s] - o["lse"]) <= 2.0 ** -15 + 2.0 ** -23 * np.abs(o["lse"]))
