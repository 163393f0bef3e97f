"""The operators around the head where a call can go wrong though its values are ordinary: garbage
in positions that do not count, offsets past 32 bits, graphs that share a workspace, the optional
operands one by one.

Tolerances, beside half a step of bf16 (2^-8 of the value) where a result is rounded to it: F32, a
few hundred fp32 roundings (2^-24 each) in a row's or a column's sums, relative to the largest value;
LOGIT, an absolute error of an fp32 log-sum-exp or entropy of magnitude at most 16 (2^-20 a step)
over exact logits, with the hardware exponential's 2^-22 relative and tens of additions."""
import numpy as np
import pytest

from oracle import head_ops_oracle as HO
from preference_alignment_b200 import libdpo
from preference_alignment_b200 import workloads as WL

import test_gpu_norm
from dpo_harness import DeviceWorkload, np64, to_device

pytestmark = pytest.mark.gpu

F32 = 1e-5
LOGIT = 1e-4
HALF_BF16 = 2.0 ** -8


def _space(n):
    import torch
    return torch.full((max(n, 256),), 0xAB, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unscored_positions_may_hold_anything(dtype):
    """NaN and infinities at prompt, padding and last positions, tokens out of range there: the
    same bits as with zeros."""
    import torch
    w = WL.make_custom(R=6, L=40, d=64, V=500, dtype=dtype, seed=5)
    scored = np.zeros((w.R, w.L), bool)
    for r in range(w.R):
        scored[r, w.prompt_len[r] - 1:w.prompt_len[r] - 1 + w.completion_len[r]] = True
    keep = torch.from_numpy(scored).cuda()
    target = torch.from_numpy(np.roll(scored, 1, axis=1)).cuda()       # token t + 1 of position t
    n, n_top = int(scored.sum()), 5
    got = []
    for garbage in (0.0, float("nan"), float("inf")):
        dw = DeviceWorkload(w)
        dw.H[~keep] = garbage
        if garbage:
            dw.tokens[~target] = -5
        b = dw.batch()
        o = dict(logp=torch.empty(n, device="cuda"), entropy=torch.empty(n, device="cuda"),
                 lse_state=torch.empty(n, device="cuda"), seq_logp=torch.empty(w.R, device="cuda"),
                 top_ids=torch.empty(n, n_top, dtype=torch.int32, device="cuda"),
                 top_logp=torch.empty(n, n_top, device="cuda"))
        libdpo.token_stats(b, n_top, ws=_space(libdpo.token_stats_size(b, n_top)[0]), **o)
        assert libdpo.check() == libdpo.OK
        got.append({k: v.cpu().numpy() for k, v in o.items()})
    assert np.all(np.isfinite(got[0]["logp"]))
    for g in got[1:]:
        for k, v in got[0].items():
            assert np.array_equal(v, g[k]), k


@pytest.mark.parametrize("n", [20, 200])
def test_two_graphs_share_a_workspace(n):
    """Two captured calls on one workspace, replayed in turn with their inputs swapped."""
    import torch
    d, V, n_top = 64, 3000, 20
    rng = np.random.default_rng(n)
    W = WL.encode((np.rint(rng.normal(size=(V, d)) * 8) / 64).astype(np.float32), "bf16")
    hs = [WL.encode((np.rint(rng.normal(size=(n, d)) * 8) / 8).astype(np.float32), "bf16")
          for _ in range(2)]
    Wd = to_device(W, "bf16")
    ws = _space(libdpo.token_stats_rows_size(n, d, V, n_top)[0])
    H = [to_device(h, "bf16") for h in hs]
    out = [dict(lse_state=torch.empty(n, device="cuda"),
                top_ids=torch.empty(n, n_top, dtype=torch.int32, device="cuda"),
                top_logp=torch.empty(n, n_top, device="cuda")) for _ in range(2)]
    libdpo.token_stats_rows(H[0], Wd, None, n_top, ws=ws, **out[0])
    torch.cuda.synchronize()
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            libdpo.token_stats_rows(H[k], Wd, None, n_top, ws=ws, **out[k])
        graphs.append(g)
    for swap in (0, 1):
        for k in range(2):
            H[k].copy_(to_device(hs[k ^ swap], "bf16"))
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        for k in range(2):
            o = HO.token_stats(WL.widen(hs[k ^ swap], "bf16"), WL.widen(W, "bf16"), None, n_top)
            assert np.array_equal(out[k]["top_ids"].cpu().numpy(), o["top_ids"])
            assert np.abs(np64(out[k]["lse_state"]) - o["lse"]).max() < LOGIT
    assert libdpo.check() == libdpo.OK


def test_rows_more_than_32_bits_apart():
    """Hidden rows 2^30 values apart: 2^31 bytes between neighbours."""
    import torch
    n, d, V, n_top = 3, 64, 300, 4
    for dtype, kind in (("bf16", torch.bfloat16), ("f32", torch.float32)):
        stride = 1 << 30 if dtype == "bf16" else 1 << 29
        wide = torch.zeros((n - 1) * stride + d, dtype=kind, device="cuda")
        H = wide.as_strided((n, d), (stride, 1))
        h = WL.encode((np.rint(np.random.default_rng(1).normal(size=(n, d)) * 8) / 8).astype(np.float32), dtype)
        H.copy_(to_device(h, dtype))
        W = WL.encode((np.rint(np.random.default_rng(2).normal(size=(V, d)) * 8) / 64).astype(np.float32), dtype)
        ids = torch.empty(n, n_top, dtype=torch.int32, device="cuda")
        top, ent = torch.empty(n, n_top, device="cuda"), torch.empty(n, device="cuda")
        libdpo.token_stats_rows(H, to_device(W, dtype), None, n_top, entropy=ent, top_ids=ids, top_logp=top,
                                ws=_space(libdpo.token_stats_rows_size(n, d, V, n_top, dtype)[0]))
        assert libdpo.check() == libdpo.OK
        o = HO.token_stats(WL.widen(h, dtype), WL.widen(W, dtype), None, n_top)
        assert np.array_equal(ids.cpu().numpy(), o["top_ids"])
        assert np.abs(np64(ent) - o["entropy"]).max() < LOGIT
        # and the norm over the same rows, in place
        rstd = torch.empty(n, device="cuda")
        libdpo.norm_forward(H, H, kind="rms", rstd=rstd)
        y, _, r = HO.norm_forward(WL.widen(h, dtype), kind="rms")
        assert np.abs(np64(rstd) / r - 1).max() < F32
        assert np.abs(np64(H) - y).max() <= (F32 + HALF_BF16) * np.abs(y).max()
        del wide, H


def test_more_than_32_bits_of_values():
    """2.2e9 values: the last rows are worked on as any others."""
    import torch
    rows, d = 540000, 4096
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(64, d, device="cuda").bfloat16()
    x[-64:] = tail
    held, small = libdpo.Checkpoint.empty(rows, d), libdpo.Checkpoint.empty(64, d)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    y, ys = torch.empty_like(x), torch.empty_like(tail)
    ms, rs = torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    libdpo.norm_forward(x, y, mean=mean, rstd=rstd, save=held)
    libdpo.norm_forward(tail, ys, mean=ms, rstd=rs, save=small)
    assert torch.equal(held.codes[-64:], small.codes) and torch.equal(held.scales[-64:], small.scales)
    # 64 rows run on more warps each than 540,000 do: sums in another order
    assert (mean[-64:] - ms).abs().max() < F32 and (rstd[-64:] / rs - 1).abs().max() < F32
    assert (y[-64:].float() - ys.float()).abs().max() <= (F32 + 2 * HALF_BF16) * ys.float().abs().max()
    assert (y[:-64] == 0).all()
    libdpo.checkpoint_pack(x, held)
    assert torch.equal(held.codes[-64:], small.codes)
    back, backs = torch.empty_like(x), torch.empty_like(tail)
    libdpo.checkpoint_unpack(held, back)
    libdpo.checkpoint_unpack(small, backs)
    assert torch.equal(back[-64:], backs) and (back[:-64] == 0).all()
    dw, dws = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = _space(libdpo.norm_workspace_size(rows, d))
    # dy = x: the tail's rows alone carry gradient (zero rows have xh = 0)
    libdpo.norm_backward(held, x, mean, rstd, dx=back, dweight=dw, ws=ws)
    libdpo.norm_backward(small, tail, mean[-64:].contiguous(), rstd[-64:].contiguous(), dx=backs,
                         dweight=dws, ws=ws)
    assert (back[-64:].float() - backs.float()).abs().max() <= (F32 + 2 * HALF_BF16) * backs.float().abs().max()
    assert (dw - dws).abs().max() <= F32 * dws.abs().max()


@pytest.mark.parametrize("d", [24, 264, 1000, 4096, 8200, 65536])
@pytest.mark.parametrize("with_weight,with_bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_optional_operands(d, with_weight, with_bias, dtype, wdtype):
    import torch
    rows = 7
    rng = np.random.default_rng(d)
    x = WL.encode(rng.normal(size=(rows, d)).astype(np.float32), dtype)
    w = WL.encode(rng.normal(1, 0.2, d).astype(np.float32), wdtype)
    b = WL.encode(rng.normal(0, 0.2, d).astype(np.float32), wdtype)
    dy = WL.encode(rng.normal(size=(rows, d)).astype(np.float32), dtype)
    wd, bd = (to_device(w, wdtype) if with_weight else None), (to_device(b, wdtype) if with_bias else None)
    xd = to_device(x, dtype)
    y = torch.empty_like(xd)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    libdpo.norm_forward(xd, y, weight=wd, bias=bd, mean=mean, rstd=rstd)
    o, _, _ = HO.norm_forward(WL.widen(x, dtype), WL.widen(w, wdtype) if with_weight else None,
                              WL.widen(b, wdtype) if with_bias else None)
    half = F32 + (HALF_BF16 if dtype == "bf16" else 0.0)
    assert np.abs(np64(y) - o).max() <= half * np.abs(o).max()
    dx, dw, db = torch.empty_like(xd), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    libdpo.norm_backward(xd, to_device(dy, dtype), mean, rstd, dx=dx, weight=wd, dweight=dw, dbias=db,
                         ws=_space(libdpo.norm_workspace_size(rows, d)))
    want = HO.norm_backward(WL.widen(x, dtype), WL.widen(dy, dtype), np64(mean), np64(rstd),
                            WL.widen(w, wdtype) if with_weight else None)
    for got, g, tol in zip((dx, dw, db), want, (half, F32, F32)):
        assert np.abs(np64(got) - g).max() <= tol * np.abs(g).max()


# Every group of warps works on several rows, at each length class of the backward.
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,dy_dtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,d", [(5000, 128), (9700, 136), (9700, 256), (1300, 2048), (900, 4104), (1000, 5128),
                                    (900, 6144), (900, 6152), (700, 8192)])
def test_backward_many_rows(rows, d, dtype, dy_dtype, kind):
    test_gpu_norm.test_backward(rows, d, dtype, dy_dtype, kind)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("rows,d", [(9700, 200), (1000, 5128), (700, 8192)])
def test_norm_and_checkpoint_many_rows(rows, d, kind):
    test_gpu_norm.test_norm_saves_and_reads_a_checkpoint(rows, d, "bf16", kind)


# Warps that take 1,024 values of a row or more, and short rows in one line.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(3000, 504), (1111, 512), (5000, 520), (5000, 1032), (2500, 4104), (5000, 2056),
                                    (1700, 8200), (2, 32), (1025, 8), (4097, 24)])
def test_checkpoint_many_rows(rows, d, dtype):
    test_gpu_norm.test_checkpoint_holds_the_oracles_codes(rows, d, dtype)
