"""The operators together, as a training step of the head uses them: final norm (holding its
input in 8 bits) -> token statistics -> loss -> the head's backward -> the norm's backward, against
the fp64 chain of the oracles."""
import numpy as np
import pytest

from oracle import dpo_oracle as O
from oracle import head_ops_oracle as HO
from preference_alignment_b200 import libdpo
from preference_alignment_b200 import workloads as WL

from dpo_harness import TOL_GRAD, TOL_LOSS, TOL_TOK, assert_seq_close, np64, rel_frob, to_device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_through_norm_statistics_and_checkpoint(dtype, kind):
    import torch
    layer = kind == "layer"
    w = WL.make_custom(R=6, L=60, d=256, V=1500, dtype=dtype, seed=21, full_rows=1)
    R, L, d, V, n_top = w.R, w.L, w.d, w.V, 5
    rng = np.random.default_rng(4)
    gs = WL.encode(rng.normal(1.0, 0.2, d).astype(np.float32), dtype)
    bs = WL.encode(rng.normal(0.0, 0.2, d).astype(np.float32), dtype)
    x, gamma = to_device(w.H, dtype), to_device(gs, dtype)
    beta = to_device(bs, dtype) if layer else None
    W, tokens = to_device(w.W, dtype), torch.from_numpy(w.tokens).cuda()
    f32 = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731

    H = torch.empty_like(x)
    mean, rstd = f32(R * L), f32(R * L)
    held = libdpo.Checkpoint.empty(R * L, d)
    libdpo.norm_forward(x, H, weight=gamma, bias=beta, kind=kind, mean=mean if layer else None,
                        rstd=rstd, save=held)
    batch = libdpo.BatchArgs(H, W, tokens, w.prompt_len, w.completion_len, dtype=dtype)
    n = batch.n_scored
    _, bwd, _ = libdpo.workspace_size(batch)
    ws = torch.empty(max(bwd, libdpo.token_stats_size(batch, n_top)[0],
                         libdpo.norm_workspace_size(R * L, d)), dtype=torch.uint8, device="cuda")
    logp, ent, lse, pol = f32(n), f32(n), f32(n), f32(R)
    ids, top = torch.empty(n, n_top, dtype=torch.int32, device="cuda"), f32(n, n_top)
    libdpo.token_stats(batch, n_top, ws=ws, logp=logp, entropy=ent, lse_state=lse, seq_logp=pol,
                       top_ids=ids, top_logp=top)
    B = R // 2
    loss, coef = f32(1), f32(R)
    libdpo.loss_ex(B, w.layout, pol, None, w.beta, 1.0, loss, row_coef=coef, reference_free=True)
    # H is formed again from the 8 bits where the backward needs it
    H2 = torch.empty_like(H)
    libdpo.norm_forward(held, H2.view(R * L, d), weight=gamma, bias=beta, kind=kind)
    batch2 = libdpo.BatchArgs(H2, W, tokens, w.prompt_len, w.completion_len, dtype=dtype)
    dH, dW = f32(R, L, d), f32(V, d)
    libdpo.backward(batch, lse, coef, dH, dW, False, ws)
    dx, dgamma, dbeta = torch.empty_like(x), f32(d), f32(d)
    libdpo.norm_backward(held, dH, mean if layer else None, rstd, dx=dx.view(R * L, d), weight=gamma,
                         dweight=dgamma, dbias=dbeta, kind=kind, ws=ws)
    dW2 = f32(V, d)
    libdpo.backward(batch2, lse, coef, None, dW2, False, ws)
    assert libdpo.check() == libdpo.OK

    # the head on the H the GPU formed (its rounding is checked with the norm's own tests)
    Hd, Wd = np64(H), WL.widen(w.W, dtype)
    op = O.seq_logprobs(Hd, Wd, w.tokens, w.prompt_len, w.completion_len)
    assert_seq_close(np64(pol), op["seq_logp"])
    at = [(r, t) for r in range(R)
          for t in range(w.prompt_len[r] - 1, w.prompt_len[r] - 1 + w.completion_len[r])]
    hs = np.array([Hd[r, t] for r, t in at])
    st = HO.token_stats(hs, Wd, [w.tokens[r, t + 1] for r, t in at], n_top)
    assert np.abs(np64(logp) - st["logp"]).max() <= TOL_TOK
    assert np.abs(np64(ent) - st["entropy"]).max() <= TOL_TOK
    picked = np.take_along_axis(st["z"], ids.cpu().numpy().astype(np.int64), axis=1)
    assert np.abs(picked - st["lse"][:, None] - np64(top)).max() <= TOL_TOK
    ol = O.dpo_loss(op["seq_logp"], np.zeros(R), w.beta, w.layout)
    assert abs(loss.item() - ol["loss"]) <= TOL_LOSS
    oH, oW = O.backward(Hd, Wd, w.tokens, w.prompt_len, w.completion_len, ol["row_coef"])
    assert rel_frob(np64(dH), oH) <= TOL_GRAD and rel_frob(np64(dW), oW) <= TOL_GRAD
    # the norm's backward is linear in dH: the same relative tolerance on its results
    _, _, values = HO.checkpoint(WL.widen(w.H, dtype).reshape(R * L, d))
    want = HO.norm_backward(values, oH.reshape(R * L, d), np64(mean), np64(rstd),
                            WL.widen(gs, dtype), kind)
    for got, o in zip((dx.view(R * L, d), dgamma, dbeta), want):
        assert rel_frob(np64(got), o) <= 2 * TOL_GRAD
    # H from the 8 bits: off by the codes' rounding, 2^-8 of a block's largest value at most, so
    # within 2 % of H (rms of a uniform error 2^-8 / sqrt(3) of a maximum about 2.5 sigma: 0.6 %)
    assert rel_frob(np64(H2), Hd) <= 0.02 and rel_frob(np64(dW2), oW) <= 0.05
