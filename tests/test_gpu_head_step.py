"""The training step of the head that keeps its input in 8 bits only: x packed, H formed from the
codes for the forward and again for the backward, the norm's backward on the codes; eagerly and as
a graph, against the fp64 chain of the oracles at the values held.

lse_state belongs to the H it was computed from. H formed twice from one checkpoint is the same H
(test below, bit for bit), so one log-sum-exp serves both; H formed from x and H formed from x's
checkpoint are two, and each backward takes its own."""
import numpy as np
import pytest

from oracle import dpo_oracle as O
from oracle import head_ops_oracle as HO
from preference_alignment_b200 import libdpo
from preference_alignment_b200 import workloads as WL

from dpo_harness import TOL_GRAD, TOL_LOSS, TOL_TOK, assert_seq_close, np64, rel_frob, to_device

pytestmark = pytest.mark.gpu

N_TOP = 5


class Step:
    """One batch and the buffers of its step."""

    def __init__(self, dtype, kind, seed=33):
        import torch
        self.dtype, self.kind, layer = dtype, kind, kind == "layer"
        self.w = w = WL.make_custom(R=6, L=60, d=256, V=1500, dtype=dtype, seed=seed, full_rows=1)
        R, L, d, V = w.R, w.L, w.d, w.V
        rng = np.random.default_rng(seed)
        self.gs = WL.encode(rng.normal(1.0, 0.2, d).astype(np.float32), dtype)
        self.bs = WL.encode(rng.normal(0.0, 0.2, d).astype(np.float32), dtype)
        f32 = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
        self.x = to_device(w.H, dtype)
        self.gamma = to_device(self.gs, dtype)
        self.beta = to_device(self.bs, dtype) if layer else None
        self.W, self.tokens = to_device(w.W, dtype), torch.from_numpy(w.tokens).cuda()
        self.held = libdpo.Checkpoint.empty(R * L, d)
        self.H, self.H2 = torch.empty_like(self.x), torch.empty_like(self.x)
        self.mean, self.rstd = (f32(R * L) if layer else None), f32(R * L)
        self.b1, self.b2 = (libdpo.BatchArgs(H, self.W, self.tokens, w.prompt_len, w.completion_len,
                                             dtype=dtype) for H in (self.H, self.H2))
        n = self.b1.n_scored
        need = max(libdpo.workspace_size(self.b1)[1], libdpo.token_stats_size(self.b1, N_TOP)[0],
                   libdpo.norm_workspace_size(R * L, d))
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        self.logp, self.ent, self.lse, self.pol = f32(n), f32(n), f32(n), f32(R)
        self.ids, self.top = torch.empty(n, N_TOP, dtype=torch.int32, device="cuda"), f32(n, N_TOP)
        self.loss, self.coef = f32(1), f32(R)
        self.dH, self.dW, self.dx = f32(R, L, d), f32(V, d), torch.empty_like(self.x)
        self.dgamma, self.dbeta = f32(d), f32(d)

    def norm(self, x, H, **kw):
        rows, d = self.held.rows, self.held.d
        libdpo.norm_forward(x if x is self.held else x.view(rows, d), H.view(rows, d),
                            weight=self.gamma, bias=self.beta, kind=self.kind, **kw)

    def statistics(self, batch):
        libdpo.token_stats(batch, N_TOP, ws=self.ws, logp=self.logp, entropy=self.ent,
                           lse_state=self.lse, seq_logp=self.pol, top_ids=self.ids,
                           top_logp=self.top)

    def objective(self):
        libdpo.loss_ex(self.w.R // 2, self.w.layout, self.pol, None, self.w.beta, 1.0, self.loss,
                       row_coef=self.coef, reference_free=True)

    def norm_backward(self):
        libdpo.norm_backward(self.held, self.dH, self.mean, self.rstd,
                             dx=self.dx.view(self.held.rows, self.held.d), weight=self.gamma,
                             dweight=self.dgamma, dbias=self.dbeta, kind=self.kind, ws=self.ws)

    def run(self):
        libdpo.checkpoint_pack(self.x.view(self.held.rows, self.held.d), self.held)
        self.norm(self.held, self.H, mean=self.mean, rstd=self.rstd)
        self.statistics(self.b1)
        self.objective()
        self.norm(self.held, self.H2)
        libdpo.backward(self.b2, self.lse, self.coef, self.dH, self.dW, False, self.ws)
        self.norm_backward()

    def results(self):
        return [t.clone() for t in (self.logp, self.ent, self.lse, self.pol, self.ids, self.top,
                                    self.loss, self.dH, self.dW, self.dx, self.dgamma, self.dbeta)]

    def check(self):
        w, rows = self.w, self.held.rows
        Hd, Wd = np64(self.H), WL.widen(w.W, self.dtype)
        op = O.seq_logprobs(Hd, Wd, w.tokens, w.prompt_len, w.completion_len)
        assert_seq_close(np64(self.pol), op["seq_logp"])
        at = [(r, t) for r in range(w.R)
              for t in range(w.prompt_len[r] - 1, w.prompt_len[r] - 1 + w.completion_len[r])]
        st = HO.token_stats(np.array([Hd[r, t] for r, t in at]), Wd,
                            [w.tokens[r, t + 1] for r, t in at], N_TOP)
        assert np.abs(np64(self.logp) - st["logp"]).max() <= TOL_TOK
        assert np.abs(np64(self.ent) - st["entropy"]).max() <= TOL_TOK
        assert np.abs(np64(self.lse) - st["lse"]).max() <= TOL_TOK
        ol = O.dpo_loss(op["seq_logp"], np.zeros(w.R), w.beta, w.layout)
        assert abs(self.loss.item() - ol["loss"]) <= TOL_LOSS
        oH, oW = O.backward(Hd, Wd, w.tokens, w.prompt_len, w.completion_len, ol["row_coef"])
        assert rel_frob(np64(self.dH), oH) <= TOL_GRAD and rel_frob(np64(self.dW), oW) <= TOL_GRAD
        _, _, values = HO.checkpoint(WL.widen(w.H, self.dtype).reshape(rows, w.d))
        mean = np64(self.mean) if self.mean is not None else np.zeros(rows)
        want = HO.norm_backward(values, oH.reshape(rows, w.d), mean, np64(self.rstd),
                                WL.widen(self.gs, self.dtype), self.kind)
        # linear in dH: the same relative tolerance once more
        for got, o in zip((self.dx.view(rows, w.d), self.dgamma, self.dbeta), want):
            assert rel_frob(np64(got), o) <= 2 * TOL_GRAD


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_on_held_input_eagerly_and_as_a_graph(dtype, kind):
    import torch
    s = Step(dtype, kind)
    s.run()
    assert libdpo.check() == libdpo.OK
    assert torch.equal(s.H, s.H2)                  # one checkpoint, one H: its log-sum-exp serves both
    s.check()
    eager = s.results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for t in (s.H, s.H2, s.dH, s.dW, s.dx, s.lse, s.logp):
        t.fill_(float("nan"))
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert libdpo.check() == libdpo.OK
        for a, b in zip(eager, s.results()):
            assert torch.equal(a, b)
    # other inputs through the same graph
    other = Step(dtype, kind, seed=34)
    s.x.copy_(other.x)
    s.w.H = other.w.H
    graph.replay()
    torch.cuda.synchronize()
    s.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_h_formed_from_x_and_from_its_checkpoint_have_their_own_log_sum_exp(dtype):
    """The forward ran on x and saved its checkpoint; the backward runs on the H that the codes give,
    with the statistics of that H taken first: its probabilities sum to 1 and its gradients are
    the oracle's at that H."""
    s = Step(dtype, "layer")
    s.norm(s.x, s.H, mean=s.mean, rstd=s.rstd, save=s.held)
    s.statistics(s.b1)
    s.objective()
    of_x, coef = np64(s.lse), np64(s.coef)
    s.norm(s.held, s.H2)
    s.statistics(s.b2)
    libdpo.backward(s.b2, s.lse, s.coef, s.dH, s.dW, False, s.ws)
    assert libdpo.check() == libdpo.OK
    assert np.any(np64(s.lse) != of_x)                             # two H, two states
    w = s.w
    oH, oW = O.backward(np64(s.H2), WL.widen(w.W, dtype), w.tokens, w.prompt_len, w.completion_len, coef)
    assert rel_frob(np64(s.dH), oH) <= TOL_GRAD and rel_frob(np64(s.dW), oW) <= TOL_GRAD
