"""Token statistics against the fp64 oracle: log-prob, entropy, log-sum-exp and alternatives, in
both forms (a batch's scored positions, independent rows) and both element types.

Tolerances. A logit is a sum of d products, exact in fp32 each, added in fp32: in any order its
error is at most d * 2^-23 * sum |h w| (one half-step of 2^-24 per addition, twice that for sums
cut instead of rounded): `tz`. The log-sum-exp moves by at most tz. S = sum of V positive terms:
2^x is off by 2^-22 relative (the instruction's bound), its argument by |x| 2^-24 and terms
beyond |x| = 40 weigh less than 2^-40 each: 40 * 2^-24 < 2^-18; 256 terms of a tile added in turn
256 * 2^-24 = 2^-16; the join is fp64. So S and T are off by less than 2^-15 relative, log S by
2^-15 absolute, and the outputs round by 2^-24 relative. The entropy's derivative along a change
dz of the logits is -sum p_v (log p_v + ent) dz_v, at most tz * 2 ent <= 2 tz log V."""
import numpy as np
import pytest

from oracle import head_ops_oracle as HO
from preference_alignment_b200 import libdpo
from preference_alignment_b200 import workloads as WL

from dpo_harness import DeviceWorkload, np64, to_device

pytestmark = pytest.mark.gpu


def _draw(n, d, V, dtype, seed, scale=1.0, grid=False):
    """h, W as stored arrays and float64; `grid`: on grids coarse enough that every logit is
    exact in fp32, so the alternatives' order has one answer."""
    rng = np.random.default_rng(seed)
    h, W = rng.normal(size=(n, d)), rng.normal(size=(V, d)) * scale / np.sqrt(d)
    if grid:
        h = np.clip(np.rint(h * 8), -32, 32) / 8
        step = 2.0 ** (np.round(np.log2(scale / np.sqrt(d))) - 3)
        W = np.clip(np.rint(W / step), -32, 32) * step
    h, W = WL.encode(h.astype(np.float32), dtype), WL.encode(W.astype(np.float32), dtype)
    return h, W, WL.widen(h, dtype), WL.widen(W, dtype)


class Got:
    """Output buffers filled with a mark, so that what is not written shows."""

    def __init__(self, n, n_top, R=None):
        import torch
        nan = float("nan")
        self.logp, self.entropy, self.lse = (torch.full((n,), nan, device="cuda") for _ in range(3))
        self.ids = torch.full((n, n_top), -7, dtype=torch.int32, device="cuda") if n_top else None
        self.top = torch.full((n, n_top), nan, device="cuda") if n_top else None
        self.seq = torch.full((R,), nan, device="cuda") if R else None

    def args(self):
        return dict(logp=self.logp, entropy=self.entropy, lse_state=self.lse, top_ids=self.ids,
                    top_logp=self.top)


def _space(nbytes):
    import torch
    return torch.full((max(nbytes, 256),), 0xAB, dtype=torch.uint8, device="cuda")


def run_rows(h, W, dtype, tokens, n_top, ws_bytes=None, pad=0, stream=None):
    import torch
    H = to_device(h, dtype)
    if pad:
        wide = torch.full((h.shape[0], h.shape[1] + pad), float("nan"), device="cuda", dtype=H.dtype)
        wide[:, :h.shape[1]] = H
        H = wide[:, :h.shape[1]]
    Wd = to_device(W, dtype)
    t = torch.from_numpy(np.asarray(tokens, np.int32)).cuda() if tokens is not None else None
    full, _ = libdpo.token_stats_rows_size(h.shape[0], h.shape[1], W.shape[0], n_top, dtype)
    ws = _space(full if ws_bytes is None else ws_bytes)
    g = Got(h.shape[0], n_top)
    a = g.args()
    if tokens is None:
        a["logp"] = None
    libdpo.token_stats_rows(H, Wd, t, n_top, ws=ws, stream=stream, **a)
    return g


def check(g, o, n_top, tz, exact_ids=False):
    tz = np.asarray(tz)
    ts = 2.0 ** -15

    def near(got, want, tol):
        err = np.abs(np64(got) - want)
        assert np.all(err <= tol + 2.0 ** -23 * np.abs(want)), (err.max(), np.max(tol))

    near(g.lse, o["lse"], tz + ts)
    if "logp" in o:
        near(g.logp, o["logp"], 2 * tz + ts)
    V = o["z"].shape[1]
    near(g.entropy, o["entropy"], 2 * tz * np.log(max(V, 2)) + ts * (2 + 2 * np.log(max(V, 2))))
    if not n_top:
        return
    ids, top = g.ids.cpu().numpy(), np64(g.top)
    k = min(n_top, V)
    assert np.all(ids[:, k:] == -1) and np.all(np.isneginf(top[:, k:]))
    ids, top = ids[:, :k], top[:, :k]
    if exact_ids:
        assert np.array_equal(ids, o["top_ids"][:, :k])
    assert ids.min() >= 0 and ids.max() < V
    assert all(len(set(r)) == k for r in ids)
    zt = np.take_along_axis(o["z"], ids, axis=1)
    best = -np.sort(-o["z"], axis=1)[:, :k]
    t2 = np.broadcast_to(np.asarray(tz).reshape(-1, 1) if np.ndim(tz) else tz, zt.shape)
    assert np.all(np.abs(zt - best) <= 2 * t2 + 1e-12)      # rank j holds a logit as large as the j-th
    want = zt - o["lse"][:, None]
    assert np.all(np.abs(top - want) <= 2 * t2 + ts + 2.0 ** -23 * np.abs(want))


def _tz(hd, Wd):
    d = hd.shape[1]
    return d * 2.0 ** -23 * (np.abs(hd) @ np.abs(Wd).T).max(axis=1)


CASES = [  # n, d, V, n_top
    (1, 8, 1, 1), (1, 64, 2, 5), (3, 72, 7, 8), (2, 64, 255, 9), (5, 64, 256, 1), (5, 136, 257, 32),
    (1, 512, 5000, 20), (33, 64, 1000, 0), (127, 64, 511, 8), (128, 64, 513, 7), (129, 200, 700, 32),
    (255, 64, 300, 2), (257, 128, 2050, 8), (300, 1024, 1300, 32), (700, 64, 260, 3),
    (16, 72, 1184, 8), (17, 64, 9, 20), (32, 64, 19001, 8), (64, 64, 60001, 20), (64, 320, 2368, 32),
    (65, 64, 3000, 8), (2, 64, 130000, 32), (50, 8, 40007, 1),
    (3, 65536, 300, 8), (70, 16384, 260, 8),
    # more tiles than the block join takes (1,024), and more positions (1,024): the warp join
    (70, 8, 300001, 8), (3, 8, 33100, 20), (1100, 16, 700, 32), (1100, 16, 700, 1), (1030, 8, 300, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,V,n_top", CASES)
def test_rows_against_the_oracle(n, d, V, n_top, dtype):
    h, W, hd, Wd = _draw(n, d, V, dtype, seed=n * 1000 + V, scale=3.0)
    tokens = np.random.default_rng(n).integers(0, V, n)
    g = run_rows(h, W, dtype, tokens, n_top)
    assert libdpo.check() == libdpo.OK
    check(g, HO.token_stats(hd, Wd, tokens, n_top), n_top, _tz(hd, Wd))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,V,n_top", CASES)
def test_rows_exact_ids_on_a_grid(n, d, V, n_top, dtype):
    h, W, hd, Wd = _draw(n, d, V, dtype, seed=n * 77 + V, grid=True)
    tokens = np.random.default_rng(n).integers(0, V, n)
    g = run_rows(h, W, dtype, tokens, n_top, pad=8)
    assert libdpo.check() == libdpo.OK
    check(g, HO.token_stats(hd, Wd, tokens, n_top), n_top, 0.0, exact_ids=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_top", [1, 8, 32])
@pytest.mark.parametrize("n,V", [(40, 3001), (90, 3001), (1100, 900), (3, 40000)])
def test_equal_logits_come_by_id(n, V, n_top, dtype):
    """All logits equal: every tile's list is full of ties; and two levels only."""
    d = 64
    h = WL.encode(np.ones((n, d), np.float32), dtype)
    W = np.zeros((V, d), np.float32)
    o = run_rows(h, WL.encode(W, dtype), dtype, [0] * n, n_top)
    assert np.array_equal(o.ids.cpu().numpy(), np.tile(np.arange(n_top), (n, 1)))
    W[5::7, 0] = 1.0
    Ws = WL.encode(W, dtype)
    g = run_rows(h, Ws, dtype, [0] * n, n_top)
    check(g, HO.token_stats(WL.widen(h, dtype), WL.widen(Ws, dtype), [0] * n, n_top), n_top, 0.0,
          exact_ids=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("n,V,n_top", [(130, 2900, 8), (5, 2900, 32), (20, 4000, 8), (1030, 1100, 32)])
def test_sorted_vocabulary(n, V, n_top, rising, dtype):
    """Logits that rise along the vocabulary renew the alternatives in every tile; falling ones
    never after the first."""
    d = 8
    h = np.zeros((n, d), np.float32)
    h[:, 0], h[:, 1] = 1.0, 16.0                       # z = a + 16 b, a < 16, b < 256: distinct, exact
    v = np.arange(V) if rising else np.arange(V)[::-1]
    W = np.zeros((V, d), np.float32)
    W[:, 0], W[:, 1] = (v % 16) / 32.0, (v // 16) / 32.0
    h, W = WL.encode(h, dtype), WL.encode(W, dtype)
    g = run_rows(h, W, dtype, [3] * n, n_top)
    check(g, HO.token_stats(WL.widen(h, dtype), WL.widen(W, dtype), [3] * n, n_top), n_top, 0.0,
          exact_ids=True)


def test_zero_signs_are_one_value():
    """-0 and +0 tie."""
    n, d, V = 2, 8, 600
    h = np.zeros((n, d), np.float32)
    h[0, 0], h[1, 0] = 1.0, -1.0
    W = np.zeros((V, d), np.float32)
    for dtype in ("bf16", "f32"):
        g = run_rows(WL.encode(h, dtype), WL.encode(W, dtype), dtype, [0, 1], 20)
        assert np.array_equal(g.ids.cpu().numpy(), np.tile(np.arange(20), (n, 1)))


def test_large_logits():
    """Logits of +-thousands: one token holds all the mass, or two share it."""
    n, d, V = 3, 64, 900
    h = np.zeros((n, d), np.float32)
    h[:, 0] = [1.0, 64.0, -64.0]
    W = np.zeros((V, d), np.float32)
    W[:, 0] = -64.0
    W[17, 0] = W[600, 0] = 64.0
    h, W = WL.encode(h, "bf16"), WL.encode(W, "bf16")
    o = HO.token_stats(WL.widen(h, "bf16"), WL.widen(W, "bf16"), [17, 17, 0], 4)
    g = run_rows(h, W, "bf16", [17, 17, 0], 4)
    check(g, o, 4, 0.0, exact_ids=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nonfinite_hidden_rows_stay_by_themselves(dtype):
    import torch
    n, d, V, n_top = 6, 64, 700, 8
    h, W, hd, Wd = _draw(n, d, V, dtype, seed=5, grid=True)
    H = to_device(h, dtype)
    H[1, 3] = float("nan")
    H[4, 0] = float("inf")
    g = Got(n, n_top)
    ws = _space(libdpo.token_stats_rows_size(n, d, V, n_top, dtype)[0])
    t = torch.zeros(n, dtype=torch.int32, device="cuda")
    libdpo.token_stats_rows(H, to_device(W, dtype), t, n_top, ws=ws, **g.args())
    assert libdpo.check() == libdpo.OK
    for r in (1, 4):
        assert torch.isnan(g.entropy[r]) and torch.isnan(g.lse[r])
        assert ((g.ids[r] >= -1) & (g.ids[r] < V)).all()
    keep = [0, 2, 3, 5]
    o = HO.token_stats(hd[keep], Wd, [0] * 4, n_top)
    for name, got in (("lse", g.lse), ("entropy", g.entropy), ("logp", g.logp)):
        assert np.abs(np64(got)[keep] - o[name]).max() < 1e-4
    assert np.array_equal(g.ids.cpu().numpy()[keep], o["top_ids"])


def test_infinite_weight_rows():
    """W rows of -inf or +inf against positive hidden values: -inf logits weigh nothing and are no
    alternative; fewer finite logits than asked for end in -1."""
    import torch
    n, d, V, n_top = 2, 64, 520, 8
    for dtype in ("bf16", "f32"):
        H = to_device(WL.encode(np.ones((n, d), np.float32), dtype), dtype)
        W = to_device(WL.encode(np.zeros((V, d), np.float32), dtype), dtype)
        W[:, 0] = float("-inf")
        W[7, 0], W[300, 0], W[519, 0] = 1.0, 2.0, 1.0
        g = Got(n, n_top)
        t = torch.tensor([300, 0], dtype=torch.int32, device="cuda")
        ws = _space(libdpo.token_stats_rows_size(n, d, V, n_top, dtype)[0])
        libdpo.token_stats_rows(H, W, t, n_top, ws=ws, **g.args())
        assert libdpo.check() == libdpo.OK
        z = np.array([2.0, 1.0, 1.0])
        lse = np.log(np.exp(z).sum())
        p = np.exp(z - lse)
        assert np.abs(np64(g.lse) - lse).max() < 1e-5
        assert np.abs(np64(g.entropy) + (p * np.log(p)).sum()).max() < 1e-5
        assert np.isclose(g.logp[0].item(), 2 - lse, atol=1e-5) and g.logp[1].item() == -np.inf
        assert g.ids.tolist() == [[300, 7, 519, -1, -1, -1, -1, -1]] * n
        assert np.all(np.isneginf(np64(g.top)[:, 3:]))


def test_bad_tokens_and_no_tokens():
    h, W, hd, Wd = _draw(9, 64, 300, "bf16", seed=8)
    tokens = np.array([0, -1, 5, 300, 299, 1 << 30, -(1 << 31), 7, 8])
    g = run_rows(h, W, "bf16", tokens, 3)
    assert libdpo.check() == libdpo.ERR_BAD_TARGET and libdpo.check() == libdpo.OK
    o = HO.token_stats(hd, Wd, tokens, 3)
    check(g, o, 3, _tz(hd, Wd))
    assert np.all(np64(g.logp)[[1, 3, 5, 6]] == 0)
    g2 = run_rows(h, W, "bf16", None, 3)
    assert libdpo.check() == libdpo.OK
    assert np.array_equal(np64(g2.entropy), np64(g.entropy))
    assert np.all(np.isnan(np64(g2.logp)))               # not asked for, not written


@pytest.mark.parametrize("dtype,n", [("bf16", 700), ("f32", 100)])
def test_chunks_and_runs_give_the_same_bits(dtype, n):
    h, W, _, _ = _draw(n, 64, 1500, dtype, seed=4)
    tokens = np.arange(n) % 1500
    _, least = libdpo.token_stats_rows_size(n, 64, 1500, 8, dtype)
    a = run_rows(h, W, dtype, tokens, 8)
    for ws_bytes in (None, least, 2 * least):
        b = run_rows(h, W, dtype, tokens, 8, ws_bytes=ws_bytes)
        for x, y in ((a.logp, b.logp), (a.entropy, b.entropy), (a.lse, b.lse), (a.top, b.top),
                     (a.ids, b.ids)):
            assert np.array_equal(x.cpu().numpy(), y.cpu().numpy())


def _batch_oracle(w, n_top):
    H, W = WL.widen(w.H, w.dtype), WL.widen(w.W, w.dtype)
    at = [(r, t) for r in range(w.R)
          for t in range(w.prompt_len[r] - 1, w.prompt_len[r] - 1 + w.completion_len[r])]
    h = np.array([H[r, t] for r, t in at]).reshape(-1, w.d)
    tok = np.array([w.tokens[r, t + 1] for r, t in at], np.int64)
    return at, h, HO.token_stats(h, W, tok, n_top) if at else None


@pytest.mark.parametrize("R,L,d,V,dtype,n_top", [
    (4, 40, 64, 1000, "f32", 5), (6, 50, 72, 300, "bf16", 1), (8, 130, 128, 2000, "bf16", 8),
    (2, 2, 8, 5, "bf16", 32), (2, 9, 64, 259, "f32", 0), (10, 90, 256, 513, "bf16", 20),
])
def test_batch_against_the_oracle_and_the_forward(R, L, d, V, dtype, n_top):
    w = WL.make_custom(R=R, L=L, d=d, V=V, dtype=dtype, seed=R * 100 + V, full_rows=1)
    w.completion_len[-1] = 0                              # a row that scores nothing
    dw = DeviceWorkload(w)
    b = dw.batch()
    at, h, o = _batch_oracle(w, n_top)
    full, least = libdpo.token_stats_size(b, n_top)
    for ws_bytes in (full, least):
        g = Got(len(at), n_top, R)
        libdpo.token_stats(b, n_top, ws=_space(ws_bytes), seq_logp=g.seq, **g.args())
        assert libdpo.check() == libdpo.OK
        tz = _tz(h, WL.widen(w.W, dtype))
        check(g, o, n_top, tz)
        want = np.zeros(R)
        for (r, _), v in zip(at, np64(g.logp)):
            want[r] += v
        assert np.all(np.abs(np64(g.seq) - want) <= 2.0 ** -23 * np.abs(want) + 1e-12)
    seq, _, lse = dw.forward()
    n = len(at)
    assert np.abs(np64(g.lse) - np64(lse)[:n]).max() < 1e-4      # what backward() may read
    assert np.abs(np64(g.seq) - np64(seq)).max() < 1e-3
    # sums alone, without any per-position output
    s2 = Got(n, 0, R)
    libdpo.token_stats(b, 0, ws=_space(libdpo.token_stats_size(b, 0)[0]), seq_logp=s2.seq)
    assert np.array_equal(np64(s2.seq), np64(g.seq))


def test_batch_without_scored_positions():
    import torch
    w = WL.make_custom(R=4, L=8, d=64, V=100, seed=3)
    w.completion_len[:] = 0
    b = DeviceWorkload(w).batch()
    seq = torch.full((4,), float("nan"), device="cuda")
    libdpo.token_stats(b, 3, ws=_space(libdpo.token_stats_size(b, 3)[0]), seq_logp=seq,
                       top_ids=torch.empty(1, 3, dtype=torch.int32, device="cuda"),
                       top_logp=torch.empty(1, 3, device="cuda"))
    assert libdpo.check() == libdpo.OK and np.all(np64(seq) == 0)


def test_large_batch_chunks():
    """More positions than one launch takes (8,192)."""
    n, d, V, n_top = 9000, 64, 777, 4
    h, W, hd, Wd = _draw(n, d, V, "bf16", seed=12, grid=True)
    tokens = np.arange(n) % V
    g = run_rows(h, W, "bf16", tokens, n_top)
    assert libdpo.check() == libdpo.OK
    check(g, HO.token_stats(hd, Wd, tokens, n_top), n_top, 0.0, exact_ids=True)


@pytest.mark.parametrize("n", [3, 300])
def test_captured_and_on_another_stream(n):
    """A captured call replayed with other inputs gives that input's values; a call on a side
    stream the same."""
    import torch
    d, V, n_top = 64, 2100, 8
    h, W, hd, Wd = _draw(n, d, V, "bf16", seed=31, grid=True)
    h2 = _draw(n, d, V, "bf16", seed=32, grid=True)
    tokens = np.arange(n) % V
    H, Wt = to_device(h, "bf16"), to_device(W, "bf16")
    t = torch.from_numpy(tokens.astype(np.int32)).cuda()
    ws = _space(libdpo.token_stats_rows_size(n, d, V, n_top)[0])
    g = Got(n, n_top)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        libdpo.token_stats_rows(H, Wt, t, n_top, ws=ws, **g.args())
    torch.cuda.current_stream().wait_stream(side)
    check(g, HO.token_stats(hd, Wd, tokens, n_top), n_top, 0.0, exact_ids=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        libdpo.token_stats_rows(H, Wt, t, n_top, ws=ws, **g.args())
    for src in (h2, (h, W, hd, Wd)):
        H.copy_(to_device(src[0], "bf16"))
        ws.fill_(0xCD)
        graph.replay()
        torch.cuda.synchronize()
        check(g, HO.token_stats(src[2], Wd, tokens, n_top), n_top, 0.0, exact_ids=True)
    assert libdpo.check() == libdpo.OK


def test_gemm_kernels_agree():
    """The single-CTA kernel and the static schedule give the same statistics."""
    h, W, hd, Wd = _draw(400, 128, 3000, "bf16", seed=6, grid=True)
    tokens = np.arange(400)
    o = HO.token_stats(hd, Wd, tokens, 20)
    for mask in (0, 1, 16):
        old = libdpo.set_gemm_variant(mask)
        try:
            g = run_rows(h, W, "bf16", tokens, 20)
            assert libdpo.check() == libdpo.OK
            check(g, o, 20, 0.0, exact_ids=True)
        finally:
            libdpo.set_gemm_variant(old)


def test_largest_vocabulary():
    """2^24 rows: every CTA walks 886 tiles, ids pass 2^24 - 256."""
    import torch
    n, d, V, n_top = 2, 8, 1 << 24, 8
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    W = (torch.randint(-128, 128, (V, d), generator=gen, device="cuda") / 64).bfloat16()   # exact
    H = (torch.randint(-8, 8, (n, d), generator=gen, device="cuda") / 4).bfloat16()
    t = torch.tensor([V - 1, 0], dtype=torch.int32, device="cuda")
    g = Got(n, n_top)
    libdpo.token_stats_rows(H, W, t, n_top, ws=_space(libdpo.token_stats_rows_size(n, d, V, n_top)[0]),
                            **g.args())
    assert libdpo.check() == libdpo.OK
    check(g, HO.token_stats(np64(H), np64(W), t.cpu().numpy(), n_top), n_top, 0.0, exact_ids=True)


@pytest.mark.parametrize("n_top", [4, 8, 20, 32])
@pytest.mark.parametrize("n", [16, 64])
def test_equal_logits_across_the_tiles_of_a_cta(n, n_top):
    """Levels of equal logits that fill up over two tiles of 128 rows: those of the later tile come by
    id, whichever segment of it is worked on first. Position p has its largest ones in CTA 2 p's tiles,
    in lists of very different lengths."""
    import torch
    d, tiles, ctas, rows = 64, 6, 148, 128
    V = rows * tiles * ctas
    v = np.arange(V)
    # one workspace: what an earlier call left there counts for nothing
    ws = torch.empty(libdpo.token_stats_rows_size(n, d, V, n_top)[0], dtype=torch.uint8, device="cuda")
    for seed in range(8):
        rng = np.random.default_rng(seed)
        level = v // (rows * ctas) // 2
        z = np.where(rng.random((V, d)) < 0.05 * (1 + seed % 3), level[:, None] + 1, 0).astype(np.float32)
        z[(v[:, None] // rows) % ctas == 2 * np.arange(d)[None, :]] += 8
        H = torch.eye(d, dtype=torch.bfloat16, device="cuda")[:n]      # position p's logits: column p
        ids = torch.empty(n, n_top, dtype=torch.int32, device="cuda")
        top = torch.empty(n, n_top, device="cuda")
        W = torch.from_numpy(z).cuda().bfloat16()
        want = np.stack([np.lexsort((v, -z[:, p]))[:n_top] for p in range(n)])
        for _ in range(5):
            libdpo.token_stats_rows(H, W, None, n_top, top_ids=ids, top_logp=top, ws=ws)
            assert np.array_equal(ids.cpu().numpy(), want)
    assert libdpo.check() == libdpo.OK
