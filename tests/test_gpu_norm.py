"""The norm before the head and 8-bit checkpoints against the fp64 oracle.

Tolerances. Sums over a row of d values run at most d/32 + 16 additions deep per thread and tree,
each off by half a step of its partial sum: gamma = (d / 32 + 16) * 2^-24 relative to the sum of
magnitudes. So mean is off by gamma mean|x|; the sum of squares by gamma (all terms positive) plus
twice the mean's error over the spread, which enters squared and is far below; 1 / sqrt halves
that; the steps after it round a few times (8 * 2^-24). An element (x - mu) r w + b is then off by
its own rounding, by r w times the mean's error and by its relative error in r. The gradients:
see _grad_tol. bf16 outputs round by half a step, 2^-8 relative (finfo.eps / 2), fp32 ones by
2^-24."""
import numpy as np
import pytest

from oracle import head_ops_oracle as HO
from preference_alignment_b200 import libdpo
from preference_alignment_b200 import workloads as WL

from dpo_harness import np64, to_device

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SHAPES = [(1, 8), (3, 24), (2, 40), (5, 256), (33, 264), (7, 512), (4, 1000), (300, 1024), (9, 2048),
          (5, 4104), (3, 8192), (3, 8200), (2, 16384), (2, 65536), (2000, 16), (650, 2056)]


def _gamma(d):
    return (d / 32 + 16) * 2.0 ** -24


def _rows(rows, d, dtype, seed, scale=1.0, offset=0.0):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, d)) * scale + offset
    x[:, rng.random(d) < 0.02] *= 20
    s = WL.encode(x.astype(np.float32), dtype)
    return s, WL.widen(s, dtype)


def _vec(d, dtype, seed, center):
    s = WL.encode(np.random.default_rng(seed).normal(center, 0.3, d).astype(np.float32), dtype)
    return s, WL.widen(s, dtype)


def _dev(s, dtype, pad=0):
    import torch
    t = to_device(s, dtype)
    if not pad:
        return t
    wide = torch.full((s.shape[0], s.shape[1] + pad), 9.0, device="cuda", dtype=t.dtype)
    wide[:, :s.shape[1]] = t
    return wide[:, :s.shape[1]]


def _empty(rows, d, dtype, pad=0):
    import torch
    kind = torch.bfloat16 if dtype == "bf16" else torch.float32
    return torch.full((rows, d + pad), 9.0, device="cuda", dtype=kind)[:, :d]


def _f32(n):
    import torch
    return torch.full((n,), float("nan"), device="cuda")


def _ws(rows, d):
    import torch
    return torch.full((libdpo.norm_workspace_size(rows, d),), 0xAB, dtype=torch.uint8, device="cuda")


def _check_forward(x, w, b, kind, eps, y, mean, rstd, dtype):
    oy, om, orr = HO.norm_forward(x, w, b, kind, eps)
    d = x.shape[1]
    gm = _gamma(d)
    tm = gm * np.abs(x).mean(axis=1) + 2.0 ** -24 * np.abs(om) if kind == "layer" else np.zeros(len(x))
    if mean is not None:
        assert np.all(np.abs(np64(mean) - om) <= tm)
    # the mean's error shifts every x - mu: squared in the variance, so relative to it (tm r)^2
    tr = gm + (tm * orr) ** 2 + 8 * 2.0 ** -24
    assert np.all(np.abs(np64(rstd) / orr - 1) <= tr)
    aw = np.abs(w) if w is not None else 1.0
    core = np.abs(x - om[:, None]) * orr[:, None] * aw
    tol = core * (tr[:, None] + 3 * 2.0 ** -24) + (tm * orr)[:, None] * aw
    tol = tol + 2.0 ** -24 * (np.abs(b) if b is not None else 0) + HALF[dtype] * np.abs(oy)
    # rounding a value that is off by tol adds half a step of tol
    assert np.all(np.abs(np64(y) - oy) <= tol * (1 + HALF[dtype]) + 1e-30)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward(rows, d, dtype, wdtype, kind):
    xs, x = _rows(rows, d, dtype, rows + d, offset=0.5)
    ws, w = _vec(d, wdtype, 1, 1.0)
    bs, b = _vec(d, wdtype, 2, 0.0)
    y, mean, rstd = _empty(rows, d, dtype, 16), _f32(rows), _f32(rows)
    layer = kind == "layer"
    libdpo.norm_forward(_dev(xs, dtype, 8), y, weight=to_device(ws, wdtype), bias=to_device(bs, wdtype),
                        kind=kind, eps=1e-5, mean=mean if layer else None, rstd=rstd)
    _check_forward(x, w, b, kind, 1e-5, y, mean if layer else None, rstd, dtype)
    if rows > 1:
        assert (y._base[:, d:] == 9).all()                # between the rows: as it was
    # without weight, bias, statistics; and in place
    xd = _dev(xs, dtype)
    libdpo.norm_forward(xd, xd, kind=kind, eps=0.25, rstd=rstd)
    _check_forward(x, None, None, kind, 0.25, xd, None, rstd, dtype)


def _grad_tol(x, dy, mean, rstd, w, kind, dtype, rows):
    """Bounds of dx, dweight, dbias: row sums are off by gamma of their magnitudes plus four
    roundings of each term, an element of dx by that and a few roundings of its own terms; a
    column sum over the rows by (rows + 32) half-steps of its magnitudes at most, its terms by
    three roundings each."""
    d = x.shape[1]
    g = np.abs(dy) * (np.abs(w) if w is not None else 1.0)
    mu = mean[:, None] if kind == "layer" else 0.0
    xh = np.abs(x - mu) * rstd[:, None]
    gm = _gamma(d) + 8 * 2.0 ** -24
    terms = g + xh * (g * xh).mean(axis=1, keepdims=True)
    if kind == "layer":
        terms = terms + g.mean(axis=1, keepdims=True)
    cols = (rows + 32) * 2.0 ** -24
    return (rstd[:, None] * terms * gm, (np.abs(dy) * xh).sum(axis=0) * (cols + 3 * 2.0 ** -24),
            np.abs(dy).sum(axis=0) * cols)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,dy_dtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"),
                                            ("f32", "bf16")])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_backward(rows, d, dtype, dy_dtype, kind):
    import torch
    xs, x = _rows(rows, d, dtype, rows + d + 1, offset=0.5)
    ws, w = _vec(d, dtype, 3, 1.0)
    dys, dy = _rows(rows, d, dy_dtype, 5, scale=1e-2)
    if rows > 2:
        dys[1], dy[1] = 0, 0                              # a row without gradient
    layer = kind == "layer"
    _, om, orr = HO.norm_forward(x, None, None, kind)
    mean = torch.from_numpy(om.astype(np.float32)).cuda()
    rstd = torch.from_numpy(orr.astype(np.float32)).cuda()
    dx, dw, db = _empty(rows, d, dtype, 8), _f32(d), _f32(d)
    args = dict(weight=to_device(ws, dtype), kind=kind, ws=_ws(rows, d))
    xd, dyd = _dev(xs, dtype, 16), _dev(dys, dy_dtype, 8)
    libdpo.norm_backward(xd, dyd, mean if layer else None, rstd, dx=dx, dweight=dw, dbias=db, **args)
    want = HO.norm_backward(x, dy, np64(mean), np64(rstd), w, kind)
    tol = _grad_tol(x, dy, np64(mean), np64(rstd), w, kind, dtype, rows)
    for got, o, t, half in zip((dx, dw, db), want, tol, (HALF[dtype], 2.0 ** -24, 2.0 ** -24)):
        assert np.all(np.abs(np64(got) - o) <= (t + half * np.abs(o)) * 1.01 + 1e-30)
    if rows > 2:
        assert (dx[1] == 0).all()
    if rows > 1:
        assert (dx._base[:, d:] == 9).all()
    # the same call again: the same bits; the gradients added on top; each output left out
    dx2, dw2, db2 = _empty(rows, d, dtype), dw.clone(), db.clone()
    libdpo.norm_backward(xd, dyd, mean if layer else None, rstd, dx=dx2, dweight=dw2, dbias=db2,
                         accumulate=True, **args)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw + dw) and torch.equal(db2, db + db)
    only = _f32(d)
    libdpo.norm_backward(xd, dyd, mean if layer else None, rstd, dbias=only, **args)
    assert torch.equal(only, db)
    dx3 = _empty(rows, d, dtype)
    libdpo.norm_backward(xd, dyd, mean if layer else None, rstd, dx=dx3, **args)
    assert torch.equal(dx3, dx)
    if dtype == dy_dtype:                                 # dx in dy's place
        libdpo.norm_backward(xd, dyd, mean if layer else None, rstd, dx=dyd, dweight=dw2, **args)
        assert torch.equal(dyd, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_backward_against_differences(kind):
    """The fp32 forward's differences: the objective sum(y * c) at x +- h v along directions v."""
    import torch
    rows, d = 6, 64
    rng = np.random.default_rng(11)
    x, c, v = (rng.normal(size=(rows, d)).astype(np.float32) for _ in range(3))
    w, vw = (rng.normal(size=d).astype(np.float32) for _ in range(2))

    def f(x, w):
        y = _empty(rows, d, "f32")
        libdpo.norm_forward(to_device(x, "f32"), y, weight=to_device(w, "f32"), kind=kind)
        return (np64(y) * c).sum()

    y, mean, rstd = _empty(rows, d, "f32"), _f32(rows), _f32(rows)
    libdpo.norm_forward(to_device(x, "f32"), y, weight=to_device(w, "f32"), kind=kind,
                        mean=mean if kind == "layer" else None, rstd=rstd)
    dx, dw = _empty(rows, d, "f32"), _f32(d)
    libdpo.norm_backward(to_device(x, "f32"), to_device(c, "f32"), mean if kind == "layer" else None,
                         rstd, dx=dx, weight=to_device(w, "f32"), dweight=dw, kind=kind,
                         ws=_ws(rows, d))
    h = 2.0 ** -6
    # fp32 values of size up to 4 in 384 terms: noise of f about 384^0.5 * 4 * 2^-23, over 2h about
    # 3e-4 (the sum is taken in fp64); third-order term h^2 |f'''| / 6 about 2^-12 * 100 / 6
    tol = 1e-2
    assert abs((f(x + h * v, w) - f(x - h * v, w)) / (2 * h) - (np64(dx) * v).sum()) < tol * rows
    assert abs((f(x, w + h * vw) - f(x, w - h * vw)) / (2 * h) - (np64(dw) * vw).sum()) < tol


def test_nonfinite_rows_stay_by_themselves():
    import torch
    rows, d = 5, 320
    xs, x = _rows(rows, d, "f32", 3)
    xd = to_device(xs, "f32")
    xd[2, 7] = float("nan")
    xd[4, 0] = float("inf")
    y, rstd = _empty(rows, d, "f32"), _f32(rows)
    libdpo.norm_forward(xd, y, rstd=rstd)
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[4]).any()
    keep = [0, 1, 3]
    _check_forward(x[keep], None, None, "layer", 1e-5, y[keep], None, rstd[keep], "f32")


def test_constant_row_and_zero_row():
    """No spread: rstd is 1 / sqrt(eps) and y the bias."""
    import torch
    x = torch.full((2, 512), 3.0, device="cuda")
    x[1] = 0
    y, mean, rstd = _empty(2, 512, "f32"), _f32(2), _f32(2)
    b = torch.full((512,), 0.25, device="cuda")
    libdpo.norm_forward(x, y, bias=b, eps=1e-4, mean=mean, rstd=rstd)
    assert (y == 0.25).all() and mean.tolist() == [3.0, 0.0]
    assert np.allclose(np64(rstd), 100.0, rtol=1e-6)


@pytest.mark.parametrize("d", [64, 16384])
def test_no_rows(d):
    import torch
    x = torch.empty(0, d, device="cuda")
    libdpo.norm_forward(x, x)
    dw, db = _f32(d), _f32(d)
    libdpo.norm_backward(x, x, _f32(0), _f32(0), dweight=dw, dbias=db, ws=_ws(0, d))
    assert (dw == 0).all() and (db == 0).all()
    dw.fill_(2)
    libdpo.norm_backward(x, x, _f32(0), _f32(0), dweight=dw, accumulate=True, ws=_ws(0, d))
    assert (dw == 2).all()
    libdpo.checkpoint_pack(x, libdpo.Checkpoint.empty(0, d))


# ------------------------------------------------------------------ checkpoints
def _mixed(rows, d, dtype, seed):
    """Rows of very different sizes, zeros, and values on the scale's borders."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, d)) * 2.0 ** rng.integers(-20, 20, (rows, d // 8 + 1)).repeat(8, 1)[:, :d]
    x[0, : min(d, 8)] = [127.0, 127.5, 63.5, 0.5, -0.5, 1.5, -2.5, 126.5][: min(d, 8)]
    if rows > 2:
        x[1] = 0
        x[2, ::3] = 0
    if rows > 4:
        x[3] *= 1e-38 * 2.0 ** -20
        x[4] = np.sign(x[4]) * 3.38e38
    s = WL.encode(x.astype(np.float32), dtype)
    return s, WL.widen(s, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(1, 8), (2, 24), (9, 32), (5, 40), (7, 1000), (40, 1032), (3, 2056),
                                    (6, 4096), (2, 65536), (5000, 8)])
def test_checkpoint_holds_the_oracles_codes(rows, d, dtype):
    import torch
    s, x = _mixed(rows, d, dtype, rows + d)
    if d >= 64 and rows > 4:
        s = s.copy()
        x = x.copy()
        nan = np.array([np.nan, np.inf], np.float32)
        s[0, 33:35] = WL.encode(nan, dtype)
        x[0, 33:35] = nan
    held = libdpo.Checkpoint(torch.full((rows, d), 99, dtype=torch.int8, device="cuda"),
                             torch.full((rows, -(-d // 32)), 77, dtype=torch.uint8, device="cuda"))
    libdpo.checkpoint_pack(_dev(s, dtype, 8), held)
    codes, scales, values = HO.checkpoint(x)
    assert np.array_equal(held.scales.cpu().numpy(), scales)
    assert np.array_equal(held.codes.cpu().numpy(), codes)
    for out in ("f32", "bf16"):                          # both hold the values exactly
        y = _empty(rows, d, out, 16)
        libdpo.checkpoint_unpack(held, y)
        assert np.array_equal(np64(y), values, equal_nan=True)
        if rows > 1:
            assert (y._base[:, d:] == 9).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(1, 8), (5, 40), (33, 264), (300, 1024), (4, 4104), (3, 8192),
                                    (3, 8200), (2, 65536)])
def test_norm_saves_and_reads_a_checkpoint(rows, d, dtype, kind):
    import torch
    layer = kind == "layer"
    xs, x = _rows(rows, d, dtype, rows + d + 7, offset=0.5)
    ws, w = _vec(d, dtype, 3, 1.0)
    dys, dy = _rows(rows, d, "f32", 5, scale=1e-2)
    held = libdpo.Checkpoint.empty(rows, d)
    xd, wd = _dev(xs, dtype), to_device(ws, dtype)
    y, y0 = _empty(rows, d, dtype), _empty(rows, d, dtype)
    mean, rstd = _f32(rows), _f32(rows)
    libdpo.norm_forward(xd, y0, weight=wd, kind=kind)
    libdpo.norm_forward(xd, y, weight=wd, kind=kind, mean=mean if layer else None, rstd=rstd, save=held)
    assert torch.equal(y, y0)
    codes, scales, values = HO.checkpoint(x)
    assert np.array_equal(held.codes.cpu().numpy(), codes)
    assert np.array_equal(held.scales.cpu().numpy(), scales)
    # the forward again, from what is held
    y2, mean2, rstd2 = _empty(rows, d, dtype), _f32(rows), _f32(rows)
    libdpo.norm_forward(held, y2, weight=wd, kind=kind, mean=mean2 if layer else None, rstd=rstd2)
    _check_forward(values, w, None, kind, 1e-5, y2, mean2 if layer else None, rstd2, dtype)
    # the backward from what is held, on the forward's statistics
    dx, dw, db = _empty(rows, d, dtype), _f32(d), _f32(d)
    m = mean if layer else None
    libdpo.norm_backward(held, to_device(dys, "f32"), m, rstd, dx=dx, weight=wd, dweight=dw, dbias=db,
                         kind=kind, ws=_ws(rows, d))
    om = np64(mean) if layer else np.zeros(rows)
    want = HO.norm_backward(values, dy, om, np64(rstd), w, kind)
    tol = _grad_tol(values, dy, om, np64(rstd), w, kind, dtype, rows)
    for got, o, t, half in zip((dx, dw, db), want, tol, (HALF[dtype], 2.0 ** -24, 2.0 ** -24)):
        assert np.all(np.abs(np64(got) - o) <= (t + half * np.abs(o)) * 1.01 + 1e-30)


def test_captured_together_and_on_another_stream():
    import torch
    rows, d = 500, 1024
    xs, _ = _rows(rows, d, "bf16", 1)
    x2, _ = _rows(rows, d, "bf16", 2)
    dys, _ = _rows(rows, d, "f32", 3)
    x, dy = to_device(xs, "bf16"), to_device(dys, "f32")
    w = torch.ones(d, device="cuda")
    held = libdpo.Checkpoint.empty(rows, d)
    ws = _ws(rows, d)

    def step():
        y, mean, rstd = _empty(rows, d, "bf16"), _f32(rows), _f32(rows)
        dx, dw = _empty(rows, d, "bf16"), _f32(d)
        libdpo.norm_forward(x, y, weight=w, mean=mean, rstd=rstd, save=held)
        libdpo.norm_backward(held, dy, mean, rstd, dx=dx, weight=w, dweight=dw, ws=ws)
        return y, dx, dw

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for s in (x2, xs):
        x.copy_(to_device(s, "bf16"))
        graph.replay()
        kept = [t.clone() for t in got]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, again))
