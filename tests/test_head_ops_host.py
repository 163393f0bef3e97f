"""Refusals of the token statistics, norm and checkpoint calls: every one is returned by the
host checks, before any CUDA call, so they run without a GPU."""
import ctypes

import numpy as np
import pytest

from preference_alignment_b200 import build as B
from preference_alignment_b200 import libdpo

FAKE = 0x100000     # never dereferenced: the checks fail first
INVALID, UNSUPPORTED, WORKSPACE = (libdpo.ERR_INVALID_ARG, libdpo.ERR_UNSUPPORTED,
                                   libdpo.ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return libdpo.load()


def _batch(R=4, L=32, d=64, V=1000, dtype="bf16"):
    return libdpo.BatchArgs(FAKE, FAKE, FAKE, np.full(R, 4, np.int32), np.full(R, 10, np.int32),
                            R=R, L=L, d=d, V=V, dtype=dtype)


def _out(n_top=0, ids=None, top=None, logp=FAKE):
    return libdpo.TokenStatsOut(logp, None, None, n_top, ids, top)


def _stats(lib, batch, out, ws=FAKE, nbytes=1 << 40):
    fn = libdpo._fn("dpo_token_stats", [ctypes.POINTER(libdpo.Batch),
                                        ctypes.POINTER(libdpo.TokenStatsOut), ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p])
    return fn(ctypes.byref(batch.c), ctypes.byref(out) if out is not None else None, None, ws,
              nbytes, None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_top", [0, 1, 8, 20, 32])
def test_stats_sizes(lib, dtype, n_top):
    full, least = libdpo.token_stats_size(_batch(R=64, L=600, d=64, V=3000, dtype=dtype), n_top)
    assert 0 < least <= full
    one, one_min = libdpo.token_stats_rows_size(1, 64, 3000, n_top, dtype)
    many, many_min = libdpo.token_stats_rows_size(100000, 64, 3000, n_top, dtype)
    assert one == one_min <= many_min < many
    # lists of alternatives cost room only when asked for
    assert full >= libdpo.token_stats_size(_batch(R=64, L=600, d=64, V=3000, dtype=dtype), 0)[0]


@pytest.mark.parametrize("n_top", [-1, 33])
def test_stats_refuse_n_top(lib, n_top):
    with pytest.raises(libdpo.DpoError) as e:
        libdpo.token_stats_size(_batch(), n_top)
    assert e.value.status == INVALID
    with pytest.raises(libdpo.DpoError) as e:
        libdpo.token_stats_rows_size(4, 64, 100, n_top)
    assert e.value.status == INVALID
    assert _stats(lib, _batch(), _out(n_top, FAKE, FAKE)) == INVALID


def test_stats_refusals(lib):
    b = _batch()
    assert _stats(lib, b, None) == INVALID
    assert _stats(lib, b, _out(5, None, FAKE)) == INVALID
    assert _stats(lib, b, _out(5, FAKE, None)) == INVALID
    _, least = libdpo.token_stats_size(b, 5)
    assert _stats(lib, b, _out(5, FAKE, FAKE), nbytes=least - 1) == WORKSPACE
    assert _stats(lib, b, _out(), ws=None) == WORKSPACE
    assert _stats(lib, b, _out(), ws=FAKE + 16) == WORKSPACE
    b.c.dtype = libdpo.F16
    assert _stats(lib, b, _out()) == UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), INVALID), (dict(d=60), UNSUPPORTED), (dict(d=0), INVALID), (dict(V=0), INVALID),
    (dict(V=(1 << 24) + 1), INVALID), (dict(dtype=libdpo.F16), UNSUPPORTED), (dict(dtype=9), INVALID),
    (dict(h_stride=56), INVALID), (dict(h_stride=68), UNSUPPORTED), (dict(H=FAKE + 8), INVALID),
    (dict(H=None), INVALID), (dict(W=None), INVALID), (dict(W=FAKE + 4), INVALID),
    (dict(tokens=None), INVALID),
])
def test_stats_rows_refusals(lib, kw, code):
    a = dict(n=4, d=64, V=100, dtype=libdpo.BF16, H=FAKE, h_stride=64, W=FAKE, tokens=FAKE)
    a.update(kw)
    rows = libdpo.TokenRows(*(a[k] for k in ("n", "d", "V", "dtype", "H", "h_stride", "W", "tokens")))
    fn = libdpo._fn("dpo_token_stats_rows",
                    [ctypes.POINTER(libdpo.TokenRows), ctypes.POINTER(libdpo.TokenStatsOut),
                     ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p])
    out = _out()
    assert fn(ctypes.byref(rows), ctypes.byref(out), FAKE, 1 << 40, None) == code
    rows = libdpo.TokenRows(4, 64, 100, libdpo.BF16, FAKE, 64, FAKE, FAKE)
    assert fn(ctypes.byref(rows), ctypes.byref(out), FAKE, 256, None) == WORKSPACE
    rows.n = 0                                            # nothing to do, whatever the workspace
    assert fn(ctypes.byref(rows), ctypes.byref(out), None, 0, None) == 0


def _norm(**kw):
    a = dict(kind=0, dtype=libdpo.BF16, weight_dtype=libdpo.BF16, rows=4, d=64, eps=1e-5, x=FAKE,
             x_stride=64, from_=None, weight=None, bias=None)
    a.update(kw)
    return libdpo.NormC(*(a[f[0]] for f in libdpo.NormC._fields_))


def _held(codes=FAKE + 0x400000, scales=FAKE + 0x500000):
    return ctypes.pointer(libdpo.CheckpointC(codes, scales))


def _fwd(lib, n, y=FAKE + 0x200000, y_stride=64, mean=None, rstd=None, save=None):
    fn = libdpo._fn("dpo_norm_forward",
                    [ctypes.POINTER(libdpo.NormC), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                     ctypes.c_void_p, ctypes.POINTER(libdpo.CheckpointC), ctypes.c_void_p])
    return fn(ctypes.byref(n) if n is not None else None, y, y_stride, mean, rstd, save, None)


@pytest.mark.parametrize("kw,code", [
    (dict(kind=2), INVALID), (dict(dtype=libdpo.F16), UNSUPPORTED), (dict(dtype=5), INVALID),
    (dict(weight_dtype=libdpo.F16), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(d=0), INVALID),
    (dict(d=65544), INVALID), (dict(d=60), UNSUPPORTED), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(x=None), INVALID),
    (dict(x=FAKE + 8), INVALID), (dict(x_stride=56), INVALID), (dict(x_stride=68), UNSUPPORTED),
    (dict(weight=FAKE + 2), INVALID), (dict(bias=FAKE + 2), INVALID), (dict(from_=_held()), INVALID),
    (dict(x=None, from_=_held(codes=None)), INVALID),
    (dict(x=None, from_=_held(codes=FAKE + 8)), INVALID),
])
def test_norm_forward_refusals(lib, kw, code):
    assert _fwd(lib, _norm(**kw)) == code


def test_norm_forward_refuses_outputs(lib):
    assert _fwd(lib, None) == INVALID
    assert _fwd(lib, _norm(), y=None) == INVALID
    assert _fwd(lib, _norm(), y_stride=63) == INVALID
    assert _fwd(lib, _norm(), y_stride=65) == UNSUPPORTED
    assert _fwd(lib, _norm(kind=1), mean=FAKE) == INVALID          # rms has no mean
    assert _fwd(lib, _norm(), mean=FAKE + 1) == INVALID
    assert _fwd(lib, _norm(), y=FAKE + 16) == INVALID               # shifted over x
    assert _fwd(lib, _norm(x_stride=128), y=FAKE, y_stride=64) == INVALID
    assert _fwd(lib, _norm(x_stride=128), y=FAKE + 120, y_stride=128) == INVALID   # touches x's row
    assert _fwd(lib, _norm(), save=_held(codes=FAKE)) == INVALID    # over x
    assert _fwd(lib, _norm(), save=_held(codes=FAKE + 0x200000)) == INVALID   # over y
    assert _fwd(lib, _norm(), save=_held(scales=FAKE + 0x400010)) == INVALID  # over its own codes
    assert _fwd(lib, _norm(x=None, from_=_held()), save=_held(FAKE, FAKE + 4096)) == INVALID
    assert _fwd(lib, _norm(x=None, from_=_held()), y=FAKE + 0x400000) == INVALID
    assert _fwd(lib, _norm(rows=0)) == 0


def _bwd(lib, n, ws=FAKE, nbytes=1 << 30, **kw):
    a = dict(mean=FAKE, rstd=FAKE, dy=FAKE + 0x200000, dy_dtype=libdpo.F32, dy_stride=64,
             dx=FAKE + 0x300000, dx_stride=64, dweight=None, dbias=None, accumulate=0)
    a.update(kw)
    g = libdpo.NormGradsC(*(a[f[0]] for f in libdpo.NormGradsC._fields_))
    fn = libdpo._fn("dpo_norm_backward",
                    [ctypes.POINTER(libdpo.NormC), ctypes.POINTER(libdpo.NormGradsC), ctypes.c_void_p,
                     ctypes.c_size_t, ctypes.c_void_p])
    return fn(ctypes.byref(n), ctypes.byref(g), ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rstd=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=FAKE + 2), INVALID),
    (dict(dy=None), INVALID), (dict(dy=FAKE + 4), INVALID), (dict(dy_dtype=libdpo.F16), UNSUPPORTED),
    (dict(dy_stride=32), INVALID), (dict(dy_stride=68), UNSUPPORTED), (dict(dx_stride=8), INVALID),
    (dict(dx=FAKE + 0x200010), INVALID),            # over dy, shifted
    (dict(dx=FAKE + 0x200000), INVALID),            # over dy, of another type
    (dict(dx=FAKE), INVALID),                       # over x
    (dict(dweight=FAKE + 1), INVALID), (dict(dweight=FAKE, dbias=FAKE), INVALID),
    (dict(accumulate=2), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 128), WORKSPACE),
    (dict(nbytes=1000), WORKSPACE),
])
def test_norm_backward_refusals(lib, kw, code):
    assert _bwd(lib, _norm(), **kw) == code


def test_norm_backward_refuses_a_mean_for_rms(lib):
    assert _bwd(lib, _norm(kind=1)) == INVALID
    assert _bwd(lib, _norm(x=None, from_=_held()), dx=FAKE + 0x400000) == INVALID
    assert _bwd(lib, _norm(x=None), ) == INVALID


def test_norm_workspace(lib):
    assert libdpo.norm_workspace_size(1, 64) >= 2 * 64 * 4
    for rows, d, code in ((-1, 64, INVALID), (4, 60, UNSUPPORTED), (4, 65544, INVALID)):
        with pytest.raises(libdpo.DpoError) as e:
            libdpo.norm_workspace_size(rows, d)
        assert e.value.status == code


@pytest.mark.parametrize("pack", [True, False])
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=libdpo.F16), UNSUPPORTED), (dict(dtype=4), INVALID), (dict(rows=-1), INVALID),
    (dict(d=12), UNSUPPORTED), (dict(d=0), INVALID), (dict(x=None), INVALID),
    (dict(x=FAKE + 2), INVALID), (dict(stride=32), INVALID), (dict(stride=66), UNSUPPORTED),
    (dict(stride=1 << 29), INVALID), (dict(held=None), INVALID),
    (dict(held=_held(codes=None)), INVALID), (dict(held=_held(scales=None)), INVALID),
    (dict(held=_held(codes=FAKE + 4)), INVALID), (dict(held=_held(codes=FAKE + 64)), INVALID),
])
def test_checkpoint_refusals(lib, pack, kw, code):
    a = dict(dtype=libdpo.BF16, rows=4, d=64, x=FAKE, stride=64, held=_held())
    a.update(kw)
    i32, vp, i64 = ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64
    cp = ctypes.POINTER(libdpo.CheckpointC)
    if pack:
        fn = libdpo._fn("dpo_checkpoint_pack", [i32, i32, i32, vp, i64, cp, vp])
        assert fn(a["dtype"], a["rows"], a["d"], a["x"], a["stride"], a["held"], None) == code
    else:
        fn = libdpo._fn("dpo_checkpoint_unpack", [i32, i32, i32, cp, vp, i64, vp])
        assert fn(a["dtype"], a["rows"], a["d"], a["held"], a["x"], a["stride"], None) == code


def test_binding_refuses_host_tensors_and_shapes():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    with pytest.raises((ValueError, AssertionError, RuntimeError)):
        libdpo.norm_forward(x, x)                        # not in device memory (or no device at all)
    with pytest.raises(ValueError):
        libdpo.Checkpoint(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 3, dtype=torch.uint8))
    with pytest.raises((ValueError, AssertionError, RuntimeError)):
        libdpo.token_stats_rows(x, x, None, 0, ws=x)
