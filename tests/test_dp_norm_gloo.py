"""The data-parallel backward exchange through the final norm on two CPU ranks (gloo): each rank
takes its own rows, the library's calls are replaced by their fp64 definitions, and the summed
weight gradients must equal one process' on all rows, dx each rank's own part."""
import os
import socket
import types

import numpy as np
import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

from oracle import head_ops_oracle as HO
from preference_alignment_b200 import dp as DP

WORLD, D, V = 2, 16, 24
ROWS = {0: slice(0, 5), 1: slice(5, 8)}          # unequal shares of 8 rows


def _data(kind):
    rng = np.random.default_rng(7)
    x, dy, w = rng.normal(size=(8, D)), rng.normal(size=(8, D)), rng.normal(size=D)
    dw = rng.normal(size=(WORLD, V, D))
    _, mean, rstd = HO.norm_forward(x, w, None, kind)
    return x, dy, w, dw, mean, rstd


class _Ops:
    """Stand-ins for the library's calls: the head's gradients are given, the norm's computed."""

    def __init__(self, dy, dw):
        self.dy, self.dw, self.calls = dy, dw, []

    def backward(self, batch, lse, coef, dH, dW, acc, ws):
        assert dH is None and dW is None
        self.calls.append("dz")

    def backward_dw(self, batch, v0, v1, dW, acc, ws, max_sms=0):
        dW[v0:v1] = torch.from_numpy(self.dw[v0:v1])
        self.calls.append("dw")

    def backward_dh(self, batch, dH, ws, max_sms=0):
        dH.copy_(torch.from_numpy(self.dy))
        self.calls.append("dh")

    def norm_backward(self, x, dy, mean, rstd, dx, weight, dweight, dbias, kind, ws):
        gx, gw, gb = HO.norm_backward(x, dy.numpy(), mean, rstd, weight, kind)
        for out, g in ((dx, gx), (dweight, gw), (dbias, gb)):
            if out is not None:
                out.copy_(torch.from_numpy(g))
        self.calls.append("norm")


def _worker(rank, port, kind, with_bias, q):
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    dist.init_process_group("gloo", rank=rank, world_size=WORLD)
    try:
        x, dy, w, dw, mean, rstd = _data(kind)
        s = ROWS[rank]
        f64 = lambda *n: torch.full(n, float("nan"), dtype=torch.float64)  # noqa: E731
        rows = len(x[s])
        dH, dW, dx, dg = f64(rows, D), f64(V, D), f64(rows, D), f64(D)
        db = f64(D) if with_bias else None
        norm = DP.FinalNorm(x[s], mean[s], rstd[s], dx, weight=w, dweight=dg, dbias=db, kind=kind)
        batch = types.SimpleNamespace(c=types.SimpleNamespace(V=V))
        ops = _Ops(dy[s], dw[rank])
        DP.finish(DP.backward_exchange(batch, None, None, dH, dW, None, n_buckets=2, norm=norm,
                                       ops=ops))
        with pytest.raises(ValueError):
            DP.backward_exchange(batch, None, None, None, dW, None, norm=norm, ops=ops)
        q.put((rank, ops.calls, dx.numpy(), dg.numpy(), db.numpy() if with_bias else None,
               dW.numpy()))
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("kind,with_bias", [("layer", True), ("rms", False)])
def test_exchange_through_the_final_norm(kind, with_bias):
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    procs = [ctx.Process(target=_worker, args=(r, port, kind, with_bias, q)) for r in range(WORLD)]
    for p in procs:
        p.start()
    res = {}
    for _ in range(WORLD):
        item = q.get(timeout=120)
        res[item[0]] = item[1:]
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0
    x, dy, w, dw, mean, rstd = _data(kind)
    gx, gw, gb = HO.norm_backward(x, dy, mean, rstd, w, kind)
    for r in range(WORLD):
        calls, dx, dg, db, dW = res[r]
        assert calls[0] == "dz" and calls[-2:] == ["dh", "norm"]
        np.testing.assert_allclose(dx, gx[ROWS[r]], rtol=1e-12)
        np.testing.assert_allclose(dg, gw, rtol=1e-12)
        if with_bias:
            np.testing.assert_allclose(db, gb, rtol=1e-12)
        np.testing.assert_allclose(dW, dw.sum(axis=0), rtol=1e-12)
