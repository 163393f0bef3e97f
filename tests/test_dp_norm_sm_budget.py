"""dp.backward_exchange with an SM budget: `max_sms` leaves the other SMs to the collective's kernels
while collectives are pending. The norm's backward takes every SM, so it starts behind them. Recorded
with stand-ins for the library and for torch.distributed's all-reduce, one process, no device."""
import types

import pytest
import torch
import torch.distributed as dist

from preference_alignment_b200 import dp as DP

V, D = 1024, 8


class Work:
    def __init__(self, log, name):
        self.log, self.name = log, name
        log.append(("start", name))

    def wait(self):
        self.log.append(("wait", self.name))


class Ops:
    def __init__(self, log):
        self.log = log

    def backward(self, batch, lse, coef, dH, dW, acc, ws):
        self.log.append(("dz",))

    def backward_dw(self, batch, v0, v1, dW, acc, ws, max_sms=0):
        self.log.append(("dw", max_sms))

    def backward_dh(self, batch, dH, ws, max_sms=0):
        self.log.append(("dh", max_sms))

    def norm_backward(self, x, dy, mean, rstd, dx, weight, dweight, dbias, kind, ws):
        self.log.append(("norm",))


def _run(monkeypatch, max_sms, norm):
    log = []
    names = iter(f"r{i}" for i in range(100))
    monkeypatch.setattr(dist, "all_reduce", lambda t, group=None, async_op=False: Work(log, next(names)))
    batch = types.SimpleNamespace(c=types.SimpleNamespace(V=V))
    dW, dH = torch.zeros(V, D), torch.zeros(2, 4, D)
    f = DP.FinalNorm(None, None, None, None, dweight=torch.zeros(D), dbias=torch.zeros(D)) if norm else None
    works = DP.backward_exchange(batch, None, None, dH, dW, None, n_buckets=4, max_sms=max_sms, norm=f,
                                 ops=Ops(log))
    DP.finish(works)
    return log


def _pending(log, at):
    started = [e[1] for e in log[:at] if e[0] == "start"]
    done = [e[1] for e in log[:at] if e[0] == "wait"]
    return [w for w in started if w not in done]


@pytest.mark.parametrize("max_sms", [1, 100])
def test_nothing_without_a_budget_runs_beside_a_collective(monkeypatch, max_sms):
    log = _run(monkeypatch, max_sms, norm=True)
    assert len([e for e in log if e[0] == "start"]) == 6        # 4 blocks of dW, dweight, dbias
    for i, e in enumerate(log):
        if e[0] in ("dz", "norm"):
            assert _pending(log, i) == []
        if e[0] in ("dw", "dh"):
            assert e[1] == max_sms
    # dH still overlaps the last block's all-reduce
    assert _pending(log, log.index(("dh", max_sms))) != []
    assert _pending(log, len(log)) == []


def test_without_a_budget_the_norm_overlaps_too(monkeypatch):
    log = _run(monkeypatch, 0, norm=True)
    assert _pending(log, log.index(("norm",))) == ["r0", "r1", "r2", "r3"]
    assert _pending(log, len(log)) == []


def test_no_norm_no_wait(monkeypatch):
    log = _run(monkeypatch, 100, norm=False)
    assert log[-5][0] == "dh" and [e[0] for e in log[-4:]] == ["wait"] * 4
