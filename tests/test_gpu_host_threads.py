"""Calls from a host thread that has made no CUDA call before: the device's context is current in the
main thread, not yet in this one. Same bits as from the main thread."""
import threading

import numpy as np
import pytest

from preference_alignment_b200 import libdpo
from preference_alignment_b200 import workloads as WL

from dpo_harness import DeviceWorkload

pytestmark = pytest.mark.gpu


def _norm(stream):
    import torch
    x = torch.arange(40 * 64, device="cuda").reshape(40, 64).float().sin()
    y, rstd = torch.empty_like(x), torch.empty(40, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(64, device="cuda")
    ws = torch.empty(libdpo.norm_workspace_size(40, 64), dtype=torch.uint8, device="cuda")

    def call():
        libdpo.norm_forward(x, y, kind="rms", rstd=rstd, stream=stream)
        libdpo.norm_backward(x, y, None, rstd, dx=dx, dweight=dw, kind="rms", ws=ws, stream=stream)
    return call, (y, dx, dw)


def _statistics(stream):
    import torch
    H = torch.arange(5 * 64, device="cuda").reshape(5, 64).float().sin().bfloat16()
    W = torch.arange(700 * 64, device="cuda").reshape(700, 64).float().cos().bfloat16()
    ent, ids, top = (torch.empty(5, device="cuda"), torch.empty(5, 3, dtype=torch.int32, device="cuda"),
                     torch.empty(5, 3, device="cuda"))
    ws = torch.empty(libdpo.token_stats_rows_size(5, 64, 700, 3)[0], dtype=torch.uint8, device="cuda")
    return (lambda: libdpo.token_stats_rows(H, W, None, 3, ws=ws, entropy=ent, top_ids=ids, top_logp=top,
                                            stream=stream)), (ent, ids, top)


def _forward(stream):
    import torch
    dw = DeviceWorkload(WL.make_custom(R=2, L=40, d=64, V=300, dtype="bf16", seed=5))
    b = dw.batch()
    seq = torch.empty(2, device="cuda")
    ws = torch.empty(libdpo.workspace_size(b)[0], dtype=torch.uint8, device="cuda")
    return (lambda: libdpo.seq_logprobs(b, False, seq, None, None, ws, stream=stream)), (seq,)


@pytest.mark.parametrize("make", [_norm, _statistics, _forward])
def test_first_call_of_a_thread(make):
    import torch
    stream = torch.cuda.current_stream().cuda_stream
    call, outs = make(stream)
    call()
    torch.cuda.synchronize()
    want = [o.cpu().numpy() for o in outs]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            call()
        except Exception as e:              # noqa: BLE001
            errors.append(repr(e))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not errors, errors
    assert libdpo.check() == libdpo.OK
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.cpu().numpy(), w)
