"""The largest number of rows: 2^31 - 1 of 8 values, all but a few of them zero (x and dy are one
buffer of 34 GB, read only). The weight gradient is the sum over the others; the grid's size is worked
out from a sum that passes 32 bits."""
import numpy as np
import pytest

from preference_alignment_b200 import libdpo

from dpo_harness import np64

pytestmark = pytest.mark.gpu

ROWS, D = 2 ** 31 - 1, 8
AT = [0, 12345, 2 ** 30 + 7, ROWS - 300, ROWS - 1]


def test_weight_gradient_over_the_most_rows():
    import torch
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB of free device memory")
    x = torch.zeros(ROWS, D, dtype=torch.bfloat16, device="cuda")
    some = torch.randn(len(AT), D, device="cuda").bfloat16()
    for i, r in enumerate(AT):
        x[r] = some[i]
    rstd = torch.ones(ROWS, device="cuda")
    dw, db = torch.full((D,), float("nan"), device="cuda"), torch.full((D,), float("nan"), device="cuda")
    ws = torch.empty(libdpo.norm_workspace_size(ROWS, D), dtype=torch.uint8, device="cuda")
    libdpo.norm_backward(x, x, None, rstd, dweight=dw, dbias=db, kind="rms", ws=ws)
    assert libdpo.check() == libdpo.OK
    s = np64(some)
    # sums of five terms each, the squares exact in fp32: at most 8 half-steps of the magnitudes
    assert np.all(np.abs(np64(dw) - (s * s).sum(axis=0)) <= 8 * 2.0 ** -24 * (s * s).sum(axis=0))
    assert np.all(np.abs(np64(db) - s.sum(axis=0)) <= 8 * 2.0 ** -24 * np.abs(s).sum(axis=0))
