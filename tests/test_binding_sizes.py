"""Sizes that pass the C ABI's 32 bits are refused by the binding: a C integer would take their low
bits, and the call would work on a few rows and report success. Tensors that large are stood in
for by their descriptions (no memory, no device)."""
import pytest

from preference_alignment_b200 import libdpo


class Described:
    """What the binding asks of a dense device tensor."""

    is_cuda = True

    def __init__(self, rows, d, dtype="bfloat16"):
        self.shape, self.dtype = (rows, d), dtype

    def stride(self):
        return self.shape[1], 1

    def numel(self):
        return self.shape[0] * self.shape[1]

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def element_size(self):
        return 2

    def data_ptr(self):
        return 0x100000


@pytest.fixture(autouse=True)
def device(monkeypatch):
    monkeypatch.setattr(libdpo, "_device", lambda: 0)


def _no_call(monkeypatch):
    def fn(name, argtypes):
        def call(*args):
            raise AssertionError(f"{name} was called")
        return call
    monkeypatch.setattr(libdpo, "_fn", fn)


@pytest.mark.parametrize("rows", [2 ** 31, 2 ** 32 + 5])
def test_rows_past_32_bits_are_refused(monkeypatch, rows):
    _no_call(monkeypatch)
    x = Described(rows, 8)
    held = object.__new__(libdpo.Checkpoint)
    held.rows, held.d = rows, 8
    held.codes, held.scales = Described(rows, 8, "int8"), Described(rows, 1, "uint8")
    rstd = Described(rows, 1, "float32")
    one = Described(100, 8)
    for call in (lambda: libdpo.norm_forward(x, x, kind="rms"),
                 lambda: libdpo.norm_backward(x, x, None, rstd, kind="rms", ws=0x100000, ws_bytes=1 << 20),
                 lambda: libdpo.norm_forward(held, x, kind="rms"),
                 lambda: libdpo.checkpoint_pack(x, held),
                 lambda: libdpo.checkpoint_unpack(held, x),
                 lambda: libdpo.token_stats_rows(x, one, None, 0, ws=0x100000, ws_bytes=1 << 20),
                 lambda: libdpo.token_stats_rows(one, x, None, 0, ws=0x100000, ws_bytes=1 << 20),
                 lambda: libdpo.norm_workspace_size(rows, 8),
                 lambda: libdpo.token_stats_rows_size(rows, 8, 100, 0),
                 lambda: libdpo.token_stats_rows_size(1, 8, rows, 0)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_row_length_past_32_bits_is_refused(monkeypatch):
    _no_call(monkeypatch)
    x = Described(2, 2 ** 32 + 64)
    for call in (lambda: libdpo.norm_forward(x, x, kind="rms"),
                 lambda: libdpo.norm_workspace_size(2, 2 ** 32 + 64)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_the_largest_rows_pass(monkeypatch):
    called = []
    monkeypatch.setattr(libdpo, "_fn", lambda name, argtypes: lambda *a: called.append(name) or 0)
    monkeypatch.setattr(libdpo, "_stream", lambda s: None)
    x = Described(2 ** 31 - 1, 8)
    libdpo.norm_forward(x, x, kind="rms")
    assert called == ["dpo_norm_forward"]
