"""ctypes binding of libdpo (include/dpo.h): argument marshalling only.

Every step of the DPO head path runs in the CUDA library; this module turns
Python arguments into the C ABI's plain pointers and sizes. Device buffers may
be given as torch tensors (their data_ptr() is passed) or as integer device
addresses; host row-length arrays as numpy int32 arrays. The names follow the C
entry points without the `dpo_` prefix.

The module refuses to run without the compiled library: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libdpo.so")

# dpo_status
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_BAD_TARGET, ERR_WORKSPACE = range(7)
# dpo_dtype
BF16, F32, F16 = 0, 1, 2
# dpo_layout
PAIRS_HALVES, PAIRS_ADJACENT = 0, 1

LAYOUTS = {"halves": PAIRS_HALVES, "adjacent": PAIRS_ADJACENT}
DTYPES = {"bf16": BF16, "f32": F32, "f16": F16}


class DpoError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class Batch(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("L", ctypes.c_int32), ("d", ctypes.c_int32), ("V", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("H", ctypes.c_void_p), ("W", ctypes.c_void_p), ("tokens", ctypes.c_void_p),
        ("prompt_len", ctypes.c_void_p), ("completion_len", ctypes.c_void_p),
    ]


_lib: Optional[ctypes.CDLL] = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libdpo.so (built in-tree by preference_alignment_b200.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libdpo.so is not built ({path}); run "
                           "`python -m preference_alignment_b200.build`")
    lib = ctypes.CDLL(path)
    vp, sz, i32, u32, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_uint32, ctypes.c_float
    bp = ctypes.POINTER(Batch)
    szp = ctypes.POINTER(ctypes.c_size_t)
    lib.dpo_workspace_size.argtypes = [bp, szp, szp, szp]
    lib.dpo_seq_logprobs.argtypes = [bp, ctypes.c_int, vp, vp, vp, vp, sz, vp]
    lib.dpo_loss.argtypes = [i32, i32, vp, vp, f32, f32, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.dpo_backward.argtypes = [bp, vp, vp, vp, vp, ctypes.c_int, vp, sz, vp]
    lib.dpo_check.argtypes = [vp]
    lib.dpo_set_wait_budget_ms.argtypes = [u32]
    lib.dpo_set_wait_budget_ms.restype = u32
    lib.dpo_status_string.argtypes = [ctypes.c_int]
    lib.dpo_status_string.restype = ctypes.c_char_p
    lib.dpo_version.restype = i32
    for name in ("dpo_workspace_size", "dpo_seq_logprobs", "dpo_loss", "dpo_backward", "dpo_check"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


# element types a buffer argument may have (bf16 data may also arrive as its 16-bit pattern)
_KINDS = {"f32": ("float32",), "i32": ("int32",), "f16": ("float16",),
          "bf16": ("bfloat16", "int16", "uint16")}


def _ptr(x, kind: Optional[str] = None) -> Optional[int]:
    """Device/host address of a torch tensor, numpy array or raw integer; None -> NULL.
    The C ABI reads dense row-major arrays of the element type its header names, so a
    strided view (a transpose, a column slice) or a tensor of another element type
    (`kind`: "f32", "i32", "bf16") is refused rather than passed on; a raw integer
    address is taken as it is."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        name = str(x.dtype).replace("torch.", "")
        ptr = x.data_ptr()
        dense = x.numel() == 0 or x.is_contiguous()
        shape = tuple(x.shape)
    elif isinstance(x, np.ndarray):
        name = x.dtype.name
        ptr = x.ctypes.data
        dense = bool(x.flags["C_CONTIGUOUS"])
        shape = x.shape
    else:
        raise TypeError(f"cannot take the address of {type(x)}")
    if not dense:
        raise ValueError(f"buffer of shape {shape} is not contiguous")
    if kind is not None and name not in _KINDS[kind]:
        raise TypeError(f"expected a {kind} buffer, got {name} (shape {shape})")
    return ptr


_raw_stream = None      # torch's lookup of a device's current stream as an address, once found


def _stream(s) -> Optional[int]:
    global _raw_stream
    if s is None:
        if _raw_stream is not None:
            return _raw_stream()
        try:
            import torch
            if torch.cuda.is_available():
                found = getattr(torch._C, "_cuda_getCurrentRawStream", None)
                current = torch.cuda.current_device
                if found is not None:
                    _raw_stream = lambda: found(current())  # noqa: E731
                return torch.cuda.current_stream().cuda_stream
        except Exception:
            pass
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int, where: str):
    if status != OK:
        raise DpoError(status, where)


def status_string(status: int) -> str:
    return load().dpo_status_string(int(status)).decode()


def version() -> int:
    return load().dpo_version()


def set_wait_budget_ms(ms: int) -> int:
    return load().dpo_set_wait_budget_ms(int(ms))


_HW_KIND = {BF16: "bf16", F32: "f32", F16: "f16"}


class BatchArgs:
    """A dpo_batch plus the Python objects its pointers refer to (kept alive)."""

    def __init__(self, H, W, tokens, prompt_len, completion_len, R=None, L=None, d=None, V=None,
                 dtype="bf16"):
        self.prompt_len = np.ascontiguousarray(prompt_len, dtype=np.int32)
        self.completion_len = np.ascontiguousarray(completion_len, dtype=np.int32)
        shapeH = tuple(H.shape) if hasattr(H, "shape") else None
        shapeW = tuple(W.shape) if hasattr(W, "shape") else None
        R = R if R is not None else shapeH[0]
        L = L if L is not None else shapeH[1]
        d = d if d is not None else shapeH[2]
        V = V if V is not None else shapeW[0]
        self.keep = (H, W, tokens)
        self.dtype = DTYPES.get(dtype, dtype) if isinstance(dtype, str) else int(dtype)
        self.c = Batch(int(R), int(L), int(d), int(V), self.dtype,
                       _ptr(H, _HW_KIND.get(self.dtype)), _ptr(W, _HW_KIND.get(self.dtype)),
                       _ptr(tokens, "i32"), self.prompt_len.ctypes.data,
                       self.completion_len.ctypes.data)

    @property
    def n_scored(self) -> int:
        return int(self.completion_len.sum())


def workspace_size(batch: BatchArgs):
    """(fwd_bytes, bwd_bytes, bwd_min_bytes) for this batch."""
    f, b, m = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().dpo_workspace_size(ctypes.byref(batch.c), ctypes.byref(f), ctypes.byref(b),
                                     ctypes.byref(m)), "dpo_workspace_size")
    return f.value, b.value, m.value


def _nbytes(ws, ws_bytes):
    if ws_bytes is not None:
        return int(ws_bytes)
    if hasattr(ws, "numel"):
        return ws.numel() * ws.element_size()
    raise ValueError("ws_bytes is required for a raw workspace address")


def seq_logprobs(batch: BatchArgs, want_grad: bool, seq_logp, tok_logp, lse_state, ws,
                 ws_bytes=None, stream=None):
    _check(load().dpo_seq_logprobs(ctypes.byref(batch.c), 1 if want_grad else 0,
                                   _ptr(seq_logp, "f32"), _ptr(tok_logp, "f32"),
                                   _ptr(lse_state, "f32"), _ptr(ws), _nbytes(ws, ws_bytes),
                                   _stream(stream)), "dpo_seq_logprobs")


def loss(B: int, layout, pol, ref, beta: float, grad_scale: float, loss_out, accuracy=None,
         margins=None, chosen_rewards=None, rejected_rewards=None, weights=None, row_coef=None,
         stream=None):
    lay = LAYOUTS[layout] if isinstance(layout, str) else int(layout)
    _check(load().dpo_loss(int(B), lay, _ptr(pol, "f32"), _ptr(ref, "f32"), float(beta),
                           float(grad_scale), _ptr(loss_out, "f32"), _ptr(accuracy, "f32"),
                           _ptr(margins, "f32"), _ptr(chosen_rewards, "f32"),
                           _ptr(rejected_rewards, "f32"), _ptr(weights, "f32"),
                           _ptr(row_coef, "f32"), _stream(stream)),
           "dpo_loss")


class LossOptions(ctypes.Structure):
    _fields_ = [("normalize", ctypes.c_int32), ("nll_weight", ctypes.c_float),
                ("completion_len", ctypes.c_void_p), ("pairs_total", ctypes.c_int32),
                ("nll_tokens_total", ctypes.c_int64), ("reference_free", ctypes.c_int32)]


def loss_ex(B: int, layout, pol, ref, beta: float, grad_scale: float, loss_out, accuracy=None,
            margins=None, chosen_rewards=None, rejected_rewards=None, weights=None, row_coef=None,
            nll=None, normalize=False, nll_weight=0.0, completion_len=None, pairs_total=0,
            nll_tokens_total=0, reference_free=False, stream=None):
    """dpo_loss_ex: length-normalised and/or SFT-NLL variants (completion_len: device int32 [2B]);
    pairs_total / nll_tokens_total > 0 make the outputs this rank's share of a data-parallel
    batch of that many pairs / chosen tokens; reference_free reads the reference sums as 0
    (ref is then not read and may be None)."""
    lib = load()
    fn = lib.dpo_loss_ex
    vp = ctypes.c_void_p
    fn.argtypes = [ctypes.c_int32, ctypes.c_int32, vp, vp, ctypes.c_float, ctypes.c_float,
                   ctypes.POINTER(LossOptions), vp, vp, vp, vp, vp, vp, vp, vp, vp]
    fn.restype = ctypes.c_int
    opt = LossOptions(1 if normalize else 0, float(nll_weight), _ptr(completion_len, "i32"),
                      int(pairs_total), int(nll_tokens_total), 1 if reference_free else 0)
    lay = LAYOUTS[layout] if isinstance(layout, str) else int(layout)
    _check(fn(int(B), lay, _ptr(pol, "f32"), _ptr(ref, "f32"), float(beta), float(grad_scale),
              ctypes.byref(opt), _ptr(loss_out, "f32"), _ptr(accuracy, "f32"), _ptr(margins, "f32"),
              _ptr(chosen_rewards, "f32"), _ptr(rejected_rewards, "f32"), _ptr(weights, "f32"),
              _ptr(row_coef, "f32"), _ptr(nll, "f32"), _stream(stream)),
           "dpo_loss_ex")


def backward(batch: BatchArgs, lse_state, row_coef, dH, dW, accumulate_dW: bool, ws,
             ws_bytes=None, stream=None):
    _check(load().dpo_backward(ctypes.byref(batch.c), _ptr(lse_state, "f32"),
                               _ptr(row_coef, "f32"), _ptr(dH, "f32"), _ptr(dW, "f32"),
                               1 if accumulate_dW else 0, _ptr(ws),
                               _nbytes(ws, ws_bytes), _stream(stream)), "dpo_backward")


def backward_dw(batch: BatchArgs, v_begin: int, v_end: int, dW, accumulate_dW: bool, ws,
                ws_bytes=None, max_sms: int = 0, stream=None):
    """dpo_backward_dw: rows [v_begin, v_end) of dW from the dz a preceding
    backward(dW=None) left in the workspace ws (max_sms > 0 caps the SMs it uses)."""
    lib = load()
    fn = lib.dpo_backward_dw
    vp = ctypes.c_void_p
    fn.argtypes = [ctypes.POINTER(Batch), ctypes.c_int32, ctypes.c_int32, vp, ctypes.c_int,
                   ctypes.c_int32, vp, ctypes.c_size_t, vp]
    fn.restype = ctypes.c_int
    _check(fn(ctypes.byref(batch.c), int(v_begin), int(v_end), _ptr(dW, "f32"),
              1 if accumulate_dW else 0, int(max_sms), _ptr(ws), _nbytes(ws, ws_bytes),
              _stream(stream)), "dpo_backward_dw")


def backward_dh(batch: BatchArgs, dH, ws, ws_bytes=None, max_sms: int = 0, stream=None):
    """dpo_backward_dh: dH (fully written) from the dz a preceding backward(dW=None) left in ws."""
    lib = load()
    fn = lib.dpo_backward_dh
    vp = ctypes.c_void_p
    fn.argtypes = [ctypes.POINTER(Batch), vp, ctypes.c_int32, vp, ctypes.c_size_t, vp]
    fn.restype = ctypes.c_int
    _check(fn(ctypes.byref(batch.c), _ptr(dH, "f32"), int(max_sms), _ptr(ws), _nbytes(ws, ws_bytes),
              _stream(stream)), "dpo_backward_dh")


MAX_SCATTER_RANKS = 8


class DwScatter(ctypes.Structure):
    _fields_ = [("n_ranks", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("rows_per_rank", ctypes.c_int32),
                ("recv", ctypes.c_void_p * MAX_SCATTER_RANKS)]


def backward_dw_scatter(batch: BatchArgs, n_ranks: int, rank: int, rows_per_rank: int, recv, ws,
                        ws_bytes=None, max_sms: int = 0, stream=None):
    """dpo_backward_dw_scatter: this rank's dW contribution, each row stored into its owner's
    receive buffer (recv: one device address or tensor per rank, as this process maps it)."""
    lib = load()
    fn = lib.dpo_backward_dw_scatter
    vp = ctypes.c_void_p
    fn.argtypes = [ctypes.POINTER(Batch), ctypes.POINTER(DwScatter), ctypes.c_int32, vp,
                   ctypes.c_size_t, vp]
    fn.restype = ctypes.c_int
    ptrs = [_ptr(r, "f32") for r in recv]
    if len(ptrs) != n_ranks or n_ranks > MAX_SCATTER_RANKS:
        raise ValueError("recv needs one buffer per rank (at most 8 ranks)")
    x = DwScatter(int(n_ranks), int(rank), int(rows_per_rank),
                  (ctypes.c_void_p * MAX_SCATTER_RANKS)(*(ptrs + [None] * (MAX_SCATTER_RANKS - n_ranks))))
    _check(fn(ctypes.byref(batch.c), ctypes.byref(x), int(max_sms), _ptr(ws), _nbytes(ws, ws_bytes),
              _stream(stream)), "dpo_backward_dw_scatter")


def dw_reduce_slots(recv, n_slots: int, rows: int, d: int, dW_shard, accumulate: bool = False,
                    stream=None):
    """dpo_dw_reduce_slots: dW_shard (+)= the sum of recv's n_slots slots, in slot order."""
    lib = load()
    fn = lib.dpo_dw_reduce_slots
    vp = ctypes.c_void_p
    fn.argtypes = [vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp, ctypes.c_int, vp]
    fn.restype = ctypes.c_int
    _check(fn(_ptr(recv, "f32"), int(n_slots), int(rows), int(d), _ptr(dW_shard, "f32"),
              1 if accumulate else 0,
              _stream(stream)), "dpo_dw_reduce_slots")


class IpcHandle(ctypes.Structure):
    _fields_ = [("bytes", ctypes.c_ubyte * 64)]


def ipc_export(ptr):
    """dpo_ipc_export: (64-byte handle as bytes, byte offset) of the allocation holding ptr."""
    lib = load()
    fn = lib.dpo_ipc_export
    fn.argtypes = [ctypes.c_void_p, ctypes.POINTER(IpcHandle), ctypes.POINTER(ctypes.c_size_t)]
    fn.restype = ctypes.c_int
    h, off = IpcHandle(), ctypes.c_size_t()
    _check(fn(_ptr(ptr), ctypes.byref(h), ctypes.byref(off)), "dpo_ipc_export")
    return bytes(h.bytes), off.value


def ipc_import(handle: bytes) -> int:
    """dpo_ipc_import: map another process's exported allocation; returns its base address."""
    lib = load()
    fn = lib.dpo_ipc_import
    fn.argtypes = [ctypes.POINTER(IpcHandle), ctypes.POINTER(ctypes.c_void_p)]
    fn.restype = ctypes.c_int
    h = IpcHandle((ctypes.c_ubyte * 64)(*handle))
    base = ctypes.c_void_p()
    _check(fn(ctypes.byref(h), ctypes.byref(base)), "dpo_ipc_import")
    return base.value


def ipc_close(base: int):
    lib = load()
    fn = lib.dpo_ipc_close
    fn.argtypes = [ctypes.c_void_p]
    fn.restype = ctypes.c_int
    _check(fn(base), "dpo_ipc_close")


class VocabShard(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_int32), ("total", ctypes.c_int32)]


def shard_logprob_parts(batch: BatchArgs, offset: int, total: int, shard_lse, shard_zy, ws,
                        ws_bytes=None, stream=None):
    """dpo_shard_logprob_parts: per-position (lse, target logit or -inf) over one shard's rows."""
    lib = load()
    fn = lib.dpo_shard_logprob_parts
    vp = ctypes.c_void_p
    fn.argtypes = [ctypes.POINTER(Batch), ctypes.POINTER(VocabShard), vp, vp, vp, ctypes.c_size_t, vp]
    fn.restype = ctypes.c_int
    sh = VocabShard(int(offset), int(total))
    _check(fn(ctypes.byref(batch.c), ctypes.byref(sh), _ptr(shard_lse, "f32"),
              _ptr(shard_zy, "f32"), _ptr(ws),
              _nbytes(ws, ws_bytes), _stream(stream)), "dpo_shard_logprob_parts")


def shard_combine(batch: BatchArgs, total: int, n_shards: int, shard_lse, shard_zy, seq_logp,
                  tok_logp, lse_state, ws, ws_bytes=None, stream=None):
    """dpo_shard_combine: merge gathered [n_shards, Nc] parts into sums, log-probs and lse."""
    lib = load()
    fn = lib.dpo_shard_combine
    vp = ctypes.c_void_p
    fn.argtypes = [ctypes.POINTER(Batch), ctypes.c_int32, ctypes.c_int32, vp, vp, vp, vp, vp, vp,
                   ctypes.c_size_t, vp]
    fn.restype = ctypes.c_int
    _check(fn(ctypes.byref(batch.c), int(total), int(n_shards), _ptr(shard_lse, "f32"),
              _ptr(shard_zy, "f32"), _ptr(seq_logp, "f32"), _ptr(tok_logp, "f32"),
              _ptr(lse_state, "f32"), _ptr(ws), _nbytes(ws, ws_bytes),
              _stream(stream)), "dpo_shard_combine")


def shard_backward(batch: BatchArgs, offset: int, total: int, lse_state, row_coef, dH_part,
                   dW_shard, accumulate_dW: bool, ws, ws_bytes=None, stream=None):
    """dpo_shard_backward: this shard's dW rows and a partial dH (summed over shards = dH)."""
    lib = load()
    fn = lib.dpo_shard_backward
    vp = ctypes.c_void_p
    fn.argtypes = [ctypes.POINTER(Batch), ctypes.POINTER(VocabShard), vp, vp, vp, vp, ctypes.c_int,
                   vp, ctypes.c_size_t, vp]
    fn.restype = ctypes.c_int
    sh = VocabShard(int(offset), int(total))
    _check(fn(ctypes.byref(batch.c), ctypes.byref(sh), _ptr(lse_state, "f32"),
              _ptr(row_coef, "f32"), _ptr(dH_part, "f32"), _ptr(dW_shard, "f32"),
              1 if accumulate_dW else 0, _ptr(ws),
              _nbytes(ws, ws_bytes), _stream(stream)), "dpo_shard_backward")


def logits_mean(batch: BatchArgs, layout, means, ws, ws_bytes=None, stream=None):
    """dpo_logits_mean: means (device float32 [2]) = mean logit of the chosen rows and of the
    rejected rows over every position and vocabulary entry."""
    lib = load()
    fn = lib.dpo_logits_mean
    fn.argtypes = [ctypes.POINTER(Batch), ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                   ctypes.c_size_t, ctypes.c_void_p]
    fn.restype = ctypes.c_int
    lay = LAYOUTS[layout] if isinstance(layout, str) else int(layout)
    _check(fn(ctypes.byref(batch.c), lay, _ptr(means, "f32"), _ptr(ws), _nbytes(ws, ws_bytes),
              _stream(stream)), "dpo_logits_mean")


def selftest_wait_timeout(budget_ms: int, stream=None):
    """Launch the bounded-wait self-test (records DPO_ERR_TIMEOUT after budget_ms)."""
    lib = load()
    fn = lib.dpo_selftest_wait_timeout
    fn.argtypes = [ctypes.c_uint32, ctypes.c_void_p]
    fn.restype = ctypes.c_int
    _check(fn(int(budget_ms), _stream(stream)), "dpo_selftest_wait_timeout")


def fingerprint(data, nbytes, out, stream=None):
    """dpo_fingerprint: 64-bit order-independent hash of a device buffer into out (device uint64)."""
    lib = load()
    fn = lib.dpo_fingerprint
    fn.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]
    fn.restype = ctypes.c_int
    _check(fn(_ptr(data), int(nbytes), _ptr(out), _stream(stream)), "dpo_fingerprint")


def set_gemm_variant(variant: int) -> int:
    """Mask per GEMM k (forward, dz, dH, dW): bit k runs it on the single-CTA kernel, bit 4 + k
    gives the CTA-pair kernel the static tile schedule instead of tiles claimed in raster order;
    bit 8 keeps dH from being split over the vocabulary (set it before sizing workspaces)."""
    lib = load()
    fn = lib.dpo_set_gemm_variant
    fn.argtypes = [ctypes.c_int32]
    fn.restype = ctypes.c_int32
    return fn(int(variant))


def check(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return load().dpo_check(_stream(stream))


def seq_logprobs_noalloc(batch: BatchArgs, want_grad: bool, seq_logp, tok_logp, lse_state,
                         stream=None):
    """dpo_seq_logprobs_noalloc: the forward with the library's built-in scratch.

    For callers that may not allocate device memory (no workspace argument). The
    batch's forward workspace must fit NOALLOC_SCRATCH_BYTES; calls that overlap on
    the GPU share the scratch and must be serialised.
    """
    lib = load()
    fn = lib.dpo_seq_logprobs_noalloc
    fn.argtypes = [ctypes.POINTER(Batch), ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                   ctypes.c_void_p, ctypes.c_void_p]
    fn.restype = ctypes.c_int
    _check(fn(ctypes.byref(batch.c), 1 if want_grad else 0, _ptr(seq_logp, "f32"),
              _ptr(tok_logp, "f32"), _ptr(lse_state, "f32"), _stream(stream)),
           "dpo_seq_logprobs_noalloc")


NOALLOC_SCRATCH_BYTES = 32 << 20


# ------------------------------------------------------------------ token statistics, norm, checkpoints
MAX_TOP = 32                # DPO_MAX_TOP
CHECKPOINT_BLOCK = 32       # DPO_CHECKPOINT_BLOCK
NORM_KINDS = {"layer": 0, "rms": 1}

_kinds = {}                 # torch dtype -> "bf16", "f32", "i32", "int8", "uint8" or its name
_current_device = None


def _name_of(x):
    name = _kinds.get(x.dtype)
    if name is None:
        name = str(x.dtype).replace("torch.", "")
        name = {"bfloat16": "bf16", "int16": "bf16", "uint16": "bf16", "float32": "f32",
                "int32": "i32"}.get(name, name)
        _kinds[x.dtype] = name
    return name


def _kind_of(x):
    """"bf16" or "f32" for a tensor of that element type, else a TypeError."""
    name = _name_of(x)
    if name != "bf16" and name != "f32":
        raise TypeError(f"expected a bf16 or f32 tensor, got {name}")
    return name


def _device():
    """The current device: what every buffer of a call has to be on."""
    global _current_device
    if _current_device is None:
        import torch
        _current_device = torch.cuda.current_device
    return _current_device()


def _elsewhere(x, what):
    if not x.is_cuda:
        raise ValueError(f"{what}: buffer of shape {tuple(x.shape)} is not in device memory")
    raise ValueError(f"{what}: buffer on {x.device}, but the current device is cuda:{_device()}")


def _buf(x, kind, n, what, dev):
    """Address of a dense tensor of at least n elements of `kind` on device dev; None -> NULL, an
    integer address as it is."""
    if x is None or type(x) is int:
        return x
    if not x.is_cuda or x.get_device() != dev:
        _elsewhere(x, what)
    if _kinds.get(x.dtype) != kind and _name_of(x) != kind:
        raise TypeError(f"{what}: expected a {kind} buffer, got {_name_of(x)}")
    if not x.is_contiguous():
        raise ValueError(f"{what}: buffer of shape {tuple(x.shape)} is not contiguous")
    if x.numel() < n:
        raise ValueError(f"{what}: {x.numel()} elements, {n} needed")
    return x.data_ptr()


_MOST = 2 ** 31 - 1


def _c32(n, what):
    """n as the C ABI's 32-bit integer, which would silently take the low bits of a larger one."""
    n = int(n)
    if n > _MOST or n < -_MOST - 1:
        raise ValueError(f"{what}: {n} does not fit 32 bits")
    return n


def _row_view(x, what, dev):
    """(address, rows, d, stride) of a tensor of rows: 2-D with dense rows (any row stride), or
    contiguous of any shape with its last dimension the row."""
    if not x.is_cuda or x.get_device() != dev:
        _elsewhere(x, what)
    shape = x.shape
    if len(shape) == 2:
        rows, d = shape
        stride, inner = x.stride()
        if inner == 1 and d > 0:
            if rows > _MOST or d > _MOST:
                _c32(max(rows, d), what)
            return x.data_ptr(), rows, d, (stride if rows > 1 else d)
    if len(shape) == 0 or shape[-1] < 1 or not x.is_contiguous():
        raise ValueError(f"{what}: tensor of shape {tuple(shape)} has no dense rows")
    d = shape[-1]
    return x.data_ptr(), _c32(x.numel() // d, what), _c32(d, what), d


def _work(ws, ws_bytes, dev):
    """(address, bytes) of a workspace."""
    if ws is not None and type(ws) is not int and (not ws.is_cuda or ws.get_device() != dev):
        _elsewhere(ws, "ws")
    if ws_bytes is None and type(ws) is not int and ws is not None:
        ws_bytes = ws.numel() * ws.element_size()
    return _ptr_of(ws), _nbytes(ws, ws_bytes)


def _ptr_of(ws):
    return ws if ws is None or type(ws) is int else ws.data_ptr()


_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_fns = {}


def _fn(name, argtypes):
    fn = _fns.get(name)
    if fn is None:
        fn = getattr(load(), name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_int
        _fns[name] = fn
    return fn


class TokenStatsOut(ctypes.Structure):
    _fields_ = [("logp", _vp), ("entropy", _vp), ("lse_state", _vp), ("n_top", _i32),
                ("top_ids", _vp), ("top_logp", _vp)]


class TokenRows(ctypes.Structure):
    _fields_ = [("n", _i32), ("d", _i32), ("V", _i32), ("dtype", _i32), ("H", _vp),
                ("h_stride", _i64), ("W", _vp), ("tokens", _vp)]


class CheckpointC(ctypes.Structure):
    _fields_ = [("codes", _vp), ("scales", _vp)]


class NormC(ctypes.Structure):
    _fields_ = [("kind", _i32), ("dtype", _i32), ("weight_dtype", _i32), ("rows", _i32),
                ("d", _i32), ("eps", ctypes.c_float), ("x", _vp), ("x_stride", _i64),
                ("from_", ctypes.POINTER(CheckpointC)), ("weight", _vp), ("bias", _vp)]


class NormGradsC(ctypes.Structure):
    _fields_ = [("mean", _vp), ("rstd", _vp), ("dy", _vp), ("dy_dtype", _i32),
                ("dy_stride", _i64), ("dx", _vp), ("dx_stride", _i64), ("dweight", _vp),
                ("dbias", _vp), ("accumulate", _i32)]


_szp, _batchp, _outp = ctypes.POINTER(_sz), ctypes.POINTER(Batch), ctypes.POINTER(TokenStatsOut)
_rowsp, _ckptp = ctypes.POINTER(TokenRows), ctypes.POINTER(CheckpointC)
_normp, _gradsp = ctypes.POINTER(NormC), ctypes.POINTER(NormGradsC)

_STATS_SIZE = [_batchp, _i32, _szp, _szp]
_STATS = [_batchp, _outp, _vp, _vp, _sz, _vp]
_ROWS_SIZE = [_rowsp, _i32, _szp, _szp]
_ROWS = [_rowsp, _outp, _vp, _sz, _vp]
_PACK = [_i32, _i32, _i32, _vp, _i64, _ckptp, _vp]
_UNPACK = [_i32, _i32, _i32, _ckptp, _vp, _i64, _vp]
_NORM_FWD = [_normp, _vp, _i64, _vp, _vp, _ckptp, _vp]
_NORM_WS = [_i32, _i32, _szp]
_NORM_BWD = [_normp, _gradsp, _vp, _sz, _vp]


def _stats_out(n, n_top, logp, entropy, lse_state, top_ids, top_logp, dev):
    n_top = _c32(n_top, "n_top")
    return TokenStatsOut(_buf(logp, "f32", n, "logp", dev), _buf(entropy, "f32", n, "entropy", dev),
                         _buf(lse_state, "f32", n, "lse_state", dev), n_top,
                         _buf(top_ids, "i32", n * n_top, "top_ids", dev),
                         _buf(top_logp, "f32", n * n_top, "top_logp", dev))


def token_stats_size(batch: BatchArgs, n_top: int):
    """(bytes, min_bytes) of token_stats' workspace."""
    a, b = _sz(), _sz()
    _check(_fn("dpo_token_stats_size", _STATS_SIZE)(ctypes.byref(batch.c), _c32(n_top, "n_top"),
                                                    ctypes.byref(a), ctypes.byref(b)),
           "dpo_token_stats_size")
    return a.value, b.value


def token_stats(batch: BatchArgs, n_top: int, ws, logp=None, entropy=None, lse_state=None,
                seq_logp=None, top_ids=None, top_logp=None, ws_bytes=None, stream=None):
    """dpo_token_stats: per scored position (row order) the target's log-prob, the entropy, the
    log-sum-exp that backward() reads with the same H and W, and the n_top largest logits' ids and
    log-probs; per row the sum of the log-probs. Outputs left out are not written."""
    dev = _device()
    out = _stats_out(batch.n_scored, n_top, logp, entropy, lse_state, top_ids, top_logp, dev)
    w, nbytes = _work(ws, ws_bytes, dev)
    _check(_fn("dpo_token_stats", _STATS)(ctypes.byref(batch.c), ctypes.byref(out),
                                          _buf(seq_logp, "f32", batch.c.R, "seq_logp", dev), w,
                                          nbytes, _stream(stream)), "dpo_token_stats")


def token_stats_rows_size(n: int, d: int, V: int, n_top: int, dtype="bf16"):
    """(bytes, min_bytes) of token_stats_rows' workspace."""
    a, b = _sz(), _sz()
    rows = TokenRows(_c32(n, "n"), _c32(d, "d"), _c32(V, "V"),
                     DTYPES[dtype] if isinstance(dtype, str) else int(dtype), None, int(d), None, None)
    _check(_fn("dpo_token_stats_rows_size", _ROWS_SIZE)(ctypes.byref(rows), _c32(n_top, "n_top"),
                                                        ctypes.byref(a), ctypes.byref(b)),
           "dpo_token_stats_rows_size")
    return a.value, b.value


def token_stats_rows(H, W, tokens, n_top: int, ws, logp=None, entropy=None, lse_state=None,
                     top_ids=None, top_logp=None, ws_bytes=None, stream=None):
    """dpo_token_stats_rows: token_stats for independent hidden rows, H [n, d] (any row stride)
    against W [V, d], tokens int32 [n] or None (then logp is None too)."""
    dev = _device()
    h, n, d, stride = _row_view(H, "H", dev)
    if len(W.shape) != 2 or W.shape[1] != d:
        raise ValueError(f"W of shape {tuple(W.shape)} does not fit rows of {d}")
    kind = _kind_of(H)
    rows = TokenRows(n, d, _c32(W.shape[0], "W"), DTYPES[kind], h, stride, _buf(W, kind, 0, "W", dev),
                     _buf(tokens, "i32", n, "tokens", dev))
    out = _stats_out(n, n_top, logp, entropy, lse_state, top_ids, top_logp, dev)
    w, nbytes = _work(ws, ws_bytes, dev)
    _check(_fn("dpo_token_stats_rows", _ROWS)(ctypes.byref(rows), ctypes.byref(out), w, nbytes,
                                              _stream(stream)), "dpo_token_stats_rows")


class Checkpoint:
    """Activations held in 8 bits: codes int8 [rows, d] and scales uint8 [rows, ceil(d / 32)],
    device tensors (Checkpoint.empty makes them)."""

    def __init__(self, codes, scales):
        if len(codes.shape) != 2:
            raise ValueError("codes must be [rows, d]")
        self.codes, self.scales = codes, scales
        self.rows, self.d = codes.shape
        blocks = -(-self.d // CHECKPOINT_BLOCK)
        if tuple(scales.shape) != (self.rows, blocks):
            raise ValueError(f"scales must be [{self.rows}, {blocks}], got {tuple(scales.shape)}")

    @classmethod
    def empty(cls, rows: int, d: int, device="cuda"):
        import torch
        return cls(torch.empty(rows, d, dtype=torch.int8, device=device),
                   torch.empty(rows, -(-d // CHECKPOINT_BLOCK), dtype=torch.uint8, device=device))

    def _c(self, dev):
        return CheckpointC(_buf(self.codes, "int8", 0, "codes", dev),
                           _buf(self.scales, "uint8", 0, "scales", dev))


def _fits(rows, d, what, rows2, d2):
    if rows != rows2 or d != d2:
        raise ValueError(f"{what} is {rows2} x {d2}, expected {rows} x {d}")


def checkpoint_pack(x, out: Checkpoint, stream=None):
    """dpo_checkpoint_pack: hold the rows of x (bf16 or f32, any row stride) in out."""
    dev = _device()
    p, rows, d, stride = _row_view(x, "x", dev)
    _fits(rows, d, "out", out.rows, out.d)
    c = out._c(dev)
    _check(_fn("dpo_checkpoint_pack", _PACK)(DTYPES[_kind_of(x)], rows, d, p, stride,
                                             ctypes.byref(c), _stream(stream)),
           "dpo_checkpoint_pack")


def checkpoint_unpack(held: Checkpoint, y, stream=None):
    """dpo_checkpoint_unpack: the values held, into the rows of y (bf16 or f32)."""
    dev = _device()
    p, rows, d, stride = _row_view(y, "y", dev)
    _fits(held.rows, held.d, "y", rows, d)
    c = held._c(dev)
    _check(_fn("dpo_checkpoint_unpack", _UNPACK)(DTYPES[_kind_of(y)], rows, d, ctypes.byref(c), p,
                                                 stride, _stream(stream)),
           "dpo_checkpoint_unpack")


def _norm(x, kind_out, weight, bias, kind, eps, dev):
    """(NormC, rows, d) of a norm of x, a tensor of rows or a Checkpoint (then kind_out is the
    other side's element type)."""
    if isinstance(x, Checkpoint):
        p, rows, d, stride = None, _c32(x.rows, "rows"), _c32(x.d, "d"), 0
        held = ctypes.pointer(x._c(dev))
    else:
        p, rows, d, stride = _row_view(x, "x", dev)
        held = None
        kind_out = _kind_of(x)
    wkind = _kind_of(weight) if weight is not None else "f32"
    if bias is not None:
        bkind = _kind_of(bias)
        if weight is not None and bkind != wkind:
            raise TypeError(f"weight is {wkind}, bias {bkind}")
        wkind = bkind
    n = NormC(NORM_KINDS[kind] if isinstance(kind, str) else int(kind), DTYPES[kind_out],
              DTYPES[wkind], rows, d, eps, p, stride, held,
              _buf(weight, wkind, d, "weight", dev), _buf(bias, wkind, d, "bias", dev))
    return n, rows, d


def norm_forward(x, y, weight=None, bias=None, kind="layer", eps=1e-5, mean=None, rstd=None,
                 save: Optional[Checkpoint] = None, stream=None):
    """dpo_norm_forward: y = norm(x) by rows, kind "layer" or "rms"; mean and rstd (f32 [rows])
    are what norm_backward reads; save also holds x in 8 bits. x may be a Checkpoint: the norm
    of the values it holds (not the H that was formed from x itself: backward() takes an lse_state
    of the H it is given)."""
    dev = _device()
    ykind = _kind_of(y)
    n, rows, d = _norm(x, ykind, weight, bias, kind, eps, dev)
    p, yr, yd, stride = _row_view(y, "y", dev)
    _fits(rows, d, "y", yr, yd)
    if DTYPES[ykind] != n.dtype:
        raise TypeError("y must have x's element type")
    c = None
    if save is not None:
        _fits(rows, d, "save", save.rows, save.d)
        c = ctypes.byref(save._c(dev))
    _check(_fn("dpo_norm_forward", _NORM_FWD)(ctypes.byref(n), p, stride,
                                              _buf(mean, "f32", rows, "mean", dev),
                                              _buf(rstd, "f32", rows, "rstd", dev), c,
                                              _stream(stream)), "dpo_norm_forward")


def norm_workspace_size(rows: int, d: int) -> int:
    """Workspace bytes of norm_backward."""
    b = _sz()
    _check(_fn("dpo_norm_workspace_size", _NORM_WS)(_c32(rows, "rows"), _c32(d, "d"), ctypes.byref(b)),
           "dpo_norm_workspace_size")
    return b.value


def norm_backward(x, dy, mean, rstd, dx=None, weight=None, dweight=None, dbias=None, kind="layer",
                  accumulate=False, ws=None, ws_bytes=None, stream=None):
    """dpo_norm_backward: dx (x's element type; for a Checkpoint, its own), and the fp32 weight
    and bias gradients, from the forward's x (a tensor of rows or the Checkpoint that held it),
    its statistics and dy (bf16 or f32 rows)."""
    dev = _device()
    n, rows, d = _norm(x, _kind_of(dx) if dx is not None else "bf16", weight, None, kind, 0.0, dev)
    p, yr, yd, stride = _row_view(dy, "dy", dev)
    _fits(rows, d, "dy", yr, yd)
    q, dx_stride = None, d
    if dx is not None:
        q, xr, xd, dx_stride = _row_view(dx, "dx", dev)
        _fits(rows, d, "dx", xr, xd)
        if DTYPES[_kind_of(dx)] != n.dtype:
            raise TypeError("dx must have x's element type")
    g = NormGradsC(_buf(mean, "f32", rows, "mean", dev), _buf(rstd, "f32", rows, "rstd", dev), p,
                   DTYPES[_kind_of(dy)], stride, q, dx_stride,
                   _buf(dweight, "f32", d, "dweight", dev), _buf(dbias, "f32", d, "dbias", dev),
                   1 if accumulate else 0)
    w, nbytes = _work(ws, ws_bytes, dev)
    _check(_fn("dpo_norm_backward", _NORM_BWD)(ctypes.byref(n), ctypes.byref(g), w, nbytes,
                                               _stream(stream)), "dpo_norm_backward")
