"""ctypes binding of libarcs.so (argument marshalling only).

Every computation runs in the library's HIP kernels; this module checks
tensor shapes, dtypes and devices, takes raw device pointers and the current
HIP stream from PyTorch, and calls the C ABI of include/arcs.h with the same
names.  It never falls back to any other implementation: if the library is
missing or a call fails, it raises.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libarcs.so")

DTYPE_BF16 = 0
DTYPE_F32 = 1

# C enum values of include/arcs.h
OK = 0
ERR_NULL_POINTER = -1
ERR_BAD_BATCH = -2
ERR_BAD_VOCAB = -3
ERR_BAD_STRIDE = -4
ERR_BAD_DTYPE = -5
ERR_WORKSPACE_TOO_SMALL = -6
ERR_LAUNCH = -7
ERR_MISALIGNED = -8
ERR_BAD_HISTORY = -9
ERR_BAD_TOP_N = -10
ERR_BAD_CAPACITY = -11
ERR_SCRATCH_TOO_SMALL = -12
ERR_BAD_BUDGET = -13
ERR_BAD_DRY = -14
ERR_BAD_HIDDEN = -15
ERR_BAD_GROUP = -16
ERR_BAD_ACTIVATION = -17
ERR_BAD_BIAS = -18
ERR_BAD_MASK = -19
ERR_OVERLAP = -20
ERR_BAD_NORM = -21
ERR_BAD_PLAN = -22
DRY_MAX_WINDOW = 2048
DRY_MAX_BREAKERS = 64
NOALLOC_SCRATCH_BYTES = 16384
ROW_OK = 0
ROW_BAD_TEMPERATURE = 1
ROW_BAD_TOP_P = 2
ROW_BAD_MIN_P = 3
ROW_BAD_PENALTY = 4
ROW_BAD_FLAGS = 5
ROW_TIES_WIDE = 1  # arcs_row_params.flags bit
ROW_HISTORY_TOO_LONG = 6
ROW_VOCAB_TOO_LARGE = 7
ROW_BAD_TARGET = 8
ROW_BAD_MASK = 9
ROW_NOTHING_ALLOWED = 10
#: arcs_activation by the names `linear` takes
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "softcap": 5}
MAX_HIDDEN = 65536  # ARCS_MAX_HIDDEN
MAX_HISTORY = 4096
MAX_PENALTY_VOCAB = 262144
TOP_LOGPROBS_MAX_VOCAB = 262144  # ARCS_TOP_LOGPROBS_MAX_VOCAB

PATH_GREEDY = 1
PATH_SORT_SKIP = 2
PATH_CUTOFF = 4
PATH_MINP_FLOOR = 8
PATH_TIE_SPLIT = 16
PATH_PENALTY = 32
PATH_SPECIAL = 64
PATH_RESIDENT = 128
PATH_REREAD = 256

# struct arcs_row_params (32 bytes)
ROW_PARAMS_DTYPE = np.dtype(
    [("temperature", "<f4"), ("top_k", "<i4"), ("top_p", "<f4"), ("min_p", "<f4"),
     ("presence", "<f4"), ("frequency", "<f4"), ("repetition", "<f4"), ("flags", "<i4")]
)
# struct arcs_row_stats (64 bytes)
ROW_STATS_DTYPE = np.dtype(
    [("id", "<i4"), ("argmax", "<i4"), ("kept", "<i4"), ("cut_index", "<i4"),
     ("cut_value", "<f4"), ("max_logit", "<f4"), ("status", "<i4"), ("path", "<u4"),
     ("mass_total", "<f8"), ("mass_kept", "<f8"), ("uniform", "<f8"), ("reserved", "<u8")]
)
# struct arcs_tensor (32 bytes)
TENSOR_DTYPE = np.dtype([("data", "<u8"), ("out", "<u8"), ("count", "<i8"), ("dtype", "<i4"), ("out_dtype", "<i4")])
assert TENSOR_DTYPE.itemsize == 32
assert ROW_PARAMS_DTYPE.itemsize == 32 and ROW_STATS_DTYPE.itemsize == 64


class ArcsError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: arcs status {code} ({status_string(code)})")


_lib = None


def library() -> ctypes.CDLL:
    """Load libarcs.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(LIB_PATH)
        c_i64, c_u64, c_p, c_i = ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_int
        lib.arcs_argmax.argtypes = [c_p, c_i, c_i64, c_i64, c_i64, c_p, c_p]
        lib.arcs_argmax.restype = c_i
        lib.arcs_sample.argtypes = [c_p, c_i, c_i64, c_i64, c_i64, c_p, c_p, c_p, c_u64, c_u64,
                                    c_p, c_p, c_p, ctypes.c_size_t, c_p]
        lib.arcs_sample.restype = c_i
        lib.arcs_sample_debug.argtypes = [c_p, c_i, c_i64, c_i64, c_i64, c_p, c_p, c_p, c_u64, c_u64,
                                          c_p, c_p, c_p, ctypes.c_size_t, c_p, c_p, c_p, c_p]
        lib.arcs_sample_debug.restype = c_i
        lib.arcs_sample_dry.argtypes = [c_p, c_i, c_i64, c_i64, c_i64, c_p, c_p, c_p, c_p, c_p, c_i, c_u64,
                                         c_u64, c_p, c_p, c_p, c_u64, c_p]
        lib.arcs_sample_dry.restype = c_i
        lib.arcs_sample_hybrid_nucleus.argtypes = [c_p, c_i, c_i64, c_i64, c_i64, c_p, c_p, c_i, c_u64, c_u64,
                                                    c_p, c_p, c_p, c_p]
        lib.arcs_sample_hybrid_nucleus.restype = c_i
        lib.arcs_sample_noalloc.argtypes = [c_p, c_i, c_i64, c_i64, c_i64, c_p, c_p, c_p, c_u64, c_u64,
                                             c_p, c_p, c_p]
        lib.arcs_sample_noalloc.restype = c_i
        lib.arcs_sample_keyed.argtypes = [c_p, c_i, c_i64, c_i64, c_i64, c_p, c_p, c_p, c_p, c_i,
                                          c_p, c_p, c_p, ctypes.c_size_t, c_p]
        lib.arcs_sample_keyed.restype = c_i
        lib.arcs_top_logprobs.argtypes = [c_p, c_i, c_i64, c_i64, c_i64, c_p, c_i, c_p, c_p, c_p, c_p]
        lib.arcs_top_logprobs.restype = c_i
        lib.arcs_commit_tokens.argtypes = [c_p, c_i64, c_i64, c_p, c_p, c_p, c_u64, c_p, c_p, c_p, c_p]
        lib.arcs_commit_tokens.restype = c_i
        lib.arcs_w4_logits.argtypes = [c_p, c_i64, c_i64, c_i64, c_p, c_i64, c_i64, c_p, c_i, c_i64, c_p, c_i64,
                                       c_i, c_p, c_i, c_i64, c_p, ctypes.c_size_t, c_p]
        lib.arcs_w4_logits.restype = c_i
        lib.arcs_w4_logits_workspace_bytes.argtypes = [c_i64, c_i64, c_i]
        lib.arcs_w4_logits_workspace_bytes.restype = ctypes.c_size_t
        lib.arcs_linear_cross_entropy.argtypes = [c_p, c_i64, c_p, c_i64, c_i, c_i64, c_i64, c_i64, c_p,
                                                  ctypes.c_int32, c_p, c_p, c_p, c_p, c_p, ctypes.c_size_t, c_p]
        lib.arcs_linear_cross_entropy.restype = c_i
        lib.arcs_linear_cross_entropy_backward.argtypes = [c_p, c_i64, c_p, c_i64, c_i, c_i64, c_i64, c_i64, c_p,
                                                           ctypes.c_int32, c_p, c_p, c_p, c_p, c_p, c_p,
                                                           ctypes.c_size_t, c_p]
        lib.arcs_linear_cross_entropy_backward.restype = c_i
        lib.arcs_linear_cross_entropy_workspace_bytes.argtypes = [c_i64, c_i64, c_i64, c_i, c_i]
        lib.arcs_linear_cross_entropy_workspace_bytes.restype = ctypes.c_size_t
        lib.arcs_linear.argtypes = [c_p, c_i64, c_p, c_i64, c_i, c_i64, c_i64, c_i64, c_p, c_i, ctypes.c_float, c_p,
                                    c_i64, c_p, c_i, c_i64, c_p, c_p, ctypes.c_size_t, c_p]
        lib.arcs_linear.restype = c_i
        lib.arcs_linear_backward.argtypes = [c_p, c_i64, c_p, c_i64, c_i, c_i64, c_i64, c_i64, c_i, ctypes.c_float,
                                             c_p, c_p, c_i, c_i64, c_p, c_p, c_p, c_p, ctypes.c_size_t, c_p]
        lib.arcs_linear_backward.restype = c_i
        for name in ("arcs_linear_workspace_bytes", "arcs_linear_backward_workspace_bytes"):
            getattr(lib, name).argtypes = [c_i64, c_i64, c_i64, c_i, c_i]
            getattr(lib, name).restype = ctypes.c_size_t
        lib.arcs_adjust_logits.argtypes = [c_p, c_i, c_i64, c_i64, c_i64, c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_i64,
                                           c_i64, c_p, c_p, c_i, c_i64, c_p, c_p]
        lib.arcs_adjust_logits.restype = c_i
        lib.arcs_gradient_plan.argtypes = [c_p, c_i64, c_p, ctypes.c_size_t]
        lib.arcs_gradient_plan.restype = c_i
        lib.arcs_gradient_plan_bytes.argtypes = [c_p, c_i64]
        lib.arcs_gradient_plan_bytes.restype = ctypes.c_size_t
        lib.arcs_gradient_norm.argtypes = [c_p, ctypes.c_size_t, c_p, c_p, ctypes.c_size_t, c_p]
        lib.arcs_gradient_norm.restype = c_i
        lib.arcs_clip_gradients.argtypes = [c_p, ctypes.c_size_t, ctypes.c_double, c_p, c_p, ctypes.c_size_t, c_p]
        lib.arcs_clip_gradients.restype = c_i
        lib.arcs_gradient_workspace_bytes.argtypes = [ctypes.c_size_t]
        lib.arcs_gradient_workspace_bytes.restype = ctypes.c_size_t
        lib.arcs_sample_workspace_bytes.argtypes = [c_i64, c_i64, c_i]
        lib.arcs_sample_workspace_bytes.restype = ctypes.c_size_t
        lib.arcs_long_history_workspace_bytes.argtypes = [c_i64, c_i64]
        lib.arcs_long_history_workspace_bytes.restype = ctypes.c_size_t
        lib.arcs_status_string.argtypes = [c_i]
        lib.arcs_status_string.restype = ctypes.c_char_p
        lib.arcs_version.argtypes = []
        lib.arcs_version.restype = c_i
        _lib = lib
    return _lib


def status_string(code: int) -> str:
    return library().arcs_status_string(int(code)).decode()


def version() -> int:
    return int(library().arcs_version())


def workspace_bytes(B: int, V: int, dtype: int) -> int:
    return int(library().arcs_sample_workspace_bytes(int(B), int(V), int(dtype)))


def long_history_workspace_bytes(B: int, V: int) -> int:
    return int(library().arcs_long_history_workspace_bytes(int(B), int(V)))


@functools.lru_cache(maxsize=256)
def w4_logits_workspace_bytes(B: int, D: int, group_size: int) -> int:
    return int(library().arcs_w4_logits_workspace_bytes(int(B), int(D), int(group_size)))


@functools.lru_cache(maxsize=256)
def linear_cross_entropy_workspace_bytes(N: int, V: int, D: int, dtype: int, backward: bool = False) -> int:
    return int(library().arcs_linear_cross_entropy_workspace_bytes(int(N), int(V), int(D), int(dtype),
                                                                   1 if backward else 0))


@functools.lru_cache(maxsize=256)
def linear_workspace_bytes(N: int, V: int, D: int, dtype: int, rows_aligned: bool = False,
                           backward: bool = False) -> int:
    call = library().arcs_linear_backward_workspace_bytes if backward else library().arcs_linear_workspace_bytes
    return int(call(int(N), int(V), int(D), int(dtype), 1 if rows_aligned else 0))


# --------------------------------------------------------------------------
# torch-facing helpers
#
# `stream=` is the torch stream a call is enqueued on (the current one if it is
# None).  The caller orders it against the streams that make the inputs and read
# the results; tensors may be dropped as soon as the call returns.
# --------------------------------------------------------------------------
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_ptr(stream) -> int:
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _used_on(stream, *tensors) -> None:
    """After a call on a given stream: tells the allocator that the stream uses these
    tensors, so that one dropped right after the call (a workspace of the call's own
    among them) is not handed out again while the kernels run."""
    if isinstance(stream, _torch().cuda.Stream):
        for t in tensors:
            if t is not None and t.is_cuda:
                t.record_stream(stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float32:
        return DTYPE_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _check_logits(logits):
    if not logits.is_cuda:
        raise ValueError("logits must be a device tensor")
    if logits.dim() != 2:
        raise ValueError("logits must be [B, V]")
    if logits.stride(1) != 1:
        raise ValueError("logits rows must be contiguous (stride(1) == 1)")
    return logits.shape[0], logits.shape[1], logits.stride(0)


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _list_ptr(t) -> Optional[int]:
    """_ptr of a list that may be given without elements, which torch has no address for:
    the library tells it from one that is not given."""
    return None if t is None else int(t.data_ptr()) or 256


def params_to_device(params: np.ndarray, device="cuda"):
    """Copy a structured array of arcs_row_params records to the device (uint8 [B, 32])."""
    torch = _torch()
    arr = np.ascontiguousarray(params).view(np.uint8).reshape(len(params), 32)
    return torch.from_numpy(arr.copy()).to(device)


def _check_out(t, dtype, n: int, name: str):
    """A caller-provided device buffer: dtype, element count and a dense layout
    (the kernels write from the base pointer in row order)."""
    torch = _torch()
    if t.dtype != dtype or t.numel() != n or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device {dtype} tensor of {n} elements")


def argmax(logits, out=None, stream=None):
    """out[b] = lowest index of the row maximum of logits[b] (int32, on device)."""
    torch = _torch()
    B, V, stride = _check_logits(logits)
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=logits.device)
    _check_out(out, torch.int32, B, "out")
    st = library().arcs_argmax(_ptr(logits), _dtype_code(logits), B, V, stride, _ptr(out), _stream_ptr(stream))
    if st != OK:
        raise ArcsError(st, "arcs_argmax")
    _used_on(stream, logits, out)
    return out


def top_logprobs(logits, n: int, temperature=None, out_ids=None, out_logprobs=None, out_status=None,
                 stream=None):
    """arcs_top_logprobs: (ids int32 [B, n], logprobs float32 [B, n]) on device.

    ``temperature`` is a device float32 tensor of B values or None (T = 1);
    ``out_status`` an optional device int32 tensor of B values.
    """
    torch = _torch()
    B, V, stride = _check_logits(logits)
    dev = logits.device
    if temperature is not None and (temperature.dtype != torch.float32 or not temperature.is_cuda
                                    or temperature.numel() != B or not temperature.is_contiguous()):
        raise ValueError("temperature must be a contiguous device float32 tensor of B elements")
    if out_ids is None:
        out_ids = torch.empty((B, n), dtype=torch.int32, device=dev)
    if out_logprobs is None:
        out_logprobs = torch.empty((B, n), dtype=torch.float32, device=dev)
    if out_ids.dtype != torch.int32 or out_ids.numel() != B * n or not out_ids.is_cuda or not out_ids.is_contiguous():
        raise ValueError("out_ids must be a device int32 tensor of B * n elements")
    if (out_logprobs.dtype != torch.float32 or out_logprobs.numel() != B * n or not out_logprobs.is_cuda
            or not out_logprobs.is_contiguous()):
        raise ValueError("out_logprobs must be a device float32 tensor of B * n elements")
    if out_status is not None:
        _check_out(out_status, torch.int32, B, "out_status")
    st = library().arcs_top_logprobs(_ptr(logits), _dtype_code(logits), B, V, stride, _ptr(temperature),
                                     int(n), _ptr(out_ids), _ptr(out_logprobs), _ptr(out_status),
                                     _stream_ptr(stream))
    if st != OK:
        raise ArcsError(st, "arcs_top_logprobs")
    _used_on(stream, logits, temperature, out_ids, out_logprobs, out_status)
    return out_ids, out_logprobs


def commit_tokens(ids, V: int, position, ring, published, drained, fault, next_input=None, stream=None):
    """arcs_commit_tokens: publish one step's tokens into a pinned host ring.

    ``ids`` device int32 [B]; ``position`` device int64 [1]; ``ring`` pinned
    CPU int32 [capacity, B]; ``published`` and ``drained`` pinned CPU int64
    [1]; ``fault`` pinned CPU int32 [1]; ``next_input`` device int32 [B] or None.
    """
    torch = _torch()
    B = ids.numel()
    if not ids.is_cuda or ids.dtype != torch.int32 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous device int32 tensor")
    _check_out(position, torch.int64, 1, "position")
    for name, t, dt in (("ring", ring, torch.int32), ("published", published, torch.int64),
                        ("drained", drained, torch.int64), ("fault", fault, torch.int32)):
        if t.is_cuda or not t.is_pinned() or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous pinned CPU tensor of {dt}")
    if ring.numel() % B != 0:
        raise ValueError("ring must hold capacity * B elements")
    if next_input is not None:
        _check_out(next_input, torch.int32, B, "next_input")
    st = library().arcs_commit_tokens(_ptr(ids), B, int(V), _ptr(next_input), _ptr(position), _ptr(ring),
                                      ring.numel() // B, _ptr(published), _ptr(drained), _ptr(fault),
                                      _stream_ptr(stream))
    if st != OK:
        raise ArcsError(st, "arcs_commit_tokens")
    _used_on(stream, ids, position, next_input)


def _check_params(params, B):
    torch = _torch()
    if not params.is_cuda or params.dtype != torch.uint8 or params.numel() != 32 * B or not params.is_contiguous():
        raise ValueError("params must be a contiguous device uint8 tensor of B * 32 bytes")


def _check_hist(hist_ids, hist_offsets, B):
    torch = _torch()
    if (hist_ids is None) != (hist_offsets is None):
        raise ValueError("hist_ids and hist_offsets go together")
    if hist_ids is not None:
        if hist_ids.dtype != torch.int32 or not hist_ids.is_cuda or not hist_ids.is_contiguous():
            raise ValueError("hist_ids must be a contiguous device int32 tensor")
        _check_out(hist_offsets, torch.int64, B + 1, "hist_offsets")


def sample(logits, params, hist_ids=None, hist_offsets=None, seed: int = 0, step: int = 0,
           out=None, out_status=None, workspace=None, stream=None):
    """One token per row (int32, on device); see arcs_sample in include/arcs.h."""
    torch = _torch()
    B, V, stride = _check_logits(logits)
    _check_params(params, B)
    _check_hist(hist_ids, hist_offsets, B)
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=logits.device)
    _check_out(out, torch.int32, B, "out")
    if out_status is not None:
        _check_out(out_status, torch.int32, B, "out_status")
    ws_need = workspace_bytes(B, V, _dtype_code(logits))
    if workspace is not None and (not workspace.is_cuda or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous device tensor")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if ws_need and workspace is None:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=logits.device)
        ws_bytes = ws_need
    st = library().arcs_sample(_ptr(logits), _dtype_code(logits), B, V, stride, _ptr(params),
                               _ptr(hist_ids), _ptr(hist_offsets), int(seed) & (2**64 - 1),
                               int(step) & (2**64 - 1), _ptr(out), _ptr(out_status), _ptr(workspace),
                               ws_bytes, _stream_ptr(stream))
    if st != OK:
        raise ArcsError(st, "arcs_sample")
    _used_on(stream, logits, params, hist_ids, hist_offsets, out, out_status, workspace)
    return out


def sample_noalloc(logits, params, hist_ids=None, hist_offsets=None, seed: int = 0, step: int = 0,
                   out=None, out_status=None, stream=None):
    """arcs_sample_noalloc: as sample, with the library's own device scratch
    instead of a workspace (the C call allocates nothing; pass `out` to keep
    this wrapper from allocating it)."""
    torch = _torch()
    B, V, stride = _check_logits(logits)
    _check_params(params, B)
    _check_hist(hist_ids, hist_offsets, B)
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=logits.device)
    _check_out(out, torch.int32, B, "out")
    if out_status is not None:
        _check_out(out_status, torch.int32, B, "out_status")
    st = library().arcs_sample_noalloc(_ptr(logits), _dtype_code(logits), B, V, stride, _ptr(params),
                                       _ptr(hist_ids), _ptr(hist_offsets), int(seed) & (2**64 - 1),
                                       int(step) & (2**64 - 1), _ptr(out), _ptr(out_status), _stream_ptr(stream))
    if st != OK:
        raise ArcsError(st, "arcs_sample_noalloc")
    _used_on(stream, logits, params, hist_ids, hist_offsets, out, out_status)
    return out


def dry_to_device(dry, device="cuda"):
    """A DRY_DTYPE structured numpy array (workloads.make_dry) as device bytes."""
    torch = _torch()
    arr = np.ascontiguousarray(dry).view(np.uint8).reshape(len(dry), 16)
    return torch.from_numpy(arr.copy()).to(device)


def sample_dry(logits, params, hist_ids, hist_offsets, dry, breakers=None, seed: int = 0, step: int = 0,
               out=None, out_status=None, workspace=None, stream=None):
    """arcs_sample_dry: arcs_sample with per-row DRY records (device bytes from
    dry_to_device) and optional device int32 sequence breakers."""
    torch = _torch()
    B, V, stride = _check_logits(logits)
    _check_params(params, B)
    _check_hist(hist_ids, hist_offsets, B)
    if dry is not None and (not dry.is_cuda or dry.dtype != torch.uint8 or dry.numel() != 16 * B
                            or not dry.is_contiguous()):
        raise ValueError("dry must be contiguous device bytes of B DRY records (dry_to_device)")
    nb = 0
    if breakers is not None:
        nb = breakers.numel()
        _check_out(breakers, torch.int32, nb, "breakers")
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=logits.device)
    _check_out(out, torch.int32, B, "out")
    if out_status is not None:
        _check_out(out_status, torch.int32, B, "out_status")
    ws_need = workspace_bytes(B, V, _dtype_code(logits))
    if ws_need and workspace is None:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=logits.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = library().arcs_sample_dry(_ptr(logits), _dtype_code(logits), B, V, stride, _ptr(params), _ptr(hist_ids),
                                   _ptr(hist_offsets), _ptr(dry), _ptr(breakers), nb, int(seed) & (2**64 - 1),
                                   int(step) & (2**64 - 1), _ptr(out), _ptr(out_status), _ptr(workspace),
                                   ws_bytes, _stream_ptr(stream))
    if st != OK:
        raise ArcsError(st, "arcs_sample_dry")
    _used_on(stream, logits, params, hist_ids, hist_offsets, dry, breakers, out, out_status, workspace)
    return out


def sample_hybrid_nucleus(logits, temperature, top_p, budget: int = 32, seed: int = 0, step: int = 0,
                          out=None, out_kept=None, out_status=None, stream=None):
    """arcs_sample_hybrid_nucleus: the baseline enumeration / bisection nucleus
    sampler (per-row float32 temperature and top_p on the device)."""
    torch = _torch()
    B, V, stride = _check_logits(logits)
    for name, t in (("temperature", temperature), ("top_p", top_p)):
        _check_out(t, torch.float32, B, name)
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=logits.device)
    _check_out(out, torch.int32, B, "out")
    for name, t in (("out_kept", out_kept), ("out_status", out_status)):
        if t is not None:
            _check_out(t, torch.int32, B, name)
    st = library().arcs_sample_hybrid_nucleus(_ptr(logits), _dtype_code(logits), B, V, stride, _ptr(temperature),
                                              _ptr(top_p), int(budget), int(seed) & (2**64 - 1),
                                              int(step) & (2**64 - 1), _ptr(out), _ptr(out_kept),
                                              _ptr(out_status), _stream_ptr(stream))
    if st != OK:
        raise ArcsError(st, "arcs_sample_hybrid_nucleus")
    _used_on(stream, logits, temperature, top_p, out, out_kept, out_status)
    return out


def make_key(seed: int = 0, step: int = 0, device="cuda"):
    """A device RNG key {seed, step} for sample_keyed (int64 storage of the
    two uint64 words)."""
    torch = _torch()
    words = [int(seed) & (2**64 - 1), int(step) & (2**64 - 1)]
    words = [w - 2**64 if w >= 2**63 else w for w in words]
    return torch.tensor(words, dtype=torch.int64, device=device)


def sample_keyed(logits, params, key, hist_ids=None, hist_offsets=None, advance: bool = True,
                 out=None, out_status=None, workspace=None, stream=None):
    """arcs_sample_keyed: seed and step read from the device key (see make_key);
    with `advance` the key's step moves on by one after the draw."""
    torch = _torch()
    B, V, stride = _check_logits(logits)
    _check_params(params, B)
    _check_hist(hist_ids, hist_offsets, B)
    if not key.is_cuda or key.dtype != torch.int64 or key.numel() != 2 or not key.is_contiguous():
        raise ValueError("key must be a contiguous device int64 tensor of 2 elements (seed, step)")
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=logits.device)
    _check_out(out, torch.int32, B, "out")
    if out_status is not None:
        _check_out(out_status, torch.int32, B, "out_status")
    ws_need = workspace_bytes(B, V, _dtype_code(logits))
    if workspace is not None and (not workspace.is_cuda or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous device tensor")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if ws_need and workspace is None:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=logits.device)
        ws_bytes = ws_need
    st = library().arcs_sample_keyed(_ptr(logits), _dtype_code(logits), B, V, stride, _ptr(params),
                                     _ptr(hist_ids), _ptr(hist_offsets), _ptr(key), 1 if advance else 0,
                                     _ptr(out), _ptr(out_status), _ptr(workspace), ws_bytes,
                                     _stream_ptr(stream))
    if st != OK:
        raise ArcsError(st, "arcs_sample_keyed")
    _used_on(stream, logits, params, key, hist_ids, hist_offsets, out, out_status, workspace)
    return out


def sample_debug(logits, params, hist_ids=None, hist_offsets=None, seed: int = 0, step: int = 0,
                 uniforms=None, want_probs: bool = False, workspace=None, stream=None):
    """arcs_sample_debug: returns (ids, status, stats[B] numpy structured, probs or None)."""
    torch = _torch()
    B, V, stride = _check_logits(logits)
    _check_params(params, B)
    _check_hist(hist_ids, hist_offsets, B)
    dev = logits.device
    out = torch.empty(B, dtype=torch.int32, device=dev)
    status = torch.empty(B, dtype=torch.int32, device=dev)
    stats = torch.zeros(B * ROW_STATS_DTYPE.itemsize, dtype=torch.uint8, device=dev)
    probs = torch.empty((B, V), dtype=torch.float32, device=dev) if want_probs else None
    if uniforms is not None:
        _check_out(uniforms, torch.float64, B, "uniforms")
    ws_need = workspace_bytes(B, V, _dtype_code(logits))
    if workspace is not None and (not workspace.is_cuda or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous device tensor")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if ws_need and workspace is None:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=dev)
        ws_bytes = ws_need
    st = library().arcs_sample_debug(_ptr(logits), _dtype_code(logits), B, V, stride, _ptr(params),
                                     _ptr(hist_ids), _ptr(hist_offsets), int(seed) & (2**64 - 1),
                                     int(step) & (2**64 - 1), _ptr(out), _ptr(status), _ptr(workspace),
                                     ws_bytes, _ptr(uniforms), _ptr(probs), _ptr(stats), _stream_ptr(stream))
    if st != OK:
        raise ArcsError(st, "arcs_sample_debug")
    torch.cuda.synchronize(dev)
    st_np = stats.cpu().numpy().view(ROW_STATS_DTYPE)
    return out, status, st_np, probs


# --------------------------------------------------------------------------
# the vocabulary head: 4-bit logits and the linear cross entropy
# --------------------------------------------------------------------------
_NO_CONTEXT = contextlib.nullcontext()


def _head_stream(stream, device) -> int:
    """_stream_ptr of a head call.  Building a Stream object takes 3 us, a fourth of a
    one-row call; the raw handle of the current one takes none of that where torch gives it."""
    if stream is not None:
        return int(stream.cuda_stream)
    raw = getattr(_torch()._C, "_cuda_getCurrentRawStream", None)
    return raw(device.index) if raw is not None else _stream_ptr(None)


def _work_on(device, stream):
    """The device and stream a head call runs on: the given stream, which has to
    be one of the tensors' device, or that device's current stream.  What the
    call allocates then belongs to that stream; _head_used says who else uses it."""
    torch = _torch()
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
        return torch.cuda.stream(stream)
    if torch.cuda.current_device() != device.index:
        return torch.cuda.device(device)
    return _NO_CONTEXT


def _head_used(stream, device, inputs, outputs) -> None:
    """_used_on of a head call on a given stream, whose outputs, allocated on that
    stream, the caller's current stream may go on with (ordered by the caller)."""
    if stream is not None:
        _used_on(stream, *inputs, *outputs)
        _used_on(_torch().cuda.current_stream(device), *outputs)


def _matrix(t, name: str, dtype, rows: int, cols: int, device):
    """A device matrix with unit column stride; returns its row stride."""
    if t.dtype != dtype or t.shape != (rows, cols) or t.device != device:
        raise ValueError(f"{name} must be a [{rows}, {cols}] {dtype} tensor on {device}")
    row, column = t.stride()
    if column != 1 and cols > 1:
        raise ValueError(f"{name} rows must be contiguous (stride(1) == 1)")
    return cols if rows == 1 else row


def _vector(t, name: str, dtype, n: int, device):
    if t.dtype != dtype or t.numel() != n or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on {device}")


def _hidden_shape(hidden):
    if not hidden.is_cuda:
        raise ValueError("hidden must be a device tensor")
    if hidden.dim() != 2:
        raise ValueError("hidden must be [rows, D]")
    rows, D = hidden.shape
    return rows, D, hidden.device


def w4_logits(hidden, qweight, scales, group_size: int, zeros=None, out=None, out_dtype=None, workspace=None,
              stream=None):
    """arcs_w4_logits: [B, V] logits of a 4-bit head, ready for argmax, sample and top_logprobs.

    ``hidden`` bfloat16 [B, D]; ``qweight`` uint8 [V, D / 2], the even weight in
    the low nibble; ``scales`` bfloat16 or float32 [V, D / group_size]; ``zeros``
    uint8 [V, D / group_size] or None (8).  ``out`` [B, V] bfloat16 or float32
    with contiguous rows, or None: a new tensor of ``out_dtype`` (bfloat16).
    """
    torch = _torch()
    B, D, dev = _hidden_shape(hidden)
    V, G = qweight.shape[0], int(group_size)
    groups = D // G if G > 0 else 0
    hs = _matrix(hidden, "hidden", torch.bfloat16, B, D, dev)
    qs = _matrix(qweight, "qweight", torch.uint8, V, D // 2, dev)
    sdt = _dtype_code_of(scales, "scales")
    ss = _matrix(scales, "scales", scales.dtype, V, groups, dev)
    zs = 0 if zeros is None else _matrix(zeros, "zeros", torch.uint8, V, groups, dev)
    with _work_on(dev, stream):
        if out is None:
            out = torch.empty((B, V), dtype=torch.bfloat16 if out_dtype is None else out_dtype, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out is not of out_dtype")
        odt = _dtype_code_of(out, "out")
        ls = _matrix(out, "out", out.dtype, B, V, dev)
        workspace, ws_bytes = _head_workspace(workspace, w4_logits_workspace_bytes(B, D, G), dev)
        st = library().arcs_w4_logits(_ptr(hidden), B, D, hs, _ptr(qweight), V, qs, _ptr(scales), sdt, ss,
                                      _ptr(zeros), zs, G, _ptr(out), odt, ls, _ptr(workspace), ws_bytes,
                                      _head_stream(stream, dev))
    if st != OK:
        raise ArcsError(st, "arcs_w4_logits")
    _head_used(stream, dev, (hidden, qweight, scales, zeros, workspace), (out,))
    return out


def _dtype_code_of(t, name: str) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    if t.dtype == torch.float32:
        return DTYPE_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _cross_entropy_inputs(hidden, weight, targets, temperature, ignore_index):
    torch = _torch()
    N, D, dev = _hidden_shape(hidden)
    dt = _dtype_code_of(hidden, "hidden")
    hs = _matrix(hidden, "hidden", hidden.dtype, N, D, dev)
    V = weight.shape[0]
    ws = _matrix(weight, "weight", hidden.dtype, V, D, dev)
    _vector(targets, "targets", torch.int32, N, dev)
    if temperature is not None:
        _vector(temperature, "temperature", torch.float32, N, dev)
    if not -2**31 <= ignore_index < 2**31:
        raise ValueError("ignore_index must fit int32")
    return N, V, D, dev, dt, hs, ws


def _head_workspace(workspace, need: int, dev):
    """The caller's workspace, or one of the needed size (sizes the library
    refuses need none: the call itself reports them)."""
    torch = _torch()
    if workspace is None:
        return (None, 0) if need == 0 else (torch.empty(need, dtype=torch.uint8, device=dev), need)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace, workspace.numel() * workspace.element_size()


def linear_cross_entropy(hidden, weight, targets, temperature=None, ignore_index: int = -100, out_loss=None,
                         out_lse=None, out_status=None, workspace=None, stream=None):
    """arcs_linear_cross_entropy: (loss, lse), float32 [N] each, of int32 ``targets`` under
    softmax(hidden weight^T / temperature), without the [N, V] logits.

    -loss is each target's log-probability; lse goes to
    linear_cross_entropy_backward.  The result has no autograd graph: gradients
    are computed by that call.
    """
    torch = _torch()
    N, V, D, dev, dt, hs, ws = _cross_entropy_inputs(hidden, weight, targets, temperature, ignore_index)
    with _work_on(dev, stream):
        if out_loss is None:
            out_loss = torch.empty(N, dtype=torch.float32, device=dev)
        if out_lse is None:
            out_lse = torch.empty(N, dtype=torch.float32, device=dev)
        _vector(out_loss, "out_loss", torch.float32, N, dev)
        _vector(out_lse, "out_lse", torch.float32, N, dev)
        if out_status is not None:
            _vector(out_status, "out_status", torch.int32, N, dev)
        workspace, ws_bytes = _head_workspace(
            workspace, linear_cross_entropy_workspace_bytes(N, V, D, dt, False), dev)
        st = library().arcs_linear_cross_entropy(_ptr(hidden), hs, _ptr(weight), ws, dt, N, V, D, _ptr(targets),
                                                 int(ignore_index), _ptr(temperature), _ptr(out_loss),
                                                 _ptr(out_lse), _ptr(out_status), _ptr(workspace), ws_bytes,
                                                 _head_stream(stream, dev))
    if st != OK:
        raise ArcsError(st, "arcs_linear_cross_entropy")
    _head_used(stream, dev, (hidden, weight, targets, temperature, workspace), (out_loss, out_lse, out_status))
    return out_loss, out_lse


def linear_cross_entropy_backward(hidden, weight, targets, lse, grad_loss, temperature=None,
                                  ignore_index: int = -100, out_dhidden=None, out_dweight=None,
                                  want_hidden: bool = True, want_weight: bool = True, workspace=None, stream=None):
    """arcs_linear_cross_entropy_backward: (dhidden [N, D], dweight [V, D]) of
    sum(grad_loss * loss), in the inputs' type; None in place of one not wanted.
    ``lse`` is the forward call's, ``grad_loss`` float32 [N]."""
    torch = _torch()
    N, V, D, dev, dt, hs, ws = _cross_entropy_inputs(hidden, weight, targets, temperature, ignore_index)
    _vector(lse, "lse", torch.float32, N, dev)
    _vector(grad_loss, "grad_loss", torch.float32, N, dev)
    with _work_on(dev, stream):
        if want_hidden and out_dhidden is None:
            out_dhidden = torch.empty((N, D), dtype=hidden.dtype, device=dev)
        if want_weight and out_dweight is None:
            out_dweight = torch.empty((V, D), dtype=hidden.dtype, device=dev)
        if out_dhidden is not None:
            _vector(out_dhidden, "out_dhidden", hidden.dtype, N * D, dev)
        if out_dweight is not None:
            _vector(out_dweight, "out_dweight", hidden.dtype, V * D, dev)
        workspace, ws_bytes = _head_workspace(
            workspace, linear_cross_entropy_workspace_bytes(N, V, D, dt, True), dev)
        st = library().arcs_linear_cross_entropy_backward(
            _ptr(hidden), hs, _ptr(weight), ws, dt, N, V, D, _ptr(targets), int(ignore_index), _ptr(temperature),
            _ptr(lse), _ptr(grad_loss), _ptr(out_dhidden), _ptr(out_dweight), _ptr(workspace), ws_bytes,
            _head_stream(stream, dev))
    if st != OK:
        raise ArcsError(st, "arcs_linear_cross_entropy_backward")
    _head_used(stream, dev, (hidden, weight, targets, temperature, lse, grad_loss, workspace),
               (out_dhidden, out_dweight))
    return out_dhidden, out_dweight


# --------------------------------------------------------------------------
# linear layers
# --------------------------------------------------------------------------
# One token's call takes as long on the host as on the card, so what follows looks each
# attribute up once and checks only what the caller gave.
def _linear_inputs(hidden, weight, activation, softcap):
    """Sizes, device, type code and strides of the two matrices, the activation's code, and
    whether their rows are on the 16-byte grid as arcs_linear_workspace_bytes asks."""
    if not hidden.is_cuda:
        raise ValueError("hidden must be a device tensor")
    if hidden.dim() != 2 or weight.dim() != 2:
        raise ValueError("hidden must be [rows, D] and weight [V, D]")
    N, D = hidden.shape
    V = weight.shape[0]
    dev, dtype = hidden.device, hidden.dtype
    dt = _dtype_code_of(hidden, "hidden")
    hs = _matrix(hidden, "hidden", dtype, N, D, dev)
    ws = _matrix(weight, "weight", dtype, V, D, dev)
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}")
    size = 4 if dt == DTYPE_F32 else 2
    aligned = ((hidden.data_ptr() | weight.data_ptr() | (hs | ws | D) * size) & 15) == 0 and max(hs, ws) * size < 2**23
    return N, V, D, dev, dtype, dt, hs, ws, act, aligned


def linear(hidden, weight, bias=None, activation: str = "none", softcap: float = 0.0, residual=None, out=None,
           out_dtype=None, out_pre=None, want_pre: bool = False, workspace=None, stream=None):
    """arcs_linear: residual + act(hidden weight^T + bias), [N, V], in one pass: a head's
    logits, ready for argmax, sample and top_logprobs, or a block in front of it.

    ``hidden`` [N, D] and ``weight`` [V, D] bfloat16 or float32; ``bias`` [V] and
    ``residual`` [N, V] of their type or None; ``activation`` one of ACTIVATIONS
    ("softcap": softcap * tanh(z / softcap)).  ``out`` [N, V] bfloat16 or float32 with
    contiguous rows (the residual itself is allowed), or None: a new tensor of ``out_dtype``
    (the inputs' type).  With ``want_pre`` or ``out_pre`` (dense [N, V] of the inputs' type)
    returns (out, pre): linear_backward needs pre where there is an activation.  The result
    has no autograd graph.
    """
    torch = _torch()
    N, V, D, dev, dtype, dt, hs, ws, act, aligned = _linear_inputs(hidden, weight, activation, softcap)
    if bias is not None:
        _vector(bias, "bias", dtype, V, dev)
    rs = 0 if residual is None else _matrix(residual, "residual", dtype, N, V, dev)
    with _work_on(dev, stream):
        if out is None:
            out = torch.empty((N, V), dtype=dtype if out_dtype is None else out_dtype, device=dev)
            os_ = V
        else:
            if out_dtype is not None and out.dtype != out_dtype:
                raise ValueError("out is not of out_dtype")
            os_ = _matrix(out, "out", out.dtype, N, V, dev)
        odt = _dtype_code_of(out, "out")
        if out_pre is not None:
            _vector(out_pre, "out_pre", dtype, N * V, dev)
        elif want_pre:
            out_pre = torch.empty((N, V), dtype=dtype, device=dev)
        workspace, ws_bytes = _head_workspace(workspace, linear_workspace_bytes(N, V, D, dt, aligned), dev)
        st = library().arcs_linear(hidden.data_ptr(), hs, weight.data_ptr(), ws, dt, N, V, D, _ptr(bias), act, softcap,
                                   _ptr(residual), rs, out.data_ptr(), odt, os_, _ptr(out_pre), _ptr(workspace),
                                   ws_bytes, _head_stream(stream, dev))
    if st != OK:
        raise ArcsError(st, "arcs_linear")
    if stream is not None:
        _head_used(stream, dev, (hidden, weight, bias, residual, workspace), (out, out_pre))
    return out if out_pre is None else (out, out_pre)


def linear_backward(hidden, weight, grad_out, pre=None, activation: str = "none", softcap: float = 0.0,
                    out_dhidden=None, out_dweight=None, out_dbias=None, want_hidden: bool = True,
                    want_weight: bool = True, want_bias: bool = False, workspace=None, stream=None):
    """arcs_linear_backward: (dhidden [N, D], dweight [V, D], dbias [V]) of
    sum(grad_out * out), in the inputs' type; None in place of one not wanted.

    ``grad_out`` [N, V] bfloat16 or float32 with contiguous rows; ``pre`` the forward
    call's (not needed without an activation).  The residual's gradient is grad_out.
    """
    torch = _torch()
    N, V, D, dev, dtype, dt, hs, ws, act, aligned = _linear_inputs(hidden, weight, activation, softcap)
    gdt = _dtype_code_of(grad_out, "grad_out")
    gs = _matrix(grad_out, "grad_out", grad_out.dtype, N, V, dev)
    if pre is not None:
        _vector(pre, "pre", dtype, N * V, dev)
    with _work_on(dev, stream):
        if want_hidden and out_dhidden is None:
            out_dhidden = torch.empty((N, D), dtype=dtype, device=dev)
        if want_weight and out_dweight is None:
            out_dweight = torch.empty((V, D), dtype=dtype, device=dev)
        if want_bias and out_dbias is None:
            out_dbias = torch.empty(V, dtype=dtype, device=dev)
        for t, name, n in ((out_dhidden, "out_dhidden", N * D), (out_dweight, "out_dweight", V * D),
                           (out_dbias, "out_dbias", V)):
            if t is not None:
                _vector(t, name, dtype, n, dev)
        workspace, ws_bytes = _head_workspace(workspace, linear_workspace_bytes(N, V, D, dt, aligned, True), dev)
        st = library().arcs_linear_backward(_ptr(hidden), hs, _ptr(weight), ws, dt, N, V, D, act, softcap, _ptr(pre),
                                            _ptr(grad_out), gdt, gs, _ptr(out_dhidden), _ptr(out_dweight),
                                            _ptr(out_dbias), _ptr(workspace), ws_bytes, _head_stream(stream, dev))
    if st != OK:
        raise ArcsError(st, "arcs_linear_backward")
    if stream is not None:
        _head_used(stream, dev, (hidden, weight, grad_out, pre, workspace), (out_dhidden, out_dweight, out_dbias))
    return out_dhidden, out_dweight, out_dbias


# --------------------------------------------------------------------------
# logits before sampling
# --------------------------------------------------------------------------
def _lists(ids, offsets, name: str, B: int, dev):
    """CSR lists of a batch: int32 ids and int64 [B + 1] offsets."""
    torch = _torch()
    if ids.dtype != torch.int32 or ids.device != dev or not ids.is_contiguous():
        raise ValueError(f"{name}_ids must be a contiguous int32 tensor on {dev}")
    _vector(offsets, f"{name}_offsets", torch.int64, B + 1, dev)


def adjust_logits(logits, params=None, hist_ids=None, hist_offsets=None, bias_ids=None, bias_values=None,
                  bias_offsets=None, mask=None, mask_rows=None, out=None, out_dtype=None, out_status=None, stream=None):
    """arcs_adjust_logits: [B, V] logits with history penalties, biases and grammar masks
    applied, ready for argmax, sample and top_logprobs (sample then takes the same
    ``params`` and no history).

    ``params`` sampling records (params_to_device), needed with a history; ``bias_ids`` int32,
    ``bias_values`` float32 and ``bias_offsets`` int64 [B + 1]; ``mask`` int32 or uint32
    [masks, >= ceil(V / 32)], bit v % 32 of word v / 32 set where token v is allowed;
    ``mask_rows`` int32 [B], the mask of each row or -1, or None: row b has mask b.
    ``out=logits`` works in place; None: a new tensor of ``out_dtype`` (the logits' type).
    ``out_status`` int32 [B] takes the rows' codes (ROW_NOTHING_ALLOWED among them).
    """
    torch = _torch()
    B, V, stride = _check_logits(logits)
    dev = logits.device
    dt = _dtype_code(logits)
    stride = V if B == 1 else stride
    if params is not None:
        _vector(params, "params", torch.uint8, 32 * B, dev)
    if (hist_ids is None) != (hist_offsets is None):
        raise ValueError("hist_ids and hist_offsets go together")
    if hist_ids is not None:
        if params is None:
            raise ValueError("a history needs params")
        _lists(hist_ids, hist_offsets, "hist", B, dev)
    if (bias_ids is None) != (bias_values is None) or (bias_ids is None) != (bias_offsets is None):
        raise ValueError("bias_ids, bias_values and bias_offsets go together")
    if bias_ids is not None:
        _lists(bias_ids, bias_offsets, "bias", B, dev)
        _vector(bias_values, "bias_values", torch.float32, bias_ids.numel(), dev)
    masks = mask_stride = 0
    if mask is not None:
        if mask.dim() != 2 or mask.element_size() != 4 or mask.dtype.is_floating_point or mask.device != dev:
            raise ValueError(f"mask must be an int32 matrix of words on {dev}")
        if mask.stride(1) != 1 and mask.shape[1] > 1:
            raise ValueError("mask rows must be contiguous (stride(1) == 1)")
        if mask.shape[1] < (V + 31) // 32:
            raise ValueError("mask rows must have a bit for every token")
        masks, mask_stride = mask.shape[0], mask.shape[1] if mask.shape[0] == 1 else mask.stride(0)
    if mask_rows is not None:
        if mask is None:
            raise ValueError("mask_rows needs a mask")
        _vector(mask_rows, "mask_rows", torch.int32, B, dev)
    with _work_on(dev, stream):
        if out is None:
            out = torch.empty((B, V), dtype=logits.dtype if out_dtype is None else out_dtype, device=dev)
            os_ = V
        else:
            if out_dtype is not None and out.dtype != out_dtype:
                raise ValueError("out is not of out_dtype")
            os_ = _matrix(out, "out", out.dtype, B, V, dev)
        odt = _dtype_code_of(out, "out")
        if out_status is not None:
            _vector(out_status, "out_status", torch.int32, B, dev)
        st = library().arcs_adjust_logits(_ptr(logits), dt, B, V, stride, _ptr(params), _list_ptr(hist_ids),
                                          _ptr(hist_offsets), _list_ptr(bias_ids), _list_ptr(bias_values),
                                          _ptr(bias_offsets), _list_ptr(mask), masks, mask_stride, _ptr(mask_rows),
                                          _ptr(out), odt, os_, _ptr(out_status), _head_stream(stream, dev))
    if st != OK:
        raise ArcsError(st, "arcs_adjust_logits")
    if stream is not None:
        _head_used(stream, dev, (logits, params, hist_ids, hist_offsets, bias_ids, bias_values, bias_offsets, mask,
                                 mask_rows), (out, out_status))
    return out


# --------------------------------------------------------------------------
# the gradients' norm and clipping
# --------------------------------------------------------------------------
class TensorList:
    """A list of gradients for gradient_norm and clip_gradients: its plan on the device,
    made once (that copy is synchronous) and good as long as the tensors stay where they are.

    ``tensors`` bfloat16 or float32, contiguous, on one device, of any shape; ``outs`` a
    tensor of as many elements for each, where clip_gradients writes, or None: in place.  The
    list keeps the tensors alive, and its plan: a captured graph that holds a call needs the list
    as long as it is replayed.  Memory that overlaps (the same tensor twice, say) is refused.
    Making a list takes the host longer than a call (86 us for 12 tensors, 4.8 ms for 1,500): it is
    for gradients that are written to the same memory in every step.
    """

    def __init__(self, tensors, outs=None):
        torch = _torch()
        self.tensors = list(tensors)
        self.outs = self.tensors if outs is None else list(outs)
        if len(self.outs) != len(self.tensors):
            raise ValueError("outs must have a tensor for each of tensors")
        if not self.tensors:
            raise ValueError("a list of gradients needs a tensor")
        self.device = self.tensors[0].device
        for t, o in zip(self.tensors, self.outs):
            for x in (t, o):
                if not x.is_cuda or x.device != self.device or not x.is_contiguous():
                    raise ValueError(f"gradients and outs must be contiguous device tensors on {self.device}")
            if o.numel() != t.numel():
                raise ValueError("each out must have as many elements as its gradient")
        records = np.zeros(len(self.tensors), TENSOR_DTYPE)
        records["data"] = [t.data_ptr() for t in self.tensors]
        records["out"] = [o.data_ptr() for o in self.outs]
        records["count"] = [t.numel() for t in self.tensors]
        records["dtype"] = [_dtype_code_of(t, "a gradient") for t in self.tensors]
        records["out_dtype"] = [_dtype_code_of(o, "an out") for o in self.outs]
        self._refuse_overlaps(records)
        n = len(records)
        size = int(library().arcs_gradient_plan_bytes(records.ctypes.data, n))
        plan = np.zeros(size, np.uint8)
        st = library().arcs_gradient_plan(records.ctypes.data, n, plan.ctypes.data, size)
        if st != OK:
            raise ArcsError(st, "arcs_gradient_plan")
        self.plan = torch.from_numpy(plan).to(self.device)
        self.plan_stream = _head_stream(None, self.device)  # whose memory it is
        self.plan_bytes = size
        self.workspace_bytes = int(library().arcs_gradient_workspace_bytes(size))

    @staticmethod
    def _refuse_overlaps(records):
        """No two gradients and no two outs may share memory, and an out only with its own gradient,
        whole."""
        size = {DTYPE_BF16: 2, DTYPE_F32: 4}
        ranges = set()
        for r in records:
            if r["count"] > 0:
                data = (int(r["data"]), int(r["data"]) + int(r["count"]) * size[int(r["dtype"])])
                out = (int(r["out"]), int(r["out"]) + int(r["count"]) * size[int(r["out_dtype"])])
                for at in {data, out}:
                    if at in ranges:
                        raise ValueError("gradients and outs must not overlap")
                    ranges.add(at)
        last = 0
        for lo, hi in sorted(ranges):
            if lo < last:
                raise ValueError("gradients and outs must not overlap")
            last = hi


def _norm_call(tensors, out_norm, workspace, stream, name, *more):
    torch = _torch()
    dev = tensors.device
    with _work_on(dev, stream):
        if out_norm is None:
            out_norm = torch.empty(1, dtype=torch.float32, device=dev)
        else:
            _vector(out_norm, "out_norm", torch.float32, 1, dev)
        workspace, ws_bytes = _head_workspace(workspace, tensors.workspace_bytes, dev)
        on = _head_stream(stream, dev)
        st = getattr(library(), name)(_list_ptr(tensors.plan), tensors.plan_bytes, *more, _ptr(out_norm),
                                      _ptr(workspace), ws_bytes, on)
    if st != OK:
        raise ArcsError(st, name)
    if stream is not None:
        _head_used(stream, dev, (tensors.plan, workspace, *tensors.tensors), (out_norm, *tensors.outs))
    elif on != tensors.plan_stream:
        # the plan is the list's own: a list dropped right after the call must not give it back yet
        _used_on(torch.cuda.current_stream(dev), tensors.plan)
    return out_norm


def gradient_norm(tensors: TensorList, out_norm=None, workspace=None, stream=None):
    """arcs_gradient_norm: sqrt(sum of all squares) of the list's gradients, float32 [1] on the device."""
    return _norm_call(tensors, out_norm, workspace, stream, "arcs_gradient_norm")


def clip_gradients(tensors: TensorList, max_norm: float, out_norm=None, workspace=None, stream=None):
    """arcs_clip_gradients: scales the list's gradients by max_norm / norm where their norm is
    above max_norm (and finite), to the list's outs or in place; returns the norm before, float32 [1]."""
    return _norm_call(tensors, out_norm, workspace, stream, "arcs_clip_gradients", float(max_norm))
