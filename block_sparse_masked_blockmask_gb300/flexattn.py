"""Thin Python binding of the C-ABI in include/flexattn.h.

Argument marshalling only: torch tensors supply device memory and
torch.cuda streams supply the cudaStream_t; every step of the path runs in
the CUDA kernels of libflexattn.so.  There is no fallback: if the library is
missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import struct
import threading

import torch

from . import _build

FLEX_OK = 0
FLEX_ERR_INVALID_ARG = -1
FLEX_ERR_UNSUPPORTED = -2
FLEX_ERR_SHAPE = -3
FLEX_ERR_ALIGNMENT = -4
FLEX_ERR_CUDA = -5
FLEX_ERR_DEVICE_TIMEOUT = -6

FLEX_MASK_CAUSAL = 0
FLEX_MASK_SLIDING_WINDOW = 1
FLEX_MASK_CAUSAL_PREFIX = 2
FLEX_MASK_DOCUMENT = 3
FLEX_MASK_ALL = 4
FLEX_MASK_WINDOW_SINKS = 5

FLEX_SCORE_IDENTITY = 0
FLEX_SCORE_SOFTCAP = 1
FLEX_SCORE_ALIBI = 2

FLEX_DTYPE_BF16 = 0
FLEX_DTYPE_FP32 = 1
FLEX_DTYPE_E4M3 = 2
FLEX_DTYPE_INT4 = 3

FLEX_ROPE_HALF = 0
FLEX_ROPE_INTERLEAVED = 1

FLEX_ROPE_SCALE_NONE = 0
FLEX_ROPE_SCALE_LINEAR = 1
FLEX_ROPE_SCALE_BASE = 2
FLEX_ROPE_SCALE_PARTS = 3

EXPORTED = ("flex_block_mask_sizes", "flex_block_mask_sizes_qkv", "flex_block_mask_create", "flex_block_mask_create_qkv",
            "flex_block_mask_transpose", "flex_attention_fwd",
            "flex_attention_fwd_opts", "flex_attention_bwd", "flex_attention_fwd_noalloc", "flex_attention_fwd_host", "flex_device_status",
            "flex_selftest_wait_timeout", "flex_status_string", "flex_rope_frequencies", "flex_rope_fwd", "flex_rope_bwd",
            "flex_kv_cache_append", "flex_kv_cache_append_packed", "flex_kv_cache_read",
            "flex_kv_cache_attention", "flex_kv_cache_attention_workspace",
            "flex_packed_plan_bytes", "flex_packed_plan_create", "flex_attention_packed_fwd")


class FlexError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {flex_status_string(code)} ({code})")


class flex_mask_params(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("prefix", ctypes.c_int32), ("doc_ids", ctypes.c_void_p)]


class flex_block_mask(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("q_len", ctypes.c_int32),
                ("kv_len", ctypes.c_int32), ("q_block", ctypes.c_int32), ("kv_block", ctypes.c_int32),
                ("nqb", ctypes.c_int32), ("nkvb", ctypes.c_int32), ("mask_kind", ctypes.c_int32),
                ("params", flex_mask_params),
                ("kv_num_blocks", ctypes.c_void_p), ("kv_indices", ctypes.c_void_p),
                ("full_kv_num_blocks", ctypes.c_void_p), ("full_kv_indices", ctypes.c_void_p)]


class flex_tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class flex_block_mask_q(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("q_len", ctypes.c_int32),
                ("kv_len", ctypes.c_int32), ("q_block", ctypes.c_int32), ("kv_block", ctypes.c_int32),
                ("nqb", ctypes.c_int32), ("nkvb", ctypes.c_int32),
                ("q_num_blocks", ctypes.c_void_p), ("q_indices", ctypes.c_void_p),
                ("full_q_num_blocks", ctypes.c_void_p), ("full_q_indices", ctypes.c_void_p)]


class flex_kernel_options(ctypes.Structure):
    _fields_ = [("prescale_qk", ctypes.c_int32), ("rows_guaranteed_safe", ctypes.c_int32),
                ("max_scores", ctypes.c_void_p)]


class flex_rope_params(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("attention_scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class flex_kv_cache(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("H", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("D", ctypes.c_int32), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class flex_packed_plan(ctypes.Structure):
    _fields_ = [("sequences", ctypes.c_int32), ("total_q", ctypes.c_int32), ("total_k", ctypes.c_int32),
                ("Hq", ctypes.c_int32), ("Hk", ctypes.c_int32), ("mask_kind", ctypes.c_int32),
                ("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("entries", ctypes.c_void_p)]


class flex_device_buffers(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("doc_ids", ctypes.c_void_p), ("kv_num_blocks", ctypes.c_void_p),
                ("kv_indices", ctypes.c_void_p), ("full_kv_num_blocks", ctypes.c_void_p),
                ("full_kv_indices", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIBRARY


def load_library():
    """Load libflexattn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; "
                                   "g.build()')")
            lib = ctypes.CDLL(path)
            i32, i64p, vp = ctypes.c_int32, ctypes.POINTER(ctypes.c_int64), ctypes.c_void_p
            lib.flex_block_mask_sizes.argtypes = [i32, i32, i32, i32, i32, i64p, i64p]
            lib.flex_block_mask_sizes.restype = ctypes.c_int
            lib.flex_block_mask_sizes_qkv.argtypes = [i32, i32, i32, i32, i32, i32, i64p, i64p]
            lib.flex_block_mask_sizes_qkv.restype = ctypes.c_int
            lib.flex_block_mask_create.argtypes = [i32, ctypes.POINTER(flex_mask_params), i32, i32, i32, i32, i32,
                                                   ctypes.POINTER(flex_block_mask), vp]
            lib.flex_block_mask_create.restype = ctypes.c_int
            lib.flex_block_mask_create_qkv.argtypes = [i32, ctypes.POINTER(flex_mask_params), i32, i32, i32, i32,
                                                       i32, i32, ctypes.POINTER(flex_block_mask), vp]
            lib.flex_block_mask_create_qkv.restype = ctypes.c_int
            tp = vp  # const flex_tensor *: packed bytes (_tensor) or a reference to a flex_tensor
            lib.flex_attention_fwd.argtypes = [tp, tp, tp, ctypes.POINTER(flex_block_mask), i32, ctypes.c_float,
                                               ctypes.c_float, vp, vp, vp]
            lib.flex_attention_fwd.restype = ctypes.c_int
            lib.flex_attention_fwd_opts.argtypes = [tp, tp, tp, ctypes.POINTER(flex_block_mask), i32,
                                                    ctypes.c_float, ctypes.c_float, vp, vp,
                                                    ctypes.POINTER(flex_kernel_options), vp]
            lib.flex_attention_fwd_opts.restype = ctypes.c_int
            lib.flex_block_mask_transpose.argtypes = [ctypes.POINTER(flex_block_mask),
                                                      ctypes.POINTER(flex_block_mask_q), vp]
            lib.flex_block_mask_transpose.restype = ctypes.c_int
            lib.flex_attention_bwd.argtypes = [tp, tp, tp, vp, vp, vp, ctypes.POINTER(flex_block_mask),
                                               ctypes.POINTER(flex_block_mask_q), i32, ctypes.c_float,
                                               ctypes.c_float, vp, vp, vp, vp, vp]
            lib.flex_attention_bwd.restype = ctypes.c_int
            lib.flex_attention_fwd_noalloc.argtypes = [tp, tp, tp, ctypes.POINTER(flex_block_mask), i32,
                                                       ctypes.c_float, ctypes.c_float, vp, vp, vp,
                                                       ctypes.POINTER(ctypes.POINTER(ctypes.c_int))]
            lib.flex_attention_fwd_noalloc.restype = ctypes.c_int
            lib.flex_attention_fwd_host.argtypes = [tp, tp, tp, i32, ctypes.POINTER(flex_mask_params), i32,
                                                    ctypes.c_float, ctypes.c_float, vp, vp,
                                                    ctypes.POINTER(flex_device_buffers), i32, vp]
            lib.flex_attention_fwd_host.restype = ctypes.c_int
            lib.flex_device_status.argtypes = [vp]
            lib.flex_device_status.restype = ctypes.c_int
            lib.flex_selftest_wait_timeout.argtypes = [ctypes.c_uint32, vp]
            lib.flex_selftest_wait_timeout.restype = ctypes.c_int
            f64 = ctypes.c_double
            lib.flex_rope_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, ctypes.POINTER(f64)]
            lib.flex_rope_frequencies.restype = ctypes.c_int
            for f in (lib.flex_rope_fwd, lib.flex_rope_bwd):
                f.argtypes = [tp, tp, vp, vp, tp, tp, vp]  # the third: packed bytes (_rope_params) or a reference
                f.restype = ctypes.c_int
            cp = ctypes.POINTER(flex_kv_cache)
            lib.flex_kv_cache_append.argtypes = [cp, tp, tp, vp, i32, vp, vp, vp, vp]
            lib.flex_kv_cache_append.restype = ctypes.c_int
            lib.flex_kv_cache_append_packed.argtypes = [cp, tp, tp, vp, i32, vp, i32, vp, vp, vp]
            lib.flex_kv_cache_append_packed.restype = ctypes.c_int
            lib.flex_kv_cache_read.argtypes = [cp, vp, i32, vp, i32, tp, tp, vp]
            lib.flex_kv_cache_read.restype = ctypes.c_int
            lib.flex_kv_cache_attention.argtypes = [tp, cp, vp, i32, vp, i32, ctypes.POINTER(flex_mask_params), i32,
                                                    ctypes.c_float, ctypes.c_float, vp, vp, vp, ctypes.c_int64, vp]
            lib.flex_kv_cache_attention.restype = ctypes.c_int
            lib.flex_kv_cache_attention_workspace.argtypes = [tp, cp, i32, i32, ctypes.POINTER(flex_mask_params), i64p]
            lib.flex_kv_cache_attention_workspace.restype = ctypes.c_int
            pp = ctypes.POINTER(flex_packed_plan)
            lib.flex_packed_plan_bytes.argtypes = [i32, i32, i32, i32, i64p]
            lib.flex_packed_plan_bytes.restype = ctypes.c_int
            lib.flex_packed_plan_create.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32,
                                                    ctypes.POINTER(flex_mask_params), pp, vp]
            lib.flex_packed_plan_create.restype = ctypes.c_int
            lib.flex_attention_packed_fwd.argtypes = [tp, tp, tp, pp, i32, ctypes.c_float, ctypes.c_float, tp, vp, vp]
            lib.flex_attention_packed_fwd.restype = ctypes.c_int
            lib.flex_status_string.argtypes = [ctypes.c_int]
            lib.flex_status_string.restype = ctypes.c_char_p
            _lib = lib
    return _lib


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream, device) -> int:
    """The cudaStream_t of a stream (None: torch's current one on the device)."""
    if stream is None:
        if _current_raw_stream is not None and device.index is not None:  # a tenth of the public call's time
            return _current_raw_stream(device.index)
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on_stream(stream, device):
    """A context in which torch allocates and works on `stream` (None: nothing to enter)."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream_handle(stream, device), device)
    return torch.cuda.stream(stream)


def _empty(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """Memory for a call on `stream`, from that stream's pool: what the pool last lent it for lies before the
    call in the stream's order (None: torch's current stream)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on_stream(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_by_token(B: int, H: int, T: int, D: int, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """_empty for a [B, H, T, D] tensor with a token's heads next to each other (in one call of torch's: transposing
    one that is empty takes 4 us more)."""
    strides = (T * H * D, D, H * D, 1)
    if stream is None:
        return torch.empty_strided((B, H, T, D), strides, dtype=dtype, device=device)
    with _on_stream(stream, device):
        return torch.empty_strided((B, H, T, D), strides, dtype=dtype, device=device)


def _device_guard(device):
    """A context in which `device` is the current CUDA device (nothing to enter when it already is)."""
    return contextlib.nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(device, f, *args) -> int:
    """f(*args) with `device` (of an existing CUDA tensor) as the current device."""
    if _current_device() == device.index:
        return f(*args)
    with torch.cuda.device(device):
        return f(*args)


def flex_status_string(code: int) -> str:
    return load_library().flex_status_string(int(code)).decode()


def flex_block_mask_sizes(B: int, H: int, q_len: int, kv_len: int, block: int = 128,
                          kv_block: int | None = None) -> tuple[int, int]:
    """Element counts of the count and index tensors (Q_BLOCK = block, KV_BLOCK = kv_block or block)."""
    n_num, n_idx = ctypes.c_int64(), ctypes.c_int64()
    if kv_block is None:
        rc = load_library().flex_block_mask_sizes(B, H, q_len, kv_len, block, ctypes.byref(n_num),
                                                  ctypes.byref(n_idx))
    else:
        rc = load_library().flex_block_mask_sizes_qkv(B, H, q_len, kv_len, block, kv_block, ctypes.byref(n_num),
                                                      ctypes.byref(n_idx))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_block_mask_sizes")
    return n_num.value, n_idx.value


def _mask_params(mask_kind: int, window: int, prefix: int, sinks: int, doc_ids=None) -> flex_mask_params:
    """The C parameters of a mask kind (the count of sinks travels in `prefix`)."""
    if sinks and mask_kind != FLEX_MASK_WINDOW_SINKS:
        raise ValueError("sinks belong to FLEX_MASK_WINDOW_SINKS")
    return flex_mask_params(window, sinks if mask_kind == FLEX_MASK_WINDOW_SINKS else prefix,
                            doc_ids.data_ptr() if doc_ids is not None else None)


class BlockMask:
    """Device BlockMask: the C struct plus the torch tensors that own its buffers."""

    def __init__(self, struct: flex_block_mask, tensors: dict, doc_ids):
        self.struct = struct
        self.kv_num_blocks = tensors["kv_num_blocks"]
        self.kv_indices = tensors["kv_indices"]
        self.full_kv_num_blocks = tensors["full_kv_num_blocks"]
        self.full_kv_indices = tensors["full_kv_indices"]
        self.doc_ids = doc_ids  # keeps the document ids alive while the mask is in use

    def as_numpy(self) -> dict:
        return {k: getattr(self, k).cpu().numpy() for k in
                ("kv_num_blocks", "kv_indices", "full_kv_num_blocks", "full_kv_indices")}


class BlockMaskQ:
    """Device q side of a BlockMask: the C struct plus the torch tensors that own its buffers."""

    KEYS = ("q_num_blocks", "q_indices", "full_q_num_blocks", "full_q_indices")

    def __init__(self, struct: flex_block_mask_q, tensors: dict):
        self.struct = struct
        for key in self.KEYS:
            setattr(self, key, tensors[key])

    def as_numpy(self) -> dict:
        return {k: getattr(self, k).cpu().numpy() for k in self.KEYS}


def flex_block_mask_transpose(block_mask: BlockMask, stream=None) -> BlockMaskQ:
    """The q side of a BlockMask, from `stream`'s pool (asynchronous on `stream`)."""
    s = block_mask.struct
    device = block_mask.kv_num_blocks.device
    t = {
        "q_num_blocks": _empty((s.B, s.H, s.nkvb), torch.int32, device, stream),
        "q_indices": _empty((s.B, s.H, s.nkvb, s.nqb), torch.int32, device, stream),
        "full_q_num_blocks": _empty((s.B, s.H, s.nkvb), torch.int32, device, stream),
        "full_q_indices": _empty((s.B, s.H, s.nkvb, s.nqb), torch.int32, device, stream),
    }
    bq = flex_block_mask_q()
    for key in BlockMaskQ.KEYS:
        setattr(bq, key, t[key].data_ptr())
    with _device_guard(device):
        rc = load_library().flex_block_mask_transpose(ctypes.byref(s), ctypes.byref(bq),
                                                      _stream_handle(stream, device))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_block_mask_transpose")
    return BlockMaskQ(bq, t)


def flex_block_mask_create(mask_kind: int, B: int, H: int, q_len: int, kv_len: int, block: int = 128,
                           window: int = 0, prefix: int = 0, doc_ids: torch.Tensor | None = None,
                           device=None, stream=None, kv_block: int | None = None, sinks: int = 0) -> BlockMask:
    """Build a BlockMask on the device, in memory of `stream`'s pool (asynchronous on `stream`).

    Tiles are block (Q_BLOCK) rows by kv_block (KV_BLOCK; default: block)
    columns; flex_block_mask_create_qkv is called when kv_block is given.
    FLEX_MASK_WINDOW_SINKS takes `window` and `sinks` (first tokens that stay
    visible).
    """
    device = torch.device(device) if device is not None else (
        doc_ids.device if doc_ids is not None else torch.device("cuda", torch.cuda.current_device()))
    n_num, n_idx = flex_block_mask_sizes(B, H, q_len, kv_len, block, kv_block)
    kvb = block if kv_block is None else kv_block
    nqb, nkvb = -(-q_len // block), -(-kv_len // kvb)  # a tail tile may reach past a length
    t = {
        "kv_num_blocks": _empty((B, H, nqb), torch.int32, device, stream),
        "kv_indices": _empty((B, H, nqb, nkvb), torch.int32, device, stream),
        "full_kv_num_blocks": _empty((B, H, nqb), torch.int32, device, stream),
        "full_kv_indices": _empty((B, H, nqb, nkvb), torch.int32, device, stream),
    }
    assert t["kv_num_blocks"].numel() == n_num and t["kv_indices"].numel() == n_idx
    if doc_ids is not None:
        with _on_stream(stream, device):
            doc_ids = doc_ids.to(device=device, dtype=torch.int32).contiguous()
    params = _mask_params(mask_kind, window, prefix, sinks, doc_ids)
    bm = flex_block_mask()
    bm.kv_num_blocks = t["kv_num_blocks"].data_ptr()
    bm.kv_indices = t["kv_indices"].data_ptr()
    bm.full_kv_num_blocks = t["full_kv_num_blocks"].data_ptr()
    bm.full_kv_indices = t["full_kv_indices"].data_ptr()
    with _device_guard(device):
        if kv_block is None:
            rc = load_library().flex_block_mask_create(mask_kind, ctypes.byref(params), B, H, q_len, kv_len, block,
                                                       ctypes.byref(bm), _stream_handle(stream, device))
        else:
            rc = load_library().flex_block_mask_create_qkv(mask_kind, ctypes.byref(params), B, H, q_len, kv_len,
                                                           block, kv_block, ctypes.byref(bm),
                                                           _stream_handle(stream, device))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_block_mask_create")
    return BlockMask(bm, t, doc_ids)


_DTYPES = {torch.bfloat16: FLEX_DTYPE_BF16, torch.float32: FLEX_DTYPE_FP32}


_pack_tensor = struct.Struct("=Qii8q").pack  # a flex_tensor's fields (a third of the time of filling the Structure)
assert struct.calcsize("=Qii8q") == ctypes.sizeof(flex_tensor)


def _tensor(x: torch.Tensor) -> bytes:
    """The flex_tensor of a [B, H, S, D] tensor, as the bytes a call takes in its place."""
    shape = x.shape
    if len(shape) != 4:
        raise ValueError("expected a [B, H, S, D] tensor")
    dtype = _DTYPES.get(x.dtype)
    if dtype is None:
        raise ValueError(f"unsupported dtype {x.dtype}")
    return _pack_tensor(x.data_ptr(), dtype, 0, *shape, *x.stride())


def flex_attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_mask: BlockMask,
                       score_kind: int = FLEX_SCORE_IDENTITY, score_param: float = 0.0,
                       scale: float | None = None, out: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None, stream=None):
    """Block-sparse attention forward; returns (out, lse), allocated from `stream`'s pool where not given.
    Asynchronous on `stream`."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    B, H, Sq, D = q.shape
    if out is None:
        out = _empty((B, H, Sq, D), q.dtype, q.device, stream)
    if lse is None:
        lse = _empty((B, H, Sq), torch.float32, q.device, stream)
    if not out.is_contiguous() or not lse.is_contiguous() or lse.dtype != torch.float32:
        raise ValueError("out and lse must be contiguous; lse float32")
    rc = _call(q.device, load_library().flex_attention_fwd, _tensor(q), _tensor(k), _tensor(v),
               ctypes.byref(block_mask.struct), score_kind, float(score_param), float(scale), out.data_ptr(),
               lse.data_ptr(), _stream_handle(stream, q.device))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_attention_fwd")
    return out, lse


def flex_attention_fwd_opts(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_mask: BlockMask,
                            score_kind: int = FLEX_SCORE_IDENTITY, score_param: float = 0.0,
                            scale: float | None = None, out: torch.Tensor | None = None,
                            lse: torch.Tensor | None = None, prescale_qk: bool = False,
                            rows_guaranteed_safe: bool = False, output_max: bool = False,
                            max_scores: torch.Tensor | None = None, stream=None):
    """flex_attention_fwd with the op's kernel options; returns (out, lse, max_scores).

    max_scores (float32 [B, H, Sq]) is allocated when output_max is set and
    none is given; it is None when OUTPUT_MAX is off.  What is allocated comes
    from `stream`'s pool.
    """
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    B, H, Sq, D = q.shape
    if out is None:
        out = _empty((B, H, Sq, D), q.dtype, q.device, stream)
    if lse is None:
        lse = _empty((B, H, Sq), torch.float32, q.device, stream)
    if max_scores is None and output_max:
        max_scores = _empty((B, H, Sq), torch.float32, q.device, stream)
    if not out.is_contiguous() or not lse.is_contiguous() or lse.dtype != torch.float32:
        raise ValueError("out and lse must be contiguous; lse float32")
    if max_scores is not None and (not max_scores.is_contiguous() or max_scores.dtype != torch.float32
                                   or max_scores.shape != (B, H, Sq)):
        raise ValueError("max_scores must be a contiguous float32 [B, H, q_len] tensor")
    opts = flex_kernel_options(int(bool(prescale_qk)), int(bool(rows_guaranteed_safe)),
                               None if max_scores is None else max_scores.data_ptr())
    tq, tk, tv = _tensor(q), _tensor(k), _tensor(v)
    with _device_guard(q.device):
        rc = load_library().flex_attention_fwd_opts(tq, tk, tv,
                                                    ctypes.byref(block_mask.struct), score_kind,
                                                    float(score_param), float(scale),
                                                    out.data_ptr(),
                                                    lse.data_ptr(), ctypes.byref(opts),
                                                    _stream_handle(stream, q.device))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_attention_fwd_opts")
    return out, lse, max_scores


def flex_attention_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
                       dout: torch.Tensor, block_mask: BlockMask, block_mask_q: BlockMaskQ,
                       score_kind: int = FLEX_SCORE_IDENTITY, score_param: float = 0.0,
                       scale: float | None = None, dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                       dv: torch.Tensor | None = None, delta: torch.Tensor | None = None, stream=None):
    """Gradients (dq, dk, dv) of sum(dout * out); asynchronous on `stream`, from whose pool they and delta are
    allocated where not given."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    B, H, Sq, D = q.shape
    Skv = k.shape[2]
    dq = _empty((B, H, Sq, D), q.dtype, q.device, stream) if dq is None else dq
    dk = _empty((B, H, Skv, D), q.dtype, q.device, stream) if dk is None else dk
    dv = _empty((B, H, Skv, D), q.dtype, q.device, stream) if dv is None else dv
    delta = _empty((B, H, Sq), torch.float32, q.device, stream) if delta is None else delta
    for name, t in (("out", out), ("dout", dout), ("dq", dq), ("dk", dk), ("dv", dv)):
        if not t.is_contiguous() or t.dtype != q.dtype:
            raise ValueError(f"{name} must be contiguous in q's dtype")
    if not lse.is_contiguous() or lse.dtype != torch.float32 or not delta.is_contiguous():
        raise ValueError("lse and delta must be contiguous float32")
    tq, tk, tv = _tensor(q), _tensor(k), _tensor(v)
    with _device_guard(q.device):
        rc = load_library().flex_attention_bwd(tq, tk, tv,
                                               out.data_ptr(), lse.data_ptr(),
                                               dout.data_ptr(), ctypes.byref(block_mask.struct),
                                               ctypes.byref(block_mask_q.struct), score_kind, float(score_param),
                                               float(scale), dq.data_ptr(),
                                               dk.data_ptr(), dv.data_ptr(),
                                               delta.data_ptr(), _stream_handle(stream, q.device))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_attention_bwd")
    return dq, dk, dv


def flex_attention_fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_mask: BlockMask,
                               out: torch.Tensor, lse: torch.Tensor, score_kind: int = FLEX_SCORE_IDENTITY,
                               score_param: float = 0.0, scale: float | None = None, stream=None):
    """flex_attention_fwd into caller-provided out/lse without any device allocation by the library.

    Returns the device address (int) of the status word the call uses; after the
    stream finishes, a nonzero word means a kernel gave up on a wait.
    """
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    tq, tk, tv = _tensor(q), _tensor(k), _tensor(v)
    status = ctypes.POINTER(ctypes.c_int)()
    with _device_guard(q.device):
        rc = load_library().flex_attention_fwd_noalloc(tq, tk, tv,
                                                       ctypes.byref(block_mask.struct), score_kind,
                                                       float(score_param), float(scale),
                                                       out.data_ptr(),
                                                       lse.data_ptr(),
                                                       _stream_handle(stream, q.device), ctypes.byref(status))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_attention_fwd_noalloc")
    return ctypes.cast(status, ctypes.c_void_p).value


class DeviceBuffers:
    """Device working memory of flex_attention_fwd_host, allocated (and owned) through torch."""

    def __init__(self, B: int, H: int, q_len: int, kv_len: int, D: int, dtype: torch.dtype,
                 document: bool = False, device=None):
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.q = torch.empty((B, H, q_len, D), dtype=dtype, device=device)
        self.k = torch.empty((B, H, kv_len, D), dtype=dtype, device=device)
        self.v = torch.empty((B, H, kv_len, D), dtype=dtype, device=device)
        self.out = torch.empty((B, H, q_len, D), dtype=dtype, device=device)
        self.lse = torch.empty((B, H, q_len), dtype=torch.float32, device=device)
        self.doc_ids = torch.empty((B, q_len), dtype=torch.int32, device=device) if document else None
        nqb, nkvb = -(-q_len // 128), -(-kv_len // 128)
        self.kv_num_blocks = torch.empty((B, H, nqb), dtype=torch.int32, device=device)
        self.kv_indices = torch.empty((B, H, nqb, nkvb), dtype=torch.int32, device=device)
        self.full_kv_num_blocks = torch.empty((B, H, nqb), dtype=torch.int32, device=device)
        self.full_kv_indices = torch.empty((B, H, nqb, nkvb), dtype=torch.int32, device=device)
        self.device = device

    def struct(self) -> flex_device_buffers:
        d = flex_device_buffers()
        for name in ("q", "k", "v", "out", "lse", "kv_num_blocks", "kv_indices", "full_kv_num_blocks",
                     "full_kv_indices"):
            setattr(d, name, getattr(self, name).data_ptr())
        d.doc_ids = self.doc_ids.data_ptr() if self.doc_ids is not None else None
        return d


def flex_attention_fwd_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, buffers: DeviceBuffers,
                            mask_kind: int, out: torch.Tensor, lse: torch.Tensor, window: int = 0, prefix: int = 0,
                            doc_ids: torch.Tensor | None = None, score_kind: int = FLEX_SCORE_IDENTITY,
                            score_param: float = 0.0, scale: float | None = None, chunks: int = 8,
                            stream=None, sinks: int = 0) -> None:
    """BlockMask build + attention from host q, k, v into host out, lse (see include/flexattn.h).

    q, k, v, out, lse (and doc_ids) are contiguous CPU tensors, pinned for the
    copies to overlap; `buffers` is the device working memory.  Asynchronous on
    `stream`: the host outputs are valid once the stream has passed the call.
    """
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    for t in (q, k, v, out, lse) + ((doc_ids,) if doc_ids is not None else ()):
        if t.device.type != "cpu" or not t.is_contiguous():
            raise ValueError("host tensors must be contiguous CPU tensors")
    if lse.dtype != torch.float32 or out.dtype != q.dtype:
        raise ValueError("out has the inputs' dtype, lse is float32")
    if doc_ids is not None and doc_ids.dtype != torch.int32:
        raise ValueError("doc_ids must be int32")
    tq, tk, tv = _tensor(q), _tensor(k), _tensor(v)
    params = _mask_params(mask_kind, window, prefix, sinks, doc_ids)
    dev = buffers.struct()
    with torch.cuda.device(buffers.device):
        rc = load_library().flex_attention_fwd_host(tq, tk, tv, mask_kind,
                                                    ctypes.byref(params), score_kind, float(score_param),
                                                    float(scale), out.data_ptr(),
                                                    lse.data_ptr(), ctypes.byref(dev), int(chunks),
                                                    _stream_handle(stream, buffers.device))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_attention_fwd_host")


def flex_rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: int = FLEX_ROPE_SCALE_NONE,
                          factor: float = 1.0, original_len: float = 0.0, low_turns: float = 1.0,
                          high_turns: float = 32.0, device=None) -> torch.Tensor:
    """Frequencies of the rotation, float64 [rotary_dim / 2], on `device` (a plan a program makes once)."""
    host = torch.empty(max(rotary_dim // 2, 1), dtype=torch.float64)
    rc = load_library().flex_rope_frequencies(rotary_dim, base, scaling, factor, original_len, low_turns, high_turns,
                                              ctypes.cast(host.data_ptr(), ctypes.POINTER(ctypes.c_double)))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_rope_frequencies")
    return host.to(torch.device("cuda", torch.cuda.current_device()) if device is None else device)


def _device_array(x: torch.Tensor | None, name: str, dtype: torch.dtype, device, shape) -> int | None:
    """The address of a contiguous tensor of this type, shape and device (None stays None)."""
    if x is None:
        return None
    if x.dtype != dtype or x.shape != shape or not x.is_contiguous() or x.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {device}")
    return x.data_ptr()


_pack_rope = struct.Struct("=Qiifi").pack
assert struct.calcsize("=Qiifi") == ctypes.sizeof(flex_rope_params)


def _rope_params(inv_freq: torch.Tensor, layout: int, attention_scale: float, device) -> bytes:
    """A flex_rope_params as the bytes a call takes in its place."""
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a float64 [rotary_dim / 2] tensor")
    n = inv_freq.shape[0]
    return _pack_rope(_device_array(inv_freq, "inv_freq", torch.float64, device, (n,)), 2 * n, layout,
                      attention_scale, 0)


def _rope(name: str, q, k, inv_freq, positions, layout, attention_scale, q_out, k_out, stream):
    device = q.device
    tq, tk, ok = _tensor(q), None, None
    if k is not None:
        tk = _tensor(k)
    elif k_out is not None:
        raise ValueError("k_out without k")
    for x in (k, q_out, k_out):
        if x is not None and x.device != device:
            raise ValueError("q, k and their outputs must be on one device")
    params = _rope_params(inv_freq, layout, attention_scale, device)
    if positions is not None:
        positions = _device_array(positions, "positions", torch.int32, device, (q.shape[0], q.shape[2]))
    if q_out is None:
        q_out = _empty(q.shape, q.dtype, device, stream)
    if k is not None:
        if k_out is None:
            k_out = _empty(k.shape, k.dtype, device, stream)
        ok = _tensor(k_out)
    rc = _call(device, getattr(load_library(), name), tq, tk, params, positions, _tensor(q_out), ok,
               _stream_handle(stream, device))
    if rc != FLEX_OK:
        raise FlexError(rc, name)
    return q_out, k_out


def flex_rope_fwd(q: torch.Tensor, k: torch.Tensor | None, inv_freq: torch.Tensor,
                  positions: torch.Tensor | None = None, layout: int = FLEX_ROPE_HALF, attention_scale: float = 1.0,
                  q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """q [B, Hq, S, D] and k [B, Hk, S, D] (or None) turned by their positions; returns (q_out, k_out).

    positions: int32 [B, S] (default 0 .. S - 1).  The outputs may be the
    inputs; those not given are allocated from `stream`'s pool.  Asynchronous
    on `stream`.
    """
    return _rope("flex_rope_fwd", q, k, inv_freq, positions, layout, attention_scale, q_out, k_out, stream)


def flex_rope_bwd(dq: torch.Tensor, dk: torch.Tensor | None, inv_freq: torch.Tensor,
                  positions: torch.Tensor | None = None, layout: int = FLEX_ROPE_HALF, attention_scale: float = 1.0,
                  dq_out: torch.Tensor | None = None, dk_out: torch.Tensor | None = None, stream=None):
    """Gradients of flex_rope_fwd's inputs from those of its outputs; same arguments."""
    return _rope("flex_rope_bwd", dq, dk, inv_freq, positions, layout, attention_scale, dq_out, dk_out, stream)


_CACHE_DTYPES = {torch.bfloat16: FLEX_DTYPE_BF16, torch.float8_e4m3fn: FLEX_DTYPE_E4M3, torch.uint8: FLEX_DTYPE_INT4}


class KVCache:
    """Paged key/value cache: the C struct plus the torch tensors that own its memory.

    k, v: contiguous [num_pages, H, page_size, D], bfloat16 or float8_e4m3fn;
    the latter with k_scale, v_scale: contiguous float32 [num_pages, H].  Or
    uint8 [num_pages, H, page_size, D / 2], two 4-bit codes a byte, with
    k_scale bfloat16 [num_pages, H, page_size, D / 32] and v_scale bfloat16
    [num_pages, H, page_size] (the order of codes is in include/flexattn.h).
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        if k.dim() != 4 or k.dtype not in _CACHE_DTYPES:
            raise ValueError("k must be a bfloat16, float8_e4m3fn or uint8 [num_pages, H, page_size, D] tensor")
        dtype = _CACHE_DTYPES[k.dtype]
        scaled = dtype != FLEX_DTYPE_BF16
        if scaled != (k_scale is not None) or scaled != (v_scale is not None):
            raise ValueError("an e4m3 or 4-bit cache needs k_scale and v_scale, a bf16 cache takes none")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        n, h, page, d = k.shape
        scales = (torch.float32, (n, h), (n, h))
        if dtype == FLEX_DTYPE_INT4:
            d *= 2
            scales = (torch.bfloat16, (n, h, page, d // 32), (n, h, page))
        self.shape = (n, h, page, d)  # pages, heads, page size, head dim
        self.struct = flex_kv_cache(n, h, page, d, dtype, 0,
                                    _device_array(k, "k", k.dtype, k.device, k.shape),
                                    _device_array(v, "v", k.dtype, k.device, k.shape),
                                    _device_array(k_scale, "k_scale", scales[0], k.device, scales[1]),
                                    _device_array(v_scale, "v_scale", scales[0], k.device, scales[2]))
        self._ref = ctypes.byref(self.struct)


def flex_kv_cache_create(num_pages: int, H: int, D: int, page_size: int = 64,
                         dtype: torch.dtype = torch.float8_e4m3fn, device=None) -> KVCache:
    """A new cache of num_pages pages (uninitialised) on `device`; dtype torch.uint8 makes one of 4-bit codes."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    row = D // 2 if dtype == torch.uint8 else D
    k, v = (torch.empty((num_pages, H, page_size, row), dtype=dtype, device=device) for _ in range(2))
    if dtype == torch.uint8:
        return KVCache(k, v, torch.empty((num_pages, H, page_size, D // 32), dtype=torch.bfloat16, device=device),
                       torch.empty((num_pages, H, page_size), dtype=torch.bfloat16, device=device))
    if dtype != torch.float8_e4m3fn:
        return KVCache(k, v)
    return KVCache(k, v, *(torch.empty((num_pages, H), dtype=torch.float32, device=device) for _ in range(2)))


def flex_kv_cache_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor,
                         cache_lens: torch.Tensor, new_lens: torch.Tensor | None = None,
                         inv_freq: torch.Tensor | None = None, layout: int = FLEX_ROPE_HALF,
                         attention_scale: float = 1.0, stream=None) -> None:
    """Write k, v [B, H, S, D] behind each sequence's cache_lens[b] tokens (asynchronous on `stream`).

    page_table int32 [B, max_pages], cache_lens and new_lens int32 [B].  k is
    rotated by its positions when inv_freq is given.
    """
    device = cache.k.device
    if k.device != device or v.device != device:
        raise ValueError("k and v must be on the cache's device")
    if page_table.dim() != 2:
        raise ValueError("page_table must be an int32 [B, max_pages] tensor")
    tk, tv = _tensor(k), _tensor(v)
    B, max_pages = k.shape[0], page_table.shape[1]
    rc = _call(device, load_library().flex_kv_cache_append, cache._ref, tk, tv,
               _device_array(page_table, "page_table", torch.int32, device, (B, max_pages)), max_pages,
               _device_array(cache_lens, "cache_lens", torch.int32, device, (B,)),
               _device_array(new_lens, "new_lens", torch.int32, device, (B,)),
               None if inv_freq is None else _rope_params(inv_freq, layout, attention_scale, device),
               _stream_handle(stream, device))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_kv_cache_append")


def _starts(starts: torch.Tensor, device) -> tuple[int, int]:
    """The address of a [sequences + 1] array of packed sequences' first tokens, and how many sequences those are."""
    if starts.dim() != 1 or starts.shape[0] < 2:
        raise ValueError("starts must be an int32 [sequences + 1] tensor")
    return _device_array(starts, "starts", torch.int32, device, starts.shape), starts.shape[0] - 1


def flex_kv_cache_append_packed(cache: KVCache, k: torch.Tensor, v: torch.Tensor, starts: torch.Tensor,
                                page_table: torch.Tensor, cache_lens: torch.Tensor,
                                inv_freq: torch.Tensor | None = None, layout: int = FLEX_ROPE_HALF,
                                attention_scale: float = 1.0, stream=None) -> None:
    """flex_kv_cache_append of packed sequences: tokens starts[b] .. starts[b + 1] - 1 of k, v [1, H, T, D] go behind
    sequence b's cache_lens[b] tokens (asynchronous on `stream`).

    starts int32 [sequences + 1], ascending; page_table int32 [sequences, max_pages], cache_lens int32 [sequences].
    """
    device = cache.k.device
    if k.device != device or v.device != device:
        raise ValueError("k and v must be on the cache's device")
    if page_table.dim() != 2:
        raise ValueError("page_table must be an int32 [sequences, max_pages] tensor")
    at, B = _starts(starts, device)
    max_pages = page_table.shape[1]
    rc = _call(device, load_library().flex_kv_cache_append_packed, cache._ref, _tensor(k), _tensor(v), at, B,
               _device_array(page_table, "page_table", torch.int32, device, (B, max_pages)), max_pages,
               _device_array(cache_lens, "cache_lens", torch.int32, device, (B,)),
               None if inv_freq is None else _rope_params(inv_freq, layout, attention_scale, device),
               _stream_handle(stream, device))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_kv_cache_append_packed")


def flex_kv_cache_read(cache: KVCache, page_table: torch.Tensor, starts: torch.Tensor, total: int | None = None,
                       dtype: torch.dtype = torch.bfloat16, k_out: torch.Tensor | None = None,
                       v_out: torch.Tensor | None = None, stream=None):
    """The cache's tokens as packed sequences: position p of sequence b is token starts[b] + p of the returned
    (k, v) [1, H, total, D], for the starts[b + 1] - starts[b] first positions of each (asynchronous on `stream`).

    page_table int32 [sequences, max_pages], starts int32 [sequences + 1].  Outputs not given are allocated
    from `stream`'s pool with `total` tokens, in `dtype` (bfloat16 or float32), a token's heads next to each other in
    memory, as flex_attention_packed_fwd and a projection have them.
    """
    device = cache.k.device
    if page_table.dim() != 2:
        raise ValueError("page_table must be an int32 [sequences, max_pages] tensor")
    at, B = _starts(starts, device)
    max_pages = page_table.shape[1]
    table = _device_array(page_table, "page_table", torch.int32, device, (B, max_pages))
    outs = []
    for x in (k_out, v_out):
        if x is None:
            if total is None:
                raise ValueError("total is needed where k_out and v_out are not both given")
            x = _empty_by_token(1, cache.shape[1], total, cache.shape[3], dtype, device, stream)
        elif x.device != device:
            raise ValueError("the outputs must be on the cache's device")
        outs.append(x)
    rc = _call(device, load_library().flex_kv_cache_read, cache._ref, table, max_pages, at, B, _tensor(outs[0]),
               _tensor(outs[1]), _stream_handle(stream, device))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_kv_cache_read")
    return outs[0], outs[1]


def flex_kv_cache_attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, kv_lens: torch.Tensor,
                            mask_kind: int = FLEX_MASK_CAUSAL, window: int = 0, sinks: int = 0,
                            score_kind: int = FLEX_SCORE_IDENTITY, score_param: float = 0.0,
                            scale: float | None = None, out: torch.Tensor | None = None,
                            lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """The newest tokens' queries q [B, Hq, Q, D] against the cache; returns (out, lse).

    kv_lens int32 [B] counts the tokens in the cache, the query tokens among
    them.  workspace: a uint8 tensor of flex_kv_cache_attention_workspace()
    bytes, not shared with calls that may run at the same time.  It and the
    outputs are allocated from `stream`'s pool when not given.  Asynchronous on
    `stream`.
    """
    device, shape = cache.k.device, q.shape
    if len(shape) != 4 or q.device != device:
        raise ValueError("q must be a [B, Hq, Q, D] tensor on the cache's device")
    B, Hq, Q, D = shape
    if page_table.dim() != 2:
        raise ValueError("page_table must be an int32 [B, max_pages] tensor")
    max_pages = page_table.shape[1]
    table = _device_array(page_table, "page_table", torch.int32, device, (B, max_pages))
    lens = _device_array(kv_lens, "kv_lens", torch.int32, device, (B,))
    if out is None:
        out = _empty(shape, q.dtype, device, stream)
    else:
        _device_array(out, "out", q.dtype, device, shape)
    if lse is None:
        lse = _empty((B, Hq, Q), torch.float32, device, stream)
    else:
        _device_array(lse, "lse", torch.float32, device, (B, Hq, Q))
    params = None if mask_kind == FLEX_MASK_CAUSAL and not sinks else \
        ctypes.byref(_mask_params(mask_kind, window, 0, sinks))
    if workspace is None:
        size = _cache_workspace_bytes(shape, cache.shape, cache.struct.dtype, max_pages, mask_kind, window, sinks)
        workspace = _empty((size,), torch.uint8, device, stream)
    else:
        _device_array(workspace, "workspace", torch.uint8, device, workspace.shape)
        size = workspace.numel()
    rc = _call(device, load_library().flex_kv_cache_attention, _tensor(q), cache._ref, table, max_pages, lens,
               mask_kind, params, score_kind, float(score_param), D**-0.5 if scale is None else float(scale),
               out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), size, _stream_handle(stream, device))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_kv_cache_attention")
    return out, lse


@functools.lru_cache(maxsize=256)
def _cache_workspace_bytes(q_shape, pool_shape, dtype: int, max_pages: int, mask_kind: int, window: int,
                           sinks: int) -> int:
    """The library's answer for these sizes (it depends on nothing else)."""
    B, Hq, Q, D = q_shape
    q = _pack_tensor(16, FLEX_DTYPE_BF16, 0, B, Hq, Q, D, Hq * Q * D, Q * D, D, 1)
    cache = flex_kv_cache(*pool_shape, dtype, 0, 16, 16, 16, 16)
    params, size = _mask_params(mask_kind, window, 0, sinks), ctypes.c_int64()
    rc = load_library().flex_kv_cache_attention_workspace(q, ctypes.byref(cache), max_pages, mask_kind,
                                                          ctypes.byref(params), ctypes.byref(size))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_kv_cache_attention_workspace")
    return size.value


def flex_kv_cache_attention_workspace(q: torch.Tensor, cache: KVCache, max_pages: int,
                                      mask_kind: int = FLEX_MASK_CAUSAL, window: int = 0, sinks: int = 0) -> int:
    """Bytes of workspace that flex_kv_cache_attention needs for these sizes."""
    if q.dim() != 4:
        raise ValueError("q must be a [B, Hq, Q, D] tensor")
    return _cache_workspace_bytes(q.shape, cache.shape, cache.struct.dtype, max_pages, mask_kind, window, sinks)


class PackedPlan:
    """The plan of a batch of packed sequences: the C struct plus the tensor that owns its entries."""

    def __init__(self, struct: flex_packed_plan, entries: torch.Tensor):
        self.struct, self.entries = struct, entries
        self._ref = ctypes.byref(struct)


def flex_packed_plan_bytes(sequences: int, total_q: int, Hq: int, Hk: int) -> int:
    """Bytes of a plan's entries."""
    size = ctypes.c_int64()
    rc = load_library().flex_packed_plan_bytes(sequences, total_q, Hq, Hk, ctypes.byref(size))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_packed_plan_bytes")
    return size.value


def flex_packed_plan_create(q_starts: torch.Tensor, k_starts: torch.Tensor | None, total_q: int, total_k: int | None,
                            Hq: int, Hk: int, mask_kind: int = FLEX_MASK_CAUSAL, window: int = 0, sinks: int = 0,
                            stream=None) -> PackedPlan:
    """Plan of a batch of packed sequences for flex_attention_packed_fwd (asynchronous on `stream`, in its pool's memory).

    Sequence b has tokens q_starts[b] .. q_starts[b + 1] - 1 of q (total_q tokens, Hq heads), and k_starts[b] ..
    k_starts[b + 1] - 1 of k and v (total_k tokens, Hk heads; None: the same as q's).  Both int32 [sequences + 1],
    ascending; they are not needed any more once `stream` has passed the call.  With more keys than queries the queries
    are the last tokens.
    """
    device = q_starts.device
    qs, sequences = _starts(q_starts, device)
    if k_starts is None:
        if total_k is not None and total_k != total_q:
            raise ValueError("total_k without k_starts")
        ks, total_k = qs, total_q
    else:
        if total_k is None:
            raise ValueError("k_starts without total_k")
        ks = _device_array(k_starts, "k_starts", torch.int32, device, (sequences + 1,))
    entries = _empty((flex_packed_plan_bytes(sequences, total_q, Hq, Hk),), torch.uint8, device, stream)
    plan = flex_packed_plan(entries=entries.data_ptr())
    rc = _call(device, load_library().flex_packed_plan_create, qs, ks, sequences, total_q, total_k, Hq, Hk, mask_kind,
               ctypes.byref(_mask_params(mask_kind, window, 0, sinks)), ctypes.byref(plan), _stream_handle(stream, device))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_packed_plan_create")
    return PackedPlan(plan, entries)


def flex_attention_packed_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, plan: PackedPlan,
                              score_kind: int = FLEX_SCORE_IDENTITY, score_param: float = 0.0, scale: float | None = None,
                              out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Attention over the packed sequences of a plan: q [1, Hq, total_q, D], k and v [1, Hk, total_k, D], bf16 with any
    strides (a projection's [tokens, heads, D] is passed transposed); returns (out, lse).

    out [1, Hq, total_q, D] may have any strides; one that is not given has a token's heads next to each other in
    memory.  lse: contiguous float32 [1, Hq, total_q].  What is not given is allocated from `stream`'s pool.
    Asynchronous on `stream`.
    """
    device, shape = plan.entries.device, q.shape
    for x in (q, k, v):
        if x.device != device:
            raise ValueError("q, k and v must be on the plan's device")
    tq, tk, tv = _tensor(q), _tensor(k), _tensor(v)
    if out is None:
        out = _empty_by_token(*shape, q.dtype, device, stream)
    elif out.device != device:
        raise ValueError("out must be on the plan's device")
    if lse is None:
        lse = _empty(shape[:3], torch.float32, device, stream)
    else:
        _device_array(lse, "lse", torch.float32, device, shape[:3])
    rc = _call(device, load_library().flex_attention_packed_fwd, tq, tk, tv, plan._ref, score_kind, float(score_param),
               shape[3] ** -0.5 if scale is None else float(scale), _tensor(out), lse.data_ptr(),
               _stream_handle(stream, device))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_attention_packed_fwd")
    return out, lse


def flex_selftest_wait_timeout(limit_ms: int = 50, stream=None, device=None) -> None:
    """Enqueue the bounded-wait failure check (see include/flexattn.h)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with _device_guard(device):
        rc = load_library().flex_selftest_wait_timeout(int(limit_ms), _stream_handle(stream, device))
    if rc != FLEX_OK:
        raise FlexError(rc, "flex_selftest_wait_timeout")


def flex_device_status(stream=None, device=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        return int(load_library().flex_device_status(_stream_handle(stream, device)))
