"""Gated DeltaNet linear-attention hot path for one GB300 (sm_103a).

A thin ctypes binding over ``libgdn.so`` (C ABI in ``include/gdn.h``).  The
functions below carry the C names; they only check and marshal PyTorch
tensors (dtype, device, contiguity, shapes) into pointers and the current CUDA
stream.  Every step of the computation runs in the library's CUDA kernels;
there is no fallback of any kind: if the library is missing, every entry
point raises.

Layouts (all row-major, device memory):
  q, k        [T][h_k][d_k]  bfloat16
  v, o        [T][h_v][d_v]  bfloat16
  g, beta     [T][h_v]       float32   (alpha = exp(g))
  state       [num_slots][h_v][d_v][d_k] float32   (S^T per slot and head)
  chunk_states [n_emit][h_v][d_v][d_k] float32

Full-attention layers beside these (bfloat16 or float16, d = 64, 128 or 256):
  q, o        [T][h_q][d];  k, v [T][h_kv][d]
  k_cache, v_cache [pages][page_size][h_kv][d], any strides with d contiguous
  block_table [requests][width] int32 page ids
Trees of drafted tokens: masks [T] int64, bit w of a node's word set for itself and the nodes above it
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import _build

__all__ = [
    "GdnError", "load_library", "library_path", "prepare_decode_packed",
    "gdn_decode_packed", "gdn_decode_packed_raw", "gdn_prep_inputs", "gdn_decode_multi",
    "gdn_prefill_varlen", "gdn_prefill_varlen_apc", "gdn_mixed_step", "gdn_mixed_step_colaunch", "gdn_prefill_num_emits", "gdn_prefill_emit_offsets", "gdn_align_block_size",
    "gdn_floor_prefix_hit", "gdn_grid_emit_every_chunks", "gdn_status_string",
    "gdn_prefill_workspace_bytes", "gdn_status_from_device",
    "gdn_paged_maps", "gdn_paged_kv_write", "gdn_paged_attention", "gdn_paged_attention_workspace_bytes",
    "gdn_tree_maps", "gdn_tree_attention", "gdn_tree_decode", "gdn_rotary", "gdn_rotary_frequencies",
    "EXPORTED_SYMBOLS", "GDN_DEV_BAD_SLOT", "GDN_DEV_TIMEOUT", "GDN_DEV_BAD_LENGTH", "GDN_DEV_NO_PAGES",
    "GDN_DEV_BAD_PARENT",
]

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA = 0, 1, 2, 3
GDN_ERR_WORKSPACE, GDN_ERR_TIMEOUT = 4, 5
GDN_DEV_BAD_SLOT, GDN_DEV_TIMEOUT, GDN_DEV_BAD_LENGTH, GDN_DEV_NO_PAGES = 0x1, 0x2, 0x4, 0x8
GDN_DEV_BAD_PARENT = 0x10
GDN_BF16, GDN_FP16 = 0, 1

EXPORTED_SYMBOLS = (
    "gdn_decode_packed", "gdn_decode_packed_raw", "gdn_prep_inputs", "gdn_decode_multi",
    "gdn_prefill_varlen", "gdn_prefill_varlen_apc", "gdn_mixed_step", "gdn_mixed_step_colaunch", "gdn_prefill_num_emits", "gdn_prefill_emit_offsets", "gdn_align_block_size",
    "gdn_floor_prefix_hit", "gdn_grid_emit_every_chunks", "gdn_status_string",
    "gdn_prefill_workspace_bytes", "gdn_status_from_device",
    "gdn_paged_maps", "gdn_paged_kv_write", "gdn_paged_attention", "gdn_paged_attention_workspace_bytes",
    "gdn_tree_maps", "gdn_tree_attention", "gdn_tree_decode", "gdn_rotary", "gdn_rotary_frequencies",
)


class GdnError(RuntimeError):
    def __init__(self, status: int, fn: str):
        self.status = status
        super().__init__(f"{fn}: {gdn_status_string(status)}")


class Dims(ctypes.Structure):
    _fields_ = [("h_k", ctypes.c_int32), ("h_v", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("scale", ctypes.c_float)]


class PagedCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("h_kv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("num_pages", ctypes.c_int64)] + [
                    (f"{s}_{n}_stride", ctypes.c_int64) for s in "kv" for n in ("page", "slot", "head")]


class RotarySide(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int32)] + [
        (f"{t}_{n}_stride", ctypes.c_int64) for t in ("x", "out") for n in ("token", "head")]


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_lib = None


def library_path() -> str:
    return _build.LIB


def load_library() -> ctypes.CDLL:
    """Load libgdn.so (built by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB):
        raise ImportError(f"libgdn.so is not built ({_build.LIB}); run __graft_entry__.build()")
    _lib = _configure(ctypes.CDLL(_build.LIB))
    return _lib


def _configure(lib: ctypes.CDLL) -> ctypes.CDLL:
    """Declare the C signatures of every entry point on a loaded library."""
    lib.gdn_decode_packed.restype = ctypes.c_int
    lib.gdn_decode_packed.argtypes = [ctypes.POINTER(Dims), _I32, _P, _P, _P, _P, _P, _P, _I64,
                                      _P, _P, _P, _P, _P]
    lib.gdn_decode_packed_raw.restype = ctypes.c_int
    lib.gdn_decode_packed_raw.argtypes = [ctypes.POINTER(Dims), _I32, _P, _P, _P, _P, _P, _P, _P,
                                          ctypes.c_float, _P, _I64, _P, _P, _P, _P, _P]
    lib.gdn_prep_inputs.restype = ctypes.c_int
    lib.gdn_prep_inputs.argtypes = [ctypes.POINTER(Dims), _I64, _P, _P, _P, _P, _P, _P, ctypes.c_float,
                                    _P, _P, _P, _P, _P]
    lib.gdn_decode_multi.restype = ctypes.c_int
    lib.gdn_decode_multi.argtypes = [ctypes.POINTER(Dims), _I32, _I32, _P, _P, _P, _P, _P, _P, _I64,
                                     _P, _P, _P, _P, _P]
    lib.gdn_prefill_varlen.restype = ctypes.c_int
    lib.gdn_prefill_varlen.argtypes = [ctypes.POINTER(Dims), _I32, _P, _P, _P, _P, _P, _P, _P,
                                       _P, _I64, _P, _P, _P, _P, _I32, _I64, _P, _SZ, _P, _P]
    lib.gdn_prefill_varlen_apc.restype = ctypes.c_int
    lib.gdn_prefill_varlen_apc.argtypes = [ctypes.POINTER(Dims), _I32, _P, _P, _P, _P, _P, _P, _P,
                                           _P, _I64, _P, _P, _P, _I32, _P, _I32, _P, _P, _SZ, _P, _P]
    lib.gdn_mixed_step.restype = ctypes.c_int
    lib.gdn_mixed_step.argtypes = [ctypes.POINTER(Dims), _I32, _I32, _P, _P, _P, _P, _P, _P, _P,
                                   _P, _I64, _P, _P, _P, _P, _P, _P, _I32, _I64, _P, _SZ, _P, _P]
    lib.gdn_mixed_step_colaunch.restype = ctypes.c_int
    lib.gdn_mixed_step_colaunch.argtypes = lib.gdn_mixed_step.argtypes + [_P, _P, _P]
    lib.gdn_prefill_workspace_bytes.restype = _SZ
    lib.gdn_prefill_workspace_bytes.argtypes = [ctypes.POINTER(Dims), _I32, _I64]
    lib.gdn_status_from_device.restype = ctypes.c_int
    lib.gdn_status_from_device.argtypes = [_I32]
    _F32 = ctypes.c_float
    lib.gdn_paged_maps.restype = ctypes.c_int
    lib.gdn_paged_maps.argtypes = [_I32, _I32, _I64, _P, _P, _P, _I32, _I64, _P, _I32, _P, _P, _P, _P, _I64,
                                   _P, _P, _P, _P]
    lib.gdn_paged_kv_write.restype = ctypes.c_int
    lib.gdn_paged_kv_write.argtypes = [_P, _I64,  # the cache: a PagedCache by reference, or its bytes
                                       _P, _I64, _I64, _P, _I64, _I64,
                                       _P, _P, _P]
    lib.gdn_paged_attention.restype = ctypes.c_int
    lib.gdn_paged_attention.argtypes = [_P, _I32, _I64, _I32, _F32, _I32, _I64,
                                        _P, _I64, _P, _I32, _I64, _P, _P, _P, _P, _SZ, _P, _P]
    lib.gdn_paged_attention_workspace_bytes.restype = _SZ
    lib.gdn_paged_attention_workspace_bytes.argtypes = [_I32, _I32, _I32, _I32, _I64, _I64]
    lib.gdn_tree_maps.restype = ctypes.c_int
    lib.gdn_tree_maps.argtypes = [_I32, _I64, _P, _P, _P, _P, _P, _P, _P]
    lib.gdn_tree_attention.restype = ctypes.c_int
    lib.gdn_tree_attention.argtypes = [_P, _I32, _I64, _I32, _F32, _I64, _P, _I64, _P, _I32, _I64, _P, _P, _P, _P, _P,
                                       _SZ, _P, _P]
    lib.gdn_tree_decode.restype = ctypes.c_int
    lib.gdn_tree_decode.argtypes = [ctypes.POINTER(Dims), _I32, _I32, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _P, _P,
                                    _P, _P]
    lib.gdn_rotary.restype = ctypes.c_int
    lib.gdn_rotary.argtypes = [_I32, _I64, _I32, _I32, _I32, _F32, _P, _P,
                               _P, _P,  # the sides: a RotarySide by reference, its bytes, or None
                               _P]
    lib.gdn_rotary_frequencies.restype = ctypes.c_int
    lib.gdn_rotary_frequencies.argtypes = [_I32, ctypes.c_double, _I32, ctypes.c_double, _I64, ctypes.c_double,
                                           ctypes.c_double, _P]
    lib.gdn_prefill_num_emits.restype = _I64
    lib.gdn_prefill_num_emits.argtypes = [_P, _I32, _I32]
    lib.gdn_prefill_emit_offsets.restype = ctypes.c_int
    lib.gdn_prefill_emit_offsets.argtypes = [_P, _I32, _I32, _P]
    lib.gdn_align_block_size.restype = _I32
    lib.gdn_align_block_size.argtypes = [_I32]
    lib.gdn_floor_prefix_hit.restype = _I64
    lib.gdn_floor_prefix_hit.argtypes = [_I64, _I64, _I32]
    lib.gdn_grid_emit_every_chunks.restype = _I32
    lib.gdn_grid_emit_every_chunks.argtypes = [_I32]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_status_string.argtypes = [ctypes.c_int]
    return lib


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _dev(t, name, dtype, ndim=None, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    # the common case in one expression; the checks below name what is wrong
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and (ndim is None or t.dim() == ndim)):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return t


def _ptr(t):
    # a plain int: the argtypes (c_void_p) convert it
    return None if t is None else t.data_ptr()


# The current stream's handle without building a Stream object (a third of
# a small call's Python time); the public route where torch lacks it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(_current_device())
    return torch.cuda.current_stream().cuda_stream


def _host_i32(x, name):
    if isinstance(x, torch.Tensor):
        if x.is_cuda:
            raise ValueError(f"{name} must live in host memory")
        x = x.to(torch.int32).contiguous()
        return x, ctypes.c_void_p(x.data_ptr())
    arr = (ctypes.c_int32 * len(x))(*[int(v) for v in x])
    return arr, ctypes.cast(arr, ctypes.c_void_p)


def _workspace(ws, dims, num_seqs, total_tokens):
    """(pointer, bytes) of a caller workspace; checks it against the library's need."""
    need = load_library().gdn_prefill_workspace_bytes(ctypes.byref(dims), int(num_seqs), int(total_tokens))
    if ws is None:
        if need:
            raise ValueError(f"this prefill needs a {need}-byte workspace (gdn_prefill_workspace_bytes)")
        return None, 0
    ws = _dev(ws, "workspace", torch.uint8)
    return _ptr(ws), ws.numel()


def _check(status, fn):
    if status != GDN_OK:
        raise GdnError(status, fn)


_dims_cache = {}


def _dims(q, v, scale):
    key = (q.shape[1], v.shape[1], q.shape[2], v.shape[2], float(scale))
    d = _dims_cache.get(key)
    if d is None:  # read-only on the C side, so one object per shape serves every call
        d = _dims_cache[key] = Dims(*key)
    return d


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def gdn_decode_packed(q, k, v, g, beta, state, src_slot, o, dst_slot=None, dev_status=None,
                      scale: float = 1.0, stream=None) -> None:
    """Packed recurrent decode of ``q.shape[0]`` cached rows (see gdn.h)."""
    lib = load_library()
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    q, k, v = _dev(q, "q", bf, 3), _dev(k, "k", bf, 3), _dev(v, "v", bf, 3)
    g, beta = _dev(g, "g", f32, 2), _dev(beta, "beta", f32, 2)
    state = _dev(state, "state", f32, 4)
    src_slot = _dev(src_slot, "src_slot", i32, 1)
    dst_slot = _dev(dst_slot, "dst_slot", i32, 1, optional=True)
    o = _dev(o, "o", bf, 3)
    dev_status = _dev(dev_status, "dev_status", i32, optional=True)
    rows = q.shape[0]
    if not (k.shape == q.shape and v.shape[0] == rows and o.shape == v.shape
            and g.shape == (rows, v.shape[1]) and beta.shape == g.shape
            and src_slot.shape[0] == rows and (dst_slot is None or dst_slot.shape[0] == rows)
            and state.shape[1:] == (v.shape[1], v.shape[2], q.shape[2])):
        raise ValueError("inconsistent decode shapes")
    d = _dims(q, v, scale)
    _check(lib.gdn_decode_packed(ctypes.byref(d), rows, _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                 _ptr(beta), _ptr(state), state.shape[0], _ptr(src_slot),
                                 _ptr(dst_slot), _ptr(o), _ptr(dev_status), _stream(stream)),
           "gdn_decode_packed")


class _PreparedCall:
    """A C-ABI call whose arguments were checked and marshalled once: calling
    it issues the same call again on the same buffers (whatever they hold by
    then) and the same stream, with no per-call checks in Python.  The
    buffers must stay alive and keep their shapes and storage."""

    def __init__(self, fn, args, name, keep):
        self._fn, self._args, self._name, self._keep = fn, args, name, keep

    def __call__(self) -> None:
        status = self._fn(*self._args)
        if status != GDN_OK:
            raise GdnError(status, self._name)


def prepare_decode_packed(q, k, v, g, beta, state, src_slot, o, dst_slot=None, dev_status=None,
                          scale: float = 1.0, stream=None) -> _PreparedCall:
    """``gdn_decode_packed`` on fixed buffers, checked once: returns a callable
    that repeats the call (a serving loop refills q, k, v, g, beta and the
    slot lists in place between steps).  The stream is the one given, or the
    current stream at preparation."""
    lib = load_library()
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    q, k, v = _dev(q, "q", bf, 3), _dev(k, "k", bf, 3), _dev(v, "v", bf, 3)
    g, beta = _dev(g, "g", f32, 2), _dev(beta, "beta", f32, 2)
    state = _dev(state, "state", f32, 4)
    src_slot = _dev(src_slot, "src_slot", i32, 1)
    dst_slot = _dev(dst_slot, "dst_slot", i32, 1, optional=True)
    o = _dev(o, "o", bf, 3)
    dev_status = _dev(dev_status, "dev_status", i32, optional=True)
    rows = q.shape[0]
    if not (k.shape == q.shape and v.shape[0] == rows and o.shape == v.shape
            and g.shape == (rows, v.shape[1]) and beta.shape == g.shape
            and src_slot.shape[0] == rows and (dst_slot is None or dst_slot.shape[0] == rows)
            and state.shape[1:] == (v.shape[1], v.shape[2], q.shape[2])):
        raise ValueError("inconsistent decode shapes")
    d = _dims(q, v, scale)
    args = (ctypes.byref(d), rows, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
            state.shape[0], _ptr(src_slot), _ptr(dst_slot), _ptr(o), _ptr(dev_status), _stream(stream))
    keep = (d, q, k, v, g, beta, state, src_slot, dst_slot, o, dev_status)
    return _PreparedCall(lib.gdn_decode_packed, args, "gdn_decode_packed", keep)


def gdn_prep_inputs(q_raw, k_raw, a, b, A_log, dt_bias, q, k, g, beta, eps: float = 1e-6,
                    stream=None) -> None:
    """Input preparation: normalised q, k (bf16) and g, beta (fp32) from raw
    projections (see gdn.h).  q, k may alias q_raw, k_raw."""
    lib = load_library()
    bf, f32 = torch.bfloat16, torch.float32
    q_raw, k_raw = _dev(q_raw, "q_raw", bf, 3), _dev(k_raw, "k_raw", bf, 3)
    q, k = _dev(q, "q", bf, 3), _dev(k, "k", bf, 3)
    a, b, g, beta = (_dev(x, n, f32, 2) for x, n in ((a, "a"), (b, "b"), (g, "g"), (beta, "beta")))
    A_log, dt_bias = _dev(A_log, "A_log", f32, 1), _dev(dt_bias, "dt_bias", f32, 1)
    T, h_v = a.shape
    if not (k_raw.shape == q_raw.shape == q.shape == k.shape and q.shape[0] == T and b.shape == a.shape
            and g.shape == a.shape and beta.shape == a.shape and A_log.shape == (h_v,)
            and dt_bias.shape == (h_v,)):
        raise ValueError("inconsistent input-preparation shapes")
    d = Dims(q.shape[1], h_v, q.shape[2], q.shape[2], 1.0)
    _check(lib.gdn_prep_inputs(ctypes.byref(d), T, _ptr(q_raw), _ptr(k_raw), _ptr(a), _ptr(b), _ptr(A_log),
                               _ptr(dt_bias), float(eps), _ptr(q), _ptr(k), _ptr(g), _ptr(beta),
                               _stream(stream)),
           "gdn_prep_inputs")


def gdn_decode_packed_raw(q_raw, k_raw, v, a, b, A_log, dt_bias, state, src_slot, o, dst_slot=None,
                          dev_status=None, eps: float = 1e-6, scale: float = 1.0, stream=None) -> None:
    """Packed decode with the input preparation fused in (see gdn.h)."""
    lib = load_library()
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    q_raw, k_raw, v = _dev(q_raw, "q_raw", bf, 3), _dev(k_raw, "k_raw", bf, 3), _dev(v, "v", bf, 3)
    a, b = _dev(a, "a", f32, 2), _dev(b, "b", f32, 2)
    A_log, dt_bias = _dev(A_log, "A_log", f32, 1), _dev(dt_bias, "dt_bias", f32, 1)
    state = _dev(state, "state", f32, 4)
    src_slot = _dev(src_slot, "src_slot", i32, 1)
    dst_slot = _dev(dst_slot, "dst_slot", i32, 1, optional=True)
    o = _dev(o, "o", bf, 3)
    dev_status = _dev(dev_status, "dev_status", i32, optional=True)
    rows = q_raw.shape[0]
    if not (k_raw.shape == q_raw.shape and v.shape[0] == rows and o.shape == v.shape
            and a.shape == (rows, v.shape[1]) and b.shape == a.shape
            and A_log.shape == (v.shape[1],) and dt_bias.shape == A_log.shape
            and src_slot.shape[0] == rows and (dst_slot is None or dst_slot.shape[0] == rows)
            and state.shape[1:] == (v.shape[1], v.shape[2], q_raw.shape[2])):
        raise ValueError("inconsistent decode shapes")
    d = _dims(q_raw, v, scale)
    _check(lib.gdn_decode_packed_raw(ctypes.byref(d), rows, _ptr(q_raw), _ptr(k_raw), _ptr(v), _ptr(a),
                                     _ptr(b), _ptr(A_log), _ptr(dt_bias), float(eps), _ptr(state),
                                     state.shape[0], _ptr(src_slot), _ptr(dst_slot), _ptr(o),
                                     _ptr(dev_status), _stream(stream)),
           "gdn_decode_packed_raw")


def gdn_decode_multi(tokens_per_row: int, q, k, v, g, beta, state, src_slot, o, dst_slots=None,
                     dev_status=None, scale: float = 1.0, stream=None) -> None:
    """Multi-token decode: ``q.shape[0] // tokens_per_row`` rows of
    ``tokens_per_row`` consecutive tokens each (see gdn.h)."""
    lib = load_library()
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    q, k, v = _dev(q, "q", bf, 3), _dev(k, "k", bf, 3), _dev(v, "v", bf, 3)
    g, beta = _dev(g, "g", f32, 2), _dev(beta, "beta", f32, 2)
    state = _dev(state, "state", f32, 4)
    src_slot = _dev(src_slot, "src_slot", i32, 1)
    dst_slots = _dev(dst_slots, "dst_slots", i32, 1, optional=True)
    o = _dev(o, "o", bf, 3)
    dev_status = _dev(dev_status, "dev_status", i32, optional=True)
    T = int(tokens_per_row)
    ntok = q.shape[0]
    if T < 1 or ntok % T:
        raise ValueError("q.shape[0] must be a multiple of tokens_per_row >= 1")
    rows = ntok // T
    if not (k.shape == q.shape and v.shape[0] == ntok and o.shape == v.shape
            and g.shape == (ntok, v.shape[1]) and beta.shape == g.shape
            and src_slot.shape[0] == rows and (dst_slots is None or dst_slots.shape[0] == ntok)
            and state.shape[1:] == (v.shape[1], v.shape[2], q.shape[2])):
        raise ValueError("inconsistent multi-token decode shapes")
    d = _dims(q, v, scale)
    _check(lib.gdn_decode_multi(ctypes.byref(d), rows, T, _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                _ptr(beta), _ptr(state), state.shape[0], _ptr(src_slot),
                                _ptr(dst_slots), _ptr(o), _ptr(dev_status), _stream(stream)),
           "gdn_decode_multi")


def gdn_prefill_varlen(q, k, v, g, beta, cu_seqlens, cu_seqlens_host, o, state=None,
                       src_slot=None, dst_slot=None, chunk_states=None, emit_every_chunks: int = 0,
                       dev_status=None, scale: float = 1.0, stream=None, workspace=None) -> None:
    """Chunked varlen prefill (see gdn.h).  ``cu_seqlens_host`` is a host
    sequence (list or CPU tensor) with the same values as ``cu_seqlens``;
    ``workspace`` an optional uint8 device tensor (see
    ``gdn_prefill_workspace_bytes``)."""
    lib = load_library()
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    q, k, v = _dev(q, "q", bf, 3), _dev(k, "k", bf, 3), _dev(v, "v", bf, 3)
    g, beta = _dev(g, "g", f32, 2), _dev(beta, "beta", f32, 2)
    o = _dev(o, "o", bf, 3)
    cu_seqlens = _dev(cu_seqlens, "cu_seqlens", i32, 1)
    state = _dev(state, "state", f32, 4, optional=True)
    src_slot = _dev(src_slot, "src_slot", i32, 1, optional=True)
    dst_slot = _dev(dst_slot, "dst_slot", i32, 1, optional=True)
    chunk_states = _dev(chunk_states, "chunk_states", f32, 4, optional=True)
    dev_status = _dev(dev_status, "dev_status", i32, optional=True)
    keep, cu_h = _host_i32(cu_seqlens_host, "cu_seqlens_host")
    n = cu_seqlens.shape[0] - 1
    if len(keep) != n + 1:
        raise ValueError("cu_seqlens_host must have num_seqs + 1 entries")
    T = q.shape[0]
    if not (k.shape == q.shape and v.shape[0] == T and o.shape == v.shape
            and g.shape == (T, v.shape[1]) and beta.shape == g.shape):
        raise ValueError("inconsistent prefill shapes")
    d = _dims(q, v, scale)
    cap = 0 if chunk_states is None else chunk_states.shape[0]
    ws, ws_bytes = _workspace(workspace, d, n, T)
    _check(lib.gdn_prefill_varlen(ctypes.byref(d), n, _ptr(cu_seqlens), cu_h, _ptr(q), _ptr(k),
                                  _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
                                  0 if state is None else state.shape[0], _ptr(src_slot),
                                  _ptr(dst_slot), _ptr(o), _ptr(chunk_states),
                                  int(emit_every_chunks), cap, ws, ws_bytes, _ptr(dev_status),
                                  _stream(stream)),
           "gdn_prefill_varlen")


def gdn_prefill_varlen_apc(q, k, v, g, beta, cu_seqlens, cu_seqlens_host, o, state, block_table,
                           block_first, emit_every_chunks: int, src_slot=None, dst_slot=None,
                           dev_status=None, scale: float = 1.0, stream=None, workspace=None) -> None:
    """Chunked varlen prefill emitting into cache blocks: ``block_table``
    int32 [num_seqs][max_blocks], ``block_first`` int32 [num_seqs] (see gdn.h)."""
    lib = load_library()
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    q, k, v = _dev(q, "q", bf, 3), _dev(k, "k", bf, 3), _dev(v, "v", bf, 3)
    g, beta = _dev(g, "g", f32, 2), _dev(beta, "beta", f32, 2)
    o = _dev(o, "o", bf, 3)
    cu_seqlens = _dev(cu_seqlens, "cu_seqlens", i32, 1)
    state = _dev(state, "state", f32, 4)
    block_table = _dev(block_table, "block_table", i32, 2)
    block_first = _dev(block_first, "block_first", i32, 1)
    src_slot = _dev(src_slot, "src_slot", i32, 1, optional=True)
    dst_slot = _dev(dst_slot, "dst_slot", i32, 1, optional=True)
    dev_status = _dev(dev_status, "dev_status", i32, optional=True)
    keep, cu_h = _host_i32(cu_seqlens_host, "cu_seqlens_host")
    n = cu_seqlens.shape[0] - 1
    if len(keep) != n + 1 or block_table.shape[0] != n or block_first.shape[0] != n:
        raise ValueError("cu_seqlens_host, block_table and block_first must cover num_seqs sequences")
    T = q.shape[0]
    if not (k.shape == q.shape and v.shape[0] == T and o.shape == v.shape
            and g.shape == (T, v.shape[1]) and beta.shape == g.shape):
        raise ValueError("inconsistent prefill shapes")
    d = _dims(q, v, scale)
    ws, ws_bytes = _workspace(workspace, d, n, T)
    _check(lib.gdn_prefill_varlen_apc(ctypes.byref(d), n, _ptr(cu_seqlens), cu_h, _ptr(q), _ptr(k),
                                      _ptr(v), _ptr(g), _ptr(beta), _ptr(state), state.shape[0],
                                      _ptr(src_slot), _ptr(dst_slot), _ptr(o), int(emit_every_chunks),
                                      _ptr(block_table), block_table.shape[1], _ptr(block_first),
                                      ws, ws_bytes, _ptr(dev_status), _stream(stream)),
           "gdn_prefill_varlen_apc")


def _mixed_args(num_decodes, q, k, v, g, beta, cu_seqlens_p, cu_seqlens_p_host, state, dec_src_slot, o,
                dec_dst_slot, pre_src_slot, pre_dst_slot, chunk_states, emit_every_chunks, dev_status,
                scale, stream, workspace):
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    q, k, v = _dev(q, "q", bf, 3), _dev(k, "k", bf, 3), _dev(v, "v", bf, 3)
    g, beta = _dev(g, "g", f32, 2), _dev(beta, "beta", f32, 2)
    o = _dev(o, "o", bf, 3)
    state = _dev(state, "state", f32, 4)
    dec_src_slot = _dev(dec_src_slot, "dec_src_slot", i32, 1, optional=num_decodes == 0)
    dec_dst_slot = _dev(dec_dst_slot, "dec_dst_slot", i32, 1, optional=True)
    pre_src_slot = _dev(pre_src_slot, "pre_src_slot", i32, 1, optional=True)
    pre_dst_slot = _dev(pre_dst_slot, "pre_dst_slot", i32, 1, optional=True)
    chunk_states = _dev(chunk_states, "chunk_states", f32, 4, optional=True)
    dev_status = _dev(dev_status, "dev_status", i32, optional=True)
    cu_seqlens_p = _dev(cu_seqlens_p, "cu_seqlens_p", i32, 1, optional=True)
    n_p = 0 if cu_seqlens_p is None else cu_seqlens_p.shape[0] - 1
    keep, cu_h = _host_i32(cu_seqlens_p_host if cu_seqlens_p_host is not None else [0], "cu_seqlens_p_host")
    if n_p and len(keep) != n_p + 1:
        raise ValueError("cu_seqlens_p_host must have num_prefills + 1 entries")
    T = q.shape[0]
    if not (k.shape == q.shape and v.shape[0] == T and o.shape == v.shape
            and g.shape == (T, v.shape[1]) and beta.shape == g.shape):
        raise ValueError("inconsistent mixed-step shapes")
    if n_p and int(keep[-1]) + num_decodes != T:
        raise ValueError("token count does not match num_decodes + cu_seqlens_p_host[-1]")
    d = _dims(q, v, scale)
    cap = 0 if chunk_states is None else chunk_states.shape[0]
    ws, ws_bytes = _workspace(workspace, d, n_p, T - int(num_decodes))
    # `keep` and `d` hold the memory that cu_h and byref(d) point into.
    return (keep, d), [ctypes.byref(d), int(num_decodes), n_p, _ptr(cu_seqlens_p), cu_h,
                       _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
                       state.shape[0], _ptr(dec_src_slot), _ptr(dec_dst_slot),
                       _ptr(pre_src_slot), _ptr(pre_dst_slot), _ptr(o), _ptr(chunk_states),
                       int(emit_every_chunks), cap, ws, ws_bytes, _ptr(dev_status), _stream(stream)]


def gdn_mixed_step(num_decodes: int, q, k, v, g, beta, cu_seqlens_p, cu_seqlens_p_host, state,
                   dec_src_slot, o, dec_dst_slot=None, pre_src_slot=None, pre_dst_slot=None,
                   chunk_states=None, emit_every_chunks: int = 0, dev_status=None,
                   scale: float = 1.0, stream=None, workspace=None) -> None:
    """Mixed step: decode rows [0, num_decodes) then prefill sequences."""
    lib = load_library()
    _keep, args = _mixed_args(num_decodes, q, k, v, g, beta, cu_seqlens_p, cu_seqlens_p_host, state,
                              dec_src_slot, o, dec_dst_slot, pre_src_slot, pre_dst_slot, chunk_states,
                              emit_every_chunks, dev_status, scale, stream, workspace)
    _check(lib.gdn_mixed_step(*args), "gdn_mixed_step")


def _event_handle(ev, stream):
    # torch creates the CUDA event on its first record; recording it once on
    # `stream` here is harmless because the library records it again.
    if ev.cuda_event == 0:
        ev.record(stream if stream is not None else torch.cuda.current_stream())
    return ctypes.c_void_p(ev.cuda_event)


def gdn_mixed_step_colaunch(num_decodes: int, q, k, v, g, beta, cu_seqlens_p, cu_seqlens_p_host, state,
                            dec_src_slot, o, aux_stream, fork_event, join_event, dec_dst_slot=None,
                            pre_src_slot=None, pre_dst_slot=None, chunk_states=None,
                            emit_every_chunks: int = 0, dev_status=None, scale: float = 1.0,
                            stream=None, workspace=None) -> None:
    """Mixed step with the decode rows on `aux_stream` (a torch.cuda.Stream)
    running beside the prefill on `stream`; `fork_event` and `join_event` are
    torch.cuda.Event objects the call records (fork on `stream`, join on
    `aux_stream`).  The decode and prefill slots must not overlap."""
    lib = load_library()
    _keep, args = _mixed_args(num_decodes, q, k, v, g, beta, cu_seqlens_p, cu_seqlens_p_host, state,
                              dec_src_slot, o, dec_dst_slot, pre_src_slot, pre_dst_slot, chunk_states,
                              emit_every_chunks, dev_status, scale, stream, workspace)
    if aux_stream is None:
        extra = [None, None, None]
    else:
        extra = [ctypes.c_void_p(aux_stream.cuda_stream), _event_handle(fork_event, stream),
                 _event_handle(join_event, stream)]
    _check(lib.gdn_mixed_step_colaunch(*args, *extra), "gdn_mixed_step_colaunch")


# ---------------------------------------------------------------------------
# full-attention layers over a paged K/V cache
# ---------------------------------------------------------------------------

_PAGED_DTYPES = {torch.bfloat16: GDN_BF16, torch.float16: GDN_FP16}
_Tensor, _i32 = torch.Tensor, torch.int32
_pack_cache = struct.Struct("=QQiiii7q").pack  # the bytes of a PagedCache, in a third of its constructor's time


# These calls' device work takes microseconds, so the checks of a good call are
# one expression each and give the pointer at once; the slow way names what is
# wrong.
def _i32_vec(t, name):
    if t.__class__ is _Tensor and t.dtype is _i32 and t.is_cuda and t.dim() == 1 and t.is_contiguous():
        return t.data_ptr()
    return _dev(t, name, _i32, 1).data_ptr()


def _i32_word(t, name):
    return None if t is None else _dev(t, name, _i32).data_ptr()


def _strided(t, name, dtype, ndim):
    """A CUDA tensor whose last dimension is contiguous; its other strides are
    free.  Gives its strides."""
    if t.__class__ is _Tensor and t.is_cuda and t.dtype is dtype and t.dim() == ndim:
        st = t.stride()
        if st[-1] == 1:
            return st
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.stride()


def _paged_cache(k_cache, v_cache):
    """The C description of a cache (its bytes), and its shape."""
    dtype = getattr(k_cache, "dtype", None)
    code = _PAGED_DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"k_cache must be bfloat16 or float16, got {dtype}")
    ks, vs = _strided(k_cache, "k_cache", dtype, 4), _strided(v_cache, "v_cache", dtype, 4)
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    pages, page_size, h_kv, d = shape
    return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), code, page_size, h_kv, d, pages,
                       ks[0], ks[1], ks[2], vs[0], vs[1], vs[2]), shape


def _block_table(t):
    """Pointer, rows, width and row stride (one row's stride says nothing: its width stands for it)."""
    st = _strided(t, "block_table", _i32, 2)
    rows, width = t.shape
    return t.data_ptr(), rows, width, st[0] if rows > 1 else width


def gdn_paged_maps(context_lens, new_lens, block_table, page_size: int, num_pages: int, cu_seqlens, kv_lens,
                   slot_map, positions, free_pages=None, free_head=None, free_head_out=None, dev_status=None,
                   stream=None) -> None:
    """Maps of a step from its request lengths: pages from the free list into
    ``block_table`` (in place), ``cu_seqlens``, ``kv_lens``, and the slot and
    position of every new token (see gdn.h).  ``free_head_out`` defaults to
    ``free_head``, which then advances in place."""
    lib = _lib or load_library()
    ctx, new = _i32_vec(context_lens, "context_lens"), _i32_vec(new_lens, "new_lens")
    table, rows, width, table_stride = _block_table(block_table)
    cu, kv = _i32_vec(cu_seqlens, "cu_seqlens"), _i32_vec(kv_lens, "kv_lens")
    slots, pos = _i32_vec(slot_map, "slot_map"), _i32_vec(positions, "positions")
    n, capacity = context_lens.numel(), slot_map.numel()
    if not (new_lens.numel() == n and rows == n and cu_seqlens.numel() == n + 1 and kv_lens.numel() == n
            and positions.numel() == capacity):
        raise ValueError("inconsistent paged-maps shapes")
    pages = head = head_out = None
    num_free = 0
    if free_pages is not None:
        num_free = free_pages.numel()
        # an empty list serves no page, unlike no list at all: any non-null pointer stands for it
        pages = _i32_vec(free_pages, "free_pages") or cu
        head = _dev(free_head, "free_head", _i32).data_ptr()
        head_out = head if free_head_out is None else _dev(free_head_out, "free_head_out", _i32).data_ptr()
    _check(lib.gdn_paged_maps(n, page_size, num_pages, ctx, new, table, width, table_stride, pages, num_free, head,
                              head_out, cu, kv, capacity, slots, pos, _i32_word(dev_status, "dev_status"),
                              _stream(stream)), "gdn_paged_maps")


def gdn_paged_kv_write(k, v, k_cache, v_cache, slot_map, dev_status=None, stream=None) -> None:
    """Rows of ``k`` and ``v`` ([T][h_kv][d]) into the caches' slots
    ``slot_map`` (see gdn.h).  The caches are viewed as
    [pages][page_size][h_kv][d]; any strides with a contiguous last dimension."""
    lib = _lib or load_library()
    cache, shape = _paged_cache(k_cache, v_cache)
    ks, vs = _strided(k, "k", k_cache.dtype, 3), _strided(v, "v", k_cache.dtype, 3)
    slots = _i32_vec(slot_map, "slot_map")
    T, h_kv, d = rows = k.shape
    if not (rows == v.shape and h_kv == shape[2] and d == shape[3] and slot_map.numel() == T):
        raise ValueError("inconsistent K/V write shapes")
    _check(lib.gdn_paged_kv_write(cache, T, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
                                  slots, _i32_word(dev_status, "dev_status"), _stream(stream)),
           "gdn_paged_kv_write")


def gdn_paged_attention_workspace_bytes(h_q: int, h_kv: int, d: int, num_reqs: int, num_tokens: int,
                                        max_kv_len: int) -> int:
    """Device scratch (bytes) of a ``gdn_paged_attention`` call of these sizes.  ``max_kv_len``: the call's bound; for a
    call without one, what its block table holds, or 0, which is enough for any table."""
    n = load_library().gdn_paged_attention_workspace_bytes(int(h_q), int(h_kv), int(d), int(num_reqs),
                                                           int(num_tokens), int(max_kv_len))
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("invalid paged-attention sizes")
    return int(n)


def gdn_paged_attention(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, o, scale=None, window: int = 0,
                        max_kv_len: int = 0, workspace=None, dev_status=None, stream=None) -> None:
    """Attention of each request's new tokens over its cached ones (see
    gdn.h).  ``q`` is [T][h_q][d] (rows may be slices of a wider tensor), ``o``
    dense; ``scale`` defaults to d ** -0.5; ``max_kv_len`` bounds ``kv_lens``
    (0: what the block table can hold); ``workspace`` is a uint8 tensor of
    ``gdn_paged_attention_workspace_bytes`` for that bound."""
    lib = _lib or load_library()
    cache, shape = _paged_cache(k_cache, v_cache)
    qs = _strided(q, "q", k_cache.dtype, 3)
    o = _dev(o, "o", k_cache.dtype, 3)
    table, rows, width, table_stride = _block_table(block_table)
    cu, kv = _i32_vec(cu_seqlens, "cu_seqlens"), _i32_vec(kv_lens, "kv_lens")
    T, h_q, d = q.shape
    n = kv_lens.numel()
    if not (o.shape == q.shape and d == shape[3] and cu_seqlens.numel() == n + 1 and rows == n):
        raise ValueError("inconsistent paged-attention shapes")
    if qs[1] != d and h_q > 1:
        raise ValueError("q's heads must be adjacent")
    ws = ws_bytes = 0
    if workspace is not None:
        workspace = _dev(workspace, "workspace", torch.uint8)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel()
    _check(lib.gdn_paged_attention(cache, n, T, h_q, d ** -0.5 if scale is None else scale, window,
                                   max_kv_len, q.data_ptr(), qs[0], table, width, table_stride, cu, kv, o.data_ptr(),
                                   ws, ws_bytes, _i32_word(dev_status, "dev_status"), _stream(stream)),
           "gdn_paged_attention")


# The calls on trees and gdn_rotary are made for steps of a few microseconds, so the checks of a good call are one
# expression for all of its tensors; where it does not hold, the slow way names what is wrong.
_i64, _bf16, _f32, _one = torch.int64, torch.bfloat16, torch.float32, (1,)
_dims_refs = {}


def _words(t, name):
    if t.__class__ is _Tensor and t.dtype is torch.int64 and t.is_cuda and t.dim() == 1 and t.is_contiguous():
        return t.data_ptr()
    return _dev(t, name, torch.int64, 1).data_ptr()


def gdn_tree_maps(parents, cu_seqlens, kv_lens, masks, positions, dev_status=None, stream=None) -> None:
    """Words (``masks``, int64) and positions of the nodes of each request's
    tree from their ``parents`` (see gdn.h); ``cu_seqlens`` and ``kv_lens`` as
    ``gdn_paged_maps`` gives them."""
    lib = _lib or load_library()
    if not (parents.__class__ is cu_seqlens.__class__ is kv_lens.__class__ is masks.__class__ is positions.__class__ is _Tensor
            and parents.dtype is cu_seqlens.dtype is kv_lens.dtype is positions.dtype is _i32 and masks.dtype is _i64
            and parents.is_cuda and cu_seqlens.is_cuda and kv_lens.is_cuda and masks.is_cuda and positions.is_cuda
            and parents.stride() == cu_seqlens.stride() == kv_lens.stride() == masks.stride() == positions.stride() == _one):
        _i32_vec(parents, "parents"), _i32_vec(cu_seqlens, "cu_seqlens"), _i32_vec(kv_lens, "kv_lens")
        _words(masks, "masks"), _i32_vec(positions, "positions")
    n, T = kv_lens.numel(), parents.numel()
    if not (cu_seqlens.numel() == n + 1 and masks.numel() == T and positions.numel() == T):
        raise ValueError("inconsistent tree-maps shapes")
    status = lib.gdn_tree_maps(n, T, parents.data_ptr(), cu_seqlens.data_ptr(), kv_lens.data_ptr(), masks.data_ptr(),
                               positions.data_ptr(), None if dev_status is None else _i32_word(dev_status, "dev_status"),
                               _raw_stream(_current_device()) if stream is None and _raw_stream else _stream(stream))
    if status:
        raise GdnError(status, "gdn_tree_maps")


def gdn_tree_attention(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, masks, o, scale=None,
                       max_kv_len: int = 0, workspace=None, dev_status=None, stream=None) -> None:
    """Attention of each request's nodes over its cached tokens and the nodes
    that their words name (see gdn.h); arguments as ``gdn_paged_attention``'s,
    and the ``masks`` of ``gdn_tree_maps``."""
    lib = _lib or load_library()
    cache, shape = _paged_cache(k_cache, v_cache)
    qs = _strided(q, "q", k_cache.dtype, 3)
    o = _dev(o, "o", k_cache.dtype, 3)
    table, rows, width, table_stride = _block_table(block_table)
    cu, kv, words = _i32_vec(cu_seqlens, "cu_seqlens"), _i32_vec(kv_lens, "kv_lens"), _words(masks, "masks")
    T, h_q, d = q.shape
    n = kv_lens.numel()
    if not (o.shape == q.shape and d == shape[3] and cu_seqlens.numel() == n + 1 and rows == n and masks.numel() == T):
        raise ValueError("inconsistent tree-attention shapes")
    if qs[1] != d and h_q > 1:
        raise ValueError("q's heads must be adjacent")
    ws = ws_bytes = 0
    if workspace is not None:
        workspace = _dev(workspace, "workspace", torch.uint8)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel()
    _check(lib.gdn_tree_attention(cache, n, T, h_q, d ** -0.5 if scale is None else scale, max_kv_len, q.data_ptr(),
                                  qs[0], table, width, table_stride, cu, kv, words, o.data_ptr(), ws, ws_bytes,
                                  _i32_word(dev_status, "dev_status"), _stream(stream)), "gdn_tree_attention")


def gdn_tree_decode(q, k, v, g, beta, state, src_slot, cu_seqlens, masks, o, max_nodes: int = 64, dev_status=None,
                    scale: float = 1.0, stream=None) -> None:
    """The gated delta rule along each row's tree of drafted tokens, from the
    state of its slot, which stays as it is (see gdn.h).  ``max_nodes`` bounds
    a row's nodes."""
    lib = _lib or load_library()
    bf, f32 = _bf16, _f32
    if not (q.__class__ is k.__class__ is v.__class__ is o.__class__ is g.__class__ is beta.__class__ is state.__class__
            is src_slot.__class__ is cu_seqlens.__class__ is masks.__class__ is _Tensor
            and q.dtype is k.dtype is v.dtype is o.dtype is bf and g.dtype is beta.dtype is state.dtype is f32
            and src_slot.dtype is cu_seqlens.dtype is _i32 and masks.dtype is _i64
            and q.is_cuda and k.is_cuda and v.is_cuda and o.is_cuda and g.is_cuda and beta.is_cuda and state.is_cuda
            and src_slot.is_cuda and cu_seqlens.is_cuda and masks.is_cuda
            and q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and o.is_contiguous() and g.is_contiguous()
            and beta.is_contiguous() and state.is_contiguous()
            and src_slot.stride() == cu_seqlens.stride() == masks.stride() == _one):
        for t, name, dtype, ndim in ((q, "q", bf, 3), (k, "k", bf, 3), (v, "v", bf, 3), (g, "g", f32, 2), (beta, "beta", f32, 2),
                                     (state, "state", f32, 4), (o, "o", bf, 3), (src_slot, "src_slot", _i32, 1),
                                     (cu_seqlens, "cu_seqlens", _i32, 1), (masks, "masks", _i64, 1)):
            _dev(t, name, dtype, ndim)
    n = src_slot.numel()
    qs, vs, ss = q.shape, v.shape, state.shape
    if not (len(qs) == len(vs) == 3 and len(ss) == 4):
        _dev(q, "q", bf, 3), _dev(v, "v", bf, 3), _dev(state, "state", f32, 4)
    T, h_k, d = qs
    _, h_v, d_v = vs
    slots_n = ss[0]
    gates = (T, h_v)
    if not (k.shape == qs and vs[0] == T and o.shape == vs and g.shape == gates and beta.shape == gates
            and cu_seqlens.numel() == n + 1 and masks.numel() == T and ss == (slots_n, h_v, d_v, d)):
        raise ValueError("inconsistent tree-decode shapes")
    key = (h_k, h_v, d, d_v, float(scale))
    dims = _dims_refs.get(key)
    if dims is None:
        dims = _dims_refs[key] = ctypes.byref(_dims(q, v, scale))
    status = lib.gdn_tree_decode(dims, n, max_nodes, T, cu_seqlens.data_ptr(), masks.data_ptr(), q.data_ptr(), k.data_ptr(),
                                 v.data_ptr(), g.data_ptr(), beta.data_ptr(), state.data_ptr(), slots_n, src_slot.data_ptr(),
                                 o.data_ptr(), None if dev_status is None else _i32_word(dev_status, "dev_status"),
                                 _raw_stream(_current_device()) if stream is None and _raw_stream else _stream(stream))
    if status:
        raise GdnError(status, "gdn_tree_decode")


_ROTARY_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
_pack_side = struct.Struct("@PPiqqqq").pack  # RotarySide's layout


def _rotary_side(x, out, name, dtype, T, d):
    """The C description of one side (its bytes)."""
    if x.__class__ is _Tensor and x.is_cuda and x.dtype is dtype:
        xt, xh, one = x.stride() if x.dim() == 3 else (0, 0, 0)
    else:
        one = 0
    if one != 1:
        xt, xh, _ = _strided(x, name, dtype, 3)
    tokens, h, size = shape = x.shape
    if tokens != T or size != d:
        raise ValueError("inconsistent rotary shapes")
    p = x.data_ptr()
    if out is None:
        return _pack_side(p, p, h, xt, xh, xt, xh)
    if out.__class__ is _Tensor and out.is_cuda and out.dtype is dtype and out.shape == shape:
        ot, oh, one = out.stride()
        if one == 1:
            return _pack_side(p, out.data_ptr(), h, xt, xh, ot, oh)
    ot, oh, _ = _strided(out, f"{name}_out", dtype, 3)
    if out.shape != shape:
        raise ValueError("inconsistent rotary shapes")
    return _pack_side(p, out.data_ptr(), h, xt, xh, ot, oh)


def gdn_rotary(q, k, positions, frequencies, q_out=None, k_out=None, interleaved: bool = False,
               magnitude: float = 1.0, stream=None) -> None:
    """Rotary positions of ``q`` ([T][h_q][d]) and ``k`` ([T][h_kv][d]; None for
    either: the other alone), into ``q_out`` and ``k_out`` or, where those are None, in place (see
    gdn.h).  The first 2 * len(frequencies) elements of each head turn, in
    halves or ``interleaved`` pairs; ``frequencies`` is the tensor of
    ``gdn_rotary_frequencies``, on the device.  Any strides with a contiguous
    last dimension."""
    lib = _lib or load_library()
    some = k if q is None else q
    dtype = getattr(some, "dtype", None)
    code = _PAGED_DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"{'k' if q is None else 'q'} must be bfloat16 or float16, got {dtype}")
    if not (positions.__class__ is frequencies.__class__ is _Tensor and positions.dtype is _i32 and frequencies.dtype is _i64
            and positions.is_cuda and frequencies.is_cuda and positions.stride() == frequencies.stride() == _one):
        _i32_vec(positions, "positions"), _words(frequencies, "frequencies")
    T, d = positions.numel(), some.shape[-1]
    status = lib.gdn_rotary(code, T, d, 2 * frequencies.numel(), 1 if interleaved else 0, magnitude, positions.data_ptr(),
                            frequencies.data_ptr(), None if q is None else _rotary_side(q, q_out, "q", dtype, T, d),
                            None if k is None else _rotary_side(k, k_out, "k", dtype, T, d),
                            _raw_stream(_current_device()) if stream is None and _raw_stream else _stream(stream))
    if status:
        raise GdnError(status, "gdn_rotary")


# ---------------------------------------------------------------------------
# host-only helpers
# ---------------------------------------------------------------------------

def gdn_rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                           original_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0) -> torch.Tensor:
    """Frequencies of the ``rotary_dim`` / 2 pairs for ``gdn_rotary``, an int64
    CPU tensor (bits of 64-bit fractions of a turn; move it to the device
    once).  ``scaling``: "none", "linear", "ntk" or "yarn" (see gdn.h)."""
    if scaling not in _ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_ROTARY_SCALINGS)}, got {scaling!r}")
    out = torch.empty(max(int(rotary_dim), 0) // 2, dtype=torch.int64)
    _check(load_library().gdn_rotary_frequencies(int(rotary_dim), float(base), _ROTARY_SCALINGS[scaling], float(factor),
                                                 int(original_length), float(beta_fast), float(beta_slow),
                                                 out.data_ptr() or None), "gdn_rotary_frequencies")
    return out


def gdn_prefill_num_emits(cu_seqlens_host, emit_every_chunks: int) -> int:
    keep, p = _host_i32(cu_seqlens_host, "cu_seqlens_host")
    n = load_library().gdn_prefill_num_emits(p, len(keep) - 1, int(emit_every_chunks))
    if n < 0:
        raise ValueError("invalid cu_seqlens_host")
    return int(n)


def gdn_prefill_emit_offsets(cu_seqlens_host, emit_every_chunks: int) -> list[int]:
    keep, p = _host_i32(cu_seqlens_host, "cu_seqlens_host")
    out = (ctypes.c_int64 * len(keep))()
    _check(load_library().gdn_prefill_emit_offsets(p, len(keep) - 1, int(emit_every_chunks),
                                                   ctypes.cast(out, ctypes.c_void_p)),
           "gdn_prefill_emit_offsets")
    return [int(x) for x in out]


def gdn_align_block_size(block_size: int) -> int:
    return int(load_library().gdn_align_block_size(int(block_size)))


def gdn_floor_prefix_hit(hit_tokens: int, prompt_tokens: int, block_size: int) -> int:
    return int(load_library().gdn_floor_prefix_hit(int(hit_tokens), int(prompt_tokens), int(block_size)))


def gdn_grid_emit_every_chunks(block_size: int) -> int:
    return int(load_library().gdn_grid_emit_every_chunks(int(block_size)))


def gdn_prefill_workspace_bytes(h_k: int, h_v: int, d: int, num_seqs: int, total_tokens: int) -> int:
    """Device scratch (bytes) a prefill of ``num_seqs`` sequences needs."""
    dims = Dims(int(h_k), int(h_v), int(d), int(d), 1.0)
    n = load_library().gdn_prefill_workspace_bytes(ctypes.byref(dims), int(num_seqs), int(total_tokens))
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("invalid prefill dims or sizes")
    return int(n)


def gdn_status_from_device(word: int) -> int:
    """Status of a finished call from the device status word it wrote."""
    return int(load_library().gdn_status_from_device(int(word)))


def gdn_status_string(status: int) -> str:
    return load_library().gdn_status_string(int(status)).decode()
