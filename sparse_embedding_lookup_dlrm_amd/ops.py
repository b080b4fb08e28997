"""Thin ctypes binding over libdlrm_embbag.so (C ABI: include/dlrm_embbag.h and, for the
attention over user histories, include/dlrm_history.h).

Only argument marshalling happens here: torch supplies device memory and the
current HIP stream; every step of the computation runs in the library's HIP
kernels. The names mirror the C entry points. If the library is missing or
cannot be loaded, every call raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from typing import List, Optional, Sequence, Tuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdlrm_embbag.so")
INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
HEADERS = [os.path.join(INCLUDE, "dlrm_embbag.h"), os.path.join(INCLUDE, "dlrm_probe.h"),
           os.path.join(INCLUDE, "dlrm_history.h")]

DLRM_F32, DLRM_F16, DLRM_BF16 = 0, 1, 2
PAIRS_SELF, WITH_EMBEDDINGS = 1, 2  # interaction layout bits
STATUS_BAD_INDEX = 1
STATUS_BAD_OFFSETS = 2
STATUS_BAD_PAGE = 4
MAX_TABLES = 128
MAX_AXES = 8

_TORCH_DT = {torch.float32: DLRM_F32, torch.float16: DLRM_F16, torch.bfloat16: DLRM_BF16}

_c_void_p = ctypes.c_void_p
_i32, _i64, _f32, _size_t = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_P = ctypes.POINTER

# argument groups of dlrm_history.h: a tensor of heads (address, token and head stride), and the
# rotation and norm (positions .. interleaved)
_HEADS = [_c_void_p, _i64, _i64]
_TURN = [_c_void_p, _i64, _i32, _P(_i32), _c_void_p, _c_void_p, _c_void_p, _f32, _i32]

_SIGNATURES = {
    "dlrm_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "dlrm_version": (ctypes.c_int, []),
    "dlrm_lengths_to_offsets": (ctypes.c_int, [_i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "dlrm_embbag_fwd": (ctypes.c_int, [_i32, _i32, _i32, _i32, _P(_c_void_p), _P(_i64), _c_void_p, _c_void_p, _i64,
                                       _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "dlrm_embbag_fwd_ex": (ctypes.c_int, [_i32, _i32, _i32, _i32, _P(_c_void_p), _P(_i64), _c_void_p, _c_void_p,
                                          _i64, _c_void_p, _c_void_p, _c_void_p, _i32, _c_void_p, _c_void_p]),
    "dlrm_embbag_fwd_q4": (ctypes.c_int, [_i32, _i32, _i32, _P(_c_void_p), _P(_i64), _c_void_p, _c_void_p, _i64,
                                          _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "dlrm_embbag_fwd_q8t": (ctypes.c_int, [_i32, _i32, _i32, _P(_c_void_p), _P(_f32), _P(_i64), _c_void_p,
                                           _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                           _c_void_p]),
    "dlrm_interact": (ctypes.c_int, [_i32, _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "dlrm_interact_ex": (ctypes.c_int, [_i32, _i32, _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "dlrm_interact_bwd": (ctypes.c_int, [_i32, _i32, _i32, _i32, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                         _c_void_p, _c_void_p]),
    "dlrm_embbag_bwd_workspace_bytes": (ctypes.c_int, [_i32, _i32, _i32, _i64, _P(_i64), _P(_size_t)]),
    "dlrm_embbag_bwd_update": (ctypes.c_int, [_i32, _i32, _i32, _i32, _P(_c_void_p), _P(_i64), _c_void_p, _c_void_p,
                                              _i64, _c_void_p, _c_void_p, _c_void_p, _f32, _c_void_p, _c_void_p,
                                              _c_void_p, _c_void_p, _c_void_p, _c_void_p, _size_t, _c_void_p,
                                              _c_void_p]),
    "dlrm_embbag_bwd_update_adagrad": (ctypes.c_int, [_i32, _i32, _i32, _i32, _P(_c_void_p), _P(_i64), _c_void_p,
                                                      _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p, _f32, _f32,
                                                      _P(_c_void_p), _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                                      _c_void_p, _c_void_p, _size_t, _c_void_p, _c_void_p]),
    "dlrm_validate_bags": (ctypes.c_int, [_i32, _i32, _P(_i64), _P(_i32), _P(_i32), _i64]),
    "dlrm_embbag_bwd_update_ex": (ctypes.c_int, [_i32, _i32, _i32, _i32, _P(_c_void_p), _P(_i64), _c_void_p,
                                                 _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p, _i32, _f32, _f32,
                                                 _P(_c_void_p), _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                                 _c_void_p, _c_void_p, _size_t, _c_void_p, _c_void_p]),
    "dlrm_embbag_bwd_plan": (ctypes.c_int, [_i32, _i32, _i32, _i64, _P(_i64), _i32, _P(_i32)]),
    "dlrm_probe_row_gather": (ctypes.c_int, [_i32, _i32, _i32, _P(_c_void_p), _P(_i64), _P(_i64), _c_void_p, _i64,
                                             _c_void_p, _c_void_p]),
    "dlrm_embbag_bwd_update_noalloc": (ctypes.c_int, [_i32, _i32, _i32, _i32, _P(_c_void_p), _P(_i64), _c_void_p,
                                                      _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p, _f32,
                                                      _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                                      _c_void_p, _c_void_p]),
    "dlrm_qk_norm_rope": (ctypes.c_int, [_i64, _i32, _i32, _i32, _i32, _i32, *_HEADS, *_HEADS, *_TURN, _c_void_p,
                                         _c_void_p, _c_void_p]),
    "dlrm_qk_norm_rope_bwd_workspace_bytes": (ctypes.c_int, [_i64, _i32, _i32, _P(_size_t)]),
    "dlrm_qk_norm_rope_bwd": (ctypes.c_int, [_i64, _i32, _i32, _i32, _i32, _i32, *_HEADS, *_HEADS, *_HEADS, *_HEADS,
                                             *_TURN, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _size_t,
                                             _c_void_p]),
    "dlrm_kv_append": (ctypes.c_int, [_i64, _i32, _i32, _i32, _i32, _i32, _i32, *_HEADS, *_HEADS, *_HEADS, *_TURN,
                                      _c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i32, _i64, _i64, _i64, _c_void_p,
                                      _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "dlrm_paged_attn_workspace_bytes": (ctypes.c_int, [_i64, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                                       _P(_size_t)]),
    "dlrm_paged_attn": (ctypes.c_int, [_i64, _i32, _i32, _i32, _i32, _i32, *_HEADS, _c_void_p, _c_void_p, _i32, _i64,
                                       _i64, _i64, _c_void_p, _c_void_p, _c_void_p, _i64, _i32, _i32, _i32, _f32, _i32,
                                       _i32, _c_void_p, _c_void_p, _c_void_p, _size_t, _c_void_p, _c_void_p]),
}

_lib: Optional[ctypes.CDLL] = None


class DlrmError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {status_string(code)} ({code})")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libdlrm_embbag.so (built in-tree). Raises if it is absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m sparse_embedding_lookup_dlrm_amd.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
    return _lib


def header_functions() -> List[str]:
    """Names of the functions declared in the library's headers (include/*.h)."""
    names = set()
    for h in HEADERS:
        with open(h) as f:
            text = f.read()
        text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
        names |= set(re.findall(r"\b(dlrm_[a-z0-9_]+)\s*\(", text))
    return sorted(names)


def status_string(code: int) -> str:
    return lib().dlrm_status_string(code).decode()


def version() -> int:
    return lib().dlrm_version()


def _check(code: int, where: str) -> None:
    if code != 0:
        raise DlrmError(code, where)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _require_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("device tensors must be contiguous CUDA (HIP) tensors")


def _expect(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, numel: int, at_least: bool = False) -> None:
    """Size and dtype of a tensor handed to the C ABI, which takes raw pointers and cannot
    see an undersized buffer: checked here, before any call."""
    if t is None:
        return
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    n = t.numel()
    if (n < numel) if at_least else (n != numel):
        raise ValueError(f"{name} has {n} elements, needs {'at least ' if at_least else ''}{numel}")


def _check_bags(offsets: torch.Tensor, indices: torch.Tensor, T: int, B: int) -> None:
    _expect(offsets, "offsets", torch.int32, T * B + 1)
    if indices.dtype != torch.int32:
        raise ValueError(f"indices must be torch.int32, got {indices.dtype}")


def _table_args(tables: Sequence[torch.Tensor]):
    T = len(tables)
    if T < 1:
        raise ValueError("need at least one table")
    dt = tables[0].dtype
    if dt not in _TORCH_DT:
        raise ValueError(f"unsupported table dtype {dt}")
    D = tables[0].shape[1]
    for t in tables:
        if t.dtype != dt or t.dim() != 2 or t.shape[1] != D:
            raise ValueError("all tables must be 2-D with the same dtype and width")
    ptrs = (_c_void_p * T)(*[t.data_ptr() for t in tables])
    rows = (_i64 * T)(*[t.shape[0] for t in tables])
    return T, D, _TORCH_DT[dt], ptrs, rows


def pair_count(T: int, self_pairs: bool = False) -> int:
    F = T + 1
    return F * (F + 1) // 2 if self_pairs else F * (F - 1) // 2


def layout_bits(self_pairs: bool = False, with_embeddings: bool = False) -> int:
    return (PAIRS_SELF if self_pairs else 0) | (WITH_EMBEDDINGS if with_embeddings else 0)


def out_width(T: int, D: int, layout: int = 0) -> int:
    """Floats per sample of the interaction output in a layout."""
    return (T + 1) * D * bool(layout & WITH_EMBEDDINGS) + D * (not layout & WITH_EMBEDDINGS) + \
        pair_count(T, bool(layout & PAIRS_SELF))


def lengths_to_offsets(lengths: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """int32 bag lengths (device) -> int32 CSR offsets (device, n + 1 entries)."""
    _expect(lengths, "lengths", torch.int32, lengths.numel())
    n = lengths.numel()
    _expect(offsets, "offsets", torch.int32, n + 1)
    _expect(status, "status", torch.int32, 1, at_least=True)
    _require_cuda(lengths, offsets, status)
    if offsets is None:
        offsets = torch.empty(n + 1, dtype=torch.int32, device=lengths.device)
    _check(lib().dlrm_lengths_to_offsets(n, _ptr(lengths), _ptr(offsets), _ptr(status), _stream(stream)),
           "dlrm_lengths_to_offsets")
    return offsets


def _check_fwd_buffers(T, B, D, offsets, indices, e0, out_pooled, out_inter, status, layout=0):
    _check_bags(offsets, indices, T, B)
    _expect(e0, "e0", torch.float32, B * D)
    _expect(out_pooled, "out_pooled", torch.float32, B * T * D)
    _expect(out_inter, "out_inter", torch.float32, B * out_width(T, D, layout))
    _expect(status, "status", torch.int32, 1, at_least=True)


def embbag_fwd(tables: Sequence[torch.Tensor], offsets: torch.Tensor, indices: torch.Tensor, B: int,
               e0: Optional[torch.Tensor] = None, *, want_pooled: bool = False, want_inter: bool = True,
               out_pooled: Optional[torch.Tensor] = None, out_inter: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, stream=None,
               layout: int = 0) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Embedding-bag forward; returns (pooled [B,T,D] or None, interaction output [B, W] or None):
    [e0 | dots] with layout 0 (dlrm_embbag_fwd), else the layout bits PAIRS_SELF and
    WITH_EMBEDDINGS (dlrm_embbag_fwd_ex)."""
    T, D, dt, ptrs, rows = _table_args(tables)
    _check_fwd_buffers(T, B, D, offsets, indices, e0, out_pooled, out_inter, status, layout)
    _require_cuda(*tables, offsets, indices, e0, out_pooled, out_inter, status)
    dev = tables[0].device
    if want_pooled and out_pooled is None:
        out_pooled = torch.empty((B, T, D), dtype=torch.float32, device=dev)
    if want_inter and out_inter is None:
        out_inter = torch.empty((B, out_width(T, D, layout)), dtype=torch.float32, device=dev)
    if layout == 0:
        _check(lib().dlrm_embbag_fwd(T, B, D, dt, ptrs, rows, _ptr(offsets), _ptr(indices), indices.numel(),
                                     _ptr(e0), _ptr(out_pooled), _ptr(out_inter), _ptr(status), _stream(stream)),
               "dlrm_embbag_fwd")
    else:
        _check(lib().dlrm_embbag_fwd_ex(T, B, D, dt, ptrs, rows, _ptr(offsets), _ptr(indices), indices.numel(),
                                        _ptr(e0), _ptr(out_pooled), _ptr(out_inter), layout, _ptr(status),
                                        _stream(stream)),
               "dlrm_embbag_fwd_ex")
    return out_pooled, out_inter


def embbag_fwd_q4(tables: Sequence[torch.Tensor], offsets: torch.Tensor, indices: torch.Tensor, B: int,
                  e0: torch.Tensor, *, want_pooled: bool = False, out_pooled: Optional[torch.Tensor] = None,
                  out_inter: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                  stream=None) -> Tuple[Optional[torch.Tensor], torch.Tensor]:
    """Fused forward on row-wise 4-bit tables: uint8 [rows, D] per table (D = 128, 256 or 512;
    a row is D/2 code bytes, its fp32 scale and bias, then padding: synth.pack_q4_rows builds
    them); returns (pooled or None, [e0 | dots])."""
    T = len(tables)
    if T < 1:
        raise ValueError("need at least one table")
    D = tables[0].shape[1]
    for t in tables:
        if t.dtype != torch.uint8 or t.dim() != 2 or t.shape[1] != D or not t.is_contiguous():
            raise ValueError("4-bit tables must be contiguous uint8 [rows, D] with the same D")
    _check_fwd_buffers(T, B, D, offsets, indices, e0, out_pooled, out_inter, status)
    _require_cuda(*tables, offsets, indices, e0, out_pooled, out_inter, status)
    ptrs = (_c_void_p * T)(*[t.data_ptr() for t in tables])
    rows = (_i64 * T)(*[t.shape[0] for t in tables])
    dev = tables[0].device
    if want_pooled and out_pooled is None:
        out_pooled = torch.empty((B, T, D), dtype=torch.float32, device=dev)
    if out_inter is None:
        out_inter = torch.empty((B, D + pair_count(T)), dtype=torch.float32, device=dev)
    _check(lib().dlrm_embbag_fwd_q4(T, B, D, ptrs, rows, _ptr(offsets), _ptr(indices), indices.numel(), _ptr(e0),
                                    _ptr(out_pooled), _ptr(out_inter), _ptr(status), _stream(stream)),
           "dlrm_embbag_fwd_q4")
    return out_pooled, out_inter


def embbag_fwd_q8t(tables: Sequence[torch.Tensor], scale_bias, offsets: torch.Tensor, indices: torch.Tensor,
                   B: int, e0: torch.Tensor, *, want_pooled: bool = False,
                   out_pooled: Optional[torch.Tensor] = None, out_inter: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None) -> Tuple[Optional[torch.Tensor], torch.Tensor]:
    """Fused forward on table-wise 8-bit tables: uint8 [rows, D] codes per table and one
    (scale, bias) pair per table (host sequence of T pairs); returns (pooled or None, [e0 | dots])."""
    T = len(tables)
    if T < 1:
        raise ValueError("need at least one table")
    D = tables[0].shape[1]
    for t in tables:
        if t.dtype != torch.uint8 or t.dim() != 2 or t.shape[1] != D or not t.is_contiguous():
            raise ValueError("8-bit tables must be contiguous uint8 [rows, D] with the same D")
    sb = [float(v) for pair in scale_bias for v in pair]
    if len(sb) != 2 * T:
        raise ValueError("need one (scale, bias) pair per table")
    _check_fwd_buffers(T, B, D, offsets, indices, e0, out_pooled, out_inter, status)
    _require_cuda(*tables, offsets, indices, e0, out_pooled, out_inter, status)
    ptrs = (_c_void_p * T)(*[t.data_ptr() for t in tables])
    rows = (_i64 * T)(*[t.shape[0] for t in tables])
    dev = tables[0].device
    if want_pooled and out_pooled is None:
        out_pooled = torch.empty((B, T, D), dtype=torch.float32, device=dev)
    if out_inter is None:
        out_inter = torch.empty((B, D + pair_count(T)), dtype=torch.float32, device=dev)
    _check(lib().dlrm_embbag_fwd_q8t(T, B, D, ptrs, (_f32 * (2 * T))(*sb), rows, _ptr(offsets), _ptr(indices),
                                     indices.numel(), _ptr(e0), _ptr(out_pooled), _ptr(out_inter), _ptr(status),
                                     _stream(stream)),
           "dlrm_embbag_fwd_q8t")
    return out_pooled, out_inter


def interact(e0: torch.Tensor, pooled: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None,
             self_pairs: bool = False, with_embeddings: bool = False) -> torch.Tensor:
    """[e0 | lower-triangle dots of Z = [e0; pooled]] from pooled [B, T, D] fp32: pairs i > j
    (dlrm_interact); i >= j with self_pairs, and [Z rows | dots] with with_embeddings
    (dlrm_interact_ex)."""
    B, T, D = pooled.shape
    layout = layout_bits(self_pairs, with_embeddings)
    W = out_width(T, D, layout)
    _expect(pooled, "pooled", torch.float32, B * T * D)
    _expect(e0, "e0", torch.float32, B * D)
    _expect(out, "out", torch.float32, B * W)
    _require_cuda(e0, pooled, out)
    if out is None:
        out = torch.empty((B, W), dtype=torch.float32, device=pooled.device)
    if layout:
        _check(lib().dlrm_interact_ex(T, B, D, layout, _ptr(e0), _ptr(pooled), _ptr(out), _stream(stream)),
               "dlrm_interact_ex")
    else:
        _check(lib().dlrm_interact(T, B, D, _ptr(e0), _ptr(pooled), _ptr(out), _stream(stream)), "dlrm_interact")
    return out


def interact_bwd(e0: torch.Tensor, pooled: torch.Tensor, d_out: torch.Tensor, self_pairs: bool = False,
                 d_e0: Optional[torch.Tensor] = None, d_pooled: Optional[torch.Tensor] = None,
                 want_d_e0: bool = True, stream=None,
                 with_embeddings: bool = False) -> Tuple[Optional[torch.Tensor], torch.Tensor]:
    """(dL/de0, dL/dpooled) of the interaction from dL/dout (dlrm_interact_bwd)."""
    B, T, D = pooled.shape
    layout = layout_bits(self_pairs, with_embeddings)
    _expect(pooled, "pooled", torch.float32, B * T * D)
    _expect(e0, "e0", torch.float32, B * D)
    _expect(d_out, "d_out", torch.float32, B * out_width(T, D, layout))
    _expect(d_e0, "d_e0", torch.float32, B * D)
    _expect(d_pooled, "d_pooled", torch.float32, B * T * D)
    _require_cuda(e0, pooled, d_out, d_e0, d_pooled)
    if d_pooled is None:
        d_pooled = torch.empty((B, T, D), dtype=torch.float32, device=pooled.device)
    if d_e0 is None and want_d_e0:
        d_e0 = torch.empty((B, D), dtype=torch.float32, device=pooled.device)
    _check(lib().dlrm_interact_bwd(T, B, D, layout, _ptr(e0), _ptr(pooled), _ptr(d_out), _ptr(d_e0),
                                   _ptr(d_pooled), _stream(stream)), "dlrm_interact_bwd")
    return d_e0, d_pooled


def bwd_workspace_bytes(T: int, B: int, D: int, nnz: int, rows: Sequence[int]) -> int:
    r = (_i64 * T)(*rows)
    out = _size_t(0)
    _check(lib().dlrm_embbag_bwd_workspace_bytes(T, B, D, nnz, r, ctypes.byref(out)),
           "dlrm_embbag_bwd_workspace_bytes")
    return out.value


def _check_bwd_buffers(T, B, D, offsets, indices, e0, pooled, d_out, d_e0, status, layout=0):
    _check_bags(offsets, indices, T, B)
    _expect(e0, "e0", torch.float32, B * D)
    _expect(pooled, "pooled", torch.float32, B * T * D)
    _expect(d_out, "d_out", torch.float32, B * out_width(T, D, layout))
    _expect(d_e0, "d_e0", torch.float32, B * D)
    _expect(status, "status", torch.int32, 1, at_least=True)


def bwd_plan(T: int, B: int, D: int, nnz: int, rows: Sequence[int], want_segments: bool = True) -> dict:
    """How the sparse backward will run for these sizes (dlrm_embbag_bwd_plan; host only)."""
    plan = (_i32 * 5)()
    _check(lib().dlrm_embbag_bwd_plan(T, B, D, nnz, (_i64 * T)(*rows), 1 if want_segments else 0, plan),
           "dlrm_embbag_bwd_plan")
    return {"radix_bits": plan[0], "passes": plan[1], "interact_bwd_shared": bool(plan[2]), "max_lds": plan[3],
            "table_sort": bool(plan[4])}


def embbag_bwd_update(tables: Sequence[torch.Tensor], offsets: torch.Tensor, indices: torch.Tensor, B: int,
                      e0: torch.Tensor, pooled: torch.Tensor, d_out: torch.Tensor, lr: float, *,
                      want_d_e0: bool = True, want_segments: bool = True, workspace: Optional[torch.Tensor] = None,
                      status: Optional[torch.Tensor] = None, stream=None,
                      row_state: Optional[Sequence[torch.Tensor]] = None, eps: float = 1e-8,
                      layout: int = 0) -> dict:
    """Sparse backward + update of the touched rows (tables are updated in place): SGD, or
    row-wise AdaGrad when row_state (one fp32 [rows_t] tensor per table, updated in
    place) is given (dlrm_embbag_bwd_update_adagrad); d_out in the interaction layout
    `layout` (dlrm_embbag_bwd_update_ex when it is not 0)."""
    T, D, dt, ptrs, rows = _table_args(tables)
    _check_bwd_buffers(T, B, D, offsets, indices, e0, pooled, d_out, None, status, layout)
    if row_state is not None:
        if len(row_state) != T:
            raise ValueError("row_state needs one tensor per table")
        for st_, t in zip(row_state, tables):
            _require_cuda(st_)
            if st_.dtype != torch.float32 or st_.numel() != t.shape[0] or not st_.is_contiguous():
                raise ValueError("row_state[t] must be a contiguous fp32 tensor with one value per row")
    nnz = indices.numel()
    dev = tables[0].device
    need = bwd_workspace_bytes(T, B, D, nnz, [t.shape[0] for t in tables])
    _expect(workspace, "workspace", torch.uint8, need, at_least=True)
    _require_cuda(*tables, offsets, indices, e0, pooled, d_out, workspace, status)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    res = {"d_e0": torch.empty((B, D), dtype=torch.float32, device=dev) if want_d_e0 else None}
    if want_segments:
        res["unique_keys"] = torch.empty(max(nnz, 1), dtype=torch.int32, device=dev)
        res["seg_offsets"] = torch.empty(nnz + 1, dtype=torch.int32, device=dev)
        res["num_unique"] = torch.empty(1, dtype=torch.int32, device=dev)
        res["perm"] = torch.empty(max(nnz, 1), dtype=torch.int32, device=dev)
    g = res.get
    if layout != 0:
        sptr = (_c_void_p * T)(*[s_.data_ptr() for s_ in row_state]) if row_state is not None else None
        _check(lib().dlrm_embbag_bwd_update_ex(T, B, D, dt, ptrs, rows, _ptr(offsets), _ptr(indices), nnz, _ptr(e0),
                                               _ptr(pooled), _ptr(d_out), int(layout), float(lr), float(eps), sptr,
                                               _ptr(g("d_e0")), _ptr(g("unique_keys")), _ptr(g("seg_offsets")),
                                               _ptr(g("num_unique")), _ptr(g("perm")), _ptr(workspace),
                                               workspace.numel(), _ptr(status), _stream(stream)),
               "dlrm_embbag_bwd_update_ex")
    elif row_state is None:
        _check(lib().dlrm_embbag_bwd_update(T, B, D, dt, ptrs, rows, _ptr(offsets), _ptr(indices), nnz, _ptr(e0),
                                            _ptr(pooled), _ptr(d_out), float(lr), _ptr(g("d_e0")),
                                            _ptr(g("unique_keys")), _ptr(g("seg_offsets")), _ptr(g("num_unique")),
                                            _ptr(g("perm")), _ptr(workspace), workspace.numel(), _ptr(status),
                                            _stream(stream)),
               "dlrm_embbag_bwd_update")
    else:
        sptr = (_c_void_p * T)(*[s_.data_ptr() for s_ in row_state])
        _check(lib().dlrm_embbag_bwd_update_adagrad(T, B, D, dt, ptrs, rows, _ptr(offsets), _ptr(indices), nnz,
                                                    _ptr(e0), _ptr(pooled), _ptr(d_out), float(lr), float(eps), sptr,
                                                    _ptr(g("d_e0")), _ptr(g("unique_keys")), _ptr(g("seg_offsets")),
                                                    _ptr(g("num_unique")), _ptr(g("perm")), _ptr(workspace),
                                                    workspace.numel(), _ptr(status), _stream(stream)),
               "dlrm_embbag_bwd_update_adagrad")
    return res


PROBE_SINK_FLOATS = 4096 * 256


class ProbeGatherPlan:
    """dlrm_probe_row_gather (measurement kernel: the bare random-row gather of a batch)
    with its arguments marshalled once. table_start: host CSR position of each table's
    first occurrence, T + 1 entries."""

    def __init__(self, tables, table_start: Sequence[int], indices: torch.Tensor, sink: torch.Tensor, stream=None):
        T, D, dt, ptrs, rows = _table_args(tables)
        if len(table_start) != T + 1:
            raise ValueError("table_start needs T + 1 entries")
        _expect(sink, "sink", torch.float32, PROBE_SINK_FLOATS, at_least=True)
        _require_cuda(*tables, indices, sink)
        starts = (_i64 * (T + 1))(*[int(x) for x in table_start])
        self._keep = (tables, indices, sink, ptrs, rows, starts)
        self._args = (T, D, dt, ptrs, rows, starts, _ptr(indices), indices.numel(), _ptr(sink), _stream(stream))
        self._fn = lib().dlrm_probe_row_gather

    def run(self):
        _check(self._fn(*self._args), "dlrm_probe_row_gather")


NOALLOC_SCRATCH_BYTES = 64 << 20


def embbag_bwd_update_noalloc(tables: Sequence[torch.Tensor], offsets: torch.Tensor, indices: torch.Tensor, B: int,
                              e0: torch.Tensor, pooled: torch.Tensor, d_out: torch.Tensor, lr: float, *,
                              d_e0: Optional[torch.Tensor] = None, unique_keys: Optional[torch.Tensor] = None,
                              seg_offsets: Optional[torch.Tensor] = None, num_unique: Optional[torch.Tensor] = None,
                              perm: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                              stream=None) -> None:
    """dlrm_embbag_bwd_update_noalloc: the SGD backward with the library's own static scratch
    (no workspace). Every output is a caller tensor (or None); this call allocates nothing."""
    T, D, dt, ptrs, rows = _table_args(tables)
    nnz = indices.numel()
    _check_bwd_buffers(T, B, D, offsets, indices, e0, pooled, d_out, d_e0, status)
    _expect(unique_keys, "unique_keys", torch.int32, nnz, at_least=True)
    _expect(seg_offsets, "seg_offsets", torch.int32, nnz + 1, at_least=True)
    _expect(num_unique, "num_unique", torch.int32, 1, at_least=True)
    _expect(perm, "perm", torch.int32, nnz, at_least=True)
    _require_cuda(*tables, offsets, indices, e0, pooled, d_out, d_e0, unique_keys, seg_offsets, num_unique, perm,
                  status)
    _check(lib().dlrm_embbag_bwd_update_noalloc(T, B, D, dt, ptrs, rows, _ptr(offsets), _ptr(indices), nnz, _ptr(e0),
                                                _ptr(pooled), _ptr(d_out), float(lr), _ptr(d_e0), _ptr(unique_keys),
                                                _ptr(seg_offsets), _ptr(num_unique), _ptr(perm), _ptr(status),
                                                _stream(stream)),
           "dlrm_embbag_bwd_update_noalloc")


def validate_bags(T: int, B: int, rows: Sequence[int], offsets, indices) -> int:
    """Host check of a bag description (numpy/int sequences); returns the status bits."""
    import numpy as np

    off = np.ascontiguousarray(offsets, dtype=np.int32)
    idx = np.ascontiguousarray(indices, dtype=np.int32)
    r = (_i64 * T)(*rows)
    return lib().dlrm_validate_bags(T, B, r, off.ctypes.data_as(_P(_i32)), idx.ctypes.data_as(_P(_i32)), len(idx))


class FwdPlan:
    """dlrm_embbag_fwd with its arguments marshalled once, for repeated calls on
    resident inputs (same tensors every call)."""

    def __init__(self, tables, offsets, indices, B, e0=None, *, out_pooled=None, out_inter=None, status=None,
                 stream=None, layout: int = 0):
        T, D, dt, ptrs, rows = _table_args(tables)
        _check_fwd_buffers(T, B, D, offsets, indices, e0, out_pooled, out_inter, status, layout)
        _require_cuda(*tables, offsets, indices, e0, out_pooled, out_inter, status)
        self._keep = (tables, offsets, indices, e0, out_pooled, out_inter, status, ptrs, rows)
        if layout == 0:
            self._args = (T, B, D, dt, ptrs, rows, _ptr(offsets), _ptr(indices), indices.numel(), _ptr(e0),
                          _ptr(out_pooled), _ptr(out_inter), _ptr(status), _stream(stream))
            self._name = "dlrm_embbag_fwd"
        else:
            self._args = (T, B, D, dt, ptrs, rows, _ptr(offsets), _ptr(indices), indices.numel(), _ptr(e0),
                          _ptr(out_pooled), _ptr(out_inter), layout, _ptr(status), _stream(stream))
            self._name = "dlrm_embbag_fwd_ex"
        self._fn = getattr(lib(), self._name)

    def run(self):
        _check(self._fn(*self._args), self._name)


class BwdPlan:
    """dlrm_embbag_bwd_update (or, with row_state, dlrm_embbag_bwd_update_adagrad) with its
    arguments marshalled once (tables, and the row states, updated in place each run)."""

    def __init__(self, tables, offsets, indices, B, e0, pooled, d_out, lr, *, d_e0=None, workspace=None,
                 status=None, stream=None, row_state=None, eps: float = 1e-8):
        T, D, dt, ptrs, rows = _table_args(tables)
        nnz = indices.numel()
        dev = tables[0].device
        self.unique_keys = torch.empty(max(nnz, 1), dtype=torch.int32, device=dev)
        self.seg_offsets = torch.empty(nnz + 1, dtype=torch.int32, device=dev)
        self.num_unique = torch.empty(1, dtype=torch.int32, device=dev)
        self.perm = torch.empty(max(nnz, 1), dtype=torch.int32, device=dev)
        need = bwd_workspace_bytes(T, B, D, nnz, [t.shape[0] for t in tables])
        _expect(workspace, "workspace", torch.uint8, need, at_least=True)
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        _check_bwd_buffers(T, B, D, offsets, indices, e0, pooled, d_out, d_e0, status)
        _require_cuda(*tables, offsets, indices, e0, pooled, d_out, d_e0, workspace, status)
        opt = ()
        sptr = None
        self._name = "dlrm_embbag_bwd_update"
        if row_state is not None:
            if len(row_state) != T:
                raise ValueError("row_state needs one tensor per table")
            for st_, t in zip(row_state, tables):
                _require_cuda(st_)
                if st_.dtype != torch.float32 or st_.numel() != t.shape[0] or not st_.is_contiguous():
                    raise ValueError("row_state[t] must be a contiguous fp32 tensor with one value per row")
            sptr = (_c_void_p * T)(*[s_.data_ptr() for s_ in row_state])
            opt = (float(eps), sptr)
            self._name = "dlrm_embbag_bwd_update_adagrad"
        self._keep = (tables, offsets, indices, e0, pooled, d_out, d_e0, workspace, status, ptrs, rows, row_state,
                      sptr)
        self._args = (T, B, D, dt, ptrs, rows, _ptr(offsets), _ptr(indices), nnz, _ptr(e0), _ptr(pooled),
                      _ptr(d_out), float(lr), *opt, _ptr(d_e0), _ptr(self.unique_keys), _ptr(self.seg_offsets),
                      _ptr(self.num_unique), _ptr(self.perm), _ptr(workspace), workspace.numel(), _ptr(status),
                      _stream(stream))
        self._fn = getattr(lib(), self._name)

    def run(self):
        _check(self._fn(*self._args), self._name)


# Attention over user histories (include/dlrm_history.h). As the rest of this module, these calls are not recorded
# for autograd: a gradient of qk_norm_rope is taken with qk_norm_rope_bwd, the attention has none.


# The checks of these calls cost more host time than a small launch takes on the GPU, so they read each
# property of a tensor once and compare devices by number (-1: a host tensor).
# ctypes cuts a number that is too long for its type.
_I32_MAX = 0x7FFFFFFF
_I32_ARRAY = [_i32 * n for n in range(MAX_AXES + 1)]


def _heads_of(t: torch.Tensor, name: str, like: Optional[torch.Tensor] = None, shape=None,
              heads: Optional[int] = None):
    """Checks a tensor of heads [tokens, heads, dim], the elements of a head contiguous; like, shape: the
    tensor whose tokens, dim, dtype and device it has to share, and its shape. Returns its shape, and its
    address and strides."""
    own, strides = t.shape, t.stride()
    if len(own) != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim], got {tuple(own)}")
    n, many, width = own
    if like is None:
        if t.dtype not in _TORCH_DT:
            raise ValueError(f"unsupported dtype {t.dtype} of {name}")
    else:
        if t.dtype is not like.dtype:
            raise ValueError(f"{name} must be {like.dtype}, got {t.dtype}")
        if n != shape[0] or width != shape[2]:
            raise ValueError(f"{name} is {tuple(own)}, needs [{shape[0]}, heads, {shape[2]}]")
        if t.get_device() != like.get_device():
            raise ValueError(f"{name} is on {t.device}, not on {like.device}")
    if heads is not None and many != heads:
        raise ValueError(f"{name} has {many} heads, needs {heads}")
    a, b, c = strides
    if c != 1 and width != 1:
        raise ValueError(f"the elements of a head of {name} must be contiguous")
    # a stride over one token or head is never taken, and may be any number
    return (n, many, width), (t.data_ptr(), a if n > 1 else 0, b if many > 1 else 0)


def _plain(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, numel: int, dev: int, at_least: bool = False):
    """Checks a contiguous tensor's dtype, size and device; returns its address, None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != numel:
        _expect(t, name, dtype, numel, at_least)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on device {dev}")
    return t.data_ptr()


def _turn_args(dev, positions, inv_freq, w_q, w_k, eps, sections, interleaved, tokens: int, dim: int):
    """rot, and the arguments from positions to interleaved."""
    if inv_freq is None:
        rot, pos, stride, axes, secs, freq = 0, None, 0, 0, None, None
    else:
        half = inv_freq.numel()
        rot, freq = 2 * half, _plain(inv_freq, "inv_freq", torch.float32, half, dev)
        if positions is None or positions.dtype != torch.int32 or positions.dim() not in (1, 2):
            raise ValueError("positions must be torch.int32 [tokens] or [axes, tokens]")
        shape, strides = positions.shape, positions.stride()
        axes, stride = (shape[0], strides[0]) if len(shape) == 2 else (1, 0)
        if shape[-1] != tokens or (tokens > 1 and strides[-1] != 1):
            raise ValueError(f"positions must be [axes, {tokens}] with the tokens contiguous, got "
                             f"{tuple(shape)} with strides {strides}")
        if positions.get_device() != dev:
            raise ValueError(f"positions is on {positions.device}, not on device {dev}")
        if sections is None:
            if axes != 1:
                raise ValueError("sections are needed with more than one axis of positions")
            sections = (half,)
        if len(sections) != axes:
            raise ValueError(f"{len(sections)} sections for {axes} axes of positions")
        secs = (_I32_ARRAY[axes] if axes <= MAX_AXES else _i32 * axes)(*sections)
        if secs[:] != list(sections):
            raise ValueError(f"sections {tuple(sections)} do not fit 32 bits")
        pos = positions.data_ptr()
    if (w_q is None) != (w_k is None):
        raise ValueError("w_q and w_k come together")
    return rot, (pos, stride, axes, secs, freq, _plain(w_q, "w_q", torch.float32, dim, dev),
                 _plain(w_k, "w_k", torch.float32, dim, dev), eps, 1 if interleaved else 0)


# The handle of a device's current stream without the Stream object around it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _Here:
    """The calling thread's current stream on a device that is already the current one."""

    __slots__ = ("raw",)

    def __init__(self, raw: int):
        self.raw = raw

    def __enter__(self) -> int:
        return self.raw

    def __exit__(self, *exc):
        pass


class _There:
    """Another stream or device: buffers made within belong to that stream, so that one freed on return is
    not handed out again before the stream has passed the call."""

    def __init__(self, outer, raw):
        self.outer, self.raw = outer, raw

    def __enter__(self) -> int:
        self.outer.__enter__()
        return self.raw()

    def __exit__(self, *exc):
        self.outer.__exit__(*exc)


def _on(dev: int, where: torch.device, stream):
    """The device and stream a call works on, as a context that gives the stream's handle."""
    if dev < 0:
        raise ValueError("device tensors must be CUDA (HIP) tensors")
    if stream is None:
        if _current_device() == dev:
            return _Here(_raw_stream(dev))
        return _There(torch.cuda.device(where), lambda: torch.cuda.current_stream(where).cuda_stream)
    if stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {where}")
    return _There(torch.cuda.stream(stream), lambda: stream.cuda_stream)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: Optional[torch.Tensor],
                 inv_freq: Optional[torch.Tensor], w_q: Optional[torch.Tensor] = None,
                 w_k: Optional[torch.Tensor] = None, *, eps: float = 1e-6, sections: Optional[Sequence[int]] = None,
                 interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Norm of each head of q [N, Hq, D] and k [N, Hk, D] (with w_q, w_k fp32 [D]) and the position
    rotation of its first 2 * len(inv_freq) elements (dlrm_qk_norm_rope); returns contiguous (q, k).
    positions is int32 [N] or, with `sections` pairs to each axis, [axes, N]; inv_freq None: no rotation."""
    shape, qa = _heads_of(q, "q")
    (_, Hk, _), ka = _heads_of(k, "k", q, shape)
    N, Hq, D = shape
    dt, dev, where = q.dtype, q.get_device(), q.device
    rot, turn = _turn_args(dev, positions, inv_freq, w_q, w_k, eps, sections, interleaved, N, D)
    if q_out is not None:
        _plain(q_out, "q_out", dt, N * Hq * D, dev)
    if k_out is not None:
        _plain(k_out, "k_out", dt, N * Hk * D, dev)
    with _on(dev, where, stream) as s:
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        _check(lib().dlrm_qk_norm_rope(N, Hq, Hk, D, rot, _TORCH_DT[dt], *qa, *ka, *turn, q_out.data_ptr(),
                                       k_out.data_ptr(), s), "dlrm_qk_norm_rope")
    return q_out, k_out


@functools.lru_cache(maxsize=1024)
def qk_norm_rope_bwd_workspace_bytes(N: int, D: int, norm: bool) -> int:
    out = _size_t(0)
    _check(lib().dlrm_qk_norm_rope_bwd_workspace_bytes(N, D, 1 if norm else 0, ctypes.byref(out)),
           "dlrm_qk_norm_rope_bwd_workspace_bytes")
    return out.value


def qk_norm_rope_bwd(d_q_out: torch.Tensor, d_k_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                     positions: Optional[torch.Tensor], inv_freq: Optional[torch.Tensor],
                     w_q: Optional[torch.Tensor] = None, w_k: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                     sections: Optional[Sequence[int]] = None, interleaved: bool = False,
                     workspace: Optional[torch.Tensor] = None, stream=None
                     ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients of qk_norm_rope from those of its outputs (dlrm_qk_norm_rope_bwd); q, k and what
    follows as in the forward. Returns (d_q, d_k, d_w_q, d_w_k), the weights' fp32, None without a norm."""
    shape, qa = _heads_of(q, "q")
    (_, Hk, _), ka = _heads_of(k, "k", q, shape)
    N, Hq, D = shape
    _, dqa = _heads_of(d_q_out, "d_q_out", q, shape, Hq)
    _, dka = _heads_of(d_k_out, "d_k_out", q, shape, Hk)
    dt, dev, where = q.dtype, q.get_device(), q.device
    rot, turn = _turn_args(dev, positions, inv_freq, w_q, w_k, eps, sections, interleaved, N, D)
    need = qk_norm_rope_bwd_workspace_bytes(N, D, w_q is not None)
    if workspace is not None:
        _plain(workspace, "workspace", torch.uint8, need, dev, at_least=True)
    with _on(dev, where, stream) as s:
        d_q = torch.empty_like(q, memory_format=torch.contiguous_format)
        d_k = torch.empty_like(k, memory_format=torch.contiguous_format)
        d_w_q = d_w_k = None
        if w_q is not None:
            d_w_q = torch.empty(D, dtype=torch.float32, device=where)
            d_w_k = torch.empty(D, dtype=torch.float32, device=where)
            if workspace is None:
                workspace = torch.empty(need, dtype=torch.uint8, device=where)
        _check(lib().dlrm_qk_norm_rope_bwd(N, Hq, Hk, D, rot, _TORCH_DT[dt], *dqa, *dka, *qa, *ka, *turn,
                                           d_q.data_ptr(), d_k.data_ptr(), _ptr(d_w_q), _ptr(d_w_k), _ptr(workspace),
                                           0 if workspace is None else workspace.numel(), s),
               "dlrm_qk_norm_rope_bwd")
    return d_q, d_k, d_w_q, d_w_k


def _paged_args(dtype, dev: int, k_cache, v_cache, q_offsets, kv_lens, page_table, status, Hk: int, D: int):
    """Checks the cache and the sequences. Returns (seqs, page, pages, page and head stride, table stride and
    width) and the addresses (q_offsets, kv_lens, page_table, status)."""
    shape, strides = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or shape[1] != Hk or shape[3] != D:
        raise ValueError(f"k_cache must be [pages, {Hk}, page, {D}], got {tuple(shape)}")
    if v_cache.shape != shape or (v_cache.stride() != strides and any(
            a != b and n > 1 for a, b, n in zip(v_cache.stride(), strides, shape))):
        raise ValueError("v_cache must have k_cache's shape and strides")
    if k_cache.dtype != dtype or v_cache.dtype != dtype:
        raise ValueError(f"the caches must be {dtype}, got {k_cache.dtype} and {v_cache.dtype}")
    table = page_table.shape
    if len(table) != 2 or page_table.dtype != torch.int32:
        raise ValueError("page_table must be torch.int32 [sequences, pages]")
    S, width = table
    by_seq, by_entry = page_table.stride()
    if width > 1 and by_entry != 1:
        raise ValueError("the entries of a row of page_table must be contiguous")
    where = (_plain(q_offsets, "q_offsets", torch.int32, S + 1, dev), _plain(kv_lens, "kv_lens", torch.int32, S, dev),
             page_table.data_ptr(),
             None if status is None else _plain(status, "status", torch.int32, 1, dev, at_least=True))
    if k_cache.get_device() != dev or v_cache.get_device() != dev or page_table.get_device() != dev:
        raise ValueError(f"the caches and page_table must be on device {dev}, are on {k_cache.device}, "
                         f"{v_cache.device} and {page_table.device}")
    if shape[0] > 0 and (strides[2] != D or strides[3] != 1):
        raise ValueError("a page's entries of a head must be contiguous in the caches")
    # a stride over one page or head is never taken, and may be any number
    by_page, by_head = strides[0] if shape[0] > 1 else 0, strides[1] if Hk > 1 else 0
    return (S, shape[2], shape[0], by_page, by_head, by_seq, width), where


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              q_offsets: torch.Tensor, kv_lens: torch.Tensor, page_table: torch.Tensor, *,
              q: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
              inv_freq: Optional[torch.Tensor] = None, w_q: Optional[torch.Tensor] = None,
              w_k: Optional[torch.Tensor] = None, eps: float = 1e-6, sections: Optional[Sequence[int]] = None,
              interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
              status: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Appends k (normed and rotated as by qk_norm_rope) and v, [N, Hk, D], to the paged caches
    [pages, Hk, page, D] in place, and norms and rotates q in the same launch (dlrm_kv_append).
    Sequence s has tokens q_offsets[s] .. q_offsets[s + 1], the last entries of its kv_lens[s].
    Returns the new q, contiguous, or None without q (then w_q is not taken)."""
    shape, ka = _heads_of(k, "k")
    N, Hk, D = shape
    _, va = _heads_of(v, "v", k, shape, Hk)
    Hq, qa = 0, (None, 0, 0)
    if q is not None:
        (_, Hq, _), qa = _heads_of(q, "q", k, shape)
    elif q_out is not None:
        raise ValueError("q_out without q")
    elif w_q is not None:
        raise ValueError("w_q without q")
    dt, dev, where = k.dtype, k.get_device(), k.device
    rot, turn = _turn_args(dev, positions, inv_freq, w_k if q is None else w_q, w_k, eps, sections, interleaved, N, D)
    if q is None:
        turn = turn[:5] + (None,) + turn[6:]
    (S, page, pages, by_page, by_head, by_seq, width), (offsets_at, lens_at, table_at, status_at) = _paged_args(
        dt, dev, k_cache, v_cache, q_offsets, kv_lens, page_table, status, Hk, D)
    if q_out is not None:
        _plain(q_out, "q_out", dt, N * Hq * D, dev)
    with _on(dev, where, stream) as s:
        if q is not None and q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        _check(lib().dlrm_kv_append(N, S, Hq, Hk, D, rot, _TORCH_DT[dt], *qa, *ka, *va, *turn, offsets_at, lens_at,
                                    table_at, by_seq, width, page, pages, by_page, by_head, k_cache.data_ptr(),
                                    v_cache.data_ptr(), _ptr(q_out), status_at, s), "dlrm_kv_append")
    return q_out


@functools.lru_cache(maxsize=1024)
def paged_attn_workspace_bytes(N: int, S: int, Hq: int, Hk: int, D: int, causal: bool, window: int, max_q: int,
                               max_kv: int) -> int:
    out = _size_t(0)
    _check(lib().dlrm_paged_attn_workspace_bytes(N, S, Hq, Hk, D, 1 if causal else 0, window, max_q, max_kv,
                                                 ctypes.byref(out)), "dlrm_paged_attn_workspace_bytes")
    return out.value


def paged_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, q_offsets: torch.Tensor,
               kv_lens: torch.Tensor, page_table: torch.Tensor, *, causal: bool = True, window: int = 0,
               scale: Optional[float] = None, max_q: Optional[int] = None, max_kv: Optional[int] = None,
               want_lse: bool = False, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """Attention of the new tokens q [N, Hq, D] over the paged caches [pages, Hk, page, D]
    (dlrm_paged_attn); the sequences as in kv_append. window > 0 (with causal): a token sees the last
    `window` entries up to its own. max_q, max_kv: the most new tokens and the longest history of a
    sequence, for how the work is cut; without them N and the page table's width are taken, which is
    right for one sequence and slow for many of one token each. Returns
    out [N, Hq, D], or (out, lse [N, Hq] fp32) with want_lse."""
    shape, qa = _heads_of(q, "q")
    N, Hq, D = shape
    dt, dev, where = q.dtype, q.get_device(), q.device
    Hk = k_cache.shape[1] if k_cache.dim() == 4 else 0
    (S, page, pages, by_page, by_head, by_seq, width), (offsets_at, lens_at, table_at, status_at) = _paged_args(
        dt, dev, k_cache, v_cache, q_offsets, kv_lens, page_table, status, Hk, D)
    if max_q is None:
        max_q = N
    if max_kv is None:
        max_kv = min(width * page, _I32_MAX)
    if scale is None:
        scale = D ** -0.5 if D > 0 else 1.0
    if window > _I32_MAX or max_q > _I32_MAX or max_kv > _I32_MAX or window < 0 or max_q < 0 or max_kv < 0:
        raise ValueError(f"window {window}, max_q {max_q} and max_kv {max_kv} must lie between 0 and {_I32_MAX}")
    need = paged_attn_workspace_bytes(N, S, Hq, Hk, D, causal, window, max_q, max_kv)
    if out is not None:
        _plain(out, "out", dt, N * Hq * D, dev)
    if lse is not None:
        _plain(lse, "lse", torch.float32, N * Hq, dev)
    if workspace is not None:
        _plain(workspace, "workspace", torch.uint8, need, dev, at_least=True)
    with _on(dev, where, stream) as s:
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        if lse is None and want_lse:
            lse = q.new_empty((N, Hq), dtype=torch.float32)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=where)
        _check(lib().dlrm_paged_attn(N, S, Hq, Hk, D, _TORCH_DT[dt], *qa, k_cache.data_ptr(), v_cache.data_ptr(), page,
                                     pages, by_page, by_head, offsets_at, lens_at, table_at, by_seq, width,
                                     1 if causal else 0, window, scale, max_q, max_kv, out.data_ptr(), _ptr(lse),
                                     _ptr(workspace), 0 if workspace is None else workspace.numel(), status_at, s),
               "dlrm_paged_attn")
    return (out, lse) if want_lse else out
