"""Python binding of libsv: speculative-decoding draft verification and D-cut depth scheduling
on GB300 (sm_103a).

This module only marshals arguments: every step of verification and scheduling runs in the
CUDA kernels of ``libsv.so`` (built in-tree by ``build.build()``).  PyTorch supplies device
memory and streams.  There is no CPU fallback: if the library is missing or cannot be loaded,
every call raises.

The ``sv_*`` functions mirror the C ABI in ``include/sv.h`` one to one (tensors in place of
pointers, ``None`` for NULL).  The lower-case helpers (``verify_greedy``, ``verify_sample``,
``verify_ragged``, ``verify_tree``, ``schedule_depth``, ``sample``, ``tree_attention``) and ``PagedCache``
derive sizes and strides from the tensors and allocate outputs and workspaces.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsv.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "sv.h")

SV_OK, SV_ERR_INVALID_ARG, SV_ERR_WORKSPACE, SV_ERR_CUDA, SV_ERR_DEVICE_INPUT, SV_ERR_TIMEOUT = range(6)
SV_BF16, SV_F32 = 0, 1
SV_OP_VERIFY, SV_OP_SCHEDULE, SV_OP_TREE = 0, 1, 2
SV_OBJ_THROUGHPUT, SV_OBJ_NET = 0, 1
SV_PHASE_STATS, SV_PHASE_ACCEPT, SV_PHASE_WEIGHTS, SV_PHASE_PICK = range(4)
(SV_DEV_BAD_TOKEN, SV_DEV_BAD_TEMPERATURE, SV_DEV_BAD_KEEP_LEN, SV_DEV_BAD_OFFSETS, SV_DEV_NO_DRAFT_ROWS,
 SV_DEV_BAD_ALPHA, SV_DEV_BAD_DRAFT_LEN, SV_DEV_TIMEOUT, SV_DEV_BAD_PARENT, SV_DEV_BAD_LOGIT, SV_DEV_BAD_FILTER,
 SV_DEV_BAD_PAGE, SV_DEV_OUT_OF_PAGES, SV_DEV_BAD_SEQ, SV_DEV_BAD_NODES) = (1 << b for b in range(15))
SV_STATUS_BYTES, SV_MAX_BATCH = 256, 4096
SV_CACHE_WORKSPACE_BYTES = SV_STATUS_BYTES + 8 * SV_MAX_BATCH
SV_FLAG_Q_ZERO, SV_FLAG_Z_ZERO, SV_FLAG_INVALID = 1, 2, 4
(SV_KERNEL_ROW_STATS, SV_KERNEL_COMBINE, SV_KERNEL_SCHEDULE, SV_KERNEL_MASS, SV_KERNEL_PICK, SV_KERNEL_TREE_WALK,
 SV_NUM_KERNELS) = range(7)
KERNEL_NAMES = ("row_stats", "combine", "schedule", "mass", "pick", "tree_walk")
# kernels of the round's other operators (sv_profile_collect_ids reports them too)
(SV_KERNEL_SAMPLE, SV_KERNEL_CACHE_PAGES, SV_KERNEL_CACHE_ROWS, SV_KERNEL_ATTENTION, SV_KERNEL_ATTENTION_JOIN,
 SV_NUM_KERNEL_IDS) = range(6, 12)
OPERATOR_KERNEL_NAMES = KERNEL_NAMES + ("sample", "cache_pages", "cache_rows", "attention", "attention_join")

_c = ctypes
_vp, _i32, _i64, _u32, _u64, _f32, _sz = (_c.c_void_p, _c.c_int32, _c.c_int64, _c.c_uint32, _c.c_uint64,
                                         _c.c_float, _c.c_size_t)

_SIGS = {
    "sv_abi_version": (_c.c_int, []),
    "sv_workspace_size": (_sz, [_c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int]),
    "sv_verify_greedy": (_c.c_int, [_vp, _i64, _vp, _i64, _vp, _c.c_int, _c.c_int, _c.c_int, _c.c_int,
                                    _vp, _vp, _vp, _sz, _vp]),
    "sv_verify_sample": (_c.c_int, [_vp, _i64, _vp, _i64, _vp, _vp, _u64, _u32, _vp, _c.c_int, _c.c_int,
                                    _c.c_int, _c.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sv_verify_ragged": (_c.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _c.c_int, _vp, _vp,
                                    _u64, _u32, _vp, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _vp, _vp, _vp,
                                    _vp, _vp, _vp, _sz, _vp]),
    "sv_verify_sample_noalloc": (_c.c_int, [_vp, _i64, _vp, _i64, _vp, _vp, _u64, _u32, _vp, _c.c_int,
                                            _c.c_int, _c.c_int, _c.c_int, _vp, _vp, _vp, _vp, _vp, _vp]),
    "sv_schedule_depth": (_c.c_int, [_vp, _c.c_int, _vp, _c.c_int, _c.c_int, _f32, _f32, _c.c_int, _vp,
                                     _c.c_int, _c.c_int, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sv_schedule_depth_table": (_c.c_int, [_vp, _c.c_int, _vp, _c.c_int, _c.c_int, _vp, _vp, _c.c_int,
                                           _c.c_int, _vp, _c.c_int, _c.c_int, _vp, _vp, _vp, _vp, _vp, _sz,
                                           _vp]),
    "sv_verify_tree": (_c.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _u64, _u32, _vp, _c.c_int,
                                  _c.c_int, _c.c_int, _c.c_int, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sv_vocab_chunks": (_c.c_int, [_c.c_int, _c.c_int, _c.POINTER(_c.c_int), _c.POINTER(_c.c_int)]),
    "sv_verify_regions": (_c.c_int, [_c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.POINTER(_sz), _c.POINTER(_sz),
                                     _c.POINTER(_sz), _c.POINTER(_sz), _c.POINTER(_sz)]),
    "sv_verify_sample_phase": (_c.c_int, [_vp, _i64, _vp, _i64, _vp, _vp, _u64, _u32, _vp, _c.c_int, _c.c_int,
                                          _c.c_int, _c.c_int, _c.c_int, _c.c_int, _c.c_int, _vp, _vp, _vp, _vp,
                                          _vp, _vp, _sz, _vp]),
    "sv_sample_workspace_size": (_sz, [_c.c_int, _c.c_int]),
    "sv_sample_rows": (_c.c_int, [_vp, _i64, _c.c_int, _c.c_int, _c.c_int, _vp, _vp, _vp, _vp, _vp, _c.c_int, _vp, _vp,
                                  _vp, _i64, _vp, _sz, _vp]),
    "sv_cache_reserve": (_c.c_int, [_vp, _vp, _c.c_int, _vp, _vp, _c.c_int, _vp, _vp, _sz, _vp]),
    "sv_cache_append": (_c.c_int, [_vp, _c.c_int, _c.c_int, _vp, _c.c_int, _vp, _vp, _i64, _vp, _vp, _i64, _i64, _c.c_int,
                                   _vp, _sz, _vp]),
    "sv_cache_commit": (_c.c_int, [_vp, _vp, _c.c_int, _vp, _vp, _vp, _vp, _c.c_int, _c.c_int, _vp, _vp, _sz, _vp]),
    "sv_cache_fork": (_c.c_int, [_vp, _vp, _c.c_int, _c.c_int, _vp, _vp, _vp, _c.c_int, _vp, _vp, _sz, _vp]),
    "sv_cache_release": (_c.c_int, [_vp, _vp, _c.c_int, _c.c_int, _vp, _vp, _c.c_int, _vp, _sz, _vp]),
    "sv_attention_workspace_size": (_sz, [_vp, _c.c_int]),
    "sv_tree_attention": (_c.c_int, [_vp, _c.c_int, _vp, _i64, _i64, _c.c_int, _vp, _c.c_int, _vp, _vp, _i64, _vp, _c.c_int,
                                     _c.c_int, _f32, _c.c_int, _c.c_int, _vp, _i64, _i64, _vp, _vp, _sz, _vp]),
    "sv_test_stall_next_verify": (None, [_c.c_int]),
    "sv_query_status": (_c.c_int, [_vp, _vp, _c.POINTER(_u32)]),
    "sv_status_string": (_c.c_char_p, [_c.c_int]),
    "sv_last_error_string": (_c.c_char_p, []),
    "sv_profile_enable": (None, [_c.c_int]),
    "sv_profile_collect": (_c.c_int, [_c.POINTER(_c.c_double), _c.POINTER(_i64)]),
    "sv_profile_collect_ids": (_c.c_int, [_c.POINTER(_c.c_double), _c.POINTER(_i64), _c.c_int]),
    "sv_profile_reset": (None, []),
    "sv_launch_count": (_i64, []),
}

_lib = None


class sv_cache(_c.Structure):
    """The C struct of the same name: a paged key/value cache (see include/sv.h)."""
    _fields_ = [("k", _vp), ("v", _vp), ("layer_stride", _i64), ("page_stride", _i64), ("slot_stride", _i64),
                ("head_stride", _i64), ("layers", _i32), ("pages", _i32), ("page_size", _i32), ("kv_heads", _i32),
                ("head_dim", _i32), ("page_refs", _vp)]


class SVError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"libsv status {status}: {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libsv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() (nvcc, sm_103a)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def header_symbols() -> list[str]:
    """Function names declared in include/sv.h."""
    with open(HEADER) as f:
        txt = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[\w\s\*]*?\b(sv_\w+)\s*\(", txt, re.M)))


def _check(status: int) -> None:
    if status != SV_OK:
        L = lib()
        raise SVError(status, L.sv_last_error_string().decode() or L.sv_status_string(status).decode())


def _p(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("libsv takes device tensors")
    return t.data_ptr()


def _need(t, name: str, dtype, count: int = 0) -> None:
    """Host check of one array argument before its pointer reaches the kernels: its dtype, and
    at least `count` elements of its storage from its data pointer on (the kernels index past
    a view's shape when a stride says so).  Raw integer pointers are the caller's affair."""
    if t is None or isinstance(t, int):
        return
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if count > 0 and not (count <= t.numel() and t.is_contiguous()):  # (a contiguous tensor holds its elements)
        avail = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
        if avail < count:
            raise ValueError(f"{name} holds {avail} elements from its data pointer, the call reads {count}")


def _logit_dtype(dt: int):
    return {SV_BF16: torch.bfloat16, SV_F32: torch.float32}.get(dt)


def _need_rows(t, name: str, dt: int, rows: int, stride: int, V: int) -> None:
    """Logit rows: rows x V elements at the given row stride."""
    _need(t, name, _logit_dtype(dt), (rows - 1) * stride + V if rows > 0 and stride >= V > 0 else 0)


def _ws_bytes(ws) -> int:
    return 0 if ws is None else ws.numel() * ws.element_size()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():  # without building a Stream object
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float32:
        return SV_F32
    raise ValueError(f"logits must be bfloat16 or float32, got {t.dtype}")


# ------------------------------------------------------------------------------------------
# one-to-one C ABI (tensors for pointers, None for NULL); each raises SVError on failure
# ------------------------------------------------------------------------------------------

def sv_workspace_size(op: int, B: int, Kmax: int, V: int, dt: int) -> int:
    return int(lib().sv_workspace_size(op, B, Kmax, V, dt))


def sv_verify_greedy(target, t_row_stride, draft, d_row_stride, draft_tokens, dt, B, K, V, out_tokens,
                     out_accept_len, ws, stream=None) -> None:
    if B > 0 and K >= 0:
        _need_rows(target, "target", dt, B * (K + 1), t_row_stride, V)
        _need_rows(draft, "draft", dt, B * K, d_row_stride, V)
        _need(draft_tokens, "draft_tokens", torch.int32, B * K)
        _need(out_tokens, "out_tokens", torch.int32, B * (K + 1))
        _need(out_accept_len, "out_accept_len", torch.int32, B)
    _check(lib().sv_verify_greedy(_p(target), t_row_stride, _p(draft), d_row_stride, _p(draft_tokens), dt, B,
                                  K, V, _p(out_tokens), _p(out_accept_len), _p(ws),
                                  _ws_bytes(ws), _stream(stream)))


def sv_verify_sample(target, t_row_stride, draft, d_row_stride, draft_tokens, temperature, seed, round_,
                     request_ids, dt, B, K, V, out_tokens, out_accept_len, out_p, out_q, out_flags, ws,
                     stream=None) -> None:
    if B > 0 and K >= 0:
        _need_rows(target, "target", dt, B * (K + 1), t_row_stride, V)
        _need_rows(draft, "draft", dt, B * K, d_row_stride, V)
        _need(draft_tokens, "draft_tokens", torch.int32, B * K)
        _need(temperature, "temperature", torch.float32, B)
        _need(request_ids, "request_ids", torch.int32, B)
        _need(out_tokens, "out_tokens", torch.int32, B * (K + 1))
        _need(out_accept_len, "out_accept_len", torch.int32, B)
        _need(out_p, "out_p", torch.float32, B * K)
        _need(out_q, "out_q", torch.float32, B * K)
        _need(out_flags, "out_flags", torch.uint8, B)
    _check(lib().sv_verify_sample(_p(target), t_row_stride, _p(draft), d_row_stride, _p(draft_tokens),
                                  _p(temperature), seed & (2 ** 64 - 1), round_, _p(request_ids), dt, B, K, V,
                                  _p(out_tokens), _p(out_accept_len), _p(out_p), _p(out_q), _p(out_flags),
                                  _p(ws), _ws_bytes(ws), _stream(stream)))


def sv_verify_ragged(target, t_row_stride, t_row_offsets, t_rows, draft, d_row_stride, d_row_offsets, d_rows,
                     draft_tokens, tok_stride, keep_len, temperature, seed, round_, request_ids, dt, B, Kmax, V,
                     out_tokens, out_accept_len, out_p, out_q, out_flags, ws, stream=None) -> None:
    if B > 0 and Kmax >= 0:
        # the packed arrays hold t_rows / d_rows rows; the kernels bound every request's rows by them
        _need_rows(target, "target", dt, t_rows, t_row_stride, V)
        if draft is not None:
            _need_rows(draft, "draft", dt, d_rows, d_row_stride, V)
        _need(t_row_offsets, "t_row_offsets", torch.int32, B + 1)
        _need(d_row_offsets, "d_row_offsets", torch.int32, B + 1)
        _need(draft_tokens, "draft_tokens", torch.int32,
              (B - 1) * tok_stride + Kmax if Kmax > 0 and tok_stride >= Kmax else 0)
        _need(keep_len, "keep_len", torch.int32, B)
        _need(temperature, "temperature", torch.float32, B)
        _need(request_ids, "request_ids", torch.int32, B)
        _need(out_tokens, "out_tokens", torch.int32, B * (Kmax + 1))
        _need(out_accept_len, "out_accept_len", torch.int32, B)
        _need(out_p, "out_p", torch.float32, B * Kmax)
        _need(out_q, "out_q", torch.float32, B * Kmax)
        _need(out_flags, "out_flags", torch.uint8, B)
    _check(lib().sv_verify_ragged(_p(target), t_row_stride, _p(t_row_offsets), t_rows, _p(draft), d_row_stride,
                                  _p(d_row_offsets), d_rows, _p(draft_tokens), tok_stride, _p(keep_len),
                                  _p(temperature), seed & (2 ** 64 - 1), round_, _p(request_ids), dt, B, Kmax,
                                  V, _p(out_tokens), _p(out_accept_len), _p(out_p), _p(out_q), _p(out_flags),
                                  _p(ws), _ws_bytes(ws), _stream(stream)))


def sv_verify_sample_noalloc(target, t_row_stride, draft, d_row_stride, draft_tokens, temperature, seed, round_,
                             request_ids, dt, B, K, V, out_tokens, out_accept_len, out_p, out_q, out_flags,
                             stream=None) -> None:
    """sv_verify_sample on the library's built-in scratch (no workspace argument)."""
    if B > 0 and K >= 0:
        _need_rows(target, "target", dt, B * (K + 1), t_row_stride, V)
        _need_rows(draft, "draft", dt, B * K, d_row_stride, V)
        _need(draft_tokens, "draft_tokens", torch.int32, B * K)
        _need(temperature, "temperature", torch.float32, B)
        _need(request_ids, "request_ids", torch.int32, B)
        _need(out_tokens, "out_tokens", torch.int32, B * (K + 1))
        _need(out_accept_len, "out_accept_len", torch.int32, B)
        _need(out_p, "out_p", torch.float32, B * K)
        _need(out_q, "out_q", torch.float32, B * K)
        _need(out_flags, "out_flags", torch.uint8, B)
    _check(lib().sv_verify_sample_noalloc(_p(target), t_row_stride, _p(draft), d_row_stride, _p(draft_tokens),
                                          _p(temperature), seed & (2 ** 64 - 1), round_, _p(request_ids), dt, B,
                                          K, V, _p(out_tokens), _p(out_accept_len), _p(out_p), _p(out_q),
                                          _p(out_flags), _stream(stream)))


def sv_schedule_depth(alpha, alpha_stride, draft_len, B, Dmax, cost_a, cost_b, budget, ratios, objective,
                      out_keep_len, out_row_offsets, out_total_K, out_utility_q48, ws, stream=None) -> None:
    if B > 0 and Dmax >= 0:
        _need(alpha, "alpha", torch.float32, (B - 1) * alpha_stride + Dmax if Dmax > 0 and alpha_stride >= Dmax else 0)
        _need(draft_len, "draft_len", torch.int32, B)
        _need(out_keep_len, "out_keep_len", torch.int32, B)
        _need(out_row_offsets, "out_row_offsets", torch.int32, B + 1)
        _need(out_total_K, "out_total_K", torch.int32, 1)
        _need(out_utility_q48, "out_utility_q48", torch.int64, 1)
    rat = None
    n = 0
    if ratios is not None:
        n = len(ratios)
        rat = (ctypes.c_float * n)(*[float(r) for r in ratios])
    _check(lib().sv_schedule_depth(_p(alpha), alpha_stride, _p(draft_len), B, Dmax, float(cost_a),
                                   float(cost_b), budget, ctypes.cast(rat, ctypes.c_void_p) if rat else None,
                                   n, objective, _p(out_keep_len), _p(out_row_offsets), _p(out_total_K),
                                   _p(out_utility_q48), _p(ws), _ws_bytes(ws),
                                   _stream(stream)))


def sv_schedule_depth_table(alpha, alpha_stride, draft_len, B, Dmax, cost_K, cost_c, budget, ratios, objective,
                            out_keep_len, out_row_offsets, out_total_K, out_utility_q48, ws, stream=None) -> None:
    if B > 0 and Dmax >= 0:
        _need(alpha, "alpha", torch.float32, (B - 1) * alpha_stride + Dmax if Dmax > 0 and alpha_stride >= Dmax else 0)
        _need(draft_len, "draft_len", torch.int32, B)
        _need(out_keep_len, "out_keep_len", torch.int32, B)
        _need(out_row_offsets, "out_row_offsets", torch.int32, B + 1)
        _need(out_total_K, "out_total_K", torch.int32, 1)
        _need(out_utility_q48, "out_utility_q48", torch.int64, 1)
    rat = None
    n = 0
    if ratios is not None:
        n = len(ratios)
        rat = (ctypes.c_float * n)(*[float(r) for r in ratios])
    nk = len(cost_K)
    if len(cost_c) != nk:
        raise SVError(SV_ERR_INVALID_ARG, "cost_K and cost_c differ in length")
    ks = (ctypes.c_int32 * max(nk, 1))(*[int(k) for k in cost_K])
    cs = (ctypes.c_double * max(nk, 1))(*[float(c) for c in cost_c])
    _check(lib().sv_schedule_depth_table(_p(alpha), alpha_stride, _p(draft_len), B, Dmax,
                                         ctypes.cast(ks, ctypes.c_void_p), ctypes.cast(cs, ctypes.c_void_p), nk,
                                         budget, ctypes.cast(rat, ctypes.c_void_p) if rat else None, n, objective,
                                         _p(out_keep_len), _p(out_row_offsets), _p(out_total_K),
                                         _p(out_utility_q48), _p(ws), _ws_bytes(ws),
                                         _stream(stream)))


def sv_verify_tree(target, t_row_stride, draft, d_row_stride, node_offsets, n_rows, parent, tokens, temperature,
                   seed, round_, request_ids, dt, B, Nmax, V, out_path, out_tokens, out_accept_len, out_flags, ws,
                   stream=None) -> None:
    if B > 0:
        # the packed arrays hold n_rows rows; the kernels bound every request's rows by it
        _need_rows(target, "target", dt, n_rows, t_row_stride, V)
        if draft is not None:
            _need_rows(draft, "draft", dt, n_rows, d_row_stride, V)
        _need(node_offsets, "node_offsets", torch.int32, B + 1)
        _need(parent, "parent", torch.int32, n_rows)
        _need(tokens, "tokens", torch.int32, n_rows)
        _need(temperature, "temperature", torch.float32, B)
        _need(request_ids, "request_ids", torch.int32, B)
        _need(out_path, "out_path", torch.int32, B * Nmax)
        _need(out_tokens, "out_tokens", torch.int32, B * Nmax)
        _need(out_accept_len, "out_accept_len", torch.int32, B)
        _need(out_flags, "out_flags", torch.uint8, B)
    _check(lib().sv_verify_tree(_p(target), t_row_stride, _p(draft), d_row_stride, _p(node_offsets), n_rows,
                                _p(parent), _p(tokens), _p(temperature), seed & (2 ** 64 - 1), round_,
                                _p(request_ids), dt, B, Nmax, V, _p(out_path), _p(out_tokens), _p(out_accept_len),
                                _p(out_flags), _p(ws), _ws_bytes(ws), _stream(stream)))


def sv_vocab_chunks(V: int, dt: int) -> tuple[int, int]:
    cl, nc = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().sv_vocab_chunks(V, dt, ctypes.byref(cl), ctypes.byref(nc)))
    return cl.value, nc.value


def sv_verify_regions(B: int, K: int, V: int, dt: int) -> dict:
    """Workspace byte offsets and sizes of the chunk records and the two range-sum arrays."""
    v = [ctypes.c_size_t(0) for _ in range(5)]
    _check(lib().sv_verify_regions(B, K, V, dt, *(ctypes.byref(x) for x in v)))
    return {"rec_offset": v[0].value, "rec_bytes": v[1].value, "mass_offset": v[2].value,
            "mass_p_offset": v[3].value, "mass_bytes": v[4].value}


def sv_verify_sample_phase(target, t_row_stride, draft, d_row_stride, draft_tokens, temperature, seed, round_,
                           request_ids, dt, B, K, V, c_begin, c_end, phase, out_tokens, out_accept_len, out_p,
                           out_q, out_flags, ws, stream=None) -> None:
    if B > 0 and K >= 0:
        # the arrays hold the shard's columns: those of chunks [c_begin, c_end)
        cl, nc = sv_vocab_chunks(V, dt)
        v_local = min(V, c_end * cl) - c_begin * cl if 0 <= c_begin < c_end <= nc else 0
        _need_rows(target, "target", dt, B * (K + 1), t_row_stride, v_local)
        _need_rows(draft, "draft", dt, B * K, d_row_stride, v_local)
        _need(draft_tokens, "draft_tokens", torch.int32, B * K)
        _need(temperature, "temperature", torch.float32, B)
        _need(request_ids, "request_ids", torch.int32, B)
        _need(out_tokens, "out_tokens", torch.int32, B * (K + 1))
        _need(out_accept_len, "out_accept_len", torch.int32, B)
        _need(out_p, "out_p", torch.float32, B * K)
        _need(out_q, "out_q", torch.float32, B * K)
        _need(out_flags, "out_flags", torch.uint8, B)
    _check(lib().sv_verify_sample_phase(_p(target), t_row_stride, _p(draft), d_row_stride, _p(draft_tokens),
                                        _p(temperature), seed & (2 ** 64 - 1), round_, _p(request_ids), dt, B, K, V,
                                        c_begin, c_end, phase, _p(out_tokens), _p(out_accept_len), _p(out_p),
                                        _p(out_q), _p(out_flags), _p(ws), _ws_bytes(ws), _stream(stream)))


def sv_sample_workspace_size(R: int, V: int) -> int:
    return int(lib().sv_sample_workspace_size(R, V))


def sv_sample_rows(logits, row_stride, dt, R, V, temperature, top_k, top_p, min_p, uniforms, M, out_tokens, out_probs,
                   out_rows, out_stride, ws, stream=None) -> None:
    if R > 0:
        _need_rows(logits, "logits", dt, R, row_stride, V)
        _need(temperature, "temperature", torch.float32, R)
        _need(top_k, "top_k", torch.int32, R)
        _need(top_p, "top_p", torch.float32, R)
        _need(min_p, "min_p", torch.float32, R)
        _need(uniforms, "uniforms", torch.float32, R * M)
        _need(out_tokens, "out_tokens", torch.int32, R * M)
        _need(out_probs, "out_probs", torch.float32, R * M)
        _need_rows(out_rows, "out_rows", dt, R, out_stride, V)
    _check(lib().sv_sample_rows(_p(logits), row_stride, dt, R, V, _p(temperature), _p(top_k), _p(top_p), _p(min_p),
                                _p(uniforms), M, _p(out_tokens), _p(out_probs), _p(out_rows), out_stride, _p(ws),
                                _ws_bytes(ws), _stream(stream)))


def _need_table(page_table, table_width: int, rows: int, **per_row) -> None:
    _need(page_table, "page_table", torch.int32, rows * table_width if table_width > 0 else 0)
    for name, t in per_row.items():
        _need(t, name, torch.int32, rows)


def sv_cache_reserve(cache, page_table, table_width, seq_len, extra, B, out_ok, ws, stream=None) -> None:
    if B > 0:
        _need_table(page_table, table_width, B, seq_len=seq_len, extra=extra, out_ok=out_ok)
    _check(lib().sv_cache_reserve(_c.addressof(cache), _p(page_table), table_width, _p(seq_len), _p(extra), B, _p(out_ok),
                                  _p(ws), _ws_bytes(ws), _stream(stream)))


def sv_cache_append(cache, layer, layers, page_table, table_width, seq_len, node_offsets, n_rows, k_new, v_new,
                    new_layer_stride, new_row_stride, B, ws, stream=None) -> None:
    if B > 0 and layers > 0 and n_rows > 0:
        _need_table(page_table, table_width, B, seq_len=seq_len)
        _need(node_offsets, "node_offsets", torch.int32, B + 1)
        last = (layers - 1) * new_layer_stride + (n_rows - 1) * new_row_stride + cache.kv_heads * cache.head_dim
        _need(k_new, "k_new", torch.bfloat16, last)
        _need(v_new, "v_new", torch.bfloat16, last)
    _check(lib().sv_cache_append(_c.addressof(cache), layer, layers, _p(page_table), table_width, _p(seq_len),
                                 _p(node_offsets), n_rows, _p(k_new), _p(v_new), new_layer_stride, new_row_stride, B,
                                 _p(ws), _ws_bytes(ws), _stream(stream)))


def sv_cache_commit(cache, page_table, table_width, seq_len, node_offsets, path, accept_len, B, Nmax, out_len, ws,
                    stream=None) -> None:
    if B > 0:
        _need_table(page_table, table_width, B, seq_len=seq_len, accept_len=accept_len, out_len=out_len)
        _need(node_offsets, "node_offsets", torch.int32, B + 1)
        _need(path, "path", torch.int32, B * Nmax)
    _check(lib().sv_cache_commit(_c.addressof(cache), _p(page_table), table_width, _p(seq_len), _p(node_offsets), _p(path),
                                 _p(accept_len), B, Nmax, _p(out_len), _p(ws), _ws_bytes(ws), _stream(stream)))


def sv_cache_fork(cache, page_table, table_width, rows, seq_len, src, dst, n, out_ok, ws, stream=None) -> None:
    if n > 0:
        _need_table(page_table, table_width, rows, seq_len=seq_len)
        _need(src, "src", torch.int32, n)
        _need(dst, "dst", torch.int32, n)
        _need(out_ok, "out_ok", torch.int32, n)
    _check(lib().sv_cache_fork(_c.addressof(cache), _p(page_table), table_width, rows, _p(seq_len), _p(src), _p(dst), n,
                               _p(out_ok), _p(ws), _ws_bytes(ws), _stream(stream)))


def sv_cache_release(cache, page_table, table_width, rows, seq_len, seqs, n, ws, stream=None) -> None:
    if n > 0:
        _need_table(page_table, table_width, rows, seq_len=seq_len)
        _need(seqs, "seqs", torch.int32, n)
    _check(lib().sv_cache_release(_c.addressof(cache), _p(page_table), table_width, rows, _p(seq_len), _p(seqs), n, _p(ws),
                                  _ws_bytes(ws), _stream(stream)))


def sv_attention_workspace_size(cache, q_heads: int) -> int:
    return int(lib().sv_attention_workspace_size(_c.addressof(cache), q_heads))


def sv_tree_attention(cache, layer, q, q_row_stride, q_head_stride, q_heads, page_table, table_width, seq_len,
                      node_offsets, n_rows, parent, B, Nmax, scale, window, sinks, out, out_row_stride,
                      out_head_stride, out_lse, ws, stream=None) -> None:
    if B > 0 and n_rows > 0:
        _need_table(page_table, table_width, B, seq_len=seq_len)
        _need(node_offsets, "node_offsets", torch.int32, B + 1)
        _need(parent, "parent", torch.int32, n_rows)
        _need(q, "q", torch.bfloat16, (n_rows - 1) * q_row_stride + (q_heads - 1) * q_head_stride + cache.head_dim)
        _need(out, "out", torch.bfloat16, (n_rows - 1) * out_row_stride + (q_heads - 1) * out_head_stride + cache.head_dim)
        _need(out_lse, "out_lse", torch.float32, n_rows * q_heads)
    _check(lib().sv_tree_attention(_c.addressof(cache), layer, _p(q), q_row_stride, q_head_stride, q_heads,
                                   _p(page_table), table_width, _p(seq_len), _p(node_offsets), n_rows, _p(parent), B,
                                   Nmax, scale, window, sinks, _p(out), out_row_stride, out_head_stride, _p(out_lse),
                                   _p(ws), _ws_bytes(ws), _stream(stream)))


def sv_test_stall_next_verify(wait_limit_ms: int) -> None:
    lib().sv_test_stall_next_verify(int(wait_limit_ms))


def sv_query_status(ws, stream=None) -> tuple[int, int]:
    v = ctypes.c_uint32(0)
    st = lib().sv_query_status(_p(ws), _stream(stream), ctypes.byref(v))
    if st not in (SV_OK, SV_ERR_DEVICE_INPUT, SV_ERR_TIMEOUT):
        _check(st)
    return st, int(v.value)


def sv_profile_enable(on: bool) -> None:
    lib().sv_profile_enable(1 if on else 0)


def sv_profile_collect() -> tuple[list[float], list[int]]:
    ms = (ctypes.c_double * SV_NUM_KERNELS)()
    n = (ctypes.c_int64 * SV_NUM_KERNELS)()
    _check(lib().sv_profile_collect(ms, n))
    return list(ms), list(n)


def sv_profile_collect_ids(n: int = SV_NUM_KERNEL_IDS) -> tuple[list[float], list[int]]:
    ms = (ctypes.c_double * n)()
    launches = (ctypes.c_int64 * n)()
    _check(lib().sv_profile_collect_ids(ms, launches, n))
    return list(ms), list(launches)


def sv_profile_reset() -> None:
    lib().sv_profile_reset()


def sv_launch_count() -> int:
    return int(lib().sv_launch_count())


# ------------------------------------------------------------------------------------------
# convenience wrappers
# ------------------------------------------------------------------------------------------

def _side_stream(stream, device) -> torch.cuda.Stream:
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream(stream), device=device)


def _empty(shape, dtype, device, stream=None) -> torch.Tensor:
    """A new tensor for a call on `stream` to write.  It comes from that stream's memory, so whatever the block was used for
    before is done when the call runs (a block of the current stream's may still be waited for there), and it goes back
    only when the current stream, on which the caller may read it, is done with it too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    s, now = _side_stream(stream, device), torch.cuda.current_stream(device)
    with torch.cuda.stream(s):
        t = torch.empty(shape, dtype=dtype, device=device)
    if s != now:
        t.record_stream(now)
    return t


def _workspace(nbytes: int, device, stream=None, zeros=False) -> torch.Tensor:
    """A workspace whose first SV_STATUS_BYTES (or all) are zero, from the memory of `stream` and the fill ordered before a
    call on it."""
    if stream is not None:
        with torch.cuda.stream(_side_stream(stream, device)):
            return _workspace(nbytes, device, zeros=zeros)
    if zeros:
        return torch.zeros(nbytes, dtype=torch.uint8, device=device)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:SV_STATUS_BYTES] = 0
    return ws


def workspace(op: int, B: int, Kmax: int, V: int, dt: int, device="cuda", stream=None) -> torch.Tensor:
    """Zero-filled workspace (torch allocations are 512-byte aligned) for calls on `stream` (None: the current one)."""
    n = sv_workspace_size(op, B, Kmax, V, dt)
    if n == 0:
        raise ValueError("invalid sizes for sv_workspace_size")
    return _workspace(n, device, stream, zeros=True)


def _rows(x: torch.Tensor):
    """(base tensor, row stride) for [..., V] logits with a contiguous last dimension."""
    if x.numel() == 0:
        return x, x.shape[-1]
    if x.stride(-1) != 1:
        raise ValueError("logit rows must be contiguous")
    return x, (x.stride(-2) if x.dim() >= 2 else x.shape[-1])


def num_rows(x: torch.Tensor) -> int:
    """Rows of V logits in a [..., V] tensor."""
    return x.numel() // x.shape[-1] if x.shape[-1] > 0 else 0


def verify_greedy(target, K, *, draft=None, draft_tokens=None, ws=None, stream=None):
    """target [B*(K+1), V] (or [B, K+1, V]); draft [B*K, V] or draft_tokens [B, K]."""
    V = target.shape[-1]
    B = target.numel() // V // (K + 1)
    dt = _dt(target)
    _, ts = _rows(target)
    ds = _rows(draft)[1] if draft is not None else V
    out_tok = _empty((B, K + 1), torch.int32, target.device, stream)
    out_len = _empty(B, torch.int32, target.device, stream)
    if ws is None:
        ws = workspace(SV_OP_VERIFY, B, K, V, dt, target.device, stream)
    sv_verify_greedy(target, ts, draft, ds, draft_tokens, dt, B, K, V, out_tok, out_len, ws, stream)
    return out_tok, out_len


def verify_sample(target, draft, draft_tokens, temperature, K, *, seed=0, round_=0, request_ids=None,
                  ws=None, stream=None, want_pq=True):
    V = target.shape[-1]
    B = target.numel() // V // (K + 1)
    dt = _dt(target)
    dev = target.device
    out_tok = _empty((B, K + 1), torch.int32, dev, stream)
    out_len = _empty(B, torch.int32, dev, stream)
    out_p = _empty((B, K), torch.float32, dev, stream) if want_pq else None
    out_q = _empty((B, K), torch.float32, dev, stream) if want_pq else None
    out_f = _empty(B, torch.uint8, dev, stream)
    if ws is None:
        ws = workspace(SV_OP_VERIFY, B, K, V, dt, dev, stream)
    ds = _rows(draft)[1] if draft is not None else V
    sv_verify_sample(target, _rows(target)[1], draft, ds, draft_tokens, temperature, seed, round_, request_ids,
                     dt, B, K, V, out_tok, out_len, out_p, out_q, out_f, ws, stream)
    return out_tok, out_len, out_p, out_q, out_f


def verify_tree(target, draft, node_offsets, parent, tokens, temperature, Nmax, *, seed=0, round_=0,
                request_ids=None, ws=None, stream=None, out=None):
    """Token-tree verification.  target / draft [rows, V]: node c of request i is row
    node_offsets[i] + c; parent / tokens [rows] int32 per node; temperature [B].  Returns
    (path [B, Nmax], tokens [B, Nmax], accept_len [B], flags [B])."""
    V = target.shape[-1]
    B = node_offsets.numel() - 1
    dt = _dt(target)
    dev = target.device
    if out is None:
        out = (_empty((B, Nmax), torch.int32, dev, stream),
               _empty((B, Nmax), torch.int32, dev, stream),
               _empty(B, torch.int32, dev, stream),
               _empty(B, torch.uint8, dev, stream))
    if ws is None:
        ws = workspace(SV_OP_TREE, B, Nmax, V, dt, dev, stream)
    ds = _rows(draft)[1] if draft is not None else V
    sv_verify_tree(target, _rows(target)[1], draft, ds, node_offsets, num_rows(target), parent, tokens, temperature,
                   seed, round_, request_ids, dt, B, Nmax, V, *out, ws, stream)
    return out


def verify_ragged(target, t_row_offsets, draft, d_row_offsets, draft_tokens, keep_len, temperature, Kmax, *,
                  seed=0, round_=0, request_ids=None, ws=None, stream=None, want_pq=True, out=None):
    V = target.shape[-1]
    B = keep_len.numel()
    dt = _dt(target)
    dev = target.device
    if out is None:
        out = (_empty((B, Kmax + 1), torch.int32, dev, stream),
               _empty(B, torch.int32, dev, stream),
               _empty((B, Kmax), torch.float32, dev, stream) if want_pq else None,
               _empty((B, Kmax), torch.float32, dev, stream) if want_pq else None,
               _empty(B, torch.uint8, dev, stream))
    if ws is None:
        ws = workspace(SV_OP_VERIFY, B, Kmax, V, dt, dev, stream)
    ds = _rows(draft)[1] if draft is not None else V
    ts_ = draft_tokens.stride(0) if draft_tokens is not None else Kmax
    sv_verify_ragged(target, _rows(target)[1], t_row_offsets, num_rows(target), draft, ds, d_row_offsets,
                     num_rows(draft) if draft is not None else 0, draft_tokens, ts_, keep_len, temperature, seed,
                     round_, request_ids, dt, B, Kmax, V, *out, ws, stream)
    return out


def schedule_depth(alpha, cost_a, cost_b, budget, *, draft_len=None, ratios=None, objective=SV_OBJ_THROUGHPUT,
                   ws=None, stream=None, out=None, cost_table=None):
    """alpha [B, Dmax] float32 (device).  Returns (keep_len [B], row_offsets [B+1], total_K [1], U_q48 [1]).
    cost_table = (token counts, latencies), e.g. from cost_table.profile_cost_table, replaces the linear
    cost cost_a + cost_b * K (sv_schedule_depth_table)."""
    B, Dmax = alpha.shape
    dev = alpha.device
    if out is None:
        out = (_empty(B, torch.int32, dev, stream), _empty(B + 1, torch.int32, dev, stream),
               _empty(1, torch.int32, dev, stream), _empty(1, torch.int64, dev, stream))
    if ws is None:
        ws = workspace(SV_OP_SCHEDULE, B, Dmax, 1, SV_F32, dev, stream)
    if cost_table is not None:
        sv_schedule_depth_table(alpha, alpha.stride(0), draft_len, B, Dmax, cost_table[0], cost_table[1], budget,
                                ratios, objective, *out, ws, stream)
    else:
        sv_schedule_depth(alpha, alpha.stride(0), draft_len, B, Dmax, cost_a, cost_b, budget, ratios, objective,
                          *out, ws, stream)
    return out


# ------------------------------------------------------------------------------------------
# the round around verification: sampling, the paged cache, tree attention
# ------------------------------------------------------------------------------------------

def _array(t, name: str, dtype, count: int) -> int | None:
    """Pointer of a contiguous device array of at least `count` elements (None = NULL)."""
    if t is None:
        return None
    if t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.numel() >= count:
        return t.data_ptr()
    _need(t, name, dtype, count)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < count:
        raise ValueError(f"{name} holds {t.numel()} elements, the call reads {count}")
    return _p(t)


def _row_stride(x: torch.Tensor) -> int:
    """Row stride of logits [R, V].  A row's logits have to lie side by side however many rows there are; a dimension of
    size 1 is never stepped along, and its stride may be any."""
    R, V = x.shape
    if V > 1 and R > 0 and x.stride(1) != 1:
        raise ValueError("logit rows must be contiguous")
    return x.stride(0) if R > 1 else V


def sample_workspace(rows: int, vocab: int, device="cuda") -> torch.Tensor:
    """Workspace of sample() for that many rows (its first word is the device status word)."""
    n = sv_sample_workspace_size(rows, vocab)
    if n == 0:
        raise ValueError("invalid sizes for sv_sample_workspace_size")
    return _workspace(n, device)


def sample(logits, temperature, uniforms, *, top_k=None, top_p=None, min_p=None, probs=True, filtered=None, out=None,
           ws=None, stream=None):
    """Draws from rows of logits.  logits [R, V] (bf16 or float32; rows may be strided); temperature [R]
    float32; uniforms [R, M] float32 in [0, 1); top_k [R] int32, top_p / min_p [R] float32 or None.  filtered: None,
    True, or a tensor like logits (it may be logits itself) that receives the rows with everything that cannot be
    drawn set to -inf: these are the rows to verify with.  Returns (tokens [R, M] int32, probs [R, M] float32 or None,
    filtered or None); out = (tokens, probs) takes the place of new tensors."""
    if logits.dim() != 2 or uniforms.dim() != 2 or uniforms.shape[0] != logits.shape[0]:
        raise ValueError("sample() takes logits [R, V] and uniforms [R, M]")
    R, V = logits.shape
    M = uniforms.shape[1]
    dt = _dt(logits)
    dev = logits.device
    if out is None:
        out = (_empty((R, M), torch.int32, dev, stream),
               _empty((R, M), torch.float32, dev, stream) if probs else None)
    row_stride = _row_stride(logits)
    out_stride = V
    if filtered is not None:
        if filtered is True:
            filtered = _empty((R, V), logits.dtype, dev, stream)
        if filtered.shape != logits.shape or filtered.dtype != logits.dtype:
            raise ValueError("filtered must have the shape and type of logits")
        out_stride = _row_stride(filtered)
    if ws is None:
        ws = _workspace(sv_sample_workspace_size(R, V), dev, stream)
    n = R * M
    f32, i32 = torch.float32, torch.int32
    _check((_lib or lib()).sv_sample_rows(
        _p(logits), row_stride, dt, R, V, _array(temperature, "temperature", f32, R), _array(top_k, "top_k", i32, R),
        _array(top_p, "top_p", f32, R), _array(min_p, "min_p", f32, R), _array(uniforms, "uniforms", f32, n), M,
        _array(out[0], "tokens", i32, n), _array(out[1], "probs", f32, n), _p(filtered), out_stride, _p(ws), _ws_bytes(ws),
        _stream(stream)))
    return out[0], out[1], filtered


class PagedCache:
    """A paged key/value cache on the device (the C struct sv_cache and the sequences' page table).

    k, v        [layers, pages, page_size, kv_heads, head_dim] bf16, the same strides, the last
                dimension contiguous (so [..., kv_heads, page_size, ...] pools come as transposed views)
    page_refs   [pages] int32, how many sequences hold a page (0 = free)
    page_table  [sequences, entries] int32, contiguous: a sequence's pages in order, then -1

    The methods take the sequences' lengths as a device tensor; they work on the table's first B rows, B
    from their arguments.  Everything stays on the device and on `stream`; errors that only the device sees go
    to the status word of `ws` (sv_query_status(cache.ws)).  One cache belongs to one stream at a time.
    """

    def __init__(self, k, v, page_refs, page_table, ws=None):
        if k.dim() != 5 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must be [layers, pages, page_size, kv_heads, head_dim] alike")
        _need(k, "k", torch.bfloat16)
        if k.stride(4) != 1:
            raise ValueError("the head dimension must be contiguous")
        if page_table.dim() != 2:
            raise ValueError("page_table must be [sequences, entries]")
        self.k, self.v, self.page_refs, self.page_table = k, v, page_refs, page_table
        self.rows, self.width = page_table.shape
        L, P, S, H, D = k.shape
        # a dimension of size 1 is never stepped along: its stride only has to be a valid one
        st = [k.stride(i) if k.shape[i] > 1 else max(8, D) for i in range(4)]
        self.kv_heads, self.head_dim = H, D
        self.c = sv_cache(k=_p(k), v=_p(v), layer_stride=st[0], page_stride=st[1], slot_stride=st[2], head_stride=st[3],
                          layers=L, pages=P, page_size=S, kv_heads=H, head_dim=D,
                          page_refs=_array(page_refs, "page_refs", torch.int32, P))
        self.ws = torch.zeros(SV_CACHE_WORKSPACE_BYTES, dtype=torch.uint8, device=k.device) if ws is None else ws
        # what every call passes: the struct, the table, the workspace
        self._c = _c.addressof(self.c)
        self._table = _array(page_table, "page_table", torch.int32, self.rows * self.width)
        self._ws, self._ws_bytes = _p(self.ws), _ws_bytes(self.ws)

    @classmethod
    def empty(cls, layers, pages, page_size, kv_heads, head_dim, sequences, entries, device="cuda"):
        """A cache of free pages and empty sequences."""
        shape = (layers, pages, page_size, kv_heads, head_dim)
        return cls(torch.zeros(shape, dtype=torch.bfloat16, device=device),
                   torch.zeros(shape, dtype=torch.bfloat16, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device),
                   torch.full((sequences, entries), -1, dtype=torch.int32, device=device))

    def _batch(self, B: int) -> int:
        if B > self.rows:
            raise ValueError(f"{B} requests, but the page table has {self.rows} rows")
        return B

    def reserve(self, seq_len, extra, *, ok=None, stream=None):
        """Pages for slots [0, seq_len + extra) of rows 0..B-1, B = extra.numel().  Returns ok [B] int32: 1 where
        served."""
        B = self._batch(extra.numel())
        i32 = torch.int32
        if ok is None:
            ok = _empty(B, i32, extra.device, stream)
        _check((_lib or lib()).sv_cache_reserve(
            self._c, self._table, self.width, _array(seq_len, "seq_len", i32, B), _array(extra, "extra", i32, B), B,
            _array(ok, "ok", i32, B), self._ws, self._ws_bytes, _stream(stream)))
        return ok

    def append(self, k_new, v_new, seq_len, node_offsets, layer=0, *, stream=None):
        """Writes the nodes' keys and values, [layers, rows, kv_heads, head_dim] from `layer` on or [rows, kv_heads,
        head_dim] for one layer: node c of request i (row node_offsets[i] + c) to slot seq_len[i] + c."""
        if k_new.dim() == 3:
            k_new, v_new = k_new.unsqueeze(0), v_new.unsqueeze(0)
        if k_new.dim() != 4 or k_new.shape != v_new.shape or k_new.shape[2] != self.kv_heads or k_new.shape[3] != self.head_dim:
            raise ValueError("k_new and v_new must be [layers, rows, kv_heads, head_dim] of this cache's heads")
        L, n, H, D = k_new.shape
        st = k_new.stride()
        if L * n and (st != v_new.stride() or st[3] != 1 or (H > 1 and st[2] != D)):
            raise ValueError("k_new and v_new need the same strides and contiguous [kv_heads, head_dim]")
        if k_new.dtype is not torch.bfloat16 or v_new.dtype is not torch.bfloat16:
            raise ValueError("k_new and v_new must be torch.bfloat16")
        B = self._batch(node_offsets.numel() - 1)
        i32 = torch.int32
        _check((_lib or lib()).sv_cache_append(
            self._c, layer, L, self._table, self.width, _array(seq_len, "seq_len", i32, B),
            _array(node_offsets, "node_offsets", i32, B + 1), n, _p(k_new), _p(v_new), st[0] if L > 1 else 0,
            st[1] if n > 1 else H * D, B, self._ws, self._ws_bytes, _stream(stream)))

    def commit(self, seq_len, node_offsets, path, accept_len, *, out_len=None, stream=None):
        """Keeps the accepted path (verify_tree's outputs path [B, Nmax] and accept_len [B]) in every layer and gives
        the pages past it back.  Returns the new lengths (written to out_len; it may be seq_len)."""
        if path.dim() != 2:
            raise ValueError("path must be [B, Nmax]")
        B, Nmax = path.shape
        self._batch(B)
        i32 = torch.int32
        if out_len is None:
            out_len = _empty(B, i32, path.device, stream)
        _check((_lib or lib()).sv_cache_commit(
            self._c, self._table, self.width, _array(seq_len, "seq_len", i32, B),
            _array(node_offsets, "node_offsets", i32, B + 1), _array(path, "path", i32, B * Nmax),
            _array(accept_len, "accept_len", i32, B), B, Nmax, _array(out_len, "out_len", i32, B), self._ws, self._ws_bytes,
            _stream(stream)))
        return out_len

    def fork(self, seq_len, src, dst, *, ok=None, stream=None):
        """Rows dst become copies of rows src (full pages shared); seq_len is updated.  Returns ok [n] int32."""
        n = src.numel()
        i32 = torch.int32
        if ok is None:
            ok = _empty(n, i32, src.device, stream)
        _check((_lib or lib()).sv_cache_fork(
            self._c, self._table, self.width, self.rows, _array(seq_len, "seq_len", i32, self.rows),
            _array(src, "src", i32, n), _array(dst, "dst", i32, n), n, _array(ok, "ok", i32, n), self._ws, self._ws_bytes,
            _stream(stream)))
        return ok

    def release(self, seq_len, seqs, *, stream=None):
        """Gives the pages of rows seqs back and empties them (seq_len = 0)."""
        n = seqs.numel()
        i32 = torch.int32
        _check((_lib or lib()).sv_cache_release(
            self._c, self._table, self.width, self.rows, _array(seq_len, "seq_len", i32, self.rows),
            _array(seqs, "seqs", i32, n), n, self._ws, self._ws_bytes, _stream(stream)))


def attention_workspace(cache: PagedCache, q_heads: int) -> torch.Tensor:
    """Workspace of tree_attention() on this cache (its first word is the device status word)."""
    return _workspace(attention_workspace_size(cache, q_heads), cache.k.device, zeros=True)


def attention_workspace_size(cache: PagedCache, q_heads: int) -> int:
    n = sv_attention_workspace_size(cache.c, q_heads)
    if n == 0:
        raise ValueError(lib().sv_last_error_string().decode() or "invalid sizes for sv_attention_workspace_size")
    return n


def tree_attention(q, cache: PagedCache, layer, seq_len, node_offsets, parent, Nmax, *, scale=None, window=0, sinks=0,
                   out=None, lse=True, ws=None, stream=None):
    """Attention of every request's token tree over its cached sequence in one layer.  q [rows, q_heads, head_dim]
    bf16, row node_offsets[i] + c for node c of request i, whose keys and values are in the cache at slot seq_len[i] +
    c (cache.append); parent [rows] int32 as in verify_tree, or None for chains; at most Nmax nodes a request.  window,
    sinks: a sliding window of that many positions and the first positions that stay visible.  Returns (out like q,
    lse [rows, q_heads] float32, or None with lse=False)."""
    bf16, i32 = torch.bfloat16, torch.int32
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError("q must be [rows, q_heads, head_dim] of the cache's head_dim")
    n, H, D = q.shape
    if out is None:
        out = _empty((n, H, D), bf16, q.device, stream)
    if out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    if q.dtype is not bf16 or out.dtype is not bf16:
        raise ValueError("q and out must be torch.bfloat16")
    if lse is True:
        lse = _empty((n, H), torch.float32, q.device, stream)
    elif lse is False:
        lse = None
    if ws is None:
        ws = _workspace(attention_workspace_size(cache, H), q.device, stream, zeros=True)
    qs, os = q.stride(), out.stride()
    if n * H and (qs[2] != 1 or os[2] != 1):
        raise ValueError("the head dimension of q and out must be contiguous")
    B = cache._batch(node_offsets.numel() - 1)
    # a dimension of size 1 is never stepped along: its stride only has to be a valid one
    _check((_lib or lib()).sv_tree_attention(
        cache._c, layer, _p(q), qs[0] if n > 1 else H * D, qs[1] if H > 1 else D, H, cache._table, cache.width,
        _array(seq_len, "seq_len", i32, B), _array(node_offsets, "node_offsets", i32, B + 1), n,
        _array(parent, "parent", i32, n), B, Nmax, D ** -0.5 if scale is None else scale, window, sinks, _p(out),
        os[0] if n > 1 else H * D, os[1] if H > 1 else D, _array(lse, "lse", torch.float32, n * H), _p(ws), _ws_bytes(ws),
        _stream(stream)))
    return out, lse
