"""Thin Python binding of libssa (the C ABI in include/ssa.h).

Two layers, both argument marshalling only (the second one, for the calls of a
decode loop, in ``csrc/marshal.cpp``):

* ``ssa_*`` functions with the C names and signatures; pointers and the
  stream are plain integers.
* ``select_blocks``, ``attn_fwd_dual``, ``align_loss``, ``attn_bwd``,
  ``attn_fwd_sparse``, ``diagnostics`` and ``DecodeCache`` (a key/value cache
  with its pooled keys, for ``ssa_decode_pool`` / ``ssa_decode_step``);
  ``window_fwd`` and ``window_bwd`` (sliding-window attention with sinks),
  ``cache_append``, ``paged_decode``, ``prefix_decode`` and ``PagedCache`` (a
  paged key/value cache and the attention that reads it): take
  torch CUDA tensors, allocate the outputs and the workspace with torch, pass
  raw device pointers and torch's current stream to the C entry point and
  raise ``SsaError`` on a non-zero status.

Every compute step runs in the library's CUDA kernels.  There is no fallback:
importing this module without a built ``libssa.so`` raises, and so does the
first call that needs ``_marshal.so`` without that.
"""
from __future__ import annotations

import ctypes
import math
import os
from ctypes import POINTER, c_float, c_int, c_longlong, c_size_t, c_uint, c_void_p

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libssa.so")

SSA_OK, SSA_ERR_INVALID_ARG, SSA_ERR_UNSUPPORTED = 0, -1, -2
SSA_ERR_WORKSPACE, SSA_ERR_CUDA, SSA_ERR_TIMEOUT = -3, -4, -5
SSA_F32, SSA_BF16 = 0, 1
SSA_FLAG_FORCE_SINK, SSA_FLAG_FORCE_SIMT = 1, 2
SSA_WS_SELECT, SSA_WS_FWD, SSA_WS_LOSS, SSA_WS_BWD, SSA_WS_FWD_SPARSE, SSA_WS_DECODE = range(6)

# every symbol include/ssa.h declares
EXPORTS = (
    "ssa_workspace_size", "ssa_select_blocks", "ssa_select_blocks_noalloc",
    "ssa_attn_fwd_dual", "ssa_attn_fwd_sparse", "ssa_attn_diagnostics", "ssa_attn_fwd_dual_diag",
    "ssa_decode_pool",
    "ssa_decode_step", "ssa_align_loss",
    "ssa_attn_bwd",
    "ssa_window_workspace_size", "ssa_window_fwd", "ssa_window_bwd",
    "ssa_cache_append", "ssa_cache_workspace_size", "ssa_paged_decode", "ssa_prefix_decode",
    "ssa_device_status", "ssa_status_string", "ssa_last_error",
    "ssa_kernel_path", "ssa_bwd_heads_per_group", "ssa_selftest_math", "ssa_selftest_wait_timeout",
    "ssa_debug_set_wait_limit_ns", "ssa_debug_set_ds_budget_bytes", "ssa_debug_set_kernel_events",
    "ssa_version",
)


class SsaError(RuntimeError):
    def __init__(self, where: str, status: int, detail: str):
        super().__init__(f"{where}: {status_string(status)} ({status}): {detail}")
        self.status = status


class ssa_params_t(ctypes.Structure):
    _fields_ = [("B", c_int), ("H", c_int), ("T", c_int), ("D", c_int), ("block", c_int),
                ("topk", c_int), ("dtype", c_int), ("sm_scale", c_float), ("flags", c_uint)]

    def __repr__(self):
        return (type(self).__name__ + "(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_)
                + ")")


class ssa_view_t(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("stride_b", c_longlong), ("stride_h", c_longlong),
                ("stride_t", c_longlong)]


class ssa_window_params_t(ctypes.Structure):
    _fields_ = [("B", c_int), ("Hq", c_int), ("Hkv", c_int), ("T", c_int), ("D", c_int),
                ("window", c_int), ("sinks", c_int), ("dtype", c_int), ("sm_scale", c_float),
                ("flags", c_uint)]
    __repr__ = ssa_params_t.__repr__


class ssa_cache_params_t(ctypes.Structure):
    _fields_ = [("B", c_int), ("Hq", c_int), ("Hkv", c_int), ("D", c_int), ("page", c_int),
                ("n_pages", c_int), ("max_pages", c_int), ("window", c_int), ("sinks", c_int),
                ("dtype", c_int), ("sm_scale", c_float), ("flags", c_uint),
                ("page_stride", c_longlong)]
    __repr__ = ssa_params_t.__repr__


_P = POINTER(ssa_params_t)
# ssa_window_params_t, ssa_cache_params_t and ssa_view_t arguments take ctypes.byref(...)
_SIGNATURES = {
    "ssa_workspace_size": (c_size_t, [_P, c_int]),
    "ssa_select_blocks": (c_int, [_P, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_size_t, c_void_p]),
    "ssa_select_blocks_noalloc": (c_int, [_P, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                          c_void_p]),
    "ssa_attn_fwd_dual": (c_int, [_P, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_size_t, c_void_p]),
    "ssa_attn_fwd_sparse": (c_int, [_P, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                    c_void_p, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "ssa_attn_diagnostics": (c_int, [_P, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p]),
    "ssa_attn_fwd_dual_diag": (c_int, [_P, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                       c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                                       c_void_p]),
    "ssa_decode_pool": (c_int, [_P, c_int, c_int, c_void_p, c_void_p, c_void_p]),
    "ssa_decode_step": (c_int, [_P, c_int, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "ssa_align_loss": (c_int, [_P, c_void_p, c_float, c_float, c_void_p, c_void_p, c_size_t,
                               c_void_p]),
    "ssa_attn_bwd": (c_int, [_P, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                             c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                             c_float, c_float, c_void_p, c_void_p, c_void_p, c_void_p,
                             c_size_t, c_void_p]),
    "ssa_window_workspace_size": (c_size_t, [c_void_p]),
    "ssa_window_fwd": (c_int, [c_void_p] * 8),
    "ssa_window_bwd": (c_int, [c_void_p] * 12 + [c_size_t, c_void_p]),
    "ssa_cache_append": (c_int, [c_void_p, c_int] + [c_void_p] * 10 + [c_int] * 3 + [c_void_p] * 3),
    "ssa_cache_workspace_size": (c_size_t, [c_void_p, c_int]),
    "ssa_paged_decode": (c_int, [c_void_p] * 9 + [c_size_t, c_void_p]),
    "ssa_prefix_decode": (c_int, [c_void_p] * 5 + [c_int] + [c_void_p] * 5 + [c_size_t, c_void_p]),
    "ssa_device_status": (c_int, [c_void_p]),
    "ssa_status_string": (ctypes.c_char_p, [c_int]),
    "ssa_last_error": (ctypes.c_char_p, []),
    "ssa_kernel_path": (c_int, [_P]),
    "ssa_bwd_heads_per_group": (c_int, [_P]),
    "ssa_selftest_math": (c_int, [c_void_p, c_int, c_void_p, c_void_p, c_void_p, c_void_p]),
    "ssa_version": (c_int, []),
    "ssa_debug_set_wait_limit_ns": (None, [ctypes.c_ulonglong]),
    "ssa_debug_set_ds_budget_bytes": (None, [ctypes.c_ulonglong]),
    "ssa_debug_set_kernel_events": (c_int, [c_void_p, c_int]),
    "ssa_selftest_wait_timeout": (c_int, [ctypes.c_ulonglong, c_void_p, c_void_p]),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; build it with "
                          "`python -m block_sparse_full_b200.build` (no fallback exists)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


_lib = _load()


class _Marshal:
    """Stands for the module _marshal (tensor checks and calls of the paged cache and window
    attention) until its first use: the other calls do without it."""

    def __getattr__(self, name):
        global _marshal
        try:
            from . import _marshal as module
        except ImportError as e:
            raise ImportError(f"the paged cache and window attention need _marshal.so, built for this torch and Python "
                              f"with `python -m block_sparse_full_b200.build` ({e})") from e
        _marshal = module
        return getattr(module, name)


_marshal = _Marshal()


def lib() -> ctypes.CDLL:
    return _lib


# ------------------------------------------------------------ C-named entry points

def ssa_workspace_size(params, which):
    return _lib.ssa_workspace_size(ctypes.byref(params), which)


def ssa_select_blocks(params, q, k, idx, cnt, mask, ws, ws_bytes, stream):
    return _lib.ssa_select_blocks(ctypes.byref(params), q, k, idx, cnt, mask, ws, ws_bytes,
                                  stream)


def ssa_select_blocks_noalloc(params, q, k, idx, cnt, mask, stream):
    """Selection with the library's built-in scratch (no workspace argument)."""
    return _lib.ssa_select_blocks_noalloc(ctypes.byref(params), q, k, idx, cnt, mask, stream)


def ssa_attn_fwd_dual(params, q, k, v, idx, cnt, mask, h_full, h_sparse, delta, lse_full,
                      lse_sparse, sqdiff_rows, ws, ws_bytes, stream):
    return _lib.ssa_attn_fwd_dual(ctypes.byref(params), q, k, v, idx, cnt, mask, h_full,
                                  h_sparse, delta, lse_full, lse_sparse, sqdiff_rows, ws,
                                  ws_bytes, stream)


def ssa_attn_fwd_sparse(params, q, k, v, idx, cnt, mask, h_sparse, lse_sparse, ws, ws_bytes,
                        stream):
    return _lib.ssa_attn_fwd_sparse(ctypes.byref(params), q, k, v, idx, cnt, mask, h_sparse,
                                    lse_sparse, ws, ws_bytes, stream)


def ssa_attn_diagnostics(params, q, k, lse_full, delta, sink_rows, head_stats, stream):
    return _lib.ssa_attn_diagnostics(ctypes.byref(params), q, k, lse_full, delta, sink_rows,
                                     head_stats, stream)


def ssa_attn_fwd_dual_diag(params, q, k, v, idx, cnt, mask, h_full, h_sparse, delta, lse_full,
                           lse_sparse, sqdiff_rows, sink_rows, head_stats, ws, ws_bytes, stream):
    return _lib.ssa_attn_fwd_dual_diag(ctypes.byref(params), q, k, v, idx, cnt, mask, h_full,
                                       h_sparse, delta, lse_full, lse_sparse, sqdiff_rows,
                                       sink_rows, head_stats, ws, ws_bytes, stream)


def ssa_decode_pool(params, j0, j1, k_cache, kbar, stream):
    return _lib.ssa_decode_pool(ctypes.byref(params), j0, j1, k_cache, kbar, stream)


def ssa_decode_step(params, t, q, k_cache, v_cache, kbar, h, lse, idx, ws, ws_bytes, stream):
    return _lib.ssa_decode_step(ctypes.byref(params), t, q, k_cache, v_cache, kbar, h, lse, idx, ws,
                                ws_bytes, stream)


def ssa_align_loss(params, sqdiff_rows, w_sparsity, w_commit, loss_out, ws, ws_bytes, stream):
    return _lib.ssa_align_loss(ctypes.byref(params), sqdiff_rows, w_sparsity, w_commit,
                               loss_out, ws, ws_bytes, stream)


def ssa_attn_bwd(params, q, k, v, idx, cnt, mask, h_full, h_sparse, lse_full, lse_sparse,
                 dh_full, dh_sparse, w_sparsity, w_commit, dq, dk, dv, ws, ws_bytes, stream):
    return _lib.ssa_attn_bwd(ctypes.byref(params), q, k, v, idx, cnt, mask, h_full, h_sparse,
                             lse_full, lse_sparse, dh_full, dh_sparse, w_sparsity, w_commit,
                             dq, dk, dv, ws, ws_bytes, stream)


def _ref(x):
    return None if x is None else ctypes.byref(x)


def ssa_window_workspace_size(params):
    return _lib.ssa_window_workspace_size(_ref(params))


def ssa_window_fwd(params, q, k, v, lens, h, lse, stream):
    return _lib.ssa_window_fwd(_ref(params), _ref(q), _ref(k), _ref(v), lens, _ref(h), lse, stream)


def ssa_window_bwd(params, q, k, v, lens, h, lse, dh, dq, dk, dv, ws, ws_bytes, stream):
    return _lib.ssa_window_bwd(_ref(params), _ref(q), _ref(k), _ref(v), lens, _ref(h), lse, _ref(dh),
                               _ref(dq), _ref(dk), _ref(dv), ws, ws_bytes, stream)


def ssa_cache_append(params, n_tokens, k, v, q, k_pages, v_pages, table, lens, new_lens, q_start,
                     inv_freq, rot_dim, interleaved, pos_offset, q_out, k_out, stream):
    return _lib.ssa_cache_append(_ref(params), n_tokens, _ref(k), _ref(v), _ref(q), k_pages, v_pages,
                                 table, lens, new_lens, q_start, inv_freq, rot_dim, interleaved,
                                 pos_offset, _ref(q_out), _ref(k_out), stream)


def ssa_cache_workspace_size(params, prefix_len):
    return _lib.ssa_cache_workspace_size(_ref(params), prefix_len)


def ssa_paged_decode(params, q, k_pages, v_pages, table, lens, h, lse, ws, ws_bytes, stream):
    return _lib.ssa_paged_decode(_ref(params), _ref(q), k_pages, v_pages, table, lens, _ref(h), lse,
                                 ws, ws_bytes, stream)


def ssa_prefix_decode(params, q, k_pages, v_pages, prefix_pages, prefix_len, table, lens, h, lse, ws,
                      ws_bytes, stream):
    return _lib.ssa_prefix_decode(_ref(params), _ref(q), k_pages, v_pages, prefix_pages, prefix_len,
                                  table, lens, _ref(h), lse, ws, ws_bytes, stream)


def ssa_device_status(stream):
    return _lib.ssa_device_status(stream)


def ssa_status_string(status):
    return _lib.ssa_status_string(status).decode()


def ssa_last_error():
    return _lib.ssa_last_error().decode()


def ssa_kernel_path(params):
    return _lib.ssa_kernel_path(ctypes.byref(params))


def ssa_selftest_math(x, n, exp2_poly, exp2_mufu, bf16_alu, stream):
    return _lib.ssa_selftest_math(x, n, exp2_poly, exp2_mufu, bf16_alu, stream)


def ssa_selftest_wait_timeout(limit_ns, gave_up, stream):
    return _lib.ssa_selftest_wait_timeout(limit_ns, gave_up, stream)


def ssa_debug_set_wait_limit_ns(ns):
    _lib.ssa_debug_set_wait_limit_ns(ns)


def ssa_debug_set_ds_budget_bytes(nbytes):
    _lib.ssa_debug_set_ds_budget_bytes(nbytes)


def ssa_bwd_heads_per_group(params):
    return _lib.ssa_bwd_heads_per_group(ctypes.byref(params))


def ssa_debug_set_kernel_events(events, n):
    return _lib.ssa_debug_set_kernel_events(events, n)


def ssa_version():
    return _lib.ssa_version()


status_string = ssa_status_string


def check(status: int, where: str):
    if status != SSA_OK:
        raise SsaError(where, status, ssa_last_error())


# ------------------------------------------------------------ tensor-level helpers

_DT = {torch.float32: SSA_F32, torch.bfloat16: SSA_BF16}


def make_params(B, H, T, D, block, topk, dtype, sm_scale=None, flags=0) -> ssa_params_t:
    if isinstance(dtype, torch.dtype):
        dtype = _DT[dtype]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    return ssa_params_t(B, H, T, D, block, topk, dtype, sm_scale, flags)


def params_for(q: torch.Tensor, block: int, topk: int, sm_scale=None, flags=0) -> ssa_params_t:
    B, H, T, D = q.shape
    return make_params(B, H, T, D, block, topk, q.dtype, sm_scale, flags)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, name: str):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def workspace(params, which, device) -> torch.Tensor:
    n = ssa_workspace_size(params, which)
    if n == ctypes.c_size_t(-1).value:
        raise SsaError("ssa_workspace_size", SSA_ERR_INVALID_ARG, ssa_last_error())
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device)


def select_blocks(params, q, k, ws=None):
    """Selection sets of the sparse stream -> (idx, cnt, mask) int32/int32/int32-bits."""
    _need(q, "q"), _need(k, "k")
    B, H, n = params.B, params.H, params.T // params.block
    words = (n + 31) // 32
    dev = q.device
    idx = torch.empty((B, H, n, params.topk), dtype=torch.int32, device=dev)
    cnt = torch.empty((B, H, n), dtype=torch.int32, device=dev)
    mask = torch.empty((B, H, n, words), dtype=torch.int32, device=dev)  # uint32 bits
    ws = workspace(params, SSA_WS_SELECT, dev) if ws is None else ws
    check(ssa_select_blocks(params, _ptr(q), _ptr(k), _ptr(idx), _ptr(cnt), _ptr(mask),
                            _ptr(ws), ws.numel(), _stream(dev)), "ssa_select_blocks")
    return idx, cnt, mask


def attn_fwd_dual(params, q, k, v, mask, idx=None, cnt=None, ws=None, out=None):
    """Both streams -> dict(h_full, h_sparse, delta, lse_full, lse_sparse, sqdiff)."""
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (mask, "mask")):
        _need(t, nm)
    dev = q.device
    rows = (params.B, params.H, params.T)
    if out is None:
        out = {
            "h_full": torch.empty_like(q), "h_sparse": torch.empty_like(q),
            **{nm: torch.empty(rows, dtype=torch.float32, device=dev)
               for nm in ("delta", "lse_full", "lse_sparse", "sqdiff")},
        }
    ws = workspace(params, SSA_WS_FWD, dev) if ws is None else ws
    check(ssa_attn_fwd_dual(params, _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(cnt),
                            _ptr(mask), _ptr(out["h_full"]), _ptr(out["h_sparse"]),
                            _ptr(out["delta"]), _ptr(out["lse_full"]),
                            _ptr(out["lse_sparse"]), _ptr(out["sqdiff"]), _ptr(ws),
                            ws.numel(), _stream(dev)), "ssa_attn_fwd_dual")
    return out


def attn_fwd_sparse(params, q, k, v, mask, idx=None, cnt=None, ws=None, out=None):
    """The sparse stream alone (inference) -> dict(h_sparse, lse_sparse)."""
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (mask, "mask")):
        _need(t, nm)
    dev = q.device
    if out is None:
        out = {"h_sparse": torch.empty_like(q),
               "lse_sparse": torch.empty((params.B, params.H, params.T), dtype=torch.float32,
                                         device=dev)}
    ws = workspace(params, SSA_WS_FWD_SPARSE, dev) if ws is None else ws
    check(ssa_attn_fwd_sparse(params, _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(cnt),
                              _ptr(mask), _ptr(out["h_sparse"]), _ptr(out["lse_sparse"]),
                              _ptr(ws), ws.numel(), _stream(dev)), "ssa_attn_fwd_sparse")
    return out


def diagnostics(params, q, k, fwd):
    """Sink mass per row and per-head means of delta and sink -> dict(sink, head_stats)."""
    _need(q, "q"), _need(k, "k")
    dev = q.device
    sink = torch.empty((params.B, params.H, params.T), dtype=torch.float32, device=dev)
    stats = torch.empty((params.B, params.H, 2), dtype=torch.float32, device=dev)
    check(ssa_attn_diagnostics(params, _ptr(q), _ptr(k), _ptr(fwd["lse_full"]), _ptr(fwd["delta"]),
                               _ptr(sink), _ptr(stats), _stream(dev)), "ssa_attn_diagnostics")
    return {"sink": sink, "head_stats": stats}


def attn_fwd_dual_diag(params, q, k, v, mask, idx=None, cnt=None, ws=None, out=None):
    """Both streams plus the diagnostics in one call -> the dict of
    ``attn_fwd_dual`` with ``sink`` [B,H,T] and ``head_stats`` [B,H,2] added."""
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (mask, "mask")):
        _need(t, nm)
    dev = q.device
    rows = (params.B, params.H, params.T)
    if out is None:
        out = {
            "h_full": torch.empty_like(q), "h_sparse": torch.empty_like(q),
            **{nm: torch.empty(rows, dtype=torch.float32, device=dev)
               for nm in ("delta", "lse_full", "lse_sparse", "sqdiff", "sink")},
            "head_stats": torch.empty((params.B, params.H, 2), dtype=torch.float32, device=dev),
        }
    ws = workspace(params, SSA_WS_FWD, dev) if ws is None else ws
    check(ssa_attn_fwd_dual_diag(params, _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(cnt),
                                 _ptr(mask), _ptr(out["h_full"]), _ptr(out["h_sparse"]),
                                 _ptr(out["delta"]), _ptr(out["lse_full"]),
                                 _ptr(out["lse_sparse"]), _ptr(out["sqdiff"]), _ptr(out["sink"]),
                                 _ptr(out["head_stats"]), _ptr(ws), ws.numel(), _stream(dev)),
          "ssa_attn_fwd_dual_diag")
    return out


class DecodeCache:
    """Key/value cache of capacity params.T and the pooled keys of its completed
    blocks, for ssa_decode_step.  Tensors are allocated on ``device``."""

    def __init__(self, params, device, dtype):
        B, H, T, D = params.B, params.H, params.T, params.D
        self.params = params
        self.k = torch.zeros((B, H, T, D), dtype=dtype, device=device)
        self.v = torch.zeros_like(self.k)
        self.kbar = torch.zeros((B, H, T // params.block, D), dtype=torch.float64, device=device)
        self.pooled = 0  # completed blocks whose pooled keys are in kbar
        self.ws = workspace(params, SSA_WS_DECODE, device)

    def pool_upto(self, n_blocks):
        if n_blocks > self.pooled:
            check(ssa_decode_pool(self.params, self.pooled, n_blocks, _ptr(self.k), _ptr(self.kbar),
                                  _stream(self.k.device)), "ssa_decode_pool")
            self.pooled = n_blocks

    def step(self, t, q_t, idx=True):
        """Attend q_t [B,H,D] at position t (keys/values 0..t already written)."""
        p = self.params
        self.pool_upto(t // p.block)
        h = torch.empty((p.B, p.H, p.D), dtype=self.k.dtype, device=self.k.device)
        lse = torch.empty((p.B, p.H), dtype=torch.float32, device=self.k.device)
        ix = torch.empty((p.B, p.H, p.topk), dtype=torch.int32, device=self.k.device) if idx else None
        check(ssa_decode_step(p, t, _ptr(q_t), _ptr(self.k), _ptr(self.v), _ptr(self.kbar), _ptr(h),
                              _ptr(lse), _ptr(ix), _ptr(self.ws), self.ws.numel(),
                              _stream(self.k.device)), "ssa_decode_step")
        return {"h": h, "lse": lse, "idx": ix}


def align_loss(params, sqdiff, w_sparsity=1.0, w_commit=1.0, ws=None, out=None):
    """(w_s * L_sparsity, w_c * L_commit) as a float32 CUDA tensor of 2."""
    _need(sqdiff, "sqdiff")
    dev = sqdiff.device
    out = torch.empty(2, dtype=torch.float32, device=dev) if out is None else out
    ws = workspace(params, SSA_WS_LOSS, dev) if ws is None else ws
    check(ssa_align_loss(params, _ptr(sqdiff), w_sparsity, w_commit, _ptr(out), _ptr(ws),
                         ws.numel(), _stream(dev)), "ssa_align_loss")
    return out


def attn_bwd(params, q, k, v, mask, fwd, dh_full=None, dh_sparse=None, w_sparsity=0.0,
             w_commit=0.0, ws=None, out=None):
    """Gradients (dq, dk, dv) of both streams plus the alignment terms."""
    dev = q.device
    if out is None:
        out = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    dq, dk, dv = out
    ws = workspace(params, SSA_WS_BWD, dev) if ws is None else ws
    check(ssa_attn_bwd(params, _ptr(q), _ptr(k), _ptr(v), None, None, _ptr(mask),
                       _ptr(fwd["h_full"]), _ptr(fwd["h_sparse"]), _ptr(fwd["lse_full"]),
                       _ptr(fwd["lse_sparse"]), _ptr(dh_full), _ptr(dh_sparse), w_sparsity,
                       w_commit, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), ws.numel(),
                       _stream(dev)), "ssa_attn_bwd")
    return dq, dk, dv


def device_status(device=None):
    """Waits for torch's current stream of ``device`` (None: the current device) and raises
    ``SsaError`` if a kernel on that device has recorded an error since the last call."""
    with torch.cuda.device(device):  # the records are each device's own
        check(ssa_device_status(_stream(device)), "ssa_device_status")


# ------------------------------------------------------------ paged cache and window attention

def window_params(B, Hq, Hkv, T, D, window, sinks, dtype, sm_scale=None, flags=0) -> ssa_window_params_t:
    """Shape of sliding-window attention (``window`` 0: every earlier token)."""
    if isinstance(dtype, torch.dtype):
        dtype = _DT[dtype]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    return ssa_window_params_t(B, Hq, Hkv, T, D, window, sinks, dtype, sm_scale, flags)


def window_params_for(q, k, window, sinks=0, sm_scale=None, flags=0) -> ssa_window_params_t:
    """For q [B,Hq,T,D] and k [B,Hkv,T,D]."""
    return _marshal.window_params_for(ssa_window_params_t, q, k, window, sinks, sm_scale, flags)


def cache_params(B, Hq, Hkv, D, page, n_pages, max_pages, dtype, window=0, sinks=0, sm_scale=None,
                 page_stride=None) -> ssa_cache_params_t:
    """Shape of a paged cache and of the queries that read it."""
    if isinstance(dtype, torch.dtype):
        dtype = _DT[dtype]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    if page_stride is None:
        page_stride = Hkv * page * D
    return ssa_cache_params_t(B, Hq, Hkv, D, page, n_pages, max_pages, window, sinks, dtype, sm_scale, 0,
                              page_stride)


def cache_params_for(q, k_pages, table, window=0, sinks=0, sm_scale=None) -> ssa_cache_params_t:
    """For q [..., Hq, D], k_pages [n_pages, Hkv, page, D] and table [B, max_pages]."""
    return _marshal.cache_params_for(ssa_cache_params_t, q, k_pages, table, window, sinks, sm_scale)


_NO_PAIR = (None, None)


def window_fwd(params, q, k, v, lens=None, out=None):
    """Sliding-window attention with sinks -> dict(h [B,Hq,T,D], lse [B,Hq,T] float32).

    q [B,Hq,T,D], k and v [B,Hkv,T,D] may be strided views (the last axis
    contiguous); ``lens`` [B] int32 are the lengths of a padded batch, rows
    behind a length get h = 0 and lse = -inf.  h is laid out like q where q
    fills its memory, else contiguous.
    """
    r = _marshal.window_fwd(params, q, k, v, lens, *(_NO_PAIR if out is None else (out["h"], out["lse"])))
    if r.__class__ is int:
        check(r, "ssa_window_fwd")
    return {"h": r[0], "lse": r[1]} if out is None else out


def window_bwd(params, q, k, v, fwd, dh, lens=None, ws=None, out=None):
    """Gradients (dq, dk, dv) of <dh, h>, from the inputs and the result of ``window_fwd``."""
    r = _marshal.window_bwd(params, q, k, v, lens, fwd["h"], fwd["lse"], dh, ws, *(out or (None, None, None)))
    if r.__class__ is int:
        check(r, "ssa_window_bwd")
    return r


def cache_append(params, k_pages, v_pages, table, lens, k, v, q=None, inv_freq=None, interleaved=False,
                 q_start=None, pos_offset=0, new_lens=None, q_out=None, k_out=None):
    """Rotates new keys (and queries) to their positions and appends keys and values to the pages
    -> dict(q, lens): the rotated queries and the sequences' new lengths.

    k, v [N,Hkv,D] and q [N,Hq,D] hold the sequences' new tokens one after the
    other: ``q_start`` [B+1] int32 says where each begins, without it every
    sequence has N / B.  ``lens`` [B] int32 are the lengths before.  ``inv_freq``
    [rot/2] float64 holds the rotation's angles per position.  ``new_lens`` may
    be ``lens`` (advanced in place), ``q_out`` may be q, ``k_out`` (k itself or
    another tensor) also receives the rotated keys.
    """
    r = _marshal.cache_append(params, k_pages, v_pages, table, lens, k, v, q, inv_freq, interleaved, q_start, pos_offset,
                              new_lens, q_out, k_out)
    if r.__class__ is int:
        check(r, "ssa_cache_append")
    return {"q": r[0], "lens": r[1]}


def paged_decode(params, q, k_pages, v_pages, table, lens, ws=None, out=None):
    """Attention of one token per sequence, q [B,Hq,D], over the paged cache
    -> dict(h [B,Hq,D], lse [B,Hq] float32).  ``lens`` count the token itself."""
    r = _marshal.decode(params, q, k_pages, v_pages, None, -1, table, lens, ws,
                        *(_NO_PAIR if out is None else (out["h"], out["lse"])))
    if r.__class__ is int:
        check(r, "ssa_paged_decode")
    return {"h": r[0], "lse": r[1]} if out is None else out


def prefix_decode(params, q, k_pages, v_pages, prefix_pages, prefix_len, table, lens, ws=None, out=None):
    """``paged_decode`` for a batch behind one shared prefix: every query sees the first
    ``prefix_len`` tokens of ``prefix_pages`` and the ``lens`` tokens of its own pages."""
    if prefix_len < 0:
        raise ValueError(f"prefix_len must not be negative, got {prefix_len}")
    r = _marshal.decode(params, q, k_pages, v_pages, prefix_pages, prefix_len, table, lens, ws,
                        *(_NO_PAIR if out is None else (out["h"], out["lse"])))
    if r.__class__ is int:
        check(r, "ssa_prefix_decode")
    return {"h": r[0], "lse": r[1]} if out is None else out


class PagedCache:
    """Pages for B sequences of up to ``capacity`` tokens each, their table and
    lengths.  ``append`` advances the lengths in place and ``attend`` reads the
    cache up to them, so that one captured decode step can be replayed.  The
    table gives every sequence pages of its own, in order; ``table`` may be
    overwritten with other page numbers.  ``prefix_pages`` (of the same pool) and
    ``prefix_len`` put one shared prefix before every sequence (without a window)."""

    def __init__(self, B, Hq, Hkv, D, capacity, dtype, device, page=64, window=0, sinks=0, sm_scale=None,
                 inv_freq=None, interleaved=False, prefix_len=0):
        width, shared = max(1, -(-capacity // page)), -(-prefix_len // page)
        self.params = cache_params(B, Hq, Hkv, D, page, B * width + shared, width, dtype, window, sinks, sm_scale)
        if ssa_cache_workspace_size(self.params, prefix_len) == ctypes.c_size_t(-1).value:
            raise SsaError("ssa_cache_workspace_size", SSA_ERR_INVALID_ARG, ssa_last_error())
        shape = (B * width + shared, Hkv, page, D)
        self.k_pages = torch.zeros(shape, dtype=dtype, device=device)
        self.v_pages = torch.zeros_like(self.k_pages)
        self.table = torch.arange(B * width, dtype=torch.int32, device=device).view(B, width)
        self.lens = torch.zeros(B, dtype=torch.int32, device=device)
        self.prefix_len = prefix_len
        self.prefix_pages = B * width + torch.arange(shared, dtype=torch.int32, device=device)
        self.inv_freq, self.interleaved = inv_freq, interleaved

    def append(self, k, v, q=None, q_start=None, q_out=None, k_out=None):
        """Appends new tokens (see ``cache_append``) -> the rotated queries."""
        return cache_append(self.params, self.k_pages, self.v_pages, self.table, self.lens, k, v, q, self.inv_freq,
                            self.interleaved, q_start, self.prefix_len, self.lens, q_out, k_out)["q"]

    def fill_prefix(self, k, v, k_out=None):
        """Writes the shared prefix's keys and values [prefix_len, Hkv, D], rotated to 0, 1, ..."""
        if not self.prefix_len:
            raise ValueError("this cache has no shared prefix")
        for name, x in (("k", k), ("v", v)):
            if x.shape[:1] != (self.prefix_len,):
                raise ValueError(f"{name} must hold the prefix's {self.prefix_len} tokens, got shape {tuple(x.shape)}")
        p, dev = self.params, self.k_pages.device
        one = cache_params(1, p.Hq, p.Hkv, p.D, p.page, p.n_pages, max(1, self.prefix_pages.numel()), p.dtype)
        cache_append(one, self.k_pages, self.v_pages, self.prefix_pages.view(1, -1),
                     torch.zeros(1, dtype=torch.int32, device=dev), k, v, None, self.inv_freq, self.interleaved,
                     k_out=k_out)

    def attend(self, q, out=None):
        """Attention of each sequence's newest token, q [B,Hq,D] rotated -> dict(h, lse)."""
        if self.prefix_len:
            return prefix_decode(self.params, q, self.k_pages, self.v_pages, self.prefix_pages, self.prefix_len,
                                 self.table, self.lens, None, out)
        return paged_decode(self.params, q, self.k_pages, self.v_pages, self.table, self.lens, None, out)
