"""Thin Python binding over the kvattn C ABI (argument marshalling only).

Every function with a ``kvattn_`` name calls the C entry point of the same name; torch
tensors are passed by ``data_ptr()``, streams by their ``cuda_stream`` handle, and a
non-OK status raises :class:`KvattnError`.  The convenience wrappers at the end
(``decode``, ``merge``, ``WindowTail``; ``rope``, ``norm_rope``, ``step_maps``, ``cache_write``,
``cache_read``, ``prefill``, ``prefill_chunk``) only allocate outputs and workspaces with torch and infer sizes from tensor
shapes; all arithmetic runs in the library's kernels.  A wrapper's ``stream`` (default: torch's
current one) is where it launches, and where the tensors that it makes belong, as under
``torch.cuda.stream(stream)``: work on another stream waits for it before it uses them, and the
call is ordered behind whatever makes its inputs by the program.

Importing this module loads ``_lib/libkvattn.so`` and raises if it has not been built
(``python -m kv_cache_decode_02_gb300._build``): there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os

import numpy as np

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libkvattn.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with "
                      "`python -m kv_cache_decode_02_gb300._build` (no fallback exists)")
lib = ctypes.CDLL(_LIB_PATH)

KVATTN_OK = 0
KVATTN_ERR_INVALID_ARG = -1
KVATTN_ERR_UNSUPPORTED = -2
KVATTN_ERR_WORKSPACE = -3
KVATTN_ERR_CAPACITY = -4
KVATTN_ERR_CUDA = -5
KVATTN_ERR_TIMEOUT = -6
KVATTN_KV_F16 = 0
KVATTN_KV_Q8_0 = 1
KVATTN_KV_Q8_0_Q4_0 = 2
KVATTN_KV_Q4_0 = 3
KVATTN_DEVICE_WAIT_TIMEOUT = 1
KVATTN_DEVICE_BAD_PLAN_ENTRY = 2
KVATTN_DEVICE_NO_ROOM = 4
KVATTN_TAIL_PREFETCH = 1
KVATTN_ROPE_HALF = 0
KVATTN_ROPE_INTERLEAVED = 1
KVATTN_ROPE_PLAIN = 0
KVATTN_ROPE_LINEAR = 1
KVATTN_ROPE_YARN = 2
KVATTN_AXES_BLOCKS = 0
KVATTN_AXES_CYCLE = 1

EXPORTED = (
    "kvattn_status_string", "kvattn_version", "kvattn_build_cell_plan", "kvattn_build_descriptors",
    "kvattn_decode_workspace_bytes", "kvattn_decode", "kvattn_decode_partials", "kvattn_merge",
    "kvattn_tail_ctx_create",
    "kvattn_tail_ctx_destroy", "kvattn_window_tail_workspace_bytes", "kvattn_decode_window_tail",
    "kvattn_tail_wait", "kvattn_workspace_status", "kvattn_decode_noalloc",
    "kvattn_window_tail_direct_workspace_bytes", "kvattn_decode_window_tail_direct",
    "kvattn_select_split_for", "kvattn_select_split", "kvattn_decode_multi_workspace_bytes",
    "kvattn_decode_multi", "kvattn_tail_ctx_set_flags", "kvattn_rope_table", "kvattn_rope", "kvattn_cache_write",
    "kvattn_cache_read", "kvattn_prefill_workspace_bytes", "kvattn_prefill", "kvattn_prefill_chunk_workspace_bytes",
    "kvattn_prefill_chunk", "kvattn_rope_axes", "kvattn_norm_rope", "kvattn_step_maps", "kvattn_prefill_window",
    "kvattn_prefill_chunk_window", "kvattn_prefill_chunk_shared_workspace_bytes", "kvattn_prefill_chunk_shared",
)

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float

lib.kvattn_status_string.argtypes = [_I]
lib.kvattn_status_string.restype = ctypes.c_char_p
lib.kvattn_version.argtypes = []
lib.kvattn_version.restype = _I
lib.kvattn_build_cell_plan.argtypes = [_P, _P, _I, _I64, _P, _I64, _P]
lib.kvattn_build_cell_plan.restype = _I
lib.kvattn_build_descriptors.argtypes = [_P, _I64, _P, _I, _I64, _I, _I64, _P, _P]
lib.kvattn_build_descriptors.restype = _I
lib.kvattn_decode_workspace_bytes.argtypes = [_I, _I, _I, _I64, _I]
lib.kvattn_decode_workspace_bytes.restype = _SZ
lib.kvattn_decode_multi_workspace_bytes.argtypes = [_I, _I, _I, _I, _I64, _I]
lib.kvattn_decode_multi_workspace_bytes.restype = _SZ
lib.kvattn_decode_multi.argtypes = [_P, _P, _P, _P, _P, _I, _I64, _P, _I64, _P, _I, _I64, _I, _I, _I, _I, _I, _F,
                                    _P, _P, _P, _SZ, _P]
lib.kvattn_decode_multi.restype = _I
lib.kvattn_select_split_for.argtypes = [_I, _I64, _I, _I64]
lib.kvattn_select_split_for.restype = _I
lib.kvattn_select_split.argtypes = [_I, _I, _I64, _I, _I]
lib.kvattn_select_split.restype = _I
lib.kvattn_decode.argtypes = [_P, _P, _P, _P, _P, _I, _I64, _P, _I64, _P, _I, _I64, _I, _I, _I, _I,
                              _F, _P, _P, _P, _SZ, _P]
lib.kvattn_decode.restype = _I
lib.kvattn_decode_partials.argtypes = lib.kvattn_decode.argtypes
lib.kvattn_decode_partials.restype = _I
lib.kvattn_decode_noalloc.argtypes = [_P, _P, _P, _P, _P, _I, _I64, _P, _I64, _P, _I, _I64, _I, _I, _I, _I,
                                      _F, _P, _P, _P]
lib.kvattn_decode_noalloc.restype = _I
KVATTN_NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024
lib.kvattn_merge.argtypes = [_P, _P, _I, _I, _I, _P, _P, _P]
lib.kvattn_merge.restype = _I
lib.kvattn_tail_ctx_create.argtypes = [ctypes.POINTER(_P)]
lib.kvattn_tail_ctx_create.restype = _I
lib.kvattn_tail_ctx_destroy.argtypes = [_P]
lib.kvattn_tail_ctx_destroy.restype = _I
lib.kvattn_tail_ctx_set_flags.argtypes = [_P, ctypes.c_uint32]
lib.kvattn_tail_ctx_set_flags.restype = _I
lib.kvattn_window_tail_workspace_bytes.argtypes = [_I, _I, _I, _I64, _I64, _I, _I64, _I]
lib.kvattn_window_tail_workspace_bytes.restype = _SZ
lib.kvattn_decode_window_tail.argtypes = [_P, _P, _P, _P, _I64, _P, _P, _I64, _I64, _I, _I, _I, _I,
                                          _I, _F, _P, _P, _P, _SZ, _P, _P]
lib.kvattn_decode_window_tail.restype = _I
lib.kvattn_window_tail_direct_workspace_bytes.argtypes = [_I, _I, _I, _I64, _I64, _I, _I]
lib.kvattn_window_tail_direct_workspace_bytes.restype = _SZ
lib.kvattn_decode_window_tail_direct.argtypes = [_P, _P, _P, _I64, _P, _P, _I64, _I, _I, _I, _I, _I, _F, _P,
                                                 _P, _P, _SZ, _P]
lib.kvattn_decode_window_tail_direct.restype = _I
lib.kvattn_tail_wait.argtypes = [_P, _I]
lib.kvattn_tail_wait.restype = _I
lib.kvattn_workspace_status.argtypes = [_P, ctypes.POINTER(ctypes.c_uint32), _I, _P]
lib.kvattn_workspace_status.restype = _I
lib.kvattn_rope_table.argtypes = [_I, ctypes.c_double, _I, ctypes.c_double, _I64, _P, ctypes.POINTER(_F)]
lib.kvattn_rope_table.restype = _I
lib.kvattn_rope.argtypes = [_P, _I64, _I, _P, _I64, _I, _P, _P, _F, _I, _I, _I64, _I, _P, _I64, _P, _I64, _P]
lib.kvattn_rope.restype = _I
lib.kvattn_cache_write.argtypes = [_P, _I64, _P, _I64, _P, _I64, _I, _I, _I, _P, _P, _P, _P, _I64, _P, _P]
lib.kvattn_cache_write.restype = _I
lib.kvattn_cache_read.argtypes = [_P, _P, _P, _P, _I, _I64, _P, _I64, _I, _I, _P, _I64, _P, _I64, _P, _P]
lib.kvattn_cache_read.restype = _I
lib.kvattn_prefill_workspace_bytes.argtypes = [_I64, _I, _I, _I, _I]
lib.kvattn_prefill_workspace_bytes.restype = _SZ
lib.kvattn_prefill.argtypes = [_P, _I64, _P, _I64, _P, _I64, _P, _I, _I64, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]
lib.kvattn_prefill.restype = _I
lib.kvattn_prefill_chunk_workspace_bytes.argtypes = [_I64, _I, _I, _I, _I, _I64]
lib.kvattn_prefill_chunk_workspace_bytes.restype = _SZ
lib.kvattn_prefill_chunk.argtypes = [_P, _I64, _P, _I64, _P, _P, _P, _P, _I, _I64, _P, _I64, _P, _I, _I64, _I, _I, _I, _F,
                                     _P, _P, _P, _SZ, _P]
lib.kvattn_prefill_chunk.restype = _I
lib.kvattn_prefill_window.argtypes = [_P, _I64, _P, _I64, _P, _I64, _P, _I, _I64, _I, _I, _I, _F, _I64, _I64, _P, _P, _P, _SZ, _P]
lib.kvattn_prefill_window.restype = _I
lib.kvattn_prefill_chunk_window.argtypes = [_P, _I64, _P, _I64, _P, _P, _P, _P, _I, _I64, _P, _I64, _P, _I, _I64, _I, _I, _I, _F,
                                            _I64, _I64, _P, _P, _P, _SZ, _P]
lib.kvattn_prefill_chunk_window.restype = _I
lib.kvattn_prefill_chunk_shared_workspace_bytes.argtypes = [_I64, _I, _I, _I, _I, _I64]
lib.kvattn_prefill_chunk_shared_workspace_bytes.restype = _SZ
lib.kvattn_prefill_chunk_shared.argtypes = [_P, _I64, _P, _I64, _P, _P, _P, _P, _I, _I64, _P, _I64, _P, _I, _I64, _I, _I, _I, _F,
                                            _I64, _P, _P, _P, _SZ, _P]
lib.kvattn_prefill_chunk_shared.restype = _I
lib.kvattn_rope_axes.argtypes = [_I, _P, _I, _I, _P]
lib.kvattn_rope_axes.restype = _I
lib.kvattn_norm_rope.argtypes = [_P, _I64, _I, _P, _P, _I64, _I, _P, _F, _P, _I64, _I, _P, _P, _F, _I, _I, _I64, _I,
                                 _P, _I64, _P, _I64, _P]
lib.kvattn_norm_rope.restype = _I
lib.kvattn_step_maps.argtypes = [_P, _P, _I, _P, _I64, _I, _P, _I64, _P, _I64, _I64, _P, _P, _P, _P, _P, _P, _I64, _I, _P, _P]
lib.kvattn_step_maps.restype = _I


class KvattnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {kvattn_status_string(status)} ({status})")


# What the prompt wrappers use of torch, looked up at the first call (callers of the C binding alone
# do not wait for torch's import) and once (an import statement and a Stream object cost 0.3 and 4 us
# in every call).
_torch = _F16 = _I32 = _current_raw_stream = _current_device = None


def _bind_torch():
    global _torch, _F16, _I32, _current_raw_stream, _current_device
    import torch
    if _current_device is None:
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda device: torch.cuda.current_stream(device).cuda_stream)
    _F16, _I32 = torch.float16, torch.int32
    _torch = torch


def _ptr(x):
    """Address of a torch tensor / numpy array / int / None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if isinstance(x, np.ndarray):
        return x.ctypes.data
    return x.data_ptr()


def _stream(s):
    if s is None:
        if _torch is None:
            _bind_torch()
        return _current_raw_stream(_current_device())
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(rc: int, where: str) -> None:
    if rc != KVATTN_OK:
        raise KvattnError(rc, where)


# ----------------------------- same names as the C ABI -----------------------------

def kvattn_status_string(status: int) -> str:
    return lib.kvattn_status_string(status).decode()


def kvattn_version() -> int:
    return lib.kvattn_version()


def kvattn_build_cell_plan(cells, offsets, n_seq, capacity_cells, plan, plan_stride, seq_lens):
    """Host arrays (numpy int64 / int32).  ``plan`` may be None to only size the rows."""
    rc = lib.kvattn_build_cell_plan(_ptr(cells), _ptr(offsets), n_seq, capacity_cells, _ptr(plan),
                                    plan_stride, _ptr(seq_lens))
    _check(rc, "kvattn_build_cell_plan")


def kvattn_build_descriptors(cell_plan, plan_stride, seq_lens, n_seq, max_len, split, n_cells, desc,
                             stream=None):
    rc = lib.kvattn_build_descriptors(_ptr(cell_plan), plan_stride, _ptr(seq_lens), n_seq, max_len,
                                      split, n_cells, _ptr(desc), _stream(stream))
    _check(rc, "kvattn_build_descriptors")


def kvattn_decode_workspace_bytes(n_seq, n_head, head_dim, max_len, split) -> int:
    return lib.kvattn_decode_workspace_bytes(n_seq, n_head, head_dim, max_len, split)


def kvattn_decode_multi_workspace_bytes(n_seq, n_q, n_head, head_dim, max_len, split) -> int:
    return lib.kvattn_decode_multi_workspace_bytes(n_seq, n_q, n_head, head_dim, max_len, split)


def kvattn_decode_multi(q, k_cache, v_cache, k_scales, v_scales, kv_type, n_cells, cell_plan, plan_stride, seq_lens,
                        n_seq, max_len, n_q, n_head, n_head_kv, head_dim, split, scale, out, lse, ws, ws_bytes,
                        stream=None):
    rc = lib.kvattn_decode_multi(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scales), _ptr(v_scales), kv_type,
                                 n_cells, _ptr(cell_plan), plan_stride, _ptr(seq_lens), n_seq, max_len, n_q, n_head,
                                 n_head_kv, head_dim, split, scale, _ptr(out), _ptr(lse), _ptr(ws), ws_bytes,
                                 _stream(stream))
    _check(rc, "kvattn_decode_multi")


def kvattn_select_split_for(n_seq, max_len, n_head_kv, resident_ctas) -> int:
    rc = lib.kvattn_select_split_for(n_seq, max_len, n_head_kv, resident_ctas)
    if rc < 0:
        raise KvattnError(rc, "kvattn_select_split_for")
    return rc


def kvattn_select_split(kv_type, n_seq, max_len, n_head_kv, head_dim) -> int:
    rc = lib.kvattn_select_split(kv_type, n_seq, max_len, n_head_kv, head_dim)
    if rc < 0:
        raise KvattnError(rc, "kvattn_select_split")
    return rc


def kvattn_decode(q, k_cache, v_cache, k_scales, v_scales, kv_type, n_cells, cell_plan, plan_stride,
                  seq_lens, n_seq, max_len, n_head, n_head_kv, head_dim, split, scale, out, lse, ws,
                  ws_bytes, stream=None):
    rc = lib.kvattn_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scales), _ptr(v_scales),
                           kv_type, n_cells, _ptr(cell_plan), plan_stride, _ptr(seq_lens), n_seq,
                           max_len, n_head, n_head_kv, head_dim, split, scale, _ptr(out), _ptr(lse),
                           _ptr(ws), ws_bytes, _stream(stream))
    _check(rc, "kvattn_decode")


def kvattn_decode_partials(q, k_cache, v_cache, k_scales, v_scales, kv_type, n_cells, cell_plan,
                           plan_stride, seq_lens, n_seq, max_len, n_head, n_head_kv, head_dim, split,
                           scale, part_o, part_lse, ws, ws_bytes, stream=None):
    rc = lib.kvattn_decode_partials(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scales),
                                    _ptr(v_scales), kv_type, n_cells, _ptr(cell_plan), plan_stride,
                                    _ptr(seq_lens), n_seq, max_len, n_head, n_head_kv, head_dim, split,
                                    scale, _ptr(part_o), _ptr(part_lse), _ptr(ws), ws_bytes,
                                    _stream(stream))
    _check(rc, "kvattn_decode_partials")


def kvattn_decode_noalloc(q, k_cache, v_cache, k_scales, v_scales, kv_type, n_cells, cell_plan,
                          plan_stride, seq_lens, n_seq, max_len, n_head, n_head_kv, head_dim, split, scale,
                          out, lse, stream=None):
    """kvattn_decode without a workspace, for callers that cannot allocate device memory:
    the library keeps the scratch in its own fixed-size device array (see kvattn.h)."""
    rc = lib.kvattn_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scales),
                                   _ptr(v_scales), kv_type, n_cells, _ptr(cell_plan), plan_stride,
                                   _ptr(seq_lens), n_seq, max_len, n_head, n_head_kv, head_dim, split,
                                   scale, _ptr(out), _ptr(lse), _stream(stream))
    _check(rc, "kvattn_decode_noalloc")


def kvattn_merge(partials, lses, n_parts, n_rows, head_dim, out, lse, stream=None):
    rc = lib.kvattn_merge(_ptr(partials), _ptr(lses), n_parts, n_rows, head_dim, _ptr(out),
                          _ptr(lse), _stream(stream))
    _check(rc, "kvattn_merge")


def kvattn_tail_ctx_create() -> int:
    h = _P()
    _check(lib.kvattn_tail_ctx_create(ctypes.byref(h)), "kvattn_tail_ctx_create")
    return h.value


def kvattn_tail_ctx_destroy(ctx: int) -> None:
    _check(lib.kvattn_tail_ctx_destroy(ctx), "kvattn_tail_ctx_destroy")


def kvattn_tail_ctx_set_flags(ctx: int, flags: int) -> None:
    _check(lib.kvattn_tail_ctx_set_flags(ctx, flags), "kvattn_tail_ctx_set_flags")


def kvattn_window_tail_workspace_bytes(n_head, n_head_kv, head_dim, n_win, n_tail, split, tile_cells,
                                       tail_split) -> int:
    return lib.kvattn_window_tail_workspace_bytes(n_head, n_head_kv, head_dim, n_win, n_tail, split,
                                                  tile_cells, tail_split)


def kvattn_decode_window_tail(ctx, q, k_win, v_win, n_win, k_tail_host, v_tail_host, n_tail,
                              tile_cells, n_head, n_head_kv, head_dim, split, tail_split, scale,
                              out, lse, ws, ws_bytes, compute_stream=None, copy_stream=None):
    rc = lib.kvattn_decode_window_tail(ctx, _ptr(q), _ptr(k_win), _ptr(v_win), n_win,
                                       _ptr(k_tail_host), _ptr(v_tail_host), n_tail, tile_cells,
                                       n_head, n_head_kv, head_dim, split, tail_split, scale,
                                       _ptr(out), _ptr(lse), _ptr(ws), ws_bytes,
                                       _stream(compute_stream), _stream(copy_stream))
    _check(rc, "kvattn_decode_window_tail")


def kvattn_window_tail_direct_workspace_bytes(n_head, n_head_kv, head_dim, n_win, n_tail, split,
                                              tail_split) -> int:
    return lib.kvattn_window_tail_direct_workspace_bytes(n_head, n_head_kv, head_dim, n_win, n_tail, split,
                                                         tail_split)


def kvattn_decode_window_tail_direct(q, k_win, v_win, n_win, k_tail_host, v_tail_host, n_tail, n_head,
                                     n_head_kv, head_dim, split, tail_split, scale, out, lse, ws, ws_bytes,
                                     stream=None):
    rc = lib.kvattn_decode_window_tail_direct(_ptr(q), _ptr(k_win), _ptr(v_win), n_win, _ptr(k_tail_host),
                                              _ptr(v_tail_host), n_tail, n_head, n_head_kv, head_dim, split,
                                              tail_split, scale, _ptr(out), _ptr(lse), _ptr(ws), ws_bytes,
                                              _stream(stream))
    _check(rc, "kvattn_decode_window_tail_direct")


def window_tail_direct(q, k_win, v_win, k_tail_host, v_tail_host, *, split, tail_split, scale=None,
                       out=None, lse=None, ws=None, stream=None):
    """Window in HBM + tail read in place from pinned host memory.  q: half [H][D]."""
    import torch
    H, D = q.shape[-2], q.shape[-1]
    Hk = k_win.shape[-2] if k_win is not None else k_tail_host.shape[-2]
    n_win = k_win.shape[0] if k_win is not None else 0
    n_tail = k_tail_host.shape[0] if k_tail_host is not None else 0
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((H, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((H,), dtype=torch.float32, device=q.device)
    if ws is None:
        nbytes = kvattn_window_tail_direct_workspace_bytes(H, Hk, D, n_win, n_tail, split, tail_split)
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    kvattn_decode_window_tail_direct(q, k_win, v_win, n_win, k_tail_host, v_tail_host, n_tail, H, Hk, D, split,
                                     tail_split, scale, out, lse, ws, ws.numel(), stream)
    return out, lse


def kvattn_tail_wait(ctx: int, timeout_ms: int) -> None:
    _check(lib.kvattn_tail_wait(ctx, timeout_ms), "kvattn_tail_wait")


def kvattn_workspace_status(ws, clear: bool = False, stream=None) -> int:
    flags = ctypes.c_uint32(0)
    _check(lib.kvattn_workspace_status(_ptr(ws), ctypes.byref(flags), int(clear), _stream(stream)),
           "kvattn_workspace_status")
    return flags.value


def kvattn_rope_table(n_rot, base, scaling, factor, original_len, turns) -> float:
    """``turns``: host uint64 [n_rot // 2] (numpy).  Returns the gain."""
    gain = _F(0.0)
    _check(lib.kvattn_rope_table(n_rot, base, scaling, factor, original_len, _ptr(turns), ctypes.byref(gain)),
           "kvattn_rope_table")
    return gain.value


def kvattn_rope(q, q_stride, n_head, k, k_stride, n_head_kv, positions, turns, gain, n_rot, layout, n_tok, head_dim, q_out,
                q_out_stride, k_out, k_out_stride, stream=None):
    rc = lib.kvattn_rope(_ptr(q), q_stride, n_head, _ptr(k), k_stride, n_head_kv, _ptr(positions), _ptr(turns), gain, n_rot,
                         layout, n_tok, head_dim, _ptr(q_out), q_out_stride, _ptr(k_out), k_out_stride, _stream(stream))
    _check(rc, "kvattn_rope")


def kvattn_cache_write(k, k_stride, v, v_stride, slots, n_tok, n_head_kv, head_dim, kv_type, k_cache, v_cache, k_scales,
                       v_scales, n_cells, status, stream=None):
    rc = lib.kvattn_cache_write(_ptr(k), k_stride, _ptr(v), v_stride, _ptr(slots), n_tok, n_head_kv, head_dim, kv_type,
                                _ptr(k_cache), _ptr(v_cache), _ptr(k_scales), _ptr(v_scales), n_cells, _ptr(status),
                                _stream(stream))
    _check(rc, "kvattn_cache_write")


def kvattn_cache_read(k_cache, v_cache, k_scales, v_scales, kv_type, n_cells, slots, n_tok, n_head_kv, head_dim, k, k_stride,
                      v, v_stride, status, stream=None):
    rc = lib.kvattn_cache_read(_ptr(k_cache), _ptr(v_cache), _ptr(k_scales), _ptr(v_scales), kv_type, n_cells, _ptr(slots),
                               n_tok, n_head_kv, head_dim, _ptr(k), k_stride, _ptr(v), v_stride, _ptr(status),
                               _stream(stream))
    _check(rc, "kvattn_cache_read")


def kvattn_prefill_workspace_bytes(n_tok, n_seq, n_head, n_head_kv, head_dim) -> int:
    return lib.kvattn_prefill_workspace_bytes(n_tok, n_seq, n_head, n_head_kv, head_dim)


def kvattn_prefill(q, q_stride, k, k_stride, v, v_stride, offsets, n_seq, n_tok, n_head, n_head_kv, head_dim, scale, out, lse,
                   ws, ws_bytes, stream=None):
    rc = lib.kvattn_prefill(_ptr(q), q_stride, _ptr(k), k_stride, _ptr(v), v_stride, _ptr(offsets), n_seq, n_tok, n_head,
                            n_head_kv, head_dim, scale, _ptr(out), _ptr(lse), _ptr(ws), ws_bytes, _stream(stream))
    _check(rc, "kvattn_prefill")


def kvattn_prefill_chunk_workspace_bytes(n_tok, n_seq, n_head, n_head_kv, head_dim, max_len) -> int:
    return lib.kvattn_prefill_chunk_workspace_bytes(n_tok, n_seq, n_head, n_head_kv, head_dim, max_len)


def kvattn_prefill_chunk(q, q_stride, offsets, n_tok, k_cache, v_cache, k_scales, v_scales, kv_type, n_cells, cell_plan,
                         plan_stride, seq_lens, n_seq, max_len, n_head, n_head_kv, head_dim, scale, out, lse, ws,
                         ws_bytes, stream=None):
    rc = lib.kvattn_prefill_chunk(_ptr(q), q_stride, _ptr(offsets), n_tok, _ptr(k_cache), _ptr(v_cache), _ptr(k_scales),
                                  _ptr(v_scales), kv_type, n_cells, _ptr(cell_plan), plan_stride, _ptr(seq_lens), n_seq,
                                  max_len, n_head, n_head_kv, head_dim, scale, _ptr(out), _ptr(lse), _ptr(ws), ws_bytes,
                                  _stream(stream))
    _check(rc, "kvattn_prefill_chunk")


def kvattn_prefill_window(q, q_stride, k, k_stride, v, v_stride, offsets, n_seq, n_tok, n_head, n_head_kv, head_dim, scale,
                          window, sinks, out, lse, ws, ws_bytes, stream=None):
    rc = lib.kvattn_prefill_window(_ptr(q), q_stride, _ptr(k), k_stride, _ptr(v), v_stride, _ptr(offsets), n_seq, n_tok, n_head,
                                   n_head_kv, head_dim, scale, window, sinks, _ptr(out), _ptr(lse), _ptr(ws), ws_bytes,
                                   _stream(stream))
    _check(rc, "kvattn_prefill_window")


def kvattn_prefill_chunk_window(q, q_stride, offsets, n_tok, k_cache, v_cache, k_scales, v_scales, kv_type, n_cells, cell_plan,
                                plan_stride, seq_lens, n_seq, max_len, n_head, n_head_kv, head_dim, scale, window, sinks, out,
                                lse, ws, ws_bytes, stream=None):
    rc = lib.kvattn_prefill_chunk_window(_ptr(q), q_stride, _ptr(offsets), n_tok, _ptr(k_cache), _ptr(v_cache), _ptr(k_scales),
                                         _ptr(v_scales), kv_type, n_cells, _ptr(cell_plan), plan_stride, _ptr(seq_lens), n_seq,
                                         max_len, n_head, n_head_kv, head_dim, scale, window, sinks, _ptr(out), _ptr(lse),
                                         _ptr(ws), ws_bytes, _stream(stream))
    _check(rc, "kvattn_prefill_chunk_window")


def kvattn_prefill_chunk_shared_workspace_bytes(n_tok, n_seq, n_head, n_head_kv, head_dim, max_len) -> int:
    return lib.kvattn_prefill_chunk_shared_workspace_bytes(n_tok, n_seq, n_head, n_head_kv, head_dim, max_len)


def kvattn_prefill_chunk_shared(q, q_stride, offsets, n_tok, k_cache, v_cache, k_scales, v_scales, kv_type, n_cells, cell_plan,
                                plan_stride, seq_lens, n_seq, max_len, n_head, n_head_kv, head_dim, scale, prefix_cells, out,
                                lse, ws, ws_bytes, stream=None):
    rc = lib.kvattn_prefill_chunk_shared(_ptr(q), q_stride, _ptr(offsets), n_tok, _ptr(k_cache), _ptr(v_cache), _ptr(k_scales),
                                         _ptr(v_scales), kv_type, n_cells, _ptr(cell_plan), plan_stride, _ptr(seq_lens), n_seq,
                                         max_len, n_head, n_head_kv, head_dim, scale, prefix_cells, _ptr(out), _ptr(lse),
                                         _ptr(ws), ws_bytes, _stream(stream))
    _check(rc, "kvattn_prefill_chunk_shared")


def kvattn_rope_axes(n_rot, sections, n_axes, order, axis) -> None:
    """``sections``: host int32 [n_axes], ``axis``: host uint8 [n_rot // 2] (numpy)."""
    _check(lib.kvattn_rope_axes(n_rot, _ptr(sections), n_axes, order, _ptr(axis)), "kvattn_rope_axes")


def kvattn_norm_rope(q, q_stride, n_head, q_weight, k, k_stride, n_head_kv, k_weight, eps, positions, pos_stride, n_axes, axis,
                     turns, gain, n_rot, layout, n_tok, head_dim, q_out, q_out_stride, k_out, k_out_stride, stream=None):
    rc = lib.kvattn_norm_rope(_ptr(q), q_stride, n_head, _ptr(q_weight), _ptr(k), k_stride, n_head_kv, _ptr(k_weight), eps,
                              _ptr(positions), pos_stride, n_axes, _ptr(axis), _ptr(turns), gain, n_rot, layout, n_tok, head_dim,
                              _ptr(q_out), q_out_stride, _ptr(k_out), k_out_stride, _stream(stream))
    _check(rc, "kvattn_norm_rope")


def kvattn_step_maps(lens, n_new, n_seq, tables, table_stride, block_cells, free_blocks, n_list, n_free, n_cells, n_tok, offsets,
                     seq_lens, positions, slots, n_free_out, cell_plan, plan_stride, whole_plan, status, stream=None):
    rc = lib.kvattn_step_maps(_ptr(lens), _ptr(n_new), n_seq, _ptr(tables), table_stride, block_cells, _ptr(free_blocks), n_list,
                              _ptr(n_free), n_cells, n_tok, _ptr(offsets), _ptr(seq_lens), _ptr(positions), _ptr(slots),
                              _ptr(n_free_out), _ptr(cell_plan), plan_stride, int(whole_plan), _ptr(status), _stream(stream))
    _check(rc, "kvattn_step_maps")


# ----------------------------- torch conveniences -----------------------------

def _other_stream(stream):
    """Whether ``stream`` is another one than torch's current stream."""
    return stream is not None and _stream(stream) != _stream(None)


def _made_on(stream):
    """A context in which torch allocates, and zeroes, in ``stream``'s order.  What a wrapper makes for
    a call on another stream than the current one has to be that stream's: a block of the current
    stream may still be in use there, would be zeroed there at any time, and goes to the next
    allocation there while the call still runs."""
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        # (1 is the legacy default stream's other handle)
        stream = torch.cuda.default_stream() if handle in (0, 1) else torch.cuda.ExternalStream(handle)
    if stream.device_index != torch.cuda.current_device():
        raise ValueError("stream: a stream of the current device is wanted")
    return torch.cuda.stream(stream)


def decode_workspace(n_seq, n_head, head_dim, max_len, split, device="cuda"):
    import torch
    nbytes = kvattn_decode_workspace_bytes(n_seq, n_head, head_dim, max_len, split)
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)


def decode(q, k_cache, v_cache, seq_lens, *, split, max_len=None, cell_plan=None, k_scales=None,
           v_scales=None, scale=None, n_cells=None, out=None, lse=None, ws=None, stream=None, kv_type=None):
    """q: half [S][H][D] (cuda); K/V as the C ABI describes; seq_lens int32 [S] (cuda).

    ``kv_type`` defaults to f16 without scales, to Q4_0 when K's rows hold head_dim / 2 bytes,
    to Q8_0_Q4_0 when only V's do, and to Q8_0 otherwise.  ``n_cells`` defaults to K's cell dimension (dim 0 for a
    unified cache or a single sequence, dim 1 for a per-sequence [S][N][Hk][D] cache).
    Returns (out, lse).
    """
    import torch
    if (out is None or lse is None or ws is None) and _other_stream(stream):
        with _made_on(stream):
            return decode(q, k_cache, v_cache, seq_lens, split=split, max_len=max_len, cell_plan=cell_plan, k_scales=k_scales,
                          v_scales=v_scales, scale=scale, n_cells=n_cells, out=out, lse=lse, ws=ws, kv_type=kv_type)
    S, H, D = q.shape
    if kv_type is None:
        if k_scales is None:
            kv_type = KVATTN_KV_F16
        else:
            if k_cache.shape[-1] * 2 == D:
                kv_type = KVATTN_KV_Q4_0
            else:
                kv_type = KVATTN_KV_Q8_0_Q4_0 if v_cache.shape[-1] * 2 == D else KVATTN_KV_Q8_0
    Hk = k_cache.shape[-2]
    if n_cells is None:
        n_cells = k_cache.shape[1] if (k_cache.dim() == 4) else k_cache.shape[0]
    plan_stride = 0
    if cell_plan is not None:
        plan_stride = cell_plan.shape[-1]
    if max_len is None:
        max_len = plan_stride if cell_plan is not None else n_cells
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((S, H, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((S, H), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = decode_workspace(S, H, D, max_len, split, device=q.device)
    kvattn_decode(q, k_cache, v_cache, k_scales, v_scales, kv_type, n_cells, cell_plan, plan_stride,
                  seq_lens, S, max_len, H, Hk, D, split, scale, out, lse, ws, ws.numel(), stream)
    return out, lse


def decode_multi(q, k_cache, v_cache, seq_lens, *, split, max_len=None, cell_plan=None, scale=None, n_cells=None,
                 out=None, lse=None, ws=None, stream=None, k_scales=None, v_scales=None):
    """q: half [S][n_q][H][D] (cuda); f16 K/V, or a quantised cache with k_scales / v_scales
    (the type inferred from the row widths as in decode), as the C ABI describes.  Returns
    (out, lse)."""
    import torch
    if (out is None or lse is None or ws is None) and _other_stream(stream):
        with _made_on(stream):
            return decode_multi(q, k_cache, v_cache, seq_lens, split=split, max_len=max_len, cell_plan=cell_plan, scale=scale,
                                n_cells=n_cells, out=out, lse=lse, ws=ws, k_scales=k_scales, v_scales=v_scales)
    S, n_q, H, D = q.shape
    Hk = k_cache.shape[-2]
    if n_cells is None:
        n_cells = k_cache.shape[1] if (k_cache.dim() == 4) else k_cache.shape[0]
    plan_stride = cell_plan.shape[-1] if cell_plan is not None else 0
    if max_len is None:
        max_len = plan_stride if cell_plan is not None else n_cells
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((S, n_q, H, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((S, n_q, H), dtype=torch.float32, device=q.device)
    if ws is None:
        nbytes = kvattn_decode_multi_workspace_bytes(S, n_q, H, D, max_len, split)
        ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    if k_scales is None:
        kv_type = KVATTN_KV_F16
    elif k_cache.shape[-1] * 2 == D:
        kv_type = KVATTN_KV_Q4_0
    else:
        kv_type = KVATTN_KV_Q8_0_Q4_0 if v_cache.shape[-1] * 2 == D else KVATTN_KV_Q8_0
    kvattn_decode_multi(q, k_cache, v_cache, k_scales, v_scales, kv_type, n_cells, cell_plan, plan_stride, seq_lens,
                        S, max_len, n_q, H, Hk, D, split, scale, out, lse, ws, ws.numel(), stream)
    return out, lse


def merge(partials, lses, out=None, lse=None, stream=None):
    """partials float [P][R][D], lses float [P][R] (cuda) -> (out [R][D], lse [R])."""
    import torch
    if (out is None or lse is None) and _other_stream(stream):
        with _made_on(stream):
            return merge(partials, lses, out=out, lse=lse)
    P, R, D = partials.shape
    if out is None:
        out = torch.empty((R, D), dtype=torch.float32, device=partials.device)
    if lse is None:
        lse = torch.empty((R,), dtype=torch.float32, device=partials.device)
    kvattn_merge(partials, lses, P, R, D, out, lse, stream)
    return out, lse


def build_cell_plan(encoded_per_seq, capacity_cells, plan_stride=None):
    """Host helper: list of int64 arrays -> (plan int32 [S][stride], seq_lens int32 [S])."""
    n_seq = len(encoded_per_seq)
    offsets = np.zeros(n_seq + 1, dtype=np.int64)
    for i, e in enumerate(encoded_per_seq):
        offsets[i + 1] = offsets[i] + len(e)
    cells = (np.concatenate([np.asarray(e, dtype=np.int64) for e in encoded_per_seq])
             if n_seq and offsets[-1] else np.zeros(1, dtype=np.int64))
    lens = np.zeros(max(n_seq, 1), dtype=np.int32)
    if plan_stride is None:
        kvattn_build_cell_plan(cells, offsets, n_seq, capacity_cells, None, 0, lens)
        plan_stride = int(lens[:n_seq].max(initial=0))
    plan = np.full((max(n_seq, 1), max(plan_stride, 1)), -1, dtype=np.int32)
    kvattn_build_cell_plan(cells, offsets, n_seq, capacity_cells, plan, plan_stride, lens)
    return plan[:n_seq, :plan_stride], lens[:n_seq]


# The wrappers below are on the path of single decode steps, where the host's time counts: each
# reads a tensor's shape and strides once, and calls the library itself with addresses.

def _rows(x, name):
    """(tokens, heads, head_dim, token stride) of half rows [T][heads][D]; the heads of a token must
    be contiguous, the tokens may be strided (a slice of a fused projection)."""
    if x.dtype is not _F16 or x.dim() != 3:
        raise ValueError(f"{name}: half rows [tokens][heads][head_dim] are wanted")
    t, h, d = x.shape
    st, sh, sd = x.stride()
    if (sd != 1 or (h > 1 and sh != d)) and x.numel():
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t, h, d, (st if t > 1 else h * d)


def _ints(x, name, n=None):
    if x.dtype is not _I32 or not x.is_contiguous() or (n is not None and x.numel() != n):
        raise ValueError(f"{name}: contiguous int32" + ("" if n is None else f" of {n} values") + " is wanted")
    return x.data_ptr()


def _here(x, name):
    """The device of x; refuses a host tensor, or one of another device than the current one, whose
    stream is used."""
    d = x.get_device()
    if d < 0 or d != _current_device():
        raise ValueError(f"{name}: a tensor of the current CUDA device is wanted")
    return d


def _elsewhere(dev, **tensors):
    """Names the tensor that is not on device ``dev`` (or the workspace's or status word's other fault)."""
    for name, x in tensors.items():
        if x is not None and x.get_device() != dev:
            raise ValueError(f"{name}: a tensor of the current CUDA device is wanted")
    raise ValueError("ws is contiguous; status holds a 32-bit word")


def _off(x, dev):
    return x is not None and x.get_device() != dev


def _bad_word(status, dev):
    return status is not None and (status.get_device() != dev or status.numel() * status.element_size() < 4)


def _bad_ws(ws, dev):
    return ws.get_device() != dev or not ws.is_contiguous()


def _raw(x):
    return None if x is None else x.data_ptr()


def _new_out(out, name, shape, like, dtype=None):
    """A contiguous result tensor: the caller's, checked, or a new one."""
    dtype = _F16 if dtype is None else dtype
    if out is None:
        return _torch.empty(shape, dtype=dtype, device=like.device)
    if out.shape != shape or out.dtype is not dtype or not out.is_contiguous():
        raise ValueError(f"{name}: contiguous {dtype} of shape {tuple(shape)} is wanted")
    return out


_QUANTISED = {(8, 8): KVATTN_KV_Q8_0, (8, 4): KVATTN_KV_Q8_0_Q4_0, (4, 4): KVATTN_KV_Q4_0}  # by bits of K and V


def _cache_type(k_cache, v_cache, k_scales, v_scales, head_dim):
    """(kv_type, KV heads, cells) from the planes, the type by the row widths as in decode; checks
    the planes' shapes, types and layout."""
    ks, vs = k_cache.shape, v_cache.shape
    if k_scales is None and v_scales is None:
        kv_type = KVATTN_KV_F16
        good = ks == vs and ks[-1] == head_dim and k_cache.dtype is v_cache.dtype is _F16
    elif k_scales is None or v_scales is None:
        raise ValueError("k_scales and v_scales go together")
    else:
        kb = 8 if ks[-1] == head_dim else 4
        vb = 8 if vs[-1] == head_dim else 4
        kv_type = _QUANTISED.get((kb, vb))
        want = ks[:-1] + (head_dim // 32,)
        good = (kv_type is not None and ks[:-1] == vs[:-1] and ks[-1] * 8 == head_dim * kb and vs[-1] * 8 == head_dim * vb
                and k_cache.dtype is (_torch.int8 if kb == 8 else _torch.uint8)
                and v_cache.dtype is (_torch.int8 if vb == 8 else _torch.uint8)
                and k_scales.dtype is v_scales.dtype is _F16 and k_scales.shape == want and v_scales.shape == want
                and k_scales.is_contiguous() and v_scales.is_contiguous())
    if len(ks) < 3 or not good or not k_cache.is_contiguous() or not v_cache.is_contiguous():
        raise ValueError("the cache planes are contiguous [cells][kv heads][row] of one type's rows, codes int8 or packed "
                         "uint8, scales half [cells][kv heads][head_dim / 32]")
    return kv_type, ks[-2], math.prod(ks[:-2])


class RopeTable:
    """Angles per position of a model's rotary pairs (``turns``, device uint64 kept as int64: 2^64
    theta / (2 pi)) and the gain on cosine and sine; with several axes of positions also each pair's
    ``axis`` (device uint8).  Made by :func:`rope_table`, or by a program from frequencies of its own."""

    def __init__(self, turns, gain, n_rot, axis=None, n_axes=1):
        self.turns, self.gain, self.n_rot, self.axis, self.n_axes = turns, gain, n_rot, axis, n_axes


def rope_table(n_rot, *, base=10000.0, scaling="none", factor=1.0, original=0, sections=None, order="blocks", restart=False,
               device="cuda"):
    """``scaling``: "none", "linear" or "yarn" (``factor`` times the ``original`` context; the paper's
    ramp, see kvattn_rope_table: a model trained with another one needs a RopeTable of its own).
    ``sections``: pairs of each axis of positions (one to four axes, n_rot / 2 pairs in all), in
    consecutive blocks or dealt out in turn (``order`` "blocks" or "cycle"); ``restart``: each axis has
    the frequencies of a head of its own pairs alone, instead of the pairs' own."""
    import torch
    kind = {"none": KVATTN_ROPE_PLAIN, "linear": KVATTN_ROPE_LINEAR, "yarn": KVATTN_ROPE_YARN}[scaling]
    host = np.zeros(n_rot // 2, dtype=np.uint64)
    gain = kvattn_rope_table(n_rot, base, kind, factor, original, host)
    axis, n_axes = None, 1
    if sections is not None:
        n_axes, counts, of = len(sections), np.array(sections, dtype=np.int32), np.zeros(n_rot // 2, dtype=np.uint8)
        kvattn_rope_axes(n_rot, counts, n_axes, {"blocks": KVATTN_AXES_BLOCKS, "cycle": KVATTN_AXES_CYCLE}[order], of)
        if restart:
            for a, count in enumerate(sections):
                own = np.zeros(count, dtype=np.uint64)
                if count:
                    kvattn_rope_table(2 * count, base, kind, factor, original, own)
                host[of == a] = own
        axis = torch.from_numpy(of).to(device)
    return RopeTable(torch.from_numpy(host.view(np.int64)).to(device), gain, n_rot, axis, n_axes)


def rope(q, k, positions, table, *, layout="half", q_out=None, k_out=None, stream=None):
    """q: half [T][H][D], k: half [T][Hk][D] (either may be None), positions int32 [T], or [axes][T] with
    a table of several axes.  Rotated rows go to new tensors, or to ``q_out`` / ``k_out`` (which may be q
    and k themselves).  Returns (q, k)."""
    if table.axis is not None:
        return norm_rope(q, k, positions, table, layout=layout, q_out=q_out, k_out=k_out, stream=stream)
    if _torch is None:
        _bind_torch()
    code = KVATTN_ROPE_HALF if layout == "half" else {"interleaved": KVATTN_ROPE_INTERLEAVED}[layout]
    if q is None and k is None:
        raise ValueError("q or k is wanted")
    if ((q is not None and q_out is None) or (k is not None and k_out is None)) and _other_stream(stream):
        with _made_on(stream):
            return rope(q, k, positions, table, layout=layout, q_out=q_out, k_out=k_out)
    T = D = None
    qa = ka = (None, 0, 0, None, 0)
    if q is not None:
        if q_out is None:
            q_out = _torch.empty(q.shape, dtype=_F16, device=q.device)
        T, h, D, st = _rows(q, "q")
        to, ho, do, so = _rows(q_out, "q_out")
        if to != T or ho != h or do != D:
            raise ValueError("q_out: q's shape is wanted")
        qa = (q.data_ptr(), st, h, q_out.data_ptr(), so)
    if k is not None:
        if k_out is None:
            k_out = _torch.empty(k.shape, dtype=_F16, device=k.device)
        t, h, d, st = _rows(k, "k")
        to, ho, do, so = _rows(k_out, "k_out")
        if to != t or ho != h or do != d or (q is not None and (t != T or d != D)):
            raise ValueError("k, k_out: shapes do not agree")
        T, D = t, d
        ka = (k.data_ptr(), st, h, k_out.data_ptr(), so)
    at, turns = _ints(positions, "positions", T), table.turns
    d = _here(k if q is None else q, "k" if q is None else "q")
    if positions.get_device() != d or turns.get_device() != d or _off(k, d) or _off(q_out, d) or _off(k_out, d):
        _elsewhere(d, k=k, positions=positions, table=turns, q_out=q_out, k_out=k_out)
    if turns.numel() * 2 < table.n_rot or turns.element_size() != 8 or not turns.is_contiguous():
        raise ValueError("table: n_rot / 2 contiguous 64-bit angles are wanted")
    _check(lib.kvattn_rope(qa[0], qa[1], qa[2], ka[0], ka[1], ka[2], at, turns.data_ptr(), table.gain, table.n_rot, code,
                           T, D, qa[3], qa[4], ka[3], ka[4], _stream(stream)), "kvattn_rope")
    return q_out if q is not None else None, k_out if k is not None else None


def _weight(w, name, n):
    if w.dtype is not _F16 or w.numel() != n or not w.is_contiguous():
        raise ValueError(f"{name}: contiguous half of head_dim values is wanted")
    return w.data_ptr()


def norm_rope(q, k, positions, table, *, q_weight=None, k_weight=None, eps=1e-6, layout="half", q_out=None, k_out=None,
              stream=None):
    """:func:`rope` of heads that are normed first, in the same pass: ``q_weight`` / ``k_weight`` half
    [D] (None: that side is not normed), ``eps`` beside the mean square.  ``positions`` as there: a row of
    tokens for each axis, [axes][T]."""
    if _torch is None:
        _bind_torch()
    code = KVATTN_ROPE_HALF if layout == "half" else {"interleaved": KVATTN_ROPE_INTERLEAVED}[layout]
    if q is None and k is None:
        raise ValueError("q or k is wanted")
    if ((q is not None and q_out is None) or (k is not None and k_out is None)) and _other_stream(stream):
        with _made_on(stream):
            return norm_rope(q, k, positions, table, q_weight=q_weight, k_weight=k_weight, eps=eps, layout=layout, q_out=q_out,
                             k_out=k_out)
    T = D = None
    qa = ka = (None, 0, 0, None, 0)
    if q is not None:
        if q_out is None:
            q_out = _torch.empty(q.shape, dtype=_F16, device=q.device)
        T, h, D, st = _rows(q, "q")
        to, ho, do, so = _rows(q_out, "q_out")
        if to != T or ho != h or do != D:
            raise ValueError("q_out: q's shape is wanted")
        qa = (q.data_ptr(), st, h, q_out.data_ptr(), so)
    if k is not None:
        if k_out is None:
            k_out = _torch.empty(k.shape, dtype=_F16, device=k.device)
        t, h, d, st = _rows(k, "k")
        to, ho, do, so = _rows(k_out, "k_out")
        if to != t or ho != h or do != d or (q is not None and (t != T or d != D)):
            raise ValueError("k, k_out: shapes do not agree")
        T, D = t, d
        ka = (k.data_ptr(), st, h, k_out.data_ptr(), so)
    turns, axis, n_axes, n_rot = table.turns, table.axis, table.n_axes, table.n_rot
    at = _ints(positions, "positions", T * n_axes)
    if n_axes > 1 and tuple(positions.shape) != (n_axes, T):   # (not [T][axes], which holds as many)
        raise ValueError(f"positions: [axes][T] is wanted, {n_axes} rows of {T} tokens")
    d = _here(k if q is None else q, "k" if q is None else "q")
    if (positions.get_device() != d or turns.get_device() != d or _off(k, d) or _off(q_out, d) or _off(k_out, d)
            or _off(q_weight, d) or _off(k_weight, d) or _off(axis, d)):
        _elsewhere(d, k=k, positions=positions, table=turns, axis=axis, q_weight=q_weight, k_weight=k_weight, q_out=q_out,
                   k_out=k_out)
    qw = kw = None
    if q_weight is not None:
        qw = _weight(q_weight, "q_weight", D)
    if k_weight is not None:
        kw = _weight(k_weight, "k_weight", D)
    if turns.numel() * 2 < n_rot or turns.element_size() != 8 or not turns.is_contiguous():
        raise ValueError("table: n_rot / 2 contiguous 64-bit angles are wanted")
    if n_axes > 1 and (axis is None or axis.numel() * 2 < n_rot or axis.element_size() != 1 or not axis.is_contiguous()):
        raise ValueError("table: n_rot / 2 contiguous 8-bit axes are wanted")
    _check(lib.kvattn_norm_rope(qa[0], qa[1], qa[2], qw, ka[0], ka[1], ka[2], kw, eps, at, T, n_axes,
                                _raw(axis), turns.data_ptr(), table.gain, n_rot, code, T, D, qa[3], qa[4], ka[3], ka[4],
                                _stream(stream)), "kvattn_norm_rope")
    return q_out if q is not None else None, k_out if k is not None else None


class StepMaps:
    """What :func:`step_maps` makes: int32 ``offsets`` [S + 1], ``seq_lens`` [S], ``positions`` [T],
    ``slots`` [T] and ``n_free`` [1]; made by :func:`step_maps_buffers`, and written by any number of
    steps.  A step without a free list leaves ``n_free`` as it is: 0 in new buffers, None in what
    :func:`step_maps` made for such a step."""
    __slots__ = ("_all", "_at", "_no_count")

    def __init__(self, n_seq, n_tok, device):
        import torch
        # one allocation; each tensor on 16 bytes
        counts = (n_seq + 1, n_seq, n_tok, n_tok, 1)
        room = torch.empty(sum(-(-n // 4) * 4 for n in counts), dtype=torch.int32, device=device)
        views, at = [], 0
        for n in counts:
            views.append(room[at:at + n])
            at += -(-n // 4) * 4
        self._all = tuple(views)
        self._at = (n_seq, n_tok, room.get_device()) + tuple(room.data_ptr() + 4 * x.storage_offset() for x in views)
        self._no_count = False

    offsets = property(lambda self: self._all[0])
    seq_lens = property(lambda self: self._all[1])
    positions = property(lambda self: self._all[2])
    slots = property(lambda self: self._all[3])
    n_free = property(lambda self: None if self._no_count else self._all[4])


def step_maps_buffers(n_seq, n_tok, device="cuda"):
    """A StepMaps for steps of ``n_seq`` sequences and at most ``n_tok`` tokens."""
    made = StepMaps(n_seq, n_tok, device)
    made.n_free.zero_()
    return made


def step_maps(lens, n_new, tables, free_blocks=None, n_free=None, *, block_cells, n_cells, n_tok=None, plan=None,
              whole_plan=True, status=None, out=None, stream=None):
    """A step's maps from the sequences' lengths and new tokens (int32 [S]): blocks of ``block_cells``
    cells are taken from the end of ``free_blocks`` (int32, the first ``n_free`` [1] of them free; None:
    nothing is taken) into ``tables`` (int32 [S][stride], in place), and the offsets, lengths, positions
    and slots of ``n_tok`` packed rows follow (rows behind the last token: slot -1).  ``plan`` (int32
    [S][stride]): the cell plan, whole rows or the new tokens' entries.  ``out``: a StepMaps to write
    (of a step before: its ``seq_lens`` must not be this one's ``lens``, nor its ``n_free``).  Returns a
    StepMaps."""
    if _torch is None:
        _bind_torch()
    if out is None:
        if n_tok is None:
            raise ValueError("n_tok or out is wanted")
        if _other_stream(stream):
            with _made_on(stream):
                out = StepMaps(lens.numel(), n_tok, lens.device)
        else:
            out = StepMaps(lens.numel(), n_tok, lens.device)
        out._no_count = True   # (until a step counts)
    S, T, d, offsets, seq_lens, positions, slots, left = out._at
    if n_tok is not None and n_tok != T:
        raise ValueError("n_tok: out has other rows")
    _here(lens, "lens")
    shape = tables.shape
    if len(shape) != 2 or shape[0] != S:
        raise ValueError("tables: a row for each sequence is wanted")
    if (lens.get_device() != d or n_new.get_device() != d or tables.get_device() != d or _off(free_blocks, d)
            or _off(n_free, d) or _off(plan, d) or (status is not None and _bad_word(status, d))):
        _elsewhere(d, lens=lens, n_new=n_new, tables=tables, free_blocks=free_blocks, n_free=n_free, plan=plan, status=status)
    a, b, tab = _ints(lens, "lens", S), _ints(n_new, "n_new", S), _ints(tables, "tables")
    pl, stride, free, count, n_list = None, 0, None, None, 0
    if plan is not None:
        pl, rows = _ints(plan, "plan"), plan.shape
        if len(rows) != 2 or rows[0] != S:
            raise ValueError("plan: a row for each sequence is wanted")
        stride = rows[1]
    if free_blocks is not None and n_free is not None:
        free, count, n_list = _ints(free_blocks, "free_blocks"), _ints(n_free, "n_free", 1), free_blocks.numel()
        if n_list == 0:
            free = count   # (torch gives an empty list no address; nothing is read of it)
    elif free_blocks is not None or n_free is not None:
        raise ValueError("free_blocks and n_free go together")
    else:
        left = None
    if left is not None:
        out._no_count = False
    _check(lib.kvattn_step_maps(a, b, S, tab, shape[1], block_cells, free, n_list, count, n_cells, T, offsets, seq_lens, positions,
                                slots, left, pl, stride, 1 if whole_plan else 0, _raw(status), _stream(stream)), "kvattn_step_maps")
    return out


def cache_write(k, v, slots, k_cache, v_cache, *, k_scales=None, v_scales=None, status=None, stream=None):
    """k, v: half [T][Hk][D] into cells ``slots`` (int32 [T], -1: skipped; None: cells 0 .. T - 1) of a
    cache whose type follows from its planes.  ``status``: an int32 tensor whose first word collects
    the KVATTN_DEVICE_* bits."""
    if _torch is None:
        _bind_torch()
    T, Hk, D, ks = _rows(k, "k")
    vt, vh, vd, vs = _rows(v, "v")
    kv_type, heads, n_cells = _cache_type(k_cache, v_cache, k_scales, v_scales, D)
    if (vt, vh, vd) != (T, Hk, D) or heads != Hk:
        raise ValueError("k, v and the cache do not agree")
    at = None if slots is None else _ints(slots, "slots", T)
    d = _here(k, "k")
    if (v.get_device() != d or k_cache.get_device() != d or v_cache.get_device() != d or _off(slots, d) or _off(k_scales, d)
            or _off(v_scales, d) or _bad_word(status, d)):
        _elsewhere(d, v=v, k_cache=k_cache, v_cache=v_cache, slots=slots, k_scales=k_scales, v_scales=v_scales, status=status)
    _check(lib.kvattn_cache_write(k.data_ptr(), ks, v.data_ptr(), vs, at, T, Hk, D, kv_type, k_cache.data_ptr(),
                                  v_cache.data_ptr(), _raw(k_scales), _raw(v_scales), n_cells, _raw(status), _stream(stream)),
           "kvattn_cache_write")


def cache_read(k_cache, v_cache, slots=None, *, head_dim, k_scales=None, v_scales=None, k_out=None, v_out=None, status=None,
               stream=None):
    """Cells ``slots`` (int32 [T], e.g. a row of a cell plan; -1 gives zeros; None: every cell) as
    half [T][Hk][head_dim] rows.  Returns (k, v)."""
    if _torch is None:
        _bind_torch()
    if (k_out is None or v_out is None) and _other_stream(stream):
        with _made_on(stream):
            return cache_read(k_cache, v_cache, slots, head_dim=head_dim, k_scales=k_scales, v_scales=v_scales, k_out=k_out,
                              v_out=v_out, status=status)
    kv_type, Hk, n_cells = _cache_type(k_cache, v_cache, k_scales, v_scales, head_dim)
    T, at = (n_cells, None) if slots is None else (slots.numel(), _ints(slots, "slots"))
    if k_out is None:
        k_out = _torch.empty((T, Hk, head_dim), dtype=_F16, device=k_cache.device)
    if v_out is None:
        v_out = _torch.empty((T, Hk, head_dim), dtype=_F16, device=k_cache.device)
    d = _here(k_cache, "k_cache")
    if (v_cache.get_device() != d or k_out.get_device() != d or v_out.get_device() != d or _off(slots, d) or _off(k_scales, d)
            or _off(v_scales, d) or _bad_word(status, d)):
        _elsewhere(d, v_cache=v_cache, slots=slots, k_scales=k_scales, v_scales=v_scales, k_out=k_out, v_out=v_out,
                   status=status)
    kt, kh, kd, ks = _rows(k_out, "k_out")
    vt, vh, vd, vs = _rows(v_out, "v_out")
    if (kt, kh, kd) != (T, Hk, head_dim) or (vt, vh, vd) != (T, Hk, head_dim):
        raise ValueError("k_out and v_out are half [slots][kv heads][head_dim]")
    _check(lib.kvattn_cache_read(k_cache.data_ptr(), v_cache.data_ptr(), _raw(k_scales), _raw(v_scales), kv_type, n_cells, at,
                                 T, Hk, head_dim, k_out.data_ptr(), ks, v_out.data_ptr(), vs, _raw(status), _stream(stream)),
           "kvattn_cache_read")
    return k_out, v_out


def prefill_workspace(n_tok, n_seq, n_head, n_head_kv, head_dim, device="cuda"):
    import torch
    nbytes = kvattn_prefill_workspace_bytes(n_tok, n_seq, n_head, n_head_kv, head_dim)
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)


def prefill(q, k, v, offsets, *, scale=None, window=None, sinks=0, out=None, lse=None, ws=None, stream=None):
    """Causal attention of packed prompts: q half [T][H][D], k and v half [T][Hk][D], offsets int32
    [S + 1].  With a ``window`` a token sees its sequence's last ``window`` tokens (its own among them)
    and the first ``sinks``.  Returns (out half [T][H][D], lse float [T][H])."""
    if _torch is None:
        _bind_torch()
    if (out is None or lse is None or ws is None) and _other_stream(stream):
        with _made_on(stream):
            return prefill(q, k, v, offsets, scale=scale, window=window, sinks=sinks, out=out, lse=lse, ws=ws)
    T, H, D, qs = _rows(q, "q")
    kt, Hk, kd, ks = _rows(k, "k")
    vt, vh, vd, vs = _rows(v, "v")
    if (kt, kd) != (T, D) or (vt, vh, vd) != (T, Hk, D):
        raise ValueError("q, k and v do not agree")
    off, S = _ints(offsets, "offsets"), offsets.numel() - 1
    d = _here(q, "q")
    out = _new_out(out, "out", (T, H, D), q)
    lse = _new_out(lse, "lse", (T, H), q, _torch.float32)
    if ws is None:
        ws = prefill_workspace(T, S, H, Hk, D, q.device)
    if (k.get_device() != d or v.get_device() != d or offsets.get_device() != d or out.get_device() != d
            or lse.get_device() != d or _bad_ws(ws, d)):
        _elsewhere(d, k=k, v=v, offsets=offsets, out=out, lse=lse, ws=ws)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if window is not None:
        _check(lib.kvattn_prefill_window(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, off, S, T, H, Hk, D, scale, window,
                                         sinks, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)),
               "kvattn_prefill_window")
        return out, lse
    if sinks:
        raise ValueError("sinks: with a window only")
    _check(lib.kvattn_prefill(q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, off, S, T, H, Hk, D, scale, out.data_ptr(),
                              lse.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)), "kvattn_prefill")
    return out, lse


def prefill_chunk_workspace(n_tok, n_seq, n_head, n_head_kv, head_dim, max_len, device="cuda", shared=0):
    """For calls with ``shared`` cells, whatever their number, when ``shared`` is not 0."""
    import torch
    query = kvattn_prefill_chunk_shared_workspace_bytes if shared else kvattn_prefill_chunk_workspace_bytes
    nbytes = query(n_tok, n_seq, n_head, n_head_kv, head_dim, max_len)
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)


def prefill_chunk(q, offsets, k_cache, v_cache, seq_lens, *, max_len=None, n_cells=None, cell_plan=None, k_scales=None,
                  v_scales=None, scale=None, window=None, sinks=0, shared=0, out=None, lse=None, ws=None, stream=None):
    """Causal attention of new tokens over caches that hold their cells: q half [T][H][D] (the
    sequences' tokens packed, offsets int32 [S + 1]), the cache as in decode: one unified cache with
    a ``cell_plan`` (int32 [S][stride]), a per-sequence [S][N][Hk][D] cache, or one [cells][Hk][D]
    whose ``n_cells`` are each sequence's.  With a ``window`` a token sees its sequence's last ``window``
    cells (its own among them) and the first ``sinks``; with ``shared`` the sequences' first ``shared``
    cells hold the same and are read once for all of them (one or the other), which pays for steps of a few
    tokens each and not for prompts (see kvattn_prefill_chunk_shared).  Returns (out half [T][H][D],
    lse: the given tensor or None)."""
    if _torch is None:
        _bind_torch()
    if (out is None or ws is None) and _other_stream(stream):
        with _made_on(stream):
            return prefill_chunk(q, offsets, k_cache, v_cache, seq_lens, max_len=max_len, n_cells=n_cells, cell_plan=cell_plan,
                                 k_scales=k_scales, v_scales=v_scales, scale=scale, window=window, sinks=sinks, shared=shared,
                                 out=out, lse=lse, ws=ws)
    T, H, D, qs = _rows(q, "q")
    off, S = _ints(offsets, "offsets"), offsets.numel() - 1
    lens = _ints(seq_lens, "seq_lens", S)
    kv_type, Hk, rows = _cache_type(k_cache, v_cache, k_scales, v_scales, D)
    if n_cells is None:
        per_sequence = k_cache.dim() == 4 and cell_plan is None
        n_cells = k_cache.shape[1] if per_sequence else rows
    plan, stride = None, 0
    if cell_plan is not None:
        stride = cell_plan.shape[-1]
        plan = _ints(cell_plan, "cell_plan", S * stride)
    if (n_cells if plan is not None else n_cells * S) > rows:
        raise ValueError("the cache has fewer cells than n_cells says")
    if max_len is None:
        max_len = stride if plan is not None else n_cells
    d = _here(q, "q")
    out = _new_out(out, "out", (T, H, D), q)
    if lse is not None:
        _new_out(lse, "lse", (T, H), q, _torch.float32)
    if ws is None:
        ws = prefill_chunk_workspace(T, S, H, Hk, D, max_len, q.device, shared)
    if (k_cache.get_device() != d or v_cache.get_device() != d or offsets.get_device() != d or seq_lens.get_device() != d
            or out.get_device() != d or _off(cell_plan, d) or _off(k_scales, d) or _off(v_scales, d) or _off(lse, d)
            or _bad_ws(ws, d)):
        _elsewhere(d, k_cache=k_cache, v_cache=v_cache, offsets=offsets, seq_lens=seq_lens, cell_plan=cell_plan,
                   k_scales=k_scales, v_scales=v_scales, out=out, lse=lse, ws=ws)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if window is None and not shared:
        if sinks:
            raise ValueError("sinks: with a window only")
        _check(lib.kvattn_prefill_chunk(q.data_ptr(), qs, off, T, k_cache.data_ptr(), v_cache.data_ptr(), _raw(k_scales),
                                        _raw(v_scales), kv_type, n_cells, plan, stride, lens, S, max_len, H, Hk, D, scale,
                                        out.data_ptr(), _raw(lse), ws.data_ptr(), ws.numel(), _stream(stream)),
               "kvattn_prefill_chunk")
    elif window is not None:
        if shared:
            raise ValueError("window or shared, not both")
        _check(lib.kvattn_prefill_chunk_window(q.data_ptr(), qs, off, T, k_cache.data_ptr(), v_cache.data_ptr(), _raw(k_scales),
                                               _raw(v_scales), kv_type, n_cells, plan, stride, lens, S, max_len, H, Hk, D, scale,
                                               window, sinks, out.data_ptr(), _raw(lse), ws.data_ptr(), ws.numel(),
                                               _stream(stream)), "kvattn_prefill_chunk_window")
    else:
        if sinks:
            raise ValueError("sinks: with a window only")
        _check(lib.kvattn_prefill_chunk_shared(q.data_ptr(), qs, off, T, k_cache.data_ptr(), v_cache.data_ptr(), _raw(k_scales),
                                               _raw(v_scales), kv_type, n_cells, plan, stride, lens, S, max_len, H, Hk, D, scale,
                                               shared, out.data_ptr(), _raw(lse), ws.data_ptr(), ws.numel(), _stream(stream)),
               "kvattn_prefill_chunk_shared")
    return out, lse


class WindowTail:
    """Owns a tail context (events only) and runs kvattn_decode_window_tail.

    ``prefetch=True`` sets KVATTN_TAIL_PREFETCH: one context serves every layer of a model,
    and a layer's tail copies wait only for the decode that last read their staging slot,
    not for the layers before it."""

    def __init__(self, prefetch=False):
        self.ctx = kvattn_tail_ctx_create()
        if prefetch:
            kvattn_tail_ctx_set_flags(self.ctx, KVATTN_TAIL_PREFETCH)

    def close(self):
        if self.ctx:
            kvattn_tail_ctx_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def workspace(n_head, n_head_kv, head_dim, n_win, n_tail, split, tile_cells, tail_split,
                  device="cuda"):
        import torch
        nbytes = kvattn_window_tail_workspace_bytes(n_head, n_head_kv, head_dim, n_win, n_tail,
                                                    split, tile_cells, tail_split)
        if nbytes == 0:
            raise KvattnError(KVATTN_ERR_INVALID_ARG, "kvattn_window_tail_workspace_bytes")
        return torch.zeros(nbytes, dtype=torch.uint8, device=device)

    def __call__(self, q, k_win, v_win, k_tail_host, v_tail_host, *, split, tile_cells, tail_split,
                 scale=None, out=None, lse=None, ws=None, compute_stream=None, copy_stream=None):
        import torch
        if (out is None or lse is None or ws is None) and _other_stream(compute_stream):
            copy_stream = _stream(copy_stream)   # (None: the current one here)
            with _made_on(compute_stream):
                return self(q, k_win, v_win, k_tail_host, v_tail_host, split=split, tile_cells=tile_cells,
                            tail_split=tail_split, scale=scale, out=out, lse=lse, ws=ws, copy_stream=copy_stream)
        H, D = q.shape[-2], q.shape[-1]
        Hk = k_win.shape[-2] if k_win is not None else k_tail_host.shape[-2]
        n_win = k_win.shape[0] if k_win is not None else 0
        n_tail = k_tail_host.shape[0] if k_tail_host is not None else 0
        if scale is None:
            scale = 1.0 / math.sqrt(D)
        if out is None:
            out = torch.empty((H, D), dtype=torch.float32, device=q.device)
        if lse is None:
            lse = torch.empty((H,), dtype=torch.float32, device=q.device)
        if ws is None:
            ws = self.workspace(H, Hk, D, n_win, n_tail, split, tile_cells, tail_split, q.device)
        kvattn_decode_window_tail(self.ctx, q, k_win, v_win, n_win, k_tail_host, v_tail_host, n_tail,
                                  tile_cells, H, Hk, D, split, tail_split, scale, out, lse, ws,
                                  ws.numel(), compute_stream, copy_stream)
        return out, lse
