"""DSA Lightning Indexer scoring fused with exact top-K on MI355X (gfx950).

Thin ctypes binding of libidxtopk.so (C ABI in include/idx_topk.h).  This
module only marshals arguments: torch supplies device memory and the current
stream; every step of the computation runs in the library's HIP kernels.
Importing raises if the library has not been built (run
``python scoring_exact_top_amd/build.py`` or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libidxtopk.so")

HEADS = 64
DIM = 128
KMAX = 2048
PAGE = 64

if not os.path.exists(LIB_PATH):
    raise ImportError("libidxtopk.so is not built at %s; run python scoring_exact_top_amd/build.py"
                      % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)
_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_sz = ctypes.c_size_t


class Opts(ctypes.Structure):
    _fields_ = [("force_tau", ctypes.c_int32), ("tau_value", ctypes.c_float),
                ("cand_cap", ctypes.c_int32),
                ("ev_main_start", ctypes.c_void_p), ("ev_main_stop", ctypes.c_void_p),
                ("main_reps", ctypes.c_int32), ("row_status", ctypes.c_void_p),
                ("clock_out", ctypes.c_void_p), ("math_only", ctypes.c_int32)]


# Row outcomes written to row_status (idx_topk.h IDX_ROW_*).
ROW_FAST, ROW_UNDERFLOW, ROW_OVERFLOW, ROW_BAD = 0, 1, 2, -1


class Stats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in
                ("rows", "fast_ok", "underflow", "overflow", "many_cands", "repaired", "trivial",
                 "bad_rows")]

    def asdict(self):
        return {n: int(getattr(self, n)) for n, _ in self._fields_}


_lib.idx_topk_prefill_workspace.restype = _sz
_lib.idx_topk_prefill_workspace.argtypes = [_i32, _i32, _i32]
_lib.idx_topk_prefill_geometry.restype = _i32
_lib.idx_topk_prefill_geometry.argtypes = [_i32, _i32, ctypes.POINTER(_i32), ctypes.POINTER(_i32), ctypes.POINTER(_i32)]
_lib.idx_topk_prefill.restype = ctypes.c_int
_lib.idx_topk_prefill.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _vp, _sz,
                                  _vp]
_lib.idx_topk_prefill_debug.restype = ctypes.c_int
_lib.idx_topk_prefill_debug.argtypes = _lib.idx_topk_prefill.argtypes + [_vp, _vp,
                                                                          ctypes.POINTER(Opts)]
_lib.idx_topk_prefill_unfused_workspace.restype = _sz
_lib.idx_topk_prefill_unfused_workspace.argtypes = [_i32, _i32, _i32]
_lib.idx_topk_prefill_unfused.restype = ctypes.c_int
_lib.idx_topk_prefill_unfused.argtypes = _lib.idx_topk_prefill.argtypes + [ctypes.POINTER(Opts)]
_lib.idx_topk_rows.restype = ctypes.c_int
_lib.idx_topk_rows.argtypes = [_vp, ctypes.c_int64, _vp, _vp, _i32, _vp, _i32, _i32, _vp]
_lib.idx_topk_scan_bf16_workspace.restype = _sz
_lib.idx_topk_scan_bf16_workspace.argtypes = [_i32, _i32, _i32]
_lib.idx_topk_scan_bf16.restype = ctypes.c_int
_lib.idx_topk_scan_bf16.argtypes = [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _sz, _vp,
                                    ctypes.POINTER(Opts)]
_lib.idx_topk_scan_bf16_scores.restype = ctypes.c_void_p
_lib.idx_topk_scan_bf16_scores.argtypes = [_vp, _i32, _i32]
_lib.idx_topk_stream_floor.restype = ctypes.c_int
_lib.idx_topk_stream_floor.argtypes = [_vp, ctypes.c_int64, _vp, _vp]
_lib.idx_topk_decode_workspace.restype = _sz
_lib.idx_topk_decode_workspace.argtypes = [_i32, _i32, _i32, _i32]
_lib.idx_topk_decode_paged.restype = ctypes.c_int
_lib.idx_topk_decode_paged.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                       _i32, _vp, _vp, _sz, _vp]
_lib.idx_topk_decode_paged_debug.restype = ctypes.c_int
_lib.idx_topk_decode_paged_debug.argtypes = _lib.idx_topk_decode_paged.argtypes + [_vp, ctypes.POINTER(Opts)]
_lib.idx_topk_decode_paged_noalloc.restype = ctypes.c_int
_lib.idx_topk_decode_paged_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp]
_lib.idx_topk_read_stats.restype = ctypes.c_int
_lib.idx_topk_read_stats.argtypes = [_vp, ctypes.POINTER(Stats), _vp]
_lib.idx_topk_strerror.restype = ctypes.c_char_p
_lib.idx_topk_strerror.argtypes = [ctypes.c_int]


class IdxTopkError(RuntimeError):
    def __init__(self, code: int):
        super().__init__("idx_topk error %d: %s" % (code, _lib.idx_topk_strerror(code).decode()))
        self.code = code


def _check(rc: int):
    if rc != 0:
        raise IdxTopkError(rc)


def _ptr(t: Optional[torch.Tensor], dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError("expected dtype %s, got %s" % (dtype, t.dtype))
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def prefill_workspace_bytes(Q: int, N: int, K: int) -> int:
    return int(_lib.idx_topk_prefill_workspace(Q, N, K))


def prefill_geometry(Q: int, N: int):
    """(shared, splits, segments) of the main kernel's walk for Q rows over
    N keys; see idx_topk_prefill_geometry in include/idx_topk.h."""
    sh, sp, sg = _i32(), _i32(), _i32()
    _check(_lib.idx_topk_prefill_geometry(Q, N, ctypes.byref(sh), ctypes.byref(sp), ctypes.byref(sg)))
    return int(sh.value), int(sp.value), int(sg.value)


def prefill_unfused_workspace_bytes(Q: int, N: int, K: int) -> int:
    return int(_lib.idx_topk_prefill_unfused_workspace(Q, N, K))


def scan_bf16_workspace_bytes(B: int, N: int, K: int) -> int:
    return int(_lib.idx_topk_scan_bf16_workspace(B, N, K))


def decode_workspace_bytes(B: int, max_pages: int, page_size: int, K: int) -> int:
    return int(_lib.idx_topk_decode_workspace(B, max_pages, page_size, K))


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _q_k(q8, k8):
    if q8.dtype == torch.float8_e4m3fn:
        q8 = q8.view(torch.uint8)
    if k8.dtype == torch.float8_e4m3fn:
        k8 = k8.view(torch.uint8)
    return q8, k8


def prefill(q8, q_scale, k8, k_scale, w, row_start, row_end, K: int, out=None, workspace=None,
            stream=None):
    """Top-K key ids per query row; see idx_topk_prefill in include/idx_topk.h.

    q8 [Q,64,128] uint8 (or float8_e4m3fn), q_scale [Q,64] f32 or None,
    k8 [N,128], k_scale [N] f32, w [Q,64] f32, row_start/row_end [Q] int32.
    Returns out [Q,K] int32 (absolute ids, unsorted, -1 padded).
    """
    return _prefill(q8, q_scale, k8, k_scale, w, row_start, row_end, K, out, workspace, stream,
                    debug=False)


def prefill_debug(q8, q_scale, k8, k_scale, w, row_start, row_end, K: int, out=None,
                  workspace=None, stream=None, scores_out=None, tau_out=None,
                  force_tau: Optional[float] = None, cand_cap: int = 0,
                  main_events=None, main_reps: int = 1, row_status=None, clock_out=None,
                  math_only: bool = False):
    """idx_topk_prefill_debug: also emits FP32 scores [Q,N] and thresholds [Q].

    main_events: optional (start, stop) pair of torch.cuda.Event(enable_timing=True)
    recorded around the fused main kernel; main_reps > 1 launches that kernel
    so many times back to back inside the pair (timing only).  row_status [Q]
    int32 receives each row's ROW_* outcome; clock_out [2] int64 (zeroed by
    the caller) accumulates the main kernel's shader-clock cycles and
    wall-clock ticks; math_only runs the control build of the main kernel
    (no selection, out is not written)."""
    ev0 = ev1 = None
    if main_events is not None:
        ev0, ev1 = (ctypes.c_void_p(e.cuda_event) for e in main_events)
    opts = Opts(1 if force_tau is not None else 0, float(force_tau or 0.0), int(cand_cap),
                ev0, ev1, int(main_reps), _ptr(row_status, torch.int32),
                _ptr(clock_out, torch.int64), 1 if math_only else 0)
    return _prefill(q8, q_scale, k8, k_scale, w, row_start, row_end, K, out, workspace, stream,
                    debug=True, scores_out=scores_out, tau_out=tau_out, opts=opts)


def _prefill(q8, q_scale, k8, k_scale, w, row_start, row_end, K, out, workspace, stream, debug,
             scores_out=None, tau_out=None, opts=None):
    q8, k8 = _q_k(q8, k8)
    Q, N = int(q8.shape[0]), int(k8.shape[0])
    if q8.shape[1:] != (HEADS, DIM) or k8.shape[1:] != (DIM,):
        raise ValueError("q8 must be [Q,64,128] and k8 [N,128]")
    dev = q8.device
    if out is None:
        out = torch.empty((Q, K), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(prefill_workspace_bytes(Q, N, K), dev)
    args = [_ptr(q8, torch.uint8), _ptr(q_scale, torch.float32), _ptr(k8, torch.uint8),
            _ptr(k_scale, torch.float32), _ptr(w, torch.float32), _ptr(row_start, torch.int32),
            _ptr(row_end, torch.int32), int(K), _ptr(out, torch.int32), Q, N, _ptr(workspace),
            int(workspace.numel()), _stream(stream)]
    if debug:
        _check(_lib.idx_topk_prefill_debug(*args, _ptr(scores_out, torch.float32),
                                           _ptr(tau_out, torch.float32), ctypes.byref(opts)))
    else:
        _check(_lib.idx_topk_prefill(*args))
    return out


def prefill_unfused(q8, q_scale, k8, k_scale, w, row_start, row_end, K: int, out=None,
                    workspace=None, stream=None, main_events=None, main_reps: int = 1):
    """idx_topk_prefill_unfused: the same scores written to an explicit [Q,N]
    matrix in the workspace, then a separate top-K over it (the comparator of
    the fused path).  main_events: optional (start, stop) event pair around
    the scoring kernel."""
    q8, k8 = _q_k(q8, k8)
    Q, N = int(q8.shape[0]), int(k8.shape[0])
    if q8.shape[1:] != (HEADS, DIM) or k8.shape[1:] != (DIM,):
        raise ValueError("q8 must be [Q,64,128] and k8 [N,128]")
    dev = q8.device
    if out is None:
        out = torch.empty((Q, K), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(prefill_unfused_workspace_bytes(Q, N, K), dev)
    ev0 = ev1 = None
    if main_events is not None:
        ev0, ev1 = (ctypes.c_void_p(e.cuda_event) for e in main_events)
    opts = Opts(0, 0.0, 0, ev0, ev1, int(main_reps))
    _check(_lib.idx_topk_prefill_unfused(
        _ptr(q8, torch.uint8), _ptr(q_scale, torch.float32), _ptr(k8, torch.uint8),
        _ptr(k_scale, torch.float32), _ptr(w, torch.float32), _ptr(row_start, torch.int32),
        _ptr(row_end, torch.int32), int(K), _ptr(out, torch.int32), Q, N, _ptr(workspace),
        int(workspace.numel()), _stream(stream), ctypes.byref(opts)))
    return out


def topk_rows(scores, row_start, row_end, K: int, out=None, stream=None):
    """idx_topk_rows: exact top-K positions of each row of a dense FP32
    matrix scores [Q, ld] over [row_start, row_end) (ties to the lowest
    positions; rows with fewer than K positions are -1 padded)."""
    if scores.dim() != 2:
        raise ValueError("scores must be [Q, N]")
    Q, N = int(scores.shape[0]), int(scores.shape[1])
    if out is None:
        out = torch.empty((Q, K), dtype=torch.int32, device=scores.device)
    _check(_lib.idx_topk_rows(_ptr(scores, torch.float32), N, _ptr(row_start, torch.int32),
                              _ptr(row_end, torch.int32), int(K), _ptr(out, torch.int32), Q, N,
                              _stream(stream)))
    return out


def scan_bf16(q16, w, k16, lens, K: int, out=None, workspace=None, stream=None, main_events=None,
              main_reps: int = 1):
    """idx_topk_scan_bf16: q16 [B,64,128] and k16 [B,N,128] as torch.bfloat16 or
    uint16/int16 bit patterns, w [B,64] f32, lens [B] int32 (device).  Returns
    out [B,K] int32 key positions.  main_events / main_reps: timing of the
    scoring kernel."""
    if q16.dtype == torch.bfloat16:
        q16 = q16.view(torch.int16)
    if k16.dtype == torch.bfloat16:
        k16 = k16.view(torch.int16)
    B, N = int(k16.shape[0]), int(k16.shape[1])
    if q16.shape != (B, HEADS, DIM) or k16.shape[2:] != (DIM,):
        raise ValueError("q16 must be [B,64,128] and k16 [B,N,128]")
    dev = q16.device
    if out is None:
        out = torch.empty((B, K), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(scan_bf16_workspace_bytes(B, N, K), dev)
    ev0 = ev1 = None
    if main_events is not None:
        ev0, ev1 = (ctypes.c_void_p(e.cuda_event) for e in main_events)
    opts = Opts(0, 0.0, 0, ev0, ev1, int(main_reps))
    _check(_lib.idx_topk_scan_bf16(_ptr(q16), _ptr(w, torch.float32), _ptr(k16), _ptr(lens, torch.int32),
                                   B, N, int(K), _ptr(out, torch.int32), _ptr(workspace),
                                   int(workspace.numel()), _stream(stream), ctypes.byref(opts)))
    return out


def scan_bf16_scores(workspace: torch.Tensor, B: int, N: int) -> torch.Tensor:
    """The [B,N] FP32 score rows inside a scan workspace (a copy; tests only)."""
    addr = _lib.idx_topk_scan_bf16_scores(_ptr(workspace), int(B), int(N))
    off = int(addr) - workspace.data_ptr()
    return workspace[off: off + 4 * B * N].view(torch.float32).view(B, N).clone()


_lib.idx_topk_graph_begin.restype = ctypes.c_int
_lib.idx_topk_graph_begin.argtypes = [_vp]
_lib.idx_topk_graph_end.restype = ctypes.c_int
_lib.idx_topk_graph_end.argtypes = [_vp, ctypes.POINTER(_vp)]
_lib.idx_topk_graph_launch.restype = ctypes.c_int
_lib.idx_topk_graph_launch.argtypes = [_vp, _vp]
_lib.idx_topk_graph_destroy.restype = ctypes.c_int
_lib.idx_topk_graph_destroy.argtypes = [_vp]


class Graph:
    """A recorded chain of library calls (idx_topk_graph_*); launch() replays it."""

    def __init__(self, handle):
        self._h = handle

    def launch(self, stream=None):
        if not self._h:
            raise ValueError("graph is destroyed")
        _check(_lib.idx_topk_graph_launch(self._h, _stream(stream)))

    def destroy(self):
        if self._h:
            h, self._h = self._h, None
            _check(_lib.idx_topk_graph_destroy(h))

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def capture(fn, stream=None) -> Graph:
    """Record the library calls that fn() makes into a graph.  fn runs with a
    side stream (or `stream`) current; it must pass its own output and
    workspace buffers (nothing may allocate during the capture) and no
    timing events."""
    s = stream if stream is not None else torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _check(_lib.idx_topk_graph_begin(_stream(s)))
        h = _vp()
        try:
            fn()
        except BaseException:
            _lib.idx_topk_graph_end(_stream(s), ctypes.byref(h))
            if h:
                _lib.idx_topk_graph_destroy(h)
            raise
        _check(_lib.idx_topk_graph_end(_stream(s), ctypes.byref(h)))
    return Graph(h)


def stream_floor(src: torch.Tensor, out=None, stream=None):
    """idx_topk_stream_floor over src viewed as 256-byte records."""
    nbytes = src.numel() * src.element_size()
    n = nbytes // 256
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=src.device)
    _check(_lib.idx_topk_stream_floor(_ptr(src), int(n), _ptr(out, torch.float32), _stream(stream)))
    return out


def decode_paged(q8, q_scale, k_cache, k_scale, w, page_table, seq_lens, K: int, out=None,
                 workspace=None, stream=None, force_tau: Optional[float] = None, main_events=None,
                 main_reps: int = 1, scores_out=None):
    """Top-K physical cache slots per sequence; see idx_topk_decode_paged.

    q8 [B,64,128], q_scale [B,64] or None, k_cache [P,64,128], k_scale [P,64],
    w [B,64], page_table [B,max_pages] int32, seq_lens [B] int32 (device).
    main_events selects idx_topk_decode_paged_debug with a (start, stop)
    torch.cuda.Event pair around the scoring kernel; scores_out
    [B, max_pages*64] f32 (debug entry too) receives the scores the
    selection read; force_tau is passed through so that the library's
    rejection of it (decode has no threshold knob) can be tested.
    """
    q8, k_cache = _q_k(q8, k_cache)
    B = int(q8.shape[0])
    P, page = int(k_cache.shape[0]), int(k_cache.shape[1])
    max_pages = int(page_table.shape[1])
    dev = q8.device
    if out is None:
        out = torch.empty((B, K), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(decode_workspace_bytes(B, max_pages, page, K), dev)
    args = [_ptr(q8, torch.uint8), _ptr(q_scale, torch.float32), _ptr(k_cache, torch.uint8),
            _ptr(k_scale, torch.float32), _ptr(w, torch.float32), _ptr(page_table, torch.int32),
            _ptr(seq_lens, torch.int32), B, max_pages, page, P, int(K), _ptr(out, torch.int32),
            _ptr(workspace), int(workspace.numel()), _stream(stream)]
    if force_tau is None and main_events is None and main_reps == 1 and scores_out is None:
        _check(_lib.idx_topk_decode_paged(*args))
    else:
        ev0 = ev1 = None
        if main_events is not None:
            ev0, ev1 = (ctypes.c_void_p(e.cuda_event) for e in main_events)
        opts = Opts(1 if force_tau is not None else 0, float(force_tau or 0.0), 0, ev0, ev1,
                    int(main_reps))
        _check(_lib.idx_topk_decode_paged_debug(*args, _ptr(scores_out, torch.float32), ctypes.byref(opts)))
    return out


# ------------------------------------------------------- operators around the indexer

LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128
LATENT_ROW = LATENT + ROPE
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}

_i64, _f32 = ctypes.c_int64, ctypes.c_float
_lib.idx_topk_latent_selected_workspace.restype = _sz
_lib.idx_topk_latent_selected_workspace.argtypes = [_i32, _i32, _i32]
_lib.idx_topk_latent_selected.restype = ctypes.c_int
_lib.idx_topk_latent_selected.argtypes = [_vp, _i64, _i64, _vp, _i64, _vp, _i32, _i32, _i32, _f32, _i32, _vp, _vp, _vp,
                                          _sz, _vp]
_lib.idx_topk_latent_paged_workspace.restype = _sz
_lib.idx_topk_latent_paged_workspace.argtypes = [_i32, _i32, _i32, _i32]
_lib.idx_topk_latent_paged.restype = ctypes.c_int
_lib.idx_topk_latent_paged.argtypes = [_vp, _i64, _i64, _i64, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _f32, _i32,
                                       _vp, _vp, _vp, _sz, _vp]
_lib.idx_topk_latent_expanded_workspace.restype = _sz
_lib.idx_topk_latent_expanded_workspace.argtypes = [_i32, _i32, _i32, _i32, _i32]
_lib.idx_topk_latent_expanded.restype = ctypes.c_int
_lib.idx_topk_latent_expanded.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _i32,
                                          _i32, _i32, _f32, _i32, _i32, _vp, _vp, _vp, _sz, _vp]
_lib.idx_topk_norm_quant.restype = ctypes.c_int
_lib.idx_topk_norm_quant.argtypes = [_vp, _i64, _vp, _i64, _vp, _f32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp]
_lib.idx_topk_cache_append.restype = ctypes.c_int
_lib.idx_topk_cache_append.argtypes = [_vp, _i64, _vp, _i64, _vp, _i32, _i32, _vp, _vp, _vp, _i64, _vp]
_lib.idx_topk_latent_tree_workspace.restype = _sz
_lib.idx_topk_latent_tree_workspace.argtypes = [_i32, _i32, _i32, _i32]
_lib.idx_topk_latent_tree.restype = ctypes.c_int
_lib.idx_topk_latent_tree.argtypes = [_vp, _i64, _i64, _i64, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _f32,
                                      _i32, _vp, _vp, _vp, _sz, _vp]
_lib.idx_topk_norm_rotate.restype = ctypes.c_int
_lib.idx_topk_norm_rotate.argtypes = [_vp, _i64, _i64, _i32, _vp, _vp, _f32, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                                      _vp, _i64, _i64, _vp, _vp, _vp]
_lib.idx_topk_cache_append_rotary.restype = ctypes.c_int
_lib.idx_topk_cache_append_rotary.argtypes = [_vp, _i64, _i32, _vp, _f32, _i32, _vp, _i64, _i32, _vp, _vp, _f32, _i32, _i32, _vp, _vp,
                                              _vp, _i32, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _vp]
_lib.idx_topk_matmul_e4m3.restype = ctypes.c_int
_lib.idx_topk_matmul_e4m3.argtypes = [_vp, _i64, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i64, _vp]


def latent_selected_workspace_bytes(T: int, H: int, K: int) -> int:
    return int(_lib.idx_topk_latent_selected_workspace(T, H, K))


def latent_paged_workspace_bytes(B: int, S: int, H: int, max_pages: int) -> int:
    return int(_lib.idx_topk_latent_paged_workspace(B, S, H, max_pages))


def latent_tree_workspace_bytes(B: int, S: int, H: int, max_pages: int) -> int:
    return int(_lib.idx_topk_latent_tree_workspace(B, S, H, max_pages))


def latent_expanded_workspace_bytes(Tq: int, B: int, max_q: int, max_k: int, H: int) -> int:
    return int(_lib.idx_topk_latent_expanded_workspace(Tq, B, max_q, max_k, H))


def _dtype16(t: torch.Tensor) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError("expected bfloat16 or float16, got %s" % t.dtype)
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    return code


# The checks below cost a few hundred nanoseconds a call in all: a decode step's
# launches wait for them.

def _int32(n: int) -> None:
    """n: sizes of a call, or'ed together, and not all of them small ones.  The library takes them in 32 bits, of
    which ctypes would drop the rest; negative ones it refuses itself."""
    if n >> 31 != -1:
        raise ValueError("a size of this call is outside 32 bits")


def _at(t: torch.Tensor, dtype, dev) -> int:
    """Address of a contiguous tensor of this type on this device."""
    if t.dtype != dtype:
        raise ValueError("expected dtype %s, got %s" % (dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("expected all tensors on cuda:%d, got one on %s" % (dev, t.device))
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _rows_at(t: torch.Tensor, dtype, dev, shape) -> int:
    """Address of a strided input of this shape whose last dimension is contiguous."""
    if t.dtype != dtype:
        raise ValueError("expected dtype %s, got %s" % (dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("expected all tensors on cuda:%d, got one on %s" % (dev, t.device))
    if t.shape != shape:
        raise ValueError("expected shape %s, got %s" % (list(shape), list(t.shape)))
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError("expected unit stride along the last dimension")
    return t.data_ptr()


def _strides(t: torch.Tensor):
    """Strides in numbers but the last; a dimension of one has none that matters."""
    if 1 not in t.shape:
        return t.stride()[:-1]
    return [n if size > 1 else 0 for n, size in zip(t.stride(), t.shape)][:-1]


def _empty(shape, dtype, dev, stream):
    """A new tensor that belongs to the stream it is written on: one of the
    current stream's could be memory that work still pending there uses."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _out(t: Optional[torch.Tensor], shape, dtype, dev, stream):
    """The caller's output, checked, or a new one; and its address."""
    if t is None:
        t = _empty(shape, dtype, dev, stream)
        return t, t.data_ptr()
    if t.shape != shape:
        raise ValueError("expected an output of shape %s, got %s" % (list(shape), list(t.shape)))
    return t, _at(t, dtype, dev)


def _scratch(workspace: Optional[torch.Tensor], need: int, dev, stream):
    """Address and size of the caller's workspace or a new one (and the tensor, to hold it)."""
    if workspace is None:
        workspace = _empty(max(need, 256), torch.uint8, dev, stream)
        return workspace.data_ptr(), max(need, 256), workspace
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("expected a contiguous workspace on cuda:%d" % dev)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _on(stream, dev) -> int:
    """Handle of `stream`, or of the current stream; the launch goes to the current device."""
    if dev != torch._C._cuda_getDevice():
        raise ValueError("expected tensors on the current device, got cuda:%d" % dev)
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _cache_at(cache: torch.Tensor, width: int, dtype, dev):
    if cache.shape[-1] != width:
        raise ValueError("expected a cache of rows of %d, got shape %s" % (width, list(cache.shape)))
    return _at(cache, dtype, dev), cache.numel() // width


def latent_selected(q, cache, slots, scale: float, out=None, lse=None, workspace=None, stream=None):
    """Latent attention over listed slots; see idx_topk_latent_selected in
    include/idx_topk.h.

    q [T,H,576] bf16 or f16 (strided), cache [...,576] contiguous, slots [T,K]
    int32 (the output of prefill or decode_paged: -1 entries are skipped).
    Returns (out [T,H,512], lse [T,H] f32).
    """
    dt, dev, dtype = _dtype16(q), q.get_device(), q.dtype
    if q.dim() != 3 or slots.dim() != 2 or slots.shape[0] != q.shape[0]:
        raise ValueError("expected q [T,H,576] and slots [T,K], got %s and %s" % (list(q.shape), list(slots.shape)))
    T, H, _ = q.shape
    K = slots.shape[1]
    if (T | H | K) >> 31:
        _int32(T | H | K)
    q_at = _rows_at(q, dtype, dev, (T, H, LATENT_ROW))
    q_token, q_head = _strides(q)
    cache_at, num_slots = _cache_at(cache, LATENT_ROW, dtype, dev)
    out, out_at = _out(out, (T, H, LATENT), dtype, dev, stream)
    lse, lse_at = _out(lse, (T, H), torch.float32, dev, stream)
    ws_at, ws_bytes, ws = _scratch(workspace, _lib.idx_topk_latent_selected_workspace(T, H, K), dev, stream)
    _check(_lib.idx_topk_latent_selected(q_at, q_token, q_head, cache_at, num_slots, _at(slots, torch.int32, dev), K, T, H,
                                         scale, dt, out_at, lse_at, ws_at, ws_bytes, _on(stream, dev)))
    return out, lse


def latent_paged(q, cache, page_table, seq_lens, scale: float, out=None, lse=None, workspace=None, stream=None):
    """Latent attention over whole paged sequences; see idx_topk_latent_paged.

    q [B,S,H,576] (strided; S tokens at the end of each sequence), cache
    [P,64,576], page_table [B,max_pages] int32, seq_lens [B] int32 (device).
    Returns (out [B,S,H,512], lse [B,S,H] f32).
    """
    dt, dev, dtype = _dtype16(q), q.get_device(), q.dtype
    if q.dim() != 4 or cache.dim() != 3 or cache.shape[1] != PAGE:
        raise ValueError("expected q [B,S,H,576] and a cache [pages,64,576], got %s and %s" % (list(q.shape), list(cache.shape)))
    B, S, H, _ = q.shape
    if page_table.dim() != 2 or page_table.shape[0] != B or seq_lens.shape != (B,):
        raise ValueError("expected page_table [%d, max_pages] and seq_lens [%d]" % (B, B))
    max_pages = page_table.shape[1]
    if (B | S | H | max_pages | cache.shape[0]) >> 31:
        _int32(B | S | H | max_pages | cache.shape[0])
    q_at = _rows_at(q, dtype, dev, (B, S, H, LATENT_ROW))
    q_seq, q_token, q_head = _strides(q)
    cache_at, num_slots = _cache_at(cache, LATENT_ROW, dtype, dev)
    out, out_at = _out(out, (B, S, H, LATENT), dtype, dev, stream)
    lse, lse_at = _out(lse, (B, S, H), torch.float32, dev, stream)
    ws_at, ws_bytes, ws = _scratch(workspace, _lib.idx_topk_latent_paged_workspace(B, S, H, max_pages), dev, stream)
    _check(_lib.idx_topk_latent_paged(q_at, q_seq, q_token, q_head, cache_at, num_slots // PAGE,
                                      _at(page_table, torch.int32, dev), max_pages, _at(seq_lens, torch.int32, dev), B, S, H,
                                      scale, dt, out_at, lse_at, ws_at, ws_bytes, _on(stream, dev)))
    return out, lse


def latent_tree(q, cache, page_table, prefix_lens, counts, masks, scale: float, out=None, lse=None, workspace=None, stream=None):
    """Latent attention of drafted tokens that form a tree; see idx_topk_latent_tree.

    q [B,S,H,576] (strided), cache [P,64,576], page_table [B,max_pages] int32,
    prefix_lens [B] and counts [B] (or None: S each) int32, masks int64 [B,S] or
    [S] (one tree for all sequences): bit i of a node's mask says whether it sees
    node i.  Returns (out [B,S,H,512], lse [B,S,H] f32).
    """
    dt, dev, dtype = _dtype16(q), q.get_device(), q.dtype
    if q.dim() != 4 or cache.dim() != 3 or cache.shape[1] != PAGE:
        raise ValueError("expected q [B,S,H,576] and a cache [pages,64,576], got %s and %s" % (list(q.shape), list(cache.shape)))
    B, S, H, _ = q.shape
    if page_table.dim() != 2 or page_table.shape[0] != B or prefix_lens.shape != (B,) or (counts is not None and counts.shape != (B,)):
        raise ValueError("expected page_table [%d, max_pages], prefix_lens [%d] and counts [%d]" % (B, B, B))
    if masks.shape != (S,) and masks.shape != (B, S):
        raise ValueError("expected masks [%d, %d] or [%d], got %s" % (B, S, S, list(masks.shape)))
    max_pages = page_table.shape[1]
    if (B | S | H | max_pages | cache.shape[0]) >> 31:
        _int32(B | S | H | max_pages | cache.shape[0])
    q_at = _rows_at(q, dtype, dev, (B, S, H, LATENT_ROW))
    q_seq, q_token, q_head = _strides(q)
    cache_at, num_slots = _cache_at(cache, LATENT_ROW, dtype, dev)
    out, out_at = _out(out, (B, S, H, LATENT), dtype, dev, stream)
    lse, lse_at = _out(lse, (B, S, H), torch.float32, dev, stream)
    ws_at, ws_bytes, ws = _scratch(workspace, _lib.idx_topk_latent_tree_workspace(B, S, H, max_pages), dev, stream)
    _check(_lib.idx_topk_latent_tree(q_at, q_seq, q_token, q_head, cache_at, num_slots // PAGE, _at(page_table, torch.int32, dev),
                                     max_pages, _at(prefix_lens, torch.int32, dev),
                                     None if counts is None else _at(counts, torch.int32, dev), _at(masks, torch.int64, dev),
                                     S if masks.dim() == 2 else 0, B, S, H, scale, dt, out_at, lse_at, ws_at, ws_bytes,
                                     _on(stream, dev)))
    return out, lse


def latent_expanded(q, kv, k_rope, cu_q, cu_k, max_q: int, max_k: int, scale: float, causal: bool = True, out=None,
                    lse=None, workspace=None, stream=None):
    """Causal attention over packed prompts with expanded keys and values; see
    idx_topk_latent_expanded.

    q [Tq,H,192], kv [Tk,H,256] (128 key numbers, then 128 value numbers),
    k_rope [Tk,64], all strided; cu_q, cu_k [B+1] int32 (device) running token
    counts, max_q and max_k the longest prompt's query tokens and keys.
    Returns (out [Tq,H,128], lse [Tq,H] f32).
    """
    dt, dev, dtype = _dtype16(q), q.get_device(), q.dtype
    if q.dim() != 3 or kv.dim() != 3:
        raise ValueError("expected q [Tq,H,192] and kv [Tk,H,256], got %s and %s" % (list(q.shape), list(kv.shape)))
    Tq, H, _ = q.shape
    Tk = kv.shape[0]
    q_at = _rows_at(q, dtype, dev, (Tq, H, NOPE + ROPE))
    kv_at = _rows_at(kv, dtype, dev, (Tk, H, NOPE + VALUE))
    rope_at = _rows_at(k_rope, dtype, dev, (Tk, ROPE))
    if cu_q.dim() != 1 or cu_q.shape != cu_k.shape or cu_q.shape[0] < 1:
        raise ValueError("expected cu_q and cu_k of shape [B+1]")
    B = cu_q.shape[0] - 1
    if (B | Tq | Tk | H | max_q | max_k) >> 31:
        _int32(B | Tq | Tk | H | max_q | max_k)
    out, out_at = _out(out, (Tq, H, VALUE), dtype, dev, stream)
    lse, lse_at = _out(lse, (Tq, H), torch.float32, dev, stream)
    ws_at, ws_bytes, ws = _scratch(workspace, _lib.idx_topk_latent_expanded_workspace(Tq, B, max_q, max_k, H), dev, stream)
    _check(_lib.idx_topk_latent_expanded(q_at, *_strides(q), kv_at, *_strides(kv), rope_at, *_strides(k_rope),
                                         _at(cu_q, torch.int32, dev), _at(cu_k, torch.int32, dev), B, Tq, Tk, max_q, max_k,
                                         H, scale, 1 if causal else 0, dt, out_at, lse_at, ws_at, ws_bytes, _on(stream, dev)))
    return out, lse


def norm_quant(x, weight, eps: float, residual=None, group: int = 0, codes=None, scales=None, residual_out=None,
               stream=None):
    """Root-mean-square norm of x + residual to e4m3 codes and scales; see
    idx_topk_norm_quant.

    x, residual [R,W] bf16 or f16 (strided rows) and weight [W] or None; group 0 (one
    scale a row) or 128.  Returns (codes [R,W] float8_e4m3fn, scales [R,W/group]
    f32, x + residual or None): the last one is residual_out, or with a
    residual and no residual_out a new tensor.
    """
    dt, dev, dtype = _dtype16(x), x.get_device(), x.dtype
    if x.dim() != 2:
        raise ValueError("expected x [R,W], got %s" % list(x.shape))
    R, W = shape = x.shape
    if (R | W | group) >> 31:
        _int32(R | W | group)
    x_at = _rows_at(x, dtype, dev, shape)
    res_at, res_stride = None, 0
    if residual is not None:
        res_at = _rows_at(residual, dtype, dev, shape)
        res_stride, = _strides(residual)
    if weight is not None and weight.shape != (W,):
        raise ValueError("expected a weight of shape [%d], got %s" % (W, list(weight.shape)))
    codes, codes_at = _out(codes, shape, torch.float8_e4m3fn, dev, stream)
    scales, scales_at = _out(scales, (R, W // group if group > 0 else 1), torch.float32, dev, stream)
    out_at = None
    if residual is not None or residual_out is not None:
        residual_out, out_at = _out(residual_out, shape, dtype, dev, stream)
    _check(_lib.idx_topk_norm_quant(x_at, *_strides(x), res_at, res_stride, None if weight is None else _at(weight, dtype, dev),
                                    eps, R, W, group, dt, codes_at, scales_at, out_at, _on(stream, dev)))
    return codes, scales, residual_out


def cache_append(latents, index_keys, slots, latent_cache, k_cache, k_scale, stream=None):
    """Store new tokens in the caches; see idx_topk_cache_append.

    latents [T,576] and index_keys [T,128] bf16 or f16 (strided rows), slots [T]
    int32 (-1: not stored), latent_cache [...,576], k_cache [...,128] uint8 or
    float8_e4m3fn, k_scale [...] f32.  latents with latent_cache, or index_keys
    with k_cache and k_scale, may be None together.
    """
    one = latents if latents is not None else index_keys
    if one is None:
        raise ValueError("expected latents, index_keys or both")
    dt, dev, dtype, T = _dtype16(one), one.get_device(), one.dtype, one.shape[0]
    if (latents is None) != (latent_cache is None) or (index_keys is None) != (k_cache is None) or (k_cache is None) != (k_scale is None):
        raise ValueError("latents come with latent_cache, index_keys with k_cache and k_scale")
    if slots.shape != (T,):
        raise ValueError("expected slots of shape [%d], got %s" % (T, list(slots.shape)))
    if T >> 31:
        _int32(T)
    lat_at = cache_at = key_at = kc_at = ks_at = None
    lat_stride = key_stride = 0
    num = n = None
    if latents is not None:
        lat_at = _rows_at(latents, dtype, dev, (T, LATENT_ROW))
        lat_stride, = _strides(latents)
        cache_at, num = _cache_at(latent_cache, LATENT_ROW, dtype, dev)
    if index_keys is not None:
        key_at = _rows_at(index_keys, dtype, dev, (T, DIM))
        key_stride, = _strides(index_keys)
        kc_at, n = _cache_at(k_cache, DIM, torch.float8_e4m3fn if k_cache.dtype == torch.float8_e4m3fn else torch.uint8, dev)
        ks_at = _at(k_scale, torch.float32, dev)
        if k_scale.numel() != n or (num is not None and num != n):
            raise ValueError("the caches hold different numbers of slots: %s" % [num, n, k_scale.numel()])
    _check(_lib.idx_topk_cache_append(lat_at, lat_stride, key_at, key_stride, _at(slots, torch.int32, dev), T, dt, cache_at,
                                      kc_at, ks_at, n if num is None else num, _on(stream, dev)))


NORMS = {"none": 0, "rms": 1, "layer": 2}


def _norm(name: str) -> int:
    code = NORMS.get(name)
    if code is None:
        raise ValueError("expected a norm of %s, got %r" % (sorted(NORMS), name))
    return code


def _vector(t: Optional[torch.Tensor], n: int, dtype, dev):
    """Address of a weight or bias [n], or None."""
    if t is None:
        return None
    if t.shape != (n,):
        raise ValueError("expected a weight or bias of shape [%d], got %s" % (n, list(t.shape)))
    return _at(t, dtype, dev)


def _angles(positions, table, T: int, dev):
    """Addresses of the positions and the table of angles, and the table's rows."""
    if positions.shape != (T,):
        raise ValueError("expected positions of shape [%d], got %s" % (T, list(positions.shape)))
    shape = table.shape
    if len(shape) != 2 or shape[1] != ROPE:
        raise ValueError("expected a table [positions,%d], got %s" % (ROPE, list(shape)))
    P = shape[0]
    if P >> 31:
        _int32(P)
    return _at(positions, torch.int32, dev), _at(table, torch.float32, dev), P


def _head_rows(x, rope_at: int):
    """What norm_rotate and norm_rotate_quant take of x [T,H,D]."""
    dt, dev, dtype, shape = _dtype16(x), x.get_device(), x.dtype, x.shape
    if len(shape) != 3:
        raise ValueError("expected x [T,H,D], got %s" % list(shape))
    T, H, D = shape
    if (T | H | D | rope_at) >> 31:
        _int32(T | H | D | rope_at)
    token, head, unit = x.stride()
    if unit != 1 and D > 1:
        raise ValueError("expected unit stride along the last dimension")
    return dt, dev, dtype, T, H, D, x.data_ptr(), (token if T > 1 else 0, head if H > 1 else 0)


def norm_rotate(x, positions, table, rope_at: int, interleaved: bool = False, norm: str = "none", weight=None, bias=None,
                eps: float = 1e-6, out=None, stream=None):
    """Norm of each head and rotation of its numbers rope_at .. rope_at + 64; see
    idx_topk_norm_rotate.

    x [T,H,D] bf16 or f16 (strided), positions [T] int32 (outside the table:
    padding, not written), table [P,64] f32 (32 cosines, 32 sines a
    position), norm "none", "rms" or "layer" with weight and bias [D] or None.
    Returns out [T,H,D]: a new tensor, or the caller's (strided; may be x).
    """
    dt, dev, dtype, T, H, D, x_at, x_strides = _head_rows(x, rope_at)
    if out is None:
        out = _empty((T, H, D), dtype, dev, stream)
        out_at, out_strides = out.data_ptr(), (H * D, D)
    else:
        out_at, out_strides = _rows_at(out, dtype, dev, (T, H, D)), _strides(out)
    pos_at, table_at, P = _angles(positions, table, T, dev)
    _check(_lib.idx_topk_norm_rotate(x_at, *x_strides, _norm(norm), _vector(weight, D, dtype, dev), _vector(bias, D, dtype, dev), eps,
                                     pos_at, table_at, P, rope_at, 1 if interleaved else 0, T, H, D, dt, out_at, *out_strides, None, None,
                                     _on(stream, dev)))
    return out


def norm_rotate_quant(x, positions, table, rope_at: int, interleaved: bool = False, norm: str = "none", weight=None, bias=None,
                      eps: float = 1e-6, codes=None, scales=None, stream=None):
    """norm_rotate to e4m3 codes with one scale a head: the indexer's queries from
    projected ones.  Returns (codes [T,H,D] float8_e4m3fn, scales [T,H] f32).
    """
    dt, dev, dtype, T, H, D, x_at, x_strides = _head_rows(x, rope_at)
    codes, codes_at = _out(codes, (T, H, D), torch.float8_e4m3fn, dev, stream)
    scales, scales_at = _out(scales, (T, H), torch.float32, dev, stream)
    pos_at, table_at, P = _angles(positions, table, T, dev)
    _check(_lib.idx_topk_norm_rotate(x_at, *x_strides, _norm(norm), _vector(weight, D, dtype, dev), _vector(bias, D, dtype, dev), eps,
                                     pos_at, table_at, P, rope_at, 1 if interleaved else 0, T, H, D, dt, None, 0, 0, codes_at,
                                     scales_at, _on(stream, dev)))
    return codes, scales


def cache_append_rotary(latents, index_keys, slots, positions, table, latent_cache, k_cache, k_scale, latent_norm: str = "rms",
                        latent_weight=None, latent_eps: float = 1e-6, latent_interleaved: bool = True, key_norm: str = "layer",
                        key_weight=None, key_bias=None, key_eps: float = 1e-6, key_rope_at: int = 0, key_interleaved: bool = False,
                        latents_out=None, stream=None):
    """Norm, rotate and store new tokens in the caches; see idx_topk_cache_append_rotary.

    As cache_append, with positions [T] int32 and table [P,64] f32 as in
    norm_rotate.  latents_out [T,576] (or None) also receives the finished
    latent rows of the tokens that are stored.
    """
    one = latents if latents is not None else index_keys
    if one is None:
        raise ValueError("expected latents, index_keys or both")
    dt, dev, dtype, T = _dtype16(one), one.get_device(), one.dtype, one.shape[0]
    if (latents is None) != (latent_cache is None) or (index_keys is None) != (k_cache is None) or (k_cache is None) != (k_scale is None):
        raise ValueError("latents come with latent_cache, index_keys with k_cache and k_scale")
    if slots.shape != (T,):
        raise ValueError("expected slots of shape [%d], got %s" % (T, list(slots.shape)))
    if (T | key_rope_at) >> 31:
        _int32(T | key_rope_at)
    lat_at = cache_at = out_at = key_at = kc_at = ks_at = None
    lat_stride = key_stride = 0
    num = n = None
    if latents is not None:
        lat_at = _rows_at(latents, dtype, dev, (T, LATENT_ROW))
        lat_stride = latents.stride(0) if T > 1 else 0
        cache_at, num = _cache_at(latent_cache, LATENT_ROW, dtype, dev)
    if latents_out is not None:
        _, out_at = _out(latents_out, (T, LATENT_ROW), dtype, dev, stream)
    if index_keys is not None:
        key_at = _rows_at(index_keys, dtype, dev, (T, DIM))
        key_stride = index_keys.stride(0) if T > 1 else 0
        kc_at, n = _cache_at(k_cache, DIM, torch.float8_e4m3fn if k_cache.dtype == torch.float8_e4m3fn else torch.uint8, dev)
        ks_at = _at(k_scale, torch.float32, dev)
        if k_scale.numel() != n or (num is not None and num != n):
            raise ValueError("the caches hold different numbers of slots: %s" % [num, n, k_scale.numel()])
    pos_at, table_at, P = _angles(positions, table, T, dev)
    _check(_lib.idx_topk_cache_append_rotary(lat_at, lat_stride, _norm(latent_norm), _vector(latent_weight, LATENT, dtype, dev), latent_eps,
                                             1 if latent_interleaved else 0, key_at, key_stride, _norm(key_norm),
                                             _vector(key_weight, DIM, dtype, dev), _vector(key_bias, DIM, dtype, dev), key_eps,
                                             key_rope_at, 1 if key_interleaved else 0, _at(slots, torch.int32, dev), pos_at, table_at,
                                             P, T, dt, cache_at, kc_at, ks_at, n if num is None else num, out_at, _on(stream, dev)))


_CODES = (torch.float8_e4m3fn, torch.uint8)


def matmul_e4m3(x, x_scale, w, w_scale, dtype=torch.bfloat16, out=None, stream=None):
    """Product x @ w.T of e4m3 operands with block scales; see idx_topk_matmul_e4m3.

    x [M,K] float8_e4m3fn or uint8 (strided rows) with x_scale [M,ceil(K/128)]
    or [M,1] f32, as norm_quant returns them; w [N,K] with w_scale
    [ceil(N/128),ceil(K/128)] f32.  Returns out [M,N] in `dtype` (bf16 or f16): a
    new tensor, or the caller's (strided rows).
    """
    if not x.is_cuda:
        raise ValueError("expected a device tensor")
    dev, shape, w_shape = x.get_device(), x.shape, w.shape
    if len(shape) != 2 or len(w_shape) != 2 or shape[1] != w_shape[1]:
        raise ValueError("expected x [M,K] and w [N,K], got %s and %s" % (list(shape), list(w_shape)))
    (M, K), N = shape, w_shape[0]
    if (M | N | K) >> 31:
        _int32(M | N | K)
    x_type, w_type = x.dtype, w.dtype
    if x_type not in _CODES or w_type not in _CODES:
        raise ValueError("expected float8_e4m3fn or uint8, got %s and %s" % (x_type, w_type))
    blocks = (K + 127) // 128
    groups = x_scale.shape
    if groups != (M, blocks) and groups != (M, 1):
        raise ValueError("expected x_scale [%d,%d] or [%d,1], got %s" % (M, blocks, M, list(groups)))
    if w_scale.shape != ((N + 127) // 128, blocks):
        raise ValueError("expected w_scale [%d,%d], got %s" % ((N + 127) // 128, blocks, list(w_scale.shape)))
    kind = _DTYPES.get(dtype)
    if kind is None:
        raise ValueError("expected an output of bfloat16 or float16, got %s" % dtype)
    x_row, unit = x.stride()
    if unit != 1 and K > 1:
        raise ValueError("expected unit stride along the last dimension")
    if out is None:
        out = _empty((M, N), dtype, dev, stream)
        out_at, out_row = out.data_ptr(), N
    else:
        out_at, (out_row,) = _rows_at(out, dtype, dev, (M, N)), _strides(out)
    _check(_lib.idx_topk_matmul_e4m3(x.data_ptr(), x_row if M > 1 else 0, _at(x_scale, torch.float32, dev), 128 if groups[1] == blocks else 0,
                                     _at(w, w_type, dev), _at(w_scale, torch.float32, dev), M, N, K, kind, out_at, out_row,
                                     _on(stream, dev)))
    return out


NOALLOC_SCRATCH_BYTES = 16 << 20


def decode_paged_noalloc(q8, q_scale, k_cache, k_scale, w, page_table, seq_lens, K: int, out, stream=None):
    """idx_topk_decode_paged_noalloc: paged decode with the library's static
    per-GPU scratch (no workspace, nothing allocated); `out` [B,K] int32 is
    the caller's."""
    q8, k_cache = _q_k(q8, k_cache)
    B = int(q8.shape[0])
    P, page = int(k_cache.shape[0]), int(k_cache.shape[1])
    _check(_lib.idx_topk_decode_paged_noalloc(
        _ptr(q8, torch.uint8), _ptr(q_scale, torch.float32), _ptr(k_cache, torch.uint8),
        _ptr(k_scale, torch.float32), _ptr(w, torch.float32), _ptr(page_table, torch.int32),
        _ptr(seq_lens, torch.int32), B, int(page_table.shape[1]), page, P, int(K), _ptr(out, torch.int32),
        _stream(stream)))
    return out


def read_stats(workspace: torch.Tensor, stream=None) -> dict:
    st = Stats()
    _check(_lib.idx_topk_read_stats(_ptr(workspace), ctypes.byref(st), _stream(stream)))
    return st.asdict()


def raw_library():
    """The loaded ctypes library (for ABI-level tests)."""
    return _lib
