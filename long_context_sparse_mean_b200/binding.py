"""Python binding of libmisa.so: argument marshalling only.

Each function has the name of the C entry point it calls (include/misa.h) and passes torch
tensors' device pointers and the current CUDA stream through ctypes.  Every step of the indexer
runs in the library's CUDA kernels; there is no fallback.  If libmisa.so is missing the import
of this module fails.

Workspaces: a call given no Workspace uses a default buffer of its device and stream, shared only by
calls ordered on that stream, so calls on different streams never share scratch.  A Workspace passed
explicitly must likewise serve one stream at a time.  Default buffers are kept for the life of the
process, each as large as the largest call made on its stream; release_default_workspaces() frees
them.

Tensor conventions (all on one CUDA device, contiguous):
  q [T, H_I, 128] bf16 or fp32, w [T, H_I] fp32, n [T] int32 (prefix lengths),
  k [L, 128] (one cache shared by all queries) or [T, L, 128] (cache t for query t), same dtype as q,
  kbar [M, 128] or [T, M, 128] fp32 with M = ceil(L / B).
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
# MISA_LIBRARY=checked selects the bounds-checked build (libmisa_checked.so, misa.h).
LIB_PATH = os.path.join(PKG, "libmisa_checked.so" if os.environ.get("MISA_LIBRARY") == "checked" else "libmisa.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE_TIMEOUT, ERR_BAD_INDEX = range(7)
BF16, F32 = 0, 1
(OP_ROUTE, OP_SCORE_TOPK, OP_RERANK, OP_DENSE_TOPK, OP_TOPK_SELECT, OP_BLOCK_FILTER, OP_ROUTE_PAGED,
 OP_SCORE_TOPK_PAGED, OP_RERANK_PAGED, OP_SCORE_TOPK_FUSED, OP_HIER_FUSED,
 OP_KV4_ATTENTION, OP_KV4_COMPACT, OP_KEYS_COMPACT_PAGED, OP_PROMPT_ATTENTION) = range(15)
MAX_KP = 16384

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built: run `python -m long_context_sparse_mean_b200.build`")


class MisaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {_lib.misa_status_str(status).decode()} (status {status})")
        self.status = status


def _setup(lib):
    P, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sigs = {
        "misa_version": ([], i32),
        "misa_device_check": ([], i32),
        "misa_checked_build": ([], i32),
        "misa_bad_index_counts": ([P], i32),
        "misa_status_str": ([i32], ctypes.c_char_p),
        "misa_workspace_bytes": ([i32, i32, i32, i32, i32, i32, i32, i32], sz),
        "misa_pool_keys": ([P, i64, i32, i32, i32, i32, i32, P, i64, i32, i32, P], i32),
        "misa_route": ([P, P, P, i64, P, i64, P, i32, i32, i32, i32, i32, i32, i32, P, P, P, sz, P], i32),
        "misa_token_scores": ([P, P, P, i64, P, P, i32, i32, i32, i32, i32, i32, P, i64, i32, P, sz, P], i32),
        "misa_topk_select": ([P, i64, P, i32, i32, i32, P, P, P, sz, i32, P], i32),
        "misa_score_topk": ([P, P, P, i64, P, P, i32, i32, i32, i32, i32, i32, i32, P, P, P, P, sz, P], i32),
        "misa_hier_rerank": ([P, P, P, i64, P, P, i32, i32, i32, i32, i32, i32, i32, P, P, P, sz, P], i32),
        "dsa_dense_topk": ([P, P, P, i64, P, i32, i32, i32, i32, i32, i32, P, P, P, sz, P], i32),
        "misa_block_filter_topk": ([P, P, P, i64, P, i64, P, P, i32, i32, i32, i32, i32, i32, i32, i32, i32, P,
                                    i64, P, P, P, P, sz, P], i32),
        "misa_pool_keys_paged": ([P, i64, i32, P, i64, i32, i32, i32, i32, i32, P, i64, i32, i32, P], i32),
        "misa_route_paged": ([P, P, P, i64, i32, P, i64, P, i64, P, i32, i32, i32, i32, i32, i32, i32, P, P, P, sz,
                              P], i32),
        "misa_score_topk_paged": ([P, P, P, i64, i32, P, i64, P, P, i32, i32, i32, i32, i32, i32, i32, P, P, P, sz,
                                   P], i32),
        "misa_hier_rerank_paged": ([P, P, P, i64, i32, P, i64, P, P, i32, i32, i32, i32, i32, i32, i32, P, P, P, sz,
                                    P], i32),
        "misa_score_topk_fused": ([P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, P, P, P, sz, P], i32),
        "misa_hier_topk_fused": ([P, P, P, i64, P, P, i32, i32, i32, i32, i32, i32, i32, i32, P, P, P, sz, P], i32),
        "misa_kv4_append": ([P, P, i64, i64, i32, f32, f32, P, i64, i32, P, i64, P, P, i32, i32, i32, i32, P], i32),
        "misa_kv4_read": ([P, i64, i32, P, i64, P, P, i32, i32, i32, i32, i32, f32, f32, P, P, P], i32),
        "misa_kv4_attention": ([P, P, i64, i32, P, i64, P, P, i32, i32, i32, i32, i32, i32, i32, f32, f32, f32, P, P,
                                P, i64, P, sz, P], i32),
        "misa_kv4_attention_cols": ([P, P, i64, i32, P, i64, P, P, i32, i32, i32, i32, i32, i32, i32, f32, f32, f32, P, P,
                                     P, i32, i64, P, sz, P], i32),
        "misa_evict_select": ([P, i64, P, i32, i32, i32, i32, i32, P, P, P, i64, P], i32),
        "misa_kv4_compact": ([P, i64, i32, P, i64, P, i32, i32, i32, i32, P, sz, P], i32),
        "misa_keys_compact_paged": ([P, i64, i32, P, i64, P, i32, i32, i32, i32, P, sz, P], i32),
        "misa_prompt_attention": ([P, P, P, i64, i64, i64, P, P, i32, i32, i32, i32, i32, i32, i32, f32, P, P, P, sz,
                                   P], i32),
    }
    for name, (args, res) in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    return lib


_lib = _setup(ctypes.CDLL(LIB_PATH))


def library() -> ctypes.CDLL:
    return _lib


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream] = None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, status: int):
    if status != OK:
        raise MisaError(fn, status)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"q/k must be bfloat16 or float32, got {t.dtype}")


def _need(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _need_opt(t: Optional[torch.Tensor], name: str, dtype=None):
    if t is not None:
        _need(t, name, dtype)


def _on_device(*ts):
    """Every given tensor is on the current CUDA device, where the library launches."""
    cur = torch.cuda.current_device()
    for t in ts:
        if t is not None and t.get_device() != cur:
            raise ValueError(f"every tensor must be on the current device cuda:{cur}; one is on {t.device}")


def _cache_geometry(k: torch.Tensor, T: int):
    """(L, d, k_seq_stride) of a shared [L, d] or per-query [T, L, d] key cache."""
    s = k.shape
    if len(s) == 2:
        return s[0], s[1], 0
    if len(s) == 3:
        if s[0] != T:
            raise ValueError(f"per-query cache needs k.shape[0] == T ({T}), got {s[0]}")
        return s[1], s[2], s[1] * s[2]
    raise ValueError("k must be [L, d] or [T, L, d]")


# Shape checks.  The C library sees only pointers and sizes, so a tensor smaller than the sizes
# passed with it would be read or written past its end; these run before any device check.
def _matrix(t, name: str, rows: int, cols: Optional[int] = None, min_cols: Optional[int] = None):
    """t is 2-D with at least `rows` rows and exactly `cols` (or at least `min_cols`) columns."""
    s = t.shape
    if len(s) != 2 or s[0] < rows or (cols is not None and s[1] != cols) or \
            (min_cols is not None and s[1] < min_cols):
        c = cols if cols is not None else (f">= {min_cols}" if min_cols is not None else "*")
        raise ValueError(f"{name} must be [>= {rows}, {c}], got {tuple(t.shape)}")


def _queries(q, w, n):
    """(T, H_I, d) of a query batch q [T, H_I, d] with w [>= T, H_I] and n [>= T]."""
    s = q.shape
    if len(s) != 3:
        raise ValueError(f"q must be [T, H_I, d], got {tuple(s)}")
    T, H_I, d = s
    _matrix(w, "w", T, H_I)
    ns = n.shape
    if len(ns) != 1 or ns[0] < T:
        raise ValueError(f"n must be [>= {T}], got {tuple(ns)}")
    return T, H_I, d


def _cache(k, T: int, d: int):
    """(L, k_seq_stride) of the key cache of a query batch whose vectors have d elements."""
    L, dk, kss = _cache_geometry(k, T)
    if dk != d:
        raise ValueError(f"k rows have {dk} elements, q rows {d}")
    return L, kss


def _pooled(kbar, k, T: int, L: int, B: int):
    """kbar matches the cache: [>= ceil(L/B), d] for a shared cache, [>= T, >= ceil(L/B), d] for
    per-query caches.  Returns the pooled caches' stride in floats (0 when shared)."""
    M = -(-L // B)
    ks, bs = k.shape, kbar.shape
    d = ks[-1]
    if not (len(bs) == len(ks) and bs[-2] >= M and bs[-1] == d and (len(bs) == 2 or bs[0] >= T)):
        want = f"[{M}, {d}]" if len(ks) == 2 else f"[{T}, {M}, {d}]"
        raise ValueError(f"kbar must be {want} for this cache and B = {B}, got {tuple(bs)}")
    return 0 if len(bs) == 2 else bs[1] * bs[2]


def _outputs(T: int, topk: int, idx, vals):
    """Caller-provided selection outputs hold [>= T, topk]."""
    if idx is not None:
        _matrix(idx, "idx", T, topk)
    if vals is not None:
        _matrix(vals, "vals", T, topk)


def misa_device_check() -> None:
    """Waits for the device, then raises MisaError if a tensor-core kernel stopped early on a
    wait that ran out since the last check (its outputs are then incomplete)."""
    _check("misa_device_check", _lib.misa_device_check())


def misa_bad_index_counts():
    """Counts of skipped out-of-range ids since the last read, (heads, candidates, pages); all zero
    unless the bounds-checked library is loaded.  Waits for the device; clears the counts."""
    out = (ctypes.c_uint * 3)()
    _check("misa_bad_index_counts", _lib.misa_bad_index_counts(out))
    return tuple(int(x) for x in out)


def checked_build() -> bool:
    return bool(_lib.misa_checked_build())


def misa_workspace_bytes(op: int, T: int, L: int, H_I: int, B: int = 1, h: int = 0, topk: int = 0,
                         kp: int = 0) -> int:
    return int(_lib.misa_workspace_bytes(op, T, L, H_I, B, h, topk, kp))


class Workspace:
    """A reusable, 256-byte aligned device scratch buffer (grown on demand).  One Workspace serves
    calls that are ordered on one stream; give each stream that may overlap another its own.

    The buffer is allocated on the stream of the call that needs it, so the caching allocator
    hands its memory to no other tensor while that stream's kernels may still use it.  A call on
    another stream marks the buffer as used there too (record_stream, outside graph capture), so
    a buffer that is replaced later returns to the allocator only after the work of every stream
    that used it.  A buffer that a captured call used is kept beside the one that replaces it, since the
    graph uses it at every replay: a Workspace lives as long as the graphs that were captured with it."""

    def __init__(self, device=None):
        self.device = device
        self.buf = None
        self._in_graph = False  # a captured call uses buf
        self._kept = []  # replaced buffers that captured calls use
        self._home = None  # raw handle of the stream the buffer was allocated on

    def get(self, nbytes: int, stream=None) -> Optional[torch.Tensor]:
        if nbytes <= 0:
            return None
        st = stream if stream is not None else torch.cuda.current_stream(self.device)
        if self.buf is None or self.buf.numel() < nbytes:
            if self._in_graph:
                self._kept.append(self.buf)
                self._in_graph = False
            with torch.cuda.stream(st):
                self.buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device or "cuda")
            self._home = int(st.cuda_stream)
        elif int(st.cuda_stream) != self._home and not torch.cuda.is_current_stream_capturing():
            self.buf.record_stream(st)
        if torch.cuda.is_current_stream_capturing():
            self._in_graph = True
        return self.buf

    def release(self) -> None:
        """Drop the buffers (their memory goes back to torch's caching allocator); graphs that were captured
        with this Workspace are not replayed after it."""
        self.buf = None
        self._home = None
        self._in_graph = False
        self._kept = []


_default_ws = {}


def _ws(ws: Optional[Workspace], device, stream=None) -> Workspace:
    """The caller's Workspace, or the default one of (device, stream): calls ordered on one stream
    share it, calls on different streams never do.  Default workspaces stay allocated (each as
    large as the largest call made on its stream) until release_default_workspaces()."""
    if ws is not None:
        return ws
    st = stream if stream is not None else torch.cuda.current_stream(device)
    key = (str(device), int(st.cuda_stream))
    w = _default_ws.get(key)
    if w is None:
        w = _default_ws[key] = Workspace(device)
    return w


def release_default_workspaces() -> None:
    """Free every default workspace (for example after a run on many external streams, whose
    handles could otherwise be reused by unrelated streams that then inherit a large buffer).
    Synchronises the device first, so no kernel still uses them; graphs of calls that were captured
    without a Workspace and do not keep their scratch themselves are not replayed after it."""
    if _default_ws:
        torch.cuda.synchronize()
    _default_ws.clear()
    _by_handle.clear()


def misa_pool_keys(k: torch.Tensor, B: int, kbar: Optional[torch.Tensor] = None, block_begin: int = 0,
                   block_end: Optional[int] = None, stream=None) -> torch.Tensor:
    """Block means of every cache: k [L,d] or [S,L,d] -> kbar [M,d] or [S,M,d] (fp32)."""
    if k.dim() not in (2, 3):
        raise ValueError(f"k must be [L, d] or [S, L, d], got {tuple(k.shape)}")
    shared = k.dim() == 2
    S = 1 if shared else k.shape[0]
    L, d = k.shape[-2], k.shape[-1]
    M = -(-L // B)
    if kbar is not None and tuple(kbar.shape) != ((M, d) if shared else (S, M, d)):
        raise ValueError(f"kbar must be {[M, d] if shared else [S, M, d]}, got {tuple(kbar.shape)}")
    _need(k, "k")
    if kbar is None:
        kbar = torch.empty((M, d) if shared else (S, M, d), dtype=torch.float32, device=k.device)
    _need(kbar, "kbar", torch.float32)
    _on_device(k, kbar)
    block_end = M if block_end is None else block_end
    _check("misa_pool_keys", _lib.misa_pool_keys(
        _p(k), 0 if shared else L * d, S, L, d, B, _dtype_code(k), _p(kbar), 0 if shared else M * d,
        block_begin, block_end, _stream(stream)))
    return kbar


def misa_route(q, w, k, kbar, n, B: int, h: int, heads=None, r=None, ws: Optional[Workspace] = None,
               want_r: bool = False, stream=None):
    """Routed heads [T, h] (descending router score) and, if asked, router scores r [T, H_I]."""
    T, H_I, d = _queries(q, w, n)
    L, kss = _cache(k, T, d)
    kbss = _pooled(kbar, k, T, L, B)
    if heads is not None:
        _matrix(heads, "heads", T, h)
    if r is not None:
        _matrix(r, "r", T, H_I)
    _need(q, "q")
    _need(k, "k", q.dtype)
    _need(w, "w", torch.float32)
    _need(n, "n", torch.int32)
    _need(kbar, "kbar", torch.float32)
    _need_opt(heads, "heads", torch.int32)
    _need_opt(r, "r", torch.float32)
    _on_device(q, k, w, n, kbar, heads, r)
    if heads is None:
        heads = torch.empty((T, h), dtype=torch.int32, device=q.device)
    if r is None and want_r:
        r = torch.empty((T, H_I), dtype=torch.float32, device=q.device)
    nbytes = misa_workspace_bytes(OP_ROUTE, T, L, H_I, B, h)
    buf = _ws(ws, q.device, stream).get(nbytes, stream)
    _check("misa_route", _lib.misa_route(
        _p(q), _p(w), _p(k), kss, _p(kbar), kbss, _p(n), T, L, H_I, d, B, h, _dtype_code(q), _p(heads), _p(r),
        _p(buf), nbytes, _stream(stream)))
    return heads, r


def misa_token_scores(q, w, k, n, heads=None, out=None, select_topk: int = 0, select_ws=None, stream=None):
    """Scores [T, L] fp32 (entries s >= n_t untouched); heads None = all heads (dense score).
    With select_topk > 0 and a Workspace, a top-select_topk selection of the scores is prepared in
    that workspace (for one bf16 cache per query: a sampled cut and the candidate list of every
    query) for misa_topk_select(..., ws=<same>, ws_prepared=True)."""
    T, H_I, d = _queries(q, w, n)
    L, kss = _cache(k, T, d)
    if heads is not None:
        _matrix(heads, "heads", T)
    if out is not None:
        _matrix(out, "out", T, min_cols=L)
    _need(q, "q")
    _need(k, "k", q.dtype)
    _need(w, "w", torch.float32)
    _need(n, "n", torch.int32)
    _need_opt(out, "out", torch.float32)
    h = 0
    if heads is not None:
        _need(heads, "heads", torch.int32)
        h = heads.shape[1]
    _on_device(q, k, w, n, heads, out)
    if out is None:
        out = torch.empty((T, L), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32)
    buf, nbytes = None, 0
    if select_topk > 0:
        if select_ws is None:
            raise ValueError("select_topk needs select_ws")
        nbytes = misa_workspace_bytes(OP_TOPK_SELECT, T, L, H_I)
        buf = select_ws.get(nbytes, stream)
    _check("misa_token_scores", _lib.misa_token_scores(
        _p(q), _p(w), _p(k), kss, _p(n), _p(heads), T, L, H_I, d, h, _dtype_code(q), _p(out), out.shape[1],
        select_topk, _p(buf), nbytes, _stream(stream)))
    return out


def misa_topk_select(scores, n, topk: int, L: Optional[int] = None, idx=None, vals=None, want_vals=True,
                     ws: Optional[Workspace] = None, ws_prepared: bool = False, stream=None):
    """Top-k per row of scores [T, ld] over entries s < min(n_t, L) -> (idx [T, k], vals [T, k])."""
    if scores.dim() != 2:
        raise ValueError(f"scores must be [T, ld], got {tuple(scores.shape)}")
    T, ld = scores.shape
    if n.dim() != 1 or n.shape[0] < T:
        raise ValueError(f"n must be [>= {T}], got {tuple(n.shape)}")
    if idx is not None:
        _matrix(idx, "idx", T, topk)
    if vals is not None:
        _matrix(vals, "vals", T, topk)
    _need(scores, "scores", torch.float32)
    _need(n, "n", torch.int32)
    _need_opt(idx, "idx", torch.int32)
    _need_opt(vals, "vals", torch.float32)
    _on_device(scores, n, idx, vals)
    L = ld if L is None else L
    if idx is None:
        idx = torch.empty((T, topk), dtype=torch.int32, device=scores.device)
    if vals is None and want_vals:
        vals = torch.empty((T, topk), dtype=torch.float32, device=scores.device)
    nbytes = misa_workspace_bytes(OP_TOPK_SELECT, T, L, 8)
    buf = _ws(ws, scores.device, stream).get(nbytes, stream)
    _check("misa_topk_select", _lib.misa_topk_select(
        _p(scores), ld, _p(n), T, L, topk, _p(idx), _p(vals), _p(buf), nbytes, int(ws_prepared), _stream(stream)))
    return idx, vals


def misa_score_topk(q, w, k, n, heads, topk: int, idx=None, vals=None, scores_full=None, want_vals=True,
                    ws: Optional[Workspace] = None, stream=None):
    """Routed scoring + top-k -> (idx [T, k], vals [T, k]); the index order is not specified."""
    T, H_I, d = _queries(q, w, n)
    L, kss = _cache(k, T, d)
    _matrix(heads, "heads", T)
    _outputs(T, topk, idx, vals)
    if scores_full is not None:
        _matrix(scores_full, "scores_full", T, L)
    _need(q, "q")
    _need(k, "k", q.dtype)
    _need(w, "w", torch.float32)
    _need(n, "n", torch.int32)
    _need(heads, "heads", torch.int32)
    _need_opt(idx, "idx", torch.int32)
    _need_opt(vals, "vals", torch.float32)
    _need_opt(scores_full, "scores_full", torch.float32)
    _on_device(q, k, w, n, heads, idx, vals, scores_full)
    h = heads.shape[1]
    if idx is None:
        idx = torch.empty((T, topk), dtype=torch.int32, device=q.device)
    if vals is None and want_vals:
        vals = torch.empty((T, topk), dtype=torch.float32, device=q.device)
    op = OP_TOPK_SELECT if scores_full is not None else OP_SCORE_TOPK
    nbytes = misa_workspace_bytes(op, T, L, H_I, 1, h, topk)
    buf = _ws(ws, q.device, stream).get(nbytes, stream)
    _check("misa_score_topk", _lib.misa_score_topk(
        _p(q), _p(w), _p(k), kss, _p(n), _p(heads), T, L, H_I, d, h, topk, _dtype_code(q), _p(idx), _p(vals),
        _p(scores_full), _p(buf), nbytes, _stream(stream)))
    return idx, vals


def misa_score_topk_fused(q, w, k, n, heads, topk: int, idx=None, vals=None, want_vals=True,
                          ws: Optional[Workspace] = None, stream=None):
    """misa_score_topk for queries sharing one bf16 cache k [L, d], without score rows (sampled cut,
    candidate lists, exact redo of the queries whose list fell short or overflowed) -> (idx, vals)."""
    T, H_I, d = _queries(q, w, n)
    if k.dim() != 2:
        raise ValueError(f"k must be one shared cache [L, d], got {tuple(k.shape)}")
    L, _ = _cache(k, T, d)
    _matrix(heads, "heads", T)
    _outputs(T, topk, idx, vals)
    _need(q, "q", torch.bfloat16)
    _need(k, "k", torch.bfloat16)
    _need(w, "w", torch.float32)
    _need(n, "n", torch.int32)
    _need(heads, "heads", torch.int32)
    _need_opt(idx, "idx", torch.int32)
    _need_opt(vals, "vals", torch.float32)
    _on_device(q, k, w, n, heads, idx, vals)
    h = heads.shape[1]
    if idx is None:
        idx = torch.empty((T, topk), dtype=torch.int32, device=q.device)
    if vals is None and want_vals:
        vals = torch.empty((T, topk), dtype=torch.float32, device=q.device)
    nbytes = misa_workspace_bytes(OP_SCORE_TOPK_FUSED, T, L, H_I, 0, h, topk)
    buf = _ws(ws, q.device, stream).get(nbytes, stream)
    _check("misa_score_topk_fused", _lib.misa_score_topk_fused(
        _p(q), _p(w), _p(k), _p(n), _p(heads), T, L, H_I, d, h, topk, BF16, _p(idx), _p(vals), _p(buf), nbytes,
        _stream(stream)))
    return idx, vals


def misa_hier_topk_fused(q, w, k, n, heads, kp: int, topk: int, idx=None, vals=None, want_vals=True,
                         ws: Optional[Workspace] = None, stream=None):
    """MISA-dagger for per-query bf16 caches k [T, L, d] in one call: routed scores, top-k' by them,
    dense scores of those k' kept while the keys are read once, top-k of the dense score ->
    (idx [T, k], vals [T, k])."""
    T, H_I, d = _queries(q, w, n)
    if k.dim() != 3:
        raise ValueError(f"k must be per-query caches [T, L, d], got {tuple(k.shape)}")
    L, kss = _cache(k, T, d)
    _matrix(heads, "heads", T)
    _outputs(T, topk, idx, vals)
    _need(q, "q", torch.bfloat16)
    _need(k, "k", torch.bfloat16)
    _need(w, "w", torch.float32)
    _need(n, "n", torch.int32)
    _need(heads, "heads", torch.int32)
    _need_opt(idx, "idx", torch.int32)
    _need_opt(vals, "vals", torch.float32)
    _on_device(q, k, w, n, heads, idx, vals)
    h = heads.shape[1]
    if idx is None:
        idx = torch.empty((T, topk), dtype=torch.int32, device=q.device)
    if vals is None and want_vals:
        vals = torch.empty((T, topk), dtype=torch.float32, device=q.device)
    nbytes = misa_workspace_bytes(OP_HIER_FUSED, T, L, H_I, 0, h, topk, kp)
    buf = _ws(ws, q.device, stream).get(nbytes, stream)
    _check("misa_hier_topk_fused", _lib.misa_hier_topk_fused(
        _p(q), _p(w), _p(k), kss, _p(n), _p(heads), T, L, H_I, d, h, kp, topk, BF16, _p(idx), _p(vals), _p(buf),
        nbytes, _stream(stream)))
    return idx, vals


def misa_hier_rerank(q, w, k, n, cand, topk: int, idx=None, vals=None, want_vals=True,
                     ws: Optional[Workspace] = None, stream=None):
    """MISA-dagger fine stage: dense re-score of cand [T, k'] -> (idx [T, k], vals [T, k])."""
    T, H_I, d = _queries(q, w, n)
    L, kss = _cache(k, T, d)
    _matrix(cand, "cand", T)
    _outputs(T, topk, idx, vals)
    _need(q, "q")
    _need(k, "k", q.dtype)
    _need(w, "w", torch.float32)
    _need(n, "n", torch.int32)
    _need(cand, "cand", torch.int32)
    _need_opt(idx, "idx", torch.int32)
    _need_opt(vals, "vals", torch.float32)
    _on_device(q, k, w, n, cand, idx, vals)
    kp = cand.shape[1]
    if idx is None:
        idx = torch.empty((T, topk), dtype=torch.int32, device=q.device)
    if vals is None and want_vals:
        vals = torch.empty((T, topk), dtype=torch.float32, device=q.device)
    nbytes = misa_workspace_bytes(OP_RERANK, T, L, H_I, 1, 0, topk, kp)
    buf = _ws(ws, q.device, stream).get(nbytes, stream)
    _check("misa_hier_rerank", _lib.misa_hier_rerank(
        _p(q), _p(w), _p(k), kss, _p(n), _p(cand), T, L, H_I, d, kp, topk, _dtype_code(q), _p(idx), _p(vals),
        _p(buf), nbytes, _stream(stream)))
    return idx, vals


def dsa_dense_topk(q, w, k, n, topk: int, idx=None, vals=None, want_vals=True, ws: Optional[Workspace] = None,
                   stream=None):
    """Dense all-head indexer -> (idx [T, k], vals [T, k]); the index order is not specified."""
    T, H_I, d = _queries(q, w, n)
    L, kss = _cache(k, T, d)
    _outputs(T, topk, idx, vals)
    _need(q, "q")
    _need(k, "k", q.dtype)
    _need(w, "w", torch.float32)
    _need(n, "n", torch.int32)
    _need_opt(idx, "idx", torch.int32)
    _need_opt(vals, "vals", torch.float32)
    _on_device(q, k, w, n, idx, vals)
    if idx is None:
        idx = torch.empty((T, topk), dtype=torch.int32, device=q.device)
    if vals is None and want_vals:
        vals = torch.empty((T, topk), dtype=torch.float32, device=q.device)
    nbytes = misa_workspace_bytes(OP_DENSE_TOPK, T, L, H_I, 1, 0, topk)
    buf = _ws(ws, q.device, stream).get(nbytes, stream)
    _check("dsa_dense_topk", _lib.dsa_dense_topk(
        _p(q), _p(w), _p(k), kss, _p(n), T, L, H_I, d, topk, _dtype_code(q), _p(idx), _p(vals), _p(buf), nbytes,
        _stream(stream)))
    return idx, vals


def misa_block_filter_topk(q, w, k, kbar, n, heads, B: int, m: int, topk: int, idx=None, vals=None,
                           blocks=None, block_scores=None, want_vals=True, want_block_scores=False,
                           ws: Optional[Workspace] = None, stream=None):
    """Block filter + routed refinement: block scores with the routed heads, the m best blocks,
    then top-k over their tokens -> dict with idx [T, k], vals [T, k] (or None), blocks [T, m]
    (-1 padded; order not specified) and, if asked, block_scores [T, ceil(L/B)]."""
    T, H_I, d = _queries(q, w, n)
    L, kss = _cache(k, T, d)
    kbss = _pooled(kbar, k, T, L, B)
    M = -(-L // B)
    _matrix(heads, "heads", T)
    _outputs(T, topk, idx, vals)
    if blocks is not None:
        _matrix(blocks, "blocks", T, m)
    if block_scores is not None:
        _matrix(block_scores, "block_scores", T, min_cols=M)
    _need(q, "q")
    _need(k, "k", q.dtype)
    _need(w, "w", torch.float32)
    _need(n, "n", torch.int32)
    _need(kbar, "kbar", torch.float32)
    _need(heads, "heads", torch.int32)
    _need_opt(idx, "idx", torch.int32)
    _need_opt(vals, "vals", torch.float32)
    _need_opt(blocks, "blocks", torch.int32)
    _need_opt(block_scores, "block_scores", torch.float32)
    _on_device(q, k, w, n, kbar, heads, idx, vals, blocks, block_scores)
    h = heads.shape[1]
    if idx is None:
        idx = torch.empty((T, topk), dtype=torch.int32, device=q.device)
    if vals is None and want_vals:
        vals = torch.empty((T, topk), dtype=torch.float32, device=q.device)
    if blocks is None:
        blocks = torch.empty((T, m), dtype=torch.int32, device=q.device)
    if block_scores is None and want_block_scores:
        block_scores = torch.empty((T, M), dtype=torch.float32, device=q.device)
    ld_bs = 0 if block_scores is None else block_scores.shape[1]
    nbytes = misa_workspace_bytes(OP_BLOCK_FILTER, T, L, H_I, B, h, topk, m)
    buf = _ws(ws, q.device, stream).get(nbytes, stream)
    _check("misa_block_filter_topk", _lib.misa_block_filter_topk(
        _p(q), _p(w), _p(k), kss, _p(kbar), kbss, _p(n), _p(heads), T, L, H_I, d, B, h, m, topk, _dtype_code(q),
        _p(block_scores), ld_bs, _p(blocks), _p(idx), _p(vals), _p(buf), nbytes, _stream(stream)))
    return {"idx": idx, "vals": vals, "blocks": blocks, "block_scores": block_scores}


def misa_indexer(q, w, k, kbar, n, B: int, h: int, topk: int, kp: Optional[int] = None,
                 ws: Optional[Workspace] = None, stream=None, m: Optional[int] = None):
    """The whole indexer for one batch: route -> routed scoring -> top-k (MISA), or with kp given
    route -> routed scoring -> top-k' candidates -> dense re-rank -> top-k (MISA-dagger), or with
    m given route -> block filter keeping m blocks -> routed scoring of their tokens -> top-k.
    Returns a dict with idx [T, k], vals [T, k], heads [T, h], (MISA-dagger) cand [T, k'] and
    (block filter) blocks [T, m]."""
    if kp is not None and m is not None:
        raise ValueError("give kp (MISA-dagger) or m (block filter), not both")
    heads, _ = misa_route(q, w, k, kbar, n, B, h, ws=ws, stream=stream)
    if m is not None:
        res = misa_block_filter_topk(q, w, k, kbar, n, heads, B, m, topk, ws=ws, stream=stream)
        return {"idx": res["idx"], "vals": res["vals"], "heads": heads, "blocks": res["blocks"]}
    if kp is None:
        idx, vals = misa_score_topk(q, w, k, n, heads, topk, ws=ws, stream=stream)
        return {"idx": idx, "vals": vals, "heads": heads}
    cand, _ = misa_score_topk(q, w, k, n, heads, kp, want_vals=False, ws=ws, stream=stream)
    idx, vals = misa_hier_rerank(q, w, k, n, cand, topk, ws=ws, stream=stream)
    return {"idx": idx, "vals": vals, "heads": heads, "cand": cand}


_lib.misa_hier_rerank_static.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int64] + [ctypes.c_void_p] * 2 + \
    [ctypes.c_int] * 7 + [ctypes.c_void_p] * 3
_lib.misa_hier_rerank_static.restype = ctypes.c_int
STATIC_RERANK_SCRATCH_FLOATS = 1 << 20


def misa_hier_rerank_static(q, w, k, n, cand, topk: int, idx=None, vals=None, want_vals=True, stream=None):
    """misa_hier_rerank for callers that cannot allocate device memory: the library's fixed
    scratch array replaces the workspace (T * k' <= STATIC_RERANK_SCRATCH_FLOATS).  Calls that
    overlap on the GPU share that array and must be ordered on one stream."""
    T, H_I, d = _queries(q, w, n)
    L, kss = _cache(k, T, d)
    _matrix(cand, "cand", T)
    _outputs(T, topk, idx, vals)
    _need(q, "q")
    _need(k, "k", q.dtype)
    _need(w, "w", torch.float32)
    _need(n, "n", torch.int32)
    _need(cand, "cand", torch.int32)
    _need_opt(idx, "idx", torch.int32)
    _need_opt(vals, "vals", torch.float32)
    _on_device(q, k, w, n, cand, idx, vals)
    kp = cand.shape[1]
    if idx is None:
        idx = torch.empty((T, topk), dtype=torch.int32, device=q.device)
    if vals is None and want_vals:
        vals = torch.empty((T, topk), dtype=torch.float32, device=q.device)
    _check("misa_hier_rerank_static", _lib.misa_hier_rerank_static(
        _p(q), _p(w), _p(k), kss, _p(n), _p(cand), T, L, H_I, d, kp, topk, _dtype_code(q), _p(idx), _p(vals),
        _stream(stream)))
    return idx, vals


# ---- paged key caches: pool [num_pages, page_size, d], page_table [T, max_pages] int32 ----------

def _paged_geometry(pool, page_table, T: int, d: int, L: Optional[int]):
    """(num_pages, page_size, max_pages, L) of a paged cache; L defaults to what the table covers."""
    if pool.dim() != 3 or pool.shape[2] != d:
        raise ValueError(f"pool must be [num_pages, page_size, {d}], got {tuple(pool.shape)}")
    _matrix(page_table, "page_table", T)
    num_pages, page_size = pool.shape[0], pool.shape[1]
    max_pages = page_table.shape[1]
    L = max_pages * page_size if L is None else L
    if L > max_pages * page_size:
        raise ValueError(f"a table of {max_pages} pages of {page_size} keys cannot hold L = {L}")
    return num_pages, page_size, max_pages, L


def misa_pool_keys_paged(pool, page_table, B: int, L: Optional[int] = None, kbar=None, block_begin: int = 0,
                         block_end: Optional[int] = None, stream=None):
    """Block means of every sequence's logical cache through its page table -> kbar [S, M, d]."""
    S = page_table.shape[0]
    num_pages, page_size, max_pages, L = _paged_geometry(pool, page_table, S, pool.shape[-1], L)
    d = pool.shape[2]
    M = -(-L // B)
    if kbar is not None and tuple(kbar.shape) != (S, M, d):
        raise ValueError(f"kbar must be {[S, M, d]}, got {tuple(kbar.shape)}")
    _need(pool, "pool")
    _need(page_table, "page_table", torch.int32)
    if kbar is None:
        kbar = torch.empty((S, M, d), dtype=torch.float32, device=pool.device)
    _need(kbar, "kbar", torch.float32)
    _on_device(pool, page_table, kbar)
    block_end = M if block_end is None else block_end
    _check("misa_pool_keys_paged", _lib.misa_pool_keys_paged(
        _p(pool), num_pages, page_size, _p(page_table), max_pages, S, L, d, B, _dtype_code(pool), _p(kbar), M * d,
        block_begin, block_end, _stream(stream)))
    return kbar


def misa_route_paged(q, w, pool, page_table, kbar, n, B: int, h: int, L: Optional[int] = None, heads=None, r=None,
                     ws: Optional[Workspace] = None, want_r: bool = False, stream=None):
    """misa_route on paged caches -> (heads [T, h], r [T, H_I] or None)."""
    T, H_I, d = _queries(q, w, n)
    num_pages, page_size, max_pages, L = _paged_geometry(pool, page_table, T, d, L)
    M = -(-L // B)
    if kbar.dim() != 3 or kbar.shape[0] < T or kbar.shape[1] < M or kbar.shape[2] != d:
        raise ValueError(f"kbar must be [{T}, {M}, {d}], got {tuple(kbar.shape)}")
    if heads is not None:
        _matrix(heads, "heads", T, h)
    if r is not None:
        _matrix(r, "r", T, H_I)
    _need(q, "q")
    _need(pool, "pool", q.dtype)
    _need(w, "w", torch.float32)
    _need(n, "n", torch.int32)
    _need(kbar, "kbar", torch.float32)
    _need(page_table, "page_table", torch.int32)
    _need_opt(heads, "heads", torch.int32)
    _need_opt(r, "r", torch.float32)
    _on_device(q, pool, w, n, kbar, page_table, heads, r)
    if heads is None:
        heads = torch.empty((T, h), dtype=torch.int32, device=q.device)
    if r is None and want_r:
        r = torch.empty((T, H_I), dtype=torch.float32, device=q.device)
    nbytes = misa_workspace_bytes(OP_ROUTE_PAGED, T, L, H_I, B, h)
    buf = _ws(ws, q.device, stream).get(nbytes, stream)
    _check("misa_route_paged", _lib.misa_route_paged(
        _p(q), _p(w), _p(pool), num_pages, page_size, _p(page_table), max_pages, _p(kbar),
        kbar.shape[1] * kbar.shape[2], _p(n), T, L, H_I, d, B, h, _dtype_code(q), _p(heads), _p(r), _p(buf), nbytes,
        _stream(stream)))
    return heads, r


def misa_score_topk_paged(q, w, pool, page_table, n, heads, topk: int, L: Optional[int] = None, idx=None, vals=None,
                          want_vals=True, ws: Optional[Workspace] = None, stream=None):
    """misa_score_topk on paged caches -> (idx [T, k], vals [T, k]); logical token indices."""
    T, H_I, d = _queries(q, w, n)
    num_pages, page_size, max_pages, L = _paged_geometry(pool, page_table, T, d, L)
    _matrix(heads, "heads", T)
    _outputs(T, topk, idx, vals)
    _need(q, "q")
    _need(pool, "pool", q.dtype)
    _need(w, "w", torch.float32)
    _need(n, "n", torch.int32)
    _need(heads, "heads", torch.int32)
    _need(page_table, "page_table", torch.int32)
    _need_opt(idx, "idx", torch.int32)
    _need_opt(vals, "vals", torch.float32)
    _on_device(q, pool, w, n, heads, page_table, idx, vals)
    h = heads.shape[1]
    if idx is None:
        idx = torch.empty((T, topk), dtype=torch.int32, device=q.device)
    if vals is None and want_vals:
        vals = torch.empty((T, topk), dtype=torch.float32, device=q.device)
    nbytes = misa_workspace_bytes(OP_SCORE_TOPK_PAGED, T, L, H_I, 0, h, topk)
    buf = _ws(ws, q.device, stream).get(nbytes, stream)
    _check("misa_score_topk_paged", _lib.misa_score_topk_paged(
        _p(q), _p(w), _p(pool), num_pages, page_size, _p(page_table), max_pages, _p(n), _p(heads), T, L, H_I, d, h,
        topk, _dtype_code(q), _p(idx), _p(vals), _p(buf), nbytes, _stream(stream)))
    return idx, vals


def misa_hier_rerank_paged(q, w, pool, page_table, n, cand, topk: int, L: Optional[int] = None, idx=None,
                           vals=None, want_vals=True, ws: Optional[Workspace] = None, stream=None):
    """misa_hier_rerank on paged caches: dense re-score of logical candidates cand [T, k']."""
    T, H_I, d = _queries(q, w, n)
    num_pages, page_size, max_pages, L = _paged_geometry(pool, page_table, T, d, L)
    _matrix(cand, "cand", T)
    _outputs(T, topk, idx, vals)
    _need(q, "q")
    _need(pool, "pool", q.dtype)
    _need(w, "w", torch.float32)
    _need(n, "n", torch.int32)
    _need(cand, "cand", torch.int32)
    _need(page_table, "page_table", torch.int32)
    _need_opt(idx, "idx", torch.int32)
    _need_opt(vals, "vals", torch.float32)
    _on_device(q, pool, w, n, cand, page_table, idx, vals)
    kp = cand.shape[1]
    if idx is None:
        idx = torch.empty((T, topk), dtype=torch.int32, device=q.device)
    if vals is None and want_vals:
        vals = torch.empty((T, topk), dtype=torch.float32, device=q.device)
    nbytes = misa_workspace_bytes(OP_RERANK_PAGED, T, L, H_I, 0, 0, topk, kp)
    buf = _ws(ws, q.device, stream).get(nbytes, stream)
    _check("misa_hier_rerank_paged", _lib.misa_hier_rerank_paged(
        _p(q), _p(w), _p(pool), num_pages, page_size, _p(page_table), max_pages, _p(n), _p(cand), T, L, H_I, d, kp,
        topk, _dtype_code(q), _p(idx), _p(vals), _p(buf), nbytes, _stream(stream)))
    return idx, vals


def misa_indexer_paged(q, w, pool, page_table, kbar, n, B: int, h: int, topk: int, kp: Optional[int] = None,
                       L: Optional[int] = None, ws: Optional[Workspace] = None, stream=None):
    """misa_indexer on paged caches (MISA, or MISA-dagger with kp given)."""
    heads, _ = misa_route_paged(q, w, pool, page_table, kbar, n, B, h, L=L, ws=ws, stream=stream)
    if kp is None:
        idx, vals = misa_score_topk_paged(q, w, pool, page_table, n, heads, topk, L=L, ws=ws, stream=stream)
        return {"idx": idx, "vals": vals, "heads": heads}
    cand, _ = misa_score_topk_paged(q, w, pool, page_table, n, heads, kp, L=L, want_vals=False, ws=ws,
                                    stream=stream)
    idx, vals = misa_hier_rerank_paged(q, w, pool, page_table, n, cand, topk, L=L, ws=ws, stream=stream)
    return {"idx": idx, "vals": vals, "heads": heads, "cand": cand}


# ---- attention beside the indexer: 4-bit caches, their attention and eviction, prompt attention ------
#
# Decode steps make these calls every few microseconds, so their marshalling is kept short: one check per
# tensor, raw stream handles, pointers passed as integers.

def _current(t: torch.Tensor, name: str) -> int:
    """Index of the current CUDA device, where the library launches (t: the call's first tensor)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return torch._C._cuda_getDevice()


def _ready(t: Optional[torch.Tensor], name: str, dtype, cur: int):
    """Data pointer of a contiguous tensor of this type on the current device (None for None)."""
    if t is None:
        return None
    if t.get_device() != cur or t.dtype is not dtype or not t.is_contiguous():
        _need(t, name, dtype)
        _on_device(t)
    return t.data_ptr()


def _handle(stream, cur: int) -> int:
    return torch._C._cuda_getCurrentRawStream(cur) if stream is None else stream.cuda_stream


_by_handle = {}  # (device index, stream handle) -> the default Workspace of that stream


def _capturing(stream) -> bool:
    """Whether a call on this stream (None: the current one) is being captured."""
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _scratch(ws: Optional["Workspace"], t: torch.Tensor, cur: int, nbytes: int, stream, handle: int):
    """nbytes of scratch for one call: the caller's Workspace, or the stream's default one, or, for a call
    that is captured without a Workspace, a buffer of the graph's own (two graphs that were captured on one
    stream may be replayed on two, and no later call can take the buffer away)."""
    if nbytes == 0:
        return None
    capturing = _capturing(stream)
    if ws is None:
        if capturing:
            return _new((nbytes,), torch.uint8, t.device, stream)
        ws = _by_handle.get((cur, handle))
        if ws is None:
            ws = _by_handle[(cur, handle)] = _ws(None, t.device, stream)
    if ws.buf is None or ws.buf.numel() < nbytes or ws._home != handle:
        ws.get(nbytes, stream)
    if capturing:
        ws._in_graph = True
    return ws.buf


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """An output of a call on `stream`, whose memory is that stream's."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _beside(stream, cur: int, handle: int, *tensors) -> None:
    """Tells the caching allocator that a call on a stream other than the current one uses these tensors, and
    that the current one will use what the call gave them (their owner does not hold them for long enough)."""
    if handle == torch._C._cuda_getCurrentRawStream(cur) or torch.cuda.is_current_stream_capturing():
        return
    now = torch.cuda.current_stream(cur)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
            t.record_stream(now)


def _address(buf) -> Optional[int]:
    return None if buf is None else buf.data_ptr()


@functools.lru_cache(maxsize=4096)
def _ws_bytes(*sizes) -> int:
    return int(_lib.misa_workspace_bytes(*sizes))


def misa_kv4_pool(num_pages: int, page_size: int, H_kv: int, d: int, device="cuda") -> torch.Tensor:
    """An empty pool of 4-bit key and value pages, uint8 [num_pages, H_kv, 2, page_size * 9 d / 16]."""
    if d not in (64, 128) or page_size < 16 or page_size % 16:
        raise ValueError(f"a 4-bit pool needs d of 64 or 128 and pages of a multiple of 16 rows, got d = {d}, "
                         f"page_size = {page_size}")
    return torch.zeros((num_pages, H_kv, 2, page_size * 9 * d // 16), dtype=torch.uint8, device=device)


def _kv4_geometry(pool, page_table, rows: int, d: int):
    """(num_pages, H_kv, page_size, max_pages) of a 4-bit pool with heads of d elements."""
    s = pool.shape
    if len(s) != 4 or s[2] != 2 or s[3] <= 0 or (s[3] * 16) % (9 * d) != 0:
        raise ValueError(f"pool must be [num_pages, H_kv, 2, page_size * {9 * d} / 16], got {tuple(s)}")
    ts = page_table.shape
    if len(ts) != 2 or ts[0] < rows:
        _matrix(page_table, "page_table", rows)
    return s[0], s[1], s[3] * 16 // (9 * d), ts[1]


def _packed_rows(t, name: str) -> int:
    """Row stride in elements of packed rows [rows, H, d]: rows may be strided (a slice of a fused
    projection), the elements of a row may not."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [rows, H, d], got {tuple(t.shape)}")
    rows, H, d = t.shape
    if t.is_contiguous() or t.numel() == 0 or (rows == 1 and t[0].is_contiguous()):
        return H * d
    if t.stride(2) != 1 or (H > 1 and t.stride(1) != d) or t.stride(0) < H * d or t.stride(0) * t.element_size() % 16:
        raise ValueError(f"{name} must have contiguous rows at a stride of a multiple of 16 bytes, got strides "
                         f"{tuple(t.stride())}")
    return t.stride(0)


def _rows_ready(t, name: str, dtype, cur: int) -> int:
    """Data pointer of packed rows that _packed_rows has looked over."""
    if t.get_device() != cur or t.dtype is not dtype:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        _on_device(t)
    return t.data_ptr()


def _packed(cu, start, name: str = "cu") -> int:
    """Number of sequences of cu [S + 1] (and start [>= S])."""
    if cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError(f"{name} must be [S + 1], got {tuple(cu.shape)}")
    S = cu.shape[0] - 1
    if start is not None and (start.dim() != 1 or start.shape[0] < S):
        raise ValueError(f"start must be [>= {S}], got {tuple(start.shape)}")
    return S


def _lengths(n, T: int) -> None:
    if n.dim() != 1 or n.shape[0] < T:
        raise ValueError(f"n must be [>= {T}], got {tuple(n.shape)}")


def misa_kv4_append(k, v, pool, page_table, cu, start, k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """Write packed rows k, v [rows, H_kv, d] into a 4-bit cache: row r of sequence b (cu[b] <= r <
    cu[b + 1]) at its logical position start[b] + r - cu[b].  k_scale and v_scale: one factor per
    tensor, the same in every call on this cache."""
    ldk, ldv = _packed_rows(k, "k"), _packed_rows(v, "v")
    if k.shape != v.shape:
        raise ValueError(f"k and v must have one shape, got {tuple(k.shape)} and {tuple(v.shape)}")
    rows, H_kv, d = k.shape
    S = _packed(cu, start)
    num_pages, Hp, page_size, max_pages = _kv4_geometry(pool, page_table, S, d)
    if Hp != H_kv:
        raise ValueError(f"the pool holds {Hp} kv heads, k has {H_kv}")
    cur = _current(k, "k")
    code, h = _dtype_code(k), _handle(stream, cur)
    _check("misa_kv4_append", _lib.misa_kv4_append(
        _rows_ready(k, "k", k.dtype, cur), _rows_ready(v, "v", k.dtype, cur), ldk, ldv, code, k_scale, v_scale,
        _ready(pool, "pool", torch.uint8, cur), num_pages, page_size, _ready(page_table, "page_table", torch.int32, cur),
        max_pages, _ready(cu, "cu", torch.int32, cur), _ready(start, "start", torch.int32, cur), S, rows, H_kv, d,
        h))
    if stream is not None:
        _beside(stream, cur, h, k, v, pool, page_table, cu, start)


def misa_kv4_read(pool, page_table, cu, start, rows: int, d: int, dtype=torch.bfloat16, k_scale: float = 1.0,
                  v_scale: float = 1.0, k=None, v=None, stream=None):
    """Rows of a 4-bit cache as packed k, v [rows, H_kv, d] (bf16 or fp32); the inverse of misa_kv4_append.
    Rows outside [cu[0], cu[S]) of given k and v are left as they are."""
    S = _packed(cu, start)
    num_pages, H_kv, page_size, max_pages = _kv4_geometry(pool, page_table, S, d)
    for t, name in ((k, "k"), (v, "v")):
        if t is not None and tuple(t.shape) != (rows, H_kv, d):
            raise ValueError(f"{name} must be {[rows, H_kv, d]}, got {tuple(t.shape)}")
    cur = _current(pool, "pool")
    pp, tp = _ready(pool, "pool", torch.uint8, cur), _ready(page_table, "page_table", torch.int32, cur)
    cp, sp = _ready(cu, "cu", torch.int32, cur), _ready(start, "start", torch.int32, cur)
    if k is None:
        k = _new((rows, H_kv, d), dtype, pool.device, stream)
    if v is None:
        v = _new((rows, H_kv, d), dtype, pool.device, stream)
    h = _handle(stream, cur)
    _check("misa_kv4_read", _lib.misa_kv4_read(
        pp, num_pages, page_size, tp, max_pages, cp, sp, S, rows, H_kv, d, _dtype_code(k), k_scale, v_scale,
        _ready(k, "k", dtype, cur), _ready(v, "v", dtype, cur), h))
    if stream is not None:
        _beside(stream, cur, h, k, v, pool, page_table, cu, start)
    return k, v


def misa_kv4_attention(q, pool, page_table, n, idx=None, L: Optional[int] = None, scale: Optional[float] = None,
                       k_scale: float = 1.0, v_scale: float = 1.0, out=None, lse=None, want_lse: bool = False,
                       acc=None, ws: Optional[Workspace] = None, stream=None):
    """Attention of one query token per sequence, q [T, H_q, d] (bf16 or fp32), over its 4-bit cache:
    over the whole prefix, or with idx [T, P] over the tokens listed there (the indexer's selection, -1
    for empty slots) -> (out [T, H_q, d], lse [T, H_q] or None).  scale defaults to 1 / sqrt(d).  acc
    [T, >= L] fp32: every token's softmax weight, summed over the heads, is added to it.  L, the longest
    prefix (a longer one is cut to it), defaults to what the page table reaches; acc may then end inside
    the table's last page, where the weights of tokens behind its end are not kept."""
    if q.dim() != 3:
        raise ValueError(f"q must be [T, H_q, d], got {tuple(q.shape)}")
    T, H_q, d = q.shape
    num_pages, H_kv, page_size, max_pages = _kv4_geometry(pool, page_table, T, d)
    reach = max_pages * page_size
    cols = reach - page_size + 1 if L is None else L  # fewest columns of acc
    L = reach if L is None else L
    _lengths(n, T)
    if idx is not None:
        _matrix(idx, "idx", T, min_cols=1)  # a list of no width has no address and would mean the whole prefix
    if out is not None and tuple(out.shape) != (T, H_q, d):
        raise ValueError(f"out must be {[T, H_q, d]}, got {tuple(out.shape)}")
    if lse is not None:
        _matrix(lse, "lse", T, H_q)
    if acc is not None:
        _matrix(acc, "acc", T, min_cols=cols)
    cur = _current(q, "q")
    code = _dtype_code(q)
    qp, pp = _ready(q, "q", q.dtype, cur), _ready(pool, "pool", torch.uint8, cur)
    tp, np_ = _ready(page_table, "page_table", torch.int32, cur), _ready(n, "n", torch.int32, cur)
    ip, ap = _ready(idx, "idx", torch.int32, cur), _ready(acc, "acc", torch.float32, cur)
    P = 0 if idx is None else idx.shape[1]
    if out is None:
        out = torch.empty_like(q) if stream is None else _new((T, H_q, d), q.dtype, q.device, stream)
    if lse is None and want_lse:
        lse = _new((T, H_q), torch.float32, q.device, stream)
    h = _handle(stream, cur)
    nbytes = _ws_bytes(OP_KV4_ATTENTION, T, L, H_q, H_kv, d, P, int(acc is not None))
    buf = _scratch(ws, q, cur, nbytes, stream, h)
    ld = 0 if acc is None else acc.shape[1]
    _check("misa_kv4_attention", _lib.misa_kv4_attention_cols(
        qp, pp, num_pages, page_size, tp, max_pages, np_, ip, T, L, P, H_q, H_kv, d, code,
        d ** -0.5 if scale is None else scale, k_scale, v_scale, _ready(out, "out", q.dtype, cur),
        _ready(lse, "lse", torch.float32, cur), ap, min(L, ld), ld, _address(buf), nbytes, h))
    if stream is not None:
        _beside(stream, cur, h, q, pool, page_table, n, idx, out, lse, acc)
    return out, lse


def misa_evict_select(acc, n, keep: int, sink: int = 0, recent: int = 0, L: Optional[int] = None, idx=None,
                      n_out=None, acc_out=None, want_acc: bool = False, stream=None):
    """Tokens that stay when every cache is thinned to `keep` by summed attention weight acc [T, >= L]:
    the first `sink`, the last `recent`, and the heaviest of the others -> (idx [T, keep] ascending and
    -1 padded, n_out [T], acc_out [T, >= keep] the weights in that order and zeros behind them, or None).
    n_out may be n itself: the lengths are then updated in place.  L defaults to acc's width; a longer
    prefix is cut to it, its last tokens lost.  To go on summing, give an acc_out as wide as acc:
    want_acc makes one of keep columns, which has none for the tokens appended next."""
    if acc.dim() != 2:
        raise ValueError(f"acc must be [T, ld], got {tuple(acc.shape)}")
    T, ld = acc.shape
    L = ld if L is None else L
    _lengths(n, T)
    if idx is not None:
        _matrix(idx, "idx", T, keep)
    if n_out is not None and (n_out.dim() != 1 or n_out.shape[0] < T):
        raise ValueError(f"n_out must be [>= {T}], got {tuple(n_out.shape)}")
    if acc_out is not None:
        _matrix(acc_out, "acc_out", T, min_cols=keep)
    cur = _current(acc, "acc")
    ap, np_ = _ready(acc, "acc", torch.float32, cur), _ready(n, "n", torch.int32, cur)
    if idx is None:
        idx = _new((T, keep), torch.int32, acc.device, stream)
    if n_out is None:
        n_out = _new((T,), torch.int32, acc.device, stream)
    if acc_out is None and want_acc:
        acc_out = _new((T, keep), torch.float32, acc.device, stream)
    h = _handle(stream, cur)
    _check("misa_evict_select", _lib.misa_evict_select(
        ap, ld, np_, T, L, keep, sink, recent, _ready(idx, "idx", torch.int32, cur),
        _ready(n_out, "n_out", torch.int32, cur), _ready(acc_out, "acc_out", torch.float32, cur),
        0 if acc_out is None else acc_out.shape[1], h))
    if stream is not None:
        _beside(stream, cur, h, acc, n, idx, n_out, acc_out)
    return idx, n_out, acc_out


def misa_kv4_compact(pool, page_table, idx, d: int, ws: Optional[Workspace] = None, stream=None) -> None:
    """Close up a 4-bit cache in place: row idx[t, j] of sequence t moves to row j (idx [T, keep]
    ascending, -1 padded, as misa_evict_select gives it)."""
    if idx.dim() != 2:
        raise ValueError(f"idx must be [T, keep], got {tuple(idx.shape)}")
    T, keep = idx.shape
    num_pages, H_kv, page_size, max_pages = _kv4_geometry(pool, page_table, T, d)
    cur = _current(pool, "pool")
    pp, tp = _ready(pool, "pool", torch.uint8, cur), _ready(page_table, "page_table", torch.int32, cur)
    ip, h = _ready(idx, "idx", torch.int32, cur), _handle(stream, cur)
    nbytes = _ws_bytes(OP_KV4_COMPACT, T, 0, H_kv, 0, d, keep, 0)
    buf = _scratch(ws, pool, cur, nbytes, stream, h)
    _check("misa_kv4_compact", _lib.misa_kv4_compact(
        pp, num_pages, page_size, tp, max_pages, ip, T, keep, H_kv, d,
        _address(buf), nbytes, h))
    if stream is not None:
        _beside(stream, cur, h, pool, page_table, idx)


def misa_keys_compact_paged(pool, page_table, idx, ws: Optional[Workspace] = None, stream=None) -> None:
    """misa_kv4_compact for the indexer's paged keys, pool [num_pages, page_size, 128] (bf16 or fp32).
    Block means are to be pooled again (misa_pool_keys_paged)."""
    if pool.dim() != 3:
        raise ValueError(f"pool must be [num_pages, page_size, d], got {tuple(pool.shape)}")
    if idx.dim() != 2:
        raise ValueError(f"idx must be [T, keep], got {tuple(idx.shape)}")
    T, keep = idx.shape
    _matrix(page_table, "page_table", T)
    cur = _current(pool, "pool")
    code = _dtype_code(pool)
    pp, tp = _ready(pool, "pool", pool.dtype, cur), _ready(page_table, "page_table", torch.int32, cur)
    ip, h = _ready(idx, "idx", torch.int32, cur), _handle(stream, cur)
    num_pages, page_size, d = pool.shape
    nbytes = _ws_bytes(OP_KEYS_COMPACT_PAGED, T, 0, 0, 0, d * pool.element_size(), keep, 0)
    buf = _scratch(ws, pool, cur, nbytes, stream, h)
    _check("misa_keys_compact_paged", _lib.misa_keys_compact_paged(
        pp, num_pages, page_size, tp, page_table.shape[1], ip, T, keep, d, code,
        _address(buf), nbytes, h))
    if stream is not None:
        _beside(stream, cur, h, pool, page_table, idx)


def misa_prompt_attention(q, k, v, cu_q, cu_k=None, scale: Optional[float] = None, out=None, lse=None,
                          want_lse: bool = False, ws: Optional[Workspace] = None, stream=None):
    """Causal attention of packed prompts, q [Tq, H_q, d] and k, v [Tk, H_kv, d] in bf16: sequence b has
    queries cu_q[b] .. cu_q[b + 1] and keys cu_k[b] .. cu_k[b + 1] (cu_k defaults to cu_q), its queries
    being its last tokens -> (out [Tq, H_q, d], lse [Tq, H_q] or None).  scale defaults to 1 / sqrt(d).
    Rows of q, k and v may be strided (views of a fused projection); rows of given out and lse outside
    the sequences are left as they are."""
    ldq, ldk, ldv = _packed_rows(q, "q"), _packed_rows(k, "k"), _packed_rows(v, "v")
    Tq, H_q, d = q.shape
    Tk, H_kv, dk = k.shape
    if k.shape != v.shape or dk != d:
        raise ValueError(f"k and v must be [Tk, H_kv, {d}], got {tuple(k.shape)} and {tuple(v.shape)}")
    cu_k = cu_q if cu_k is None else cu_k
    S = _packed(cu_q, None, "cu_q")
    if cu_k.shape != cu_q.shape:
        raise ValueError(f"cu_k must be {list(cu_q.shape)}, got {tuple(cu_k.shape)}")
    if out is not None and tuple(out.shape) != (Tq, H_q, d):
        raise ValueError(f"out must be {[Tq, H_q, d]}, got {tuple(out.shape)}")
    if lse is not None and tuple(lse.shape) != (Tq, H_q):
        raise ValueError(f"lse must be {[Tq, H_q]}, got {tuple(lse.shape)}")
    cur, bf = _current(q, "q"), torch.bfloat16
    qp, kp, vp = _rows_ready(q, "q", bf, cur), _rows_ready(k, "k", bf, cur), _rows_ready(v, "v", bf, cur)
    cq, ck = _ready(cu_q, "cu_q", torch.int32, cur), _ready(cu_k, "cu_k", torch.int32, cur)
    if out is None:
        out = _new((Tq, H_q, d), bf, q.device, stream)
    if lse is None and want_lse:
        lse = _new((Tq, H_q), torch.float32, q.device, stream)
    h = _handle(stream, cur)
    nbytes = _ws_bytes(OP_PROMPT_ATTENTION, Tq, Tk, H_q, S, d, 0, 0)
    buf = _scratch(ws, q, cur, nbytes, stream, h)
    _check("misa_prompt_attention", _lib.misa_prompt_attention(
        qp, kp, vp, ldq, ldk, ldv, cq, ck, S, Tq, Tk, H_q, H_kv, d, BF16, d ** -0.5 if scale is None else scale,
        _ready(out, "out", bf, cur), _ready(lse, "lse", torch.float32, cur),
        _address(buf), nbytes, h))
    if stream is not None:
        _beside(stream, cur, h, q, k, v, cu_q, cu_k, out, lse)
    return out, lse
