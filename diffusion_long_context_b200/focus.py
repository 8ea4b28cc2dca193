"""Thin ctypes binding of libfocus.so (argument marshalling only).

Every function here has the name of the C entry point it calls and takes torch tensors
that already live on the GPU; it checks dtype / shape / contiguity, passes raw device
pointers and the current (or given) CUDA stream, and raises FocusError on a non-zero
status. All arithmetic happens in the library's kernels. Importing this module loads
the library and raises ImportError when it has not been built.
"""
from __future__ import annotations

import ctypes
import math
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfocus.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "focus.h")


class FocusError(RuntimeError):
    pass


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m diffusion_long_context_b200.build`")

lib = ctypes.CDLL(LIB_PATH)

_i, _f, _p, _sz, _u64 = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint64
_SIGS = {
    "focus_status_string": (ctypes.c_char_p, [_i]),
    "focus_last_error": (ctypes.c_char_p, []),
    "focus_launch_count": (_u64, []),
    "focus_device_error": (_i, [ctypes.POINTER(ctypes.c_int)]),
    "focus_select_queries": (_i, [_p, _p, _i, _i, _i, _i, _i, _f, _i, _p, _p, _i, _p, _p, _i, _p]),
    "focus_gather_rows": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _i, _p, _p]),
    "focus_scatter_rows": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _i, _p, _p]),
    "focus_block_means": (_i, [_p, _i, _i, _i, _i, _i, _i, _p, _p]),
    "focus_block_select": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _i, _i, _p, _p, _p]),
    "focus_dense_attention": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _f, _p, _p, _p, _sz, _p]),
    "focus_dense_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "focus_dense_attention_sinks": (_i, [_p, _p, _p, _p, _i, _i, _i, _i, _i, _i, _f, _p, _p, _i, _p, _p, _sz, _p]),
    "focus_full_refresh": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _f, _p, _i, _i, _p, _p, _sz, _p]),
    "focus_sink_identify": (_i, [_p, _i, _i, _i, _i, _p, _p]),
    "focus_sparse_attention": (_i, [_p, _p, _p, _p, _p, _i, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i, _f,
                                    _p, _p, _sz, _p]),
    "focus_sparse_workspace_bytes": (_sz, [_i] * 12),
    "focus_sparse_attention_noalloc": (_i, [_p, _p, _p, _p, _p, _i, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                                            _i, _f, _p, _p]),
    "focus_sparse_attention_fused": (_i, [_p, _p, _p, _p, _p, _i, _i, _p, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                                          _i, _f, _p, _p, _p, _sz, _p]),
    "focus_cache_store": (_i, [_p, _p, _i, _i, _p, _p, _i, _p, _p]),
    "focus_cache_scatter_rows": (_i, [_p, _p, _p, _p, _i, _i, _p, _p, _i, _p, _p]),
    "focus_cache_load": (_i, [_p, _p, _i, _p, _i, _i, _i, _p, _p, _p]),
    "focus_cache_attention": (_i, [_p, _p, _p, _p, _i, _p, _i, _i, _i, _f, _p, _p, _sz, _p]),
    "focus_cache_sparse_attention": (_i, [_p, _p, _p, _p, _i, _p, _p, _i, _p, _i, _p, _i, _i, _i, _i, _f, _p, _p, _sz,
                                          _p]),
    "focus_cache_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "focus_pages_reserve": (_i, [_p, _p, _p, _i, _p, _p]),
    "focus_pages_fork": (_i, [_p, _p, _p, _p, _i, _p]),
    "focus_pages_own": (_i, [_p, _p, _p, _p, _i, _p, _i, _p, _p, _p]),
    "focus_pages_release": (_i, [_p, _p, _p, _i, _p]),
    "focus_pages_compact": (_i, [_p, _p, _i, _p, _p, _p]),
    "focus_pages_copy": (_i, [_p, _p, _p, _i, _p]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def header_symbols():
    """Names of the entry points declared in include/focus.h."""
    with open(HEADER_PATH) as f:
        return re.findall(r"FOCUS_API\s+[\w\s\*]+?\b(focus_\w+)\s*\(", f.read())


def launch_count() -> int:
    return int(lib.focus_launch_count())


def last_error() -> str:
    return lib.focus_last_error().decode()


def device_error() -> int:
    """Synchronises, returns and clears the device error word (0 = none)."""
    code = ctypes.c_int(0)
    st = lib.focus_device_error(ctypes.byref(code))
    if st not in (0, -5):
        raise FocusError(f"focus_device_error: {last_error()}")
    return code.value


def _check(status: int, name: str):
    if status != 0:
        raise FocusError(f"{name}: {lib.focus_status_string(status).decode()}: {last_error()}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream, device=None):
    if stream is None:                   # (torch.cuda.current_stream() builds an object: 3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device is None else device)
    return stream.cuda_stream


def _need(t, dtype, name, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")


# ----------------------------------------------------------------------------- calls
def focus_select_queries(conf_prev, mask, g0, g1, n_t, rho, w, i_focus, n_focus, i_active, n_active, stream=None):
    _need(conf_prev, torch.float32, "conf_prev", 2)
    _need(mask, torch.uint8, "mask", 2)
    for t, n in ((i_focus, "i_focus"), (n_focus, "n_focus"), (i_active, "i_active"), (n_active, "n_active")):
        _need(t, torch.int32, n)
    B, L = mask.shape
    st = lib.focus_select_queries(_ptr(conf_prev), _ptr(mask), B, L, g0, g1, n_t, float(rho), w, _ptr(i_focus),
                                  _ptr(n_focus), i_focus.shape[-1], _ptr(i_active), _ptr(n_active),
                                  i_active.shape[-1], _stream(stream))
    _check(st, "focus_select_queries")


def focus_gather_rows(X, rows, n_rows, X_rows, stream=None):
    """X [n_mat, B, H, L, d] (or [B, H, L, d]) -> X_rows [..., cap, d]."""
    _need(X, torch.bfloat16, "X")
    _need(X_rows, torch.bfloat16, "X_rows")
    _need(rows, torch.int32, "rows", 2)
    _need(n_rows, torch.int32, "n_rows", 1)
    x = X if X.dim() == 5 else X.unsqueeze(0)
    n_mat, B, H, L, d = x.shape
    cap = rows.shape[1]
    st = lib.focus_gather_rows(_ptr(X), _ptr(rows), _ptr(n_rows), n_mat, B, H, L, d, cap, _ptr(X_rows),
                               _stream(stream))
    _check(st, "focus_gather_rows")


def focus_scatter_rows(X, rows, n_rows, X_rows, stream=None):
    """Approximate-KV-cache refresh: X[..., rows[b, i], :] = X_rows[..., i, :] for i < n_rows[b].

    X [n_mat, B, H, L, d] (or [B, H, L, d]) is updated in place from X_rows [..., cap, d]."""
    _need(X, torch.bfloat16, "X")
    _need(X_rows, torch.bfloat16, "X_rows")
    _need(rows, torch.int32, "rows", 2)
    _need(n_rows, torch.int32, "n_rows", 1)
    x = X if X.dim() == 5 else X.unsqueeze(0)
    n_mat, B, H, L, d = x.shape
    cap = rows.shape[1]
    st = lib.focus_scatter_rows(_ptr(X), _ptr(rows), _ptr(n_rows), n_mat, B, H, L, d, cap, _ptr(X_rows),
                                _stream(stream))
    _check(st, "focus_scatter_rows")


def focus_block_means(K, P, bs, kbar, stream=None):
    _need(K, torch.bfloat16, "K", 4)
    _need(kbar, torch.float32, "kbar", 4)
    B, Hkv, L, d = K.shape
    st = lib.focus_block_means(_ptr(K), B, Hkv, L, d, P, bs, _ptr(kbar), _stream(stream))
    _check(st, "focus_block_means")


def focus_block_select(Q_active, n_active, kbar, C, blocks, scores=None, stream=None):
    _need(Q_active, torch.bfloat16, "Q_active", 4)
    _need(n_active, torch.int32, "n_active", 1)
    _need(kbar, torch.float32, "kbar", 4)
    _need(blocks, torch.int32, "blocks", 3)
    if scores is not None:
        _need(scores, torch.float32, "scores", 3)
    B, Hq, acap, d = Q_active.shape
    Hkv, nb = kbar.shape[1], kbar.shape[2]
    st = lib.focus_block_select(_ptr(Q_active), _ptr(n_active), _ptr(kbar), B, Hq, Hkv, d, acap, nb, C,
                                _ptr(blocks), _ptr(scores), _stream(stream))
    _check(st, "focus_block_select")


def dense_workspace_bytes(B, Hq, Hkv, L, d, qcap, want_colsum):
    return int(lib.focus_dense_workspace_bytes(B, Hq, Hkv, L, d, qcap, 1 if want_colsum else 0))


def sparse_workspace_bytes(B, Hq, Hkv, L, d, acap, S, C, bs, P, g0, g1):
    return int(lib.focus_sparse_workspace_bytes(B, Hq, Hkv, L, d, acap, S, C, bs, P, g0, g1))


def _workspace(nbytes, device, ws, stream=None):
    """The caller's workspace, or one that lives as long as the call's binding. That one is taken from
    the memory of the stream that the kernels run on: only there is what comes after ordered behind them."""
    if nbytes == 0:
        return None, 0
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError(f"workspace needs {nbytes} bytes")
        return ws, ws.numel() * ws.element_size()
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def focus_dense_attention(Q, n_q, K, V, O, scale=None, colsum=None, ws=None, stream=None):
    _need(Q, torch.bfloat16, "Q", 4)
    _need(K, torch.bfloat16, "K", 4)
    _need(V, torch.bfloat16, "V", 4)
    _need(O, torch.bfloat16, "O", 4)
    if n_q is not None:
        _need(n_q, torch.int32, "n_q", 1)
    if colsum is not None:
        _need(colsum, torch.float32, "colsum", 3)
    B, Hq, qcap, d = Q.shape
    Hkv, L = K.shape[1], K.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    need = dense_workspace_bytes(B, Hq, Hkv, L, d, qcap, colsum is not None)
    ws, ws_bytes = _workspace(need, Q.device, ws, stream)
    st = lib.focus_dense_attention(_ptr(Q), _ptr(n_q), _ptr(K), _ptr(V), B, Hq, Hkv, L, d, qcap, float(scale),
                                   _ptr(O), _ptr(colsum), _ptr(ws), ws_bytes, _stream(stream))
    _check(st, "focus_dense_attention")


def focus_dense_attention_sinks(Q, n_q, K, V, O, colsum, sinks, scale=None, ws=None, stream=None):
    """The sink layer: dense attention, column sums and the top-S sinks (S = sinks.shape[2])."""
    _need(Q, torch.bfloat16, "Q", 4)
    _need(K, torch.bfloat16, "K", 4)
    _need(V, torch.bfloat16, "V", 4)
    _need(O, torch.bfloat16, "O", 4)
    _need(colsum, torch.float32, "colsum", 3)
    _need(sinks, torch.int32, "sinks", 3)
    if n_q is not None:
        _need(n_q, torch.int32, "n_q", 1)
    B, Hq, qcap, d = Q.shape
    Hkv, L = K.shape[1], K.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    need = dense_workspace_bytes(B, Hq, Hkv, L, d, qcap, True)
    ws, ws_bytes = _workspace(need, Q.device, ws, stream)
    st = lib.focus_dense_attention_sinks(_ptr(Q), _ptr(n_q), _ptr(K), _ptr(V), B, Hq, Hkv, L, d, qcap, float(scale),
                                         _ptr(O), _ptr(colsum), sinks.shape[2], _ptr(sinks), _ptr(ws), ws_bytes,
                                         _stream(stream))
    _check(st, "focus_dense_attention_sinks")


def focus_full_refresh(Q, K, V, O, P, bs, kbar, scale=None, ws=None, stream=None):
    """Block entry: dense attention of every query (O [B, Hq, L, d]) and the prompt's block
    means kbar [B, Hkv, ceil(P / bs), d] fp32, in one launch where the kernel serves it."""
    _need(Q, torch.bfloat16, "Q", 4)
    _need(K, torch.bfloat16, "K", 4)
    _need(V, torch.bfloat16, "V", 4)
    _need(O, torch.bfloat16, "O", 4)
    _need(kbar, torch.float32, "kbar", 4)
    B, Hq, L, d = Q.shape
    Hkv = K.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    need = dense_workspace_bytes(B, Hq, Hkv, L, d, L, False)
    ws, ws_bytes = _workspace(need, Q.device, ws, stream)
    st = lib.focus_full_refresh(_ptr(Q), _ptr(K), _ptr(V), B, Hq, Hkv, L, d, float(scale), _ptr(O), P, bs, _ptr(kbar),
                                _ptr(ws), ws_bytes, _stream(stream))
    _check(st, "focus_full_refresh")


def focus_sink_identify(colsum, S, sinks, stream=None):
    _need(colsum, torch.float32, "colsum", 3)
    _need(sinks, torch.int32, "sinks", 3)
    B, Hkv, L = colsum.shape
    st = lib.focus_sink_identify(_ptr(colsum), B, Hkv, L, S, _ptr(sinks), _stream(stream))
    _check(st, "focus_sink_identify")


def focus_sparse_attention(Q_active, n_active, K, V, sinks, blocks, bs, P, g0, g1, O_active, scale=None, ws=None,
                           stream=None):
    _need(Q_active, torch.bfloat16, "Q_active", 4)
    _need(n_active, torch.int32, "n_active", 1)
    _need(K, torch.bfloat16, "K", 4)
    _need(V, torch.bfloat16, "V", 4)
    _need(O_active, torch.bfloat16, "O_active", 4)
    _need(blocks, torch.int32, "blocks", 3)
    if sinks is not None:
        _need(sinks, torch.int32, "sinks", 3)
    B, Hq, acap, d = Q_active.shape
    Hkv, L = K.shape[1], K.shape[2]
    S = 0 if sinks is None else sinks.shape[2]
    C = blocks.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    need = sparse_workspace_bytes(B, Hq, Hkv, L, d, acap, S, C, bs, P, g0, g1)
    ws, ws_bytes = _workspace(need, Q_active.device, ws, stream)
    st = lib.focus_sparse_attention(_ptr(Q_active), _ptr(n_active), _ptr(K), _ptr(V), _ptr(sinks), S,
                                    _ptr(blocks), C, bs, P, g0, g1, B, Hq, Hkv, L, d, acap, float(scale),
                                    _ptr(O_active), _ptr(ws), ws_bytes, _stream(stream))
    _check(st, "focus_sparse_attention")


def focus_sparse_attention_fused(Q_active, n_active, K, V, kbar, C, sinks, bs, P, g0, g1, blocks, O_active, scale=None,
                                 ws=None, stream=None):
    """Block relevance + top-C + sparse attention of one layer (blocks receives the kept blocks)."""
    _need(Q_active, torch.bfloat16, "Q_active", 4)
    _need(n_active, torch.int32, "n_active", 1)
    _need(K, torch.bfloat16, "K", 4)
    _need(V, torch.bfloat16, "V", 4)
    _need(kbar, torch.float32, "kbar", 4)
    _need(blocks, torch.int32, "blocks", 3)
    _need(O_active, torch.bfloat16, "O_active", 4)
    if sinks is not None:
        _need(sinks, torch.int32, "sinks", 3)
    B, Hq, acap, d = Q_active.shape
    Hkv, L = K.shape[1], K.shape[2]
    nb = kbar.shape[2]
    S = 0 if sinks is None else sinks.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    need = sparse_workspace_bytes(B, Hq, Hkv, L, d, acap, S, C, bs, P, g0, g1)
    ws, ws_bytes = _workspace(need, Q_active.device, ws, stream)
    st = lib.focus_sparse_attention_fused(_ptr(Q_active), _ptr(n_active), _ptr(K), _ptr(V), _ptr(kbar), nb, C,
                                          _ptr(sinks), S, bs, P, g0, g1, B, Hq, Hkv, L, d, acap, float(scale),
                                          _ptr(blocks), _ptr(O_active), _ptr(ws), ws_bytes, _stream(stream))
    _check(st, "focus_sparse_attention_fused")


# ----------------------------------------------------------------------------- 8-bit paged cache
class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p), ("n_mat", _i), ("n_pages", _i), ("Hkv", _i),
                ("page", _i), ("d", _i), ("format", _i)]


class _PagesStruct(ctypes.Structure):
    _fields_ = [("refs", _p), ("table", _p), ("held", _p), ("n_pages", _i), ("n_seq", _i), ("table_cols", _i)]


CACHE_FORMATS = {torch.float8_e4m3fn: 0, torch.int8: 1}


def _here(name, *tensors):
    """The tensors of a call lie on the current device (whose stream and error word it uses); its index."""
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != cur:
            raise ValueError(f"{name}: tensor on {t.device}, the current device is cuda:{cur}")
    return cur


class Cache:
    """The tensors of an 8-bit paged key/value cache: codes k, v [n_mat, n_pages, Hkv, page, d]
    (torch.float8_e4m3fn or torch.int8) and scales k_scale, v_scale [n_mat, n_pages, Hkv] fp32.

    Holds the tensors, so their memory stays while the handle lives; layer(m) is the handle of
    one layer, which the attention calls take."""

    def __init__(self, k, v, k_scale, v_scale):
        if not isinstance(k, torch.Tensor) or k.dtype not in CACHE_FORMATS:
            raise TypeError("cache codes must be torch.float8_e4m3fn or torch.int8 tensors")
        _need(k, k.dtype, "k", 5)
        _need(v, k.dtype, "v", 5)
        _need(k_scale, torch.float32, "k_scale", 3)
        _need(v_scale, torch.float32, "v_scale", 3)
        if v.shape != k.shape or k_scale.shape != k.shape[:3] or v_scale.shape != k.shape[:3]:
            raise ValueError(f"cache shapes differ: k {tuple(k.shape)}, v {tuple(v.shape)}, k_scale "
                             f"{tuple(k_scale.shape)}, v_scale {tuple(v_scale.shape)}")
        if not (k.device == v.device == k_scale.device == v_scale.device):
            raise ValueError("cache tensors lie on different devices")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_mat, self.n_pages, self.Hkv, self.page, self.d = k.shape
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), *k.shape,
                                    CACHE_FORMATS[k.dtype])
        self._ref = ctypes.byref(self._struct)

    def layer(self, m):
        return Cache(self.k[m:m + 1], self.v[m:m + 1], self.k_scale[m:m + 1], self.v_scale[m:m + 1])


class Pages:
    """The page accounting of a cache: refs [n_pages], table [n_seq, cols], held [n_seq] (int32)."""

    def __init__(self, refs, table, held):
        _need(refs, torch.int32, "refs", 1)
        _need(table, torch.int32, "table", 2)
        _need(held, torch.int32, "held", 1)
        if held.shape[0] != table.shape[0]:
            raise ValueError(f"held has {held.shape[0]} sequences, table {table.shape[0]}")
        if not (refs.device == table.device == held.device):
            raise ValueError("page tensors lie on different devices")
        self.refs, self.table, self.held = refs, table, held
        self.n_pages, (self.n_seq, self.table_cols) = refs.shape[0], table.shape
        self._struct = _PagesStruct(refs.data_ptr(), table.data_ptr(), held.data_ptr(), refs.shape[0], *table.shape)
        self._ref = ctypes.byref(self._struct)


def _shape(t, want, name):
    if t.shape != want:
        raise ValueError(f"{name} must be {tuple(want)}, got {tuple(t.shape)}")


def _cache_rows(X, Y, names, cache):
    """bf16 rows [n_mat, B, Hkv, n, d] (or without n_mat for one layer) that fit the cache -> (B, n)."""
    _need(X, torch.bfloat16, names[0])
    _need(Y, torch.bfloat16, names[1])
    n_mat, B, Hkv, n, d = X.shape if X.dim() == 5 else (1, *X.shape) if X.dim() == 4 else (0, 0, 0, 0, 0)
    if n_mat != cache.n_mat or Hkv != cache.Hkv or d != cache.d:
        raise ValueError(f"{names[0]} {tuple(X.shape)} does not fit a cache of {cache.n_mat} layers, {cache.Hkv} heads, "
                         f"d = {cache.d}")
    _shape(Y, X.shape, names[1])
    return B, n


def _table(table, B):
    _need(table, torch.int32, "table", 2)
    if table.shape[0] != B:
        raise ValueError(f"table must name the pages of {B} sequences, got {tuple(table.shape)}")
    return table.shape[1]


def _i32_list(t, n, name):
    _need(t, torch.int32, name, 1)
    if t.shape[0] != n:
        raise ValueError(f"{name} must be ({n},), got {tuple(t.shape)}")


def focus_cache_store(K, V, cache, table, lens=None, stream=None):
    """Positions [0, lens[b]) (all L without lens) of K, V [n_mat, B, Hkv, L, d] into the cache."""
    B, L = _cache_rows(K, V, ("K", "V"), cache)
    cols = _table(table, B)
    if lens is not None:
        _i32_list(lens, B, "lens")
    cur = _here("focus_cache_store", K, V, cache.k, table, lens)
    st = lib.focus_cache_store(_ptr(K), _ptr(V), B, L, _ptr(lens), _ptr(table), cols, cache._ref, _stream(stream, cur))
    _check(st, "focus_cache_store")


def focus_cache_scatter_rows(K_rows, V_rows, rows, n_rows, cache, table, lens, stream=None):
    """Position rows[b, i] takes K_rows[..., b, :, i], V_rows[..., b, :, i] for i < n_rows[b]
    (K_rows, V_rows [n_mat, B, Hkv, cap, d]); lens [B] = positions held before the call."""
    B, cap = _cache_rows(K_rows, V_rows, ("K_rows", "V_rows"), cache)
    _need(rows, torch.int32, "rows", 2)
    _shape(rows, (B, cap), "rows")
    _i32_list(n_rows, B, "n_rows")
    _i32_list(lens, B, "lens")
    cols = _table(table, B)
    cur = _here("focus_cache_scatter_rows", K_rows, V_rows, rows, n_rows, cache.k, table, lens)
    st = lib.focus_cache_scatter_rows(_ptr(K_rows), _ptr(V_rows), _ptr(rows), _ptr(n_rows), B, cap, _ptr(lens),
                                      _ptr(table), cols, cache._ref, _stream(stream, cur))
    _check(st, "focus_cache_scatter_rows")


def focus_cache_load(cache, table, lens, start, K, V, stream=None):
    """K, V [n_mat, B, Hkv, L, d] = the cached values of positions [start, min(start + L, lens[b]))."""
    B, L = _cache_rows(K, V, ("K", "V"), cache)
    _i32_list(lens, B, "lens")
    cols = _table(table, B)
    cur = _here("focus_cache_load", K, V, cache.k, table, lens)
    st = lib.focus_cache_load(cache._ref, _ptr(table), cols, _ptr(lens), B, start, L, _ptr(K), _ptr(V),
                              _stream(stream, cur))
    _check(st, "focus_cache_load")


def cache_workspace_bytes(B, Hq, Hkv, d, qcap):
    return int(lib.focus_cache_workspace_bytes(B, Hq, Hkv, d, qcap))


def _cache_queries(Q, n_q, cache, O, ws, stream):
    _need(Q, torch.bfloat16, "Q", 4)
    _need(O, torch.bfloat16, "O", 4)
    B, Hq, qcap, d = Q.shape
    if d != cache.d:
        raise ValueError(f"Q has d = {d}, the cache {cache.d}")
    _shape(O, Q.shape, "O")
    if n_q is not None:
        _i32_list(n_q, B, "n_q")
    ws, ws_bytes = _workspace(cache_workspace_bytes(B, Hq, cache.Hkv, d, qcap), Q.device, ws, stream)
    return B, Hq, qcap, d, ws, ws_bytes


def focus_cache_attention(Q, n_q, cache, table, lens, O, scale=None, ws=None, stream=None):
    """Dense attention of Q [B, Hq, qcap, d] over positions [0, lens[b]) of a one-layer cache."""
    B, Hq, qcap, d, ws, ws_bytes = _cache_queries(Q, n_q, cache, O, ws, stream)
    _i32_list(lens, B, "lens")
    cols = _table(table, B)
    cur = _here("focus_cache_attention", Q, n_q, cache.k, table, lens, O, ws)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    st = lib.focus_cache_attention(_ptr(Q), _ptr(n_q), cache._ref, _ptr(table), cols, _ptr(lens), B, Hq, qcap,
                                   float(scale), _ptr(O), _ptr(ws), ws_bytes, _stream(stream, cur))
    _check(st, "focus_cache_attention")


def focus_cache_sparse_attention(Q_active, n_active, cache, table, P, g0, G, sinks, blocks, O_active, scale=None,
                                 ws=None, stream=None):
    """Sparse attention from a one-layer cache over sinks U kept blocks (of a page each) U [g0, g0 + G);
    P, g0 [B] int32, sinks [B, Hkv, S] or None, blocks [B, Hkv, C]."""
    B, Hq, qcap, d, ws, ws_bytes = _cache_queries(Q_active, n_active, cache, O_active, ws, stream)
    _i32_list(P, B, "P")
    _i32_list(g0, B, "g0")
    _need(blocks, torch.int32, "blocks", 3)
    C = blocks.shape[2]
    _shape(blocks, (B, cache.Hkv, C), "blocks")
    S = 0
    if sinks is not None:
        _need(sinks, torch.int32, "sinks", 3)
        S = sinks.shape[2]
        _shape(sinks, (B, cache.Hkv, S), "sinks")
    cols = _table(table, B)
    cur = _here("focus_cache_sparse_attention", Q_active, n_active, cache.k, table, P, g0, sinks, blocks, O_active, ws)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    st = lib.focus_cache_sparse_attention(_ptr(Q_active), _ptr(n_active), cache._ref, _ptr(table), cols, _ptr(P),
                                          _ptr(g0), G, _ptr(sinks), S, _ptr(blocks), C, B, Hq, qcap, float(scale),
                                          _ptr(O_active), _ptr(ws), ws_bytes, _stream(stream, cur))
    _check(st, "focus_cache_sparse_attention")


def focus_pages_reserve(pages, seqs, want, status, stream=None):
    """Sequences seqs[i] grow to want[i] pages; status [1] = pages missing (then nothing changed)."""
    _need(seqs, torch.int32, "seqs", 1)
    n = seqs.shape[0]
    _i32_list(want, n, "want")
    _i32_list(status, 1, "status")
    cur = _here("focus_pages_reserve", pages.refs, seqs, want, status)
    st = lib.focus_pages_reserve(pages._ref, _ptr(seqs), _ptr(want), n, _ptr(status), _stream(stream, cur))
    _check(st, "focus_pages_reserve")


def focus_pages_fork(pages, src, dst, keep, stream=None):
    """Empty sequences dst[i] share the first keep[i] pages of src[i]."""
    _need(src, torch.int32, "src", 1)
    n = src.shape[0]
    _i32_list(dst, n, "dst")
    _i32_list(keep, n, "keep")
    cur = _here("focus_pages_fork", pages.refs, src, dst, keep)
    st = lib.focus_pages_fork(pages._ref, _ptr(src), _ptr(dst), _ptr(keep), n, _stream(stream, cur))
    _check(st, "focus_pages_fork")


def _pairs(pairs, n_pairs):
    _need(pairs, torch.int32, "pairs", 2)
    _shape(pairs, (pairs.shape[0], 2), "pairs")
    _i32_list(n_pairs, 1, "n_pairs")
    return pairs.shape[0]


def focus_pages_own(pages, seqs, first, last, pairs, n_pairs, status, stream=None):
    """Pages first[i] <= j < last[i] of seqs[i] that others share are replaced by free ones; pairs
    [cap, 2], n_pairs [1] then name what focus_pages_copy has to copy."""
    _need(seqs, torch.int32, "seqs", 1)
    n = seqs.shape[0]
    _i32_list(first, n, "first")
    _i32_list(last, n, "last")
    _i32_list(status, 1, "status")
    cap = _pairs(pairs, n_pairs)
    cur = _here("focus_pages_own", pages.refs, seqs, first, last, pairs, n_pairs, status)
    st = lib.focus_pages_own(pages._ref, _ptr(seqs), _ptr(first), _ptr(last), n, _ptr(pairs), cap, _ptr(n_pairs),
                             _ptr(status), _stream(stream, cur))
    _check(st, "focus_pages_own")


def focus_pages_release(pages, seqs, keep, stream=None):
    """Sequences seqs[i] give up their pages behind the first keep[i]."""
    _need(seqs, torch.int32, "seqs", 1)
    n = seqs.shape[0]
    _i32_list(keep, n, "keep")
    cur = _here("focus_pages_release", pages.refs, seqs, keep)
    st = lib.focus_pages_release(pages._ref, _ptr(seqs), _ptr(keep), n, _stream(stream, cur))
    _check(st, "focus_pages_release")


def focus_pages_compact(pages, pairs, n_pairs, remap, stream=None):
    """Live pages move to the front of the pool; pairs, n_pairs name what focus_pages_copy has to
    copy, remap [n_pages] = each page's new index (-1: free)."""
    cap = _pairs(pairs, n_pairs)
    _i32_list(remap, pages.n_pages, "remap")
    cur = _here("focus_pages_compact", pages.refs, pairs, n_pairs, remap)
    st = lib.focus_pages_compact(pages._ref, _ptr(pairs), cap, _ptr(n_pairs), _ptr(remap), _stream(stream, cur))
    _check(st, "focus_pages_compact")


def focus_pages_copy(cache, pairs, n_pairs, stream=None):
    """Codes and scales of page pairs[r, 0] to page pairs[r, 1] in every layer, r < n_pairs[0]."""
    cap = _pairs(pairs, n_pairs)
    cur = _here("focus_pages_copy", cache.k, pairs, n_pairs)
    st = lib.focus_pages_copy(cache._ref, _ptr(pairs), _ptr(n_pairs), cap, _stream(stream, cur))
    _check(st, "focus_pages_copy")
