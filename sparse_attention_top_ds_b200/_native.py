"""ctypes binding of libdstopk.so: argument marshalling only.

Every step of the selection runs in the library's CUDA kernels.  If the shared
library is missing or cannot be loaded, every call raises; there is no
fallback implementation.
"""

import ctypes
import math
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
# DS_TOPK_LIB may name another build, such as libdstopk_debug.so (device range checks)
_LIB_PATH = os.environ.get("DS_TOPK_LIB", os.path.join(_PKG, "libdstopk.so"))
DEBUG_LIB_PATH = os.path.join(_PKG, "libdstopk_debug.so")

DS_F32 = 0
DS_BF16 = 1
DS_E4M3 = 2
DS_I8 = 3

DS_OK = 0
DS_ERR_ARG = -1
DS_ERR_CUDA = -2
DS_ERR_TIMEOUT = -3
DS_ERR_UNSUPPORTED = -4
DS_ERR_NOMEM = -5
DS_ERR_RANGE = -6

DS_MAX_K = 2048
DS_INDEXER_DIM = 128
DS_INDEXER_MAX_HEADS = 64
DS_ATTN_MAX_DIM = 512
DS_ATTN_MAX_WINDOW = 4096
DS_ATTN_MAX_HEADS = 4096
DS_CACHE_MAX_BLOCK = 128
DS_CACHE_MAX_ARRAYS = 8

_lib = None


# ds_cache_array of the header: src, dst, their batch strides, item_bytes, per_block
_CACHE_ARRAY = "QQqqqi4x"


class DsError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {strerror(code) if _lib is not None else code}")


def lib_path():
    return _LIB_PATH


def load():
    """Load the shared library once; raise if it is not there."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"libdstopk.so not found at {_LIB_PATH}; build it with "
            "`python -m sparse_attention_top_ds_b200.build` (there is no CPU fallback)")
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i32, i32p = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
    lib.ds_topk.argtypes = [vp, i32, i32, i32, i32, i32p, vp, vp, i32, i32, vp]
    lib.ds_topk.restype = i32
    lib.ds_indexer_score.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32p, vp, vp]
    lib.ds_indexer_score.restype = i32
    lib.ds_indexer_topk.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32p, i32, vp, vp, vp]
    lib.ds_indexer_topk.restype = i32
    lib.ds_indexer_topk_noalloc.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32p, i32, vp, vp, vp]
    lib.ds_indexer_topk_noalloc.restype = i32
    lib.ds_sparse_attention.argtypes = [vp, vp, ctypes.c_int64, i32, i32p, i32, vp, i32, i32p, vp,
                                        i32, i32, i32, ctypes.c_float, vp, vp, vp]
    lib.ds_sparse_attention.restype = i32
    lib.ds_indexer_topk_ex.argtypes = [vp, vp, ctypes.c_int64, vp, i32, i32, i32, i32, i32p, i32, i32, vp, vp, vp]
    lib.ds_indexer_topk_ex.restype = i32
    lib.ds_compress_fold.argtypes = [vp, i32, i32, ctypes.c_int64, vp, vp, ctypes.c_int64, vp]
    lib.ds_compress_fold.restype = i32
    lib.ds_indexer_qproj.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp]
    lib.ds_indexer_qproj.restype = i32
    lib.ds_get_device_status.argtypes = [vp]
    lib.ds_get_device_status.restype = i32
    lib.ds_strerror.argtypes = [i32]
    lib.ds_strerror.restype = ctypes.c_char_p
    lib.ds_release.argtypes = []
    lib.ds_release.restype = None
    lib.ds_set_wait_limit.argtypes = [ctypes.c_int64]
    lib.ds_set_wait_limit.restype = i32
    lib.ds_plant_wait_fault.argtypes = [i32]
    lib.ds_plant_wait_fault.restype = i32
    lib.ds_debug_build.argtypes = []
    lib.ds_debug_build.restype = i32
    lib.ds_debug_stash_stamps.argtypes = [vp, i32]
    lib.ds_debug_stash_stamps.restype = i32
    lib.ds_read_floor.argtypes = [vp, ctypes.c_int64, i32, vp]
    lib.ds_read_floor.restype = i32
    i64, f32 = ctypes.c_int64, ctypes.c_float
    lib.ds_cache_quantize.argtypes = [vp, i64, i64, i32, i32, i32, i32, i32, i32, i32p, i32p, vp, i64, vp, i64, i32, vp]
    lib.ds_cache_quantize.restype = i32
    lib.ds_sparse_attention_q8.argtypes = [vp, vp, i64, vp, i64, i32, i32, i32, i32p, i32, vp, i32, i32p, vp,
                                           i32, i32, i32, i32, f32, vp, vp, vp]
    lib.ds_sparse_attention_q8.restype = i32
    lib.ds_attention_mass.argtypes = [vp, vp, i64, vp, i64, i32, i32, i32, i32p, i32, vp, i32, i32, i32, i32, f32,
                                      vp, i64, vp]
    lib.ds_attention_mass.restype = i32
    lib.ds_cache_evict.argtypes = [vp, i64, i32, i32, i32p, i32, i32, i32, i32, i32p, i32p, vp]
    lib.ds_cache_evict.restype = i32
    lib.ds_cache_compact.argtypes = [vp, i32, i32p, i32, i32p, i32, i32, i32, vp]
    lib.ds_cache_compact.restype = i32
    _lib = lib
    return lib


def strerror(code):
    return load().ds_strerror(int(code)).decode()


def _check(code, where):
    if code != DS_OK:
        raise DsError(code, where)


# ------------------------------------------------------------------ raw pointer calls (C ABI)

def ds_topk_raw(scores, batch, n, k, dtype, valid_len, out_idx, out_val, return_value, sorted_index, stream):
    return load().ds_topk(scores, batch, n, k, dtype, valid_len, out_idx, out_val,
                          int(return_value), int(sorted_index), stream)


def ds_indexer_score_raw(q, kcache, w, batch, heads, d, S, valid_len, out_score, stream):
    return load().ds_indexer_score(q, kcache, w, batch, heads, d, S, valid_len, out_score, stream)


def ds_indexer_topk_raw(q, kcache, w, batch, heads, d, S, valid_len, k, out_idx, out_score, stream):
    return load().ds_indexer_topk(q, kcache, w, batch, heads, d, S, valid_len, k, out_idx, out_score, stream)


def ds_indexer_topk_noalloc_raw(q, kcache, w, batch, heads, d, S, valid_len, k, out_idx, out_score, stream):
    """The allocation-free variant (score rows in the library's fixed array)."""
    return load().ds_indexer_topk_noalloc(q, kcache, w, batch, heads, d, S, valid_len, k, out_idx, out_score,
                                          stream)


def ds_sparse_attention_raw(q, kv, kv_batch_stride, T, idx, k, win, W, win_len, sink, batch, heads, d, scale,
                            out, lse, stream):
    return load().ds_sparse_attention(q, kv, int(kv_batch_stride), T, idx, k, win, W, win_len, sink,
                                      batch, heads, d, float(scale), out, lse, stream)


def ds_indexer_qproj_raw(x, wq, ww, T, d_in, heads, d, q_out, w_out, stream):
    return load().ds_indexer_qproj(x, wq, ww, T, d_in, heads, d, q_out, w_out, stream)


def ds_get_device_status(stream=None):
    return load().ds_get_device_status(_stream_ptr(stream))


def ds_release():
    load().ds_release()


def ds_set_wait_limit(ns):
    """Limit of the kernels' bounded waits in ns (0: the default of one second)."""
    _check(load().ds_set_wait_limit(int(ns)), "ds_set_wait_limit")


def ds_plant_wait_fault(launches):
    """Testing the failure detection: the next `launches` launches of the scorer,
    the 8-bit cache's attention and account and the copy kernel of ds_cache_compact
    each make one of their bounded waits run out (DS_ERR_TIMEOUT in the status)."""
    _check(load().ds_plant_wait_fault(int(launches)), "ds_plant_wait_fault")


def ds_debug_build():
    """True for the DS_DEBUG build (device range checks -> DS_ERR_RANGE)."""
    return bool(load().ds_debug_build())


def ds_debug_stash_stamps(ctas):
    """DS_DEBUG build: the stash top-k kernel's phase stamps (ns), [ctas, 10] uint64."""
    import numpy as np
    out = np.zeros((ctas, 10), dtype=np.uint64)
    _check(load().ds_debug_stash_stamps(ctypes.c_void_p(out.ctypes.data), int(ctas)), "ds_debug_stash_stamps")
    return out


def ds_read_floor(x, ctas, stream=None):
    """Enqueue a read-only pass over the CUDA tensor x (its bytes split over ctas CTAs)."""
    _check(load().ds_read_floor(_ptr(x), x.numel() * x.element_size(), int(ctas), _stream_ptr(stream)),
           "ds_read_floor")


# ------------------------------------------------------------------ torch-tensor front end

def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _require(t, dtype, name, device=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def ds_topk(scores, k, valid_len=None, return_value=True, sorted_index=False,
            out_idx=None, out_val=None, stream=None):
    """Top-k of every row of a [batch, n] float32 / bfloat16 CUDA tensor.

    Returns (idx int32 [batch, k], val [batch, k] or None).  Without
    ``sorted_index`` the order of a row's selection is unspecified.
    """
    import torch
    if scores.dtype == torch.float32:
        dt = DS_F32
    elif scores.dtype == torch.bfloat16:
        dt = DS_BF16
    else:
        raise TypeError("scores must be float32 or bfloat16")
    _require(scores, None, "scores")
    if scores.dim() != 2:
        raise ValueError("scores must be [batch, n]")
    batch, n = scores.shape
    dev = scores.device
    if valid_len is not None:
        _require(valid_len, torch.int32, "valid_len", dev)
    if out_idx is None:
        out_idx = torch.empty((batch, k), dtype=torch.int32, device=dev)
    _require(out_idx, torch.int32, "out_idx", dev)
    if return_value and out_val is None:
        out_val = torch.empty((batch, k), dtype=scores.dtype, device=dev)
    with torch.cuda.device(dev):
        rc = ds_topk_raw(_ptr(scores), batch, n, k, dt, _ptr(valid_len), _ptr(out_idx),
                         _ptr(out_val) if return_value else None, return_value, sorted_index,
                         _stream_ptr(stream))
    _check(rc, "ds_topk")
    return out_idx, (out_val if return_value else None)


def _indexer_args(q, kcache, w, valid_len):
    import torch
    _require(q, torch.bfloat16, "q")
    dev = q.device
    _require(kcache, torch.bfloat16, "kcache", dev)
    _require(w, torch.float32, "w", dev)
    if q.dim() != 3 or kcache.dim() != 2 or w.dim() != 2:
        raise ValueError("q [batch,heads,d], kcache [S,d], w [batch,heads]")
    batch, heads, d = q.shape
    S = kcache.shape[0]
    if kcache.shape[1] != d or tuple(w.shape) != (batch, heads):
        raise ValueError("shape mismatch between q, kcache and w")
    if valid_len is not None:
        _require(valid_len, torch.int32, "valid_len", dev)
    return dev, batch, heads, d, S


def ds_indexer_score(q, kcache, w, valid_len=None, out=None, stream=None):
    """Indexer score rows [batch, S] float32 (-inf at positions >= valid_len)."""
    import torch
    dev, batch, heads, d, S = _indexer_args(q, kcache, w, valid_len)
    if out is None:
        out = torch.empty((batch, S), dtype=torch.float32, device=dev)
    _require(out, torch.float32, "out", dev)
    with torch.cuda.device(dev):
        rc = ds_indexer_score_raw(_ptr(q), _ptr(kcache), _ptr(w), batch, heads, d, S,
                                  _ptr(valid_len), _ptr(out), _stream_ptr(stream))
    _check(rc, "ds_indexer_score")
    return out


def ds_indexer_topk(q, kcache, w, k, valid_len=None, return_score=False,
                    out_idx=None, out_score=None, stream=None):
    """Top-k positions of every indexer score row: (idx int32 [batch,k], score f32 [batch,k] or None)."""
    import torch
    dev, batch, heads, d, S = _indexer_args(q, kcache, w, valid_len)
    if out_idx is None:
        out_idx = torch.empty((batch, k), dtype=torch.int32, device=dev)
    _require(out_idx, torch.int32, "out_idx", dev)
    if return_score and out_score is None:
        out_score = torch.empty((batch, k), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        rc = ds_indexer_topk_raw(_ptr(q), _ptr(kcache), _ptr(w), batch, heads, d, S,
                                 _ptr(valid_len), k, _ptr(out_idx),
                                 _ptr(out_score) if return_score else None, _stream_ptr(stream))
    _check(rc, "ds_indexer_topk")
    return out_idx, (out_score if return_score else None)


def ds_indexer_topk_noalloc(q, kcache, w, k, valid_len=None, return_score=False,
                            out_idx=None, out_score=None, stream=None):
    """ds_indexer_topk through the allocation-free entry point (batch * S <= 262144)."""
    import torch
    dev, batch, heads, d, S = _indexer_args(q, kcache, w, valid_len)
    if out_idx is None:
        out_idx = torch.empty((batch, k), dtype=torch.int32, device=dev)
    _require(out_idx, torch.int32, "out_idx", dev)
    if return_score and out_score is None:
        out_score = torch.empty((batch, k), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        rc = ds_indexer_topk_noalloc_raw(_ptr(q), _ptr(kcache), _ptr(w), batch, heads, d, S,
                                         _ptr(valid_len), k, _ptr(out_idx),
                                         _ptr(out_score) if return_score else None, _stream_ptr(stream))
    _check(rc, "ds_indexer_topk_noalloc")
    return out_idx, (out_score if return_score else None)


def ds_sparse_attention(q, kv, idx, scale=None, win=None, win_len=None, sink=None, return_lse=False,
                        out=None, lse=None, stream=None):
    """Multi-query attention of every query head over the selected cache rows
    plus a sliding window.

    q    bf16 [batch, heads, d];  kv  bf16 [T, d] (one cache for every batch
    row) or [batch, T, d];  idx  int32 [batch, k] or None (window only);
    win  bf16 [batch, W, d] or None;  win_len  int32 [batch] or None (= W);
    sink float32 [heads] or None;  scale  default 1/sqrt(d).
    Returns out bf16 [batch, heads, d], or (out, lse float32 [batch, heads]).
    """
    import math
    import torch
    _require(q, torch.bfloat16, "q")
    dev = q.device
    _require(kv, torch.bfloat16, "kv", dev)
    if q.dim() != 3:
        raise ValueError("q must be [batch, heads, d]")
    batch, heads, d = q.shape
    if kv.dim() == 2:
        T, stride = kv.shape[0], 0
    elif kv.dim() == 3 and kv.shape[0] == batch:
        T, stride = kv.shape[1], kv.shape[1]
    else:
        raise ValueError("kv must be [T, d] or [batch, T, d]")
    if kv.shape[-1] != d:
        raise ValueError("kv and q differ in d")
    k = 0
    if idx is not None:
        _require(idx, torch.int32, "idx", dev)
        if idx.dim() != 2 or idx.shape[0] != batch:
            raise ValueError("idx must be [batch, k]")
        k = idx.shape[1]
    W = 0
    if win is not None:
        _require(win, torch.bfloat16, "win", dev)
        if win.dim() != 3 or win.shape[0] != batch or win.shape[2] != d:
            raise ValueError("win must be [batch, W, d]")
        W = win.shape[1]
    if win_len is not None:
        _require(win_len, torch.int32, "win_len", dev)
    if sink is not None:
        _require(sink, torch.float32, "sink", dev)
        if sink.numel() != heads:
            raise ValueError("sink must hold one logit per head")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((batch, heads, d), dtype=torch.bfloat16, device=dev)
    _require(out, torch.bfloat16, "out", dev)
    if return_lse and lse is None:
        lse = torch.empty((batch, heads), dtype=torch.float32, device=dev)
    if lse is not None:
        _require(lse, torch.float32, "lse", dev)
    with torch.cuda.device(dev):
        rc = ds_sparse_attention_raw(_ptr(q), _ptr(kv), stride, T, _ptr(idx), k, _ptr(win), W, _ptr(win_len),
                                     _ptr(sink), batch, heads, d, scale, _ptr(out), _ptr(lse),
                                     _stream_ptr(stream))
    _check(rc, "ds_sparse_attention")
    return (out, lse) if return_lse else out


def ds_indexer_qproj(x, wq, ww=None, heads=None, q_out=None, w_out=None, stream=None):
    """Indexer queries and per-head weights from one input row per token.

    x bf16 [T, d_in];  wq bf16 [heads * 128, d_in];  ww bf16 [heads, d_in] or None.
    Returns (q bf16 [T, heads, 128], w float32 [T, heads] or None).
    """
    import torch
    _require(x, torch.bfloat16, "x")
    dev = x.device
    _require(wq, torch.bfloat16, "wq", dev)
    if x.dim() != 2 or wq.dim() != 2 or wq.shape[1] != x.shape[1] or wq.shape[0] % DS_INDEXER_DIM:
        raise ValueError("x [T, d_in], wq [heads * 128, d_in]")
    T, d_in = x.shape
    H = wq.shape[0] // DS_INDEXER_DIM if heads is None else int(heads)
    if ww is not None:
        _require(ww, torch.bfloat16, "ww", dev)
        if tuple(ww.shape) != (H, d_in):
            raise ValueError("ww must be [heads, d_in]")
    if q_out is None:
        q_out = torch.empty((T, H, DS_INDEXER_DIM), dtype=torch.bfloat16, device=dev)
    _require(q_out, torch.bfloat16, "q_out", dev)
    if ww is not None and w_out is None:
        w_out = torch.empty((T, H), dtype=torch.float32, device=dev)
    if w_out is not None:
        _require(w_out, torch.float32, "w_out", dev)
    with torch.cuda.device(dev):
        rc = ds_indexer_qproj_raw(_ptr(x), _ptr(wq), _ptr(ww), T, d_in, H, DS_INDEXER_DIM, _ptr(q_out),
                                  _ptr(w_out) if ww is not None else None, _stream_ptr(stream))
    _check(rc, "ds_indexer_qproj")
    return q_out, (w_out if ww is not None else None)


def ds_indexer_topk_ex(q, kcache, w, k, valid_len=None, sorted_index=False, return_score=False,
                       out_idx=None, out_score=None, stream=None):
    """ds_indexer_topk with kcache [S, d] (shared) or [batch, S, d] (one cache per
    row), and optional position-sorted output."""
    import torch
    _require(q, torch.bfloat16, "q")
    dev = q.device
    _require(kcache, torch.bfloat16, "kcache", dev)
    _require(w, torch.float32, "w", dev)
    batch, heads, d = q.shape
    if kcache.dim() == 2:
        S, stride = kcache.shape[0], 0
    elif kcache.dim() == 3 and kcache.shape[0] == batch:
        S, stride = kcache.shape[1], kcache.shape[1]
    else:
        raise ValueError("kcache must be [S, d] or [batch, S, d]")
    if kcache.shape[-1] != d or tuple(w.shape) != (batch, heads):
        raise ValueError("shape mismatch between q, kcache and w")
    if valid_len is not None:
        _require(valid_len, torch.int32, "valid_len", dev)
    if out_idx is None:
        out_idx = torch.empty((batch, k), dtype=torch.int32, device=dev)
    _require(out_idx, torch.int32, "out_idx", dev)
    if return_score and out_score is None:
        out_score = torch.empty((batch, k), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        rc = load().ds_indexer_topk_ex(_ptr(q), _ptr(kcache), int(stride), _ptr(w), batch, heads, d, S,
                                       _ptr(valid_len), k, int(bool(sorted_index)), _ptr(out_idx),
                                       _ptr(out_score) if return_score else None, _stream_ptr(stream))
    _check(rc, "ds_indexer_topk_ex")
    return out_idx, (out_score if return_score else None)


def ds_compress_fold(rows, gate, out=None, stream=None):
    """Fold each batch row's 4 rows into 1 (gated weighted sum).

    rows bf16 [batch, 4, D] (any batch stride, rows contiguous within a batch
    row); gate bf16 [D]; out bf16 [batch, D] or a strided [batch, D] view (for
    instance cache[:, j, :]).  Returns out.
    """
    import torch
    if not isinstance(rows, torch.Tensor) or rows.dtype != torch.bfloat16 or not rows.is_cuda:
        raise TypeError("rows must be a CUDA bfloat16 tensor")
    if rows.dim() != 3 or rows.shape[1] != 4 or rows.stride(2) != 1 or rows.stride(1) != rows.shape[2]:
        raise ValueError("rows must be [batch, 4, D] with contiguous rows")
    dev = rows.device
    batch, _, D = rows.shape
    _require(gate, torch.bfloat16, "gate", dev)
    if gate.numel() != D:
        raise ValueError("gate must hold D elements")
    if out is None:
        out = torch.empty((batch, D), dtype=torch.bfloat16, device=dev)
    if out.dtype != torch.bfloat16 or out.device != dev or out.dim() != 2 or out.stride(1) != 1 or out.shape[1] != D:
        raise ValueError("out must be a [batch, D] bfloat16 view with contiguous rows")
    with torch.cuda.device(dev):
        rc = load().ds_compress_fold(_ptr(rows), batch, D, rows.stride(0), _ptr(gate), _ptr(out), out.stride(0),
                                     _stream_ptr(stream))
    _check(rc, "ds_compress_fold")
    return out


# ------------------------------------------------------------------ the 8-bit cache
#
# These calls run on ``stream`` (default: the tensors' device's current stream).
# Given another stream, what they return is allocated on it, and every tensor is
# recorded there, so that freeing a tensor does not hand out its memory early;
# the caller orders the two streams, as for any other work.
#
# A decode step makes several of these calls per layer, and the smallest run for a
# few microseconds.  The usual call (the current stream and device, contiguous
# tensors) is therefore marshalled by the extension _front, which returns None for
# any other; that is marshalled here, each check in one comparison, and the reason
# for a refusal is worked out only once there is one.

_front = None


def _load_front():
    """Import the extension once and give it the library's addresses."""
    global _front
    import torch  # noqa: F401  (loads the libraries that the extension is linked to)
    lib = load()
    from . import build
    made = build.front_built_for()
    if made not in (None, build.front_tag()):  # loading it could end the process
        raise RuntimeError(f"_front.so was built for {made}, not for {build.front_tag()}; build it with "
                           "`python -m sparse_attention_top_ds_b200.build`")
    try:
        from . import _front as front
    except ImportError as e:
        raise RuntimeError(
            f"_front.so cannot be loaded ({e}); build it with `python -m sparse_attention_top_ds_b200.build`") from e
    front.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.ds_cache_quantize, lib.ds_sparse_attention_q8, lib.ds_attention_mass, lib.ds_cache_evict, lib.ds_cache_compact)))
    _front = front
    return front


def _refuse(t, dtype, shape, dev, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _arg(t, dtype, shape, dev, name):
    """Address of a contiguous tensor argument."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.shape == shape:
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, dtype, shape, dev, name)


def _opt(t, dtype, shape, dev, name):
    return None if t is None else _arg(t, dtype, shape, dev, name)


def _rows_arg(t, dtype, shape, dev, name, lead=1):
    """Address of an argument that is contiguous behind its first ``lead``
    dimensions (sizes of one have no stride)."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape:
            if not t.is_contiguous():
                step = 1
                for n, st in zip(reversed(t.shape[lead:]), reversed(t.stride()[lead:])):
                    if n != 1 and st != step:
                        raise ValueError(f"{name} must be contiguous behind dimension {lead}")
                    step *= n
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, dtype, shape, dev, name)


def _batch_step(t, unit, name):
    """Batch stride of t [batch, ...] in units of ``unit`` elements."""
    st = t.stride(0) if t.shape[0] > 1 else t.numel()
    if st % unit:
        raise ValueError(f"{name}: the batch stride must be whole rows")
    return st // unit


def _lead(t, dims, name):
    """Device (its index) of the argument that says where a call runs."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {list(t.shape)}")
    return t.get_device()


def _size(t, dims, i, name):
    """Size i of an argument of ``dims`` dimensions."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {list(t.shape)}")
    return t.shape[i]


def _new(like, shape, dtype, stream):
    """A new tensor on the device of ``like``, of the stream that will write it."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    import torch
    dev = like.device
    here = torch.cuda.current_stream(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, expected {dev}")
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    if here != stream:
        t.record_stream(here)
    return t


def _run(where, fn, args, dev, stream, tensors):
    import torch
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, expected cuda:{dev}")
    else:
        raw = stream.cuda_stream
    if torch.cuda.current_device() == dev:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, raw)
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    if rc != DS_OK:
        raise DsError(rc, where)


def _cache8(codes, scales, block, batch, dev):
    """(dtype, T, kv_heads, d, addresses and batch strides) of an 8-bit cache."""
    import torch
    if not isinstance(codes, torch.Tensor):
        raise TypeError("codes must be a torch.Tensor")
    if codes.dtype is torch.float8_e4m3fn:
        dt = DS_E4M3
    elif codes.dtype is torch.int8:
        dt = DS_I8
    else:
        raise TypeError(f"codes must be torch.float8_e4m3fn or torch.int8, got {codes.dtype}")
    if not isinstance(block, int) or block < 1:
        raise ValueError("block must be a positive int")
    shape = codes.shape
    if len(shape) == 4 and shape[0] == batch:
        _, T, kv_heads, d = shape
        nb = (T + block - 1) // block
        c = _rows_arg(codes, codes.dtype, shape, dev, "codes")
        s = _rows_arg(scales, torch.float32, (batch, nb, kv_heads), dev, "scales")
        return dt, T, kv_heads, d, c, _batch_step(codes, max(1, kv_heads * d), "codes"), s, _batch_step(
            scales, max(1, kv_heads), "scales")
    if len(shape) == 3:
        T, kv_heads, d = shape
        c = _arg(codes, codes.dtype, shape, dev, "codes")
        return dt, T, kv_heads, d, c, 0, _arg(scales, torch.float32, ((T + block - 1) // block, kv_heads), dev, "scales"), 0
    raise ValueError(f"codes must be [T, kv_heads, d] or [{batch}, T, kv_heads, d], got {list(shape)}")


def ds_cache_quantize(rows, codes, scales, block, pos=None, length=None, stream=None):
    """Write bfloat16 rows into an 8-bit cache, in place.

    rows    bf16 [batch, n, kv_heads, d], 16-byte aligned; its batch stride (0 too) and its row
            stride (kv_heads * d or more) are multiples of 8 elements;
    codes   float8_e4m3fn or int8 [batch, T, kv_heads, d];
    scales  float32 [batch, ceil(T / block), kv_heads];
    block   rows that share a scale: 1, 2, 4 .. 128;
    pos     int32 [batch] or None (= 0): where the first row goes, a multiple of block;
    length  int32 [batch] or None (= n): how many rows are written.
    Returns (codes, scales).
    """
    if stream is None:
        r = (_front or _load_front()).quantize(rows, codes, scales, block, pos, length)
        if r is not None:
            return r
    import torch
    dev = _lead(rows, 4, "rows")
    batch, n, kv_heads, d = rows.shape
    dt, T, ch, cd, c, cstep, s, sstep = _cache8(codes, scales, block, batch, dev)
    if ch != kv_heads or cd != d or codes.dim() != 4:
        raise ValueError("codes must be [batch, T, kv_heads, d] with the rows' kv_heads and d")
    x = _rows_arg(rows, torch.bfloat16, rows.shape, dev, "rows", 2)
    if (batch > 1 and rows.stride(0) % 8) or (n > 1 and (rows.stride(1) % 8 or rows.stride(1) < kv_heads * d)):
        raise ValueError("rows: the batch and row strides must be multiples of 8 elements, the row stride at least "
                         f"kv_heads * d, got strides {list(rows.stride())}")
    args = (x, rows.stride(0) if batch > 1 else 0, rows.stride(1) if n > 1 else kv_heads * d, batch, n, kv_heads, d, dt, block,
            _opt(pos, torch.int32, (batch,), dev, "pos"), _opt(length, torch.int32, (batch,), dev, "length"), c, cstep, s,
            sstep, T)
    _run("ds_cache_quantize", load().ds_cache_quantize, args, dev, stream, (rows, codes, scales, pos, length))
    return codes, scales


def ds_sparse_attention_q8(q, codes, scales, idx, block, scale=None, win=None, win_len=None, sink=None,
                           return_lse=False, out=None, lse=None, stream=None):
    """ds_sparse_attention over an 8-bit cache with KV heads.

    q      bf16 [batch, heads, d];
    codes  float8_e4m3fn or int8 [T, kv_heads, d] (one cache for every batch row)
           or [batch, T, kv_heads, d];
    scales float32 [ceil(T / block), kv_heads], with the batch in front as in codes;
    idx    int32 [batch, k] or None (window only);  block  rows that share a scale;
    win    bf16 [batch, W, kv_heads, d] or None;  win_len  int32 [batch] or None (= W);
    sink   float32 [heads] or None;  scale  default 1/sqrt(d).
    Query head h reads KV head h // (heads // kv_heads).
    The weights carry 16 bits into the weighted sum, or 8 (bfloat16) in calls of more than
    64 rows with more than 32 query heads to a KV head.
    Returns out bf16 [batch, heads, d], or (out, lse float32 [batch, heads]).
    """
    if stream is None and out is None and lse is None:
        r = (_front or _load_front()).attention(q, codes, scales, idx, block, scale, win, win_len, sink, bool(return_lse))
        if r is not None:
            return r
    import torch
    dev = _lead(q, 3, "q")
    batch, heads, d = shape = q.shape
    dt, T, kv_heads, cd, c, cstep, s, sstep = _cache8(codes, scales, block, batch, dev)
    if cd != d:
        raise ValueError("codes and q differ in d")
    qp = _arg(q, torch.bfloat16, shape, dev, "q")
    k = W = 0
    ip = wp = None
    if idx is not None:
        k = _size(idx, 2, 1, "idx")
        ip = _arg(idx, torch.int32, (batch, k), dev, "idx") if k else None
    if win is not None:
        W = _size(win, 4, 1, "win")
        wp = _arg(win, torch.bfloat16, (batch, W, kv_heads, d), dev, "win") if W else None
    lp, sp = _opt(win_len, torch.int32, (batch,), dev, "win_len"), _opt(sink, torch.float32, (heads,), dev, "sink")
    if out is None:
        out = _new(q, shape, torch.bfloat16, stream)
        op = out.data_ptr()
    else:
        op = _arg(out, torch.bfloat16, shape, dev, "out")
    if lse is None and return_lse:
        lse = _new(q, (batch, heads), torch.float32, stream)
        ep = lse.data_ptr()
    else:
        ep = _opt(lse, torch.float32, (batch, heads), dev, "lse")
    args = (qp, c, cstep, s, sstep, dt, block, T, ip, k, wp, W, lp, sp, batch, heads, kv_heads, d,
            d ** -0.5 if scale is None else float(scale), op, ep)
    _run("ds_sparse_attention_q8", load().ds_sparse_attention_q8, args, dev, stream,
         (q, codes, scales, idx, win, win_len, sink, out, lse))
    return (out, lse) if return_lse else out


def ds_attention_mass(q, cache, idx, lse, mass, scales=None, block=1, scale=None, stream=None):
    """Add the attention weight that every selected row received, summed over
    the query heads, to the rows' accounts, in place.

    q      bf16 [batch, heads, d];  idx  int32 [batch, k];
    cache  an 8-bit cache as in ds_sparse_attention_q8, with its scales and block; or
           a bf16 cache [T, d], [batch, T, d] or [batch, T, kv_heads, d], scales None;
    lse    float32 [batch, heads] of the attention;  scale  default 1/sqrt(d);
    mass   float32 [batch, T], rows contiguous.
    Returns mass.
    """
    if stream is None:
        r = (_front or _load_front()).mass(q, cache, idx, lse, mass, scales, block, scale)
        if r is not None:
            return r
    import torch
    dev = _lead(q, 3, "q")
    batch, heads, d = shape = q.shape
    if scales is not None:
        dt, T, kv_heads, cd, c, cstep, s, sstep = _cache8(cache, scales, block, batch, dev)
    else:
        if not isinstance(cache, torch.Tensor) or cache.dim() not in (2, 3, 4) or (cache.dim() > 2 and cache.shape[0] != batch):
            raise ValueError("a bf16 cache must be [T, d], [batch, T, d] or [batch, T, kv_heads, d]")
        T, kv_heads = (cache.shape[1], cache.shape[2]) if cache.dim() == 4 else (cache.shape[-2], 1)
        dt, cd, s, sstep, block = DS_BF16, cache.shape[-1], None, 0, 1
        c = _rows_arg(cache, torch.bfloat16, cache.shape, dev, "cache", 0 if cache.dim() == 2 else 1)
        cstep = 0 if cache.dim() == 2 else _batch_step(cache, max(1, kv_heads * cd), "cache")
    if cd != d:
        raise ValueError("cache and q differ in d")
    k = _size(idx, 2, 1, "idx")
    args = (_arg(q, torch.bfloat16, shape, dev, "q"), c, cstep, s, sstep, dt, block, T,
            _arg(idx, torch.int32, (batch, k), dev, "idx") if k else None, k,
            _arg(lse, torch.float32, (batch, heads), dev, "lse"), batch, heads, kv_heads, d,
            d ** -0.5 if scale is None else float(scale), _rows_arg(mass, torch.float32, (batch, T), dev, "mass"),
            _batch_step(mass, 1, "mass"))
    _run("ds_attention_mass", load().ds_attention_mass, args, dev, stream, (q, cache, scales, idx, lse, mass))
    return mass


def ds_cache_evict(mass, budget, block=1, length=None, keep_first=0, keep_last=1, kept=None, new_length=None,
                   stream=None):
    """Which blocks of each batch row's cache stay, by accumulated attention weight.

    mass    float32 [batch, T], rows contiguous;  length  int32 [batch] or None (= T);
    budget  blocks that stay at most: the first ``keep_first`` and the last
            ``keep_last``, then those whose rows' weights sum to the most.
    Returns (kept int32 [batch, budget]: the blocks that stay, ascending, then -1;
    new_length int32 [batch]: the rows in them).
    """
    if stream is None and kept is None and new_length is None:
        r = (_front or _load_front()).evict(mass, budget, block, length, keep_first, keep_last)
        if r is not None:
            return r
    import torch
    dev = _lead(mass, 2, "mass")
    batch, T = shape = mass.shape
    m = _rows_arg(mass, torch.float32, shape, dev, "mass")
    if not isinstance(budget, int) or not isinstance(block, int) or budget < 1:
        raise ValueError("budget and block must be positive ints")
    if kept is None:
        kept = _new(mass, (batch, budget), torch.int32, stream)
        kp = kept.data_ptr()
    else:
        kp = _arg(kept, torch.int32, (batch, budget), dev, "kept")
    if new_length is None:
        new_length = _new(mass, (batch,), torch.int32, stream)
        np_ = new_length.data_ptr()
    else:
        np_ = _arg(new_length, torch.int32, (batch,), dev, "new_length")
    args = (m, _batch_step(mass, 1, "mass"), batch, T, _opt(length, torch.int32, (batch,), dev, "length"), block, budget,
            int(keep_first), int(keep_last), kp, np_)
    _run("ds_cache_evict", load().ds_cache_evict, args, dev, stream, (mass, length, kept, new_length))
    return kept, new_length


def ds_cache_compact(kept, block=1, length=None, rows=(), blocks=(), stream=None):
    """Move the blocks of a list (ds_cache_evict's) to the front of other buffers.

    kept    int32 [batch, budget];  length  int32 [batch] or None: the lengths
            before the eviction;
    rows    pairs (src, dst) of arrays with one entry for each row, [batch, T, ...]
            and [batch, at least min(T, budget * block), ...] (codes, keys, accounts);
    blocks  pairs with one entry for each block, [batch, ceil(T / block), ...] and
            [batch, at least budget, ...] (scales).
    The arrays are contiguous behind the batch; a pair has one dtype and trailing
    shape, and no dst has a byte of a src or of another dst (two halves of one buffer
    may be src and dst: buf[:, 0] and buf[:, 1]).  Rows of dst behind what stays are
    left as they were.
    """
    if stream is None and (_front or _load_front()).compact(kept, block, length, rows, blocks):
        return
    import torch
    dev = _lead(kept, 2, "kept")
    batch, budget = kept.shape
    if not isinstance(block, int) or block < 1:
        raise ValueError("block must be a positive int")
    n = len(rows) + len(blocks)
    if not 1 <= n <= DS_CACHE_MAX_ARRAYS:
        raise ValueError(f"1 to {DS_CACHE_MAX_ARRAYS} arrays can be moved")
    first = rows[0][0] if rows else blocks[0][0]
    if not isinstance(first, torch.Tensor) or first.dim() < 2:
        raise TypeError("src must be a tensor [batch, items, ...]")
    T = first.shape[1] if rows else first.shape[1] * block
    arrays, tensors = [], [kept, length]
    for per_block, pairs, items, least in ((0, rows, T, min(T, budget * block)), (1, blocks, (T + block - 1) // block, budget)):
        for src, dst in pairs:
            if not isinstance(src, torch.Tensor) or not isinstance(dst, torch.Tensor):
                raise TypeError("src and dst must be tensors")
            shape, dt, size = src.shape, src.dtype, src.element_size()
            rest, to = shape[2:], dst.shape
            if len(to) < 2 or to[1] < least:
                raise ValueError(f"dst must be [{batch}, at least {least}, ...] like src, got {list(to)}")
            arrays += (_rows_arg(src, dt, (batch, items) + rest, dev, "src"), _rows_arg(dst, dt, (batch, to[1]) + rest, dev, "dst"),
                       src.stride(0) * size, dst.stride(0) * size, math.prod(rest) * size, per_block)
            if stream is not None:
                tensors += [src, dst]
    arrays = struct.pack(_CACHE_ARRAY * n, *arrays)
    args = (arrays, n, _arg(kept, torch.int32, (batch, budget), dev, "kept"), budget,
            _opt(length, torch.int32, (batch,), dev, "length"), batch, T, block)
    _run("ds_cache_compact", load().ds_cache_compact, args, dev, stream, tensors)
