"""Python binding of libcacheblend (the GB300 CacheBlend blend-step library).

Argument marshalling only: every step of the blend runs in the CUDA library behind the C ABI
declared in ``include/cacheblend.h``.  PyTorch is used for device memory and streams.  There is
no fallback: if ``libcacheblend.so`` is missing or cannot be loaded, every call raises.

Entry points (same names as the C ABI): ``cb_model_create``, ``cb_model_destroy``,
``cb_rerope``, ``cb_blend``, ``cb_blend_gradual``, ``cb_selected_count``, ``cb_last_error``;
``BlendModel`` bundles a handle with the device tensors it borrows, ``KV8Cache`` an 8-bit paged K/V cache
with the operators on it (write, append, read, attention, attention_shared, evict), and ``cb_sample`` takes the next
tokens from rows of logits.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcacheblend.so")

CB_OK, CB_ERR_INVALID_ARG, CB_ERR_UNSUPPORTED, CB_ERR_OOM, CB_ERR_CUDA, CB_ERR_INTERNAL = 0, -1, -2, -3, -4, -5
CB_F32, CB_BF16 = 0, 1
CB_PREC_SPLIT, CB_PREC_BF16 = 0, 1
CB_MAX_CHUNKS = 1024
EXPORTED = ("cb_model_create", "cb_model_destroy", "cb_rerope", "cb_blend", "cb_blend_gradual", "cb_blend_streamed",
            "cb_selected_count", "cb_last_error", "cb_profile_enable", "cb_profile_read", "cb_model_status",
            "cb_rerope_static", "cb_model_diag", "cb_load_time", "cb_controller_ratio", "cb_pick_storage",
            "cb_blend_paged", "cb_kv_gather_pages", "cb_kv_scatter_pages", "cb_pages_create", "cb_pages_destroy",
            "cb_pages_alloc", "cb_pages_retain", "cb_pages_release", "cb_pages_plan_write", "cb_pages_count",
            "cb_pages_free", "cb_index_create", "cb_index_destroy", "cb_index_size", "cb_index_match",
            "cb_select_hkvd", "cb_blend_hkvd", "cb_gradual_layout", "cb_kv8_create", "cb_kv8_destroy", "cb_kv8_status",
            "cb_kv8_write", "cb_kv8_read", "cb_kv8_attention", "cb_kv8_evict", "cb_blend_kv8", "cb_kv8_append",
            "cb_kv8_attention_shared", "cb_sample")
CB_STATIC_MAX_CHUNKS = 256
CB_SAMPLE_MAX_VOCAB = 393216
_I32 = 1 << 31
CB_STATUS_BAD_TOKEN, CB_STATUS_WAIT_TIMEOUT, CB_STATUS_BAD_ROW = 1, 2, 4


class CbConfig(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("d_model", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("ffn_hidden", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("rope_theta", ctypes.c_double), ("rms_eps", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("max_chunks", ctypes.c_int32),
                ("precision", ctypes.c_int32)]


_PP = ctypes.POINTER(ctypes.c_void_p)


class CbWeights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("final_norm", ctypes.c_void_p), ("lm_head", ctypes.c_void_p),
                ("attn_norm", _PP), ("wq", _PP), ("wk", _PP), ("wv", _PP), ("wo", _PP), ("mlp_norm", _PP),
                ("w_gate", _PP), ("w_up", _PP), ("w_down", _PP)]


class CbChunk(ctypes.Structure):
    _fields_ = [("src_pos", ctypes.c_int32), ("dst_pos", ctypes.c_int32), ("len", ctypes.c_int32)]


class CbStats(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("n_ctx", ctypes.c_int32), ("n_selected", ctypes.c_int32),
                ("n_recompute", ctypes.c_int32), ("kernel_launches", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("gemm_flops", ctypes.c_double), ("attn_flops", ctypes.c_double),
                ("kv_bytes_moved", ctypes.c_double)]


class CbLayerIO(ctypes.Structure):
    _fields_ = [("cached_kv_host", ctypes.c_void_p), ("out_kv_host", ctypes.c_void_p), ("copy_stream", ctypes.c_void_p),
                ("copy_back_stream", ctypes.c_void_p)]


class CbPagedKV(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("src_table", ctypes.c_void_p), ("dst_table", ctypes.c_void_p)]


class CbKV8Config(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", ctypes.c_int64), ("weight_cells", ctypes.c_int64)]


class CbKV8Seqs(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("table", ctypes.c_void_p), ("table_ld", ctypes.c_int32),
                ("lens", ctypes.c_void_p), ("max_len", ctypes.c_int32)]


class CbKernelProfile(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 24), ("launches", ctypes.c_int32), ("ms", ctypes.c_double),
                ("flops", ctypes.c_double), ("bytes", ctypes.c_double)]


class CacheBlendError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


_lib = None


def build(force: bool = False) -> str:
    from . import buildlib
    return buildlib.build(force=force)


def lib() -> ctypes.CDLL:
    """Load libcacheblend.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libcacheblend.so is not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        L.cb_model_create.restype = ctypes.c_int
        L.cb_model_create.argtypes = [ctypes.POINTER(CbConfig), ctypes.POINTER(CbWeights), ctypes.POINTER(vp)]
        L.cb_model_destroy.restype = ctypes.c_int
        L.cb_model_destroy.argtypes = [vp]
        L.cb_rerope.restype = ctypes.c_int
        L.cb_rerope.argtypes = [vp, vp, i64, ctypes.POINTER(CbChunk), i32, vp]
        L.cb_blend.restype = ctypes.c_int
        L.cb_blend.argtypes = [vp, vp, i32, vp, ctypes.POINTER(CbChunk), i32, ctypes.c_double, vp, vp, vp, vp,
                               ctypes.POINTER(CbStats), vp]
        L.cb_blend_gradual.restype = ctypes.c_int
        L.cb_blend_gradual.argtypes = [vp, vp, i32, vp, ctypes.POINTER(CbChunk), i32, ctypes.POINTER(ctypes.c_double),
                                       i32, vp, vp, vp, vp, ctypes.POINTER(CbStats), vp]
        L.cb_blend_streamed.restype = ctypes.c_int
        L.cb_blend_streamed.argtypes = [vp, vp, i32, ctypes.POINTER(CbLayerIO), ctypes.POINTER(CbChunk), i32,
                                        ctypes.POINTER(ctypes.c_double), i32, vp, vp, vp, vp, ctypes.POINTER(CbStats), vp]
        L.cb_load_time.restype = ctypes.c_double
        L.cb_load_time.argtypes = [ctypes.c_double, i64, ctypes.c_double]
        L.cb_controller_ratio.restype = ctypes.c_double
        L.cb_controller_ratio.argtypes = [ctypes.c_double, ctypes.c_double, ctypes.c_double]
        L.cb_pick_storage.restype = i32
        L.cb_pick_storage.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double), i32,
                                      ctypes.c_double, i64, ctypes.c_double, ctypes.c_double]
        L.cb_blend_paged.restype = ctypes.c_int
        L.cb_blend_paged.argtypes = [vp, vp, i32, ctypes.POINTER(CbPagedKV), ctypes.POINTER(CbChunk), i32,
                                     ctypes.POINTER(ctypes.c_double), i32, vp, vp, vp, vp, ctypes.POINTER(CbStats), vp]
        L.cb_kv_gather_pages.restype = ctypes.c_int
        L.cb_kv_gather_pages.argtypes = [vp, ctypes.POINTER(CbPagedKV), i32, vp, vp]
        L.cb_kv_scatter_pages.restype = ctypes.c_int
        L.cb_kv_scatter_pages.argtypes = [vp, vp, i32, ctypes.POINTER(CbPagedKV), vp]
        ip = ctypes.POINTER(ctypes.c_int32)
        L.cb_pages_create.restype = ctypes.c_int
        L.cb_pages_create.argtypes = [i64, ctypes.POINTER(vp)]
        L.cb_pages_destroy.restype = ctypes.c_int
        L.cb_pages_destroy.argtypes = [vp]
        L.cb_pages_alloc.restype = ctypes.c_int
        L.cb_pages_alloc.argtypes = [vp, i32, ip]
        L.cb_pages_retain.restype = ctypes.c_int
        L.cb_pages_retain.argtypes = [vp, ip, i32]
        L.cb_pages_release.restype = ctypes.c_int
        L.cb_pages_release.argtypes = [vp, ip, i32]
        L.cb_pages_plan_write.restype = i32
        L.cb_pages_plan_write.argtypes = [vp, ip, i32, ip]
        L.cb_pages_count.restype = i32
        L.cb_pages_count.argtypes = [vp, i32]
        L.cb_pages_free.restype = i64
        L.cb_pages_free.argtypes = [vp]
        L.cb_index_create.restype = ctypes.c_int
        L.cb_index_create.argtypes = [i32, vp, vp, vp, vp, i32, i32, ctypes.POINTER(vp)]
        L.cb_index_destroy.restype = ctypes.c_int
        L.cb_index_destroy.argtypes = [vp]
        L.cb_index_size.restype = i32
        L.cb_index_size.argtypes = [vp, i32]
        L.cb_index_match.restype = ctypes.c_int
        L.cb_index_match.argtypes = [vp, vp, i32, i32, i32, i32, vp, i32, vp, vp]
        L.cb_selected_count.restype = i32
        L.cb_selected_count.argtypes = [i32, ctypes.c_double]
        L.cb_gradual_layout.restype = i32
        L.cb_gradual_layout.argtypes = [i32, ctypes.POINTER(ctypes.c_double), i32, vp, vp, vp, i32]
        L.cb_select_hkvd.restype = ctypes.c_int
        L.cb_select_hkvd.argtypes = [vp, i32, i32, vp, vp]
        L.cb_sample.restype = ctypes.c_int
        L.cb_sample.argtypes = [vp, i32, i32, i32, i64, vp, vp, vp, vp, vp, vp, vp, vp]
        L.cb_blend_hkvd.restype = ctypes.c_int
        L.cb_blend_hkvd.argtypes = [vp, vp, i32, vp, ctypes.POINTER(CbChunk), i32, vp, i32, vp, vp,
                                    ctypes.POINTER(CbStats), vp]
        sq = ctypes.POINTER(CbKV8Seqs)
        L.cb_kv8_create.restype = ctypes.c_int
        L.cb_kv8_create.argtypes = [ctypes.POINTER(CbKV8Config), vp, vp, ctypes.POINTER(vp)]
        L.cb_kv8_destroy.restype = ctypes.c_int
        L.cb_kv8_destroy.argtypes = [vp]
        L.cb_kv8_status.restype = ctypes.c_int
        L.cb_kv8_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), i32]
        for f in (L.cb_kv8_write, L.cb_kv8_read):
            f.restype = ctypes.c_int
            f.argtypes = [vp, sq, i32, i32, vp, vp, i64, i64, vp, i32, vp]
        L.cb_kv8_append.restype = ctypes.c_int
        L.cb_kv8_append.argtypes = [vp, sq, i32, vp, i64, vp, i64, vp, vp, i64, vp, ctypes.c_double, vp, i32, vp]
        L.cb_kv8_attention.restype = ctypes.c_int
        L.cb_kv8_attention.argtypes = [vp, sq, i32, vp, i64, vp, i32, ctypes.c_float, vp, i64, vp, i32, i32, vp]
        L.cb_kv8_attention_shared.restype = ctypes.c_int
        L.cb_kv8_attention_shared.argtypes = [vp, sq, vp, sq, i32, vp, i64, vp, i32, ctypes.c_float, vp, i64, vp]
        L.cb_kv8_evict.restype = ctypes.c_int
        L.cb_kv8_evict.argtypes = [vp, sq, vp, i32, i32, i32, vp, i32, i32, i32, i32, vp, vp, vp, vp]
        L.cb_blend_kv8.restype = ctypes.c_int
        L.cb_blend_kv8.argtypes = [vp, vp, i32, vp, vp, vp, ctypes.POINTER(CbChunk), i32, ctypes.POINTER(ctypes.c_double),
                                   i32, vp, vp, vp, vp, ctypes.POINTER(CbStats), vp]
        L.cb_profile_enable.restype = ctypes.c_int
        L.cb_profile_enable.argtypes = [vp, i32, i32]
        L.cb_profile_read.restype = i32
        L.cb_profile_read.argtypes = [vp, ctypes.POINTER(CbKernelProfile), i32]
        L.cb_rerope_static.restype = ctypes.c_int
        L.cb_rerope_static.argtypes = [vp, i64, i32, i32, i32, ctypes.c_double, i32, ctypes.POINTER(CbChunk), i32, vp]
        L.cb_model_diag.restype = ctypes.c_int
        L.cb_model_diag.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
        L.cb_model_status.restype = ctypes.c_int
        L.cb_model_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), i32]
        L.cb_last_error.restype = ctypes.c_char_p
        L.cb_last_error.argtypes = []
        _lib = L
    return _lib


def cb_last_error() -> str:
    return lib().cb_last_error().decode()


def _check(code: int):
    if code != CB_OK:
        raise CacheBlendError(code, cb_last_error())


def cb_selected_count(n_ctx: int, ratio: float) -> int:
    return int(lib().cb_selected_count(n_ctx, ratio))


def cb_gradual_layout(n_ctx: int, ratios):
    """The comparing layers of a gradual schedule as a list of (layer, kept rows, compared rows), in the order
    cb_blend_gradual writes out_selected and out_dev.  Raises on an invalid schedule."""
    r = (ctypes.c_double * len(ratios))(*[float(x) for x in ratios])
    cap = len(ratios)
    lay, kept, cmp_ = (ctypes.c_int32 * cap)(), (ctypes.c_int32 * cap)(), (ctypes.c_int32 * cap)()
    n = int(lib().cb_gradual_layout(int(n_ctx), r, len(ratios), ctypes.addressof(lay), ctypes.addressof(kept),
                                    ctypes.addressof(cmp_), cap))
    if n < 0:
        raise ValueError(f"cb_gradual_layout: invalid schedule (status {n})")
    return [(int(lay[i]), int(kept[i]), int(cmp_[i])) for i in range(n)]


def cb_select_hkvd(dev, n: int, k: int, out_rows, stream=None) -> None:
    """The k rows of largest dev[0..n) (ties to the lower row), ascending, into out_rows (device tensors)."""
    _check(lib().cb_select_hkvd(_ptr(dev), n, k, _ptr(out_rows), _stream(stream)))


def cb_sample(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None, out_tokens=None, out_probs=None, stream=None):
    """The next token of each row of logits (device float32 or bfloat16 [n_rows][vocab], or [vocab] for one row; a row's
    elements contiguous) from uniform (device float32 [n_rows]); temperature, top_p and min_p (float32) and top_k (int32) are
    [n_rows] or None.  Returns out_tokens (int32 [n_rows]); out_probs (float32 [n_rows]) receives the tokens' probabilities.
    Asynchronous on `stream` (default: the current one of the logits' device), without synchronisation or scratch.  A tensor
    of another shape, type or device raises ValueError before anything is enqueued."""
    import torch
    if logits.dim() == 1:
        logits = logits[None]
    dtype, dev = logits.dtype, logits.get_device()
    if logits.dim() != 2 or dev < 0 or (dtype is not torch.float32 and dtype is not torch.bfloat16):
        raise ValueError("logits must be a float32 or bfloat16 device tensor [n_rows][vocab]")
    n, vocab = logits.shape
    stride = logits.stride()
    if vocab > 1 and stride[1] != 1:
        raise ValueError("the logits of a row must be contiguous")

    def of(t, name, want):
        if t is None:
            return None
        if t.dtype is not want or t.get_device() != dev or t.shape != (n,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {want} tensor [{n}] on {logits.device}")
        return t.data_ptr()
    f32, i32 = torch.float32, torch.int32
    if uniform is None:
        raise ValueError("uniform is missing")
    settings = of(temperature, "temperature", f32), of(top_k, "top_k", i32), of(top_p, "top_p", f32), of(min_p, "min_p", f32)
    drawn, probs = of(uniform, "uniform", f32), of(out_probs, "out_probs", f32)
    here = torch.cuda.current_device()
    with contextlib.nullcontext() if here == dev else torch.cuda.device(dev):
        raw = torch._C._cuda_getCurrentRawStream(dev)
        at = raw if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
        if out_tokens is None:
            # made on the call's stream
            other = None if at == raw else torch.cuda.ExternalStream(at, device=dev) if at else torch.cuda.default_stream(dev)
            with torch.cuda.stream(other):
                out_tokens = uniform.new_empty(n, dtype=i32)
        code = lib().cb_sample(logits.data_ptr(), CB_BF16 if dtype is torch.bfloat16 else CB_F32, n, vocab, stride[0] if n > 1 else vocab,
                               *settings, drawn, of(out_tokens, "out_tokens", i32), probs, at)
    if code:
        _check(code)
    return out_tokens


def _chunks(chunks):
    arr = (CbChunk * max(1, len(chunks)))()
    for i, (s, d, n) in enumerate(chunks):
        arr[i] = CbChunk(int(s), int(d), int(n))
    return arr


def _ptr(t) -> int:
    if t is None:
        return 0
    return t if isinstance(t, int) else int(t.data_ptr())


def _stream(stream) -> int:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return stream if isinstance(stream, int) else int(stream.cuda_stream)


def cb_model_create(config: dict, weights: dict) -> int:
    """config: shape dict (n_layers, d_model, n_heads, n_kv_heads, head_dim, ffn_hidden, vocab, rope_theta,
    rms_eps, dtype 'bf16'|'f32', max_tokens, max_chunks, precision 'split'|'bf16'); weights: device pointers / tensors with keys
    embed, final_norm, lm_head and 'layers' (list of dicts of per-layer tensors)."""
    cfg = CbConfig(config["n_layers"], config["d_model"], config["n_heads"], config["n_kv_heads"],
                   config["head_dim"], config["ffn_hidden"], config["vocab"], float(config["rope_theta"]),
                   float(config.get("rms_eps", 1e-5)), CB_BF16 if config["dtype"] == "bf16" else CB_F32,
                   int(config["max_tokens"]), int(config.get("max_chunks", 256)),
                   CB_PREC_BF16 if config.get("precision", "split") == "bf16" else CB_PREC_SPLIT)
    L = config["n_layers"]
    tabs = {}
    for name in ("attn_norm", "wq", "wk", "wv", "wo", "mlp_norm", "w_gate", "w_up", "w_down"):
        tabs[name] = (ctypes.c_void_p * L)(*[_ptr(weights["layers"][i][name]) for i in range(L)])
    w = CbWeights(_ptr(weights["embed"]), _ptr(weights["final_norm"]), _ptr(weights["lm_head"]),
                  *[ctypes.cast(tabs[n], _PP) for n in ("attn_norm", "wq", "wk", "wv", "wo", "mlp_norm",
                                                         "w_gate", "w_up", "w_down")])
    h = ctypes.c_void_p()
    _check(lib().cb_model_create(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(h)))
    return h.value


def cb_model_destroy(handle: int) -> None:
    _check(lib().cb_model_destroy(handle))


def cb_rerope(handle: int, kv, n_rows: int, chunks, stream=None) -> None:
    _check(lib().cb_rerope(handle, _ptr(kv), int(n_rows), _chunks(chunks), len(chunks), _stream(stream)))


def cb_rerope_static(kv, n_rows: int, n_layers: int, n_kv_heads: int, head_dim: int, rope_theta: float, dtype: str,
                     chunks, stream=None) -> None:
    """In-place re-RoPE without a model handle and without any device allocation (see the header)."""
    _check(lib().cb_rerope_static(_ptr(kv), int(n_rows), int(n_layers), int(n_kv_heads), int(head_dim),
                                  float(rope_theta), CB_BF16 if dtype == "bf16" else CB_F32, _chunks(chunks),
                                  len(chunks), _stream(stream)))


def cb_blend(handle: int, tokens, n_tokens: int, cached_kv, chunks, ratio: float, out_kv, out_logits,
             out_selected=None, out_dev=None, stream=None, stats: bool = False):
    st = CbStats()
    _check(lib().cb_blend(handle, _ptr(tokens), int(n_tokens), _ptr(cached_kv), _chunks(chunks), len(chunks),
                          float(ratio), _ptr(out_kv), _ptr(out_logits), _ptr(out_selected), _ptr(out_dev),
                          ctypes.byref(st) if stats else None, _stream(stream)))
    if stats:
        return {f: getattr(st, f) for f, _ in CbStats._fields_}
    return None


def cb_blend_hkvd(handle: int, tokens, n_tokens: int, cached_kv, chunks, hkvd, k: int, out_kv, out_logits,
                  stream=None, stats: bool = False):
    """A blend whose recomputed context rows are the caller's (device int32 [k], ascending)."""
    st = CbStats()
    _check(lib().cb_blend_hkvd(handle, _ptr(tokens), int(n_tokens), _ptr(cached_kv), _chunks(chunks), len(chunks),
                               _ptr(hkvd), int(k), _ptr(out_kv), _ptr(out_logits), ctypes.byref(st) if stats else None,
                               _stream(stream)))
    if stats:
        return {f: getattr(st, f) for f, _ in CbStats._fields_}
    return None


def cb_blend_gradual(handle: int, tokens, n_tokens: int, cached_kv, chunks, ratios, out_kv, out_logits,
                     out_selected=None, out_dev=None, stream=None, stats: bool = False):
    """Gradual filtering: ratios[l - 1] is the ratio of layer l (n_layers - 1 entries, non-increasing counts)."""
    st = CbStats()
    r = (ctypes.c_double * max(1, len(ratios)))(*[float(x) for x in ratios])
    _check(lib().cb_blend_gradual(handle, _ptr(tokens), int(n_tokens), _ptr(cached_kv), _chunks(chunks), len(chunks),
                                  r, len(ratios), _ptr(out_kv), _ptr(out_logits), _ptr(out_selected), _ptr(out_dev),
                                  ctypes.byref(st) if stats else None, _stream(stream)))
    if stats:
        return {f: getattr(st, f) for f, _ in CbStats._fields_}
    return None


def cb_blend_streamed(handle: int, tokens, n_tokens: int, cached_kv_host, chunks, ratios, out_kv, out_logits,
                      out_kv_host=None, out_selected=None, out_dev=None, stream=None, copy_stream=None,
                      copy_back_stream=None, stats: bool = False):
    """Layer-wise load pipeline: the chunk caches come from pinned host memory (cached_kv_host), one layer
    per copy on copy_stream; out_kv_host (optional, pinned) receives each finished layer."""
    st = CbStats()
    r = (ctypes.c_double * max(1, len(ratios)))(*[float(x) for x in ratios])
    io = CbLayerIO(_ptr(cached_kv_host) or None, _ptr(out_kv_host) or None, _stream(copy_stream),
                   _stream(copy_back_stream) if copy_back_stream is not None else None)
    _check(lib().cb_blend_streamed(handle, _ptr(tokens), int(n_tokens), ctypes.byref(io), _chunks(chunks), len(chunks),
                                   r, len(ratios), _ptr(out_kv), _ptr(out_logits), _ptr(out_selected), _ptr(out_dev),
                                   ctypes.byref(st) if stats else None, _stream(stream)))
    if stats:
        return {f: getattr(st, f) for f, _ in CbStats._fields_}
    return None


def _paged(pool, n_pages, page_size, src_table=None, dst_table=None):
    return CbPagedKV(_ptr(pool) or None, int(n_pages), int(page_size), _ptr(src_table) or None, _ptr(dst_table) or None)


def cb_blend_paged(handle: int, tokens, n_tokens: int, pool, n_pages: int, page_size: int, src_table, dst_table, chunks,
                   ratios, work_kv, out_logits, out_selected=None, out_dev=None, stream=None, stats: bool = False):
    """Blend over a paged pool: chunk caches read through src_table, blended K/V written through dst_table
    (device int32 tables); work_kv is the caller's contiguous working copy."""
    st = CbStats()
    r = (ctypes.c_double * max(1, len(ratios)))(*[float(x) for x in ratios])
    pg = _paged(pool, n_pages, page_size, src_table, dst_table)
    _check(lib().cb_blend_paged(handle, _ptr(tokens), int(n_tokens), ctypes.byref(pg), _chunks(chunks), len(chunks),
                                r, len(ratios), _ptr(work_kv), _ptr(out_logits), _ptr(out_selected), _ptr(out_dev),
                                ctypes.byref(st) if stats else None, _stream(stream)))
    if stats:
        return {f: getattr(st, f) for f, _ in CbStats._fields_}
    return None


def cb_kv_gather_pages(handle: int, pool, n_pages: int, page_size: int, table, n_rows: int, out_kv, stream=None):
    pg = _paged(pool, n_pages, page_size, table, None)
    _check(lib().cb_kv_gather_pages(handle, ctypes.byref(pg), int(n_rows), _ptr(out_kv), _stream(stream)))


def cb_kv_scatter_pages(handle: int, kv, n_rows: int, pool, n_pages: int, page_size: int, table, stream=None):
    pg = _paged(pool, n_pages, page_size, None, table)
    _check(lib().cb_kv_scatter_pages(handle, _ptr(kv), int(n_rows), ctypes.byref(pg), _stream(stream)))


class Pages:
    """Host-side page bookkeeping of a pool (cb_pages_*): reference counts, allocation, copy-on-write plans."""

    def __init__(self, n_pages: int):
        h = ctypes.c_void_p()
        _check(lib().cb_pages_create(int(n_pages), ctypes.byref(h)))
        self.h = h.value

    @staticmethod
    def _arr(ids):
        return (ctypes.c_int32 * max(1, len(ids)))(*[int(i) for i in ids])

    def alloc(self, n: int) -> list:
        a = (ctypes.c_int32 * max(1, n))()
        _check(lib().cb_pages_alloc(self.h, int(n), a))
        return [a[i] for i in range(n)]

    def retain(self, ids):
        _check(lib().cb_pages_retain(self.h, self._arr(ids), len(ids)))

    def release(self, ids):
        _check(lib().cb_pages_release(self.h, self._arr(ids), len(ids)))

    def plan_write(self, table) -> tuple:
        """(dst table, number of copy-on-write pages)."""
        d = (ctypes.c_int32 * max(1, len(table)))()
        n = int(lib().cb_pages_plan_write(self.h, self._arr(table), len(table), d))
        if n < 0:
            raise CacheBlendError(n, cb_last_error())
        return [d[i] for i in range(len(table))], n

    def count(self, i: int) -> int:
        return int(lib().cb_pages_count(self.h, int(i)))

    def free(self) -> int:
        return int(lib().cb_pages_free(self.h))

    def close(self):
        if self.h:
            lib().cb_pages_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def cb_blend_kv8(handle: int, tokens, n_tokens: int, cache: "KV8Cache", src_table, dst_table, chunks, ratios, work_kv,
                 out_logits, out_selected=None, out_dev=None, stream=None, stats: bool = False):
    """Blend over an 8-bit paged pool: chunk caches read through src_table, blended K/V written through dst_table
    (device int32 tables); work_kv is the caller's contiguous working copy."""
    st = CbStats()
    r = (ctypes.c_double * max(1, len(ratios)))(*[float(x) for x in ratios])
    _check(lib().cb_blend_kv8(handle, _ptr(tokens), int(n_tokens), cache.handle, _ptr(src_table), _ptr(dst_table),
                              _chunks(chunks), len(chunks), r, len(ratios), _ptr(work_kv), _ptr(out_logits),
                              _ptr(out_selected), _ptr(out_dev), ctypes.byref(st) if stats else None, _stream(stream)))
    if stats:
        return {f: getattr(st, f) for f, _ in CbStats._fields_}
    return None


class KV8Cache:
    """An 8-bit paged K/V cache (cb_kv8_*): the caller's pool and the operators on it.

    codes: device uint8 (or float8_e4m3fn) [n_layers][2][n_pages][n_kv_heads][page_size][head_dim]; scales: device
    float32 [n_layers][2][n_pages][n_kv_heads].  ``KV8Cache.empty`` allocates both.  dtype ('bf16' | 'f32') is that of
    the K/V rows, queries and outputs.  weight_cells: scratch of attention calls that return weights (``cells``).

    Every call takes the batch as ``table`` (device int32 [n_seqs][pages]) and ``lens`` (device int32 [n_seqs], or None:
    max_len each); ``max_len`` bounds the lengths (default: all the table can hold).  Calls are asynchronous on `stream`
    (default: the current one) and allocate nothing, so they can be captured into a graph.  A tensor of another shape,
    type or device raises ValueError before anything is enqueued.  An output that is left to a call is made on the call's
    stream: another stream that uses it waits for that one first (and Tensor.record_stream tells the allocator so)."""

    def __init__(self, codes, scales, n_heads: int, dtype: str = "bf16", weight_cells: int = 0):
        import torch
        self.handle = None
        if codes.dim() != 6 or codes.shape[1] != 2 or codes.element_size() != 1 or not codes.is_contiguous() or not codes.is_cuda:
            raise ValueError("codes must be a contiguous device tensor of bytes [n_layers][2][n_pages][n_kv_heads][page_size][head_dim]")
        if scales.dtype != torch.float32 or scales.shape != codes.shape[:4] or not scales.is_contiguous() or scales.device != codes.device:
            raise ValueError("scales must be contiguous float32 [n_layers][2][n_pages][n_kv_heads] on the codes' device")
        if dtype not in ("bf16", "f32"):
            raise ValueError("dtype must be 'bf16' or 'f32'")
        self.codes, self.scales = codes, scales               # borrowed by the handle
        self.n_layers, _, self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = codes.shape
        self.n_heads, self.device = int(n_heads), codes.device
        self.dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        self._i32, self._f32, self._dev = torch.int32, torch.float32, codes.get_device()
        self._kv_row, self._kv_width = (self.n_kv_heads, self.head_dim), self.n_kv_heads * self.head_dim
        self._q_row, self._q_width = (self.n_heads, self.head_dim), self.n_heads * self.head_dim
        self._scale = self.head_dim ** -0.5
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        self._lib = lib()
        cfg = CbKV8Config(self.n_layers, self.n_heads, self.n_kv_heads, self.head_dim, CB_BF16 if dtype == "bf16" else CB_F32,
                          self.page_size, self.n_pages, int(weight_cells))
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(self._lib.cb_kv8_create(ctypes.byref(cfg), codes.data_ptr(), scales.data_ptr(), ctypes.byref(h)))
        self.handle = h.value

    @classmethod
    def empty(cls, n_layers: int, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, n_heads: int,
              dtype: str = "bf16", weight_cells: int = 0, device="cuda"):
        """A cache over a new pool (all blocks zero)."""
        import torch
        codes = torch.zeros((n_layers, 2, n_pages, n_kv_heads, page_size, head_dim), dtype=torch.uint8, device=device)
        scales = torch.zeros((n_layers, 2, n_pages, n_kv_heads), dtype=torch.float32, device=device)
        return cls(codes, scales, n_heads, dtype, weight_cells)

    @staticmethod
    def cells(n_q: int, n_heads: int, max_len: int) -> int:
        """weight_cells that an attention call of n_q query rows over at most max_len keys needs to return weights."""
        return n_q * n_heads * (-(-max_len // 128) * 128 + 1)

    @staticmethod
    def shared_cells(n_q: int, n_heads: int, head_dim: int) -> int:
        """weight_cells that an attention_shared call of n_q query rows needs."""
        return n_q * n_heads * (2 * head_dim + 6)

    # A decoding step calls write and attention once per layer, so the checks below stay within a few microseconds.
    def _int(self, t, name, *shape):
        if t.dtype is not self._i32 or t.get_device() != self._dev or not t.is_contiguous() or t.shape != shape:
            raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on {self.device}")
        return t.data_ptr()

    def _seqs(self, table, lens, max_len, layer, n_layers=1):
        shape = table.shape
        if len(shape) != 2:
            raise ValueError("table must be int32 [n_seqs][pages]")
        n, ld = shape
        if max_len is None:
            max_len = ld * self.page_size
        # (ctypes would take the lower 32 bits of a larger number)
        if not (-_I32 <= max_len < _I32 and -_I32 <= layer < _I32 and -_I32 <= n_layers < _I32):
            raise ValueError(f"max_len {max_len}, layer {layer} or n_layers {n_layers} passes 32 bits")
        return CbKV8Seqs(n, self._int(table, "table", n, ld), ld, None if lens is None else self._int(lens, "lens", n), max_len)

    def _stream(self, stream):
        if stream is None:
            return self._raw_stream(self._dev)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _made_on(self, stream):
        """Outputs that a call makes are made on its stream: a fill is then in order with the kernels, and the memory is
        none that the current stream still uses."""
        raw = self._stream(stream)
        if stream is None or raw == self._raw_stream(self._dev):
            return contextlib.nullcontext()
        import torch
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(raw, device=self.device) if raw else torch.cuda.default_stream(self.device)
        return torch.cuda.stream(stream)

    def _kv(self, t, name, n_layers):
        """(pointer, layer stride, row stride, rows) of K/V rows [n_layers][rows][n_kv_heads][head_dim] (or without the
        layers when there is one)."""
        shape, stride = t.shape, t.stride()
        if len(shape) == 3 and n_layers == 1:
            shape, stride = (1, *shape), (0, *stride)
        if t.dtype is not self.dtype or t.get_device() != self._dev or len(shape) != 4 or shape[0] != n_layers or \
                shape[2:] != self._kv_row:
            raise ValueError(f"{name} must be {self.dtype} [{n_layers}][rows][{self.n_kv_heads}][{self.head_dim}] on {self.device}")
        if stride[3] != 1 or (stride[2] != self.head_dim and self.n_kv_heads > 1):
            raise ValueError(f"{name}: the heads of a row must be contiguous")
        return t.data_ptr(), stride[0] if n_layers > 1 else 0, stride[1] if shape[1] > 1 else self._kv_width, shape[1]

    def _io(self, f, table, lens, k, v, layer, n_layers, row_start, max_len, stream):
        kp, *lay = self._kv(k, "k", n_layers)
        vp, *lay_v = self._kv(v, "v", n_layers)
        if lay != lay_v:
            raise ValueError("k and v must have the same number of rows and the same strides")
        sq = self._seqs(table, lens, max_len, layer, n_layers)
        code = f(self.handle, sq, layer, n_layers, kp, vp, lay[0], lay[1],
                 None if row_start is None else self._int(row_start, "row_start", sq.n_seqs + 1), lay[2], self._stream(stream))
        if code:
            _check(code)

    def write(self, table, lens, k, v, layer: int = 0, n_layers: int = 1, row_start=None, max_len=None, stream=None):
        """k and v ([n_layers][n_rows][n_kv_heads][head_dim]) become the last rows of their sequences (lens counts them
        already), quantised into their blocks.  row_start (device int32 [n_seqs + 1]) gives each sequence its rows; None
        shares them evenly."""
        self._io(self._lib.cb_kv8_write, table, lens, k, v, layer, n_layers, row_start, max_len, stream)

    def read(self, table, lens, k, v, layer: int = 0, n_layers: int = 1, row_start=None, max_len=None, stream=None):
        """The last rows of each sequence as values, into k and v (as for write)."""
        self._io(self._lib.cb_kv8_read, table, lens, k, v, layer, n_layers, row_start, max_len, stream)

    def _q(self, t, name):
        shape, stride = t.shape, t.stride()
        if t.dtype is not self.dtype or t.get_device() != self._dev or len(shape) != 3 or shape[1:] != self._q_row:
            raise ValueError(f"{name} must be {self.dtype} [n_q][{self.n_heads}][{self.head_dim}] on {self.device}")
        if stride[2] != 1 or (stride[1] != self.head_dim and self.n_heads > 1):
            raise ValueError(f"{name}: the heads of a row must be contiguous")
        return t.data_ptr(), stride[0] if shape[0] > 1 else self._q_width, shape[0]

    def append(self, table, lens, q, k, v, rope_theta: float, out_q=None, layer: int = 0, positions=None, row_start=None,
               max_len=None, stream=None):
        """New rows of one layer, q and k not yet rotated: k ([n_rows][n_kv_heads][head_dim]) is rotated at its rows'
        positions, and k and v become the last rows of their sequences (as write puts them there); q ([n_rows][n_heads]
        [head_dim], or None) is rotated into out_q, which may be q itself; returns out_q.  positions: device int32 [n_rows];
        None: a row's place in its sequence.  row_start as for write.  Rows of no sequence are left as they were."""
        shape, stride, dt, dev = k.shape, k.stride(), self.dtype, self._dev
        if k.dtype is not dt or v.dtype is not dt or k.get_device() != dev or v.get_device() != dev or len(shape) != 3 or \
                shape[1:] != self._kv_row or stride[2] != 1 or (stride[1] != self.head_dim and self.n_kv_heads > 1) or \
                v.shape != shape or v.stride() != stride:
            # (a single row's stride, and a single head's, say nothing)
            if self._kv(k, "k", 1)[1:] != self._kv(v, "v", 1)[1:] or len(shape) != 3 or v.dim() != 3:
                raise ValueError("k and v must be [n_rows][n_kv_heads][head_dim] with the same number of rows and the same strides")
        n = shape[0]
        qp, qs, op, os_ = None, 0, None, 0
        if q is not None:
            if out_q is None:
                with self._made_on(stream):
                    # rows that belong to no sequence are not written: zeros there
                    out_q = q.new_empty(q.shape) if row_start is None else q.new_zeros(q.shape)
            qp, qs, n_q = self._q(q, "q")
            op, os_, n_out = (qp, qs, n_q) if out_q is q else self._q(out_q, "out_q")
            if n_q != n or n_out != n:
                raise ValueError(f"q and out_q must have k's {n} rows")
        elif out_q is not None:
            raise ValueError("out_q without q")
        sq = self._seqs(table, lens, max_len, layer)
        code = self._lib.cb_kv8_append(self.handle, sq, layer, qp, qs, op, os_, k.data_ptr(), v.data_ptr(),
                                       stride[0] if n > 1 else self._kv_width,
                                       None if positions is None else self._int(positions, "positions", n), rope_theta,
                                       None if row_start is None else self._int(row_start, "row_start", sq.n_seqs + 1), n,
                                       self._stream(stream))
        if code:
            _check(code)
        return out_q

    def attention(self, table, lens, q, out=None, layer: int = 0, q_start=None, scale=None, weights=None, add: bool = False,
                  max_len=None, stream=None):
        """softmax(q k * scale) v of the query rows q [n_q][n_heads][head_dim], each sequence's last rows, over its cache
        (causal); returns out.  weights (device float32 [n_seqs][n_kv_heads][ld >= max_len]) receives, or with add
        accumulates, the weight of every key.  q_start as row_start of write; scale defaults to head_dim ** -0.5.  Rows of
        a sequence whose length is out of range are not written."""
        if out is None:
            with self._made_on(stream):
                # rows that belong to no sequence are not written: zeros there
                out = q.new_empty(q.shape) if q_start is None else q.new_zeros(q.shape)
        qp, qs, n = self._q(q, "q")
        op, os_, n_out = self._q(out, "out")
        if n_out != n:
            raise ValueError(f"out must have q's {n} rows")
        sq = self._seqs(table, lens, max_len, layer)
        wp, ld = None, 0
        if weights is not None:
            ld = weights.shape[-1]
            if weights.dtype is not self._f32 or weights.get_device() != self._dev or not weights.is_contiguous() or \
                    weights.shape != (sq.n_seqs, self.n_kv_heads, ld):
                raise ValueError(f"weights must be contiguous float32 [{sq.n_seqs}][{self.n_kv_heads}][keys] on {self.device}")
            wp = weights.data_ptr()
        code = self._lib.cb_kv8_attention(self.handle, sq, layer, qp, qs,
                                          None if q_start is None else self._int(q_start, "q_start", sq.n_seqs + 1), n,
                                          self._scale if scale is None else scale, op, os_, wp, ld, add, self._stream(stream))
        if code:
            _check(code)
        return out

    def attention_shared(self, prefix_table, prefix_lens, table, lens, q, out=None, layer: int = 0, prefix_start=None, q_start=None,
                         scale=None, prefix_max_len=None, max_len=None, stream=None):
        """attention where groups of sequences share rows that stand in front of their own: prefix_table (device int32
        [groups][pages]) and prefix_lens ([groups]) name each group's, which are read once for all its sequences; prefix_start
        (device int32 [groups + 1]) gives the groups their sequences, None shares them evenly.  A query row sees its whole
        prefix and then its own sequence's rows as in attention.  The cache needs weight_cells >= shared_cells(n_q, ..)."""
        if out is None:
            with self._made_on(stream):
                out = q.new_empty(q.shape) if q_start is None else q.new_zeros(q.shape)
        qp, qs, n = self._q(q, "q")
        op, os_, n_out = self._q(out, "out")
        if n_out != n:
            raise ValueError(f"out must have q's {n} rows")
        pre = self._seqs(prefix_table, prefix_lens, prefix_max_len, layer)
        sq = self._seqs(table, lens, max_len, layer)
        code = self._lib.cb_kv8_attention_shared(
            self.handle, pre, None if prefix_start is None else self._int(prefix_start, "prefix_start", pre.n_seqs + 1), sq, layer,
            qp, qs, None if q_start is None else self._int(q_start, "q_start", sq.n_seqs + 1), n,
            self._scale if scale is None else scale, op, os_, self._stream(stream))
        if code:
            _check(code)
        return out

    def evict(self, table, lens, dst_table, weights, n_keep: int, n_sink: int = 0, n_recent: int = 0, out_rows=None,
              out_lens=None, out_weights=None, layer: int = 0, n_layers: int = 1, max_len=None, stream=None):
        """Every KV head keeps n_keep rows of each sequence: the first n_sink, the last n_recent and of the others those of
        largest weight (weights: device float32 [n_layers][n_seqs][n_kv_heads][ld]).  The kept rows move to dst_table
        (table itself: in place; else pages that table does not name).  Returns dict(rows, lens, weights); out_weights
        defaults to weights itself, out_lens may be lens."""
        sq = self._seqs(table, lens, max_len, layer, n_layers)
        if not (-_I32 <= n_keep < _I32 and -_I32 <= n_sink < _I32 and -_I32 <= n_recent < _I32):
            raise ValueError(f"n_keep {n_keep}, n_sink {n_sink} or n_recent {n_recent} passes 32 bits")
        n = sq.n_seqs
        if dst_table.dim() != 2:
            raise ValueError("dst_table must be int32 [n_seqs][pages]")
        dst_ld = dst_table.shape[1]
        dp = self._int(dst_table, "dst_table", n, dst_ld)
        if out_weights is None:
            out_weights = weights
        with self._made_on(stream):
            if out_lens is None:
                out_lens = table.new_empty(n)
            if out_rows is None:
                out_rows = table.new_empty((n_layers, n, self.n_kv_heads, max(int(n_keep), 0)))
        ld = weights.shape[-1]
        for t, name in ((weights, "weights"),) if out_weights is weights else ((weights, "weights"), (out_weights, "out_weights")):
            if t.dtype is not self._f32 or t.get_device() != self._dev or not t.is_contiguous() or \
                    t.shape != (n_layers, n, self.n_kv_heads, ld):
                raise ValueError(f"{name} must be contiguous float32 [{n_layers}][{n}][{self.n_kv_heads}][rows] on {self.device}")
        code = self._lib.cb_kv8_evict(self.handle, sq, dp, dst_ld, layer, n_layers, weights.data_ptr(), ld, n_keep, n_sink,
                                      n_recent, out_weights.data_ptr(),
                                      self._int(out_rows, "out_rows", n_layers, n, self.n_kv_heads, n_keep),
                                      self._int(out_lens, "out_lens", n), self._stream(stream))
        if code:
            _check(code)
        return dict(rows=out_rows, lens=out_lens, weights=out_weights)

    def status(self, clear: bool = False) -> int:
        """Device status bits (CB_STATUS_*) recorded by the kernels; synchronises."""
        v = ctypes.c_uint32()
        _check(self._lib.cb_kv8_status(self.handle, ctypes.byref(v), 1 if clear else 0))
        return v.value

    def close(self):
        if self.handle:
            self._lib.cb_kv8_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class FragmentIndex:
    """cb_index_*: an immutable fragment index on the device (built from host arrays) and its matcher."""

    def __init__(self, chunk_size: int, tokens, occ_ids, old_st, ns, max_tokens: int):
        t = np.ascontiguousarray(tokens, dtype=np.uint32).reshape(-1)
        o, s_, n_ = (np.ascontiguousarray(a, dtype=np.int32) for a in (occ_ids, old_st, ns))
        h = ctypes.c_void_p()
        _check(lib().cb_index_create(int(chunk_size), t.ctypes.data, o.ctypes.data, s_.ctypes.data, n_.ctypes.data,
                                     len(o), int(max_tokens), ctypes.byref(h)))
        self.h, self.chunk_size = h.value, chunk_size

    def size(self, what: int) -> int:
        return int(lib().cb_index_size(self.h, int(what)))

    def match_async(self, tokens, ns: int, out, out_count, stride: int = 1, greedy: bool = True, stream=None):
        """Enqueue a match: out (device int32 [max][3]) and out_count (device int32 [1])."""
        _check(lib().cb_index_match(self.h, _ptr(tokens), int(tokens.shape[0]), int(ns), int(stride),
                                    1 if greedy else 0, _ptr(out), int(out.shape[0]), _ptr(out_count),
                                    _stream(stream)))

    def match(self, tokens, ns: int, stride: int = 1, greedy: bool = True, max_out: int = 4096) -> list:
        """Matches as (occupant id, old_st, cur_st) triples (synchronises)."""
        import torch
        out = torch.empty((max_out, 3), dtype=torch.int32, device=tokens.device)
        cnt = torch.zeros(1, dtype=torch.int32, device=tokens.device)
        self.match_async(tokens, ns, out, cnt, stride, greedy)
        n = int(cnt.item())
        return [tuple(int(v) for v in r) for r in out[:min(n, max_out)].cpu().tolist()]

    def close(self):
        if self.h:
            lib().cb_index_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def cb_load_time(per_token_kv_bytes: float, n_tokens: int, throughput_bytes_per_s: float) -> float:
    return float(lib().cb_load_time(float(per_token_kv_bytes), int(n_tokens), float(throughput_bytes_per_s)))


def cb_controller_ratio(t_prefill_s: float, t_load_s: float, r_min: float = 0.15) -> float:
    return float(lib().cb_controller_ratio(float(t_prefill_s), float(t_load_s), float(r_min)))


def cb_pick_storage(devices, per_token_kv_bytes: float, n_tokens: int, t_prefill_s: float, r_min: float = 0.15) -> int:
    """devices: list of (throughput bytes/s, cost per GB); returns the chosen index."""
    n = len(devices)
    bw = (ctypes.c_double * max(1, n))(*[float(d[0]) for d in devices])
    cost = (ctypes.c_double * max(1, n))(*[float(d[1]) for d in devices])
    i = int(lib().cb_pick_storage(bw, cost, n, float(per_token_kv_bytes), int(n_tokens), float(t_prefill_s),
                                  float(r_min)))
    if i < 0:
        raise CacheBlendError(i, cb_last_error())
    return i


def cb_model_status(handle: int, clear: bool = False) -> int:
    """Device status bits (CB_STATUS_*) recorded by the kernels; synchronises."""
    v = ctypes.c_uint32()
    _check(lib().cb_model_status(handle, ctypes.byref(v), 1 if clear else 0))
    return v.value


def cb_model_diag(handle: int) -> list:
    """16 diagnostic words (status bits, then the first bounded wait that gave up); synchronises."""
    w = (ctypes.c_uint32 * 16)()
    _check(lib().cb_model_diag(handle, w))
    return list(w)


def cb_profile_enable(handle: int, enable: bool = True, max_launches: int = 65536) -> None:
    _check(lib().cb_profile_enable(handle, 1 if enable else 0, int(max_launches)))


def cb_profile_read(handle: int) -> list:
    """Per kernel class: name, launches, ms, flops, bytes since the last read (synchronises)."""
    arr = (CbKernelProfile * 32)()
    n = lib().cb_profile_read(handle, arr, 32)
    if n < 0:
        raise CacheBlendError(n, cb_last_error())
    return [dict(name=arr[i].name.decode(), launches=arr[i].launches, ms=arr[i].ms, flops=arr[i].flops,
                 bytes=arr[i].bytes) for i in range(n)]


# ------------------------------------------------------------------------------------------------
# convenience: a model handle that owns the device copies of its weights
# ------------------------------------------------------------------------------------------------
def to_device(a: np.ndarray, device="cuda"):
    """numpy float32 or bfloat16-bit-pattern (uint16) array -> torch tensor on the device."""
    import torch
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16)
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


class BlendModel:
    """A cb_model handle plus the device weights it borrows."""

    def __init__(self, shape: dict, weights: dict, max_tokens: int, max_chunks: int = 256, device="cuda",
                 precision: str = "split"):
        import torch
        self.shape = dict(shape)
        self.device = torch.device(device)
        self.weights = {k: to_device(weights[k], device) for k in ("embed", "final_norm", "lm_head")}
        self.weights["layers"] = [{k: to_device(v, device) for k, v in lw.items()} for lw in weights["layers"]]
        cfg = dict(shape, max_tokens=max_tokens, max_chunks=max_chunks, precision=precision)
        self.handle = cb_model_create(cfg, self.weights)
        self.max_tokens = max_tokens
        self.kv_dtype = torch.bfloat16 if shape["dtype"] == "bf16" else torch.float32

    def status(self, clear: bool = False) -> int:
        return cb_model_status(self.handle, clear)

    def close(self):
        if self.handle:
            cb_model_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def kv_buffer(self, n_rows: int):
        import torch
        s = self.shape
        return torch.empty((s["n_layers"], 2, n_rows, s["n_kv_heads"], s["head_dim"]), dtype=self.kv_dtype,
                           device=self.device)

    def blend(self, tokens, cached_kv, chunks, ratio, out_kv=None, stream=None, want_dev=False, stats=False):
        """Run cb_blend; returns dict(out_kv, logits, selected, dev?, stats?).  Asynchronous on `stream`."""
        import torch
        n = int(tokens.shape[0])
        n_ctx = sum(c[2] for c in chunks)
        k = cb_selected_count(n_ctx, ratio)
        if out_kv is None:
            out_kv = self.kv_buffer(n)
        logits = torch.empty(self.shape["vocab"], dtype=torch.float32, device=self.device)
        sel = torch.empty(max(k, 1), dtype=torch.int32, device=self.device)
        dev = torch.empty(max(n_ctx, 1), dtype=torch.float32, device=self.device) if want_dev else None
        st = cb_blend(self.handle, tokens, n, cached_kv, chunks, ratio, out_kv, logits,
                      sel if k > 0 else None, dev, stream, stats)
        out = dict(out_kv=out_kv, logits=logits, selected=sel[:k], k=k)
        if want_dev:
            out["dev"] = dev[:n_ctx]
        if stats:
            out["stats"] = st
        return out

    def blend_hkvd(self, tokens, cached_kv, chunks, hkvd, out_kv=None, stream=None):
        """Run cb_blend_hkvd with the given recomputed context rows (device int32, ascending); returns
        dict(out_kv, logits).  Asynchronous on `stream`."""
        import torch
        n = int(tokens.shape[0])
        if out_kv is None:
            out_kv = self.kv_buffer(n)
        logits = torch.empty(self.shape["vocab"], dtype=torch.float32, device=self.device)
        cb_blend_hkvd(self.handle, tokens, n, cached_kv, chunks, hkvd, int(hkvd.numel()), out_kv, logits, stream)
        return dict(out_kv=out_kv, logits=logits)

    def blend_gradual(self, tokens, cached_kv, chunks, ratios, out_kv=None, stream=None, want_dev=False,
                      stats=False):
        """Run cb_blend_gradual; returns dict(out_kv, logits, counts [k_1..k_{L-1}], sets {layer: positions} for
        the check layer and every shrinking layer, devs {layer: deviations}?, stats?).  The sets and
        deviations are device tensors (asynchronous on `stream`)."""
        import torch
        n = int(tokens.shape[0])
        n_ctx = sum(c[2] for c in chunks)
        counts = [cb_selected_count(n_ctx, r) for r in ratios]
        try:
            layout = cb_gradual_layout(n_ctx, ratios)      # the library's own order of the outputs
        except ValueError:
            layout = []                                    # cb_blend_gradual below rejects it with its own error
        n_sel = sum(kept for _, kept, _ in layout)
        n_dev = sum(cmp_ for _, _, cmp_ in layout)
        if out_kv is None:
            out_kv = self.kv_buffer(n)
        logits = torch.empty(self.shape["vocab"], dtype=torch.float32, device=self.device)
        sel = torch.empty(max(n_sel, 1), dtype=torch.int32, device=self.device)
        dev = torch.empty(max(n_dev, 1), dtype=torch.float32, device=self.device) if want_dev else None
        st = cb_blend_gradual(self.handle, tokens, n, cached_kv, chunks, ratios, out_kv, logits,
                              sel if n_sel > 0 else None, dev, stream, stats)
        sets, devs, at, dat = {}, {}, 0, 0
        for l, kept, nd in layout:
            sets[l] = sel[at:at + kept]
            at += kept
            if want_dev:
                devs[l] = dev[dat:dat + nd]
                dat += nd
        out = dict(out_kv=out_kv, logits=logits, counts=counts, sets=sets)
        if want_dev:
            out["devs"] = devs
        if stats:
            out["stats"] = st
        return out

    def blend_streamed(self, tokens, cached_kv_host, chunks, ratios, out_kv=None, out_kv_host=None, stream=None,
                       copy_stream=None, copy_back_stream=None, stats=False):
        """Run cb_blend_streamed (chunk caches in pinned host memory, loaded layer by layer); returns
        dict(out_kv, out_kv_host, logits, stats?).  Asynchronous on `stream`."""
        import torch
        n = int(tokens.shape[0])
        if out_kv is None:
            out_kv = self.kv_buffer(n)
        logits = torch.empty(self.shape["vocab"], dtype=torch.float32, device=self.device)
        if copy_stream is None:
            copy_stream = torch.cuda.Stream(self.device)
        st = cb_blend_streamed(self.handle, tokens, n, cached_kv_host, chunks, ratios, out_kv, logits,
                               out_kv_host=out_kv_host, stream=stream, copy_stream=copy_stream,
                               copy_back_stream=copy_back_stream, stats=stats)
        out = dict(out_kv=out_kv, out_kv_host=out_kv_host, logits=logits)
        if stats:
            out["stats"] = st
        return out

    def prefill_chunk(self, tokens, stream=None):
        """A chunk prefilled alone at positions 0..len-1 (cb_blend with no cached chunks): its K/V cache."""
        return self.blend(tokens, None, [], 0.0, stream=stream)["out_kv"]
