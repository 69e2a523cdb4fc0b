"""Thin ctypes binding over libdiffattn.so (``include/diffattn.h``).

Every function here has the name of the C entry point it wraps and only
marshals arguments: torch tensors (device memory allocated by PyTorch) are
passed as raw pointers together with their sizes, on the current CUDA
stream.  All arithmetic happens in the library's CUDA kernels.  There is no
fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdiffattn.so")

DA_OK = 0
DA_ERR_INVALID_ARG = -1
DA_ERR_UNSUPPORTED = -2
DA_ERR_ALIGNMENT = -3
DA_ERR_WORKSPACE = -4
DA_ERR_CUDA = -5
DA_ERR_DEVICE_TIMEOUT = -6
DA_ERR_SCHEDULE = -7
DA_ERR_PAGE = -8
DA_ERR_CACHE_FULL = -9
DA_BF16 = 0
DA_FP32 = 1

# Every symbol include/diffattn.h declares.
EXPORTS = (
    "diffattn_status_string",
    "diffattn_lambda_init",
    "lambda_from_params",
    "diffattn_v1_fwd",
    "diffattn_v2_prefill",
    "diffattn_v2_decode_workspace_size",
    "diffattn_v2_decode",
    "diffattn_v2_decode_noalloc",
    "diffattn_v1_decode_workspace_size",
    "diffattn_v1_decode",
    "diffattn_v1_fwd_window",
    "diffattn_v2_prefill_window",
    "diffattn_v2_decode_window",
    "diffattn_v1_decode_window",
    "diffattn_v1_bwd_workspace_size",
    "diffattn_v1_bwd",
    "diffattn_v2_bwd_workspace_size",
    "diffattn_v2_bwd",
    "lambda_from_params_bwd",
    "diffattn_v1_fwd_train_saves_size",
    "diffattn_v1_fwd_train",
    "diffattn_v1_bwd_saved_workspace_size",
    "diffattn_v1_bwd_saved",
    "diffattn_v2_prefill_train_saves_size",
    "diffattn_v2_prefill_train",
    "diffattn_v2_bwd_saved_workspace_size",
    "diffattn_v2_bwd_saved",
    "diffattn_v2_prefill_oproj_workspace_size",
    "diffattn_v2_prefill_oproj",
    "diffattn_page_plan_workspace_size",
    "diffattn_page_plan",
    "diffattn_page_release",
    "diffattn_kv4_page_bytes",
    "diffattn_kv4_append",
    "diffattn_kv4_read",
    "diffattn_v2_decode_kv4_workspace_size",
    "diffattn_v2_decode_kv4",
    "diffattn_v1_decode_kv4_workspace_size",
    "diffattn_v1_decode_kv4",
    "diffattn_qk_norm_rope",
    "diffattn_qk_norm_rope_bwd_workspace_size",
    "diffattn_qk_norm_rope_bwd",
    "diffattn_reset_tile_counters",
    "diffattn_selftest_hold_tile_counter",
    "diffattn_selftest_keep_tile_counter",
    "diffattn_selftest_wait_timeout",
)


class DiffAttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (fn, status_string(status), status))


_lib = None
_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t
_ll = ctypes.c_longlong


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the library (once).  Raises if it is missing: there is no
    CPU or library fallback for the operator."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError("libdiffattn.so not built (run __graft_entry__.build() or "
                          "python -m differential_attention_sm_b200.build)")
    lib = ctypes.CDLL(p)
    lib.diffattn_status_string.restype = ctypes.c_char_p
    lib.diffattn_status_string.argtypes = [_i]
    lib.diffattn_lambda_init.restype = ctypes.c_double
    lib.diffattn_lambda_init.argtypes = [_i]
    lib.lambda_from_params.restype = _i
    lib.lambda_from_params.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp]
    lib.diffattn_v1_fwd.restype = _i
    lib.diffattn_v1_fwd.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _i, _i,
                                    _vp, _f, _f, _vp, _vp]
    lib.diffattn_v2_prefill.restype = _i
    lib.diffattn_v2_prefill.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _i,
                                        _vp, _vp]
    lib.diffattn_v2_decode_workspace_size.restype = _sz
    lib.diffattn_v2_decode_workspace_size.argtypes = [_i, _i, _i, _i, _i]
    lib.diffattn_v2_decode.restype = _i
    lib.diffattn_v2_decode.argtypes = [_vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _vp,
                                       _vp, _sz, _vp, _vp]
    lib.diffattn_v2_decode_noalloc.restype = _i
    lib.diffattn_v2_decode_noalloc.argtypes = [_vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _vp,
                                               _vp, _vp]
    lib.diffattn_v1_decode_workspace_size.restype = _sz
    lib.diffattn_v1_decode_workspace_size.argtypes = [_i, _i, _i, _i, _i]
    lib.diffattn_v1_decode.restype = _i
    lib.diffattn_v1_decode.argtypes = [_vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _vp,
                                       _i, _vp, _f, _f, _vp, _sz, _vp, _vp]
    lib.diffattn_v1_fwd_window.restype = _i
    lib.diffattn_v1_fwd_window.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _i,
                                           _i, _i, _vp, _f, _f, _vp, _vp]
    lib.diffattn_v2_prefill_window.restype = _i
    lib.diffattn_v2_prefill_window.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp,
                                               _i, _i, _vp, _vp]
    lib.diffattn_v2_decode_window.restype = _i
    lib.diffattn_v2_decode_window.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _vp, _i, _i, _i, _i,
                                              _i, _vp, _vp, _sz, _vp, _vp]
    lib.diffattn_v1_decode_window.restype = _i
    lib.diffattn_v1_decode_window.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _vp, _i, _i, _i, _i,
                                              _i, _vp, _i, _vp, _f, _f, _vp, _sz, _vp, _vp]
    lib.diffattn_v1_bwd_workspace_size.restype = _sz
    lib.diffattn_v1_bwd_workspace_size.argtypes = [_i, _i, _i, _i, _i]
    lib.diffattn_v1_bwd.restype = _i
    lib.diffattn_v1_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                                    _i, _vp, _f, _f, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp,
                                    _vp]
    lib.diffattn_v2_bwd_workspace_size.restype = _sz
    lib.diffattn_v2_bwd_workspace_size.argtypes = [_i, _i, _i, _i, _i]
    lib.diffattn_v2_bwd.restype = _i
    lib.diffattn_v2_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                                    _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]
    lib.lambda_from_params_bwd.restype = _i
    lib.lambda_from_params_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp,
                                           _vp]
    for name in ("diffattn_v1_fwd_train_saves_size", "diffattn_v1_bwd_saved_workspace_size",
                 "diffattn_v2_prefill_train_saves_size", "diffattn_v2_bwd_saved_workspace_size"):
        getattr(lib, name).restype = _sz
        getattr(lib, name).argtypes = [_i, _i, _i]
    lib.diffattn_v1_fwd_train.restype = _i
    lib.diffattn_v1_fwd_train.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _i,
                                          _i, _i, _vp, _f, _f, _vp, _sz, _vp, _vp]
    lib.diffattn_v1_bwd_saved.restype = _i
    lib.diffattn_v1_bwd_saved.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                                          _i, _i, _vp, _f, _f, _vp, _sz, _vp, _vp, _vp, _vp,
                                          _vp, _vp, _sz, _vp, _vp]
    lib.diffattn_v2_prefill_train.restype = _i
    lib.diffattn_v2_prefill_train.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp,
                                              _i, _i, _vp, _sz, _vp, _vp]
    lib.diffattn_v2_bwd_saved.restype = _i
    lib.diffattn_v2_bwd_saved.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                                          _i, _vp, _sz, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]
    lib.diffattn_v2_prefill_oproj_workspace_size.restype = _sz
    lib.diffattn_v2_prefill_oproj_workspace_size.argtypes = [_i, _i, _i, _i]
    lib.diffattn_v2_prefill_oproj.restype = _i
    lib.diffattn_v2_prefill_oproj.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                                              _i, _i, _i, _i, _vp, _sz, _vp, _vp]
    lib.diffattn_page_plan.restype = _i
    lib.diffattn_page_plan.argtypes = [_vp] * 5 + [_i] * 5 + [_vp] * 7 + [_sz, _vp, _vp]
    lib.diffattn_page_plan_workspace_size.restype = _sz
    lib.diffattn_page_plan_workspace_size.argtypes = [_i, _i]
    lib.diffattn_page_release.restype = _i
    lib.diffattn_page_release.argtypes = [_vp] * 5 + [_i] * 4 + [_vp] * 2
    lib.diffattn_kv4_page_bytes.restype = _sz
    lib.diffattn_kv4_page_bytes.argtypes = [_i, _i, _i]
    lib.diffattn_kv4_append.restype = _i
    lib.diffattn_kv4_append.argtypes = [_vp, _ll, _vp, _ll, _i, _vp, _i, _i, _i, _vp, _i, _i, _vp,
                                        _vp]
    lib.diffattn_kv4_read.restype = _i
    lib.diffattn_kv4_read.argtypes = [_vp, _i, _i, _vp, _i, _i, _i, _vp, _vp, _i, _vp, _vp]
    lib.diffattn_v2_decode_kv4_workspace_size.restype = _sz
    lib.diffattn_v2_decode_kv4_workspace_size.argtypes = [_i, _i, _i]
    lib.diffattn_v2_decode_kv4.restype = _i
    lib.diffattn_v2_decode_kv4.argtypes = [_vp, _vp, _i, _i, _vp, _i, _vp, _i, _vp, _i, _i, _i,
                                           _i, _i, _vp, _vp, _sz, _vp, _vp]
    lib.diffattn_v1_decode_kv4_workspace_size.restype = _sz
    lib.diffattn_v1_decode_kv4_workspace_size.argtypes = [_i, _i]
    lib.diffattn_v1_decode_kv4.restype = _i
    lib.diffattn_v1_decode_kv4.argtypes = [_vp, _vp, _i, _i, _vp, _i, _vp, _i, _vp, _i, _i, _i,
                                           _i, _i, _vp, _i, _vp, _f, _f, _vp, _sz, _vp, _vp]
    lib.diffattn_qk_norm_rope.restype = _i
    lib.diffattn_qk_norm_rope.argtypes = [_vp, _ll, _vp, _ll, _i, _i, _i, _i, _i, _vp, _vp, _f,
                                          _vp, _vp, _i, _i, _vp, _ll, _vp, _ll, _vp]
    lib.diffattn_qk_norm_rope_bwd_workspace_size.restype = _sz
    lib.diffattn_qk_norm_rope_bwd_workspace_size.argtypes = [_i, _i, _i, _i]
    lib.diffattn_qk_norm_rope_bwd.restype = _i
    lib.diffattn_qk_norm_rope_bwd.argtypes = [_vp, _ll, _vp, _ll, _i, _vp, _ll, _vp, _ll, _i, _i,
                                              _i, _i, _vp, _vp, _f, _vp, _vp, _i, _i, _vp, _vp,
                                              _vp, _vp, _vp, _sz, _vp]
    lib.diffattn_reset_tile_counters.restype = _i
    lib.diffattn_reset_tile_counters.argtypes = [_vp]
    lib.diffattn_selftest_hold_tile_counter.restype = _i
    lib.diffattn_selftest_hold_tile_counter.argtypes = [_i, ctypes.c_uint, ctypes.c_uint, _vp]
    lib.diffattn_selftest_keep_tile_counter.restype = _i
    lib.diffattn_selftest_keep_tile_counter.argtypes = [_i, ctypes.c_uint, ctypes.c_uint, _vp]
    lib.diffattn_selftest_wait_timeout.restype = _i
    lib.diffattn_selftest_wait_timeout.argtypes = [ctypes.c_uint, _vp, _vp, _vp]
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().diffattn_status_string(int(status)).decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return DA_BF16
    if t.dtype == torch.float32:
        return DA_FP32
    raise TypeError("unsupported dtype %s" % t.dtype)


def _check(fn: str, status: int) -> None:
    if status != DA_OK:
        raise DiffAttnError(fn, status)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not isinstance(t, int):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("tensors must be contiguous CUDA tensors")


def diffattn_lambda_init(layer: int) -> float:
    return float(load().diffattn_lambda_init(int(layer)))


def lambda_from_params(lq1, lk1, lq2, lk2, layer: int, out=None, stream=None):
    """lambda [H] (fp32, device) from four [H, dim] fp32 device vectors."""
    _need_cuda(lq1, lk1, lq2, lk2)
    H, dim = lq1.shape
    if out is None:
        out = torch.empty(H, dtype=torch.float32, device=lq1.device)
    _check("lambda_from_params", load().lambda_from_params(
        _ptr(lq1), _ptr(lk1), _ptr(lq2), _ptr(lk2), H, dim, int(layer), _ptr(out),
        _stream(stream)))
    return out


def diffattn_v1_fwd(q, k, v, lam, *, causal=True, apply_norm=False, norm_weight=None,
                    norm_eps=1e-5, lambda_init=0.0, out=None, dev_status=None, stream=None):
    """V1 prefill.  q, k [B, N, H, 2d]; v [B, N, H, dv]; lam [H] fp32."""
    _need_cuda(q, k, v, lam, norm_weight, dev_status)
    B, N, H, d2 = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty(B, N, H, dv, dtype=q.dtype, device=q.device)
    _check("diffattn_v1_fwd", load().diffattn_v1_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _dtype_code(q), B, N, H, d2 // 2, dv,
        _ptr(lam), int(bool(causal)), int(bool(apply_norm)), _ptr(norm_weight),
        float(norm_eps), float(lambda_init), _ptr(dev_status), _stream(stream)))
    return out


def diffattn_v2_prefill(q, k, v, lam, *, causal=True, out=None, dev_status=None, stream=None):
    """V2 prefill.  q [B, N, Hq, d]; k, v [B, N, Hkv, d]; lam [Hq/2] fp32."""
    _need_cuda(q, k, v, lam, dev_status)
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    if out is None:
        out = torch.empty(B, N, Hq // 2, d, dtype=q.dtype, device=q.device)
    _check("diffattn_v2_prefill", load().diffattn_v2_prefill(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _dtype_code(q), B, N, Hq, Hkv, d, _ptr(lam),
        int(bool(causal)), _ptr(dev_status), _stream(stream)))
    return out


def diffattn_v2_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, max_len) -> int:
    return int(load().diffattn_v2_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim,
                                                        max_len))


def diffattn_v2_decode(q, k_cache, v_cache, lam, *, cache_lens=None, workspace=None, out=None,
                       dev_status=None, stream=None):
    """V2 decode.  q [B, Hq, d]; caches [B, L, Hkv, d]; lam [Hq/2] fp32;
    cache_lens int32 [B] or None; workspace a uint8 device tensor or None
    (allocated here from the size query)."""
    _need_cuda(q, k_cache, v_cache, lam, cache_lens, dev_status)
    B, Hq, d = q.shape
    L, Hkv = k_cache.shape[1], k_cache.shape[2]
    ws_need = diffattn_v2_decode_workspace_size(B, Hq, Hkv, d, L)
    if workspace is None and ws_need:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if out is None:
        out = torch.empty(B, Hq // 2, d, dtype=q.dtype, device=q.device)
    _check("diffattn_v2_decode", load().diffattn_v2_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cache_lens), L, _ptr(out), _dtype_code(q),
        B, Hq, Hkv, d, _ptr(lam), _ptr(workspace), ws_bytes, _ptr(dev_status),
        _stream(stream)))
    return out


def diffattn_v2_decode_noalloc(q, k_cache, v_cache, lam, *, cache_lens=None, out=None,
                               dev_status=None, stream=None):
    """V2 decode without a workspace (bf16, head_dim 128): for callers that
    cannot allocate device memory.  The split-KV partials live in the
    library's fixed 8 MiB device array; calls that overlap on the GPU race
    on it.  Note that this wrapper still allocates `out` through PyTorch when
    it is not given."""
    _need_cuda(q, k_cache, v_cache, lam, cache_lens, dev_status)
    B, Hq, d = q.shape
    L, Hkv = k_cache.shape[1], k_cache.shape[2]
    if out is None:
        out = torch.empty(B, Hq // 2, d, dtype=q.dtype, device=q.device)
    _check("diffattn_v2_decode_noalloc", load().diffattn_v2_decode_noalloc(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cache_lens), L, _ptr(out), B, Hq, Hkv,
        _ptr(lam), _ptr(dev_status), _stream(stream)))
    return out


def diffattn_v1_decode_workspace_size(batch, n_heads, d_qk, d_v, max_len) -> int:
    return int(load().diffattn_v1_decode_workspace_size(batch, n_heads, d_qk, d_v, max_len))


def diffattn_v1_decode(q, k_cache, v_cache, lam, *, cache_lens=None, apply_norm=False,
                       norm_weight=None, norm_eps=1e-5, lambda_init=0.0, workspace=None,
                       out=None, dev_status=None, stream=None):
    """V1 decode.  q [B, H, 2d]; k_cache [B, L, H, 2d]; v_cache [B, L, H, dv]."""
    _need_cuda(q, k_cache, v_cache, lam, cache_lens, norm_weight, dev_status)
    B, H, d2 = q.shape
    L, dv = k_cache.shape[1], v_cache.shape[-1]
    ws_need = diffattn_v1_decode_workspace_size(B, H, d2 // 2, dv, L)
    if workspace is None and ws_need:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if out is None:
        out = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    _check("diffattn_v1_decode", load().diffattn_v1_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cache_lens), L, _ptr(out), _dtype_code(q),
        B, H, d2 // 2, dv, _ptr(lam), int(bool(apply_norm)), _ptr(norm_weight),
        float(norm_eps), float(lambda_init), _ptr(workspace), ws_bytes, _ptr(dev_status),
        _stream(stream)))
    return out


# ---- sliding-window variants: query i sees keys (i - window, i]; a decode
# query the last `window` cache entries (window 0 = no window) -------------
def diffattn_v1_fwd_window(q, k, v, lam, window, *, causal=True, apply_norm=False,
                           norm_weight=None, norm_eps=1e-5, lambda_init=0.0, out=None,
                           dev_status=None, stream=None):
    """V1 prefill with a sliding window.  Shapes as diffattn_v1_fwd."""
    _need_cuda(q, k, v, lam, norm_weight, dev_status)
    B, N, H, d2 = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty(B, N, H, dv, dtype=q.dtype, device=q.device)
    _check("diffattn_v1_fwd_window", load().diffattn_v1_fwd_window(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _dtype_code(q), B, N, H, d2 // 2, dv,
        _ptr(lam), int(bool(causal)), int(window), int(bool(apply_norm)), _ptr(norm_weight),
        float(norm_eps), float(lambda_init), _ptr(dev_status), _stream(stream)))
    return out


def diffattn_v2_prefill_window(q, k, v, lam, window, *, causal=True, out=None, dev_status=None,
                               stream=None):
    """V2 prefill with a sliding window.  Shapes as diffattn_v2_prefill."""
    _need_cuda(q, k, v, lam, dev_status)
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    if out is None:
        out = torch.empty(B, N, Hq // 2, d, dtype=q.dtype, device=q.device)
    _check("diffattn_v2_prefill_window", load().diffattn_v2_prefill_window(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _dtype_code(q), B, N, Hq, Hkv, d, _ptr(lam),
        int(bool(causal)), int(window), _ptr(dev_status), _stream(stream)))
    return out


def _span(L, window):
    return min(int(window), L) if window and window > 0 else L


def diffattn_v2_decode_window(q, k_cache, v_cache, lam, window, *, cache_lens=None,
                              workspace=None, out=None, dev_status=None, stream=None):
    """V2 decode over the last `window` cache entries.  Shapes as
    diffattn_v2_decode; the workspace is sized for min(window, L) entries."""
    _need_cuda(q, k_cache, v_cache, lam, cache_lens, dev_status)
    B, Hq, d = q.shape
    L, Hkv = k_cache.shape[1], k_cache.shape[2]
    ws_need = diffattn_v2_decode_workspace_size(B, Hq, Hkv, d, _span(L, window))
    if workspace is None and ws_need:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if out is None:
        out = torch.empty(B, Hq // 2, d, dtype=q.dtype, device=q.device)
    _check("diffattn_v2_decode_window", load().diffattn_v2_decode_window(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cache_lens), L, int(window), _ptr(out),
        _dtype_code(q), B, Hq, Hkv, d, _ptr(lam), _ptr(workspace), ws_bytes, _ptr(dev_status),
        _stream(stream)))
    return out


def diffattn_v1_decode_window(q, k_cache, v_cache, lam, window, *, cache_lens=None,
                              apply_norm=False, norm_weight=None, norm_eps=1e-5,
                              lambda_init=0.0, workspace=None, out=None, dev_status=None,
                              stream=None):
    """V1 decode over the last `window` cache entries.  Shapes as
    diffattn_v1_decode; the workspace is sized for min(window, L) entries."""
    _need_cuda(q, k_cache, v_cache, lam, cache_lens, norm_weight, dev_status)
    B, H, d2 = q.shape
    L, dv = k_cache.shape[1], v_cache.shape[-1]
    ws_need = diffattn_v1_decode_workspace_size(B, H, d2 // 2, dv, _span(L, window))
    if workspace is None and ws_need:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if out is None:
        out = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    _check("diffattn_v1_decode_window", load().diffattn_v1_decode_window(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cache_lens), L, int(window), _ptr(out),
        _dtype_code(q), B, H, d2 // 2, dv, _ptr(lam), int(bool(apply_norm)),
        _ptr(norm_weight), float(norm_eps), float(lambda_init), _ptr(workspace), ws_bytes,
        _ptr(dev_status), _stream(stream)))
    return out


# ---- backward ---------------------------------------------------------------
def diffattn_v1_bwd_workspace_size(batch, seqlen, n_heads, d_qk, d_v) -> int:
    return int(load().diffattn_v1_bwd_workspace_size(batch, seqlen, n_heads, d_qk, d_v))


def diffattn_v1_bwd(q, k, v, dout, lam, *, causal=True, window=0, apply_norm=False,
                    norm_weight=None, norm_eps=1e-5, lambda_init=0.0, workspace=None,
                    out=None, dev_status=None, stream=None):
    """V1 gradients.  Returns dict of fp32 device tensors dq, dk (like q),
    dv (like v), dlambda [H] and, with the norm, dnorm_weight [dv]; `out`
    may supply any of them (caller-owned, written in place)."""
    _need_cuda(q, k, v, dout, lam, norm_weight)
    B, N, H, d2 = q.shape
    dvw = v.shape[-1]
    if workspace is None:
        workspace = torch.empty(diffattn_v1_bwd_workspace_size(B, N, H, d2 // 2, dvw),
                                dtype=torch.uint8, device=q.device)
    f32 = dict(dtype=torch.float32, device=q.device)
    res = {"dq": torch.empty(q.shape, **f32), "dk": torch.empty(k.shape, **f32),
           "dv": torch.empty(v.shape, **f32), "dlambda": torch.empty(H, **f32),
           "dnorm_weight": torch.empty(dvw, **f32) if apply_norm else None}
    res.update(out or {})
    _check("diffattn_v1_bwd", load().diffattn_v1_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(lam), _dtype_code(q), B, N, H, d2 // 2,
        dvw, int(bool(causal)), int(window), int(bool(apply_norm)), _ptr(norm_weight),
        float(norm_eps), float(lambda_init), _ptr(res["dq"]), _ptr(res["dk"]), _ptr(res["dv"]),
        _ptr(res["dlambda"]), _ptr(res["dnorm_weight"]), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream(stream)))
    return res


def diffattn_v2_bwd_workspace_size(batch, seqlen, n_q_heads, n_kv_heads, head_dim) -> int:
    return int(load().diffattn_v2_bwd_workspace_size(batch, seqlen, n_q_heads, n_kv_heads,
                                                     head_dim))


def diffattn_v2_bwd(q, k, v, dout, lam, *, causal=True, window=0, workspace=None,
                    out=None, dev_status=None, stream=None):
    """V2 gradients.  Returns dict of fp32 device tensors dq (like q), dk,
    dv (like k) and dlambda [Hq/2]; `out` may supply any of them."""
    _need_cuda(q, k, v, dout, lam)
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    if workspace is None:
        workspace = torch.empty(diffattn_v2_bwd_workspace_size(B, N, Hq, Hkv, d),
                                dtype=torch.uint8, device=q.device)
    f32 = dict(dtype=torch.float32, device=q.device)
    res = {"dq": torch.empty(q.shape, **f32), "dk": torch.empty(k.shape, **f32),
           "dv": torch.empty(v.shape, **f32), "dlambda": torch.empty(Hq // 2, **f32)}
    res.update(out or {})
    _check("diffattn_v2_bwd", load().diffattn_v2_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(lam), _dtype_code(q), B, N, Hq, Hkv, d,
        int(bool(causal)), int(window), _ptr(res["dq"]), _ptr(res["dk"]), _ptr(res["dv"]),
        _ptr(res["dlambda"]), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(dev_status), _stream(stream)))
    return res


# ---- training forward with saves, and the backward from the saves ----------
def _nbytes(t):
    return t.numel() * t.element_size()


def diffattn_v1_fwd_train(q, k, v, lam, *, causal=True, window=0, apply_norm=False,
                          norm_weight=None, norm_eps=1e-5, lambda_init=0.0, out=None,
                          saves=None, dev_status=None, stream=None):
    """V1 forward that also writes the saves the backward reads.  Returns
    (out, saves); saves is a uint8 device tensor (allocated here if None)."""
    _need_cuda(q, k, v, lam, norm_weight, dev_status)
    B, N, H, d2 = q.shape
    dvw = v.shape[-1]
    if saves is None:
        saves = torch.empty(int(load().diffattn_v1_fwd_train_saves_size(B, N, H)),
                            dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty(B, N, H, dvw, dtype=q.dtype, device=q.device)
    _check("diffattn_v1_fwd_train", load().diffattn_v1_fwd_train(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _dtype_code(q), B, N, H, d2 // 2, dvw, _ptr(lam),
        int(bool(causal)), int(window), int(bool(apply_norm)), _ptr(norm_weight),
        float(norm_eps), float(lambda_init), _ptr(saves), _nbytes(saves), _ptr(dev_status),
        _stream(stream)))
    return out, saves


def diffattn_v1_bwd_saved(q, k, v, dout, lam, saves, *, causal=True, window=0,
                          apply_norm=False, norm_weight=None, norm_eps=1e-5, lambda_init=0.0,
                          workspace=None, out=None, dev_status=None, stream=None):
    """V1 gradients from the saves of diffattn_v1_fwd_train (same dict as
    diffattn_v1_bwd)."""
    _need_cuda(q, k, v, dout, lam, saves, norm_weight)
    B, N, H, d2 = q.shape
    dvw = v.shape[-1]
    if workspace is None:
        workspace = torch.empty(int(load().diffattn_v1_bwd_saved_workspace_size(B, N, H)),
                                dtype=torch.uint8, device=q.device)
    f32 = dict(dtype=torch.float32, device=q.device)
    res = {"dq": torch.empty(q.shape, **f32), "dk": torch.empty(k.shape, **f32),
           "dv": torch.empty(v.shape, **f32), "dlambda": torch.empty(H, **f32),
           "dnorm_weight": torch.empty(dvw, **f32) if apply_norm else None}
    res.update(out or {})
    _check("diffattn_v1_bwd_saved", load().diffattn_v1_bwd_saved(
        _ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(lam), _dtype_code(q), B, N, H, d2 // 2,
        dvw, int(bool(causal)), int(window), int(bool(apply_norm)), _ptr(norm_weight),
        float(norm_eps), float(lambda_init), _ptr(saves), _nbytes(saves), _ptr(res["dq"]),
        _ptr(res["dk"]), _ptr(res["dv"]), _ptr(res["dlambda"]), _ptr(res["dnorm_weight"]),
        _ptr(workspace), _nbytes(workspace), _ptr(dev_status), _stream(stream)))
    return res


def diffattn_v2_prefill_train(q, k, v, lam, *, causal=True, window=0, out=None, saves=None,
                              dev_status=None, stream=None):
    """V2 prefill that also writes the saves the backward reads.  Returns
    (out, saves)."""
    _need_cuda(q, k, v, lam, dev_status)
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    if saves is None:
        saves = torch.empty(int(load().diffattn_v2_prefill_train_saves_size(B, N, Hq)),
                            dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty(B, N, Hq // 2, d, dtype=q.dtype, device=q.device)
    _check("diffattn_v2_prefill_train", load().diffattn_v2_prefill_train(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _dtype_code(q), B, N, Hq, Hkv, d, _ptr(lam),
        int(bool(causal)), int(window), _ptr(saves), _nbytes(saves), _ptr(dev_status),
        _stream(stream)))
    return out, saves


def diffattn_v2_bwd_saved(q, k, v, dout, lam, saves, *, causal=True, window=0, workspace=None,
                          out=None, dev_status=None, stream=None):
    """V2 gradients from the saves of diffattn_v2_prefill_train (same dict
    as diffattn_v2_bwd)."""
    _need_cuda(q, k, v, dout, lam, saves)
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    if workspace is None:
        workspace = torch.empty(int(load().diffattn_v2_bwd_saved_workspace_size(B, N, Hq)),
                                dtype=torch.uint8, device=q.device)
    f32 = dict(dtype=torch.float32, device=q.device)
    res = {"dq": torch.empty(q.shape, **f32), "dk": torch.empty(k.shape, **f32),
           "dv": torch.empty(v.shape, **f32), "dlambda": torch.empty(Hq // 2, **f32)}
    res.update(out or {})
    _check("diffattn_v2_bwd_saved", load().diffattn_v2_bwd_saved(
        _ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(lam), _dtype_code(q), B, N, Hq, Hkv, d,
        int(bool(causal)), int(window), _ptr(saves), _nbytes(saves), _ptr(res["dq"]),
        _ptr(res["dk"]), _ptr(res["dv"]), _ptr(res["dlambda"]), _ptr(workspace),
        _nbytes(workspace), _ptr(dev_status), _stream(stream)))
    return res


def lambda_from_params_bwd(lq1, lk1, lq2, lk2, dlambda, stream=None):
    """Gradients of the four lambda vectors: dict of fp32 [H, dim] tensors."""
    _need_cuda(lq1, lk1, lq2, lk2, dlambda)
    H, dim = lq1.shape
    outs = {n: torch.empty(H, dim, dtype=torch.float32, device=lq1.device)
            for n in ("dlq1", "dlk1", "dlq2", "dlk2")}
    _check("lambda_from_params_bwd", load().lambda_from_params_bwd(
        _ptr(lq1), _ptr(lk1), _ptr(lq2), _ptr(lk2), _ptr(dlambda), H, dim,
        *(_ptr(outs[n]) for n in ("dlq1", "dlk1", "dlq2", "dlk2")), _stream(stream)))
    return outs


# ---- V2 prefill + output projection ------------------------------------------
def diffattn_v2_prefill_oproj_workspace_size(batch, seqlen, n_q_heads, head_dim) -> int:
    return int(load().diffattn_v2_prefill_oproj_workspace_size(batch, seqlen, n_q_heads,
                                                                head_dim))


def diffattn_v2_prefill_oproj(q, k, v, lam, w_o, *, causal=True, window=0, workspace=None,
                              out=None, dev_status=None, stream=None):
    """V2 prefill followed by out = o . w_o.  q [B, N, Hq, d]; k, v
    [B, N, Hkv, d]; w_o [Hq/2 * d, d_model] bf16.  Returns [B, N, d_model]."""
    _need_cuda(q, k, v, lam, w_o, dev_status)
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    d_model = w_o.shape[1]
    if workspace is None:
        workspace = torch.empty(diffattn_v2_prefill_oproj_workspace_size(B, N, Hq, d),
                                dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty(B, N, d_model, dtype=q.dtype, device=q.device)
    _check("diffattn_v2_prefill_oproj", load().diffattn_v2_prefill_oproj(
        _ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(w_o), _ptr(out), _dtype_code(q), B, N, Hq,
        Hkv, d, d_model, int(bool(causal)), int(window), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream(stream)))
    return out


def diffattn_selftest_wait_timeout(timeout_us, dev_status, waited_ns=None, stream=None):
    """Run the bounded-wait path to its timeout (see the header); the status
    word then holds DA_ERR_DEVICE_TIMEOUT."""
    _need_cuda(dev_status, waited_ns)
    _check("diffattn_selftest_wait_timeout", load().diffattn_selftest_wait_timeout(
        int(timeout_us), _ptr(dev_status), _ptr(waited_ns), _stream(stream)))


# ---- serving: page plan, 4-bit paged cache, decode over it; QK norm + rotation
# These calls take microseconds on the GPU, as long as a few checks take here.
# So each call first asks in one expression whether all is as it should be, and
# only otherwise goes through the named checks, which say what is not; devices
# are compared by index, and switched only when the device is not the current.
_I32, _U8, _F32, _BF16 = torch.int32, torch.uint8, torch.float32, torch.bfloat16
_CODES = {_BF16: DA_BF16, _F32: DA_FP32}


def _need(name, t, dtype, shape=None):
    """A dense tensor of one type and shape (None: any)."""
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, not %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), shape))


def _one_device(first, *others):
    """Index of the device that all tensors of a call lie on."""
    at = first.get_device()
    if at < 0:
        raise ValueError("tensors must be CUDA tensors")
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError("tensors lie on different devices (cuda:%d, %s)" % (at, t.device))
    return at


def _run(fn, at, stream, *args):
    """Calls an entry point with device `at` current, on `stream` (None: that
    device's current stream)."""
    if torch._C._cuda_getDevice() != at:
        with torch.cuda.device(at):
            status = fn(*args, _stream(stream))
    else:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(at) if stream is None
                    else _stream(stream))
    if status != DA_OK:
        raise DiffAttnError(fn.__name__, status)


def _token_stride(name, t, tokens=None, dtype=None):
    """Token stride of t [T, H, d], whose heads of a token lie in a row."""
    if t.dim() != 3 or (tokens is not None and t.shape[0] != tokens):
        raise ValueError("%s must be [tokens, heads, width], got %s" % (name, tuple(t.shape)))
    if dtype is not None and t.dtype is not dtype:
        raise TypeError("%s must be %s, not %s" % (name, dtype, t.dtype))
    T, H, d = t.shape
    st, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (H > 1 and sh != d):
        raise ValueError("%s: the heads of a token must lie in a row" % name)
    return st if T > 1 else max(1, H) * d


def _code(name, t):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError("%s: unsupported dtype %s" % (name, t.dtype))
    return code


def _workspace(workspace, need, at, stream):
    if workspace is None:
        device = torch.device("cuda", at)
        workspace = torch.empty(max(need, 1), dtype=_U8, device=device)
        if stream is not None:   # freed on return: kept from reuse until that stream is past it
            workspace.record_stream(torch.cuda.ExternalStream(_stream(stream), device=device))
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def _kv4_cache(cache):
    """(pages, KV heads, page size) of a cache [n_pages, n_kv_heads, page_size * 144]."""
    if cache.dtype is not _U8 or not cache.is_contiguous():
        _need("cache", cache, _U8)
    if cache.dim() == 3:
        pages, heads, nbytes = cache.shape
        if nbytes % 144 == 0:
            return pages, heads, nbytes // 144
    raise ValueError("cache must be [n_pages, n_kv_heads, page_size * 144], not %s"
                     % (tuple(cache.shape),))


def _page_lists(first, cache_lens, block_table, free_pages, free_count):
    """(requests, max_pages, n_pages), all checked."""
    R = first.numel()
    if (first.dtype is _I32 and cache_lens.dtype is _I32 and block_table.dtype is _I32 and
            free_pages.dtype is _I32 and free_count.dtype is _I32 and first.is_contiguous() and
            cache_lens.is_contiguous() and block_table.is_contiguous() and
            free_pages.is_contiguous() and free_count.numel() == 1 and
            first.dim() == cache_lens.dim() == free_pages.dim() == free_count.dim() == 1 and
            cache_lens.numel() == R and block_table.dim() == 2):
        rows, max_pages = block_table.shape
        if rows == R:
            return R, max_pages, free_pages.numel()
    _need("new_lens or release", first, _I32, (R,))
    _need("cache_lens", cache_lens, _I32, (R,))
    _need("block_table", block_table, _I32)
    _need("free_pages", free_pages, _I32)
    _need("free_count", free_count, _I32, (1,))
    if block_table.dim() != 2 or block_table.shape[0] != R:
        raise ValueError("block_table must be [%d, max_pages], not %s"
                         % (R, tuple(block_table.shape)))
    if free_pages.dim() != 1:
        raise ValueError("free_pages must be [n_pages]")
    return R, block_table.shape[1], free_pages.shape[0]


def diffattn_page_plan_workspace_size(requests, n_slots) -> int:
    return int(load().diffattn_page_plan_workspace_size(requests, n_slots))


def diffattn_page_plan(new_lens, cache_lens, block_table, free_pages, free_count, page_size,
                       n_slots, *, out=None, workspace=None, dev_status=None, stream=None):
    """Pages, slots and positions of a step's new tokens.  new_lens,
    cache_lens int32 [R]; block_table int32 [R, max_pages] (new pages written
    in place); free_pages int32 [n_pages], a stack of which free_count int32
    [1] are free.  Returns a dict: slots, positions [n_slots], offsets
    [R + 1], served, cache_lens [R], free_count [1] (int32).  `out`, such a
    dict, is written instead of new tensors; its cache_lens and free_count
    may be the arguments themselves."""
    R, max_pages, n_pages = _page_lists(new_lens, cache_lens, block_table, free_pages, free_count)
    if n_slots < 0:
        raise ValueError("n_slots is negative")
    need = 0
    if workspace is None and n_slots > 1024:   # none below
        need = diffattn_page_plan_workspace_size(R, n_slots)
    if out is None:
        at = _one_device(new_lens, cache_lens, block_table, free_pages, free_count, workspace,
                         dev_status)
        slots, positions, offsets, served, lens, count = new_lens.new_empty(
            2 * n_slots + 3 * R + 2).split_with_sizes((n_slots, n_slots, R + 1, R, R, 1))
        out = {"slots": slots, "positions": positions, "offsets": offsets, "served": served,
               "cache_lens": lens, "free_count": count}
    else:
        for name, n in (("slots", n_slots), ("positions", n_slots), ("offsets", R + 1),
                        ("served", R), ("cache_lens", R), ("free_count", 1)):
            _need(name, out[name], _I32, (n,))
        slots, positions, offsets, served, lens, count = (out[name] for name in (
            "slots", "positions", "offsets", "served", "cache_lens", "free_count"))
        at = _one_device(new_lens, cache_lens, block_table, free_pages, free_count, workspace,
                         dev_status, slots, positions, offsets, served, lens, count)
    if need:
        workspace = _workspace(None, need, at, stream)
    _run((_lib or load()).diffattn_page_plan, at, stream, new_lens.data_ptr(), cache_lens.data_ptr(),
         block_table.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(), R, max_pages,
         n_pages, int(page_size), int(n_slots), slots.data_ptr(), positions.data_ptr(), offsets.data_ptr(),
         served.data_ptr(), lens.data_ptr(), count.data_ptr(), _ptr(workspace),
         0 if workspace is None else workspace.nbytes, _ptr(dev_status))
    return out


def diffattn_page_release(release, cache_lens, block_table, free_pages, free_count, page_size, *,
                          dev_status=None, stream=None):
    """Gives the pages of requests with release[r] != 0 back (int32 [R]);
    cache_lens, block_table, free_pages and free_count are changed in place."""
    R, max_pages, n_pages = _page_lists(release, cache_lens, block_table, free_pages, free_count)
    at = _one_device(release, cache_lens, block_table, free_pages, free_count, dev_status)
    _run((_lib or load()).diffattn_page_release, at, stream, release.data_ptr(), cache_lens.data_ptr(),
         block_table.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(), R, max_pages,
         n_pages, int(page_size), _ptr(dev_status))


def diffattn_kv4_page_bytes(n_kv_heads, head_dim, page_size) -> int:
    return int(load().diffattn_kv4_page_bytes(n_kv_heads, head_dim, page_size))


def diffattn_kv4_append(k, v, slots, cache, *, dev_status=None, stream=None):
    """Writes rows k, v [T, Hkv, 128] (bf16 or fp32; slices of a fused
    projection are taken as they are) into the 4-bit cache
    [n_pages, Hkv, page_size * 144] uint8 at slots int32 [T] (negative: skipped)."""
    if v.shape != k.shape:
        raise ValueError("k and v differ in shape")
    dtype = _code("k", k)
    ks, vs = _token_stride("k", k), _token_stride("v", v, None, k.dtype)
    T, H, d = k.shape
    if slots.dtype is not _I32 or slots.shape != (T,) or not slots.is_contiguous():
        _need("slots", slots, _I32, (T,))
    pages, heads, ps = _kv4_cache(cache)
    if heads != H:
        raise ValueError("cache holds %d heads, k %d" % (heads, H))
    at = _one_device(k, v, slots, cache, dev_status)
    _run((_lib or load()).diffattn_kv4_append, at, stream, k.data_ptr(), ks, v.data_ptr(), vs, dtype,
         slots.data_ptr(), T, H, d, cache.data_ptr(), pages, ps, _ptr(dev_status))
    return cache


def diffattn_kv4_read(cache, slots, *, out=None, dtype=torch.bfloat16, dev_status=None,
                      stream=None):
    """Rows (k, v) [T, Hkv, 128] held at slots int32 [T].  Rows of negative
    slots are left as they were in `out` = (k, v), or are 0 in new tensors."""
    pages, H, ps = _kv4_cache(cache)
    if slots.dtype is not _I32 or slots.dim() != 1 or not slots.is_contiguous():
        _need("slots", slots, _I32, (slots.numel(),))
    T = slots.shape[0]
    if out is None:
        out = tuple(torch.zeros(T, H, 128, dtype=dtype, device=cache.device) for _ in "kv")
    k, v = out
    code = _code("k", k)
    shape = (T, H, 128)
    if (v.dtype is not k.dtype or k.shape != shape or v.shape != shape or
            not k.is_contiguous() or not v.is_contiguous()):
        _need("k", k, k.dtype, shape)
        _need("v", v, k.dtype, shape)
    at = _one_device(cache, slots, k, v, dev_status)
    _run((_lib or load()).diffattn_kv4_read, at, stream, cache.data_ptr(), pages, ps, slots.data_ptr(), T, H, 128,
         k.data_ptr(), v.data_ptr(), code, _ptr(dev_status))
    return k, v


def diffattn_v2_decode_kv4_workspace_size(batch, n_q_heads, n_kv_heads) -> int:
    return int(load().diffattn_v2_decode_kv4_workspace_size(batch, n_q_heads, n_kv_heads))


def diffattn_v2_decode_kv4(q, cache, block_table, cache_lens, lam, *, window=0, workspace=None,
                           out=None, dev_status=None, stream=None):
    """V2 decode over the 4-bit cache.  q [B, Hq, 128] bf16; cache
    [n_pages, Hkv, page_size * 144] uint8; block_table int32 [B, max_pages];
    cache_lens int32 [B]; lam [Hq/2] fp32; out [B, Hq/2, 128]."""
    code = _code("q", q)
    B, Hq, d = q.shape
    _need("q", q, q.dtype)
    pages, Hkv, ps = _kv4_cache(cache)
    max_pages = _decode_lists(B, block_table, cache_lens, lam, Hq // 2)
    at = _one_device(q, cache, block_table, cache_lens, lam, workspace, out, dev_status)
    if out is None:
        out = q.new_empty((B, Hq // 2, d))
    else:
        _need("out", out, q.dtype, (B, Hq // 2, d))
    ws = _workspace(workspace, 0 if workspace is not None else
                    diffattn_v2_decode_kv4_workspace_size(B, Hq, Hkv), at, stream)
    _run((_lib or load()).diffattn_v2_decode_kv4, at, stream, q.data_ptr(), cache.data_ptr(), pages, ps,
         block_table.data_ptr(), max_pages, cache_lens.data_ptr(), int(window), out.data_ptr(), code, B,
         Hq, Hkv, d, lam.data_ptr(), ws.data_ptr(), ws.nbytes, _ptr(dev_status))
    return out


def _decode_lists(B, block_table, cache_lens, lam, n_lam):
    """max_pages of a decode's tables, all checked."""
    if (block_table.dtype is not _I32 or cache_lens.dtype is not _I32 or lam.dtype is not _F32 or
            cache_lens.shape != (B,) or lam.shape != (n_lam,) or
            not block_table.is_contiguous() or not cache_lens.is_contiguous() or
            not lam.is_contiguous()):
        _need("block_table", block_table, _I32)
        _need("cache_lens", cache_lens, _I32, (B,))
        _need("lam", lam, _F32, (n_lam,))
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [%d, max_pages], not %s"
                         % (B, tuple(block_table.shape)))
    return block_table.shape[1]


def diffattn_v1_decode_kv4_workspace_size(batch, n_heads) -> int:
    return int(load().diffattn_v1_decode_kv4_workspace_size(batch, n_heads))


def diffattn_v1_decode_kv4(q, cache, block_table, cache_lens, lam, *, window=0, apply_norm=False,
                           norm_weight=None, norm_eps=1e-5, lambda_init=0.0, workspace=None,
                           out=None, dev_status=None, stream=None):
    """V1 decode over the 4-bit cache.  q [B, H, 128] bf16 (two 64-wide
    branches); cache [n_pages, H, page_size * 144] uint8; out [B, H, 128]."""
    code = _code("q", q)
    B, H, d2 = q.shape
    _need("q", q, q.dtype)
    pages, heads, ps = _kv4_cache(cache)
    if heads != H:
        raise ValueError("cache holds %d heads, q %d" % (heads, H))
    max_pages = _decode_lists(B, block_table, cache_lens, lam, H)
    if norm_weight is not None:
        _need("norm_weight", norm_weight, _F32, (128,))
    at = _one_device(q, cache, block_table, cache_lens, lam, norm_weight, workspace, out,
                     dev_status)
    if out is None:
        out = torch.empty_like(q)
    else:
        _need("out", out, q.dtype, (B, H, 128))
    ws = _workspace(workspace, 0 if workspace is not None else
                    diffattn_v1_decode_kv4_workspace_size(B, H), at, stream)
    _run((_lib or load()).diffattn_v1_decode_kv4, at, stream, q.data_ptr(), cache.data_ptr(), pages, ps,
         block_table.data_ptr(), max_pages, cache_lens.data_ptr(), int(window), out.data_ptr(), code, B,
         H, d2 // 2, 128, lam.data_ptr(), int(bool(apply_norm)), _ptr(norm_weight), float(norm_eps),
         float(lambda_init), ws.data_ptr(), ws.nbytes, _ptr(dev_status))
    return out


def _norm_rope_args(q, k, positions, inv_freq, q_weight, k_weight):
    dtype = q.dtype
    code = _code("q", q)
    T, Hq, d = q.shape
    qs, sh, sd = q.stride()
    if sd != 1 or sh != d or T < 2:
        qs = _token_stride("q", q)
    Hk = ks = 0
    if k is not None:
        Tk, Hk, dk = k.shape
        ks, sh, sd = k.stride()
        if sd != 1 or sh != d or Tk != T or T < 2 or k.dtype is not dtype:
            ks = _token_stride("k", k, T, dtype)
        if dk != d:
            raise ValueError("q and k differ in width")
    if q_weight is not None and (q_weight.dtype is not _F32 or q_weight.shape != (d,) or
                                 not q_weight.is_contiguous()):
        _need("q_weight", q_weight, _F32, (d,))
    if k_weight is not None and (k_weight.dtype is not _F32 or k_weight.shape != (d,) or
                                 not k_weight.is_contiguous()):
        _need("k_weight", k_weight, _F32, (d,))
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        if (inv_freq.dtype is not _F32 or inv_freq.dim() != 1 or
                not inv_freq.is_contiguous()):
            _need("inv_freq", inv_freq, _F32, (rot // 2,))
    if positions is not None and (positions.dtype is not _I32 or positions.shape != (T,) or
                                  not positions.is_contiguous()):
        _need("positions", positions, _I32, (T,))
    return code, T, Hq, Hk, d, qs, ks, rot


def diffattn_qk_norm_rope(q, k, positions, inv_freq, *, q_weight=None, k_weight=None,
                          norm_eps=1e-6, interleaved=False, out=None, stream=None):
    """RMS norm of every head of q [T, Hq, d] and k [T, Hk, d] (bf16 or fp32;
    slices of a fused projection are taken as they are) with weights fp32 [d]
    (None: ones), then the rotation of the first 2 * len(inv_freq) features by
    positions int32 [T] * inv_freq fp32 (inv_freq None: no rotation).  k may
    be None.  Returns (q, k); `out` = (q, k) may be the arguments themselves."""
    code, T, Hq, Hk, d, qs, ks, rot = _norm_rope_args(q, k, positions, inv_freq, q_weight,
                                                      k_weight)
    ko, kos = None, 0
    if out is None:
        # dense, since a token's heads lie in a row and tokens do not overlap
        qo, qos = torch.empty_like(q), Hq * d
        if k is not None:
            ko, kos = torch.empty_like(k), Hk * d
        at = _one_device(q, k, positions, inv_freq, q_weight, k_weight)
    else:
        qo, ko = out
        if qo.shape != q.shape or (k is not None and ko.shape != k.shape):
            raise ValueError("outputs must have the inputs' shapes")
        qos = _token_stride("q out", qo, T, q.dtype)
        if k is not None:
            kos = _token_stride("k out", ko, T, q.dtype)
        at = _one_device(q, k, positions, inv_freq, q_weight, k_weight, qo, ko)
    _run((_lib or load()).diffattn_qk_norm_rope, at, stream, q.data_ptr(), qs, _ptr(k), ks, code, T, Hq, Hk, d,
         _ptr(q_weight), _ptr(k_weight), float(norm_eps), _ptr(positions), _ptr(inv_freq), rot,
         int(bool(interleaved)), qo.data_ptr(), qos, _ptr(ko), kos)
    return qo, ko


def diffattn_qk_norm_rope_bwd_workspace_size(tokens, n_q_heads, n_k_heads, head_dim) -> int:
    return int(load().diffattn_qk_norm_rope_bwd_workspace_size(tokens, n_q_heads, n_k_heads,
                                                               head_dim))


def diffattn_qk_norm_rope_bwd(q, k, dq_out, dk_out, positions, inv_freq, *, q_weight=None,
                              k_weight=None, norm_eps=1e-6, interleaved=False, workspace=None,
                              stream=None):
    """Gradients of diffattn_qk_norm_rope: q, k are its inputs, dq_out, dk_out
    (fp32) the gradients of its outputs.  Returns a dict of fp32 tensors: dq,
    dk, dq_weight, dk_weight (None where the input is None)."""
    code, T, Hq, Hk, d, qs, ks, rot = _norm_rope_args(q, k, positions, inv_freq, q_weight,
                                                      k_weight)
    if dq_out.shape != q.shape or (k is not None and dk_out.shape != k.shape):
        raise ValueError("the gradients must have the inputs' shapes")
    if dq_out.dtype is _F32 and dq_out.is_contiguous():
        gqs = Hq * d
    else:
        gqs = _token_stride("dq_out", dq_out, T, _F32)
    if k is None:
        gks = 0
    elif dk_out.dtype is _F32 and dk_out.is_contiguous():
        gks = Hk * d
    else:
        gks = _token_stride("dk_out", dk_out, T, _F32)
    at = _one_device(q, k, dq_out, dk_out, positions, inv_freq, q_weight, k_weight, workspace)
    r = {"dq": torch.empty_like(dq_out), "dk": None if k is None else torch.empty_like(dk_out),
         "dq_weight": None if q_weight is None else torch.empty_like(q_weight),
         "dk_weight": None if k is None or k_weight is None else torch.empty_like(k_weight)}
    ws = _workspace(workspace, 0 if workspace is not None else
                    diffattn_qk_norm_rope_bwd_workspace_size(T, Hq, Hk, d), at, stream)
    _run((_lib or load()).diffattn_qk_norm_rope_bwd, at, stream, q.data_ptr(), qs, _ptr(k), ks, code,
         dq_out.data_ptr(), gqs, _ptr(dk_out), gks, T, Hq, Hk, d, _ptr(q_weight), _ptr(k_weight),
         float(norm_eps), _ptr(positions), _ptr(inv_freq), rot, int(bool(interleaved)),
         r["dq"].data_ptr(), _ptr(r["dk"]), _ptr(r["dq_weight"]), _ptr(r["dk_weight"]),
         ws.data_ptr(), ws.nbytes)
    return r


def diffattn_reset_tile_counters(stream=None):
    """Free every tile counter of the tensor-core prefill on the current
    device (see the header)."""
    _check("diffattn_reset_tile_counters",
           load().diffattn_reset_tile_counters(_stream(stream)))


def diffattn_selftest_hold_tile_counter(slot, tag, count, stream=None):
    """Test hook: set tile counter `slot` to (tag, count) and make the next
    tensor-core prefill launch take it (see the header)."""
    _check("diffattn_selftest_hold_tile_counter", load().diffattn_selftest_hold_tile_counter(
        int(slot), int(tag), int(count), _stream(stream)))


def diffattn_selftest_keep_tile_counter(slot, tag, duration_ms, stream=None):
    """Test hook: keep tile counter `slot` held by `tag`, as a launch in
    flight would, for `duration_ms` (see the header)."""
    _check("diffattn_selftest_keep_tile_counter", load().diffattn_selftest_keep_tile_counter(
        int(slot), int(tag), int(duration_ms), _stream(stream)))
