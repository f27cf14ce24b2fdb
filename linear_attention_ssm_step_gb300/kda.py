"""Thin ctypes binding of libkda_gb300.so (include/kda.h, kda_fp8.h, kda_prefill.h, kda_paged.h,
kda_paged_fp8.h).

Argument marshalling only: torch tensors supply device pointers, strides and
the current CUDA stream; every step of the computation runs in the library's
kernels. There is no CPU or fallback path: if the library is missing or a
call is rejected, this module raises.
"""

import collections
import ctypes
import os

import torch

from . import _build

KDA_OK, KDA_EINVAL, KDA_EUNSUPPORTED, KDA_ELAUNCH = 0, 1, 2, 3
KDA_ERR_HIST_LEN = 1
KDA_ERR_TIMEOUT = 2
KDA_ERR_CACHE_BASE = 4
KDA_ERR_SEQLENS = 8
KDA_ERR_PAGES = 16
KDA_ERR_LENGTHS = 32
KDA_MAX_REQUESTS = 4096
KDA_ATTENTION_WORKSPACE_ZEROED = 4096
KDA_FP8_SCALE_TOKENS = 16
KDA_ROPE_PLAIN, KDA_ROPE_LINEAR, KDA_ROPE_BASE, KDA_ROPE_PARTS = 0, 1, 2, 3
KDA_MAX_T = 16
KDA_GATE_RAW, KDA_GATE_PRECOMPUTED = 0, 1
STATUS_NAMES = {0: "KDA_OK", 1: "KDA_EINVAL", 2: "KDA_EUNSUPPORTED", 3: "KDA_ELAUNCH"}


class KdaError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class KdaView(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("b_stride", ctypes.c_int64),
                ("t_stride", ctypes.c_int64), ("h_stride", ctypes.c_int64)]


class KdaParams(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("K", ctypes.c_int32),
        ("V", ctypes.c_int32), ("N", ctypes.c_int32),
        ("q", KdaView), ("k", KdaView), ("v", KdaView), ("g_raw", KdaView),
        ("beta_logit", KdaView),
        ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
        ("lower_bound", ctypes.c_float), ("scale", ctypes.c_float),
        ("state", ctypes.c_void_p), ("state_slot_stride", ctypes.c_int64),
        ("state_indices", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("out_b_stride", ctypes.c_int64),
        ("out_t_stride", ctypes.c_int64), ("out_h_stride", ctypes.c_int64),
        ("error_word", ctypes.c_void_p), ("config_override", ctypes.c_int32),
        ("gate_mode", ctypes.c_int32),
    ]


class KdaRingParams(ctypes.Structure):
    _fields_ = [
        ("k_cache", ctypes.c_void_p), ("u_cache", ctypes.c_void_p), ("g_cache", ctypes.c_void_p),
        ("k_slot_stride", ctypes.c_int64), ("u_slot_stride", ctypes.c_int64),
        ("g_slot_stride", ctypes.c_int64),
        ("hist_len", ctypes.c_void_p), ("W", ctypes.c_int32), ("flush_min", ctypes.c_int32),
        ("restart_hist_on_flush", ctypes.c_int32), ("cache_base", ctypes.c_void_p),
    ]


class KdaFp8Pool(ctypes.Structure):
    """kda_fp8_pool of include/kda_fp8.h."""

    _fields_ = [("scale", ctypes.c_void_p), ("scale_slot_stride", ctypes.c_int64)]


class KdaSeqs(ctypes.Structure):
    """kda_seqs of include/kda_prefill.h."""

    _fields_ = [("cu_seqlens", ctypes.c_void_p), ("num_seqs", ctypes.c_int32)]


class KdaPages(ctypes.Structure):
    """kda_pages of include/kda_paged.h."""

    _fields_ = [("ptr", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class KdaPagedCache(ctypes.Structure):
    """kda_paged_cache of include/kda_paged.h."""

    _fields_ = [("k", KdaPages), ("v", KdaPages), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class KdaPlanParams(ctypes.Structure):
    """kda_plan_params of include/kda_paged.h."""

    _fields_ = [
        ("num_requests", ctypes.c_int32), ("num_tokens", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("cached", ctypes.c_void_p), ("new_len", ctypes.c_void_p),
        ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int32),
        ("free_pages", ctypes.c_void_p), ("free_capacity", ctypes.c_int32),
        ("free_count", ctypes.c_void_p), ("free_count_out", ctypes.c_void_p),
        ("cu_new", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
        ("positions", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("error_word", ctypes.c_void_p),
    ]


class KdaRopeParams(ctypes.Structure):
    """kda_rope_params of include/kda_paged.h."""

    _fields_ = [
        ("num_tokens", ctypes.c_int32), ("num_q_heads", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32), ("mscale", ctypes.c_float),
        ("q", KdaView), ("k", KdaView), ("v", KdaView),
        ("q_out", ctypes.c_void_p), ("q_out_b_stride", ctypes.c_int64), ("q_out_h_stride", ctypes.c_int64),
        ("positions", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("freqs", ctypes.c_void_p),
        ("cache", KdaPagedCache), ("error_word", ctypes.c_void_p),
    ]


class KdaAttentionParams(ctypes.Structure):
    """kda_attention_params of include/kda_paged.h."""

    _fields_ = [
        ("num_requests", ctypes.c_int32), ("num_tokens", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
        ("window", ctypes.c_int32), ("scale", ctypes.c_float), ("q", KdaView),
        ("out", ctypes.c_void_p), ("out_b_stride", ctypes.c_int64), ("out_h_stride", ctypes.c_int64),
        ("lse", ctypes.c_void_p), ("cu_new", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
        ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int32),
        ("cache", KdaPagedCache), ("error_word", ctypes.c_void_p),
    ]


class KdaPageScales(ctypes.Structure):
    """kda_page_scales of include/kda_paged_fp8.h."""

    _fields_ = [("ptr", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("block_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class KdaPagedScales(ctypes.Structure):
    """kda_paged_scales of include/kda_paged_fp8.h."""

    _fields_ = [("k", KdaPageScales), ("v", KdaPageScales)]


class KdaReadParams(ctypes.Structure):
    """kda_read_params of include/kda_paged_fp8.h."""

    _fields_ = [
        ("num_requests", ctypes.c_int32), ("num_tokens", ctypes.c_int32),
        ("k_out", ctypes.c_void_p), ("k_out_b_stride", ctypes.c_int64), ("k_out_h_stride", ctypes.c_int64),
        ("v_out", ctypes.c_void_p), ("v_out_b_stride", ctypes.c_int64), ("v_out_h_stride", ctypes.c_int64),
        ("cu_rows", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
        ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int32),
        ("cache", KdaPagedCache), ("error_word", ctypes.c_void_p),
    ]


EXPORTS = {
    "kda_decode": ([ctypes.POINTER(KdaParams), ctypes.c_void_p], ctypes.c_int),
    "kda_decode_fp8": ([ctypes.POINTER(KdaParams), ctypes.POINTER(KdaFp8Pool), ctypes.c_void_p], ctypes.c_int),
    "kda_verify_fp8": ([ctypes.POINTER(KdaParams), ctypes.c_int32, ctypes.POINTER(KdaFp8Pool), ctypes.c_void_p],
                       ctypes.c_int),
    "kda_verify_ring_fp8": ([ctypes.POINTER(KdaParams), ctypes.c_int32, ctypes.POINTER(KdaRingParams),
                             ctypes.POINTER(KdaFp8Pool), ctypes.c_void_p], ctypes.c_int),
    "kda_verify": ([ctypes.POINTER(KdaParams), ctypes.c_int32, ctypes.c_void_p], ctypes.c_int),
    "kda_prefill": ([ctypes.POINTER(KdaParams), ctypes.POINTER(KdaSeqs), ctypes.c_void_p], ctypes.c_int),
    "kda_select_prefill_config": ([ctypes.c_int32, ctypes.c_int32], ctypes.c_int32),
    "kda_prefill_ws": ([ctypes.POINTER(KdaParams), ctypes.POINTER(KdaSeqs), ctypes.c_void_p, ctypes.c_size_t,
                        ctypes.c_void_p], ctypes.c_int),
    "kda_prefill_workspace_bytes": ([ctypes.c_int32, ctypes.c_int32, ctypes.c_int32], ctypes.c_size_t),
    "kda_prefill_static": ([ctypes.POINTER(KdaParams), ctypes.POINTER(KdaSeqs), ctypes.c_void_p], ctypes.c_int),
    "kda_select_prefill_ws_config": ([ctypes.c_int32, ctypes.c_int32, ctypes.c_int32], ctypes.c_int32),
    "kda_verify_ring": ([ctypes.POINTER(KdaParams), ctypes.c_int32, ctypes.POINTER(KdaRingParams),
                         ctypes.c_void_p], ctypes.c_int),
    "kda_num_configs": ([], ctypes.c_int32),
    "kda_config_tile_v": ([ctypes.c_int32], ctypes.c_int32),
    "kda_select_config": ([ctypes.c_int32, ctypes.c_int32], ctypes.c_int32),
    "kda_select_ring_config": ([ctypes.c_int32, ctypes.c_int32], ctypes.c_int32),
    "kda_last_error": ([], ctypes.c_char_p),
    "kda_paged_plan": ([ctypes.POINTER(KdaPlanParams), ctypes.c_void_p], ctypes.c_int),
    "kda_rope_append": ([ctypes.POINTER(KdaRopeParams), ctypes.c_void_p], ctypes.c_int),
    "kda_rope_freqs": ([ctypes.c_void_p, ctypes.c_int32, ctypes.c_double, ctypes.c_int32, ctypes.c_double,
                        ctypes.c_double, ctypes.c_double, ctypes.c_double], ctypes.c_int),
    "kda_paged_attention": ([ctypes.POINTER(KdaAttentionParams), ctypes.c_void_p, ctypes.c_size_t,
                             ctypes.c_void_p], ctypes.c_int),
    "kda_paged_attention_workspace_bytes": ([ctypes.c_int32], ctypes.c_size_t),
    "kda_rope_append_fp8": ([ctypes.POINTER(KdaRopeParams), ctypes.POINTER(KdaPagedScales), ctypes.c_void_p],
                            ctypes.c_int),
    "kda_paged_attention_fp8": ([ctypes.POINTER(KdaAttentionParams), ctypes.POINTER(KdaPagedScales), ctypes.c_void_p,
                                 ctypes.c_size_t, ctypes.c_void_p], ctypes.c_int),
    "kda_paged_read_fp8": ([ctypes.POINTER(KdaReadParams), ctypes.POINTER(KdaPagedScales), ctypes.c_void_p],
                           ctypes.c_int),
}

_lib = None


def lib_path():
    return _build.LIB_PATH


def bind_library(path):
    """Open a build of the library at `path` with the C signatures of EXPORTS set."""
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run __graft_entry__.build() first")
    lib = ctypes.CDLL(path)
    for name, (args, res) in EXPORTS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


def load_library():
    """Load libkda_gb300.so (built by __graft_entry__.build()); raise if it is absent."""
    global _lib
    if _lib is None:
        _lib = bind_library(lib_path())
    return _lib


def _check(status):
    if status != KDA_OK:
        raise KdaError(status, load_library().kda_last_error().decode())


def _need(t, name, dtype):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _view(t, name, has_T, D):
    """KdaView of [B, H, D] (has_T False) or [B, T, H, D]; D == 1 drops the last dim."""
    _need(t, name, torch.bfloat16)
    want = (3 if has_T else 2) + (1 if D > 1 else 0)
    if t.dim() != want:
        raise ValueError(f"{name} must have {want} dims, got shape {tuple(t.shape)}")
    if D > 1 and (t.shape[-1] != D or t.stride(-1) != 1):
        raise ValueError(f"{name} must have a contiguous last dim of {D}")
    s = t.stride()
    if has_T:
        return KdaView(t.data_ptr(), s[0], s[1], s[2])
    return KdaView(t.data_ptr(), s[0], 0, s[1])


def _stream_handle(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _empty(shape, dtype, device, stream):
    """What a call allocates for itself (its outputs, a workspace), from the pool of the call's stream: memory of the
    current stream's pool may still be in use by that stream's earlier work. The current stream, which may use it
    later, is noted, so that the memory is not handed out again while either stream has work with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if stream.cuda_stream != current.cuda_stream:
        t.record_stream(current)
    return t


def _params(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out, T,
            lower_bound, scale, error_word, config_override, gate_mode, state_dtype=torch.bfloat16,
            n_indices=None):
    has_T = T is not None
    B = q.shape[0]
    n_idx = B if n_indices is None else n_indices
    H = q.shape[-2]
    _need(state, "state", state_dtype)
    if state.dim() != 4 or state.shape[1:] != (H, 128, 128):
        raise ValueError(f"state must be [N, {H}, 128, 128], got {tuple(state.shape)}")
    if state.stride()[1:] != (128 * 128, 128, 1):
        raise ValueError("each state slot must be contiguous [H][V][K]")
    _need(state_indices, "state_indices", torch.int32)
    if state_indices.shape != (n_idx,) or (n_idx > 0 and state_indices.stride(0) != 1):
        raise ValueError(f"state_indices must be a contiguous [{n_idx}] tensor")
    if gate_mode == KDA_GATE_RAW or A_log is not None:
        _need(A_log, "A_log", torch.float32)
        if A_log.numel() != H or not A_log.is_contiguous():
            raise ValueError("A_log must be a contiguous [H] tensor")
    if gate_mode == KDA_GATE_RAW or dt_bias is not None:
        _need(dt_bias, "dt_bias", torch.float32)
        if dt_bias.numel() != H * 128 or not dt_bias.is_contiguous():
            raise ValueError("dt_bias must be a contiguous [H, 128] tensor")
    _need(out, "out", torch.bfloat16)
    if out.stride(-1) != 1:
        raise ValueError("out must have a contiguous last dim")
    so = out.stride()
    p = KdaParams()
    p.B, p.H, p.K, p.V, p.N = B, H, 128, 128, state.shape[0]
    p.q = _view(q, "q", has_T, 128)
    p.k = _view(k, "k", has_T, 128)
    p.v = _view(v, "v", has_T, 128)
    p.g_raw = _view(g_raw, "g_raw", has_T, 128)
    p.beta_logit = _view(beta_logit, "beta_logit", has_T, 1)
    p.A_log = None if A_log is None else A_log.data_ptr()
    p.dt_bias = None if dt_bias is None else dt_bias.data_ptr()
    p.lower_bound = lower_bound
    p.scale = scale
    p.state = state.data_ptr()
    p.state_slot_stride = state.stride(0)
    p.state_indices = state_indices.data_ptr()
    p.out = out.data_ptr()
    if has_T:
        p.out_b_stride, p.out_t_stride, p.out_h_stride = so[0], so[1], so[2]
    else:
        p.out_b_stride, p.out_t_stride, p.out_h_stride = so[0], 0, so[1]
    if error_word is not None:
        _need(error_word, "error_word", torch.int32)
        p.error_word = error_word.data_ptr()
    p.config_override = config_override
    p.gate_mode = gate_mode
    return p


def kda_decode(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out=None,
               lower_bound=-5.0, scale=1.0, error_word=None, config_override=-1, gate_mode=KDA_GATE_RAW,
               stream=None):
    """T=1 decode. q, k, v, g_raw: bf16 [B, H, 128] views (any row and head stride);
    beta_logit: bf16 [B, H]; state: bf16 [N, H, 128, 128] pool updated in place;
    returns out bf16 [B, H, 128]. With gate_mode=KDA_GATE_PRECOMPUTED, g_raw holds
    log-space g, beta_logit holds beta, and A_log / dt_bias may be None."""
    if out is None:
        out = _empty((q.shape[0], q.shape[1], 128), torch.bfloat16, q.device, stream)
    p = _params(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out, None,
                lower_bound, scale, error_word, config_override, gate_mode)
    _check(load_library().kda_decode(ctypes.byref(p), _stream_handle(stream, q.device)))
    return out


class PreparedCall:
    """A library call bound to fixed tensors: argument checks and the C parameter
    struct are done once, and each call() launches the kernel on the tensors'
    current contents, on the stream given (or current) at preparation. The bound
    tensors must stay alive and keep their storage; `out` is the output tensor.
    For serving loops that refill the same input buffers every step."""

    def __init__(self, fn, args, out, keep):
        self._fn, self._args = fn, args  # ctypes arguments, structs passed by reference
        self.out = out
        self._keep = keep  # the structs and bound tensors, kept alive with the call

    def __call__(self):
        _check(self._fn(*self._args))
        return self.out


def prepare_decode(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out=None,
                   lower_bound=-5.0, scale=1.0, error_word=None, config_override=-1, gate_mode=KDA_GATE_RAW,
                   stream=None):
    """kda_decode bound to these tensors (see PreparedCall); same arguments."""
    if out is None:
        out = _empty((q.shape[0], q.shape[1], 128), torch.bfloat16, q.device, stream)
    p = _params(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out, None,
                lower_bound, scale, error_word, config_override, gate_mode)
    keep = (p, state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, error_word)
    return PreparedCall(load_library().kda_decode, (ctypes.byref(p), _stream_handle(stream, q.device)), out, keep)


def kda_decode_fp8(codes, scales, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out=None,
                   lower_bound=-5.0, scale=1.0, error_word=None, config_override=-1, gate_mode=KDA_GATE_RAW,
                   stream=None):
    """T=1 decode on an fp8 state pool (include/kda_fp8.h): codes uint8
    [N, H, 128, 128] (E4M3) and scales fp32 [N, H, 128] (powers of two), both
    updated in place for active rows; other arguments as kda_decode."""
    if out is None:
        out = _empty((q.shape[0], q.shape[1], 128), torch.bfloat16, q.device, stream)
    p = _params(codes, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out, None,
                lower_bound, scale, error_word, config_override, gate_mode, state_dtype=torch.uint8)
    f = _fp8_pool(codes, scales)
    _check(load_library().kda_decode_fp8(ctypes.byref(p), ctypes.byref(f), _stream_handle(stream, q.device)))
    return out


def kda_verify_fp8(codes, scales, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out=None,
                   lower_bound=-5.0, scale=1.0, error_word=None, config_override=-1, gate_mode=KDA_GATE_RAW,
                   stream=None):
    """T-token verify on an fp8 state pool (include/kda_fp8.h): the pool as for
    kda_decode_fp8, the token views and output as for kda_verify
    ([B, T, H, 128]); equal to T kda_decode_fp8 calls, bit for bit."""
    B, T, H = q.shape[0], q.shape[1], q.shape[2]
    if out is None:
        out = _empty((B, T, H, 128), torch.bfloat16, q.device, stream)
    p = _params(codes, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out, T,
                lower_bound, scale, error_word, config_override, gate_mode, state_dtype=torch.uint8)
    f = _fp8_pool(codes, scales)
    _check(load_library().kda_verify_fp8(ctypes.byref(p), T, ctypes.byref(f), _stream_handle(stream, q.device)))
    return out


def kda_verify_ring_fp8(codes, scales, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias,
                        k_cache, u_cache, g_cache, hist_len, flush_min, restart_hist_on_flush=True,
                        out=None, lower_bound=-5.0, scale=1.0, error_word=None, config_override=-1,
                        gate_mode=KDA_GATE_RAW, stream=None, cache_base=None):
    """Ring-cache verify with replay and fold on an fp8 checkpoint pool
    (include/kda_fp8.h): codes and scales as kda_decode_fp8's (a fold
    requantizes the checkpoint in place), the ring and the rest as
    kda_verify_ring's."""
    B, T, H = q.shape[0], q.shape[1], q.shape[2]
    if out is None:
        out = _empty((B, T, H, 128), torch.bfloat16, q.device, stream)
    p = _params(codes, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out, T,
                lower_bound, scale, error_word, config_override, gate_mode, state_dtype=torch.uint8)
    r = _ring_params(codes, H, k_cache, u_cache, g_cache, hist_len, flush_min, restart_hist_on_flush, cache_base)
    f = _fp8_pool(codes, scales)
    _check(load_library().kda_verify_ring_fp8(ctypes.byref(p), T, ctypes.byref(r), ctypes.byref(f),
                                              _stream_handle(stream, q.device)))
    return out


def _fp8_pool(codes, scales):
    _need(scales, "scales", torch.float32)
    if scales.dim() != 3 or scales.shape != codes.shape[:3] or scales.stride()[1:] != (128, 1):
        raise ValueError(f"scales must be [N, H, 128] with contiguous slots, got {tuple(scales.shape)}")
    return KdaFp8Pool(scales.data_ptr(), scales.stride(0))


def prepare_decode_fp8(codes, scales, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out=None,
                       lower_bound=-5.0, scale=1.0, error_word=None, config_override=-1, gate_mode=KDA_GATE_RAW,
                       stream=None):
    """kda_decode_fp8 bound to these tensors (see PreparedCall); same arguments."""
    if out is None:
        out = _empty((q.shape[0], q.shape[1], 128), torch.bfloat16, q.device, stream)
    p = _params(codes, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out, None,
                lower_bound, scale, error_word, config_override, gate_mode, state_dtype=torch.uint8)
    f = _fp8_pool(codes, scales)
    keep = (p, f, codes, scales, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, error_word)
    args = (ctypes.byref(p), ctypes.byref(f), _stream_handle(stream, q.device))
    return PreparedCall(load_library().kda_decode_fp8, args, out, keep)


def kda_verify(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out=None,
               lower_bound=-5.0, scale=1.0, error_word=None, config_override=-1, gate_mode=KDA_GATE_RAW,
               stream=None):
    """T-token verify. q, k, v, g_raw: bf16 [B, T, H, 128]; beta_logit: bf16 [B, T, H];
    returns out bf16 [B, T, H, 128]."""
    B, T, H = q.shape[0], q.shape[1], q.shape[2]
    if out is None:
        out = _empty((B, T, H, 128), torch.bfloat16, q.device, stream)
    p = _params(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out, T,
                lower_bound, scale, error_word, config_override, gate_mode)
    _check(load_library().kda_verify(ctypes.byref(p), T, _stream_handle(stream, q.device)))
    return out


def prepare_verify(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out=None,
                   lower_bound=-5.0, scale=1.0, error_word=None, config_override=-1, gate_mode=KDA_GATE_RAW,
                   stream=None):
    """kda_verify bound to these tensors (see PreparedCall); same arguments."""
    B, T, H = q.shape[0], q.shape[1], q.shape[2]
    if out is None:
        out = _empty((B, T, H, 128), torch.bfloat16, q.device, stream)
    p = _params(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out, T,
                lower_bound, scale, error_word, config_override, gate_mode)
    keep = (p, state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, error_word)
    return PreparedCall(load_library().kda_verify, (ctypes.byref(p), T, _stream_handle(stream, q.device)), out,
                        keep)


def kda_verify_ring(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias,
                    k_cache, u_cache, g_cache, hist_len, flush_min, restart_hist_on_flush=True,
                    out=None, lower_bound=-5.0, scale=1.0, error_word=None, config_override=-1,
                    gate_mode=KDA_GATE_RAW, stream=None, cache_base=None):
    """Ring-cache verify with replay and fold. k_cache, u_cache: bf16 [N, H, W, 128];
    g_cache: fp32 [N, H, W, 128]; hist_len: int32 [N]; cache_base: optional int32 [N]
    (ring position P of slot n is entry (cache_base[n] + P) mod W). Returns out
    bf16 [B, T, H, 128]."""
    B, T, H = q.shape[0], q.shape[1], q.shape[2]
    if out is None:
        out = _empty((B, T, H, 128), torch.bfloat16, q.device, stream)
    p = _params(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out, T,
                lower_bound, scale, error_word, config_override, gate_mode)
    r = _ring_params(state, H, k_cache, u_cache, g_cache, hist_len, flush_min, restart_hist_on_flush, cache_base)
    _check(load_library().kda_verify_ring(ctypes.byref(p), T, ctypes.byref(r),
                                          _stream_handle(stream, q.device)))
    return out


def prepare_verify_ring(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias,
                        k_cache, u_cache, g_cache, hist_len, flush_min, restart_hist_on_flush=True,
                        out=None, lower_bound=-5.0, scale=1.0, error_word=None, config_override=-1,
                        gate_mode=KDA_GATE_RAW, stream=None, cache_base=None):
    """kda_verify_ring bound to these tensors (see PreparedCall); same arguments."""
    B, T, H = q.shape[0], q.shape[1], q.shape[2]
    if out is None:
        out = _empty((B, T, H, 128), torch.bfloat16, q.device, stream)
    p = _params(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out, T,
                lower_bound, scale, error_word, config_override, gate_mode)
    r = _ring_params(state, H, k_cache, u_cache, g_cache, hist_len, flush_min, restart_hist_on_flush, cache_base)
    keep = (p, r, state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, k_cache, u_cache, g_cache,
            hist_len, cache_base, error_word)
    args = (ctypes.byref(p), T, ctypes.byref(r), _stream_handle(stream, q.device))
    return PreparedCall(load_library().kda_verify_ring, args, out, keep)


def _ring_params(state, H, k_cache, u_cache, g_cache, hist_len, flush_min, restart_hist_on_flush, cache_base):
    _need(k_cache, "k_cache", torch.bfloat16)
    _need(u_cache, "u_cache", torch.bfloat16)
    _need(g_cache, "g_cache", torch.float32)
    _need(hist_len, "hist_len", torch.int32)
    W = k_cache.shape[2]
    for name, t in (("k_cache", k_cache), ("u_cache", u_cache), ("g_cache", g_cache)):
        if t.dim() != 4 or t.shape[1:] != (H, W, 128) or t.stride()[1:] != (W * 128, 128, 1):
            raise ValueError(f"{name} must be [N, {H}, {W}, 128] with contiguous slots")
    if hist_len.shape != (state.shape[0],) or not hist_len.is_contiguous():
        raise ValueError("hist_len must be a contiguous [N] tensor")
    if cache_base is not None:
        _need(cache_base, "cache_base", torch.int32)
        if cache_base.shape != (state.shape[0],) or not cache_base.is_contiguous():
            raise ValueError("cache_base must be a contiguous [N] tensor")
    r = KdaRingParams()
    r.k_cache, r.u_cache, r.g_cache = k_cache.data_ptr(), u_cache.data_ptr(), g_cache.data_ptr()
    r.k_slot_stride, r.u_slot_stride, r.g_slot_stride = k_cache.stride(0), u_cache.stride(0), g_cache.stride(0)
    r.hist_len = hist_len.data_ptr()
    r.W, r.flush_min, r.restart_hist_on_flush = W, flush_min, int(bool(restart_hist_on_flush))
    r.cache_base = None if cache_base is None else cache_base.data_ptr()
    return r


def kda_prefill(state, state_indices, cu_seqlens, q, k, v, g_raw, beta_logit, A_log, dt_bias, out=None,
                lower_bound=-5.0, scale=1.0, error_word=None, config_override=-1, gate_mode=KDA_GATE_RAW,
                stream=None, workspace=None):
    """Varlen prefill (include/kda_prefill.h). q, k, v, g_raw: bf16 [L, H, 128]
    views with one row per token (any row and head stride); beta_logit: bf16
    [L, H]; cu_seqlens: int32 [S + 1] on the device, sequence i owning rows
    cu_seqlens[i] .. cu_seqlens[i+1]-1; state_indices: int32 [S], one slot per
    sequence; state: bf16 [N, H, 128, 128] pool, read as each sequence's
    initial state and overwritten with its final state. Returns out bf16
    [L, H, 128] (rows no sequence covers are left as they were).
    workspace: None (kda_prefill, configurations 0-4) or a device byte tensor
    of at least prefill_workspace_bytes(L, S, H) (kda_prefill_ws, which may
    then choose the two-stage configuration 5)."""
    if out is None:
        out = _empty((q.shape[0], q.shape[1], 128), torch.bfloat16, q.device, stream)
    fn, args, _ = _prefill_call(state, state_indices, cu_seqlens, q, k, v, g_raw, beta_logit, A_log, dt_bias,
                                out, lower_bound, scale, error_word, config_override, gate_mode, stream, workspace)
    _check(fn(*args))
    return out


def _prefill_call(state, state_indices, cu_seqlens, q, k, v, g_raw, beta_logit, A_log, dt_bias, out,
                  lower_bound, scale, error_word, config_override, gate_mode, stream, workspace):
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous [S + 1] tensor")
    S = cu_seqlens.shape[0] - 1
    p = _params(state, state_indices, q, k, v, g_raw, beta_logit, A_log, dt_bias, out, None,
                lower_bound, scale, error_word, config_override, gate_mode, n_indices=S)
    sq = KdaSeqs(cu_seqlens.data_ptr(), S)
    keep = (p, sq, state, state_indices, cu_seqlens, q, k, v, g_raw, beta_logit, A_log, dt_bias, error_word,
            workspace)
    lib = load_library()
    handle = _stream_handle(stream, q.device)
    if workspace is None:
        return lib.kda_prefill, (ctypes.byref(p), ctypes.byref(sq), handle), keep
    _need(workspace, "workspace", torch.uint8)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous byte tensor")
    return lib.kda_prefill_ws, (ctypes.byref(p), ctypes.byref(sq), workspace.data_ptr(), workspace.numel(),
                                handle), keep


def prepare_prefill(state, state_indices, cu_seqlens, q, k, v, g_raw, beta_logit, A_log, dt_bias, out=None,
                    lower_bound=-5.0, scale=1.0, error_word=None, config_override=-1, gate_mode=KDA_GATE_RAW,
                    stream=None, workspace=None):
    """kda_prefill bound to these tensors (see PreparedCall); same arguments. The
    sequence count is fixed by cu_seqlens' length; its contents may change."""
    if out is None:
        out = _empty((q.shape[0], q.shape[1], 128), torch.bfloat16, q.device, stream)
    fn, args, keep = _prefill_call(state, state_indices, cu_seqlens, q, k, v, g_raw, beta_logit, A_log, dt_bias,
                                   out, lower_bound, scale, error_word, config_override, gate_mode, stream,
                                   workspace)
    return PreparedCall(fn, args, out, keep)


def prefill_workspace_bytes(B, num_seqs, H):
    """Bytes of the workspace kda_prefill_ws needs (include/kda_prefill.h)."""
    return int(load_library().kda_prefill_workspace_bytes(B, num_seqs, H))


def prefill_workspace(B, num_seqs, H, device):
    """A device workspace for prefill calls of up to B token rows and num_seqs sequences of H heads."""
    return torch.empty(max(16, prefill_workspace_bytes(B, num_seqs, H)), dtype=torch.uint8, device=device)


def kda_select_prefill_ws_config(B, num_seqs, H=12):
    return int(load_library().kda_select_prefill_ws_config(B, num_seqs, H))


def kda_select_prefill_config(num_seqs, H=12):
    return int(load_library().kda_select_prefill_config(num_seqs, H))


def kda_select_config(B, T=1):
    return load_library().kda_select_config(B, T)


def kda_select_ring_config(B, T=8):
    return load_library().kda_select_ring_config(B, T)


def kda_num_configs():
    return load_library().kda_num_configs()


def kda_config_tile_v(config):
    return load_library().kda_config_tile_v(config)


def kda_last_error():
    return load_library().kda_last_error().decode()


def _ints(t, name, shape):
    _need(t, name, torch.int32)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor, got {tuple(t.shape)}")
    return t.data_ptr()


def _error_word(error_word):
    if error_word is None:
        return None
    _need(error_word, "error_word", torch.int32)
    return error_word.data_ptr()


def _table(block_table, num_requests):
    _need(block_table, "block_table", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] != num_requests or (
            num_requests > 0 and block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError(f"block_table must be [{num_requests}, pages] with contiguous rows, "
                         f"got {tuple(block_table.shape)}")
    return block_table.data_ptr(), block_table.stride(0), block_table.shape[1]


def _paged_cache(k_cache, v_cache, num_heads=None, head_dim=None, dtype=torch.bfloat16):
    """KdaPagedCache of k_cache and v_cache, views [pages, page_size, heads, head_dim] with any strides."""
    c = KdaPagedCache()
    kind = "codes" if dtype == torch.uint8 else "cache"
    for name, t in (("k_" + kind, k_cache), ("v_" + kind, v_cache)):
        _need(t, name, dtype)
        if t.dim() != 4 or (t.shape[3] > 1 and t.stride(3) != 1):
            raise ValueError(f"{name} must be [pages, page_size, heads, head_dim] with a contiguous last dim")
        if t.shape != k_cache.shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, k_{kind} {tuple(k_cache.shape)}")
        if (num_heads is not None and t.shape[2] != num_heads) or (head_dim is not None and t.shape[3] != head_dim):
            raise ValueError(f"{name} must have heads of {head_dim}, got {tuple(t.shape)}")
    c.k = KdaPages(k_cache.data_ptr(), *k_cache.stride()[:3])
    c.v = KdaPages(v_cache.data_ptr(), *v_cache.stride()[:3])
    c.num_pages, c.page_size, c.num_heads, c.head_dim = k_cache.shape
    return c


def _scales(k_scales, v_scales, cache):
    """KdaPagedScales of fp32 views [pages, blocks of 16 tokens a page, heads] with any strides."""
    blocks = -(-cache.page_size // KDA_FP8_SCALE_TOKENS)
    want = (cache.num_pages, blocks, cache.num_heads)
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        _need(t, name, torch.float32)
        if tuple(t.shape) != want:
            raise ValueError(f"{name} must be {list(want)} (pages, blocks of {KDA_FP8_SCALE_TOKENS} tokens, heads), "
                             f"got {tuple(t.shape)}")
    return KdaPagedScales(KdaPageScales(k_scales.data_ptr(), *k_scales.stride()),
                          KdaPageScales(v_scales.data_ptr(), *v_scales.stride()))


def _rows(t, name, num_tokens=None, num_heads=None, head_dim=None):
    _need(t, name, torch.bfloat16)
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name} must be [tokens, heads, head_dim] with a contiguous last dim")
    for got, want in zip(t.shape, (num_tokens, num_heads, head_dim)):
        if want is not None and got != want:
            raise ValueError(f"{name} must be [{num_tokens}, {num_heads or 'heads'}, {head_dim}], got {tuple(t.shape)}")
    return KdaView(t.data_ptr(), t.stride(0), 0, t.stride(1))


PagedPlan = collections.namedtuple("PagedPlan", "cu_new kv_len positions slots free_count")


def prepare_paged_plan(cached, new_len, block_table, free_pages, free_count, page_size, num_pages, num_tokens,
                       out=None, error_word=None, stream=None):
    """kda_paged_plan bound to these tensors (see PreparedCall); same arguments. out is its PagedPlan."""
    _need(cached, "cached", torch.int32)
    R = cached.shape[0] if cached.dim() == 1 else -1
    p = KdaPlanParams()
    p.num_requests, p.num_tokens, p.page_size, p.num_pages = R, num_tokens, page_size, num_pages
    p.cached, p.new_len = _ints(cached, "cached", (R,)), _ints(new_len, "new_len", (R,))
    p.table, p.table_stride, p.table_width = _table(block_table, R)
    _need(free_pages, "free_pages", torch.int32)
    p.free_pages, p.free_capacity = _ints(free_pages, "free_pages", (free_pages.numel(),)), free_pages.numel()
    p.free_count = _ints(free_count, "free_count", (1,))
    if out is None:
        new = lambda n: _empty(n, torch.int32, cached.device, stream)  # noqa: E731
        out = PagedPlan(new(R + 1), new(R), new(num_tokens), new(num_tokens), new(1))
    p.cu_new, p.kv_len = _ints(out.cu_new, "out.cu_new", (R + 1,)), _ints(out.kv_len, "out.kv_len", (R,))
    p.positions = _ints(out.positions, "out.positions", (num_tokens,))
    p.slots = _ints(out.slots, "out.slots", (num_tokens,))
    p.free_count_out = _ints(out.free_count, "out.free_count", (1,))
    p.error_word = _error_word(error_word)
    keep = (p, cached, new_len, block_table, free_pages, free_count, error_word)
    return PreparedCall(load_library().kda_paged_plan, (ctypes.byref(p), _stream_handle(stream, cached.device)), out,
                        keep)


def kda_paged_plan(cached, new_len, block_table, free_pages, free_count, page_size, num_pages, num_tokens,
                   out=None, error_word=None, stream=None):
    """The page plan of a step (include/kda_paged.h). cached, new_len: int32 [R],
    tokens each request has in the cache and brings; block_table: int32 [R, W],
    updated in place; free_pages: int32 list of free pages, of which the first
    free_count[0] are free (taken from the end); num_tokens: rows of positions
    and slots (at least the sum of new_len; rows beyond it get -1). Returns
    PagedPlan(cu_new [R + 1], kv_len [R], positions, slots [num_tokens],
    free_count [1]), all int32; pass the returned free_count to the next call.
    Pages of tokens that are not kept (rejected drafts, requests that end) are
    put back at the end of the free list by the caller, before the next call."""
    return prepare_paged_plan(cached, new_len, block_table, free_pages, free_count, page_size, num_pages, num_tokens,
                              out, error_word, stream)()


def rope_freqs(rotary_dim, base=10000.0, scaling=KDA_ROPE_PLAIN, factor=1.0, original_len=0.0, low=1.0, high=32.0,
               device="cuda"):
    """kda_rope_freqs as an int64 device tensor [rotary_dim / 2] for kda_rope_append
    (the bits of the library's uint64 turns per position)."""
    host = torch.empty(max(1, rotary_dim // 2), dtype=torch.int64)
    _check(load_library().kda_rope_freqs(host.data_ptr(), rotary_dim, base, scaling, factor, original_len, low, high))
    return host.to(device)


def prepare_rope_append(q, k, v, positions, slots, freqs, k_cache, v_cache, q_out=None, interleaved=False, mscale=1.0,
                        error_word=None, stream=None):
    """kda_rope_append bound to these tensors (see PreparedCall); same arguments. out is q_out."""
    p, q_out, keep = _rope_params(q, k, v, positions, slots, freqs, k_cache, v_cache, q_out, interleaved, mscale,
                                  error_word, stream, torch.bfloat16)
    return PreparedCall(load_library().kda_rope_append, (ctypes.byref(p), _stream_handle(stream, q.device)), q_out,
                        keep)


def _rope_params(q, k, v, positions, slots, freqs, k_cache, v_cache, q_out, interleaved, mscale, error_word, stream,
                 dtype):
    p = KdaRopeParams()
    p.q = _rows(q, "q")
    T, Hq, D = q.shape
    p.cache = _paged_cache(k_cache, v_cache, head_dim=D, dtype=dtype)
    Hkv = p.cache.num_heads
    p.num_tokens, p.num_q_heads = T, Hq
    p.k, p.v = _rows(k, "k", T, Hkv, D), _rows(v, "v", T, Hkv, D)
    if q_out is None:
        q_out = _empty((T, Hq, D), torch.bfloat16, q.device, stream)
    o = _rows(q_out, "q_out", T, Hq, D)
    p.q_out, p.q_out_b_stride, p.q_out_h_stride = o.ptr, o.b_stride, o.h_stride
    p.positions, p.slots = _ints(positions, "positions", (T,)), _ints(slots, "slots", (T,))
    _need(freqs, "freqs", torch.int64)
    if freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous [rotary_dim / 2] tensor")
    p.freqs, p.rotary_dim = freqs.data_ptr(), 2 * freqs.shape[0]
    p.interleaved, p.mscale = int(bool(interleaved)), mscale
    p.error_word = _error_word(error_word)
    return p, q_out, (p, q, k, v, positions, slots, freqs, k_cache, v_cache, error_word)


def kda_rope_append(q, k, v, positions, slots, freqs, k_cache, v_cache, q_out=None, interleaved=False, mscale=1.0,
                    error_word=None, stream=None):
    """Rotary positions and the append to the cache (include/kda_paged.h). q: bf16
    [T, Hq, D]; k, v: bf16 [T, Hkv, D] (any row and head strides); positions,
    slots: int32 [T] (kda_paged_plan's); freqs: int64 [rotary_dim / 2]
    (rope_freqs); k_cache, v_cache: bf16 [pages, page_size, Hkv, D] views with
    any strides, written at the slots. Returns q_out bf16 [T, Hq, D] (q itself
    turns in place)."""
    return prepare_rope_append(q, k, v, positions, slots, freqs, k_cache, v_cache, q_out, interleaved, mscale,
                               error_word, stream)()


def paged_attention_workspace_bytes(head_dim):
    """Bytes of the workspace kda_paged_attention needs (include/kda_paged.h)."""
    return int(load_library().kda_paged_attention_workspace_bytes(head_dim))


def paged_attention_workspace(head_dim, device, stream=None):
    """A device workspace for kda_paged_attention calls on one stream (the current one when None), with the part that
    its first use needs zeroed there. Calls on a stream other than that one must be ordered behind the zeroing."""
    device = torch.device(device)
    with torch.cuda.device(device):
        ws = _empty(max(16, paged_attention_workspace_bytes(head_dim)), torch.uint8, device, stream)
        with torch.cuda.stream(stream):  # no change when None
            ws[:KDA_ATTENTION_WORKSPACE_ZEROED].zero_()
        return ws


def prepare_paged_attention(q, k_cache, v_cache, block_table, cu_new, kv_len, out=None, lse=None, scale=None,
                            window=0, workspace=None, error_word=None, stream=None):
    """kda_paged_attention bound to these tensors (see PreparedCall); same arguments."""
    p, out, workspace, keep = _attention_params(q, k_cache, v_cache, block_table, cu_new, kv_len, out, lse, scale,
                                                window, workspace, error_word, stream, torch.bfloat16)
    args = (ctypes.byref(p), workspace.data_ptr(), workspace.numel(), _stream_handle(stream, q.device))
    return PreparedCall(load_library().kda_paged_attention, args, out, keep)


def _attention_params(q, k_cache, v_cache, block_table, cu_new, kv_len, out, lse, scale, window, workspace, error_word,
                      stream, dtype):
    p = KdaAttentionParams()
    p.q = _rows(q, "q")
    T, Hq, D = q.shape
    p.cache = _paged_cache(k_cache, v_cache, head_dim=D, dtype=dtype)
    _need(kv_len, "kv_len", torch.int32)
    R = kv_len.numel()
    p.num_requests, p.num_tokens, p.num_q_heads, p.window = R, T, Hq, window
    p.scale = D ** -0.5 if scale is None else scale
    if out is None:
        out = _empty((T, Hq, D), torch.bfloat16, q.device, stream)
    o = _rows(out, "out", T, Hq, D)
    p.out, p.out_b_stride, p.out_h_stride = o.ptr, o.b_stride, o.h_stride
    if lse is not None:
        _need(lse, "lse", torch.float32)
        if lse.shape != (T, Hq) or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous [{T}, {Hq}] tensor, got {tuple(lse.shape)}")
        p.lse = lse.data_ptr()
    p.cu_new, p.kv_len = _ints(cu_new, "cu_new", (R + 1,)), _ints(kv_len, "kv_len", (R,))
    p.table, p.table_stride, p.table_width = _table(block_table, R)
    p.error_word = _error_word(error_word)
    if workspace is None:
        workspace = paged_attention_workspace(D, q.device, stream)
    _need(workspace, "workspace", torch.uint8)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous byte tensor")
    return p, out, workspace, (p, q, k_cache, v_cache, block_table, cu_new, kv_len, lse, workspace, error_word)


def kda_paged_attention(q, k_cache, v_cache, block_table, cu_new, kv_len, out=None, lse=None, scale=None, window=0,
                        workspace=None, error_word=None, stream=None):
    """Attention of each request's new tokens over the paged cache
    (include/kda_paged.h). q: bf16 [T, Hq, D], request r owning rows cu_new[r]
    .. cu_new[r+1]-1; k_cache, v_cache: bf16 [pages, page_size, Hkv, D] views
    with any strides, holding the new tokens' keys and values too; block_table:
    int32 [R, W]; kv_len: int32 [R]; lse: optional fp32 [T, Hq], written;
    scale: D ** -0.5 when None; window: keys a row sees at most (0: all);
    workspace: a paged_attention_workspace kept between calls (allocated and
    zeroed on the call's stream when None). Returns out bf16 [T, Hq, D]."""
    return prepare_paged_attention(q, k_cache, v_cache, block_table, cu_new, kv_len, out, lse, scale, window,
                                   workspace, error_word, stream)()


def paged_fp8_cache(num_pages, page_size, num_heads, head_dim, device, stream=None):
    """An empty cache in 8 bits, (k_codes, v_codes, k_scales, v_scales): uint8 [num_pages, page_size, num_heads,
    head_dim] and fp32 [num_pages, blocks of 16 tokens, num_heads]. Nothing of it needs a first value."""
    device = torch.device(device)
    codes = (num_pages, page_size, num_heads, head_dim)
    scales = (num_pages, -(-page_size // KDA_FP8_SCALE_TOKENS), num_heads)
    return tuple(_empty(shape, dtype, device, stream)
                 for shape, dtype in ((codes, torch.uint8), (codes, torch.uint8), (scales, torch.float32), (scales, torch.float32)))


def prepare_rope_append_fp8(q, k, v, positions, slots, freqs, k_codes, v_codes, k_scales, v_scales, q_out=None,
                            interleaved=False, mscale=1.0, error_word=None, stream=None):
    """kda_rope_append_fp8 bound to these tensors (see PreparedCall); same arguments. out is q_out."""
    p, q_out, keep = _rope_params(q, k, v, positions, slots, freqs, k_codes, v_codes, q_out, interleaved, mscale,
                                  error_word, stream, torch.uint8)
    sc = _scales(k_scales, v_scales, p.cache)
    args = (ctypes.byref(p), ctypes.byref(sc), _stream_handle(stream, q.device))
    return PreparedCall(load_library().kda_rope_append_fp8, args, q_out, keep + (sc, k_scales, v_scales))


def kda_rope_append_fp8(q, k, v, positions, slots, freqs, k_codes, v_codes, k_scales, v_scales, q_out=None,
                        interleaved=False, mscale=1.0, error_word=None, stream=None):
    """Rotary positions and the append to a cache in 8 bits (include/kda_paged_fp8.h).
    As kda_rope_append, with k_codes, v_codes: uint8 [pages, page_size, Hkv, D]
    and k_scales, v_scales: fp32 [pages, blocks of 16 tokens, Hkv], views with
    any strides, written at the slots and their blocks. Returns q_out."""
    return prepare_rope_append_fp8(q, k, v, positions, slots, freqs, k_codes, v_codes, k_scales, v_scales, q_out,
                                   interleaved, mscale, error_word, stream)()


def prepare_paged_attention_fp8(q, k_codes, v_codes, k_scales, v_scales, block_table, cu_new, kv_len, out=None,
                                lse=None, scale=None, window=0, workspace=None, error_word=None, stream=None):
    """kda_paged_attention_fp8 bound to these tensors (see PreparedCall); same arguments."""
    p, out, workspace, keep = _attention_params(q, k_codes, v_codes, block_table, cu_new, kv_len, out, lse, scale,
                                                window, workspace, error_word, stream, torch.uint8)
    sc = _scales(k_scales, v_scales, p.cache)
    args = (ctypes.byref(p), ctypes.byref(sc), workspace.data_ptr(), workspace.numel(),
            _stream_handle(stream, q.device))
    return PreparedCall(load_library().kda_paged_attention_fp8, args, out, keep + (sc, k_scales, v_scales))


def kda_paged_attention_fp8(q, k_codes, v_codes, k_scales, v_scales, block_table, cu_new, kv_len, out=None, lse=None,
                            scale=None, window=0, workspace=None, error_word=None, stream=None):
    """Attention of each request's new tokens over a paged cache in 8 bits
    (include/kda_paged_fp8.h). As kda_paged_attention, with the cache of
    kda_rope_append_fp8. Returns out bf16 [T, Hq, D]."""
    return prepare_paged_attention_fp8(q, k_codes, v_codes, k_scales, v_scales, block_table, cu_new, kv_len, out, lse,
                                       scale, window, workspace, error_word, stream)()


PagedRead = collections.namedtuple("PagedRead", "k v")


def prepare_paged_read_fp8(k_codes, v_codes, k_scales, v_scales, block_table, cu_rows, kv_len, num_tokens, out=None,
                           error_word=None, stream=None):
    """kda_paged_read_fp8 bound to these tensors (see PreparedCall); same arguments. out is its PagedRead."""
    p = KdaReadParams()
    p.cache = _paged_cache(k_codes, v_codes, dtype=torch.uint8)
    sc = _scales(k_scales, v_scales, p.cache)
    H, D = p.cache.num_heads, p.cache.head_dim
    _need(kv_len, "kv_len", torch.int32)
    R = kv_len.numel()
    p.num_requests, p.num_tokens = R, num_tokens
    if out is None:
        out = PagedRead(*(_empty((num_tokens, H, D), torch.bfloat16, k_codes.device, stream) for _ in range(2)))
    k, v = _rows(out.k, "out.k", num_tokens, H, D), _rows(out.v, "out.v", num_tokens, H, D)
    p.k_out, p.k_out_b_stride, p.k_out_h_stride = k.ptr, k.b_stride, k.h_stride
    p.v_out, p.v_out_b_stride, p.v_out_h_stride = v.ptr, v.b_stride, v.h_stride
    p.cu_rows, p.kv_len = _ints(cu_rows, "cu_rows", (R + 1,)), _ints(kv_len, "kv_len", (R,))
    p.table, p.table_stride, p.table_width = _table(block_table, R)
    p.error_word = _error_word(error_word)
    keep = (p, sc, k_codes, v_codes, k_scales, v_scales, block_table, cu_rows, kv_len, error_word)
    args = (ctypes.byref(p), ctypes.byref(sc), _stream_handle(stream, k_codes.device))
    return PreparedCall(load_library().kda_paged_read_fp8, args, out, keep)


def kda_paged_read_fp8(k_codes, v_codes, k_scales, v_scales, block_table, cu_rows, kv_len, num_tokens, out=None,
                       error_word=None, stream=None):
    """Cached tokens of a cache in 8 bits read back as packed bf16 rows
    (include/kda_paged_fp8.h): request r has rows cu_rows[r] .. cu_rows[r+1]-1,
    its last tokens up to kv_len[r]. Returns PagedRead(k, v), bf16
    [num_tokens, Hkv, D]."""
    return prepare_paged_read_fp8(k_codes, v_codes, k_scales, v_scales, block_table, cu_rows, kv_len, num_tokens, out,
                                  error_word, stream)()
