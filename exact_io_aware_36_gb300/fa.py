"""Thin ctypes binding of libfa (include/fa.h).

Only argument marshalling happens here: torch tensors become device pointers
and the current CUDA stream becomes a ``cudaStream_t``.  Every step of the
attention computation runs in the library's CUDA kernels.  There is no other
implementation behind these functions: if the library is missing or fails
to load, the calls raise.

Raw entry points with the C names (``fa_fwd``, ``fa_bwd``,
``fa_bwd_workspace_size``, ``fa_check_device_error``, ``fa_status_string``)
take integer pointers; ``attention_forward`` / ``attention_backward`` take
torch tensors and allocate the outputs with torch.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libfa.so")

FA_BF16, FA_FP32 = 0, 1
STATUS = {
    0: "FA_OK", 1: "FA_ERR_NULL", 2: "FA_ERR_SHAPE", 3: "FA_ERR_UNSUPPORTED", 4: "FA_ERR_ALIGN",
    5: "FA_ERR_WORKSPACE", 6: "FA_ERR_CUDA", 7: "FA_ERR_DEVICE_TIMEOUT", 8: "FA_ERR_CU_SEQLENS",
    9: "FA_ERR_PAGE", 10: "FA_ERR_POSITION",
}
EXPORTS = ("fa_fwd", "fa_bwd", "fa_bwd_stage", "fa_bwd_workspace_size", "fa_check_device_error",
           "fa_status_string", "fa_version", "fa_bwd_static_scratch", "fa_selftest_wait_timeout",
           "fa_decode", "fa_decode_workspace_size", "fa_fp8_layout_get", "fa_fp8_quantize",
           "fa_fwd_fp8", "fa_host_cache_stats", "fa_bwd_workspace_size_gqa", "fa_bwd_dkdv_split",
           "fa_qk_norm_rope", "fa_qk_norm_rope_bwd", "fa_qk_norm_rope_bwd_workspace_size",
           "fa_qk_norm_rope_append", "fa_cache_append", "fa_cache_copy", "fa_fwd_paged",
           "fa_fwd_paged_workspace_size", "fa_cache_append_fp8", "fa_qk_norm_rope_append_fp8",
           "fa_cache_copy_fp8", "fa_fwd_paged_fp8", "fa_fwd_paged_fp8_workspace_size")
FA_BWD_PREPROCESS, FA_BWD_DKDV, FA_BWD_DQ_CONVERT = 0, 1, 2


class FAError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        name = STATUS.get(status, str(status))
        msg = f"{what}: {name}" if what else name
        try:
            msg += f" ({fa_status_string(status)})"
        except Exception:
            pass
        super().__init__(msg)


_lib = None


class FP8Layout(ctypes.Structure):
    """fa_fp8_layout: byte offsets of the FP8 codes and scales in one buffer."""
    _fields_ = [("q8", ctypes.c_size_t), ("k8", ctypes.c_size_t), ("v8t", ctypes.c_size_t),
                ("q_scale", ctypes.c_size_t), ("k_scale", ctypes.c_size_t),
                ("v_scale", ctypes.c_size_t), ("v_scale_max", ctypes.c_size_t),
                ("total", ctypes.c_size_t), ("nblk", ctypes.c_int)]


def load(path: Optional[str] = None):
    """Load libfa (once) and declare the C signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise FAError(6, f"libfa not built ({p} missing); run exact_io_aware_36_gb300.build")
    lib = ctypes.CDLL(p)
    vp, i, f, ll, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong, ctypes.c_size_t
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, ll, vp, i, i, vp]
    lib.fa_fwd.restype = i
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, ll, vp,
                           i, i, i, vp, sz, vp]
    lib.fa_bwd.restype = i
    lib.fa_bwd_stage.argtypes = [i] + lib.fa_bwd.argtypes
    lib.fa_bwd_stage.restype = i
    lib.fa_bwd_workspace_size.argtypes = [i, i, i, i, ll]
    lib.fa_bwd_workspace_size.restype = sz
    lib.fa_bwd_workspace_size_gqa.argtypes = [i, i, i, i, i, ll]
    lib.fa_bwd_workspace_size_gqa.restype = sz
    lib.fa_decode_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.fa_decode_workspace_size.restype = sz
    lib.fa_decode.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp, i, vp, sz, vp]
    lib.fa_decode.restype = i
    lib.fa_fp8_layout_get.argtypes = [i, i, i, i, i, ll, ctypes.POINTER(FP8Layout)]
    lib.fa_fp8_layout_get.restype = i
    lib.fa_fp8_quantize.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp, ll, vp, sz, vp]
    lib.fa_fp8_quantize.restype = i
    lib.fa_fwd_fp8.argtypes = [vp, sz, vp, vp, i, i, i, i, i, f, i, i, vp, ll, vp, i, vp]
    lib.fa_fwd_fp8.restype = i
    lib.fa_qk_norm_rope.argtypes = [vp, vp, vp, vp, ll, ll, vp, vp, f, vp, vp, vp, ll, i, i, i, i, i, i, i, vp]
    lib.fa_qk_norm_rope.restype = i
    lib.fa_qk_norm_rope_bwd_workspace_size.argtypes = [i]
    lib.fa_qk_norm_rope_bwd_workspace_size.restype = sz
    lib.fa_qk_norm_rope_bwd.argtypes = [vp, vp, vp, vp, ll, ll, vp, vp, f, vp, vp, vp, vp, vp, ll, ll, vp, vp,
                                        ll, i, i, i, i, i, i, i, vp, sz, vp]
    lib.fa_qk_norm_rope_bwd.restype = i
    lib.fa_cache_append.argtypes = [vp, vp, vp, vp, ll, ll, vp, vp, vp, i, i, i, i, ll, i, i, i, vp]
    lib.fa_cache_append.restype = i
    lib.fa_qk_norm_rope_append.argtypes = [vp, vp, vp, vp, vp, vp, ll, ll, ll, vp, vp, f, vp, vp, vp, vp, vp,
                                           i, i, i, i, i, ll, i, i, i, i, i, i, vp]
    lib.fa_qk_norm_rope_append.restype = i
    lib.fa_fwd_paged_workspace_size.argtypes = [i, i, i, i]
    lib.fa_fwd_paged_workspace_size.restype = sz
    lib.fa_fwd_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, ll, i, i, i, f, i, i, vp, i,
                                 vp, sz, vp]
    lib.fa_fwd_paged.restype = i
    lib.fa_cache_copy.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.fa_cache_copy.restype = i
    # the calls over a cache in 8 bits: two more pointers, the scales, behind the pages
    for name, pages in (("fa_cache_append", 4), ("fa_qk_norm_rope_append", 6), ("fa_cache_copy", 2), ("fa_fwd_paged", 3)):
        a = getattr(lib, name).argtypes
        getattr(lib, name + "_fp8").argtypes = a[:pages] + [vp, vp] + a[pages:]
        getattr(lib, name + "_fp8").restype = i
    lib.fa_fwd_paged_fp8_workspace_size.argtypes = [i, i, i, i, ll]
    lib.fa_fwd_paged_fp8_workspace_size.restype = sz
    lib.fa_check_device_error.argtypes = [vp]
    lib.fa_check_device_error.restype = i
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_version.argtypes = []
    lib.fa_version.restype = i
    if path is None:
        _lib = lib
    return lib


# ------------------------------------------------------------ raw C entry points

def fa_fwd(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, causal, window, cu_seqlens, total_tokens,
           alibi_slopes, dtype, o_dtype, stream) -> int:
    return load().fa_fwd(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, int(causal), int(window),
                         cu_seqlens, total_tokens, alibi_slopes, dtype, o_dtype, stream)


def fa_bwd(q, k, v, o, dO, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, causal, window, cu_seqlens,
           total_tokens, alibi_slopes, dtype, o_dtype, deterministic, workspace, workspace_bytes,
           stream) -> int:
    return load().fa_bwd(q, k, v, o, dO, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, int(causal),
                         int(window), cu_seqlens, total_tokens, alibi_slopes, dtype, o_dtype,
                         int(deterministic), workspace, workspace_bytes, stream)


def fa_bwd_stage(stage, q, k, v, o, dO, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, causal, window,
                 cu_seqlens, total_tokens, alibi_slopes, dtype, o_dtype, deterministic, workspace,
                 workspace_bytes, stream) -> int:
    return load().fa_bwd_stage(stage, q, k, v, o, dO, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale,
                               int(causal), int(window), cu_seqlens, total_tokens, alibi_slopes,
                               dtype, o_dtype, int(deterministic), workspace, workspace_bytes,
                               stream)


FA_BWD_STATIC_SCRATCH_BYTES = 64 << 20


def fa_bwd_static_scratch(q, k, v, o, dO, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, causal,
                          window, cu_seqlens, total_tokens, alibi_slopes, dtype, o_dtype,
                          deterministic, stream) -> int:
    """fa_bwd without a workspace argument, for callers that cannot allocate
    device memory: the scratch lives in a fixed array of
    FA_BWD_STATIC_SCRATCH_BYTES inside the library (see include/fa.h)."""
    lib = load()
    fn = lib.fa_bwd_static_scratch
    if fn.restype is not ctypes.c_int or not fn.argtypes:
        fn.argtypes = lib.fa_bwd.argtypes[:23] + [ctypes.c_void_p]
        fn.restype = ctypes.c_int
    return fn(q, k, v, o, dO, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, int(causal), int(window),
              cu_seqlens, total_tokens, alibi_slopes, dtype, o_dtype, int(deterministic), stream)


def fa_decode_workspace_size(B, Hq, Hkv, S_max, q_len, d) -> int:
    return load().fa_decode_workspace_size(B, Hq, Hkv, S_max, q_len, d)


def fa_decode(q, k_cache, v_cache, cache_seqlens, o, lse, B, Hq, Hkv, S_max, q_len, d, scale,
              window, alibi_slopes, o_dtype, workspace, workspace_bytes, stream) -> int:
    return load().fa_decode(q, k_cache, v_cache, cache_seqlens, o, lse, B, Hq, Hkv, S_max, q_len,
                            d, scale, int(window), alibi_slopes, o_dtype, workspace,
                            workspace_bytes, stream)


def fa_fp8_layout_get(B, Hq, Hkv, N, d, total_tokens):
    """(status, FP8Layout)."""
    lay = FP8Layout()
    st = load().fa_fp8_layout_get(B, Hq, Hkv, N, d, total_tokens, ctypes.byref(lay))
    return st, lay


def fa_fp8_quantize(q, k, v, signs, B, Hq, Hkv, N, d, cu_seqlens, total_tokens, fp8_buf,
                    fp8_bytes, stream) -> int:
    return load().fa_fp8_quantize(q, k, v, signs, B, Hq, Hkv, N, d, cu_seqlens, total_tokens,
                                  fp8_buf, fp8_bytes, stream)


def fa_fwd_fp8(fp8_buf, fp8_bytes, o, lse, B, Hq, Hkv, N, d, scale, causal, window, cu_seqlens,
               total_tokens, alibi_slopes, o_dtype, stream) -> int:
    return load().fa_fwd_fp8(fp8_buf, fp8_bytes, o, lse, B, Hq, Hkv, N, d, scale, int(causal),
                             int(window), cu_seqlens, total_tokens, alibi_slopes, o_dtype, stream)


def fa_qk_norm_rope(q, k, q_out, k_out, q_stride, k_stride, q_weight, k_weight, eps, cos, sin,
                    positions, T, Hq, Hkv, d, rot_dim, max_pos, interleaved, dtype, stream) -> int:
    return load().fa_qk_norm_rope(q, k, q_out, k_out, q_stride, k_stride, q_weight, k_weight, eps,
                                  cos, sin, positions, T, Hq, Hkv, d, rot_dim, max_pos,
                                  int(interleaved), dtype, stream)


def fa_qk_norm_rope_bwd_workspace_size(d) -> int:
    return load().fa_qk_norm_rope_bwd_workspace_size(d)


def fa_qk_norm_rope_bwd(q, k, dq_out, dk_out, q_stride, k_stride, q_weight, k_weight, eps, cos,
                        sin, positions, dq, dk, dq_stride, dk_stride, dq_weight, dk_weight, T, Hq,
                        Hkv, d, rot_dim, max_pos, interleaved, dtype, workspace, workspace_bytes,
                        stream) -> int:
    return load().fa_qk_norm_rope_bwd(q, k, dq_out, dk_out, q_stride, k_stride, q_weight, k_weight,
                                      eps, cos, sin, positions, dq, dk, dq_stride, dk_stride,
                                      dq_weight, dk_weight, T, Hq, Hkv, d, rot_dim, max_pos,
                                      int(interleaved), dtype, workspace, workspace_bytes, stream)


def fa_cache_append(k, v, k_pages, v_pages, k_stride, v_stride, block_table, cache_seqlens,
                    cu_seqlens, B, Hkv, N, d, total_tokens, page_size, num_pages, max_pages,
                    stream) -> int:
    return load().fa_cache_append(k, v, k_pages, v_pages, k_stride, v_stride, block_table,
                                  cache_seqlens, cu_seqlens, B, Hkv, N, d, total_tokens, page_size,
                                  num_pages, max_pages, stream)


def fa_qk_norm_rope_append(q, k, v, q_out, k_pages, v_pages, q_stride, k_stride, v_stride,
                           q_weight, k_weight, eps, cos, sin, block_table, cache_seqlens,
                           cu_seqlens, B, Hq, Hkv, N, d, total_tokens, rot_dim, max_pos,
                           interleaved, page_size, num_pages, max_pages, stream) -> int:
    return load().fa_qk_norm_rope_append(q, k, v, q_out, k_pages, v_pages, q_stride, k_stride,
                                         v_stride, q_weight, k_weight, eps, cos, sin, block_table,
                                         cache_seqlens, cu_seqlens, B, Hq, Hkv, N, d, total_tokens,
                                         rot_dim, max_pos, int(interleaved), page_size, num_pages,
                                         max_pages, stream)


def fa_cache_copy(k_pages, v_pages, src, dst, n, num_pages, page_size, Hkv, d, stream) -> int:
    return load().fa_cache_copy(k_pages, v_pages, src, dst, n, num_pages, page_size, Hkv, d, stream)


def fa_fwd_paged_workspace_size(Hq, Hkv, N, d) -> int:
    return load().fa_fwd_paged_workspace_size(Hq, Hkv, N, d)


def fa_fwd_paged(q, k_pages, v_pages, block_table, cache_seqlens, cu_seqlens, o, lse, B, Hq, Hkv,
                 N, d, total_tokens, page_size, num_pages, max_pages, scale, causal, window,
                 alibi_slopes, o_dtype, workspace, workspace_bytes, stream) -> int:
    return load().fa_fwd_paged(q, k_pages, v_pages, block_table, cache_seqlens, cu_seqlens, o, lse,
                               B, Hq, Hkv, N, d, total_tokens, page_size, num_pages, max_pages,
                               scale, int(causal), int(window), alibi_slopes, o_dtype, workspace,
                               workspace_bytes, stream)


def fa_cache_append_fp8(k, v, k_pages, v_pages, k_scales, v_scales, k_stride, v_stride, block_table,
                        cache_seqlens, cu_seqlens, B, Hkv, N, d, total_tokens, page_size, num_pages,
                        max_pages, stream) -> int:
    return load().fa_cache_append_fp8(k, v, k_pages, v_pages, k_scales, v_scales, k_stride, v_stride,
                                      block_table, cache_seqlens, cu_seqlens, B, Hkv, N, d,
                                      total_tokens, page_size, num_pages, max_pages, stream)


def fa_qk_norm_rope_append_fp8(q, k, v, q_out, k_pages, v_pages, k_scales, v_scales, q_stride,
                               k_stride, v_stride, q_weight, k_weight, eps, cos, sin, block_table,
                               cache_seqlens, cu_seqlens, B, Hq, Hkv, N, d, total_tokens, rot_dim,
                               max_pos, interleaved, page_size, num_pages, max_pages, stream) -> int:
    return load().fa_qk_norm_rope_append_fp8(q, k, v, q_out, k_pages, v_pages, k_scales, v_scales,
                                             q_stride, k_stride, v_stride, q_weight, k_weight, eps, cos,
                                             sin, block_table, cache_seqlens, cu_seqlens, B, Hq, Hkv, N,
                                             d, total_tokens, rot_dim, max_pos, int(interleaved),
                                             page_size, num_pages, max_pages, stream)


def fa_cache_copy_fp8(k_pages, v_pages, k_scales, v_scales, src, dst, n, num_pages, page_size, Hkv, d,
                      stream) -> int:
    return load().fa_cache_copy_fp8(k_pages, v_pages, k_scales, v_scales, src, dst, n, num_pages,
                                    page_size, Hkv, d, stream)


def fa_fwd_paged_fp8_workspace_size(Hq, Hkv, N, d, total_tokens) -> int:
    return load().fa_fwd_paged_fp8_workspace_size(Hq, Hkv, N, d, total_tokens)


def fa_fwd_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, block_table, cache_seqlens, cu_seqlens, o,
                     lse, B, Hq, Hkv, N, d, total_tokens, page_size, num_pages, max_pages, scale, causal,
                     window, alibi_slopes, o_dtype, workspace, workspace_bytes, stream) -> int:
    return load().fa_fwd_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, block_table, cache_seqlens,
                                   cu_seqlens, o, lse, B, Hq, Hkv, N, d, total_tokens, page_size,
                                   num_pages, max_pages, scale, int(causal), int(window), alibi_slopes,
                                   o_dtype, workspace, workspace_bytes, stream)


def fa_bwd_workspace_size(B, Hq, N, d, total_tokens) -> int:
    return load().fa_bwd_workspace_size(B, Hq, N, d, total_tokens)


def fa_bwd_workspace_size_gqa(B, Hq, Hkv, N, d, total_tokens) -> int:
    return load().fa_bwd_workspace_size_gqa(B, Hq, Hkv, N, d, total_tokens)


def fa_bwd_dkdv_split(B, Hq, Hkv, N, d, causal, window, cu_seqlens, workspace_bytes) -> int:
    lib = load()
    fn = lib.fa_bwd_dkdv_split
    fn.argtypes = [ctypes.c_int] * 7 + [ctypes.c_void_p, ctypes.c_size_t]
    fn.restype = ctypes.c_int
    return fn(B, Hq, Hkv, N, d, int(causal), int(window), cu_seqlens, workspace_bytes)


def fa_selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    """Launch one block whose bounded wait can never complete (see fa.h)."""
    lib = load()
    fn = lib.fa_selftest_wait_timeout
    fn.argtypes = [ctypes.c_ulonglong, ctypes.c_void_p]
    fn.restype = ctypes.c_int
    return fn(limit_ns, stream)


def fa_host_cache_stats():
    """(descriptors encoded, descriptors reused, shared-memory limits set)."""
    lib = load()
    fn = lib.fa_host_cache_stats
    u = ctypes.c_ulonglong
    fn.argtypes = [ctypes.POINTER(u)] * 3
    fn.restype = None
    a, b, c = u(), u(), u()
    fn(ctypes.byref(a), ctypes.byref(b), ctypes.byref(c))
    return a.value, b.value, c.value


def fa_check_device_error(stream=None) -> int:
    return load().fa_check_device_error(stream)


def fa_status_string(status: int) -> str:
    return load().fa_status_string(status).decode()


# ------------------------------------------------------------ torch wrappers

def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(status: int, what: str):
    if status != 0:
        raise FAError(status, what)


def _sizes(q, k, cu_seqlens, max_seqlen, batch):
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    if cu_seqlens is not None:
        B = cu_seqlens.numel() - 1
        if max_seqlen is None:
            raise ValueError("max_seqlen is required with cu_seqlens")
        N = int(max_seqlen)
    else:
        B = int(batch) if batch is not None else 1
        N = T // B if B else 0
    return T, B, Hq, Hkv, N, d


def _dtype_code(dt):
    import torch
    return FA_BF16 if dt == torch.bfloat16 else FA_FP32 if dt == torch.float32 else -1


def attention_forward(q, k, v, *, causal: bool, scale: Optional[float] = None, cu_seqlens=None,
                      max_seqlen: Optional[int] = None, batch: Optional[int] = None,
                      alibi_slopes=None, window: Optional[int] = None, out=None, lse=None,
                      out_dtype=None, stream=None, check: bool = False):
    """O, LSE = attention(q, k, v) through ``fa_fwd``.

    q: [T, Hq, d], k/v: [T, Hkv, d] (bf16 or fp32, contiguous, on the GPU).
    Dense batches pass ``batch`` (T = batch * N); packed batches pass int32
    ``cu_seqlens`` [B+1] and ``max_seqlen``.  Returns (o [T, Hq, d] of
    ``out_dtype`` (default: ``out``'s dtype, else q's), lse float32 [Hq, T]).
    ``window`` w (causal only): query i sees keys i - w .. i; None: no window.
    """
    import torch
    T, B, Hq, Hkv, N, d = _sizes(q, k, cu_seqlens, max_seqlen, batch)
    dtype = _dtype_code(q.dtype)
    if dtype < 0:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype or q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    st = fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, N, d, float(scale),
                causal, -1 if window is None else window, _ptr(cu_seqlens), T,
                _ptr(alibi_slopes), dtype, _dtype_code(out.dtype), _stream(stream))
    _check(st, "fa_fwd")
    if check:
        _check(fa_check_device_error(_stream(stream)), "fa_fwd (device)")
    return out, lse


def attention_backward(q, k, v, o, dO, lse, *, causal: bool, scale: Optional[float] = None,
                       cu_seqlens=None, max_seqlen: Optional[int] = None,
                       batch: Optional[int] = None, alibi_slopes=None,
                       window: Optional[int] = None, deterministic: bool = False,
                       workspace=None, dq=None, dk=None, dv=None, stream=None,
                       check: bool = False):
    """dQ, dK, dV through ``fa_bwd`` (bf16).  ``workspace`` (uint8 device
    tensor of at least ``fa_bwd_workspace_size`` bytes; the default is
    ``fa_bwd_workspace_size_gqa``'s size, which lets grouped-query problems
    split their dK/dV work) is allocated when not given.  ``window`` as in attention_forward; ``deterministic`` selects
    the backward whose results do not vary from run to run."""
    import torch
    T, B, Hq, Hkv, N, d = _sizes(q, k, cu_seqlens, max_seqlen, batch)
    if q.dtype != torch.bfloat16:
        raise TypeError("fa_bwd takes bf16 tensors")
    if scale is None:
        scale = d ** -0.5
    need = fa_bwd_workspace_size_gqa(B, Hq, Hkv, N, d, T)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    st = fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq), _ptr(dk),
                _ptr(dv), B, Hq, Hkv, N, d, float(scale), causal,
                -1 if window is None else window, _ptr(cu_seqlens), T, _ptr(alibi_slopes),
                FA_BF16, _dtype_code(o.dtype), deterministic, _ptr(workspace),
                workspace.numel(), _stream(stream))
    _check(st, "fa_bwd")
    if check:
        _check(fa_check_device_error(_stream(stream)), "fa_bwd (device)")
    return dq, dk, dv


def attention_decode(q, k_cache, v_cache, *, cache_seqlens=None, q_len: int = 1,
                     scale: Optional[float] = None, alibi_slopes=None,
                     window: Optional[int] = None, out=None, lse=None, out_dtype=None,
                     workspace=None, stream=None, check: bool = False):
    """O, LSE of the q_len newest tokens of each sequence through ``fa_decode``.

    q: bf16 [B * q_len, Hq, d]; k_cache, v_cache: bf16 [B, S_max, Hkv, d];
    cache_seqlens: int32 [B] on the GPU (None: every cache holds S_max).
    Returns (o [B * q_len, Hq, d] of ``out_dtype`` (default fp32), lse
    float32 [Hq, B * q_len]).
    """
    import torch
    B, S_max, Hkv, d = k_cache.shape
    Hq = q.shape[1]
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype or torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((Hq, q.shape[0]), dtype=torch.float32, device=q.device)
    need = fa_decode_workspace_size(B, Hq, Hkv, S_max, q_len, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = fa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cache_seqlens), _ptr(out), _ptr(lse),
                   B, Hq, Hkv, S_max, q_len, d, float(scale), -1 if window is None else window,
                   _ptr(alibi_slopes), _dtype_code(out.dtype), _ptr(workspace), workspace.numel(),
                   _stream(stream))
    _check(st, "fa_decode")
    if check:
        _check(fa_check_device_error(_stream(stream)), "fa_decode (device)")
    return out, lse


def attention_forward_fp8(q, k, v, signs, *, causal: bool, scale: Optional[float] = None,
                          cu_seqlens=None, max_seqlen: Optional[int] = None,
                          batch: Optional[int] = None, alibi_slopes=None,
                          window: Optional[int] = None, out=None, lse=None, out_dtype=None,
                          fp8_buf=None, stream=None, check: bool = False):
    """O, LSE through ``fa_fp8_quantize`` and ``fa_fwd_fp8`` (d = 128).

    q: bf16 [T, Hq, 128], k/v: bf16 [T, Hkv, 128]; signs: float32 [128] of
    +-1 on the GPU.  Returns (o, lse, fp8_buf, layout): the buffer holds the
    codes and scales at the layout's offsets.
    """
    import torch
    T, B, Hq, Hkv, N, d = _sizes(q, k, cu_seqlens, max_seqlen, batch)
    if scale is None:
        scale = d ** -0.5
    st, lay = fa_fp8_layout_get(B, Hq, Hkv, N, d, T if cu_seqlens is not None else 0)
    _check(st, "fa_fp8_layout_get")
    if fp8_buf is None:
        fp8_buf = torch.empty(max(lay.total, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty(q.shape, dtype=out_dtype or torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    sp = _stream(stream)
    _check(fa_fp8_quantize(_ptr(q), _ptr(k), _ptr(v), _ptr(signs), B, Hq, Hkv, N, d,
                           _ptr(cu_seqlens), T, _ptr(fp8_buf), fp8_buf.numel(), sp), "fa_fp8_quantize")
    _check(fa_fwd_fp8(_ptr(fp8_buf), fp8_buf.numel(), _ptr(out), _ptr(lse), B, Hq, Hkv, N, d,
                      float(scale), causal, -1 if window is None else window, _ptr(cu_seqlens), T,
                      _ptr(alibi_slopes), _dtype_code(out.dtype), sp), "fa_fwd_fp8")
    if check:
        _check(fa_check_device_error(sp), "fa_fwd_fp8 (device)")
    return out, lse, fp8_buf, lay


# ------------------------------------------- norm, rotation and a cache in pages

# Single-token calls are as short as a few microseconds on the GPU, so what runs
# before them here is kept lean: devices are compared by index, shapes as
# tuples, and a message is made only for a call that is refused.

_INT_MAX = 2**31 - 1    # ctypes cuts a larger int to its low 32 bits without a word

_torch = None


def _import_torch():
    """torch, imported by the first call that needs it."""
    global _torch
    import torch
    _torch = torch
    return torch


def _refuse(name, t, dtype, index, shape, contiguous=True):
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {dtype} expected, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {shape} expected, got {tuple(t.shape)}")
    if contiguous:
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name}: [T, H, d] with the heads of a token contiguous expected")


def _checked(name, t, dtype, index, shape=None):
    """The pointer of a contiguous tensor of `dtype` on GPU `index` (and of `shape`), else TypeError / ValueError."""
    if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous() or \
            (shape is not None and t.shape != shape):
        _refuse(name, t, dtype, index, shape)
    return t.data_ptr()


def _rows(name, t, dtype, index, shape=None):
    """(pointer, token stride) of a [T, H, d] tensor whose tokens may lie apart."""
    if t.dtype is not dtype or t.get_device() != index or t.dim() != 3 or (shape is not None and t.shape != shape):
        _refuse(name, t, dtype, index, shape, False)
    T, H, d = t.shape
    st, sh, sd = t.stride()
    if (sd != 1 or (H > 1 and sh != d)) and t.numel():
        _refuse(name, t, dtype, index, shape, False)
    return t.data_ptr(), (st if T > 1 else H * d)


def _gpu(t, stream):
    """Index of the GPU that `t` is on; `stream` (if any) must be there too."""
    index = t.get_device()
    if index < 0:
        raise ValueError("tensors must be on a GPU")
    if stream is not None and stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
    return index


def _out(name, t, like, shape, dtype, index, stream):
    """(tensor, pointer) of an output: the one given, checked, or a new one that belongs to `stream` (None: the current one)."""
    if t is not None:
        return t, _checked(name, t, dtype, index, shape)
    if stream is None:
        t = _torch.empty(shape, dtype=dtype, device=like.device)
    else:
        with _torch.cuda.stream(stream):
            t = _torch.empty(shape, dtype=dtype, device=like.device)
    return t, t.data_ptr()


def _run(what, index, stream, check, *args):
    """The library's `what`(*args, stream) with GPU `index` current; raises on a status that is not FA_OK."""
    torch = _torch or _import_torch()
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _run(what, index, stream, check, *args)
    # the raw handle of the current stream, without a Stream object around it
    sp = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    st = getattr(_lib or load(), what)(*args, sp)
    if st:
        raise FAError(st, what)
    if check:
        _check(fa_check_device_error(sp), what + " (device)")


def _angles(q_weight, k_weight, cos, sin, d, index):
    """Pointers of the weights and of the angles, rot_dim and max_pos."""
    f32 = (_torch or _import_torch()).float32
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    qw = kw = None
    if q_weight is not None:
        qw, kw = _checked("q_weight", q_weight, f32, index, (d,)), _checked("k_weight", k_weight, f32, index, (d,))
    if cos is None:
        return qw, kw, None, None, 0, 0
    if cos.dim() != 2:
        raise ValueError("cos: [max_pos, rot_dim / 2] expected")
    shape = cos.shape
    return qw, kw, _checked("cos", cos, f32, index), _checked("sin", sin, f32, index, shape), 2 * shape[1], shape[0]


def qk_norm_rope(q, k, *, q_weight=None, k_weight=None, eps: float = 1e-6, cos=None, sin=None,
                 positions=None, interleaved: bool = False, q_out=None, k_out=None, stream=None,
                 check: bool = False):
    """RMS norm of every head of q and k and rotation by position through ``fa_qk_norm_rope``.

    q: [T, Hq, d], k: [T, Hkv, d] (bf16 or fp32; both may be parts of one
    projection's output: only the heads of a token have to be contiguous).
    q_weight, k_weight: float32 [d] (None: no norm); cos, sin: float32
    [max_pos, rot_dim / 2] with positions int32 [T] (None: no rotation).
    Pairs are (i, i + rot_dim / 2), or (2 i, 2 i + 1) with ``interleaved``.
    Returns (q_out, k_out), contiguous, of q's type.  For training the result
    goes to ``attention_forward`` and ``attention_backward``'s dq, dk to
    ``qk_norm_rope_backward``.
    """
    torch = _torch or _import_torch()
    index = _gpu(q, stream)
    qp, qs = _rows("q", q, q.dtype, index)
    kp, ks = _rows("k", k, q.dtype, index)
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    if k.shape[0] != T or k.shape[2] != d:
        raise ValueError("q and k must have the same tokens and head dimension")
    ang = _angles(q_weight, k_weight, cos, sin, d, index)
    pos = None
    if cos is not None:
        if positions is None:
            raise ValueError("positions are required with cos and sin")
        pos = _checked("positions", positions, torch.int32, index, (T,))
    q_out, qop = _out("q_out", q_out, q, (T, Hq, d), q.dtype, index, stream)
    k_out, kop = _out("k_out", k_out, q, (T, Hkv, d), q.dtype, index, stream)
    _run("fa_qk_norm_rope", index, stream, check, qp, kp, qop, kop, qs, ks, ang[0], ang[1], float(eps),
         ang[2], ang[3], pos, T, Hq, Hkv, d, ang[4], ang[5], interleaved, _dtype_code(q.dtype))
    return q_out, k_out


def qk_norm_rope_backward(q, k, dq_out, dk_out, *, q_weight=None, k_weight=None,
                          eps: float = 1e-6, cos=None, sin=None, positions=None,
                          interleaved: bool = False, dq=None, dk=None, workspace=None,
                          stream=None, check: bool = False):
    """Gradient of ``qk_norm_rope`` through ``fa_qk_norm_rope_bwd``.

    q, k and the other arguments as given to ``qk_norm_rope``; dq_out, dk_out:
    gradients of its results (contiguous).  dq, dk may be parts of one buffer, as
    q and k.  Returns (dq, dk, dq_weight, dk_weight); the weights' gradients are
    float32 [d], or None without norm.  Results do not vary from run to run.
    """
    torch = _torch or _import_torch()
    index = _gpu(q, stream)
    qp, qs = _rows("q", q, q.dtype, index)
    kp, ks = _rows("k", k, q.dtype, index)
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    if k.shape[0] != T or k.shape[2] != d:
        raise ValueError("q and k must have the same tokens and head dimension")
    ang = _angles(q_weight, k_weight, cos, sin, d, index)
    pos = None
    if cos is not None:
        if positions is None:
            raise ValueError("positions are required with cos and sin")
        pos = _checked("positions", positions, torch.int32, index, (T,))
    if dq is None:
        dqs, (dq, dqp) = Hq * d, _out("dq", None, q, (T, Hq, d), q.dtype, index, stream)
    else:
        dqp, dqs = _rows("dq", dq, q.dtype, index, (T, Hq, d))
    if dk is None:
        dks, (dk, dkp) = Hkv * d, _out("dk", None, q, (T, Hkv, d), q.dtype, index, stream)
    else:
        dkp, dks = _rows("dk", dk, q.dtype, index, (T, Hkv, d))
    dqw = dkw = dqwp = dkwp = wp = None
    wbytes = 0
    if q_weight is not None:
        dqw, dqwp = _out("", None, q, (d,), torch.float32, index, stream)
        dkw, dkwp = _out("", None, q, (d,), torch.float32, index, stream)
        wbytes = fa_qk_norm_rope_bwd_workspace_size(d) if workspace is None else workspace.numel()
        workspace, wp = _out("workspace", workspace, q, (wbytes,), torch.uint8, index, stream)
    _run("fa_qk_norm_rope_bwd", index, stream, check, qp, kp,
         _checked("dq_out", dq_out, q.dtype, index, (T, Hq, d)),
         _checked("dk_out", dk_out, q.dtype, index, (T, Hkv, d)), qs, ks, ang[0], ang[1], float(eps),
         ang[2], ang[3], pos, dqp, dkp, dqs, dks, dqwp, dkwp, T, Hq, Hkv, d, ang[4], ang[5],
         interleaved, _dtype_code(q.dtype), wp, wbytes)
    return dq, dk, dqw, dkw


def _pages(k_pages, v_pages, index):
    """(k pointer, v pointer, num_pages, page_size, Hkv, d) of the two pools."""
    torch = _torch or _import_torch()
    if k_pages.dim() != 4:
        raise ValueError("k_pages: [num_pages, page_size, Hkv, d] expected")
    kp = _checked("k_pages", k_pages, torch.bfloat16, index)
    vp = _checked("v_pages", v_pages, torch.bfloat16, index, k_pages.shape)
    return (kp, vp, *k_pages.shape)


def _table(block_table, cache_seqlens, cu_seqlens, max_seqlen, T, index):
    """(table, cache_seqlens, cu_seqlens pointers, B, N, max_pages)."""
    torch = _torch or _import_torch()
    if block_table.dim() != 2:
        raise ValueError("block_table: [B, max_pages] expected")
    B, max_pages = block_table.shape
    tp = _checked("block_table", block_table, torch.int32, index)
    cp = _checked("cache_seqlens", cache_seqlens, torch.int32, index, (B,))
    if cu_seqlens is not None:
        if max_seqlen is None:
            raise ValueError("max_seqlen is required with cu_seqlens")
        return tp, cp, _checked("cu_seqlens", cu_seqlens, torch.int32, index, (B + 1,)), B, \
            max(-1, min(int(max_seqlen), _INT_MAX)), max_pages
    N = T // B if B else 0
    if T != B * N:
        raise ValueError("without cu_seqlens every sequence brings the same number of tokens")
    return tp, cp, None, B, N, max_pages


def cache_append(k, v, k_pages, v_pages, block_table, cache_seqlens, *, cu_seqlens=None,
                 max_seqlen: Optional[int] = None, stream=None, check: bool = False):
    """Write the new tokens' k and v into the pages of a cache through ``fa_cache_append``.

    k, v: bf16 [T, Hkv, d] (the heads of a token contiguous); k_pages, v_pages:
    bf16 [num_pages, page_size, Hkv, d]; block_table: int32 [B, max_pages];
    cache_seqlens: int32 [B], the new tokens included.  Sequence b's new tokens
    are rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (int32 [B + 1], with
    ``max_seqlen`` their largest number), or T / B each without it.
    """
    torch = _torch or _import_torch()
    index = _gpu(k, stream)
    kp, ks = _rows("k", k, torch.bfloat16, index)
    vp, vs = _rows("v", v, torch.bfloat16, index, k.shape)
    T, Hkv, d = k.shape
    kpool, vpool, num_pages, page_size, Hp, dp = _pages(k_pages, v_pages, index)
    if (Hp, dp) != (Hkv, d):
        raise ValueError("the pages have other heads than k")
    tp, cp, cup, B, N, max_pages = _table(block_table, cache_seqlens, cu_seqlens, max_seqlen, T, index)
    _run("fa_cache_append", index, stream, check, kp, vp, kpool, vpool, ks, vs, tp,
         cp, cup, B, Hkv, N, d, T, page_size, num_pages, max_pages)


def qk_norm_rope_append(q, k, v, k_pages, v_pages, block_table, cache_seqlens, *, cu_seqlens=None,
                        max_seqlen: Optional[int] = None, q_weight=None, k_weight=None,
                        eps: float = 1e-6, cos=None, sin=None, interleaved: bool = False,
                        q_out=None, stream=None, check: bool = False):
    """``qk_norm_rope`` of new tokens and ``cache_append`` of their k and v in
    one launch (``fa_qk_norm_rope_append``).  A token's position is its place
    in its sequence's cache.  Returns q_out [T, Hq, d], ready for
    ``attention_forward_paged`` over the same pages."""
    torch = _torch or _import_torch()
    index = _gpu(q, stream)
    qp, qs = _rows("q", q, torch.bfloat16, index)
    kp, ks = _rows("k", k, torch.bfloat16, index)
    vp, vs = _rows("v", v, torch.bfloat16, index, k.shape)
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    kpool, vpool, num_pages, page_size, Hp, dp = _pages(k_pages, v_pages, index)
    if k.shape[0] != T or k.shape[2] != d or (Hp, dp) != (Hkv, d):
        raise ValueError("q, k and the pages must have the same tokens, key heads and head dimension")
    tp, cp, cup, B, N, max_pages = _table(block_table, cache_seqlens, cu_seqlens, max_seqlen, T, index)
    ang = _angles(q_weight, k_weight, cos, sin, d, index)
    q_out, qop = _out("q_out", q_out, q, (T, Hq, d), q.dtype, index, stream)
    _run("fa_qk_norm_rope_append", index, stream, check, qp, kp, vp, qop, kpool, vpool, qs, ks, vs, ang[0],
         ang[1], float(eps), ang[2], ang[3], tp, cp, cup, B, Hq, Hkv, N, d, T, ang[4], ang[5],
         interleaved, page_size, num_pages, max_pages)
    return q_out


def cache_copy(k_pages, v_pages, src, dst, *, stream=None, check: bool = False):
    """Copy pages src[i] to dst[i] (int32 [n], on the GPU) of both pools through
    ``fa_cache_copy``: the fork of a sequence's last page, a compaction's moves.
    The copies run in no order; see include/fa.h on pairs that clash."""
    torch = _torch or _import_torch()
    index = _gpu(k_pages, stream)
    kpool, vpool, num_pages, page_size, Hkv, d = _pages(k_pages, v_pages, index)
    n = src.numel()
    _run("fa_cache_copy", index, stream, check, kpool, vpool,
         _checked("src", src, torch.int32, index, (n,)), _checked("dst", dst, torch.int32, index, (n,)),
         n, num_pages, page_size, Hkv, d)


def attention_forward_paged(q, k_pages, v_pages, block_table, cache_seqlens, *, cu_seqlens=None,
                            max_seqlen: Optional[int] = None, causal: bool = True,
                            scale: Optional[float] = None, alibi_slopes=None,
                            window: Optional[int] = None, out=None, lse=None, out_dtype=None,
                            workspace=None, stream=None, check: bool = False):
    """O, LSE of each sequence's newest tokens over its pages through ``fa_fwd_paged``.

    q: bf16 [T, Hq, d]; pools, table, lengths and ``cu_seqlens`` / ``max_seqlen``
    as ``cache_append`` (which has put the new tokens' k and v there).  Causal:
    the last new token sees the whole sequence, the one before all but one
    key; otherwise every row sees all of its sequence's keys.  Returns
    (o [T, Hq, d] of ``out_dtype`` (default: ``out``'s dtype, else q's), lse
    float32 [Hq, T]).
    """
    torch = _torch or _import_torch()
    index = _gpu(q, stream)
    if q.dim() != 3:
        raise ValueError("q: [T, Hq, d] expected")
    T, Hq, d = q.shape
    qp = _checked("q", q, torch.bfloat16, index)
    kpool, vpool, num_pages, page_size, Hkv, dp = _pages(k_pages, v_pages, index)
    if dp != d:
        raise ValueError("q and the pages must have the same head dimension")
    tp, cp, cup, B, N, max_pages = _table(block_table, cache_seqlens, cu_seqlens, max_seqlen, T, index)
    slopes = None if alibi_slopes is None else _checked("alibi_slopes", alibi_slopes, torch.float32, index, (Hq,))
    out, op = _out("out", out, q, (T, Hq, d), (out_dtype or q.dtype) if out is None else out.dtype, index, stream)
    lse, lp = _out("lse", lse, q, (Hq, T), torch.float32, index, stream)
    wbytes = fa_fwd_paged_workspace_size(Hq, Hkv, N, d) if workspace is None else workspace.numel()
    workspace, wp = _out("workspace", workspace, q, (wbytes,), torch.uint8, index, stream)
    _run("fa_fwd_paged", index, stream, check, qp, kpool, vpool, tp, cp, cup, op, lp, B, Hq, Hkv, N, d, T,
         page_size, num_pages, max_pages, float(d ** -0.5 if scale is None else scale), causal,
         -1 if window is None else max(-1, min(window, _INT_MAX)), slopes, _dtype_code(out.dtype), wp, wbytes)
    return out, lse


def _pages_fp8(k_pages, v_pages, k_scales, v_scales, index):
    """(the four pointers, num_pages, page_size, Hkv, d) of pools of codes and their scales."""
    torch = _torch or _import_torch()
    if k_pages.dim() != 4:
        raise ValueError("k_pages: [num_pages, page_size, Hkv, d] expected")
    codes = torch.uint8 if k_pages.dtype is torch.uint8 else torch.float8_e4m3fn
    scale = torch.uint8 if k_scales.dtype is torch.uint8 else torch.float8_e8m0fnu
    num_pages, page_size, Hkv, d = k_pages.shape
    shape = (num_pages, page_size // 16, Hkv)
    return (_checked("k_pages", k_pages, codes, index), _checked("v_pages", v_pages, codes, index, k_pages.shape),
            _checked("k_scales", k_scales, scale, index, shape), _checked("v_scales", v_scales, scale, index, shape),
            num_pages, page_size, Hkv, d)


def cache_append_fp8(k, v, k_pages, v_pages, k_scales, v_scales, block_table, cache_seqlens, *,
                     cu_seqlens=None, max_seqlen: Optional[int] = None, stream=None,
                     check: bool = False):
    """Quantize the new tokens' k and v into the pages of a cache in 8 bits
    through ``fa_cache_append_fp8``.

    k_pages, v_pages: codes, float8_e4m3fn or uint8 [num_pages, page_size, Hkv,
    d]; k_scales, v_scales: the exponents (plus 127) of the powers of two of every
    16 slots and head, float8_e8m0fnu or uint8 [num_pages, page_size / 16, Hkv].
    The other arguments as ``cache_append``.  A block of 16 slots that gets
    tokens takes the least scale that holds them and the older tokens before
    them (see include/fa.h).
    """
    torch = _torch or _import_torch()
    index = _gpu(k, stream)
    kp, ks = _rows("k", k, torch.bfloat16, index)
    vp, vs = _rows("v", v, torch.bfloat16, index, k.shape)
    T, Hkv, d = k.shape
    *pools, num_pages, page_size, Hp, dp = _pages_fp8(k_pages, v_pages, k_scales, v_scales, index)
    if (Hp, dp) != (Hkv, d):
        raise ValueError("the pages have other heads than k")
    tp, cp, cup, B, N, max_pages = _table(block_table, cache_seqlens, cu_seqlens, max_seqlen, T, index)
    _run("fa_cache_append_fp8", index, stream, check, kp, vp, *pools, ks, vs, tp, cp, cup, B, Hkv, N, d, T,
         page_size, num_pages, max_pages)


def qk_norm_rope_append_fp8(q, k, v, k_pages, v_pages, k_scales, v_scales, block_table, cache_seqlens, *,
                            cu_seqlens=None, max_seqlen: Optional[int] = None, q_weight=None,
                            k_weight=None, eps: float = 1e-6, cos=None, sin=None,
                            interleaved: bool = False, q_out=None, stream=None, check: bool = False):
    """``qk_norm_rope`` of new tokens and ``cache_append_fp8`` of their k and v in
    one launch (``fa_qk_norm_rope_append_fp8``); k is quantized from float32.
    Returns q_out [T, Hq, d] in bf16, ready for ``attention_forward_paged_fp8``
    over the same pages."""
    torch = _torch or _import_torch()
    index = _gpu(q, stream)
    qp, qs = _rows("q", q, torch.bfloat16, index)
    kp, ks = _rows("k", k, torch.bfloat16, index)
    vp, vs = _rows("v", v, torch.bfloat16, index, k.shape)
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    *pools, num_pages, page_size, Hp, dp = _pages_fp8(k_pages, v_pages, k_scales, v_scales, index)
    if k.shape[0] != T or k.shape[2] != d or (Hp, dp) != (Hkv, d):
        raise ValueError("q, k and the pages must have the same tokens, key heads and head dimension")
    tp, cp, cup, B, N, max_pages = _table(block_table, cache_seqlens, cu_seqlens, max_seqlen, T, index)
    ang = _angles(q_weight, k_weight, cos, sin, d, index)
    q_out, qop = _out("q_out", q_out, q, (T, Hq, d), q.dtype, index, stream)
    _run("fa_qk_norm_rope_append_fp8", index, stream, check, qp, kp, vp, qop, *pools, qs, ks, vs, ang[0],
         ang[1], float(eps), ang[2], ang[3], tp, cp, cup, B, Hq, Hkv, N, d, T, ang[4], ang[5],
         interleaved, page_size, num_pages, max_pages)
    return q_out


def cache_copy_fp8(k_pages, v_pages, k_scales, v_scales, src, dst, *, stream=None, check: bool = False):
    """``cache_copy`` of pages of codes and their scales through ``fa_cache_copy_fp8``."""
    torch = _torch or _import_torch()
    index = _gpu(k_pages, stream)
    *pools, num_pages, page_size, Hkv, d = _pages_fp8(k_pages, v_pages, k_scales, v_scales, index)
    n = src.numel()
    _run("fa_cache_copy_fp8", index, stream, check, *pools,
         _checked("src", src, torch.int32, index, (n,)), _checked("dst", dst, torch.int32, index, (n,)),
         n, num_pages, page_size, Hkv, d)


def attention_forward_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, block_table, cache_seqlens, *,
                                cu_seqlens=None, max_seqlen: Optional[int] = None, causal: bool = True,
                                scale: Optional[float] = None, alibi_slopes=None,
                                window: Optional[int] = None, out=None, lse=None, out_dtype=None,
                                workspace=None, stream=None, check: bool = False):
    """``attention_forward_paged`` over a cache in 8 bits (pools and scales as
    ``cache_append_fp8``) through ``fa_fwd_paged_fp8``.  q: bf16 [T, Hq, d].
    Returns (o, lse) as ``attention_forward_paged``."""
    torch = _torch or _import_torch()
    index = _gpu(q, stream)
    if q.dim() != 3:
        raise ValueError("q: [T, Hq, d] expected")
    T, Hq, d = q.shape
    qp = _checked("q", q, torch.bfloat16, index)
    *pools, num_pages, page_size, Hkv, dp = _pages_fp8(k_pages, v_pages, k_scales, v_scales, index)
    if dp != d:
        raise ValueError("q and the pages must have the same head dimension")
    tp, cp, cup, B, N, max_pages = _table(block_table, cache_seqlens, cu_seqlens, max_seqlen, T, index)
    slopes = None if alibi_slopes is None else _checked("alibi_slopes", alibi_slopes, torch.float32, index, (Hq,))
    out, op = _out("out", out, q, (T, Hq, d), (out_dtype or q.dtype) if out is None else out.dtype, index, stream)
    lse, lp = _out("lse", lse, q, (Hq, T), torch.float32, index, stream)
    wbytes = fa_fwd_paged_fp8_workspace_size(Hq, Hkv, N, d, T) if workspace is None else workspace.numel()
    workspace, wp = _out("workspace", workspace, q, (wbytes,), torch.uint8, index, stream)
    _run("fa_fwd_paged_fp8", index, stream, check, qp, *pools, tp, cp, cup, op, lp, B, Hq, Hkv, N, d, T,
         page_size, num_pages, max_pages, float(d ** -0.5 if scale is None else scale), causal,
         -1 if window is None else max(-1, min(window, _INT_MAX)), slopes, _dtype_code(out.dtype), wp, wbytes)
    return out, lse
