"""attention_rank_additive_b200 -- attention with a low-rank additive bias on B200.

Python binding of libflashbias (the C ABI in include/flashbias.h). The
functions named ``fb_*`` mirror the C entry points one to one and take raw
integers for pointers; the helpers below them (``attn``, ``attn_dense_bias``,
``factors_sandwich``, ``factors_alibi``, ``svd_factors``, and for serving
``rope``, ``cache_write``, ``cache_read``, ``attn_cache``) only marshal torch
tensors: every step of the computation runs in the library's kernels.

There is no fallback: importing works without a GPU, but the first call that
needs the library raises if ``libflashbias.so`` has not been built
(``python -m attention_rank_additive_b200.build``).
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

__all__ = [
    "FB_OK", "FB_ERR_INVALID_ARG", "FB_ERR_UNSUPPORTED", "FB_ERR_RANGE", "FB_ERR_WORKSPACE", "FB_ERR_CUDA",
    "FB_ERR_TIMEOUT", "FB_F32", "FB_BF16", "FB_F16", "FlashBiasError", "lib", "lib_path", "EXPORTED",
    "fb_status_str", "fb_version", "fb_attn_workspace_bytes", "fb_attn_fwd", "fb_attn_dense_bias_fwd",
    "fb_factors_sandwich", "fb_factors_alibi", "fb_svd_factors_host", "fb_check_device_error",
    "fb_selftest_wait_timeout", "fb_attn_fwd_noalloc", "fb_attn_prepare_factors", "fb_attn_fwd_prepared",
    "fb_attn_mul_bias_workspace_bytes", "fb_attn_mul_bias_fwd", "attn_mul_bias", "attn",
    "fb_svd_device_workspace_bytes", "fb_svd_factors_device", "svd_factors_device",
    "fb_attn_neural_workspace_bytes", "fb_attn_neural_fwd", "attn_neural",
    "PreparedBias", "attn_dense_bias", "factors_sandwich", "factors_alibi", "svd_factors",
    "attn_flops", "FB_E4M3", "fb_rope_fwd", "fb_rope_bwd", "fb_rope_turns_host", "fb_rope_frequencies_host",
    "fb_cache_write", "fb_cache_read", "fb_cache_bias_bytes", "fb_cache_bias_prepare",
    "fb_attn_cache_workspace_bytes", "fb_attn_cache_fwd", "fb_call", "Rope", "rope", "rope_bwd", "PagedCache",
    "cache_write", "cache_read", "CacheBias", "cache_workspace", "attn_cache",
]

FB_OK, FB_ERR_INVALID_ARG, FB_ERR_UNSUPPORTED, FB_ERR_RANGE, FB_ERR_WORKSPACE, FB_ERR_CUDA, FB_ERR_TIMEOUT = range(7)
FB_F32, FB_BF16, FB_F16, FB_E4M3 = 0, 1, 2, 3

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libflashbias.so")

# Every symbol include/flashbias.h declares.
EXPORTED = (
    "fb_status_str", "fb_version", "fb_attn_workspace_bytes", "fb_attn_fwd", "fb_attn_dense_bias_fwd",
    "fb_factors_sandwich", "fb_factors_alibi", "fb_svd_factors_host", "fb_check_device_error",
    "fb_selftest_wait_timeout", "fb_attn_fwd_noalloc", "fb_attn_prepare_factors", "fb_attn_fwd_prepared",
    "fb_attn_mul_bias_workspace_bytes", "fb_attn_mul_bias_fwd", "fb_svd_device_workspace_bytes",
    "fb_svd_factors_device", "fb_attn_neural_workspace_bytes", "fb_attn_neural_fwd", "fb_attn_bwd_workspace_bytes",
    "fb_attn_bwd", "fb_attn_neural_bwd_workspace_bytes", "fb_attn_neural_bwd", "fb_rope_fwd", "fb_rope_bwd",
    "fb_rope_turns_host", "fb_rope_frequencies_host", "fb_cache_write", "fb_cache_read", "fb_cache_bias_bytes",
    "fb_cache_bias_prepare", "fb_attn_cache_workspace_bytes", "fb_attn_cache_fwd", "fb_call",
)


class FlashBiasError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fb_status_str(status)} ({status})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libflashbias; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise RuntimeError(f"libflashbias.so is missing at {lib_path}; build it with "
                               "`python -m attention_rank_additive_b200.build`")
        L = ctypes.CDLL(lib_path)
        i32, i64, sz, vp, f32 = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
        L.fb_status_str.argtypes, L.fb_status_str.restype = [i32], ctypes.c_char_p
        L.fb_version.argtypes, L.fb_version.restype = [], i32
        L.fb_attn_workspace_bytes.argtypes = [i32, i32, i32, i32, i64, i64]
        L.fb_attn_workspace_bytes.restype = sz
        L.fb_attn_fwd.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, i32, vp, vp, i64, i64, f32, i32, vp, vp, vp,
                                  sz, vp]
        L.fb_attn_fwd.restype = i32
        L.fb_attn_fwd_noalloc.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, i32, vp, vp, i64, i64, f32, i32, vp,
                                          vp, vp]
        L.fb_attn_fwd_noalloc.restype = i32
        L.fb_attn_prepare_factors.argtypes = [i32, i32, i32, i32, vp, vp, i64, i64, f32, vp, sz, vp]
        L.fb_attn_prepare_factors.restype = i32
        L.fb_attn_fwd_prepared.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, i32, i64, i64, f32, i32, vp, vp, vp,
                                           sz, vp]
        L.fb_attn_fwd_prepared.restype = i32
        L.fb_attn_mul_bias_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.fb_attn_mul_bias_workspace_bytes.restype = sz
        L.fb_attn_mul_bias_fwd.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, i32, vp, vp, i64, i64, f32, i32, vp,
                                           vp, vp, sz, vp]
        L.fb_attn_mul_bias_fwd.restype = i32
        L.fb_svd_device_workspace_bytes.argtypes = [i32, i32, i32, i32]
        L.fb_svd_device_workspace_bytes.restype = sz
        L.fb_svd_factors_device.argtypes = [i32, i32, i32, i32, i32, ctypes.c_uint64, vp, vp, vp, vp, vp, sz, vp]
        L.fb_svd_factors_device.restype = i32
        L.fb_attn_neural_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.fb_attn_neural_workspace_bytes.restype = sz
        L.fb_attn_neural_fwd.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, f32, i32, vp,
                                         vp, vp, sz, vp]
        L.fb_attn_neural_fwd.restype = i32
        L.fb_attn_bwd_workspace_bytes.argtypes = [i32, i32, i32, i32, i64, i64]
        L.fb_attn_bwd_workspace_bytes.restype = sz
        L.fb_attn_bwd.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, i32, vp, vp, i64, i64, f32, i32, vp, vp, vp,
                                  vp, vp, vp, vp, vp, vp, sz, vp]
        L.fb_attn_bwd.restype = i32
        L.fb_attn_neural_bwd_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.fb_attn_neural_bwd_workspace_bytes.restype = sz
        L.fb_attn_neural_bwd.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp, f32, i32, vp,
                                         vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.fb_attn_neural_bwd.restype = i32
        L.fb_attn_dense_bias_fwd.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, vp, i64, i64, f32, i32, vp, vp, vp]
        L.fb_attn_dense_bias_fwd.restype = i32
        L.fb_factors_sandwich.argtypes, L.fb_factors_sandwich.restype = [i32, i32, vp, vp, vp], i32
        L.fb_factors_alibi.argtypes, L.fb_factors_alibi.restype = [i32, i32, vp, vp, vp], i32
        L.fb_svd_factors_host.argtypes = [vp, i32, i32, i32, i32, ctypes.c_uint64, vp, vp, vp, vp]
        L.fb_svd_factors_host.restype = i32
        rope_args = [i32, i32, i32, i32, i32, i32, vp, f32, vp, i64] + 2 * [i32, vp, i64, i64, i64, vp, i64, i64, i64]
        L.fb_rope_fwd.argtypes, L.fb_rope_fwd.restype = rope_args + [vp], i32
        L.fb_rope_bwd.argtypes, L.fb_rope_bwd.restype = rope_args + [vp], i32
        L.fb_rope_turns_host.argtypes, L.fb_rope_turns_host.restype = [i32, vp, vp], i32
        f64 = ctypes.c_double
        L.fb_rope_frequencies_host.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp, vp]
        L.fb_rope_frequencies_host.restype = i32
        L.fb_cache_write.argtypes = [i32, i32, i32, i32, i32, i32, vp, i64, i64, i64, vp, i64, i64, i64, vp, vp, vp, vp,
                                     i32, i32, vp, i32, vp, vp, vp]
        L.fb_cache_write.restype = i32
        L.fb_cache_read.argtypes = [i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp]
        L.fb_cache_read.restype = i32
        L.fb_cache_bias_bytes.argtypes, L.fb_cache_bias_bytes.restype = [i32, i32, i32, i32], sz
        L.fb_cache_bias_prepare.argtypes = [i32, i32, i32, i32, vp, vp, vp, sz, vp]
        L.fb_cache_bias_prepare.restype = i32
        L.fb_attn_cache_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.fb_attn_cache_workspace_bytes.restype = sz
        L.fb_attn_cache_fwd.argtypes = [i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, i32, i32, vp, i32, vp, vp, vp,
                                        i32, vp, i32, i32, i32, i32, vp, f32, vp, vp, vp, sz, vp]
        L.fb_attn_cache_fwd.restype = i32
        L.fb_call.argtypes, L.fb_call.restype = [i32, ctypes.c_char_p, i32], i32
        L.fb_check_device_error.argtypes, L.fb_check_device_error.restype = [vp], i32
        L.fb_selftest_wait_timeout.argtypes, L.fb_selftest_wait_timeout.restype = [i32, vp], i32
        _lib = L
    return _lib


# ---------------------------------------------------------------- raw C ABI

def fb_status_str(status: int) -> str:
    return lib().fb_status_str(int(status)).decode()


def fb_version() -> int:
    return lib().fb_version()


def fb_attn_workspace_bytes(B, H, N, R, phi_bstride, phi_hstride) -> int:
    return lib().fb_attn_workspace_bytes(B, H, N, R, phi_bstride, phi_hstride)


def fb_attn_fwd(dt, B, H, N, d, Q, K, V, R, phi_q, phi_k, phi_bstride, phi_hstride, scale, causal, O, LSE,
                workspace, workspace_bytes, stream) -> int:
    return lib().fb_attn_fwd(dt, B, H, N, d, Q, K, V, R, phi_q, phi_k, phi_bstride, phi_hstride, scale, causal, O,
                             LSE, workspace, workspace_bytes, stream)


def fb_attn_prepare_factors(B, H, N, R, phi_q, phi_k, phi_bstride, phi_hstride, scale, workspace, workspace_bytes,
                            stream) -> int:
    return lib().fb_attn_prepare_factors(B, H, N, R, phi_q, phi_k, phi_bstride, phi_hstride, scale, workspace,
                                         workspace_bytes, stream)


def fb_attn_fwd_prepared(dt, B, H, N, d, Q, K, V, R, phi_bstride, phi_hstride, scale, causal, O, LSE, workspace,
                         workspace_bytes, stream) -> int:
    return lib().fb_attn_fwd_prepared(dt, B, H, N, d, Q, K, V, R, phi_bstride, phi_hstride, scale, causal, O, LSE,
                                      workspace, workspace_bytes, stream)


def fb_attn_mul_bias_workspace_bytes(B, H, N, d, R) -> int:
    return lib().fb_attn_mul_bias_workspace_bytes(B, H, N, d, R)


def fb_attn_mul_bias_fwd(dt, B, H, N, d, Q, K, V, R, phi_q, phi_k, phi_bstride, phi_hstride, scale, causal, O, LSE,
                         workspace, workspace_bytes, stream) -> int:
    return lib().fb_attn_mul_bias_fwd(dt, B, H, N, d, Q, K, V, R, phi_q, phi_k, phi_bstride, phi_hstride, scale,
                                      causal, O, LSE, workspace, workspace_bytes, stream)


def fb_svd_device_workspace_bytes(H, N, R, oversample) -> int:
    return lib().fb_svd_device_workspace_bytes(H, N, R, oversample)


def fb_svd_factors_device(H, N, R, oversample, power_iters, seed, bias, phi_q, phi_k, err_energy, workspace,
                          workspace_bytes, stream) -> int:
    return lib().fb_svd_factors_device(H, N, R, oversample, power_iters, seed, bias, phi_q, phi_k, err_energy,
                                       workspace, workspace_bytes, stream)


def svd_factors_device(bias, R: int, oversample: int = 16, power_iters: int = 2, seed: int = 0):
    """Truncated SVD of dense biases on the GPU (fb_svd_factors_device).

    bias: fp32 CUDA tensor [N, N] or [H, N, N]. Returns (phi_q, phi_k, err_energy)
    with phi [.., N, R] fp32 on the device and err_energy a [H, 2] fp64 device
    tensor (relative Frobenius error, captured energy per head)."""
    import torch
    squeeze = bias.dim() == 2
    b = bias[None] if squeeze else bias
    assert b.is_cuda and b.dtype == torch.float32 and b.is_contiguous()
    H, N, _ = b.shape
    pq = torch.empty((H, N, R), device=b.device, dtype=torch.float32)
    pk = torch.empty_like(pq)
    ee = torch.empty((H, 2), device=b.device, dtype=torch.float64)
    nb = fb_svd_device_workspace_bytes(H, N, R, oversample)
    ws = torch.empty(max(nb, 1), device=b.device, dtype=torch.uint8)
    _check(fb_svd_factors_device(H, N, R, oversample, power_iters, seed, b.data_ptr(), pq.data_ptr(), pk.data_ptr(),
                                 ee.data_ptr(), ws.data_ptr(), nb, _stream(b.device)), "fb_svd_factors_device")
    if squeeze:
        return pq[0], pk[0], ee
    return pq, pk, ee


def fb_attn_neural_workspace_bytes(B, H, N, F, R) -> int:
    return lib().fb_attn_neural_workspace_bytes(B, H, N, F, R)


def fb_attn_neural_fwd(dt, B, H, N, d, Q, K, V, F, R, X_q, X_k, W_q, W_k, scale, causal, O, LSE, workspace,
                       workspace_bytes, stream) -> int:
    return lib().fb_attn_neural_fwd(dt, B, H, N, d, Q, K, V, F, R, X_q, X_k, W_q, W_k, scale, causal, O, LSE,
                                    workspace, workspace_bytes, stream)


def attn_neural(q, k, v, x_q, x_k, w_q, w_k, scale=None, causal=False, out=None, lse=None):
    """Attention whose bias factors come from linear layers on token features
    (fb_attn_neural_fwd): phi_q[b, h] = x_q[b] w_q[h], phi_k[b, h] = x_k[b] w_k[h].

    q, k, v: bf16 CUDA [B, H, N, d]; x_q, x_k: fp32 [B, N, F]; w_q, w_k: fp32
    [H, F, R]. Returns (O, LSE)."""
    import torch
    assert q.is_cuda and q.dtype == torch.bfloat16 and q.is_contiguous() and k.is_contiguous() \
        and v.is_contiguous()
    for t in (x_q, x_k, w_q, w_k):
        assert t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()
    B, H, N, d = q.shape
    F, R = w_q.shape[1], w_q.shape[2]
    assert x_q.shape == (B, N, F) and x_k.shape == (B, N, F) and w_k.shape == (H, F, R)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, H, N), device=q.device, dtype=torch.float32) if lse is None else lse
    nb = fb_attn_neural_workspace_bytes(B, H, N, F, R)
    ws = torch.empty(max(nb, 1), device=q.device, dtype=torch.uint8)
    _check(fb_attn_neural_fwd(FB_BF16, B, H, N, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), F, R, x_q.data_ptr(),
                              x_k.data_ptr(), w_q.data_ptr(), w_k.data_ptr(), scale, int(bool(causal)), o.data_ptr(),
                              l.data_ptr(), ws.data_ptr(), nb, _stream(q.device)), "fb_attn_neural_fwd")
    return o, l


def fb_attn_bwd_workspace_bytes(B, H, N, R, phi_bstride, phi_hstride) -> int:
    return lib().fb_attn_bwd_workspace_bytes(B, H, N, R, phi_bstride, phi_hstride)


def fb_attn_bwd(dt, B, H, N, d, Q, K, V, R, phi_q, phi_k, phi_bstride, phi_hstride, scale, causal, O, LSE, dO,
                dQ, dK, dV, dphi_q, dphi_k, workspace, workspace_bytes, stream) -> int:
    return lib().fb_attn_bwd(dt, B, H, N, d, Q, K, V, R, phi_q, phi_k, phi_bstride, phi_hstride, scale, causal, O,
                             LSE, dO, dQ, dK, dV, dphi_q, dphi_k, workspace, workspace_bytes, stream)


def attn_bwd(q, k, v, phi_q, phi_k, o, lse, do, scale=None, causal=False, workspace=None, factor_grads=True):
    """Gradients of attn's O for an upstream gradient do (fb_attn_bwd).

    q, k, v, o, do: bf16 CUDA [B, H, N, d] contiguous; lse: fp32 [B, H, N]
    from the forward; phi_q, phi_k as for attn (or None). Returns
    (dq, dk, dv, dphi_q, dphi_k): bf16 [B, H, N, d] and fp32 gradients shaped
    like phi_q, phi_k (None without factors, or with factor_grads=False for
    fixed factors, whose gradient products are then skipped)."""
    import torch
    for t in (q, k, v, o, do):
        assert t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()
    B, H, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    R, bs, hs, pq, pk, gq, gk = 0, 0, 0, 0, 0, 0, 0
    dpq = dpk = None
    if phi_q is not None:
        assert phi_q.dtype == torch.float32 and phi_k.dtype == torch.float32
        assert phi_q.shape == phi_k.shape and phi_q.stride() == phi_k.stride() and phi_q.is_contiguous()
        R = phi_q.shape[-1]
        bs, hs = _factor_strides(phi_q, B, H, N, R)
        pq, pk = phi_q.data_ptr(), phi_k.data_ptr()
        if factor_grads:
            dpq, dpk = torch.empty_like(phi_q), torch.empty_like(phi_k)
            gq, gk = dpq.data_ptr(), dpk.data_ptr()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nb = fb_attn_bwd_workspace_bytes(B, H, N, R, bs, hs)
    if workspace is None:
        workspace = torch.empty(max(nb, 1), device=q.device, dtype=torch.uint8)
    _check(fb_attn_bwd(FB_BF16, B, H, N, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), R, pq, pk, bs, hs, scale,
                       int(bool(causal)), o.data_ptr(), lse.data_ptr(), do.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                       dv.data_ptr(), gq, gk, workspace.data_ptr(), nb, _stream(q.device)), "fb_attn_bwd")
    return dq, dk, dv, dpq, dpk


def fb_attn_neural_bwd_workspace_bytes(B, H, N, F, R) -> int:
    return lib().fb_attn_neural_bwd_workspace_bytes(B, H, N, F, R)


def fb_attn_neural_bwd(dt, B, H, N, d, Q, K, V, F, R, X_q, X_k, W_q, W_k, scale, causal, O, LSE, dO, dQ, dK, dV,
                       dX_q, dX_k, dW_q, dW_k, workspace, workspace_bytes, stream) -> int:
    return lib().fb_attn_neural_bwd(dt, B, H, N, d, Q, K, V, F, R, X_q, X_k, W_q, W_k, scale, causal, O, LSE, dO, dQ,
                                    dK, dV, dX_q, dX_k, dW_q, dW_k, workspace, workspace_bytes, stream)


def attn_neural_bwd(q, k, v, x_q, x_k, w_q, w_k, o, lse, do, scale=None, causal=False, feature_grads=True):
    """Gradients of attn_neural's O for an upstream gradient do
    (fb_attn_neural_bwd). Returns (dq, dk, dv, dx_q, dx_k, dw_q, dw_k); dx
    are None with feature_grads=False."""
    import torch
    for t in (q, k, v, o, do):
        assert t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()
    for t in (x_q, x_k, w_q, w_k):
        assert t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()
    B, H, N, d = q.shape
    F, R = w_q.shape[1], w_q.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dwq, dwk = torch.empty_like(w_q), torch.empty_like(w_k)
    dxq = torch.empty_like(x_q) if feature_grads else None
    dxk = torch.empty_like(x_k) if feature_grads else None
    nb = fb_attn_neural_bwd_workspace_bytes(B, H, N, F, R)
    ws = torch.empty(max(nb, 1), device=q.device, dtype=torch.uint8)
    _check(fb_attn_neural_bwd(FB_BF16, B, H, N, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), F, R, x_q.data_ptr(),
                              x_k.data_ptr(), w_q.data_ptr(), w_k.data_ptr(), scale, int(bool(causal)), o.data_ptr(),
                              lse.data_ptr(), do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                              dxq.data_ptr() if dxq is not None else 0, dxk.data_ptr() if dxk is not None else 0,
                              dwq.data_ptr(), dwk.data_ptr(), ws.data_ptr(), nb, _stream(q.device)),
           "fb_attn_neural_bwd")
    return dq, dk, dv, dxq, dxk, dwq, dwk


def fb_attn_fwd_noalloc(dt, B, H, N, d, Q, K, V, R, phi_q, phi_k, phi_bstride, phi_hstride, scale, causal, O, LSE,
                        stream) -> int:
    """fb_attn_fwd without a caller workspace, for callers that cannot allocate
    device memory: the prepared factors go to the library's fixed 8 MiB device
    array (larger needs return FB_ERR_WORKSPACE). Calls that overlap on the GPU
    share that array and must be serialised by the caller."""
    return lib().fb_attn_fwd_noalloc(dt, B, H, N, d, Q, K, V, R, phi_q, phi_k, phi_bstride, phi_hstride, scale,
                                     causal, O, LSE, stream)


def fb_attn_dense_bias_fwd(dt, B, H, N, d, Q, K, V, Bias, bias_bstride, bias_hstride, scale, causal, O, LSE,
                           stream) -> int:
    return lib().fb_attn_dense_bias_fwd(dt, B, H, N, d, Q, K, V, Bias, bias_bstride, bias_hstride, scale, causal, O,
                                        LSE, stream)


def fb_factors_sandwich(N, C, phi_q, phi_k, stream) -> int:
    return lib().fb_factors_sandwich(N, C, phi_q, phi_k, stream)


def fb_factors_alibi(H, N, phi_q, phi_k, stream) -> int:
    return lib().fb_factors_alibi(H, N, phi_q, phi_k, stream)


def fb_svd_factors_host(bias_host, N, R, oversample, power_iters, seed, phi_q_host, phi_k_host, rel_fro_err,
                        energy) -> int:
    return lib().fb_svd_factors_host(bias_host, N, R, oversample, power_iters, seed, phi_q_host, phi_k_host,
                                     rel_fro_err, energy)


def fb_rope_fwd(dt, B, N, d, rot, interleaved, turns, factor, positions, pos_bstride, Hq, Q, q_bstride, q_hstride,
                q_nstride, Q_out, qo_bstride, qo_hstride, qo_nstride, Hk, K, k_bstride, k_hstride, k_nstride, K_out,
                ko_bstride, ko_hstride, ko_nstride, stream) -> int:
    return lib().fb_rope_fwd(dt, B, N, d, rot, interleaved, turns, factor, positions, pos_bstride, Hq, Q, q_bstride,
                             q_hstride, q_nstride, Q_out, qo_bstride, qo_hstride, qo_nstride, Hk, K, k_bstride,
                             k_hstride, k_nstride, K_out, ko_bstride, ko_hstride, ko_nstride, stream)


def fb_rope_bwd(dt, B, N, d, rot, interleaved, turns, factor, positions, pos_bstride, Hq, dQ_out, q_bstride, q_hstride,
                q_nstride, dQ, qo_bstride, qo_hstride, qo_nstride, Hk, dK_out, k_bstride, k_hstride, k_nstride, dK,
                ko_bstride, ko_hstride, ko_nstride, stream) -> int:
    return lib().fb_rope_bwd(dt, B, N, d, rot, interleaved, turns, factor, positions, pos_bstride, Hq, dQ_out,
                             q_bstride, q_hstride, q_nstride, dQ, qo_bstride, qo_hstride, qo_nstride, Hk, dK_out,
                             k_bstride, k_hstride, k_nstride, dK, ko_bstride, ko_hstride, ko_nstride, stream)


def fb_rope_turns_host(pairs, freq_host, turns_host) -> int:
    return lib().fb_rope_turns_host(pairs, freq_host, turns_host)


def fb_rope_frequencies_host(rot, base, scaling, factor, trained, fast, slow, freq_host, out_factor_host) -> int:
    return lib().fb_rope_frequencies_host(rot, base, scaling, factor, trained, fast, slow, freq_host, out_factor_host)


def fb_cache_write(dt, cache_dt, B, H, T, d, K, k_bstride, k_hstride, k_tstride, V, v_bstride, v_hstride, v_tstride,
                   k_pages, v_pages, k_scale, v_scale, num_pages, page_size, block_table, max_pages, starts, counts,
                   stream) -> int:
    return lib().fb_cache_write(dt, cache_dt, B, H, T, d, K, k_bstride, k_hstride, k_tstride, V, v_bstride, v_hstride,
                                v_tstride, k_pages, v_pages, k_scale, v_scale, num_pages, page_size, block_table,
                                max_pages, starts, counts, stream)


def fb_cache_read(dt, cache_dt, B, H, N, d, k_pages, v_pages, k_scale, v_scale, num_pages, page_size, block_table,
                  max_pages, starts, counts, K, V, stream) -> int:
    return lib().fb_cache_read(dt, cache_dt, B, H, N, d, k_pages, v_pages, k_scale, v_scale, num_pages, page_size,
                               block_table, max_pages, starts, counts, K, V, stream)


def fb_cache_bias_bytes(Hq, H, P, R) -> int:
    return lib().fb_cache_bias_bytes(Hq, H, P, R)


def fb_cache_bias_prepare(Hq, H, P, R, phi_q, phi_k, prepared, prepared_bytes, stream) -> int:
    return lib().fb_cache_bias_prepare(Hq, H, P, R, phi_q, phi_k, prepared, prepared_bytes, stream)


def fb_attn_cache_workspace_bytes(B, Hq, H, T, d) -> int:
    return lib().fb_attn_cache_workspace_bytes(B, Hq, H, T, d)


def fb_attn_cache_fwd(cache_dt, B, Hq, H, T, d, Q, k_pages, v_pages, k_scale, v_scale, num_pages, page_size,
                      block_table, max_pages, prefix, counts, tree_mask, mask_words, depths, R, P, phi_q_heads,
                      phi_k_heads, prepared_bias, scale, O, LSE, workspace, workspace_bytes, stream) -> int:
    return lib().fb_attn_cache_fwd(cache_dt, B, Hq, H, T, d, Q, k_pages, v_pages, k_scale, v_scale, num_pages,
                                   page_size, block_table, max_pages, prefix, counts, tree_mask, mask_words, depths, R,
                                   P, phi_q_heads, phi_k_heads, prepared_bias, scale, O, LSE, workspace,
                                   workspace_bytes, stream)


def fb_call(entry, words, count) -> int:
    """words: the arguments packed by the struct module, 8 bytes each (a bytes object)."""
    return lib().fb_call(entry, words, count)


def fb_check_device_error(stream) -> int:
    return lib().fb_check_device_error(stream)


def fb_selftest_wait_timeout(limit_ms, stream) -> int:
    return lib().fb_selftest_wait_timeout(limit_ms, stream)


# ------------------------------------------------- torch-tensor marshalling

def _check(status: int, where: str):
    if status != FB_OK:
        raise FlashBiasError(status, where)


def _stream(device=None) -> int:
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return FB_BF16
    if t.dtype == torch.float32:
        return FB_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16 or float32")


def _factor_strides(phi, B, H, N, R):
    """Element strides (b, h) of a factor tensor broadcastable to [B, H, N, R]."""
    if phi.dim() == 2:  # [N, R]: shared by every head and batch
        return 0, 0
    if phi.dim() == 3:  # [H, N, R]: shared by the batch
        return 0, (phi.stride(0) if phi.shape[0] == H and H > 1 else 0)
    bs = phi.stride(0) if phi.shape[0] == B and B > 1 else 0
    hs = phi.stride(1) if phi.shape[1] == H and H > 1 else 0
    return bs, hs


def attn(q, k, v, phi_q=None, phi_k=None, scale=None, causal=False, out=None, lse=None, workspace=None):
    """O, LSE = softmax(scale q k^T + phi_q phi_k^T [+ causal]) v through fb_attn_fwd.

    q, k, v: CUDA tensors [B, H, N, d] (bf16 or fp32, contiguous).
    phi_q, phi_k: fp32 factors [N, R], [H, N, R] or [B, H, N, R] (last two dims
    contiguous), or None for plain attention. Returns (O, LSE).
    """
    import torch
    assert q.is_cuda and q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
    B, H, N, d = q.shape
    dt = _dtype_code(q)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    R, bs, hs, pq, pk = 0, 0, 0, 0, 0
    if phi_q is not None:
        assert phi_q.dtype == torch.float32 and phi_k.dtype == torch.float32
        assert phi_q.shape == phi_k.shape and phi_q.stride() == phi_k.stride()
        assert phi_q.stride(-1) == 1 and phi_q.stride(-2) == phi_q.shape[-1]
        R = phi_q.shape[-1]
        bs, hs = _factor_strides(phi_q, B, H, N, R)
        pq, pk = phi_q.data_ptr(), phi_k.data_ptr()
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, H, N), device=q.device, dtype=torch.float32) if lse is None else lse
    ws_bytes = fb_attn_workspace_bytes(B, H, N, R, bs, hs) if dt == FB_BF16 else 0
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, device=q.device, dtype=torch.uint8)
    ws_ptr = workspace.data_ptr() if (workspace is not None and ws_bytes) else 0
    _check(fb_attn_fwd(dt, B, H, N, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), R, pq, pk, bs, hs, scale,
                       int(bool(causal)), o.data_ptr(), l.data_ptr(), ws_ptr, ws_bytes, _stream(q.device)),
           "fb_attn_fwd")
    return o, l


def attn_mul_bias(q, k, v, phi_q, phi_k, scale=None, causal=False, out=None, lse=None, workspace=None):
    """O, LSE = softmax(scale (q k^T) o (phi_q phi_k^T) [+ causal]) v through
    fb_attn_mul_bias_fwd (multiplicative low-rank bias; bf16 q, k, v).

    phi_q, phi_k: fp32 [N, R], [H, N, R] or [B, H, N, R] (last two dims
    contiguous). Returns (O, LSE)."""
    import torch
    assert q.is_cuda and q.dtype == torch.bfloat16 and q.is_contiguous() and k.is_contiguous() \
        and v.is_contiguous()
    assert phi_q.dtype == torch.float32 and phi_k.dtype == torch.float32
    assert phi_q.shape == phi_k.shape and phi_q.stride() == phi_k.stride()
    assert phi_q.stride(-1) == 1 and phi_q.stride(-2) == phi_q.shape[-1]
    B, H, N, d = q.shape
    R = phi_q.shape[-1]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    bs, hs = _factor_strides(phi_q, B, H, N, R)
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, H, N), device=q.device, dtype=torch.float32) if lse is None else lse
    ws_bytes = fb_attn_mul_bias_workspace_bytes(B, H, N, d, R)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), device=q.device, dtype=torch.uint8)
    _check(fb_attn_mul_bias_fwd(FB_BF16, B, H, N, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), R, phi_q.data_ptr(),
                                phi_k.data_ptr(), bs, hs, scale, int(bool(causal)), o.data_ptr(), l.data_ptr(),
                                workspace.data_ptr(), ws_bytes, _stream(q.device)), "fb_attn_mul_bias_fwd")
    return o, l


class PreparedBias:
    """Factors prepared once (fb_attn_prepare_factors) for many bf16 calls.

    phi_q, phi_k as for attn(); B, H, N the shape of the q tensors it will be
    used with; scale the softmax scale (it is folded into the prepared
    factors). Call it as attn(q, k, v, causal=...) -> (O, LSE)."""

    def __init__(self, phi_q, phi_k, B: int, H: int, N: int, d: int, scale=None):
        import torch
        assert phi_q.dtype == torch.float32 and phi_k.dtype == torch.float32
        assert phi_q.shape == phi_k.shape and phi_q.stride() == phi_k.stride()
        assert phi_q.stride(-1) == 1 and phi_q.stride(-2) == phi_q.shape[-1]
        self.B, self.H, self.N, self.d = B, H, N, d
        self.R = phi_q.shape[-1]
        self.scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
        self.bs, self.hs = _factor_strides(phi_q, B, H, N, self.R)
        self.ws_bytes = fb_attn_workspace_bytes(B, H, N, self.R, self.bs, self.hs)
        self.workspace = torch.empty(max(self.ws_bytes, 1), device=phi_q.device, dtype=torch.uint8)
        _check(fb_attn_prepare_factors(B, H, N, self.R, phi_q.data_ptr(), phi_k.data_ptr(), self.bs, self.hs,
                                       self.scale, self.workspace.data_ptr(), self.ws_bytes,
                                       _stream(phi_q.device)), "fb_attn_prepare_factors")

    def attn(self, q, k, v, causal=False, out=None, lse=None):
        import torch
        assert q.is_cuda and q.dtype == torch.bfloat16 and q.is_contiguous() and k.is_contiguous() \
            and v.is_contiguous()
        B, H, N, d = q.shape
        assert (B, H, N, d) == (self.B, self.H, self.N, self.d)
        o = torch.empty_like(q) if out is None else out
        l = torch.empty((B, H, N), device=q.device, dtype=torch.float32) if lse is None else lse
        _check(fb_attn_fwd_prepared(FB_BF16, B, H, N, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), self.R, self.bs,
                                    self.hs, self.scale, int(bool(causal)), o.data_ptr(), l.data_ptr(),
                                    self.workspace.data_ptr(), self.ws_bytes, _stream(q.device)),
               "fb_attn_fwd_prepared")
        return o, l


def attn_dense_bias(q, k, v, bias, scale=None, causal=False, out=None, lse=None):
    """The dense-bias comparison path through fb_attn_dense_bias_fwd.

    bias: [N, N], [H, N, N] or [B, H, N, N] tensor of q's dtype (last two dims
    contiguous). Returns (O, LSE).
    """
    import torch
    B, H, N, d = q.shape
    dt = _dtype_code(q)
    assert bias.dtype == q.dtype and bias.stride(-1) == 1 and bias.stride(-2) == N
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if bias.dim() == 2:
        bs, hs = 0, 0
    elif bias.dim() == 3:
        bs, hs = 0, (bias.stride(0) if H > 1 else 0)
    else:
        bs = bias.stride(0) if (bias.shape[0] == B and B > 1) else 0
        hs = bias.stride(1) if (bias.shape[1] == H and H > 1) else 0
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, H, N), device=q.device, dtype=torch.float32) if lse is None else lse
    _check(fb_attn_dense_bias_fwd(dt, B, H, N, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), bias.data_ptr(), bs, hs,
                                  scale, int(bool(causal)), o.data_ptr(), l.data_ptr(), _stream(q.device)),
           "fb_attn_dense_bias_fwd")
    return o, l


def factors_sandwich(N: int, C: int, device="cuda"):
    """Exact Sandwich factors phi [N, C] fp32 (phi_q = phi_k); one kernel."""
    import torch
    phi = torch.empty((N, C), device=device, dtype=torch.float32)
    _check(fb_factors_sandwich(N, C, phi.data_ptr(), phi.data_ptr(), _stream(phi.device)), "fb_factors_sandwich")
    return phi


def factors_alibi(H: int, N: int, device="cuda"):
    """Exact rank-2 ALiBi factors (phi_q, phi_k), each [H, N, 2] fp32; one kernel."""
    import torch
    pq = torch.empty((H, N, 2), device=device, dtype=torch.float32)
    pk = torch.empty((H, N, 2), device=device, dtype=torch.float32)
    _check(fb_factors_alibi(H, N, pq.data_ptr(), pk.data_ptr(), _stream(pq.device)), "fb_factors_alibi")
    return pq, pk


def svd_factors(bias, R: int, oversample: int = 16, power_iters: int = 2, seed: int = 0):
    """Host truncated SVD of one head's bias (numpy float64 [N, N]).

    Returns (phi_q [N, R] fp32, phi_k [N, R] fp32, rel_fro_err, energy) as numpy.
    """
    import numpy as np
    b = np.ascontiguousarray(bias, dtype=np.float64)
    N = b.shape[0]
    assert b.shape == (N, N)
    pq = np.empty((N, R), dtype=np.float32)
    pk = np.empty((N, R), dtype=np.float32)
    err, en = ctypes.c_double(), ctypes.c_double()
    _check(fb_svd_factors_host(b.ctypes.data, N, R, oversample, power_iters, seed, pq.ctypes.data, pk.ctypes.data,
                               ctypes.addressof(err), ctypes.addressof(en)), "fb_svd_factors_host")
    return pq, pk, err.value, en.value


def attn_flops(B: int, H: int, N: int, d: int, R: int, causal: bool) -> float:
    """Counted FLOPs: 4 N^2 d + 2 N^2 R per head, halved when causal."""
    f = float(B) * H * (4.0 * N * N * d + 2.0 * N * N * R)
    return f / 2.0 if causal else f


# ------------------------------------------------- serving: rotary positions, paged cache, attention over it

class _Entry:
    """One entry of fb_call. Called with the device and the arguments but the stream, which is the device's current one;
    the device is made the current one for the call where it is not."""

    def __init__(self, entry: int, where: str, words: str):
        self.entry, self.where, self.count = entry, where, len(words) + 1
        self.pack = struct.Struct("=" + words + "q").pack

    def __call__(self, index: int, *args):
        import torch
        words = self.pack(*args, torch._C._cuda_getCurrentRawStream(index))
        L = _lib or lib()
        now = torch.cuda.current_device()
        if now == index:
            status = L.fb_call(self.entry, words, self.count)
        else:
            with torch.cuda.device(index):
                status = L.fb_call(self.entry, words, self.count)
        if status != FB_OK:
            raise FlashBiasError(status, self.where)


_rope_fwd = _Entry(0, "fb_rope_fwd", 7 * "q" + "d" + 20 * "q")
_rope_bwd = _Entry(1, "fb_rope_bwd", 7 * "q" + "d" + 20 * "q")
_cache_write = _Entry(2, "fb_cache_write", 24 * "q")
_cache_read = _Entry(3, "fb_cache_read", 18 * "q")
_attn_cache = _Entry(4, "fb_attn_cache_fwd", 25 * "q" + "d" + 4 * "q")


def _code(dtype):
    """FB_BF16, FB_F32, or None."""
    import torch
    return FB_BF16 if dtype is torch.bfloat16 else (FB_F32 if dtype is torch.float32 else None)


def _ints(t, shape, index: int, what: str) -> int:
    """Pointer of a contiguous int32 tensor of this shape on CUDA device `index` (0 for None)."""
    import torch
    if t is None:
        return 0
    if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous int32 tensor {tuple(shape)} on cuda:{index}")
    return t.data_ptr()


class Rope:
    """Rotary positions: the angle per position of each rotated pair.

    frequencies: rot / 2 numbers; the first rot values of a head turn, pair p
    being (2p, 2p + 1) when interleaved, else (p, p + rot / 2). factor
    multiplies the turned values. Rope.scaled makes the usual frequencies."""

    SCALINGS = ("none", "linear", "base", "yarn", "bands")

    def __init__(self, frequencies, interleaved=False, factor=1.0, device="cuda"):
        import torch
        pairs = len(frequencies)
        if not (pairs >= 1):
            raise ValueError("Rope: at least one pair")
        freq = (ctypes.c_double * pairs)(*[float(w) for w in frequencies])
        turns = (ctypes.c_uint64 * pairs)()
        _check(fb_rope_turns_host(pairs, ctypes.addressof(freq), ctypes.addressof(turns)), "fb_rope_turns_host")
        self.frequencies = list(freq)
        self.rot, self.interleaved, self.factor = 2 * pairs, bool(interleaved), float(factor)
        if not (math.isfinite(self.factor) and self.factor != 0.0):
            raise ValueError("Rope: factor finite and not 0")
        # 2^-64 turns as two's complement: torch's uint64 has few operations
        signed = [t - (1 << 64) if t >> 63 else t for t in turns]
        self.turns = torch.tensor(signed, dtype=torch.int64, device=device)
        self.index, self.pointer = self.turns.get_device(), self.turns.data_ptr()

    @classmethod
    def scaled(cls, rot: int, base=10000.0, scaling="none", by=1.0, trained=4096.0, fast=32.0, slow=1.0,
               interleaved=False, factor=None, device="cuda"):
        """base^(-2p / rot), for contexts `by` times the trained length (fb_rope_frequencies_host)."""
        if not (scaling in cls.SCALINGS):
            raise ValueError(f"Rope.scaled: scaling one of {cls.SCALINGS}")
        freq, out = (ctypes.c_double * max(rot // 2, 1))(), ctypes.c_double()
        _check(fb_rope_frequencies_host(rot, base, cls.SCALINGS.index(scaling), by, trained, fast, slow,
                                        ctypes.addressof(freq), ctypes.addressof(out)), "fb_rope_frequencies_host")
        return cls(freq, interleaved, out.value if factor is None else factor, device)


def _side(x, what: str):
    """Heads, pointer and strides of a [B, H, N, d] tensor with d contiguous."""
    if x.dim() != 4:
        raise ValueError(f"{what}: a tensor [B, H, N, d]")
    sb, sh, sn, sd = x.stride()
    if sd != 1 and x.shape[3] > 1:
        raise ValueError(f"{what}: the last dimension contiguous")
    return x.data_ptr(), sb, sh, sn


def _rope(call, q, k, rope, positions, out):
    import torch
    B, Hq, N, d = q.shape
    index, dt = q.get_device(), _code(q.dtype)
    if dt is None or index < 0:
        raise ValueError(f"{call.where}: q a bfloat16 or float32 CUDA tensor [B, H, N, d]")
    if rope.index != index:
        raise ValueError(f"{call.where}: the Rope is on another device")
    if out is None:
        qo, ko = torch.empty_like(q), None if k is None else torch.empty_like(k)
    else:
        qo, ko = out
        for x, y in ((q, qo), (k, ko)):
            if (x is None) != (y is None) or x is not None and not (
                    y.shape == x.shape and y.dtype is x.dtype and y.get_device() == index
                    and all(s > 0 or n <= 1 for s, n in zip(y.stride(), y.shape))):
                raise ValueError(f"{call.where}: out like q and k, with a place of its own for every value")
    qp, qb, qh, qn = _side(q, "q")
    op, ob, oh, on = _side(qo, "q's output")
    if k is None:
        Hk = kp = kb = kh = kn = rp = rb = rh = rn = 0
    else:
        Bk, Hk, Nk, dk = k.shape
        if Bk != B or Nk != N or dk != d or k.dtype is not q.dtype or k.get_device() != index:
            raise ValueError(f"{call.where}: k [B, Hk, N, d] like q")
        kp, kb, kh, kn = _side(k, "k")
        rp, rb, rh, rn = _side(ko, "k's output")
    pos = pos_bs = 0
    if positions is not None:
        shape = positions.shape
        if not (positions.dtype is torch.int32 and positions.get_device() == index and shape[-1] == N
                and (N == 1 or positions.stride(-1) == 1)
                and (len(shape) == 1 or len(shape) == 2 and shape[0] in (1, B))):
            raise ValueError(f"{call.where}: positions int32 [N], [1, N] or [B, N] on q's device, contiguous along N")
        pos = positions.data_ptr()
        if len(shape) == 2 and shape[0] > 1:
            pos_bs = positions.stride(0)
    call(index, dt, B, N, d, rope.rot, rope.interleaved, rope.pointer, rope.factor, pos, pos_bs, Hq, qp, qb, qh, qn, op,
         ob, oh, on, Hk, kp, kb, kh, kn, rp, rb, rh, rn)
    return qo, ko


def rope(q, k, rope, positions=None, out=None):
    """Queries and keys turned by their positions (fb_rope_fwd); returns (q, k).

    q, k: bf16 or fp32 CUDA [B, H, N, d] in any order of the first three
    dimensions (d contiguous); k may be None. positions: int32 [N], [1, N] or
    [B, N], or None for 0 .. N - 1. out: (q, k) to write to, which may be the
    inputs themselves."""
    return _rope(_rope_fwd, q, k, rope, positions, out)


def rope_bwd(dq, dk, rope, positions=None, out=None):
    """Gradients of rope's inputs from those of its outputs (fb_rope_bwd); arguments as for rope."""
    return _rope(_rope_bwd, dq, dk, rope, positions, out)


class PagedCache:
    """A paged key/value cache: pools k, v [pages, H, page, d], bf16 or e4m3.

    An e4m3 cache has k_scale, v_scale [pages, H, page] (float8_e8m0fnu or
    uint8, 2^(byte - 127)). The tensors are used as they are, not copied."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        if not (k.is_cuda and k.dim() == 4 and k.dtype in (torch.bfloat16, torch.float8_e4m3fn) and k.is_contiguous()):
            raise ValueError("PagedCache: k a contiguous CUDA tensor [pages, H, page, d], bfloat16 or float8_e4m3fn")
        if not (v.shape == k.shape and v.dtype == k.dtype and v.device == k.device and v.is_contiguous()):
            raise ValueError("PagedCache: v like k")
        self.dt = FB_E4M3 if k.dtype == torch.float8_e4m3fn else FB_BF16
        for s in (k_scale, v_scale):
            if not ((s is None) == (self.dt == FB_BF16)):
                raise ValueError("PagedCache: scales for float8_e4m3fn, none for bfloat16")
            if s is not None:
                if not (s.dtype in (torch.float8_e8m0fnu, torch.uint8) and s.shape == k.shape[:3]
                        and s.device == k.device and s.is_contiguous()):
                    raise ValueError("PagedCache: scales float8_e8m0fnu or uint8 [pages, H, page]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.index = k.device, k.get_device()
        self.num_pages, self.heads, self.page, self.d = k.shape

    @classmethod
    def empty(cls, num_pages: int, heads: int, page: int, d: int, dtype=None, device="cuda"):
        """A cache of its own memory, its contents undefined (dtype: bfloat16, or float8_e4m3fn)."""
        import torch
        dtype = torch.bfloat16 if dtype is None else dtype
        kv = [torch.empty((num_pages, heads, page, d), dtype=dtype, device=device) for _ in range(2)]
        if dtype != torch.float8_e4m3fn:
            return cls(*kv)
        return cls(*kv, *[torch.empty((num_pages, heads, page), dtype=torch.uint8, device=device).view(
            torch.float8_e8m0fnu) for _ in range(2)])

    def _pointers(self):
        # afresh at each call: the tensors are the user's, who may have resized or moved them
        if self.dt == FB_BF16:
            return self.k.data_ptr(), self.v.data_ptr(), 0, 0, self.num_pages, self.page
        return (self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(), self.num_pages,
                self.page)

    def _table(self, table, B):
        import torch
        if not (table.dtype is torch.int32 and table.dim() == 2 and table.shape[0] == B
                and table.get_device() == self.index and table.is_contiguous()):
            raise ValueError(f"block table: a contiguous int32 tensor [{B}, pages] on cuda:{self.index}")
        return table.data_ptr(), table.shape[1]


def cache_write(cache: PagedCache, k, v, table, starts, counts=None):
    """New keys and values into the cache (fb_cache_write): row n < counts[b] of
    k, v [B, H, N, d] (bf16 or fp32, any order of the first three dimensions)
    becomes token starts[b] + n of sequence b. table: int32 [B, max_pages];
    starts, counts: int32 [B] (counts None: every row)."""
    B, H, N, d = k.shape
    index, dt = cache.index, _code(k.dtype)
    if (H != cache.heads or d != cache.d or dt is None or k.get_device() != index or v.shape != k.shape
            or v.dtype is not k.dtype or v.get_device() != index):
        raise ValueError(f"cache_write: k, v bfloat16 or float32 [B, {cache.heads}, N, {cache.d}] on cuda:{index}")
    if starts is None:
        raise ValueError("cache_write: starts")
    kx, kb, kh, kn = _side(k, "k")
    vx, vb, vh, vn = _side(v, "v")
    tab, width = cache._table(table, B)
    kp, vp, ks, vs, pages, page = cache._pointers()
    _cache_write(index, dt, cache.dt, B, H, N, d, kx, kb, kh, kn, vx, vb, vh, vn, kp, vp, ks, vs, pages, page, tab,
                 width, _ints(starts, (B,), index, "starts"), _ints(counts, (B,), index, "counts"))


def cache_read(cache: PagedCache, table, starts, counts, tokens: int, dtype=None, out=None):
    """Tokens starts[b] .. starts[b] + counts[b] - 1 of each sequence as (k, v)
    [B, H, tokens, d] (fb_cache_read), rows past counts[b] zero; dtype bfloat16
    (the default) or float32. starts None: from 0; counts None: all tokens."""
    import torch
    B, index = table.shape[0], cache.index
    tab, width = cache._table(table, B)
    shape = (B, cache.heads, tokens, cache.d)
    if out is None:
        dtype = torch.bfloat16 if dtype is None else dtype
        k = torch.empty(shape, dtype=dtype, device=cache.device)
        v = torch.empty_like(k)
    else:
        k, v = out
        if not (all(t.shape == shape and t.get_device() == index and t.is_contiguous() and t.dtype is k.dtype
                    for t in (k, v)) and dtype in (None, k.dtype)):
            raise ValueError(f"cache_read: out two contiguous tensors {shape}")
    dt = _code(k.dtype)
    if dt is None:
        raise ValueError("cache_read: dtype bfloat16 or float32")
    kp, vp, ks, vs, pages, page = cache._pointers()
    _cache_read(index, dt, cache.dt, B, cache.heads, tokens, cache.d, kp, vp, ks, vs, pages, page, tab, width,
                _ints(starts, (B,), index, "starts"), _ints(counts, (B,), index, "counts"), k.data_ptr(), v.data_ptr())
    return k, v


class CacheBias:
    """Bias factors laid out once for attn_cache (fb_cache_bias_prepare).

    phi_q [Hq, P, R] and phi_k [H, P, R], or [1, P, R] or [P, R] where all heads
    share them, fp32, over positions 0 .. P - 1. The factors are copied."""

    def __init__(self, phi_q, phi_k):
        import torch
        phi_q, phi_k = (x[None] if x.dim() == 2 else x for x in (phi_q, phi_k))
        for x in (phi_q, phi_k):
            if not (x.is_cuda and x.dim() == 3 and x.dtype == torch.float32):
                raise ValueError("CacheBias: fp32 CUDA factors [heads, P, R]")
        if not (phi_q.shape[1:] == phi_k.shape[1:] and phi_q.device == phi_k.device):
            raise ValueError("CacheBias: factors of one length, rank and device")
        phi_q, phi_k = phi_q.contiguous(), phi_k.contiguous()
        self.device = phi_q.device
        self.q_heads, self.P, self.R = phi_q.shape
        self.k_heads = phi_k.shape[0]
        nb = fb_cache_bias_bytes(self.q_heads, self.k_heads, self.P, self.R)
        self.prepared = torch.empty(max(nb, 1), device=self.device, dtype=torch.uint8)
        with torch.cuda.device(self.device):
            _check(fb_cache_bias_prepare(self.q_heads, self.k_heads, self.P, self.R, phi_q.data_ptr(), phi_k.data_ptr(),
                                         self.prepared.data_ptr(), nb, _stream(self.device)), "fb_cache_bias_prepare")
        self.index = phi_q.get_device()
        # the five words that a call takes
        self.words = self.R, self.P, self.q_heads, self.k_heads, self.prepared.data_ptr()


def cache_workspace(B: int, Hq: int, H: int, T: int, d: int, device="cuda"):
    """A workspace for attn_cache calls of these sizes (one per call that can run at the same time)."""
    import torch
    nb = fb_attn_cache_workspace_bytes(B, Hq, H, T, d)
    if not (nb > 0):
        raise ValueError(f"cache_workspace: unsupported sizes B={B} Hq={Hq} H={H} T={T} d={d}")
    return torch.zeros(nb, device=device, dtype=torch.uint8)


def attn_cache(q, cache: PagedCache, table, prefix, counts=None, tree_mask=None, depths=None, bias=None, scale=None,
               workspace=None, out=None, lse=None):
    """Attention of new tokens over the cache (fb_attn_cache_fwd); returns (O, LSE).

    q: bf16 [B, Hq, T, d] contiguous, T = 1 for a decode step. table: int32
    [B, max_pages]; prefix: int32 [B], each sequence's context, its new tokens
    being cache tokens prefix[b] + t; counts: int32 [B], how many of the T it
    brings (None: T). tree_mask: int32 [B, T, words], bit u of row t set where
    new token t sees new token u (None: u <= t); depths: int32 [B, T], a new
    token's position after the prefix (None: t). bias: a CacheBias, or None.
    workspace: of cache_workspace (None: allocated here, at the cost of a
    memset)."""
    import torch
    B, Hq, T, d = q.shape
    index, H = cache.index, cache.heads
    if q.dtype is not torch.bfloat16 or q.get_device() != index or d != cache.d or not q.is_contiguous():
        raise ValueError(f"attn_cache: q a contiguous bfloat16 tensor [B, Hq, T, {cache.d}] on cuda:{index}")
    tab, width = cache._table(table, B)
    mask = words = 0
    if tree_mask is not None:
        words = tree_mask.shape[-1]
        mask = _ints(tree_mask, (B, T, words), index, "tree_mask")
    R = P = fq = fk = pb = 0
    if bias is not None:
        if bias.index != index:
            raise ValueError("attn_cache: the bias is on another device")
        R, P, fq, fk, pb = bias.words
    if out is None:
        out = torch.empty_like(q)
    elif not (out.shape == q.shape and out.dtype is q.dtype and out.get_device() == index and out.is_contiguous()):
        raise ValueError("attn_cache: out like q")
    if lse is None:
        lse = torch.empty((B, Hq, T), device=cache.device, dtype=torch.float32)
    elif not (lse.shape == (B, Hq, T) and lse.dtype is torch.float32 and lse.get_device() == index
              and lse.is_contiguous()):
        raise ValueError("attn_cache: lse a contiguous float32 tensor [B, Hq, T]")
    if workspace is None:
        nb = fb_attn_cache_workspace_bytes(B, Hq, H, T, d)
        workspace = torch.zeros(max(nb, 1), device=cache.device, dtype=torch.uint8)
    if workspace.dtype is not torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("attn_cache: a workspace of cache_workspace")
    kp, vp, ks, vs, pages, page = cache._pointers()
    _attn_cache(index, cache.dt, B, Hq, H, T, d, q.data_ptr(), kp, vp, ks, vs, pages, page, tab, width,
                _ints(prefix, (B,), index, "prefix"), _ints(counts, (B,), index, "counts"), mask, words,
                _ints(depths, (B, T), index, "depths"), R, P, fq, fk, pb, d ** -0.5 if scale is None else scale,
                out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel())
    return out, lse
