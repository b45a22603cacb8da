"""ctypes binding of libspa.so: argument marshalling only.

Torch tensors supply data pointers, shapes and the current CUDA stream; the
functions raise ``SpaError`` on any non-zero status.  Names follow the C ABI.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_PKG, "libspa.so")

if not os.path.exists(lib_path):
    raise ImportError(
        f"libspa.so is not built ({lib_path}); build it with "
        "`python -m projected_feature_efficient_gb300.build` (needs nvcc)")

lib = ctypes.CDLL(lib_path)

SPA_F32, SPA_BF16 = 0, 1
SPA_OK, SPA_ERR_TIMEOUT = 0, 8  # spa_status values (include/spa.h)
_vp, _i, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t

lib.spa_status_str.argtypes = [_i]
lib.spa_status_str.restype = ctypes.c_char_p
lib.spa_version.argtypes = []
lib.spa_version.restype = _i
lib.spa_project.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]
lib.spa_project.restype = _i
lib.spa_attention_fwd.argtypes = [_vp] * 5 + [_i] * 8 + [_vp]
lib.spa_attention_fwd.restype = _i
lib.spa_attention_workspace_size.argtypes = [_i] * 7 + [ctypes.POINTER(_sz)]
lib.spa_attention_workspace_size.restype = _i
lib.spa_attention_fwd_ws.argtypes = [_vp] * 5 + [_i] * 8 + [_vp, _sz, _vp]
lib.spa_attention_fwd_ws.restype = _i
lib.spa_attention_fwd_host.argtypes = [_vp] * 5 + [_i] * 8 + [_vp]
lib.spa_attention_fwd_host.restype = _i
lib.spa_attention_prepare.argtypes = [_vp] * 3 + [_i] * 7 + [_vp, _sz, _vp]
lib.spa_attention_prepare.restype = _i
lib.spa_attention_apply.argtypes = [_vp] * 2 + [_i] * 8 + [_vp, _sz, _vp]
lib.spa_attention_apply.restype = _i
lib.spa_attention_fwd_noalloc.argtypes = [_vp] * 5 + [_i] * 8 + [_vp]
lib.spa_attention_fwd_noalloc.restype = _i
lib.spa_device_error.argtypes = [ctypes.POINTER(_i)]
lib.spa_device_error.restype = _i
lib.spa_selftest_wait_timeout.argtypes = [_i]
lib.spa_selftest_wait_timeout.restype = _i
lib.spa_selftest_bwd_wait_timeout.argtypes = [_i]
lib.spa_selftest_bwd_wait_timeout.restype = _i
lib.spa_selftest_proj_wait_timeout.argtypes = [_i, _i]
lib.spa_selftest_proj_wait_timeout.restype = _i
lib.spa_selftest_copy_wait_timeout.argtypes = [_i, _i]
lib.spa_selftest_copy_wait_timeout.restype = _i
lib.spa_selftest_decode_wait_timeout.argtypes = [_i, _i]
lib.spa_selftest_decode_wait_timeout.restype = _i
lib.spa_attention_bwd.argtypes = [_vp] * 10 + [_i] * 8 + [_vp]
lib.spa_attention_bwd.restype = _i
lib.spa_host_pool_trim.argtypes = []
lib.spa_host_pool_trim.restype = _i
lib.spa_attention_bwd_lse.argtypes = [_vp] * 11 + [_i] * 8 + [_vp]
lib.spa_attention_bwd_lse.restype = _i
lib.spa_attention_fwd_lse.argtypes = [_vp] * 6 + [_i] * 8 + [_vp]
lib.spa_attention_fwd_lse.restype = _i
lib.spa_attention_bwd_workspace_size.argtypes = [_i] * 7 + [ctypes.POINTER(_sz)]
lib.spa_attention_bwd_workspace_size.restype = _i
lib.spa_attention_bwd_prepare.argtypes = [_vp] * 6 + [_i] * 7 + [_vp, _sz, _vp]
lib.spa_attention_bwd_prepare.restype = _i
lib.spa_attention_bwd_apply.argtypes = [_vp] * 3 + [_i] * 8 + [_vp, _sz, _vp]
lib.spa_attention_bwd_apply.restype = _i
lib.spa_attention_bwd_finish.argtypes = [_vp] * 6 + [_i] * 7 + [_vp, _sz, _vp]
lib.spa_attention_bwd_finish.restype = _i
lib.spa_topk_features.argtypes = [_vp, _vp, ctypes.c_longlong, _i, _i, _i, _vp]
lib.spa_topk_features.restype = _i
lib.spa_sfa_attention_fwd.argtypes = [_vp] * 4 + [_i] * 8 + [_vp]
lib.spa_sfa_attention_fwd.restype = _i
lib.spa_kcache_append.argtypes = [_vp] * 4 + [_i] * 8 + [_vp]
lib.spa_kcache_append.restype = _i
lib.spa_attention_decode.argtypes = [_vp] * 6 + [_i] * 8 + [_vp]
lib.spa_attention_decode.restype = _i
_d, _ll, _pd = ctypes.c_double, ctypes.c_longlong, ctypes.POINTER(ctypes.c_double)
lib.spa_rope_frequencies.argtypes = [_pd, _i, _d, _i, _d, _d, _d, _d]
lib.spa_rope_frequencies.restype = _i
lib.spa_rope_table.argtypes = [_pd, _i, ctypes.POINTER(ctypes.c_ulonglong)]
lib.spa_rope_table.restype = _i
lib.spa_rope.argtypes = ([_vp] * 4 + [ctypes.POINTER(_ll), _vp, _i, _vp] + [_i] * 8 +
                         [ctypes.c_float, _i, _vp])
lib.spa_rope.restype = _i
lib.spa_kcache_append_ragged.argtypes = [_vp] * 11 + [_i] * 8 + [_vp]
lib.spa_kcache_append_ragged.restype = _i
lib.spa_attention_decode_shared_workspace_size.argtypes = [_i] * 9 + [ctypes.POINTER(_sz)]
lib.spa_attention_decode_shared_workspace_size.restype = _i
lib.spa_attention_decode_shared.argtypes = [_vp] * 12 + [_i] * 10 + [_vp, _sz, _vp]
lib.spa_attention_decode_shared.restype = _i
lib.spa_kcache_evict_workspace_size.argtypes = [_i] * 4 + [ctypes.POINTER(_sz)]
lib.spa_kcache_evict_workspace_size.restype = _i
lib.spa_kcache_evict.argtypes = [_vp] * 10 + [_i] * 8 + [_vp, _sz, _vp]
lib.spa_kcache_evict.restype = _i


class SpaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)}")


def status_str(status: int) -> str:
    return lib.spa_status_str(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise SpaError(status, where)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return SPA_BF16
    if t.dtype == torch.float32:
        return SPA_F32
    raise TypeError(f"unsupported dtype {t.dtype}: use torch.bfloat16 or torch.float32")


def _stream_ptr(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _shapes(q, k, v, P):
    B, H, N, d = q.shape
    dv = v.shape[-1]
    m = P.shape[-1]
    if tuple(k.shape) != (B, H, N, d) or tuple(v.shape) != (B, H, N, dv) or \
            tuple(P.shape) != (H, d, m):
        raise ValueError("shapes: q,k [B,H,N,d]; v [B,H,N,dv]; P [H,d,m]")
    for t in (q, k, v, P):
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
    if len({t.dtype for t in (q, k, v, P)}) != 1:
        raise TypeError("q, k, v and P must share one dtype")
    return B, H, N, d, m, dv


def spa_project(x, P, out=None, stream=None):
    """x [B,H,N,d] @ P [H,d,m] -> fp32 [B,H,N,m] (device tensors)."""
    import torch
    B, H, N, d = x.shape
    m = P.shape[-1]
    if tuple(P.shape) != (H, d, m) or x.dtype != P.dtype:
        raise ValueError("P must be [H,d,m] with x's dtype")
    if out is None:
        out = torch.empty((B, H, N, m), dtype=torch.float32, device=x.device)
    _check(lib.spa_project(_ptr(x), _ptr(P), _ptr(out), B, H, N, d, m, _dtype_code(x),
                           _stream_ptr(stream)), "spa_project")
    return out


def spa_attention_fwd(q, k, v, P, causal=False, out=None, stream=None):
    """Forward on device tensors; returns fp32 [B,H,N,dv]."""
    import torch
    B, H, N, d, m, dv = _shapes(q, k, v, P)
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=torch.float32, device=q.device)
    _check(lib.spa_attention_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(P), _ptr(out), B, H, N, d, m,
                                 dv, int(bool(causal)), _dtype_code(q), _stream_ptr(stream)),
           "spa_attention_fwd")
    return out


def spa_attention_workspace_size(B, H, N, d, m, dv, dtype_code) -> int:
    n = _sz(0)
    _check(lib.spa_attention_workspace_size(B, H, N, d, m, dv, dtype_code, ctypes.byref(n)),
           "spa_attention_workspace_size")
    return int(n.value)


def spa_attention_fwd_ws(q, k, v, P, workspace, causal=False, out=None, stream=None):
    """Forward with a caller-provided device workspace (uint8 tensor)."""
    import torch
    B, H, N, d, m, dv = _shapes(q, k, v, P)
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=torch.float32, device=q.device)
    _check(lib.spa_attention_fwd_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(P), _ptr(out), B, H, N, d, m,
                                    dv, int(bool(causal)), _dtype_code(q), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _stream_ptr(stream)), "spa_attention_fwd_ws")
    return out


def spa_attention_prepare(q, k, P, dv, workspace, stream=None):
    """Stage 1 of the forward: project q and k into `workspace` (uint8 device tensor)."""
    B, H, N, d = q.shape
    m = P.shape[-1]
    if tuple(k.shape) != (B, H, N, d) or tuple(P.shape) != (H, d, m):
        raise ValueError("shapes: q,k [B,H,N,d]; P [H,d,m]")
    _check(lib.spa_attention_prepare(_ptr(q), _ptr(k), _ptr(P), B, H, N, d, m, dv,
                                     _dtype_code(q), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(),
                                     _stream_ptr(stream)), "spa_attention_prepare")


def spa_attention_apply(v, workspace, B, H, N, d, m, causal=False, out=None, stream=None,
                        dtype_code=None):
    """Stage 2 of the forward from a prepared workspace; returns fp32 [B,H,N,dv]."""
    import torch
    dv = v.shape[-1]
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=torch.float32, device=v.device)
    code = _dtype_code(v) if dtype_code is None else dtype_code
    _check(lib.spa_attention_apply(_ptr(v), _ptr(out), B, H, N, d, m, dv, int(bool(causal)),
                                   code, _ptr(workspace),
                                   workspace.numel() * workspace.element_size(),
                                   _stream_ptr(stream)), "spa_attention_apply")
    return out


def spa_attention_fwd_host(q, k, v, P, causal=False, out=None, stream=None):
    """End-to-end form on host (CPU) tensors: copies in, computes, copies out."""
    import torch
    B, H, N, d, m, dv = _shapes(q, k, v, P)
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=torch.float32)
    _check(lib.spa_attention_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(P), _ptr(out), B, H, N, d,
                                      m, dv, int(bool(causal)), _dtype_code(q),
                                      _stream_ptr(stream)), "spa_attention_fwd_host")
    return out


def spa_attention_bwd(q, k, v, P, out, dO, causal=False, stream=None):
    """Gradients (dq, dk, dv, dP) of spa_attention_fwd for the upstream gradient
    dO (same type as q), given the forward's fp32 output `out`."""
    import torch
    B, H, N, d, m, dv = _shapes(q, k, v, P)
    dev = q.device
    dq = torch.empty((B, H, N, d), dtype=torch.float32, device=dev)
    dk = torch.empty((B, H, N, d), dtype=torch.float32, device=dev)
    dvo = torch.empty((B, H, N, dv), dtype=torch.float32, device=dev)
    dP = torch.empty((H, d, m), dtype=torch.float32, device=dev)
    _check(lib.spa_attention_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(P), _ptr(out), _ptr(dO), _ptr(dq),
                                 _ptr(dk), _ptr(dvo), _ptr(dP), B, H, N, d, m, dv,
                                 int(bool(causal)), _dtype_code(q), _stream_ptr(stream)),
           "spa_attention_bwd")
    return dq, dk, dvo, dP


def spa_attention_fwd_lse(q, k, v, P, causal=False, out=None, lse=None, stream=None):
    """Forward that also returns the row log-sum-exp of the logits: (out, lse),
    out fp32 [B,H,N,dv], lse fp32 [B,H,N]."""
    import torch
    B, H, N, d, m, dv = _shapes(q, k, v, P)
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check(lib.spa_attention_fwd_lse(_ptr(q), _ptr(k), _ptr(v), _ptr(P), _ptr(out), _ptr(lse), B,
                                     H, N, d, m, dv, int(bool(causal)), _dtype_code(q),
                                     _stream_ptr(stream)), "spa_attention_fwd_lse")
    return out, lse


def spa_attention_bwd_lse(q, k, v, P, out, lse, dO, causal=False, grads=None, stream=None):
    """Gradients (dq, dk, dv, dP) given the forward's output and row log-sum-exp
    (from spa_attention_fwd_lse).  `grads` may supply the four fp32 output tensors."""
    import torch
    B, H, N, d, m, dv = _shapes(q, k, v, P)
    dev = q.device
    if grads is None:
        grads = (torch.empty((B, H, N, d), dtype=torch.float32, device=dev),
                 torch.empty((B, H, N, d), dtype=torch.float32, device=dev),
                 torch.empty((B, H, N, dv), dtype=torch.float32, device=dev),
                 torch.empty((H, d, m), dtype=torch.float32, device=dev))
    dq, dk, dvo, dP = grads
    _check(lib.spa_attention_bwd_lse(_ptr(q), _ptr(k), _ptr(v), _ptr(P), _ptr(out), _ptr(lse),
                                     _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dvo), _ptr(dP), B, H, N, d,
                                     m, dv, int(bool(causal)), _dtype_code(q),
                                     _stream_ptr(stream)), "spa_attention_bwd_lse")
    return dq, dk, dvo, dP


def spa_attention_bwd_workspace_size(B, H, N, d, m, dv, dtype_code) -> int:
    n = _sz(0)
    _check(lib.spa_attention_bwd_workspace_size(B, H, N, d, m, dv, dtype_code, ctypes.byref(n)),
           "spa_attention_bwd_workspace_size")
    return int(n.value)


def spa_attention_bwd_prepare(q, k, P, out, lse, dO, workspace, stream=None):
    """Fused backward stage 1 into `workspace` (uint8 device tensor)."""
    B, H, N, d = q.shape
    m, dv = P.shape[-1], dO.shape[-1]
    _check(lib.spa_attention_bwd_prepare(_ptr(q), _ptr(k), _ptr(P), _ptr(out), _ptr(lse), _ptr(dO),
                                         B, H, N, d, m, dv, _dtype_code(q), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(),
                                         _stream_ptr(stream)), "spa_attention_bwd_prepare")


def spa_attention_bwd_apply(v, dO, dv_out, workspace, B, H, N, d, m, causal=False, stream=None):
    """Fused backward stage 2: the tensor-core kernel; writes dv_out (fp32)."""
    dv = v.shape[-1]
    _check(lib.spa_attention_bwd_apply(_ptr(v), _ptr(dO), _ptr(dv_out), B, H, N, d, m, dv,
                                       int(bool(causal)), _dtype_code(v), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(),
                                       _stream_ptr(stream)), "spa_attention_bwd_apply")


def spa_attention_bwd_finish(q, k, P, dq, dk, dP, dv, workspace, stream=None):
    """Fused backward stage 3: dq, dk, dP (fp32) from the workspace; dv = d_v."""
    B, H, N, d = q.shape
    m = P.shape[-1]
    _check(lib.spa_attention_bwd_finish(_ptr(q), _ptr(k), _ptr(P), _ptr(dq), _ptr(dk), _ptr(dP), B,
                                        H, N, d, m, int(dv), _dtype_code(q), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _stream_ptr(stream)), "spa_attention_bwd_finish")


def spa_topk_features(x, k, out=None, stream=None):
    """Row-wise Top-k over the last dimension of x (bf16 or fp32 CUDA tensor)."""
    import torch
    if out is None:
        out = torch.empty_like(x)
    d = x.shape[-1]
    rows = x.numel() // d if d else 0
    _check(lib.spa_topk_features(_ptr(x), _ptr(out), rows, d, int(k), _dtype_code(x),
                                 _stream_ptr(stream)), "spa_topk_features")
    return out


def spa_sfa_attention_fwd(q, k, v, topk, causal=False, out=None, stream=None):
    """softmax(Topk(q) Topk(k)^T / sqrt(d)) v; q, k [B,H,N,d], v [B,H,N,dv]."""
    import torch
    B, H, N, d = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=torch.float32, device=q.device)
    _check(lib.spa_sfa_attention_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, N, d, dv,
                                     int(topk), int(bool(causal)), _dtype_code(q),
                                     _stream_ptr(stream)), "spa_sfa_attention_fwd")
    return out


def kcache_new(B, H, cap, m, device="cuda"):
    """Empty projected key cache: (kc [B,H,cap,m] int16 holding fp16 bits,
    kc_mul [B,H,cap] float32)."""
    import torch
    return (torch.zeros((B, H, cap, m), dtype=torch.int16, device=device),
            torch.zeros((B, H, cap), dtype=torch.float32, device=device))


def spa_kcache_append(k, P, kc, kc_mul, pos, stream=None):
    """Project k [B,H,T,d] (bf16) with P [H,d,m] into cache rows pos..pos+T-1."""
    B, H, T, d = k.shape
    m = P.shape[2]
    cap = kc.shape[2]
    _check(lib.spa_kcache_append(_ptr(k), _ptr(P), _ptr(kc), _ptr(kc_mul), B, H, T, d, m, pos,
                                 cap, _dtype_code(k), _stream_ptr(stream)), "spa_kcache_append")


def spa_attention_decode(q, P, kc, kc_mul, v, L, out=None, stream=None):
    """One query per (b, h): q [B,H,d] bf16 against cache rows 0..L-1 with the
    value cache v [B,H,cap,dv] bf16; returns out [B,H,dv] float32."""
    import torch
    B, H, d = q.shape
    m = P.shape[2]
    cap, dv = v.shape[2], v.shape[3]
    if out is None:
        out = torch.empty((B, H, dv), dtype=torch.float32, device=q.device)
    _check(lib.spa_attention_decode(_ptr(q), _ptr(P), _ptr(kc), _ptr(kc_mul), _ptr(v), _ptr(out),
                                    B, H, L, d, m, dv, cap, _dtype_code(q), _stream_ptr(stream)),
           "spa_attention_decode")
    return out


SPA_ROPE_PLAIN, SPA_ROPE_LINEAR, SPA_ROPE_BASE, SPA_ROPE_RAMP = 0, 1, 2, 3


_here = contextlib.nullcontext()


def _on(device, stream):
    """The raw stream of a call and the context for it: the arguments' device is
    current, and `stream` (default: the device's current one) is the stream of
    the call's launches and of the tensors it allocates."""
    import torch
    if stream is not None:
        if stream.device_index != device.index:
            raise ValueError("the stream belongs to another device than the tensors")
        return stream.cuda_stream, torch.cuda.stream(stream)
    raw = torch._C._cuda_getCurrentRawStream(device.index)
    if torch._C._cuda_getDevice() != device.index:
        return raw, torch.cuda.device(device.index)
    return raw, _here


def _device_of(t):
    if not t.is_cuda:
        raise ValueError("the tensors of this call are CUDA tensors")
    return t.device


def _arg(name, t, shape, dtype, device):
    """A dense tensor of this shape, type and device; its address."""
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _workspace(t, device):
    """Address and size of a caller's workspace (None: the library takes its own)."""
    if t is None:
        return None, 0
    if t.device != device:
        raise ValueError(f"workspace must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.data_ptr(), t.nbytes


def rope_frequencies(rot, base=10000.0, scaling=SPA_ROPE_PLAIN, factor=1.0, trained=0.0, slow=1.0,
                     fast=32.0):
    """The rot/2 frequencies base^(-2i/rot) as a float64 CPU tensor, stretched
    for long contexts (scaling: SPA_ROPE_LINEAR, _BASE or _RAMP; see spa.h)."""
    import torch
    f = torch.empty(max(int(rot), 0) // 2, dtype=torch.float64)
    _check(lib.spa_rope_frequencies(ctypes.cast(f.data_ptr(), _pd), int(rot), base, int(scaling),
                                    factor, trained, slow, fast), "spa_rope_frequencies")
    return f


def rope_table(inv_freq, device="cuda"):
    """The table that spa_rope takes, from the rot/2 frequencies (radians per
    position): an int64 tensor on `device` of advances in units of 2^-64 turns."""
    import torch
    f = torch.as_tensor(inv_freq, dtype=torch.float64, device="cpu").contiguous()
    if f.dim() != 1:
        raise ValueError("inv_freq must have one dimension")
    t = torch.empty(f.shape, dtype=torch.int64)
    _check(lib.spa_rope_table(ctypes.cast(f.data_ptr(), _pd), 2 * f.numel(),
                              ctypes.cast(t.data_ptr(), ctypes.POINTER(ctypes.c_ulonglong))),
           "spa_rope_table")
    return t.to(device)


_Strides = _ll * 12


def spa_rope(q, table, pos=None, *, k=None, rot=None, interleaved=False, inverse=False, scale=1.0,
             pos0=0, out=None, k_out=None, stream=None):
    """Rotary positions of q [B,H,N,d] and, in the same launch, k [B,Hk,N,d]
    (bf16 or fp32, any strides with adjacent features); returns the rotated
    tensor, or both.  pos is [B,N] int32 (default: pos0 + n).  inverse=True maps
    the outputs' gradients to the inputs'."""
    import torch
    device = _device_of(q)
    B, H, N, d = q.shape
    rot = 2 * table.numel() if rot is None else int(rot)
    ptable = _arg("table", table, (rot // 2,), torch.int64, device)
    ppos = None if pos is None else _arg("pos", pos, (B, N), torch.int32, device)
    code = _dtype_code(q)
    Hk = 0
    if k is not None:
        Hk = k.shape[1]
        if k.shape != (B, Hk, N, d):
            raise ValueError("k must be [B,Hk,N,d] with q's B, N and d")
        if k.dtype != q.dtype:
            raise TypeError("q and k must share one dtype")
        if k.device != device:
            raise ValueError(f"k must be on {device}, got {k.device}")
    elif k_out is not None:
        raise ValueError("k_out without k")
    raw, context = _on(device, stream)
    with context:
        if out is None:
            out = torch.empty((B, H, N, d), dtype=q.dtype, device=device)
        if k is not None and k_out is None:
            k_out = torch.empty((B, Hk, N, d), dtype=q.dtype, device=device)
        for x, y in ((q, out), (k, k_out)):
            if x is None:
                continue
            if y.shape != x.shape or y.dtype != x.dtype or y.device != device:
                raise ValueError("an output must have its input's shape, dtype and device")
            if (x.stride(3) != 1 or y.stride(3) != 1) and d > 1:
                raise ValueError("the features of a row must be adjacent")
        a, c = q.stride(), out.stride()
        b, e = (k.stride(), k_out.stride()) if k is not None else ((0, 0, 0), (0, 0, 0))
        strides = _Strides(a[0], a[1], a[2], b[0], b[1], b[2], c[0], c[1], c[2], e[0], e[1], e[2])
        _check(lib.spa_rope(q.data_ptr(), k.data_ptr() if Hk else None, out.data_ptr(),
                            k_out.data_ptr() if Hk else None, strides, ppos, pos0, ptable, B, H, Hk,
                            N, d, rot, bool(interleaved), bool(inverse), scale, code, raw),
               "spa_rope")
    return out if k is None else (out, k_out)


def spa_kcache_append_ragged(k, v, P, kc, kc_mul, vc, pos, count=None, acc=None, row_pos=None,
                             token=None, stream=None):
    """The first count[b] (default: T) rows of k [B,H,T,d] (projected with P
    [H,d,m]) and v [B,H,T,dv], bf16, into cache rows pos[b].. of every sequence;
    acc and row_pos (for spa_kcache_evict) start at 0 and token[b] + t."""
    import torch
    device = _device_of(k)
    B, H, T, d = k.shape
    m, cap, dv = P.shape[-1], kc.shape[2], v.shape[-1]
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    row = (B, H, cap)
    args = (_arg("k", k, (B, H, T, d), bf16, device), _arg("v", v, (B, H, T, dv), bf16, device),
            _arg("P", P, (H, d, m), bf16, device),
            _arg("kc", kc, (B, H, cap, m), torch.int16, device),
            _arg("kc_mul", kc_mul, row, f32, device),
            _arg("vc", vc, (B, H, cap, dv), bf16, device),
            _arg("pos", pos, (B,), i32, device),
            None if count is None else _arg("count", count, (B,), i32, device),
            None if acc is None else _arg("acc", acc, row, f32, device),
            None if row_pos is None else _arg("row_pos", row_pos, row, i32, device),
            None if token is None else _arg("token", token, (B,), i32, device))
    raw, context = _on(device, stream)
    with context:
        _check(lib.spa_kcache_append_ragged(*args, B, H, T, d, m, dv, cap, SPA_BF16, raw),
               "spa_kcache_append_ragged")


def spa_attention_decode_shared_workspace_size(B, H, Hk, plen, d, m, dv, cap, weights=False) -> int:
    n = _sz(0)
    _check(lib.spa_attention_decode_shared_workspace_size(B, H, Hk, plen, d, m, dv, cap,
                                                          bool(weights), ctypes.byref(n)),
           "spa_attention_decode_shared_workspace_size")
    return int(n.value)


def spa_attention_decode_shared(q, P, kc, kc_mul, v, lens, *, prefix=None, plen=None, acc=None,
                                acc_out=None, out=None, workspace=None, stream=None):
    """One query per (sequence, head), q [B,H,d] bf16, against a prefix shared by
    the batch, prefix = (kc [Hk,pcap,m], kc_mul [Hk,pcap], v [Hk,pcap,dv]) of
    which plen rows (default: all) count, and rows 0..lens[b]-1 of the own
    caches kc [B,Hk,cap,m], kc_mul, v; returns bf16 [B,H,dv].  With acc
    [B,Hk,cap] the step's attention weights are added to it (into acc_out,
    default: acc itself)."""
    import torch
    device = _device_of(q)
    B, H, d = q.shape
    Hk, m = P.shape[0], P.shape[-1]
    cap, dv = v.shape[2], v.shape[3]
    bf16, f32, i16 = torch.bfloat16, torch.float32, torch.int16
    own = (_arg("q", q, (B, H, d), bf16, device), _arg("P", P, (Hk, d, m), bf16, device),
           _arg("kc", kc, (B, Hk, cap, m), i16, device),
           _arg("kc_mul", kc_mul, (B, Hk, cap), f32, device),
           _arg("v", v, (B, Hk, cap, dv), bf16, device),
           _arg("lens", lens, (B,), torch.int32, device))
    shared, pcap = (None, None, None), 0
    if prefix is not None:
        pkc, pmul, pv = prefix
        pcap = pkc.shape[1]
        shared = (_arg("prefix kc", pkc, (Hk, pcap, m), i16, device),
                  _arg("prefix kc_mul", pmul, (Hk, pcap), f32, device),
                  _arg("prefix v", pv, (Hk, pcap, dv), bf16, device))
    plen = pcap if plen is None else int(plen)
    if acc_out is None:
        acc_out = acc
    weights = (None if acc is None else _arg("acc", acc, (B, Hk, cap), f32, device),
               None if acc_out is None else _arg("acc_out", acc_out, (B, Hk, cap), f32, device))
    raw, context = _on(device, stream)
    with context:
        if out is None:
            out = torch.empty((B, H, dv), dtype=bf16, device=device)
        pout = _arg("out", out, (B, H, dv), bf16, device)
        ws, size = _workspace(workspace, device)
        _check(lib.spa_attention_decode_shared(*own, *shared, pout, *weights, B, H, Hk, plen, pcap,
                                               d, m, dv, cap, SPA_BF16, ws, size, raw),
               "spa_attention_decode_shared")
    return out


def spa_kcache_evict_workspace_size(B, H, cap, budget) -> int:
    n = _sz(0)
    _check(lib.spa_kcache_evict_workspace_size(B, H, cap, budget, ctypes.byref(n)),
           "spa_kcache_evict_workspace_size")
    return int(n.value)


def spa_kcache_evict(kc, kc_mul, v, acc, row_pos, lens, budget, sink=0, recent=0, acc_out=None,
                     row_pos_out=None, lens_out=None, src=None, workspace=None, stream=None):
    """Brings the cache (kc [B,H,cap,m], kc_mul, v) down to `budget` rows per
    (sequence, head), in place: the first `sink` positions, the newest `recent`
    ones and the rows of largest acc stay.  acc, row_pos and lens are updated
    in place unless *_out tensors are given.  Returns src [B,H,budget] int32:
    the row that each row was before (-1 behind the new length)."""
    import torch
    device = _device_of(kc)
    B, H, cap, m = kc.shape
    dv, budget = v.shape[-1], int(budget)
    f32, i32 = torch.float32, torch.int32
    row = (B, H, cap)
    acc_out = acc if acc_out is None else acc_out
    row_pos_out = row_pos if row_pos_out is None else row_pos_out
    lens_out = lens if lens_out is None else lens_out
    args = (_arg("kc", kc, (B, H, cap, m), torch.int16, device),
            _arg("kc_mul", kc_mul, row, f32, device),
            _arg("v", v, (B, H, cap, dv), torch.bfloat16, device),
            _arg("acc", acc, row, f32, device), _arg("row_pos", row_pos, row, i32, device),
            _arg("lens", lens, (B,), i32, device), _arg("acc_out", acc_out, row, f32, device),
            _arg("row_pos_out", row_pos_out, row, i32, device),
            _arg("lens_out", lens_out, (B,), i32, device))
    raw, context = _on(device, stream)
    with context:
        if src is None:
            src = torch.empty((B, H, max(budget, 0)), dtype=i32, device=device)
        psrc = _arg("src", src, (B, H, max(budget, 0)), i32, device)
        ws, size = _workspace(workspace, device)
        _check(lib.spa_kcache_evict(*args, psrc, B, H, m, dv, cap, budget, int(sink), int(recent),
                                    ws, size, raw), "spa_kcache_evict")
    return src


def selftest_wait_timeout(limit_ms: int = 50) -> int:
    """Run the failure-detection self-test; returns the spa_status code
    (SPA_ERR_TIMEOUT when the withheld barrier was detected, as expected)."""
    return int(lib.spa_selftest_wait_timeout(int(limit_ms)))


def selftest_bwd_wait_timeout(limit_ms: int = 50) -> int:
    """The same self-test for the fused backward kernel (returns the status code)."""
    return int(lib.spa_selftest_bwd_wait_timeout(int(limit_ms)))


def selftest_proj_wait_timeout(limit_ms: int = 50, m: int = 64) -> int:
    """The same self-test for the tensor-core projection kernels (m = 32: the
    per-CTA kernel, m = 64: the warp-specialised one); returns the status code."""
    return int(lib.spa_selftest_proj_wait_timeout(int(limit_ms), int(m)))


def selftest_copy_wait_timeout(limit_ms: int = 50, kernel: int = 0) -> int:
    """The same self-test for the kernels that wait on their own copies
    (kernel 0: the backward's statistics, 1: its finish, 2: the Top-k);
    returns the status code."""
    return int(lib.spa_selftest_copy_wait_timeout(int(limit_ms), int(kernel)))


def selftest_decode_wait_timeout(limit_ms: int = 50, kernel: int = 0) -> int:
    """The same self-test for the shared-prefix decode (kernel 0: the prefix
    kernel, 1: the kernel of the sequences' own rows); returns the status code."""
    return int(lib.spa_selftest_decode_wait_timeout(int(limit_ms), int(kernel)))


def device_error() -> int:
    """Read and clear the device error word (0 or SPA_ERR_TIMEOUT)."""
    c = _i(0)
    _check(lib.spa_device_error(ctypes.byref(c)), "spa_device_error")
    return int(c.value)


def host_pool_trim() -> None:
    """Release the current device's unused memory kept by the library's pool."""
    _check(lib.spa_host_pool_trim(), "spa_host_pool_trim")
