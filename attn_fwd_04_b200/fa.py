"""ctypes binding of libfa.so (include/fa.h), one Python function per C entry
point, same names.  Argument marshalling only: every step of the computation
runs in the library's CUDA kernels.  PyTorch supplies device memory and the
stream; there is no fallback -- a missing library or a non-CUDA tensor is an
error.
"""
import ctypes
import functools
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfa.so")

FA_OK = 0
FA_ERR_NULL = -1
FA_ERR_SHAPE = -2
FA_ERR_UNSUPPORTED = -3
FA_ERR_ALIGN = -4
FA_ERR_CUDA = -5
FA_ERR_DEVICE_TIMEOUT = -6
FA_ERR_NOMEM = -7
FA_ERR_DEVICE_BAD_INPUT = -8

# every symbol include/fa.h declares
EXPORTS = ("fa_fwd", "fa_fwd_gqa", "fa_fwd_rope", "fa_bwd", "fa_bwd_gqa", "fa_bwd_varlen",
           "fa_fwd_varlen", "fa_fwd_varlen_gqa",
           "fa_decode_paged",
           "fa_decode_paged_gqa", "fa_decode_paged_strided",
           "fa_decode_paged_noalloc", "fa_append_paged", "fa_prefill_paged",
           "fa_gather_paged",
           "fa_rope_table", "fa_qk_norm_rope", "fa_qk_norm_rope_bwd",
           "fa_qk_norm_rope_bwd_workspace", "fa_append_paged_rope", "fa_append_paged_fp8",
           "fa_decode_paged_fp8", "fa_decode_paged_fp8_workspace",
           "fa_get_device_error", "fa_selftest_bounded_wait", "fa_selftest_fwd_stall",
           "fa_selftest_decode_stall",
           "fa_release_workspace", "fa_status_str", "fa_version", "fa_fwd_set_cta_pairs")

_lib = None


class FaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {fa_status_str(status)} ({status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libfa.so (built in-tree by attn_fwd_04_b200.build); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libfa.so not found at {LIB_PATH}; build it with "
                              "`python -m attn_fwd_04_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.fa_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, F, P]
        L.fa_fwd_gqa.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, P]
        L.fa_fwd_varlen.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, P]
        L.fa_fwd_varlen_gqa.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, F, P]
        L.fa_fwd_rope.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P]
        L.fa_bwd.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, F, P]
        L.fa_bwd_gqa.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P]
        L.fa_bwd_varlen.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P]
        L.fa_decode_paged.argtypes = [P, P, P, P, P, P, I, I, I, I, P]
        L.fa_decode_paged_gqa.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P]
        L.fa_decode_paged_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, I, P]
        L.fa_decode_paged_strided.argtypes = [P, P, P, P, I, P, P, I, I, I, I, I, I, P]
        L.fa_gather_paged.argtypes = [P, P, P, P, I, I, I, I, P]
        L.fa_append_paged.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, P]
        L.fa_prefill_paged.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, P]
        D = ctypes.c_double
        L.fa_rope_table.argtypes = [P, P, I, I, D, I, D, I, D, D, D, P]
        L.fa_qk_norm_rope.argtypes = [P] * 6 + [I, P, P, I, I, I, P] + [I] * 10 + [F, P]
        L.fa_qk_norm_rope_bwd.argtypes = ([P] * 10 + [I, P, P, I, I, I, P] + [I] * 12 +
                                          [F, P, I, P])
        L.fa_qk_norm_rope_bwd_workspace.argtypes = [I] * 5 + [ctypes.POINTER(ctypes.c_int)]
        L.fa_append_paged_rope.argtypes = ([P] * 8 + [I, I] + [P] * 3 + [I, P, P] + [I] * 13 +
                                           [F, P])
        L.fa_append_paged_fp8.argtypes = ([P] * 9 + [I, P, I, I] + [P] * 3 + [I, P, P] +
                                          [I] * 13 + [F, P])
        L.fa_decode_paged_fp8.argtypes = ([P] * 5 + [I, P, I, I] + [P] * 3 + [I] * 6 +
                                          [F, P, I, P])
        L.fa_decode_paged_fp8_workspace.argtypes = [I] * 4 + [ctypes.POINTER(ctypes.c_int)]
        L.fa_get_device_error.argtypes = [ctypes.POINTER(ctypes.c_int), P]
        L.fa_selftest_bounded_wait.argtypes = [P]
        L.fa_selftest_fwd_stall.argtypes = [P, P, P, P, P, I, I, I, I, I, I, P]
        L.fa_selftest_decode_stall.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P]
        L.fa_release_workspace.argtypes = []
        L.fa_status_str.argtypes = [I]
        L.fa_status_str.restype = ctypes.c_char_p
        L.fa_version.argtypes = []
        L.fa_fwd_set_cta_pairs.argtypes = [I]
        for name in ("fa_fwd", "fa_fwd_gqa", "fa_fwd_rope", "fa_bwd", "fa_bwd_gqa", "fa_bwd_varlen",
                     "fa_fwd_varlen", "fa_fwd_varlen_gqa",
                     "fa_decode_paged",
                     "fa_decode_paged_gqa", "fa_decode_paged_strided", "fa_decode_paged_noalloc",
                     "fa_append_paged",
                     "fa_prefill_paged", "fa_gather_paged",
                     "fa_rope_table", "fa_qk_norm_rope", "fa_qk_norm_rope_bwd",
                     "fa_qk_norm_rope_bwd_workspace", "fa_append_paged_rope",
                     "fa_append_paged_fp8", "fa_decode_paged_fp8",
                     "fa_decode_paged_fp8_workspace",
                     "fa_get_device_error", "fa_selftest_bounded_wait", "fa_selftest_fwd_stall",
                     "fa_selftest_decode_stall",
                     "fa_release_workspace", "fa_version", "fa_fwd_set_cta_pairs"):
            getattr(L, name).restype = I
        _lib = L
    return _lib


def fa_status_str(status: int) -> str:
    return lib().fa_status_str(int(status)).decode()


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# device types the wrappers accept (the library reads device memory only)
_DEVICE_TYPES = ("cuda",)


def _check(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int):
    if not isinstance(t, torch.Tensor) or t.device.type not in _DEVICE_TYPES:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _expect(t, name: str, dtype: torch.dtype, shape, device):
    """t must be a contiguous CUDA tensor of this dtype and exact shape on
    `device` (the device of the call's first input)."""
    _check(t, name, dtype, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's inputs on {device}")


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, the call's inputs on {device}")


def _pages(k_pages, v_pages, page_size: int, d: int, heads=None):
    """k_pages, v_pages: the same [P, heads, page_size, d] shape."""
    if v_pages.shape != k_pages.shape:
        raise ValueError("k_pages and v_pages must have the same shape")
    want = (heads if heads is not None else k_pages.shape[1], int(page_size), d)
    if tuple(k_pages.shape[1:]) != want:
        raise ValueError(f"pages must be [P, {want[0]}, {want[1]}, {want[2]}], got "
                         f"{tuple(k_pages.shape)}")


def _raise_if(status: int, what: str):
    if status != FA_OK:
        raise FaError(status, what)


def fa_fwd(q, k, v, causal: bool, scale: Optional[float] = None, o=None, lse=None, stream=None):
    """Fused attention forward over [B,H,N,d] bf16 tensors -> (o, lse [B,H,N] fp32)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, torch.bfloat16, 4)
    B, H, N, d = q.shape
    if k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must have the same [B,H,N,d] shape")
    _same_device(q.device, k=k, v=v)
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _expect(o, "o", torch.bfloat16, q.shape, q.device)
    _expect(lse, "lse", torch.float32, (B, H, N), q.device)
    rc = lib().fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                      B, H, N, d, int(bool(causal)), float(scale), _stream(stream))
    _raise_if(rc, "fa_fwd")
    return o, lse


def fa_fwd_gqa(q, k, v, causal: bool, scale: Optional[float] = None, o=None, lse=None,
               stream=None):
    """Grouped-query forward: q [B,H,N,d], k/v [B,H_kv,N,d] bf16 with H a
    multiple of H_kv -> (o [B,H,N,d], lse [B,H,N] fp32)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, torch.bfloat16, 4)
    B, H, N, d = q.shape
    H_kv = k.shape[1]
    if k.shape != (B, H_kv, N, d) or v.shape != k.shape:
        raise ValueError("k, v must be [B,H_kv,N,d] with q's B, N, d")
    _same_device(q.device, k=k, v=v)
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _expect(o, "o", torch.bfloat16, q.shape, q.device)
    _expect(lse, "lse", torch.float32, (B, H, N), q.device)
    rc = lib().fa_fwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                          B, H, H_kv, N, d, int(bool(causal)), float(scale), _stream(stream))
    _raise_if(rc, "fa_fwd_gqa")
    return o, lse


def fa_fwd_rope(q, k, v, rope_cos, rope_sin, causal: bool, scale: Optional[float] = None,
                o=None, lse=None, stream=None):
    """Forward with rotary embedding applied in the kernel: q [B,H,N,d],
    k/v [B,H_kv,N,d] bf16 (unrotated), tables [max_pos,d/2] fp32 ->
    (o [B,H,N,d], lse [B,H,N])."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, torch.bfloat16, 4)
    _check(rope_cos, "rope_cos", torch.float32, 2)
    _check(rope_sin, "rope_sin", torch.float32, 2)
    B, H, N, d = q.shape
    H_kv = k.shape[1]
    if k.shape != (B, H_kv, N, d) or v.shape != k.shape:
        raise ValueError("k, v must be [B,H_kv,N,d] with q's B, N, d")
    if rope_cos.shape[1] != d // 2 or rope_sin.shape != rope_cos.shape:
        raise ValueError("rope tables must be [max_pos, d/2]")
    _same_device(q.device, k=k, v=v, rope_cos=rope_cos, rope_sin=rope_sin)
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _expect(o, "o", torch.bfloat16, q.shape, q.device)
    _expect(lse, "lse", torch.float32, (B, H, N), q.device)
    rc = lib().fa_fwd_rope(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                           rope_cos.data_ptr(), rope_sin.data_ptr(), rope_cos.shape[0], B, H,
                           H_kv, N, d, int(bool(causal)), float(scale), _stream(stream))
    _raise_if(rc, "fa_fwd_rope")
    return o, lse


def fa_bwd(q, k, v, o, lse, dout, causal: bool, scale: Optional[float] = None, dq=None,
           dk=None, dv=None, stream=None):
    """Gradients of fa_fwd: (dq, dk, dv), each [B,H,N,d] bf16, from q, k, v, o,
    dout [B,H,N,d] bf16 and lse [B,H,N] fp32 (as fa_fwd returned them)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _check(t, n, torch.bfloat16, 4)
        if t.shape != q.shape:
            raise ValueError(f"{n} must have q's shape")
    B, H, N, d = q.shape
    _expect(lse, "lse", torch.float32, (B, H, N), q.device)
    _same_device(q.device, k=k, v=v, o=o, dout=dout)
    if scale is None:
        scale = d ** -0.5
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _expect(t, n, torch.bfloat16, q.shape, q.device)
    rc = lib().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                      dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d,
                      int(bool(causal)), float(scale), _stream(stream))
    _raise_if(rc, "fa_bwd")
    return dq, dk, dv


def fa_bwd_gqa(q, k, v, o, lse, dout, causal: bool, scale: Optional[float] = None, dq=None,
               dk=None, dv=None, stream=None):
    """Gradients of fa_fwd_gqa: dq [B,H,N,d] and dk, dv [B,H_kv,N,d] bf16, from
    q, o, dout [B,H,N,d], k, v [B,H_kv,N,d] bf16 and lse [B,H,N] fp32."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _check(t, n, torch.bfloat16, 4)
    B, H, N, d = q.shape
    H_kv = k.shape[1]
    if o.shape != q.shape or dout.shape != q.shape or k.shape != (B, H_kv, N, d) or \
            v.shape != k.shape:
        raise ValueError("q, o, dout must be [B,H,N,d] and k, v [B,H_kv,N,d]")
    _expect(lse, "lse", torch.float32, (B, H, N), q.device)
    _same_device(q.device, k=k, v=v, o=o, dout=dout)
    if scale is None:
        scale = d ** -0.5
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _expect(dq, "dq", torch.bfloat16, q.shape, q.device)
    _expect(dk, "dk", torch.bfloat16, k.shape, q.device)
    _expect(dv, "dv", torch.bfloat16, k.shape, q.device)
    rc = lib().fa_bwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                          dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H,
                          H_kv, N, d, int(bool(causal)), float(scale), _stream(stream))
    _raise_if(rc, "fa_bwd_gqa")
    return dq, dk, dv


def fa_bwd_varlen(q, k, v, o, lse, dout, cu_seqlens, max_seqlen: int, causal: bool,
                  scale: Optional[float] = None, dq=None, dk=None, dv=None, stream=None):
    """Gradients of fa_fwd_varlen over packed sequences: dq [total,H,d] and dk, dv
    [total,H_kv,d] bf16, from q, o, dout [total,H,d], k, v [total,H_kv,d] bf16 and
    lse [H,total] fp32 (as fa_fwd_varlen returned it)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _check(t, n, torch.bfloat16, 3)
    _check(cu_seqlens, "cu_seqlens", torch.int32, 1)
    total, H, d = q.shape
    H_kv = k.shape[1]
    if o.shape != q.shape or dout.shape != q.shape or k.shape != (total, H_kv, d) or \
            v.shape != k.shape:
        raise ValueError("q, o, dout must be [total,H,d] and k, v [total,H_kv,d]")
    _expect(lse, "lse", torch.float32, (H, total), q.device)
    _same_device(q.device, k=k, v=v, o=o, dout=dout, cu_seqlens=cu_seqlens)
    B = cu_seqlens.numel() - 1
    if scale is None:
        scale = d ** -0.5
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _expect(dq, "dq", torch.bfloat16, q.shape, q.device)
    _expect(dk, "dk", torch.bfloat16, k.shape, q.device)
    _expect(dv, "dv", torch.bfloat16, k.shape, q.device)
    rc = lib().fa_bwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                             lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                             dv.data_ptr(), cu_seqlens.data_ptr(), B, H, H_kv, total,
                             int(max_seqlen), d, int(bool(causal)), float(scale), _stream(stream))
    _raise_if(rc, "fa_bwd_varlen")
    return dq, dk, dv


def fa_fwd_varlen(q, k, v, cu_seqlens, max_seqlen: int, causal: bool,
                  scale: Optional[float] = None, o=None, lse=None, stream=None):
    """Forward over packed [total,H,d] sequences -> (o, lse [H,total] fp32)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, torch.bfloat16, 3)
    _check(cu_seqlens, "cu_seqlens", torch.int32, 1)
    total, H, d = q.shape
    if k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must have the same [total,H,d] shape")
    _same_device(q.device, k=k, v=v, cu_seqlens=cu_seqlens)
    B = cu_seqlens.numel() - 1
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((H, total), dtype=torch.float32, device=q.device)
    _expect(o, "o", torch.bfloat16, q.shape, q.device)
    _expect(lse, "lse", torch.float32, (H, total), q.device)
    rc = lib().fa_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                             lse.data_ptr(), cu_seqlens.data_ptr(), B, H, total,
                             int(max_seqlen), d, int(bool(causal)), float(scale),
                             _stream(stream))
    _raise_if(rc, "fa_fwd_varlen")
    return o, lse


def fa_fwd_varlen_gqa(q, k, v, cu_seqlens, max_seqlen: int, causal: bool,
                      scale: Optional[float] = None, o=None, lse=None, stream=None):
    """Forward over packed sequences with grouped K/V heads: q [total,H,d], k, v
    [total,H_kv,d] -> (o [total,H,d], lse [H,total] fp32)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, torch.bfloat16, 3)
    _check(cu_seqlens, "cu_seqlens", torch.int32, 1)
    total, H, d = q.shape
    H_kv = k.shape[1]
    if k.shape != (total, H_kv, d) or v.shape != k.shape:
        raise ValueError("k, v must be [total,H_kv,d]")
    _same_device(q.device, k=k, v=v, cu_seqlens=cu_seqlens)
    B = cu_seqlens.numel() - 1
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((H, total), dtype=torch.float32, device=q.device)
    _expect(o, "o", torch.bfloat16, q.shape, q.device)
    _expect(lse, "lse", torch.float32, (H, total), q.device)
    rc = lib().fa_fwd_varlen_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                 lse.data_ptr(), cu_seqlens.data_ptr(), B, H, H_kv, total,
                                 int(max_seqlen), d, int(bool(causal)), float(scale),
                                 _stream(stream))
    _raise_if(rc, "fa_fwd_varlen_gqa")
    return o, lse


def fa_decode_paged(q, k_pages, v_pages, page_table, seq_lens, page_size: int = 256, o=None,
                    stream=None):
    """Single-token decode over a paged cache -> o [B,H,d] bf16."""
    _check(q, "q", torch.bfloat16, 3)
    _check(k_pages, "k_pages", torch.bfloat16, 4)
    _check(v_pages, "v_pages", torch.bfloat16, 4)
    _check(page_table, "page_table", torch.int32, 1)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    B, H, d = q.shape
    # the multi-head call takes no pool size, so the pool's layout is checked
    # here: a cache of another head count or page size would be misread
    _pages(k_pages, v_pages, page_size, d, heads=H)
    if seq_lens.numel() != B:
        raise ValueError(f"seq_lens must hold one length per sequence ({B})")
    _same_device(q.device, k_pages=k_pages, v_pages=v_pages, page_table=page_table,
                 seq_lens=seq_lens)
    if o is None:
        o = torch.empty_like(q)
    _expect(o, "o", torch.bfloat16, q.shape, q.device)
    rc = lib().fa_decode_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                               page_table.data_ptr(), seq_lens.data_ptr(), o.data_ptr(),
                               B, H, d, int(page_size), _stream(stream))
    _raise_if(rc, "fa_decode_paged")
    return o


def fa_decode_paged_gqa(q, k_pages, v_pages, page_table, seq_lens, page_size: int = 256, o=None,
                        stream=None):
    """Decode with grouped K/V heads: q [B,H,d], pages [P,H_kv,page_size,d]
    -> o [B,H,d] bf16.  The pool size P bounds the page indices read."""
    _check(q, "q", torch.bfloat16, 3)
    _check(k_pages, "k_pages", torch.bfloat16, 4)
    _check(v_pages, "v_pages", torch.bfloat16, 4)
    _check(page_table, "page_table", torch.int32, 1)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    B, H, d = q.shape
    H_kv = k_pages.shape[1]
    _pages(k_pages, v_pages, page_size, d)
    if H_kv == 0 or H % H_kv != 0:
        raise ValueError(f"H ({H}) must be a multiple of the cache's K/V heads ({H_kv})")
    if seq_lens.numel() != B:
        raise ValueError(f"seq_lens must hold one length per sequence ({B})")
    _same_device(q.device, k_pages=k_pages, v_pages=v_pages, page_table=page_table,
                 seq_lens=seq_lens)
    if o is None:
        o = torch.empty_like(q)
    _expect(o, "o", torch.bfloat16, q.shape, q.device)
    rc = lib().fa_decode_paged_gqa(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                   page_table.data_ptr(), seq_lens.data_ptr(), o.data_ptr(),
                                   B, H, H_kv, k_pages.shape[0], d, int(page_size),
                                   _stream(stream))
    _raise_if(rc, "fa_decode_paged_gqa")
    return o


def fa_decode_paged_strided(q, k_pages, v_pages, block_table, seq_lens, page_size: int = 256,
                            o=None, stream=None):
    """Decode through a block table [B, max_pages] int32 (row b lists sequence
    b's pages): q [B,H,d], pages [P,H_kv,page_size,d] -> o [B,H,d] bf16."""
    _check(q, "q", torch.bfloat16, 3)
    _check(k_pages, "k_pages", torch.bfloat16, 4)
    _check(v_pages, "v_pages", torch.bfloat16, 4)
    _check(block_table, "block_table", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    B, H, d = q.shape
    H_kv = k_pages.shape[1]
    if block_table.shape[0] != B:
        raise ValueError("block_table must have one row per sequence")
    _pages(k_pages, v_pages, page_size, d)
    if H_kv == 0 or H % H_kv != 0:
        raise ValueError(f"H ({H}) must be a multiple of the cache's K/V heads ({H_kv})")
    if seq_lens.numel() != B:
        raise ValueError(f"seq_lens must hold one length per sequence ({B})")
    _same_device(q.device, k_pages=k_pages, v_pages=v_pages, block_table=block_table,
                 seq_lens=seq_lens)
    if o is None:
        o = torch.empty_like(q)
    _expect(o, "o", torch.bfloat16, q.shape, q.device)
    rc = lib().fa_decode_paged_strided(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                       block_table.data_ptr(), block_table.shape[1],
                                       seq_lens.data_ptr(), o.data_ptr(), B, H, H_kv,
                                       k_pages.shape[0], d, int(page_size), _stream(stream))
    _raise_if(rc, "fa_decode_paged_strided")
    return o


def fa_decode_paged_noalloc(q, k_pages, v_pages, page_table, seq_lens, page_size: int = 256,
                            o=None, stream=None):
    """fa_decode_paged without any device allocation by the library (its scratch
    is a fixed 16 MiB device array).  `o` should be preallocated by callers that
    cannot allocate; it is created here only as a convenience."""
    _check(q, "q", torch.bfloat16, 3)
    _check(k_pages, "k_pages", torch.bfloat16, 4)
    _check(v_pages, "v_pages", torch.bfloat16, 4)
    _check(page_table, "page_table", torch.int32, 1)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    B, H, d = q.shape
    # the multi-head call takes no pool size, so the pool's layout is checked
    # here: a cache of another head count or page size would be misread
    _pages(k_pages, v_pages, page_size, d, heads=H)
    if seq_lens.numel() != B:
        raise ValueError(f"seq_lens must hold one length per sequence ({B})")
    _same_device(q.device, k_pages=k_pages, v_pages=v_pages, page_table=page_table,
                 seq_lens=seq_lens)
    if o is None:
        o = torch.empty_like(q)
    _expect(o, "o", torch.bfloat16, q.shape, q.device)
    rc = lib().fa_decode_paged_noalloc(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                       page_table.data_ptr(), seq_lens.data_ptr(), o.data_ptr(),
                                       B, H, d, int(page_size), _stream(stream))
    _raise_if(rc, "fa_decode_paged_noalloc")
    return o


def fa_append_paged(k_new, v_new, cu_new, k_pages, v_pages, page_table, seq_lens,
                    page_size: int = 256, stream=None):
    """Write new rows [total_new,H_kv,d] into the [P,H_kv,page_size,d] pages
    (in place) as the last tokens of their sequences; seq_lens are the
    lengths after the append."""
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _check(t, n, torch.bfloat16, 3)
    _check(k_pages, "k_pages", torch.bfloat16, 4)
    _check(v_pages, "v_pages", torch.bfloat16, 4)
    _check(cu_new, "cu_new", torch.int32, 1)
    _check(page_table, "page_table", torch.int32, 1)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    total_new, H_kv, d = k_new.shape
    if v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must have the same shape")
    _pages(k_pages, v_pages, page_size, d, heads=H_kv)
    if seq_lens.numel() != cu_new.numel() - 1:
        raise ValueError("seq_lens must hold one length per sequence of cu_new")
    _same_device(k_new.device, v_new=v_new, cu_new=cu_new, k_pages=k_pages, v_pages=v_pages,
                 page_table=page_table, seq_lens=seq_lens)
    rc = lib().fa_append_paged(k_new.data_ptr(), v_new.data_ptr(), cu_new.data_ptr(),
                               k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
                               seq_lens.data_ptr(), cu_new.numel() - 1, H_kv, total_new,
                               k_pages.shape[0], d, int(page_size), _stream(stream))
    _raise_if(rc, "fa_append_paged")


def fa_prefill_paged(q, k_pages, v_pages, page_table, seq_lens, cu_q, max_q: int, causal: bool,
                     scale: Optional[float] = None, page_size: int = 256, o=None, lse=None,
                     stream=None):
    """Queries [total_q,H,d] that end their cached sequences, attending
    through the page table -> (o [total_q,H,d], lse [H,total_q] fp32)."""
    _check(q, "q", torch.bfloat16, 3)
    _check(k_pages, "k_pages", torch.bfloat16, 4)
    _check(v_pages, "v_pages", torch.bfloat16, 4)
    _check(page_table, "page_table", torch.int32, 1)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    _check(cu_q, "cu_q", torch.int32, 1)
    total_q, H, d = q.shape
    _pages(k_pages, v_pages, page_size, d)
    if k_pages.shape[1] == 0 or H % k_pages.shape[1] != 0:
        raise ValueError(f"H ({H}) must be a multiple of the cache's K/V heads "
                         f"({k_pages.shape[1]})")
    if seq_lens.numel() != cu_q.numel() - 1:
        raise ValueError("seq_lens must hold one length per sequence of cu_q")
    _same_device(q.device, k_pages=k_pages, v_pages=v_pages, page_table=page_table,
                 seq_lens=seq_lens, cu_q=cu_q)
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((H, total_q), dtype=torch.float32, device=q.device)
    _expect(o, "o", torch.bfloat16, q.shape, q.device)
    _expect(lse, "lse", torch.float32, (H, total_q), q.device)
    rc = lib().fa_prefill_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                page_table.data_ptr(), seq_lens.data_ptr(), cu_q.data_ptr(),
                                o.data_ptr(), lse.data_ptr(), cu_q.numel() - 1, H,
                                k_pages.shape[1], total_q, int(max_q), k_pages.shape[0], d,
                                int(page_size), int(bool(causal)), float(scale), _stream(stream))
    _raise_if(rc, "fa_prefill_paged")
    return o, lse


def fa_gather_paged(pages, page_table, seq_lens, total_tokens: int, page_size: int = 256,
                    out=None, stream=None):
    """Copy cached tokens out of [P,H,page_size,d] pages -> [total_tokens,H,d]."""
    _check(pages, "pages", torch.bfloat16, 4)
    _check(page_table, "page_table", torch.int32, 1)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    _, H, _, d = pages.shape
    if pages.shape[2] != int(page_size):
        raise ValueError(f"pages must hold {page_size} tokens each, got {pages.shape[2]}")
    B = seq_lens.numel()
    _same_device(pages.device, page_table=page_table, seq_lens=seq_lens)
    if out is None:
        out = torch.empty((total_tokens, H, d), dtype=torch.bfloat16, device=pages.device)
    _expect(out, "out", torch.bfloat16, (total_tokens, H, d), pages.device)
    rc = lib().fa_gather_paged(pages.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(),
                               out.data_ptr(), B, H, d, int(page_size), _stream(stream))
    _raise_if(rc, "fa_gather_paged")
    return out


# ---- rotary tables, norms with the rotation, appends with both, the 8-bit cache ----

_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "turns": 3, "yarn": 4}
_FP8 = torch.float8_e4m3fn


# What _calls.so (csrc/calls.cpp) binds, in its order.
_SHORT = ("fa_rope_table", "fa_qk_norm_rope", "fa_qk_norm_rope_bwd",
          "fa_qk_norm_rope_bwd_workspace", "fa_append_paged_rope", "fa_append_paged_fp8",
          "fa_decode_paged_fp8", "fa_decode_paged_fp8_workspace")
_short_calls = None


def _short():
    """The short way into these calls: checks, outputs and scratch in C++, for
    the ordinary case (contiguous tensors of the current GPU, its current
    stream).  It answers None for any other, and the wrapper goes on by itself."""
    global _short_calls
    if _short_calls is None:
        L = lib()
        try:
            from . import _calls
            _same_torch(_calls.torch_version)
        except (ImportError, AttributeError) as e:
            raise ImportError("the binding's _calls.so is missing or of another torch; build "
                              "it with `python -m attn_fwd_04_b200.build`") from e
        _calls.bind(tuple(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in _SHORT))
        _short_calls = _calls
    return _short_calls


def _same_torch(built_for: str):
    """Tensors are read through torch's own C++ classes: one version's only."""
    if not torch.__version__.startswith(built_for):
        raise ImportError(f"built for torch {built_for}, this is {torch.__version__}")


def _answer(out, name: str):
    """A short call's outputs, or the error of the status it stands for."""
    if out.__class__ is tuple:
        return out
    raise FaError(out, name)


# The current stream of a GPU as a handle, without a Stream object around it
# (1.2 us of a call that may take 10).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _call(name: str, dev: int, stream, *args):
    """The library's `name` on `stream` (None: the current one of GPU `dev`, which
    holds the tensors), with that GPU current for the call."""
    fn = getattr(lib(), name)
    if stream is None:
        handle = _raw_stream(dev)
    elif stream.device.index == dev:
        handle = stream.cuda_stream
    else:
        raise ValueError(f"the stream is on {stream.device}, the call's inputs on GPU {dev}")
    if torch.cuda.current_device() == dev:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc != FA_OK:
        raise FaError(rc, name)


@functools.lru_cache(maxsize=256)
def _bytes(name: str, dev: int, *sizes) -> int:
    """The scratch that `name` gives for a call's sizes on GPU `dev`."""
    n = ctypes.c_int(0)
    fn = getattr(lib(), name)
    with torch.cuda.device(dev):
        _raise_if(fn(*sizes, ctypes.byref(n)), name)
    return n.value


def _empty(shape, dtype, device, stream):
    """Memory of the call's own stream (scratch and outputs may be freed, and
    handed out again, in that stream's order)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_like(t, stream):
    # (of a tensor with gaps it makes a dense one, in the same order)
    if stream is None:
        return torch.empty_like(t)
    with torch.cuda.stream(stream):
        return torch.empty_like(t)


def _ptr(t):
    return None if t is None else t.data_ptr()


# These calls take a dozen tensors each, and a decode step's kernels are short:
# a tensor that is as it should be is told by one expression, and what is wrong
# with one that is not is found out afterwards.

def _want(t, name: str, dtype, shape, dev: int):
    """t: contiguous, of this type and shape, on GPU `dev`."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and \
            t.get_device() == dev and t.is_contiguous():
        return
    _check(t, name, dtype, len(shape))
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call's inputs on GPU {dev}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _token_rows(t, name: str, dev=None, shape=None) -> int:
    """t: bf16 [tokens, heads, d] whose rows [heads, d] are contiguous, tokens
    any stride apart; returns that stride."""
    if not isinstance(t, torch.Tensor) or (dev is None and t.device.type not in _DEVICE_TYPES):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    mine = t.shape
    if len(mine) != 3 or (shape is not None and mine != shape):
        raise ValueError(f"{name} must have shape {shape or '[tokens, heads, d]'}, got "
                         f"{tuple(mine)}")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call's inputs on GPU {dev}")
    tokens, heads, d = mine
    st, sh, sd = t.stride()
    # (torch gives a dimension of one any stride)
    if sd == 1 and (sh == d or heads == 1) and heads * d <= st < 1 << 31 and st % 8 == 0:
        return st
    if (sd != 1 and d > 1) or (sh != d and heads > 1):
        raise ValueError(f"{name}: the [heads, d] part of a token must be contiguous")
    if tokens <= 1:
        return heads * d
    raise ValueError(f"{name}: tokens must be a multiple of 8 elements apart, without "
                     f"overlap and less than 2^31; got a stride of {st}")


def _norm_weights(q_weight, k_weight, d: int, dev: int) -> int:
    """The weights' type (FA_WEIGHT_*): [d] bf16 or fp32, one type, or None."""
    if q_weight is None and k_weight is None:
        return 0
    dtype = (k_weight if q_weight is None else q_weight).dtype
    if dtype is not torch.float32:
        dtype = torch.bfloat16
    if q_weight is not None:
        _want(q_weight, "q_weight", dtype, (d,), dev)
    if k_weight is not None:
        _want(k_weight, "k_weight", dtype, (d,), dev)
    return int(dtype is torch.float32)


def _rope(rope_cos, rope_sin, dev: int):
    """(max_pos, rotary_dim) of the tables; (0, 0) without them."""
    if rope_cos is None and rope_sin is None:
        return 0, 0
    if rope_cos is None or rope_sin is None:
        raise ValueError("rope_cos and rope_sin come together")
    if not isinstance(rope_cos, torch.Tensor) or rope_cos.dim() != 2:
        _check(rope_cos, "rope_cos", torch.float32, 2)
    shape = rope_cos.shape
    _want(rope_cos, "rope_cos", torch.float32, shape, dev)
    _want(rope_sin, "rope_sin", torch.float32, shape, dev)
    return shape[0], 2 * shape[1]


def fa_rope_table(max_pos: int, rotary_dim: int, base: float = 10000.0, scaling: str = "none",
                  factor: float = 1.0, original_len: int = 0, low: float = 1.0,
                  high: float = 4.0, mscale: float = 1.0, rope_cos=None, rope_sin=None,
                  device=None, stream=None):
    """Rotary tables (cos, sin), each [max_pos, rotary_dim/2] fp32: mscale times
    the cosine and sine of p * w_i, with the frequencies w_i = base^(-2i/R)
    scaled for long contexts: "none", "linear", "ntk", "turns" (blended by the
    turns within original_len, between low and high) or "yarn" (a ramp over the
    pairs between them)."""
    if rope_cos is None and rope_sin is None and device is None and stream is None:
        out = _short().rope_table(max_pos, rotary_dim, base, _SCALINGS.get(scaling), factor,
                                  original_len, low, high, mscale)
        if out is not None:
            return _answer(out, "fa_rope_table")
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}, got {scaling!r}")
    shape = (int(max_pos), int(rotary_dim) // 2)
    if shape[0] < 1 or shape[1] < 1 or rotary_dim % 2 != 0:
        raise ValueError(f"max_pos must be positive and rotary_dim even, got {max_pos}, "
                         f"{rotary_dim}")
    if rope_cos is None:
        if device is None:
            device = rope_sin.device if rope_sin is not None else \
                stream.device if stream is not None else "cuda"
        rope_cos = _empty(shape, torch.float32, device, stream)
    if rope_sin is None:
        rope_sin = _empty_like(rope_cos, stream)
    dev = rope_cos.get_device()
    _check(rope_cos, "rope_cos", torch.float32, 2)
    _want(rope_cos, "rope_cos", torch.float32, shape, dev)
    _want(rope_sin, "rope_sin", torch.float32, shape, dev)
    _call("fa_rope_table", dev, stream, rope_cos.data_ptr(),
          rope_sin.data_ptr(), shape[0], int(rotary_dim), float(base), _SCALINGS[scaling],
          float(factor), int(original_len), float(low), float(high), float(mscale))
    return rope_cos, rope_sin


def _qk_rows(q, k, positions):
    """What the calls on queries and keys share: (GPU, layout, B, N, H, H_kv, d,
    stride of q, stride of k), positions checked."""
    if isinstance(q, torch.Tensor) and q.dim() == 4:
        _check(q, "q", torch.bfloat16, 4)
        dev = q.get_device()
        B, H, N, d = q.shape
        _check(k, "k", torch.bfloat16, 4)
        H_kv = k.shape[1]
        _want(k, "k", torch.bfloat16, (B, H_kv, N, d), dev)
        if positions is not None:
            _want(positions, "positions", torch.int32, (B, N), dev)
        return dev, 1, B, N, H, H_kv, d, 0, 0
    q_stride = _token_rows(q, "q")
    dev = q.get_device()
    k_stride = _token_rows(k, "k", dev)
    N, H, d = q.shape
    M, H_kv, dk = k.shape
    if M != N or dk != d:
        raise ValueError(f"k must have q's tokens and d, got {tuple(k.shape)} and "
                         f"{tuple(q.shape)}")
    if positions is not None:
        _want(positions, "positions", torch.int32, (N,), dev)
    return dev, 0, 1, N, H, H_kv, d, q_stride, k_stride


def _row_arg(t, name: str, like, layout: int, stream):
    """An output or a gradient of the same shape as `like` and its stride; made
    contiguous on the call's stream where it is None."""
    if t is None:
        return _empty_like(like, stream), 0
    if layout == 1:
        _want(t, name, torch.bfloat16, like.shape, like.get_device())
        return t, 0
    return t, _token_rows(t, name, like.get_device(), like.shape)


def fa_qk_norm_rope(q, k, q_weight=None, k_weight=None, rope_cos=None, rope_sin=None,
                    positions=None, eps: float = 1e-6, interleaved: bool = False, q_out=None,
                    k_out=None, stream=None):
    """Queries and keys normed for each head (weights [d] bf16 or fp32, None: no
    norm) and rotated (tables [max_pos, R/2] fp32 over the first R values, None:
    no rotation) in one pass -> (q_out, k_out).  q [tokens,H,d] and k
    [tokens,H_kv,d] bf16, tokens any stride apart, positions [tokens] int32; or
    [B,H,N,d] and [B,H_kv,N,d] contiguous, positions [B,N].  No positions:
    token n is at position n.  The outputs may be the inputs."""
    if stream is None:
        out = _short().norm(q, k, q_weight, k_weight, rope_cos, rope_sin, positions, eps,
                            interleaved, q_out, k_out)
        if out is not None:
            return _answer(out, "fa_qk_norm_rope")
    dev, layout, B, N, H, H_kv, d, q_st, k_st = _qk_rows(q, k, positions)
    wt = _norm_weights(q_weight, k_weight, d, dev)
    max_pos, rot = _rope(rope_cos, rope_sin, dev)
    q_out, qo_st = _row_arg(q_out, "q_out", q, layout, stream)
    k_out, ko_st = _row_arg(k_out, "k_out", k, layout, stream)
    if B * N == 0:
        return q_out, k_out
    _call("fa_qk_norm_rope", dev, stream, q.data_ptr(), k.data_ptr(),
          q_out.data_ptr(), k_out.data_ptr(), _ptr(q_weight), _ptr(k_weight), wt, _ptr(rope_cos),
          _ptr(rope_sin), max_pos, rot, bool(interleaved), _ptr(positions), layout, B, N, H, H_kv,
          d, q_st, k_st, qo_st, ko_st, eps)
    return q_out, k_out


def fa_qk_norm_rope_bwd_workspace(B: int, N: int, H: int, H_kv: int, d: int) -> int:
    """Bytes of scratch of fa_qk_norm_rope_bwd on the current GPU."""
    n = ctypes.c_int(0)
    _raise_if(lib().fa_qk_norm_rope_bwd_workspace(B, N, H, H_kv, d, ctypes.byref(n)),
              "fa_qk_norm_rope_bwd_workspace")
    return n.value


def fa_qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, rope_cos=None,
                        rope_sin=None, positions=None, eps: float = 1e-6,
                        interleaved: bool = False, dq=None, dk=None, dq_weight=None,
                        dk_weight=None, stream=None):
    """Gradients of fa_qk_norm_rope: (dq, dk, dq_weight, dk_weight) from its
    inputs and its outputs' gradients; the weights' gradients are fp32 [d], None
    where there is no weight."""
    if stream is None:
        out = _short().norm_bwd(q, k, dq_out, dk_out, q_weight, k_weight, rope_cos, rope_sin,
                                positions, eps, interleaved, dq, dk, dq_weight, dk_weight)
        if out is not None:
            return _answer(out, "fa_qk_norm_rope_bwd")
    dev, layout, B, N, H, H_kv, d, q_st, k_st = _qk_rows(q, k, positions)
    wt = _norm_weights(q_weight, k_weight, d, dev)
    max_pos, rot = _rope(rope_cos, rope_sin, dev)
    for t, n in ((dq_out, "dq_out"), (dk_out, "dk_out")):
        if t is None:
            raise TypeError(f"{n} must be a CUDA tensor")
    dq_out, gq_st = _row_arg(dq_out, "dq_out", q, layout, stream)
    dk_out, gk_st = _row_arg(dk_out, "dk_out", k, layout, stream)
    dq, dq_st = _row_arg(dq, "dq", q, layout, stream)
    dk, dk_st = _row_arg(dk, "dk", k, layout, stream)
    grads = []
    for w, g, n in ((q_weight, dq_weight, "dq_weight"), (k_weight, dk_weight, "dk_weight")):
        if g is not None:
            if w is None:
                raise ValueError(f"{n} given without its weight")
            _want(g, n, torch.float32, (d,), dev)
        elif w is not None:
            g = _empty((d,), torch.float32, q.device, stream)
        grads.append(g)
    if B * N == 0:
        with torch.cuda.stream(stream):
            for g in grads:
                if g is not None:
                    g.zero_()
        return dq, dk, grads[0], grads[1]
    ws, n = None, 0
    if q_weight is not None or k_weight is not None:
        n = _bytes("fa_qk_norm_rope_bwd_workspace", dev, B, N, H, H_kv, d)
        ws = _empty((n,), torch.uint8, q.device, stream)
    _call("fa_qk_norm_rope_bwd", dev, stream, q.data_ptr(), k.data_ptr(),
          dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), _ptr(grads[0]),
          _ptr(grads[1]), _ptr(q_weight), _ptr(k_weight), wt, _ptr(rope_cos), _ptr(rope_sin),
          max_pos, rot, bool(interleaved), _ptr(positions), layout, B, N, H, H_kv, d, q_st, k_st,
          gq_st, gk_st, dq_st, dk_st, eps, _ptr(ws), n)
    return dq, dk, grads[0], grads[1]


def _table(page_table, B: int, dev: int):
    """(entries, entries of a row) of a packed page table [n] (rows 0) or a
    block table [B, max_pages]."""
    rows = isinstance(page_table, torch.Tensor) and page_table.dim() == 2
    if not rows:
        _check(page_table, "page_table", torch.int32, 1)
    shape = page_table.shape
    if rows and shape[0] != B:
        raise ValueError("a block table must have one row per sequence")
    _want(page_table, "page_table", torch.int32, shape, dev)
    return page_table.numel(), shape[1] if rows else 0


def _pool(k_pages, v_pages, dtype, page_size: int, d: int, heads, dev: int):
    """(pages, K/V heads) of a pool [P, heads, page_size, d], heads given or any."""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        _check(k_pages, "k_pages", dtype, 4)
    shape = k_pages.shape
    P, H_kv = shape[0], shape[1]
    _want(k_pages, "k_pages", dtype, shape, dev)
    if v_pages.shape != shape or shape[2] != page_size or shape[3] != d or \
            (heads is not None and H_kv != heads):
        _pages(k_pages, v_pages, page_size, d, heads=heads)
    _want(v_pages, "v_pages", dtype, shape, dev)
    return P, H_kv


def _scale_block(k_scales, v_scales, P: int, H_kv: int, page_size: int, dev: int) -> int:
    """Tokens that share a scale: scales [P, H_kv, page_size / block] fp32."""
    _check(k_scales, "k_scales", torch.float32, 3)
    shape = k_scales.shape
    n = shape[2]
    if shape[0] != P or shape[1] != H_kv or n < 1 or page_size % n != 0:
        raise ValueError(f"scales must be [{P}, {H_kv}, {page_size} / block], got "
                         f"{tuple(shape)}")
    _want(k_scales, "k_scales", torch.float32, shape, dev)
    _want(v_scales, "v_scales", torch.float32, shape, dev)
    return page_size // n


def _append(name, q_new, k_new, v_new, cu_new, k_pages, v_pages, scales, page_table, seq_lens,
            rope_cos, rope_sin, q_weight, k_weight, eps, interleaved, page_size, q_out, stream):
    """Checks and call of both appends; `scales`: (k_scales, v_scales) or ()."""
    if stream is None:
        out = _short().append(q_new, k_new, v_new, cu_new, k_pages, v_pages,
                              *(scales or (None, None)), page_table, seq_lens, rope_cos, rope_sin,
                              q_weight, k_weight, eps, interleaved, page_size, q_out)
        if out is not None:
            return _answer(out, name)[0]
    k_st = _token_rows(k_new, "k_new")
    dev = k_new.get_device()
    total, H_kv, d = shape = k_new.shape
    v_st = _token_rows(v_new, "v_new", dev, shape)
    H, q_st = 0, 0
    if q_new is not None:
        q_st = _token_rows(q_new, "q_new", dev)
        q_shape = q_new.shape
        H = q_shape[1]
        if q_shape[0] != total or q_shape[2] != d:
            raise ValueError(f"q_new must have k_new's tokens and d, got {tuple(q_shape)}")
        if q_out is None:
            q_out = _empty_like(q_new, stream)
        else:
            _want(q_out, "q_out", torch.bfloat16, q_shape, dev)
    elif q_out is not None or q_weight is not None:
        raise ValueError("q_out and q_weight need q_new")
    P, _ = _pool(k_pages, v_pages, _FP8 if scales else torch.bfloat16, page_size, d, H_kv, dev)
    _check(cu_new, "cu_new", torch.int32, 1)
    B = cu_new.numel() - 1
    _want(cu_new, "cu_new", torch.int32, (B + 1,), dev)
    _want(seq_lens, "seq_lens", torch.int32, (B,), dev)
    table_len, max_pages = _table(page_table, B, dev)
    block = (_scale_block(*scales, P, H_kv, page_size, dev),) if scales else ()
    wt = _norm_weights(q_weight, k_weight, d, dev)
    max_pos, rot = _rope(rope_cos, rope_sin, dev)
    if total == 0:
        return q_out
    _call(name, dev, stream, _ptr(q_new), k_new.data_ptr(), v_new.data_ptr(),
          cu_new.data_ptr(), _ptr(q_out), k_pages.data_ptr(), v_pages.data_ptr(),
          *[s.data_ptr() for s in scales], *block, page_table.data_ptr() or seq_lens.data_ptr(),
          table_len, max_pages, seq_lens.data_ptr(), _ptr(q_weight), _ptr(k_weight), wt,
          _ptr(rope_cos), _ptr(rope_sin), max_pos, rot, bool(interleaved), B, H, H_kv, total, P,
          d, page_size, q_st, k_st, v_st, eps)
    return q_out


def fa_append_paged_rope(q_new, k_new, v_new, cu_new, k_pages, v_pages, page_table, seq_lens,
                         rope_cos=None, rope_sin=None, q_weight=None, k_weight=None,
                         eps: float = 1e-6, interleaved: bool = False, page_size: int = 256,
                         q_out=None, stream=None):
    """fa_append_paged with the norms and the rotation on the way: new rows
    [tokens, heads, d] bf16 (any stride between tokens) of sequences cu_new; keys
    normed, rotated and written to their pages, values written as they are,
    queries normed and rotated -> q_out (None without q_new).  page_table packed
    [n] or a block table [B, max_pages]; seq_lens after the append."""
    return _append("fa_append_paged_rope", q_new, k_new, v_new, cu_new, k_pages, v_pages, (),
                   page_table, seq_lens, rope_cos, rope_sin, q_weight, k_weight, eps,
                   interleaved, page_size, q_out, stream)


def fa_append_paged_fp8(q_new, k_new, v_new, cu_new, k_pages, v_pages, k_scales, v_scales,
                        page_table, seq_lens, rope_cos=None, rope_sin=None, q_weight=None,
                        k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                        page_size: int = 256, q_out=None, stream=None):
    """fa_append_paged_rope into pages of torch.float8_e4m3fn values with scales
    [P, H_kv, 256 / block] fp32, one for each block of tokens and head (updated
    in place with the pages) -> q_out."""
    return _append("fa_append_paged_fp8", q_new, k_new, v_new, cu_new, k_pages, v_pages,
                   (k_scales, v_scales), page_table, seq_lens, rope_cos, rope_sin, q_weight,
                   k_weight, eps, interleaved, page_size, q_out, stream)


def fa_decode_paged_fp8_workspace(B: int, H: int, H_kv: int, d: int) -> int:
    """Bytes of scratch of fa_decode_paged_fp8 on the current GPU."""
    n = ctypes.c_int(0)
    _raise_if(lib().fa_decode_paged_fp8_workspace(B, H, H_kv, d, ctypes.byref(n)),
              "fa_decode_paged_fp8_workspace")
    return n.value


def fa_decode_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, page_table, seq_lens,
                        page_size: int = 256, scale: Optional[float] = None, o=None, lse=None,
                        stream=None):
    """Decode over the 8-bit cache: q [B,H,d] bf16, pages [P,H_kv,page_size,d]
    torch.float8_e4m3fn with scales [P,H_kv,page_size/block] fp32, page_table
    packed [n] or a block table [B, max_pages] -> o [B,H,d] bf16; `lse` [B,H]
    fp32 is filled where it is given."""
    if stream is None:
        out = _short().decode(q, k_pages, v_pages, k_scales, v_scales, page_table, seq_lens,
                              page_size, scale, o, lse)
        if out is not None:
            return _answer(out, "fa_decode_paged_fp8")[0]
    _check(q, "q", torch.bfloat16, 3)
    dev = q.get_device()
    B, H, d = shape = q.shape
    P, H_kv = _pool(k_pages, v_pages, _FP8, page_size, d, None, dev)
    if H_kv == 0 or H % H_kv != 0:
        raise ValueError(f"H ({H}) must be a multiple of the cache's K/V heads ({H_kv})")
    _want(seq_lens, "seq_lens", torch.int32, (B,), dev)
    block = _scale_block(k_scales, v_scales, P, H_kv, page_size, dev)
    table_len, max_pages = _table(page_table, B, dev)
    if o is None:
        o = _empty_like(q, stream)
    else:
        _want(o, "o", torch.bfloat16, shape, dev)
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, H), dev)
    if B == 0:
        return o
    n = _bytes("fa_decode_paged_fp8_workspace", dev, B, H, H_kv, d)
    ws = _empty((n,), torch.uint8, q.device, stream)
    _call("fa_decode_paged_fp8", dev, stream, q.data_ptr(), k_pages.data_ptr(),
          v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), block,
          page_table.data_ptr() or seq_lens.data_ptr(), table_len, max_pages,
          seq_lens.data_ptr(), o.data_ptr(), _ptr(lse), B, H, H_kv, P, d, page_size,
          d ** -0.5 if scale is None else scale, ws.data_ptr(), n)
    return o


def fa_get_device_error(stream=None) -> int:
    """Synchronise the stream, read and clear the device error word (FA_* code)."""
    code = ctypes.c_int(0)
    rc = lib().fa_get_device_error(ctypes.byref(code), _stream(stream))
    _raise_if(rc, "fa_get_device_error")
    return code.value


def fa_selftest_bounded_wait(stream=None) -> None:
    """Launch the bounded-wait self test; read the result with fa_get_device_error."""
    _raise_if(lib().fa_selftest_bounded_wait(_stream(stream)), "fa_selftest_bounded_wait")


def fa_selftest_fwd_stall(q, k, v, withheld: int, wait_us: int, o=None, lse=None,
                          stream=None):
    """Launch the causal forward pass with K/V copy `withheld` never issued and
    every wait bounded by wait_us; read the outcome with fa_get_device_error."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, torch.bfloat16, 4)
    B, H, N, d = q.shape
    if k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must have the same [B,H,N,d] shape")
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _expect(o, "o", torch.bfloat16, q.shape, q.device)
    _expect(lse, "lse", torch.float32, (B, H, N), q.device)
    rc = lib().fa_selftest_fwd_stall(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                     lse.data_ptr(), B, H, N, d, int(withheld), int(wait_us),
                                     _stream(stream))
    _raise_if(rc, "fa_selftest_fwd_stall")
    return o, lse


def fa_selftest_decode_stall(q, k_pages, v_pages, page_table, seq_lens, withheld: int,
                             wait_us: int, page_size: int = 256, o=None, stream=None):
    """Launch the paged decode with no copy issued from ring use `withheld` on
    and every wait bounded by wait_us; read the outcome with
    fa_get_device_error."""
    _check(q, "q", torch.bfloat16, 3)
    _check(k_pages, "k_pages", torch.bfloat16, 4)
    _check(v_pages, "v_pages", torch.bfloat16, 4)
    _check(page_table, "page_table", torch.int32, 1)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    B, H, d = q.shape
    _pages(k_pages, v_pages, page_size, d, heads=H)
    if seq_lens.numel() != B:
        raise ValueError(f"seq_lens must hold one length per sequence ({B})")
    _same_device(q.device, k_pages=k_pages, v_pages=v_pages, page_table=page_table,
                 seq_lens=seq_lens)
    o = torch.empty_like(q) if o is None else o
    _expect(o, "o", torch.bfloat16, q.shape, q.device)
    rc = lib().fa_selftest_decode_stall(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                        page_table.data_ptr(), seq_lens.data_ptr(), o.data_ptr(),
                                        B, H, d, int(page_size), int(withheld), int(wait_us),
                                        _stream(stream))
    _raise_if(rc, "fa_selftest_decode_stall")
    return o


def fa_release_workspace() -> None:
    _raise_if(lib().fa_release_workspace(), "fa_release_workspace")


def fa_version() -> int:
    return lib().fa_version()


def fa_fwd_set_cta_pairs(enable: bool) -> bool:
    """Select the CTA-pair (True) or single-CTA (False, default) forward kernel
    for d = 128; returns the previous setting."""
    return bool(lib().fa_fwd_set_cta_pairs(int(bool(enable))))
