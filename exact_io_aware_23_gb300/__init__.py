"""Python binding of libfa, the exact-attention C ABI (include/fa.h), for GB300 (sm_103a).

This module only marshals arguments: it checks tensor placement, dtype and shape, passes raw
device pointers and the current CUDA stream to the C functions, and turns a non-OK status into
an exception.  Every step of the computation runs in the library's CUDA kernels.  Importing
fails loudly when the library has not been built (``__graft_entry__.build()``); there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
from typing import Optional, Tuple

import torch

__all__ = ["forward", "forward_splitkv", "backward", "backward_noalloc", "backward_workspace_size",
           "backward_fused_workspace_size", "check_device_status", "set_fault_injection",
           "set_wait_limit_ms", "FaError", "LIB_PATH", "lib", "rotary", "rotary_backward",
           "rotary_frequencies", "append_paged", "forward_paged", "forward_paged_workspace_size",
           "select_pages", "select_pages_workspace_size", "assign_pages"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(5)
FA_BF16, FA_FP32, FA_FP16 = 0, 1, 2
_DTYPES = {torch.bfloat16: FA_BF16, torch.float32: FA_FP32, torch.float16: FA_FP16}


class FaDropout(ctypes.Structure):
    """fa_dropout: dropout probability, generator key and counter offset."""
    _fields_ = [("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint32)]


class FaScoreMod(ctypes.Structure):
    """fa_score_mod: cap of the scores, distance slopes and prefix lengths (device pointers)."""
    _fields_ = [("softcap", ctypes.c_float), ("alibi_slopes", ctypes.c_void_p),
                ("prefix_lens", ctypes.c_void_p)]


class FaPagedCache(ctypes.Structure):
    """fa_paged_cache: where a paged cache's keys and values lie."""
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("n_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("block_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("max_pages", ctypes.c_int),
                ("kv_lens", ctypes.c_void_p)]


class FaPageStore(ctypes.Structure):
    """fa_page_store: the pages' format, their scales and the bounds of their keys."""
    _fields_ = [("format", ctypes.c_int), ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("k_bounds", ctypes.c_void_p), ("bound_scales", ctypes.c_void_p)]


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib.fa_status_string(status).decode()}")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libfa.so is not built ({LIB_PATH}); run __graft_entry__.build()")
    L = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.fa_forward.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, i, vp, vp]
    L.fa_forward.restype = i
    L.fa_backward_workspace_size.argtypes = [i, i, i, i]
    L.fa_backward_workspace_size.restype = sz
    L.fa_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, i, vp,
                              vp, sz, vp]
    L.fa_backward.restype = i
    L.fa_check_device_status.argtypes = [vp]
    L.fa_check_device_status.restype = i
    L.fa_status_string.argtypes = [i]
    L.fa_status_string.restype = ctypes.c_char_p
    L.fa_debug_set_fault_injection.argtypes = [i]
    L.fa_debug_set_fault_injection.restype = None
    L.fa_debug_set_wait_limit_ms.argtypes = [ctypes.c_uint32]
    L.fa_debug_set_wait_limit_ms.restype = None
    L.fa_version.argtypes = []
    L.fa_version.restype = i
    L.fa_forward_gqa.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, i, vp, vp]
    L.fa_forward_gqa.restype = i
    L.fa_forward_blocksparse.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, i, vp, vp, sz, vp]
    L.fa_forward_blocksparse.restype = i
    L.fa_forward_blocksparse_workspace_size.argtypes = [i, i, i, i]
    L.fa_forward_blocksparse_workspace_size.restype = sz
    L.fa_backward_gqa.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, i,
                                  vp, vp, sz, vp]
    L.fa_backward_gqa.restype = i
    L.fa_backward_deterministic.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f,
                                            i, vp, i, vp, vp, sz, vp]
    L.fa_backward_deterministic.restype = i
    L.fa_backward_deterministic_workspace_size.argtypes = [i, i, i]
    L.fa_backward_deterministic_workspace_size.restype = sz
    L.fa_forward_varlen.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp]
    L.fa_forward_varlen.restype = i
    L.fa_backward_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f,
                                     i, i, vp, sz, vp]
    L.fa_backward_varlen.restype = i
    dp = ctypes.POINTER(FaDropout)
    L.fa_forward_dropout.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, i, vp, dp, vp]
    L.fa_forward_dropout.restype = i
    L.fa_backward_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, i,
                                      vp, dp, vp, sz, vp]
    L.fa_backward_dropout.restype = i
    L.fa_backward_fused.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, i,
                                    vp, vp, sz, vp]
    L.fa_backward_fused.restype = i
    L.fa_backward_fused_workspace_size.argtypes = [i, i, i, i]
    L.fa_backward_fused_workspace_size.restype = sz
    L.fa_forward_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, i, i, vp, sz, vp]
    L.fa_forward_splitkv_gqa.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp, i, i, vp, sz, vp]
    L.fa_forward_splitkv_gqa.restype = i
    L.fa_forward_splitkv.restype = i
    L.fa_forward_splitkv_workspace_size.argtypes = [i, i, i, i, i]
    L.fa_forward_splitkv_workspace_size.restype = sz
    L.fa_forward_splitkv_auto_splits.argtypes = [i, i, i, i]
    L.fa_forward_splitkv_auto_splits.restype = i
    L.fa_backward_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, i,
                                      vp, vp]
    L.fa_backward_noalloc.restype = i
    L.fa_backward_noalloc_max_workspace.argtypes = []
    L.fa_backward_noalloc_max_workspace.restype = sz
    st3, i64 = ctypes.c_int64 * 3, ctypes.c_int64
    L.fa_rotary.argtypes = [vp, st3, vp, st3, i, i, i, i, vp, i64, vp, i, i, f, i, vp]
    L.fa_rotary.restype = i
    L.fa_rotary_backward.argtypes = L.fa_rotary.argtypes
    L.fa_rotary_backward.restype = i
    cp, mp = ctypes.POINTER(FaPagedCache), ctypes.POINTER(FaScoreMod)
    L.fa_forward_scored.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, mp, vp]
    L.fa_forward_scored.restype = i
    L.fa_backward_scored.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, mp, vp, sz, vp]
    L.fa_backward_scored.restype = i
    L.fa_forward_varlen_scored.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, mp, vp]
    L.fa_forward_varlen_scored.restype = i
    L.fa_backward_varlen_scored.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i,
                                            mp, vp, sz, vp]
    L.fa_backward_varlen_scored.restype = i
    L.fa_append_paged.argtypes = [cp, vp, st3, vp, st3, vp, st3, vp, i, i, i, i, i, vp, vp, i, i, f, i, vp]
    L.fa_append_paged.restype = i
    L.fa_forward_paged_workspace_size.argtypes = [i, i, i, i, i, i]
    L.fa_forward_paged_workspace_size.restype = sz
    L.fa_forward_paged.argtypes = [vp, cp, vp, vp, i, i, i, i, i, f, vp, mp, i, vp, sz, vp]
    L.fa_forward_paged.restype = i
    fp = ctypes.POINTER(FaPageStore)
    L.fa_append_paged_store.argtypes = [cp, fp, vp, st3, vp, st3, vp, st3, vp, i, i, i, i, i, vp, vp, i, i, f, i, vp]
    L.fa_append_paged_store.restype = i
    L.fa_forward_paged_store.argtypes = [vp, cp, fp, vp, i, vp, vp, i, i, i, i, i, f, vp, mp, i, vp, sz, vp]
    L.fa_forward_paged_store.restype = i
    L.fa_select_pages_workspace_size.argtypes = [i, i, i, i]
    L.fa_select_pages_workspace_size.restype = sz
    L.fa_select_pages.argtypes = [vp, cp, fp, vp, i, i, i, i, i, vp, i, i, i, i, vp, sz, vp]
    L.fa_select_pages.restype = i
    L.fa_assign_pages.argtypes = [vp, i64, i, i, i, vp, vp, vp, i, vp, vp, vp, vp, vp, vp, i, vp]
    L.fa_assign_pages.restype = i
    for packed in (L.fa_append_paged_store_packed, L.fa_forward_paged_store_packed, L.fa_select_pages_packed, L.fa_assign_pages_packed, L.fa_forward_scored_packed, L.fa_backward_scored_packed, L.fa_rotary_packed,
                   L.fa_rotary_backward_packed, L.fa_append_paged_packed, L.fa_forward_paged_packed):
        packed.argtypes = [ctypes.c_char_p]
        packed.restype = i
    return L


lib = _load()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check_qkv(q, k, v):
    """q: [B, H, N, d]; k, v: [B, Hkv, N, d] with Hkv dividing H (grouped-query attention when
    Hkv < H).  Returns (B, H, N, d, Hkv)."""
    qshape, kshape, dtype = q.shape, k.shape, q.dtype
    if not (q.is_cuda and k.is_cuda and v.is_cuda and q.is_contiguous() and k.is_contiguous()
            and v.is_contiguous() and len(qshape) == len(kshape) == v.dim() == 4):
        for name, t in (("q", q), ("k", k), ("v", v)):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous CUDA tensor")
            if t.dim() != 4:
                raise ValueError(f"{name} must be [B, H, N, d]")
    B, H, N, d = qshape
    Bk, Hkv, Nk, dk = kshape
    if kshape != v.shape or Bk != B or Nk != N or dk != d or H % Hkv != 0:
        raise ValueError("k, v must be [B, Hkv, N, d] with Hkv dividing the query heads")
    if not (dtype == k.dtype == v.dtype):
        raise ValueError("q, k, v must share a dtype")
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    return B, H, N, d, Hkv


def _masks(block_mask, kv_lens, B, N, device):
    if block_mask is not None:
        T = (N + 127) // 128
        if block_mask.dtype != torch.uint8 or tuple(block_mask.shape) != (T, T):
            raise ValueError(f"block_mask must be uint8 [{T}, {T}]")
        block_mask = block_mask.to(device).contiguous()
    if kv_lens is not None:
        if kv_lens.dtype != torch.int32 or tuple(kv_lens.shape) != (B,):
            raise ValueError(f"kv_lens must be int32 [{B}]")
        kv_lens = (kv_lens if kv_lens.device == device else kv_lens.to(device)).contiguous()
    return block_mask, kv_lens


def forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, causal: bool = False,
            scale: Optional[float] = None, block_mask: Optional[torch.Tensor] = None,
            kv_lens: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None,
            lse: Optional[torch.Tensor] = None, stream=None, dropout_p: float = 0.0,
            seed: int = 0, offset: int = 0, balanced: bool = True,
            workspace: Optional[torch.Tensor] = None, softcap: float = 0.0,
            alibi_slopes: Optional[torch.Tensor] = None,
            prefix_lens: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """O, LSE = attention forward (fa_forward; fa_forward_gqa when k, v have fewer heads;
    fa_forward_dropout when dropout_p > 0; with a block mask and 16-bit inputs,
    fa_forward_blocksparse unless balanced=False).  q: [B, H, N, d]; k, v: [B, Hkv, N, d];
    bf16, fp16 or fp32 on CUDA.  With softcap > 0 (scores capped by softcap * tanh(. / softcap)),
    alibi_slopes (fp32 [H]: scores lowered by the slope times |i - j|) or prefix_lens (int32 [B]:
    leading keys seen in spite of causal), fa_forward_scored: bf16 or fp16, no block mask or
    dropout."""
    if softcap != 0.0 or alibi_slopes is not None or prefix_lens is not None:
        if block_mask is not None or dropout_p > 0.0:
            raise ValueError("score modifications take no block mask and no dropout")
        return _forward_scored(q, k, v, causal, scale, kv_lens, o, lse, stream, softcap, alibi_slopes, prefix_lens)
    B, H, N, d, Hkv = _check_qkv(q, k, v)
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    if block_mask is not None or kv_lens is not None:
        block_mask, kv_lens = _masks(block_mask, kv_lens, B, N, q.device)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    if dropout_p > 0.0:
        drop = FaDropout(float(dropout_p), int(seed), int(offset))
        st = lib.fa_forward_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, N, d,
                                    scale, int(bool(causal)), _ptr(block_mask), _DTYPES[q.dtype],
                                    _ptr(kv_lens), ctypes.byref(drop), _stream(stream))
        if st != FA_OK:
            raise FaError(st, "fa_forward_dropout")
        return o, lse
    if block_mask is not None and balanced and q.dtype != torch.float32:
        need = int(lib.fa_forward_blocksparse_workspace_size(B, H, N, d))
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
        st = lib.fa_forward_blocksparse(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, N,
                                        d, scale, int(bool(causal)), _ptr(block_mask),
                                        _DTYPES[q.dtype], _ptr(kv_lens), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream))
        if st != FA_OK:
            raise FaError(st, "fa_forward_blocksparse")
        return o, lse
    if Hkv == H:
        st = lib.fa_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, scale,
                            int(bool(causal)), _ptr(block_mask), _DTYPES[q.dtype], _ptr(kv_lens),
                            _stream(stream))
    else:
        st = lib.fa_forward_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, N, d,
                                scale, int(bool(causal)), _ptr(block_mask), _DTYPES[q.dtype],
                                _ptr(kv_lens), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_forward")
    return o, lse


def _check_packed(q, k, v, cu_seqlens):
    """q: [H, total, d]; k, v: [Hkv, total, d]; cu_seqlens: int32 [n_seqs + 1] on q's device."""
    qshape, kshape, dtype = q.shape, k.shape, q.dtype
    if not (q.is_cuda and k.is_cuda and v.is_cuda and q.is_contiguous() and k.is_contiguous()
            and v.is_contiguous() and len(qshape) == len(kshape) == v.dim() == 3):
        for name, t in (("q", q), ("k", k), ("v", v)):
            if not t.is_cuda or not t.is_contiguous() or t.dim() != 3:
                raise ValueError(f"{name} must be a contiguous CUDA tensor [heads, total, d]")
    H, T, d = qshape
    Hkv, Tk, dk = kshape
    if kshape != v.shape or Tk != T or dk != d or H % Hkv != 0:
        raise ValueError("k, v must be [Hkv, total, d] with Hkv dividing the query heads")
    if not (dtype == k.dtype == v.dtype) or dtype not in _DTYPES:
        raise ValueError("q, k, v must share a supported dtype")
    if (cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1
            or cu_seqlens.device != q.device or not cu_seqlens.is_contiguous()):
        raise ValueError("cu_seqlens must be a contiguous int32 [n_seqs + 1] tensor on q's device")
    return H, Hkv, T, d, cu_seqlens.numel() - 1


def forward_varlen(q, k, v, cu_seqlens, max_seqlen: int, *, causal: bool = False,
                   scale: Optional[float] = None, stream=None, softcap: float = 0.0,
                   alibi_slopes: Optional[torch.Tensor] = None,
                   prefix_lens: Optional[torch.Tensor] = None):
    """fa_forward_varlen: sequences packed along the token axis (q [H, total, d], k, v
    [Hkv, total, d], offsets cu_seqlens); returns O [H, total, d] and LSE [H, total].  softcap,
    alibi_slopes and prefix_lens (int32 [n_seqs]) as in ``forward`` (fa_forward_varlen_scored);
    distances and prefixes count within a sequence."""
    H, Hkv, T, d, S = _check_packed(q, k, v, cu_seqlens)
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    o = torch.empty_like(q)
    lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    if softcap != 0.0 or alibi_slopes is not None or prefix_lens is not None:
        dev, slopes, prefix = _score_args(q, k, v, None, None, None, alibi_slopes, prefix_lens, H, S)
        st = lib.fa_forward_scored_packed(_SCORED.pack(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), 0, 0, 0, 0, 0,
            cu_seqlens.data_ptr(), slopes, prefix, 0, 0, _handle(stream, dev, o, lse),
            S, H, Hkv, int(max_seqlen), T, d, 1 if causal else 0, _DTYPES[q.dtype], scale, softcap))
        if st != FA_OK:
            raise FaError(st, "fa_forward_varlen_scored")
        return o, lse
    st = lib.fa_forward_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens), S,
                               int(max_seqlen), T, H, Hkv, d, scale, int(bool(causal)),
                               _DTYPES[q.dtype], _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_forward_varlen")
    return o, lse


def backward_varlen(q, k, v, o, lse, do, cu_seqlens, max_seqlen: int, *, causal: bool = False,
                    scale: Optional[float] = None, stream=None, softcap: float = 0.0,
                    alibi_slopes: Optional[torch.Tensor] = None,
                    prefix_lens: Optional[torch.Tensor] = None):
    """fa_backward_varlen: dQ [H, total, d], dK, dV [Hkv, total, d] for packed sequences
    (fa_backward_varlen_scored with the score arguments of ``forward_varlen``)."""
    H, Hkv, T, d, S = _check_packed(q, k, v, cu_seqlens)
    for name, t in (("o", o), ("do", do)):
        if t.shape != q.shape or t.dtype != q.dtype or not t.is_contiguous():
            raise ValueError(f"{name} must match q")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (H, T):
        raise ValueError("lse must be fp32 [H, total]")
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    need = backward_deterministic_workspace_size(1, H, T)
    workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    if softcap != 0.0 or alibi_slopes is not None or prefix_lens is not None:
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
        dev, slopes, prefix = _score_args(q, k, v, o, lse, do, alibi_slopes, prefix_lens, H, S)
        st = lib.fa_backward_scored_packed(_SCORED.pack(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), do.data_ptr(), dq.data_ptr(),
            dk.data_ptr(), dv.data_ptr(), 0, cu_seqlens.data_ptr(), slopes, prefix, workspace.data_ptr(),
            workspace.numel(), _handle(stream, dev, dq, dk, dv, workspace),
            S, H, Hkv, int(max_seqlen), T, d, 1 if causal else 0, _DTYPES[q.dtype], scale, softcap))
        if st != FA_OK:
            raise FaError(st, "fa_backward_varlen_scored")
        return dq, dk, dv
    st = lib.fa_backward_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                                _ptr(dk), _ptr(dv), _ptr(cu_seqlens), S, int(max_seqlen), T, H,
                                Hkv, d, scale, int(bool(causal)), _DTYPES[q.dtype],
                                _ptr(workspace), workspace.numel(), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_backward_varlen")
    return dq, dk, dv


def forward_splitkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
                    scale: Optional[float] = None, kv_lens: Optional[torch.Tensor] = None,
                    n_splits: int = 0, o: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """O, LSE with the key sequence cut into ranges merged afterwards (fa_forward_splitkv;
    fa_forward_splitkv_gqa when k, v have fewer heads).  q: [B, H, Nq, d]; k, v: [B, Hkv, Nk, d]
    with Hkv dividing H; bf16 or fp16; no causal or tile mask."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous 4-D CUDA tensor")
    B, H, Nq, d = q.shape
    Nk, Hkv = k.shape[2], k.shape[1]
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != d or H % Hkv != 0:
        raise ValueError("k, v must be [B, Hkv, Nk, d] with Hkv dividing the query heads")
    if not (q.dtype == k.dtype == v.dtype) or q.dtype not in _DTYPES:
        raise ValueError("q, k, v must share a supported dtype")
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    _, kv_lens = _masks(None, kv_lens, B, Nq, q.device)
    G = H // Hkv                       # a group's query heads run as one block of G * Nq rows
    splits = (int(lib.fa_forward_splitkv_auto_splits(B, Hkv, G * Nq, Nk)) if n_splits == 0
              else int(n_splits))
    splits = max(1, min(splits, (Nk + 127) // 128 or 1))
    need = int(lib.fa_forward_splitkv_workspace_size(B, H, Nq, d, splits))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    if Hkv == H:
        st = lib.fa_forward_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk, d,
                                    scale, _ptr(kv_lens), _DTYPES[q.dtype], splits, _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream))
    else:
        st = lib.fa_forward_splitkv_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, Nq,
                                        Nk, d, scale, _ptr(kv_lens), _DTYPES[q.dtype], splits,
                                        _ptr(workspace), workspace.numel() * workspace.element_size(),
                                        _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_forward_splitkv")
    return o, lse


def backward_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(lib.fa_backward_workspace_size(B, H, N, d))


def backward_deterministic_workspace_size(B: int, H: int, N: int) -> int:
    return int(lib.fa_backward_deterministic_workspace_size(B, H, N))


def backward_fused_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(lib.fa_backward_fused_workspace_size(B, H, N, d))


def backward(q, k, v, o, lse, do, *, causal: bool = False, scale: Optional[float] = None,
             block_mask=None, kv_lens=None, dq=None, dk=None, dv=None, workspace=None,
             stream=None, deterministic: bool = False, fused: bool = False,
             dropout_p: float = 0.0, seed: int = 0, offset: int = 0, softcap: float = 0.0,
             alibi_slopes: Optional[torch.Tensor] = None,
             prefix_lens: Optional[torch.Tensor] = None):
    """dQ, dK, dV = recompute-based attention backward (fa_backward; fa_backward_gqa when k, v
    have fewer heads than q; fa_backward_deterministic, bit-reproducible, when asked;
    fa_backward_fused, the single-pass atomic-dQ variant, when asked; fa_backward_scored,
    bit-reproducible too, with the score arguments of ``forward``)."""
    if softcap != 0.0 or alibi_slopes is not None or prefix_lens is not None:
        if block_mask is not None or dropout_p > 0.0 or fused:
            raise ValueError("score modifications take no block mask, no dropout and no fused backward")
        return _backward_scored(q, k, v, o, lse, do, causal, scale, kv_lens, dq, dk, dv, workspace, stream, softcap,
                                alibi_slopes, prefix_lens)
    B, H, N, d, Hkv = _check_qkv(q, k, v)
    shape, dtype = q.shape, q.dtype
    if o.shape != shape or o.dtype != dtype or not o.is_contiguous():
        raise ValueError("o must match q")
    if do.shape != shape or do.dtype != dtype or not do.is_contiguous():
        raise ValueError("do must match q")
    if lse.dtype != torch.float32 or lse.shape != (B, H, N):
        raise ValueError("lse must be fp32 [B, H, N]")
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    if block_mask is not None or kv_lens is not None:
        block_mask, kv_lens = _masks(block_mask, kv_lens, B, N, q.device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if fused and (deterministic or dropout_p > 0.0):
        raise ValueError("the fused backward has no deterministic or dropout form")
    need = (backward_fused_workspace_size(B, H, N, d) if fused
            else backward_deterministic_workspace_size(B, H, N) if deterministic or dropout_p > 0.0
            else backward_workspace_size(B, H, N, d))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv))
    tail = (d, scale, int(bool(causal)), _ptr(block_mask), _DTYPES[q.dtype], _ptr(kv_lens),
            _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if dropout_p > 0.0:
        drop = FaDropout(float(dropout_p), int(seed), int(offset))
        st = lib.fa_backward_dropout(*args, B, H, Hkv, N, d, scale, int(bool(causal)),
                                     _ptr(block_mask), _DTYPES[q.dtype], _ptr(kv_lens),
                                     ctypes.byref(drop), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream))
        if st != FA_OK:
            raise FaError(st, "fa_backward_dropout")
        return dq, dk, dv
    if deterministic:
        st = lib.fa_backward_deterministic(*args, B, H, Hkv, N, *tail)
        if st != FA_OK:
            raise FaError(st, "fa_backward_deterministic")
        return dq, dk, dv
    if fused:
        st = lib.fa_backward_fused(*args, B, H, Hkv, N, *tail)
        if st != FA_OK:
            raise FaError(st, "fa_backward_fused")
        return dq, dk, dv
    if Hkv == H:
        st = lib.fa_backward(*args, B, H, N, *tail)
    else:
        st = lib.fa_backward_gqa(*args, B, H, Hkv, N, *tail)
    if st != FA_OK:
        raise FaError(st, "fa_backward")
    return dq, dk, dv


def check_device_status(stream=None) -> int:
    """Synchronise the stream and return the device status (FA_OK or FA_ERR_TIMEOUT/CUDA)."""
    return int(lib.fa_check_device_status(_stream(stream)))


def set_fault_injection(mode: int) -> None:
    lib.fa_debug_set_fault_injection(int(mode))


def set_wait_limit_ms(ms: int) -> None:
    lib.fa_debug_set_wait_limit_ms(int(ms))


def backward_noalloc(q, k, v, o, lse, do, *, causal: bool = False, scale: Optional[float] = None,
                     block_mask=None, kv_lens=None, dq=None, dk=None, dv=None, stream=None):
    """fa_backward_noalloc: the backward with the library's built-in scratch instead of a
    workspace (for callers that cannot allocate device memory).  Output tensors may be passed
    in so that the call itself allocates nothing."""
    B, H, N, d, Hkv = _check_qkv(q, k, v)
    if Hkv != H:
        raise ValueError("fa_backward_noalloc takes one key/value head per query head")
    scale = 1.0 / d ** 0.5 if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    st = lib.fa_backward_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse),
                                 _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, scale,
                                 int(bool(causal)), _ptr(block_mask), _DTYPES[q.dtype],
                                 _ptr(kv_lens), _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_backward_noalloc")
    return dq, dk, dv


def noalloc_max_workspace() -> int:
    return int(lib.fa_backward_noalloc_max_workspace())


# ---- rotary positions, the paged cache, score modifications ------------------------------------------
#
# These calls are made once per layer and token: their host time is most of a short call, so the
# checks read each property of a tensor once, names for a message are found only when one is
# raised, and the arguments cross as one packed structure (one token over a short cache: 13.7 us a
# call, 18 with an argument each and the workspace's size asked for every time; its write into the
# cache 12.9 and 17.7).

_CACHE_FORMAT = "PPqqqiiPqiP"                                     # fa_paged_cache
_SCORED = struct.Struct("14PNP8iff")                              # fa_scored_call
_ROTARY = struct.Struct("PPPPP7q7if")                             # fa_rotary_call
_APPEND = struct.Struct(_CACHE_FORMAT + "7P9q8if0q")              # fa_append_paged_call
_PAGED = struct.Struct(_CACHE_FORMAT + "6PNP6iff")                # fa_forward_paged_call
_STORE_FORMAT = "iPPPP"                                           # fa_page_store
_APPEND_STORE = struct.Struct(_CACHE_FORMAT + "7P9q8if0q" + _STORE_FORMAT)          # fa_append_paged_store_call
_PAGED_STORE = struct.Struct(_CACHE_FORMAT + "6PNP6iff0q" + _STORE_FORMAT + "Pi0q")  # fa_forward_paged_store_call
_SELECT = struct.Struct(_CACHE_FORMAT + _STORE_FORMAT + "4PNP9i0q")  # fa_select_pages_call
_ASSIGN = struct.Struct("Pq10P5i0q")                              # fa_assign_pages_call
_16_BIT = (torch.bfloat16, torch.float16)
_PLAIN_STORE = (0, 0, 0, 0, 0)                                    # 16-bit pages
_PAGE_FORMATS = {torch.float8_e4m3fn: 1, torch.int8: 2}           # fa_page_format; 0: the queries' type
# of PyTorch's module for CUDA, without the wrappers around them (absent from builds without CUDA)
_device, _raw_stream = (getattr(torch._C, name, None) for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"))


def _refuse_place(**tensors) -> None:
    """The library launches on the current device: says which tensor is not there."""
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.get_device() != torch.cuda.current_device():
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")


def _current_device(t: torch.Tensor) -> int:
    """The current device's index, when t is there; -1 otherwise (tensors elsewhere give -1 too)."""
    dev = t.get_device()
    return dev if dev >= 0 and dev == _device() else -1


def _handle(stream, dev: int, *allocated) -> int:
    """The stream's handle.  Memory allocated here (None: given by the caller) belongs to the current
    stream: for a call on another one, that stream first waits for what the current one still does
    with it, and it is not reused before that stream is done with it."""
    current = _raw_stream(dev)
    if stream is None or stream.cuda_stream == current:
        return current
    mine = [t for t in allocated if t is not None]
    if mine:
        stream.wait_stream(torch.cuda.current_stream(dev))
    for t in mine:
        t.record_stream(stream)
    return stream.cuda_stream


def _int32(name: str, t: torch.Tensor, shape) -> None:
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor")


def _strides(name: str, t: torch.Tensor) -> Tuple[int, int, int]:
    """Strides (batch, head, token) of a [B, heads, N, d] tensor whose last axis adjoins."""
    b, h, n, last = t.stride()
    if last != 1:
        raise ValueError(f"the values of a head must adjoin in {name}")
    return b, h, n


def _rotated(inv_freq: Optional[torch.Tensor]) -> int:
    """The rotated values of a head (0: none)."""
    if inv_freq is None:
        return 0
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 [rotary_dim / 2] tensor")
    return 2 * inv_freq.numel()


def _span(t: torch.Tensor) -> Tuple[int, int]:
    """The bytes a tensor lies in."""
    last = sum((n - 1) * st for n, st in zip(t.shape, t.stride())) if t.numel() else -1
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _apart(a: str, x: torch.Tensor, b: str, y: torch.Tensor, same: bool) -> None:
    """x may be y itself (``same``); otherwise the two must not share memory."""
    if same and x.data_ptr() == y.data_ptr() and x.stride() == y.stride():
        return
    (x0, x1), (y0, y1) = _span(x), _span(y)
    if x0 < y1 and y0 < x1:
        raise ValueError(f"{a} and {b} overlap")


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, *, factor: float = 1.0,
                       method: str = "linear", trained_len: Optional[int] = None,
                       fast: float = 32.0, slow: float = 1.0, device="cuda") -> Tuple[torch.Tensor, float]:
    """inv_freq (float64 [rotary_dim / 2], radians per position) and mscale for ``rotary``:
    base ** (-2 p / rotary_dim), stretched for contexts ``factor`` times longer by one of
      "linear"  every frequency divided by the factor (positions interpolated);
      "ntk"     the base raised by factor ** (rotary_dim / (rotary_dim - 2)): the slowest pair is
                divided by the factor, the fastest kept;
      "ramp"    pairs that turn more than ``fast`` times in ``trained_len`` positions kept, those
                that turn less than ``slow`` times divided by the factor, a linear ramp between,
                and mscale = 0.1 ln(factor) + 1."""
    if rotary_dim <= 0 or rotary_dim % 2 != 0:
        raise ValueError("rotary_dim must be positive and even")
    if not base > 0.0 or not factor >= 1.0:
        raise ValueError("base must be positive and factor at least 1")
    p = torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim
    mscale = 1.0
    if method == "ntk":
        if rotary_dim > 2:
            base = base * factor ** (rotary_dim / (rotary_dim - 2))
        inv = base ** -p
    elif method == "linear":
        inv = base ** -p / factor
    elif method == "ramp":
        if trained_len is None or trained_len <= 0 or not fast > slow:
            raise ValueError("the ramp needs trained_len > 0 and fast > slow")
        inv = base ** -p
        keep = ((trained_len * inv / (2.0 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        inv = inv * keep + inv / factor * (1.0 - keep)
        mscale = 0.1 * math.log(factor) + 1.0
    else:
        raise ValueError(f"unknown method {method!r}")
    return inv.to(device), mscale


def _rotary(fn, where, x, positions, inv_freq, interleaved, mscale, out, stream):
    dev = _current_device(x)
    if dev < 0 or positions.get_device() != dev or inv_freq.get_device() != dev:
        _refuse_place(x=x, positions=positions, inv_freq=inv_freq)
    shape, dtype = x.shape, x.dtype
    if len(shape) == 4:
        B, H, N, d = shape
        x4 = x
    elif len(shape) == 3:
        H, N, d = shape
        B, x4 = 1, x.unsqueeze(0)
    else:
        raise ValueError("x must be [B, H, N, d] or [H, N, d]")
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}")
    xs = _strides("x", x4)
    rot = _rotated(inv_freq)
    per_batch = positions.dim() == 2
    _int32("positions", positions, (B, N) if per_batch else (N,))
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
        ys = (H * N * d, N * d, d)
        s = _handle(stream, dev, out)
    else:
        _refuse_place(out=out)
        if out.shape != shape or out.dtype != dtype:
            raise ValueError("out must have x's shape and type")
        _apart("x", x, "out", out, True)
        ys = _strides("out", out if len(shape) == 4 else out.unsqueeze(0))
        s = _handle(stream, dev)
    st = fn(_ROTARY.pack(x.data_ptr(), out.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(), s, *xs, *ys,
                         N if per_batch else 0, B, H, N, d, rot, 1 if interleaved else 0, code, mscale))
    if st != FA_OK:
        raise FaError(st, where)
    return out


def rotary(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, *, interleaved: bool = False,
           mscale: float = 1.0, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fa_rotary: x with the first 2 * inv_freq.numel() values of every head turned by their
    positions.  x: [B, H, N, d] or packed [H, total, d], any strides whose last axis adjoins (a
    projection's [B, N, H, d] seen as [B, H, N, d], say); positions: int32 [N] or [B, N]; inv_freq:
    float64, from ``rotary_frequencies``; out: a new contiguous tensor, or given (x itself for a
    rotation in place).  bf16, fp16 or fp32."""
    return _rotary(lib.fa_rotary_packed, "fa_rotary", x, positions, inv_freq, interleaved, mscale, out, stream)


def rotary_backward(dy: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, *,
                    interleaved: bool = False, mscale: float = 1.0,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fa_rotary_backward: the gradient of ``rotary``'s input, given that of its output."""
    return _rotary(lib.fa_rotary_backward_packed, "fa_rotary_backward", dy, positions, inv_freq, interleaved,
                   mscale, out, stream)


def _cache(k_cache, v_cache, block_table, kv_lens, B, Hkv, d, dtype) -> tuple:
    """Checks a paged cache ([n_pages, Hkv, page_size, d], any strides) and gives fa_paged_cache's fields."""
    shape, strides = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or shape[1] != Hkv or shape[3] != d or k_cache.dtype != dtype or v_cache.dtype != dtype:
        raise ValueError(f"k_cache and v_cache must be {dtype} [n_pages, {Hkv}, page_size, {d}]")
    if strides[3] != 1:
        raise ValueError("the values of a head must adjoin in k_cache")
    if v_cache.shape != shape or v_cache.stride() != strides:
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    table, row, width, lens = _table(block_table, kv_lens, B)
    return (k_cache.data_ptr(), v_cache.data_ptr(), strides[0], strides[1], strides[2], shape[0], shape[2],
            table, row, width, lens)


def _table(block_table, kv_lens, B) -> Tuple[int, int, int, int]:
    """Checks a block table and the lengths that go with it: its address, row stride and width, theirs."""
    tshape = block_table.shape
    if block_table.dtype != torch.int32 or len(tshape) != 2 or tshape[0] != B:
        raise ValueError(f"block_table must be int32 [{B}, max_pages]")
    row, entry = block_table.stride()
    width = tshape[1]
    if width > 1 and entry != 1:
        raise ValueError("the entries of a row must adjoin in block_table")
    if B <= 1 or width == 0:
        row = width                                   # no other row to step to
    elif row < width:
        raise ValueError("the rows of block_table overlap (one row seen as many, say): they must lie apart")
    if kv_lens.dtype != torch.int32 or kv_lens.shape != (B,) or not kv_lens.is_contiguous():
        raise ValueError(f"kv_lens must be a contiguous int32 [{B}] tensor")
    return block_table.data_ptr(), row, width, kv_lens.data_ptr()


def _scales(name: str, t: Optional[torch.Tensor], dev: int, shape) -> int:
    if t is not None and t.get_device() == dev and t.dtype is torch.float32 and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t is None:
        raise ValueError(f"8-bit pages (and bounds) need {name}")
    _refuse_place(**{name: t})
    raise ValueError(f"{name} must be a contiguous float32 {list(shape)} tensor")


def _bounds(k_bounds, bound_scales, dev: int, n_pages: int, Hkv: int, d: int) -> Tuple[int, int]:
    if k_bounds.get_device() != dev:
        _refuse_place(k_bounds=k_bounds)
    if k_bounds.dtype != torch.int8 or k_bounds.shape != (n_pages, Hkv, 2, d) or not k_bounds.is_contiguous():
        raise ValueError(f"k_bounds must be a contiguous int8 [{n_pages}, {Hkv}, 2, {d}] tensor")
    return k_bounds.data_ptr(), _scales("bound_scales", bound_scales, dev, (n_pages, Hkv))


def _store(k_cache, k_scales, v_scales, k_bounds, bound_scales, dtype, dev: int, Hkv: int, d: int):
    """The type of the pages' elements, and fa_page_store's fields (None: 16-bit pages without bounds)."""
    if k_scales is None and v_scales is None and k_bounds is None and bound_scales is None and k_cache.dtype is dtype:
        return dtype, None
    fmt = _PAGE_FORMATS.get(k_cache.dtype, 0)
    if fmt == 0:
        if k_scales is not None or v_scales is not None:
            raise ValueError("16-bit pages have no scales")
        if k_bounds is None and bound_scales is None:
            return dtype, None
        ks = vs = 0
    else:
        shape = (k_cache.shape[0], Hkv)
        ks, vs = _scales("k_scales", k_scales, dev, shape), _scales("v_scales", v_scales, dev, shape)
        dtype = k_cache.dtype
    kb = bs = 0
    if k_bounds is not None:
        kb, bs = _bounds(k_bounds, bound_scales, dev, k_cache.shape[0], Hkv, d)
    elif bound_scales is not None:
        raise ValueError("bound_scales without k_bounds")
    return dtype, (fmt, ks, vs, kb, bs)


def append_paged(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 block_table: torch.Tensor, kv_lens: torch.Tensor, *, q: Optional[torch.Tensor] = None,
                 q_lens: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None,
                 interleaved: bool = False, mscale: float = 1.0, q_out: Optional[torch.Tensor] = None,
                 k_scales: Optional[torch.Tensor] = None, v_scales: Optional[torch.Tensor] = None,
                 k_bounds: Optional[torch.Tensor] = None, bound_scales: Optional[torch.Tensor] = None,
                 stream=None) -> Optional[torch.Tensor]:
    """fa_append_paged: writes new tokens k, v [B, Hkv, T, d] into the pages, keys rotated when
    inv_freq is given, and returns the rotated queries [B, H, T, d] when q is.  kv_lens (int32 [B])
    counts the new tokens already; q_lens (int32 [B]) says how many of the T are real (default all).
    k_cache, v_cache: [n_pages, Hkv, page_size, d], any strides whose last axis adjoins;
    block_table: int32 [B, max_pages], rows that lie apart.
    The pages are of k's type, or int8 or float8_e4m3fn with k_scales and v_scales (float32 [n_pages, Hkv],
    a power of two for each page and head, written too; what they hold of pages without tokens does not
    matter).  k_bounds (int8 [n_pages, Hkv, 2, d]) and bound_scales (float32 [n_pages, Hkv]): bounds of
    each page's keys, before they go to 8 bits, for ``select_pages``, kept when given (fa_append_paged_store)."""
    dev = _current_device(k)
    if (dev < 0 or v.get_device() != dev or k_cache.get_device() != dev or v_cache.get_device() != dev
            or block_table.get_device() != dev or kv_lens.get_device() != dev
            or (q is not None and q.get_device() != dev) or (q_lens is not None and q_lens.get_device() != dev)
            or (inv_freq is not None and inv_freq.get_device() != dev)):
        _refuse_place(k=k, v=v, k_cache=k_cache, v_cache=v_cache, block_table=block_table, kv_lens=kv_lens,
                      q=q, q_lens=q_lens, inv_freq=inv_freq)
    shape, dtype = k.shape, k.dtype
    if len(shape) != 4 or dtype not in _16_BIT:
        raise ValueError("k must be bf16 or fp16 [B, Hkv, T, d]")
    if v.shape != shape or v.dtype != dtype:
        raise ValueError("v must have k's shape and type")
    B, Hkv, T, d = shape
    pages, store = _store(k_cache, k_scales, v_scales, k_bounds, bound_scales, dtype, dev, Hkv, d)
    cache = _cache(k_cache, v_cache, block_table, kv_lens, B, Hkv, d, pages)
    if store is not None and store[0]:
        size = 4 * cache[5] * Hkv
        if abs(store[1] - store[2]) < size or (store[4] and min(abs(store[1] - store[4]), abs(store[2] - store[4])) < size):
            raise ValueError("the scales overlap")
    rot = _rotated(inv_freq)
    if q_lens is not None:
        _int32("q_lens", q_lens, (B,))
    H, qs = Hkv, (0, 0, 0)
    s = None
    if q is not None:
        qshape = q.shape
        H = qshape[1] if len(qshape) == 4 else 0
        if Hkv == 0 or H == 0 or H % Hkv != 0 or qshape != (B, H, T, d) or q.dtype != dtype:
            raise ValueError("q must be [B, H, T, d] of k's type, the key heads dividing H")
        qs = _strides("q", q)
        if q_out is None:
            q_out = torch.empty(qshape, dtype=dtype, device=q.device)
            s = _handle(stream, dev, q_out)
        else:
            _refuse_place(q_out=q_out)
            if q_out.shape != qshape or q_out.dtype != dtype or not q_out.is_contiguous():
                raise ValueError("q_out must be contiguous, of q's shape and type")
            _apart("q", q, "q_out", q_out, True)
            _apart("k", k, "q_out", q_out, False)
            _apart("v", v, "q_out", q_out, False)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if s is None:
        s = _handle(stream, dev)
    call = (
        *cache, k.data_ptr(), v.data_ptr(), 0 if q is None else q.data_ptr(), 0 if q_out is None else q_out.data_ptr(),
        0 if q_lens is None else q_lens.data_ptr(), 0 if inv_freq is None else inv_freq.data_ptr(), s,
        *_strides("k", k), *_strides("v", v), *qs, B, H, Hkv, T, d, rot, 1 if interleaved else 0, _DTYPES[dtype], mscale)
    if store is None:
        st = lib.fa_append_paged_packed(_APPEND.pack(*call))
    else:
        st = lib.fa_append_paged_store_packed(_APPEND_STORE.pack(*call, *store))
    if st != FA_OK:
        raise FaError(st, "fa_append_paged")
    return q_out


def forward_paged_workspace_size(B: int, H: int, Hkv: int, T: int, d: int, max_keys: int) -> int:
    """max_keys: entries of a block table's row times the page size."""
    return int(lib.fa_forward_paged_workspace_size(B, H, Hkv, T, d, max_keys))


@functools.lru_cache(maxsize=1024)
def _paged_workspace_size(dev, *sizes) -> int:
    """forward_paged_workspace_size, which the device and the sizes determine: one call into the library
    for each of them."""
    return lib.fa_forward_paged_workspace_size(*sizes)


def _check_slopes(alibi_slopes, H) -> None:
    if alibi_slopes.dtype != torch.float32 or alibi_slopes.shape != (H,) or not alibi_slopes.is_contiguous():
        raise ValueError(f"alibi_slopes must be a contiguous float32 [{H}] tensor")


def _score_args(q, k, v, o, lse, do, alibi_slopes, prefix_lens, H, n_seqs) -> Tuple[int, int, int]:
    """Checks the score arguments (slopes fp32 [H], prefix lengths int32 [n_seqs]) and where the
    tensors are; the current device, and the two addresses (0: not given)."""
    dev = _current_device(q)
    if (dev < 0 or k.get_device() != dev or v.get_device() != dev
            or (do is not None and not (o.get_device() == lse.get_device() == do.get_device() == dev))
            or (alibi_slopes is not None and alibi_slopes.get_device() != dev)
            or (prefix_lens is not None and prefix_lens.get_device() != dev)):
        _refuse_place(q=q, k=k, v=v, o=o, lse=lse, do=do, alibi_slopes=alibi_slopes, prefix_lens=prefix_lens)
    slopes = prefix = 0
    if alibi_slopes is not None:
        _check_slopes(alibi_slopes, H)
        slopes = alibi_slopes.data_ptr()
    if prefix_lens is not None:
        _int32("prefix_lens", prefix_lens, (n_seqs,))
        prefix = prefix_lens.data_ptr()
    return dev, slopes, prefix


def _given(name: str, t: torch.Tensor, shape, dtype) -> None:
    """Checks an output that the caller gives."""
    _refuse_place(**{name: t})
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor")


def _workspace_bytes(t: torch.Tensor) -> int:
    """The bytes of a workspace that the caller gives: its elements adjoin, so its size is its memory's."""
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.numel() * t.element_size()


def _kv_lens(kv_lens, B, dev, q):
    """The key lengths where and as the library takes them, and the copy made for that (or None), which
    is memory allocated here like an output."""
    if kv_lens is None:
        return None, None
    if kv_lens.get_device() != dev or kv_lens.dtype != torch.int32 or kv_lens.shape != (B,) or not kv_lens.is_contiguous():
        kv_lens = _masks(None, kv_lens, B, 0, q.device)[1]
        return kv_lens, kv_lens
    return kv_lens, None


@functools.lru_cache(maxsize=1024)
def _backward_workspace_size(B, H, N, d) -> int:
    """backward_workspace_size, which the sizes determine: one call into the library for each of them."""
    return max(lib.fa_backward_workspace_size(B, H, N, d), 256)


def _forward_scored(q, k, v, causal, scale, kv_lens, o, lse, stream, softcap, alibi_slopes, prefix_lens):
    B, H, N, d, Hkv = _check_qkv(q, k, v)
    dev, slopes, prefix = _score_args(q, k, v, None, None, None, alibi_slopes, prefix_lens, H, B)
    dtype = q.dtype
    kv_lens, kv_new = _kv_lens(kv_lens, B, dev, q)
    o_new = lse_new = None
    if o is None:
        o = o_new = torch.empty_like(q)
    else:
        _given("o", o, q.shape, dtype)
    if lse is None:
        lse = lse_new = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    else:
        _given("lse", lse, (B, H, N), torch.float32)
    st = lib.fa_forward_scored_packed(_SCORED.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), 0, 0, 0, 0,
        0 if kv_lens is None else kv_lens.data_ptr(), 0, slopes, prefix, 0, 0, _handle(stream, dev, o_new, lse_new, kv_new),
        B, H, Hkv, N, 0, d, 1 if causal else 0, _DTYPES[dtype], 1.0 / d ** 0.5 if scale is None else scale, softcap))
    if st != FA_OK:
        raise FaError(st, "fa_forward_scored")
    return o, lse


def _backward_scored(q, k, v, o, lse, do, causal, scale, kv_lens, dq, dk, dv, workspace, stream, softcap,
                     alibi_slopes, prefix_lens):
    B, H, N, d, Hkv = _check_qkv(q, k, v)
    dev, slopes, prefix = _score_args(q, k, v, o, lse, do, alibi_slopes, prefix_lens, H, B)
    shape, dtype = q.shape, q.dtype
    if o.shape != shape or o.dtype != dtype or not o.is_contiguous():
        raise ValueError("o must match q")
    if do.shape != shape or do.dtype != dtype or not do.is_contiguous():
        raise ValueError("do must match q")
    if lse.dtype != torch.float32 or lse.shape != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [B, H, N]")
    kv_lens, kv_new = _kv_lens(kv_lens, B, dev, q)
    dq_new = dk_new = dv_new = ws_new = None
    if dq is None:
        dq = dq_new = torch.empty_like(q)
    else:
        _given("dq", dq, shape, dtype)
    if dk is None:
        dk = dk_new = torch.empty_like(k)
    else:
        _given("dk", dk, k.shape, dtype)
    if dv is None:
        dv = dv_new = torch.empty_like(v)
    else:
        _given("dv", dv, k.shape, dtype)
    if workspace is None:
        workspace = ws_new = torch.empty(_backward_workspace_size(B, H, N, d), dtype=torch.uint8, device=q.device)
    else:
        _refuse_place(workspace=workspace)
    st = lib.fa_backward_scored_packed(_SCORED.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), do.data_ptr(), dq.data_ptr(),
        dk.data_ptr(), dv.data_ptr(), 0 if kv_lens is None else kv_lens.data_ptr(), 0, slopes, prefix,
        workspace.data_ptr(), _workspace_bytes(workspace),
        _handle(stream, dev, dq_new, dk_new, dv_new, ws_new, kv_new),
        B, H, Hkv, N, 0, d, 1 if causal else 0, _DTYPES[dtype], 1.0 / d ** 0.5 if scale is None else scale, softcap))
    if st != FA_OK:
        raise FaError(st, "fa_backward_scored")
    return dq, dk, dv


def forward_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                  kv_lens: torch.Tensor, *, scale: Optional[float] = None,
                  q_lens: Optional[torch.Tensor] = None, softcap: float = 0.0,
                  alibi_slopes: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  k_scales: Optional[torch.Tensor] = None, v_scales: Optional[torch.Tensor] = None,
                  pages: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """O, LSE of T new tokens per sequence over a paged cache that holds them (fa_forward_paged).
    q: [B, H, T, d] contiguous, bf16 or fp16; the cache, block_table, kv_lens and q_lens as in
    ``append_paged``.  Token t of a sequence's n new ones sees the keys up to its own place
    kv_lens - n + t; scores capped by softcap * tanh(. / softcap) when softcap > 0 and lowered by
    alibi_slopes[h] (fp32 [H]) times the distance.
    k_scales, v_scales: of int8 or float8_e4m3fn pages.  pages (int32 [B, Hkv, n]): only these pages are seen,
    by their number in the sequence, -1 for none (``select_pages``; fa_forward_paged_store)."""
    dev = _current_device(q)
    if (dev < 0 or k_cache.get_device() != dev or v_cache.get_device() != dev
            or block_table.get_device() != dev or kv_lens.get_device() != dev
            or (q_lens is not None and q_lens.get_device() != dev)
            or (alibi_slopes is not None and alibi_slopes.get_device() != dev)):
        _refuse_place(q=q, k_cache=k_cache, v_cache=v_cache, block_table=block_table, kv_lens=kv_lens, q_lens=q_lens,
                      alibi_slopes=alibi_slopes)
    shape, dtype = q.shape, q.dtype
    if len(shape) != 4 or dtype not in _16_BIT or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 or fp16 [B, H, T, d] tensor")
    B, H, T, d = shape
    Hkv = k_cache.shape[1] if k_cache.dim() == 4 else 0
    if Hkv == 0 or H % Hkv != 0:
        raise ValueError("k_cache must be [n_pages, Hkv, page_size, d] with Hkv dividing the query heads")
    page_type, store = _store(k_cache, k_scales, v_scales, None, None, dtype, dev, Hkv, d)
    cache = _cache(k_cache, v_cache, block_table, kv_lens, B, Hkv, d, page_type)
    span = cache[6] * cache[9]
    picks = 0
    if pages is not None:
        if pages.get_device() != dev:
            _refuse_place(pages=pages)
        picks = pages.shape[2] if pages.dim() == 3 else 0
        if picks == 0 or pages.shape != (B, Hkv, picks) or pages.dtype != torch.int32 or not pages.is_contiguous():
            raise ValueError(f"pages must be a contiguous int32 [{B}, {Hkv}, n] tensor, n > 0")
        span = min(span, cache[6] * picks)
    if q_lens is not None:
        _int32("q_lens", q_lens, (B,))
    if alibi_slopes is not None:
        _check_slopes(alibi_slopes, H)
    if o is None:
        o = o_new = torch.empty_like(q)
    else:
        o_new = None
        _refuse_place(o=o)
        if o.shape != shape or o.dtype != dtype or not o.is_contiguous():
            raise ValueError("o must be contiguous, of q's shape and type")
        _apart("q", q, "o", o, False)
    if lse is None:
        lse = lse_new = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    else:
        lse_new = None
        _refuse_place(lse=lse)
        if lse.shape != (B, H, T) or lse.dtype != torch.float32 or not lse.is_contiguous():
            raise ValueError("lse must be contiguous float32 [B, H, T]")
    ws_new = None
    if workspace is None:
        need = _paged_workspace_size(dev, B, H, Hkv, T, d, min(span, 0x7fffffff))
        if need > 0:
            workspace = ws_new = torch.empty((need,), dtype=torch.uint8, device=q.device)
    else:
        _refuse_place(workspace=workspace)
    call = (
        *cache, q.data_ptr(), o.data_ptr(), lse.data_ptr(), 0 if q_lens is None else q_lens.data_ptr(),
        0 if alibi_slopes is None else alibi_slopes.data_ptr(), 0 if workspace is None else workspace.data_ptr(),
        0 if workspace is None else _workspace_bytes(workspace), _handle(stream, dev, o_new, lse_new, ws_new),
        B, H, Hkv, T, d, _DTYPES[dtype], 1.0 / d ** 0.5 if scale is None else scale, softcap)
    if store is None and pages is None:
        st = lib.fa_forward_paged_packed(_PAGED.pack(*call))
    else:
        st = lib.fa_forward_paged_store_packed(_PAGED_STORE.pack(*call, *(_PLAIN_STORE if store is None else store),
                                                                 0 if pages is None else pages.data_ptr(), picks))
    if st != FA_OK:
        raise FaError(st, "fa_forward_paged")
    return o, lse


def select_pages_workspace_size(B: int, Hkv: int, max_pages: int, n_select: int) -> int:
    """max_pages: entries of a block table's row."""
    return int(lib.fa_select_pages_workspace_size(B, Hkv, max_pages, n_select))


@functools.lru_cache(maxsize=1024)
def _select_workspace_size(dev, *sizes) -> int:
    """select_pages_workspace_size, which the device and the sizes determine."""
    return lib.fa_select_pages_workspace_size(*sizes)


def select_pages(q: torch.Tensor, k_bounds: torch.Tensor, bound_scales: torch.Tensor, block_table: torch.Tensor,
                 kv_lens: torch.Tensor, n_select: int, page_size: int, *, q_lens: Optional[torch.Tensor] = None,
                 first: int = 1, last: int = 1, pages: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fa_select_pages: for each sequence and key head the n_select pages whose key bounds promise the
    highest scores to its new tokens q [B, H, T, d] (contiguous, bf16 or fp16; rotated like the keys),
    the first and the last ones among them: int32 [B, Hkv, n_select], ascending, -1 behind.  (For this q goes to
    whole numbers of 8 bits, row by row.)  k_bounds and bound_scales as ``append_paged`` keeps them; block_table, kv_lens and q_lens as there."""
    dev = _current_device(q)
    if (dev < 0 or block_table.get_device() != dev or kv_lens.get_device() != dev
            or (q_lens is not None and q_lens.get_device() != dev)):
        _refuse_place(q=q, block_table=block_table, kv_lens=kv_lens, q_lens=q_lens)
    shape, dtype = q.shape, q.dtype
    if len(shape) != 4 or dtype not in _16_BIT or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 or fp16 [B, H, T, d] tensor")
    B, H, T, d = shape
    n_pages, Hkv = k_bounds.shape[:2] if k_bounds.dim() == 4 else (0, 0)
    if Hkv == 0 or H % Hkv != 0:
        raise ValueError("k_bounds must be [n_pages, Hkv, 2, d] with Hkv dividing the query heads")
    kb, bs = _bounds(k_bounds, bound_scales, dev, n_pages, Hkv, d)
    table, row, width, lens = _table(block_table, kv_lens, B)
    if q_lens is not None:
        _int32("q_lens", q_lens, (B,))
    if n_select <= 0:
        raise ValueError("n_select must be positive")
    pages_new = ws_new = None
    if pages is None:
        pages = pages_new = torch.empty((B, Hkv, n_select), dtype=torch.int32, device=q.device)
    else:
        _given("pages", pages, (B, Hkv, n_select), torch.int32)
    if workspace is None:
        need = _select_workspace_size(dev, B, Hkv, width, n_select)
        if need > 0:
            workspace = ws_new = torch.empty((need,), dtype=torch.uint8, device=q.device)
    else:
        _refuse_place(workspace=workspace)
    st = lib.fa_select_pages_packed(_SELECT.pack(
        0, 0, 0, 0, 0, n_pages, page_size, table, row, width, lens, 0, 0, 0, kb, bs, q.data_ptr(), pages.data_ptr(),
        0 if q_lens is None else q_lens.data_ptr(), 0 if workspace is None else workspace.data_ptr(),
        0 if workspace is None else _workspace_bytes(workspace), _handle(stream, dev, pages_new, ws_new),
        B, H, Hkv, T, d, n_select, first, last, _DTYPES[dtype]))
    if st != FA_OK:
        raise FaError(st, "fa_select_pages")
    return pages


def _check_assigned(given, B, max_new, **read) -> None:
    """Outputs of ``assign_pages`` that the caller gives: they lie apart from one another and from what is read,
    but for lens and state, which may be their inputs."""
    for i, (name, t) in enumerate(given):
        shape = (B, max_new) if name in ("slots", "positions") else (2,) if name == "state" else (B,)
        _given(name, t, shape, torch.int64 if name == "slots" else torch.int32)
        for other, x in given[:i]:
            _apart(name, t, other, x, False)
        for other, x in read.items():
            _apart(name, t, other, x, (name, other) in (("lens", "old_lens"), ("lens", "new_lens"), ("state", "free_state")))


def assign_pages(block_table: torch.Tensor, old_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
                 free_state: torch.Tensor, page_size: int, max_new: int = 0, *, lens: Optional[torch.Tensor] = None,
                 q_lens: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                 positions: Optional[torch.Tensor] = None, state: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """fa_assign_pages: takes the sequences from old_lens to new_lens tokens (int32 [B]); pages they need come
    from free_pages (int32, a ring with a place for every page; free_state int32 [2]: its first entry and
    their number) into block_table [B, max_pages], pages they no longer need go back.  Returns
    (lens, q_lens, slots, positions, state): the lengths now and the new tokens of each sequence (``kv_lens`` and
    ``q_lens`` of the paged calls), slots (int64) and positions (int32) [B, max_new] of the first max_new of
    them, -1 where there is none, and the ring's state.  All may be given; lens may be old_lens or new_lens,
    and state free_state.  When the free pages do not suffice nothing changes (lens are old_lens then) and
    ``check_device_status`` tells."""
    dev = _current_device(old_lens)
    if (dev < 0 or block_table.get_device() != dev or new_lens.get_device() != dev or free_pages.get_device() != dev
            or free_state.get_device() != dev):
        _refuse_place(block_table=block_table, old_lens=old_lens, new_lens=new_lens, free_pages=free_pages,
                      free_state=free_state)
    B = old_lens.shape[0] if old_lens.dim() == 1 else -1
    table, row, width, old = _table(block_table, old_lens, B)
    _int32("new_lens", new_lens, (B,))
    _int32("free_state", free_state, (2,))
    n_free = free_pages.numel()
    _int32("free_pages", free_pages, (n_free,))
    if max_new < 0:
        raise ValueError("max_new must not be negative")
    given = [(n, t) for n, t in (("lens", lens), ("q_lens", q_lens), ("slots", slots), ("positions", positions), ("state", state))
             if t is not None]
    if given:
        _check_assigned(given, B, max_new, block_table=block_table, free_pages=free_pages, old_lens=old_lens, new_lens=new_lens,
                        free_state=free_state)
    mine = []
    if slots is None:
        slots = torch.empty((B, max_new), dtype=torch.int64, device=old_lens.device)
        mine.append(slots)
    if positions is None:
        positions = torch.empty((B, max_new), dtype=torch.int32, device=old_lens.device)
        mine.append(positions)
    if lens is None:
        lens = torch.empty_like(old_lens)
        mine.append(lens)
    if q_lens is None:
        q_lens = torch.empty_like(old_lens)
        mine.append(q_lens)
    if state is None:
        state = torch.empty_like(free_state)
        mine.append(state)
    st = lib.fa_assign_pages_packed(_ASSIGN.pack(
        table, row, old, new_lens.data_ptr(), free_pages.data_ptr(), free_state.data_ptr(), state.data_ptr(), lens.data_ptr(),
        q_lens.data_ptr(), slots.data_ptr(), positions.data_ptr(), _handle(stream, dev, *mine), B, width, page_size, n_free,
        max_new))
    if st != FA_OK:
        raise FaError(st, "fa_assign_pages")
    return lens, q_lens, slots, positions, state
