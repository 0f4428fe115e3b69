"""ctypes binding of libfa_fwd.so (see include/fa_fwd.h for the contract)."""
from __future__ import annotations

import ctypes
import math
import operator
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(PKG, "libfa_fwd.so")

FA_MASK_NONE = 0
FA_MASK_CAUSAL = 1
FA_MASK_CAUSAL_DIAG_BLOCK = 2
FA_DTYPE_FP16 = 0x100
FA_V_FROM_K = 0x200
FA_V_FP16 = 0x400
FA_FP8_E4M3 = 0
FA_FP8_E5M2 = 1

FA_OK = 0
FA_ERR_NULL = -1
FA_ERR_SHAPE = -2
FA_ERR_UNSUPPORTED = -3
FA_ERR_ALIGN = -4
FA_ERR_THRESHOLD = -5
FA_ERR_CUDA = -6
FA_ERR_DEVICE_TIMEOUT = -7
FA_ERR_RANGE = -8
FA_ERR_SCRATCH = -9
FA_ERR_INDEX = -10


class FaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"fa_fwd error {code}: {msg}")
        self.code = code


class fa_block_sparse_t(ctypes.Structure):
    _fields_ = [("idx", ctypes.c_void_p), ("max_sel", ctypes.c_int32), ("block", ctypes.c_int32),
                ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64)]


class fa_topk_t(ctypes.Structure):
    _fields_ = [("idx", ctypes.c_void_p), ("topk", ctypes.c_int32), ("stride_b", ctypes.c_int64)]


class fa_extras_t(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("pre_tokens", ctypes.c_int32),
                ("next_tokens", ctypes.c_int32), ("alibi", ctypes.c_int32),
                ("atten_mask", ctypes.c_void_p), ("mask_stride_b", ctypes.c_int64),
                ("mask_stride_h", ctypes.c_int64), ("mask_stride_q", ctypes.c_int64),
                ("pse", ctypes.c_void_p), ("pse_stride_b", ctypes.c_int64),
                ("pse_stride_h", ctypes.c_int64), ("pse_stride_q", ctypes.c_int64),
                ("pse_type", ctypes.c_int32), ("keep_prob", ctypes.c_float),
                ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64)]


class fa_paged_kv_t(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_stride_page", ctypes.c_int64), ("k_stride_head", ctypes.c_int64),
                ("k_stride_slot", ctypes.c_int64), ("v_stride_page", ctypes.c_int64),
                ("v_stride_head", ctypes.c_int64), ("v_stride_slot", ctypes.c_int64),
                ("k_min", ctypes.c_void_p), ("k_max", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("max_pages", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class fa_kv_new_t(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q", ctypes.c_void_p),
                ("q_out", ctypes.c_void_p),
                ("k_stride_b", ctypes.c_int64), ("k_stride_h", ctypes.c_int64),
                ("k_stride_s", ctypes.c_int64), ("v_stride_b", ctypes.c_int64),
                ("v_stride_h", ctypes.c_int64), ("v_stride_s", ctypes.c_int64),
                ("q_stride_b", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
                ("q_stride_s", ctypes.c_int64), ("qo_stride_b", ctypes.c_int64),
                ("qo_stride_h", ctypes.c_int64), ("qo_stride_s", ctypes.c_int64),
                ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("max_pos", ctypes.c_int32)]


_lib = None


def library_path() -> str:
    return _LIB_PATH


def library() -> ctypes.CDLL:
    """Load libfa_fwd.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise OSError(f"{_LIB_PATH} is missing: build it with "
                          "`python -m attention_forward_fa_gb300.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        lib.fa_fwd.restype = ctypes.c_int
        lib.fa_fwd.argtypes = [ctypes.c_void_p] * 4 + [ctypes.c_void_p] + [ctypes.c_int] * 7 + [
            ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(fa_block_sparse_t),
            ctypes.POINTER(fa_topk_t), ctypes.c_float, ctypes.c_void_p]
        lib.fa_fwd_noalloc.restype = ctypes.c_int
        lib.fa_fwd_noalloc.argtypes = lib.fa_fwd.argtypes
        lib.fa_fwd_fp8.restype = ctypes.c_int
        lib.fa_fwd_fp8.argtypes = [ctypes.c_void_p] * 6 + [ctypes.c_int, ctypes.c_void_p,
                                                           ctypes.c_void_p] + [ctypes.c_int] * 7 + [
            ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(fa_extras_t),
            ctypes.c_float, ctypes.c_void_p]
        lib.fa_fwd_ext.restype = ctypes.c_int
        lib.fa_fwd_ext.argtypes = [ctypes.c_void_p] * 4 + [ctypes.c_void_p] + [ctypes.c_int] * 7 + [
            ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(fa_extras_t),
            ctypes.c_float, ctypes.c_void_p]
        lib.fa_fwd_o_lo.restype = ctypes.c_int
        lib.fa_fwd_o_lo.argtypes = lib.fa_fwd.argtypes[:4] + [ctypes.c_void_p] + lib.fa_fwd.argtypes[4:]
        lib.fa_bwd.restype = ctypes.c_int
        lib.fa_bwd.argtypes = [ctypes.c_void_p] * 10 + [ctypes.c_int] * 7 + [
            ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
        lib.fa_convert_v_fp16.restype = ctypes.c_int
        lib.fa_convert_v_fp16.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                          ctypes.c_void_p]
        lib.fa_kv_append.restype = ctypes.c_int
        lib.fa_kv_append.argtypes = [ctypes.POINTER(fa_paged_kv_t), ctypes.POINTER(fa_kv_new_t)] + [
            ctypes.c_int] * 6 + [ctypes.c_void_p] * 3
        lib.fa_decode.restype = ctypes.c_int
        lib.fa_decode.argtypes = [ctypes.c_void_p, ctypes.POINTER(fa_paged_kv_t), ctypes.c_void_p,
                                  ctypes.c_void_p] + [ctypes.c_int] * 5 + [
            ctypes.c_float, ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
            ctypes.c_int, ctypes.c_void_p]
        lib.fa_select_pages.restype = ctypes.c_int
        lib.fa_select_pages.argtypes = [ctypes.c_void_p, ctypes.POINTER(fa_paged_kv_t),
                                        ctypes.c_void_p] + [ctypes.c_int] * 6 + [
            ctypes.c_void_p] + [ctypes.c_int] * 3 + [ctypes.c_void_p]
        lib.fa_check_status.restype = ctypes.c_int
        lib.fa_check_status.argtypes = [ctypes.c_void_p]
        lib.fa_set_wait_timeout_ns.restype = None
        lib.fa_set_wait_timeout_ns.argtypes = [ctypes.c_int64]
        lib.fa_set_max_kv_split.restype = ctypes.c_int
        lib.fa_set_max_kv_split.argtypes = [ctypes.c_int]
        lib.fa_wait_probe.restype = ctypes.c_int
        lib.fa_wait_probe.argtypes = [ctypes.c_void_p]
        lib.fa_strerror.restype = ctypes.c_char_p
        lib.fa_strerror.argtypes = [ctypes.c_int]
        lib.fa_last_cuda_error.restype = ctypes.c_int
        lib.fa_last_cuda_error_string.restype = ctypes.c_char_p
        _lib = lib
    return _lib


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def fa_strerror(code: int) -> str:
    return library().fa_strerror(code).decode()


def fa_fwd(q, k, v, o, lse, B: int, Hq: int, Hkv: int, Sq: int, Skv: int, D: int, Dv: int,
           scale: float, mask_mode: int, seqlens=None, kv_block_idx=None, topk_idx=None,
           rescale_threshold: float = 0.0, stream=None) -> int:
    """Direct call of the C entry point.  Tensors (or raw device pointers) for
    q, k, v, o, lse, seqlens; kv_block_idx = (idx, max_sel, block, stride_b,
    stride_h) and topk_idx = (idx, topk, stride_b) with device index arrays.
    Returns the FA_* code."""
    lib = library()
    bs = None
    if kv_block_idx is not None:
        idx, max_sel, block, sb, sh = kv_block_idx
        bs = ctypes.pointer(fa_block_sparse_t(_ptr(idx), max_sel, block, sb, sh))
    tk = None
    if topk_idx is not None:
        idx, topk, sb = topk_idx
        tk = ctypes.pointer(fa_topk_t(_ptr(idx), topk, sb))
    return lib.fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Sq, Skv, D, Dv,
                      float(scale), int(mask_mode), _ptr(seqlens), bs, tk,
                      float(rescale_threshold), _stream(stream))


def fa_fwd_o_lo(q, k, v, o, o_lo, lse, B: int, Hq: int, Hkv: int, Sq: int, Skv: int, D: int,
                Dv: int, scale: float, mask_mode: int, seqlens=None, kv_block_idx=None,
                topk_idx=None, rescale_threshold: float = 0.0, stream=None) -> int:
    """fa_fwd that also writes o_lo = fp32(O) - O rounded to o's type (same
    type and layout as o).  Same arguments as fa_fwd plus o_lo after o."""
    lib = library()
    bs = None
    if kv_block_idx is not None:
        idx, max_sel, block, sb, sh = kv_block_idx
        bs = ctypes.pointer(fa_block_sparse_t(_ptr(idx), max_sel, block, sb, sh))
    tk = None
    if topk_idx is not None:
        idx, topk, sb = topk_idx
        tk = ctypes.pointer(fa_topk_t(_ptr(idx), topk, sb))
    return lib.fa_fwd_o_lo(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(o_lo), _ptr(lse), B, Hq, Hkv,
                           Sq, Skv, D, Dv, float(scale), int(mask_mode), _ptr(seqlens), bs, tk,
                           float(rescale_threshold), _stream(stream))


def fa_bwd(q, k, v, o, o_lo, lse, dout, dq, dk, dv, B: int, Hq: int, Hkv: int, Sq: int, Skv: int,
           D: int, Dv: int, scale: float, mask_mode: int, seqlens=None, stream=None) -> int:
    """Direct call of the backward entry point (see include/fa_fwd.h); o_lo
    may be None.  Returns the FA_* code."""
    return library().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(o_lo), _ptr(lse), _ptr(dout),
                            _ptr(dq), _ptr(dk), _ptr(dv), B, Hq, Hkv, Sq, Skv, D, Dv, float(scale),
                            int(mask_mode), _ptr(seqlens), _stream(stream))


def fa_fwd_ext(q, k, v, o, lse, B: int, Hq: int, Hkv: int, Sq: int, Skv: int, D: int, Dv: int,
               scale: float, mask_mode: int, seqlens, extras, rescale_threshold: float = 0.0,
               stream=None) -> int:
    """Direct call of fa_fwd_ext (see include/fa_fwd.h).  extras: an
    fa_extras_t (or None, which the library rejects).  Returns the FA_* code."""
    return library().fa_fwd_ext(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Sq, Skv,
                                D, Dv, float(scale), int(mask_mode), _ptr(seqlens),
                                ctypes.byref(extras) if extras is not None else None,
                                float(rescale_threshold), _stream(stream))


def fa_fwd_fp8(q8, k8, v8, d_scale_q, d_scale_k, d_scale_v, fp8_format: int, o, lse, B: int,
               Hq: int, Hkv: int, Sq: int, Skv: int, D: int, Dv: int, scale: float,
               mask_mode: int, seqlens=None, extras=None, rescale_threshold: float = 0.0,
               stream=None) -> int:
    """Direct call of fa_fwd_fp8 (see include/fa_fwd.h).  Returns the FA_* code."""
    return library().fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(d_scale_q), _ptr(d_scale_k),
                                _ptr(d_scale_v), int(fp8_format), _ptr(o), _ptr(lse), B, Hq, Hkv,
                                Sq, Skv, D, Dv, float(scale), int(mask_mode), _ptr(seqlens),
                                ctypes.byref(extras) if extras is not None else None,
                                float(rescale_threshold), _stream(stream))


def flash_attention_forward_fp8(q8, k8, v8, d_scale_q, d_scale_k, d_scale_v, *, fp8_format="e4m3",
                                scale: Optional[float] = None, causal: bool = False, seqlens=None,
                                rescale_threshold: float = 0.0, stream=None):
    """Allocating wrapper over fa_fwd_fp8: q8 / k8 / v8 CUDA tensors of fp8 bytes
    (torch float8_e4m3fn / float8_e5m2 or uint8) [B, H, S, D], d_scale_* fp32
    [B, H, ceil(S / 128)].  Returns (o fp16, lse)."""
    import torch
    B, Hq, Sq, D = q8.shape
    _, Hkv, Skv, _ = k8.shape
    Dv = v8.shape[-1]
    for t in (q8, k8, v8, d_scale_q, d_scale_k, d_scale_v):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("FP8 inputs and scales must be contiguous CUDA tensors")
    fmt = {"e4m3": FA_FP8_E4M3, "e5m2": FA_FP8_E5M2}[fp8_format]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    out = torch.empty((B, Hq, Sq, Dv), dtype=torch.float16, device=q8.device)
    lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q8.device)
    _raise(fa_fwd_fp8(q8, k8, v8, d_scale_q, d_scale_k, d_scale_v, fmt, out, lse, B, Hq, Hkv, Sq,
                      Skv, D, Dv, scale, FA_MASK_CAUSAL if causal else FA_MASK_NONE, seqlens, None,
                      rescale_threshold, stream))
    return out, lse


def fa_fwd_noalloc(q, k, v, o, lse, B: int, Hq: int, Hkv: int, Sq: int, Skv: int, D: int,
                   Dv: int, scale: float, mask_mode: int, seqlens=None, kv_block_idx=None,
                   topk_idx=None, rescale_threshold: float = 0.0, stream=None) -> int:
    """fa_fwd without any memory allocation (fixed 32 MiB scratch inside the
    library; bf16 V larger than that is rejected with FA_ERR_SCRATCH).  Same
    arguments as fa_fwd.  Calls that overlap on the GPU race on the scratch."""
    lib = library()
    bs = None
    if kv_block_idx is not None:
        idx, max_sel, block, sb, sh = kv_block_idx
        bs = ctypes.pointer(fa_block_sparse_t(_ptr(idx), max_sel, block, sb, sh))
    tk = None
    if topk_idx is not None:
        idx, topk, sb = topk_idx
        tk = ctypes.pointer(fa_topk_t(_ptr(idx), topk, sb))
    return lib.fa_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Sq, Skv,
                              D, Dv, float(scale), int(mask_mode), _ptr(seqlens), bs, tk,
                              float(rescale_threshold), _stream(stream))


def fa_convert_v_fp16(v_bf16, v_fp16, n_elems: int, stream=None) -> int:
    """fp16 copy of a bf16 V (see include/fa_fwd.h); returns the FA_* code."""
    return library().fa_convert_v_fp16(_ptr(v_bf16), _ptr(v_fp16), int(n_elems), _stream(stream))


def fa_check_status(stream=None) -> int:
    return library().fa_check_status(_stream(stream))


def fa_set_wait_timeout_ns(ns: int) -> None:
    library().fa_set_wait_timeout_ns(int(ns))


def fa_set_max_kv_split(n: int) -> int:
    """Most KV pieces per unit for under-filled dense problems (1 = never split)."""
    return library().fa_set_max_kv_split(int(n))


def fa_wait_probe(stream=None) -> int:
    return library().fa_wait_probe(_stream(stream))


def _raise(code: int):
    if code != FA_OK:
        lib = library()
        msg = lib.fa_strerror(code).decode()
        if code == -6:
            msg += f" ({lib.fa_last_cuda_error_string().decode()})"
        raise FaError(code, msg)


def flash_attention_forward(q, k, v=None, *, scale: Optional[float] = None, causal: bool = False,
                            mask_mode: Optional[int] = None, seqlens=None, block_idx=None,
                            topk_idx=None, rescale_threshold: float = 0.0, out=None, lse=None,
                            o_lo=None, window=None, bottom_right_causal: bool = False,
                            atten_mask=None, alibi: bool = False, pse=None, pse_type: int = 0,
                            dropout=None, stream=None):
    """Allocating convenience wrapper over fa_fwd.

    q [B,Hq,Sq,D], k [B,Hkv,Skv,D], v [B,Hkv,Skv,Dv] (or None with top-k and a
    shared latent), bf16 or fp16 CUDA tensors.  block_idx: int32 tensor
    [B, Hq or 1, ceil(Sq/128), max_sel]; topk_idx: int32 [B, Sq, W].
    o_lo: True (allocate) or a tensor like out to also receive the output's
    rounding residual (fa_fwd_o_lo).  Returns (o, lse), or (o, lse, o_lo).

    The operator's optional terms go through fa_fwd_ext: window=(pre_tokens,
    next_tokens) (sparse_mode 0), bottom_right_causal (sparse_mode 3),
    atten_mask (bool or uint8 CUDA tensor [..., Sq, Skv] broadcastable to
    [B, Hq, Sq, Skv], True / nonzero = masked; its last dimension contiguous),
    alibi (True or 2: pse_type 2, -slope |i - j|; 3: pse_type 3, -slope
    sqrt|i - j|), pse (a bias tensor of q's type [..., Sq, Skv]
    broadcastable like atten_mask, last dim contiguous) with pse_type 0
    (added after the scale) or 1 (before), dropout=(keep_prob, seed, offset)
    (the Philox mask of include/fa_fwd.h)."""
    import torch
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("q, k, v must be bf16 or fp16")
    for t in (q, k, v):
        if t is not None and (not t.is_cuda or not t.is_contiguous() or t.dtype != q.dtype):
            raise ValueError("q, k, v must be contiguous CUDA tensors of one dtype")
    B, Hq, Sq, D = q.shape
    _, Hkv, Skv, _ = k.shape
    v_from_k = v is None
    Dv = v.shape[-1] if v is not None else 512
    if mask_mode is None:
        mask_mode = FA_MASK_CAUSAL if causal else FA_MASK_NONE
    if q.dtype == torch.float16:
        mask_mode |= FA_DTYPE_FP16
    if v_from_k:
        mask_mode |= FA_V_FROM_K
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty((B, Hq, Sq, Dv), dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    bs = None
    if block_idx is not None:
        assert block_idx.dtype == torch.int32 and block_idx.is_contiguous()
        nb, hh, nqb, ms = block_idx.shape
        bs = (block_idx, ms, 128, hh * nqb * ms, nqb * ms if hh > 1 else 0)
    tk = None
    if topk_idx is not None:
        assert topk_idx.dtype == torch.int32 and topk_idx.is_contiguous()
        tk = (topk_idx, topk_idx.shape[-1], topk_idx.shape[-2] * topk_idx.shape[-1])
    if seqlens is not None:
        assert seqlens.dtype == torch.int32 and seqlens.is_cuda
    if (window is not None or bottom_right_causal or atten_mask is not None or alibi
            or pse is not None or dropout is not None):
        if o_lo not in (None, False) or bs is not None or tk is not None:
            raise ValueError("the optional terms apply to dense problems without o_lo")
        ex = fa_extras_t()
        ex.window = 1 if window is not None else (2 if bottom_right_causal else 0)
        if window is not None and bottom_right_causal:
            raise ValueError("window and bottom_right_causal are exclusive")
        ex.pre_tokens, ex.next_tokens = (int(window[0]), int(window[1])) if window is not None else (0, 0)
        ex.alibi = {False: 0, True: 1, 2: 1, 3: 2}[alibi]   # True = pse_type 2
        if dropout is not None:
            ex.keep_prob, ex.seed, ex.offset = float(dropout[0]), int(dropout[1]), int(dropout[2])
        keep = None
        if atten_mask is not None:
            m = atten_mask
            if m.dtype == torch.bool:
                m = m.view(torch.uint8)
            if m.dtype != torch.uint8 or not m.is_cuda or m.stride(-1) != 1:
                raise ValueError("atten_mask must be a bool / uint8 CUDA tensor with a contiguous last dim")
            while m.dim() < 4:
                m = m.unsqueeze(0)
            def st(d):
                return 0 if m.shape[d] == 1 else m.stride(d)
            ex.atten_mask = m.data_ptr()
            ex.mask_stride_b, ex.mask_stride_h, ex.mask_stride_q = st(0), st(1), st(2)
            keep = m
        keep_pse = None
        if pse is not None:
            b_ = pse
            if b_.dtype != q.dtype or not b_.is_cuda or b_.stride(-1) != 1:
                raise ValueError("pse must be a CUDA tensor of q's dtype with a contiguous last dim")
            while b_.dim() < 4:
                b_ = b_.unsqueeze(0)
            def stp(d):
                return 0 if b_.shape[d] == 1 else b_.stride(d)
            ex.pse = b_.data_ptr()
            ex.pse_stride_b, ex.pse_stride_h, ex.pse_stride_q = stp(0), stp(1), stp(2)
            ex.pse_type = int(pse_type)
            keep_pse = b_
        code = fa_fwd_ext(q, k, v, out, lse, B, Hq, Hkv, Sq, Skv, D, Dv, scale, mask_mode, seqlens,
                          ex, rescale_threshold, stream)
        del keep, keep_pse
        _raise(code)
        return out, lse
    if o_lo is None or o_lo is False:
        code = fa_fwd(q, k, v, out, lse, B, Hq, Hkv, Sq, Skv, D, Dv, scale, mask_mode, seqlens, bs,
                      tk, rescale_threshold, stream)
        _raise(code)
        return out, lse
    if o_lo is True:
        o_lo = torch.empty_like(out)
    code = fa_fwd_o_lo(q, k, v, out, o_lo, lse, B, Hq, Hkv, Sq, Skv, D, Dv, scale, mask_mode,
                       seqlens, bs, tk, rescale_threshold, stream)
    _raise(code)
    return out, lse, o_lo


def flash_attention_backward(q, k, v, o, lse, dout, *, o_lo=None, scale: Optional[float] = None,
                             causal: bool = False, seqlens=None, dq=None, dk=None, dv=None,
                             stream=None):
    """Allocating wrapper over fa_bwd: q, o, dout [B,Hq,Sq,D], k, v
    [B,Hkv,Skv,D] (D = 64 or 128; bf16 or fp16 CUDA tensors, contiguous), lse [B,Hq,Sq]
    fp32 from the forward, o_lo its residual (recommended).  Returns
    (dq, dk, dv) in the inputs' type."""
    import torch
    for t in (q, k, v, o, dout) + ((o_lo,) if o_lo is not None else ()):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != q.dtype:
            raise ValueError("q, k, v, o, dout (and o_lo) must be contiguous CUDA tensors of one dtype")
    B, Hq, Sq, D = q.shape
    _, Hkv, Skv, _ = k.shape
    Dv = v.shape[-1]
    mask_mode = FA_MASK_CAUSAL if causal else FA_MASK_NONE
    if q.dtype == torch.float16:
        mask_mode |= FA_DTYPE_FP16
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _raise(fa_bwd(q, k, v, o, o_lo, lse, dout, dq, dk, dv, B, Hq, Hkv, Sq, Skv, D, Dv, scale,
                  mask_mode, seqlens, stream))
    return dq, dk, dv


# ------------------------------------------------------------------ paged key-value cache
def _int(x) -> int:
    """x as the library's 32-bit ints hold it: what does not fit is the nearest that does (ctypes would
    take its lowest 32 bits: a window of 2**32 tokens would become one of none)."""
    x = operator.index(x)
    return -2**31 if x < -2**31 else 2**31 - 1 if x > 2**31 - 1 else x


def fa_kv_append(kv: fa_paged_kv_t, x: fa_kv_new_t, B: int, Hq: int, Hkv: int, Snew: int, D: int,
                 mask_mode: int, kv_lens, new_lens=None, stream=None) -> int:
    """Direct call of the C entry point (see include/fa_fwd.h).  Returns the FA_* code."""
    return library().fa_kv_append(kv, x, *map(_int, (B, Hq, Hkv, Snew, D, int(mask_mode))), _ptr(kv_lens),
                                  _ptr(new_lens), _stream(stream))


def fa_decode(q, kv: fa_paged_kv_t, o, lse, B: int, Hq: int, Hkv: int, Sq: int, D: int,
              scale: float, mask_mode: int, kv_lens, pre_tokens: int = -1, page_idx=None,
              max_sel: int = 0, stream=None) -> int:
    """Direct call of the C entry point (see include/fa_fwd.h).  Returns the FA_* code."""
    return library().fa_decode(_ptr(q), kv, _ptr(o), _ptr(lse), *map(_int, (B, Hq, Hkv, Sq, D)), float(scale),
                               _int(int(mask_mode)), _ptr(kv_lens), _int(int(pre_tokens)), _ptr(page_idx),
                               _int(int(max_sel)), _stream(stream))


def fa_select_pages(q, kv: fa_paged_kv_t, page_idx, B: int, Hq: int, Hkv: int, Sq: int, D: int,
                    mask_mode: int, kv_lens, max_sel: int, first: int = 1, last: int = 1,
                    stream=None) -> int:
    """Direct call of the C entry point (see include/fa_fwd.h).  Returns the FA_* code."""
    return library().fa_select_pages(_ptr(q), kv, _ptr(page_idx),
                                     *map(_int, (B, Hq, Hkv, Sq, D, int(mask_mode))), _ptr(kv_lens),
                                     *map(_int, map(int, (max_sel, first, last))), _stream(stream))


class PagedKV:
    """A paged key-value cache: what the paged calls need to know of it.

    k_pages, v_pages: bf16 or fp16 CUDA tensors [num_pages, Hkv, page_size, D], any strides with a
    contiguous last dimension (a [num_pages, page_size, Hkv, D] pool enters as
    ``pool.transpose(1, 2)``); page_size 16, 32, 64, 128 or 256; D 64 or 128.
    page_table: int32 [B, max_pages], column p the page of sequence b's tokens
    [p * page_size, (p + 1) * page_size); entries past a sequence's last page are never read.
    k_min, k_max: None, or contiguous [num_pages, Hkv, D] of the cache's type: the page bounds that
    paged_kv_append keeps and select_kv_pages reads.

    Holds the tensors, no copies: what is written into them between calls counts.  The object
    itself is never changed by a call and may serve several streams."""

    __slots__ = ("k_pages", "v_pages", "page_table", "k_min", "k_max", "dtype", "device", "B",
                 "Hkv", "D", "page_size", "num_pages", "max_pages", "_flags", "_c")

    def __init__(self, k_pages, v_pages, page_table, k_min=None, k_max=None):
        import torch
        if k_pages.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("the cache must be bf16 or fp16")
        if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
            raise ValueError("k_pages and v_pages must be [num_pages, Hkv, page_size, D], of one shape")
        if (k_min is None) != (k_max is None):
            raise ValueError("k_min and k_max go together")
        if page_table.dtype != torch.int32 or page_table.dim() != 2 or (
                page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table must be int32 [B, max_pages] with a contiguous last dimension")
        self.num_pages, self.Hkv, self.page_size, self.D = k_pages.shape
        self.B, self.max_pages = page_table.shape
        bounds = () if k_min is None else (k_min, k_max)
        for t in (k_pages, v_pages, page_table) + bounds:
            if not t.is_cuda or t.device != k_pages.device:
                raise ValueError("the cache's tensors must be on one CUDA device")
        for t in (v_pages,) + bounds:
            if t.dtype != k_pages.dtype:
                raise ValueError("k_pages, v_pages, k_min and k_max must be of one type")
        for t in (k_pages, v_pages):
            if t.stride(3) != 1:
                raise ValueError("k_pages and v_pages must have a contiguous last dimension")
        for t in bounds:
            if t.shape != (self.num_pages, self.Hkv, self.D) or not t.is_contiguous():
                raise ValueError("k_min and k_max must be contiguous [num_pages, Hkv, D]")
        if self.D not in (64, 128) or self.page_size not in (16, 32, 64, 128, 256):
            raise ValueError("D must be 64 or 128, page_size 16, 32, 64, 128 or 256")
        self.k_pages, self.v_pages, self.page_table = k_pages, v_pages, page_table
        self.k_min, self.k_max = k_min, k_max
        self.dtype, self.device = k_pages.dtype, k_pages.device
        self._flags = FA_DTYPE_FP16 if self.dtype == torch.float16 else 0
        self._c = fa_paged_kv_t(
            k_pages.data_ptr(), v_pages.data_ptr(), *k_pages.stride()[:3], *v_pages.stride()[:3],
            _ptr(k_min), _ptr(k_max), page_table.data_ptr(), page_table.stride(0), _int(self.max_pages),
            _int(self.num_pages), self.page_size)


def _int32_of(t, shape, device, name):
    import torch
    if t.dtype != torch.int32 or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {tuple(shape)} on the cache's device")


def _query_of(q, cache):
    if q.dtype != cache.dtype or q.device != cache.device or q.dim() != 4:
        raise ValueError("q must be [B, Hq, Sq, D] of the cache's type, on its device")
    B, Hq, Sq, D = q.shape
    if B != cache.B or D != cache.D or Hq % cache.Hkv:
        raise ValueError("q does not fit the cache: B, D or Hq % Hkv")
    return B, Hq, Sq, D


def _raw_here(device) -> Optional[int]:
    """The raw current stream where `device` is the current device, else None."""
    import torch
    if torch.cuda.current_device() != device.index:
        return None
    fast = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # a tenth of current_stream()'s time
    return torch.cuda.current_stream().cuda_stream if fast is None else fast(device.index)


def _elsewhere(device, stream, call):
    """call(raw stream) with `device` current and, for a given stream, that stream current too, so
    that what the call allocates belongs to it."""
    import torch
    if stream is None:
        with torch.cuda.device(device):
            return call(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    if stream.device != device:
        raise ValueError("the stream is of another device than the cache")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def paged_kv_append(cache: PagedKV, kv_lens, k, v, *, new_lens=None, q=None, q_out=None, cos=None,
                    sin=None, interleaved: bool = False, stream=None):
    """New tokens into a paged cache, rotated on the way (fa_kv_append).

    k, v [B, Hkv, S, D] of the cache's type, any strides with a contiguous last dimension; token i
    of sequence b takes position kv_lens[b] + i (kv_lens int32 [B], the tokens in the cache before;
    the caller adds the new ones).  new_lens: int32 [B], how many of the S are real (None: all).
    q [B, Hq, S, D]: rotated by the same positions into q_out (allocated where None; may be q).
    cos, sin: fp32 [max_pos, r / 2] of the rotated channels r <= D, r a multiple of 16; None: no
    rotation.  interleaved: pairs (2j, 2j + 1) instead of (j, j + r / 2).
    Updates cache.k_min / k_max where the cache has them (then no two sequences may append to one
    page).  Returns q_out (rows past new_lens as they were: undefined in an allocated one), or None
    without q.  A sequence's rows are its first new_lens[b], flash_attention_decode wants them as the
    last: where new_lens differ, row i moves to row i + S - new_lens[b] in between.

    stream, of this and the other calls on a cache: as under torch.cuda.stream(stream); the caller
    orders it behind what makes the inputs and keeps them until it has run."""
    import torch
    if k.dim() != 4 or k.shape != v.shape:
        raise ValueError("k and v must be [B, Hkv, S, D], of one shape")
    B, Hkv, S, D = k.shape
    if B != cache.B or Hkv != cache.Hkv or D != cache.D:
        raise ValueError("k and v do not fit the cache: B, Hkv or D")
    _int32_of(kv_lens, (B,), cache.device, "kv_lens")
    if new_lens is not None:
        _int32_of(new_lens, (B,), cache.device, "new_lens")
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
        Hq = Hkv
    else:
        _query_of(q, cache)
        Hq = q.shape[1]
        if q.shape[2] != S or (q_out is not None and q_out.shape != q.shape):
            raise ValueError("q and q_out must be [B, Hq, S, D] with k's S")
    for t in (k, v) + (() if q is None else (q,)) + (() if q_out is None else (q_out,)):
        if t.dtype != cache.dtype or t.device != cache.device or t.stride(3) != 1:
            raise ValueError("k, v, q, q_out must be of the cache's type, on its device, with a contiguous last dimension")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    rot, max_pos = 0, 0
    if cos is not None:
        if cos.shape != sin.shape or cos.dim() != 2:
            raise ValueError("cos and sin must be [max_pos, rotated channels / 2]")
        for t in (cos, sin):
            if t.dtype != torch.float32 or t.device != cache.device or not t.is_contiguous():
                raise ValueError("cos and sin must be contiguous fp32 tensors on the cache's device")
        max_pos, rot = _int(cos.shape[0]), _int(2 * cos.shape[1])

    def call(raw):
        qo = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q is not None and q_out is None else q_out
        none = (0, 0, 0)
        x = fa_kv_new_t(k.data_ptr(), v.data_ptr(), _ptr(q), _ptr(qo), *k.stride()[:3], *v.stride()[:3],
                        *(none if q is None else q.stride()[:3]), *(none if q is None else qo.stride()[:3]),
                        _ptr(cos), _ptr(sin), rot, 1 if interleaved else 0, max_pos)
        _raise(library().fa_kv_append(cache._c, x, B, Hq, Hkv, S, D, cache._flags, kv_lens.data_ptr(),
                                      _ptr(new_lens), raw))
        return qo

    raw = _raw_here(cache.device) if stream is None else None
    return _elsewhere(cache.device, stream, call) if raw is None else call(raw)


def flash_attention_decode(q, cache: PagedKV, kv_lens, *, scale: Optional[float] = None,
                           pre_tokens: Optional[int] = None, page_idx=None, out=None, lse=None,
                           stream=None):
    """Attention of each sequence's newest tokens over a paged cache (fa_decode).

    q [B, Hq, Sq, D] contiguous, of the cache's type: the Sq newest tokens of each sequence, which
    are in the cache already; kv_lens int32 [B], the tokens in the cache.  Row i is token
    t = kv_lens[b] - Sq + i and sees keys max(0, t - pre_tokens) .. t (pre_tokens None: from 0); a
    row that sees none gets 0 and LSE +inf.  A sequence with fewer new tokens has them in its last
    rows (paged_kv_append leaves them in the first).  page_idx: int32 [B, Hkv, max_sel] (select_kv_pages):
    only these pages of each sequence are read (of a list, as many entries count as the sequence
    has pages: invalid ones belong at the end).  Returns (o, lse fp32 [B, Hq, Sq])."""
    import torch
    B, Hq, Sq, D = _query_of(q, cache)
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    _int32_of(kv_lens, (B,), cache.device, "kv_lens")
    max_sel = 0
    if page_idx is not None:
        max_sel = page_idx.shape[-1]
        _int32_of(page_idx, (B, cache.Hkv, max_sel), cache.device, "page_idx")
    if pre_tokens is not None and pre_tokens < 0:
        raise ValueError("pre_tokens must be >= 0 (None: unbounded)")
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype or out.device != q.device
                            or not out.is_contiguous()):
        raise ValueError("out must be contiguous, of q's shape and type, on its device")
    if lse is not None and (lse.shape != (B, Hq, Sq) or lse.dtype != torch.float32
                            or lse.device != q.device or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 tensor [B, Hq, Sq] on q's device")

    def call(raw):
        o = torch.empty_like(q) if out is None else out
        e = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device) if lse is None else lse
        _raise(library().fa_decode(q.data_ptr(), cache._c, o.data_ptr(), e.data_ptr(), B, Hq, cache.Hkv,
                                   Sq, D, 1.0 / math.sqrt(D) if scale is None else scale, cache._flags,
                                   kv_lens.data_ptr(), -1 if pre_tokens is None else _int(pre_tokens),
                                   _ptr(page_idx), max_sel, raw))
        return o, e

    raw = _raw_here(cache.device) if stream is None else None
    return _elsewhere(cache.device, stream, call) if raw is None else call(raw)


def select_kv_pages(q, cache: PagedKV, kv_lens, max_sel: int, *, first: int = 1, last: int = 1,
                    out=None, stream=None):
    """The pages of each sequence whose keys can score highest (fa_select_pages), as the page_idx
    of flash_attention_decode: int32 [B, Hkv, max_sel], ascending, -1 behind the last.  The cache
    needs page bounds (k_min, k_max).  first, last: so many first and last pages are always
    chosen."""
    import torch
    B, Hq, Sq, D = _query_of(q, cache)
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    if cache.k_min is None:
        raise ValueError("the cache has no page bounds (k_min, k_max)")
    _int32_of(kv_lens, (B,), cache.device, "kv_lens")
    shape = (B, cache.Hkv, max_sel)
    if out is not None:
        _int32_of(out, shape, cache.device, "out")

    def call(raw):
        idx = torch.empty(shape, dtype=torch.int32, device=q.device) if out is None else out
        _raise(library().fa_select_pages(q.data_ptr(), cache._c, idx.data_ptr(), B, Hq, cache.Hkv, Sq, D,
                                         cache._flags, kv_lens.data_ptr(), max_sel, _int(first), _int(last), raw))
        return idx

    raw = _raw_here(cache.device) if stream is None else None
    return _elsewhere(cache.device, stream, call) if raw is None else call(raw)
