"""Thin Python binding of libtm (ctypes).

Argument marshalling only: every step of tile-routed attention runs in the
library's CUDA kernels.  PyTorch supplies device memory and the current
stream; outputs are allocated here with torch and passed to the library as
raw pointers.  There is no CPU fallback: if libtm.so is missing the import
fails, and a CUDA tensor is required wherever the library expects device
memory.
"""

from __future__ import annotations

import ctypes
import math
import os
import re
import struct

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtm.so")
HEADER = os.path.join(_HERE, "..", "include", "tm.h")

TM_OK, TM_ERR_INVALID_ARG, TM_ERR_UNSUPPORTED, TM_ERR_CUDA, TM_ERR_TIMEOUT = range(5)
TM_SCALE_NONE, TM_SCALE_TILE, TM_SCALE_TOKEN = range(3)


class TmError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {_lib().tm_status_string(status).decode()} (status {status}"
                         + (f", cuda {_lib().tm_last_cuda_error()})" if status == TM_ERR_CUDA else ")"))


class TmRopeFreqs(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("mscale", ctypes.c_float), ("turns", ctypes.c_uint64 * 64)]


class TmPagedKv(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scales", "v_scales")]
                + [(n, ctypes.c_int32) for n in ("num_pages", "page_size", "H", "d")]
                + [(n, ctypes.c_int64) for n in ("stride_page", "stride_t", "stride_h", "scale_stride_page",
                                                 "scale_stride_t", "scale_stride_h")])


class TmTensor(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("T", ctypes.c_int64), ("H", ctypes.c_int64), ("d", ctypes.c_int64),
        ("stride_t", ctypes.c_int64), ("stride_h", ctypes.c_int64),
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("scale_kind", ctypes.c_int32),
    ]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libtm.so not built at {LIB_PATH}; run "
                              "`python -m mixed_precision_attention_tm_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        P, I32, I64, U64, D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_double
        TP = ctypes.POINTER(TmTensor)
        RP, KP, F = ctypes.POINTER(TmRopeFreqs), ctypes.POINTER(TmPagedKv), ctypes.c_float
        sig = {
            "tm_quantize_qk": (I32, [TP, TP, P, P, P, P, P, I32, I32, I32, I32, P]),
            "tm_mask_words": (I32, [I64, I32, I32]),
            "tm_count_tiles": (I64, [P, I32, I64, I32]),
            "tm_build_mask": (I32, [P, I32, P, I32, I32, I64, I64, I32, I32, I32, I32, D, U64, I32, I32,
                                    I64, P]),
            "tm_build_mask_host": (I32, [P, I32, P, I32, I64, I64, I32, I32, I32, I32, D, U64, I32, I32]),
            "tm_build_mask_scale_policy": (I32, [P, I32, I32, P, I32, I32, I64, I64, I32, I32, I32, I32, P, P,
                                                 ctypes.c_float, I32, I32, I64, P]),
            "tm_build_mask_scale_policy_varlen": (I32, [P, I32, I32, P, P, I32, I32, I32, I32, I32, I32, I32,
                                                        P, P, ctypes.c_float, I32, I32, I64, P]),
            "tm_key_tile_scales": (I32, [P, P, I32, P, I32, I32, I64, I32, P]),
            "tm_cache_workspace_bytes": (I64, [I64, I32, I32]),
            "tm_attn_fwd_cache_ws": (I32, [TP, TP, TP, TP, P, P, I32, I32, I32, P, I64, I32, I32, I32, I32, P, I64,
                                           P]),
            "tm_route_stats": (I32, [P, I64, I32, P, I32, I64, I64, I32, I32, I32, I32,
                                     ctypes.POINTER(D), ctypes.POINTER(D)]),
            "tm_attn_fwd": (I32, [TP, TP, TP, TP, P, I32, I32, P, I64, I32, I32, I32, I32, P]),
            "tm_attn_fwd_varlen": (I32, [TP, TP, TP, TP, P, P, I32, I32, I32, P, I64, I32, I32, I32, I32, P]),
            "tm_quantize_qk_varlen": (I32, [TP, TP, P, P, P, P, P, P, I32, I32, I32, I32, I32, P]),
            "tm_build_mask_varlen": (I32, [P, I32, P, P, I32, I32, I32, I32, I32, I32, I32, D, U64, I32, I32,
                                           I64, P]),
            "tm_route_stats_varlen": (I32, [P, I64, I32, P, P, I32, I32, I32, I32, I32,
                                            ctypes.POINTER(D), ctypes.POINTER(D)]),
            "tm_attn_fwd_routed_noalloc": (I32, [TP, TP, TP, TP, I32, I32, I32, I32, D, U64, I32, I32, P]),
            "tm_selftest_wait_timeout": (I32, [U64, P]),
            "tm_get_device_error": (I32, [P]),
            "tm_status_string": (ctypes.c_char_p, [I32]),
            "tm_last_cuda_error": (I32, []),
            "tm_version": (ctypes.c_char_p, []),
            "tm_probe_scratch_bytes": (I64, []),
            "tm_probe_rates": (I32, [ctypes.POINTER(D), I32, P, I64, P]),
            "tm_merge_head_shards": (I32, [P, I64, P, I64, I32, I32, I32, I32, P, P]),
            "tm_set_attn_kernel": (I32, [I32]),
            "tm_attn_kernel_choice": (I32, [I64, I64, I32, I32, I32, I32, I32, I32]),
            "tm_quantize_qk_fp8": (I32, [TP, TP, P, P, P, P, P, I32, I32, I32, I32, P]),
            "tm_rope_init": (I32, [RP, I32, I32, I32, D, I32, D, D, D, D]),
            "tm_rope": (I32, [P, P, P, P, RP, P, I64, P]),          # tensors from _thd
            "tm_qk_norm_rope": (I32, [P, P, P, P, P, P, F, RP, P, I64, P]),
            "tm_block_table_check": (I32, [P, I64, I32, P, I32, I32, I32, P]),
            "tm_kv_append": (I32, [P, P, KP, P, I64, I32, P, P, I32, RP, I64, P, P, P, P, F, P]),
            "tm_kv_gather": (I32, [KP, P, I64, I32, P, I32, P, P, P]),
            "tm_attn_shared_prefix_workspace": (I64, [I64, I32, I32, I32, I32, I32, I64, I64]),
            "tm_attn_shared_prefix": (I32, [P, KP, P, P, I64, I32, P, P, I32, I32, P, I64, I64, I32, P, I64, P]),
            "tm_attn_fwd_fp8": (I32, [TP, TP, TP, TP, P, I32, I32, P, P, I64, P, P, P, P, I32, I32, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _LIB = lib
    return _LIB


def header_functions():
    """Names of the functions declared in include/tm.h."""
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(tm_[a-z0-9_]+)\s*\(", src)))


def _check(st, what):
    if st != TM_OK:
        raise TmError(st, what)


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _cuda(t, name):
    if t is not None and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _desc(x, codes=None, scales=None, scale_kind=TM_SCALE_NONE, shape_from=None):
    """tm_tensor for a [T, H, d] tensor (x may be None for an INT8 cache)."""
    ref = x if x is not None else shape_from
    T, H, d = ref.shape
    if x is not None:
        if x.dtype != torch.float16:
            raise ValueError("fp16 tensor expected")
        if x.stride(2) != 1:
            raise ValueError("innermost dimension must be contiguous")
        st, sh = x.stride(0), x.stride(1)
    else:
        st, sh = H * d, d
    return TmTensor(None if x is None else x.data_ptr(), T, H, d, st, sh,
                    None if codes is None else codes.data_ptr(),
                    None if scales is None else scales.data_ptr(), scale_kind)


def _cu_host(cu_seqlens, cu_seqlens_host=None):
    """Host int32 copy of cu_seqlens.  Callers that run many steps pass the
    host copy they keep (cu_seqlens_host) so no step reads the device array
    back (a blocking copy)."""
    if cu_seqlens is None:
        return None
    if cu_seqlens_host is not None:
        return torch.as_tensor(cu_seqlens_host, dtype=torch.int32).contiguous()
    return cu_seqlens.detach().to("cpu", torch.int32).contiguous()


def _check_buf(t, shape, dtype, name):
    if t is None or tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)}")


def count_tiles(L=None, tile=128, cu_seqlens_host=None):
    lib = _lib()
    if cu_seqlens_host is not None:
        cu = np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int32))
        return int(lib.tm_count_tiles(cu.ctypes.data, len(cu) - 1, 0, tile))
    return int(lib.tm_count_tiles(None, 0, int(L), tile))


def mask_words(max_lk, tile_n, g):
    return int(_lib().tm_mask_words(int(max_lk), int(tile_n), int(g)))


def _need(t, n, dtype, name):
    """t holds at least n contiguous elements of dtype."""
    if t is None or t.dtype != dtype or not t.is_contiguous() or t.numel() < n:
        got = "None" if t is None else f"{tuple(t.shape)} {t.dtype}"
        raise ValueError(f"{name}: at least {n} contiguous {dtype} elements expected, got {got}")


def _check_routing(Tq, Hq, Tk, Hkv, d, tile_m, tile_n, g, maxk, cu_h, ck_h, bitmask, mask_head_stride,
                   q_quant, k_quant, codes_dtype=torch.int8, what=""):
    """Sizes of the buffers an attention launch reads (the library receives
    plain pointers): codes [T, H, d]; tile scales n_tiles x H fp32, tiles
    counted per sequence; mask words (Hm - 1) x head stride + n_qtiles x W,
    W = mask_words(longest key row, tile_n, g) as the kernels compute it.
    ck_h: host key offsets (cu_h when keys share the query offsets), or None
    when only the device holds them (then the key scales are not counted)."""
    nqt = count_tiles(Tq, tile_m, None if cu_h is None else cu_h.numpy())
    if bitmask is not None:
        rows = nqt * mask_words(maxk, tile_n, g)
        _need(bitmask, rows + (Hq - 1) * int(mask_head_stride or 0), torch.int32, what + "bitmask")
    if q_quant is not None:
        _need(q_quant[0], Tq * Hq * d, codes_dtype, what + "q codes")
        _need(q_quant[1], nqt * Hq, torch.float32, what + "q scales")
    if k_quant is not None:
        _need(k_quant[0], Tk * Hkv * d, codes_dtype, what + "k codes")
        if ck_h is not None or cu_h is None:
            nkt = count_tiles(Tk, tile_n, None if ck_h is None else ck_h.numpy())
            _need(k_quant[1], nkt * Hkv, torch.float32, what + "k scales")


# ---------------------------------------------------------------- quantise
def quantize_qk(q, k=None, *, tile_m=128, tile_n=128, cu_seqlens=None, max_seqlen=None,
                cu_seqlens_host=None, out=None, cu_seqlens_k=None, max_seqlen_k=None, cu_seqlens_k_host=None):
    """Per-tile INT8 codes and fp32 scales of Q (tile_m rows) and K (tile_n
    rows): returns (q_codes [Tq,Hq,d] int8, q_scales [n_qt, Hq] fp32,
    k_codes, k_scales) (the K pair is None when k is None).  out: the same
    4-tuple of preallocated tensors to write into (reused across steps)."""
    _cuda(q, "q")
    _cuda(k, "k")
    lib = _lib()
    cu_h = _cu_host(cu_seqlens, cu_seqlens_host)
    batch = 0 if cu_h is None else cu_h.numel() - 1
    if cu_seqlens is not None and max_seqlen is None:
        max_seqlen = int((cu_h[1:] - cu_h[:-1]).max()) if batch else 0
    nqt = count_tiles(q.shape[0], tile_m, None if cu_h is None else cu_h.numpy())
    ck_h = cu_h if cu_seqlens_k is None else _cu_host(cu_seqlens_k, cu_seqlens_k_host)
    if cu_seqlens_k is not None and max_seqlen_k is None:
        max_seqlen_k = int((ck_h[1:] - ck_h[:-1]).max()) if batch else 0
    if out is not None:
        qc, qs, kc, ks = out
        _check_buf(qc, q.shape, torch.int8, "q_codes")
        _check_buf(qs, (nqt, q.shape[1]), torch.float32, "q_scales")
        if k is None:
            kc = ks = None
    else:
        qc = torch.empty(q.shape, dtype=torch.int8, device=q.device)
        qs = torch.empty((nqt, q.shape[1]), dtype=torch.float32, device=q.device)
        kc = ks = None
    if k is not None and out is not None:
        nkt = count_tiles(k.shape[0], tile_n, None if ck_h is None else ck_h.numpy())
        _check_buf(kc, k.shape, torch.int8, "k_codes")
        _check_buf(ks, (nkt, k.shape[1]), torch.float32, "k_scales")
    elif k is not None:
        nkt = count_tiles(k.shape[0], tile_n, None if ck_h is None else ck_h.numpy())
        kc = torch.empty(k.shape, dtype=torch.int8, device=k.device)
        ks = torch.empty((nkt, k.shape[1]), dtype=torch.float32, device=k.device)
    qd = _desc(q)
    kd = _desc(k) if k is not None else None
    if cu_seqlens_k is not None:       # separate key offsets (prefix-cached prefill)
        st = lib.tm_quantize_qk_varlen(ctypes.byref(qd), None if kd is None else ctypes.byref(kd),
                                       _ptr(qc), _ptr(qs), _ptr(kc), _ptr(ks), _ptr(cu_seqlens), _ptr(cu_seqlens_k),
                                       batch, int(max_seqlen or 0), int(max_seqlen_k or 0), tile_m, tile_n,
                                       _stream())
        _check(st, "tm_quantize_qk_varlen")
        return qc, qs, kc, ks
    st = lib.tm_quantize_qk(ctypes.byref(qd), None if kd is None else ctypes.byref(kd),
                            _ptr(qc), _ptr(qs), _ptr(kc), _ptr(ks), _ptr(cu_seqlens), batch,
                            int(max_seqlen or 0), tile_m, tile_n, _stream())
    _check(st, "tm_quantize_qk")
    return qc, qs, kc, ks


def quantize_qk_fp8(q, k=None, *, tile_m=128, tile_n=128, cu_seqlens=None, max_seqlen=None,
                    cu_seqlens_host=None, out=None):
    """Per-tile FP8 E4M3 codes and fp32 scales of Q and K (the third
    precision; tm_quantize_qk_fp8): returns (q_codes [Tq,Hq,d] uint8,
    q_scales [n_qt, Hq] fp32, k_codes, k_scales); the K pair is None when k
    is None.  out: the same 4-tuple of preallocated tensors."""
    _cuda(q, "q")
    _cuda(k, "k")
    cu_h = _cu_host(cu_seqlens, cu_seqlens_host)
    batch = 0 if cu_h is None else cu_h.numel() - 1
    if cu_seqlens is not None and max_seqlen is None:
        max_seqlen = int((cu_h[1:] - cu_h[:-1]).max()) if batch else 0
    cu_np = None if cu_h is None else cu_h.numpy()
    nqt = count_tiles(q.shape[0], tile_m, cu_np)
    if out is not None:
        qc, qs, kc, ks = out
        _check_buf(qc, q.shape, torch.uint8, "q_codes")
        _check_buf(qs, (nqt, q.shape[1]), torch.float32, "q_scales")
    else:
        qc = torch.empty(q.shape, dtype=torch.uint8, device=q.device)
        qs = torch.empty((nqt, q.shape[1]), dtype=torch.float32, device=q.device)
        kc = ks = None
    if k is not None:
        nkt = count_tiles(k.shape[0], tile_n, cu_np)
        if out is not None:
            _check_buf(kc, k.shape, torch.uint8, "k_codes")
            _check_buf(ks, (nkt, k.shape[1]), torch.float32, "k_scales")
        else:
            kc = torch.empty(k.shape, dtype=torch.uint8, device=k.device)
            ks = torch.empty((nkt, k.shape[1]), dtype=torch.float32, device=k.device)
    else:
        kc = ks = None
    qd = _desc(q)
    kd = _desc(k) if k is not None else None
    st = _lib().tm_quantize_qk_fp8(ctypes.byref(qd), None if kd is None else ctypes.byref(kd), _ptr(qc), _ptr(qs),
                                   _ptr(kc), _ptr(ks), _ptr(cu_seqlens), batch, int(max_seqlen or 0), tile_m,
                                   tile_n, _stream())
    _check(st, "tm_quantize_qk_fp8")
    return qc, qs, kc, ks


# ---------------------------------------------------------------- mask
def build_mask(Hq, *, tile_m, tile_n, g, causal, p, seed, force_diag=False, force_sink=False,
               Lq=None, Lk=None, cu_seqlens=None, max_seqlen=None, device="cuda",
               cu_seqlens_host=None, out=None, cu_seqlens_k=None, max_seqlen_k=None, cu_seqlens_k_host=None):
    """Seeded routing bitmask on the device, int32 view [Hq, n_qt, W] of the
    uint32 words (bit 1 = INT8).  The library writes every word, so the
    buffer (out, or a new one) needs no initialisation."""
    lib = _lib()
    cu_h = _cu_host(cu_seqlens, cu_seqlens_host)
    batch = 0 if cu_h is None else cu_h.numel() - 1
    if cu_h is not None:
        lens = (cu_h[1:] - cu_h[:-1])
        maxk = int(lens.max()) if batch else 0
        if max_seqlen is None:
            max_seqlen = maxk
        nqt = count_tiles(None, tile_m, cu_h.numpy())
        if cu_seqlens_k is not None:       # key lengths from the key offsets
            ck_h = _cu_host(cu_seqlens_k, cu_seqlens_k_host)
            maxk = int((ck_h[1:] - ck_h[:-1]).max()) if batch else 0
            if max_seqlen_k is None:
                max_seqlen_k = maxk
            maxk = max_seqlen_k
    else:
        maxk = Lk
        nqt = count_tiles(Lq, tile_m)
    W = mask_words(maxk, tile_n, g)
    if out is None:
        out = torch.empty((Hq, nqt, W), dtype=torch.int32, device=device)
    else:
        _check_buf(out, (Hq, nqt, W), torch.int32, "bitmask")
    if cu_seqlens_k is not None:
        st = lib.tm_build_mask_varlen(_ptr(out), Hq, _ptr(cu_seqlens), _ptr(cu_seqlens_k), batch,
                                      int(max_seqlen or 0), int(max_seqlen_k or 0), tile_m, tile_n, g,
                                      int(bool(causal)), float(p), ctypes.c_uint64(int(seed) & (2 ** 64 - 1)),
                                      int(bool(force_diag)), int(bool(force_sink)), nqt * W, _stream())
        _check(st, "tm_build_mask_varlen")
        return out
    st = lib.tm_build_mask(_ptr(out), Hq, _ptr(cu_seqlens), batch, int(max_seqlen or 0),
                           int(Lq or 0), int(Lk or 0), tile_m, tile_n, g, int(bool(causal)),
                           float(p), ctypes.c_uint64(int(seed) & (2 ** 64 - 1)),
                           int(bool(force_diag)), int(bool(force_sink)), nqt * W, _stream())
    _check(st, "tm_build_mask")
    return out


def build_mask_scale_policy(q_scales, k_scales, Hq, Hkv, *, tile_m, tile_n, g, causal, tau, force_diag=False,
                            force_sink=False, Lq=None, Lk=None, cu_seqlens=None, max_seqlen=None,
                            cu_seqlens_host=None, out=None, cu_seqlens_k=None, max_seqlen_k=None,
                            cu_seqlens_k_host=None):
    """Content-driven routing bitmask (int32 view [Hq, n_qt, W]): group G of
    query tile I goes INT8 iff s_q[I] * max s_k over its visible key tiles
    <= tau (see tm_build_mask_scale_policy).  q_scales / k_scales: the device
    tile scales from quantize_qk, or k_scales from key_tile_scales for an INT8
    cache.  cu_seqlens_k: key offsets when they differ from cu_seqlens."""
    _cuda(q_scales, "q_scales")
    _cuda(k_scales, "k_scales")
    lib = _lib()
    cu_h = _cu_host(cu_seqlens, cu_seqlens_host)
    batch = 0 if cu_h is None else cu_h.numel() - 1
    if cu_seqlens_k is not None and cu_h is None:
        raise ValueError("cu_seqlens_k needs cu_seqlens")
    if cu_h is not None:
        maxk = int((cu_h[1:] - cu_h[:-1]).max()) if batch else 0
        if max_seqlen is None:
            max_seqlen = maxk
        nqt = count_tiles(None, tile_m, cu_h.numpy())
        if cu_seqlens_k is not None:
            ck_h = _cu_host(cu_seqlens_k, cu_seqlens_k_host)
            if max_seqlen_k is None:
                max_seqlen_k = int((ck_h[1:] - ck_h[:-1]).max()) if batch else 0
            maxk = max_seqlen_k
    else:
        maxk = Lk
        nqt = count_tiles(Lq, tile_m)
    W = mask_words(maxk, tile_n, g)
    if out is None:
        out = torch.empty((Hq, nqt, W), dtype=torch.int32, device=q_scales.device)
    else:
        _check_buf(out, (Hq, nqt, W), torch.int32, "bitmask")
    if cu_seqlens_k is not None:
        st = lib.tm_build_mask_scale_policy_varlen(
            _ptr(out), Hq, Hkv, _ptr(cu_seqlens), _ptr(cu_seqlens_k), batch, int(max_seqlen or 0),
            int(max_seqlen_k or 0), tile_m, tile_n, g, int(bool(causal)), _ptr(q_scales), _ptr(k_scales),
            float(tau), int(bool(force_diag)), int(bool(force_sink)), nqt * W, _stream())
        _check(st, "tm_build_mask_scale_policy_varlen")
        return out
    st = lib.tm_build_mask_scale_policy(_ptr(out), Hq, Hkv, _ptr(cu_seqlens), batch, int(max_seqlen or 0),
                                        int(Lq or 0), int(Lk or 0), tile_m, tile_n, g, int(bool(causal)),
                                        _ptr(q_scales), _ptr(k_scales), float(tau), int(bool(force_diag)),
                                        int(bool(force_sink)), nqt * W, _stream())
    _check(st, "tm_build_mask_scale_policy")
    return out


def key_tile_scales(k_token_scales, *, tile_n, cu_seqlens_k=None, max_seqlen_k=None, cu_seqlens_k_host=None,
                    out=None):
    """Largest per-token key scale of every key tile and kv head (fp32
    [n_ktiles, Hkv]) from an INT8 cache's fp16 scales [Tk, Hkv]: the k_scales
    of the scale policy for that cache (see tm_key_tile_scales)."""
    _cuda(k_token_scales, "k_token_scales")
    if k_token_scales.dtype != torch.float16 or k_token_scales.dim() != 2 or not k_token_scales.is_contiguous():
        raise ValueError("k_token_scales: contiguous fp16 [Tk, Hkv]")
    Tk, Hkv = k_token_scales.shape
    lib = _lib()
    ck_h = _cu_host(cu_seqlens_k, cu_seqlens_k_host)
    batch = 0 if ck_h is None else ck_h.numel() - 1
    if ck_h is not None:
        if max_seqlen_k is None:
            max_seqlen_k = int((ck_h[1:] - ck_h[:-1]).max()) if batch else 0
        nkt = count_tiles(None, tile_n, ck_h.numpy())
    else:
        nkt = count_tiles(Tk, tile_n)
    if out is None:
        out = torch.empty((nkt, Hkv), dtype=torch.float32, device=k_token_scales.device)
    else:
        _check_buf(out, (nkt, Hkv), torch.float32, "k_tile_scales")
    st = lib.tm_key_tile_scales(_ptr(out), _ptr(k_token_scales), Hkv, _ptr(cu_seqlens_k), batch,
                                int(max_seqlen_k or 0), int(Tk), tile_n, _stream())
    _check(st, "tm_key_tile_scales")
    return out


def build_mask_host(Hq, *, tile_m, tile_n, g, causal, p, seed, force_diag=False, force_sink=False,
                    Lq=None, Lk=None, cu_seqlens_host=None):
    """Host twin of build_mask: numpy uint32 [Hq, n_qt, W]."""
    lib = _lib()
    cu = None if cu_seqlens_host is None else np.ascontiguousarray(np.asarray(cu_seqlens_host, np.int32))
    batch = 0 if cu is None else len(cu) - 1
    if cu is not None:
        maxk = int((cu[1:] - cu[:-1]).max()) if batch else 0
        nqt = count_tiles(None, tile_m, cu)
    else:
        maxk = Lk
        nqt = count_tiles(Lq, tile_m)
    W = mask_words(maxk, tile_n, g)
    out = np.zeros((Hq, nqt, W), dtype=np.uint32)
    st = lib.tm_build_mask_host(out.ctypes.data, Hq, None if cu is None else cu.ctypes.data, batch,
                                int(Lq or 0), int(Lk or 0), tile_m, tile_n, g, int(bool(causal)),
                                float(p), ctypes.c_uint64(int(seed) & (2 ** 64 - 1)),
                                int(bool(force_diag)), int(bool(force_sink)))
    _check(st, "tm_build_mask_host")
    return out


def route_stats(mask_host, *, Hq, tile_m, tile_n, g, causal, Lq=None, Lk=None, cu_seqlens_host=None,
                cu_seqlens_k_host=None):
    """(n_vis, e8) from a host mask (numpy uint32 [Hm, n_qt, W]) or None."""
    lib = _lib()
    cu = None if cu_seqlens_host is None else np.ascontiguousarray(np.asarray(cu_seqlens_host, np.int32))
    if cu_seqlens_k_host is not None:
        ck = np.ascontiguousarray(np.asarray(cu_seqlens_k_host, np.int32))
        nv, e8 = ctypes.c_double(), ctypes.c_double()
        ptr, hs = None, 0
        if mask_host is not None:
            m = np.ascontiguousarray(mask_host.astype(np.uint32, copy=False))
            ptr, hs = m.ctypes.data, (0 if m.shape[0] == 1 else m.shape[1] * m.shape[2])
        st = lib.tm_route_stats_varlen(ptr, hs, Hq, cu.ctypes.data, ck.ctypes.data, len(cu) - 1, tile_m, tile_n,
                                       g, int(bool(causal)), ctypes.byref(nv), ctypes.byref(e8))
        _check(st, "tm_route_stats_varlen")
        return nv.value, e8.value
    batch = 0 if cu is None else len(cu) - 1
    nv, e8 = ctypes.c_double(), ctypes.c_double()
    ptr, hs = None, 0
    if mask_host is not None:
        m = np.ascontiguousarray(mask_host.astype(np.uint32, copy=False))
        ptr = m.ctypes.data
        hs = 0 if m.shape[0] == 1 else m.shape[1] * m.shape[2]
    st = lib.tm_route_stats(ptr, hs, Hq, None if cu is None else cu.ctypes.data, batch, int(Lq or 0),
                            int(Lk or 0), tile_m, tile_n, g, int(bool(causal)), ctypes.byref(nv),
                            ctypes.byref(e8))
    _check(st, "tm_route_stats")
    return nv.value, e8.value


# ---------------------------------------------------------------- attention
def attn_fwd(q, k=None, v=None, *, out=None, tile_m=128, tile_n=128, g=1, causal=False,
             bitmask=None, mask_head_stride=None, q_quant=None, k_quant=None, kv_cache=None,
             cu_seqlens=None, max_seqlen=None, cu_seqlens_host=None, cu_seqlens_k=None, max_seqlen_k=None,
             cache_workspace=None):
    """Fused tile-routed attention.  q: fp16 [Tq,Hq,d]; k, v: fp16 [Tk,Hkv,d]
    (or kv_cache = (k_codes, k_scale16, v_codes, v_scale16)); bitmask: int32
    view [Hm, n_qt, W] (Hm = Hq or 1) or None (all FP16); q_quant / k_quant:
    (codes, scales) from quantize_qk, needed with a bitmask.
    cache_workspace: with kv_cache, a uint8 device tensor of at least
    cache_workspace_bytes(...) bytes; the cache is then expanded into it once
    and read from there (tm_attn_fwd_cache_ws).  Returns out."""
    _cuda(q, "q")
    lib = _lib()
    if out is None:
        out = torch.empty_like(q)
    cu_h = _cu_host(cu_seqlens, cu_seqlens_host)
    batch = 0 if cu_h is None else cu_h.numel() - 1
    if cu_seqlens is not None and max_seqlen is None:
        max_seqlen = int((cu_h[1:] - cu_h[:-1]).max()) if batch else 0
    if bitmask is not None and mask_head_stride is None:
        mask_head_stride = 0 if bitmask.shape[0] == 1 else bitmask.shape[1] * bitmask.shape[2]
    ck_h = None
    if cu_seqlens_k is not None and max_seqlen_k is None:
        ck_h = _cu_host(cu_seqlens_k, None)
        max_seqlen_k = int((ck_h[1:] - ck_h[:-1]).max()) if batch else 0
    kshape = (kv_cache[0] if kv_cache is not None else k).shape
    maxk = (max_seqlen_k if cu_seqlens_k is not None else max_seqlen) if cu_seqlens is not None else kshape[0]
    _check_routing(q.shape[0], q.shape[1], kshape[0], kshape[1], q.shape[2], tile_m, tile_n, g, maxk or 0, cu_h,
                   ck_h if cu_seqlens_k is not None else cu_h, bitmask, mask_head_stride, q_quant, k_quant)
    qd = _desc(q, *(q_quant if q_quant is not None else (None, None)),
               scale_kind=TM_SCALE_TILE if q_quant is not None else TM_SCALE_NONE)
    if kv_cache is not None:
        kcod, ksc, vcod, vsc = kv_cache
        kd = _desc(None, kcod, ksc, TM_SCALE_TOKEN, shape_from=kcod)
        vd = _desc(None, vcod, vsc, TM_SCALE_TOKEN, shape_from=vcod)
    else:
        _cuda(k, "k")
        _cuda(v, "v")
        kd = _desc(k, *(k_quant if k_quant is not None else (None, None)),
                   scale_kind=TM_SCALE_TILE if k_quant is not None else TM_SCALE_NONE)
        vd = _desc(v)
    od = _desc(out)
    if cache_workspace is not None:
        if kv_cache is None:
            raise ValueError("cache_workspace is for an INT8 K/V cache")
        _cuda(cache_workspace, "cache_workspace")
        need = cache_workspace_bytes(kshape[0], kshape[1], batch)
        if cache_workspace.dtype != torch.uint8 or cache_workspace.numel() < need \
                or not cache_workspace.is_contiguous():
            raise ValueError(f"cache_workspace: contiguous uint8 of at least {need} bytes expected")
        st = lib.tm_attn_fwd_cache_ws(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), ctypes.byref(od),
                                      _ptr(cu_seqlens), _ptr(cu_seqlens_k), batch, int(max_seqlen or 0),
                                      int(max_seqlen_k or 0), _ptr(bitmask), int(mask_head_stride or 0), tile_m,
                                      tile_n, g, int(bool(causal)), _ptr(cache_workspace),
                                      int(cache_workspace.numel()), _stream())
        _check(st, "tm_attn_fwd_cache_ws")
        return out
    if cu_seqlens_k is not None:
        st = lib.tm_attn_fwd_varlen(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), ctypes.byref(od),
                                    _ptr(cu_seqlens), _ptr(cu_seqlens_k), batch, int(max_seqlen or 0),
                                    int(max_seqlen_k or 0), _ptr(bitmask), int(mask_head_stride or 0), tile_m,
                                    tile_n, g, int(bool(causal)), _stream())
        _check(st, "tm_attn_fwd_varlen")
        return out
    st = lib.tm_attn_fwd(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), ctypes.byref(od),
                         _ptr(cu_seqlens), batch, int(max_seqlen or 0), _ptr(bitmask),
                         int(mask_head_stride or 0), tile_m, tile_n, g, int(bool(causal)), _stream())
    _check(st, "tm_attn_fwd")
    return out


def cache_workspace_bytes(Tk, Hkv, batch=0):
    """Bytes of the workspace tm_attn_fwd_cache_ws needs for a cache of Tk
    tokens and Hkv heads (batch: sequences, 0 for one without offsets)."""
    n = int(_lib().tm_cache_workspace_bytes(int(Tk), int(Hkv), int(batch)))
    if n < 0:
        raise ValueError("bad cache shape")
    return n


def attn_fwd_fp8(q, k, v, *, bitmask_fp8, qf8_quant, kf8_quant, out=None, g=1, causal=False, bitmask=None,
                 q_quant=None, k_quant=None, cu_seqlens=None, max_seqlen=None, cu_seqlens_host=None):
    """Attention with the FP8 third precision (tm_attn_fwd_fp8): d = 128,
    128 x 128 tiles; bitmask_fp8 (int32 view [Hm, n_qt, W], layout of the
    INT8 bitmask) routes a group to FP8 when its INT8 bit (bitmask, may be
    None) is clear; qf8_quant / kf8_quant = (codes, scales) from
    quantize_qk_fp8; q_quant / k_quant the INT8 (codes, scales) when bitmask
    is given.  Returns out."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (bitmask_fp8, "bitmask_fp8")):
        _cuda(t, n)
    if out is None:
        out = torch.empty_like(q)
    cu_h = _cu_host(cu_seqlens, cu_seqlens_host)
    batch = 0 if cu_h is None else cu_h.numel() - 1
    if cu_seqlens is not None and max_seqlen is None:
        max_seqlen = int((cu_h[1:] - cu_h[:-1]).max()) if batch else 0
    qd = _desc(q, *(q_quant if q_quant is not None else (None, None)),
               scale_kind=TM_SCALE_TILE if q_quant is not None else TM_SCALE_NONE)
    kd = _desc(k, *(k_quant if k_quant is not None else (None, None)),
               scale_kind=TM_SCALE_TILE if k_quant is not None else TM_SCALE_NONE)
    vd, od = _desc(v), _desc(out)
    mhs = 0 if bitmask_fp8.shape[0] == 1 else bitmask_fp8.shape[1] * bitmask_fp8.shape[2]
    if bitmask is not None and tuple(bitmask.shape) != tuple(bitmask_fp8.shape):
        raise ValueError("bitmask and bitmask_fp8 must have the same layout")
    maxk = max_seqlen if cu_seqlens is not None else k.shape[0]
    _check_routing(q.shape[0], q.shape[1], k.shape[0], k.shape[1], q.shape[2], 128, 128, g, maxk or 0, cu_h, cu_h,
                   bitmask, mhs, q_quant, k_quant)
    _check_routing(q.shape[0], q.shape[1], k.shape[0], k.shape[1], q.shape[2], 128, 128, g, maxk or 0, cu_h, cu_h,
                   bitmask_fp8, mhs, qf8_quant, kf8_quant, codes_dtype=torch.uint8, what="fp8 ")
    st = _lib().tm_attn_fwd_fp8(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), ctypes.byref(od),
                                _ptr(cu_seqlens), batch, int(max_seqlen or 0), _ptr(bitmask), _ptr(bitmask_fp8), mhs,
                                _ptr(qf8_quant[0]), _ptr(qf8_quant[1]), _ptr(kf8_quant[0]), _ptr(kf8_quant[1]),
                                g, int(bool(causal)), _stream())
    _check(st, "tm_attn_fwd_fp8")
    return out


def attn_fwd_routed_noalloc(q, k, v, *, out=None, tile_m=128, tile_n=128, g=1, causal=False, p=0.5,
                            seed=0, force_diag=False, force_sink=False):
    """Routed prefill (quantise, mask, attend) for one sequence with the
    library's fixed device scratch array instead of caller-allocated codes,
    scales and mask; only out is allocated here (by torch) when not given."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _cuda(t, n)
    if out is None:
        out = torch.empty_like(q)
    qd, kd, vd, od = _desc(q), _desc(k), _desc(v), _desc(out)
    st = _lib().tm_attn_fwd_routed_noalloc(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), ctypes.byref(od),
                                           tile_m, tile_n, g, int(bool(causal)), float(p),
                                           ctypes.c_uint64(int(seed) & (2 ** 64 - 1)), int(bool(force_diag)),
                                           int(bool(force_sink)), _stream())
    _check(st, "tm_attn_fwd_routed_noalloc")
    return out


ATTN_KERNEL_AUTO, ATTN_KERNEL_TWO_TILE, ATTN_KERNEL_ONE_TILE = 0, 1, 2


def set_attn_kernel(choice):
    """Kernel for 128 x 128-tile attention with fp16 K / V, d = 64 or 128
    (tm_set_attn_kernel): ATTN_KERNEL_AUTO (default), ATTN_KERNEL_TWO_TILE or
    ATTN_KERNEL_ONE_TILE.  Process-wide."""
    _check(_lib().tm_set_attn_kernel(int(choice)), "tm_set_attn_kernel")


def attn_kernel_choice(max_q, max_k, hq, d, *, batch=1, routed=False, causal=True, sm_count=0):
    """Kernel tm_attn_fwd would run for 128 x 128 tiles with fp16 K / V
    (tm_attn_kernel_choice): ATTN_KERNEL_TWO_TILE or ATTN_KERNEL_ONE_TILE.
    sm_count 0 queries the current device."""
    r = int(_lib().tm_attn_kernel_choice(int(max_q), int(max_k), int(batch), int(hq), int(d), int(bool(routed)),
                                         int(bool(causal)), int(sm_count)))
    if r == 0:
        raise ValueError("tm_attn_kernel_choice: invalid arguments")
    return r


def merge_head_shards(out, gathered, head_start):
    """Interleave the all-gathered output slices of a head-sharded prefill
    back into token-major order (tm_merge_head_shards): gathered fp16
    [world, T, h_cap, d] contiguous, rank r's heads head_start[r] ..
    head_start[r+1]-1 in its first slots; out fp16 [T, Hq, d] (heads
    contiguous, rows may be strided).  Returns out."""
    _cuda(out, "out")
    _cuda(gathered, "gathered")
    if out.dtype != torch.float16 or gathered.dtype != torch.float16:
        raise ValueError("fp16 tensors expected")
    if gathered.dim() != 4 or not gathered.is_contiguous():
        raise ValueError("gathered: contiguous [world, T, h_cap, d] expected")
    world, T, h_cap, d = gathered.shape
    if out.dim() != 3 or out.shape[0] != T or out.shape[2] != d or out.stride(2) != 1 or out.stride(1) != d:
        raise ValueError("out: [T, Hq, d] with contiguous heads expected")
    hs = np.ascontiguousarray(np.asarray(head_start, dtype=np.int32))
    if hs.shape != (world + 1,):
        raise ValueError("head_start must hold world + 1 entries")
    st = _lib().tm_merge_head_shards(_ptr(out), int(out.stride(0)), _ptr(gathered), int(T), int(out.shape[1]),
                                     int(d), int(world), int(h_cap), hs.ctypes.data, _stream())
    _check(st, "tm_merge_head_shards")
    return out


# ------------------------------------------------- serving over a paged cache
ROPE_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


class Rope:
    """Rotary positions of heads of d values (tm_rope_init): the first rot_dim
    of them turned (default all; a multiple of 16), in pairs (i, i +
    rot_dim / 2), or (2i, 2i + 1) when interleaved.  scaling for contexts
    longer than original_max: None, "linear", "ntk", "yarn" or "bands" (see
    tm_rope_scaling in include/tm.h), by factor; fast / slow default to 32 / 1
    for "yarn" and 4 / 1 for "bands".  Host object; keep one for each model."""

    def __init__(self, d, rot_dim=None, *, theta=10000.0, interleaved=False, scaling=None, factor=1.0,
                 original_max=4096, fast=None, slow=None):
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling: one of {tuple(ROPE_SCALINGS)} expected")
        self.d, self.rot_dim = int(d), int(d if rot_dim is None else rot_dim)
        self.struct = TmRopeFreqs()
        fast = (4.0 if scaling == "bands" else 32.0) if fast is None else fast
        _check(_lib().tm_rope_init(ctypes.byref(self.struct), self.d, self.rot_dim, int(bool(interleaved)), float(theta),
                                   ROPE_SCALINGS[scaling], float(factor), float(original_max), float(fast),
                                   float(1.0 if slow is None else slow)), "tm_rope_init")


class PagedKV:
    """A pool of K/V pages (tm_paged_kv): k, v [num_pages, page_size, Hkv, d],
    fp16, or INT8 codes with fp16 scales [num_pages, page_size, Hkv] for each
    slot and head.  Any strides with the innermost dimension contiguous (heads
    before slots, say), the same for K and V.  Wraps the caller's tensors and
    keeps them alive; page_size in {16, 32, 64, 128, 256}, d in {64, 128}."""

    def __init__(self, k, v, k_scales=None, v_scales=None):
        if k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride() or v.dtype != k.dtype:
            raise ValueError("k, v: [num_pages, page_size, Hkv, d] of one shape, type and layout expected")
        if k.stride(3) != 1:
            raise ValueError("innermost dimension must be contiguous")
        self.int8 = k.dtype == torch.int8
        if self.int8 != (k_scales is not None) or self.int8 != (v_scales is not None):
            raise ValueError("INT8 pages come with k_scales and v_scales, fp16 pages without")
        if not self.int8 and k.dtype != torch.float16:
            raise ValueError("fp16 or int8 pages expected")
        for t, n in ((k, "k"), (v, "v"), (k_scales, "k_scales"), (v_scales, "v_scales")):
            _cuda(t, n)
            if t is not None and t.device != k.device:
                raise ValueError(f"{n}: all of a cache lies on one device")
        st = (0, 0, 0)
        if self.int8:
            for t in (k_scales, v_scales):
                if t.dtype != torch.float16 or t.shape != k.shape[:3] or t.stride() != k_scales.stride():
                    raise ValueError("k_scales, v_scales: fp16 [num_pages, page_size, Hkv] of one layout expected")
            st = k_scales.stride()
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.device, self.index = k.device, k.get_device()
        self.num_pages, self.page_size, self.H, self.d = k.shape
        if self.d not in (64, 128) or self.page_size not in (16, 32, 64, 128, 256):
            raise ValueError("page_size in {16, 32, 64, 128, 256} and d in {64, 128} expected")
        if min(k.stride()[:3]) <= 0 or (self.int8 and min(st) <= 0):
            raise ValueError("pages, slots and heads must not share memory")
        self.struct = TmPagedKv(k.data_ptr(), v.data_ptr(), k_scales.data_ptr() if self.int8 else None,
                                v_scales.data_ptr() if self.int8 else None, *k.shape, *k.stride()[:3], *st)


# The current stream's handle without a Stream object around it (0.1 us instead of 3.4).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_HALF, _INT32 = torch.float16, torch.int32
# A tm_tensor of an fp16 operand (no codes, no scales) as bytes: 0.1 us, where a ctypes.Structure takes 0.4.
_tensor_bytes = struct.Struct(f"P5q{ctypes.sizeof(TmTensor) - 48}x").pack


def _call(index, name, *args):
    """A library entry on the current stream of CUDA device `index`, whichever device is current."""
    fn = getattr(_LIB or _lib(), name)
    if index == _current_device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st != TM_OK:
        raise TmError(st, name)


def _on(x, name, index):
    """x lies on CUDA device `index` (-1: x is what the call goes by, and is not on one)."""
    if x.get_device() != index or index < 0:
        _cuda(x, name)
        raise ValueError(f"{name}: on {x.device}, the call is on cuda:{index}")


def _thd(x, name, index, T=None, H=None, d=None):
    """tm_tensor (as bytes) of an fp16 [T, H, d] operand on CUDA device `index`."""
    shape = x.shape
    if x.dtype is not _HALF or len(shape) != 3:
        raise ValueError(f"{name}: fp16 [T, H, d] expected")
    if x.get_device() != index or index < 0:
        _on(x, name, index)
    a, b, c = shape
    st, sh, sd = x.stride()
    if sd != 1 and c != 1:
        raise ValueError(f"{name}: innermost dimension must be contiguous")
    if (T is not None and a != T) or (H is not None and b != H) or (d is not None and c != d):
        raise ValueError(f"{name}: {(a, b, c)} where {(T, H, d)} is expected")
    return _tensor_bytes(x.data_ptr(), a, b, c, st, sh)


def _int32(t, name, index, n=None):
    """Device address of a contiguous int32 vector of at least n elements (None passes)."""
    if t is None:
        return None
    shape = t.shape
    if t.dtype is not _INT32 or len(shape) != 1 or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous int32 vector expected")
    if t.get_device() != index:
        _on(t, name, index)
    if n is not None and shape[0] < n:
        raise ValueError(f"{name}: at least {n} elements expected, got {shape[0]}")
    return t.data_ptr()


def _weight(w, name, index, d):
    if w is None:
        return None
    if w.dtype is not _HALF or w.shape != (d,) or not w.is_contiguous():
        raise ValueError(f"{name}: contiguous fp16 [{d}] expected")
    if w.get_device() != index:
        _on(w, name, index)
    return w.data_ptr()


def _table(block_table, kv, batch=None):
    """(address, row stride, columns) of an int32 [batch, columns] block table."""
    shape = block_table.shape
    if block_table.dtype is not _INT32 or len(shape) != 2:
        raise ValueError("block_table: int32 [batch, columns] expected")
    if block_table.get_device() != kv.index:
        _on(block_table, "block_table", kv.index)
    n, cols = shape
    stride, one = block_table.stride()
    if n < 1 or cols < 1 or (cols > 1 and one != 1):
        raise ValueError("block_table: at least one row and column, columns contiguous")
    if batch is not None and n < batch:
        raise ValueError(f"block_table: {batch} rows expected, got {n}")
    return block_table.data_ptr(), stride, cols


def _rope_call(name, q, k, out, rope, positions, pos_offset, *weights):
    dev = q.get_device()
    T, hq, d = q.shape
    if rope is not None and rope.d != d:
        raise ValueError(f"rope is for heads of {rope.d}, q has {d}")
    if out is None:
        out = (torch.empty(q.shape, dtype=q.dtype, device=q.device),
               None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device))
    elif isinstance(out, torch.Tensor):
        out = (out, None)
    qo, ko = out
    if k is not None and ko is None:
        raise ValueError("out: a pair (q, k) expected")
    qd, qod = _thd(q, "q", dev), _thd(qo, "q out", dev, T, hq, d)
    kd = kod = None
    if k is not None:
        kd, kod = _thd(k, "k", dev, T, None, d), _thd(ko, "k out", dev, T, k.shape[1], d)
    _call(dev, name, qd, kd, qod, kod, *weights, None if rope is None else rope.struct,
          _int32(positions, "positions", dev, T), int(pos_offset))
    return qo if k is None else (qo, ko)


def rope(q, k=None, *, rope, positions=None, pos_offset=0, out=None):
    """Rotary positions (tm_rope) of q, and of k in the same launch: fp16 [T,
    H, d], row t at position positions[t] + pos_offset (int32 [T]), or t +
    pos_offset without positions.  out: tensors to write, (q, k) themselves
    for in place.  Returns the rotated q, or (q, k)."""
    if rope is None:
        raise ValueError("rope: a Rope expected")
    return _rope_call("tm_rope", q, k, out, rope, positions, pos_offset)


def qk_norm_rope(q, k=None, *, q_weight, k_weight=None, eps=1e-6, rope=None, positions=None, pos_offset=0, out=None):
    """Norm of each head of q (and k), x / sqrt(mean(x^2) + eps) * weight
    (fp16 [d]), and the rotation, in one pass (tm_qk_norm_rope); rope None:
    the norm alone.  Other arguments as for rope()."""
    if q_weight is None or (k is not None and k_weight is None):
        raise ValueError("a weight for each of q and k expected")
    d = q.shape[2]
    return _rope_call("tm_qk_norm_rope", q, k, out, rope, positions, pos_offset,
                      _weight(q_weight, "q_weight", q.get_device(), d),
                      _weight(k_weight if k is not None else None, "k_weight", q.get_device(), d), float(eps))


def block_table_check(block_table, kv_lens, num_pages, page_size):
    """Raises ValueError where a host block table (int32 [batch, columns])
    does not hold kv_lens[b] tokens of each sequence in pages 0 ..
    num_pages - 1 (tm_block_table_check): the test that the kernels make of
    each page, before anything is launched."""
    # to 32 bits: what lies outside is no page, and longer than any table
    t, n = (torch.as_tensor(x, dtype=torch.int64, device="cpu").clamp(-1, 2 ** 31 - 1).to(torch.int32).contiguous()
            for x in (block_table, kv_lens))
    if t.dim() != 2 or n.dim() != 1 or n.shape[0] > t.shape[0]:
        raise ValueError("block_table [batch, columns] and kv_lens [batch] expected")
    bad = (ctypes.c_int32 * 2)(-1, -1)
    st = _lib().tm_block_table_check(t.data_ptr(), t.shape[1], t.shape[1], n.data_ptr(), n.shape[0], int(num_pages),
                                     int(page_size), bad)
    if st == TM_ERR_INVALID_ARG and bad[0] >= 0:
        raise ValueError(f"block_table: sequence {bad[0]}, column {bad[1]}: no usable page")
    _check(st, "tm_block_table_check")


def kv_append(k, v, kv, block_table, kv_lens, *, cu_seqlens=None, rope=None, pos_offset=0, k_weight=None, q=None,
              q_weight=None, eps=1e-6, q_out=None):
    """New tokens' k and v (fp16 [T, Hkv, d]) into the pages of kv, K normed
    (k_weight) and rotated (rope) on the way, and their queries q normed and
    rotated in the same launch (tm_kv_append).  kv_lens: int32 [batch], each
    sequence's own length AFTER the append; rows are packed by cu_seqlens
    (int32 [batch + 1]) or T / batch for each sequence.  pos_offset: length of
    a shared prefix.  Returns q_out (a new tensor if not given), or None
    without q."""
    dev = kv.index
    T = k.shape[0]
    batch = kv_lens.shape[0]
    ptr, stride, cols = _table(block_table, kv, batch)
    if cu_seqlens is None and T % max(batch, 1):
        raise ValueError(f"{T} rows for {batch} sequences: cu_seqlens expected")
    if rope is not None and rope.d != kv.d:
        raise ValueError(f"rope is for heads of {rope.d}, the cache holds {kv.d}")
    kd, vd = _thd(k, "k", dev, T, kv.H, kv.d), _thd(v, "v", dev, T, kv.H, kv.d)
    qd = qod = None
    if q is not None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        qd, qod = _thd(q, "q", dev, T, None, kv.d), _thd(q_out, "q_out", dev, T, q.shape[1], kv.d)
    elif q_out is not None or q_weight is not None:
        raise ValueError("q_out and q_weight come with q")
    _call(dev, "tm_kv_append", kd, vd, kv.struct, ptr, stride, cols, _int32(kv_lens, "kv_lens", dev),
          _int32(cu_seqlens, "cu_seqlens", dev, batch + 1), batch, None if rope is None else rope.struct, int(pos_offset),
          qd, qod, _weight(q_weight, "q_weight", dev, kv.d), _weight(k_weight, "k_weight", dev, kv.d),
          float(eps))
    return q_out


def kv_gather(kv, block_table, cu_seqlens_k, *, out):
    """The cached rows of each sequence as contiguous fp16 (tm_kv_gather): out
    = (k, v) [T, Hkv, d], rows cu_seqlens_k[b] .. cu_seqlens_k[b + 1] (int32
    [batch + 1]) sequence b's tokens in order: the keys and values of attn_fwd
    with cu_seqlens_k.  Returns out."""
    k, v = out
    dev = kv.index
    batch = cu_seqlens_k.shape[0] - 1
    if batch < 1:
        raise ValueError("cu_seqlens_k: int32 [batch + 1] expected")
    ptr, stride, cols = _table(block_table, kv, batch)
    kd, vd = _thd(k, "k", dev, None, kv.H, kv.d), _thd(v, "v", dev, k.shape[0], kv.H, kv.d)
    _call(dev, "tm_kv_gather", kv.struct, ptr, stride, cols, _int32(cu_seqlens_k, "cu_seqlens_k", dev), batch,
          kd, vd)
    return out


def shared_prefix_workspace_bytes(kv, batch, T, Hq, *, max_seqlen=None, prefix_len=0, max_kv_len):
    """Bytes of the workspace attn_shared_prefix needs for these sizes."""
    if batch < 1:
        raise ValueError("at least one sequence expected")
    n = int(_lib().tm_attn_shared_prefix_workspace(int(T), int(Hq), kv.H, kv.d, int(batch),
                                                   int(-(-T // batch) if max_seqlen is None else min(max_seqlen, T)),
                                                   int(prefix_len), int(max_kv_len)))
    if n < 0:
        raise ValueError("bad sizes")
    return n


def attn_shared_prefix(q, kv, block_table, kv_lens, *, prefix_pages=None, prefix_len=0, cu_seqlens=None,
                       max_seqlen=None, max_kv_len=None, causal=True, workspace=None, out=None):
    """Attention of a batch over a paged cache (tm_attn_shared_prefix): q fp16
    [T, Hq, d], packed by cu_seqlens (int32 [batch + 1]; max_seqlen bounds the
    rows of a sequence) or T / batch rows each.  Every row sees the prefix_len
    tokens in prefix_pages (int32), read once for the whole batch, and, bottom-right
    causal, its sequence's own kv_lens[b] tokens (int32 [batch]) in
    block_table's pages.  max_kv_len: a bound on kv_lens (default: what the
    table holds) that sizes the launch, so it may stay while a captured graph's
    kv_lens grow.  workspace: uint8, shared_prefix_workspace_bytes(...), one
    for each call that may run at the same time; allocated here when None.
    Returns out (a new tensor if not given)."""
    dev = kv.index
    T, Hq = q.shape[0], q.shape[1]
    batch = kv_lens.shape[0]
    if batch < 1:
        raise ValueError("kv_lens: int32 [batch] expected")
    ptr, stride, cols = _table(block_table, kv, batch)
    if max_kv_len is None:
        max_kv_len = cols * kv.page_size
    if cu_seqlens is None:
        if T % batch:
            raise ValueError(f"{T} rows for {batch} sequences: cu_seqlens expected")
        max_seqlen = T // batch
    elif max_seqlen is None:
        raise ValueError("max_seqlen comes with cu_seqlens")
    else:
        max_seqlen = min(max_seqlen, T)
    if Hq % kv.H:
        raise ValueError(f"{Hq} query heads over {kv.H} K/V heads")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if workspace is None:
        workspace = torch.empty(shared_prefix_workspace_bytes(kv, batch, T, Hq, max_seqlen=max_seqlen,
                                                              prefix_len=prefix_len, max_kv_len=max_kv_len),
                                dtype=torch.uint8, device=kv.device)
    elif workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError(f"workspace: contiguous uint8 on {kv.device} expected")
    qd, od = _thd(q, "q", dev, T, Hq, kv.d), _thd(out, "out", dev, T, Hq, kv.d)
    _call(dev, "tm_attn_shared_prefix", qd, kv.struct, od, ptr, stride, cols,
          _int32(kv_lens, "kv_lens", dev), _int32(cu_seqlens, "cu_seqlens", dev, batch + 1), batch, int(max_seqlen),
          _int32(prefix_pages, "prefix_pages", dev, -(-int(prefix_len) // kv.page_size)) if prefix_len else None,
          int(prefix_len), int(max_kv_len), int(bool(causal)), workspace.data_ptr(), workspace.numel())
    return out


def probe_rates():
    """Instruction rates behind the kernels' secondary bounds, measured on the
    current GPU (see tm_probe_rates in include/tm.h): cycles per warp
    instruction per SM sub-partition for MUFU ex2, cvt int32->fp32 and the
    kernels' exact conversion; cycles per tcgen05 MMA (f16 M128N128K16, i8
    M128N128K32) on one SM."""
    lib = _lib()
    n = int(lib.tm_probe_scratch_bytes())
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = (ctypes.c_double * 5)()
    _check(lib.tm_probe_rates(out, 5, _ptr(scratch), n, _stream()), "tm_probe_rates")
    keys = ("ex2_cycles_per_warp_instr", "cvt_s32_f32_cycles_per_warp_instr", "magic_conversion_cycles_per_warp_value",
            "mma_f16_m128n128k16_cycles", "mma_i8_m128n128k32_cycles")
    return dict(zip(keys, list(out)))


def selftest_wait_timeout(limit_ns=1_000_000):
    """Launch the bounded-wait self-test (a wait that must time out)."""
    _check(_lib().tm_selftest_wait_timeout(int(limit_ns), _stream()), "tm_selftest_wait_timeout")


def get_device_error():
    return int(_lib().tm_get_device_error(_stream()))


def sm_scale(d):
    return 1.0 / math.sqrt(d)
