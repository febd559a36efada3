"""Thin Python binding of libfattn (ctypes): argument marshalling only.

Every step of the computation runs in the library's CUDA kernels; this module
checks tensor shapes/dtypes, allocates outputs with PyTorch when the caller
does not pass them, and forwards raw device pointers and the current CUDA
stream. There is no fallback: if ``libfattn.so`` is missing or fails to load,
every call raises.

``stream=s`` runs a call on another stream than the current one. Workspaces that are not passed then come
from the memory of ``s``; outputs that are not passed come from the current stream's, as the caller's own tensors
do, so ``s`` has to be ordered behind the current stream (``s.wait_stream``) as for the inputs.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfattn.so")

FATTN_OK = 0
FATTN_ERR_INVALID_ARG = 1
FATTN_ERR_UNSUPPORTED = 2
FATTN_ERR_WORKSPACE = 3
FATTN_ERR_CUDA = 4
FATTN_ERR_TIMEOUT = 5
FATTN_ERR_DEVICE_CHECK = 6
FATTN_BF16 = 0
FATTN_FP32 = 1

# Every entry point declared in include/fattn.h: name -> (restype, argtypes)
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
SIGNATURES = {
    "fattn_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _i, _vp]),
    "fattn_fwd_block_sparse": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _vp]),
    "fattn_fwd_masked": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, ctypes.c_longlong,
                              ctypes.c_longlong, _i, _vp]),
    "fattn_fwd_fp8": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _f, _f, _f, _vp]),
    "fattn_fwd_paged": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i, _f,
                             _vp]),
    "fattn_bwd_workspace_size": (_sz, [_i, _i, _i]),
    "fattn_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]),
    "fattn_decode_workspace_size": (_sz, [_i, _i, _i, _i]),
    "fattn_decode_paged": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _sz,
                                _vp]),
    "fattn_decode_paged_static": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f,
                                       _vp]),
    "fattn_merge_partials": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "fattn_status_string": (ctypes.c_char_p, [_i]),
    "fattn_debug_read_status": (_i, [_vp]),
    "fattn_debug_set_wait_limit": (None, [ctypes.c_ulonglong, _i]),
}

# Every entry point declared in include/fattn_ops.h
_ll = ctypes.c_longlong
SIGNATURES_OPS = {
    "fattn_rope": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _ll, _ll, _ll, _ll, _ll, _ll, _ll, _ll,
                        _i, _i, _f, _i, _vp]),
    "fattn_rope_append_paged": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                                     _i, _i, _ll, _ll, _ll, _ll, _ll, _ll, _i, _f, _vp]),
    "fattn_fwd_shaped": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _f, _vp, _i, _vp, _vp, _vp]),
    "fattn_fwd_paged_shaped_workspace_size": (_sz, [_i, _i, _i, _i]),
    "fattn_fwd_paged_shaped": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i, _f,
                                    _f, _vp, _i, _vp, _vp, _i, _vp, _sz, _vp]),
    "fattn_bwd_shaped_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "fattn_bwd_shaped": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _f, _vp, _i,
                              _vp, _vp, _vp, _sz, _vp]),
    "fattn_decode_paged_shaped": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _f, _vp,
                                       _i, _vp, _sz, _vp]),
    "fattn_key_weights_paged": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _ll, _ll, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                                     _i, _i, _f, _f, _vp, _i, _f, _vp]),
    "fattn_evict_paged": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i,
                               _vp]),
}

_lib = None


class FattnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} (status {status})")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfattn.so and declare its C signatures; raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libfattn.so not found at {path}: build it with __graft_entry__.build() "
                           "or python -m exact_tiled_attention_fattn_gb300.build")
    lib = ctypes.CDLL(path)
    for name, (res, args) in {**SIGNATURES, **SIGNATURES_OPS}.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().fattn_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != FATTN_OK:
        raise FattnError(fn, status)


def _stream_handle(stream) -> int:
    if stream is None:  # the handle without a Stream object around it (0.3 us against 2.9)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if stream.device.index != torch.cuda.current_device():
        raise ValueError(f"stream is on {stream.device} but the current CUDA device is cuda:{torch.cuda.current_device()}")
    return int(stream.cuda_stream)


def _scratch(need: int, device, stream):
    """A workspace that the caller never sees, from the memory of the stream that the call runs on: dropped at return, it
    goes to what that stream does next. (From the current stream's memory the next tensor there could have it
    while ``stream`` still writes to it.)"""
    if stream is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(max(need, 1), dtype=torch.uint8, device=device)


def _ptr(t):
    """Address for a c_void_p argument (an int: ctypes converts it without an object of its own)."""
    return None if t is None else t.data_ptr()


def _dtype_code(dt) -> int:
    if dt == torch.bfloat16:
        return FATTN_BF16
    if dt == torch.float32:
        return FATTN_FP32
    raise TypeError(f"unsupported dtype {dt}: bf16 or fp32 only")


def _need_cuda(*ts, contiguous: bool = True):
    """All given tensors are contiguous CUDA tensors on one device, the current one
    (the library launches on the current device, so a tensor elsewhere would be an
    invalid address there). ``contiguous=False``: for calls that take strides."""
    dev = -1
    for t in ts:
        if t is None:
            continue
        d = t.get_device()
        if d < 0:
            raise ValueError("all tensors must be CUDA tensors")
        if contiguous and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
        if d != dev:
            if dev >= 0:
                raise ValueError(f"all tensors must be on one device (got cuda:{dev} and {t.device})")
            dev = d
    if dev >= 0 and dev != torch.cuda.current_device():
        raise ValueError(f"tensors are on cuda:{dev} but the current CUDA device is cuda:{torch.cuda.current_device()}; "
                         f"call under torch.cuda.device({dev})")


def _expect(t, shape, name, dtype=None):
    """Shape (and dtype) check of an argument the library will read or write in full."""
    if t is None:
        return
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def fwd(q, k, v, causal: bool = False, scale: float | None = None, cu_seqlens=None, max_seqlen: int | None = None,
        out=None, lse=None, want_lse: bool = True, stream=None):
    """Prefill attention. Dense q [B,N,Hq,d] / k,v [B,N,Hkv,d]; varlen q [T,Hq,d] with
    int32 ``cu_seqlens`` [B+1] on the device and ``max_seqlen`` (host int).
    Returns (O, lse): lse is [B,Hq,N] (dense) or [Hq,T] (varlen), fp32, natural log.
    """
    lib = load_library()
    _need_cuda(q, k, v, cu_seqlens, out, lse)
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k and v must share a dtype")
    d = q.shape[-1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if cu_seqlens is None:
        if q.dim() != 4:
            raise ValueError("dense q must be [B, N, Hq, d]")
        B, N, Hq, _ = q.shape
        if k.dim() != 4:
            raise ValueError("dense k must be [B, N, Hkv, d]")
        Hkv = k.shape[2]
        kv_shape, o_shape = (B, N, Hkv, d), (B, N, Hq, d)
        T = B * N
        lse_shape = (B, Hq, N)
    else:
        if q.dim() != 3 or max_seqlen is None:
            raise ValueError("varlen q must be [T, Hq, d] and max_seqlen must be given")
        if cu_seqlens.dtype != torch.int32:
            raise TypeError("cu_seqlens must be int32")
        T, Hq, _ = q.shape
        if k.dim() != 3:
            raise ValueError("varlen k must be [T, Hkv, d]")
        Hkv = k.shape[1]
        kv_shape, o_shape = (T, Hkv, d), (T, Hq, d)
        B = cu_seqlens.numel() - 1
        N = int(max_seqlen)
        lse_shape = (Hq, T)
    _expect(k, kv_shape, "k")
    _expect(v, kv_shape, "v")
    _expect(out, o_shape, "out", q.dtype)
    _expect(lse, lse_shape, "lse", torch.float32)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
    st = lib.fattn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, N, d, 1 if causal else 0,
                       float(scale), _ptr(cu_seqlens), T if cu_seqlens is not None else 0, _dtype_code(q.dtype),
                       _stream_handle(stream))
    _check("fattn_fwd", st)
    return out, lse


SPARSE_BLOCK = 128  # FATTN_SPARSE_BLOCK: rows/keys per block-mask entry


def fwd_block_sparse(q, k, v, block_mask, causal: bool = False, scale: float | None = None, out=None, lse=None,
                     want_lse: bool = True, stream=None):
    """Prefill restricted by a block mask. q [B,N,Hq,d], k/v [B,N,Hkv,d] bf16;
    block_mask uint8 [mask_heads, nb, nb] on the device, nb = ceil(N/128), mask_heads 1 or Hq.
    Returns (O, lse [B,Hq,N]); rows that keep no key get O = 0, lse = -inf."""
    lib = load_library()
    _need_cuda(q, k, v, block_mask, out, lse)
    if not (q.dtype == k.dtype == v.dtype == torch.bfloat16):
        raise TypeError("block-sparse prefill takes bf16 q, k, v")
    if block_mask.dtype != torch.uint8 or block_mask.dim() != 3:
        raise TypeError("block_mask must be uint8 [mask_heads, nb, nb]")
    B, N, Hq, d = q.shape
    if k.dim() != 4:
        raise ValueError("k must be [B, N, Hkv, d]")
    _expect(k, (B, N, k.shape[2], d), "k")
    _expect(v, k.shape, "v")
    _expect(out, q.shape, "out", q.dtype)
    _expect(lse, (B, Hq, N), "lse", torch.float32)
    nb = -(-N // SPARSE_BLOCK)
    if block_mask.shape[1] != nb or block_mask.shape[2] != nb:
        raise ValueError(f"block_mask must be [mask_heads, {nb}, {nb}]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    st = lib.fattn_fwd_block_sparse(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, k.shape[2], N, d,
                                    1 if causal else 0, float(scale), _ptr(block_mask), block_mask.shape[0],
                                    _stream_handle(stream))
    _check("fattn_fwd_block_sparse", st)
    return out, lse


def fwd_masked(q, k, v, mask, causal: bool = False, scale: float | None = None, out=None, lse=None,
               want_lse: bool = True, stream=None):
    """Prefill with an additive bf16 mask: O = softmax(scale Q K^T + M) V.
    q [B,N,Hq,d], k/v [B,N,Hkv,d] bf16; mask [Bm, Hm, N, L] bf16 on the device with
    Bm in {1, B}, Hm in {1, Hq} (size 1 is shared) and row length L >= N, L a multiple of 8
    (entries past N are ignored). Returns (O, lse [B,Hq,N]); a row with no key gets
    O = 0, lse = -inf."""
    lib = load_library()
    _need_cuda(q, k, v, mask, out, lse)
    if not (q.dtype == k.dtype == v.dtype == mask.dtype == torch.bfloat16):
        raise TypeError("masked prefill takes bf16 q, k, v and mask")
    if q.dim() != 4 or k.dim() != 4 or mask.dim() != 4:
        raise ValueError("q [B,N,Hq,d], k [B,N,Hkv,d] and mask [Bm,Hm,N,L] expected")
    B, N, Hq, d = q.shape
    _expect(k, (B, N, k.shape[2], d), "k")
    _expect(v, k.shape, "v")
    _expect(out, q.shape, "out", q.dtype)
    _expect(lse, (B, Hq, N), "lse", torch.float32)
    Bm, Hm, Nm, L = mask.shape
    if Bm not in (1, B) or Hm not in (1, Hq) or Nm != N or L < N or L % 8:
        raise ValueError(f"mask must be [1 or {B}, 1 or {Hq}, {N}, L] with L >= {N}, L % 8 == 0")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    sb = 0 if Bm == 1 else Hm * N * L
    sh = 0 if Hm == 1 else N * L
    st = lib.fattn_fwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, k.shape[2], N, d,
                              1 if causal else 0, float(scale), _ptr(mask), sb, sh, L,
                              _stream_handle(stream))
    _check("fattn_fwd_masked", st)
    return out, lse


def fwd_fp8(q8, k8, v8, q_descale: float, k_descale: float, v_descale: float, causal: bool = False,
            scale: float | None = None, out=None, lse=None, want_lse: bool = True, stream=None):
    """FP8 prefill. q8 [B,N,Hq,d], k8/v8 [B,N,Hkv,d] E4M3 (torch.float8_e4m3fn or uint8 codes),
    d = 128; the inputs are descale * e4m3. Returns (O bf16 [B,N,Hq,d], lse [B,Hq,N])."""
    lib = load_library()
    _need_cuda(q8, k8, v8, out, lse)
    for t in (q8, k8, v8):
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
            raise TypeError("fp8 prefill takes E4M3 tensors (float8_e4m3fn or uint8 codes)")
    if q8.dim() != 4 or k8.dim() != 4:
        raise ValueError("q [B,N,Hq,d] and k [B,N,Hkv,d] expected")
    B, N, Hq, d = q8.shape
    _expect(k8, (B, N, k8.shape[2], d), "k")
    _expect(v8, k8.shape, "v")
    _expect(out, q8.shape, "out", torch.bfloat16)
    _expect(lse, (B, Hq, N), "lse", torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty(q8.shape, dtype=torch.bfloat16, device=q8.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q8.device)
    st = lib.fattn_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(out), _ptr(lse), B, Hq, k8.shape[2], N, d,
                           1 if causal else 0, float(scale), float(q_descale), float(k_descale), float(v_descale),
                           _stream_handle(stream))
    _check("fattn_fwd_fp8", st)
    return out, lse


def fwd_paged(q, kcache, vcache, block_table, seqlens_k, cu_seqlens_q, max_seqlen_q: int, causal: bool = True,
              scale: float | None = None, out=None, lse=None, want_lse: bool = True, stream=None):
    """Prefill of query chunks against a paged KV cache. q [Tq,Hq,d] bf16 packed by
    int32 ``cu_seqlens_q`` [B+1]; chunk b holds the last Lq_b positions of sequence b's
    ``seqlens_k[b]`` context tokens; kcache/vcache [pages, page_size, Hkv, d] bf16;
    block_table int32 [B, max_pages_per_seq]. Returns (O [Tq,Hq,d], lse [Hq,Tq])."""
    lib = load_library()
    _need_cuda(q, kcache, vcache, block_table, seqlens_k, cu_seqlens_q, out, lse)
    if not (q.dtype == kcache.dtype == vcache.dtype == torch.bfloat16):
        raise TypeError("paged prefill takes bf16 q and caches")
    if block_table.dtype != torch.int32 or seqlens_k.dtype != torch.int32 or cu_seqlens_q.dtype != torch.int32:
        raise TypeError("block_table, seqlens_k and cu_seqlens_q must be int32")
    if q.dim() != 3 or kcache.dim() != 4:
        raise ValueError("q must be [Tq, Hq, d] and kcache [pages, page_size, Hkv, d]")
    Tq, Hq, d = q.shape
    num_pages, page_size, Hkv, _ = kcache.shape
    B = cu_seqlens_q.numel() - 1
    _expect(kcache, (num_pages, page_size, Hkv, d), "kcache")
    _expect(vcache, kcache.shape, "vcache")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must be [{B}, max_pages_per_seq]")
    _expect(seqlens_k, (B,), "seqlens_k")
    _expect(out, q.shape, "out", q.dtype)
    _expect(lse, (Hq, Tq), "lse", torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((Hq, Tq), dtype=torch.float32, device=q.device)
    st = lib.fattn_fwd_paged(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(block_table), _ptr(seqlens_k),
                             _ptr(cu_seqlens_q), _ptr(out), _ptr(lse), B, Hq, Hkv, d, page_size,
                             block_table.shape[1], num_pages, Tq, int(max_seqlen_q), 1 if causal else 0,
                             float(scale), _stream_handle(stream))
    _check("fattn_fwd_paged", st)
    return out, lse


def bwd_workspace_size(B: int, Hq: int, N: int) -> int:
    return int(load_library().fattn_bwd_workspace_size(B, Hq, N))


def bwd(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None, dq=None, dk=None, dv=None,
        workspace=None, stream=None):
    """Attention backward. q, o, dout [B,N,Hq,d], k, v [B,N,Hkv,d] bf16; lse [B,Hq,N] fp32 from
    ``fwd`` on the same inputs. Returns (dq, dk, dv) in the input layouts (bf16)."""
    lib = load_library()
    _need_cuda(q, k, v, o, lse, dout, dq, dk, dv, workspace)
    if not (q.dtype == k.dtype == v.dtype == o.dtype == dout.dtype == torch.bfloat16):
        raise TypeError("backward takes bf16 q, k, v, o and dout")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, N, Hq, d] and k [B, N, Hkv, d]")
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    _expect(k, (B, N, Hkv, d), "k")
    _expect(v, k.shape, "v")
    _expect(o, q.shape, "o")
    _expect(dout, q.shape, "dout")
    _expect(lse, (B, Hq, N), "lse", torch.float32)
    _expect(dq, q.shape, "dq", q.dtype)
    _expect(dk, k.shape, "dk", q.dtype)
    _expect(dv, k.shape, "dv", q.dtype)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = bwd_workspace_size(B, Hq, N)
    if workspace is None:
        workspace = _scratch(need, q.device, stream)
    st = lib.fattn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                       B, Hq, Hkv, N, d, 1 if causal else 0, float(scale), _ptr(workspace),
                       workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check("fattn_bwd", st)
    return dq, dk, dv


def decode_workspace_size(B: int, Hq: int, d: int, num_splits: int) -> int:
    return int(load_library().fattn_decode_workspace_size(B, Hq, d, num_splits))


def choose_num_splits(batch: int, hkv: int, max_pages_per_seq: int, num_sms: int | None = None,
                      chunk_pages: int = 256) -> int:
    """A split count that cuts contexts into ~``chunk_pages``-page chunks and gives at
    least two work items per SM over the batch. Larger chunks amortise each item's
    fixed cost (Q load, pipeline fill, partial write); smaller ones balance better.
    On the 8 x 64k-context decode workload, 256-page chunks (16 splits) read the KV
    cache at 85.6 % of the measured HBM bandwidth against 81 % for 128-page chunks
    (32 splits), 83 % for 12 splits and 63 % for 8."""
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    by_chunk = -(-max_pages_per_seq // chunk_pages)
    by_fill = -(-2 * num_sms // max(1, batch * hkv))
    return max(1, min(max_pages_per_seq, max(by_chunk, by_fill)))


def decode_paged(q, kcache, vcache, block_table, seqlens, num_splits: int, scale: float | None = None,
                 out=None, lse=None, workspace=None, want_lse: bool = True, stream=None):
    """Split-KV paged decode. q [B,Hq,d] bf16; kcache/vcache [pages, page_size, Hkv, d] bf16;
    block_table int32 [B, max_pages_per_seq]; seqlens int32 [B]. Returns (O [B,Hq,d], lse [B,Hq])."""
    lib = load_library()
    _need_cuda(q, kcache, vcache, block_table, seqlens, out, lse, workspace)
    if block_table.dtype != torch.int32 or seqlens.dtype != torch.int32:
        raise TypeError("block_table and seqlens must be int32")
    if not (q.dtype == kcache.dtype == vcache.dtype == torch.bfloat16):
        raise TypeError("q, kcache and vcache must be bfloat16 (the decode kernels read bf16 only)")
    B, Hq, d = q.shape
    num_pages, page_size, Hkv, _ = kcache.shape
    _expect(kcache, (num_pages, page_size, Hkv, d), "kcache")
    _expect(vcache, kcache.shape, "vcache")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must be [{B}, max_pages_per_seq]")
    _expect(seqlens, (B,), "seqlens")
    _expect(out, q.shape, "out", q.dtype)
    _expect(lse, (B, Hq), "lse", torch.float32)
    maxp = block_table.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    need = decode_workspace_size(B, Hq, d, num_splits)
    if workspace is None:
        workspace = _scratch(need, q.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib.fattn_decode_paged(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(block_table), _ptr(seqlens), num_splits,
                                _ptr(out), _ptr(lse), B, Hq, Hkv, d, page_size, maxp, num_pages, float(scale),
                                _ptr(workspace), ws_bytes, _stream_handle(stream))
    _check("fattn_decode_paged", st)
    return out, lse


# Size of the fixed device scratch behind decode_paged_static (FATTN_DECODE_STATIC_SCRATCH_BYTES).
DECODE_STATIC_SCRATCH_BYTES = 32 << 20


def decode_paged_static(q, kcache, vcache, block_table, seqlens, num_splits: int, scale: float | None = None,
                        out=None, lse=None, want_lse: bool = True, stream=None):
    """decode_paged for callers that cannot allocate a device workspace: the split
    partials live in the library's fixed 32 MiB device scratch. Calls share that
    scratch, so calls that overlap on the GPU race; the first call on a device
    looks up the scratch address and should come before any stream capture."""
    lib = load_library()
    _need_cuda(q, kcache, vcache, block_table, seqlens, out, lse)
    if block_table.dtype != torch.int32 or seqlens.dtype != torch.int32:
        raise TypeError("block_table and seqlens must be int32")
    if not (q.dtype == kcache.dtype == vcache.dtype == torch.bfloat16):
        raise TypeError("q, kcache and vcache must be bfloat16 (the decode kernels read bf16 only)")
    B, Hq, d = q.shape
    num_pages, page_size, Hkv, _ = kcache.shape
    _expect(kcache, (num_pages, page_size, Hkv, d), "kcache")
    _expect(vcache, kcache.shape, "vcache")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must be [{B}, max_pages_per_seq]")
    _expect(seqlens, (B,), "seqlens")
    _expect(out, q.shape, "out", q.dtype)
    _expect(lse, (B, Hq), "lse", torch.float32)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    st = lib.fattn_decode_paged_static(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(block_table), _ptr(seqlens),
                                       num_splits, _ptr(out), _ptr(lse), B, Hq, Hkv, d, page_size,
                                       block_table.shape[1], num_pages, float(scale),
                                       _stream_handle(stream))
    _check("fattn_decode_paged_static", st)
    return out, lse


def split_workspace(workspace, B: int, Hq: int, d: int, num_splits: int):
    """Views (lse_part [B,Hq,S], o_part [B,Hq,S,d]) of a decode workspace (fp32)."""
    rows = B * Hq * num_splits
    lse_bytes = (rows * 4 + 255) // 256 * 256
    flat = workspace.view(torch.uint8)
    lse_part = flat[: rows * 4].view(torch.float32).view(B, Hq, num_splits)
    o_part = flat[lse_bytes: lse_bytes + rows * d * 4].view(torch.float32).view(B, Hq, num_splits, d)
    return lse_part, o_part


def merge_partials(o_part, lse_part, out_dtype=torch.bfloat16, out=None, lse=None, want_lse: bool = True,
                   stream=None):
    """Merge split partials: o_part [B,Hq,S,d] fp32, lse_part [B,Hq,S] fp32 -> (O [B,Hq,d], lse [B,Hq])."""
    lib = load_library()
    _need_cuda(o_part, lse_part, out, lse)
    B, Hq, S, d = o_part.shape
    _expect(lse_part, (B, Hq, S), "lse_part", torch.float32)
    if o_part.dtype != torch.float32:
        raise TypeError("o_part must be float32")
    _expect(out, (B, Hq, d), "out")
    _expect(lse, (B, Hq), "lse", torch.float32)
    if out is None:
        out = torch.empty((B, Hq, d), dtype=out_dtype, device=o_part.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=o_part.device)
    st = lib.fattn_merge_partials(_ptr(o_part), _ptr(lse_part), _ptr(out), _ptr(lse), B, Hq, S, d,
                                  _dtype_code(out.dtype), _stream_handle(stream))
    _check("fattn_merge_partials", st)
    return out, lse


def debug_read_status(stream=None) -> int:
    """Synchronise the stream, then read and clear the device status word."""
    return int(load_library().fattn_debug_read_status(_stream_handle(stream)))


def debug_set_wait_limit(limit_ns: int = 0, stall: bool = False) -> None:
    """Test hook: limit of every pipeline wait in later tensor-core launches (0 = the
    default, 2 s); with ``stall`` their softmax / element-wise warps first wait on a
    barrier nothing arrives on, so each launch times out (FATTN_ERR_TIMEOUT) and
    returns without writing its outputs. Reset with debug_set_wait_limit(0, False)."""
    load_library().fattn_debug_set_wait_limit(int(limit_ns), 1 if stall else 0)


# ------------------------------------------------------------------ rotary positions
_INT_MAX = 2 ** 31 - 1


def _int(x, name: str) -> int:
    """A C int argument (ctypes would take the lowest 32 bits of a larger one)."""
    x = int(x)
    if not -_INT_MAX - 1 <= x <= _INT_MAX:
        raise ValueError(f"{name} must fit 32 bits, got {x}")
    return x


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_length: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """(inv_freq float64 [rotary_dim / 2], amplitude) for ``rope``: angle per position of
    pair i is base^(-2i / rotary_dim), then, for contexts ``factor`` times longer than trained,

    * ``scaling="linear"``: every frequency divided by ``factor``;
    * ``scaling="base"``: the base raised so that the lowest frequency is divided by ``factor``
      and the highest stays;
    * ``scaling="bands"``: pairs that turn more than ``beta_fast`` times over ``original_length``
      keep their frequency, pairs that turn less than ``beta_slow`` times have it divided by
      ``factor``, a linear ramp over the pair index between; the amplitude is 0.1 ln(factor) + 1.
    """
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be positive and even")
    if not (base > 0 and factor >= 1.0):
        raise ValueError("base must be positive and factor at least 1")
    half = rotary_dim // 2
    i = torch.arange(half, dtype=torch.float64)
    if scaling == "base" and half > 1:
        base = base * factor ** (half / (half - 1))
    f = float(base) ** (-i / half)
    amplitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":
        def pair(turns):  # index (real) of the pair that turns `turns` times over the original length
            return half * math.log(original_length / (2.0 * math.pi * turns)) / math.log(base)
        lo, hi = math.floor(pair(beta_fast)), math.ceil(pair(beta_slow))  # (outside the head too: the ramp keeps its slope)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        f = f * (1.0 - ramp) + f / factor * ramp
        amplitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"unknown scaling {scaling!r}: None, 'linear', 'base' or 'bands'")
    return f.to(device) if device is not None else f, amplitude


def _row_strides(t, name):
    """(row stride, head stride) of [..., H, d] whose leading dimensions are one uniform run of rows."""
    if t.dim() not in (3, 4):
        raise ValueError(f"{name} must be [T, H, d] or [B, N, H, d]")
    stride = t.stride()
    if stride[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    row = stride[-3]
    if len(stride) == 4 and t.shape[0] > 1:
        if t.shape[1] == 1:
            row = stride[0]
        elif stride[0] != t.shape[1] * row:
            raise ValueError(f"{name}: the batch stride must be N row strides")
    return row, stride[-2]


def _no_overlap(t, name):
    """An output: distinct elements have distinct addresses."""
    row, head = _row_strides(t, name)
    extent = t.shape[-1]
    for stride, n in sorted([(row, t.shape[:-2].numel()), (head, t.shape[-2])]):
        if n > 1:
            if stride < extent:
                raise ValueError(f"{name}: rows or heads overlap")
            extent += (n - 1) * stride


def _check_freq(inv_freq, d):
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous float64 vector of rotary_dim / 2 frequencies")
    rot = 2 * inv_freq.numel()
    if rot > d:
        raise ValueError(f"inv_freq has {inv_freq.numel()} frequencies for heads of {d} elements")
    return rot


def rope(q, k=None, inv_freq=None, positions=None, interleaved: bool = False, amplitude: float = 1.0,
         inverse: bool = False, out_q=None, out_k=None, stream=None):
    """Rotary positions on q [T,Hq,d] or [B,N,Hq,d] (bf16 or fp32; any row and head strides, so
    slices of a packed projection serve as they are) and, in the same launch, k with the same
    leading dimensions. ``inv_freq`` float64 [rotary_dim / 2] on the device (``rope_frequencies``);
    pairs are (i, i + rotary_dim / 2), or (2i, 2i + 1) if ``interleaved``; the rest of the head is
    copied. ``positions`` int32, [T] or [B,N]; None: the index along T (N). ``inverse=True`` with the
    other arguments unchanged is the gradient: it maps (dq', dk') to (dq, dk). ``out_q`` / ``out_k``
    may be q / k themselves. Returns q', or (q', k')."""
    lib = load_library()
    if inv_freq is None:
        raise ValueError("inv_freq must be given (rope_frequencies)")
    _need_cuda(q, k, inv_freq, positions, out_q, out_k, contiguous=False)
    if q.dim() not in (3, 4):
        raise ValueError("q must be [T, H, d] or [B, N, H, d]")
    code, d, lead = _dtype_code(q.dtype), q.shape[-1], tuple(q.shape[:-2])
    rot = _check_freq(inv_freq, d)
    if k is not None:
        if k.dtype != q.dtype:
            raise TypeError("q and k must share a dtype")
        if k.dim() != q.dim() or tuple(k.shape[:-2]) != lead or k.shape[-1] != d:
            raise ValueError("k must have q's leading dimensions and head size")
    elif out_k is not None:
        raise ValueError("out_k without k")
    if positions is not None:
        _expect(positions, lead, "positions", torch.int32)
        if not positions.is_contiguous():
            raise ValueError("positions must be contiguous")
    rows = math.prod(lead)
    if rows > _INT_MAX:
        raise ValueError("at most 2^31 - 1 rows")
    Hq, Hk = q.shape[-2], 0 if k is None else k.shape[-2]
    strides = [*_row_strides(q, "q")]
    if out_q is None:
        out_q = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        strides += [Hq * d, d]
    else:
        _expect(out_q, q.shape, "out_q", q.dtype)
        _no_overlap(out_q, "out_q")
        strides += _row_strides(out_q, "out_q")
    if k is None:
        strides += [0, 0, 0, 0]
    else:
        strides += _row_strides(k, "k")
        if out_k is None:
            out_k = torch.empty(k.shape, dtype=q.dtype, device=q.device)
            strides += [Hk * d, d]
        else:
            _expect(out_k, k.shape, "out_k", q.dtype)
            _no_overlap(out_k, "out_k")
            strides += _row_strides(out_k, "out_k")
    st = lib.fattn_rope(_ptr(q), _ptr(out_q), _ptr(k), _ptr(out_k), _ptr(positions), lead[-1] if rows else 1,
                        _ptr(inv_freq), rows, Hq, Hk, d, rot, *strides,
                        1 if interleaved else 0, 1 if inverse else 0, float(amplitude), code,
                        _stream_handle(stream))
    _check("fattn_rope", st)
    return out_q if k is None else (out_q, out_k)


def _check_paged_cache(kcache, vcache, block_table, B):
    if kcache.dim() != 4:
        raise ValueError("kcache must be [pages, page_size, Hkv, d]")
    if vcache is not None:
        _expect(vcache, kcache.shape, "vcache", kcache.dtype)
    if block_table.dtype != torch.int32:
        raise TypeError("block_table must be int32")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must be [{B}, max_pages_per_seq]")


def rope_append_paged(q, k, v, kcache, vcache, block_table, seqlens_k, cu_seqlens_q, inv_freq, positions=None,
                      interleaved: bool = False, amplitude: float = 1.0, out=None, stream=None):
    """One serving step before the attention: q [Tq,Hq,d] (or None) and k [Tq,Hkv,d] of new tokens
    rotated, k and v [Tq,Hkv,d] written into their slots of the paged cache, one launch. bf16; q, k and v
    may have any row and head strides. Chunks are packed as in ``fwd_paged`` (one token each for
    decoding): chunk b holds the last tokens of the ``seqlens_k[b]`` context tokens, the new ones
    included. ``positions`` int32 [Tq]; None: each token's index in its sequence. Rows past the last
    chunk are left alone. Returns the rotated q [Tq,Hq,d], packed (None without q)."""
    lib = load_library()
    _need_cuda(q, k, v, inv_freq, contiguous=False)
    _need_cuda(kcache, vcache, block_table, seqlens_k, cu_seqlens_q, positions, out)
    if not (k.dtype == v.dtype == kcache.dtype == vcache.dtype == torch.bfloat16) or (
            q is not None and q.dtype != torch.bfloat16):
        raise TypeError("rope_append_paged takes bf16 q, k, v and caches")
    if k.dim() != 3 or v.shape != k.shape:
        raise ValueError("k and v must be [Tq, Hkv, d]")
    Tq, Hkv, d = k.shape
    rot = _check_freq(inv_freq, d)
    if seqlens_k.dtype != torch.int32 or cu_seqlens_q.dtype != torch.int32:
        raise TypeError("seqlens_k and cu_seqlens_q must be int32")
    B = cu_seqlens_q.numel() - 1
    _expect(seqlens_k, (B,), "seqlens_k")
    _check_paged_cache(kcache, vcache, block_table, B)
    _expect(kcache, (*kcache.shape[:2], Hkv, d), "kcache")
    if positions is not None:
        _expect(positions, (Tq,), "positions", torch.int32)
    Hq = 0
    qs = (0, 0)
    if q is not None:
        if q.dim() != 3 or q.shape[0] != Tq or q.shape[2] != d:
            raise ValueError(f"q must be [{Tq}, Hq, {d}]")
        Hq = q.shape[1]
        qs = _row_strides(q, "q")
        _expect(out, q.shape, "out", q.dtype)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif out is not None:
        raise ValueError("out without q")
    st = lib.fattn_rope_append_paged(_ptr(q), _ptr(out), _ptr(k), _ptr(v), _ptr(kcache), _ptr(vcache),
                                     _ptr(block_table), _ptr(seqlens_k), _ptr(cu_seqlens_q), _ptr(positions),
                                     _ptr(inv_freq), B, Tq, Hq, Hkv, d, rot, kcache.shape[1], block_table.shape[1],
                                     kcache.shape[0], *qs, *_row_strides(k, "k"), *_row_strides(v, "v"),
                                     1 if interleaved else 0, float(amplitude), _stream_handle(stream))
    _check("fattn_rope_append_paged", st)
    return out


_sms: dict = {}


def _num_sms(device: int) -> int:
    """SM count of a device (a property of the machine, looked up once)."""
    if device not in _sms:
        _sms[device] = torch.cuda.get_device_properties(device).multi_processor_count
    return _sms[device]


# ------------------------------------------------------------------ shaped scores
def document_ranges(doc_ids, prefix_len=None):
    """Key ranges (key_begin, key_end), int32 [B, N], of packed documents: ``doc_ids`` [B, N] names
    each row's document, equal ids are contiguous; an id < 0 is padding, which sees nothing and is seen by
    nobody. Every row sees its document; with ``prefix_len`` (tokens of every document that all of
    it sees, an int) row i sees max(i + 1, document start + prefix_len), and without
    ``causal`` in the call. Made once per batch, for every layer."""
    if doc_ids.dim() != 2:
        raise ValueError("doc_ids must be [B, N]")
    B, N = doc_ids.shape
    i = torch.arange(N, device=doc_ids.device).expand(B, N)
    edge = torch.ones(B, N, dtype=torch.bool, device=doc_ids.device)
    edge[:, 1:] = doc_ids[:, 1:] != doc_ids[:, :-1]
    begin = torch.where(edge, i, 0).cummax(1)[0]
    last = torch.ones_like(edge)
    last[:, :-1] = edge[:, 1:]
    end = torch.where(last, i + 1, N).flip(1).cummin(1)[0].flip(1)
    if prefix_len is not None:
        end = torch.minimum(end, torch.maximum(i + 1, begin + int(prefix_len)))
    end = torch.where(doc_ids < 0, begin, end)
    return begin.to(torch.int32).contiguous(), end.to(torch.int32).contiguous()


def _check_shape(slopes, Hq, key_begin, key_end, range_shape):
    _need_cuda(slopes, key_begin, key_end)
    _expect(slopes, (Hq,), "slopes", torch.float32)
    _expect(key_begin, range_shape, "key_begin", torch.int32)
    _expect(key_end, range_shape, "key_end", torch.int32)


def fwd_shaped(q, k, v, causal: bool = False, scale: float | None = None, softcap: float = 0.0, slopes=None,
               window: int = 0, key_begin=None, key_end=None, out=None, lse=None, want_lse: bool = True, stream=None):
    """Prefill with shaped scores: s = scale q.k, then s = softcap tanh(s / softcap) (softcap > 0), then
    s -= slopes[h] |i - j| (slopes fp32 [Hq]); key j is visible iff j <= i (causal), |i - j| < window
    (window > 0) and key_begin[b, i] <= j < key_end[b, i] (int32 [B, N], non-decreasing along N:
    ``document_ranges``). q [B,N,Hq,d], k, v [B,N,Hkv,d] bf16, d 64 or 128. Returns (O, lse [B,Hq,N]); a row that
    sees no key gets O = 0, lse = -inf."""
    lib = load_library()
    _need_cuda(q, k, v, out, lse)
    if not (q.dtype == k.dtype == v.dtype == torch.bfloat16):
        raise TypeError("shaped prefill takes bf16 q, k, v")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q [B,N,Hq,d] and k [B,N,Hkv,d] expected")
    B, N, Hq, d = q.shape
    _expect(k, (B, N, k.shape[2], d), "k")
    _expect(v, k.shape, "v")
    _expect(out, q.shape, "out", q.dtype)
    _expect(lse, (B, Hq, N), "lse", torch.float32)
    _check_shape(slopes, Hq, key_begin, key_end, (B, N))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    st = lib.fattn_fwd_shaped(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, k.shape[2], N, d,
                              1 if causal else 0, float(scale), float(softcap), _ptr(slopes), _int(min(window, _INT_MAX), "window"),
                              _ptr(key_begin), _ptr(key_end), _stream_handle(stream))
    _check("fattn_fwd_shaped", st)
    return out, lse


def fwd_paged_shaped_workspace_size(total_q: int, Hq: int, d: int, num_splits: int) -> int:
    return int(load_library().fattn_fwd_paged_shaped_workspace_size(total_q, Hq, d, num_splits))


def choose_chunk_splits(batch: int, Hq: int, d: int, max_seqlen_q: int, max_context: int,
                        num_sms: int | None = None) -> int:
    """Split count of ``fwd_paged_shaped``, 16 at most: the S whose estimate is lowest, in units of a step of one SM
    over 128 keys (about 1.7 us): rounds of items over the SMs, each of its run's steps and 2 more, and for S > 1 the
    joining launch (4) with the fp32 partials' way through memory (1 per million elements).

    Measured, S = 1 against the choice: 16 queries over 32768 keys, 8 heads 476 -> 51 us (S 16); 256 over 32768, 32 heads
    673 -> 186 (4); 2 x 512 over 4096, 16 heads 74 -> 57 (2); 3 x 517 over 9000, 16 heads stay at 1 (135; 2: 147)."""
    items = batch * Hq * -(-max_seqlen_q // 256)
    if items <= 0:
        return 1
    if num_sms is None:
        num_sms = _num_sms(torch.cuda.current_device())
    if items >= 4 * num_sms:
        return 1
    steps, join = max_context / 128, batch * max_seqlen_q * Hq * d * 1e-6
    best, best_cost = 1, -(-items // num_sms) * (steps + 2)
    for S in range(2, min(16, -(-max_context // 128)) + 1):
        cost = -(-items * S // num_sms) * (steps / S + 2) + 4 + S * join
        if cost < best_cost:
            best, best_cost = S, cost
    return best


def fwd_paged_shaped(q, kcache, vcache, block_table, seqlens_k, cu_seqlens_q, max_seqlen_q: int, causal: bool = True,
                     scale: float | None = None, softcap: float = 0.0, slopes=None, window: int = 0, key_begin=None,
                     key_end=None, out=None, lse=None, want_lse: bool = True, num_splits: int | None = None,
                     workspace=None, stream=None):
    """``fwd_paged`` with the shaped scores of ``fwd_shaped``; a chunk's queries sit at the last positions
    of their sequence's context. key_begin / key_end int32 [Tq], keys of the row's sequence. ``num_splits`` cuts
    every query tile's keys into runs that are joined at the end (None: ``choose_chunk_splits``); their partials
    take a ``workspace`` of fwd_paged_shaped_workspace_size bytes (allocated when None).
    Returns (O [Tq,Hq,d], lse [Hq,Tq])."""
    lib = load_library()
    _need_cuda(q, kcache, vcache, block_table, seqlens_k, cu_seqlens_q, out, lse)
    if not (q.dtype == kcache.dtype == vcache.dtype == torch.bfloat16):
        raise TypeError("paged prefill takes bf16 q and caches")
    if seqlens_k.dtype != torch.int32 or cu_seqlens_q.dtype != torch.int32:
        raise TypeError("seqlens_k and cu_seqlens_q must be int32")
    if q.dim() != 3:
        raise ValueError("q must be [Tq, Hq, d]")
    Tq, Hq, d = q.shape
    B = cu_seqlens_q.numel() - 1
    _check_paged_cache(kcache, vcache, block_table, B)
    num_pages, page_size, Hkv, _ = kcache.shape
    _expect(kcache, (num_pages, page_size, Hkv, d), "kcache")
    _expect(seqlens_k, (B,), "seqlens_k")
    _expect(out, q.shape, "out", q.dtype)
    _expect(lse, (Hq, Tq), "lse", torch.float32)
    _check_shape(slopes, Hq, key_begin, key_end, (Tq,))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((Hq, Tq), dtype=torch.float32, device=q.device)
    if num_splits is None:
        context = block_table.shape[1] * page_size
        if window > 0:
            context = min(context, int(window) + int(max_seqlen_q))
        num_splits = choose_chunk_splits(B, Hq, d, int(max_seqlen_q), context)
    num_splits = _int(num_splits, "num_splits")
    _need_cuda(workspace)
    if workspace is None and num_splits > 1:
        workspace = _scratch(fwd_paged_shaped_workspace_size(Tq, Hq, d, num_splits), q.device, stream)
    st = lib.fattn_fwd_paged_shaped(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(block_table), _ptr(seqlens_k),
                                    _ptr(cu_seqlens_q), _ptr(out), _ptr(lse), B, Hq, Hkv, d, page_size,
                                    block_table.shape[1], num_pages, Tq, _int(max_seqlen_q, "max_seqlen_q"), 1 if causal else 0,
                                    float(scale), float(softcap), _ptr(slopes), _int(min(window, _INT_MAX), "window"), _ptr(key_begin),
                                    _ptr(key_end), num_splits, _ptr(workspace),
                                    0 if workspace is None else workspace.numel() * workspace.element_size(),
                                    _stream_handle(stream))
    _check("fattn_fwd_paged_shaped", st)
    return out, lse


def bwd_shaped_workspace_size(B: int, Hq: int, Hkv: int, N: int, d: int) -> int:
    return int(load_library().fattn_bwd_shaped_workspace_size(B, Hq, Hkv, N, d))


def bwd_shaped(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None, softcap: float = 0.0,
               slopes=None, window: int = 0, key_begin=None, key_end=None, dq=None, dk=None, dv=None, workspace=None,
               stream=None):
    """Gradients of ``fwd_shaped`` (same arguments; o and lse are its outputs) with respect to q, k and v;
    the slopes are constants. Returns (dq, dk, dv), bf16 in the input layouts."""
    lib = load_library()
    _need_cuda(q, k, v, o, lse, dout, dq, dk, dv, workspace)
    if not (q.dtype == k.dtype == v.dtype == o.dtype == dout.dtype == torch.bfloat16):
        raise TypeError("backward takes bf16 q, k, v, o and dout")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, N, Hq, d] and k [B, N, Hkv, d]")
    B, N, Hq, d = q.shape
    Hkv = k.shape[2]
    _expect(k, (B, N, Hkv, d), "k")
    _expect(v, k.shape, "v")
    _expect(o, q.shape, "o")
    _expect(dout, q.shape, "dout")
    _expect(lse, (B, Hq, N), "lse", torch.float32)
    _expect(dq, q.shape, "dq", q.dtype)
    _expect(dk, k.shape, "dk", q.dtype)
    _expect(dv, k.shape, "dv", q.dtype)
    _check_shape(slopes, Hq, key_begin, key_end, (B, N))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = _scratch(bwd_shaped_workspace_size(B, Hq, Hkv, N, d), q.device, stream)
    st = lib.fattn_bwd_shaped(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                              B, Hq, Hkv, N, d, 1 if causal else 0, float(scale), float(softcap), _ptr(slopes),
                              _int(min(window, _INT_MAX), "window"), _ptr(key_begin), _ptr(key_end), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check("fattn_bwd_shaped", st)
    return dq, dk, dv


def decode_paged_shaped(q, kcache, vcache, block_table, seqlens, num_splits: int, scale: float | None = None,
                        softcap: float = 0.0, slopes=None, window: int = 0, out=None, lse=None, workspace=None,
                        want_lse: bool = True, stream=None):
    """``decode_paged`` with the cap, distance bias and window of ``fwd_shaped`` (the query is the
    sequence's last token). With a window, num_splits cuts the pages that it touches: pass
    choose_num_splits their count, min(max_pages, (window + page_size - 2) // page_size + 1).
    Returns (O [B,Hq,d], lse [B,Hq])."""
    lib = load_library()
    _need_cuda(q, kcache, vcache, block_table, seqlens, out, lse, workspace)
    if not (q.dtype == kcache.dtype == vcache.dtype == torch.bfloat16):
        raise TypeError("q, kcache and vcache must be bfloat16 (the decode kernels read bf16 only)")
    if seqlens.dtype != torch.int32:
        raise TypeError("block_table and seqlens must be int32")
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, d]")
    B, Hq, d = q.shape
    _check_paged_cache(kcache, vcache, block_table, B)
    num_pages, page_size, Hkv, _ = kcache.shape
    _expect(kcache, (num_pages, page_size, Hkv, d), "kcache")
    _expect(seqlens, (B,), "seqlens")
    _expect(out, q.shape, "out", q.dtype)
    _expect(lse, (B, Hq), "lse", torch.float32)
    _check_shape(slopes, Hq, None, None, None)
    num_splits = _int(num_splits, "num_splits")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _scratch(decode_workspace_size(B, Hq, d, num_splits), q.device, stream)
    st = lib.fattn_decode_paged_shaped(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(block_table), _ptr(seqlens),
                                       num_splits, _ptr(out), _ptr(lse), B, Hq, Hkv, d, page_size,
                                       block_table.shape[1], num_pages, float(scale), float(softcap), _ptr(slopes),
                                       _int(min(window, _INT_MAX), "window"), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                       _stream_handle(stream))
    _check("fattn_decode_paged_shaped", st)
    return out, lse


# ------------------------------------------------------------------ a budget for the cache
def key_weights_paged(q, kcache, block_table, seqlens_k, cu_seqlens_q, max_seqlen_q: int, lse, weights=None,
                      decay: float = 1.0, causal: bool = True, scale: float | None = None, softcap: float = 0.0,
                      slopes=None, window: int = 0, out=None, stream=None):
    """Attention weight that cached tokens received: out[b, hkv, t] = decay * weights[b, hkv, t] + the sum over
    the heads of the group and the queries of chunk b of exp(s - lse), fp32 [B, Hkv, max_pages * page_size].
    q [Tq,Hq,d] and the chunk arguments as in ``fwd_paged``; ``lse`` [Hq,Tq] from the attention call, any strides
    (``lse.t()`` of ``decode_paged``). ``weights`` None starts from zero; ``out`` may be ``weights`` (which a call
    whose bounded waits ran out leaves partly updated). Slots past a sequence's length are 0, or, with ``out`` the
    same tensor as ``weights``, left as they are."""
    lib = load_library()
    _need_cuda(q, kcache, block_table, seqlens_k, cu_seqlens_q, weights, out)
    _need_cuda(lse, contiguous=False)
    if not (q.dtype == kcache.dtype == torch.bfloat16):
        raise TypeError("key_weights_paged takes bf16 q and cache")
    if seqlens_k.dtype != torch.int32 or cu_seqlens_q.dtype != torch.int32:
        raise TypeError("seqlens_k and cu_seqlens_q must be int32")
    if q.dim() != 3:
        raise ValueError("q must be [Tq, Hq, d]")
    Tq, Hq, d = q.shape
    B = cu_seqlens_q.numel() - 1
    _check_paged_cache(kcache, None, block_table, B)
    num_pages, page_size, Hkv, _ = kcache.shape
    _expect(kcache, (num_pages, page_size, Hkv, d), "kcache")
    _expect(seqlens_k, (B,), "seqlens_k")
    _expect(lse, (Hq, Tq), "lse", torch.float32)
    shape = (B, Hkv, block_table.shape[1] * page_size)
    _expect(weights, shape, "weights", torch.float32)
    _expect(out, shape, "out", torch.float32)
    _check_shape(slopes, Hq, None, None, None)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=q.device)
    st = lib.fattn_key_weights_paged(_ptr(q), _ptr(kcache), _ptr(block_table), _ptr(seqlens_k), _ptr(cu_seqlens_q),
                                     _ptr(lse), lse.stride(0), lse.stride(1), _ptr(weights), _ptr(out), B, Hq, Hkv, d,
                                     page_size, block_table.shape[1], num_pages, Tq, _int(max_seqlen_q, "max_seqlen_q"),
                                     1 if causal else 0, float(scale), float(softcap), _ptr(slopes), _int(min(window, _INT_MAX), "window"),
                                     float(decay), _stream_handle(stream))
    _check("fattn_key_weights_paged", st)
    return out


def evict_paged(kcache, vcache, block_table, seqlens, weights, keep: int, recent: int = 0, first: int = 0,
                dst_table=None, out_weights=None, out_seqlens=None, kept=None, stream=None):
    """Cuts every KV head of every sequence down to ``keep`` tokens: the first ``first``, the last ``recent`` and the
    heaviest of the others by ``weights`` fp32 [B,Hkv,max_pages*page_size] (``key_weights_paged``; ties to the lowest
    index). The kept tokens move, in order, to slots 0, 1, ... of the sequence's own pages, or of the unused pages
    ``dst_table`` int32 [B, dst_pages] of the same pool. Shared pages must not be evicted in place.
    Returns (seqlens [B], weights [B,Hkv,dst_pages*page_size], kept indices int32 [B,Hkv,keep], -1 past the end)."""
    lib = load_library()
    _need_cuda(kcache, vcache, block_table, seqlens, weights, dst_table, out_weights, out_seqlens, kept)
    if not (kcache.dtype == vcache.dtype == torch.bfloat16):
        raise TypeError("evict_paged takes bf16 caches")
    if seqlens.dtype != torch.int32:
        raise TypeError("seqlens must be int32")
    keep, recent, first = _int(keep, "keep"), _int(recent, "recent"), _int(first, "first")
    B = seqlens.numel()
    _expect(seqlens, (B,), "seqlens")
    _check_paged_cache(kcache, vcache, block_table, B)
    num_pages, page_size, Hkv, d = kcache.shape
    if dst_table is not None:
        if dst_table.dtype != torch.int32:
            raise TypeError("dst_table must be int32")
        if dst_table.dim() != 2 or dst_table.shape[0] != B:
            raise ValueError(f"dst_table must be [{B}, dst_pages]")
    maxp = block_table.shape[1]
    dst_pages = maxp if dst_table is None else dst_table.shape[1]
    _expect(weights, (B, Hkv, maxp * page_size), "weights", torch.float32)
    _expect(out_weights, (B, Hkv, dst_pages * page_size), "out_weights", torch.float32)
    _expect(out_seqlens, (B,), "out_seqlens", torch.int32)
    _expect(kept, (B, Hkv, keep), "kept", torch.int32)
    if out_weights is None:
        out_weights = torch.empty((B, Hkv, dst_pages * page_size), dtype=torch.float32, device=kcache.device)
    if out_seqlens is None:
        out_seqlens = torch.empty_like(seqlens)
    if kept is None:
        kept = torch.empty((B, Hkv, max(keep, 0)), dtype=torch.int32, device=kcache.device)
    st = lib.fattn_evict_paged(_ptr(kcache), _ptr(vcache), _ptr(block_table), _ptr(seqlens), _ptr(weights),
                               _ptr(dst_table), _ptr(out_seqlens), _ptr(out_weights), _ptr(kept), B, Hkv, d, page_size,
                               maxp, num_pages, dst_pages, keep, recent, first,
                               _stream_handle(stream))
    _check("fattn_evict_paged", st)
    return out_seqlens, out_weights, kept
