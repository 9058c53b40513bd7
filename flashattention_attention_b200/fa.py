"""Thin ctypes binding of libfa.so (include/fa.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  torch supplies device memory and the current
stream.  Importing this module loads ``lib/libfa.so`` and raises ImportError
when it is missing -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional, Sequence, Tuple

import torch

# FA_LIBRARY may name another build of the same library (e.g. one compiled
# with different tuning constants); by default the in-tree build is loaded.
_LIB_PATH = os.environ.get("FA_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib",
                                                          "libfa.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libfa.so not built ({_LIB_PATH}); run __graft_entry__.build() "
                      "or python flashattention_attention_b200/build.py")
lib = ctypes.CDLL(_LIB_PATH)

# --- fa.h mirrors -------------------------------------------------------------
FA_OK, FA_ERR_INVALID, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_WORKSPACE = range(6)
FA_F32, FA_BF16, FA_I8, FA_I4 = 0, 1, 2, 3
FA_EPI_MUL, FA_EPI_ADD = 1, 2
FA_MAX_EPILOGUE = 8
FA_ACC_FIRST, FA_ACC_LAST = 1, 2


class EpiOp(ctypes.Structure):
    _fields_ = [("op", ctypes.c_int32), ("value", ctypes.c_float)]


class FwdParams(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("q_dtype", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("seqlen_q", ctypes.c_int32), ("seqlen_k", ctypes.c_int32),
                ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
                ("total_q", ctypes.c_int32), ("total_k", ctypes.c_int32),
                ("max_seqlen_q", ctypes.c_int32), ("max_seqlen_k", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("window", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("n_epilogue", ctypes.c_int32),
                ("epilogue", EpiOp * FA_MAX_EPILOGUE)]


class DecodeParams(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("cache_seqlens", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("kv_dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("hq", ctypes.c_int32),
                ("hkv", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("max_seqlen", ctypes.c_int32), ("window", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("split_keys", ctypes.c_int32),
                ("n_epilogue", ctypes.c_int32), ("epilogue", EpiOp * FA_MAX_EPILOGUE),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class MergeParams(ctypes.Structure):
    _fields_ = [("o_acc", ctypes.c_void_p), ("lse_acc", ctypes.c_void_p), ("o_part", ctypes.c_void_p),
                ("part_dtype", ctypes.c_int32), ("lse_part", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("head_dim", ctypes.c_int32), ("out", ctypes.c_void_p), ("out_dtype", ctypes.c_int32),
                ("n_epilogue", ctypes.c_int32), ("epilogue", EpiOp * FA_MAX_EPILOGUE)]


class TqCompressParams(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_dtype", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("head_dim", ctypes.c_int32), ("bits", ctypes.c_int32), ("signs", ctypes.c_void_p),
                ("levels", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("norms", ctypes.c_void_p)]


class TqDecodeParams(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k_codes", ctypes.c_void_p), ("k_norms", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_norms", ctypes.c_void_p), ("k_levels", ctypes.c_void_p),
                ("v_levels", ctypes.c_void_p), ("signs", ctypes.c_void_p), ("cache_seqlens", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("capacity", ctypes.c_int32), ("k_bits", ctypes.c_int32),
                ("v_bits", ctypes.c_int32), ("softmax_scale", ctypes.c_float), ("out", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("n_epilogue", ctypes.c_int32), ("epilogue", EpiOp * FA_MAX_EPILOGUE)]


class KvPages(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("max_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32)]


class KvAppendParams(ctypes.Structure):
    _fields_ = [("k_new", ctypes.c_void_p), ("v_new", ctypes.c_void_p), ("x_dtype", ctypes.c_int32),
                ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("cache_dtype", ctypes.c_int32), ("cur_pos", ctypes.c_void_p),
                ("cache_seqlens", ctypes.c_void_p), ("batch", ctypes.c_int32), ("hkv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("capacity", ctypes.c_int32)]


_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class KvAppendRopeParams(ctypes.Structure):
    _fields_ = [("k_new", _P), ("v_new", _P), ("q", _P), ("q_out", _P),
                ("k_token_stride", _I64), ("k_head_stride", _I64), ("v_token_stride", _I64), ("v_head_stride", _I64),
                ("q_token_stride", _I64), ("q_head_stride", _I64),
                ("q_out_token_stride", _I64), ("q_out_head_stride", _I64),
                ("rope_table", _P), ("k_cache", _P), ("v_cache", _P), ("k_scales", _P), ("v_scales", _P),
                ("key_bounds", _P), ("cu_seqlens", _P), ("cur_pos", _P), ("cache_seqlens", _P),
                ("x_dtype", _I32), ("cache_dtype", _I32), ("batch", _I32), ("total", _I32), ("hq", _I32),
                ("hkv", _I32), ("head_dim", _I32), ("rot_dim", _I32), ("interleaved", _I32), ("rope_rows", _I32)]


class KvReadParams(ctypes.Structure):
    _fields_ = [("k_cache", _P), ("v_cache", _P), ("k_scales", _P), ("v_scales", _P), ("k_out", _P), ("v_out", _P),
                ("cu_seqlens", _P), ("start", _P), ("cache_dtype", _I32), ("out_dtype", _I32), ("batch", _I32),
                ("total", _I32), ("hkv", _I32), ("head_dim", _I32)]


class PageSelectParams(ctypes.Structure):
    _fields_ = [("q", _P), ("key_bounds", _P), ("cache_seqlens", _P), ("selected", _P), ("batch", _I32), ("hq", _I32),
                ("hkv", _I32), ("head_dim", _I32), ("top_k", _I32), ("n_first", _I32), ("n_recent", _I32),
                ("workspace", _P), ("workspace_bytes", ctypes.c_size_t)]


lib.fa_kv_append_rope_paged.restype = ctypes.c_int
lib.fa_kv_append_rope_paged.argtypes = [ctypes.POINTER(KvAppendRopeParams), ctypes.POINTER(KvPages), _P]
lib.fa_rope_table.restype = ctypes.c_int
lib.fa_rope_table.argtypes = [_I32, _I32, ctypes.c_double, _P]
lib.fa_kv_read_paged.restype = ctypes.c_int
lib.fa_kv_read_paged.argtypes = [ctypes.POINTER(KvReadParams), ctypes.POINTER(KvPages), _P]
lib.fa_page_select_workspace_size.restype = ctypes.c_size_t
lib.fa_page_select_workspace_size.argtypes = [_I32] * 3
lib.fa_page_select.restype = ctypes.c_int
lib.fa_page_select.argtypes = [ctypes.POINTER(PageSelectParams), ctypes.POINTER(KvPages), _P]
lib.fa_decode_pages_workspace_size.restype = ctypes.c_size_t
lib.fa_decode_pages_workspace_size.argtypes = [ctypes.POINTER(DecodeParams), ctypes.POINTER(KvPages), _I32]
lib.fa_attention_decode_selected.restype = ctypes.c_int
lib.fa_attention_decode_selected.argtypes = [ctypes.POINTER(DecodeParams), ctypes.POINTER(KvPages), _P, _I32, _P]
lib.fa_compress_kv.restype = ctypes.c_int
lib.fa_compress_kv.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int32,
                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
lib.fa_attention_fwd.restype = ctypes.c_int
lib.fa_attention_fwd.argtypes = [ctypes.POINTER(FwdParams), ctypes.c_void_p]
lib.fa_decode_workspace_size.restype = ctypes.c_size_t
lib.fa_decode_workspace_size.argtypes = [ctypes.c_int32] * 4
lib.fa_attention_decode.restype = ctypes.c_int
lib.fa_attention_decode.argtypes = [ctypes.POINTER(DecodeParams), ctypes.c_void_p]
lib.fa_attention_fwd_lse.restype = ctypes.c_int
lib.fa_attention_fwd_lse.argtypes = [ctypes.POINTER(FwdParams), ctypes.c_void_p, ctypes.c_void_p]
lib.fa_attention_fwd_acc.restype = ctypes.c_int
lib.fa_attention_fwd_acc.argtypes = [ctypes.POINTER(FwdParams), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                     ctypes.c_void_p]
lib.fa_attention_merge.restype = ctypes.c_int
lib.fa_attention_merge.argtypes = [ctypes.POINTER(MergeParams), ctypes.c_void_p]
lib.fa_attention_fwd_paged.restype = ctypes.c_int
lib.fa_attention_fwd_paged.argtypes = [ctypes.POINTER(FwdParams), ctypes.POINTER(KvPages), ctypes.c_void_p]
lib.fa_attention_decode_paged.restype = ctypes.c_int
lib.fa_attention_decode_paged.argtypes = [ctypes.POINTER(DecodeParams), ctypes.POINTER(KvPages), ctypes.c_void_p]
lib.fa_kv_append.restype = ctypes.c_int
lib.fa_kv_append.argtypes = [ctypes.POINTER(KvAppendParams), ctypes.c_void_p]
lib.fa_kv_append_paged.restype = ctypes.c_int
lib.fa_kv_append_paged.argtypes = [ctypes.POINTER(KvAppendParams), ctypes.POINTER(KvPages), ctypes.c_void_p]
lib.fa_tq_codebook.restype = ctypes.c_int
lib.fa_tq_codebook.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p]
lib.fa_tq_compress.restype = ctypes.c_int
lib.fa_tq_compress.argtypes = [ctypes.POINTER(TqCompressParams), ctypes.c_void_p]
lib.fa_tq_decode_workspace_size.restype = ctypes.c_size_t
lib.fa_tq_decode_workspace_size.argtypes = [ctypes.c_int32] * 4
lib.fa_tq_attention_decode.restype = ctypes.c_int
lib.fa_tq_attention_decode.argtypes = [ctypes.POINTER(TqDecodeParams), ctypes.c_void_p]
lib.fa_status_string.restype = ctypes.c_char_p
lib.fa_status_string.argtypes = [ctypes.c_int]
lib.fa_check_device_error.restype = ctypes.c_int
lib.fa_check_device_error.argtypes = [ctypes.c_void_p]
lib.fa_selftest_watchdog.restype = ctypes.c_int
lib.fa_selftest_watchdog.argtypes = [ctypes.c_uint64, ctypes.c_void_p]
lib.fa_kernel_variants_used.restype = ctypes.c_int32
lib.fa_kernel_variants_used.argtypes = []
lib.fa_kernel_launches.restype = ctypes.c_int64
lib.fa_kernel_launches.argtypes = []


class FAError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {lib.fa_status_string(status).decode()} (status {status})")
        self.status = status


def _check(status: int, what: str):
    if status != FA_OK:
        raise FAError(status, what)


_DT = {torch.float32: FA_F32, torch.bfloat16: FA_BF16, torch.int8: FA_I8}


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _fill_epilogue(arr, epilogue: Sequence[Tuple[str, float]]) -> int:
    if len(epilogue) > FA_MAX_EPILOGUE:
        raise ValueError(f"at most {FA_MAX_EPILOGUE} epilogue ops")
    for i, (op, val) in enumerate(epilogue):
        name = op.lower() if isinstance(op, str) else op
        arr[i].op = {"mul": FA_EPI_MUL, "add": FA_EPI_ADD}.get(name, name)
        arr[i].value = float(val)
    return len(epilogue)


def _shape(t, want, name: str):
    """ValueError unless t has the shape `want` (None: any extent).  The C
    ABI sees only pointers and sizes, so a tensor smaller than its sizes say
    must be caught here, before a kernel reads past it."""
    got = tuple(t.shape)
    if len(got) != len(want) or any(w is not None and g != w for g, w in zip(got, want)):
        shown = tuple("*" if w is None else w for w in want)
        raise ValueError(f"{name} has shape {got}, expected {shown}")


def _int32(t, name: str):
    if t is not None and t.dtype != torch.int32:
        raise ValueError(f"{name} must be int32")


def _contig_cuda(t: torch.Tensor, name: str):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


# --- API ----------------------------------------------------------------------

def compress_kv(x: torch.Tensor, codes: Optional[torch.Tensor] = None,
                scales: Optional[torch.Tensor] = None, stream=None):
    """Per-row int8 codes + fp32 scales of x [..., d] (bf16 or fp32)."""
    _contig_cuda(x, "x")
    d = x.shape[-1]
    rows = x.numel() // d if d else 0
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    if scales is None:
        scales = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _check(lib.fa_compress_kv(_ptr(x), _DT[x.dtype], rows, d, _ptr(codes), _ptr(scales), _stream(stream)),
           "fa_compress_kv")
    return codes, scales


def fwd_params(q, k, v, out, *, hq, hkv, causal=False, window=0, scale=None, epilogue=(),
               k_scales=None, v_scales=None, cu_seqlens_q=None, cu_seqlens_k=None,
               max_seqlen_q=None, max_seqlen_k=None) -> FwdParams:
    d = q.shape[-1]
    if hq <= 0 or hkv <= 0:
        raise ValueError("hq and hkv must be positive")
    if cu_seqlens_q is None:
        if len(q.shape) != 3 or q.shape[0] % hq:
            raise ValueError(f"dense q must be [batch*hq, s_q, d]; got {tuple(q.shape)} with hq={hq}")
        _shape(k, (q.shape[0] // hq * hkv, None, d), "k")
    else:
        _int32(cu_seqlens_q, "cu_seqlens_q")
        _int32(cu_seqlens_k, "cu_seqlens_k")
        _shape(q, (hq, None, d), "q")
        _shape(k, (hkv, None, d), "k")
        if cu_seqlens_k is not None:
            _shape(cu_seqlens_k, (cu_seqlens_q.numel(),), "cu_seqlens_k")
    _shape(v, tuple(k.shape), "v")
    _shape(out, tuple(q.shape), "out")
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        if t is not None:
            _shape(t, tuple(k.shape[:2]), name)
    p = FwdParams()
    p.q, p.k, p.v, p.out = q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr()
    p.k_scales = None if k_scales is None else k_scales.data_ptr()
    p.v_scales = None if v_scales is None else v_scales.data_ptr()
    p.q_dtype, p.kv_dtype = _DT[q.dtype], _DT[k.dtype]
    p.hq, p.hkv, p.head_dim = hq, hkv, q.shape[-1]
    if cu_seqlens_q is None:
        p.batch = q.shape[0] // hq
        p.seqlen_q, p.seqlen_k = q.shape[1], k.shape[1]
    else:
        p.batch = cu_seqlens_q.numel() - 1
        p.cu_seqlens_q = cu_seqlens_q.data_ptr()
        p.cu_seqlens_k = None if cu_seqlens_k is None else cu_seqlens_k.data_ptr()
        p.total_q, p.total_k = q.shape[1], k.shape[1]
        p.max_seqlen_q = int(max_seqlen_q)
        p.max_seqlen_k = int(max_seqlen_k if max_seqlen_k is not None else max_seqlen_q)
    p.causal, p.window = int(bool(causal)), int(window)
    p.softmax_scale = float(scale if scale is not None else 1.0 / math.sqrt(q.shape[-1]))
    p.n_epilogue = _fill_epilogue(p.epilogue, epilogue)
    return p


def attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, hq: int, hkv: int,
                  causal: bool = False, window: int = 0, scale: Optional[float] = None,
                  epilogue: Sequence[Tuple[str, float]] = (), k_scales=None, v_scales=None,
                  cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q=None, max_seqlen_k=None,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Fused attention forward; layouts and semantics as fa_attention_fwd in fa.h."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        _contig_cuda(t, name)
    if out is None:
        out = torch.empty_like(q)
    p = fwd_params(q, k, v, out, hq=hq, hkv=hkv, causal=causal, window=window, scale=scale,
                   epilogue=epilogue, k_scales=k_scales, v_scales=v_scales, cu_seqlens_q=cu_seqlens_q,
                   cu_seqlens_k=cu_seqlens_k, max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k)
    _check(lib.fa_attention_fwd(ctypes.byref(p), _stream(stream)), "fa_attention_fwd")
    return out


def attention_fwd_lse(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, hq: int, hkv: int,
                      causal: bool = False, window: int = 0, scale: Optional[float] = None,
                      k_scales=None, v_scales=None, cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q=None,
                      max_seqlen_k=None, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      stream=None):
    """Partial attention result (bf16 path): (out, lse) with lse the natural
    log-sum-exp of each row's scaled scores (-inf and out = 0 for a row
    without keys).  As fa_attention_fwd_lse in fa.h; no epilogue."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        _contig_cuda(t, name)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    p = fwd_params(q, k, v, out, hq=hq, hkv=hkv, causal=causal, window=window, scale=scale, epilogue=(),
                   k_scales=k_scales, v_scales=v_scales, cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k,
                   max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k)
    _check(lib.fa_attention_fwd_lse(ctypes.byref(p), _ptr(lse), _stream(stream)), "fa_attention_fwd_lse")
    return out, lse


def attention_fwd_acc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o_acc: torch.Tensor,
                      lse_acc: torch.Tensor, *, hq: int, hkv: int, causal: bool = False, window: int = 0,
                      scale: Optional[float] = None, first: bool = False, last: bool = False,
                      out: Optional[torch.Tensor] = None, epilogue: Sequence[Tuple[str, float]] = (),
                      k_scales=None, v_scales=None, cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q=None,
                      max_seqlen_k=None, stream=None) -> Optional[torch.Tensor]:
    """Attention of q over these keys merged into the fp32 accumulator
    (o_acc [..., d] like q, lse_acc [...]) in the kernel's epilogue.  first:
    the accumulator is empty and not read; last: the merged rows go to `out`
    (allocated in q's dtype if None) after the epilogue and are returned,
    the accumulator is left as it was.  As fa_attention_fwd_acc in fa.h."""
    for name, t in (("q", q), ("k", k), ("v", v), ("o_acc", o_acc), ("lse_acc", lse_acc)):
        _contig_cuda(t, name)
    if o_acc.dtype != torch.float32 or lse_acc.dtype != torch.float32:
        raise ValueError("the accumulator is fp32")
    if o_acc.shape != q.shape or lse_acc.shape != q.shape[:-1]:
        raise ValueError("o_acc must have q's shape and lse_acc q's shape without the last dim")
    if last and out is None:
        out = torch.empty_like(q)
    p = fwd_params(q, k, v, out if last else q, hq=hq, hkv=hkv, causal=causal, window=window, scale=scale,
                   epilogue=epilogue, k_scales=k_scales, v_scales=v_scales, cu_seqlens_q=cu_seqlens_q,
                   cu_seqlens_k=cu_seqlens_k, max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k)
    if not last:
        p.out = None
    flags = (FA_ACC_FIRST if first else 0) | (FA_ACC_LAST if last else 0)
    _check(lib.fa_attention_fwd_acc(ctypes.byref(p), _ptr(o_acc), _ptr(lse_acc), flags, _stream(stream)),
           "fa_attention_fwd_acc")
    return out if last else None


def attention_merge(o_acc: torch.Tensor, lse_acc: torch.Tensor, o_part: Optional[torch.Tensor] = None,
                    lse_part: Optional[torch.Tensor] = None, *, out: Optional[torch.Tensor] = None,
                    epilogue: Sequence[Tuple[str, float]] = (), stream=None) -> Optional[torch.Tensor]:
    """Fold the partial result (o_part, lse_part) into the fp32 accumulator
    (o_acc [..., d], lse_acc [...]) in place; with `out`, also write the
    merged rows after the epilogue.  As fa_attention_merge in fa.h."""
    _contig_cuda(o_acc, "o_acc")
    _contig_cuda(lse_acc, "lse_acc")
    _shape(lse_acc, tuple(o_acc.shape[:-1]), "lse_acc")
    if o_part is not None:
        _shape(o_part, tuple(o_acc.shape), "o_part")
        if lse_part is None:
            raise ValueError("lse_part is required with o_part")
        _shape(lse_part, tuple(lse_acc.shape), "lse_part")
    if out is not None:
        _shape(out, tuple(o_acc.shape), "out")
    p = MergeParams()
    p.o_acc, p.lse_acc = o_acc.data_ptr(), lse_acc.data_ptr()
    if o_part is not None:
        _contig_cuda(o_part, "o_part")
        _contig_cuda(lse_part, "lse_part")
        p.o_part, p.part_dtype, p.lse_part = o_part.data_ptr(), _DT[o_part.dtype], lse_part.data_ptr()
    p.head_dim = o_acc.shape[-1]
    p.rows = o_acc.numel() // p.head_dim
    if out is not None:
        _contig_cuda(out, "out")
        p.out, p.out_dtype = out.data_ptr(), _DT[out.dtype]
    p.n_epilogue = _fill_epilogue(p.epilogue, epilogue)
    _check(lib.fa_attention_merge(ctypes.byref(p), _stream(stream)), "fa_attention_merge")
    return out


def _pool_shapes(k_pages, v_pages, k_scales, v_scales, hkv: int, d: int):
    """Page pools [num_pages, hkv, page_size, d] and their scales
    [num_pages, hkv, page_size]."""
    _shape(k_pages, (None, hkv, None, d), "k_pages")
    _shape(v_pages, tuple(k_pages.shape), "v_pages")
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        if t is not None:
            _shape(t, tuple(k_pages.shape[:3]), name)


def _cache_shapes(q, k_cache, v_cache, k_scales, v_scales, cache_seqlens, out, hq: int, hkv: int):
    """Decode operands: q [batch*hq, d] or [batch*hq, 1, d], dense caches
    [batch*hkv, capacity, d] and scales [batch*hkv, capacity]."""
    _int32(cache_seqlens, "cache_seqlens")
    batch, d = cache_seqlens.numel(), q.shape[-1]
    if q.numel() != batch * hq * d:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected batch*hq = {batch * hq} rows of {d}")
    if k_cache is not None:
        _shape(k_cache, (batch * hkv, None, d), "k_cache")
        _shape(v_cache, tuple(k_cache.shape), "v_cache")
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if t is not None:
                _shape(t, tuple(k_cache.shape[:2]), name)
    if out is not None:
        _shape(out, tuple(q.shape), "out")


def attention_fwd_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                        cu_seqlens_k: torch.Tensor, block_table: torch.Tensor, *, hq: int, hkv: int,
                        causal: bool = False, window: int = 0, scale: Optional[float] = None,
                        epilogue: Sequence[Tuple[str, float]] = (), k_scales=None, v_scales=None,
                        cu_seqlens_q=None, max_seqlen_q=None, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """Prefill over page pools k_pages/v_pages [num_pages, hkv, page_size, d]
    (int8 with scales [num_pages, hkv, page_size], or bf16) through a device
    int32 block_table [B, max_pages]; q dense [B*hq, s_q, d] or varlen
    [hq, total_q, d] with cu_seqlens_q.  As fa_attention_fwd_paged in fa.h."""
    for name, t in (("q", q), ("k_pages", k_pages), ("v_pages", v_pages), ("cu_seqlens_k", cu_seqlens_k),
                    ("block_table", block_table)):
        _contig_cuda(t, name)
    d = q.shape[-1]
    _pool_shapes(k_pages, v_pages, k_scales, v_scales, hkv, d)
    for name, t in (("cu_seqlens_k", cu_seqlens_k), ("block_table", block_table), ("cu_seqlens_q", cu_seqlens_q)):
        _int32(t, name)
    batch = cu_seqlens_k.numel() - 1
    _shape(block_table, (batch, None), "block_table")
    if cu_seqlens_q is None:
        _shape(q, (batch * hq, None, d), "q")
    else:
        _shape(q, (hq, None, d), "q")
        _shape(cu_seqlens_q, (batch + 1,), "cu_seqlens_q")
    if out is not None:
        _shape(out, tuple(q.shape), "out")
    if out is None:
        out = torch.empty_like(q)
    p = FwdParams()
    p.q, p.k, p.v, p.out = q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr()
    p.k_scales = None if k_scales is None else k_scales.data_ptr()
    p.v_scales = None if v_scales is None else v_scales.data_ptr()
    p.q_dtype, p.kv_dtype = _DT[q.dtype], _DT[k_pages.dtype]
    p.hq, p.hkv, p.head_dim = hq, hkv, q.shape[-1]
    p.batch = cu_seqlens_k.numel() - 1
    p.cu_seqlens_k = cu_seqlens_k.data_ptr()
    if cu_seqlens_q is None:
        p.seqlen_q = q.shape[1]
    else:
        p.cu_seqlens_q = cu_seqlens_q.data_ptr()
        p.total_q = q.shape[1]
        p.max_seqlen_q = int(max_seqlen_q)
    p.causal, p.window = int(bool(causal)), int(window)
    p.softmax_scale = float(scale if scale is not None else 1.0 / math.sqrt(q.shape[-1]))
    p.n_epilogue = _fill_epilogue(p.epilogue, epilogue)
    num_pages, _, page_size, _ = k_pages.shape
    pg = KvPages(block_table.data_ptr(), block_table.shape[1], page_size, num_pages)
    _check(lib.fa_attention_fwd_paged(ctypes.byref(p), ctypes.byref(pg), _stream(stream)), "fa_attention_fwd_paged")
    return out


def decode_workspace_size(batch: int, hq: int, capacity: int, head_dim: int) -> int:
    return int(lib.fa_decode_workspace_size(batch, hq, capacity, head_dim))


def decode_params(q, k_cache, v_cache, cache_seqlens, out, workspace, *, hq, hkv, k_scales=None,
                  v_scales=None, window=0, scale=None, epilogue=(), max_seqlen=0,
                  split_keys=0) -> DecodeParams:
    p = DecodeParams()
    p.q, p.k_cache, p.v_cache = q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    p.k_scales = None if k_scales is None else k_scales.data_ptr()
    p.v_scales = None if v_scales is None else v_scales.data_ptr()
    p.cache_seqlens, p.out = cache_seqlens.data_ptr(), out.data_ptr()
    p.kv_dtype = _DT[k_cache.dtype]
    p.batch = cache_seqlens.numel()
    p.hq, p.hkv, p.head_dim, p.capacity = hq, hkv, q.shape[-1], k_cache.shape[1]
    p.max_seqlen, p.window = int(max_seqlen), int(window)
    p.softmax_scale = float(scale if scale is not None else 1.0 / math.sqrt(q.shape[-1]))
    p.split_keys = int(split_keys)
    p.n_epilogue = _fill_epilogue(p.epilogue, epilogue)
    p.workspace = workspace.data_ptr()
    p.workspace_bytes = workspace.numel() * workspace.element_size()
    return p


def attention_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     cache_seqlens: torch.Tensor, *, hq: int, hkv: int, k_scales=None, v_scales=None,
                     window: int = 0, scale: Optional[float] = None,
                     epilogue: Sequence[Tuple[str, float]] = (), max_seqlen: int = 0,
                     split_keys: int = 0, workspace: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """s_q = 1 decode; q [B*hq, d] (or [B*hq, 1, d]) bf16, caches [B*hkv, cap, d]."""
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache),
                    ("cache_seqlens", cache_seqlens)):
        _contig_cuda(t, name)
    _cache_shapes(q, k_cache, v_cache, k_scales, v_scales, cache_seqlens, out, hq, hkv)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        nbytes = decode_workspace_size(cache_seqlens.numel(), hq, k_cache.shape[1], q.shape[-1])
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    p = decode_params(q, k_cache, v_cache, cache_seqlens, out, workspace, hq=hq, hkv=hkv,
                      k_scales=k_scales, v_scales=v_scales, window=window, scale=scale,
                      epilogue=epilogue, max_seqlen=max_seqlen, split_keys=split_keys)
    _check(lib.fa_attention_decode(ctypes.byref(p), _stream(stream)), "fa_attention_decode")
    return out


def attention_decode_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                           cache_seqlens: torch.Tensor, block_table: torch.Tensor, *, hq: int, hkv: int,
                           k_scales=None, v_scales=None, window: int = 0, scale: Optional[float] = None,
                           epilogue: Sequence[Tuple[str, float]] = (), max_seqlen: int = 0,
                           split_keys: int = 0, workspace: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """s_q = 1 decode over page pools k_pages/v_pages [num_pages, hkv, page_size, d]
    (int8 with scales [num_pages, hkv, page_size], or bf16) through a device
    int32 block_table [B, max_pages]; as fa_attention_decode_paged in fa.h.
    uint8 pools [num_pages, hkv, page_size, d/2] hold 4-bit codes, with scales
    [num_pages, hkv, page_size, 2] of (step, offset); split_keys must be 0."""
    if k_pages.dtype == torch.uint8:
        if split_keys != 0:
            raise ValueError("split_keys does not apply to a 4-bit cache")
        return _decode_pages(q, k_pages, v_pages, cache_seqlens, block_table, None, hq, hkv, k_scales, v_scales, window,
                             scale, epilogue, max_seqlen, workspace, out, stream)
    for name, t in (("q", q), ("k_pages", k_pages), ("v_pages", v_pages), ("cache_seqlens", cache_seqlens),
                    ("block_table", block_table)):
        _contig_cuda(t, name)
    _pool_shapes(k_pages, v_pages, k_scales, v_scales, hkv, q.shape[-1])
    _cache_shapes(q, None, None, None, None, cache_seqlens, out, hq, hkv)
    _int32(block_table, "block_table")
    _shape(block_table, (cache_seqlens.numel(), None), "block_table")
    num_pages, _, page_size, d = k_pages.shape
    max_pages = block_table.shape[1]
    capacity = max_pages * page_size
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        nbytes = decode_workspace_size(cache_seqlens.numel(), hq, capacity, d)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    p = decode_params(q, k_pages, v_pages, cache_seqlens, out, workspace, hq=hq, hkv=hkv,
                      k_scales=k_scales, v_scales=v_scales, window=window, scale=scale,
                      epilogue=epilogue, max_seqlen=max_seqlen, split_keys=split_keys)
    p.capacity = capacity
    pg = KvPages(block_table.data_ptr(), max_pages, page_size, num_pages)
    _check(lib.fa_attention_decode_paged(ctypes.byref(p), ctypes.byref(pg), _stream(stream)),
           "fa_attention_decode_paged")
    return out


def kv_append(k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              cur_pos: torch.Tensor, *, hkv: int, k_scales=None, v_scales=None, cache_seqlens=None,
              stream=None) -> None:
    """Write one new token per sequence (k_new, v_new [B*hkv, d]) into the
    caches [B*hkv, cap, d] at slot cur_pos[b] (device int32 [B]); an int8
    cache is quantised on the way in (scales required), a bf16 one stored
    as bf16.  cache_seqlens (device int32 [B]), if given, becomes cur_pos + 1.
    Layouts and semantics as fa_kv_append in fa.h."""
    _append_shapes(k_new, v_new, cur_pos, cache_seqlens, hkv)
    _shape(k_cache, (cur_pos.numel() * hkv, None, k_new.shape[-1]), "k_cache")
    _shape(v_cache, tuple(k_cache.shape), "v_cache")
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        if t is not None:
            _shape(t, tuple(k_cache.shape[:2]), name)
    p = _append_params(k_new, v_new, k_cache, v_cache, cur_pos, hkv, k_scales, v_scales, cache_seqlens)
    _check(lib.fa_kv_append(ctypes.byref(p), _stream(stream)), "fa_kv_append")


def kv_append_paged(k_new: torch.Tensor, v_new: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                    cur_pos: torch.Tensor, block_table: torch.Tensor, *, hkv: int, k_scales=None,
                    v_scales=None, cache_seqlens=None, stream=None) -> None:
    """kv_append into page pools [num_pages, hkv, page_size, d] through a
    device int32 block_table [B, max_pages]; as fa_kv_append_paged in fa.h."""
    _contig_cuda(block_table, "block_table")
    _append_shapes(k_new, v_new, cur_pos, cache_seqlens, hkv)
    _pool_shapes(k_pages, v_pages, k_scales, v_scales, hkv, k_new.shape[-1])
    _int32(block_table, "block_table")
    _shape(block_table, (cur_pos.numel(), None), "block_table")
    p = _append_params(k_new, v_new, k_pages, v_pages, cur_pos, hkv, k_scales, v_scales, cache_seqlens)
    num_pages, _, page_size, d = k_pages.shape
    p.head_dim, p.capacity = d, block_table.shape[1] * page_size
    pg = KvPages(block_table.data_ptr(), block_table.shape[1], page_size, num_pages)
    _check(lib.fa_kv_append_paged(ctypes.byref(p), ctypes.byref(pg), _stream(stream)), "fa_kv_append_paged")


def _append_shapes(k_new, v_new, cur_pos, cache_seqlens, hkv: int):
    _int32(cur_pos, "cur_pos")
    _int32(cache_seqlens, "cache_seqlens")
    _shape(k_new, (cur_pos.numel() * hkv, None), "k_new")
    _shape(v_new, tuple(k_new.shape), "v_new")
    if cache_seqlens is not None:
        _shape(cache_seqlens, (cur_pos.numel(),), "cache_seqlens")


def _append_params(k_new, v_new, k_cache, v_cache, cur_pos, hkv, k_scales, v_scales, cache_seqlens):
    for name, t in (("k_new", k_new), ("v_new", v_new), ("k_cache", k_cache), ("v_cache", v_cache),
                    ("cur_pos", cur_pos)):
        _contig_cuda(t, name)
    p = KvAppendParams()
    p.k_new, p.v_new, p.x_dtype = k_new.data_ptr(), v_new.data_ptr(), _DT[k_new.dtype]
    p.k_cache, p.v_cache, p.cache_dtype = k_cache.data_ptr(), v_cache.data_ptr(), _DT[k_cache.dtype]
    p.k_scales = None if k_scales is None else k_scales.data_ptr()
    p.v_scales = None if v_scales is None else v_scales.data_ptr()
    p.cur_pos = cur_pos.data_ptr()
    p.cache_seqlens = None if cache_seqlens is None else cache_seqlens.data_ptr()
    p.batch, p.hkv = cur_pos.numel(), hkv
    p.head_dim, p.capacity = k_cache.shape[-1], k_cache.shape[1]
    return p


# --- rotated append, page selection and attention over page pools -----------------
#
# A decode step makes a few of these calls per layer, so their checks are
# written for their cost: each call tests all of its tensors in one expression
# and looks for the one at fault (_refuse) only when the expression fails.

_CACHE_DT = {torch.bfloat16: FA_BF16, torch.int8: FA_I8, torch.uint8: FA_I4}
_BF16, _F32, _INT32 = torch.bfloat16, torch.float32, torch.int32
# torch's own accessors, several times as fast as the public ones; a torch
# without them (one built without CUDA) still imports this module
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _packer(cls):
    """cls(*fields) as bytes with the structure's layout: a quarter of the cost of
    making the structure (an array field is given as bytes)."""
    codes = {ctypes.c_void_p: "P", ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_size_t: "N", ctypes.c_float: "f"}
    s = struct.Struct("@" + "".join(codes.get(c) or f"{ctypes.sizeof(c)}s" for _, c in cls._fields_) + "0P")
    assert s.size == ctypes.sizeof(cls)
    return s.pack


_pack_append, _pack_read, _pack_select = _packer(KvAppendRopeParams), _packer(KvReadParams), _packer(PageSelectParams)
_pack_decode, _pack_pages = _packer(DecodeParams), _packer(KvPages)


def _packed(name: str):
    """The library's function for structures packed as bytes (lib.<name> itself takes the structures only)."""
    fn = lib[name]  # another object than lib.<name>
    typed = getattr(lib, name)
    fn.restype, fn.argtypes = typed.restype, [_P if issubclass(a, ctypes._Pointer) else a for a in typed.argtypes]
    return fn


_append_call, _read_call = _packed("fa_kv_append_rope_paged"), _packed("fa_kv_read_paged")
_select_call, _decode_size_call = _packed("fa_page_select"), _packed("fa_decode_pages_workspace_size")
_decode_call, _selected_call = _packed("fa_attention_decode_paged"), _packed("fa_attention_decode_selected")
_NO_EPILOGUE = bytes(ctypes.sizeof(EpiOp) * FA_MAX_EPILOGUE)


def _on_device(dev: int, stream, what: str, fn, *args) -> None:
    """Call fn(*args, stream) with CUDA device `dev` current: on `stream`, or
    on dev's current stream (torch.cuda.current_stream(dev), without the
    object that costs more than the rest of the call)."""
    if stream is None:
        raw = _raw_stream(dev)
    else:
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
        raw = stream.cuda_stream
    if _current_device() == dev:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status != FA_OK:
        raise FAError(status, what)


def _new(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    """A tensor on like's device for a call on `stream`: allocated on that
    stream, so that memory freed when the call returns is only reused in its order."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _refuse(dev: int, *operands) -> None:
    """ValueError for the first operand (tensor, name, dtype, shape) that is not a
    contiguous tensor of that dtype and shape on CUDA device dev."""
    for t, name, dtype, shape in operands:
        if t is None:
            continue
        if t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor on cuda:{dev}")
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def _operand(t, name: str, dev: int, dtype, shape) -> int:
    """The address of a contiguous tensor on CUDA device dev with this dtype and shape (0 for None)."""
    if t is None:
        return 0
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
        _refuse(dev, (t, name, dtype, shape))
    return t.data_ptr()


def _pool_operands(k_pages, v_pages, k_scales, v_scales, block_table, batch: int, hkv: int, d: int, dev: int):
    """(cache dtype, packed KvPages, pool and scale addresses) of page pools; ValueError where they do not fit together."""
    dtype, shape, table_shape = k_pages.dtype, k_pages.shape, block_table.shape
    kind = _CACHE_DT.get(dtype)
    if kind is None:
        raise ValueError(f"a page pool is bfloat16, int8 or uint8 (4-bit codes), not {dtype}")
    if len(shape) != 4 or len(table_shape) != 2:
        raise ValueError(f"a page pool has 4 dimensions and a block table 2; got {tuple(shape)} and {tuple(table_shape)}")
    num_pages, heads, page_size, width = shape
    want = d >> 1 if kind == FA_I4 else d
    if not (heads == hkv and width == want and table_shape[0] == batch and v_pages.dtype is dtype
            and v_pages.shape == shape and block_table.dtype is _INT32 and k_pages.get_device() == dev
            and v_pages.get_device() == dev and block_table.get_device() == dev and k_pages.is_contiguous()
            and v_pages.is_contiguous() and block_table.is_contiguous()):
        pool = (num_pages, hkv, page_size, want)
        _refuse(dev, (k_pages, "k_pages", dtype, pool), (v_pages, "v_pages", dtype, pool),
                (block_table, "block_table", _INT32, (batch, table_shape[1])))
    pages = _pack_pages(block_table.data_ptr(), table_shape[1], page_size, num_pages)
    if kind == FA_BF16:
        if k_scales is not None or v_scales is not None:
            raise ValueError("a bfloat16 cache has no scales")
        return kind, pages, k_pages.data_ptr(), v_pages.data_ptr(), 0, 0
    if k_scales is None or v_scales is None:
        raise ValueError("k_scales and v_scales are required with a quantised cache")
    rows = (num_pages, hkv, page_size, 2) if kind == FA_I4 else (num_pages, hkv, page_size)
    if not (k_scales.dtype is _F32 and v_scales.dtype is _F32 and k_scales.shape == rows and v_scales.shape == rows
            and k_scales.get_device() == dev and v_scales.get_device() == dev and k_scales.is_contiguous()
            and v_scales.is_contiguous()):
        _refuse(dev, (k_scales, "k_scales", _F32, rows), (v_scales, "v_scales", _F32, rows))
    return kind, pages, k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr()


def _int(x, name: str, lo: int = 0) -> int:
    """x as an int of the C ABI's 32 bits, at least lo."""
    x = int(x)
    if not lo <= x < 2147483648:
        raise ValueError(f"{name} = {x} is out of range")
    return x


def _cuda_device(t, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _rows_operand(t, name: str, dev: int, dtype, shape):
    """(address, token stride, head stride) of rows [tokens, heads, d] whose last dimension is contiguous."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == dev):
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} on cuda:{dev}; got {t.dtype} {tuple(t.shape)} on {t.device}")
    tokens, heads, channels = t.stride()
    if channels != 1 and shape[2] > 1:
        raise ValueError(f"{name}: the channels of a row must be contiguous")
    # a dimension of one row has no stride of its own
    return t.data_ptr(), tokens if shape[0] > 1 else 0, heads if shape[1] > 1 else 0


def rope_table(rows: int, rot_dim: int, base: float = 10000.0) -> torch.Tensor:
    """The rotation table [rows, rot_dim] (fp32, CPU): cos then sin of
    p * base^(-2i/rot_dim), computed in double.  As fa_rope_table in fa.h."""
    if rows < 0 or rot_dim < 1:
        raise ValueError("rows must not be negative, rot_dim positive")
    out = torch.empty((rows, rot_dim), dtype=torch.float32)
    _check(lib.fa_rope_table(rows, rot_dim, float(base), out.data_ptr()), "fa_rope_table")
    return out


def kv_append_rope_paged(k_new: torch.Tensor, v_new: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                         cur_pos: torch.Tensor, block_table: torch.Tensor, *, q: Optional[torch.Tensor] = None,
                         q_out: Optional[torch.Tensor] = None, rope_table: Optional[torch.Tensor] = None,
                         interleaved: bool = False, k_scales=None, v_scales=None,
                         key_bounds: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                         cache_seqlens: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Append new tokens to page pools, keys (and the queries q) rotated to
    their positions.  k_new, v_new [total, hkv, d] and q [total, hq, d] (bf16
    or fp32) may be slices of one projection: any token and head strides.
    Without cu_seqlens one token per sequence, else device int32 [B+1]; the
    first goes to slot cur_pos[b] (device int32 [B]).  rope_table fp32
    [rows, rot_dim] (None: no rotation).  Pools as attention_decode_paged:
    bf16, int8 or uint8 (4-bit).  key_bounds bf16 [num_pages, hkv, 2, d] is
    kept up to date for page_select; cache_seqlens becomes the new lengths.
    Returns the rotated queries in bf16 in the layout the attention calls
    take: [B*hq, d] without cu_seqlens, else [hq, total, d] (`q_out` of that
    shape if given), or None without q.  As fa_kv_append_rope_paged in fa.h."""
    dev = _cuda_device(k_pages, "k_pages")
    rows, pos_shape = k_new.shape, cur_pos.shape
    if len(rows) != 3 or len(pos_shape) != 1:
        raise ValueError(f"k_new must be [total, hkv, d] and cur_pos [batch]; got {tuple(rows)} and {tuple(pos_shape)}")
    total, hkv, d = rows
    batch = pos_shape[0]
    xt = k_new.dtype
    if xt is not _BF16 and xt is not _F32:
        raise ValueError(f"k_new must be bfloat16 or float32, not {xt}")
    if cu_seqlens is None and total != batch:
        raise ValueError(f"without cu_seqlens there is one token per sequence: {total} tokens, {batch} sequences")
    kn, kts, khs = _rows_operand(k_new, "k_new", dev, xt, rows)
    vn, vts, vhs = _rows_operand(v_new, "v_new", dev, xt, rows)
    kind, pg, kp, vp, ks, vs = _pool_operands(k_pages, v_pages, k_scales, v_scales, block_table, batch, hkv, d, dev)
    bounds = _operand(key_bounds, "key_bounds", dev, _BF16, (k_pages.shape[0], hkv, 2, d))
    pos = _operand(cur_pos, "cur_pos", dev, _INT32, pos_shape)
    cu = _operand(cu_seqlens, "cu_seqlens", dev, _INT32, (batch + 1,))
    lens = _operand(cache_seqlens, "cache_seqlens", dev, _INT32, pos_shape)
    table = table_rows = rot = 0
    if rope_table is not None:
        shape = rope_table.shape
        if len(shape) != 2:
            raise ValueError(f"rope_table has shape {tuple(shape)}, expected 2 dimensions")
        table_rows, rot = shape
        table = _operand(rope_table, "rope_table", dev, _F32, shape)
    qp = qo = qts = qhs = ots = ohs = hq = 0
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
    else:
        shape = q.shape
        if len(shape) != 3 or shape[0] != total or shape[2] != d:
            raise ValueError(f"q must be [{total}, hq, {d}]; got {tuple(shape)}")
        hq = shape[1]
        qp, qts, qhs = _rows_operand(q, "q", dev, xt, shape)
        if cu_seqlens is None:
            out_shape, ots, ohs = (total * hq, d), hq * d, d
        else:
            out_shape, ots, ohs = (hq, total, d), d, total * d
        if q_out is None:
            q_out = _new(q, out_shape, _BF16, stream)
            qo = q_out.data_ptr()
        else:
            qo = _operand(q_out, "q_out", dev, _BF16, out_shape)
    p = _pack_append(kn, vn, qp, qo, kts, khs, vts, vhs, qts, qhs, ots, ohs, table, kp, vp, ks, vs, bounds, cu, pos,
                     lens, FA_BF16 if xt is _BF16 else FA_F32, kind, batch, total, hq, hkv, d, rot,
                     1 if interleaved else 0, table_rows)
    _on_device(dev, stream, "fa_kv_append_rope_paged", _append_call, p, pg)
    return q_out


def kv_read_paged(k_pages: torch.Tensor, v_pages: torch.Tensor, cu_seqlens: torch.Tensor, block_table: torch.Tensor, *,
                  total: int, start: Optional[torch.Tensor] = None, k_scales=None, v_scales=None,
                  out_dtype: torch.dtype = torch.bfloat16, k_out: Optional[torch.Tensor] = None,
                  v_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(k, v) [hkv, total, d] of the cached rows start[b] .. of each sequence
    (start None: from slot 0), cu_seqlens[b+1] - cu_seqlens[b] of them, as bf16
    or fp32 values in attention_fwd's varlen layout.  As fa_kv_read_paged in fa.h."""
    dev = _cuda_device(k_pages, "k_pages")
    if len(cu_seqlens.shape) != 1 or cu_seqlens.shape[0] < 1 or len(k_pages.shape) != 4:
        raise ValueError("cu_seqlens must be [batch + 1] and k_pages [num_pages, hkv, page_size, d]")
    batch, hkv = cu_seqlens.shape[0] - 1, k_pages.shape[1]
    d = k_pages.shape[3] * (2 if k_pages.dtype is torch.uint8 else 1)
    kind, pg, kp, vp, ks, vs = _pool_operands(k_pages, v_pages, k_scales, v_scales, block_table, batch, hkv, d, dev)
    if out_dtype is not _BF16 and out_dtype is not _F32:
        raise ValueError(f"out_dtype must be bfloat16 or float32, not {out_dtype}")
    shape = (hkv, _int(total, "total"), d)
    if k_out is None:
        k_out = _new(k_pages, shape, out_dtype, stream)
        ko = k_out.data_ptr()
    else:
        ko = _operand(k_out, "k_out", dev, out_dtype, shape)
    if v_out is None:
        v_out = torch.empty_like(k_out) if stream is None else _new(k_pages, shape, out_dtype, stream)
        vo = v_out.data_ptr()
    else:
        vo = _operand(v_out, "v_out", dev, out_dtype, shape)
    p = _pack_read(kp, vp, ks, vs, ko, vo, _operand(cu_seqlens, "cu_seqlens", dev, _INT32, (batch + 1,)),
                   _operand(start, "start", dev, _INT32, (batch,)), kind, FA_BF16 if out_dtype is _BF16 else FA_F32,
                   batch, shape[1], hkv, d)
    _on_device(dev, stream, "fa_kv_read_paged", _read_call, p, pg)
    return k_out, v_out


def _decode_queries(q, cache_seqlens, hq: int, hkv: int, dev: int):
    """(batch, d, address of q, address of cache_seqlens) of a decode step's operands."""
    if hq < 1 or hkv < 1 or hq % hkv:
        raise ValueError(f"hq = {hq} must be a positive multiple of hkv = {hkv}")
    shape, lens_shape = q.shape, cache_seqlens.shape
    if len(lens_shape) != 1:
        raise ValueError(f"cache_seqlens has shape {tuple(lens_shape)}, expected 1 dimension")
    batch, d = lens_shape[0], shape[-1]
    if shape != (batch * hq, d) and shape != (batch * hq, 1, d):
        raise ValueError(f"q has shape {tuple(shape)}, expected batch*hq = {batch * hq} rows")
    if not (q.dtype is _BF16 and cache_seqlens.dtype is _INT32 and cache_seqlens.get_device() == dev
            and q.is_contiguous() and cache_seqlens.is_contiguous()):
        _refuse(dev, (q, "q", _BF16, shape), (cache_seqlens, "cache_seqlens", _INT32, lens_shape))
    return batch, d, q.data_ptr(), cache_seqlens.data_ptr()


def _workspace(t, dev: int) -> int:
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return t.data_ptr()


def page_select(q: torch.Tensor, key_bounds: torch.Tensor, cache_seqlens: torch.Tensor, block_table: torch.Tensor, *,
                hq: int, hkv: int, page_size: int, top_k: int, n_first: int = 1, n_recent: int = 1,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """int32 [B, hkv, top_k]: the logical pages each sequence's query (q
    [B*hq, d] bf16) is most likely to need, by the bounds
    kv_append_rope_paged keeps; ascending, -1 behind the last.  The first
    n_first and last n_recent pages are always among them.  As fa_page_select
    in fa.h."""
    dev = _cuda_device(q, "q")
    batch, d, qp, lens = _decode_queries(q, cache_seqlens, hq, hkv, dev)
    bounds_shape, table_shape = key_bounds.shape, block_table.shape
    if len(bounds_shape) != 4 or len(table_shape) != 2:
        raise ValueError("key_bounds must be [num_pages, hkv, 2, d] and block_table [batch, max_pages]")
    num_pages, max_pages = bounds_shape[0], table_shape[1]
    bounds = _operand(key_bounds, "key_bounds", dev, _BF16, (num_pages, hkv, 2, d))
    table = _operand(block_table, "block_table", dev, _INT32, (batch, max_pages))
    top_k = _int(top_k, "top_k", 1)
    shape = (batch, hkv, top_k)
    if out is None:
        out = _new(q, shape, _INT32, stream)
        selected = out.data_ptr()
    else:
        selected = _operand(out, "out", dev, _INT32, shape)
    nbytes = ws = 0
    if workspace is None:
        if max_pages > 128:  # shorter tables need none
            if _current_device() == dev:
                nbytes = lib.fa_page_select_workspace_size(batch, hkv, max_pages)
            else:
                with torch.cuda.device(dev):  # its count of SMs enters the size
                    nbytes = lib.fa_page_select_workspace_size(batch, hkv, max_pages)
        if nbytes:
            workspace = _new(q, nbytes, torch.uint8, stream)
            ws = workspace.data_ptr()
    else:
        nbytes, ws = workspace.numel() * workspace.element_size(), _workspace(workspace, dev)
    p = _pack_select(qp, bounds, lens, selected, batch, hq, hkv, d, top_k, _int(n_first, "n_first"),
                     _int(n_recent, "n_recent"), ws, nbytes)
    _on_device(dev, stream, "fa_page_select", _select_call, p,
               _pack_pages(table, max_pages, _int(page_size, "page_size", 1), num_pages))
    return out


def attention_decode_selected(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                              cache_seqlens: torch.Tensor, block_table: torch.Tensor, selected: torch.Tensor, *,
                              hq: int, hkv: int, k_scales=None, v_scales=None, scale: Optional[float] = None,
                              epilogue: Sequence[Tuple[str, float]] = (), workspace: Optional[torch.Tensor] = None,
                              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """attention_decode_paged (bf16, int8 or uint8 4-bit pools) over the pages
    `selected` (device int32 [B, hkv, top_k] of logical page numbers; -1: none)
    only.  As fa_attention_decode_selected in fa.h."""
    return _decode_pages(q, k_pages, v_pages, cache_seqlens, block_table, selected, hq, hkv, k_scales, v_scales, 0, scale,
                         epilogue, 0, workspace, out, stream)


def _decode_pages(q, k_pages, v_pages, cache_seqlens, block_table, selected, hq, hkv, k_scales, v_scales, window, scale,
                  epilogue, max_seqlen, workspace, out, stream):
    dev = _cuda_device(q, "q")
    batch, d, qp, lens = _decode_queries(q, cache_seqlens, hq, hkv, dev)
    kind, pg, kp, vp, ks, vs = _pool_operands(k_pages, v_pages, k_scales, v_scales, block_table, batch, hkv, d, dev)
    capacity = block_table.shape[1] * k_pages.shape[2]
    if out is None:
        out = torch.empty_like(q) if stream is None else _new(q, q.shape, _BF16, stream)
        op = out.data_ptr()
    else:
        op = _operand(out, "out", dev, _BF16, q.shape)
    n_epilogue, ops = 0, _NO_EPILOGUE
    if epilogue:
        array = (EpiOp * FA_MAX_EPILOGUE)()
        n_epilogue = _fill_epilogue(array, epilogue)
        ops = bytes(array)
    fields = (qp, kp, vp, ks, vs, lens, op, kind, batch, hq, hkv, d, _int(capacity, "max_pages * page_size"),
              _int(max_seqlen, "max_seqlen"), _int(window, "window") if window > 0 else 0,
              1.0 / math.sqrt(d) if scale is None else ctypes.c_float(scale).value, 0, n_epilogue, ops)
    if selected is None:
        top_k, what, fn, more = 0, "fa_attention_decode_paged", _decode_call, ()
    else:
        shape = selected.shape
        if len(shape) != 3 or shape[0] != batch or shape[1] != hkv:
            raise ValueError(f"selected must be [{batch}, {hkv}, top_k]; got {tuple(shape)}")
        top_k, what, fn = shape[2], "fa_attention_decode_selected", _selected_call
        more = (_operand(selected, "selected", dev, _INT32, shape), top_k)
    if workspace is not None:
        p = _pack_decode(*fields, _workspace(workspace, dev), workspace.numel() * workspace.element_size())
    else:
        # only problems too long for one kernel need a workspace (the count of SMs decides)
        p = _pack_decode(*fields, 0, 0)
        if _current_device() == dev:
            nbytes = _decode_size_call(p, pg, top_k)
        else:
            with torch.cuda.device(dev):
                nbytes = _decode_size_call(p, pg, top_k)
        if nbytes:
            workspace = _new(q, nbytes, torch.uint8, stream)
            p = _pack_decode(*fields, workspace.data_ptr(), nbytes)
    _on_device(dev, stream, what, fn, p, pg, *more)
    return out


def check_device_error(stream=None) -> int:
    """Synchronise and return (then clear) the device status: FA_OK,
    FA_ERR_TIMEOUT, or FA_ERR_INVALID (a device-side argument was out of range)."""
    return int(lib.fa_check_device_error(_stream(stream)))


def selftest_watchdog(budget_cycles: int, stream=None) -> int:
    return int(lib.fa_selftest_watchdog(budget_cycles, _stream(stream)))


def kernel_variants_used() -> int:
    return int(lib.fa_kernel_variants_used())


def kernel_launches() -> int:
    return int(lib.fa_kernel_launches())


# --- TurboQuant KV cache -------------------------------------------------------

def tq_codebook(head_dim: int, bits: int) -> torch.Tensor:
    """The 2^bits Lloyd-Max levels (fp32, CPU) of the Beta(head_dim/2,
    head_dim/2) law in u-space.  As fa_tq_codebook in fa.h."""
    out = (ctypes.c_float * (1 << bits))()
    _check(lib.fa_tq_codebook(head_dim, bits, ctypes.cast(out, ctypes.c_void_p)), "fa_tq_codebook")
    return torch.tensor(list(out), dtype=torch.float32)


def tq_compress(x: torch.Tensor, signs: torch.Tensor, levels: torch.Tensor, bits: int,
                codes: Optional[torch.Tensor] = None, norms: Optional[torch.Tensor] = None, stream=None):
    """(codes uint8 [..., d*bits/8], norms fp32 [...]) of rows x [..., d]
    (bf16 or fp32).  signs / levels: fp32 CUDA tensors.  As fa_tq_compress."""
    for name, t in (("x", x), ("signs", signs), ("levels", levels)):
        _contig_cuda(t, name)
    d = x.shape[-1]
    _shape(signs, (d,), "signs")
    _shape(levels, (1 << bits,), "levels")
    if codes is None:
        codes = torch.empty(x.shape[:-1] + (d * bits // 8,), dtype=torch.uint8, device=x.device)
    if norms is None:
        norms = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _shape(codes, tuple(x.shape[:-1]) + (d * bits // 8,), "codes")
    _shape(norms, tuple(x.shape[:-1]), "norms")
    p = TqCompressParams()
    p.x, p.x_dtype, p.rows, p.head_dim, p.bits = x.data_ptr(), _DT[x.dtype], x.numel() // d if d else 0, d, bits
    p.signs, p.levels, p.codes, p.norms = signs.data_ptr(), levels.data_ptr(), codes.data_ptr(), norms.data_ptr()
    _check(lib.fa_tq_compress(ctypes.byref(p), _stream(stream)), "fa_tq_compress")
    return codes, norms


def tq_decode_workspace_size(batch: int, hq: int, head_dim: int, capacity: int) -> int:
    return int(lib.fa_tq_decode_workspace_size(batch, hq, head_dim, capacity))


def tq_attention_decode(q: torch.Tensor, k_codes: torch.Tensor, k_norms: torch.Tensor, v_codes: torch.Tensor,
                        v_norms: torch.Tensor, cache_seqlens: torch.Tensor, *, hq: int, hkv: int, k_bits: int,
                        v_bits: int, k_levels: torch.Tensor, v_levels: torch.Tensor, signs: torch.Tensor,
                        scale: Optional[float] = None, epilogue: Sequence[Tuple[str, float]] = (),
                        out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """One decode step over a TurboQuant cache: q [B*hq, d] (or [B*hq, 1, d])
    bf16, codes [B*hkv, capacity, d*bits/8], norms [B*hkv, capacity].  As
    fa_tq_attention_decode in fa.h."""
    for name, t in (("q", q), ("k_codes", k_codes), ("k_norms", k_norms), ("v_codes", v_codes),
                    ("v_norms", v_norms), ("cache_seqlens", cache_seqlens), ("k_levels", k_levels),
                    ("v_levels", v_levels), ("signs", signs)):
        _contig_cuda(t, name)
    d = q.shape[-1]
    batch = cache_seqlens.numel()
    _cache_shapes(q, None, None, None, None, cache_seqlens, out, hq, hkv)
    _shape(k_codes, (batch * hkv, None, d * k_bits // 8), "k_codes")
    cap = k_codes.shape[1]
    _shape(v_codes, (batch * hkv, cap, d * v_bits // 8), "v_codes")
    _shape(k_norms, (batch * hkv, cap), "k_norms")
    _shape(v_norms, (batch * hkv, cap), "v_norms")
    _shape(k_levels, (1 << k_bits,), "k_levels")
    _shape(v_levels, (1 << v_bits,), "v_levels")
    _shape(signs, (d,), "signs")
    if out is None:
        out = torch.empty_like(q)
    need = tq_decode_workspace_size(batch, hq, d, cap)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    p = TqDecodeParams()
    p.q, p.k_codes, p.k_norms, p.v_codes, p.v_norms = (q.data_ptr(), k_codes.data_ptr(), k_norms.data_ptr(),
                                                       v_codes.data_ptr(), v_norms.data_ptr())
    p.k_levels, p.v_levels, p.signs, p.cache_seqlens = (k_levels.data_ptr(), v_levels.data_ptr(), signs.data_ptr(),
                                                        cache_seqlens.data_ptr())
    p.batch, p.hq, p.hkv, p.head_dim, p.capacity, p.k_bits, p.v_bits = batch, hq, hkv, d, cap, k_bits, v_bits
    p.softmax_scale = float(scale if scale is not None else 1.0 / math.sqrt(d))
    p.out, p.workspace, p.workspace_bytes = out.data_ptr(), workspace.data_ptr(), workspace.numel()
    p.n_epilogue = _fill_epilogue(p.epilogue, epilogue)
    _check(lib.fa_tq_attention_decode(ctypes.byref(p), _stream(stream)), "fa_tq_attention_decode")
    return out

