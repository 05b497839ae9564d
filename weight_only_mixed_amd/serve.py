"""Serving operators of libslq (include/slq_serve.h): the paged 8-bit key/value
cache (write, read, attention) and token sampling.

The same thin marshalling as the package's other entry points: device tensors
in, the current stream of their device, no fallback.  Each call takes its
workspace from torch's allocator, so calls on several streams, and captured
graphs, never share one.
"""
from __future__ import annotations

import ctypes
import math

import torch

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32

SLQ_KV_INT8, SLQ_KV_E4M3 = 0, 1
SLQ_F32, SLQ_BF16, SLQ_F16 = 0, 1, 2
_DTYPE = {torch.float32: SLQ_F32, torch.bfloat16: SLQ_BF16, torch.float16: SLQ_F16}


class _Cache(ctypes.Structure):
    _fields_ = [("format", _i32), ("heads", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("pages", _i64), ("page_stride", _i64), ("head_stride", _i64),
                ("token_stride", _i64), ("k_codes", _vp), ("v_codes", _vp), ("k_scales", _vp),
                ("v_scales", _vp)]


class _Seqs(ctypes.Structure):
    _fields_ = [("batch", _i32), ("max_pages", _i32), ("table_stride", _i64), ("table", _vp),
                ("lens", _vp), ("cu", _vp)]


def declare(L):
    """Argument types of the entry points of slq_serve.h."""
    L.slq_kv_write.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int, _i64, _i64, _i64, _i64, _i64, _i64, _vp]
    L.slq_kv_read.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int, _i64, _i64, _vp]
    L.slq_kv_attention_workspace_bytes.argtypes = [_vp, _vp, _i64, _i32, _i32, _i64, _i64]
    L.slq_kv_attention_workspace_bytes.restype = ctypes.c_size_t
    L.slq_kv_attention.argtypes = [_vp, _vp, _vp, ctypes.c_int, _i64, _i32, _i64, _i64,
                                   ctypes.c_float, _i32, _i64, _i64, _vp, _vp, _vp, _vp]
    L.slq_sample_workspace_bytes.argtypes = [_i64, _i64]
    L.slq_sample_workspace_bytes.restype = ctypes.c_size_t
    L.slq_sample.argtypes = [_vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                             _vp, _vp]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        from . import lib
        _LIB = lib()
    return _LIB


def _need(ok: bool, what: str):
    if not ok:
        from . import SLQ_EINVAL, SlqError
        raise SlqError(SLQ_EINVAL, what)


_raw_stream = torch._C._cuda_getCurrentRawStream   # the current stream's handle, without a Stream object


def _call(device, what: str, fn, *args):
    """fn(*args, current stream) with `device` current; raises on any status but SLQ_OK."""
    index = device.index
    if torch.cuda.current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        from . import SlqError
        raise SlqError(status, what)


class KvCache:
    """A paged 8-bit cache.  k_codes, v_codes: uint8 [pages, heads, page_size,
    head_dim], the last dimension contiguous, any order of heads and slots,
    equal strides; k_scales, v_scales: float32 [pages, heads], contiguous.
    Describes the caller's tensors and holds them; nothing is copied."""

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scales: torch.Tensor,
                 v_scales: torch.Tensor, fmt: int):
        shape, strides, dev = k_codes.shape, k_codes.stride(), k_codes.device
        if not (k_codes.dtype == v_codes.dtype == torch.uint8 and len(shape) == 4):
            _need(False, "KvCache: codes are uint8 [pages, heads, page_size, head_dim]")
        if not (v_codes.shape == shape and v_codes.stride() == strides and strides[3] == 1):
            _need(False, "KvCache: k and v codes need equal shapes and strides, the last dimension contiguous")
        pages, heads, page_size, dim = shape
        for s in (k_scales, v_scales):
            if not (s.dtype == torch.float32 and s.shape == (pages, heads) and s.is_contiguous() and
                    s.device == dev):
                _need(False, "KvCache: scales are contiguous float32 [pages, heads] on the codes' GPU")
        if not (k_codes.is_cuda and v_codes.device == dev):
            _need(False, "KvCache: all tensors on one GPU")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.fmt, self.device = fmt, dev
        self.pages, self.heads, self.page_size, self.head_dim = pages, heads, page_size, dim
        self._c = _Cache(fmt, heads, dim, page_size, pages, strides[0], strides[1], strides[2],
                         k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(),
                         v_scales.data_ptr())
        self._ref = ctypes.addressof(self._c)


def alloc_kv_cache(pages: int, heads: int, head_dim: int, page_size: int = 64,
                   fmt: int = SLQ_KV_INT8, device="cuda") -> KvCache:
    """A cache in newly allocated tensors (contents unset, as free pages are)."""
    codes = [torch.empty((pages, heads, page_size, head_dim), dtype=torch.uint8, device=device)
             for _ in range(2)]
    scales = [torch.empty((pages, heads), dtype=torch.float32, device=device) for _ in range(2)]
    return KvCache(*codes, *scales, fmt)


class KvSeqs:
    """A ragged batch: table int32 [batch, max_pages], lens int32 [batch]
    (tokens of each sequence after this step), cu int32 [batch + 1] (row
    offsets of this step's tokens, the last ones of each sequence)."""

    def __init__(self, table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor):
        if not (table.dtype == lens.dtype == cu.dtype == torch.int32):
            _need(False, "KvSeqs: int32 tensors")
        shape, batch = table.shape, lens.shape[0] if lens.dim() == 1 else -1
        if not (len(shape) == 2 and shape[0] == batch and cu.shape == (batch + 1,)):
            _need(False, "KvSeqs: table [batch, max_pages], lens [batch], cu [batch + 1]")
        width, strides, dev = shape[1], table.stride(), table.device
        if not ((width <= 1 or strides[1] == 1) and lens.is_contiguous() and cu.is_contiguous()):
            _need(False, "KvSeqs: table rows, lens and cu contiguous")
        if not (table.is_cuda and lens.device == dev and cu.device == dev):
            _need(False, "KvSeqs: one GPU")
        self.table, self.lens, self.cu, self.device = table, lens, cu, dev
        self.batch, self.max_pages = batch, width
        self._c = _Seqs(batch, width, strides[0] if batch > 1 else width, table.data_ptr(),
                        lens.data_ptr(), cu.data_ptr())
        self._ref = ctypes.addressof(self._c)


def _rows(t: torch.Tensor, cache: KvCache, what: str):
    if not (t.dim() == 3 and t.shape[2] == cache.head_dim and t.dtype in _DTYPE and
            t.device == cache.device and t.stride(2) == 1):
        _need(False, f"{what}: [rows, heads, head_dim], the last dimension contiguous, on the cache's GPU")


def slq_kv_write(cache: KvCache, seqs: KvSeqs, k: torch.Tensor, v: torch.Tensor,
                 max_new: int | None = None) -> None:
    """Quantize the new rows k, v [rows, heads, head_dim] (fp32, bf16 or fp16;
    strided) into the cache as the last tokens of each sequence.  max_new: the
    most rows of one sequence, if known (a hint for the grid)."""
    _rows(k, cache, "slq_kv_write: k")
    _rows(v, cache, "slq_kv_write: v")
    _need(k.shape == v.shape and k.dtype == v.dtype and k.shape[1] == cache.heads and
          seqs.device == cache.device, "slq_kv_write: k and v of one shape and type, cache heads")
    rows = k.shape[0]
    ks, vs = k.stride(), v.stride()
    _call(cache.device, "slq_kv_write", _lib().slq_kv_write, cache._ref, seqs._ref, k.data_ptr(),
          v.data_ptr(), _DTYPE[k.dtype], rows, ks[0], ks[1], vs[0], vs[1],
          max(1, rows) if max_new is None else max_new)


def slq_kv_read(cache: KvCache, seqs: KvSeqs, rows: int, dtype: torch.dtype = torch.bfloat16,
                max_rows: int | None = None, out=None):
    """Read the last cu[b+1] - cu[b] tokens of each sequence back: (k, v), each
    [rows, heads, head_dim] of dtype.  out: a pair of such tensors to fill; rows
    that belong to no sequence keep their contents."""
    _need(dtype in _DTYPE and seqs.device == cache.device, "slq_kv_read: dtype or device")
    shape = (rows, cache.heads, cache.head_dim)
    if out is None:
        out = (torch.empty(shape, dtype=dtype, device=cache.device),
               torch.empty(shape, dtype=dtype, device=cache.device))
    for t in out:
        _need(tuple(t.shape) == shape and t.dtype == dtype and t.device == cache.device and
              t.is_contiguous(), "slq_kv_read: out is contiguous [rows, heads, head_dim] of dtype")
    k, v = out
    _call(cache.device, "slq_kv_read", _lib().slq_kv_read, cache._ref, seqs._ref, k.data_ptr(),
          v.data_ptr(), _DTYPE[dtype], rows, max(1, rows) if max_rows is None else max_rows)
    return k, v


def slq_kv_attention(cache: KvCache, seqs: KvSeqs, q: torch.Tensor, scale: float | None = None,
                     window: int = 0, max_q: int | None = None, max_len: int | None = None,
                     out: torch.Tensor | None = None, with_lse: bool = False):
    """Causal attention of q [rows, heads_q, head_dim] (bf16 or fp16; strided),
    the last tokens of each sequence, over the cache: out of q's type, and with
    with_lse also the log of each row's softmax sum, fp32 [rows, heads_q].
    scale: 1 / sqrt(head_dim) by default.  window: tokens a query sees back,
    itself included (0: all).  max_q, max_len: the most rows and the longest
    length of one sequence, if known (hints for the grid)."""
    _rows(q, cache, "slq_kv_attention: q")
    _need(seqs.device == cache.device, "slq_kv_attention: one GPU")
    rows, hq, dim = q.shape
    if out is None:
        out = torch.empty((rows, hq, dim), dtype=q.dtype, device=q.device)
    else:
        _need(out.shape == q.shape and out.dtype == q.dtype and out.device == q.device and
              out.is_contiguous(), "slq_kv_attention: out is contiguous, of q's shape and type")
    lse = torch.empty((rows, hq), dtype=torch.float32, device=q.device) if with_lse else None
    mq = max(1, rows) if max_q is None else max_q
    ml = max(1, seqs.max_pages * cache.page_size) if max_len is None else max_len
    L = _lib()
    nbytes = L.slq_kv_attention_workspace_bytes(cache._ref, seqs._ref, rows, hq, window, mq, ml)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
    qs = q.stride()
    _call(cache.device, "slq_kv_attention", L.slq_kv_attention, cache._ref, seqs._ref, q.data_ptr(),
          _DTYPE[q.dtype], rows, hq, qs[0], qs[1], 1.0 / math.sqrt(dim) if scale is None else scale,
          window, mq, ml, out.data_ptr(), None if lse is None else lse.data_ptr(),
          None if ws is None else ws.data_ptr())
    return (out, lse) if with_lse else out


def slq_sample(logits: torch.Tensor, u: torch.Tensor, temperature: torch.Tensor | None = None,
               top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
               min_p: torch.Tensor | None = None):
    """One token per row of logits [rows, vocab] (fp32, bf16 or fp16; rows may be
    strided) from uniform numbers u float32 [rows]: (tokens int32 [rows],
    logprobs float32 [rows]).  temperature, top_p, min_p float32 [rows], top_k
    int32 [rows]; None leaves a cut out (temperature: 1)."""
    _need(logits.dim() == 2 and logits.dtype in _DTYPE and logits.device.type == "cuda" and
          logits.shape[1] >= 1 and (logits.shape[1] == 1 or logits.stride(1) == 1),
          "slq_sample: logits [rows, vocab] on a GPU, rows contiguous")
    rows, vocab = logits.shape
    dev = logits.device
    for t, ty in ((u, torch.float32), (temperature, torch.float32), (top_k, torch.int32),
                  (top_p, torch.float32), (min_p, torch.float32)):
        _need((t is None and t is not u) or (t is not None and t.dtype == ty and
              tuple(t.shape) == (rows,) and t.device == dev and t.is_contiguous()),
              "slq_sample: u, temperature, top_p, min_p float32 and top_k int32, contiguous [rows]")
    tokens = torch.empty(rows, dtype=torch.int32, device=dev)
    logprobs = torch.empty(rows, dtype=torch.float32, device=dev)
    L = _lib()
    nbytes = L.slq_sample_workspace_bytes(rows, vocab)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None

    def ptr(t):
        return None if t is None else t.data_ptr()

    _call(dev, "slq_sample", L.slq_sample, logits.data_ptr(), _DTYPE[logits.dtype], rows, vocab,
          logits.stride(0), u.data_ptr(), ptr(temperature), ptr(top_k), ptr(top_p), ptr(min_p),
          tokens.data_ptr(), logprobs.data_ptr(), ptr(ws))
    return tokens, logprobs


__all__ = ["KvCache", "KvSeqs", "alloc_kv_cache", "slq_kv_write", "slq_kv_read", "slq_kv_attention",
           "slq_sample", "SLQ_KV_INT8", "SLQ_KV_E4M3", "SLQ_F32", "SLQ_BF16", "SLQ_F16"]
