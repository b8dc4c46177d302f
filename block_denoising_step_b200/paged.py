"""The paged KV cache's operators (the dgen_paged_* calls of include/dgen.h) on torch tensors.

PagedCache describes one layer's cache; paged_append rotates new tokens and writes them into its pages;
paged_attention is the new tokens' attention over it.  Arguments that do not fit raise DgenError (EINVAL)
before anything is launched.  Calls run on the given stream (a cudaStream_t as an int), by default torch's
current stream of the cache's device, and return without waiting.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import DGEN_EINVAL, DgenError, PagedCacheStruct, _check, _lib

_append, _attention = _lib.dgen_paged_append, _lib.dgen_paged_attention
_pack = struct.Struct("Qqq").pack
_stream_of = torch._C._cuda_getCurrentRawStream  # torch.cuda.current_stream() without the object around it
_ROW_TYPES = {torch.bfloat16: 0, torch.float16: 1}
_SMALLEST = 2.0 ** -149  # fp32's: less would reach the C call as 0
_CACHE_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}


def _need(ok: bool, call: str, what: str) -> None:
    if not ok:
        raise DgenError(call, DGEN_EINVAL, what)


def _count(call: str, name: str, value: int) -> int:
    _need(value < 1 << 31, call, f"{name}: {value} does not fit 32 bits")
    return value


class PagedCache:
    """One layer's cache: k, v [n_pages][n_kv_heads][page_size][head_dim] contiguous (bf16, fp16 or
    float8_e4m3fn), page_table [batch][pages] int32 (entries outside [0, n_pages) mean no page), kv_len
    [batch] int32 (lengths, the new tokens of a call included); for float8_e4m3fn k_scale and v_scale
    [n_kv_heads] fp32.  Keeps the tensors; table and lengths may be changed in place between calls."""

    def __init__(self, k, v, page_table, kv_len, k_scale=None, v_scale=None):
        call = "PagedCache"
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype, call, "k and v: two alike 4-d tensors")
        _need(k.dtype in _CACHE_TYPES, call, f"no cache of {k.dtype}")
        _need(k.is_contiguous() and v.is_contiguous(), call, "k and v must be contiguous")
        _need(page_table.dim() == 2 and page_table.dtype == torch.int32 and
              (page_table.stride(1) == 1 or page_table.shape[1] == 1), call, "page_table: [batch][pages] int32")
        _need(page_table.shape[0] > 0, call, "page_table: no sequence")
        _need(kv_len.shape == page_table.shape[:1] and kv_len.dtype == torch.int32 and kv_len.is_contiguous(), call,
              "kv_len: [batch] int32")
        e4m3 = k.dtype == torch.float8_e4m3fn
        for s in (k_scale, v_scale):
            _need((s is not None) == e4m3, call, "scales come with float8_e4m3fn and only with it")
            if s is not None:
                _need(s.shape == k.shape[1:2] and s.dtype == torch.float32 and s.is_contiguous(), call,
                      "scales: [n_kv_heads] fp32")
        tensors = [t for t in (k, v, page_table, kv_len, k_scale, v_scale) if t is not None]
        _need(all(t.device == k.device and t.is_cuda for t in tensors), call, "every tensor on one CUDA device")
        self.k, self.v, self.page_table, self.kv_len = k, v, page_table, kv_len
        self.k_scale, self.v_scale = k_scale, v_scale
        self.device, self.dtype = k.device, k.dtype
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.batch = page_table.shape[0]
        # a row of a one-row table may have any stride
        stride = max(page_table.stride(0), page_table.shape[1])
        _need(self.batch == 1 or stride == page_table.stride(0), call, "page_table's rows overlap")
        self._c = PagedCacheStruct(
            k.data_ptr(), v.data_ptr(), *(None if s is None else s.data_ptr() for s in (k_scale, v_scale)),
            page_table.data_ptr(), kv_len.data_ptr(), _CACHE_TYPES[k.dtype],
            *(_count(call, n, x) for n, x in zip(("n_pages", "n_kv_heads", "page_size", "head_dim"), k.shape)),
            _count(call, "batch", self.batch), _count(call, "table_pages", page_table.shape[1]),
            _count(call, "table_stride", stride))
        self._ref = ctypes.addressof(self._c)
        self._dev = k.get_device()
        self._scale = 1.0 / math.sqrt(self.head_dim)
        self._row_types = _ROW_TYPES if e4m3 else (k.dtype,)


def paged_workspace(device=None):
    """A workspace for paged_attention on `device` (default: the current one), zeroed on its current stream: a
    call on another stream waits for that first.  Calls that can overlap on the GPU (other streams, replays of
    captured graphs) each need one of their own."""
    return torch.zeros(_lib.dgen_paged_workspace_bytes(), dtype=torch.uint8,
                       device="cuda" if device is None else device)


def paged_synchronize(workspace, stream: int | None = None) -> None:
    """Wait for the stream; raises DgenError (EDEVICE) if a device-side bounded wait ran out in a call with this
    workspace (a paged_workspace()) since the last check: outputs since then are not valid."""
    _need(workspace.is_cuda and workspace.dtype == torch.uint8 and workspace.is_contiguous() and
          workspace.numel() >= _lib.dgen_paged_workspace_bytes(), "dgen_paged_synchronize",
          "workspace: wants a paged_workspace()")
    st = torch.cuda.current_stream(workspace.device).cuda_stream if stream is None else stream
    _off_device("dgen_paged_synchronize", workspace.device, workspace.data_ptr(), st)


def _bad(call: str, what: str):
    raise DgenError(call, DGEN_EINVAL, what)


def _check_rows(call, cache, name, t, shape, dtype):
    """Raises for token rows that are not [tokens][heads][head_dim] of this shape, type and device."""
    if t.dtype not in _ROW_TYPES:
        _bad(call, f"{name}: rows are bf16 or fp16, not {t.dtype}")
    if t.get_device() != cache._dev:
        _bad(call, f"{name}: on {t.device}, the cache on {cache.device}")
    if t.dim() != 3 or t.shape[2] != cache.head_dim or t.stride(2) != 1:
        _bad(call, f"{name}: wants [tokens][heads][{cache.head_dim}] with a contiguous last dimension")
    if t.shape != shape or t.dtype != dtype:
        _bad(call, f"{name}: {tuple(t.shape)} {t.dtype} where {tuple(shape)} {dtype} belongs")
    _bad(call, f"{name}: does not fit the cache")


def _check_cu(call, cache, cu):
    if cu.shape != (cache.batch + 1,) or cu.dtype != torch.int32 or not cu.is_contiguous() or \
            cu.get_device() != cache._dev:
        _bad(call, f"cu_new: wants [{cache.batch + 1}] int32 on the cache's device")


def _off_device(call, device, *args):
    with torch.cuda.device(device):
        _check(call, getattr(_lib, call)(*args))


# The two calls below run once per layer and step of a serving loop, where their host time counts: the checks
# are plain comparisons, messages are made only on failure, and a view of token rows goes to C as packed bytes
# (struct dgen_token_rows).

def paged_append(cache: PagedCache, k, v, q=None, q_out=None, cu_new=None, rope_base: float = 0.0,
                 stream: int | None = None) -> None:
    """Write the new tokens' keys and values, k and v [tokens][n_kv_heads][head_dim], into their pages; with
    rope_base > 0 keys are rotated by their positions on the way, and queries q [tokens][heads][head_dim]
    into q_out (q_out may be q).  Rows belong to sequences by cu_new [batch + 1] (None: the same number
    each); see dgen_paged_append."""
    dev, dtype, shape, st = cache._dev, k.dtype, k.shape, k.stride()
    if (len(shape) != 3 or shape[1] != cache.n_kv_heads or shape[2] != cache.head_dim or st[2] != 1 or
            dtype not in cache._row_types or k.get_device() != dev):
        _check_rows("dgen_paged_append", cache, "k", k, (shape[0] if len(shape) else 0, cache.n_kv_heads,
                                                         cache.head_dim), dtype)
    n = shape[0]
    if n >> 31:
        _bad("dgen_paged_append", "counts of rows are 32 bits")
    sv = v.stride()
    if v.shape != shape or sv[2] != 1 or v.dtype != dtype or v.get_device() != dev:
        _check_rows("dgen_paged_append", cache, "v", v, shape, dtype)
    kr, vr = _pack(k.data_ptr(), st[0], st[1]), _pack(v.data_ptr(), sv[0], sv[1])
    heads, qr, qor = 0, None, None
    if q is not None:
        if q_out is None:
            _bad("dgen_paged_append", "q and q_out come together")
        qs, sq, so = q.shape, q.stride(), q_out.stride()
        if len(qs) != 3 or qs[0] != n or qs[2] != shape[2] or sq[2] != 1 or q.dtype != dtype or q.get_device() != dev:
            _check_rows("dgen_paged_append", cache, "q", q, (n, qs[1] if len(qs) > 1 else 0, shape[2]), dtype)
        if q_out.shape != qs or so[2] != 1 or q_out.dtype != dtype or q_out.get_device() != dev:
            _check_rows("dgen_paged_append", cache, "q_out", q_out, qs, dtype)
        heads = qs[1]
        if heads >> 31:
            _bad("dgen_paged_append", "counts of heads are 32 bits")
        qr, qor = _pack(q.data_ptr(), sq[0], sq[1]), _pack(q_out.data_ptr(), so[0], so[1])
    elif q_out is not None:
        _bad("dgen_paged_append", "q and q_out come together")
    cu = None
    if cu_new is not None:
        _check_cu("dgen_paged_append", cache, cu_new)
        cu = cu_new.data_ptr()
    elif cache.batch < 1 or n % cache.batch:
        _bad("dgen_paged_append", "without cu_new every sequence has the same number of rows")
    if 0.0 < rope_base < _SMALLEST:
        _bad("dgen_paged_append", "rope_base: fp32 has no such number")
    args = (cache._ref, n, cu, _ROW_TYPES[dtype], kr, vr, heads, qr, qor, rope_base,
            _stream_of(dev) if stream is None else stream)
    if dev != torch.cuda.current_device():
        return _off_device("dgen_paged_append", cache.device, *args)
    status = _append(*args)
    if status:
        raise DgenError("dgen_paged_append", status)


def paged_attention(cache: PagedCache, q, out, workspace, cu_new=None, scale: float | None = None,
                    causal: bool = True, window: int = 0, cap: float = 0.0, lse=None,
                    stream: int | None = None) -> None:
    """out [tokens][heads][head_dim] = attention of the new tokens' queries q (rotated already) over their
    sequences' cached keys: scale (default 1 / sqrt(head_dim)), causal or all keys, a window of positions
    (0: none), scores capped as cap tanh(s / cap) (0: not), lse [tokens][heads] fp32 if given.  workspace:
    paged_workspace() of the cache's device; see dgen_paged_attention."""
    dev, dtype, shape, st, so = cache._dev, q.dtype, q.shape, q.stride(), out.stride()
    if (len(shape) != 3 or shape[2] != cache.head_dim or st[2] != 1 or dtype not in cache._row_types or
            q.get_device() != dev):
        _check_rows("dgen_paged_attention", cache, "q", q,
                    (*shape[:2], cache.head_dim) if len(shape) == 3 else (0, 0, cache.head_dim), dtype)
    if out.shape != shape or so[2] != 1 or out.dtype != dtype or out.get_device() != dev:
        _check_rows("dgen_paged_attention", cache, "out", out, shape, dtype)
    n, heads = shape[0], shape[1]
    if (n | heads) >> 31:
        _bad("dgen_paged_attention", "counts of rows and heads are 32 bits")
    lse_at = None
    if lse is not None:
        if lse.shape != (n, heads) or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.get_device() != dev:
            _bad("dgen_paged_attention", "lse: wants [tokens][heads] fp32 on the cache's device")
        lse_at = lse.data_ptr()
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != dev:
        _bad("dgen_paged_attention", "workspace: wants paged_workspace() of the cache's device")
    cu = None
    if cu_new is not None:
        _check_cu("dgen_paged_attention", cache, cu_new)
        cu = cu_new.data_ptr()
    elif cache.batch < 1 or n % cache.batch:
        _bad("dgen_paged_attention", "without cu_new every sequence has the same number of rows")
    if not 0 <= window < 1 << 31:
        _bad("dgen_paged_attention", "window: wants 0 (none) or a count of positions below 2^31")
    if 0.0 < cap < _SMALLEST:
        _bad("dgen_paged_attention", "cap: fp32 has no such number")
    args = (cache._ref, n, cu, _ROW_TYPES[dtype], heads, _pack(q.data_ptr(), st[0], st[1]),
            _pack(out.data_ptr(), so[0], so[1]), cache._scale if scale is None else scale, 1 if causal else 0, window,
            cap, lse_at, workspace.data_ptr(), workspace.numel(),
            _stream_of(dev) if stream is None else stream)
    if dev != torch.cuda.current_device():
        return _off_device("dgen_paged_attention", cache.device, *args)
    status = _attention(*args)
    if status:
        raise DgenError("dgen_paged_attention", status)
