"""The paged KV cache's operators (the dgen_paged_* calls of include/dgen.h) on torch tensors.

PagedCache describes one layer's cache; paged_append rotates new tokens and writes them into its pages;
paged_attention is the new tokens' attention over it.  Arguments that do not fit raise DgenError (EINVAL)
before anything is launched.  Calls run on the given stream (a cudaStream_t as an int), by default torch's
current stream of the cache's device, and return without waiting.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import DGEN_EINVAL, DgenError, PagedCacheStruct, TokenRows, _check, _lib

_ROW_TYPES = {torch.bfloat16: 0, torch.float16: 1}
_CACHE_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}


def _need(ok: bool, call: str, what: str) -> None:
    if not ok:
        raise DgenError(call, DGEN_EINVAL, what)


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
            page_table.data_ptr(), kv_len.data_ptr(), _CACHE_TYPES[k.dtype], *k.shape[:3], k.shape[3], self.batch,
            page_table.shape[1], stride)
        self._ref = ctypes.addressof(self._c)


def paged_workspace(device=None):
    """A zeroed workspace for paged_attention on `device` (default: the current one).  Calls that can overlap
    on the GPU (other streams, replays of captured graphs) each need one of their own."""
    return torch.zeros(_lib.dgen_paged_workspace_bytes(), dtype=torch.uint8,
                       device="cuda" if device is None else device)


def paged_synchronize(workspace, stream: int | None = None) -> None:
    """Wait for the stream; raises DgenError (EDEVICE) if a device-side bounded wait ran out in a call with this
    workspace since the last check."""
    st = torch.cuda.current_stream(workspace.device).cuda_stream if stream is None else stream
    _launch("dgen_paged_synchronize", workspace.device, workspace.data_ptr(), st)


def _rows(call, cache, name, t, tokens=None, heads=None, dtype=None):
    """The C view of token rows [tokens][heads][head_dim]."""
    _need(t.dim() == 3 and t.shape[2] == cache.head_dim and t.dtype in _ROW_TYPES and t.device == cache.device, call,
          f"{name}: [tokens][heads][{cache.head_dim}] bf16 or fp16 on the cache's device")
    _need((tokens is None or t.shape[0] == tokens) and (heads is None or t.shape[1] == heads) and
          (dtype is None or t.dtype == dtype), call, f"{name}: shape {tuple(t.shape)} or {t.dtype} does not fit")
    st, sh, se = t.stride()
    _need(se == 1, call, f"{name}: the last dimension must be contiguous")
    return TokenRows(t.data_ptr(), st, sh)


def _common(call, cache, rows, cu_new, stream):
    _need(cache.dtype in (rows.dtype, torch.float8_e4m3fn), call, f"{rows.dtype} rows, a cache of {cache.dtype}")
    if cu_new is None:
        _need(rows.shape[0] % cache.batch == 0, call, "without cu_new every sequence has the same number of rows")
        cu = None
    else:
        _need(cu_new.shape == (cache.batch + 1,) and cu_new.dtype == torch.int32 and cu_new.is_contiguous() and
              cu_new.device == cache.device, call, "cu_new: [batch + 1] int32 on the cache's device")
        cu = cu_new.data_ptr()
    if stream is None:
        stream = torch.cuda.current_stream(cache.device).cuda_stream
    return cu, stream


def _launch(call, device, *args):
    if device.index == torch.cuda.current_device():
        _check(call, getattr(_lib, call)(*args))
    else:
        with torch.cuda.device(device):
            _check(call, getattr(_lib, call)(*args))


def paged_append(cache: PagedCache, k, v, q=None, q_out=None, cu_new=None, rope_base: float = 0.0,
                 stream: int | None = None) -> None:
    """Write the new tokens' keys and values, k and v [tokens][n_kv_heads][head_dim], into their pages; with
    rope_base > 0 keys are rotated by their positions on the way, and queries q [tokens][heads][head_dim]
    into q_out (q_out may be q).  Rows belong to sequences by cu_new [batch + 1] (None: the same number
    each); see dgen_paged_append."""
    call = "dgen_paged_append"
    n = k.shape[0]
    kr = _rows(call, cache, "k", k, heads=cache.n_kv_heads)
    vr = _rows(call, cache, "v", v, n, cache.n_kv_heads, k.dtype)
    _need((q is None) == (q_out is None), call, "q and q_out come together")
    heads, qr, qor = 0, None, None
    if q is not None:
        heads = q.shape[1]
        qr = ctypes.byref(_rows(call, cache, "q", q, n, None, k.dtype))
        qor = ctypes.byref(_rows(call, cache, "q_out", q_out, n, heads, k.dtype))
    cu, st = _common(call, cache, k, cu_new, stream)
    _launch(call, cache.device, cache._ref, n, cu, _ROW_TYPES[k.dtype], ctypes.byref(kr), ctypes.byref(vr), heads, qr,
            qor, rope_base, st)


def paged_attention(cache: PagedCache, q, out, workspace, cu_new=None, scale: float | None = None,
                    causal: bool = True, window: int = 0, cap: float = 0.0, lse=None,
                    stream: int | None = None) -> None:
    """out [tokens][heads][head_dim] = attention of the new tokens' queries q (rotated already) over their
    sequences' cached keys: scale (default 1 / sqrt(head_dim)), causal or all keys, a window of positions
    (0: none), scores capped as cap tanh(s / cap) (0: not), lse [tokens][heads] fp32 if given.  workspace:
    paged_workspace() of the cache's device; see dgen_paged_attention."""
    call = "dgen_paged_attention"
    qr = _rows(call, cache, "q", q)
    n, heads = q.shape[0], q.shape[1]
    outr = _rows(call, cache, "out", out, n, heads, q.dtype)
    if lse is not None:
        _need(lse.shape == (n, heads) and lse.dtype == torch.float32 and lse.is_contiguous() and
              lse.device == cache.device, call, "lse: [tokens][heads] fp32")
    _need(workspace.dtype == torch.uint8 and workspace.is_contiguous() and workspace.device == cache.device, call,
          "workspace: paged_workspace() of the cache's device")
    cu, st = _common(call, cache, q, cu_new, stream)
    _launch(call, cache.device, cache._ref, n, cu, _ROW_TYPES[q.dtype], heads, ctypes.byref(qr), ctypes.byref(outr),
            1.0 / math.sqrt(cache.head_dim) if scale is None else scale, 1 if causal else 0, window, cap,
            None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(), st)
