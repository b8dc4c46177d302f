"""The paged cache's operators, what needs no GPU: refusals of the C entries and of the binding, and the
64-bit reference itself."""
import ctypes
import math

import pytest
import torch

import block_denoising_step_b200 as dg
from tests import paged_reference as ref

A = 0x10000  # an aligned address that nothing touches: every call here is refused first


def _cache(**kw):
    c = dict(k_dev=A, v_dev=A, k_scale_dev=None, v_scale_dev=None, page_table_dev=A, kv_len_dev=A, type=0, n_pages=8,
             n_kv_heads=2, page_size=16, head_dim=64, batch=2, table_pages=4, table_stride=4)
    c.update(kw)
    return dg.PagedCacheStruct(**c)


def _rows(dev=A, ts=256, hs=64):
    return ctypes.byref(dg.TokenRows(dev, ts, hs))


def _append(cache=None, n=2, cu=None, type=0, k=None, v=None, heads=4, q=None, q_out=None, base=1e4):
    r = _rows()
    return dg._lib.dgen_paged_append(ctypes.byref(cache or _cache()), n, cu, type, k or r, v or r, heads, q or r,
                                     q_out or r, base, None)


def _attend(cache=None, n=2, cu=None, type=0, heads=4, q=None, out=None, scale=0.125, causal=1, window=0, cap=0.0,
            ws=A, ws_bytes=None):
    r = _rows()
    size = dg._lib.dgen_paged_workspace_bytes() if ws_bytes is None else ws_bytes
    return dg._lib.dgen_paged_attention(ctypes.byref(cache or _cache()), n, cu, type, heads, q or r, out or r, scale,
                                        causal, window, cap, None, ws, size, None)


BAD_CACHES = [dict(k_dev=None), dict(v_dev=A + 8), dict(page_table_dev=None), dict(kv_len_dev=None), dict(type=3),
              dict(type=2), dict(type=2, k_scale_dev=A), dict(k_scale_dev=A, v_scale_dev=A), dict(head_dim=96),
              dict(n_pages=0), dict(n_kv_heads=0), dict(page_size=0), dict(batch=0), dict(table_pages=0),
              dict(table_stride=3), dict(n_pages=1 << 30, page_size=16), dict(page_size=1 << 30, table_pages=4)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_caches_are_refused(bad):
    assert _append(_cache(**bad)) == dg.DGEN_EINVAL
    assert _attend(_cache(**bad)) == dg.DGEN_EINVAL


@pytest.mark.parametrize("bad", [dict(n=-1), dict(n=3), dict(type=1), dict(type=2), dict(k=_rows(A + 2)),
                                 dict(v=_rows(ts=100)), dict(q=_rows(hs=63)), dict(q_out=_rows(None)), dict(heads=0),
                                 dict(heads=-4), dict(base=-1.0), dict(base=math.nan), dict(base=math.inf)])
def test_append_refuses(bad):
    assert _append(**bad) == dg.DGEN_EINVAL


@pytest.mark.parametrize("bad", [dict(n=-1), dict(n=3), dict(type=1), dict(type=2), dict(q=_rows(A + 2)),
                                 dict(out=_rows(ts=100)), dict(heads=3), dict(heads=0), dict(scale=math.inf),
                                 dict(scale=math.nan), dict(scale=0.0), dict(scale=-1.0), dict(causal=2), dict(window=-1), dict(cap=-1.0),
                                 dict(cap=math.nan), dict(cap=math.inf), dict(ws=None), dict(ws=A + 8),
                                 dict(n=1 << 30)])
def test_attention_refuses(bad):
    assert _attend(**bad) == dg.DGEN_EINVAL


def test_small_workspace_is_refused():
    assert _attend(ws_bytes=16) == dg.DGEN_ESCRATCH


def test_synchronize_refuses_a_bad_workspace():
    assert dg._lib.dgen_paged_synchronize(None, None) == dg.DGEN_EINVAL
    assert dg._lib.dgen_paged_synchronize(A + 4, None) == dg.DGEN_EINVAL


def test_strides_of_single_rows_do_not_matter():
    one = _cache(batch=1, n_kv_heads=1)
    r = _rows(ts=3, hs=5)
    assert _append(one, n=1, k=r, v=r, heads=1, q=r, q_out=_rows(None, 3, 5)) == dg.DGEN_EINVAL  # for the null alone
    assert _attend(one, n=1, heads=1, q=r, out=r, ws_bytes=16) == dg.DGEN_ESCRATCH


def test_no_tokens_is_nothing_to_do():
    assert _append(n=0) == dg.DGEN_OK
    assert _attend(n=0) == dg.DGEN_OK
    assert dg._lib.dgen_paged_append(None, 0, None, 0, None, None, 0, None, None, 0.0, None) == dg.DGEN_EINVAL
    assert dg._lib.dgen_paged_attention(None, 0, None, 0, 1, None, None, 1.0, 0, 0, 0.0, None, None, 0,
                                        None) == dg.DGEN_EINVAL


def test_cache_struct_matches_the_header():
    assert ctypes.sizeof(dg.PagedCacheStruct) == 6 * 8 + 8 * 4
    assert ctypes.sizeof(dg.TokenRows) == 24


def test_binding_refuses_what_is_not_a_cuda_cache():
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for args in ((k, k, table, lens), (k.float(), k.float(), table, lens), (k[0], k[0], table, lens),
                 (k, k.half(), table, lens), (k, k, table.long(), lens), (k, k, table, lens[:0]),
                 (k.transpose(1, 2), k.transpose(1, 2), table, lens)):
        with pytest.raises(dg.DgenError) as e:
            dg.PagedCache(*args)
        assert e.value.status == dg.DGEN_EINVAL


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32 + 5, -2 ** 32 + 5, -1])
def test_binding_refuses_windows_beyond_32_bits(window):
    """They would reach the C call as another window (2^32 + 5 as 5)."""
    cache = object.__new__(dg.paged.PagedCache)
    cache._dev, cache._row_types, cache.head_dim, cache.batch = -1, (torch.bfloat16,), 64, 1
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(dg.DgenError) as e:
        dg.paged_attention(cache, q, q.clone(), torch.zeros(64, dtype=torch.uint8), window=window)
    assert e.value.status == dg.DGEN_EINVAL


class _Cpu:
    def __init__(self, k, v, table, lens):
        self.k, self.v, self.page_table, self.kv_len, self.k_scale, self.v_scale = k, v, table, lens, None, None


def test_reference_attention_by_hand():
    """One head, keys in three pages out of order, against a direct evaluation."""
    g = torch.Generator().manual_seed(1)
    k = torch.randn(4, 1, 2, 64, generator=g, dtype=torch.float64)
    v = torch.randn(4, 1, 2, 64, generator=g, dtype=torch.float64)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32)
    q = torch.randn(2, 1, 64, generator=g, dtype=torch.float64)
    out, lse, _ = ref.attention(_Cpu(k, v, table, torch.tensor([5])), q, [2])
    keys = torch.stack([k[2, 0, 0], k[2, 0, 1], k[0, 0, 0], k[0, 0, 1], k[3, 0, 0]])
    vals = torch.stack([v[2, 0, 0], v[2, 0, 1], v[0, 0, 0], v[0, 0, 1], v[3, 0, 0]])
    for i, n in ((0, 4), (1, 5)):
        s = (keys[:n] @ q[i, 0]) / 8
        assert torch.allclose(lse[i, 0], torch.logsumexp(s, 0), atol=1e-12)
        assert torch.allclose(out[i, 0], torch.softmax(s, 0) @ vals[:n], atol=1e-12)


def test_reference_attention_masks():
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(2, 1, 8, 64, generator=g, dtype=torch.float64) for _ in range(2))
    q = torch.randn(1, 1, 64, generator=g, dtype=torch.float64)
    table = torch.tensor([[1, -1]], dtype=torch.int32)
    out, lse, _ = ref.attention(_Cpu(k, v, table, torch.tensor([12])), q, [1], window=4)
    assert lse[0, 0] == -math.inf and not out.any()  # the window lies in the absent page
    out, lse, _ = ref.attention(_Cpu(k, v, table, torch.tensor([12])), q, [1], window=5)
    assert torch.allclose(out[0, 0], v[1, 0, 7])  # one key left


def test_reference_rotation_turns_by_the_position():
    x = torch.zeros(1, 1, 64, dtype=torch.float64)
    x[..., 0] = 1
    y = ref.rotate(x, torch.tensor([3]), 10000.0)
    assert torch.allclose(y[0, 0, 0], torch.cos(torch.tensor(3.0, dtype=torch.float64)))
    assert torch.allclose(y[0, 0, 32], torch.sin(torch.tensor(3.0, dtype=torch.float64)))
