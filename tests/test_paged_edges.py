"""The paged cache's calls at the edges of what they allow, what needs no GPU."""
import ctypes
import os
import subprocess

import pytest
import torch

import block_denoising_step_b200 as dg
from block_denoising_step_b200 import build
from tests.test_paged import A, _append, _attend, _cache, _rows


# ------------------------------------------------------------------ output rows that overlap

# (token stride, head stride) of two rows of four heads of 64
OVERLAPPING = [(256, 0), (0, 64), (192, 64), (256, 56), (64, 64), (0, 0), (72, 128), (-192, 64)]
APART = [(256, 64), (264, 64), (512, 128), (64, 128), (-256, 64), (256, -64)]


@pytest.mark.parametrize("ts,hs", OVERLAPPING)
def test_output_rows_that_overlap_are_refused(ts, hs):
    r = _rows(ts=ts, hs=hs)
    assert _attend(out=r) == dg.DGEN_EINVAL
    assert _append(q_out=r) == dg.DGEN_EINVAL


@pytest.mark.parametrize("ts,hs", APART)
def test_output_rows_that_do_not_overlap_pass(ts, hs):
    """(The small workspace is what the call is refused for.)"""
    assert _attend(out=_rows(ts=ts, hs=hs), ws_bytes=16) == dg.DGEN_ESCRATCH


def test_inputs_may_overlap():
    """One row for all tokens or heads is read as often as it is named."""
    assert _attend(q=_rows(ts=0, hs=0), ws_bytes=16) == dg.DGEN_ESCRATCH


# ------------------------------------------------------------------ counts at their ends

@pytest.mark.parametrize("heads", [65537, 1 << 29, 1 << 30])
def test_more_kv_heads_than_query_heads_may_be_are_refused(heads):
    """The append counts a token's items in 32 bits: 2^30 heads of 64 would come to none, and be divided by."""
    c, r = _cache(n_pages=1, n_kv_heads=heads, page_size=1), _rows()
    assert dg._lib.dgen_paged_append(ctypes.byref(c), 2, None, 0, r, r, 0, None, None, 0.0, None) == dg.DGEN_EINVAL
    assert _attend(c, heads=heads) == dg.DGEN_EINVAL


# ------------------------------------------------------------------ alignment of what is read by 32-bit words

@pytest.mark.parametrize("field", ["page_table_dev", "kv_len_dev", "k_scale_dev", "v_scale_dev"])
def test_misaligned_words_of_the_cache_are_refused(field):
    c = dict(type=2, k_scale_dev=A, v_scale_dev=A) if "scale" in field else {}
    c[field] = A + 2
    assert _append(_cache(**c)) == dg.DGEN_EINVAL
    assert _attend(_cache(**c), ws_bytes=16) == dg.DGEN_EINVAL


def test_misaligned_counts_and_lse_are_refused():
    assert _append(cu=A + 1) == dg.DGEN_EINVAL
    assert _attend(cu=A + 1, ws_bytes=16) == dg.DGEN_EINVAL
    r = _rows()
    for at, status in ((A + 2, dg.DGEN_EINVAL), (A + 4, dg.DGEN_ESCRATCH)):
        assert dg._lib.dgen_paged_attention(ctypes.byref(_cache()), 2, None, 0, 4, r, r, 0.125, 1, 0, 0.0, at, A, 16,
                                            None) == status


# ------------------------------------------------------------------ the binding's own checks

def _binding_cache(batch=1):
    """A handle as PagedCache makes it, for tensors that no GPU holds: every call here is refused before the C entry."""
    cache = object.__new__(dg.paged.PagedCache)
    cache._dev, cache._row_types, cache.head_dim, cache.batch, cache.n_kv_heads = -1, (torch.bfloat16,), 64, batch, 2
    return cache


def _refused(f, *args, **kw):
    with pytest.raises(dg.DgenError) as e:
        f(*args, **kw)
    assert e.value.status == dg.DGEN_EINVAL


@pytest.mark.parametrize("n", [0, 2])
def test_a_batch_of_no_sequences_is_refused(n):
    q, kv = (torch.zeros(n, h, 64, dtype=torch.bfloat16) for h in (4, 2))
    _refused(dg.paged_attention, _binding_cache(0), q, q.clone(), torch.zeros(64, dtype=torch.uint8))
    _refused(dg.paged_append, _binding_cache(0), kv, kv)


def test_counts_beyond_32_bits_are_refused():
    """They would reach the C call as other counts (2^32 + 2 rows of one expanded token as 2)."""
    for n, h in ((2 ** 32 + 2, 2), (2 ** 31, 2), (2, 2 ** 32 + 2)):
        q = torch.zeros(1, 1, 64, dtype=torch.bfloat16).expand(n, h, 64)
        _refused(dg.paged_attention, _binding_cache(), q, q, torch.zeros(64, dtype=torch.uint8))
        if h == 2:
            kv = torch.zeros(1, 1, 64, dtype=torch.bfloat16).expand(n, 2, 64)
            _refused(dg.paged_append, _binding_cache(), kv, kv)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16).expand(2, 2 ** 32 + 2, 64)
    kv = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    _refused(dg.paged_append, _binding_cache(), kv, kv, q=q, q_out=q)


def test_cache_counts_beyond_32_bits_are_refused():
    """The struct's fields are 32 bits wide: a table row stride of 2^32 + 4 was kept as 4."""
    for field, value in (("table_stride", 2 ** 32 + 4), ("n_pages", 2 ** 32 + 1), ("page_size", 2 ** 31)):
        _refused(dg.paged._count, "PagedCache", field, value)
    assert dg.paged._count("PagedCache", "page_size", 2 ** 31 - 1) == 2 ** 31 - 1


@pytest.mark.parametrize("tiny", [1e-60, 1e-46, 5e-324])
def test_numbers_that_fp32_rounds_to_zero_are_refused(tiny):
    """Zero means no cap and no rotation."""
    q, kv = (torch.zeros(1, h, 64, dtype=torch.bfloat16) for h in (4, 2))
    _refused(dg.paged_attention, _binding_cache(), q, q.clone(), torch.zeros(64, dtype=torch.uint8), cap=tiny)
    _refused(dg.paged_append, _binding_cache(), kv, kv, rope_base=tiny)


def test_synchronize_refuses_what_is_no_workspace():
    """The call reads and writes the workspace's head whatever the tensor's size."""
    for ws in (torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(16, dtype=torch.uint8), torch.zeros(1 << 20)):
        _refused(dg.paged_synchronize, ws)


# ------------------------------------------------------------------ the division of a batch

def test_closed_forms_of_the_unit_walk(tmp_path):
    """Host code of csrc/paged_work.cuh, compiled with a check that sums block by block."""
    if not os.path.exists(build.NVCC):
        pytest.skip("needs nvcc")
    exe = str(tmp_path / "check")
    subprocess.check_call([build.NVCC, "-std=c++17", "-O1", "--expt-relaxed-constexpr", "-gencode",
                           "arch=compute_100a,code=sm_100a", "-I", build.SRC_DIR, "-o", exe,
                           os.path.join(os.path.dirname(os.path.abspath(__file__)), "paged_units_check.cu")])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


# ------------------------------------------------------------------ scales

def test_a_scale_beyond_fp32_in_powers_of_two_is_refused():
    """Scores are kept in powers of two: scale * log2 e is a number of fp32 too."""
    assert _attend(scale=3e38, ws_bytes=16) == dg.DGEN_EINVAL
    assert _attend(scale=2.3e38, ws_bytes=16) == dg.DGEN_ESCRATCH
