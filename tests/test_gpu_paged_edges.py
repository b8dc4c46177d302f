"""The paged cache's operators at the edges of what their calls allow, against bounds that count each rounding."""
import math

import pytest
import torch

import block_denoising_step_b200 as dg
from tests import paged_bounds as bounds
from tests import paged_reference as ref
from tests.test_gpu_paged import TYPES, _gen, cu_of, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def workspace():
    return dg.paged_workspace()


def check(cache, q, new, workspace, uniform=False, **kw):
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    dg.paged_attention(cache, q, out, workspace, cu_new=None if uniform else cu_of(new), lse=lse, **kw)
    dg.paged_synchronize(workspace)
    steps = [bounds.p_step(cache, q, n * q.shape[1] // cache.n_kv_heads) for n in new if n]
    step, half = max(s for s, _ in steps), steps[0][1]
    want, want_lse, bound, lse_bound = bounds.attention(cache, q, new, p_step=step, p_half=half, **kw)
    n = sum(new)
    bad = (out.double() - want).abs()[:n] > (ref.half_step(q.dtype, want) * (1 + 2.0 ** -7) + bound)[:n]
    assert not bad.any() and not out[:n].isnan().any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    live = want_lse[:n] > -math.inf
    assert torch.equal(lse[:n] == -math.inf, ~live)
    assert not ((lse[:n].double() - want_lse[:n]).abs()[live] > lse_bound[:n][live]).any()
    assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()
    return out, lse


# ------------------------------------------------------------------ capped scores

# (cap, scale, deviation of the queries): scores far below the cap, all about zero, saturated; powers of scale / cap
# beyond fp32's range
CAPS = [(1e5, None, 2.0), (18000.0, None, 2.0), (1e30, None, 2.0), (3e38, None, 2.0), (1e-6, None, 0.0),
        (1e-6, None, 1e-7), (1e-30, None, 2.0), (1e-42, None, 2.0), (1e-42, None, 0.0), (50.0, 1e-4, 2.0), (50.0, 3e-4, 2.0),
        (1.0, 1e-30, 2.0), (4.0, None, 2.0)]


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("cap,scale,dev", CAPS)
@pytest.mark.parametrize("new", [[70, 40], [1, 1]], ids=["many", "few"])
def test_caps_of_any_size(hd, cap, scale, dev, new, workspace):
    for kind in ("bf16", "f16"):
        cache = make_cache(kind, [300, 200], 2, hd, 16, seed=100)
        cache.page_table[1, 3] = -1
        q = (dev * torch.randn(sum(new), 6, hd, generator=_gen(101), device="cuda")).to(TYPES[kind][0])
        check(cache, q, new, workspace, cap=cap, scale=scale)
        check(cache, q, new, workspace, cap=cap, scale=scale, causal=False, window=90)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group,new", [(3, [45, 20]), (7, [60, 1]), (4, [100, 33])])
def test_capped_results_depend_on_the_sequences_alone(kind, group, new, workspace):
    """Keys behind the end, padding rows, the other sequence and earlier calls change no bit."""
    t = TYPES[kind][0]
    cache = make_cache(kind, [333, 90], 1, 128, 16, seed=110)
    cache.k.nan_to_num_(0.0), cache.v.nan_to_num_(0.0)
    ids, n = cache.page_table.cpu(), sum(new)
    q = torch.full((n + 40, group, 128), 0.0, device="cuda", dtype=t)
    q[:n] = (2 * torch.randn(n, group, 128, generator=_gen(111), device="cuda")).to(t)
    other = make_cache(kind, [1000], 1, 128, 16, seed=112, std=50.0)
    noise = (50 * torch.randn(200, group, 128, generator=_gen(113), device="cuda")).to(t)
    first = None
    for tail, pad, disturb in ((0.0, 0.0, False), (200.0, 100.0, True), (-200.0, math.nan, True), (math.nan, -3.0, False)):
        for b, length in ((0, 333), (1, 90)):
            cache.k[ids[b, length // 16], :, length % 16:] = tail
            cache.v[ids[b, length // 16], :, length % 16:] = tail
        q[n:] = pad
        if disturb:
            dg.paged_attention(other, noise, torch.empty_like(noise), workspace, cap=9.0)
        got = check(cache, q, new, workspace, cap=30.0, causal=True)
        if first is None:
            first = got
        assert torch.equal(got[0][:n], first[0][:n]) and torch.equal(got[1][:n], first[1][:n])
    q[new[0]:n] *= 100  # the other sequence's scores pass the cap
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    dg.paged_attention(cache, q, out, workspace, cu_new=cu_of(new), lse=lse, cap=30.0)
    assert torch.equal(out[:new[0]], first[0][:new[0]]) and torch.equal(lse[:new[0]], first[1][:new[0]])


# ------------------------------------------------------------------ weights in 16 bits

@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("below", [64.5, 6.5, 0.48])
def test_light_keys_beside_heavy_ones(kind, hd, new, below, workspace):
    """Every 16th key outweighs the others by 2^24 / below and has no value: the output is the light keys' alone."""
    t, ct = TYPES[kind]
    length = 640 + new
    cache = make_cache(kind, [length], 1, hd, 16, seed=120)
    g = _gen(121)
    heavy = torch.arange(16, device="cuda") % 16 == 5
    cache.k.copy_(torch.zeros(cache.k.shape, device="cuda"))
    cache.k[..., ~heavy, 0] = torch.full((1,), -1.0, device="cuda").to(ct)
    value = 64 * (1 + torch.rand(cache.v.shape, generator=g, device="cuda"))
    value[..., heavy, :] = 0
    cache.v.copy_(value)
    if cache.k_scale is not None:
        cache.k_scale.fill_(1.0), cache.v_scale.fill_(512.0)
    else:
        cache.v.mul_(16)
    q = torch.zeros(new, 2, hd, device="cuda", dtype=t)
    q[..., 0] = 1
    check(cache, q, [new], workspace, causal=False, scale=math.log(2) * math.log2(2 ** 24 / below))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_weights_of_few_rows_keep_16_bits(kind, hd, workspace):
    """Two keys whose values nearly cancel: what a weight's rounding loses is left over."""
    cache = make_cache(kind, [2], 1, hd, 8, seed=130)
    ct, page = TYPES[kind][1], int(cache.page_table[0, 0])
    cache.k[page, 0, :2], cache.v[page, 0, :2] = torch.zeros(2, hd, device="cuda").to(ct), 0.0
    if cache.k_scale is not None:
        cache.k_scale.fill_(1.0), cache.v_scale.fill_(1.0)
    cache.k[page, 0, 1, 0] = -1.0
    cache.v[page, 0, 0], cache.v[page, 0, 1] = 0.75, -1.0
    q = torch.zeros(1, 8, hd, device="cuda", dtype=TYPES[kind][0])
    q[0, :, 0] = 0.2 + 0.03 * torch.arange(8, device="cuda").to(q.dtype)
    check(cache, q, [1], workspace, scale=1.0)


@pytest.mark.parametrize("kind", ["bf16-e4m3", "f16-e4m3"])
@pytest.mark.parametrize("new", [1, 30])
@pytest.mark.parametrize("large", [2.0 ** 13, 2.0 ** 17, 2.0 ** 20])
def test_queries_with_one_large_element_over_e4m3(kind, new, large, workspace):
    """Where the large element's key coordinates are zero, the small ones make the score."""
    if kind == "f16-e4m3":
        large = min(large, 32768.0)
    cache = make_cache(kind, [200], 1, 128, 16, seed=140)
    cache.k.view(torch.uint8)[..., 0] = 0
    cache.k_scale.fill_(0.5)
    q = torch.zeros(new, 2, 128, device="cuda")
    q[..., 1:5] = 2.0 ** -10 * torch.randn(new, 2, 4, generator=_gen(141), device="cuda")
    q[..., 0] = large
    check(cache, q.to(TYPES[kind][0]), [new], workspace, scale=16.0)


@pytest.mark.parametrize("power", [-120, -60, 60, 118, 126])
def test_queries_of_any_magnitude_over_e4m3(power, workspace):
    """bf16 reaches as far as fp32: the row's scale follows it."""
    cache = make_cache("bf16-e4m3", [200], 1, 128, 16, seed=150)
    q = (torch.randn(1, 2, 128, generator=_gen(151), device="cuda").clamp(-1.9, 1.9) * 2.0 ** power).bfloat16()
    check(cache, q, [1], workspace, scale=2.0 ** -power / 8)


# ------------------------------------------------------------------ workspaces

ERROR_WORD, JOIN_LIST, HEAD = 1023, 4096, 4096 + 1023 * 64


def test_nothing_is_joined_after_a_wait_ran_out():
    """With an error in the workspace the pieces of cut row tiles are left alone: whoever wrote the list of them, the
    rows it names are not written.  The check empties the list too."""
    ws = dg.paged_workspace()
    cache = make_cache("bf16", [2304], 2, 128, 16, seed=160)
    q = torch.randn(256, 4, 128, generator=_gen(161), device="cuda").bfloat16()
    good, out = torch.empty_like(q), torch.full_like(q, 7.0)
    dg.paged_attention(cache, q, good, ws, causal=False)
    dg.paged_synchronize(ws)
    assert ws[JOIN_LIST:HEAD].any()
    ws[:JOIN_LIST].view(torch.int32)[ERROR_WORD] = 22
    dg.paged_attention(cache, q, out, ws, causal=False)
    with pytest.raises(dg.DgenError) as e:
        dg.paged_synchronize(ws)
    assert e.value.status == dg.DGEN_EDEVICE
    assert (out == 7.0).all()  # two units over all CTAs: every row tile is cut
    assert not ws[:HEAD].any()
    dg.paged_attention(cache, q, out, ws, causal=False)
    dg.paged_synchronize(ws)
    assert torch.equal(out, good)


def test_synchronize_refuses_part_of_a_workspace():
    ws = dg.paged_workspace()
    for part in (ws[:64], ws[16:], ws[:: 2]):
        with pytest.raises(dg.DgenError) as e:
            dg.paged_synchronize(part)
        assert e.value.status == dg.DGEN_EINVAL
    dg.paged_synchronize(ws)


# ------------------------------------------------------------------ the append's division

# powers of two and thirds of them (ties with many rows), both sides of 2^-100 and 2^100, the ends of fp32's range
SCALES = [1.0, 2.0 ** -7, 3.0, 1 / 3, 0.75, 0.0123, 0.0178, 17.3, 1.0000001, 0.99999994, 5e-3, 448.0, -0.5, 2.0 ** -99,
          2.0 ** -101, 1.7e-30, 3e-31, 2.0 ** 99, 1.3 * 2.0 ** 100, 1e-40, 1e38, 3e38, 0.0, math.inf]


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_e4m3_values_are_the_divisions_to_the_bit(t):
    """Every bf16 / fp16 value over every scale: the stored byte is that of x / scale in fp32, rounded and saturated."""
    hkv, hd = len(SCALES), 256
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(t).view(-1, 1, hd).expand(-1, hkv, -1)
    n = x.shape[0]
    scale = torch.tensor(SCALES)
    k = torch.zeros(n, hkv, 1, hd, dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros_like(k)
    cache = dg.PagedCache(k, v, torch.arange(n, dtype=torch.int32, device="cuda")[None],
                          torch.tensor([n], dtype=torch.int32, device="cuda"), scale.cuda(), scale.flip(0).cuda())
    rows = x.contiguous().cuda()
    dg.paged_append(cache, rows, rows)
    for got, s in ((k, scale), (v, scale.flip(0))):
        q = x.float() / s[None, :, None]
        want = q.clamp(-448, 448).to(torch.float8_e4m3fn)  # (clamp keeps NaN)
        same = got.cpu()[:, :, 0].view(torch.uint8) == want.view(torch.uint8)
        nan = want.float().isnan()
        assert torch.equal(got.cpu()[:, :, 0].float().isnan(), nan)
        assert (same | nan).all(), [(SCALES[h], int((~same & ~nan)[:, h].sum())) for h in range(hkv)]


# ------------------------------------------------------------------ batches and contexts as they are used

@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("hd,group,new", [(256, 2, 256), (256, 2, 250), (128, 4, 120), (64, 8, 64), (128, 3, 83), (64, 1, 255)])
@pytest.mark.parametrize("masks", [dict(causal=False), dict(causal=True), dict(causal=True, window=300),
                                   dict(causal=False, window=100, cap=20.0)], ids=["all", "causal", "window", "capped"])
def test_canvases_over_prompts_of_unequal_length(kind, hd, group, new, masks, workspace):
    """As many new tokens in every sequence and no cu_new: neighbouring row tiles go to teams of CTAs (two to four)."""
    lens = [new + p for p in (2048, 44, 0, 855, 1, 300)]
    cache = make_cache(kind, lens, 2, hd, 16, seed=170)
    cache.page_table[3, 5:9] = -1
    q = (2 * torch.randn(new * len(lens), 2 * group, hd, generator=_gen(171), device="cuda")).to(TYPES[kind][0])
    check(cache, q, [new] * len(lens), workspace, uniform=True, **masks)


@pytest.mark.parametrize("kind", ["bf16", "f16-e4m3"])
@pytest.mark.parametrize("new", [1, 20])
def test_batches_of_more_sequences_than_a_warp_has_lanes(kind, new, workspace):
    """Two chunks of lengths and a bit, some sequences empty in between."""
    g = torch.Generator().manual_seed(180)
    lens = torch.randint(new, 400, (71,), generator=g).tolist()
    cache = make_cache(kind, lens, 1, 64, 16, seed=181)
    q = (2 * torch.randn(71 * new, 4, 64, generator=_gen(182), device="cuda")).to(TYPES[kind][0])
    check(cache, q, [new] * 71, workspace, uniform=True, causal=True)
    counts = [new if i % 3 else 0 for i in range(71)]
    check(cache, q[:sum(counts)], counts, workspace, causal=True, window=77)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("hd,group,new,length", [(128, 8, 1, 40000), (256, 2, 1, 40000), (64, 12, 1, 40000),
                                                 (128, 4, 1, 131071), (128, 2, 64, 40000), (256, 2, 130, 20000)])
def test_long_contexts(kind, hd, group, new, length, workspace):
    """Beside the bound of every output, whose sums of tens of thousands of weights are counted at their worst: the
    root of the mean square.  A rounding spreads evenly over a step, so the output's leaves 1/sqrt(3) of the half
    step, and the weights' independent ones 1/sqrt(3) of theirs times the root of sum p^2 v^2; a quarter is left for the
    scores' errors, a few 2^-24 of scores of about ten."""
    cache = make_cache(kind, [length], 1, hd, 64, seed=190)
    q = (2 * torch.randn(new, group, hd, generator=_gen(191), device="cuda")).to(TYPES[kind][0])
    out, _ = check(cache, q, [new], workspace, uniform=True, causal=True)
    step, half = bounds.p_step(cache, q, new * group)
    want = bounds.attention(cache, q, [new], p_step=step, p_half=half)[0]
    rounding = (ref.half_step(q.dtype, want) / 3 ** 0.5).square().mean().sqrt()
    spread = step / 3 ** 0.5 * weights_spread(cache, q, new)
    assert (out.double() - want).square().mean().sqrt() <= 1.25 * (rounding ** 2 + spread ** 2).sqrt()


def weights_spread(cache, q, new):
    """Root of the mean over outputs of sum p^2 v^2, for one sequence of one KV head."""
    n_pages, _, page, hd = cache.k.shape
    total = int(cache.kv_len[0])
    j = torch.arange(total)
    ids = cache.page_table[0].cpu()[j // page].long().cuda()
    k, v = cache.k[ids, 0, (j % page).cuda()].double(), cache.v[ids, 0, (j % page).cuda()].double()
    if cache.k_scale is not None:
        k, v = k * cache.k_scale[0].double(), v * cache.v_scale[0].double()
    s = torch.einsum("nhd,ld->nhl", q.double(), k) / math.sqrt(hd)
    p = torch.arange(total - new, total, device="cuda")
    s = s.masked_fill((torch.arange(total, device="cuda") > p[:, None])[:, None], -math.inf)
    return (torch.softmax(s, -1).square() @ v.square()).mean().sqrt()


# ------------------------------------------------------------------ layouts

@pytest.mark.parametrize("page", [8, 24, 40, 48, 96, 200, 384, 1024])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_many_rows_over_pages_of_any_size_that_8_divides(page, hd, workspace):
    lens, new = [900, 129, 41, 1030], [200, 64, 41, 30]
    cache = make_cache("bf16", lens, 2, hd, page, seed=200)
    q = (2 * torch.randn(sum(new), 6, hd, generator=_gen(201), device="cuda")).bfloat16()
    check(cache, q, new, workspace, causal=True)
    check(cache, q, new, workspace, causal=False, window=130, cap=15.0)


@pytest.mark.parametrize("kind", ["bf16", "f16-e4m3"])
@pytest.mark.parametrize("group", [100, 127, 128, 129, 200])
def test_large_groups(kind, group, workspace):
    lens, new = [300, 77, 64], [5, 1, 2]
    cache = make_cache(kind, lens, 1, 128, 16, seed=210)
    q = (2 * torch.randn(sum(new), group, 128, generator=_gen(211), device="cuda")).to(TYPES[kind][0])
    check(cache, q, new, workspace, causal=True)
    check(cache, q, new, workspace, causal=False, window=40)


@pytest.mark.parametrize("kind", ["bf16", "f16-e4m3"])
@pytest.mark.parametrize("new", [1, 70])
def test_any_order_of_strides(kind, new, workspace):
    """Rows stored by head, one row for every token, one head for all, tables and lse inside larger ones, in place."""
    t, lens = TYPES[kind][0], [300, 80]
    cache = make_cache(kind, lens, 2, 64, 16, seed=220)
    n = 2 * new
    wide = torch.full((2, 40), -7, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + cache.page_table.shape[1]] = cache.page_table
    cache = dg.PagedCache(cache.k, cache.v, wide[:, 3:3 + cache.page_table.shape[1]], cache.kv_len, cache.k_scale,
                          cache.v_scale)
    rows = torch.randn(n, 4, 64, generator=_gen(221), device="cuda").to(t)
    by_head = rows.transpose(0, 1).contiguous().transpose(0, 1)
    for q in (by_head, rows[:1].expand(n, 4, 64), rows[:, :1].expand(n, 4, 64)):
        want = torch.empty_like(rows)
        dg.paged_attention(cache, q.contiguous(), want, workspace, causal=False)
        out = torch.empty(4, n, 64, dtype=t, device="cuda").transpose(0, 1)
        dg.paged_attention(cache, q, out, workspace, causal=False)
        step = bounds.p_step(cache, q, 2 * new)
        exact, _, bound, _ = bounds.attention(cache, q, [new, new], causal=False, p_step=step[0], p_half=step[1])
        for x in (want, out):
            assert ((x.double() - exact).abs() <= ref.half_step(t, exact) * (1 + 2.0 ** -7) + bound).all()
    x = rows.clone()
    dg.paged_attention(cache, x, x, workspace, causal=False)
    dg.paged_attention(cache, rows, want, workspace, causal=False)
    assert torch.equal(x, want)


def test_pages_shared_by_sequences(workspace):
    """A common prompt's pages in every table, each sequence's own behind them."""
    cache = make_cache("bf16", [160] * 5, 2, 128, 16, seed=230)
    cache.page_table[:, :8] = cache.page_table[0, :8].clone()
    cache.kv_len.copy_(torch.tensor([160, 140, 129, 150, 128]))
    for new in (1, 40):
        q = (2 * torch.randn(5 * new, 8, 128, generator=_gen(231), device="cuda")).bfloat16()
        check(cache, q, [new] * 5, workspace, uniform=True, causal=True)


@pytest.mark.parametrize("new", [1, 64])
def test_16_bit_pools_beyond_32_bit_offsets(new, workspace):
    page, hd = 64, 128
    n_pages = (1 << 32) // (page * hd) + 8
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    k = torch.empty(n_pages, 1, page, hd, dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    used = [n_pages - 1, 5, n_pages - 7, n_pages // 2 + 3]
    g = _gen(240)
    for x in (k, v):
        for i in used:
            x[i] = torch.randn(1, page, hd, generator=g, device="cuda").half()
    cache = dg.PagedCache(k, v, torch.tensor([used], dtype=torch.int32, device="cuda"),
                          torch.tensor([250], dtype=torch.int32, device="cuda"))
    rows = torch.randn(new, 6, hd, generator=g, device="cuda").half()
    dg.paged_append(cache, rows[:, 4:5], rows[:, 5:])
    at = torch.arange(250 - new, 250, device="cuda")
    ids = torch.tensor(used, device="cuda")[at // page]
    assert torch.equal(k[ids, 0, at % page], rows[:, 4]) and torch.equal(v[ids, 0, at % page], rows[:, 5])
    check(cache, rows[:, :4], [new], workspace)


# ------------------------------------------------------------------ captured calls

@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_captured_batches_follow_counts_lengths_and_pages(cap, workspace):
    """One graph of append and attention for a ragged batch: replays with other counts, lengths and tables, from one
    token each to one sequence with all of them, on a workspace that other calls use in between."""
    b, n, hq, hkv = 4, 120, 6, 2
    cache = make_cache("bf16", [1200] * b, hkv, 128, 16, seed=250)
    cache.k.nan_to_num_(0.0), cache.v.nan_to_num_(0.0)
    g = _gen(251)
    rows = torch.randn(n, hq + 2 * hkv, 128, generator=g, device="cuda").bfloat16()
    q, k, v = rows.split([hq, hkv, hkv], dim=1)
    qr, out = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty(n, hq, 128, device="cuda").bfloat16()
    lse, cu = torch.empty(n, hq, device="cuda"), cu_of([30] * b)

    def step():
        dg.paged_append(cache, k, v, q=q, q_out=qr, cu_new=cu, rope_base=10000.0)
        dg.paged_attention(cache, qr, out, workspace, cu_new=cu, cap=cap, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new, lens in (([30, 30, 30, 30], [1200, 31, 30, 700]), ([1, 1, 1, 1], [900, 1, 17, 16]),
                      ([0, 120, 0, 0], [5, 1000, 0, 3]), ([0, 0, 0, 0], [1, 2, 3, 4]), ([2, 100, 3, 10], [2, 1111, 64, 640])):
        cu.copy_(cu_of(new))
        cache.kv_len.copy_(torch.tensor(lens))
        cache.page_table.copy_(cache.page_table.roll(1, 0))
        rows.normal_(generator=g)
        out.fill_(7.0), lse.fill_(7.0), qr.fill_(1.0)
        graph.replay()
        dg.paged_synchronize(workspace)
        got, m = out.clone(), sum(new)
        assert (got[m:] == 7.0).all() and (lse[m:] == 7.0).all()
        if m:
            step_, half = max((bounds.p_step(cache, q, c * hq // hkv) for c in new if c))
            want, want_lse, bound, lse_bound = bounds.attention(cache, qr, new, cap=cap, p_step=step_, p_half=half)
            assert ((got.double() - want).abs() <= ref.half_step(q.dtype, want) * (1 + 2.0 ** -7) + bound)[:m].all()
            assert ((lse.double() - want_lse).abs() <= lse_bound)[:m].all()
        dg.paged_attention(cache, qr, out, workspace, cu_new=cu_of([30] * b), causal=False)  # the graph's own next to come


def test_two_graphs_at_once_with_a_workspace_each():
    caches = [make_cache("bf16", [2304], 2, 128, 16, seed=260 + i) for i in range(2)]
    spaces = [dg.paged_workspace() for _ in range(2)]
    qs = [torch.randn(256, 4, 128, generator=_gen(262 + i), device="cuda").bfloat16() for i in range(2)]
    outs, first = [torch.empty_like(x) for x in qs], []
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        dg.paged_attention(caches[i], qs[i], outs[i], spaces[i], causal=False)
        first.append(outs[i].clone())
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[i]):
            for _ in range(4):
                dg.paged_attention(caches[i], qs[i], outs[i], spaces[i], causal=False)
        outs[i].zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        dg.paged_synchronize(spaces[i])
        assert torch.equal(outs[i], first[i])
