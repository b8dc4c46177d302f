"""The paged cache's operators on the device against their definition in 64 bits."""
import math

import pytest
import torch

import block_denoising_step_b200 as dg
from tests import paged_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, torch.bfloat16), "f16": (torch.float16, torch.float16),
         "bf16-e4m3": (torch.bfloat16, torch.float8_e4m3fn), "f16-e4m3": (torch.float16, torch.float8_e4m3fn)}


@pytest.fixture(scope="module")
def workspace():
    return dg.paged_workspace()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make_cache(kind, lens, hkv, hd, page, seed, spare=2, std=1.0, extra_pages=0):
    """A filled cache with shuffled pages; positions behind a sequence's end hold NaN, entries behind it garbage."""
    g = _gen(seed)
    t, ct = TYPES[kind]
    need = [-(-max(n, 0) // page) for n in lens]
    n_pages = sum(need) + spare
    k, v = (torch.randn(n_pages, hkv, page, hd, generator=g, device="cuda") * std for _ in range(2))
    ks = vs = None
    if ct == torch.float8_e4m3fn:
        ks = 0.01 + 0.01 * torch.rand(hkv, generator=g, device="cuda")
        vs = 0.01 + 0.01 * torch.rand(hkv, generator=g, device="cuda")
        k, v = (k / ks[:, None, None]).clamp(-448, 448), (v / vs[:, None, None]).clamp(-448, 448)
    order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
    table = torch.full((len(lens), max(max(need), 1) + extra_pages), 1 << 30, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        ids = order[at:at + n]
        table[b, :n] = torch.tensor(ids, dtype=torch.int32)
        at += n
        if lens[b] % page and n:
            k[ids[-1], :, lens[b] % page:] = math.nan
            v[ids[-1], :, lens[b] % page:] = math.nan
    k[order[at:]] = math.nan
    v[order[at:]] = math.nan
    return dg.PagedCache(k.to(ct), v.to(ct), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), ks, vs)


def cu_of(new):
    return torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")


def check_attention(cache, q, new, workspace, **kw):
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    dg.paged_attention(cache, q, out, workspace, cu_new=cu_of(new), lse=lse, **kw)
    torch.cuda.synchronize()
    want, want_lse, slack = ref.attention(cache, q, new, **kw)
    n = sum(new)
    bound = ref.half_step(q.dtype, want) * (1 + 2.0 ** -7) + slack
    bad = (out.double() - want).abs()[:n] > bound[:n]
    assert not bad.any() and not out[:n].isnan().any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    live = want_lse[:n] > -math.inf
    assert torch.equal(lse[:n] == -math.inf, ~live)
    d = (lse[:n].double() - want_lse[:n]).abs()[live]
    # scores up to ~ 10 within their fp32 error (as the outputs), the log rounded once
    assert d.numel() == 0 or float(d.max()) < 2e-4
    assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()  # padding rows are left as they were
    return out


# (lengths, new tokens, kv heads, group, head dim, page)
SHAPES = [
    ([1], [1], 1, 1, 64, 16),
    ([0, 5, 17], [0, 1, 1], 2, 3, 64, 7),
    ([300], [1], 8, 2, 256, 64),
    ([33, 1, 64, 65, 1000], [1, 1, 1, 1, 1], 2, 8, 128, 16),
    ([2000, 3], [1, 1], 1, 5, 128, 24),
    ([129, 500], [1, 1], 2, 16, 64, 1),
    ([700, 40], [1, 0], 1, 48, 128, 32),
    ([90, 31, 12], [4, 31, 2], 2, 3, 128, 16),
    ([260, 70], [130, 70], 2, 2, 256, 64),
    ([300, 20], [200, 1], 1, 4, 64, 128),
    ([513, 256, 258], [256, 256, 256], 2, 2, 128, 64),
]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}-{s[1]}-{s[2]}x{s[3]}x{s[4]}-p{s[5]}".replace(" ", ""))
def test_attention_matches_the_formula(shape, kind, workspace):
    lens, new, hkv, group, hd, page = shape
    cache = make_cache(kind, lens, hkv, hd, page, seed=3)
    q = (2 * torch.randn(sum(new) + 3, hkv * group, hd, generator=_gen(4), device="cuda")).to(TYPES[kind][0])
    q[sum(new):] = math.nan
    check_attention(cache, q, new, workspace, causal=True)
    check_attention(cache, q, new, workspace, causal=False)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f16-e4m3"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window,cap", [(1, 0.0), (40, 0.0), (100000, 0.0), (2 ** 31 - 1, 5.0), (0, 2.0), (65, 30.0)])
def test_window_and_cap(kind, causal, window, cap, workspace):
    lens, new = [400, 90, 64, 1], [1, 90, 20, 1]
    cache = make_cache(kind, lens, 2, 128, 32, seed=5)
    q = (3 * torch.randn(sum(new), 8, 128, generator=_gen(6), device="cuda")).to(TYPES[kind][0])
    check_attention(cache, q, new, workspace, causal=causal, window=window, cap=cap)


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_many_new_tokens(hd, workspace):
    """Canvases and prompt chunks with odd counts, beside single tokens."""
    lens, new = [700, 129, 1025, 64, 2], [257, 1, 300, 64, 2]
    for kind in ("bf16", "f16"):
        cache = make_cache(kind, lens, 2, hd, 16, seed=7)
        q = (2 * torch.randn(sum(new), 6, hd, generator=_gen(8), device="cuda")).to(TYPES[kind][0])
        check_attention(cache, q, new, workspace, causal=False)
        check_attention(cache, q, new, workspace, causal=True, window=200)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 4, 8, 9, 16, 17])
def test_rows_around_the_kernels_limit(hd, group, workspace):
    """A batch whose sequences have 8, 9, 16 and 17 rows per KV head, or about: few go to one kernel, more to the other."""
    for new in ([1, 1, 1, 1, 0], [8, 9, 16, 17, 1], [2, 2, 2, 2, 2]):
        lens = [300, 19, 641, 128, 77]
        cache = make_cache("bf16", lens, 2, hd, 16, seed=70)
        q = (2 * torch.randn(sum(new), 2 * group, hd, generator=_gen(71), device="cuda")).to(torch.bfloat16)
        check_attention(cache, q, new, workspace, causal=True)
        check_attention(cache, q, new, workspace, causal=False, window=50, cap=20.0)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("kind,page,group", [("bf16-e4m3", 16, 3), ("f16-e4m3", 7, 7), ("bf16", 7, 3), ("f16", 12, 5),
                                             ("bf16", 7, 48), ("bf16", 16, 7), ("f16", 8, 3)])
def test_many_new_tokens_of_odd_groups(hd, kind, page, group, workspace):
    """Groups that do not divide a row tile, on either kernel (E4M3 caches and odd pages take the split one)."""
    lens, new = [500, 41, 316, 64], [237, 41, 100, 1]
    cache = make_cache(kind, lens, 1, hd, page, seed=60)
    q = (2 * torch.randn(sum(new), group, hd, generator=_gen(61), device="cuda")).to(TYPES[kind][0])
    check_attention(cache, q, new, workspace, causal=True)
    check_attention(cache, q, new, workspace, causal=True, window=70)
    check_attention(cache, q, new, workspace, causal=False, window=33, cap=20.0)


@pytest.mark.parametrize("new", [1, 128])
def test_absent_pages_are_masked(new, workspace):
    lens = [400, 300, 128]
    cache = make_cache("bf16", lens, 2, 128, 16, seed=9, extra_pages=3)
    cache.page_table[0, 3] = -1
    cache.page_table[0, 7] = cache.n_pages
    cache.page_table[1, :] = -1       # nothing left: zeros
    cache.page_table[2, 2:8] = -5
    q = (2 * torch.randn(new * 3, 4, 128, generator=_gen(10), device="cuda")).bfloat16()
    out = check_attention(cache, q, [new] * 3, workspace, causal=False)
    assert not out[new:2 * new].any()
    check_attention(cache, q, [new] * 3, workspace, causal=True, window=50)


@pytest.mark.parametrize("new", [1, 64])
def test_length_beyond_the_table_and_below_the_new_tokens(new, workspace):
    cache = make_cache("bf16", [100, 64], 1, 64, 16, seed=11)
    cache.kv_len.copy_(torch.tensor([150, 0]))
    cache.page_table[:, :] = torch.arange(cache.page_table.numel()).view(2, -1) % 3
    cache.k.nan_to_num_(0.0), cache.v.nan_to_num_(0.0)
    q = torch.randn(2 * new, 2, 64, generator=_gen(12), device="cuda").bfloat16()
    check_attention(cache, q, [new, new], workspace, causal=True)
    check_attention(cache, q, [new, new], workspace, causal=False)


def test_large_scores_and_scale(workspace):
    """Scores in the hundreds: one key takes all, no overflow; a scale of its own."""
    cache = make_cache("bf16", [500, 77], 2, 128, 16, seed=13, std=8.0)
    q = (16 * torch.randn(2, 8, 128, generator=_gen(14), device="cuda")).bfloat16()
    for scale in (None, 0.3):
        out = torch.empty_like(q)
        dg.paged_attention(cache, q, out, workspace, scale=scale)
        want, _, slack = ref.attention(cache, q, [1, 1], scale=scale)
        assert ((out.double() - want).abs() <= ref.half_step(q.dtype, want) * 1.01 + slack).all()


@pytest.mark.parametrize("new", [1, 40])
def test_strided_rows(new, workspace):
    """Queries inside a fused projection, the output inside a wider buffer; the gaps stay as they were."""
    lens = [200, 90]
    cache = make_cache("f16", lens, 2, 64, 16, seed=15)
    fused = torch.randn(2 * new, 8 + 4, 64, generator=_gen(16), device="cuda").half()
    q = fused[:, :8]
    wide = torch.full((2 * new, 9, 72), 5.0, device="cuda", dtype=torch.float16)
    out = wide[:, 1:, :64]
    dg.paged_attention(cache, q, out, workspace, causal=False)
    want, _, slack = ref.attention(cache, q.contiguous(), [new, new], causal=False)
    assert ((out.double() - want).abs() <= ref.half_step(q.dtype, want) * 1.01 + slack).all()
    assert (wide[:, 0] == 5).all() and (wide[:, :, 64:] == 5).all()


def test_offsets_beyond_32_bits(workspace):
    """Pages whose element offsets pass 2^32."""
    page, hd = 64, 128
    n_pages = (1 << 32) // (page * hd) // 2 * 2 + 8  # more than 2^32 elements in one head's pages
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    k = torch.empty(n_pages, 1, page, hd, dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.empty_like(k)
    used = [n_pages - 1, 5, n_pages - 7, n_pages // 2 + 3]
    g = _gen(17)
    for x in (k, v):
        for i in used:
            x[i] = torch.randn(1, page, hd, generator=g, device="cuda").to(x.dtype)
    one = torch.ones(1, device="cuda")
    table = torch.tensor([used], dtype=torch.int32, device="cuda")
    cache = dg.PagedCache(k, v, table, torch.tensor([250], dtype=torch.int32, device="cuda"), one, one)
    q = torch.randn(1, 4, hd, generator=g, device="cuda").bfloat16()
    kn, vn = (torch.randn(1, 1, hd, generator=g, device="cuda").bfloat16() for _ in range(2))
    dg.paged_append(cache, kn, vn)
    assert torch.equal(k[used[3], 0, 249 % page].float(), kn[0, 0].float().to(k.dtype).float())
    check_attention(cache, q, [1], workspace)


def _append_case(kind, lens, new, hkv, hq, hd, page, base, seed, fused=True, cu=True):
    t, ct = TYPES[kind]
    cache = make_cache(kind, lens, hkv, hd, page, seed)
    n = sum(new) + (2 if cu else 0)
    g = _gen(seed + 1)
    if fused:
        rows = torch.randn(n, hq + 2 * hkv, hd, generator=g, device="cuda").to(t)
        q, k, v = rows.split([hq, hkv, hkv], dim=1)
    else:
        q, k, v = (torch.randn(n, h, hd, generator=g, device="cuda").to(t) for h in (hq, hkv, hkv))
    before = cache.k.clone(), cache.v.clone()
    q_out = torch.full((n, hq, hd), 9.0, device="cuda", dtype=t)
    dg.paged_append(cache, k, v, q=q, q_out=q_out, cu_new=cu_of(new) if cu else None, rope_base=base)
    torch.cuda.synchronize()
    table, row = cache.page_table.cpu(), 0
    touched = torch.zeros(cache.n_pages, page, dtype=torch.bool, device="cuda")
    for b, where in enumerate(ref.positions(table, cache.kv_len, new, page)):
        for pos, pid in where:
            p = torch.tensor([pos], device="cuda")
            if pos < 0:
                assert (q_out[row] == 9.0).all()
            elif base:
                qd, kd = q[row:row + 1].double(), k[row:row + 1].double()
                want_q, want_k = ref.rotate(qd, p, base), ref.rotate(kd, p, base)
                sq, sk = ref.rotation_slack(qd, want_q), ref.rotation_slack(kd, want_k)
            else:
                want_q, want_k = q[row:row + 1].double(), k[row:row + 1].double()
                sq = sk = torch.zeros(1, device="cuda", dtype=torch.float64)
            if pos >= 0:
                assert ((q_out[row] - want_q[0]).abs() <= ref.half_step(t, want_q[0]) * 1.01 + sq[0]).all()
                if 0 <= pid < cache.n_pages:
                    touched[pid, pos % page] = True
                    for c, want, scale, sl in ((cache.k, want_k[0], cache.k_scale, sk[0]),
                                               (cache.v, v[row].double(), cache.v_scale, 0.0)):
                        got = c[pid, :, pos % page].double()
                        if scale is not None:
                            s = scale.double()[:, None]
                            got, tol = got * s, ref.half_step(ct, (want / s)) * s
                            want = want.clamp(-448 * s, 448 * s)
                        else:
                            tol = ref.half_step(ct, want)
                        assert ((got - want).abs() <= tol * 1.01 + sl).all(), (b, pos)
            row += 1
    assert (q_out[row:] == 9.0).all()
    for was, c in zip(before, (cache.k, cache.v)):  # every other row is as it was, to the bit
        a, b = was.view(torch.uint8).transpose(1, 2)[~touched], c.view(torch.uint8).transpose(1, 2)[~touched]
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shape", [([1], [1], 1, 1, 64, 16), ([70, 3, 9], [5, 0, 9], 2, 6, 128, 7),
                                   ([40, 4], [20, 4], 8, 16, 256, 64), ([33, 65, 1], [33, 1, 1], 3, 3, 64, 1)],
                         ids=str)
def test_append_matches_the_formula(shape, kind):
    lens, new, hkv, hq, hd, page = shape
    _append_case(kind, lens, new, hkv, hq, hd, page, 10000.0, seed=20)
    _append_case(kind, lens, new, hkv, hq, hd, page, 0.0, seed=21, fused=False)


def test_append_far_positions():
    """Positions near the largest cache: the angle's reduction keeps its accuracy."""
    page, far = 1 << 20, (1 << 30) - 1
    k = torch.zeros(2, 1, page, 64, dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.full((1, 1024), -1, dtype=torch.int32, device="cuda")
    table[0, 1023] = 1
    cache = dg.PagedCache(k, v, table, torch.tensor([far + 1], dtype=torch.int32, device="cuda"))
    kn = torch.randn(3, 1, 64, generator=_gen(22), device="cuda").half()
    dg.paged_append(cache, kn, kn, rope_base=500000.0)
    p = torch.arange(far - 2, far + 1, device="cuda")
    want = ref.rotate(kn.double(), p, 500000.0)
    got = k[1, 0, -3:].double()[:, None]
    # at 2^30 the reference's own fp64 angle is off by up to 2^30 * 2^-52
    assert ((got - want).abs() <= ref.half_step(k.dtype, want) * 1.01 + ref.rotation_slack(kn.double(), want) +
            2.0 ** -20).all()


def test_append_absent_pages_short_lengths_and_uniform_rows():
    cache = make_cache("bf16", [40, 3, 64], 2, 64, 16, seed=23)
    cache.page_table[0, 2] = -1           # positions 32..39 have no page
    cache.kv_len[1] = 3                   # four new tokens at positions -1..2: the first is dropped
    was = cache.k.clone()
    k, v, q = (torch.randn(12, h, 64, generator=_gen(24), device="cuda").bfloat16() for h in (2, 2, 4))
    q_in = q.clone()
    dg.paged_append(cache, k, v, q=q, q_out=q, rope_base=10000.0)  # in place
    ids = cache.page_table
    assert torch.equal(cache.k[ids[1, 0], :, 0].view(torch.uint8),
                       dg_rotated(k[5:6], 0).view(torch.uint8)[0])
    assert torch.equal(q[4], q_in[4]) and not torch.equal(q[5 + 1], q_in[5 + 1])
    changed = (cache.k.view(torch.int16) != was.view(torch.int16)).any(-1).any(1)
    where = changed.nonzero().tolist()
    want = [[int(ids[1, 0]), o] for o in range(3)] + [[int(ids[2, 3]), o] for o in range(12, 16)]
    assert sorted(where) == sorted(want)


def dg_rotated(x, pos):
    return ref.rotate(x.double(), torch.tensor([pos], device="cuda"), 10000.0).to(x.dtype)


def test_append_saturates_and_keeps_nan():
    one = torch.ones(1, device="cuda")
    k = torch.zeros(1, 1, 16, 64, dtype=torch.float8_e4m3fn, device="cuda")
    cache = dg.PagedCache(k, torch.zeros_like(k), torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                          torch.ones(1, dtype=torch.int32, device="cuda"), one, one)
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, :4] = torch.tensor([1e9, -math.inf, math.nan, 449.0])
    dg.paged_append(cache, x, x)
    got = k[0, 0, 0, :4].float()
    assert got[0] == 448 and got[1] == -448 and got[2].isnan() and got[3] == 448


@pytest.mark.parametrize("kind", ["bf16", "f16-e4m3"])
def test_prompt_canvas_and_tokens_as_a_server_runs_them(kind, workspace):
    """Two prompts of their own lengths enter in chunks, a canvas is denoised on one of them, then both go on
    token by token: append and attention together against the definition over the whole context."""
    t, ct = TYPES[kind]
    hkv, hq, hd, page, base = 2, 8, 128, 16, 10000.0
    g = _gen(30)
    cache = make_cache(kind, [400, 400], hkv, hd, page, seed=31)
    cache.kv_len.zero_()
    steps = [([90, 33], True), ([50, 0], True), ([64, 64], False), ([1, 1], True), ([1, 1], True), ([0, 3], True)]
    for new, causal in steps:
        n = sum(new)
        cache.kv_len += torch.tensor(new, dtype=torch.int32, device="cuda")
        rows = torch.randn(n, hq + 2 * hkv, hd, generator=g, device="cuda").to(t)
        q, k, v = rows.split([hq, hkv, hkv], dim=1)
        qr = torch.empty(n, hq, hd, device="cuda", dtype=t)
        dg.paged_append(cache, k, v, q=q, q_out=qr, cu_new=cu_of(new), rope_base=base)
        check_attention(cache, qr, new, workspace, causal=causal)


def test_captured_calls_follow_the_table_and_lengths(workspace):
    """Append and attention in one CUDA graph: replays see the lengths and pages of their time."""
    cache = make_cache("bf16", [200, 100], 2, 128, 16, seed=32)
    cache.k.nan_to_num_(0.0), cache.v.nan_to_num_(0.0)
    g = _gen(33)
    q, k, v = (torch.randn(2, h, 128, generator=g, device="cuda").bfloat16() for h in (4, 2, 2))
    qr, out = torch.empty_like(q), torch.empty_like(q)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        dg.paged_append(cache, k, v, q=q, q_out=qr, rope_base=10000.0)
        dg.paged_attention(cache, qr, out, workspace)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.paged_append(cache, k, v, q=q, q_out=qr, rope_base=10000.0)
        dg.paged_attention(cache, qr, out, workspace)
    for lens in ([200, 100], [17, 1], [151, 99]):
        cache.kv_len.copy_(torch.tensor(lens))
        cache.page_table.copy_(cache.page_table.flip(0))
        cache.page_table[cache.page_table == 1 << 30] = 0
        k.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        want, _, slack = ref.attention(cache, qr, [1, 1])
        assert ((out.double() - want).abs() <= ref.half_step(q.dtype, want) * 1.01 + slack).all()
        p = torch.tensor(lens, device="cuda") - 1
        rot = ref.rotate(q.double(), p, 10000.0)
        assert ((qr.double() - rot).abs() <= ref.half_step(q.dtype, rot) * 1.01 + ref.rotation_slack(q.double(), rot)).all()


def test_two_streams_at_once_with_a_workspace_each():
    caches = [make_cache("bf16", [3000, 1], 2, 128, 16, seed=40 + i) for i in range(2)]
    spaces = [dg.paged_workspace() for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    qs = [torch.randn(2, 8, 128, generator=_gen(42 + i), device="cuda").bfloat16() for i in range(2)]
    outs = [torch.empty_like(x) for x in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            dg.paged_attention(caches[i], qs[i], outs[i], spaces[i], stream=streams[i].cuda_stream)
    torch.cuda.synchronize()
    for i in range(2):
        want, _, slack = ref.attention(caches[i], qs[i], [1, 1])
        assert ((outs[i].double() - want).abs() <= ref.half_step(torch.bfloat16, want) * 1.01 + slack).all()


def test_workspace_status(workspace):
    """No wait ran out so far; a recorded device error is reported once and the workspace put back."""
    dg.paged_synchronize(workspace)
    ws = dg.paged_workspace()
    ws[:4096].view(torch.int32)[1023] = 5
    ws[:4096].view(torch.int32)[0] = 3
    with pytest.raises(dg.DgenError) as e:
        dg.paged_synchronize(ws)
    assert e.value.status == dg.DGEN_EDEVICE
    dg.paged_synchronize(ws)
    assert not ws[:4096].any()


@pytest.mark.parametrize("new", [1, 100])
def test_same_call_same_bits(new, workspace):
    cache = make_cache("bf16", [5000, 700, 2300], 2, 128, 16, seed=50)
    q = torch.randn(3 * new, 8, 128, generator=_gen(51), device="cuda").bfloat16()
    outs = []
    for _ in range(5):
        out = torch.empty_like(q)
        dg.paged_attention(cache, q, out, workspace, causal=False)
        outs.append(out)
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_binding_refusals(workspace):
    cache = make_cache("bf16", [16, 16], 2, 64, 16, seed=60)
    q = torch.zeros(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    kv = torch.zeros(2, 2, 64, device="cuda", dtype=torch.bfloat16)
    good = dict(cache=cache, q=q, out=torch.empty_like(q), workspace=workspace)
    bad_att = [dict(q=q.half()), dict(q=q[:, :3]), dict(out=q[:1]), dict(out=q.half()), dict(q=q.cpu()),
               dict(q=q.transpose(1, 2)), dict(cu_new=torch.zeros(2, dtype=torch.int32, device="cuda")),
               dict(cu_new=torch.zeros(3, dtype=torch.int64, device="cuda")), dict(lse=torch.empty(2, 3, device="cuda")),
               dict(q=q[:1], out=q[:1]), dict(workspace=workspace.cpu()), dict(q=q[..., 1:])]
    for b in bad_att:
        with pytest.raises(dg.DgenError) as e:
            dg.paged_attention(**{**good, **b})
        assert e.value.status == dg.DGEN_EINVAL
    with pytest.raises(dg.DgenError) as e:
        dg.paged_attention(**{**good, "workspace": workspace[:8192].clone()})
    assert e.value.status == dg.DGEN_ESCRATCH
    bad_app = [dict(k=kv.half()), dict(k=kv[:, :1]), dict(v=kv[:1]), dict(q=q), dict(q=q, q_out=q.half()),
               dict(k=kv[:1], v=kv[:1])]
    for b in bad_app:
        with pytest.raises(dg.DgenError) as e:
            dg.paged_append(**{**dict(cache=cache, k=kv, v=kv), **b})
        assert e.value.status == dg.DGEN_EINVAL
    with pytest.raises(dg.DgenError):
        dg.PagedCache(cache.k, cache.v, cache.page_table, cache.kv_len, k_scale=torch.ones(2, device="cuda"))
