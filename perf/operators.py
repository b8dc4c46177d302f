"""Calls of the paged KV cache's operators at sizes of real use, for measuring them.

``run`` makes one call of ``paged_append`` (rotate the new tokens' keys and queries, write keys and values
into the pages) or ``paged_attention`` (the new tokens' attention over the pages): with ``own`` false in
plain torch operations in 32 bits, with ``own`` true through block_denoising_step_b200.  ``exact`` gives the
same outputs from the definition in 64 bits.

Case fields: op "append" / "attend"; type of the token rows and cache "bf16" / "f16" with cache "same" or
"e4m3"; batch sequences; new tokens per sequence (ragged: between 1 and this many); length = keys of the
longest sequence, the new tokens included (ragged: down to the new tokens alone); kv_heads, group (query
heads per KV head), head_dim, page (keys per page); causal, window (0: none), cap (0: none).
"""
import math

import torch

own = False

_FULL = dict(type="bf16", cache="same", kv_heads=8, group=2, head_dim=256, page=64)  # the full-scale model's heads


def listed():
    plain = dict(causal=True, window=0, cap=0.0, ragged=False)
    return [
        # one sequence's next token in the full-scale model: latency alone
        dict(plain, name="append one", op="append", **_FULL, batch=1, new=1, length=2049),
        # a large decode batch of a small model with seven query heads per KV head and pages of 24 keys
        dict(plain, name="append decode f16", op="append", type="f16", cache="same", kv_heads=4, group=7, head_dim=64,
             page=24, batch=256, new=1, length=1000),
        # eight canvases of 256 tokens behind prompts of 4096 (the batched full-scale workload)
        dict(plain, name="append canvas", op="append", **_FULL, batch=8, new=256, length=4352),
        # prompts of mixed lengths entering an 8-bit cache
        dict(plain, name="append prompts e4m3", op="append", type="bf16", cache="e4m3", kv_heads=8, group=4, head_dim=128,
             page=16, batch=16, new=4096, length=4096, ragged=True),
        # a short conversation's next token
        dict(plain, name="one token short", op="attend", **_FULL, batch=1, new=1, length=301),
        # one sequence with a book-long context
        dict(plain, name="one token long", op="attend", type="bf16", cache="same", kv_heads=8, group=4, head_dim=128,
             page=64, batch=1, new=1, length=131071),
        # a decode batch of the full-scale model, lengths mixed
        dict(plain, name="decode batch", op="attend", **_FULL, batch=64, new=1, length=8192, ragged=True),
        # a decode batch over an 8-bit cache, eight query heads per KV head, small pages
        dict(plain, name="decode batch e4m3", op="attend", type="bf16", cache="e4m3", kv_heads=8, group=8, head_dim=128,
             page=16, batch=48, new=1, length=16384, ragged=True),
        # heads without sharing, a sliding window and capped scores
        dict(plain, name="decode window f16", op="attend", type="f16", cache="same", kv_heads=12, group=1, head_dim=64,
             page=32, batch=128, new=1, length=4097, ragged=True) | dict(window=1024, cap=50.0),
        # one canvas over its prompt, every canvas token sees all keys (the full-scale workload's attention)
        dict(plain, name="canvas", op="attend", **_FULL, batch=1, new=256, length=2304) | dict(causal=False),
        # eight canvases over prompts of 4096 (the batched full-scale workload's attention)
        dict(plain, name="canvas batch", op="attend", **_FULL, batch=8, new=256, length=4352) | dict(causal=False),
        # causal chunks of prompts, mixed lengths, capped scores
        dict(plain, name="prompt chunks f16", op="attend", type="f16", cache="same", kv_heads=8, group=4, head_dim=128,
             page=16, batch=6, new=1024, length=5000, ragged=True) | dict(cap=30.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend"])
    c = dict(op=op, type=rng.choice(["bf16", "f16"]), cache=rng.choice(["same", "same", "e4m3"]),
             kv_heads=rng.choice([1, 2, 4, 5, 8]), group=rng.choice([1, 2, 3, 4, 7, 8, 16]),
             head_dim=rng.choice([64, 128, 256]), page=rng.choice([7, 16, 24, 32, 64, 128]),
             batch=_log_int(rng, 1, 128), new=1, length=_log_int(rng, 1, 40000), ragged=rng.random() < 0.7,
             causal=True, window=0, cap=0.0)
    if op == "append":
        c["new"] = rng.choice([1, _log_int(rng, 2, 4096)])
    else:
        c["new"] = rng.choice([1, 1, _log_int(rng, 2, 512)])
        c["causal"] = rng.random() < 0.6
        c["window"] = rng.choice([0, 0, _log_int(rng, 16, 4096)])
        c["cap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
    c["length"] = max(c["length"], c["new"])
    top = {k: max(work(x)[k] for x in listed() if x["op"] == op) for k in ("bytes", "flops")}
    while True:  # no costlier than the largest listed case, nor the plain form's score matrix over 2 GB
        w, scores = work(c), c["batch"] * c["new"] * c["kv_heads"] * c["group"] * c["length"]
        padded = c["batch"] * c["length"] * c["kv_heads"] * c["head_dim"]
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"] and (
                padded <= 4e8 if op == "append" else scores <= 5e8 and padded <= 2e9):
            return c
        if c["batch"] > 1:
            c["batch"] = c["batch"] * 2 // 3
        else:
            c["new"] = max(1, c["new"] * 2 // 3)
            c["length"] = max(c["new"], c["length"] * 2 // 3)


def _lengths(c):
    """(new tokens, keys) of each sequence: of the case alone, spread evenly where ragged."""
    new, total = [], []
    for b in range(c["batch"]):
        u, v = (b * 0.6180339887498949) % 1.0, (b * 0.7548776662466927) % 1.0
        n = c["new"] if not c["ragged"] or b == 0 else max(1, round(c["new"] * (1 - u)))
        t = c["length"] if not c["ragged"] or b == 0 else max(n, round(c["length"] * (1 - v)))
        new.append(n)
        total.append(t)
    return new, total


def _visible(c, n, t):
    """(query, key) pairs and distinct keys that the n last tokens of t keys see."""
    w, pairs, first = c["window"], 0, t
    last = 0
    for p in range(t - n, t):
        lo = max(0, p - w + 1) if w else 0
        hi = p + 1 if c["causal"] else (min(t, p + w) if w else t)
        pairs += hi - lo
        first, last = min(first, lo), max(last, hi)
    return pairs, last - first


def work(case):
    c = case
    new, total = _lengths(c)
    tokens, hd, hkv, hq = sum(new), c["head_dim"], c["kv_heads"], c["kv_heads"] * c["group"]
    es = 1 if c["cache"] == "e4m3" else 2
    if c["op"] == "append":  # rows of q, k, v in; rotated q and the cache rows out
        b = tokens * hd * (2 * hq * 2 + 2 * hkv * (2 + es))
        return {"bytes": b, "flops": 3 * tokens * hd * (hq + hkv)}
    seen = {}
    for n, t in zip(new, total):
        if (n, t) not in seen:
            seen[n, t] = _visible(c, n, t)
    pairs = sum(seen[n, t][0] for n, t in zip(new, total))
    keys = sum(seen[n, t][1] for n, t in zip(new, total))
    b = 2 * tokens * hq * hd * 2 + tokens * hq * 4 + 2 * keys * hkv * hd * es
    return {"bytes": b, "flops": 4 * pairs * hq * hd}


_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, total = _lengths(c)
    hkv, hq, hd, page, t = c["kv_heads"], c["kv_heads"] * c["group"], c["head_dim"], c["page"], _TYPES[c["type"]]
    pages = [-(-x // page) for x in total]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    table = torch.full((c["batch"], max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (n_pages, hkv, page, hd)
    k_cache = torch.randn(shape, generator=g, device="cuda", dtype=t)
    v_cache = torch.randn(shape, generator=g, device="cuda", dtype=t)
    st = dict(c=dict(c), table=table, total=torch.tensor(total, dtype=torch.int32, device="cuda"), cu=None,
              max_total=max(total), k_scale=None, v_scale=None)
    if c["cache"] == "e4m3":
        st["k_scale"] = 0.01 + 0.02 * torch.rand(hkv, generator=g, device="cuda")
        st["v_scale"] = 0.01 + 0.02 * torch.rand(hkv, generator=g, device="cuda")
        for x, s in ((k_cache, st["k_scale"]), (v_cache, st["v_scale"])):
            x.div_(s.to(t)[None, :, None, None]).clamp_(-448, 448)
        k_cache, v_cache = k_cache.to(torch.float8_e4m3fn), v_cache.to(torch.float8_e4m3fn)
    st["k_cache"], st["v_cache"] = k_cache, v_cache
    if c["ragged"]:
        st["cu"] = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    n = sum(new)
    if c["op"] == "append":  # the rows are views of one fused projection's output
        qkv = torch.randn(n, (hq + 2 * hkv) * hd, generator=g, device="cuda", dtype=t)
        parts = qkv.split([hq * hd, hkv * hd, hkv * hd], dim=1)
        st["q"], st["k"], st["v"] = (x.unflatten(1, (h, hd)) for x, h in zip(parts, (hq, hkv, hkv)))
        st["q_out"] = torch.empty(n, hq, hd, dtype=t, device="cuda")
    else:
        # score deviation of about 2 after the 1/sqrt(hd) scale: some keys matter, none alone
        st["q"] = (2 * torch.randn(n, hq, hd, generator=g, device="cuda")).to(t)
        st["out"] = torch.empty(n, hq, hd, dtype=t, device="cuda")
        st["lse"] = torch.empty(n, hq, dtype=torch.float32, device="cuda")
        st["max_new"] = max(new)
    return st


# ------------------------------------------------------------------ the framework's calls

_workspace = None


def _own_cache(st):
    """The cache handle that a program builds once and keeps: the page table and lengths change in place."""
    global _workspace
    import block_denoising_step_b200 as dg
    if _workspace is None:
        _workspace = dg.paged_workspace()
    if "handle" not in st:
        st["handle"] = dg.PagedCache(st["k_cache"], st["v_cache"], st["table"], st["total"],
                                     k_scale=st["k_scale"], v_scale=st["v_scale"])
    return dg, st["handle"]


def _own(st):
    dg, cache = _own_cache(st)
    c = st["c"]
    if c["op"] == "append":
        dg.paged_append(cache, st["k"], st["v"], q=st["q"], q_out=st["q_out"], cu_new=st["cu"], rope_base=10000.0)
        return {"q": st["q_out"], "k": st["k_cache"], "v": st["v_cache"]}
    dg.paged_attention(cache, st["q"], st["out"], _workspace, cu_new=st["cu"], causal=c["causal"], window=c["window"],
                       cap=c["cap"], lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


# ------------------------------------------------------------------ the plain form

def _rows(st):
    """Sequence and index within it of every token row."""
    c, n = st["c"], st["q"].shape[0]
    at = torch.arange(n, device="cuda")
    if st["cu"] is None:
        return at // c["new"], at % c["new"], torch.full((c["batch"],), c["new"], device="cuda")
    seq = torch.searchsorted(st["cu"][1:].contiguous(), at.to(torch.int32), right=True)
    return seq, at - st["cu"][seq], st["cu"][1:] - st["cu"][:-1]


def _rotate(x, pos, base):
    """Rotate-half by pos * base^(-2j/hd): the angle in 64 bits, its cosine and sine and the products in 32."""
    half = x.shape[-1] // 2
    freq = base ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    ang = pos[:, None].double() * freq
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _plain_append(st):
    c, page = st["c"], st["c"]["page"]
    seq, i, new = _rows(st)
    pos = (st["total"][seq] - new[seq] + i).long()
    dst, off = st["table"][seq, pos // page].long(), pos % page
    k, v = _rotate(st["k"], pos, 10000.0), st["v"].float()
    if st["k_scale"] is not None:
        k = (k / st["k_scale"][:, None]).clamp(-448, 448)
        v = (v / st["v_scale"][:, None]).clamp(-448, 448)
    for cache, x in ((st["k_cache"], k), (st["v_cache"], v)):
        if cache.dtype == torch.float8_e4m3fn:
            cache.view(torch.uint8)[dst, :, off] = x.to(cache.dtype).view(torch.uint8)
        else:
            cache[dst, :, off] = x.to(cache.dtype)
    st["q_out"].copy_(_rotate(st["q"], pos, 10000.0))
    return {"q": st["q_out"], "k": st["k_cache"], "v": st["v_cache"]}


def _gathered(cache, scale, table, length, page):
    """[batch][length][heads][hd] in 32 bits."""
    j = torch.arange(length, device="cuda")
    at = table[:, j // page].long().clamp_min(0)
    x = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    x = x.transpose(1, 2)[at, (j % page)[None]]
    x = x.view(cache.dtype).float()
    return x if scale is None else x * scale[:, None]


def _plain_attend(st):
    c, page, length = st["c"], st["c"]["page"], st["max_total"]
    seq, i, new = _rows(st)
    b, hkv, hd, m = c["batch"], c["kv_heads"], c["head_dim"], st["max_new"]
    k = _gathered(st["k_cache"], st["k_scale"], st["table"], length, page)
    v = _gathered(st["v_cache"], st["v_scale"], st["table"], length, page)
    first = torch.zeros(b, dtype=torch.int64, device="cuda")
    first[1:] = new.cumsum(0)[:-1]
    at = torch.arange(m, device="cuda")
    q = st["q"][(first[:, None] + at).clamp_max(st["q"].shape[0] - 1)].float()
    s = torch.einsum("bnkgd,blkd->bkgnl", q.view(b, m, hkv, -1, hd) / math.sqrt(hd), k)
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    pos = (st["total"] - new)[:, None] + at
    j = torch.arange(length, device="cuda")
    ok = (j < st["total"][:, None])[:, None] & (at < new[:, None])[..., None]
    if c["causal"]:
        ok = ok & (j <= pos[..., None])
    if c["window"]:
        ok = ok & ((pos[..., None] - j).abs() < c["window"])
    s = s.masked_fill(~ok[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bkgnl,blkd->bnkgd", p / total.clamp_min(1e-37), v).reshape(b, m, -1, hd)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(b, m, -1)
    st["out"].copy_(o[seq, i])
    st["lse"].copy_(lse[seq, i])
    return {"out": st["out"], "lse": st["lse"]}


def run(state):
    if own:
        return _own(state)
    return _plain_append(state) if state["c"]["op"] == "append" else _plain_attend(state)


# ------------------------------------------------------------------ in 64 bits, one sequence at a time

def exact(case, seed):
    st = prepare(case, seed)
    c, page, group, hd = case, case["page"], case["group"], case["head_dim"]
    new, total = _lengths(c)
    outs, lses, qs = [], [], []
    kd = st["k_cache"].to(torch.float64) if c["op"] == "append" else None
    vd = st["v_cache"].to(torch.float64) if c["op"] == "append" else None
    at = 0
    for b, (n, t) in enumerate(zip(new, total)):
        rows = slice(at, at + n)
        at += n
        pages = st["table"][b, :-(-t // page)].long()
        pos = torch.arange(t - n, t, device="cuda")
        if c["op"] == "append":
            j = torch.arange(hd, device="cuda") % (hd // 2)
            ang = pos[:, None] * torch.exp(-j.double() * (2 * math.log(10000.0) / hd))
            turned = []
            for x in (st["q"][rows].double(), st["k"][rows].double()):
                other = torch.roll(x, hd // 2, dims=-1)
                other[..., :hd // 2] *= -1
                turned.append(x * torch.cos(ang)[:, None] + other * torch.sin(ang)[:, None])
            qs.append(turned[0])
            for cache, x, s in ((kd, turned[1], st["k_scale"]), (vd, st["v"][rows].double(), st["v_scale"])):
                if s is not None:
                    x = (x / s.double()[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).double()
                cache[pages[pos // page], :, pos % page] = x
            continue
        lo, hi = 0, t
        if c["window"]:
            lo = max(0, t - n - c["window"] + 1)
        key = torch.arange(lo, hi, device="cuda")
        see = torch.ones(n, hi - lo, dtype=torch.bool, device="cuda")
        if c["causal"]:
            see &= key <= pos[:, None]
        if c["window"]:
            see &= (pos[:, None] - key).abs() < c["window"]
        o = torch.empty(n, c["kv_heads"] * group, hd, dtype=torch.float64, device="cuda")
        z = torch.empty(n, c["kv_heads"] * group, dtype=torch.float64, device="cuda")
        for h in range(c["kv_heads"]):
            k = st["k_cache"][pages, h].reshape(-1, hd)[lo:hi].double()
            v = st["v_cache"][pages, h].reshape(-1, hd)[lo:hi].double()
            if st["k_scale"] is not None:
                k, v = k * st["k_scale"][h].double(), v * st["v_scale"][h].double()
            for g in range(h * group, (h + 1) * group):
                s = st["q"][rows, g].double() @ k.T / hd ** 0.5
                if c["cap"]:
                    s = torch.tanh(s / c["cap"]) * c["cap"]
                s = torch.where(see, s, -math.inf)
                z[:, g] = torch.logsumexp(s, dim=1)
                o[:, g] = torch.softmax(s, dim=1) @ v
        outs.append(o)
        lses.append(z)
    if c["op"] == "append":
        return {"q": torch.cat(qs), "k": kd, "v": vd}
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
