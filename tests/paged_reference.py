"""The paged cache's operators in 64 bits, from their definition, and bounds on what fp32 kernels may differ by."""
import math

import torch


def rotate(x, pos, base):
    """Rotate-half of x [n][heads][hd] (float64) by pos [n]."""
    half = x.shape[-1] // 2
    j = torch.arange(half, dtype=torch.float64, device=x.device)
    ang = (pos.double()[:, None] * base ** (-j / half))[:, None]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], dim=-1)


def rotation_slack(x, out):
    """|error| of a rotated element before its rounding: the fp32 fraction of a turn is off by at most 2^-25
    turns (2e-7 rad), sine and cosine by another 2^-23, the two products and their sum by 2^-24 each, all
    times at most |a| + |b|."""
    half = x.shape[-1] // 2
    m = x[..., :half].abs() + x[..., half:].abs()
    return torch.cat([m, m], dim=-1) * (2e-7 + 2.0 ** -23 + 3 * 2.0 ** -24)


def half_step(t, ref):
    """Largest rounding error of type t at ref: half a step, or half the smallest subnormal."""
    sub = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float8_e4m3fn: 2.0 ** -10}[t]
    rel = 2.0 ** -4 if t == torch.float8_e4m3fn else torch.finfo(t).eps / 2
    return ref.abs() * rel + sub


def positions(page_table, kv_len, new, page):
    """Per sequence: [(position, page id)] of its new tokens (page id -1: absent)."""
    out = []
    for b, n in enumerate(new):
        t = max(int(kv_len[b]), 0)
        row = []
        for p in range(t - n, t):
            ok = p >= 0 and p // page < page_table.shape[1]
            row.append((p, int(page_table[b, p // page]) if ok else -1))
        out.append(row)
    return out


def attention(cache, q, new, *, scale=None, causal=True, window=0, cap=0.0):
    """(out, lse, slack) in float64 for packed rows q; cache: an object with k, v, page_table, kv_len, scales.
    slack bounds the kernel's error before the output's rounding."""
    k_pages, v_pages = cache.k, cache.v
    n_pages, hkv, page, hd = k_pages.shape
    hq, dev = q.shape[1], q.device
    g = hq // hkv
    scale = 1 / math.sqrt(hd) if scale is None else scale
    out = torch.zeros(q.shape[0], hq, hd, dtype=torch.float64, device=dev)
    lse = torch.full((q.shape[0], hq), -math.inf, dtype=torch.float64, device=dev)
    slack = torch.zeros_like(out)
    table = cache.page_table.cpu()
    row = 0
    for b, n in enumerate(new):
        if n == 0:
            continue
        t = max(int(cache.kv_len[b]), 0)
        rows = slice(row, row + n)
        row += n
        lim = min(t, table.shape[1] * page)
        j = torch.arange(lim)
        ids = table[b, j // page] if lim else torch.zeros(0, dtype=torch.int32)
        have = (ids >= 0) & (ids < n_pages)
        j, ids = j[have].to(dev), ids[have].long().to(dev)
        p = torch.arange(t - n, t, device=dev)
        see = torch.ones(n, j.numel(), dtype=torch.bool, device=dev)
        if causal:
            see &= j <= p[:, None]
        if window:
            see &= (p[:, None] - j).abs() < window
        kd = k_pages[ids, :, j % page].double()
        vd = v_pages[ids, :, j % page].double()
        if cache.k_scale is not None:
            kd, vd = kd * cache.k_scale.double()[:, None], vd * cache.v_scale.double()[:, None]
        for h in range(hq):
            kh, vh, qh = kd[:, h // g], vd[:, h // g], q[rows, h].double()
            s = qh @ kh.T * scale
            mag = qh.abs() @ kh.abs().T * abs(scale)
            # fp32 accumulation of hd exact products and five more roundings on the way to the exponent;
            # with a cap also tanh's 1 - 2 / (1 + e^2x): three roundings of values up to 1, times cap
            ds = mag * (hd + 5) * 2.0 ** -24 + 2.0 ** -22
            if cap:
                s = cap * torch.tanh(s / cap)
                ds = ds + cap * 6 * 2.0 ** -24 + s.abs() * 4 * 2.0 ** -24
            s = s.masked_fill(~see, -math.inf)
            live = see.any(1)
            top = torch.where(live, s.amax(1) if j.numel() else torch.zeros(n, dtype=torch.float64, device=dev), 0.0)
            e = torch.exp(s - top[:, None])
            tot = e.sum(1)
            pr = e / tot.clamp_min(1e-300)[:, None]
            out[rows, h] = pr @ vh
            lse[rows, h] = torch.where(live, top + torch.log(tot), -math.inf)
            if j.numel():
                worst = torch.where(see, ds, 0.0).amax(1)
                # weights off by e^ds, the sum likewise; P in 16-bit halves (2^-16), or rounded once: to the row
                # type for more than 8 rows per KV head (16 at hd 64) on a 16-bit cache, to fp16 for bf16 rows
                # on an E4M3 cache; fp32 sums over the keys; fp16 weights at worst 2^-25 absolute per key
                p_step = 2.0 ** -16
                if cache.k_scale is None and n * g > (8 if hd >= 128 else 16):
                    p_step = torch.finfo(q.dtype).eps / 2
                elif cache.k_scale is not None and q.dtype == torch.bfloat16:
                    p_step = 2.0 ** -11
                c = 2 * worst + p_step + (see.sum(1) + 16) * 2.0 ** -24
                slack[rows, h] = (pr @ vh.abs()) * c[:, None]
                slack[rows, h] += (see.sum(1) * 2.0 ** -24)[:, None] * vh.abs().amax()
    return out, lse, slack
