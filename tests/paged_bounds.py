"""Attention over the paged cache in 64 bits with a bound on each output that counts the kernels' roundings one by one.

Scores are taken in powers of e.  What separates a kernel's score from the exact one:
  the dot product's fp32 sum        hd * 2^-24 * sum |q k| * scale
  the factor scale * log2 e, its product with the sum, the subtracted maximum    4 * 2^-24 * |s| (and of the maximum)
  a cap c, while |s| <= 0.6 c       the fit of tanh is 1.54e-7 |u| off at most (u + u^3 P(u^2) - tanh u over u, by
                                    evaluation in 64 bits at 2 million points), and five roundings: (1.6e-7 + 5 * 2^-24) |s|
  a cap c, any other score          c tanh = c (1 - 2 / (1 + e^2u)), values of up to c in four roundings: 6 * 2^-24 c
  queries over an E4M3 cache        as fp16 with the row's largest element at 2^14 or more: half a subnormal step is 2^-25,
                                    so each element is off by 2^-39 of the largest at most (bf16's 8 and fp16's 11 bits
                                    are exact above that), the score by that times scale * sum |k|
A weight e^s is off by twice the largest of these (its own and the maximum's), by 2^-22 for the exponential, and by
p_step for its own rounding; sums of n weights in fp32 by n * 2^-24.  fp16 weights are kept 2^7 above their
maximum, so that what a subnormal loses is at most 2^-25 * 2^-7 of the largest weight for each key."""
import math

import torch


def attention(cache, q, new, *, scale=None, causal=True, window=0, cap=0.0, p_step, p_half=False):
    """(out, lse, bound of out before its rounding, bound of lse), float64, for packed rows q."""
    n_pages, hkv, page, hd = cache.k.shape
    hq, dev = q.shape[1], q.device
    g = hq // hkv
    scale = 1 / math.sqrt(hd) if scale is None else scale
    out = torch.zeros(q.shape[0], hq, hd, dtype=torch.float64, device=dev)
    lse = torch.full((q.shape[0], hq), -math.inf, dtype=torch.float64, device=dev)
    bound, lse_bound = torch.zeros_like(out), torch.zeros(q.shape[0], hq, dtype=torch.float64, device=dev)
    table, row = cache.page_table.cpu(), 0
    for b, n in enumerate(new):
        rows = slice(row, row + n)
        row += n
        total = max(int(cache.kv_len[b]), 0)
        j = torch.arange(min(total, table.shape[1] * page))
        ids = table[b, j // page]
        have = (ids >= 0) & (ids < n_pages)
        j, ids = j[have].to(dev), ids[have].long().to(dev)
        if n == 0 or j.numel() == 0:
            continue
        p = torch.arange(total - n, total, device=dev)
        see = torch.ones(n, j.numel(), dtype=torch.bool, device=dev)
        if causal:
            see &= j <= p[:, None]
        if window:
            see &= (p[:, None] - j).abs() < window
        live = see.any(1)
        count = see.sum(1).double()
        for h in range(hkv):
            kh, vh = cache.k[ids, h, j % page].double(), cache.v[ids, h, j % page].double()
            if cache.k_scale is not None:
                kh, vh = kh * cache.k_scale[h].double(), vh * cache.v_scale[h].double()
            heads = slice(h * g, (h + 1) * g)
            qh, seen = q[rows, heads].double().transpose(0, 1), see[None]  # [group][n][hd]
            s = qh @ kh.T * scale
            off = qh.abs() @ kh.abs().T * (scale * hd * 2.0 ** -24)
            if cache.k_scale is not None:
                off += qh.abs().amax(-1, keepdim=True) * kh.abs().sum(1) * (scale * 2.0 ** -39)
            if cap:
                s = cap * torch.tanh(s / cap)
                small = bool((s.abs() <= 0.5 * cap)[seen.expand_as(s)].all())
                off += s.abs() * (1.6e-7 + 5 * 2.0 ** -24) if small else 6 * 2.0 ** -24 * cap
            s = s.masked_fill(~seen, -math.inf)
            top = torch.where(live, s.amax(-1), 0.0)
            off += torch.where(seen, s, 0.0).abs() * 2.0 ** -22 + top.abs()[..., None] * 2.0 ** -22
            worst = torch.where(seen, off, 0.0).amax(-1)
            e = torch.exp(s - top[..., None])
            tot = e.sum(-1)
            pr = e / tot.clamp_min(1e-300)[..., None]
            log_sum = torch.where(live, top + torch.log(tot), -math.inf)
            c = 2 * worst + p_step + 2.0 ** -22 + (count + 16) * 2.0 ** -24
            far = (pr @ vh.abs()) * c[..., None]
            if p_half:
                far += (count / tot.clamp_min(1.0) * 2.0 ** -32)[..., None] * vh.abs().amax()
            far_lse = 2 * worst + (count + 16) * 2.0 ** -24 + torch.where(live, log_sum.abs(), 0.0) * 2.0 ** -22 + 2.0 ** -22
            for to, x in ((out, pr @ vh), (lse, log_sum), (bound, far), (lse_bound, far_lse)):
                to[rows, heads] = x.transpose(0, 1)
    return out, lse, bound, lse_bound


def p_step(cache, q, rows):
    """(rounding of one weight, whether weights are fp16) by the row type, the cache's and a sequence's rows per KV head."""
    e4m3 = cache.k_scale is not None
    half = e4m3 or q.dtype == torch.float16
    if e4m3:
        return 2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -16, half
    one = cache.page_size % 8 == 0 and rows > (8 if cache.head_dim >= 128 else 16)
    return torch.finfo(q.dtype).eps / 2 if one else 2.0 ** -16, half
