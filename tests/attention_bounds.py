"""The 64-bit form of single-token attention with bounds counted tightly from what the kernels
round:
  query    fp16 after a power of two that brings the row's largest value to [128, 256): values
           down to 2^-24 of the largest keep their 8 bits, smaller ones are off by at most half of
           fp16's smallest step, 2^-25 / 2^7 = 2^-32 of it
  weights  p vs as fp16 of a unit whose range the row's largest weighted value sets (the largest
           over the tokens whose codes are not all zero): 2^-11 relative, and below the normal
           range half a smallest step, 2^-39 of that largest value (the largest is brought to
           2^14 and more) or, in the tcgen05 prefix kernel, 2^-25 (to 1 and more)
  float32  sums of head_dim products, the score's factors, the exponent's argument, exp2 (2 ulp),
           the sums over tokens"""

import torch

from decode_ref import U16, U32, cache_values, gather

OWN, TCGEN05 = 2.0 ** -39, 2.0 ** -25


def attention(q, cache, page_table, lengths, scale, prefix_pages=None, prefix_length=0, unit=OWN,
              score_error=0.0):
    """(out, lse, bound of |out error| before the output rounding, bound of |lse error|).
    score_error: a further relative error of the scores."""
    b, heads, d = q.shape
    n_kv, page = cache[0].shape[1:3]
    group = heads // n_kv
    kval, vval = cache_values(cache)
    codes = cache[2].view(torch.float8_e4m3fn).double()
    vscale = cache[3].double()[..., None]
    out = torch.zeros((b, heads, d), dtype=torch.float64, device=q.device)
    lse = torch.full((b, heads), -float("inf"), dtype=torch.float64, device=q.device)
    bound, lbound = torch.zeros_like(out), torch.zeros_like(lse)
    for i in range(b):
        n = max(0, min(int(lengths[i]), page_table.shape[1] * page))
        parts = [gather(a, page_table[i], n, page) for a in (kval, vval, codes, vscale)]
        if prefix_pages is not None:
            m = max(0, min(int(prefix_length), prefix_pages.numel() * page))
            parts = [torch.cat((gather(a, prefix_pages, m, page), own), 1)
                     for a, own in zip((kval, vval, codes, vscale), parts)]
        n = parts[0].shape[1]
        if n == 0:
            continue
        k, v, c, vs = (a.repeat_interleave(group, 0) for a in parts)
        qi = q[i].double()
        s = torch.einsum("hd,htd->ht", qi, k) * scale
        lse[i] = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[i][:, None])
        out[i] = torch.einsum("ht,htd->hd", p, v)
        absk = torch.einsum("hd,htd->ht", qi.abs(), k.abs()) * abs(scale)
        # a token's score: its own error, as a factor of its weight
        ds = (2.0 ** -32 * qi.abs().amax(-1)[:, None] * k.abs().sum(-1) * abs(scale)
              + (d + 8) * U32 * 2 * absk + (8 * U32 + score_error) * s.abs()
              + 4 * U32 * (s - s.amax(-1, keepdim=True)).abs() + 16 * U32)
        sums = U32 * 2 * (n / 32 + 128)
        weight = p * vs[..., 0].abs()
        some = (c != 0).any(-1)
        top = torch.where(some, weight, torch.zeros_like(weight)).amax(-1)
        dl = (p * ds).sum(-1) + sums
        pv = p[..., None] * v.abs()
        bound[i] = ((pv * (U16 + ds)[..., None]).sum(1) + pv.sum(1) * (sums + dl[:, None])
                    + unit * top[:, None] * c.abs().sum(1)) * (1 + 2.0 ** -8)
        lbound[i] = dl * (1 + 2.0 ** -8) + 4 * U32 * lse[i].abs()
    return out, lse, bound, lbound
