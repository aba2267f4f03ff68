"""Plain 64-bit forms of the attention operators, row by row, and the error
bounds that follow from the kernels' number formats.

Derivation of the bounds.  u is the 16-bit type's unit roundoff (bf16 2^-8,
fp16 2^-11); every fp32 step has relative error at most 2^-23 (truncating
accumulation included).
 * A rotated value y = n_a cos -+ n_b sin carries at most about 12 fp32 steps on
   each term (sum of squares in a tree, rsqrt, two products, the rotation):
   12 * 2^-23 < 2^-19 of |n_a cos| + |n_b sin|, then one rounding u |y|.
 * A score is a D-term fp32 sum scaled once: |ds| <= (D + 4) 2^-23 scale sum|q k|.
   exp2 and its argument add 2^-21 + |s| 2^-22.  With e = the largest such
   error of a row (|s| of the row's largest score difference counted), every
   weight is off by a factor within 1 +- 2e, the normalised ones by 4e, and
   the weights are rounded to the 16-bit type (u, or 2^-25 absolute where fp16
   is subnormal; the largest weight is at least 1, so the sum is):
   |dout| <= u |out| + (u + 4e + 2^-18) sum p|v| + n 2^-25 max|v|.
 * lse: |dlse| <= e + 2^-20 (1 + |lse|) + n 2^-24.
"""

import math

import torch

UNIT = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}


def norm_rope(x, w, positions, table, rope_dim, interleaved, eps):
    """x [T, H, D] -> (y, bound), float64 on the CPU."""
    x = x.detach().cpu().double()
    n = x
    if w is not None:
        n = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w.cpu().double()
    y, mag = n.clone(), n.abs().clone()
    half = rope_dim // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c = table[positions.cpu().long(), i].cpu().double()[:, None]
        s = table[positions.cpu().long(), half + i].cpu().double()[:, None]
        y[..., a] = n[..., a] * c - n[..., b] * s
        y[..., b] = n[..., b] * c + n[..., a] * s
        mag[..., a] = (n[..., a] * c).abs() + (n[..., b] * s).abs()
        mag[..., b] = (n[..., b] * c).abs() + (n[..., a] * s).abs()
    return y, mag


def norm_rope_bound(y, mag, dtype):
    return UNIT[dtype] * y.abs() + 2.0**-19 * mag + 2.0**-25


def positions_of(new, total):
    return torch.cat([torch.arange(b - a, b) for a, b in zip(new, total)]) if new else torch.zeros(0, dtype=torch.long)


def gather_sequence(pages, block_table, s, length):
    """The first `length` cached rows [length, heads, D] of sequence s."""
    P = pages.shape[1]
    used = block_table[s, : -(-length // P)].long().to(pages.device)
    return pages[used].flatten(0, 1)[:length]


def attention(q, k_pages, v_pages, block_table, new, total, n_kv_heads, scale, window):
    """(out, lse, out bound, lse bound): float64 on the tensors' device, a sequence and a kv head at a time."""
    T, Hq, D = q.shape
    g = Hq // n_kv_heads
    u = UNIT[q.dtype]
    dev = q.device
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=dev)
    bound = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=dev)
    lse_bound = torch.zeros_like(lse)
    t0 = 0
    for s, (a, b) in enumerate(zip(new, total)):
        if a and b > 0:
            K, V = (gather_sequence(x, block_table, s, b).double() for x in (k_pages, v_pages))
            p = torch.arange(b - a, b, device=dev)[:, None]
            j = torch.arange(b, device=dev)[None, :]
            ok = j <= p
            if window:
                ok &= j > p - window
            for h in range(Hq):
                x = q[t0:t0 + a, h].double()
                k, v = K[:, h // g], V[:, h // g]
                raw = (x @ k.T) * scale
                mag = (x.abs() @ k.abs().T) * scale
                sc = raw.masked_fill(~ok, -math.inf)
                any_key = ok.any(1)
                m = torch.where(any_key, sc.amax(1), torch.zeros(a, dtype=torch.float64, device=dev))
                w = torch.exp(sc - m[:, None])
                l = w.sum(1)
                safe = torch.where(any_key, l, torch.ones_like(l))
                pn = w / safe[:, None]
                o = pn @ v
                spread = torch.where(ok, (sc - m[:, None]).abs().clamp(max=88.0), torch.zeros_like(sc)).amax(1)
                e = (D + 4) * 2.0**-23 * torch.where(ok, mag, torch.zeros_like(mag)).amax(1) + 2.0**-21 + spread * 2.0**-22
                out[t0:t0 + a, h] = o
                lse[t0:t0 + a, h] = torch.where(any_key, m + torch.log(safe), torch.full_like(m, -math.inf))
                vmax = v.abs().amax() if b else 0.0
                bound[t0:t0 + a, h] = (u * o.abs() + (u + 4 * e + 2.0**-18)[:, None] * (pn @ v.abs())
                                       + b * 2.0**-25 * vmax)
                lse_bound[t0:t0 + a, h] = e + 2.0**-20 * (1 + torch.where(any_key, lse[t0:t0 + a, h].abs(),
                                                                          torch.zeros_like(m))) + b * 2.0**-24
        t0 += a
    return out, lse, bound, lse_bound
