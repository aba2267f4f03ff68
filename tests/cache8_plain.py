"""Plain forms of the 8-bit cache's operators, and the attention's error bounds.

The plan is whole numbers, in Python lists.  The append rounds values that are given in 16 bits: its codes are the
nearest ones, found from the grid's steps in 64 bits, so they have to be equal.  Bounds of the attention, with u the
half step of the output's type (bf16 2^-8, fp16 2^-11):
 * A score is a D-term fp32 sum times one factor; q is exact in fp16 but for values below 2^-28 of the row's largest
   (off by at most 2^-39 of that): |ds| <= (D + 4) 2^-23 scale sum|q k| + 2^-39 scale max|q| sum|k|.
 * The exponent u_j = log2(e) s_j + log2 vs_j is rounded (2^-24 of its size), log2 vs_j is off by 2^-22 and 2^-24 of its
   size, and exp2 and its argument add 2^-21 + 2^-22 times the row's largest |u_j - R|.  With e the sum of these, a weight is off
   by 1 +- 2e, a normalised one by 4e.
 * A weight is rounded to fp16: 2^-11 of it, or half of 2^-24 absolute where it is subnormal, which beside the largest
   one's 2^11 at least is 2^-36:  |dout| <= u |out| + (2^-11 + 4e + 2^-18) sum p|v| + n 2^-36 448 max vs.
 * |dlse| <= e + 2^-20 (1 + |lse|) + n 2^-24.
"""

import math

import torch

from attention_plain import UNIT

E4M3 = torch.float8_e4m3fn


# -------------------------------------------------------------------- plan ----

def plan(old, keep, new, table, stack, n_free, page):
    """Lists in, (offsets, lengths, table, stack, free, positions, slots, counts) out."""
    table, stack = [list(r) for r in table], list(stack)
    pages = lambda n: -(-n // page)  # noqa: E731
    back = take = 0
    for s, (o, k, n) in enumerate(zip(old, keep, new)):
        for e in range(pages(k + n), pages(o)):
            stack[n_free + back] = table[s][e]
            back += 1
    for s, (o, k, n) in enumerate(zip(old, keep, new)):
        for e in range(pages(o), pages(k + n)):
            table[s][e] = stack[n_free + back - 1 - take]
            take += 1
    offs, pos, slots = [0], [], []
    for s, (k, n) in enumerate(zip(keep, new)):
        for i in range(n):
            p = k + i
            pos.append(p)
            slots.append(table[s][p // page] * page + p % page)
        offs.append(offs[-1] + n)
    return offs, [k + n for k, n in zip(keep, new)], table, stack, n_free + back - take, pos, slots, [offs[-1], take, back, 0]


# ------------------------------------------------------------------ append ----

def nearest_codes(y):
    """The code's values nearest to y (float64 on the CPU, where ldexp is exact), ties to even; NaN and infinities NaN."""
    assert y.device.type == "cpu"
    z = torch.where(torch.isfinite(y), y, 0.0).clamp(-448.0, 448.0)
    _, e = torch.frexp(z.abs().clamp(min=2.0**-6))
    step = torch.ldexp(torch.ones_like(z), e - 4)
    return torch.where(torch.isfinite(y), torch.round(z / step) * step, math.nan)


def exponent_for(most):
    """Least e from -48 to 48 with most <= 448 * 2^e."""
    e = -48
    while e < 48 and most > 448.0 * 2.0**e:
        e += 1
    return e


def append(x, codes, scales, table, new, total, block):
    """x float64 [T, H, D] into codes float64 [pages, P, H, D] and scales [pages, H, P / block], in place."""
    P = codes.shape[1]
    t0 = 0
    for s, (a, b) in enumerate(zip(new, total)):
        p = b - a
        if p < 0:
            t0, p = t0 - p, 0
        while p < b:
            page, lo = int(table[s][p // P]), p % P // block * block
            end = min(b, p - p % block + block)
            for h in range(x.shape[1]):
                y = x[t0:t0 + end - p, h]
                fine = y[torch.isfinite(y)].abs()
                e = exponent_for(float(fine.max()) if fine.numel() else 0.0)
                n_old = p % block
                at = codes[page, lo:lo + block, h]
                if n_old:
                    was = float(scales[page, h, lo // block])
                    if was > 0:
                        e = max(e, min(48, math.ceil(math.log2(was))))
                    if 2.0**e != was:
                        at[:n_old] = nearest_codes(at[:n_old] * was * 2.0**-e)
                at[n_old:n_old + end - p] = nearest_codes(y * 2.0**-e)
                scales[page, h, lo // block] = 2.0**e
            t0 += end - p
            p = end


# --------------------------------------------------------------- attention ----

def values(codes, scales, block_table, s, length, head, block):
    """float64 [length, D] of one kv head, and its scales [length]."""
    P = codes.shape[1]
    used = block_table[s, : -(-length // P)].long()
    sc = scales[used, head].double().flatten().repeat_interleave(block)[:length]
    return codes.view(torch.uint8)[used, :, head].view(E4M3).double().flatten(0, 1)[:length] * sc[:, None], sc


def attention(q, k_pages, v_pages, k_scales, v_scales, block_table, new, total, n_kv_heads, scale, window):
    """(out, lse, out bound, lse bound), float64."""
    T, Hq, D = q.shape
    g = Hq // n_kv_heads
    block = k_pages.shape[1] // k_scales.shape[2]
    u = UNIT[q.dtype]
    dev = q.device
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=dev)
    bound = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=dev)
    lse_bound = torch.zeros_like(lse)
    t0 = 0
    for s, (a, b) in enumerate(zip(new, total)):
        if a and b > 0:
            p = torch.arange(b - a, b, device=dev)[:, None]
            j = torch.arange(b, device=dev)[None, :]
            ok = j <= p
            if window:
                ok &= j > p - window
            any_key = ok.any(1)
            for kv in range(n_kv_heads):
                k, _ = values(k_pages, k_scales, block_table, s, b, kv, block)
                v, vs = values(v_pages, v_scales, block_table, s, b, kv, block)
                lv = torch.log2(vs.clamp(2.0**-48, 2.0**48))
                for h in range(kv * g, kv * g + g):
                    x = q[t0:t0 + a, h].double()
                    zero = torch.zeros(a, dtype=torch.float64, device=dev)
                    sc = ((x @ k.T) * scale).masked_fill(~ok, -math.inf)
                    mag = torch.where(ok, (x.abs() @ k.abs().T) * scale, 0.0).amax(1)
                    m = torch.where(any_key, sc.amax(1), zero)
                    w = torch.exp(sc - m[:, None])
                    safe = torch.where(any_key, w.sum(1), zero + 1)
                    pn = w / safe[:, None]
                    o = pn @ v
                    uj = torch.where(ok, sc / math.log(2) + lv, -math.inf)
                    R = torch.where(any_key, uj.amax(1), zero)
                    spread = torch.where(ok, (uj - R[:, None]).abs().clamp(max=127.0), 0.0).amax(1)
                    size = torch.where(ok, uj.abs(), 0.0).amax(1)
                    e = ((D + 4) * 2.0**-23 * mag + 2.0**-39 * scale * x.abs().amax(1) * k.abs().sum(1).amax()
                         + 2.0**-21 + spread * 2.0**-22 + size * 2.0**-24 + 2.0**-22 + lv.abs().amax() * 2.0**-24)
                    out[t0:t0 + a, h] = o
                    lse[t0:t0 + a, h] = torch.where(any_key, m + torch.log(safe), zero - math.inf)
                    bound[t0:t0 + a, h] = (u * o.abs() + (2.0**-11 + 4 * e + 2.0**-18)[:, None] * (pn @ v.abs())
                                           + b * 2.0**-36 * 448 * vs.amax() + 2.0**-25 * (u == 2.0**-11))
                    size = torch.where(any_key, lse[t0:t0 + a, h].abs(), zero)
                    lse_bound[t0:t0 + a, h] = e + 2.0**-20 * (1 + size) + b * 2.0**-24
        t0 += a
    return out, lse, bound, lse_bound
