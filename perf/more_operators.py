"""Timed cases of the 8-bit cache's operators: block tables and slot maps from request lengths, the append that
quantises keys and values, attention over the cache.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()`` makes a case's inputs on the
GPU, ``run()`` is one pass (the library's calls where ``own`` is true, else elementary torch operations),
``work()`` the bytes and operations a pass cannot do without and ``exact()`` the definition in 64 bits.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6
THETA = 10000.0
SCALE_EXP = 48  # scales that the append makes lie in 2^-48 .. 2^48


def _case(op, name=None, **kw):
    c = {"op": op, "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128, "rope": 128, "interleaved": False,
         "norm": True, "page": 64, "block": 64, "seqs": 1, "new": 1, "context": 0, "ragged": False, "window": 0,
         "with_q": True, "lse": False, "drafts": 0, "ended": 0}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a decode step's tables: one token of each of 64 running requests, few of which need a page (latency)
        _case("plan", "plan_decode_64", seqs=64, new=1, context=4096),
        # a busy server's step: 512 requests of ragged chunks, one in eight just ended and gave its place to a new
        # one, the others dropping up to 7 rejected drafts; 16-token pages
        _case("plan", "plan_mixed_512", seqs=512, new=96, context=2000, ragged=True, page=16, drafts=7, ended=8),
        # prompts only: 64 new requests, 256,000 tokens in all (bandwidth of the maps)
        _case("plan", "plan_prompts_64", seqs=64, new=4000, context=0, page=64),
        # the decode step's append of 64 sequences, q rotated in the same call (latency)
        _case("append", "append8_decode_64", seqs=64, new=1, context=4096, ragged=True),
        # a long prompt's keys and values alone into pages of 64 (bandwidth)
        _case("append", "append8_prompt_32768", seqs=8, new=4096, context=1000, ragged=True, with_q=False),
        # odd sizes: ragged chunks, 96-wide heads of which 64 values rotate in interleaved pairs, pages of 48, fp16
        _case("append", "append8_odd", dtype="fp16", heads=24, kv_heads=4, dim=96, rope=64, interleaved=True, seqs=5,
              new=777, context=1500, ragged=True, page=48, block=16),
        # the smallest attention: one token of one short sequence of a narrow model (latency)
        _case("attention", "attn8_one_token", heads=4, kv_heads=2, dim=64, rope=64, page=16, block=16, context=512),
        # the decode batch of 64 sequences of unequal length up to 16,384 tokens (bandwidth)
        _case("attention", "attn8_decode_64", seqs=64, new=1, context=16384, ragged=True),
        # one long sequence: the keys of a single token are split over the whole GPU
        _case("attention", "attn8_decode_131072", seqs=1, new=1, context=131072, page=128, block=128),
        # a mixed step, odd everywhere: short chunks, 6 heads a kv head, 96-wide heads, pages of 48, fp16, with lse
        _case("attention", "attn8_mixed_odd", dtype="fp16", heads=24, kv_heads=4, dim=96, rope=96, page=48, block=16,
              seqs=9, new=333, context=3001, ragged=True, lse=True),
        # a whole prompt of 8,192 tokens (tensor cores)
        _case("attention", "attn8_prompt_8192", seqs=1, new=8192),
        # a chunk of 2,048 tokens of a prompt whose first 63,488 are in the cache
        _case("attention", "attn8_chunk_65536", seqs=1, new=2048, context=63488, block=32),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention"])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 6, 8])
    dim = rng.choice([64, 64, 96, 128, 128, 128])
    page = rng.choice([16, 32, 48, 64, 128])
    c = _case(op, dtype=rng.choice(["bf16", "bf16", "fp16"]), heads=heads, kv_heads=kv_heads, dim=dim,
              rope=rng.choice([dim, dim, 64, 32]), interleaved=rng.random() < 0.3, norm=rng.random() < 0.7, page=page,
              block=rng.choice([b for b in (16, 32, 64, 128) if page % b == 0]), ragged=rng.random() < 0.6,
              with_q=rng.random() < 0.6, lse=rng.random() < 0.3)
    if op == "plan":
        c["seqs"] = _logint(rng, 1, 1024)
        c["new"] = _logint(rng, 1, max(1, 256000 // c["seqs"]))
        c["context"] = _logint(rng, 1, 8192)
        c["drafts"] = rng.choice([0, 0, 3, 7])
        c["ended"] = rng.choice([0, 4, 16])
        return c
    if op == "append":
        tokens = _logint(rng, 64, 32768)
        c["seqs"] = min(_logint(rng, 1, 64), tokens)
        c["new"] = tokens // c["seqs"]
        c["context"] = _logint(rng, 1, 8192)
        return c
    if rng.random() < 0.5:  # single tokens
        c["seqs"] = _logint(rng, 1, 64)
        c["new"] = 1
        c["context"] = _logint(rng, 32, min(131072, 1048576 // c["seqs"]))
    else:  # chunks: at most as many scores as the listed ones
        c["seqs"] = _logint(rng, 1, 8)
        c["new"] = _logint(rng, 2, 4096 // c["seqs"])
        most = min(65536 // c["seqs"], (1 << 31) // (heads * c["new"] * c["seqs"]))
        c["context"] = _logint(rng, 1, max(2, most - c["new"]))
    if rng.random() < 0.2:
        c["window"] = _logint(rng, 16, 4096)
    return c


# ------------------------------------------------------------------ inputs ----

def _lens(c):
    """New tokens and cached tokens (the new ones among them) of each sequence; a function of the case alone."""
    new = [c["new"]] * c["seqs"]
    old = [c["context"]] * c["seqs"]
    if c["ragged"]:
        r = random.Random(c["seqs"] * 1000003 + c["new"] * 10007 + c["context"])
        for s in range(1, c["seqs"]):  # the first sequence is the longest
            if c["new"] > 1:
                new[s] = r.randint(1, c["new"])
            old[s] = r.randint(0, c["context"])
    return new, [a + b for a, b in zip(new, old)]


def _requests(c):
    """(tokens cached, tokens kept of them, tokens new) of each request; a function of the case alone."""
    new, total = _lens(c)
    r = random.Random(c["seqs"] * 7919 + c["new"])
    old = [b - a for a, b in zip(new, total)]
    keep = [max(0, n - r.randint(0, c["drafts"])) for n in old]
    if c["ended"]:
        keep = [0 if s % c["ended"] == c["ended"] - 1 else n for s, n in enumerate(keep)]
    return old, keep, new


def _randn(shape, gen, dtype, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    x.normal_(0.0, scale, generator=gen)
    return x


def _codes(shape, gen):
    """Codes of normal values whose blocks' largest comes near the type's."""
    x = torch.empty(shape, dtype=E4M3, device="cuda")
    for at in range(0, shape[0], 4096):
        y = _randn((min(4096, shape[0] - at),) + shape[1:], gen, torch.bfloat16, 100.0)
        x[at:at + 4096] = y.clamp_(-448, 448).to(E4M3)
    return x


def _prepare_plan(c, gen):
    old, keep, new = _requests(c)
    P = c["page"]
    had = [-(-a // P) for a in old]
    need = [-(-(a + b) // P) for a, b in zip(keep, new)]
    grow = sum(max(0, n - h) for h, n in zip(had, need))
    n_pages = sum(had) + grow + 5
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    width = max(had + need)
    table = torch.zeros((c["seqs"], width), dtype=torch.int32, device="cuda")
    h = torch.tensor(had, device="cuda")
    e = torch.arange(width, device="cuda")
    first = h.cumsum(0) - h
    table = torch.where(e < h[:, None], ids[(first[:, None] + e).clamp(max=n_pages - 1)], table)
    free = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    n_free = n_pages - sum(had)
    free[:n_free] = ids[sum(had):]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"case": c, "kv_len": i32(old), "keep_len": i32(keep) if c["drafts"] or c["ended"] else None,
            "new_len": i32(new), "block_table": table, "free_pages": free, "n_free": i32([n_free]), "T": sum(new)}


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if c["op"] == "plan":
        return _prepare_plan(c, gen)
    dt = DTYPES[c["dtype"]]
    new, total = _lens(c)
    T, Hq, Hk, D, P, B = sum(new), c["heads"], c["kv_heads"], c["dim"], c["page"], c["block"]
    s = {"case": c, "T": T, "max_new": max(new), "max_total": max(total)}
    offs = torch.tensor([0] + new).cumsum(0)
    s["seq_offsets"] = offs.to(torch.int64).cuda()
    s["kv_len"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    seq = torch.repeat_interleave(torch.arange(c["seqs"]), torch.tensor(new))
    pos = torch.arange(T) - offs[seq] + (torch.tensor(total) - torch.tensor(new))[seq]
    s["seq"], s["pos"] = seq.cuda(), pos.to(torch.int32).cuda()
    per = [-(-n // P) for n in total]
    n_pages = sum(per) + 3
    # the cache: codes and a scale for each block of tokens and head, as an earlier program left them
    s["k_pages"], s["v_pages"] = _codes((n_pages, P, Hk, D), gen), _codes((n_pages, P, Hk, D), gen)
    for n in ("k_scales", "v_scales"):
        x = 0.005 + 0.01 * torch.rand((n_pages, Hk, P // B), generator=gen, device="cuda")
        s[n] = x if c["op"] == "attention" else torch.exp2(torch.ceil(torch.log2(x)))
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((c["seqs"], max(per)), dtype=torch.int32)
    at, order = 0, order.cpu()
    for i, n in enumerate(per):
        table[i, :n] = order[at:at + n]
        at += n
    s["block_table"] = table.cuda()
    if c["op"] == "attention":  # normed and rotated already: heads of length about sqrt(D)
        s["q"] = _randn((T, Hq, D), gen, dt)
        return s
    # the layer's packed projection, q | k | v for each token
    s["qkv"] = _randn((T, (Hq + 2 * Hk) * D), gen, dt)
    q, k, v = s["qkv"].split([Hq * D, Hk * D, Hk * D], 1)
    s["q"], s["k"], s["v"] = q.unflatten(1, (Hq, D)), k.unflatten(1, (Hk, D)), v.unflatten(1, (Hk, D))
    for n in ("w_q", "w_k"):
        s[n] = (1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt) if c["norm"] else None
    half = c["rope"] // 2
    freq = THETA ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(max(total), dtype=torch.float64, device="cuda")[:, None] * freq
    s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    return s


# ------------------------------------------------------------------- plain ----

def _plain_plan(s):
    """Pages given back go on top of the stack in the order of (request, entry), those taken come off its top in
    that order."""
    c, table, free = s["case"], s["block_table"], s["free_pages"]
    P, T = c["page"], s["T"]
    old, new, n_free = s["kv_len"].long(), s["new_len"].long(), s["n_free"].long()
    keep = old if s["keep_len"] is None else s["keep_len"].long()
    after = keep + new
    had, need = (old + P - 1) // P, (after + P - 1) // P
    back, take = (had - need).clamp(min=0), (need - had).clamp(min=0)
    back_to, take_to = back.cumsum(0), take.cumsum(0)
    n, width = table.shape
    e = torch.arange(width, device="cuda")
    # the stack with what is given back on it; entries that are not given back go to a place past its end
    gives = (e >= need[:, None]) & (e < had[:, None])
    at = torch.where(gives, n_free + (back_to - back - need)[:, None] + e, free.numel())
    stack = torch.cat([free, free[:1]])
    stack.scatter_(0, at.flatten(), table.flatten())
    free.copy_(stack[:-1])
    takes = (e >= had[:, None]) & (e < need[:, None])
    top = n_free + back_to[-1] - 1
    at = torch.where(takes, top - ((take_to - take - had)[:, None] + e), 0)
    table.copy_(torch.where(takes, free[at], table))
    offs = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(offs, t, right=True) - 1
    pos = keep[seq] + t - offs[seq]
    slots = table[seq, pos // P].long() * P + pos % P
    left = n_free + back_to[-1:] - take_to[-1:]
    counts = torch.cat([offs[-1:], take_to[-1:], back_to[-1:], torch.zeros_like(left)])
    return {"block_table": table, "free_pages": free, "seq_offsets": offs, "kv_len": after.int(), "n_free": left.int(),
            "positions": pos.int(), "slots": slots, "counts": counts.int()}


def _norm_rope(x, w, cs, c):
    """x [T, H, D] fp32; cs [T, rope] (cosines, then sines)."""
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    r = c["rope"]
    cos, sin = cs[:, None, : r // 2], cs[:, None, r // 2:]
    rot, rest = x[..., :r], x[..., r:]
    if c["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = rot[..., : r // 2], rot[..., r // 2:]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([rot, rest], -1)


def _scale_for(most):
    """The least power of two, within its limits, whose 448-fold holds `most`."""
    m, e = torch.frexp(most)
    e = torch.where(most > 0, e - 9 + (m > 0.875), -SCALE_EXP).clamp(-SCALE_EXP, SCALE_EXP)
    return torch.ldexp(torch.ones_like(most), e)


def _quantise(x, scale):
    return (x / scale).clamp(-448, 448).to(E4M3)


def _plain_append_one(s, x, pages, scales):
    """x [T, Hk, D] (fp32) into pages; a block's scale holds its new tokens and, where it has earlier ones, is no
    smaller than before: those are rounded again if it grows."""
    c = s["case"]
    P, B = c["page"], c["block"]
    Hk, D = c["kv_heads"], c["dim"]
    seq, pos, table = s["seq"], s["pos"].long(), s["block_table"]
    page, slot = table[seq, pos // P].long(), pos % P
    blocks = pages.shape[0] * (P // B)
    by_block = scales.transpose(1, 2).reshape(blocks, Hk)
    of = page * (P // B) + slot // B
    most = torch.zeros((blocks, Hk), device="cuda")
    most.scatter_reduce_(0, of[:, None].expand(-1, Hk), x.abs().amax(-1), "amax")
    # the block that a sequence's first new token falls into, where earlier tokens are in it
    n_new = s["seq_offsets"][1:] - s["seq_offsets"][:-1]
    first = s["kv_len"].long() - n_new
    p0 = table.gather(1, (first // P)[:, None].long())[:, 0].long()
    b0 = p0 * (P // B) + first % P // B
    begun = first % B > 0
    touched = torch.zeros(blocks, dtype=torch.bool, device="cuda")
    touched[of] = True
    earlier = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    earlier.scatter_reduce_(0, b0, begun.int(), "amax")
    before = by_block.clone()
    need = _scale_for(most)
    now = torch.where(earlier[:, None] > 0, torch.maximum(need, before), need)
    now = torch.where(touched[:, None], now, before)
    scales.copy_(now.view(pages.shape[0], P // B, Hk).transpose(1, 2))
    flat = pages.view(blocks, B, Hk, D)
    values = flat[b0].float() * before[b0][:, None, :, None]
    again = _quantise(values, now[b0][:, None, :, None])
    old = (torch.arange(B, device="cuda") < (first % B)[:, None])[:, :, None, None]
    # through bytes: selecting and indexing by place is for them
    kept = torch.where(old, again.view(torch.uint8), flat[b0].view(torch.uint8))
    raw = flat.view(torch.uint8)
    raw[b0] = torch.where(begun[:, None, None, None], kept, raw[b0])
    raw[of, slot % B] = _quantise(x, now[of][:, :, None]).view(torch.uint8)


def _plain_append(s):
    c, dt = s["case"], s["q"].dtype
    cs = s["table"][s["pos"].long()]
    # keys are what a 16-bit cache would hold, then quantised
    k = _norm_rope(s["k"].float(), s["w_k"], cs, c).to(dt).float()
    _plain_append_one(s, k, s["k_pages"], s["k_scales"])
    _plain_append_one(s, s["v"].float(), s["v_pages"], s["v_scales"])
    out = {n: s[n] for n in ("k_pages", "v_pages", "k_scales", "v_scales")}
    if c["with_q"]:
        out["q"] = _norm_rope(s["q"].float(), s["w_q"], cs, c).to(dt)
    return out


def _values(s, which, pages):
    """[n, pages, P, Hk, D] fp32 values of the given pages."""
    c = s["case"]
    scale = s[which + "_scales"][pages].transpose(2, 3).repeat_interleave(c["block"], 2)
    return s[which + "_pages"].view(torch.uint8)[pages].view(E4M3).float() * scale[..., None]


def _plain_attention(s):
    c, q = s["case"], s["q"]
    T, Hq, D = q.shape
    Hk, n, mn, mt = c["kv_heads"], c["seqs"], s["max_new"], s["max_total"]
    g = Hq // Hk
    offs, total = s["seq_offsets"], s["kv_len"].long()
    pages = s["block_table"].long()
    j = torch.arange(mt, device="cuda")
    there = (j[None, :] < total[:, None])[:, :, None, None]  # [n, keys, 1, 1]
    K = _values(s, "k", pages).flatten(1, 2)[:, :mt]
    V = _values(s, "v", pages).flatten(1, 2)[:, :mt]
    K = torch.where(there, K, 0).permute(0, 2, 3, 1)  # [n, Hk, D, keys]
    V = torch.where(there, V, 0).permute(0, 2, 1, 3)  # [n, Hk, keys, D]
    i = torch.arange(mn, device="cuda")
    row = (offs[:-1, None] + i).clamp(max=T - 1)  # [n, new]
    Q = q[row].float().view(n, mn, Hk, g, D).permute(0, 2, 3, 1, 4).reshape(n, Hk, g * mn, D)
    S = torch.matmul(Q, K).mul_(1.0 / math.sqrt(D)).view(n, Hk, g, mn, mt)
    pos = (total - (offs[1:] - offs[:-1]))[:, None] + i  # [n, new]
    ok = j <= pos[..., None]
    if c["window"]:
        ok &= j > pos[..., None] - c["window"]
    S.masked_fill_(~ok[:, None, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    S.sub_(m).exp_()
    total_weight = S.sum(-1, keepdim=True)
    O = torch.matmul(S.view(n, Hk, g * mn, mt), V).view(n, Hk, g, mn, D) / total_weight
    seq, at = s["seq"], torch.arange(T, device="cuda") - offs[s["seq"]]
    out = O[seq, :, :, at].reshape(T, Hq, D).to(q.dtype)
    if not c["lse"]:
        return {"out": out}
    lse = (m + total_weight.log()).squeeze(-1)[seq, :, :, at].reshape(T, Hq)
    return {"out": out, "lse": lse}


# --------------------------------------------------------------------- run ----

def _own_plan(s):
    import engram_gram_hash_gb300 as eg

    p = eg.engram_kv_plan(s["new_len"], s["kv_len"], s["block_table"], s["free_pages"], s["n_free"],
                          page_size=s["case"]["page"], max_tokens=s["T"], keep_len=s["keep_len"])
    return {"block_table": s["block_table"], "free_pages": s["free_pages"], "seq_offsets": p.seq_offsets,
            "kv_len": p.kv_len, "n_free": p.n_free, "positions": p.positions, "slots": p.slots, "counts": p.counts}


def _handles(s):
    """What a program makes once for a layer (cfg), its cache and its batch, and keeps from call to call."""
    import engram_gram_hash_gb300 as eg

    c = s["case"]
    s["cfg"] = eg.make_attn_config(c["heads"], c["kv_heads"], c["dim"], dtype=DTYPES[c["dtype"]], rope_dim=c["rope"],
                                   rope_interleaved=c["interleaved"], norm_eps=EPS, window=c["window"])
    s["cache"] = eg.kv_cache_q8(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"])
    s["batch"] = eg.kv_batch(s["seq_offsets"], s["kv_len"], s["block_table"], s["T"])


def _own(s):
    import engram_gram_hash_gb300 as eg

    c = s["case"]
    if c["op"] == "plan":
        return _own_plan(s)
    if "cfg" not in s:
        _handles(s)
    if c["op"] == "append":
        out = {n: s[n] for n in ("k_pages", "v_pages", "k_scales", "v_scales")}
        q = eg.engram_kv_append_q8(s["cfg"], s["cache"], s["batch"], s["k"], s["v"], s["table"], w_k=s["w_k"],
                                   q=s["q"] if c["with_q"] else None, w_q=s["w_q"] if c["with_q"] else None)
        if c["with_q"]:
            out["q"] = q
        return out
    if c["lse"]:
        lse = torch.empty((s["T"], c["heads"]), dtype=torch.float32, device="cuda")
        return {"out": eg.engram_paged_attention_q8(s["cfg"], s["cache"], s["batch"], s["q"], lse=lse), "lse": lse}
    return {"out": eg.engram_paged_attention_q8(s["cfg"], s["cache"], s["batch"], s["q"])}


def _plain(s):
    return {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention}[s["case"]["op"]](s)


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work ----

def work(case):
    c = case
    if c["op"] == "plan":
        old, keep, new = _requests(c)
        P, n, T = c["page"], c["seqs"], sum(new)
        had = [-(-a // P) for a in old]
        need = [-(-(a + b) // P) for a, b in zip(keep, new)]
        moved = sum(abs(h - x) for h, x in zip(had, need))
        pages = sum(-(-(a + b) // P) - a // P for a, b in zip(keep, new) if b)  # table entries that the slots name
        ints = n * (4 if c["drafts"] or c["ended"] else 3)  # lengths in, lengths out
        return {"bytes": 4 * ints + 8 * (n + 1) + 8 * moved + 4 * pages + 12 * T, "flops": 0}
    new, total = _lens(c)
    T, Hq, Hk, D, B, e = sum(new), c["heads"], c["kv_heads"], c["dim"], c["block"], 2
    if c["op"] == "attention":
        keys = pairs = 0
        for a, b in zip(new, total):
            w = c["window"] or b
            first = b - a  # position of the first new token
            keys += b - max(0, first - w + 1)
            # sum over positions p of min(p + 1, w)
            short = max(0, min(b, w) - first)  # positions that see all keys before them
            pairs += short * (2 * first + short + 1) // 2 + (a - short) * w
        return {"bytes": 2 * T * Hq * D * e + 2 * keys * Hk * D + 8 * (-(-keys // B)) * Hk + (T * Hq * 4 if c["lse"] else 0),
                "flops": 4 * D * Hq * pairs}
    rotated = Hk + (Hq if c["with_q"] else 0)
    blocks = sum((b - 1) // B - (b - a) // B + 1 for a, b in zip(new, total))
    moved = 2 * T * Hk * D * (e + 1) + T * c["rope"] * 4 + 2 * 4 * blocks * Hk
    if c["with_q"]:
        moved += 2 * T * Hq * D * e
    return {"bytes": moved, "flops": T * rotated * (3 * c["rope"] + (4 * D if c["norm"] else 0)) + 4 * T * Hk * D}


# ------------------------------------------------------------------- exact ----

def _exact_rot(x, w, pos, table, c):
    """Head by head: norm, then each pair of values as a complex number turned by the position's angle."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + EPS) * w.double()
    r = c["rope"]
    half = r // 2
    t = table.double()[pos.long()]
    turn = torch.complex(t[:, :half], t[:, half:])[:, None, :]
    y = y.clone()
    if c["interleaved"]:
        z = torch.view_as_complex(y[..., :r].unflatten(-1, (half, 2)).contiguous()) * turn
        y[..., :r] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :half].contiguous(), y[..., half:r].contiguous()) * turn
        y[..., :half], y[..., half:r] = z.real, z.imag
    return y


def _exact_codes(y):
    """The values of the type's codes nearest to y: eight steps to a power of two, from 2^-9 on."""
    y = y.clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0**-6))) - 3)
    return torch.round(y / step) * step


def _exact_pages(s, x, pages, scales):
    """Sequence by sequence, block by block of tokens."""
    c = s["case"]
    P, B = c["page"], c["block"]
    new, total = _lens(c)
    codes, scales = pages.double(), scales.double()
    table = s["block_table"].cpu().tolist()
    t0 = 0
    for i, (a, b) in enumerate(zip(new, total)):
        p = b - a
        while p < b:
            page, lo = table[i][p // P], p % P // B * B
            end = min(b, p - p % B + B)
            n_old, n_new = p % B, end - p
            y = x[t0:t0 + n_new]
            most = y.abs().amax((0, 2))
            exponent = torch.where(most > 0, torch.ceil(torch.log2(most / 448.0)), -float(SCALE_EXP))
            scale = torch.exp2(exponent.clamp(-SCALE_EXP, SCALE_EXP))
            at = codes[page, lo:lo + B]
            if n_old:
                was = scales[page, :, lo // B]
                scale = torch.maximum(scale, was)
                at[:n_old] = _exact_codes(at[:n_old] * (was / scale)[:, None])
            at[n_old:n_old + n_new] = _exact_codes(y / scale[:, None])
            scales[page, :, lo // B] = scale
            t0 += n_new
            p = end
    return codes, scales


def _exact_attention(s):
    c, q = s["case"], s["q"]
    T, Hq, D = q.shape
    g = Hq // c["kv_heads"]
    new, total = _lens(c)
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for i, (a, b) in enumerate(zip(new, total)):
        used = s["block_table"][i, : -(-b // c["page"])].long()
        step = max(1, (1 << 27) // b)
        for kv in range(c["kv_heads"]):
            k, v = (s[n + "_pages"].view(torch.uint8)[used, :, kv].view(E4M3).double().flatten(0, 1)[:b]
                    * s[n + "_scales"].double()[used, kv].flatten().repeat_interleave(c["block"])[:b, None]
                    for n in ("k", "v"))
            for h in range(kv * g, kv * g + g):
                for x in range(0, a, step):
                    y = min(a, x + step)
                    score = (q[t0 + x:t0 + y, h].double() @ k.T) / math.sqrt(D)
                    p = torch.arange(b - a + x, b - a + y, device="cuda")[:, None]
                    key = torch.arange(b, device="cuda")[None, :]
                    hidden = key > p
                    if c["window"]:
                        hidden |= p - key >= c["window"]
                    score.masked_fill_(hidden, -math.inf)
                    lse[t0 + x:t0 + y, h] = torch.logsumexp(score, -1)
                    out[t0 + x:t0 + y, h] = torch.softmax(score, -1) @ v
        t0 += a
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    if -(-s["T"] // case["block"]) + 2 * case["seqs"] > 20000:
        return None
    k = _exact_rot(s["k"], s["w_k"], s["pos"], s["table"], case).to(s["q"].dtype).double()
    out = {}
    out["k_pages"], out["k_scales"] = _exact_pages(s, k, s["k_pages"], s["k_scales"])
    out["v_pages"], out["v_scales"] = _exact_pages(s, s["v"].double(), s["v_pages"], s["v_scales"])
    if case["with_q"]:
        out["q"] = _exact_rot(s["q"], s["w_q"], s["pos"], s["table"], case)
    return out
