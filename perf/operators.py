"""Timed cases of the attention operators: head norm + rotation, paged-cache append, paged attention.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()`` makes a case's inputs on the
GPU, ``run()`` is one pass (the library's calls where ``own`` is true, else elementary torch operations in fp32),
``work()`` the bytes and operations a pass cannot do without and ``exact()`` the definition in 64 bits.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
THETA = 10000.0


def _case(op, name=None, **kw):
    c = {"op": op, "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128, "rope": 128, "interleaved": False,
         "norm": True, "page": 64, "seqs": 1, "new": 1, "context": 0, "ragged": False, "window": 0, "with_q": True,
         "lse": False}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # head norm + rotation of a decode batch: one token of each of 64 sequences (latency)
        _case("qk_norm_rope", "qk_decode_64", seqs=64, new=1, context=4096),
        # a 32,768-token prompt of a model of width 4096 (bandwidth)
        _case("qk_norm_rope", "qk_prompt_32768", seqs=1, new=32768),
        # odd sizes: ragged prompts, 96-wide heads of which 64 values rotate in interleaved pairs, fp16
        _case("qk_norm_rope", "qk_odd", dtype="fp16", heads=24, kv_heads=4, dim=96, rope=64, interleaved=True, seqs=5,
              new=777, context=1500, ragged=True),
        # the decode step's append of 64 sequences, q rotated in the same call (latency)
        _case("kv_append", "append_decode_64", seqs=64, new=1, context=4096),
        # a long prompt's keys and values alone into pages of 64 (bandwidth)
        _case("kv_append", "append_prompt_32768", seqs=8, new=4096, context=1000, ragged=True, with_q=False),
        # the smallest attention: one token of one short sequence of a narrow model (latency)
        _case("attention", "attn_one_token", heads=4, kv_heads=2, dim=64, rope=64, page=16, context=512),
        # the decode batch of 64 sequences of unequal length up to 16,384 tokens (bandwidth)
        _case("attention", "attn_decode_64", seqs=64, new=1, context=16384, ragged=True),
        # one long sequence: the keys of a single token are split over the whole GPU
        _case("attention", "attn_decode_131072", seqs=1, new=1, context=131072, page=128),
        # a mixed step, odd everywhere: short chunks, 6 heads a kv head, 96-wide heads, pages of 48, fp16, with lse
        _case("attention", "attn_mixed_odd", dtype="fp16", heads=24, kv_heads=4, dim=96, rope=96, page=48, seqs=9,
              new=333, context=3001, ragged=True, lse=True),
        # a whole prompt of 8,192 tokens (tensor cores)
        _case("attention", "attn_prompt_8192", seqs=1, new=8192),
        # a chunk of 2,048 tokens of a prompt whose first 63,488 are in the cache
        _case("attention", "attn_chunk_65536", seqs=1, new=2048, context=63488),
        # 8 prompts under a sliding window of 128 tokens
        _case("attention", "attn_window_128", seqs=8, new=4096, window=128, ragged=True),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "kv_append", "attention", "attention"])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 6, 8])
    dim = rng.choice([64, 64, 96, 128, 128, 128])
    c = _case(op, dtype=rng.choice(["bf16", "bf16", "fp16"]), heads=heads, kv_heads=kv_heads, dim=dim,
              rope=rng.choice([dim, dim, 64, 32]), interleaved=rng.random() < 0.3, norm=rng.random() < 0.7,
              page=rng.choice([16, 32, 48, 64, 128]), ragged=rng.random() < 0.6, with_q=rng.random() < 0.6,
              lse=rng.random() < 0.3)
    if op != "attention":
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


def _randn(shape, gen, dtype, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    x.normal_(0.0, scale, generator=gen)
    return x


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    new, total = _lens(c)
    T, Hq, Hk, D, P = sum(new), c["heads"], c["kv_heads"], c["dim"], c["page"]
    s = {"case": c, "T": T, "max_new": max(new), "max_total": max(total)}
    offs = torch.tensor([0] + new).cumsum(0)
    s["seq_offsets"] = offs.to(torch.int64).cuda()
    s["kv_len"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    # the layer's packed projection, q | k | v for each token
    s["qkv"] = _randn((T, (Hq + 2 * Hk) * D), gen, dt)
    s["w_q"] = 1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda") if c["norm"] else None
    s["w_k"] = 1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda") if c["norm"] else None
    if c["norm"]:
        s["w_q"], s["w_k"] = s["w_q"].to(dt), s["w_k"].to(dt)
    seq = torch.repeat_interleave(torch.arange(c["seqs"]), torch.tensor(new))
    pos = torch.arange(T) - offs[seq] + (torch.tensor(total) - torch.tensor(new))[seq]
    s["seq"], s["pos"] = seq.cuda(), pos.to(torch.int32).cuda()
    if c["op"] != "attention":
        half = c["rope"] // 2
        freq = THETA ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        angle = torch.arange(max(total), dtype=torch.float64, device="cuda")[:, None] * freq
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    if c["op"] != "qk_norm_rope":
        per = [-(-n // P) for n in total]
        n_pages = sum(per) + 3
        s["k_pages"] = _randn((n_pages, P, Hk, D), gen, dt)
        s["v_pages"] = _randn((n_pages, P, Hk, D), gen, dt)
        order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.zeros((c["seqs"], max(per)), dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(per):
            table[i, :n] = order[at:at + n]
            at += n
        s["block_table"] = table
    if c["op"] == "attention":  # normed and rotated already: heads of length about sqrt(D)
        s["q"] = s.pop("qkv")[:, : Hq * D].view(T, Hq, D)
    else:
        q, k, v = s["qkv"].split([Hq * D, Hk * D, Hk * D], 1)
        s["q"], s["k"], s["v"] = q.unflatten(1, (Hq, D)), k.unflatten(1, (Hk, D)), v.unflatten(1, (Hk, D))
    return s


# --------------------------------------------------------------------- run ----

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


def _plain_attention(s):
    c, q, P = s["case"], s["q"], s["case"]["page"]
    T, Hq, D = q.shape
    Hk, n, mn, mt = c["kv_heads"], c["seqs"], s["max_new"], s["max_total"]
    g = Hq // Hk
    offs, total = s["seq_offsets"], s["kv_len"].long()
    pages = s["block_table"].long()
    j = torch.arange(mt, device="cuda")
    there = (j[None, :] < total[:, None])[:, :, None, None]  # [n, keys, 1, 1]
    K = s["k_pages"][pages].flatten(1, 2)[:, :mt]
    V = s["v_pages"][pages].flatten(1, 2)[:, :mt]
    K = torch.where(there, K, 0).float().permute(0, 2, 3, 1)  # [n, Hk, D, keys]
    V = torch.where(there, V, 0).float().permute(0, 2, 1, 3)  # [n, Hk, keys, D]
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


def _plain(s):
    c = s["case"]
    if c["op"] == "attention":
        return _plain_attention(s)
    cs = s["table"][s["pos"].long()]
    dt = s["q"].dtype
    k = _norm_rope(s["k"].float(), s["w_k"], cs, c).to(dt)
    if c["op"] == "qk_norm_rope":
        return {"q": _norm_rope(s["q"].float(), s["w_q"], cs, c).to(dt), "k": k}
    pos = s["pos"].long()
    page, slot = s["block_table"][s["seq"], pos // c["page"]].long(), pos % c["page"]
    s["k_pages"][page, slot] = k
    s["v_pages"][page, slot] = s["v"]
    out = {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if c["with_q"]:
        out["q"] = _norm_rope(s["q"].float(), s["w_q"], cs, c).to(dt)
    return out


def _handles(s):
    """What a program makes once for a layer (cfg), its cache and its batch, and keeps from call to call."""
    import engram_gram_hash_gb300 as eg

    c = s["case"]
    s["cfg"] = eg.make_attn_config(c["heads"], c["kv_heads"], c["dim"], dtype=DTYPES[c["dtype"]], rope_dim=c["rope"],
                                   rope_interleaved=c["interleaved"], norm_eps=EPS, window=c["window"])
    if "k_pages" in s:
        s["cache"] = eg.kv_cache(s["k_pages"], s["v_pages"])
        s["batch"] = eg.kv_batch(s["seq_offsets"], s["kv_len"], s["block_table"], s["T"])


def _own(s):
    import engram_gram_hash_gb300 as eg

    c = s["case"]
    if "cfg" not in s:
        _handles(s)
    if c["op"] == "qk_norm_rope":
        q, k = eg.engram_qk_norm_rope(s["cfg"], s["q"], s["k"], s["pos"], s["table"], w_q=s["w_q"], w_k=s["w_k"])
        return {"q": q, "k": k}
    if c["op"] == "kv_append":
        if c["with_q"]:
            q = eg.engram_kv_append(s["cfg"], s["cache"], s["batch"], s["k"], s["v"], s["table"], w_k=s["w_k"],
                                    q=s["q"], w_q=s["w_q"])
            return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "q": q}
        eg.engram_kv_append(s["cfg"], s["cache"], s["batch"], s["k"], s["v"], s["table"], w_k=s["w_k"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if c["lse"]:
        lse = torch.empty((s["T"], c["heads"]), dtype=torch.float32, device="cuda")
        return {"out": eg.engram_paged_attention(s["cfg"], s["cache"], s["batch"], s["q"], lse=lse), "lse": lse}
    return {"out": eg.engram_paged_attention(s["cfg"], s["cache"], s["batch"], s["q"])}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work ----

def work(case):
    c = case
    new, total = _lens(c)
    T, Hq, Hk, D, e = sum(new), c["heads"], c["kv_heads"], c["dim"], 2
    if c["op"] == "attention":
        keys = pairs = 0
        for a, b in zip(new, total):
            w = c["window"] or b
            first = b - a  # position of the first new token
            keys += b - max(0, first - w + 1)
            # sum over positions p of min(p + 1, w)
            short = max(0, min(b, w) - first)  # positions that see all keys before them
            pairs += short * (2 * first + short + 1) // 2 + (a - short) * w
        return {"bytes": 2 * T * Hq * D * e + 2 * keys * Hk * D * e + (T * Hq * 4 if c["lse"] else 0),
                "flops": 4 * D * Hq * pairs}
    heads = Hk + (Hq if c["op"] == "qk_norm_rope" or c["with_q"] else 0)
    moved = 2 * T * heads * D * e + T * c["rope"] * 4
    if c["op"] == "kv_append":
        moved += 2 * T * Hk * D * e
    return {"bytes": moved, "flops": T * heads * (3 * c["rope"] + (4 * D if c["norm"] else 0))}


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
        k_all, v_all = (s[n][used].flatten(0, 1)[:b] for n in ("k_pages", "v_pages"))
        step = max(1, (1 << 27) // b)
        for h in range(Hq):
            k, v = k_all[:, h // g].double(), v_all[:, h // g].double()
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
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    k = _exact_rot(s["k"], s["w_k"], s["pos"], s["table"], case)
    q = _exact_rot(s["q"], s["w_q"], s["pos"], s["table"], case)
    if case["op"] == "qk_norm_rope":
        return {"q": q, "k": k}
    pages = {"k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double()}
    at = s["pos"].long()
    where = s["block_table"].long()[s["seq"], at // case["page"]] * case["page"] + at % case["page"]
    pages["k_pages"].flatten(0, 1)[where] = k
    pages["v_pages"].flatten(0, 1)[where] = s["v"].double()
    if case["with_q"]:
        pages["q"] = q
    return pages
