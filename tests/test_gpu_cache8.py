"""The serving step over the 8-bit cache (block tables, quantising append, attention over codes) against its plain
forms (needs a GB300)."""

import math
import random

import pytest
import torch

import cache8_plain as plain

pytestmark = pytest.mark.gpu

BF16, FP16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
ERANGE, ECAPACITY = 3, 4


@pytest.fixture(scope="module")
def eg():
    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without CUDA")
    import engram_gram_hash_gb300 as eg

    eg.lib()
    return eg


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# -------------------------------------------------------------------- plan ----

class Requests:
    """Requests with pages of their own, the rest of n_pages on the stack, in a shuffled order."""

    def __init__(self, old, keep, new, page, spare, seed=0, wide=3):
        rng = random.Random(seed)
        pages = lambda n: -(-n // page)  # noqa: E731
        had = [pages(o) for o in old]
        grow = sum(max(0, pages(k + n) - h) for k, n, h in zip(keep, new, had))
        self.n_pages = sum(had) + grow + spare
        ids = list(range(self.n_pages))
        rng.shuffle(ids)
        self.width = max([pages(k + n) for k, n in zip(keep, new)] + had + [1])
        self.table = []
        for h in had:
            self.table.append([ids.pop() for _ in range(h)] + [-9] * (self.width - h))
        self.n_free = len(ids)
        self.stack = ids + [-5] * (self.n_pages - len(ids))
        self.old, self.keep, self.new, self.page = old, keep, new, page
        # the table is a slice of a wider one whose other entries stay as they are
        self.whole = torch.full((len(old), self.width + wide), -3, dtype=torch.int32, device="cuda")
        self.whole[:, : self.width] = i32(self.table).view(len(old), self.width)
        self.t_table, self.t_stack = self.whole[:, : self.width], i32(self.stack)

    def call(self, eg, max_tokens=None, **kw):
        n = sum(self.new) if max_tokens is None else max_tokens
        return eg.engram_kv_plan(i32(self.new), i32(self.old), self.t_table, self.t_stack, i32([self.n_free]), self.page, n,
                                 keep_len=None if self.keep == self.old else i32(self.keep), **kw)

    def check(self, got, max_tokens):
        offs, after, table, stack, free, pos, slots, counts = plain.plan(self.old, self.keep, self.new, self.table,
                                                                        self.stack, self.n_free, self.page)
        tail = [-1] * (max_tokens - len(pos))
        assert got.seq_offsets.tolist() == offs and got.kv_len.tolist() == after
        assert self.t_table.tolist() == table and self.t_stack.tolist() == stack
        assert bool((self.whole[:, self.width:] == -3).all())
        assert got.n_free.tolist() == [free] and got.counts.tolist() == counts
        assert got.positions.tolist() == pos + tail and got.slots.tolist() == slots + tail


def _requests(n, page, most_old, most_new, seed):
    rng = random.Random(seed)
    old = [rng.choice([0, rng.randint(0, most_old), page * rng.randint(0, max(1, most_old // page))]) for _ in range(n)]
    keep = [rng.choice([o, o, 0, rng.randint(0, o)]) for o in old]
    new = [rng.choice([0, 1, 1, rng.randint(0, most_new)]) for _ in range(n)]
    return old, keep, new


@pytest.mark.parametrize("n,page,most_old,most_new,extra", [
    (1, 16, 40, 5, 0), (1, 64, 100, 300, 7), (3, 16, 64, 200, 1), (31, 48, 500, 9, 0), (32, 32, 100, 40, 0),
    (33, 16, 100, 40, 100), (257, 128, 700, 64, 3), (1023, 16, 90, 3, 0), (1024, 16, 90, 3, 0), (1025, 16, 90, 3, 5),
    (2500, 16, 60, 2, 0), (300, 16, 200, 100, 60), (2100, 32, 90, 21, 1000), (5, 16, 3000, 2000, 0),
])
def test_plan(eg, n, page, most_old, most_new, extra):
    old, keep, new = _requests(n, page, most_old, most_new, n + page)
    r = Requests(old, keep, new, page, spare=4, seed=n)
    T = sum(new) + extra
    got = r.call(eg, T)
    assert eg.engram_last_error() == 0
    r.check(got, T)


def test_plan_takes_the_last_page(eg):
    r = Requests([16, 32, 5], [16, 0, 5], [1, 0, 12], 16, spare=0)
    got = r.call(eg)
    assert eg.engram_last_error() == 0
    r.check(got, 13)


def test_plan_of_nothing(eg):
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    got = eg.engram_kv_plan(empty, empty, empty.view(0, 0), i32([4, 2, 9]), i32([3]), 16, 2)
    assert eg.engram_last_error() == 0
    assert got.seq_offsets.tolist() == [0] and got.n_free.tolist() == [3] and got.counts.tolist() == [0] * 4
    assert got.positions.tolist() == [-1, -1] and got.slots.tolist() == [-1, -1]


@pytest.mark.parametrize("n,extra", [(3, 0), (1500, 0), (3, 9000)])
@pytest.mark.parametrize("what", ["pages", "tokens", "keep", "negative", "width", "stack"])
def test_plan_all_or_nothing(eg, what, n, extra):
    old, new = [20 + s % 30 for s in range(n)], [1 + s % 20 + (16 if what == "pages" else 0) for s in range(n)]
    keep = [o - s % 3 for s, o in enumerate(old)]
    r = Requests(old, keep, new, 16, spare=2)
    T, missing, status = sum(new) + extra, 0, ERANGE
    if what == "pages":
        counts = plain.plan(old, keep, new, r.table, r.stack, r.n_free, 16)[-1]
        missing, status = 3, ECAPACITY
        missing = min(missing, counts[1] - counts[2])
        r.n_free = counts[1] - counts[2] - missing
    elif what == "tokens":
        T, status = sum(new) - 1, ECAPACITY
    elif what == "keep":
        r.keep = keep[:-1] + [old[-1] + 1]
    elif what == "negative":
        r.new = new[:-1] + [-1]
    elif what == "width":
        r.t_table = r.whole[:, : r.width - 1]
        if n == 3:
            r.new = new[:-1] + [16 * r.width]
    else:
        r.n_free = r.n_pages + 1
    table, stack = r.whole.clone(), r.t_stack.clone()
    got = r.call(eg, T)
    assert eg.engram_last_error() == status
    assert torch.equal(r.whole, table) and torch.equal(r.t_stack, stack)
    assert got.kv_len.tolist() == old and got.n_free.tolist() == [r.n_free] and got.seq_offsets.tolist() == [0] * (n + 1)
    assert got.counts.tolist() == [0, 0, 0, missing]
    assert bool((got.positions == -1).all()) and bool((got.slots == -1).all())


def test_plan_in_place_and_replayed(eg):
    """A captured plan that works on its own lengths and free pages: replays go on from the last one."""
    n, page, steps = 40, 16, 25
    r = Requests([3 * s for s in range(n)], [3 * s for s in range(n)], [1] * n, page, spare=n * 3)
    room = r.width + 3
    table = torch.full((n, room), -9, dtype=torch.int32, device="cuda")
    table[:, : r.width] = r.t_table
    kv, free, new = i32(r.old), i32([r.n_free]), i32(r.new)
    outs = dict(kv_len_out=kv, n_free_out=free)
    eg.engram_kv_plan(new, kv, table, r.t_stack, free, page, n, **outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = eg.engram_kv_plan(new, kv, table, r.t_stack, free, page, n, **outs)
    old, t, stack, n_free = r.old, [list(x) + [-9] * (room - r.width) for x in r.table], r.stack, r.n_free
    for step in range(steps + 1):
        offs, old, t, stack, n_free, pos, slots, _ = plain.plan(old, old, [1] * n, t, stack, n_free, page)
        if step:  # the first was the eager one
            g.replay()
        if step in (1, steps):
            assert kv.tolist() == old and free.tolist() == [n_free]
            assert table.tolist() == t and got.positions.tolist() == pos and got.slots.tolist() == slots
    assert eg.engram_last_error() == 0


def test_plan_parts_left_out_and_streams(eg):
    r = Requests([10, 50], [10, 40], [100, 7], 16, spare=1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    pos = torch.full((107,), 5, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    got = r.call(eg, positions=pos, stream=side)
    side.synchronize()
    assert got.positions is pos
    r.check(got, 107)


# ------------------------------------------------------------------- cache ----

class Cache:
    """An 8-bit cache and a step's batch over it: new[s] tokens of sequences that are total[s] long with them.  What no
    sequence uses holds NaN codes and NaN scales."""

    def __init__(self, eg, dtype, heads, kv_heads, dim, page, block, new, total, order="token", seed=0, spare=2, pow2=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.page, self.block = heads, kv_heads, dim, page, block
        self.dtype, self.new, self.total = dtype, list(new), list(total)
        n, T = len(new), sum(new)
        per = [-(-max(b, 0) // page) for b in total]
        n_pages = sum(per) + spare
        ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        self.block_table = torch.full((n, max(per + [1]) + 1), -7, dtype=torch.int32, device="cuda")

        def pages():
            shape = (n_pages, page, kv_heads, dim) if order == "token" else (n_pages, kv_heads, page, dim)
            x = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
            return x if order == "token" else x.transpose(1, 2)

        self.k_pages, self.v_pages = pages(), pages()
        shape = (n_pages, kv_heads, page // block)
        self.k_scales, self.v_scales = (torch.full(shape, math.nan, device="cuda") for _ in range(2))
        at = 0
        for s, c in enumerate(per):
            self.block_table[s, :c] = ids[at:at + c]
            at += c
            for i in range(c):
                used, p = min(page, total[s] - i * page), int(self.block_table[s, i])
                blocks = -(-used // block)
                for x, sc in ((self.k_pages, self.k_scales), (self.v_pages, self.v_scales)):
                    y = 100 * torch.randn((used, kv_heads, dim), generator=g, device="cuda")
                    x.view(torch.uint8)[p, :used] = y.clamp(-448, 448).to(E4M3).view(torch.uint8)
                    z = 0.005 + 0.01 * torch.rand((kv_heads, blocks), generator=g, device="cuda")
                    sc[p, :, :blocks] = torch.exp2(torch.round(torch.log2(z))) if pow2 else z
        self.seq_offsets = torch.tensor([0] + list(new)).cumsum(0).cuda()
        self.kv_len = i32(total)
        packed = torch.randn((T, (heads + 2 * kv_heads) * dim), generator=g, device="cuda").to(dtype)
        q, k, v = packed.split([heads * dim, kv_heads * dim, kv_heads * dim], 1)
        self.q, self.k, self.v = (q.unflatten(1, (heads, dim)), k.unflatten(1, (kv_heads, dim)),
                                  v.unflatten(1, (kv_heads, dim)))
        self.handles(eg)

    def handles(self, eg):
        self.cache = eg.kv_cache_q8(self.k_pages, self.v_pages, self.k_scales, self.v_scales)
        self.batch = eg.kv_batch(self.seq_offsets, self.kv_len, self.block_table, sum(self.new))


# ------------------------------------------------------------------ append ----

def positions_of(c):
    return torch.cat([torch.arange(b - a, b) for a, b in zip(c.new, c.total)]).int().cuda()


def check_append(eg, c, rope=None, interleaved=False, norm=True, with_q=True, table_rows=None):
    rope = c.dim if rope is None else rope
    cfg = eg.make_attn_config(c.heads, c.kv_heads, c.dim, dtype=c.dtype, rope_dim=rope, rope_interleaved=interleaved)
    table = eg.rope_table(max(c.total + [1]) if table_rows is None else table_rows, rope) if rope else None
    g = torch.Generator(device="cuda").manual_seed(3)
    w_q, w_k = ((1 + 0.1 * torch.randn(c.dim, generator=g, device="cuda")).to(c.dtype) if norm else None for _ in range(2))
    pos = positions_of(c)
    live = pos >= 0
    # what a 16-bit cache would hold: its codes must be the nearest ones
    q16, k16 = eg.engram_qk_norm_rope(cfg, c.q, c.k, pos.clamp(min=0), table, w_q=w_q, w_k=w_k)
    want = {}
    for name, x, pages, scales in (("k", k16, c.k_pages, c.k_scales), ("v", c.v, c.v_pages, c.v_scales)):
        codes, sc = pages.cpu().double(), scales.cpu().double()
        plain.append(x.cpu().double(), codes, sc, c.block_table.tolist(), c.new, c.total, c.block)
        want[name] = codes, sc
    out = eg.engram_kv_append_q8(cfg, c.cache, c.batch, c.k, c.v, table, w_k=w_k, q=c.q if with_q else None, w_q=w_q)
    assert eg.engram_last_error() == 0
    for name, pages, scales in (("k", c.k_pages, c.k_scales), ("v", c.v_pages, c.v_scales)):
        codes, sc = want[name]
        assert torch.equal(scales.cpu().double().nan_to_num(-1.0), sc.nan_to_num(-1.0)), name
        got = pages.cpu().double()
        assert torch.equal(got.isnan(), codes.isnan()), name
        assert torch.equal(got.nan_to_num(0.0), codes.nan_to_num(0.0)), name
    if with_q:
        assert torch.equal(out[live], q16[live])
    else:
        assert out is None


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("heads,kv_heads,dim,page,block,new,total", [
    (4, 2, 64, 16, 16, [1], [1]),
    (4, 1, 128, 16, 16, [1, 1, 1], [16, 17, 32]),
    (8, 8, 128, 64, 64, [1] * 5, [64, 65, 100, 128, 3]),
    (10, 5, 128, 64, 16, [100, 1, 0, 17], [100, 50, 9, 17]),
    (6, 3, 96, 48, 16, [333, 2, 48], [400, 48, 96]),
    (2, 1, 16, 32, 32, [70, 31], [71, 64]),
    (12, 6, 80, 128, 128, [300, 129, 1], [301, 258, 128]),
    (9, 9, 48, 128, 64, [65, 64, 63], [130, 65, 63]),
    (2, 2, 112, 256, 128, [5, 250], [5, 500]),
])
def test_append(eg, dtype, heads, kv_heads, dim, page, block, new, total):
    c = Cache(eg, dtype, heads, kv_heads, dim, page, block, new, total, seed=dim + page)
    check_append(eg, c)


@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("rope,interleaved,norm", [(0, False, True), (64, False, True), (32, True, False), (96, True, True),
                                                   (16, False, False)])
def test_append_rotations_and_orders(eg, rope, interleaved, norm, order):
    c = Cache(eg, BF16, 6, 3, 96, 48, 48 // 3, [100, 7], [130, 90], order=order, pow2=True)
    check_append(eg, c, rope=rope, interleaved=interleaved, norm=norm, with_q=order == "token")


@pytest.mark.parametrize("n", [33, 70])
def test_append_many_sequences(eg, n):
    new = [s % 5 for s in range(n)]
    c = Cache(eg, BF16, 4, 2, 64, 32, 32, new, [a + 3 * s for s, a in enumerate(new)])
    check_append(eg, c)


def test_append_padding_and_growth(eg):
    """Tokens before a sequence's start are left out; a block that begins small and grows is rounded again."""
    c = Cache(eg, BF16, 4, 2, 64, 32, 32, [5, 1, 40], [3, 0, 50], pow2=True)
    check_append(eg, c)
    c = Cache(eg, FP16, 2, 2, 128, 64, 64, [1, 1, 1], [10, 64, 63])
    for sc in (c.k_scales, c.v_scales):
        sc.copy_(torch.where(sc.isnan(), sc, torch.tensor([0.0, 2.0**-20, 0.37], device="cuda")[torch.randint(3, sc.shape, device="cuda")]))
    check_append(eg, c)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_append_extremes(eg, dtype):
    """Zeros, infinities, NaN, values at the scale's borders, beyond its range and below the codes' steps."""
    c = Cache(eg, dtype, 2, 2, 64, 64, 16, [64 + 40], [64 + 40])
    v = c.v
    v.zero_()
    big = 3.0e38 if dtype == BF16 else 65504.0
    v[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 1.0])
    v[16, 0, 0] = math.inf
    v[32, 0, 0], v[33, 0, 1] = big, -1.0
    for i, x in enumerate([448.0, 449.0, 447.0, 450.0, 1.75, 1.76, 0.875, 2.0**-14, 2.0**-24]):
        v[48 + i, 0, i], v[48 + i, 0, 32 + i] = x, -x
    v[64:80, 0] = torch.linspace(-1.75, 1.75, 16 * 64, device="cuda").view(16, 64)
    v[80:96, 1] = 2.0**-24
    v[96:104, 1, 0] = 3.0
    check_append(eg, c, norm=False, rope=0)


def test_append_steps_and_sharing(eg):
    """Token by token a block's codes stay within half a code's step of the values at the final scale (once for each
    rounding); ranges outside the new tokens stay bit for bit."""
    T, block = 64, 64
    c = Cache(eg, BF16, 2, 1, 64, 64, block, [1], [1], spare=1)
    cfg = eg.make_attn_config(2, 1, 64, rope_dim=0)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, 1, 64), generator=g, device="cuda") * torch.exp2(torch.arange(T, device="cuda") // 6).view(T, 1, 1)
    x = x.to(BF16)
    for t in range(T):
        c.kv_len.fill_(t + 1)
        eg.engram_kv_append_q8(cfg, c.cache, c.batch, x[t:t + 1], x[t:t + 1], None)
    assert eg.engram_last_error() == 0
    page = int(c.block_table[0, 0])
    scale = float(c.k_scales[page, 0, 0])
    got = c.k_pages[page, :, 0].double() * scale
    # powers of two: only steps below the normal range move, each rounding by half a step of 2^-9 of the scale
    most = 2.0**-4 * x[:, 0].double().abs() + 12 * 2.0**-10 * scale
    assert bool(((got - x[:, 0].double()).abs() <= most).all())
    assert torch.equal(c.k_pages.view(torch.uint8)[page], c.v_pages.view(torch.uint8)[page])


def test_append_out_of_range(eg):
    c = Cache(eg, BF16, 4, 2, 64, 32, 32, [3, 3], [40, 3])
    cfg = eg.make_attn_config(4, 2, 64)
    table = eg.rope_table(39, 64)
    before = [t.clone() for t in (c.k_pages.view(torch.uint8), c.k_scales)]
    eg.engram_kv_append_q8(cfg, c.cache, c.batch, c.k, c.v, table)  # position 39 has no angles
    assert eg.engram_last_error() == ERANGE
    page, other = int(c.block_table[0, 1]), int(c.block_table[1, 0])
    now = c.k_pages.view(torch.uint8)
    assert not torch.equal(now[page, 5:7], before[0][page, 5:7]) and torch.equal(now[page, 7:], before[0][page, 7:])
    assert not torch.equal(now[other, :3], before[0][other, :3])
    for bad in (-1, c.k_pages.shape[0]):  # a page that is not there: nothing of that block is written
        c.block_table[0, 1] = bad
        now = c.k_pages.view(torch.uint8).clone()
        eg.engram_kv_append_q8(cfg, c.cache, c.batch, c.k, c.v, eg.rope_table(40, 64))
        assert eg.engram_last_error() == ERANGE
        now[other] = c.k_pages.view(torch.uint8)[other]
        assert torch.equal(now, c.k_pages.view(torch.uint8))
    c.kv_len[0] = 32 * c.block_table.shape[1] + 2  # past the table
    eg.engram_kv_append_q8(cfg, c.cache, c.batch, c.k, c.v, eg.rope_table(400, 64))
    assert eg.engram_last_error() == ERANGE


# --------------------------------------------------------------- attention ----

def check_attention(eg, c, window=0, scale=None):
    cfg = eg.make_attn_config(c.heads, c.kv_heads, c.dim, dtype=c.dtype, rope_dim=0, window=window, scale=scale)
    T = sum(c.new)
    lse = torch.full((T, c.heads), 7.0, device="cuda")
    out = torch.full((T, c.heads, c.dim), 7.0, dtype=c.dtype, device="cuda")
    got = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q, out=out, lse=lse)
    assert got is out and eg.engram_last_error() == 0
    ref, ref_lse, bound, lse_bound = plain.attention(c.q, c.k_pages, c.v_pages, c.k_scales, c.v_scales, c.block_table,
                                                     c.new, c.total, c.kv_heads, cfg.scale, window)
    assert torch.isfinite(got).all()
    off = (got.double() - ref).abs() - bound
    assert bool((off <= 0).all()), float(off.max())
    empty = ref_lse == -math.inf
    assert torch.equal(lse == -math.inf, empty) and bool((got[empty] == 0).all())
    off = (lse.double() - ref_lse).abs()[~empty] - lse_bound[~empty]
    assert bool((off <= 0).all())
    return got


DECODE = [
    ([1], [1]), ([1], [16]), ([1], [17]), ([1], [128]), ([1], [129]), ([1], [5000]),
    ([1, 1, 1], [1, 700, 130]), ([1] * 40, [37 * s + 1 for s in range(40)]), ([1, 0, 1, 1], [600, 40, 0, 3]),
    ([2, 3, 1, 5], [300, 3, 1000, 7]),
]


@pytest.mark.parametrize("new,total", DECODE)
@pytest.mark.parametrize("dtype,heads,kv_heads,dim,page,block", [
    (BF16, 8, 2, 128, 64, 64), (FP16, 4, 4, 64, 16, 16), (BF16, 12, 2, 96, 48, 16), (FP16, 8, 1, 128, 128, 128),
    (BF16, 3, 1, 16, 32, 32), (FP16, 10, 2, 80, 256, 64),
])
def test_attention_few_rows(eg, dtype, heads, kv_heads, dim, page, block, new, total):
    check_attention(eg, Cache(eg, dtype, heads, kv_heads, dim, page, block, new, total, seed=dim))


PROMPTS = [
    ([256], [256]), ([300], [1300]), ([64, 129, 1, 400], [64, 500, 2000, 401]), ([1000], [1000]),
    ([33] * 34, [33 + 20 * s for s in range(34)]), ([200, 5, 0, 90], [150, 3, 10, 91]),
]


@pytest.mark.parametrize("new,total", PROMPTS)
@pytest.mark.parametrize("dtype,heads,kv_heads,dim,page,block", [
    (BF16, 8, 2, 128, 64, 64), (FP16, 6, 2, 64, 16, 16), (BF16, 12, 2, 96, 48, 16), (FP16, 4, 1, 128, 128, 128),
    (BF16, 4, 2, 48, 32, 16),
])
def test_attention_prompts(eg, dtype, heads, kv_heads, dim, page, block, new, total):
    check_attention(eg, Cache(eg, dtype, heads, kv_heads, dim, page, block, new, total, seed=dim + 1))


@pytest.mark.parametrize("window", [1, 16, 100, 1 << 30])
@pytest.mark.parametrize("new,total", [([1, 1, 1], [700, 30, 128]), ([300, 129], [900, 129])])
@pytest.mark.parametrize("dim,page,block", [(128, 64, 16), (64, 48, 16), (128, 128, 128)])
def test_attention_window(eg, dim, page, block, new, total, window):
    check_attention(eg, Cache(eg, BF16, 8, 2, dim, page, block, new, total), window=window)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("new,total", [([1, 1], [700, 30]), ([280, 40], [700, 90])])
def test_attention_scales_far_apart(eg, dtype, new, total):
    """Value scales from 2^-40 to 2^10, zero blocks with scale 0, key scales of 0: rows whose weight lies on small
    values keep their bits (the bound's last term is absolute, so such rows are checked on their own)."""
    c = Cache(eg, dtype, 4, 2, 64, 16, 16, new, total)
    g = torch.Generator(device="cuda").manual_seed(5)
    e = torch.randint(-24, 5, c.v_scales.shape, generator=g, device="cuda").float()
    c.v_scales.copy_(torch.where(c.v_scales.isnan(), c.v_scales, torch.exp2(e)))
    check_attention(eg, c)
    zero = torch.rand(c.v_scales.shape, generator=g, device="cuda") < 0.3
    pages, _, heads, _ = c.v_pages.shape
    hit = zero[:, :, 0] & ~c.v_scales[:, :, 0].isnan()
    for p, h in hit.nonzero().tolist():
        used = ~c.v_pages[p, :, h, 0].float().isnan()
        c.v_pages.view(torch.uint8)[p, used, h] = 0
    c.v_scales[hit] = 0.0
    k0 = torch.rand(hit.shape, generator=g, device="cuda") < 0.2
    c.k_scales[k0 & ~c.k_scales[:, :, 0].isnan()] = 0.0
    check_attention(eg, c)


def test_attention_follows_small_values(eg):
    """All of a row's weight on a block whose values are 2^-30 of another block's: the result keeps its relative
    precision."""
    for new in (1, 300):
        c = Cache(eg, BF16, 2, 1, 64, 16, 16, [new], [new + 64], seed=2)
        used = c.block_table[0].tolist()
        for i, p in enumerate(used[: -(-(new + 64) // 16)]):
            c.k_scales[p] = 0.01
            c.v_scales[p] = 2.0**-30 if i == 1 else 1.0
        c.k_pages.view(torch.uint8)[used[1]] = torch.full((16, 1, 64), 240.0, device="cuda").to(E4M3).view(torch.uint8)
        c.q.fill_(20.0)  # far above the others at block 1
        cfg = eg.make_attn_config(2, 1, 64, rope_dim=0)
        got = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q).double()
        ref = plain.attention(c.q, c.k_pages, c.v_pages, c.k_scales, c.v_scales, c.block_table, c.new, c.total, 1, cfg.scale, 0)[0]
        v = plain.values(c.v_pages, c.v_scales, c.block_table, 0, 32, 0, 16)[0][16:].abs().amax()
        assert bool(((got - ref).abs() <= 2.0**-8 * ref.abs() + 2.0**-9 * v).all())


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("new,total", [([1, 1, 1], [300, 40, 1]), ([260, 30], [500, 300])])
def test_attention_query_ranges(eg, dtype, new, total):
    """Rows of zeros, of the type's largest and smallest values."""
    c = Cache(eg, dtype, 4, 2, 128, 64, 32, new, total)
    c.q[0, 0] = 0.0
    c.q[0, 1] = 2.0**-24
    c.q[1, 0] = c.q[1, 0].sign() * (2.0**60 if dtype == BF16 else 60000.0)
    c.q[1, 1] *= 2.0**-60 if dtype == BF16 else 2.0**-14
    c.k_scales[c.k_scales > 0] *= 1e-4
    big = check_attention  # the row of large queries: scores of 1e15, one key takes everything
    if dtype == FP16:
        big(eg, c)
        return
    c.q[1, 0] = c.q[1, 0].sign() * 2.0**20
    big(eg, c)


@pytest.mark.parametrize("new,total", [([1], [200]), ([5], [200]), ([200], [300]), ([40, 300], [40, 600])])
@pytest.mark.parametrize("dim,block", [(128, 64), (64, 16)])
def test_attention_nan_codes(eg, new, total, dim, block):
    """A NaN code of a key reaches the queries that see its position, of a value their result's column alone."""
    for which in ("k", "v"):
        c = Cache(eg, BF16, 4, 2, dim, 64, block, new, total, seed=9)
        s = len(new) - 1
        pos = total[s] - max(1, new[s] // 2)
        page = int(c.block_table[s, pos // 64])
        cfg = eg.make_attn_config(4, 2, dim, rope_dim=0)
        clean = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
        pages = c.k_pages if which == "k" else c.v_pages
        pages.view(torch.uint8)[page, pos % 64, 1, 5] = 0xFF
        got = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
        assert eg.engram_last_error() == 0
        first = sum(new[:s]) + pos - (total[s] - new[s])
        want = torch.zeros_like(got, dtype=torch.bool)
        if which == "k":
            want[first:sum(new[:s + 1]), 2:] = True
        else:
            want[first:sum(new[:s + 1]), 2:, 5] = True
        assert torch.equal(got.isnan(), want)
        assert torch.equal(got[~want], clean[~want])


def test_attention_bad_pages(eg):
    c = Cache(eg, BF16, 8, 2, 128, 64, 64, [1, 100], [300, 250])
    c.block_table[0, 2] = c.k_pages.shape[0]
    c.block_table[1, 0] = -1
    cfg = eg.make_attn_config(8, 2, 128, rope_dim=0)
    out = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    assert eg.engram_last_error() == ERANGE and bool(torch.isfinite(out).all())
    c.kv_len[0] = 64 * c.block_table.shape[1] + 1
    eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    assert eg.engram_last_error() == ERANGE


@pytest.mark.parametrize("new,total", [([1] * 7, [2000 * s + 5 for s in range(7)]), ([300, 700], [2300, 700])])
def test_attention_repeats_and_graphs(eg, new, total):
    """Equal bits from call to call, from a captured graph, on another stream and with a given workspace."""
    c = Cache(eg, BF16, 8, 2, 128, 64, 64, new, total)
    cfg = eg.make_attn_config(8, 2, 128, rope_dim=0)
    first = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    need = eg.engram_paged_attention_q8_workspace_bytes(cfg, c.cache, c.batch)
    ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q, workspace=ws), first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
        b = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    for _ in range(3):
        a.fill_(0)
        b.fill_(0)
        g.replay()
        assert torch.equal(a, first) and torch.equal(b, first)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q, stream=x) for x in (side, None, side)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, first) for x in got) and eg.engram_last_error() == 0


# ---------------------------------------------------------------- together ----

@pytest.mark.parametrize("dtype,page,block,dim", [(BF16, 16, 16, 64), (FP16, 64, 32, 128)])
def test_serving_run(eg, dtype, page, block, dim):
    """Requests that start, decode, drop drafts and end, by plan, append and attention alone, the lengths never leaving
    the GPU; every step's results against the plain attention over what the cache holds."""
    heads, kv_heads, n, rng = 4, 2, 6, random.Random(4)
    n_pages, width = 60, 1 + 600 // page
    pages = [torch.full((n_pages, page, kv_heads, dim), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    scales = [torch.full((n_pages, kv_heads, page // block), math.nan, device="cuda") for _ in range(2)]
    cache = eg.kv_cache_q8(*pages, *scales)
    cfg = eg.make_attn_config(heads, kv_heads, dim, dtype=dtype)
    angles = eg.rope_table(600, dim)
    kv, table = i32([0] * n), torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    stack, free = torch.arange(n_pages, dtype=torch.int32, device="cuda"), i32([n_pages])
    old = [0] * n
    g = torch.Generator(device="cuda").manual_seed(8)
    for step in range(8):
        keep = [rng.choice([o, o, max(0, o - 3), 0 if step > 3 else o]) for o in old]
        new = [rng.randint(1, 100) if k == 0 else rng.choice([0, 1, 1, 4]) for k in keep]
        T = sum(new)
        if T == 0:
            continue
        p = eg.engram_kv_plan(i32(new), kv, table, stack, free, page, T, keep_len=i32(keep), kv_len_out=kv, n_free_out=free)
        batch = eg.kv_batch(p.seq_offsets, p.kv_len, table, T)
        x = [torch.randn((T, h, dim), generator=g, device="cuda").to(dtype) for h in (heads, kv_heads, kv_heads)]
        q = eg.engram_kv_append_q8(cfg, cache, batch, x[1], x[2], angles, q=x[0])
        lse = torch.empty((T, heads), device="cuda")
        out = eg.engram_paged_attention_q8(cfg, cache, batch, q, lse=lse)
        assert eg.engram_last_error() == 0
        old = [k + m for k, m in zip(keep, new)]
        assert kv.tolist() == old and int(free) == n_pages - sum(-(-o // page) for o in old)
        used = [table[s, : -(-o // page)].tolist() for s, o in enumerate(old)]
        flat = sum(used, []) + stack[: int(free)].tolist()
        assert sorted(flat) == list(range(n_pages))  # every page has one place
        ref, ref_lse, bound, lse_bound = plain.attention(q, *pages, *scales, table, new, old, kv_heads, cfg.scale, 0)
        assert bool(((out.double() - ref).abs() <= bound).all()) and bool(((lse.double() - ref_lse).abs() <= lse_bound).all())
        # the slots name the rows that were written: v's codes there are v's nearest at their blocks' scales
        page_of, slot = p.slots // page, p.slots % page
        sc = scales[1][page_of, :, slot // block].double()
        got = pages[1].view(torch.uint8)[page_of, slot].view(E4M3).cpu().double()
        assert torch.equal(got, plain.nearest_codes((x[2].double() / sc[..., None]).cpu()))
