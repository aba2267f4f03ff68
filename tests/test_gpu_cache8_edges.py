"""The 8-bit cache's calls at their far ends: longest sequences, pages past 4 GB, unaligned outputs, one captured step, other
GPUs' tensors (needs a GB300)."""

import pytest
import torch

import cache8_plain as plain
from attention_far import Far
from test_gpu_cache8 import BF16, E4M3, FP16, Cache, check_attention, eg, i32  # noqa: F401

pytestmark = pytest.mark.gpu

PAGE, LONGEST = 65536, (1 << 31) - 1024


def codes(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (100 * torch.randn(shape, generator=g, device="cuda")).clamp(-448, 448).to(E4M3)


@pytest.mark.parametrize("heads", [4, 128])  # few rows, tiles
@pytest.mark.parametrize("dim,block", [(16, 16), (80, 128)])
def test_longest_sequences(eg, heads, dim, block):  # noqa: F811
    """One page of 65,536 tokens stands in every entry of the table, and a window keeps the work small."""
    new, window = 10, 64
    k, v = codes((1, PAGE, 1, dim), dim), codes((1, PAGE, 1, dim), dim + 1)
    ks, vs = (0.005 + 0.01 * torch.rand((1, 1, PAGE // block), device="cuda") for _ in range(2))
    q = torch.randn((new, heads, dim), device="cuda").to(BF16)
    cfg = eg.make_attn_config(heads, 1, dim, rope_dim=0, window=window)
    cache, offs = eg.kv_cache_q8(k, v, ks, vs), torch.tensor([0, new], device="cuda")
    table = torch.zeros((1, (LONGEST + 1024) // PAGE), dtype=torch.int32, device="cuda")

    def run(length):
        batch = eg.kv_batch(offs, i32([length]), table, new)
        return eg.engram_paged_attention_q8(cfg, cache, batch, q)

    ref, _, bound, _ = plain.attention(q, k, v, ks, vs, table[:, :2], [new], [PAGE + LONGEST % PAGE], 1, cfg.scale, window)
    got = run(LONGEST)
    assert eg.engram_last_error() == 0
    assert ((got.double() - ref).abs() <= bound).all()
    assert torch.equal(run(PAGE + LONGEST % PAGE), got)
    for length in (LONGEST + 1, LONGEST + 1023):  # flagged and cut
        cut = run(length)
        assert eg.engram_last_error() == 3
        assert torch.equal(cut, got)


def test_longest_append_and_plan(eg):  # noqa: F811
    block = 16
    k, v = codes((2, PAGE, 1, 16), 1), codes((2, PAGE, 1, 16), 2)
    ks, vs = (torch.ones((2, 1, PAGE // block), device="cuda") for _ in range(2))
    table = torch.zeros((1, (LONGEST + 1024) // PAGE), dtype=torch.int32, device="cuda")
    table[0, (LONGEST - 1) // PAGE] = 1
    cfg = eg.make_attn_config(1, 1, 16, rope_dim=0)
    x = torch.randn((5, 1, 16), device="cuda").to(BF16)
    before = k.view(torch.uint8).clone()
    eg.engram_kv_append_q8(cfg, eg.kv_cache_q8(k, v, ks, vs), eg.kv_batch(torch.tensor([0, 5], device="cuda"), i32([LONGEST]), table, 5), x, x, None)
    assert eg.engram_last_error() == 0
    at = (LONGEST - 5) % PAGE
    now = k.view(torch.uint8)
    assert torch.equal(now[0], before[0]) and torch.equal(now[1, :at - at % block], before[1, :at - at % block])
    sc = ks[1, 0, at // block]
    want = plain.nearest_codes((x.double() / sc.double()).cpu())
    assert torch.equal(k[1, at:at + 5].cpu().double(), want)
    # a plan of the same length: the last page is there already, one token more has none
    p = eg.engram_kv_plan(i32([3]), i32([LONGEST - 3]), table, i32([7]), i32([1]), PAGE, 3)
    assert eg.engram_last_error() == 0 and p.kv_len.tolist() == [LONGEST] and p.n_free.tolist() == [1]
    assert p.slots.tolist() == [PAGE + (LONGEST - 3 + i) % PAGE for i in range(3)]
    p = eg.engram_kv_plan(i32([4]), i32([LONGEST - 3]), table, i32([7]), i32([1]), PAGE, 4)
    assert eg.engram_last_error() == 3 and p.kv_len.tolist() == [LONGEST - 3]


@pytest.mark.parametrize("new", [1, 200])
def test_pages_past_4_gb(eg, new):  # noqa: F811
    """A cache of 6 GB a tensor whose sequence lies in its last pages, at both ends of 32 bits' reach."""
    heads, kv, dim, page, block, n_pages = 8, 8, 128, 64, 64, 92000
    small = Cache(eg, BF16, heads, kv, dim, page, block, [new], [new + 150], seed=4)
    big = []
    for x in (small.k_pages, small.v_pages):
        y = torch.empty((n_pages, page, kv, dim), dtype=torch.uint8, device="cuda")
        big.append(y)
    scales = [torch.full((n_pages, kv, 1), float("nan"), device="cuda") for _ in range(2)]
    used = small.block_table[0, : -(-(new + 150) // page)].tolist()
    table = small.block_table.clone()
    for i, p in enumerate(used):
        at = n_pages - 1 - i if i % 2 else 32768 + i
        table[0, i] = at
        for y, x, sc, s in zip(big, (small.k_pages, small.v_pages), scales, (small.k_scales, small.v_scales)):
            y[at] = x.view(torch.uint8)[p]
            sc[at] = s[p]
    cfg = eg.make_attn_config(heads, kv, dim, rope_dim=0)
    want = eg.engram_paged_attention_q8(cfg, small.cache, small.batch, small.q)
    cache = eg.kv_cache_q8(*[y.view(E4M3) for y in big], *scales)
    batch = eg.kv_batch(small.seq_offsets, small.kv_len, table, new)
    assert torch.equal(eg.engram_paged_attention_q8(cfg, cache, batch, small.q), want)
    eg.engram_kv_append_q8(cfg, small.cache, small.batch, small.k, small.v, None)
    eg.engram_kv_append_q8(cfg, cache, batch, small.k, small.v, None)
    assert eg.engram_last_error() == 0
    for i, p in enumerate(used):
        n = min(page, new + 150 - i * page)
        for y, x in zip(big, (small.k_pages, small.v_pages)):
            assert torch.equal(y[table[0, i].long(), :n], x.view(torch.uint8)[p, :n])


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("new,total", [([1, 1], [90, 3]), ([300, 20], [400, 20])])
def test_strided_heads(eg, dtype, new, total):  # noqa: F811
    """Queries and outputs as slices of wider rows, on 16-byte boundaries that are no 32-byte ones; what lies between stays."""
    c = Cache(eg, dtype, 6, 2, 96, 48, 16, new, total)
    cfg = eg.make_attn_config(6, 2, 96, dtype=dtype, rope_dim=0)
    want = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    T = sum(new)
    wide = torch.full((T, 7, 104), 5.0, dtype=dtype, device="cuda")
    out = wide[:, :6, 8:]
    got = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q.clone(), out=out)
    assert got is out and torch.equal(out, want)
    assert bool((wide[:, 6] == 5).all()) and bool((wide[:, :, :8] == 5).all())


def test_one_captured_step(eg):  # noqa: F811
    """Plan, append and attention of a decode step in one graph, its lengths and free pages in place: replays equal the
    eager steps bit for bit."""
    n, page, block, dim, heads, kv_heads, steps = 5, 16, 16, 64, 4, 2, 20

    def start():
        g = torch.Generator(device="cuda").manual_seed(6)
        s = dict(kv=i32([10 * i for i in range(n)]), free=i32([40]), stack=torch.arange(64, dtype=torch.int32, device="cuda"))
        s["table"] = torch.full((n, 8), -1, dtype=torch.int32, device="cuda")
        at = 40
        for i in range(n):
            for e in range(-(-10 * i // page)):
                s["table"][i, e] = at
                at += 1
        s["pages"] = [codes((64, page, kv_heads, dim), j) for j in (1, 2)]
        s["scales"] = [torch.full((64, kv_heads, 1), 0.0078125, device="cuda") for _ in range(2)]
        s["x"] = [torch.randn((n, h, dim), generator=g, device="cuda").to(BF16) for h in (heads, kv_heads, kv_heads)]
        return s

    cfg, angles, new = eg.make_attn_config(heads, kv_heads, dim), eg.rope_table(200, dim), i32([1] * n)

    def step(s):
        p = eg.engram_kv_plan(new, s["kv"], s["table"], s["stack"], s["free"], page, n, kv_len_out=s["kv"], n_free_out=s["free"])
        cache = eg.kv_cache_q8(*s["pages"], *s["scales"])
        batch = eg.kv_batch(p.seq_offsets, s["kv"], s["table"], n)
        q = eg.engram_kv_append_q8(cfg, cache, batch, s["x"][1], s["x"][2], angles, q=s["x"][0])
        return eg.engram_paged_attention_q8(cfg, cache, batch, q)

    eager, s = [], start()
    for _ in range(steps):
        eager.append(step(s).clone())
    assert eg.engram_last_error() == 0
    s = start()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step(s).clone()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, eager[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(s)
    for i in range(1, steps):
        g.replay()
        assert torch.equal(out, eager[i]), i
    assert eg.engram_last_error() == 0


def test_calls_on_two_streams_at_once(eg):  # noqa: F811
    """Different batches over one cache on two streams, with their own workspaces."""
    a = Cache(eg, BF16, 8, 2, 128, 64, 64, [1] * 30, [40 * s + 1 for s in range(30)], seed=1)
    b = Cache(eg, BF16, 8, 2, 128, 64, 64, [300, 200], [1300, 200], seed=2)
    cfg = eg.make_attn_config(8, 2, 128, rope_dim=0)
    want = [eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q) for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, c in enumerate((a, b)):
            got[i].append(eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q, stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])


def test_other_devices_are_refused(eg):  # noqa: F811
    c = Cache(eg, BF16, 8, 2, 128, 16, 16, [1, 1], [30, 20])
    cfg, table, w = eg.make_attn_config(8, 2, 128), eg.rope_table(64, 128), torch.ones(128, device="cuda", dtype=BF16)
    out, lse = torch.empty((2, 8, 128), dtype=BF16, device="cuda"), torch.empty((2, 8), device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    calls = {
        "append": (eg.engram_kv_append_q8, (cfg, c.cache, c.batch), dict(k=c.k, v=c.v, table=table, w_k=w, q=c.q, w_q=w, q_out=out)),
        "attention": (eg.engram_paged_attention_q8, (cfg, c.cache, c.batch), dict(q=c.q, out=out, lse=lse, workspace=ws)),
    }
    for name, (call, first, args) in calls.items():
        call(*first, **args)
        for far in args:
            with pytest.raises(ValueError, match="cuda:1"):
                call(*first, **{**args, far: Far(args[far])})
                pytest.fail(f"{name}: {far} was accepted")
    assert eg.engram_last_error() == 0


def test_prompt_and_decode_agree(eg):  # noqa: F811
    """The same cache through both kernels: each row within its bound (checked) whatever batch it comes in."""
    c = Cache(eg, FP16, 8, 2, 64, 64, 32, [500], [900])
    whole = check_attention(eg, c)
    cfg = eg.make_attn_config(8, 2, 64, dtype=FP16, rope_dim=0)
    for t in (0, 250, 499):
        batch = eg.kv_batch(torch.tensor([0, 1], device="cuda"), i32([401 + t]), c.block_table, 1)
        one = eg.engram_paged_attention_q8(cfg, c.cache, batch, c.q[t:t + 1].clone())
        _, _, bound, _ = plain.attention(c.q[t:t + 1], c.k_pages, c.v_pages, c.k_scales, c.v_scales, c.block_table, [1], [401 + t], 2,
                                         cfg.scale, 0)
        assert bool(((one.double() - whole[t:t + 1].double()).abs() <= 2 * bound).all())


def test_plan_arguments(eg):  # noqa: F811
    """Other GPUs' tensors, wrong sizes and types of every tensor of a plan."""
    i64 = lambda n: torch.zeros(n, dtype=torch.int64, device="cuda")  # noqa: E731
    good = dict(new_len=i32([1, 2]), kv_len=i32([3, 4]), block_table=torch.zeros((2, 3), dtype=torch.int32, device="cuda"),
                n_free=i32([3]), keep_len=i32([3, 4]), kv_len_out=i32([0, 0]), n_free_out=i32([0]), seq_offsets=i64(3),
                positions=i32([0, 0, 0]), slots=i64(3), counts=i32([0] * 4))
    wrong = dict(new_len=i32([1]), kv_len=i32([1]), block_table=torch.zeros((3, 3), dtype=torch.int32, device="cuda"),
                 n_free=i32([1, 2]), keep_len=i32([1]), kv_len_out=i32([1]), n_free_out=i32([1, 2]), seq_offsets=i64(2),
                 positions=i32([1, 2]), slots=i64(4), counts=i32([1, 2, 3]))
    more = dict(free_pages=i32([1, 2, 3]), page_size=16, max_tokens=3)
    eg.engram_kv_plan(**good, **more)
    assert eg.engram_last_error() == 0
    for n, t in good.items():
        with pytest.raises(ValueError, match="cuda:1"):
            eg.engram_kv_plan(**{**good, n: Far(t)}, **more)
        with pytest.raises(ValueError):
            eg.engram_kv_plan(**{**good, n: wrong[n]}, **more)
        with pytest.raises(TypeError):
            eg.engram_kv_plan(**{**good, n: t.double()}, **more)
        with pytest.raises(ValueError):
            eg.engram_kv_plan(**{**good, n: t.cpu()}, **more)
    for page_size in (8, 24, 65552):
        with pytest.raises(eg.EngramError):
            eg.engram_kv_plan(**good, **{**more, "page_size": page_size})
    with pytest.raises(ValueError, match="contiguous rows"):
        eg.engram_kv_plan(**{**good, "block_table": torch.zeros((3, 2), dtype=torch.int32, device="cuda").T}, **more)
    assert eg.engram_last_error() == 0
