"""Attention over the 8-bit cache by each of its forms, every case with the kernels that it is meant for: few rows (whole or
cut and joined), tiles converted where they are met (whole or split and joined), tiles opened beforehand.  The edges are those
of the other tests of the cache, on shapes that the choice gives to the form; bounds and plain forms as there (needs a GB300)."""

import ctypes
import re

import pytest
import torch

import cache8_plain as plain
from test_gpu_cache8 import BF16, E4M3, ERANGE, FP16, Cache, check_attention, eg, i32  # noqa: F401
from test_gpu_cache8_edges import LONGEST, PAGE, codes

pytestmark = pytest.mark.gpu

ROWS, CUT = {"rows8_kernel"}, {"rows8_kernel", "rows_join_kernel"}
TILES, SPLIT = {"tile8_kernel"}, {"tile8_kernel", "tile_join_kernel"}
OPENED, OPENED_SPLIT = TILES | {"open_kernel"}, SPLIT | {"open_kernel"}


def config(eg, c, window=0):  # noqa: F811
    return eg.make_attn_config(c.heads, c.kv_heads, c.dim, dtype=c.dtype, rope_dim=0, window=window)


def kernels(eg, cfg, cache, batch, q, tmp_path):  # noqa: F811
    """The attention kernels that a call launches, from its CUDA graph."""
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    n = eg.engram_paged_attention_q8_workspace_bytes(cfg, cache, batch)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    eg.engram_paged_attention_q8(cfg, cache, batch, q, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        eg.engram_paged_attention_q8(cfg, cache, batch, q, out=out, workspace=ws)
    dot = str(tmp_path / "graph.dot").encode()
    assert ctypes.CDLL("libcudart.so.13").cudaGraphDebugDotPrint(ctypes.c_void_p(graph.raw_cuda_graph()), dot, 0) == 0
    return set(re.findall(r"(?:rows8|tile8|open|rows_join|tile_join)_kernel", (tmp_path / "graph.dot").read_text()))


def path_of(eg, c, tmp_path, window=0):  # noqa: F811
    return kernels(eg, config(eg, c, window), c.cache, c.batch, c.q, tmp_path)


# One shape for each form, small enough for every edge below.
FORMS = {
    "rows": (ROWS, dict(dtype=BF16, heads=8, kv_heads=2, dim=128, page=64, block=64, new=[40, 3], total=[600, 300])),
    "cluster": (ROWS, dict(dtype=FP16, heads=4, kv_heads=4, dim=128, page=32, block=16, new=[5, 1], total=[700, 1900])),
    "cut": (CUT, dict(dtype=FP16, heads=32, kv_heads=8, dim=64, page=16, block=16, new=[2, 5, 1], total=[9000, 700, 3000])),
    "tiles": (TILES, dict(dtype=BF16, heads=64, kv_heads=2, dim=128, page=64, block=64, new=[100, 30], total=[700, 300])),
    "tiles_64": (TILES, dict(dtype=FP16, heads=64, kv_heads=2, dim=64, page=16, block=16, new=[100, 30], total=[700, 300])),
    "split": (SPLIT, dict(dtype=FP16, heads=64, kv_heads=2, dim=96, page=48, block=16, new=[300], total=[1300])),
    "split_64": (SPLIT, dict(dtype=BF16, heads=64, kv_heads=2, dim=64, page=16, block=16, new=[300, 7], total=[1300, 100])),
    "opened": (OPENED_SPLIT, dict(dtype=BF16, heads=64, kv_heads=2, dim=128, page=64, block=32, new=[1500], total=[3000])),
    "opened_64": (OPENED_SPLIT, dict(dtype=FP16, heads=64, kv_heads=2, dim=64, page=16, block=16, new=[1600, 300], total=[3000, 2000])),
}


def form(eg, name, tmp_path, window=0, **kw):  # noqa: F811
    path, c = FORMS[name]
    c = Cache(eg, **{**c, **kw})
    assert path_of(eg, c, tmp_path, window) == path
    return c


IN_PLACE = {
    "odd_heads": (TILES, (BF16, 36, 3, 96, 48, 16, [300, 20], [400, 20])),
    "padding": (TILES, (BF16, 48, 1, 96, 48, 16, [200, 5, 0, 90], [150, 3, 10, 91])),
    "all_padding": (TILES, (FP16, 64, 2, 64, 16, 16, [100, 40], [0, 300])),
    "dim_16": (TILES, (FP16, 128, 1, 16, 128, 128, [130], [131])),
    "dim_80": (TILES, (BF16, 64, 2, 80, 32, 32, [100, 30], [700, 300])),
    "many": (TILES, (BF16, 64, 2, 128, 64, 64, [33] * 34, [33 + 20 * s for s in range(34)])),
    "many_64": (TILES, (FP16, 64, 2, 48, 16, 16, [s % 7 * 9 for s in range(40)], [s % 7 * 9 + 15 * s for s in range(40)])),
    "single_heads": (TILES, (BF16, 8, 8, 128, 64, 128 // 2, [256, 255], [300, 255])),
    "mixed_split": (SPLIT, (BF16, 12, 2, 96, 48, 16, [64, 129, 1, 400], [64, 500, 2000, 401])),
    "many_split": (SPLIT, (FP16, 64, 1, 64, 64, 32, [9] * 40, [9 + 60 * s for s in range(40)])),
    "one_row_tile": (SPLIT, (BF16, 128, 1, 112, 256, 128, [1, 1, 1, 40], [3000, 100, 5, 2222])),
    "prompt": (SPLIT, (FP16, 8, 2, 128, 128, 64, [1000], [1000])),
}


@pytest.mark.parametrize("name", IN_PLACE)
def test_tiles_in_place(eg, name, tmp_path):  # noqa: F811
    path, shape = IN_PLACE[name]
    c = Cache(eg, *shape, seed=len(name))
    assert path_of(eg, c, tmp_path) == path
    check_attention(eg, c)


@pytest.mark.parametrize("window", [1, 16, 17, 100, 128, 300])
@pytest.mark.parametrize("name", ["tiles", "tiles_64", "split", "split_64"])
def test_windows_in_place(eg, name, window, tmp_path):  # noqa: F811
    """Tiles begin on any 16 keys; pages before every token's window have no id and their scales are not numbers."""
    c = Cache(eg, seed=window, **FORMS[name][1])
    assert path_of(eg, c, tmp_path, window) == TILES
    got = check_attention(eg, c, window=window)
    for s, (new, total) in enumerate(zip(c.new, c.total)):
        for e in range(max(0, total - new - window + 1) // c.page):
            page = int(c.block_table[s, e])
            c.k_scales[page] = c.v_scales[page] = float("nan")
            c.block_table[s, e] = -5
    assert int(c.block_table[0, 0]) == -5
    again = eg.engram_paged_attention_q8(config(eg, c, window), c.cache, c.batch, c.q)
    assert eg.engram_last_error() == 0
    assert torch.equal(again, got)


# ------------------------------------------------------------ scales, queries ----

def check_chunks(eg, c, scales, rows=16):  # noqa: F811
    """The bound of each `rows` tokens for themselves, from what these see alone: its absolute terms follow the largest value
    scale among the keys."""
    cfg = config(eg, c)
    lse = torch.empty((sum(c.new), c.heads), device="cuda")
    got = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q, lse=lse)
    assert eg.engram_last_error() == 0 and bool(torch.isfinite(got).all())
    t0 = 0
    for s, (new, total) in enumerate(zip(c.new, c.total)):
        for a in range(0, new, rows):
            n = min(rows, new - a)
            at = slice(t0 + a, t0 + a + n)
            ref, ref_lse, bound, lse_bound = plain.attention(c.q[at], c.k_pages, c.v_pages, c.k_scales, scales, c.block_table[s:s + 1], [n],
                                                             [total - new + a + n], c.kv_heads, cfg.scale, 0)
            off = (got[at].double() - ref).abs() - bound
            assert bool((off <= 0).all()), (s, a, float(off.max()))
            assert bool(((lse[at].double() - ref_lse).abs() <= lse_bound).all())
        t0 += new


def position_scales(c, of_block):
    """v_scales[...] = of_block(number of the 16-token strip in its sequence, how many it has), blocks of 16."""
    assert c.block == 16
    for s, total in enumerate(c.total):
        n = -(-total // 16)
        for i in range(n):
            c.v_scales[int(c.block_table[s, i * 16 // c.page]), :, i % (c.page // 16)] = of_block(i, n)


SCALES = {
    "growing": lambda i, n: 2.0 ** round(-48 + 96 * i / max(1, n - 1)),
    "falling": lambda i, n: 2.0 ** round(48 - 96 * i / max(1, n - 1)),
    "in_turn": lambda i, n: (2.0**-48, 1.0, 2.0**48, 3.7)[i * 7 % 4],
    "past_the_ends": lambda i, n: (0.0, 2.0**-60, 1e-30, 2.0**-46)[i % 4] if i < n // 2 else (2.0**50, 1e30, 2.0**48, 3e38)[i % 4],
}


@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("name", ["cut", "tiles_64", "split", "split_64", "opened_64"])
def test_value_scales_over_their_range(eg, name, kind, tmp_path):  # noqa: F811
    """Value scales from 2^-48 to 2^48, and beyond, where they count as these (bf16, whose outputs hold them)."""
    c = form(eg, name, tmp_path, dtype=BF16)
    position_scales(c, SCALES[kind])
    check_chunks(eg, c, c.v_scales.clamp(2.0**-48, 2.0**48))


@pytest.mark.parametrize("name", FORMS)
def test_key_scales_far_apart(eg, name, tmp_path):  # noqa: F811
    """Key scales of 0 and from 2^-40 to 2^-3."""
    c = form(eg, name, tmp_path)
    g = torch.Generator(device="cuda").manual_seed(6)
    e = torch.randint(-40, -2, c.k_scales.shape, generator=g, device="cuda").float()
    zero = torch.rand(e.shape, generator=g, device="cuda") < 0.2
    used = ~c.k_scales.isnan()
    c.k_scales[used] = torch.where(zero, 0.0, torch.exp2(e))[used]
    c.q.mul_(0.125)
    check_attention(eg, c)


@pytest.mark.parametrize("name", FORMS)
def test_query_ranges(eg, name, tmp_path):  # noqa: F811
    """Rows of zeros, of very large and very small values, side by side with ordinary ones."""
    c = form(eg, name, tmp_path)
    bf = c.dtype == BF16
    for t in range(0, sum(c.new), 7):
        h = t % c.heads
        c.q[t, h] = 0.0
        c.q[t, (h + 1) % c.heads] = 2.0**-24
        c.q[t, (h + 2) % c.heads] = c.q[t, (h + 2) % c.heads].sign() * (2.0**20 if bf else 60000.0)
        c.q[t, (h + 3) % c.heads] *= 2.0**-60 if bf else 2.0**-14
        c.q[t, (h + 4) % c.heads, 1:] *= 2.0**-20  # one value far above the rest
    c.k_scales[c.k_scales > 0] *= 1e-4
    check_attention(eg, c)


# ------------------------------------------------------------------ NaN, pages ----

@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("name", FORMS)
def test_nan_codes(eg, name, window, tmp_path):  # noqa: F811
    """A NaN code of a value reaches its column of the rows that see it, of a key all of theirs: in tiles seen whole and in
    part, by some row tiles and not by others, in every sequence."""
    c = form(eg, name, tmp_path)
    cfg = config(eg, c, window)
    g = c.heads // c.kv_heads
    clean = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    places = []
    for s, (new, total) in enumerate(zip(c.new, c.total)):
        first = total - new
        for i, pos in enumerate({0, first // 2, max(0, first - 150), first, first + new // 2, total - 1}):
            places.append((s, pos, i % c.kv_heads, (5 * i + 3) % c.dim))

    def marked(pages, which):
        want = torch.zeros_like(clean, dtype=torch.bool)
        kept = []
        for s, pos, head, col in which:
            code = pages.view(torch.uint8)[int(c.block_table[s, pos // c.page]), pos % c.page, head]
            kept.append((code, col, int(code[col])))
            code[col] = 0xFF if col % 2 else 0x7F
            t0, new = sum(c.new[:s]), c.new[s]
            rows = torch.arange(c.total[s] - new, c.total[s], device="cuda")
            sees = torch.zeros(len(clean), dtype=torch.bool, device="cuda")
            sees[t0:t0 + new] = (rows >= pos) & ((rows < pos + window) if window else (rows >= 0))
            if pages is c.v_pages:
                want[sees, head * g:(head + 1) * g, col] = True
            else:
                want[sees, head * g:(head + 1) * g] = True
        got = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
        for code, col, was in kept:
            code[col] = was
        assert eg.engram_last_error() == 0
        assert torch.equal(got.isnan(), want)
        assert torch.equal(got[~want], clean[~want])

    marked(c.v_pages, places)
    for p in places:
        marked(c.v_pages, [p])
        marked(c.k_pages, [p])


@pytest.mark.parametrize("name", FORMS)
def test_missing_pages_read_as_zeros(eg, name, tmp_path):  # noqa: F811
    """The result is that over a page of zeros, within the bound; other sequences' rows stay bit for bit."""
    c = form(eg, name, tmp_path)
    cfg = config(eg, c)
    whole = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    zeros = min(set(range(len(c.k_pages))) - set(c.block_table.flatten().tolist()))
    for x, sc in ((c.k_pages, c.k_scales), (c.v_pages, c.v_scales)):
        x.view(torch.uint8)[zeros] = 0
        sc[zeros] = 0.01
    e = (c.total[0] - c.new[0]) // c.page // 2
    for bad in (-1, len(c.k_pages), -(1 << 31), (1 << 31) - 1):
        c.block_table[0, e] = bad
        out = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
        assert eg.engram_last_error() == ERANGE
        assert torch.equal(out[c.new[0]:], whole[c.new[0]:])
        c.block_table[0, e] = zeros
        ref, _, bound, _ = plain.attention(c.q, c.k_pages, c.v_pages, c.k_scales, c.v_scales, c.block_table, c.new, c.total, c.kv_heads,
                                           cfg.scale, 0)
        assert bool(((out.double() - ref).abs() <= bound).all())
    c.kv_len[0] = c.page * c.block_table.shape[1] + 1
    eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    assert eg.engram_last_error() == ERANGE


# ------------------------------------------------------------- batches, strides ----

@pytest.mark.parametrize("name", FORMS)
def test_strided_heads(eg, name, tmp_path):  # noqa: F811
    """Outputs as slices of wider rows, on 16-byte boundaries that are no 32-byte ones; what lies between stays."""
    c = form(eg, name, tmp_path)
    cfg = config(eg, c)
    want = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    wide = torch.full((sum(c.new), c.heads + 1, c.dim + 8), 5.0, dtype=c.dtype, device="cuda")
    out = wide[:, :c.heads, 8:]
    got = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q.clone(), out=out)
    assert got is out and eg.engram_last_error() == 0 and torch.equal(out, want)
    assert bool((wide[:, c.heads] == 5).all()) and bool((wide[:, :, :8] == 5).all())


@pytest.mark.parametrize("name", FORMS)
def test_replayed_with_other_batches(eg, name, tmp_path):  # noqa: F811
    """One captured call, a workspace full of NaN; lengths and the tokens' shares among sequences change between replays."""
    c = form(eg, name, tmp_path)
    cfg, T, n = config(eg, c), sum(c.new), len(c.new)
    need = eg.engram_paged_attention_q8_workspace_bytes(cfg, c.cache, c.batch)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty((T, c.heads, c.dim), dtype=c.dtype, device="cuda")

    def call():
        eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q, out=out, workspace=ws)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    shares = [c.new, [T] + [0] * (n - 1), [0] * (n - 1) + [T], [T // n + (i < T % n) for i in range(n)]]
    for share in shares * 2:
        for total in (c.total, [max(1, t // 2) for t in c.total], [0] + c.total[1:]):
            c.new = share
            c.seq_offsets.copy_(torch.tensor([0] + share).cumsum(0))
            c.kv_len.copy_(i32(total))
            ws.fill_(0xFF)
            out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert eg.engram_last_error() == 0
            ref, _, bound, _ = plain.attention(c.q, c.k_pages, c.v_pages, c.k_scales, c.v_scales, c.block_table, share, total, c.kv_heads,
                                               cfg.scale, 0)
            assert bool(((out.double() - ref).abs() <= bound).all()), (share, total)
            again = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
            assert torch.equal(again, out)


@pytest.mark.parametrize("name", FORMS)
def test_rows_behind_the_last_sequence(eg, name, tmp_path):  # noqa: F811
    """Offsets that stop short of the step's rows are flagged; the rows behind them stay as they were."""
    c = form(eg, name, tmp_path)
    cfg, T = config(eg, c), sum(c.new)
    q = torch.cat([c.q, c.q[:5]])
    out, lse = torch.full_like(q, 7.0), torch.full((T + 5, c.heads), 7.0, device="cuda")
    eg.engram_paged_attention_q8(cfg, c.cache, eg.kv_batch(c.seq_offsets, c.kv_len, c.block_table, T + 5), q, out=out, lse=lse)
    assert eg.engram_last_error() == ERANGE
    assert bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all())
    ref, _, bound, _ = plain.attention(c.q, c.k_pages, c.v_pages, c.k_scales, c.v_scales, c.block_table, c.new, c.total, c.kv_heads, cfg.scale, 0)
    assert bool(((out[:T].double() - ref).abs() <= bound).all())


def test_two_graphs_of_one_workspace(eg, tmp_path):  # noqa: F811
    """Steps of different forms captured over one workspace, replayed in turn on one stream."""
    steps = [form(eg, n, tmp_path) for n in ("cut", "split", "opened", "tiles")]
    cfgs = [config(eg, c) for c in steps]
    want = [eg.engram_paged_attention_q8(f, c.cache, c.batch, c.q) for f, c in zip(cfgs, steps)]
    ws = torch.empty(max(eg.engram_paged_attention_q8_workspace_bytes(f, c.cache, c.batch) for f, c in zip(cfgs, steps)),
                     dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for f, c in zip(cfgs, steps):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(eg.engram_paged_attention_q8(f, c.cache, c.batch, c.q, workspace=ws))
    for i in (0, 1, 2, 3, 2, 1, 0, 3, 1):
        outs[i].fill_(7.0)
        graphs[i].replay()
        assert torch.equal(outs[i], want[i]), i


# --------------------------------------------------------------- far ends, both ----

@pytest.mark.parametrize("dim,block", [(16, 16), (80, 128)])
def test_longest_sequences_by_tiles(eg, dim, block, tmp_path):  # noqa: F811
    """One page of 65,536 tokens stands in every entry of the table, and a window keeps the work small."""
    heads, new, window = 128, 200, 64
    k, v = codes((1, PAGE, 1, dim), dim), codes((1, PAGE, 1, dim), dim + 1)
    ks, vs = (0.005 + 0.01 * torch.rand((1, 1, PAGE // block), device="cuda") for _ in range(2))
    q = torch.randn((new, heads, dim), device="cuda").to(BF16)
    cfg = eg.make_attn_config(heads, 1, dim, rope_dim=0, window=window)
    cache, offs = eg.kv_cache_q8(k, v, ks, vs), torch.tensor([0, new], device="cuda")
    table = torch.zeros((1, (LONGEST + 1024) // PAGE), dtype=torch.int32, device="cuda")
    batch = lambda n: eg.kv_batch(offs, i32([n]), table, new)  # noqa: E731
    run = lambda n: eg.engram_paged_attention_q8(cfg, cache, batch(n), q)  # noqa: E731
    assert kernels(eg, cfg, cache, batch(LONGEST), q, tmp_path) == TILES
    same = PAGE + LONGEST % PAGE  # the same keys near the start
    ref, _, bound, _ = plain.attention(q, k, v, ks, vs, table[:, :2], [new], [same], 1, cfg.scale, window)
    got = run(LONGEST)
    assert eg.engram_last_error() == 0
    assert ((got.double() - ref).abs() <= bound).all()
    assert torch.equal(run(same), got)
    for length in (LONGEST + 1, LONGEST + 1023):  # flagged and cut
        cut = run(length)
        assert eg.engram_last_error() == ERANGE
        assert torch.equal(cut, got)


@pytest.mark.parametrize("name", ["tiles", "tiles_64", "split", "opened"])
def test_prompts_and_single_tokens_agree(eg, name, tmp_path):  # noqa: F811
    """The same cache through the tile kernel and, token by token, the rows kernel: both within the bound."""
    c = form(eg, name, tmp_path)
    whole, cfg = check_attention(eg, c), config(eg, c)
    for t in (0, 1, c.new[0] // 2, c.new[0] - 1):
        length = c.total[0] - c.new[0] + t + 1
        batch = eg.kv_batch(torch.tensor([0, 1], device="cuda"), i32([length]), c.block_table[:1], 1)
        q = c.q[t:t + 1].clone()
        assert "rows8_kernel" in kernels(eg, cfg, c.cache, batch, q, tmp_path)
        one = eg.engram_paged_attention_q8(cfg, c.cache, batch, q)
        _, _, bound, _ = plain.attention(q, c.k_pages, c.v_pages, c.k_scales, c.v_scales, c.block_table, [1], [length], c.kv_heads, cfg.scale, 0)
        assert bool(((one.double() - whole[t:t + 1].double()).abs() <= 2 * bound).all())
