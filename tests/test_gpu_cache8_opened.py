"""Attention over the 8-bit cache where the codes are made fp16 tiles in the workspace first (long prompts and chunks: a rule
on sizes, seen in the workspace's size), at the edges of that form.  Bounds and the plain form as in the cache's other tests
(needs a GB300)."""

import pytest
import torch

from test_gpu_cache8 import BF16, ERANGE, FP16, Cache, check_attention, eg, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def opened(eg, cfg, c):  # noqa: F811
    """Whether the workspace holds every sequence's tiles (4 bytes a key's value)."""
    room = c.block_table.shape[1] * c.page
    tiles = len(c.new) * c.kv_heads * room * (256 if c.dim <= 64 else 512)
    return eg.engram_paged_attention_q8_workspace_bytes(cfg, c.cache, c.batch) >= tiles


def config(eg, c, window=0):  # noqa: F811
    return eg.make_attn_config(c.heads, c.kv_heads, c.dim, dtype=c.dtype, rope_dim=0, window=window)


@pytest.mark.parametrize("dtype,heads,kv_heads,dim,page,block,new,total", [
    (BF16, 64, 2, 128, 64, 64, [1500], [3000]),
    (FP16, 64, 2, 64, 16, 16, [1777], [3001]),
    (BF16, 72, 3, 96, 48, 16, [700, 0, 1, 900], [2500, 40, 7, 2111]),
    (FP16, 128, 1, 16, 128, 128, [2049], [2049]),
    (BF16, 64, 2, 80, 32, 32, [1200, 600], [1100, 3300]),  # padding before the first token
    (FP16, 8, 8, 128, 256, 128, [4000], [4100]),
])
def test_shapes(eg, dtype, heads, kv_heads, dim, page, block, new, total):  # noqa: F811
    c = Cache(eg, dtype, heads, kv_heads, dim, page, block, new, total, seed=dim)
    assert opened(eg, config(eg, c), c)
    check_attention(eg, c)


@pytest.mark.parametrize("window", [333, 700])
@pytest.mark.parametrize("dim,page,block", [(128, 16, 16), (64, 48, 16)])
def test_windows_over_pages_given_back(eg, window, dim, page, block):  # noqa: F811
    """Tiles begin on any 16 keys; pages before every token's window have no id and their scales are not numbers."""
    new, total = [3000, 2500], [3700, 2500]
    c = Cache(eg, BF16, 64, 2, dim, page, block, new, total, seed=window)
    cfg = config(eg, c, window)
    assert opened(eg, cfg, c)
    got = check_attention(eg, c, window=window)
    gone = (total[0] - new[0] - window) // page  # the first token sees positions total - new - window + 1 on
    c.block_table[0, :gone] = -5  # (none with a window of 700)
    again = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    assert eg.engram_last_error() == 0
    assert torch.equal(again, got)


@pytest.mark.parametrize("window", [0, 700])
def test_nan_codes(eg, window):  # noqa: F811
    """NaN among the values reaches its column of the rows that see the key, in tiles seen whole and in part."""
    new, total = [3000], [3500]
    c = Cache(eg, BF16, 64, 2, 64, 64, 16, new, total, seed=9)
    cfg = config(eg, c, window)
    assert opened(eg, cfg, c)
    clean = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    want = torch.zeros_like(clean, dtype=torch.bool)
    rows = torch.arange(total[0] - new[0], total[0], device="cuda")
    for pos, head, col in ((300, 0, 3), (1031, 1, 5), (2900, 0, 63), (3499, 1, 0)):
        c.v_pages.view(torch.uint8)[int(c.block_table[0, pos // 64]), pos % 64, head, col] = 0x7F
        sees = (rows >= pos) & ((rows < pos + window) if window else (rows >= 0))
        want[sees, head * 32:(head + 1) * 32, col] = True
    got = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    assert eg.engram_last_error() == 0
    assert torch.equal(got.isnan(), want)
    assert torch.equal(got[~want], clean[~want])
    # among the keys: every column of the rows that see it
    pos = 3100
    c.k_pages.view(torch.uint8)[int(c.block_table[0, pos // 64]), pos % 64, 1, 7] = 0xFF
    sees = (rows >= pos) & ((rows < pos + window) if window else (rows >= 0))
    want[sees, 32:] = True
    assert torch.equal(eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q).isnan(), want)


def test_scales_far_apart(eg):  # noqa: F811
    """Neighbouring blocks' scales a factor of 2^30 apart, scales of 0."""
    c = Cache(eg, FP16, 64, 2, 64, 16, 16, [1500], [3000], seed=4)
    g = torch.Generator(device="cuda").manual_seed(5)
    used = ~c.v_scales.isnan()
    e = torch.randint(-24, 5, c.v_scales.shape, generator=g, device="cuda").float()
    c.v_scales[used] = torch.exp2(e)[used]
    none = (torch.rand(c.k_scales.shape, generator=g, device="cuda") < 0.2) & ~c.k_scales.isnan()
    c.k_scales[none] = 0.0
    assert opened(eg, config(eg, c), c)
    check_attention(eg, c)


def test_bad_pages_and_lengths(eg):  # noqa: F811
    c = Cache(eg, BF16, 64, 2, 128, 64, 64, [1500, 600], [3000, 2900])
    cfg = config(eg, c)
    assert opened(eg, cfg, c)
    whole = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    c.block_table[0, 2] = c.k_pages.shape[0]
    out = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    assert eg.engram_last_error() == ERANGE
    assert bool(torch.isfinite(out).all()) and torch.equal(out[1500:], whole[1500:])
    c.block_table[0, 2] = -1
    c.kv_len[0] = 64 * c.block_table.shape[1] + 1
    eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    assert eg.engram_last_error() == ERANGE


def test_replayed_with_other_lengths(eg):  # noqa: F811
    """One captured call, a workspace full of NaN, lengths that change between replays; equal bits each time."""
    new, total = [1500, 700], [3000, 2800]
    c = Cache(eg, BF16, 64, 2, 128, 64, 64, new, total, seed=3)
    cfg = config(eg, c)
    assert opened(eg, cfg, c)
    need = eg.engram_paged_attention_q8_workspace_bytes(cfg, c.cache, c.batch)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c.q.contiguous())

    def call():
        eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q, out=out, workspace=ws)

    def eager(lengths):
        c.kv_len.copy_(i32(lengths))
        ws.fill_(0xFF)
        call()
        return out.clone()

    lengths = [total, [1500, 700], [2999, 1001]]
    want = [eager(n) for n in lengths]
    c.kv_len.copy_(i32(total))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for n, w in list(zip(lengths, want)) * 2:
        c.kv_len.copy_(i32(n))
        ws.fill_(0xFF)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert eg.engram_last_error() == 0
        assert torch.equal(out, w)


def test_small_workspaces_stay_small(eg):  # noqa: F811
    """Over a gigabyte of tiles the codes stay as they are; the result holds."""
    c = Cache(eg, BF16, 64, 2, 128, 64, 64, [1500], [3000])
    wide = torch.full((1, 40000), -7, dtype=torch.int32, device="cuda")
    wide[:, :c.block_table.shape[1]] = c.block_table
    c.block_table = wide
    c.handles(eg)
    cfg = config(eg, c)
    assert not opened(eg, cfg, c)
    assert eg.engram_paged_attention_q8_workspace_bytes(cfg, c.cache, c.batch) < 1 << 30
    check_attention(eg, c)
