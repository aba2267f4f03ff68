"""Paged attention with many query rows a sequence (prompts, chunks, wide head
groups: the kernel over row tiles) against its plain 64-bit form (needs a GB300).

The batches, the plain form and the bounds are those of the few-row tests; here
every case has several hundred rows of queries a sequence, so that items of two
row tiles, of one, and of a few rows stand side by side.
"""

import math

import pytest
import torch

import attention_plain as plain
import test_gpu_attention as base
from test_gpu_attention import BF16, FP16, Step, check_attention, eg  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = {
    # unsplit: at most 768 keys
    "mixed_short": dict(heads=128, kv_heads=2, dim=128, page=16, new=[1, 130, 1, 0, 64, 1], total=[700, 640, 3, 50, 64, 1]),
    "no_keys": dict(heads=64, kv_heads=1, dim=64, page=16, new=[1, 3, 2, 90], total=[0, 2, 70, 40]),
    "no_keys_128": dict(dtype=FP16, heads=64, kv_heads=1, dim=128, page=32, new=[90, 3, 2, 1], total=[40, 2, 70, 0]),
    "no_keys_at_all": dict(heads=64, kv_heads=1, dim=64, page=16, new=[100, 50], total=[0, 0]),
    "no_tokens": dict(heads=64, kv_heads=1, dim=128, page=16, new=[0, 70, 0], total=[9, 120, 0]),
    "one_key": dict(heads=64, kv_heads=1, dim=64, page=16, new=[70], total=[1]),
    "group_1": dict(dtype=FP16, heads=16, kv_heads=16, dim=72, page=48, new=[300, 7, 257], total=[300, 200, 600]),
    "group_3": dict(heads=12, kv_heads=4, dim=64, page=32, new=[500, 1, 259, 128], total=[700, 513, 260, 129]),
    "dim_8": dict(heads=32, kv_heads=2, dim=8, page=16, new=[129, 64], total=[500, 64]),
    "one_token_groups": dict(heads=128, kv_heads=1, dim=64, page=64, new=[1] * 200, total=[1 + 7 * i % 190 for i in range(200)]),
    "sequences_60": dict(heads=64, kv_heads=1, dim=128, page=16, new=[7 * i % 23 for i in range(60)],
                         total=[7 * i % 23 + 11 * i % 300 for i in range(60)]),
    # longer: items may be split and joined
    "mixed": dict(heads=128, kv_heads=2, dim=128, page=16, new=[1, 130, 1, 0, 64, 1], total=[900, 1000, 3, 50, 64, 1]),
    "group_20": dict(heads=20, kv_heads=1, dim=128, page=80, new=[65, 3, 200], total=[1500, 77, 333]),
    "fp16_96": dict(dtype=FP16, heads=24, kv_heads=4, dim=96, page=48, new=[130, 1, 333], total=[1130, 900, 2000]),
    "prompt": dict(heads=8, kv_heads=2, dim=128, page=64, new=[1100], total=[1100]),
    "prompt_64": dict(dtype=FP16, heads=4, kv_heads=4, dim=64, page=128, new=[900, 511], total=[900, 511]),
    "chunk": dict(heads=8, kv_heads=1, dim=128, page=64, new=[300], total=[9001]),
    "chunk_64": dict(heads=8, kv_heads=1, dim=64, page=256, new=[300, 200], total=[6000, 777]),
    "sequences_50": dict(heads=32, kv_heads=2, dim=64, page=16, new=[1 + 13 * i % 57 for i in range(50)],
                         total=[1 + 13 * i % 57 + 37 * i % 1300 for i in range(50)]),
}


@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("name", CASES)
def test_prompts(eg, name, order):  # noqa: F811
    check_attention(eg, Step(eg, order=order, seed=len(name), **{"dtype": BF16, **CASES[name]}))


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 128, 129, 300, 1000])
@pytest.mark.parametrize("name", ["mixed_short", "no_keys", "group_1", "fp16_96", "chunk", "chunk_64", "sequences_50"])
def test_prompts_window(eg, name, window):  # noqa: F811
    check_attention(eg, Step(eg, seed=window, **{"dtype": BF16, **CASES[name]}), window=window)


@pytest.mark.parametrize("dim", [64, 128])
def test_prompts_window_ignores_nan_before_it(eg, dim):  # noqa: F811
    """Pages that no query of the step reaches may hold NaN."""
    st = Step(eg, BF16, 64, 1, dim, 64, [70, 1, 33], [1000, 300, 700], seed=3)
    ref, _ = check_attention(eg, st, window=100)
    for s, (a, b) in enumerate(zip(st.new, st.total)):
        for i in range((b - a + 1 - 100) // 64):
            st.k_pages[st.block_table[s, i].long()] = math.nan
            st.v_pages[st.block_table[s, i].long()] = math.nan
    cfg = eg.make_attn_config(64, 1, dim, rope_dim=0, window=100)
    assert torch.equal(eg.engram_paged_attention(cfg, st.cache, st.batch, st.q), ref)


@pytest.mark.parametrize("window", [0, 50, 200])
@pytest.mark.parametrize("shape", [
    dict(dtype=BF16, heads=64, kv_heads=2, dim=128, page=64, new=[40, 1, 130], total=[100, 70, 500]),
    dict(dtype=FP16, heads=48, kv_heads=2, dim=72, page=48, new=[300, 7], total=[300, 200]),
    dict(dtype=BF16, heads=64, kv_heads=1, dim=64, page=16, new=[30, 1, 200], total=[600, 130, 200]),
    dict(dtype=BF16, heads=128, kv_heads=2, dim=128, page=16, new=[1, 60, 2], total=[900, 1700, 40]),
    dict(dtype=FP16, heads=32, kv_heads=1, dim=64, page=32, new=[100, 90], total=[2500, 90]),
])
def test_prompts_infinities_stay_with_the_rows_that_see_them(eg, shape, window):  # noqa: F811
    base.test_attention_infinities_stay_with_the_rows_that_see_them(eg, shape, window)


@pytest.mark.parametrize("dim", [64, 128])
def test_prompts_large_scores(eg, dim):  # noqa: F811
    """Scores of several hundred: the running maximum moves far, sums are rescaled and weights underflow."""
    st = Step(eg, BF16, 64, 1, dim, 64, [1, 140], [777, 1640], seed=5)
    check_attention(eg, st, scale=2.0)


@pytest.mark.parametrize("dim", [64, 128])
def test_prompts_rising_scores(eg, dim):  # noqa: F811
    """Every tile of keys has larger scores than the one before: the sums are rescaled at each."""
    st = Step(eg, BF16, 64, 1, dim, 64, [130], [1280], seed=15)
    q = st.q.clone()
    q[:] = 1.0
    st.q = q
    for i in range(20):
        st.k_pages[st.block_table[0, i].long()] = (0.1 * i)
    check_attention(eg, st, scale=1.0)


def test_prompts_strided_output_and_repeat(eg):  # noqa: F811
    """Strided output views leave their gaps alone, whatever their alignment; the same call twice gives the
    same bits."""
    st = Step(eg, BF16, 64, 2, 128, 64, [1, 40, 100], [777, 640, 9000], seed=6)
    for width, at in ((256, 0), (256, 64), (136, 8)):
        wide = torch.full((141, 64, width), 3.0, dtype=BF16, device="cuda")
        a, lse_a = check_attention(eg, st, out=wide[:, :, at:at + 128])
        assert (wide[:, :, :at] == 3.0).all() and (wide[:, :, at + 128:] == 3.0).all()
    b, lse_b = check_attention(eg, st)
    assert torch.equal(a, b) and torch.equal(lse_a, lse_b)


def test_prompts_cache_past_32_bits(eg):  # noqa: F811
    """Pages whose element offsets pass 2^32."""
    at = (1 << 32) // (64 * 8 * 128) + 1
    check_attention(eg, Step(eg, BF16, 64, 8, 128, 64, [1, 270], [130, 300], seed=7, pages_at=at))


def test_prompts_seq_offsets_base(eg):  # noqa: F811
    st = Step(eg, BF16, 64, 1, 128, 16, [30, 100], [50, 1200], seed=9)
    a, _ = check_attention(eg, st)
    st.seq_offsets += 1000
    b, _ = check_attention(eg, st)
    assert torch.equal(a, b)


@pytest.mark.parametrize("n_seqs", [3, 40])
@pytest.mark.parametrize("longest", [600, 5000])
def test_prompts_graph_streams_workspace(eg, n_seqs, longest):  # noqa: F811
    """Captured in a CUDA graph and replayed after the lengths changed; on a stream of its own; with a
    caller's workspace full of NaN."""
    new = [90, 1, 40] + [2] * (n_seqs - 3)
    total = [500, 70, longest] + [2 + 9 * i for i in range(n_seqs - 3)]
    st = Step(eg, BF16, 64, 1, 128, 16, new, total, seed=10)
    cfg = eg.make_attn_config(64, 1, 128, rope_dim=0)
    full, _ = check_attention(eg, st)
    n = eg.engram_paged_attention_workspace_bytes(cfg, st.cache, st.batch)
    assert (n > 8 << 20) == (longest == 5000)  # partial results of whole items: the row-tile kernel, split
    ws = torch.full((n // 4,), math.nan, device="cuda").view(torch.uint8) if n else None
    out = torch.empty_like(full)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eg.engram_paged_attention(cfg, st.cache, st.batch, st.q, out=out, workspace=ws)
    side.synchronize()
    assert torch.equal(out, full)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eg.engram_paged_attention(cfg, st.cache, st.batch, st.q, out=out, workspace=ws)
    st.total = [123, 30, 1] + total[3:]
    st.kv_len.copy_(torch.tensor(st.total, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    again, _ = check_attention(eg, st)
    assert torch.equal(out, again)


def test_prompts_device_errors(eg):  # noqa: F811
    """A page id out of range and a length past the block table are flagged; other sequences keep their bits."""
    st = Step(eg, BF16, 64, 1, 64, 16, [60, 70], [60, 500], seed=11)
    cfg = eg.make_attn_config(64, 1, 64, rope_dim=0)
    good = eg.engram_paged_attention(cfg, st.cache, st.batch, st.q)
    for bad in (-1, st.k_pages.shape[0]):
        keep = st.block_table[0, 1].item()
        st.block_table[0, 1] = bad
        out = eg.engram_paged_attention(cfg, st.cache, st.batch, st.q)
        assert eg.engram_last_error() == 3
        assert torch.equal(out[60:], good[60:])
        st.block_table[0, 1] = keep
    st.kv_len[0] = 16 * st.block_table.shape[1] + 1
    eg.engram_paged_attention(cfg, st.cache, st.batch, st.q)
    assert eg.engram_last_error() == 3
    st.kv_len[0] = 60
    assert torch.equal(eg.engram_paged_attention(cfg, st.cache, st.batch, st.q), good)
    assert eg.engram_last_error() == 0


@pytest.mark.parametrize("name", ["group_3", "fp16_96", "chunk_64"])
def test_prompts_rows_do_not_depend_on_the_batch(eg, name):  # noqa: F811
    """A sequence's rows are within the bounds whether it is served alone or with the others."""
    c = {"dtype": BF16, **CASES[name]}
    st = Step(eg, seed=16, **c)
    cfg = eg.make_attn_config(st.heads, st.kv_heads, st.dim, dtype=st.dtype, rope_dim=0)
    ref, _, bound, _ = plain.attention(st.q, st.k_pages, st.v_pages, st.block_table, st.new, st.total, st.kv_heads,
                                       cfg.scale, 0)
    t0 = 0
    for s, a in enumerate(st.new):
        offs = torch.tensor([0, a], device="cuda")
        one = eg.kv_batch(offs, st.kv_len[s:s + 1], st.block_table[s:s + 1], a)
        got = eg.engram_paged_attention(cfg, st.cache, one, st.q[t0:t0 + a])
        assert ((got.double() - ref[t0:t0 + a]).abs() <= bound[t0:t0 + a]).all()
        t0 += a
    assert eg.engram_last_error() == 0
