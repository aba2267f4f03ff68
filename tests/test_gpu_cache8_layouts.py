"""The 8-bit cache in other orders and places, steps without tokens, plans without maps, queries in a launch of their own
(needs a GB300)."""

import ctypes

import pytest
import torch

import cache8_plain as plain
from test_cache8_cpu import _PlanArgs
from test_gpu_cache8 import BF16, E4M3, ERANGE, FP16, Cache, Requests, check_append, check_attention, eg, i32  # noqa: F401
from test_gpu_cache8_paths import FORMS, config, form, path_of

pytestmark = pytest.mark.gpu


def laid_out(eg, c, order):  # noqa: F811
    """The same codes in another order: heads outside tokens, keys and values of a page or of a token side by side, gaps."""
    n, P, H, D = c.k_pages.shape
    if order == "head":
        pages = [torch.full((n, H, P, D), 0x7F, dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in range(2)]
    elif order == "page_pairs":
        pages = torch.full((n, 2, P, H, D), 0x7F, dtype=torch.uint8, device="cuda").unbind(1)
    elif order == "token_pairs":
        pages = torch.full((n, P, 2, H, D), 0x7F, dtype=torch.uint8, device="cuda").unbind(2)
    elif order == "head_pairs":
        pages = torch.full((n, P, H, 2, D), 0x7F, dtype=torch.uint8, device="cuda").unbind(3)
    else:  # gaps
        pages = [torch.full((n + 1, P + 2, H + 1, D + 48), 0x7F, dtype=torch.uint8, device="cuda")[1:, 1:-1, :H, 16:16 + D] for _ in range(2)]
    for to, x in zip(pages, (c.k_pages, c.v_pages)):
        to.copy_(x.view(torch.uint8))
    c.k_pages, c.v_pages = (x.view(E4M3) for x in pages)
    c.handles(eg)


ORDERS = ["head", "page_pairs", "token_pairs", "head_pairs", "gaps"]


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("name", FORMS)
def test_orders(eg, name, order, tmp_path):  # noqa: F811
    c = form(eg, name, tmp_path)
    want = eg.engram_paged_attention_q8(config(eg, c), c.cache, c.batch, c.q)
    laid_out(eg, c, order)
    assert path_of(eg, c, tmp_path) == FORMS[name][0]
    assert torch.equal(eg.engram_paged_attention_q8(config(eg, c), c.cache, c.batch, c.q), want)
    assert eg.engram_last_error() == 0


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("dtype,kv_heads,dim,page,block", [(BF16, 3, 96, 48, 16), (FP16, 2, 64, 64, 64)])
def test_append_orders(eg, dtype, kv_heads, dim, page, block, order):  # noqa: F811
    c = Cache(eg, dtype, 2 * kv_heads, kv_heads, dim, page, block, [100, 1, 30], [130, 90, 30], pow2=True)
    laid_out(eg, c, order)
    check_append(eg, c)


@pytest.mark.parametrize("name", ["tiles", "split_64", "opened", "opened_64"])
def test_pages_past_4_gb_by_tiles(eg, name, tmp_path):  # noqa: F811
    """A cache of 6 GB a tensor whose sequences lie in its last pages and at 32 bits' reach; NaN among the values there."""
    c = form(eg, name, tmp_path)
    n, P, H, D = c.k_pages.shape
    n_pages = 6 * 10**9 // (P * H * D)
    c.v_pages.view(torch.uint8)[int(c.block_table[0, 1]), 3, 1, 5] = 0x7F
    cfg = config(eg, c)
    want = eg.engram_paged_attention_q8(cfg, c.cache, c.batch, c.q)
    at = torch.tensor([n_pages - 1 - i if i % 2 else (1 << 32) // (P * H * D) - n // 2 + i for i in range(n)], device="cuda")
    pages = [torch.empty((n_pages, P, H, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((n_pages, *c.k_scales.shape[1:]), float("nan"), device="cuda") for _ in range(2)]
    for to, x, sc, y in zip(pages, (c.k_pages, c.v_pages), scales, (c.k_scales, c.v_scales)):
        to[at] = x.view(torch.uint8)
        sc[at] = y
    table = c.block_table.clone()
    used = table >= 0
    table[used] = at[table[used].long()].int()
    cache = eg.kv_cache_q8(*(x.view(E4M3) for x in pages), *scales)
    got = eg.engram_paged_attention_q8(cfg, cache, eg.kv_batch(c.seq_offsets, c.kv_len, table, sum(c.new)), c.q)
    assert eg.engram_last_error() == 0
    assert torch.equal(got.isnan(), want.isnan()) and bool(got.isnan().any())
    assert torch.equal(got.nan_to_num(), want.nan_to_num())


# ------------------------------------------------------------------ batches ----

MORE = {"many_cut": dict(dtype=FP16, heads=8, kv_heads=8, dim=64, page=16, block=16, new=[2] * 40, total=[200 * s + 2 for s in range(40)]),
        "many_tiles": dict(dtype=BF16, heads=64, kv_heads=2, dim=128, page=64, block=64, new=[33] * 34, total=[33 + 20 * s for s in range(34)])}


@pytest.mark.parametrize("name", [*FORMS, *MORE])
def test_step_of_a_plan_that_failed(eg, name):  # noqa: F811
    """A plan without room gives offsets of zero; append and attention of the step flag it and write nothing."""
    c = Cache(eg, **(MORE[name] if name in MORE else FORMS[name][1]))
    T, n = sum(c.new), len(c.new)
    p = eg.engram_kv_plan(i32(c.new), i32([t - a for t, a in zip(c.total, c.new)]), c.block_table, i32([1, 2]), i32([0]), c.page, T - 1)
    assert eg.engram_last_error() == 4 and p.seq_offsets.tolist() == [0] * (n + 1)
    batch, cfg = eg.kv_batch(p.seq_offsets, p.kv_len, c.block_table, T), config(eg, c)
    before = [t.view(torch.uint8).clone() for t in (c.k_pages, c.v_pages, c.k_scales, c.v_scales)]
    q_out = torch.full((T, c.heads, c.dim), 7.0, dtype=c.dtype, device="cuda")
    eg.engram_kv_append_q8(cfg, c.cache, batch, c.k, c.v, None, q=c.q, q_out=q_out)
    assert eg.engram_last_error() == ERANGE and bool((q_out == 7).all())
    assert all(torch.equal(t.view(torch.uint8), b) for t, b in zip((c.k_pages, c.v_pages, c.k_scales, c.v_scales), before))
    lse = torch.full((T, c.heads), 7.0, device="cuda")
    eg.engram_paged_attention_q8(cfg, c.cache, batch, c.q, out=q_out, lse=lse)
    assert eg.engram_last_error() == ERANGE and bool((q_out == 7).all()) and bool((lse == 7).all())


def test_few_tokens_among_many_sequences(eg):  # noqa: F811
    new = [0] * 1500
    for s, n in ((0, 1), (31, 2), (700, 5), (1499, 1)):
        new[s] = n
    c = Cache(eg, BF16, 8, 2, 64, 16, 16, new, [n and n + 3 * s // 10 for s, n in enumerate(new)])
    check_attention(eg, c)
    check_append(eg, c)


@pytest.mark.parametrize("dtype,heads,kv_heads,dim,block", [(BF16, 32, 4, 128, 64), (FP16, 48, 2, 64, 16), (BF16, 33, 3, 96, 128)])
def test_append_whose_queries_go_apart(eg, dtype, heads, kv_heads, dim, block):  # noqa: F811
    """Queries of so many tokens that they have a launch of their own; some tokens are padding."""
    new, total = [3000, 1, 2900], [2990, 700, 3300]
    assert sum(new) * ((heads + 3) // 4) >= torch.cuda.get_device_properties(0).multi_processor_count * 256
    check_append(eg, Cache(eg, dtype, heads, kv_heads, dim, 128, block, new, total, pow2=True))


# --------------------------------------------------------------------- plan ----

@pytest.mark.parametrize("left_out", [("positions",), ("slots",), ("positions", "slots")])
@pytest.mark.parametrize("tokens", [4096, 4097, 9000])
def test_plan_maps_left_out(eg, left_out, tokens):  # noqa: F811
    """Through the C structure, maps that are NULL are not made, on both sides of the kernel for many tokens."""
    old = [20 + s % 30 for s in range(300)]
    keep, new = [o - s % 3 for s, o in enumerate(old)], [s % 14 for s in range(300)]
    r = Requests(old, keep, new, 16, spare=2)
    assert sum(new) <= tokens
    outs = dict(kv_len_out=i32([7] * 300), n_free_out=i32([7]), seq_offsets=torch.full((301,), 7, device="cuda"), counts=i32([7] * 4),
                positions=i32([7] * tokens), slots=torch.full((tokens,), 7, device="cuda"))
    ins = dict(new_len=i32(new), keep_len=i32(keep), kv_len=i32(old), n_free=i32([r.n_free]), block_table=r.t_table, free_pages=r.t_stack)
    p = _PlanArgs()
    p.n_seqs, p.max_tokens, p.n_pages, p.page_size = 300, tokens, r.n_pages, 16
    p.table_stride, p.table_width = r.t_table.stride(0), r.width
    for name, t in {**ins, **outs}.items():
        setattr(p, name, None if name in left_out else t.data_ptr())
    assert eg.lib().engram_kv_plan(ctypes.byref(p), None) == 0
    assert eg.engram_last_error() == 0
    offs, after, table, stack, free, pos, slots, counts = plain.plan(old, keep, new, r.table, r.stack, r.n_free, 16)
    tail = [-1] * (tokens - len(pos))
    want = dict(kv_len_out=after, n_free_out=[free], seq_offsets=offs, counts=counts, positions=pos + tail, slots=slots + tail)
    for name, t in outs.items():
        assert t.tolist() == ([7] * tokens if name in left_out else want[name]), name
    assert r.t_table.tolist() == table and r.t_stack.tolist() == stack


# ------------------------------------------------------------- parts of a step ----

@pytest.mark.parametrize("first", [1, 1000, 1 << 40])
@pytest.mark.parametrize("name", FORMS)
def test_offsets_from_anywhere(eg, name, first, tmp_path):  # noqa: F811
    """A step's offsets need not begin at 0: appends and results are the same bit for bit."""
    c, d = (form(eg, name, tmp_path) for _ in range(2))
    d.seq_offsets += first
    cfg = config(eg, c)
    for x in (c, d):
        eg.engram_kv_append_q8(cfg, x.cache, x.batch, x.k, x.v, None)
    out, other = (eg.engram_paged_attention_q8(cfg, x.cache, x.batch, x.q) for x in (c, d))
    assert eg.engram_last_error() == 0 and torch.equal(out, other)
    for x, y in ((c.k_pages, d.k_pages), (c.v_pages, d.v_pages), (c.k_scales, d.k_scales), (c.v_scales, d.v_scales)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_a_step_in_two_calls(eg):  # noqa: F811
    """Single tokens and a chunk of one step, a call for each: slices of its offsets, lengths, table and queries."""
    new, total = [1] * 12 + [400], [50 * s + 1 for s in range(12)] + [1500]
    c = Cache(eg, BF16, 32, 8, 128, 64, 64, new, total)
    cfg, whole = config(eg, c), check_attention(eg, c)
    ref, _, bound, _ = plain.attention(c.q, c.k_pages, c.v_pages, c.k_scales, c.v_scales, c.block_table, new, total, 8, cfg.scale, 0)
    for lo, hi in ((0, 12), (12, 13)):
        rows = slice(sum(new[:lo]), sum(new[:hi]))
        width = -(-max(total[lo:hi]) // 64)
        batch = eg.kv_batch(c.seq_offsets[lo:hi + 1], c.kv_len[lo:hi], c.block_table[lo:hi, :width], sum(new[lo:hi]))
        part = eg.engram_paged_attention_q8(cfg, c.cache, batch, c.q[rows])
        assert eg.engram_last_error() == 0
        assert bool(((part.double() - ref[rows]).abs() <= bound[rows]).all())
        assert bool(((part.double() - whole[rows].double()).abs() <= 2 * bound[rows]).all())
