"""The attention step (head norm + rotation, cache append, paged attention)
against its plain 64-bit form (needs a GB300)."""

import math

import pytest
import torch

import attention_plain as plain

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def eg():
    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without CUDA")
    import engram_gram_hash_gb300 as eg

    eg.lib()
    return eg


class Step:
    """A step's batch over a paged cache: new[s] tokens of sequences that are total[s] long with them.
    Slots that no sequence uses hold NaN."""

    def __init__(self, eg, dtype, heads, kv_heads, dim, page, new, total, order="token", seed=0, spare=2, pages_at=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype, self.heads, self.kv_heads, self.dim, self.page = dtype, heads, kv_heads, dim, page
        self.new, self.total = list(new), list(total)
        n, T = len(new), sum(new)
        per = [-(-max(b, 0) // page) for b in total]
        n_pages = sum(per) + spare + pages_at
        shape = (n_pages, page, kv_heads, dim)

        def pages():
            if order == "token":
                x = torch.empty(shape, dtype=dtype, device="cuda")
            else:  # [page][head][token][D]
                x = torch.empty((n_pages, kv_heads, page, dim), dtype=dtype, device="cuda").transpose(1, 2)
            x[pages_at:] = math.nan
            return x

        self.k_pages, self.v_pages = pages(), pages()
        ids = (torch.randperm(sum(per) + spare, generator=g, device="cuda") + pages_at).to(torch.int32)
        self.block_table = torch.full((n, max(per + [1]) + 1), -7, dtype=torch.int32, device="cuda")
        at = 0
        for s, c in enumerate(per):
            self.block_table[s, :c] = ids[at:at + c]
            at += c
            for x in (self.k_pages, self.v_pages):
                for i in range(c):
                    used = min(page, total[s] - i * page)
                    x[self.block_table[s, i].long(), :used] = torch.randn(
                        (used, kv_heads, dim), generator=g, device="cuda").to(dtype)
        offs = torch.tensor([0] + list(new)).cumsum(0)
        self.seq_offsets = offs.cuda()
        self.kv_len = torch.tensor(total, dtype=torch.int32, device="cuda")
        self.packed = torch.randn((T, (heads + 2 * kv_heads) * dim), generator=g, device="cuda").to(dtype)
        q, k, v = self.packed.split([heads * dim, kv_heads * dim, kv_heads * dim], 1)
        self.q, self.k, self.v = (q.unflatten(1, (heads, dim)), k.unflatten(1, (kv_heads, dim)),
                                  v.unflatten(1, (kv_heads, dim)))
        self.cache = eg.kv_cache(self.k_pages, self.v_pages)
        self.batch = eg.kv_batch(self.seq_offsets, self.kv_len, self.block_table, T)


def check_attention(eg, st, window=0, scale=None, out=None):
    cfg = eg.make_attn_config(st.heads, st.kv_heads, st.dim, dtype=st.dtype, rope_dim=0, window=window, scale=scale)
    T = sum(st.new)
    lse = torch.full((T, st.heads), 7.0, device="cuda")
    if out is None:
        out = torch.full((T, st.heads, st.dim), 7.0, dtype=st.dtype, device="cuda")
    got = eg.engram_paged_attention(cfg, st.cache, st.batch, st.q, out=out, lse=lse)
    assert eg.engram_last_error() == 0
    ref, ref_lse, bound, lse_bound = plain.attention(st.q, st.k_pages, st.v_pages, st.block_table, st.new, st.total,
                                                     st.kv_heads, cfg.scale, window)
    assert torch.isfinite(got).all()
    worst = ((got.double() - ref).abs() - bound).max().item()
    assert worst <= 0, f"out is {worst} past its bound"
    empty = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
    assert (got[empty] == 0).all()
    assert ((lse.double() - ref_lse)[~empty].abs() <= lse_bound[~empty]).all()
    return got, lse


CASES = {
    "one_token": dict(heads=4, kv_heads=2, dim=64, page=16, new=[1], total=[513]),
    "one_key": dict(heads=8, kv_heads=1, dim=128, page=64, new=[1], total=[1]),
    "decode_ragged": dict(heads=32, kv_heads=8, dim=128, page=64, new=[1] * 7, total=[1, 63, 64, 65, 700, 1999, 128]),
    "decode_long": dict(heads=8, kv_heads=2, dim=128, page=128, new=[1], total=[20011]),
    "decode_long_64": dict(heads=2, kv_heads=2, dim=64, page=32, new=[1, 1], total=[9000, 5]),
    "many_sequences": dict(heads=4, kv_heads=1, dim=64, page=16, new=[1] * 400, total=[1 + 7 * i % 90 for i in range(400)]),
    "fp16_96": dict(dtype=FP16, heads=12, kv_heads=2, dim=96, page=48, new=[5, 1, 30], total=[333, 200, 30]),
    "dim_8": dict(heads=3, kv_heads=1, dim=8, page=16, new=[2, 1], total=[40, 17]),
    "dim_72": dict(heads=6, kv_heads=2, dim=72, page=80, new=[3], total=[170]),
    "group_1": dict(heads=3, kv_heads=3, dim=128, page=16, new=[17, 4], total=[100, 4]),
    "group_20": dict(heads=20, kv_heads=1, dim=128, page=64, new=[3, 1], total=[300, 77]),
    "group_128": dict(heads=128, kv_heads=1, dim=64, page=64, new=[2], total=[130]),
    "prompt": dict(heads=8, kv_heads=2, dim=128, page=64, new=[300], total=[300]),
    "prompt_fp16": dict(dtype=FP16, heads=4, kv_heads=4, dim=64, page=32, new=[129, 257, 1], total=[129, 257, 1]),
    "chunk": dict(heads=8, kv_heads=2, dim=128, page=64, new=[200, 33], total=[1500, 1033]),
    "mixed": dict(heads=12, kv_heads=4, dim=128, page=16, new=[1, 130, 1, 0, 64, 1], total=[900, 1000, 3, 50, 64, 1]),
    "no_keys": dict(heads=4, kv_heads=2, dim=128, page=16, new=[1, 3, 2], total=[0, 2, 70]),
    "no_keys_at_all": dict(heads=4, kv_heads=2, dim=64, page=16, new=[2, 1], total=[0, 0]),
    "no_tokens": dict(heads=4, kv_heads=2, dim=64, page=16, new=[0, 2, 0], total=[9, 12, 0]),
}


@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("name", CASES)
def test_attention(eg, name, order):
    c = {"dtype": BF16, **CASES[name]}
    check_attention(eg, Step(eg, order=order, seed=len(name), **c))


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 128, 1000])
@pytest.mark.parametrize("name", ["decode_ragged", "fp16_96", "prompt", "mixed", "no_keys"])
def test_attention_window(eg, name, window):
    c = {"dtype": BF16, **CASES[name]}
    check_attention(eg, Step(eg, seed=window, **c), window=window)


def test_attention_window_ignores_nan_before_it(eg):
    """Positions that no query of the step reaches may hold NaN (their pages can be reused)."""
    st = Step(eg, BF16, 8, 2, 128, 64, [1, 1], [1000, 300], seed=3)
    ref, lse = check_attention(eg, st, window=100)
    for s, b in enumerate(st.total):
        for i in range((b - 100) // 64):
            st.k_pages[st.block_table[s, i].long()] = math.nan
            st.v_pages[st.block_table[s, i].long()] = math.nan
    cfg = eg.make_attn_config(8, 2, 128, rope_dim=0, window=100)
    assert torch.equal(eg.engram_paged_attention(cfg, st.cache, st.batch, st.q), ref)


def _slot(st, s, j):
    return st.block_table[s, j // st.page].long(), j % st.page


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("shape", [
    dict(dtype=BF16, heads=8, kv_heads=2, dim=128, page=64, new=[40, 1, 130], total=[100, 70, 500]),  # tiles
    dict(dtype=FP16, heads=6, kv_heads=2, dim=72, page=48, new=[300, 7], total=[300, 200]),  # tiles
    dict(dtype=BF16, heads=4, kv_heads=2, dim=64, page=16, new=[3, 1, 2], total=[60, 130, 2]),  # few rows
    dict(dtype=FP16, heads=4, kv_heads=4, dim=128, page=32, new=[5, 1], total=[700, 1900]),  # few rows, cut
])
def test_attention_infinities_stay_with_the_rows_that_see_them(eg, shape, window):
    """Infinities and NaN among cached keys and values: a row that does not see the position is as if they
    were finite, a row that does is infinite or NaN in that column (value) or as a whole (key)."""
    st = Step(eg, seed=21, **shape)
    g = torch.Generator().manual_seed(5)
    clean_k, clean_v = st.k_pages.clone(), st.v_pages.clone()
    bad_v, bad_k = [], []
    for s, (a, b) in enumerate(zip(st.new, st.total)):
        at = {b - 1, b - a, max(b - a - 60, 0), int(torch.randint(0, b, (1,), generator=g))}
        for i, j in enumerate(sorted(at)):
            h, c = int(torch.randint(0, st.kv_heads, (1,), generator=g)), int(torch.randint(0, st.dim, (1,), generator=g))
            x = (math.inf, -math.inf, math.nan)[(i + s) % 3]
            st.v_pages[(*_slot(st, s, j), h, c)] = x
            bad_v.append((s, j, h, c, x))
    s, j, h = 0, st.total[0] - 1, 0
    st.k_pages[(*_slot(st, s, j), h, 3)] = math.nan
    bad_k.append((s, j, h))
    cfg = eg.make_attn_config(st.heads, st.kv_heads, st.dim, dtype=st.dtype, rope_dim=0, window=window)
    got = eg.engram_paged_attention(cfg, st.cache, st.batch, st.q).double()
    assert eg.engram_last_error() == 0
    finite_v = torch.where(torch.isfinite(st.v_pages), st.v_pages, torch.where(torch.isnan(clean_v), clean_v, 0))
    ref, _, bound, _ = plain.attention(st.q, clean_k, finite_v, st.block_table, st.new, st.total, st.kv_heads, cfg.scale, window)
    expect = torch.zeros_like(ref)
    pos = plain.positions_of(st.new, st.total)
    seq = torch.repeat_interleave(torch.arange(len(st.new)), torch.tensor(st.new))
    group = st.heads // st.kv_heads

    def rows_seeing(s, j):
        return ((seq == s) & (pos >= j) & ((pos < j + window) if window else (pos >= 0))).cuda()

    for s, j, h, c, x in bad_v:
        expect[rows_seeing(s, j), h * group:(h + 1) * group, c] += x
    for s, j, h in bad_k:
        expect[rows_seeing(s, j), h * group:(h + 1) * group] = math.nan
    touched = expect != 0
    assert touched.any() and not touched.all()
    assert ((got - ref).abs() <= bound)[~touched].all()
    # a weight can underflow to zero, and zero times an infinity is NaN: both are accepted where p is tiny
    assert not torch.isfinite(got[touched]).any()


def test_attention_large_scores(eg):
    """Scores of several hundred: the running maximum moves far and weights underflow."""
    st = Step(eg, BF16, 4, 1, 128, 64, [1, 40], [777, 640], seed=5)
    check_attention(eg, st, scale=2.0)


def test_attention_strided_output_and_repeat(eg):
    """A strided output view leaves its gaps alone; the same call twice gives the same bits."""
    st = Step(eg, BF16, 8, 2, 128, 64, [1, 40, 1], [777, 640, 9000], seed=6)
    wide = torch.full((42, 8, 256), 3.0, dtype=BF16, device="cuda")
    a, lse_a = check_attention(eg, st, out=wide[:, :, :128])
    assert (wide[:, :, 128:] == 3.0).all()
    b, lse_b = check_attention(eg, st)
    assert torch.equal(a, b) and torch.equal(lse_a, lse_b)


def test_attention_cache_past_32_bits(eg):
    """Pages whose element offsets pass 2^32."""
    at = (1 << 32) // (64 * 8 * 128) + 1
    st = Step(eg, BF16, 8, 8, 128, 64, [1, 70], [130, 300], seed=7, pages_at=at)
    check_attention(eg, st)


def test_attention_shared_pages(eg):
    """Two sequences whose block tables name the same prefix pages."""
    st = Step(eg, BF16, 8, 2, 128, 16, [1, 1], [200, 200], seed=8)
    st.block_table[1, :8] = st.block_table[0, :8]
    check_attention(eg, st)


def test_attention_seq_offsets_base(eg):
    """seq_offsets may start anywhere: rows count from the first offset."""
    st = Step(eg, BF16, 8, 2, 128, 16, [3, 1], [50, 20], seed=9)
    a, _ = check_attention(eg, st)
    st.seq_offsets += 1000
    b, _ = check_attention(eg, st)
    assert torch.equal(a, b)


@pytest.mark.parametrize("new, total", [
    ([1, 1, 1], [500, 70, 3000]),  # clusters, no workspace
    ([1, 1, 1], [500, 70, 5000]),  # cut and joined
    ([1, 100, 1], [500, 170, 5000]),  # tiles, split
])
def test_attention_graph_streams_workspace(eg, new, total):
    """Captured in a CUDA graph and replayed after the lengths changed; on a stream of its own; with a
    caller's workspace full of NaN."""
    st = Step(eg, BF16, 8, 2, 128, 16, new, total, seed=10)
    cfg = eg.make_attn_config(8, 2, 128, rope_dim=0)
    full, _ = check_attention(eg, st)
    n = eg.engram_paged_attention_workspace_bytes(cfg, st.cache, st.batch)
    assert (n > 0) == (total[2] == 5000)
    ws = torch.full((n // 4,), math.nan, device="cuda").view(torch.uint8)
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
    st.total = [123, total[1], 1]
    st.kv_len.copy_(torch.tensor(st.total, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    again, _ = check_attention(eg, st)
    assert torch.equal(out, again)


def test_attention_device_errors(eg):
    """A page id out of range and a length past the block table are flagged; nothing else is touched."""
    st = Step(eg, BF16, 4, 2, 64, 16, [1, 1], [60, 60], seed=11)
    cfg = eg.make_attn_config(4, 2, 64, rope_dim=0)
    good = eg.engram_paged_attention(cfg, st.cache, st.batch, st.q)
    for bad in (-1, st.k_pages.shape[0]):
        keep = st.block_table[0, 1].item()
        st.block_table[0, 1] = bad
        out = eg.engram_paged_attention(cfg, st.cache, st.batch, st.q)
        assert eg.engram_last_error() == 3
        assert torch.equal(out[1], good[1])
        st.block_table[0, 1] = keep
    st.kv_len[0] = 16 * st.block_table.shape[1] + 1
    eg.engram_paged_attention(cfg, st.cache, st.batch, st.q)
    assert eg.engram_last_error() == 3
    st.kv_len[0] = 60
    short = eg.kv_batch(st.seq_offsets, st.kv_len, st.block_table, 2)
    short.n_query = 1  # the offsets name two rows
    eg.engram_paged_attention(cfg, st.cache, short, st.q[:1])
    assert eg.engram_last_error() == 3
    assert torch.equal(eg.engram_paged_attention(cfg, st.cache, st.batch, st.q), good)
    assert eg.engram_last_error() == 0


def test_refusals_of_the_binding(eg):
    """Wrong types, shapes, devices and sizes raise before anything is enqueued; a status raises EngramError."""
    st = Step(eg, BF16, 8, 2, 128, 16, [1, 1], [30, 20], seed=13)
    cfg, table = eg.make_attn_config(8, 2, 128), eg.rope_table(64, 128)
    f16 = eg.make_attn_config(8, 2, 128, dtype=FP16)
    w = torch.ones(128, device="cuda", dtype=BF16)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    cases = [
        (TypeError, lambda: eg.engram_qk_norm_rope(f16, st.q, None, pos, table)),
        (ValueError, lambda: eg.engram_qk_norm_rope(cfg, st.k, None, pos, table)),
        (ValueError, lambda: eg.engram_qk_norm_rope(cfg, st.q[:1], st.k, pos, table)),
        (ValueError, lambda: eg.engram_qk_norm_rope(cfg, st.q, None, pos[:1], table)),
        (TypeError, lambda: eg.engram_qk_norm_rope(cfg, st.q, None, pos.long(), table)),
        (ValueError, lambda: eg.engram_qk_norm_rope(cfg, st.q, None, pos, table[:, :64].contiguous())),
        (ValueError, lambda: eg.engram_qk_norm_rope(cfg, st.q, None, pos, None)),
        (TypeError, lambda: eg.engram_qk_norm_rope(cfg, st.q, None, pos, table.half())),
        (ValueError, lambda: eg.engram_qk_norm_rope(cfg, st.q, None, pos, table, w_q=w[:64])),
        (TypeError, lambda: eg.engram_qk_norm_rope(cfg, st.q, None, pos, table, w_q=w.float())),
        (ValueError, lambda: eg.engram_qk_norm_rope(cfg, st.q, None, pos, table, q_out=torch.empty_like(st.q)[:1])),
        (eg.EngramError, lambda: eg.engram_qk_norm_rope(cfg, st.q, None, None, table)),
        (ValueError, lambda: eg.engram_kv_append(f16, st.cache, st.batch, st.k, st.v, table)),
        (ValueError, lambda: eg.engram_kv_append(cfg, st.cache, st.batch, st.k[:1], st.v, table)),
        (ValueError, lambda: eg.engram_kv_append(cfg, st.cache, st.batch, st.k, None, table)),
        (ValueError, lambda: eg.engram_paged_attention(cfg, st.cache, st.batch, st.q[:1])),
        (ValueError, lambda: eg.engram_paged_attention(cfg, st.cache, st.batch, st.q.cpu())),
        (ValueError, lambda: eg.engram_paged_attention(cfg, st.cache, st.batch, st.q, lse=torch.empty(2, 4, device="cuda"))),
        (TypeError, lambda: eg.engram_paged_attention(cfg, st.cache, st.batch, st.q, workspace=torch.empty(9, device="cuda"))),
    ]
    for i, (error, call) in enumerate(cases):
        with pytest.raises(error):
            call()
            pytest.fail(f"case {i} was accepted")
    wide = eg.kv_batch(st.seq_offsets, st.kv_len, torch.zeros((2, 1 << 14), dtype=torch.int32, device="cuda"), 2)
    with pytest.raises(eg.EngramError) as e:
        eg.engram_paged_attention(cfg, st.cache, wide, st.q, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 6  # ENGRAM_ENOMEM
    assert eg.engram_last_error() == 0


def test_calls_on_another_stream(eg):
    """With stream= the outputs and workspace made by the call belong to that stream: many calls there give
    the bits of the current stream's, with other work allocating in between."""
    st = Step(eg, BF16, 8, 2, 128, 16, [1, 60, 1], [500, 170, 6000], seed=14)
    cfg = eg.make_attn_config(8, 2, 128, rope_dim=0)
    ref = eg.engram_paged_attention(cfg, st.cache, st.batch, st.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        outs.append(eg.engram_paged_attention(cfg, st.cache, st.batch, st.q, stream=side))
        torch.full((1 << 20,), math.nan, device="cuda")
    side.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


# ------------------------------------------------------------ norm, rotation ----

HEADS = [  # dtype, heads, kv_heads, dim, rope
    (BF16, 32, 8, 128, 128),
    (BF16, 4, 2, 64, 64),
    (FP16, 24, 4, 96, 64),
    (BF16, 5, 1, 128, 32),
    (FP16, 7, 7, 80, 80),
    (BF16, 3, 3, 8, 0),
    (BF16, 9, 3, 24, 16),
    (FP16, 2, 1, 120, 112),
]


def _close(got, ref, mag, dtype, what):
    worst = ((got.detach().cpu().double() - ref).abs() - plain.norm_rope_bound(ref, mag, dtype)).max().item()
    assert worst <= 0, f"{what} is {worst} past its bound"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("shape", HEADS)
@pytest.mark.parametrize("tokens", [1, 37])
def test_qk_norm_rope(eg, shape, tokens, normed, interleaved):
    dtype, hq, hk, d, r = shape
    g = torch.Generator(device="cuda").manual_seed(tokens)
    packed = torch.randn((tokens, (hq + hk) * d), generator=g, device="cuda").to(dtype)
    q, k = packed[:, : hq * d].unflatten(1, (hq, d)), packed[:, hq * d:].unflatten(1, (hk, d))
    q.data[0, 0] = 0  # a head of zeros stays zero
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype) if normed else None for _ in range(2))
    table = eg.rope_table(5000, r) if r else None
    pos = torch.randint(0, 5000, (tokens,), generator=g, device="cuda", dtype=torch.int32) if r else None
    cfg = eg.make_attn_config(hq, hk, d, dtype=dtype, rope_dim=r, rope_interleaved=interleaved, norm_eps=1e-5)
    qo, ko = eg.engram_qk_norm_rope(cfg, q, k, pos, table, w_q=wq, w_k=wk)
    assert eg.engram_last_error() == 0
    where = pos if r else torch.zeros(tokens, dtype=torch.int32)
    t = table if r else torch.zeros((1, 0))
    for x, w, got in ((q, wq, qo), (k, wk, ko)):
        ref, mag = plain.norm_rope(x, w, where, t, r, interleaved, 1e-5)
        _close(got, ref, mag, dtype, "head")
    # in place, one of the two at a time: the same bits, the other untouched
    before = k.clone()
    eg.engram_qk_norm_rope(cfg, q, None, pos, table, w_q=wq, q_out=q)
    assert torch.equal(q, qo) and torch.equal(k, before)
    eg.engram_qk_norm_rope(cfg, None, k, pos, table, w_k=wk, k_out=k)
    assert torch.equal(k, ko)


def test_qk_norm_rope_many_tokens(eg):
    """A batch large enough for several heads per lane gives the bits of the small batches."""
    cfg = eg.make_attn_config(32, 8, 128)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((3001, 32, 128), generator=g, device="cuda").to(BF16)
    k = torch.randn((3001, 8, 128), generator=g, device="cuda").to(BF16)
    w = (1 + 0.2 * torch.randn(128, generator=g, device="cuda")).to(BF16)
    table = eg.rope_table(4000, 128)
    pos = torch.randint(0, 4000, (3001,), generator=g, device="cuda", dtype=torch.int32)
    qo, ko = eg.engram_qk_norm_rope(cfg, q, k, pos, table, w_q=w, w_k=w)
    for a in (0, 1000, 2990):
        qs, ks = eg.engram_qk_norm_rope(cfg, q[a:a + 11], k[a:a + 11], pos[a:a + 11], table, w_q=w, w_k=w)
        assert torch.equal(qs, qo[a:a + 11]) and torch.equal(ks, ko[a:a + 11])
    ref, mag = plain.norm_rope(q[:50], w, pos[:50], table, 128, False, 1e-6)
    _close(qo[:50], ref, mag, BF16, "head")


def test_qk_norm_rope_position_out_of_range(eg):
    cfg = eg.make_attn_config(2, 1, 64)
    q = torch.randn((3, 2, 64), device="cuda").to(BF16)
    table = eg.rope_table(10, 64)
    out = torch.full_like(q, 5.0)
    for bad in (-1, 10):
        pos = torch.tensor([0, bad, 9], dtype=torch.int32, device="cuda")
        eg.engram_qk_norm_rope(cfg, q, None, pos, table, q_out=out)
        assert eg.engram_last_error() == 3
        assert (out[1] == 5.0).all() and (out[0] != 5.0).any() and (out[2] != 5.0).any()


# -------------------------------------------------------------------- append ----

@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("with_q", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", [
    (BF16, 32, 8, 128, 128, 64, [1, 1, 1], [1, 64, 700]),
    (FP16, 6, 2, 96, 64, 48, [5, 0, 100, 1], [5, 9, 333, 48]),
    (BF16, 4, 4, 64, 0, 16, [33, 2], [40, 2]),
    (BF16, 8, 1, 128, 32, 16, [1] * 70, [3 + i for i in range(70)]),
    (BF16, 2, 1, 64, 64, 16, [2, 3], [0, 2]),  # padding: tokens at negative positions
])
def test_append(eg, case, interleaved, with_q, order):
    dtype, hq, hk, d, r, page, new, total = case
    st = Step(eg, dtype, hq, hk, d, page, new, total, order=order, seed=page)
    k_before, v_before = st.k_pages.clone(), st.v_pages.clone()
    g = torch.Generator(device="cuda").manual_seed(2)
    w = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype)
    table = eg.rope_table(max(total), r) if r else None
    cfg = eg.make_attn_config(hq, hk, d, dtype=dtype, rope_dim=r, rope_interleaved=interleaved)
    q_out = eg.engram_kv_append(cfg, st.cache, st.batch, st.k, st.v, table, w_k=w, q=st.q if with_q else None, w_q=w)
    assert eg.engram_last_error() == 0
    pos = plain.positions_of(new, total)
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    live = pos >= 0
    t = table if r else torch.zeros((1, 0))
    at = pos.clamp(min=0) if r else torch.zeros_like(pos)
    for kind, x in (("k", st.k), ("q", st.q)):
        ref, mag = plain.norm_rope(x, w, at, t, r, interleaved, 1e-6)
        if kind == "k":
            page_id = st.block_table.cpu()[seq, pos.clamp(min=0) // page].long()
            rows = (page_id[live], pos[live] % page)
            got = st.k_pages.cpu()[rows]
            assert torch.equal(st.v_pages.cpu()[rows], st.v.cpu()[live])
            _close(got, ref[live], mag[live], dtype, "k")
            # every other slot keeps its bits
            for now, was in ((st.k_pages, k_before), (st.v_pages, v_before)):
                now, was = now.cpu().clone(), was.cpu().clone()
                now[rows], was[rows] = 0, 0
                assert torch.equal(now.contiguous().view(torch.int16), was.contiguous().view(torch.int16))
        elif with_q:
            _close(q_out.cpu()[live], ref[live], mag[live], dtype, "q")
        else:
            assert q_out is None


def test_append_equals_norm_rope(eg):
    """The append's k and q have the bits of engram_qk_norm_rope (small and large batches)."""
    for n, new in ((40, 1), (8, 500)):
        st = Step(eg, BF16, 32, 8, 128, 64, [new] * n, [new + 11 * i for i in range(n)], seed=3)
        cfg = eg.make_attn_config(32, 8, 128)
        table = eg.rope_table(1000, 128)
        w = (1 + 0.2 * torch.randn(128, device="cuda")).to(BF16)
        pos = plain.positions_of(st.new, st.total).to(torch.int32).cuda()
        q, k = eg.engram_qk_norm_rope(cfg, st.q, st.k, pos, table, w_q=w, w_k=w)
        q2 = eg.engram_kv_append(cfg, st.cache, st.batch, st.k, st.v, table, w_k=w, q=st.q, w_q=w)
        assert torch.equal(q, q2)
        t0 = 0
        for s in range(n):
            rows = plain.gather_sequence(st.k_pages, st.block_table, s, st.total[s])[-new:]
            assert torch.equal(rows, k[t0:t0 + new])
            t0 += new


def test_append_device_errors(eg):
    st = Step(eg, BF16, 4, 2, 64, 16, [1, 1], [20, 20], seed=4)
    cfg = eg.make_attn_config(4, 2, 64)
    k_before = st.k_pages.clone()
    table = eg.rope_table(100, 64)
    st.block_table[0, 1] = st.k_pages.shape[0]
    eg.engram_kv_append(cfg, st.cache, st.batch, st.k, st.v, table)
    assert eg.engram_last_error() == 3
    st.block_table[0, 1] = -1
    eg.engram_kv_append(cfg, st.cache, st.batch, st.k, st.v, table)
    assert eg.engram_last_error() == 3
    eg.engram_kv_append(cfg, st.cache, st.batch, st.k, st.v, table[:5])  # positions past the table
    assert eg.engram_last_error() == 3
    st.kv_len[:] = 16 * st.block_table.shape[1] + 1
    eg.engram_kv_append(cfg, st.cache, st.batch, st.k, st.v, table)
    assert eg.engram_last_error() == 3
    # only sequence 1's slot was written (by the calls in which it was in range)
    changed = (st.k_pages.view(torch.int16) != k_before.view(torch.int16)).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [st.block_table[1, 1].item()]


def test_step_decode_equals_prompt(eg):
    """Appending and attending token by token gives what the whole prompt at once gives."""
    n = 40
    one = Step(eg, BF16, 8, 2, 128, 16, [n], [n], seed=12)
    cfg = eg.make_attn_config(8, 2, 128)
    table = eg.rope_table(64, 128)
    w = (1 + 0.2 * torch.randn(128, device="cuda")).to(BF16)
    q = eg.engram_kv_append(cfg, one.cache, one.batch, one.k, one.v, table, w_k=w, q=one.q, w_q=w)
    whole = eg.engram_paged_attention(cfg, one.cache, one.batch, q)
    ref, _, bound, _ = plain.attention(q, one.k_pages, one.v_pages, one.block_table, [n], [n], 2, cfg.scale, 0)
    one.k_pages.fill_(math.nan)
    one.v_pages.fill_(math.nan)
    offs = torch.tensor([0, 1], device="cuda")
    for t in range(n):
        b = eg.kv_batch(offs, torch.tensor([t + 1], dtype=torch.int32, device="cuda"), one.block_table, 1)
        qt = eg.engram_kv_append(cfg, one.cache, b, one.k[t:t + 1], one.v[t:t + 1], table, w_k=w, q=one.q[t:t + 1], w_q=w)
        assert torch.equal(qt, q[t:t + 1])
        out = eg.engram_paged_attention(cfg, one.cache, b, qt)
        assert ((out.double() - ref[t:t + 1]).abs() <= bound[t:t + 1]).all()
        assert ((whole[t:t + 1].double() - ref[t:t + 1]).abs() <= bound[t:t + 1]).all()
    assert eg.engram_last_error() == 0
