"""Scores of minus infinity (infinite keys): a row that sees nothing else has no softmax and becomes NaN with a
log-sum-exp of minus infinity; beside finite scores they weigh nothing; a row without any key stays zero (needs a GB300)."""

import math

import pytest
import torch

from test_gpu_attention import BF16, FP16, Step, eg  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = {  # the first sequence starts at position 0; the last begins with a token before its start
    "cluster": dict(heads=8, kv_heads=2, dim=128, page=64, new=[3, 2], total=[3, 1]),
    "cluster_long": dict(heads=8, kv_heads=2, dim=64, page=64, new=[1, 2], total=[1500, 1]),
    "whole": dict(dtype=FP16, heads=12, kv_heads=2, dim=96, page=48, new=[20, 1, 30], total=[20, 200, 29]),
    "cut": dict(heads=8, kv_heads=2, dim=128, page=64, new=[1, 2], total=[20011, 1]),
    "cut_many": dict(heads=8, kv_heads=2, dim=64, page=64, new=[2] * 40, total=[9000 if i == 5 else 3 for i in range(39)] + [1]),
    "tiles": dict(heads=64, kv_heads=1, dim=64, page=16, new=[90, 3], total=[90, 2]),
    "tiles_split": dict(dtype=FP16, heads=64, kv_heads=1, dim=128, page=16, new=[90, 60, 3], total=[90, 5000, 2]),
}


@pytest.mark.parametrize("name", SHAPES)
def test_minus_infinity(eg, name):  # noqa: F811
    st = Step(eg, seed=5, **{"dtype": BF16, **SHAPES[name]})
    q = st.q.clone()
    q[..., 3] = 1.0
    cfg = eg.make_attn_config(st.heads, st.kv_heads, st.dim, dtype=st.dtype, rope_dim=0)
    pos = torch.cat([torch.arange(b - a, b) for a, b in zip(st.new, st.total)]).cuda()
    seq = torch.repeat_interleave(torch.arange(len(st.new)), torch.tensor(st.new)).cuda()

    def run():
        lse = torch.zeros((sum(st.new), st.heads), device="cuda")
        out = eg.engram_paged_attention(cfg, st.cache, st.batch, q, lse=lse)
        assert eg.engram_last_error() == 0
        return out, lse

    # every sequence's first key: far below (a weight of exactly zero), then at minus infinity
    first = st.block_table[:, 0].long()[torch.tensor(st.total).cuda() > 0]
    st.k_pages[first, 0, :, 3] = -30000.0
    low, low_lse = run()
    st.k_pages[first, 0, :, 3] = -math.inf
    out, lse = run()
    alone, others = pos == 0, pos != 0
    assert torch.equal(out[others], low[others]) and torch.equal(lse[others], low_lse[others])
    assert torch.isfinite(low).all() and torch.isnan(out[alone]).all() and (lse[alone] == -math.inf).all()
    assert (out[pos < 0] == 0).all() and (lse[pos < 0] == -math.inf).all() and (pos < 0).any()

    # all keys of the sequences
    for s, b in enumerate(st.total):
        for i in range(-(-b // st.page)):
            st.k_pages[st.block_table[s, i].long(), : min(st.page, b - i * st.page), :, 3] = -math.inf
    out, lse = run()
    assert torch.isnan(out[pos >= 0]).all() and (lse == -math.inf).all() and (out[pos < 0] == 0).all()
    assert (seq[pos >= 0] == 0).any()
