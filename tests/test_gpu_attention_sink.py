"""A key far above the others whose value is zero (an attention sink): the output is what the other keys' small weights
make of it, so their bits count (needs a GB300).

The bound is the plain form's with one term sharpened.  Weights are rounded to the 16-bit type relative to the row's
largest one, w = 1: a relative u, and where fp16 is subnormal an absolute 2^-25 of the unit in which the weights are
kept.  Kept so that the largest lies between 2^11 and 2^15, that is at most 2^-36 of the largest weight per key (bf16:
its exponents reach further still), so n 2^-36 max|v| stands in the place of n 2^-25 max|v|.
"""

import pytest
import torch

import attention_plain as plain
from test_gpu_attention import BF16, FP16, Step, eg  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = {
    "cluster": dict(heads=8, kv_heads=2, dim=128, page=64, new=[1], total=[2000]),
    "whole": dict(heads=8, kv_heads=2, dim=128, page=16, new=[2], total=[120]),
    "cut": dict(heads=8, kv_heads=2, dim=128, page=64, new=[1], total=[20011]),
    "cut_64": dict(heads=4, kv_heads=4, dim=64, page=32, new=[3], total=[40000]),
    "tiles": dict(heads=64, kv_heads=1, dim=128, page=16, new=[90], total=[600]),
    "tiles_64": dict(heads=64, kv_heads=1, dim=64, page=16, new=[90], total=[600]),
    "tiles_split": dict(heads=64, kv_heads=1, dim=128, page=64, new=[60], total=[9000]),
    "tiles_split_64": dict(heads=64, kv_heads=1, dim=64, page=64, new=[60], total=[9000]),
}


@pytest.mark.parametrize("nats", [12.0, 14.0, 16.0, 18.0])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("name", SHAPES)
def test_sink(eg, name, dtype, nats):  # noqa: F811
    st = Step(eg, dtype, seed=11, **SHAPES[name])
    n, D = st.total[0], st.dim
    # scores: the first value of q and of key 0 make `nats`, the others a little around zero
    q = 0.3 * st.q
    q[..., 0] = D**0.5
    st.q = q
    st.k_pages[..., 0] = 0.0
    where = (st.block_table[0, 0].long(), 0)
    st.k_pages[where] = 0.0
    st.k_pages[(*where, slice(None), 0)] = nats
    st.v_pages.copy_(1.0 + 0.1 * torch.rand(st.v_pages.shape, device="cuda").to(dtype))
    st.v_pages[where] = 0.0
    cfg = eg.make_attn_config(st.heads, st.kv_heads, D, dtype=dtype, rope_dim=0)
    lse = torch.empty((sum(st.new), st.heads), device="cuda")
    got = eg.engram_paged_attention(cfg, st.cache, st.batch, st.q, lse=lse)
    assert eg.engram_last_error() == 0
    ref, ref_lse, bound, lse_bound = plain.attention(st.q, st.k_pages, st.v_pages, st.block_table, st.new, st.total,
                                                     st.kv_heads, cfg.scale, 0)
    used = plain.gather_sequence(st.v_pages, st.block_table, 0, n).abs().double()
    vmax = used.amax((0, 2)).repeat_interleave(st.heads // st.kv_heads)[None, :, None]
    bound = bound - n * (2.0**-25 - 2.0**-36) * vmax
    if dtype == FP16:  # the output itself may be subnormal
        bound = bound + 2.0**-25
    assert (ref > 0).all()
    worst = ((got.double() - ref).abs() / bound).max().item()
    assert worst <= 1, f"the error is {worst} times its bound"
    assert ((lse.double() - ref_lse).abs() <= lse_bound).all()
