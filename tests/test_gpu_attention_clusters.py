"""Attention calls whose CTAs exchange their parts through distributed shared memory, one behind the other: each starts
while the one before it drains, and a CTA leaves only when no other needs its memory (needs a GB300)."""

import pytest
import torch

from test_gpu_attention import BF16, FP16, Step, check_attention, eg  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [
    dict(heads=4, kv_heads=2, dim=64, page=16, new=[1], total=[513]),  # clusters of 8
    dict(dtype=FP16, heads=8, kv_heads=2, dim=128, page=16, new=[1, 1, 1], total=[500, 70, 1000]),
    dict(heads=32, kv_heads=8, dim=128, page=64, new=[1, 1, 1, 1], total=[2000, 3, 1900, 64]),  # clusters of 4
])
def test_calls_back_to_back(eg, shape):  # noqa: F811
    st = Step(eg, seed=17, **{"dtype": BF16, **shape})
    ref, _ = check_attention(eg, st)
    cfg = eg.make_attn_config(st.heads, st.kv_heads, st.dim, dtype=st.dtype, rope_dim=0)
    assert eg.engram_paged_attention_workspace_bytes(cfg, st.cache, st.batch) == 0
    outs = [torch.empty_like(ref) for _ in range(300)]
    for out in outs:
        eg.engram_paged_attention(cfg, st.cache, st.batch, st.q, out=out)
    assert eg.engram_last_error() == 0
    assert all(torch.equal(out, ref) for out in outs)
