"""Arguments of the attention step that lie on another GPU than the call's are refused before anything is enqueued
(needs a GB300; the other GPU's tensors are stand-ins without memory)."""

import pytest
import torch

from attention_far import Far
from test_gpu_attention import BF16, Step, eg  # noqa: F401

pytestmark = pytest.mark.gpu


def test_other_devices_are_refused(eg):  # noqa: F811
    st = Step(eg, BF16, 8, 2, 128, 16, [1, 1], [30, 20], seed=13)
    cfg, table = eg.make_attn_config(8, 2, 128), eg.rope_table(64, 128)
    w, pos = torch.ones(128, device="cuda", dtype=BF16), torch.zeros(2, dtype=torch.int32, device="cuda")
    out, lse = torch.empty((2, 8, 128), dtype=BF16, device="cuda"), torch.empty((2, 8), device="cuda")
    k_out, ws = torch.empty((2, 2, 128), dtype=BF16, device="cuda"), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    calls = {
        "norm_rope": (eg.engram_qk_norm_rope, (cfg,), dict(q=st.q, k=st.k, positions=pos, table=table, w_q=w, w_k=w,
                                                           q_out=out, k_out=k_out)),
        "append": (eg.engram_kv_append, (cfg, st.cache, st.batch), dict(k=st.k, v=st.v, table=table, w_k=w, q=st.q, w_q=w,
                                                                        q_out=out)),
        "attention": (eg.engram_paged_attention, (cfg, st.cache, st.batch), dict(q=st.q, out=out, lse=lse, workspace=ws)),
    }
    for name, (call, first, args) in calls.items():
        call(*first, **args)
        for far in args:
            with pytest.raises(ValueError, match="cuda:1"):
                call(*first, **{**args, far: Far(args[far])})
                pytest.fail(f"{name}: {far} was accepted")
    assert eg.engram_last_error() == 0
