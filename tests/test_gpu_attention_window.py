"""Sliding windows that hide nothing, up to the largest there is, through every way the attention kernels share keys out
(needs a GB300)."""

import pytest
import torch

import test_gpu_attention as base
from test_gpu_attention import BF16, FP16, Step, check_attention, eg  # noqa: F401

pytestmark = pytest.mark.gpu

LARGEST = (1 << 31) - 1

SHAPES = {
    "few_rows_cluster": dict(heads=8, kv_heads=2, dim=128, page=64, new=[1], total=[700]),
    "few_rows_whole": dict(dtype=FP16, heads=12, kv_heads=2, dim=96, page=48, new=[5, 1, 30], total=[333, 200, 30]),
    "few_rows_cut": dict(heads=8, kv_heads=2, dim=128, page=128, new=[1], total=[20011]),
    "few_rows_cut_padded": dict(heads=8, kv_heads=2, dim=64, page=32, new=[1, 5], total=[9000, 2]),
    "tiles": dict(heads=64, kv_heads=1, dim=64, page=16, new=[90, 3, 2, 1], total=[40, 2, 70, 0]),
    "tiles_split": dict(heads=64, kv_heads=1, dim=128, page=16, new=[90, 1, 40], total=[500, 70, 5000]),
}


@pytest.mark.parametrize("name", SHAPES)
def test_windows_past_the_room_are_causal(eg, name):  # noqa: F811
    """The bits of the plain causal call."""
    st = Step(eg, seed=len(name), **{"dtype": BF16, **SHAPES[name]})
    ref, ref_lse = check_attention(eg, st)
    room = st.block_table.shape[1] * st.page
    for window in (room, room + 1, LARGEST - 256, LARGEST - 255, LARGEST - 1, LARGEST):
        cfg = eg.make_attn_config(st.heads, st.kv_heads, st.dim, dtype=st.dtype, rope_dim=0, window=window)
        lse = torch.empty_like(ref_lse)
        out = eg.engram_paged_attention(cfg, st.cache, st.batch, st.q, lse=lse)
        assert eg.engram_last_error() == 0
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse), window


@pytest.mark.parametrize("heads", [4, 128])  # few rows, tiles
@pytest.mark.parametrize("dim", [8, 72])
def test_largest_windows_under_the_widest_table(eg, heads, dim):  # noqa: F811
    """A table with room for every position keeps the window as it is; tokens before the sequence's start (position
    minus window far below zero) see nothing, the others what they see without a window."""
    st = Step(eg, BF16, heads, 1, dim, 65536, [10, 3], [6, 3], seed=3)
    wide = torch.full((2, 32769), -7, dtype=torch.int32, device="cuda")
    wide[:, :1] = st.block_table[:, :1]
    st.block_table = wide
    st.batch = eg.kv_batch(st.seq_offsets, st.kv_len, wide, sum(st.new))
    for window in (LARGEST - 1, LARGEST - 9):
        check_attention(eg, st, window=window)
