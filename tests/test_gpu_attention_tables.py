"""Block tables that are slices of wider ones: what lies beside the slice is not the sequences' (needs a GB300)."""

import pytest
import torch

from test_gpu_attention import BF16, Step, check_attention, eg  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = {
    "few_rows": dict(heads=8, kv_heads=2, dim=128, page=16, new=[1, 1], total=[160, 100]),
    "few_rows_cut": dict(heads=8, kv_heads=2, dim=64, page=16, new=[1, 2], total=[8000, 30]),
    "tiles": dict(heads=64, kv_heads=1, dim=64, page=16, new=[60, 70], total=[160, 100]),
    "tiles_split": dict(heads=64, kv_heads=1, dim=128, page=16, new=[60, 70], total=[4000, 100]),
}


def _sliced(eg, st, at=3, right=5):  # noqa: F811
    """The step's table as columns [at, at + width) of a wider one, whose other columns name pages as well."""
    width = -(-st.total[0] // st.page)
    wide = torch.zeros((len(st.new), at + width + right), dtype=torch.int32, device="cuda")
    wide[:, at:at + width] = st.block_table[:, :width].clamp(min=0)
    st.block_table = wide[:, at:at + width]
    st.batch = eg.kv_batch(st.seq_offsets, st.kv_len, st.block_table, sum(st.new))
    return width


@pytest.mark.parametrize("name", SHAPES)
def test_attention_over_a_sliced_table(eg, name):  # noqa: F811
    """The values of the whole table; a length past the slice is flagged and cut there, as past any table."""
    st = Step(eg, BF16, seed=4, **SHAPES[name])
    width = _sliced(eg, st)
    good, _ = check_attention(eg, st)
    cfg = eg.make_attn_config(st.heads, st.kv_heads, st.dim, rope_dim=0)
    st.kv_len[0] = width * st.page
    full = eg.engram_paged_attention(cfg, st.cache, st.batch, st.q)
    assert eg.engram_last_error() == 0
    st.kv_len[0] = width * st.page + 3
    cut = eg.engram_paged_attention(cfg, st.cache, st.batch, st.q)
    assert eg.engram_last_error() == 3
    assert torch.equal(cut, full)
    st.kv_len[0] = st.total[0]
    assert torch.equal(eg.engram_paged_attention(cfg, st.cache, st.batch, st.q), good)


def test_append_under_a_sliced_table(eg):  # noqa: F811
    """A position past the slice is flagged and written nowhere."""
    st = Step(eg, BF16, 4, 2, 64, 16, [1, 1], [64, 20], seed=4)
    width = _sliced(eg, st)
    st.k_pages.zero_()
    st.v_pages.zero_()
    cfg, table = eg.make_attn_config(4, 2, 64), eg.rope_table(100, 64)
    st.kv_len[:] = torch.tensor([width * 16 + 1, width * 16], dtype=torch.int32)
    eg.engram_kv_append(cfg, st.cache, st.batch, st.k, st.v, table)
    assert eg.engram_last_error() == 3
    page = st.block_table[1, width - 1].item()
    assert st.v_pages.flatten(1).any(1).nonzero().flatten().tolist() == [page]
    assert torch.equal(st.v_pages[page, 15], st.v[1])


def test_choice_follows_the_slice(eg):  # noqa: F811
    """The workspace, and with it how the keys are shared out, is that of the slice's own width."""
    st = Step(eg, BF16, 8, 2, 128, 16, [1, 1], [160, 100], seed=4)
    cfg = eg.make_attn_config(8, 2, 128, rope_dim=0)
    wide = torch.zeros((2, 4096), dtype=torch.int32, device="cuda")
    size = [eg.engram_paged_attention_workspace_bytes(cfg, st.cache, eg.kv_batch(st.seq_offsets, st.kv_len, t, 2))
            for t in (wide, wide[:, :10], wide[:, :10].contiguous())]
    assert size[0] > 0 and size[1] == size[2] == 0
