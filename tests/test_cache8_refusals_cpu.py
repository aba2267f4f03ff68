"""Appends to the 8-bit cache that are refused before anything is launched (CPU)."""

import pytest

from test_cache8_cpu import EINVAL, Args, eg  # noqa: F401


@pytest.mark.parametrize("heads,tokens", [(65536, 1 << 22), (65536, 1 << 21), (32768, 1 << 23)])
def test_more_blocks_than_a_grid(eg, heads, tokens):  # noqa: F811
    """A step whose keys and values need more CTAs than a launch may have is refused whole: its queries, which would go in a
    launch of their own, are not written either (without a GPU that launch would answer ECUDA)."""
    a = Args(eg)
    a.cfg = eg.make_attn_config(heads, heads, 16)
    a.cache.block_tokens, a.cache.page_stride, a.cache.token_stride, a.cache.head_stride = 16, 64 * heads * 16, heads * 16, 16
    a.batch.n_query = tokens
    assert a.append(q=a.heads, q_out=a.heads) == EINVAL
    assert a.append() == EINVAL
