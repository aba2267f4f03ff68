"""Sequences as long as 32-bit lengths allow: one page of 65,536 tokens stands in every entry of the table, and a window
keeps the work small (needs a GB300)."""

import pytest
import torch

import attention_plain as plain
from test_gpu_attention import BF16, eg  # noqa: F401

pytestmark = pytest.mark.gpu

PAGE, LONGEST = 65536, (1 << 31) - 1024


@pytest.mark.parametrize("heads", [4, 128])  # few rows, tiles
@pytest.mark.parametrize("dim", [16, 72])
def test_longest_sequences(eg, heads, dim):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(dim)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(BF16)

    new, window = 10, 64
    k, v, q = randn(1, PAGE, 1, dim), randn(1, PAGE, 1, dim), randn(new, heads, dim)
    cfg = eg.make_attn_config(heads, 1, dim, rope_dim=0, window=window)
    cache, offs = eg.kv_cache(k, v), torch.tensor([0, new], device="cuda")
    table = torch.zeros((1, (LONGEST + 1024) // PAGE), dtype=torch.int32, device="cuda")

    def run(length):
        batch = eg.kv_batch(offs, torch.tensor([length], dtype=torch.int32, device="cuda"), table, new)
        return eg.engram_paged_attention(cfg, cache, batch, q)

    # the same keys are in reach of a sequence that ends at the same row of its second page
    ref, _, bound, _ = plain.attention(q, k, v, table[:, :2], [new], [PAGE + LONGEST % PAGE], 1, cfg.scale, window)
    got = run(LONGEST)
    assert eg.engram_last_error() == 0
    assert ((got.double() - ref).abs() <= bound).all()
    assert torch.equal(run(PAGE + LONGEST % PAGE), got)
    for length in (LONGEST + 1, LONGEST + 1023):  # flagged and cut
        cut = run(length)
        assert eg.engram_last_error() == 3
        assert torch.equal(cut, got)
