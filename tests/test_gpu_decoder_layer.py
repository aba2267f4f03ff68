"""The decoder-layer example: Engram read, cache append and paged attention together (needs a GB300)."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("prompts, heads, kv_heads, dim", [
    ((300, 17, 1000, 64), 8, 2, 128),
    ((5, 1), 6, 2, 64),
])
def test_decoding_equals_the_whole_prompt(prompts, heads, kv_heads, dim):
    """The residual of a decoded token and of the same token inside one long prompt.  Both round the same
    values to bf16 (u = 2^-8) at the same places: rmsnorm output, packed projection, heads, attention output,
    projection, residual.  What differs is the order of fp32 sums and the attention's rounded weights, so one
    value may round to its neighbour at each of these places: a few units of its size, h of about 1 to 4."""
    if not torch.cuda.is_available():
        pytest.fail("GPU test collected on a machine without CUDA")
    import decoder_layer

    decoded, whole = decoder_layer.run(prompts=prompts, steps=6, heads=heads, kv_heads=kv_heads, dim=dim)
    a, b = decoded.double(), whole.double()
    assert torch.isfinite(a).all()
    assert ((a - b).abs() <= 4e-2 * b.abs().clamp(min=1.0)).all()
