"""Tensors of the attention step on different GPUs are refused, without a GPU."""

import pytest
import torch

from attention_far import Far


@pytest.fixture(scope="module")
def eg():
    import engram_gram_hash_gb300 as eg

    eg.build()
    eg.lib()
    return eg


def _pages(device):
    return Far(torch.zeros((2, 16, 2, 128), dtype=torch.bfloat16), device)


def _batch(eg, *devices):
    offs, length = torch.tensor([0, 3]), torch.tensor([3], dtype=torch.int32)
    table = torch.zeros((1, 2), dtype=torch.int32)
    return eg.kv_batch(*(Far(t, d) for t, d in zip((offs, length, table), devices)), 3)


def test_descriptions_on_one_device(eg):
    eg.kv_cache(_pages("cuda:1"), _pages("cuda:1"))
    with pytest.raises(ValueError, match="one device"):
        eg.kv_cache(_pages("cuda:0"), _pages("cuda:1"))
    _batch(eg, "cuda:1", "cuda:1", "cuda:1")
    for devices in (("cuda:1", "cuda:0", "cuda:0"), ("cuda:0", "cuda:1", "cuda:0"), ("cuda:0", "cuda:0", "cuda:1")):
        with pytest.raises(ValueError, match="one device"):
            _batch(eg, *devices)


def test_calls_on_one_device(eg):
    cfg, table = eg.make_attn_config(8, 2, 128), Far(torch.zeros((10, 128)), "cuda:0")
    q, k = (Far(torch.zeros((3, h, 128), dtype=torch.bfloat16), "cuda:0") for h in (8, 2))
    far_q, far_k = Far(q), Far(k)
    near, far = eg.kv_cache(_pages("cuda:0"), _pages("cuda:0")), eg.kv_cache(_pages("cuda:1"), _pages("cuda:1"))
    batch, far_batch = _batch(eg, *["cuda:0"] * 3), _batch(eg, *["cuda:1"] * 3)
    for call in (
        lambda: eg.engram_paged_attention(cfg, far, batch, q),
        lambda: eg.engram_paged_attention(cfg, near, far_batch, q),
        lambda: eg.engram_paged_attention(cfg, far, far_batch, q),
        lambda: eg.engram_paged_attention(cfg, near, batch, far_q),
        lambda: eg.engram_kv_append(cfg, far, batch, k, k, table),
        lambda: eg.engram_kv_append(cfg, near, far_batch, k, k, table),
        lambda: eg.engram_kv_append(cfg, near, batch, far_k, k, table),
        lambda: eg.engram_kv_append(cfg, near, batch, k, far_k, table),
        lambda: eg.engram_kv_append(cfg, near, batch, k, k, table, q=far_q),
        lambda: eg.engram_qk_norm_rope(cfg, q, far_k, None, table),
    ):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
