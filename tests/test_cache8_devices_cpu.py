"""Tensors of the 8-bit cache's calls on different GPUs are refused, without a GPU."""

import pytest
import torch

from attention_far import Far

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def eg():
    import engram_gram_hash_gb300 as eg

    eg.build()
    eg.lib()
    return eg


def _cache(eg, *devices):
    codes = torch.zeros((2, 16, 2, 128), dtype=torch.uint8).view(E4M3)
    scales = torch.ones((2, 2, 1))
    return eg.kv_cache_q8(*(Far(t, d) for t, d in zip((codes, codes, scales, scales), devices)))


def _batch(eg, device):
    offs, length = torch.tensor([0, 3]), torch.tensor([3], dtype=torch.int32)
    table = torch.zeros((1, 2), dtype=torch.int32)
    return eg.kv_batch(*(Far(t, device) for t in (offs, length, table)), 3)


def test_caches_on_one_device(eg):
    _cache(eg, *["cuda:1"] * 4)
    for i in range(4):
        devices = ["cuda:0"] * 4
        devices[i] = "cuda:1"
        with pytest.raises(ValueError, match="one device"):
            _cache(eg, *devices)


def test_cache_shapes(eg):
    codes, scales = torch.zeros((4, 64, 2, 64), dtype=torch.uint8).view(E4M3), torch.ones((4, 2, 2))
    far = lambda t: Far(t, "cuda:0")  # noqa: E731
    c = eg.kv_cache_q8(far(codes), far(codes), far(scales), far(scales))
    assert (c.n_pages, c.page_size, c.block_tokens) == (4, 64, 32)
    assert (c.page_stride, c.token_stride, c.head_stride) == (64 * 128, 128, 64)
    for bad in (torch.ones((4, 2, 3)), torch.ones((3, 2, 2)), torch.ones((4, 1, 2)), torch.ones((4, 2)), torch.ones((4, 2, 0))):
        with pytest.raises(ValueError, match="scales"):
            eg.kv_cache_q8(far(codes), far(codes), far(bad), far(bad))
    with pytest.raises(ValueError, match="blocks of 16"):  # 8 tokens a block
        eg.kv_cache_q8(far(codes), far(codes), far(torch.ones((4, 2, 8))), far(torch.ones((4, 2, 8))))
    with pytest.raises(ValueError, match="alike"):
        eg.kv_cache_q8(far(codes), far(codes), far(scales), far(torch.ones((4, 2, 4))))
    with pytest.raises(ValueError, match="shape and strides"):
        eg.kv_cache_q8(far(codes), far(codes[:3]), far(scales), far(scales))
    with pytest.raises(TypeError, match="float32"):
        eg.kv_cache_q8(far(codes), far(codes), far(scales.double()), far(scales))


def test_calls_on_one_device(eg):
    cfg, table = eg.make_attn_config(8, 2, 128), Far(torch.zeros((10, 128)), "cuda:0")
    q, k = (Far(torch.zeros((3, h, 128), dtype=torch.bfloat16), "cuda:0") for h in (8, 2))
    far_q, far_k = Far(q), Far(k)
    near, far = _cache(eg, *["cuda:0"] * 4), _cache(eg, *["cuda:1"] * 4)
    batch, far_batch = _batch(eg, "cuda:0"), _batch(eg, "cuda:1")
    for call in (
        lambda: eg.engram_paged_attention_q8(cfg, far, batch, q),
        lambda: eg.engram_paged_attention_q8(cfg, near, far_batch, q),
        lambda: eg.engram_paged_attention_q8(cfg, far, far_batch, q),
        lambda: eg.engram_paged_attention_q8(cfg, near, batch, far_q),
        lambda: eg.engram_kv_append_q8(cfg, far, batch, k, k, table),
        lambda: eg.engram_kv_append_q8(cfg, near, far_batch, k, k, table),
        lambda: eg.engram_kv_append_q8(cfg, near, batch, far_k, k, table),
        lambda: eg.engram_kv_append_q8(cfg, near, batch, k, far_k, table),
        lambda: eg.engram_kv_append_q8(cfg, near, batch, k, k, table, q=far_q),
    ):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
