"""The block table's width among the attention entry points' arguments, without a GPU."""

import ctypes

import pytest

A = 4096  # an aligned stand-in address, never dereferenced


@pytest.fixture(scope="module")
def eg():
    import engram_gram_hash_gb300 as eg

    eg.build()
    eg.lib()
    return eg


def _size(eg, stride, width):
    cfg = eg.make_attn_config(8, 2, 128)
    cache = eg.engram_kv_cache(A, A, 10, 64, 64 * 256, 256, 128)
    batch = eg.engram_kv_batch(2, 5, A, A, A, stride, width)
    return eg.lib().engram_paged_attention_workspace_bytes(*(ctypes.byref(x) for x in (cfg, cache, batch)))


def test_width_decides(eg):
    assert _size(eg, 4, 0) == _size(eg, 4, 4) == 0
    assert _size(eg, 4096, 0) == _size(eg, 4096, 4096) > 0
    assert _size(eg, 4096, 4) == 0 and _size(eg, 4096, 1024) == _size(eg, 1024, 0)


@pytest.mark.parametrize("width", [-1, 5, 1 << 40])
def test_bad_widths(eg, width):
    cfg, heads = eg.make_attn_config(8, 2, 128), eg.engram_heads(A, 1024, 128)
    cache = eg.engram_kv_cache(A, A, 10, 64, 64 * 256, 256, 128)
    batch = eg.engram_kv_batch(2, 5, A, A, A, 4, width)
    ref = ctypes.byref
    assert eg.lib().engram_paged_attention(ref(cfg), ref(cache), ref(batch), ref(heads), ref(heads), None, A, 1 << 40, None) == 1
    assert eg.lib().engram_kv_append(ref(cfg), ref(cache), ref(batch), ref(heads), ref(heads), None, A, 100, None, None, None,
                                     None) == 1
