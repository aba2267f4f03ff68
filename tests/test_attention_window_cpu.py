"""Sliding windows of the attention entry points without a GPU: a window that reaches past the block table's room is
plain causal attention, with the same workspace, up to the largest window there is."""

import ctypes

import pytest

A = 4096  # an aligned stand-in address, never dereferenced
LARGEST = (1 << 31) - 1


@pytest.fixture(scope="module")
def eg():
    import engram_gram_hash_gb300 as eg

    eg.build()
    eg.lib()
    return eg


# heads, kv heads, head_dim, sequences, new tokens, table entries (pages of 64): every way of sharing keys out
SHAPES = [
    (8, 2, 128, 1, 2048, 1024), (32, 8, 128, 1, 256, 64), (32, 4, 64, 1, 4096, 512), (32, 8, 128, 64, 64, 256),
    (8, 2, 64, 1, 1, 2048), (8, 2, 128, 1, 1, 8), (8, 2, 128, 3, 3, 1), (128, 1, 128, 5, 700, 1 << 20),
    (8, 2, 128, 5, 5, 1 << 25),  # more room than any position
]


@pytest.mark.parametrize("shape", SHAPES)
def test_windows_past_the_room_are_causal(eg, shape):
    heads, kv_heads, dim, seqs, new, pages = shape
    cache = eg.engram_kv_cache(A, A, 10, 64, 64 * kv_heads * dim, kv_heads * dim, dim)
    batch = eg.engram_kv_batch(seqs, new, A, A, A, pages)

    def size(window):
        cfg = eg.make_attn_config(heads, kv_heads, dim, window=window)
        return eg.lib().engram_paged_attention_workspace_bytes(*(ctypes.byref(x) for x in (cfg, cache, batch)))

    causal, room = size(0), min(pages * 64, LARGEST)
    windows = {room, max(room, LARGEST // 2), LARGEST - 256, LARGEST - 255, LARGEST - 254, LARGEST - 1, LARGEST}
    assert {w: size(w) for w in windows if w >= room} == {w: causal for w in windows if w >= room}
