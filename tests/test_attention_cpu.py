"""The attention entry points without a GPU: every bad argument is refused
before any device work, empty batches are no-ops, the binding checks its
tensors."""

import ctypes
import math

import pytest
import torch

P = ctypes.c_void_p
A = 4096  # an aligned stand-in address, never dereferenced


@pytest.fixture(scope="module")
def eg():
    import engram_gram_hash_gb300 as eg

    eg.build()
    eg.lib()
    return eg


def _cfg(eg, **kw):
    c = eg.make_attn_config(8, 2, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _heads(eg, data=A, ts=1024, hs=128):
    return eg.engram_heads(data, ts, hs)


def _cache(eg, **kw):
    c = eg.engram_kv_cache(A, A, 10, 64, 64 * 256, 256, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _batch(eg, **kw):
    b = eg.engram_kv_batch(2, 5, A, A, A, 4)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def _ref(x):
    return None if x is None else ctypes.byref(x)


def qk(eg, cfg=None, n=5, q=True, k=True, pos=A, table=A, rows=100, w=A, qo=True, ko=True):
    h = _heads(eg)
    pick = lambda x: h if x is True else x  # noqa: E731
    return eg.lib().engram_qk_norm_rope(_ref(cfg or _cfg(eg)), n, _ref(pick(q)), _ref(pick(k)), P(pos), P(table), rows,
                                        P(w), P(w), _ref(pick(qo)), _ref(pick(ko)), None)


def append(eg, cfg=None, cache=None, batch=None, k=True, v=True, w=A, table=A, rows=100, q=True, qo=True):
    h = _heads(eg)
    pick = lambda x: h if x is True else x  # noqa: E731
    return eg.lib().engram_kv_append(_ref(cfg or _cfg(eg)), _ref(cache or _cache(eg)), _ref(batch or _batch(eg)),
                                     _ref(pick(k)), _ref(pick(v)), P(w), P(table), rows, _ref(pick(q)), P(w),
                                     _ref(pick(qo)), None)


def attend(eg, cfg=None, cache=None, batch=None, q=True, out=True, lse=A, ws=A, ws_bytes=1 << 40):
    h = _heads(eg)
    pick = lambda x: h if x is True else x  # noqa: E731
    return eg.lib().engram_paged_attention(_ref(cfg or _cfg(eg)), _ref(cache or _cache(eg)), _ref(batch or _batch(eg)),
                                           _ref(pick(q)), _ref(pick(out)), P(lse), P(ws), ws_bytes, None)


BAD_CONFIGS = [
    dict(n_heads=0), dict(n_heads=9), dict(n_kv_heads=0), dict(n_kv_heads=-2), dict(n_heads=258),
    dict(head_dim=0), dict(head_dim=4), dict(head_dim=136), dict(head_dim=100),
    dict(rope_dim=-16), dict(rope_dim=24), dict(rope_dim=144), dict(rope_layout=2), dict(dtype=2),
    dict(norm_eps=-1.0), dict(norm_eps=math.nan), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf),
    dict(scale=math.nan), dict(window=-1),
]


@pytest.mark.parametrize("bad", BAD_CONFIGS)
def test_bad_configs(eg, bad):
    c = _cfg(eg, **bad)
    assert qk(eg, cfg=c) == 1 and append(eg, cfg=c) == 1 and attend(eg, cfg=c) == 1
    assert eg.lib().engram_paged_attention_workspace_bytes(_ref(c), _ref(_cache(eg)), _ref(_batch(eg))) == 0


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(k=A + 8), dict(v=A + 2), dict(n_pages=0), dict(n_pages=1 << 31), dict(page_size=0),
    dict(page_size=8), dict(page_size=24), dict(page_size=65552), dict(page_stride=0), dict(page_stride=-256),
    dict(page_stride=260), dict(token_stride=64), dict(head_stride=120), dict(head_stride=132), dict(page_stride=1 << 39),
])
def test_bad_caches(eg, bad):
    c = _cache(eg, **bad)
    assert append(eg, cache=c) == 1 and attend(eg, cache=c) == 1


@pytest.mark.parametrize("bad", [
    dict(n_seqs=0), dict(n_seqs=-1), dict(n_query=-1), dict(n_query=1 << 31), dict(seq_offsets=None), dict(kv_len=None),
    dict(block_table=None), dict(table_stride=0), dict(table_stride=-4), dict(seq_offsets=A + 4), dict(kv_len=A + 2),
])
def test_bad_batches(eg, bad):
    b = _batch(eg, **bad)
    assert append(eg, batch=b) == 1 and attend(eg, batch=b) == 1


def test_bad_views_and_pointers(eg):
    for bad in (None, _heads(eg, data=None), _heads(eg, data=A + 8), _heads(eg, ts=1020), _heads(eg, hs=130)):
        assert append(eg, k=bad) == 1 and append(eg, v=bad) == 1 and append(eg, qo=bad) == 1
        assert attend(eg, q=bad) == 1 and attend(eg, out=bad) == 1
        assert qk(eg, qo=bad) == 1 and qk(eg, ko=bad) == 1
        if bad is not None:
            assert qk(eg, q=bad) == 1 and qk(eg, k=bad) == 1 and append(eg, q=bad) == 1
    assert qk(eg, pos=None) == 1 and qk(eg, table=None) == 1 and append(eg, table=None) == 1
    assert qk(eg, table=A + 8) == 1 and append(eg, table=A + 4) == 1 and qk(eg, w=A + 8) == 1 and append(eg, w=A + 2) == 1
    assert qk(eg, n=-1) == 1 and qk(eg, rows=-1) == 1 and append(eg, rows=-1) == 1
    long = _batch(eg, n_seqs=5, table_stride=1 << 20)  # needs a workspace
    assert attend(eg, lse=A + 2) == 1 and attend(eg, batch=long, ws=None) == 1 and attend(eg, batch=long, ws=A + 16) == 1
    assert attend(eg, batch=long, ws_bytes=16) == 6


def test_rows_times_group_must_fit(eg):
    assert attend(eg, batch=_batch(eg, n_query=(1 << 31) - 1)) == 1


def test_empty_calls_are_no_ops(eg):
    b = _batch(eg, n_query=0, seq_offsets=None, kv_len=None, block_table=None, table_stride=0)
    assert append(eg, batch=b, k=None, v=None) == 0
    assert attend(eg, batch=b, q=None, out=None, ws=None) == 0
    assert qk(eg, n=0, q=None, k=None) == 0 and qk(eg, q=None, k=None) == 0


def test_workspace_size(eg):
    """Follows from the descriptions; none for short block tables, bounded for the longest."""
    def size(**kw):
        return eg.lib().engram_paged_attention_workspace_bytes(_ref(_cfg(eg)), _ref(_cache(eg)), _ref(_batch(eg, **kw)))

    assert size(table_stride=4) == 0 and attend(eg, ws=None, ws_bytes=0, batch=_batch(eg, n_query=0)) == 0
    long = size(n_seqs=5, table_stride=1 << 20)
    assert 0 < long <= 16 << 20 and size(n_seqs=5, table_stride=1 << 24) == long
    chunk = size(n_query=2000, table_stride=1 << 20)
    assert 0 < chunk <= 256 << 20
    assert size(n_query=1 << 20, table_stride=1 << 20) == 0  # many row blocks: nothing is split
    assert size(n_query=-1) == 0 and size(n_query=0) == 0


def test_binding_checks(eg):
    with pytest.raises(TypeError):
        eg.make_attn_config(8, 2, 128, dtype=torch.float32)
    cfg = eg.make_attn_config(8, 2, 128)
    assert abs(cfg.scale - 128**-0.5) < 1e-7 and cfg.rope_dim == 128
    pages = torch.zeros((2, 16, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        eg.kv_cache(pages, pages)  # not on the GPU
    with pytest.raises(TypeError):
        eg.kv_cache(pages.float(), pages)
    q = torch.zeros((3, 8, 128), dtype=torch.bfloat16)
    table = torch.zeros((10, 128))
    pos = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        eg.engram_qk_norm_rope(cfg, q, None, pos, table)  # not on the GPU
    with pytest.raises(TypeError):
        eg.engram_qk_norm_rope(cfg, q.float(), None, pos, table)
    with pytest.raises(ValueError):
        eg.engram_qk_norm_rope(cfg, q[:, :4], None, pos, table)
    with pytest.raises(ValueError):
        eg.engram_qk_norm_rope(cfg, None, None, pos, table)
    with pytest.raises(TypeError):
        eg.engram_qk_norm_rope(cfg, [1.0], None, pos, table)


def test_rope_table(eg):
    t = eg.rope_table(7, 32, theta=100.0, device="cpu")
    assert t.shape == (7, 32) and t.dtype == torch.float32
    for p in range(7):
        for i in range(16):
            a = p * 100.0 ** (-i / 16)
            assert abs(t[p, i].item() - math.cos(a)) < 1e-7 and abs(t[p, 16 + i].item() - math.sin(a)) < 1e-7
