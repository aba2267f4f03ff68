"""The 8-bit cache's calls: structures, exports and refusals (CPU; nothing is launched)."""

import ctypes
import re

import pytest
import torch

EINVAL, ENOMEM = 1, 6
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def eg():
    import engram_gram_hash_gb300 as eg

    eg.build()
    eg.lib()
    return eg


class Args:
    """Descriptions over addresses that are never followed: the checks come before any launch."""

    def __init__(self, eg):
        self.eg = eg
        self.cfg = eg.make_attn_config(8, 2, 128)
        c = self.cache = eg.engram_kv_cache_q8()
        c.k = c.v = c.k_scales = c.v_scales = 4096
        c.n_pages, c.page_size, c.block_tokens = 10, 64, 32
        c.page_stride, c.token_stride, c.head_stride = 64 * 256, 256, 128
        b = self.batch = eg.engram_kv_batch()
        b.n_seqs, b.n_query, b.seq_offsets, b.kv_len, b.block_table, b.table_stride = 2, 3, 4096, 4096, 4096, 5
        h = self.heads = eg.engram_heads()
        h.data, h.token_stride, h.head_stride = 4096, 1024, 128

    def append(self, **kw):
        a = dict(cfg=self.cfg, cache=self.cache, batch=self.batch, k=self.heads, v=self.heads, w_k=None, table=4096,
                 rows=100, q=None, w_q=None, q_out=None)
        a.update(kw)
        r = lambda x: ctypes.byref(x) if isinstance(x, ctypes.Structure) else x  # noqa: E731
        return self.eg.lib().engram_kv_append_q8(*[r(x) for x in a.values()], None)

    def attend(self, **kw):
        a = dict(cfg=self.cfg, cache=self.cache, batch=self.batch, q=self.heads, out=self.heads, lse=None, ws=None, bytes=0)
        a.update(kw)
        r = lambda x: ctypes.byref(x) if isinstance(x, ctypes.Structure) else x  # noqa: E731
        return self.eg.lib().engram_paged_attention_q8(*[r(x) for x in a.values()], None)


@pytest.mark.parametrize("field,values", [
    ("k", [0, 4104]), ("v", [0, 8]), ("k_scales", [0, 4098]), ("v_scales", [0, 4097]), ("n_pages", [0, -1, 1 << 31]),
    ("page_size", [0, 8, 24, 65552, 48]), ("block_tokens", [0, 8, 48, 128, 256]), ("page_stride", [0, -16, 24, 64]),
    ("token_stride", [8, 250, 64]), ("head_stride", [0, 120, 64, 1 << 40]),
])
def test_caches_refused(eg, field, values):
    for x in values:
        a = Args(eg)
        setattr(a.cache, field, x)
        assert a.append() == EINVAL and a.attend() == EINVAL, (field, x)
        assert eg.engram_paged_attention_q8_workspace_bytes(a.cfg, a.cache, a.batch) == 0


@pytest.mark.parametrize("field,value", [("head_dim", 120), ("head_dim", 136), ("n_heads", 7), ("dtype", 2), ("rope_dim", 8),
                                         ("scale", 0.0), ("window", -1)])
def test_configurations_refused(eg, field, value):
    a = Args(eg)
    setattr(a.cfg, field, value)
    assert a.append() == EINVAL and a.attend() == EINVAL


@pytest.mark.parametrize("field,value", [("n_seqs", 0), ("n_seqs", -1), ("n_query", -1), ("seq_offsets", 0), ("kv_len", 2),
                                         ("block_table", 0), ("table_stride", 0), ("table_width", 6)])
def test_batches_refused(eg, field, value):
    a = Args(eg)
    setattr(a.batch, field, value)
    assert a.append() == EINVAL and a.attend() == EINVAL


def test_heads_and_pointers_refused(eg):
    a = Args(eg)
    for field, value in (("data", 0), ("data", 4104), ("token_stride", 4), ("head_stride", 12)):
        h = a.eg.engram_heads(4096, 1024, 128)
        setattr(h, field, value)
        assert a.append(k=h) == EINVAL and a.append(v=h) == EINVAL and a.append(q=h, q_out=a.heads) == EINVAL
        assert a.append(q=a.heads, q_out=h) == EINVAL and a.attend(q=h) == EINVAL and a.attend(out=h) == EINVAL
    assert a.append(k=None) == EINVAL and a.append(v=None) == EINVAL and a.append(q=a.heads) == EINVAL
    assert a.append(table=None) == EINVAL and a.append(table=4100) == EINVAL and a.append(rows=-1) == EINVAL
    assert a.append(w_k=4100) == EINVAL and a.append(w_q=4100) == EINVAL
    assert a.append(cfg=None) == EINVAL and a.append(cache=None) == EINVAL and a.append(batch=None) == EINVAL
    assert a.attend(q=None) == EINVAL and a.attend(out=None) == EINVAL and a.attend(lse=4098) == EINVAL


def test_workspace_refused(eg):
    a = Args(eg)
    a.batch.table_stride, a.batch.n_seqs, a.batch.n_query = 4000, 100, 100
    need = eg.engram_paged_attention_q8_workspace_bytes(a.cfg, a.cache, a.batch)
    assert need > 0
    assert a.attend(ws=4096, bytes=need - 1) == ENOMEM and a.attend(ws=None, bytes=need) == EINVAL
    assert a.attend(ws=4100, bytes=need) == EINVAL


def test_empty_steps(eg):
    a = Args(eg)
    a.batch.n_query = 0
    assert a.append() == 0 and a.attend() == 0


def test_structures_match_the_header(eg):
    import os

    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "engram.h")) as f:
        header = f.read()
    body = re.search(r"typedef struct \{([^}]*)\} engram_kv_cache_q8;", header).group(1)
    names = re.findall(r"(\w+);", re.sub(r"/\*.*?\*/", "", body, flags=re.S))
    assert names == [n for n, _ in eg.engram_kv_cache_q8._fields_]


def _cache_tensors(dtype=E4M3, pages=4, size=64, heads=2, dim=64, blocks=2):
    x = torch.zeros((pages, size, heads, dim), dtype=torch.uint8).view(dtype)
    return x, x.clone(), torch.ones((pages, heads, blocks)), torch.ones((pages, heads, blocks))


def test_python_caches_refused(eg):
    k, v, ks, vs = _cache_tensors()
    with pytest.raises(ValueError, match="CUDA"):
        eg.kv_cache_q8(k, v, ks, vs)
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        eg.kv_cache_q8(k.view(torch.uint8), v, ks, vs)
    with pytest.raises(ValueError, match="contiguous heads"):
        eg.kv_cache_q8(k.transpose(2, 3), v, ks, vs)


@pytest.mark.parametrize("call", ["engram_kv_append_q8", "engram_paged_attention_q8"])
def test_python_wrong_caches(eg, call):
    a = Args(eg)
    other = eg.engram_kv_cache()
    other.heads_dim, other.torch_dtype, other.device_index = (2, 128), torch.bfloat16, 0
    args = [None] * (3 if call == "engram_kv_append_q8" else 1)
    with pytest.raises(ValueError, match="kv_cache_q8"):
        getattr(eg, call)(a.cfg, other, a.batch, *args)
    a.cache.heads_dim, a.cache.torch_dtype, a.cache.device_index = (2, 64), E4M3, 0
    with pytest.raises(ValueError, match="heads"):
        getattr(eg, call)(a.cfg, a.cache, a.batch, *args)
    a.cache.heads_dim = (2, 128)
    a.batch.device_index = 0
    with pytest.raises(ValueError):  # the 16-bit calls do not take it
        eg.engram_paged_attention(a.cfg, a.cache, a.batch, None)


def test_plan_refusals(eg):
    i = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    good = dict(new_len=i(1, 2), kv_len=i(3, 4), block_table=torch.zeros((2, 3), dtype=torch.int32), free_pages=i(1, 2, 3),
                n_free=i(3), page_size=16, max_tokens=3)
    with pytest.raises(ValueError, match="CUDA"):
        eg.engram_kv_plan(**good)
    for name, value, error in [("new_len", None, ValueError), ("free_pages", torch.zeros(3), TypeError),
                               ("max_tokens", -1, ValueError), ("max_tokens", 1 << 31, ValueError),
                               ("max_tokens", "x", TypeError), ("page_size", 0, ValueError), ("block_table", None, ValueError),
                               ("free_pages", 5, TypeError)]:
        with pytest.raises(error):
            eg.engram_kv_plan(**{**good, name: value})


class _PlanArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("n_seqs", "max_tokens", "n_pages")] + [("page_size", ctypes.c_int32)] + [
        (n, ctypes.c_void_p) for n in ("new_len", "keep_len", "kv_len", "kv_len_out", "block_table")] + [
        ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int64)] + [
        (n, ctypes.c_void_p) for n in ("free_pages", "n_free", "n_free_out", "seq_offsets", "positions", "slots", "counts")]


def _plan_args(**kw):
    p = _PlanArgs()
    for n, t in p._fields_:
        if t is ctypes.c_void_p:
            setattr(p, n, 4096)
    p.n_seqs, p.max_tokens, p.n_pages, p.page_size, p.table_stride, p.table_width = 2, 3, 5, 16, 4, 0
    for n, v in kw.items():
        setattr(p, n, v)
    return p


@pytest.mark.parametrize("field,value", [
    ("n_seqs", -1), ("n_seqs", 1 << 31), ("max_tokens", -1), ("max_tokens", 1 << 31), ("n_pages", 0), ("page_size", 0),
    ("page_size", 24), ("page_size", 65552), ("new_len", 0), ("new_len", 4098), ("keep_len", 4098), ("kv_len", 0),
    ("kv_len_out", 0), ("block_table", 0), ("block_table", 4097), ("table_stride", 0), ("table_width", 5),
    ("table_width", -1), ("free_pages", 0), ("n_free", 0), ("n_free_out", 0), ("seq_offsets", 0), ("seq_offsets", 4100),
    ("positions", 4098), ("slots", 4100), ("counts", 0),
])
def test_plan_arguments_refused(eg, field, value):
    assert eg.lib().engram_kv_plan(ctypes.byref(_plan_args(**{field: value})), None) == EINVAL


def test_plan_null(eg):
    assert eg.lib().engram_kv_plan(None, None) == EINVAL
