"""Paged attention by the way its keys are shared out, each case with the kernels that it is meant for: more than 32
sequences cut into runs and joined, infinities through cuts and joins, windows over long chunks and pages of 256
(needs a GB300)."""

import ctypes
import re

import pytest
import torch

import test_gpu_attention as base
from test_gpu_attention import BF16, FP16, Step, check_attention, eg  # noqa: F401

pytestmark = pytest.mark.gpu

ROWS, CUT = {"rows_kernel"}, {"rows_kernel", "rows_join_kernel"}
TILES, SPLIT = {"tile_kernel"}, {"tile_kernel", "tile_join_kernel"}


def kernels(eg, st, tmp_path, window=0):  # noqa: F811
    """The attention kernels that a call on this step launches, from the call's CUDA graph."""
    cfg = eg.make_attn_config(st.heads, st.kv_heads, st.dim, dtype=st.dtype, rope_dim=0, window=window)
    out = torch.empty((sum(st.new), st.heads, st.dim), dtype=st.dtype, device="cuda")
    n = eg.engram_paged_attention_workspace_bytes(cfg, st.cache, st.batch)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    eg.engram_paged_attention(cfg, st.cache, st.batch, st.q, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        eg.engram_paged_attention(cfg, st.cache, st.batch, st.q, out=out, workspace=ws)
    dot = str(tmp_path / "graph.dot").encode()
    assert ctypes.CDLL("libcudart.so.13").cudaGraphDebugDotPrint(ctypes.c_void_p(graph.raw_cuda_graph()), dot, 0) == 0
    return set(re.findall(r"(?:rows|tile)_(?:join_)?kernel", (tmp_path / "graph.dot").read_text()))


def _lengths(n, most):
    """Unequal lengths, 1 and the longest among them."""
    return [1, most] + [1 + (i * 7919) % most for i in range(n - 2)]


MANY = {
    "33": (CUT, dict(heads=8, kv_heads=2, dim=128, page=64, new=[1] * 33, total=_lengths(33, 4000))),
    "64": (CUT, dict(heads=32, kv_heads=8, dim=128, page=64, new=[1] * 64, total=_lengths(64, 3000))),
    "70_64": (CUT, dict(dtype=FP16, heads=4, kv_heads=4, dim=64, page=16, new=[1] * 70, total=_lengths(70, 6000))),
    "40_72": (CUT, dict(heads=6, kv_heads=2, dim=72, page=48, new=[i % 3 for i in range(40)],
                        total=[max(t, i % 3) for i, t in enumerate(_lengths(40, 5000))])),
    "400": (CUT, dict(heads=2, kv_heads=1, dim=64, page=32, new=[1] * 400, total=_lengths(400, 2500))),
}


@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("name", MANY)
def test_many_sequences_cut(eg, name, order, tmp_path):  # noqa: F811
    path, c = MANY[name]
    st = Step(eg, order=order, seed=len(name), **{"dtype": BF16, **c})
    assert kernels(eg, st, tmp_path) == path
    check_attention(eg, st)


@pytest.mark.parametrize("window", [100, 2000])
@pytest.mark.parametrize("name", ["33", "40_72"])
def test_many_sequences_window(eg, name, window, tmp_path):  # noqa: F811
    st = Step(eg, seed=window, **{"dtype": BF16, **MANY[name][1]})
    assert kernels(eg, st, tmp_path, window) == (CUT if window == 2000 else ROWS)
    check_attention(eg, st, window=window)


INFINITE = {
    "whole": (ROWS, dict(dtype=BF16, heads=8, kv_heads=2, dim=128, page=64, new=[40, 1, 130], total=[100, 70, 500])),
    "cluster": (ROWS, dict(dtype=FP16, heads=4, kv_heads=4, dim=128, page=32, new=[5, 1], total=[700, 1900])),
    "cut": (CUT, dict(dtype=FP16, heads=4, kv_heads=4, dim=128, page=32, new=[5, 1, 2], total=[700, 9000, 2])),
    "cut_33": (CUT, dict(dtype=BF16, heads=8, kv_heads=2, dim=64, page=64, new=[2] * 33,
                         total=[max(2, t) for t in _lengths(33, 5000)])),
    "split": (SPLIT, dict(dtype=BF16, heads=64, kv_heads=1, dim=128, page=64, new=[50, 3], total=[6000, 100])),
    "split_40": (SPLIT, dict(dtype=FP16, heads=64, kv_heads=1, dim=64, page=64, new=[9] * 40,
                             total=[max(9, t) for t in _lengths(40, 6000)])),
}


@pytest.mark.parametrize("window", [0, 1000])
@pytest.mark.parametrize("name", INFINITE)
def test_infinities_stay_with_the_rows_that_see_them(eg, name, window, tmp_path):  # noqa: F811
    path, c = INFINITE[name]
    if window == 0:
        assert kernels(eg, Step(eg, seed=21, **c), tmp_path) == path
    base.test_attention_infinities_stay_with_the_rows_that_see_them(eg, c, window)


CHUNKS = {
    "chunk": dict(heads=64, kv_heads=1, dim=128, page=64, new=[300], total=[9001]),
    "chunk_64": dict(heads=64, kv_heads=1, dim=64, page=256, new=[300, 200], total=[6000, 777]),
    "chunk_256": dict(dtype=FP16, heads=32, kv_heads=1, dim=128, page=256, new=[300, 200], total=[6000, 777]),
}


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 128, 129, 300, 1000, 5000])
@pytest.mark.parametrize("name", CHUNKS)
def test_chunks_window(eg, name, window, tmp_path):  # noqa: F811
    st = Step(eg, seed=window, **{"dtype": BF16, **CHUNKS[name]})
    assert kernels(eg, st, tmp_path, window) == (TILES if window <= 300 else SPLIT)
    check_attention(eg, st, window=window)


@pytest.mark.parametrize("name", CHUNKS)
def test_chunks(eg, name, tmp_path):  # noqa: F811
    st = Step(eg, seed=1, **{"dtype": BF16, **CHUNKS[name]})
    assert kernels(eg, st, tmp_path) == SPLIT
    check_attention(eg, st)
