"""Block tables from request lengths, by both kernels (the maps of more than 4,096 tokens are a kernel of their own), where
something is missing: requests, tokens, outputs (needs a GB300)."""

import ctypes

import pytest
import torch

from test_cache8_cpu import _PlanArgs
from test_gpu_cache8 import eg, i32  # noqa: F401

pytestmark = pytest.mark.gpu

SIDES = [4096, 4097, 5000, 70000]  # of the two kernels


@pytest.mark.parametrize("tokens", SIDES)
def test_plan_of_no_requests(eg, tokens):  # noqa: F811
    """Nothing but -1 in the maps, and nothing behind them or behind the one offset is touched."""
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    pos = torch.full((tokens + 9000,), 7, dtype=torch.int32, device="cuda")
    slots = torch.full((tokens + 9000,), 7, dtype=torch.int64, device="cuda")
    offs = torch.tensor([5, 1 << 30], device="cuda")  # what lies behind the offset names tokens
    got = eg.engram_kv_plan(empty, empty, empty.view(0, 0), i32([4, 2, 9]), i32([3]), 16, tokens, seq_offsets=offs[:1],
                            positions=pos[:tokens], slots=slots[:tokens])
    assert eg.engram_last_error() == 0
    assert offs.tolist() == [0, 1 << 30] and got.n_free.tolist() == [3] and got.counts.tolist() == [0] * 4
    for t in (pos, slots):
        assert bool((t[:tokens] == -1).all()) and bool((t[tokens:] == 7).all())


@pytest.mark.parametrize("tokens", SIDES)
def test_plan_of_no_requests_in_c(eg, tokens):  # noqa: F811
    """The header's structure with nothing where no request has anything: no lengths, no table."""
    offs, counts, n_free = torch.tensor([5], device="cuda"), i32([7] * 4), i32([3])
    pos = torch.full((tokens,), 7, dtype=torch.int32, device="cuda")
    slots = torch.full((tokens,), 7, dtype=torch.int64, device="cuda")
    p = _PlanArgs()
    p.max_tokens, p.n_pages, p.page_size = tokens, 3, 16
    stack = i32([4, 2, 9])
    p.free_pages, p.n_free, p.n_free_out = stack.data_ptr(), n_free.data_ptr(), n_free.data_ptr()
    p.seq_offsets, p.positions, p.slots, p.counts = (t.data_ptr() for t in (offs, pos, slots, counts))
    assert eg.lib().engram_kv_plan(ctypes.byref(p), None) == 0
    assert eg.engram_last_error() == 0
    assert offs.tolist() == [0] and n_free.tolist() == [3] and counts.tolist() == [0] * 4 and stack.tolist() == [4, 2, 9]
    assert bool((pos == -1).all()) and bool((slots == -1).all())


def test_plan_whose_missing_outputs_are_empty(eg):  # noqa: F811
    """A step that only drops tokens: every output that has values is given, those left out have none."""
    table, stack = i32([[5, 6, 7], [8, 9, -1]]), i32([0, 1, -1, -1, -1, -1])
    offs = torch.full((3,), 7, dtype=torch.int64, device="cuda")
    kv, free, counts = i32([40, 20]), i32([2]), i32([7] * 4)
    got = eg.engram_kv_plan(i32([0, 0]), kv, table, stack, free, 16, 0, keep_len=i32([17, 0]), kv_len_out=kv, n_free_out=free,
                            seq_offsets=offs, counts=counts)
    assert eg.engram_last_error() == 0
    assert got.seq_offsets is offs and got.kv_len is kv and got.n_free is free and got.counts is counts
    assert offs.tolist() == [0, 0, 0] and kv.tolist() == [17, 0] and free.tolist() == [5] and counts.tolist() == [0, 0, 3, 0]
    assert stack.tolist() == [0, 1, 7, 8, 9, -1]
    for t, dtype in ((got.positions, torch.int32), (got.slots, torch.int64)):
        assert t.shape == (0,) and t.dtype == dtype and t.device == kv.device


@pytest.mark.parametrize("missing", ["positions", "slots", "kv_len_out"])
def test_plan_of_nothing_with_one_output_missing(eg, missing):  # noqa: F811
    """No requests and no tokens: an empty output is made whichever it is."""
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    outs = dict(kv_len_out=empty, n_free_out=i32([0]), seq_offsets=torch.zeros(1, dtype=torch.int64, device="cuda"),
                positions=empty, slots=torch.zeros(0, dtype=torch.int64, device="cuda"), counts=i32([7] * 4))
    del outs[missing]
    got = eg.engram_kv_plan(empty, empty, empty.view(0, 0), i32([4, 2]), i32([2]), 16, 0, **outs)
    assert eg.engram_last_error() == 0 and got.n_free.tolist() == [2] and got.counts.tolist() == [0] * 4
    assert all(t.numel() == 0 for t in (got.positions, got.slots, got.kv_len))
