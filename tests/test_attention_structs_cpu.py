"""The attention step's descriptions as Python objects: copies, changes and directly made ones mean what they hold."""

import copy
import pickle

import pytest
import torch


@pytest.fixture(scope="module")
def eg():
    import engram_gram_hash_gb300 as eg

    eg.build()
    eg.lib()
    return eg


def _refusal(eg, cfg, heads, dtype):
    """What the call says about q [3, heads, 128] on the CPU: refused as a CPU tensor if cfg names that shape and type."""
    q = torch.zeros((3, heads, 128), dtype=dtype)
    with pytest.raises((ValueError, TypeError)) as e:
        eg.engram_qk_norm_rope(cfg, q, None, torch.zeros(3, dtype=torch.int32), torch.zeros((10, 128)))
    return str(e.value)


@pytest.mark.parametrize("duplicate", [copy.copy, copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c))])
def test_copies_are_configurations_of_their_own(eg, duplicate):
    first = eg.make_attn_config(8, 2, 128)
    second = duplicate(first)
    second.n_heads, second.dtype = 4, 1
    assert "CUDA" in _refusal(eg, second, 4, torch.float16)
    assert "CUDA" in _refusal(eg, first, 8, torch.bfloat16)
    assert (first.torch_dtype, second.torch_dtype) == (torch.bfloat16, torch.float16)
    third = duplicate(eg.make_attn_config(8, 2, 128))  # whose first one is gone
    assert "CUDA" in _refusal(eg, third, 8, torch.bfloat16)


def test_directly_made_configurations(eg):
    c = eg.engram_attn_config(6, 2, 128, 128, 0, 1, 1e-6, 0.1, 0)
    assert c.torch_dtype is torch.float16
    assert "CUDA" in _refusal(eg, c, 6, torch.float16)


@pytest.mark.parametrize("wrong", [None, 0, 4096, b"x", "cfg"])
def test_other_objects_are_refused(eg, wrong):
    with pytest.raises(TypeError):
        eg.engram_qk_norm_rope(wrong, torch.zeros((3, 8, 128), dtype=torch.bfloat16), None, None, None)
