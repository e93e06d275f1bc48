"""Integers past 32 bits in the calls of the cache operators: the C ABI takes int, and a larger value's low 32
bits would be another, valid one. Each is refused by name, whatever else the call holds (no device here)."""
import pytest
import torch

import __graft_entry__

__graft_entry__._build_module().build()
import sparse_attention_keys_b200 as dsa  # noqa: E402

WIDE = (1 << 32) + 8                         # its low 32 bits are 8


def refused(name, call):
    with pytest.raises(ValueError, match=rf"{name}.*32 bits"):
        call()


@pytest.mark.parametrize("value", [WIDE, 1 << 31, -(1 << 32), -(1 << 31) - 1])
def test_eviction(value):
    acc, pos = torch.zeros(1, 8), torch.zeros(1, 8, dtype=torch.int32)
    n = torch.full((1,), 8, dtype=torch.int32)
    for name in ("recent", "sinks"):
        refused(name, lambda: dsa.dsa_cache_evict(acc, pos, n, 4, **{name: value}))
    if value > 0:
        refused("keep", lambda: dsa.dsa_cache_evict(acc, pos, n, value))
    else:
        with pytest.raises(ValueError):
            dsa.dsa_cache_evict(acc, pos, n, value)


def test_sizes_of_tensors():
    """A cache of more rows, a selection of more slots, more heads or features than an int counts."""
    def meta(*shape, dtype=torch.int32):
        return torch.empty(shape, dtype=dtype, device="meta")

    n = meta(1)
    refused("S", lambda: dsa.dsa_cache_evict(meta(1, WIDE, dtype=torch.float32), meta(1, WIDE), n, 4))
    refused("B", lambda: dsa.dsa_cache_evict(meta(WIDE, 1, dtype=torch.float32), meta(WIDE, 1), meta(WIDE), 4))
    q, lse = meta(1, 1, 128, 576, dtype=torch.bfloat16), meta(1, 1, 128, dtype=torch.float32)
    refused("k", lambda: dsa.dsa_mla_weights_selected(q, meta(1, 8, 576, dtype=torch.bfloat16), meta(1, 1, WIDE), lse))
    freqs = meta(4, dtype=torch.int64)
    for shape, name in (((1, WIDE, 8), "heads"), ((1, WIDE), "dim"), ((1, 1, WIDE), "dim")):
        x = meta(*shape, dtype=torch.bfloat16)
        refused(name, lambda: dsa._rope(x, n, freqs, 0, False, False, 1.0, None, 0))


@pytest.mark.parametrize("value", [WIDE, 1 << 31, -(1 << 32)])
def test_frequencies(value):
    refused("original_len", lambda: dsa.dsa_rope_freqs(8, original_len=value))
    if value > 0:
        refused("pairs", lambda: dsa.dsa_rope_freqs(value))
    with pytest.raises(ValueError):
        dsa.dsa_rope_freqs(value)


@pytest.mark.parametrize("value", [WIDE, -(1 << 32) + 8])
def test_workspace_sizes_are_zero_for_a_shape_that_no_call_takes(value):
    for i in range(4):
        shape = [2, 1, 8, 8]
        assert dsa.dsa_mla_shared_workspace_size(*shape) > 0
        shape[i] = value
        assert dsa.dsa_mla_shared_workspace_size(*shape) == 0
    for i in range(3):
        shape = [2, 8, 4]
        assert dsa.dsa_cache_evict_workspace_size(*shape) > 0
        shape[i] = value
        assert dsa.dsa_cache_evict_workspace_size(*shape) == 0
