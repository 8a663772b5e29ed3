"""Refusals of the 4-bit cache's binding (no GPU)."""
import numpy as np
import pytest

from gated_deltanet_tree_amd import binding

OFFS = np.array([0, 3], dtype=np.int32)


def test_rows_of_other_heads_or_channels_are_refused():
    """Enough elements, but not the cache's heads, or an output of other heads than q's."""
    import torch
    kv = binding.alloc_kv_cache(1, 1, 2, 64, 3, 16, 3, device="cpu")
    dev = torch.from_numpy(OFFS)

    def rows(heads, d=64):
        return torch.zeros((1, 3, heads, d))

    binding.kv_args(kv, OFFS, dev, k=rows(2), v=rows(2), q=rows(6), out=rows(6))
    binding.kv_args(kv, OFFS, dev, k=rows(2).flatten(), v=rows(2).flatten())  # no shape to compare
    for bad in (dict(k=rows(6)), dict(v=rows(6)), dict(k=rows(1, 128)), dict(v=rows(2, 128)),
                dict(q=rows(6), out=rows(8)), dict(q=rows(6), out=rows(3, 128)), dict(out=rows(4))):
        with pytest.raises(ValueError):
            binding.kv_args(kv, OFFS, dev, **bad)
