"""Refusals of the 4-bit cache's binding (no GPU)."""
import ctypes

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


def _commit(new_length, n_seqs=4):
    """gdn_kv_commit of n_seqs single tokens, every array at an address of its own; without k, so that
    a call whose lengths are accepted is refused for that and launches nothing."""
    a = binding.KvArgs()
    for k, v in dict(n_seqs=n_seqs, n_heads=2, n_kv_heads=2, head_dim=64, n_tokens=n_seqs, n_pages=4, page_tokens=64,
                     max_pages=4, n_layers=1, in_dtype=1, k=None, v=1 << 21, k_codes=1 << 22, v_codes=1 << 23,
                     k_scales=1 << 24, v_scales=1 << 25, length=0x10000, seq_offsets=0x20000, pages=0x30000).items():
        setattr(a, k, v)
    offs = np.arange(n_seqs + 1, dtype=np.int32)
    L = binding.lib()
    r = L.gdn_kv_commit(ctypes.byref(a), binding._ptr(offs), 0x40000, 2, 0x50000, new_length, None)
    return r, L.gdn_last_error()


def test_commit_refuses_lengths_that_overlap_its_inputs():
    """new_length may be the lengths or the counts themselves; shifted over them, or over the offsets,
    the pages or the rows, one sequence's result would be another's input."""
    for at in (0x10004, 0x10000 - 4, 0x1000C, 0x50004, 0x50000 - 12, 0x20000, 0x20010, 0x30000, 0x3003C, 0x40000, 0x4001C):
        r, why = _commit(at)
        assert r == -1 and b"overlap" in why, hex(at)
    for at in (0x20014, 0x10010, 0x50010, 0x20000 - 16, 0x30040, 0x40020):  # beside them
        r, why = _commit(at)
        assert r == -1 and b"k/v" in why, hex(at)
    for at in (0x10000, 0x50000):  # the lengths or the counts themselves
        assert b"k/v" in _commit(at)[1]
