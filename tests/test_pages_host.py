"""Refusals of the page tables (no GPU)."""
import ctypes

import numpy as np
import pytest

from gated_deltanet_tree_amd import binding


def _args(**edit):
    a = binding.PagesArgs()
    for k, v in dict(n_seqs=2, n_tokens=3, n_pages=10, page_tokens=16, max_pages=4, workspace_bytes=1 << 20, **{
            n: 4096 for n in ("seq_offsets", "length", "pages", "refs", "missing", "slots", "positions", "depth",
                              "workspace")}).items():
        setattr(a, k, edit.get(k, v))
    return a


SIZES = [dict(n_seqs=-1), dict(n_seqs=(1 << 20) + 1), dict(n_tokens=-1), dict(n_pages=0), dict(max_pages=0),
         dict(page_tokens=24), dict(page_tokens=0), dict(page_tokens=256, max_pages=(1 << 22) + 1)]


@pytest.mark.parametrize("edit", SIZES + [dict(pages=None), dict(refs=None)])
def test_both_calls_refuse(edit):
    L = binding.lib()
    assert L.gdn_kv_reserve(ctypes.byref(_args(**edit)), None) == -1
    assert L.gdn_kv_release(ctypes.byref(_args(**edit)), 4096, None) == -1
    assert b"gdn_kv_release" in L.gdn_last_error()


@pytest.mark.parametrize("edit", SIZES)
def test_sizes_have_no_workspace(edit):
    assert binding.lib().gdn_pages_workspace_bytes(ctypes.byref(_args(**edit))) == 0


def test_own_arguments():
    L = binding.lib()
    for edit in (dict(length=None), dict(seq_offsets=None), dict(workspace=4104)):
        assert L.gdn_kv_reserve(ctypes.byref(_args(**edit)), None) == -1
    assert L.gdn_kv_release(ctypes.byref(_args()), None, None) == -1
    assert L.gdn_kv_reserve(None, None) == -1 and L.gdn_kv_release(None, 4096, None) == -1
    assert L.gdn_pages_workspace_bytes(None) == 0
    need = L.gdn_pages_workspace_bytes(ctypes.byref(_args(pages=None, workspace=None)))
    assert need >= 4 * 12
    assert L.gdn_kv_reserve(ctypes.byref(_args(workspace=None)), None) == -4
    assert L.gdn_kv_reserve(ctypes.byref(_args(workspace_bytes=8)), None) == -4
    empty = _args(n_seqs=0, pages=None, refs=None)
    assert L.gdn_kv_reserve(ctypes.byref(empty), None) == 0 and L.gdn_kv_release(ctypes.byref(empty), 4096, None) == 0


def test_binding_checks_types_and_sizes():
    import torch
    offs = np.array([0, 2, 3], dtype=np.int32)
    i32 = dict(dtype=torch.int32)
    ok = dict(pages=torch.zeros((2, 4), **i32), length=torch.zeros(2, **i32), refs=torch.zeros(9, **i32),
              page_tokens=16, host_offsets=offs, dev_offsets=torch.from_numpy(offs))
    out = dict(missing=torch.zeros(2, **i32), slots=torch.zeros(3, dtype=torch.int64),
               positions=torch.zeros(3, **i32), depth=torch.zeros(3, **i32))
    a = binding.pages_args(**ok, **out)
    assert (a.n_seqs, a.n_tokens, a.n_pages, a.page_tokens, a.max_pages) == (2, 3, 9, 16, 4)
    assert binding.pages_workspace_bytes(a) > 0
    for bad in (dict(pages=torch.zeros((1, 4), **i32)), dict(pages=torch.zeros(8, **i32)), dict(length=torch.zeros(1, **i32)),
                dict(refs=torch.zeros(9)), dict(host_offsets=[0, 3, 2]), dict(host_offsets=[1, 2, 3]),
                dict(missing=torch.zeros(1, **i32)), dict(slots=torch.zeros(3, **i32)),
                dict(positions=torch.zeros(2, **i32)), dict(depth=torch.zeros(3)),
                dict(pages=torch.zeros((4, 2), **i32).T)):
        with pytest.raises(ValueError):
            binding.pages_args(**(ok | out | bad))
    for call in (lambda: binding.kv_reserve(a), lambda: binding.kv_release(a, ok["length"])):
        with pytest.raises(ValueError, match="GPU memory"):
            call()
    with pytest.raises(ValueError):
        binding.kv_release(a, torch.zeros(2))


def test_references_of_a_caches_tables():
    import torch
    kv = binding.alloc_kv_cache(1, 2, 1, 64, 5, 16, 3, device="cpu")
    kv.pages.copy_(torch.tensor([[4, 0, -1], [4, 7, 2]], dtype=torch.int32))
    refs = binding.alloc_kv_refs(kv)
    assert refs.tolist() == [1, 0, 1, 0, 2] and refs.dtype == torch.int32
