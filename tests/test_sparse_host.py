"""Refusals and launch plans of the sparse attention (no GPU)."""
import ctypes

import numpy as np
import pytest

from gated_deltanet_tree_amd import binding

OFFS = np.array([0, 3], dtype=np.int32)


def _kv(**edit):
    a = binding.KvArgs()
    for k, v in dict(n_seqs=1, n_heads=8, n_kv_heads=2, head_dim=128, n_tokens=3, n_pages=4, page_tokens=64,
                     max_pages=4, n_layers=1, in_dtype=1, scale=0.1, max_length=0, **{
                         n: 4096 for n in ("q", "k", "v", "out", "seq_offsets", "k_codes", "v_codes", "k_scales",
                                           "v_scales", "pages", "length")}).items():
        setattr(a, k, edit.pop(k, v))
    for k, v in edit.items():
        setattr(a, k, v)
    return a


def _sparse(**edit):
    x = binding.SparseArgs()
    for k, v in dict(top_pages=2, share_tokens=1, keep_first=0, keep_last=0, bounds=4096, selected=4096).items():
        setattr(x, k, edit.get(k, v))
    return x


def _calls(image=None):
    L, o = binding.lib(), binding._ptr(OFFS)
    image = binding.hld_schedule([np.array([-1, 0, 0])]) if image is None else image
    ref = ctypes.byref
    return {
        "bounds": lambda a, x: L.gdn_kv_bounds(ref(a), x and ref(x), o, None),
        "select": lambda a, x: L.gdn_kv_select(ref(a), x and ref(x), o, None),
        "attention": lambda a, x: L.gdn_sparse_attention(ref(a), x and ref(x), o, None),
        "tree": lambda a, x: L.gdn_sparse_tree_attention(ref(a), x and ref(x), binding._ptr(image), 4096, None),
    }


@pytest.mark.parametrize("edit", [dict(head_dim=96), dict(page_tokens=24), dict(n_pages=0), dict(max_pages=0),
                                  dict(in_dtype=3), dict(n_tokens=4), dict(n_kv_heads=0), dict(n_layers=0),
                                  dict(k_codes=None), dict(pages=None), dict(length=None), dict(n_seqs=-1),
                                  dict(layer_begin=-1)])
def test_the_cache_is_checked_as_by_the_other_calls(edit):
    for name, call in _calls().items():
        assert call(_kv(**edit), _sparse(share_tokens=0)) == -1, name
        assert binding.lib().gdn_last_error() != b""


@pytest.mark.parametrize("edit", [dict(top_pages=0), dict(top_pages=257), dict(keep_first=-1), dict(keep_last=-1),
                                  dict(keep_first=2, keep_last=1), dict(keep_first=2**31 - 1, keep_last=2**31 - 1),
                                  dict(share_tokens=-1), dict(selected=None)])
def test_selections_that_cannot_be_are_refused(edit):
    x = dict(share_tokens=0) | edit
    for name in ("select", "attention", "tree"):
        assert _calls()[name](_kv(), _sparse(**x)) == -1, name


def test_pointers():
    calls = _calls()
    for name, call in calls.items():
        assert call(_kv(), None) == -1 and b"null" in binding.lib().gdn_last_error(), name
    for bad in (None, 4104):
        assert calls["bounds"](_kv(), _sparse(bounds=bad)) == -1
        assert calls["select"](_kv(), _sparse(bounds=bad)) == -1
        assert calls["select"](_kv(q=bad), _sparse()) == -1
        assert calls["attention"](_kv(q=bad), _sparse()) == -1
        assert calls["attention"](_kv(out=bad), _sparse()) == -1
    assert calls["select"](_kv(n_heads=7), _sparse()) == -1
    assert calls["attention"](_kv(scale=0.0), _sparse()) == -1


def test_a_trees_nodes_share_one_selection():
    assert _calls()["tree"](_kv(), _sparse(share_tokens=1)) == -1 and b"share" in binding.lib().gdn_last_error()


def test_workspace_is_asked_for_and_checked():
    L, o = binding.lib(), binding._ptr(OFFS)
    a, x = _kv(max_pages=4000), _sparse(top_pages=32)
    need = L.gdn_sparse_workspace_bytes(ctypes.byref(a), ctypes.byref(x), o)
    assert need > 0
    calls = _calls()
    for name in ("select", "attention"):
        assert calls[name](a, x) == -4, name
    a.workspace, a.workspace_bytes = 4104, need
    for name in ("select", "attention"):
        assert calls[name](a, x) == -1 and b"workspace" in L.gdn_last_error(), name
    assert L.gdn_sparse_workspace_bytes(ctypes.byref(a), None, o) == 0
    assert L.gdn_sparse_workspace_bytes(ctypes.byref(a), ctypes.byref(_sparse(top_pages=0)), o) == 0


def test_too_many_selections_are_refused():
    offs = np.array([0, 1 << 20], dtype=np.int32)
    a, x = _kv(n_tokens=1 << 20, n_layers=64, n_heads=2), _sparse()
    L = binding.lib()
    for call in (L.gdn_kv_select, L.gdn_sparse_attention):
        assert call(ctypes.byref(a), ctypes.byref(x), binding._ptr(offs), None) == -1
        assert b"too many" in L.gdn_last_error()
    assert L.gdn_sparse_workspace_bytes(ctypes.byref(a), ctypes.byref(x), binding._ptr(offs)) == 0


def test_selections_fill_the_largest_grid_at_most():
    """Workgroups of 1024 threads: 2^32 of them in all, fewer selections than the attention has room for."""
    n = 1 << 20
    offs = np.array([0, n], dtype=np.int32)
    L = binding.lib()
    for layers, ok in ((3, True), (4, False), (7, False)):
        a, x = _kv(n_tokens=n, n_layers=layers, n_heads=1, n_kv_heads=1, max_pages=4), _sparse(selected=None)
        assert L.gdn_kv_select(ctypes.byref(a), ctypes.byref(x), binding._ptr(offs), None) == -1
        x.selected = 4096
        if not ok:
            assert L.gdn_kv_select(ctypes.byref(a), ctypes.byref(x), binding._ptr(offs), None) == -1
            assert b"too many" in L.gdn_last_error()


def test_binding_checks_types_and_sizes():
    import torch
    kv = binding.alloc_kv_cache(2, 1, 2, 64, 3, 16, 3, device="cpu")
    a = binding.kv_args(kv, OFFS, torch.from_numpy(OFFS), n_layers=2)
    bounds = binding.alloc_kv_bounds(kv)
    assert tuple(bounds.shape) == (2, 3, 2, 2, 64) and bounds.dtype == torch.bfloat16
    sel = torch.zeros((2, 3, 2, 4), dtype=torch.int32)
    x = binding.sparse_args(a, bounds, sel, top_pages=4, share_tokens=0, keep_first=1)
    assert (x.top_pages, x.share_tokens, x.keep_first, x.keep_last) == (4, 0, 1, 0)
    for bad in (dict(bounds=bounds.float()), dict(bounds=bounds[:1]), dict(selected=sel.long()),
                dict(selected=sel[..., :3]), dict(selected=sel[:1].contiguous()),
                dict(selected=torch.zeros((2, 6, 2, 2), dtype=torch.int32)),
                dict(bounds=torch.zeros((2, 6, 2, 1, 64), dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            binding.sparse_args(a, **(dict(bounds=bounds, selected=sel, top_pages=4) | bad))
    for call in (binding.kv_bounds, binding.kv_select, binding.sparse_attention):
        with pytest.raises(ValueError, match="GPU memory"):
            call(a, x)
