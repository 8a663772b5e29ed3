"""Host side of the 4-bit cache, its attention and the acceptance (no GPU): the address arithmetic
and argument checks under sanitizers, and every refusal through the C ABI and the binding."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from gated_deltanet_tree_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_layout_and_checks_under_sanitizers(tmp_path):
    if shutil.which(os.environ.get("CXX", "g++")) is None:
        pytest.skip("no host C++ compiler")
    from gated_deltanet_tree_amd import build_host_san  # not there where only GPU tests run
    exe = build_host_san.build_driver(os.path.join(ROOT, "tests", "host_san_kv.cpp"), str(tmp_path))
    env = dict(os.environ, ASAN_OPTIONS="halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and out.strip().endswith("ok"), out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out


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


OFFS = np.array([0, 3], dtype=np.int32)


def _calls():
    L = binding.lib()
    o = binding._ptr(OFFS)
    return {
        "append": lambda a: L.gdn_kv_append(ctypes.byref(a), o, None),
        "read": lambda a: L.gdn_kv_read(ctypes.byref(a), o, None, None),
        "commit": lambda a: L.gdn_kv_commit(ctypes.byref(a), o, 4096, 3, 4096, 4096, None),
        "attention": lambda a: L.gdn_attention(ctypes.byref(a), o, None),
    }


@pytest.mark.parametrize("edit", [dict(head_dim=96), dict(page_tokens=24), dict(n_pages=0), dict(max_pages=0),
                                  dict(in_dtype=3), dict(n_tokens=4), dict(n_kv_heads=0), dict(n_layers=0),
                                  dict(k_codes=None), dict(v_scales=4104), dict(pages=None), dict(length=None),
                                  dict(seq_offsets=None), dict(n_seqs=-1), dict(layer_begin=-1)])
def test_cache_calls_refuse_before_any_launch(edit):
    for name, call in _calls().items():
        assert call(_kv(**edit)) == -1, name
        assert binding.lib().gdn_last_error() != b""


def test_row_pointers_and_alignment():
    calls = _calls()
    for name in ("append", "read", "commit"):
        assert calls[name](_kv(k=None)) == -1 and calls[name](_kv(v=4100)) == -1
    assert calls["attention"](_kv(q=None)) == -1 and calls["attention"](_kv(out=4104)) == -1
    assert calls["attention"](_kv(n_heads=7)) == -1 and b"multiple" in binding.lib().gdn_last_error()


@pytest.mark.parametrize("scale", [0.0, -0.1, float("nan"), float("inf"), 3e38, 1e-40])
def test_attention_refuses_a_scale_that_is_not_positive_and_finite(scale):
    assert _calls()["attention"](_kv(scale=scale)) == -1 and b"scale" in binding.lib().gdn_last_error()


def test_commit_needs_its_arrays():
    L, o = binding.lib(), binding._ptr(OFFS)
    a = _kv()
    assert L.gdn_kv_commit(ctypes.byref(a), o, 4096, 0, 4096, 4096, None) == -1
    assert L.gdn_kv_commit(ctypes.byref(a), o, 4096, 3, None, 4096, None) == -1
    assert L.gdn_kv_commit(ctypes.byref(a), o, None, 0, 4096, None, None) == -1


def test_attention_workspace_is_checked():
    L, o = binding.lib(), binding._ptr(OFFS)
    a = _kv(max_pages=1000)
    need = L.gdn_attention_workspace_bytes(ctypes.byref(a), o)
    assert need > 0
    assert L.gdn_attention(ctypes.byref(a), o, None) == -4
    a.workspace, a.workspace_bytes = 4096, need - 1
    assert L.gdn_attention(ctypes.byref(a), o, None) == -4 and b"workspace" in L.gdn_last_error()
    a.workspace, a.workspace_bytes = 4104, need
    assert L.gdn_attention(ctypes.byref(a), o, None) == -1
    a.max_length = 100  # short sequences are not cut
    assert L.gdn_attention_workspace_bytes(ctypes.byref(a), o) == 0


def test_tree_attention_checks_its_image():
    L = binding.lib()
    image = binding.hld_schedule([np.array([-1, 0, 0])])
    a = _kv()
    bad = image.copy()
    bad[0] = 1
    assert L.gdn_tree_attention(ctypes.byref(a), binding._ptr(bad), 4096, None) == -1
    assert L.gdn_tree_attention(ctypes.byref(a), binding._ptr(image), None, None) == -1
    assert L.gdn_tree_attention(None, binding._ptr(image), 4096, None) == -1
    assert L.gdn_tree_attention(ctypes.byref(_kv(n_tokens=4)), binding._ptr(image), 4096, None) == -1
    assert L.gdn_tree_attention(ctypes.byref(_kv(n_seqs=2)), binding._ptr(image), 4096, None) == -1
    assert L.gdn_tree_attention(ctypes.byref(_kv(q=None, seq_offsets=None)), binding._ptr(image), 4096, None) == -1
    assert b"q/out" in L.gdn_last_error()  # the image's offsets stand in for seq_offsets


def _accept(**edit):
    a = binding.AcceptArgs()
    for k, v in dict(n_seqs=1, n_nodes=3, vocab=100, in_dtype=0, max_path=3, logit_stride=100,
                     workspace_bytes=1 << 20, **{n: 4096 for n in (
                         "logits", "tokens", "uniform", "temperature", "path", "path_len", "next_token",
                         "workspace")}).items():
        setattr(a, k, edit.get(k, v))
    return a


@pytest.mark.parametrize("edit,status", [
    (dict(n_seqs=2), -1), (dict(n_nodes=4), -1), (dict(vocab=0), -1), (dict(vocab=101), -1),
    (dict(in_dtype=2), -1), (dict(max_path=2), -4), (dict(workspace_bytes=10), -4), (dict(workspace=4104), -1),
    (dict(logits=4098), -1), (dict(logits=None), -1), (dict(tokens=None), -1), (dict(uniform=None), -1),
    (dict(temperature=None), -1), (dict(path=None), -1), (dict(path_len=None), -1), (dict(next_token=None), -1),
    (dict(workspace=None), -1)])
def test_accept_refuses_before_any_launch(edit, status):
    L = binding.lib()
    image = binding.hld_schedule([np.array([-1, 0, 0])])
    a = _accept(**edit)
    assert L.gdn_tree_accept(ctypes.byref(a), binding._ptr(image), 4096, None) == status
    assert L.gdn_last_error() != b""
    assert L.gdn_tree_accept(None, binding._ptr(image), 4096, None) == -1
    assert L.gdn_tree_accept(ctypes.byref(_accept()), binding._ptr(image), None, None) == -1


def test_padding_behind_the_last_sequence_only_in_the_last_layer():
    import torch
    kv = binding.alloc_kv_cache(2, 1, 2, 64, 3, 16, 3, device="cpu")
    dev, padded = torch.from_numpy(OFFS), torch.zeros((2, 5, 2, 64))
    a = binding.kv_args(kv, OFFS, dev, k=padded, v=padded)  # rows 3, 4 are left alone
    assert a.n_tokens == 3
    for kw in (dict(n_layers=2), dict(layer_begin=1)):  # the second layer would start inside the padding
        with pytest.raises(ValueError):
            binding.kv_args(kv, OFFS, dev, k=padded, v=padded, **kw)


def test_binding_rejects_wrong_tensors():
    import torch
    kv = binding.alloc_kv_cache(2, 1, 2, 64, 3, 16, 3, device="cpu")
    offs, dev = OFFS, torch.from_numpy(OFFS)
    rows = torch.zeros((1, 3, 2, 64))

    def refused(**kw):
        with pytest.raises(ValueError):
            binding.kv_args(kv, offs, dev, **kw)

    refused(k=rows[:, :2])                                  # too few rows
    refused(k=rows, v=rows.to(torch.bfloat16))              # two dtypes
    refused(k=rows.double())
    refused(k=torch.zeros((1, 3, 64, 2)).transpose(2, 3))   # strided
    refused(k=rows, layer_begin=2)
    refused(k=rows, layer_begin=1)                          # the second layer's rows are not there
    refused(q=torch.zeros((1, 3, 4, 32)))
    refused(q=torch.zeros((3, 4, 64)))
    with pytest.raises(ValueError):
        binding.kv_args(kv, np.array([0, 1, 3]), dev, k=rows)  # more sequences than the table
    with pytest.raises(ValueError):
        binding.kv_args(kv, offs, dev.long(), k=rows)
    kv.pages = kv.pages.long()
    refused(k=rows)
    kv.pages = kv.pages.int()
    a = binding.kv_args(kv, offs, dev, k=rows, v=rows)
    with pytest.raises(ValueError):
        binding.kv_append(a)  # host memory
    with pytest.raises(ValueError):
        binding.kv_commit(a, None, dev, torch.zeros(1))
    image = binding.hld_schedule([np.array([-1, 0, 0])])
    i32 = dict(dtype=torch.int32)
    ok = dict(logits=torch.zeros((3, 9)), tokens=torch.zeros(3, **i32), uniform=torch.zeros((1, 3)),
              temperature=torch.ones(1), path=torch.zeros((1, 3), **i32), path_len=torch.zeros(1, **i32),
              next_token=torch.zeros(1, **i32), workspace=torch.zeros(4096))
    binding.accept_args(image, **ok)
    for bad in (dict(logits=torch.zeros((2, 9))), dict(logits=torch.zeros((9, 3)).t()),
                dict(logits=torch.zeros((3, 9)).half()), dict(tokens=torch.zeros(3)), dict(uniform=torch.zeros((1, 4))),
                dict(path=torch.zeros((1, 3))), dict(temperature=torch.zeros(0))):
        with pytest.raises(ValueError):
            binding.accept_args(image, **{**ok, **bad})
    with pytest.raises(ValueError):
        binding.accept_args(image, vocab=10, **ok)
    with pytest.raises(ValueError):
        binding.tree_accept(binding.accept_args(image, **ok), image, torch.from_numpy(image))
