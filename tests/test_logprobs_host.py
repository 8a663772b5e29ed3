"""Refusals of the log probabilities (no GPU)."""
import ctypes

import pytest

from gated_deltanet_tree_amd import binding


def _args(**edit):
    a = binding.LogprobsArgs()
    for k, v in dict(n_rows=3, vocab=100, in_dtype=0, top_k=4, n_given=1, logit_stride=100, workspace_bytes=1 << 20,
                     **{n: 4096 for n in ("logits", "given", "given_logp", "top_token", "top_logp", "entropy",
                                          "workspace")}).items():
        setattr(a, k, edit.get(k, v))
    return a


@pytest.mark.parametrize("edit", [
    dict(n_rows=-1), dict(vocab=0), dict(vocab=-5), dict(logit_stride=99), dict(in_dtype=2), dict(top_k=-1),
    dict(top_k=65), dict(n_given=-1), dict(vocab=(1 << 20) + 1, logit_stride=1 << 21), dict(logits=None),
    dict(workspace=None), dict(top_token=None), dict(top_logp=None), dict(given=None), dict(given_logp=None),
    dict(logits=4098), dict(logits=4097, in_dtype=1), dict(workspace=4104)])
def test_refused_before_any_launch(edit):
    L = binding.lib()
    assert L.gdn_token_logprobs(ctypes.byref(_args(**edit)), None) == -1
    assert b"gdn_token_logprobs" in L.gdn_last_error()


def test_null_and_empty():
    L = binding.lib()
    assert L.gdn_token_logprobs(None, None) == -1
    assert L.gdn_token_logprobs(ctypes.byref(_args(n_rows=0, logits=None, workspace=None)), None) == 0


def test_workspace_is_asked_for_and_checked():
    L = binding.lib()
    need = binding.logprobs_workspace_bytes(3, 100, 4)
    assert need > 0 and need > binding.logprobs_workspace_bytes(3, 100, 0) > 0
    assert L.gdn_token_logprobs(ctypes.byref(_args(workspace_bytes=need - 1)), None) == -4
    for bad in ((-1, 100, 4), (3, 0, 4), (3, 100, 65), (3, 100, -1), (3, 1 << 30 | 1, 0)):
        assert binding.logprobs_workspace_bytes(*bad) == 0


def test_too_many_rows_are_refused():
    a = _args(n_rows=2**31 - 1, vocab=20000, logit_stride=20000, workspace_bytes=2**62)
    assert binding.lib().gdn_token_logprobs(ctypes.byref(a), None) == -1
    assert b"too many" in binding.lib().gdn_last_error()


def test_binding_checks_types_and_sizes():
    import torch
    x = torch.zeros((3, 50))
    i, f = torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2))
    a = binding.logprobs_args(x, i, f, i, f, torch.zeros(3), vocab=40)
    assert (a.n_rows, a.vocab, a.top_k, a.n_given, a.logit_stride) == (3, 40, 2, 2, 50)
    wide = torch.zeros((3, 80))[:, 5:55]
    assert binding.logprobs_args(wide).logit_stride == 80
    for bad in (lambda: binding.logprobs_args(x.T), lambda: binding.logprobs_args(x, vocab=51),
                lambda: binding.logprobs_args(x.half()), lambda: binding.logprobs_args(x[0]),
                lambda: binding.logprobs_args(x[:1].expand(3, 50)),
                lambda: binding.logprobs_args(x, given=i), lambda: binding.logprobs_args(x, given=i, given_logp=f[:, :1]),
                lambda: binding.logprobs_args(x, given=i.long(), given_logp=f),
                lambda: binding.logprobs_args(x, top_token=i[:2], top_logp=f[:2]),
                lambda: binding.logprobs_args(x, top_token=i, top_logp=f.double()),
                lambda: binding.logprobs_args(x, entropy=torch.zeros(2))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError, match="GPU memory"):
        binding.token_logprobs(a)


MOST = (2**32 - 1) // 256  # workgroups of 256 threads; one takes up to four pieces of 2048 logits of a row


@pytest.mark.parametrize("rows,vocab,top_k", [(1, 1 << 20, 64), (1, (1 << 20) + 1, 1), (1, 1 << 21, 4), (1, 1 << 21, 0),
                                              (1, 1 << 30, 0), (1, 1 << 30, 1), (MOST, 8185, 4), (MOST + 1, 8185, 4),
                                              (MOST, 8186, 4), (MOST // 2, 8186, 0), (2**31 - 1, 20000, 0)])
def test_the_size_query_and_the_call_refuse_the_same_sizes(rows, vocab, top_k):
    """No bytes exactly where the call refuses the sizes; everywhere else it asks for those bytes."""
    L = binding.lib()
    need = binding.logprobs_workspace_bytes(rows, vocab, top_k)
    a = _args(n_rows=rows, vocab=vocab, logit_stride=vocab, top_k=top_k, workspace_bytes=need - 1)
    assert L.gdn_token_logprobs(ctypes.byref(a), None) == (-4 if need > 0 else -1), L.gdn_last_error()
    refused = (top_k > 0 and vocab > 1 << 20) or rows * ((vocab + 7 + 8191) // 8192) > MOST
    assert (need == 0) == refused
