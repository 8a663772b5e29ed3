"""The log probabilities' oracle by hand and against its own identities."""
import numpy as np

from oracle import logprobs as olp


def test_three_tokens_by_hand():
    logp, h = olp.logprobs(np.log([1.0, 2.0, 5.0]))
    assert np.allclose(np.exp(logp), [1 / 8, 2 / 8, 5 / 8])
    assert np.isclose(h, -(np.log(1 / 8) / 8 + np.log(2 / 8) * 2 / 8 + np.log(5 / 8) * 5 / 8))
    tok, lp = olp.alternatives(np.log([1.0, 2.0, 5.0]), 2)
    assert tok.tolist() == [2, 1] and np.allclose(np.exp(lp), [5 / 8, 2 / 8])


def test_entropy_is_the_mean_of_minus_the_log_probability():
    x = np.random.default_rng(0).standard_normal(1000) * 4
    logp, h = olp.logprobs(x)
    assert np.isclose(np.exp(logp).sum(), 1) and np.isclose(h, -(np.exp(logp) * logp).sum())


def test_ties_and_logits_that_are_not_finite():
    tok, lp = olp.alternatives([1.0, 3.0, np.nan, 3.0, -np.inf, 1.0], 6)
    assert tok.tolist() == [1, 3, 0, 5, -1, -1] and (lp[4:] == -np.inf).all()
    tok, lp = olp.alternatives([1.0, np.inf, np.inf], 3)
    assert tok.tolist() == [1, 2, -1] and np.allclose(lp[:2], -np.log(2))
    logp, h = olp.logprobs([np.nan, -np.inf])
    assert (logp == -np.inf).all() and h == 0.0
    assert olp.alternatives([np.nan, -np.inf], 2)[0].tolist() == [-1, -1]
