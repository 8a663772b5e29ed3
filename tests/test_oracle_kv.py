"""Pins of the 4-bit cache's and the acceptance's oracles: hand-worked values, closed forms and
frequencies of the plain definition."""
import numpy as np
import pytest

from oracle import accept as oaccept
from oracle import kv as okv


@pytest.mark.parametrize("amax,e", [(0.0, -125), (4.0, 0), (6.0, 0), (7.0, 0), (7.0001, 1), (8.0, 1),
                                    (1.0, -2), (3.5, -1), (3.51, 0), (2.0 ** -140, -125), (3.4e38, 125)])
def test_block_exponent(amax, e):
    assert okv.block_exponent(amax) == e


def test_nearest_ties_go_to_the_even_code():
    y = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.0, 100.0, 0.24, 0.26]
    assert okv.nearest(y).tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0, 6.0, 0.0, 0.5]


def test_stored_blocks_are_separate_and_exact_on_grid_values():
    rng = np.random.default_rng(3)
    x = rng.choice(np.concatenate([okv.GRID, -okv.GRID]), size=(5, 64))
    x[:, 0], x[:, 32] = 6.0, 4.0
    x[:, 32:] *= 2.0 ** 20
    assert np.array_equal(okv.stored(x), x)
    noisy = rng.standard_normal((50, 128))
    err = np.abs(okv.stored(noisy) - noisy).reshape(50, 4, 32)
    amax = np.abs(noisy).reshape(50, 4, 32).max(-1, keepdims=True)
    assert np.all(err <= amax / 4 + 1e-15)  # half the widest step (2 of 8 after scaling)


def test_stored_pair_poisons_one_head_only():
    k, v = np.ones((2, 3, 64)), np.ones((2, 3, 64))
    v[1, 2, 5] = np.inf
    ks, vs = okv.stored_pair(k, v)
    assert np.isnan(ks[1, 2]).all() and (vs[1, 2] == 0).all()
    assert np.isfinite(np.delete(ks.reshape(6, 64), 5, 0)).all()


def test_attention_closed_forms():
    rng = np.random.default_rng(4)
    K, V = np.zeros((5, 2, 8)), rng.standard_normal((5, 2, 8))
    q = rng.standard_normal((3, 4, 8))
    see = okv.visible_causal(2, 3)
    out = okv.attention(q, K, V, see, 0.3)  # equal scores: the mean of what a row sees
    for i in range(3):
        for h in range(4):
            assert np.allclose(out[i, h], V[:3 + i, h // 2].mean(0))
    see[1] = False
    assert (okv.attention(q, K, V, see, 0.3)[1] == 0).all()
    tree = okv.visible_tree([-1, 0, 0, 1], 1).astype(int)
    assert tree.tolist() == [[1, 1, 0, 0, 0], [1, 1, 1, 0, 0], [1, 1, 0, 1, 0], [1, 1, 1, 0, 1]]


def test_accept_draws_from_the_target():
    """Over evenly spaced random numbers the first drawn token has the softmax's frequencies,
    whatever the children are."""
    rng = np.random.default_rng(5)
    V, T = 7, 0.8
    logits = rng.standard_normal((4, V))
    parent, tokens = [-1, 0, 0, 0], [0, 3, 3, 6]
    u = (np.arange(20000) + 0.5) / 20000
    count = np.zeros(V)
    for x in u:
        path, nxt = oaccept.accept(parent, tokens, logits, [x] * 4, T)
        count[tokens[path[1]] if len(path) > 1 else nxt] += 1
    p = np.exp(logits[0] / T)
    assert np.abs(count / 20000 - p / p.sum()).max() <= 1.0 / 20000 + 1e-12


def test_accept_walks_and_stops():
    V = 5
    logits = np.full((4, V), -np.inf)
    logits[0, 2] = logits[1, 4] = 1.0
    logits[2, 0] = logits[2, 3] = 2.0
    parent, tokens = [-1, 0, 1, 1], [0, 2, 4, 1]
    assert oaccept.accept(parent, tokens, logits, [0.9] * 4, 1.0) == ([0, 1, 2], 3)
    assert oaccept.accept(parent, tokens, logits, [0.1] * 4, 1.0) == ([0, 1, 2], 0)
    assert oaccept.accept(parent, tokens, logits, [0.9] * 4, 0.0) == ([0, 1, 2], 0)  # lowest index
    logits[2] = np.nan
    assert oaccept.accept(parent, tokens, logits, [0.1] * 4, 1.0) == ([0, 1, 2], -1)
    # only children have weight: nothing else can be drawn
    logits[1, :] = [-np.inf, 0.0, -np.inf, -np.inf, 0.0]
    for x, end in ((0.2, 2), (0.7, 3)):
        assert oaccept.accept(parent, tokens, logits, [x] * 4, 1.0)[0] == [0, 1, end]


def test_the_largest_of_a_block_is_off_by_a_fifth_at_most():
    """Half the step of 2 above 4: at 5 a fifth, at 7 and beyond a seventh; a quarter where the exponent
    is held at 125."""
    def off(x):
        row = np.zeros(32)
        row[3] = x
        return abs(okv.stored(row)[3] - x) / x
    assert off(5.0) == 0.2 and off(7.0) == 1 / 7
    assert max(off(x) for x in np.linspace(4, 8, 4097)[:-1]) == 0.2
    assert max(off(x) for x in np.linspace(7, 8, 4097)[:-1]) == pytest.approx(1 / 7)
    assert off(7.5 * 2.0 ** 124) < 0.2 and off(7.0 * 2.0 ** 125) == 1 / 7
    assert off(float(np.finfo(np.float32).max)) == pytest.approx(0.25, abs=1e-6)
