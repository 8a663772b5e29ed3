"""The sparse attention's oracle on cases small enough to see through."""
import numpy as np
import pytest

from oracle import kv as okv
from oracle import sparse as osp


def test_a_page_score_bounds_its_keys_and_is_reached_where_one_key_holds_the_limits():
    rng = np.random.default_rng(0)
    K = rng.standard_normal((8, 6))
    q = rng.standard_normal((5, 6))
    hi, lo = osp.limits(K)
    for r in q:
        assert osp.score(r[None], hi, lo) >= (K @ r).max() - 1e-12
    one = K[:1]
    assert np.isclose(osp.score(q[:1], *osp.limits(one)), float((one @ q[0])[0]))


def test_selection_takes_the_kept_pages_the_best_and_the_lower_among_equals():
    K = np.zeros((10, 1, 2))
    K[:, 0, 0] = [1, 1, 5, 5, 2, 2, 5, 5, 0, 0]  # pages of two slots: 1 5 2 5 0
    q = np.array([[[1.0, 0.0]]])
    assert osp.select(q, K, 2, 5, 2)[0].tolist() == [[1, 3]]
    assert osp.select(q, K, 2, 5, 1)[0].tolist() == [[1]]
    assert osp.select(q, K, 2, 5, 3, first=1, last=1)[0].tolist() == [[0, 1, 4]]
    assert osp.select(q, K, 2, 5, 5)[0].tolist() == [[0, 1, 2, 3, 4]]
    assert osp.select(-q, K, 2, 5, 1)[0].tolist() == [[4]]
    there = np.array([True, False, True, False, True])
    assert osp.select(q, K, 2, 5, 3, there=there)[0].tolist() == [[0, 2, 4]]


def test_shared_selections_go_by_their_best_row_and_leave_out_rows_that_are_not_finite():
    K = np.zeros((6, 1, 2))
    K[:, 0] = [[1, 0], [1, 0], [0, 2], [0, 2], [0, 0], [0, 0]]
    q = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[np.nan, 0.0]]])
    assert [s.tolist() for s in osp.select(q, K, 2, 3, 1, share=1)] == [[[0]], [[1]], [[0]]]
    assert [s.tolist() for s in osp.select(q, K, 2, 3, 1, share=0)] == [[[1]]]
    assert [s.tolist() for s in osp.select(q, K, 2, 3, 1, share=2)] == [[[1]], [[0]]]
    K[4, 0, 0] = np.nan  # a page with a key that is not a number comes first
    assert [s.tolist() for s in osp.select(q, K, 2, 3, 1, share=2)] == [[[2]], [[2]]]


def test_everything_selected_is_dense_attention():
    rng = np.random.default_rng(1)
    K, V, q = rng.standard_normal((9, 1, 4)), rng.standard_normal((9, 1, 4)), rng.standard_normal((2, 2, 4))
    see = okv.visible_causal(7, 2)
    part = osp.visible(see, [0, 1, 2], 2, 3)
    assert np.array_equal(part, see)
    fewer = osp.visible(see, [1], 2, 3)
    assert fewer[0].tolist() == [False, False, True, True, False, False, True, True, False]
    assert np.allclose(okv.attention(q, K, V, fewer, 0.5),
                       okv.attention(q, K[2:4].repeat(1, 0).tolist() + K[6:].tolist(),
                                     V[2:4].tolist() + V[6:].tolist(),
                                     np.array([[1, 1, 1, 1, 0], [1, 1, 1, 1, 1]], dtype=bool), 0.5))


@pytest.mark.parametrize("bits,spread", [(8, 35), (24, 19)])
def test_sums_of_a_rows_products_are_exact_within_a_spread(bits, spread):
    """Products of a q of so many bits (bf16, fp32) and a limit of two (a 4-bit float times a power of
    two): 256 of them within `spread` binades have the same fp64 sum in any order, and that is the exact one."""
    rng = np.random.default_rng(bits)
    most = (2 ** bits - 1) * 3
    for case in range(20):
        mant = rng.integers(most // 2, most + 1, 256)
        power = rng.integers(0, spread + 1, 256)
        if case == 0:  # the largest sum beside the smallest unit
            mant[:], power[:] = most, spread
            mant[0], power[0] = 1, 0
        exact = sum(int(m) << int(p) for m, p in zip(mant, power))
        terms = [float(int(m)) * 2.0 ** int(p) for m, p in zip(mant, power)]
        for _ in range(5):
            total = 0.0
            for i in rng.permutation(256):
                total += terms[i]
            assert int(total) == exact
            parts = [sum(terms[i] for i in range(k, 256, 16)) for k in range(16)]  # lanes first, then their sums
            assert int(sum(parts)) == exact


def test_sums_that_spread_further_round():
    assert 1.0 + 255 * 765 * 2.0 ** 38 == 255 * 765 * 2.0 ** 38
