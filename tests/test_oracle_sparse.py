"""The sparse attention's oracle on cases small enough to see through."""
import numpy as np

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
