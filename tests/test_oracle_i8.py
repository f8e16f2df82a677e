"""The 8-bit operators' 64-bit forms, pinned to hand-worked rows and to other formulations."""
import numpy as np
import pytest

from oracle import i8_oracle as ref


def test_quant_rows_by_hand():
    # units of 1/8: 127, -63.5 (to even: -64), 2.5 (to even: 2), 0.25; and a row of zeros
    q, s, _ = ref.quant_rows(np.array([[15.875, -7.9375, 0.3125, 0.03125], [0.0, 0.0, 0.0, 0.0]]))
    assert q.tolist() == [[127.0, -64.0, 2.0, 0.0], [0.0, 0.0, 0.0, 0.0]]
    assert s.tolist() == [0.125, 0.0]


def test_norm_of_a_scaled_row_is_the_weight():
    w = np.array([1.0, -2.0, 0.5, 3.0])
    v, n = ref.norm(np.full((2, 4), 7.0), np.full((2, 4), -3.0), w, 0.0)
    assert (v == 4.0).all() and np.allclose(n, w[None])


def test_linear_is_the_product_of_the_values():
    rng = np.random.default_rng(0)
    a, w = rng.integers(-127, 128, (3, 64)), rng.integers(-128, 128, (5, 64))
    sa, sw = rng.random(3), rng.random(5)
    assert np.allclose(ref.linear(a, sa, w, sw), (a * sa[:, None]) @ (w * sw[:, None]).T)


def test_scores_edges():
    inf, nan = np.inf, np.nan
    lg = np.array([[0.0, 0.0, -inf, nan], [inf, 1.0, inf, -inf], [-inf] * 4])
    assert ref.scores(lg, False).tolist() == [[0.5, 0.5, 0, 0], [0.5, 0, 0.5, 0], [0, 0, 0, 0]]
    assert ref.scores(lg, True).tolist() == [[0.5, 0.5, 0, 0], [1, 1 / (1 + np.exp(-1.0)), 1, 0],
                                             [0, 0, 0, 0]]


def test_groups_by_hand():
    # sums of two: group 0 -> 2 + 1, group 1 -> 4 + (-4), group 2 -> 1.4 + 1.5
    lg, bias = np.zeros((1, 6)), np.array([2, 1, 4, -4, 1.4, 1.5], np.float32)
    by = lambda **kw: ref.route_scored(lg, bias, 2, sigmoid=True, n_groups=3, **kw)[0].tolist()  # noqa: E731
    assert by(topk_groups=1, top2=True) == [[0, 1]]
    assert by(topk_groups=1, top2=False) == [[2, 3]]
    assert by(topk_groups=2, top2=True) == [[0, 5]]
    assert by(topk_groups=3, top2=True) == [[2, 0]]


def test_selection_equals_a_stable_sort_without_groups():
    rng = np.random.default_rng(1)
    lg = np.round(rng.normal(size=(40, 24)), 1).astype(np.float32)   # many ties
    idx, w = ref.route_scored(lg, None, 5, sigmoid=True)
    assert np.array_equal(idx, np.argsort(-lg, axis=1, kind="stable")[:, :5])
    assert np.allclose(w.sum(1), 1.0)


def test_ffn_bound_is_zero_away_from_borders():
    one = np.ones(1)
    x = np.array([[64, 0]])
    out, bound = ref.expert_ffn(x, one, (np.array([[1, 0]]), one), (np.array([[1, 0]]), one),
                                (np.array([[2]]), one))
    h = 64 * 64 / (1 + np.exp(-64.0))
    assert out[0, 0] == pytest.approx(2 * h) and bound[0, 0] <= out[0, 0] * 2 * ref.H_SHARE
