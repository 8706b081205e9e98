"""Pins of the 64-bit definitions in oracle/moe.py: hand-worked choices,
invariants, and every gradient against central differences."""
import numpy as np
import pytest

from oracle import moe

INF = float("inf")


def test_choice_by_hand():
    ids, w, _ = moe.route_row([0.0, 2.0, 2.0, 1.0], 3)
    assert ids.tolist() == [1, 2, 3]                      # equal logits: the lower index first
    e = np.exp([2.0, 2.0, 1.0])
    assert np.allclose(w, e / e.sum(), rtol=1e-15)
    ids, w, _ = moe.route_row([-INF, 5.0, -INF, -3e38], 3, renorm=False, scale=2.0)
    assert ids.tolist() == [1, 3, -1] and w.tolist() == [2.0, 0.0, 0.0]
    ids, w, _ = moe.route_row([-INF] * 4, 2, score=moe.SIGMOID)
    assert ids.tolist() == [-1, -1] and w.tolist() == [0.0, 0.0]


def test_bias_steers_the_choice_and_not_the_weights():
    l = np.array([1.0, 0.0, -1.0])
    ids, w, _ = moe.route_row(l, 1, score=moe.SIGMOID, bias=[0.0, 0.0, 0.9], renorm=False)
    assert ids.tolist() == [2] and np.isclose(w[0], 1 / (1 + np.e))
    ids, _, _ = moe.route_row(l, 3, score=moe.SIGMOID, bias=[0.0, -INF, 0.0])
    assert ids.tolist() == [0, 2, -1]


def test_a_nan_score_does_not_bring_back_what_the_bias_takes_away():
    nan = float("nan")
    for score in (moe.SOFTMAX, moe.SIGMOID):
        ids, _, _ = moe.route_row([nan, 1.0, nan, 0.0], 4, score=score, bias=[-INF, 0.0, 0.0, -INF])
        assert ids.tolist() == [1, 2, -1, -1]


def test_groups_by_hand():
    #        group 0      group 1       group 2
    l = [3.0, -9.0, 2.0, 1.9, 2.5, -INF]
    assert moe.route_row(l, 2, groups=3, top_groups=1, group_best=1)[0].tolist() == [0, 1]
    # sums of two sigmoids: group 1 leads (0.881 + 0.870), group 0 has 0.953, group 2 0.924 alone
    assert moe.route_row(l, 2, score=moe.SIGMOID, groups=3, top_groups=1, group_best=2)[0].tolist() == [2, 3]
    assert moe.route_row(l, 3, score=moe.SIGMOID, groups=3, top_groups=2, group_best=2)[0].tolist() == [0, 2, 3]
    # a group with nothing available is never one of the kept that give experts
    assert moe.route_row([-INF, -INF, 1.0, 2.0], 2, groups=2, top_groups=1)[0].tolist() == [3, 2]


def test_renormalised_scores_keep_their_proportions_where_they_underflow():
    for score in (moe.SOFTMAX, moe.SIGMOID):
        w = moe.route_row([-2000.0, -2001.0, -3000.0], 2, score=score)[1]
        assert np.allclose(w, [1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))], rtol=1e-12)


@pytest.mark.parametrize("score", [moe.SOFTMAX, moe.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(7)
    for _ in range(6):
        n, k = 9, 4
        l, dw = rng.normal(0, 2, n), rng.normal(0, 1, k)
        ids = moe.route_row(l, k, score=score)[0]
        ids[1] = -1                                       # a place without an expert
        got = moe.route_bwd_row(l, ids, dw, score, renorm, 2.5)
        for e in range(n):
            h = 1e-6
            up, down = l.copy(), l.copy()
            up[e] += h
            down[e] -= h
            d = (moe.weights_of(up, ids, score, renorm, 2.5) - moe.weights_of(down, ids, score, renorm, 2.5)) / (2 * h)
            assert abs((d * dw).sum() - got[e]) < 1e-8


def test_plan_by_hand():
    ids = np.array([[1, 0], [-1, 1], [0, 2]], dtype=np.int32)
    offsets, row_index, slot = moe.route_plan(ids, 4)
    assert offsets.tolist() == [0, 2, 4, 5, 5]
    assert row_index.tolist() == [0, 2, 0, 1, 2, 1]
    assert slot.tolist() == [[2, 0], [-1, 3], [1, 4]]


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(3)
    y, w, dout = rng.normal(size=(6, 5)), rng.random((3, 2)), rng.normal(size=(3, 5))
    slot = np.array([[4, 0], [-1, 2], [5, 9]], dtype=np.int32)

    def value(y, w):
        return (moe.combine(y, slot, w) * dout).sum()

    dy, dw = moe.combine_bwd(dout, y, slot, w)
    h = 1e-6
    for r in range(6):
        for c in range(5):
            up, down = y.copy(), y.copy()
            up[r, c] += h
            down[r, c] -= h
            want = 0.0 if np.isnan(dy[r, c]) else dy[r, c]
            assert abs((value(up, w) - value(down, w)) / (2 * h) - want) < 1e-8
    for t in range(3):
        for j in range(2):
            up, down = w.copy(), w.copy()
            up[t, j] += h
            down[t, j] -= h
            assert abs((value(y, up) - value(y, down)) / (2 * h) - dw[t, j]) < 1e-8


def test_clip_by_hand():
    assert moe.grad_norm([[3.0], [[0.0, 4.0]]]) == 5.0
    assert moe.clip_coef(5.0, 1.0) == 1.0 / (5.0 + 1e-6) and moe.clip_coef(0.5, 1.0) == 1.0
    assert moe.clip_coef(INF, 1.0) == 1.0 and moe.clip_coef(float("nan"), 1.0) == 1.0 and moe.clip_coef(2.0, 0.0) == 0.0
