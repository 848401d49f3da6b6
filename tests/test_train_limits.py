"""The oracle at log probabilities of -inf, by hand."""
import numpy as np
import pytest

import oracle.train_oracle as o

INF = float("inf")


@pytest.mark.parametrize("mean", [False, True])
def test_preference_loss_of_banned_targets(mean):
    # pairs: a rejected token of probability zero, a chosen one, none
    lp = np.array([-1.0, -INF, -2.0, -INF, -1.0, -2.0])
    start = range(7)
    loss, margin, g = o.preference_loss(lp, start, 0.5, smoothing=0.0, mean=mean)
    assert margin.tolist() == [INF, -INF, 0.0] and loss == INF
    assert g == pytest.approx(np.array([0.0, -0.5, -0.25, 0.0, 0.5, 0.25]) / 3)
    keep = [0, 2, 3, 5]                        # without the chosen one
    loss, margin, g = o.preference_loss(lp[keep], range(5), 0.5, smoothing=0.0, mean=mean)
    assert margin.tolist() == [INF, 0.0] and loss == pytest.approx(np.log(2.0) / 2)
    assert o.preference_loss(lp[[0, 3]], range(3), 0.5, smoothing=0.1)[0] == INF
    assert o.preference_loss(lp[[3, 0]], range(3), 0.5, smoothing=1.0)[0] == 0.0


def test_policy_loss_of_banned_targets():
    # a banned target, one banned by the reference alone, a ratio past the range without an advantage
    lp, old = np.array([-INF, -1.0, -1.0]), np.array([-2.0, -1.0, -1000.0])
    A, ref = np.array([1.0, 1.0, 0.0]), np.array([-2.0, -INF, -1.0])
    sums, g = o.policy_loss(lp, old, A)
    assert sums.tolist() == [-1.0, 0.0, 0.0] and g.tolist() == [0.0, -1.0, 0.0]
    sums, g = o.policy_loss(lp, old, A, None, ref, kl_coef=0.5)
    assert sums.tolist() == [INF, INF, 0.0] and g.tolist() == [-INF, -0.5, 0.0]
    sums, g = o.policy_loss(np.array([np.nan]), old[:1], np.zeros(1))    # NaN is not hidden
    assert np.isnan(sums[0])


def test_infinite_gradient_of_a_log_probability():
    x = np.array([[-INF, 0.0, -INF, 0.0], [0.0, -INF, -INF, -INF]])
    g = o.token_logprob_backward(np.array([-INF, INF]), x, np.array([0, 0]))
    assert g.tolist() == [[-INF, INF, 0.0, INF], [0.0, 0.0, 0.0, 0.0]]
