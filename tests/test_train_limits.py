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
