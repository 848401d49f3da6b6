"""The oracle's gradients of the training step's operators against central
differences of its own losses, and hand examples."""
import math

import numpy as np
import pytest

import oracle.train_oracle as o


def _differences(f, x, step=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + step
        up = f()
        x[i] = keep - step
        g[i] = (up - f()) / (2 * step)
        x[i] = keep
    return g


# central differences in 64 bits with a step of 1e-5: the truncation is about
# step^2 times the third derivative (a few units here), the cancellation about
# 2^-52 / step; both below 1e-9
TOL = 1e-8


@pytest.mark.parametrize("T,C", [(1, 1), (2, 2), (3, 7)])
def test_layer_norm_gradients(T, C):
    rng = np.random.default_rng(T * 10 + C)
    x, r = rng.normal(size=(T, C)), rng.normal(size=(T, C))
    w, b = rng.normal(size=C), rng.normal(size=C)
    gy, gh = rng.normal(size=(T, C)), rng.normal(size=(T, C))

    def loss():
        y, h, _, _ = o.layer_norm_forward(x, w, b, 0.1, r)
        return (y * gy).sum() + (h * gh).sum()

    _, h, mean, rstd = o.layer_norm_forward(x, w, b, 0.1, r)
    g_x, g_w, g_b = o.layer_norm_backward(gy, h, mean, rstd, w, gh)
    for got, at in ((g_x, x), (g_x, r), (g_w, w), (g_b, b)):
        assert np.allclose(got, _differences(loss, at), atol=TOL)


def test_token_logprob_gradient():
    rng = np.random.default_rng(1)
    x, t, g = rng.normal(size=(4, 6)), np.array([2, 5, -100, 0]), rng.normal(size=4)
    want = _differences(lambda: (o.token_logprob(x, t, 1.7)[0] * g).sum(), x)
    assert np.allclose(o.token_logprob_backward(g, x, t, 1.7), want, atol=TOL)
    assert (want[2] == 0).all()


def test_token_logprob_by_hand():
    x = np.array([[0.0, math.log(3.0)], [-np.inf, 2.0], [-np.inf, -np.inf]])
    lp, stats = o.token_logprob(x, np.array([1, 0, 1]))
    assert lp[0] == pytest.approx(math.log(0.75)) and stats[0, 1] == pytest.approx(4.0 / 3.0)
    assert lp[1] == -np.inf and tuple(stats[1]) == (2.0, 1.0)
    assert lp[2] == -np.inf and tuple(stats[2]) == (-np.inf, 0.0)


@pytest.mark.parametrize("kl", [0.0, 0.3])
def test_policy_loss_gradient(kl):
    rng = np.random.default_rng(2)
    lp, old, ref, A = (rng.normal(size=40) * 0.5 for _ in range(4))
    w = rng.uniform(size=40) * (rng.uniform(size=40) > 0.2)
    f = lambda: o.policy_loss(lp, old, A, w, ref, 0.1, 0.3, kl)[0][0]
    g = o.policy_loss(lp, old, A, w, ref, 0.1, 0.3, kl)[1]
    assert np.allclose(g, _differences(f, lp), atol=TOL)
    assert o.policy_loss(lp, old, A, w, ref, 0.1, 0.3, kl)[0][2] > 0


@pytest.mark.parametrize("mean", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_preference_loss_gradient(mean, weighted):
    rng = np.random.default_rng(3)
    lp, ref = rng.normal(size=23), rng.normal(size=23)
    start = [0, 4, 4, 11, 15, 20, 23]         # P = 3, an empty sequence among them
    w = rng.integers(0, 3, 23).astype(float) if weighted else None
    f = lambda: o.preference_loss(lp, start, 0.7, ref, w, 0.2, mean)[0]
    g = o.preference_loss(lp, start, 0.7, ref, w, 0.2, mean)[2]
    assert np.allclose(g, _differences(f, lp), atol=TOL)


def test_clip_by_hand():
    norm, out = o.clip_grad_norm([np.array([3.0]), np.array([]), np.array([0.0, -4.0])], 1.0)
    assert norm == 5.0 and out[2][1] == pytest.approx(-0.8, rel=1e-6)
    assert o.clip_grad_norm([np.array([3.0, -4.0])], 8.0, True)[0] == 4.0


def test_bf16_rounding_by_hand():
    e = 2.0 ** -8
    v = [1.0 + e, 1.0 + 3 * e, 1.0 + e + 2.0 ** -40, -(1.0 + e), 2.0 ** -140, np.inf]
    assert o.round_bf16(v).tolist() == [1.0, 1.0 + 4 * e, 1.0 + 2 * e, -1.0, 0.0, np.inf]
