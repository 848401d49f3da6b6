"""The losses at log probabilities of -inf: what scoring returns for a target
that a mask has banned, and for a row that it has banned whole."""
import math

import numpy as np
import pytest

import oracle.train_oracle as o

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = math.inf


def _say(msg):
    print(f"\n[gpu-case] {msg}", flush=True)


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, want, rel, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want)
    bad = ~((off <= rel * np.abs(want) + 1e-14) | (got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), f"{what}: {got[bad][:4]} for {want[bad][:4]} at {np.argwhere(bad)[:4]}"


@pytest.mark.parametrize("smoothing", [0.0, 0.1, 1.0])
@pytest.mark.parametrize("mean", [False, True])
@pytest.mark.parametrize("P,length", [(3, 4), (3, 600), (20, 5)])
def test_preference_loss_of_banned_targets(P, length, mean, smoothing):
    # every way through the kernels; sums in 64 bits, so an output is off by its
    # rounding and the loss by half a step more
    import torch
    import hadamard_rank_linear_amd as h
    _say(f"preference: banned targets, P={P} length={length} mean={mean} smoothing={smoothing}")
    rng = np.random.default_rng(P + length)
    T = 2 * P * length
    lp, ref = (rng.normal(size=T).astype(np.float32) - 2 for _ in range(2))
    start = np.arange(2 * P + 1) * length
    c = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()
    red = h.HLQ_MEAN if mean else h.HLQ_SUM

    def check(v):
        loss, margin, g = h.hlq_preference_loss(c(v), c(start), 0.3, c(ref),
                                                label_smoothing=smoothing, reduction=red)
        torch.cuda.synchronize()
        ol, om, og = o.preference_loss(v.astype(np.float64), start, 0.3, ref, None, smoothing,
                                       mean)
        _close(_np(margin), om, 2 * U, "margin")
        _close(_np(loss), [ol], 2 * U + 1e-10, "loss")
        _close(_np(g), og, 2 * U, "g_logprob")
        assert np.isfinite(og).all()
        return ol, om

    bad = lp.copy()
    bad[start[P + 1] + length - 1] = -INF      # in a rejected sequence
    loss, margin = check(bad)
    assert margin[1] == INF and math.isfinite(loss) == (smoothing == 0.0)
    bad = lp.copy()
    bad[start[2]] = -INF                       # in a chosen one
    loss, margin = check(bad)
    assert margin[2] == -INF and math.isfinite(loss) == (smoothing == 1.0)
