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


# ------------------------------------------------------------ policy loss

def _banned_case(T, V, name, seed):
    """Logits whose first rows have targets that nothing can sample, with the
    other inputs of the policy loss; which rows have a finite KL term."""
    import torch
    from test_gpu_train import _logits, _policy_inputs
    x, t = _logits(T, V, name, seed)
    low = torch.finfo(x.dtype).min
    s = _policy_inputs(x, t, 1.0, seed, zero=0.0)
    x[0, t[0]] = -INF                          # banned
    x[1, t[1]] = low                           # banned by the type's lowest value
    x[2] = -INF                                # nothing allowed
    x[3] = -INF                                # the target is all that is allowed
    x[3, t[3]] = 1.0
    s["old"][3], s["ref"][3] = 0.1, -0.2       # (its log probability is 0)
    s["ref"][4] = -INF                         # banned by the reference alone
    s["old"][5], s["adv"][5] = low, 0.0        # by the old policy, without an advantage
    s["w"][:] = 1.0 / T
    return x, t, s, np.isin(np.arange(T), [0, 1, 2, 4], invert=True)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(8, 5), (8, 1001), (300, 1001), (300, 4099), (8, 32003),
                                 (8, 65541), (8, 140001)])
def test_policy_loss_of_banned_targets(T, V, name):
    import torch
    import hadamard_rank_linear_amd as h
    from test_gpu_train import _clear_of_the_border, _dev, _gradient_tolerance, _logit_errors, \
        _within
    _say(f"policy: banned targets, T={T} V={V} {name}")
    x, t, s, finite = _banned_case(T, V, name, T + V)
    xn, tn = _np(x), t.numpy()
    olp = o.token_logprob(xn, tn)[0]
    assert olp[0] == -INF and olp[2] == -INF and -INF < olp[1] < -1e38 and olp[3] == 0.0
    e_lp, e_s = _logit_errors(xn, tn, 1.0)
    _clear_of_the_border(olp, s, 0.2, 0.28, 1e-3)
    c = lambda v: torch.from_numpy(v).cuda()
    for kl, keep in ((0.0, np.ones(T, bool)), (0.05, np.ones(T, bool)), (0.05, finite)):
        w = np.where(keep, s["w"], 0.0).astype(np.float32)
        ref = s["ref"] if kl else None
        osums, og = o.policy_loss(olp, s["old"], s["adv"], w, ref, 0.2, 0.28, kl)
        assert np.isfinite(osums).all() == (kl == 0.0 or not keep.all()) and not np.isnan(og).any()
        want = o.token_logprob_backward(og, xn, tn)
        args = [c(s["old"]), c(s["adv"]), c(w)]
        kw = dict(ref_logprob=c(ref) if kl else None, clip_low=0.2, clip_high=0.28, kl_coef=kl)
        out = []
        for place in (False, True):            # the second time in place of the logits
            dx = _dev(x, name, 1)
            sums, lp, g_x = h.hlq_policy_loss_logits(dx, t.cuda(), *args, g_x=dx if place else None,
                                                     **kw)
            torch.cuda.synchronize()
            out.append((sums, lp, g_x))
        assert all(torch.equal(a, b) for a, b in zip(*out))
        # the log probability's error moves the ratio and exp(d) in proportion
        live = keep & np.isfinite(og) & np.isfinite(olp) & (olp > -1e38)
        ratio = np.exp(np.where(live, np.minimum(olp - s["old"], 50.0), 0.0))
        away = np.exp(np.where(live, np.minimum(s["ref"] - olp, 50.0), 0.0))
        move = np.where(live, 1.01 * e_lp, 0.0) * w
        e_g = move * (ratio * np.abs(s["adv"]) + kl * away)
        tol = np.array([e_g.sum(), (move * np.abs(away - 1)).sum(), 0.0])
        _within(_np(sums), osums, np.where(np.isfinite(osums), 1.01 * tol + 2 * U * np.abs(osums), 0)
                + 1e-12, "sums")
        fin = np.isfinite(og)
        with np.errstate(invalid="ignore"):
            g_tol = _gradient_tolerance(xn, tn, np.where(fin, og, 0.0), e_s, 1.0, name,
                                        np.where(np.isfinite(want), want, 0.0))
            half = 2.0 ** -8 if name == "bf16" else 0.0
            for i in np.flatnonzero(live):
                g_tol[i] += (1 + half) * np.abs(want[i]) * (e_g[i] / max(abs(og[i]), 1e-30) + 2 * U)
        _within(_np(g_x), want, g_tol, "g_x")
        # through the log probabilities
        lp1, stats = h.hlq_token_logprob_forward(_dev(x, name, 1), t.cuda())
        sums2, g_lp = h.hlq_policy_loss(lp1, *args, **kw)
        g_x2 = h.hlq_token_logprob_backward(g_lp, _dev(x, name, 1), t.cuda(), stats)
        torch.cuda.synchronize()
        assert np.array_equal(np.isfinite(_np(sums2)), np.isfinite(osums))
        assert not np.isnan(_np(sums2)).any() and not np.isnan(_np(g_lp)).any()
        assert np.array_equal(_np(g_lp) == -INF, og == -INF)
        assert np.array_equal(np.isinf(_np(g_x2)), np.isinf(want)) and \
            not np.isnan(_np(g_x2)).any()
        assert (_np(g_x2)[want == 0] == 0).all()


def test_policy_loss_does_not_hide_nan():
    # an advantage of zero takes out a ratio past the range, not one that is no number
    import torch
    import hadamard_rank_linear_amd as h
    _say("policy: NaN logits under an advantage of zero")
    x, t = torch.zeros(3, 40, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    x[1, 7] = math.nan
    old, adv = torch.zeros(3, device="cuda"), torch.zeros(3, device="cuda")
    sums, lp, _ = h.hlq_policy_loss_logits(x, t, old, adv)
    sums2, _ = h.hlq_policy_loss(lp, old, adv)
    torch.cuda.synchronize()
    assert torch.isnan(lp).tolist() == [False, True, False]
    assert torch.isnan(sums[0]) and torch.isnan(sums2[0])


# ------------------------------------------------------------ many pairs

def test_preference_loss_of_more_pairs_than_a_launch_takes():
    # more workgroups than a launch holds threads for; a token a sequence, so the
    # margins are differences of single tokens
    import torch
    import hadamard_rank_linear_amd as h
    P = (1 << 22) + 5
    _say(f"preference: P={P}")
    g = torch.Generator(device="cuda").manual_seed(9)
    lp = -torch.rand(2 * P, generator=g, device="cuda")
    start = torch.arange(2 * P + 1, device="cuda")
    loss, margin, g_lp = h.hlq_preference_loss(lp, start, 0.5)
    torch.cuda.synchronize()
    d = lp.double()
    z = 0.5 * (d[:P] - d[P:])
    x = torch.exp(-z)
    want = 0.5 / P * (1.0 / (1.0 + x) - 1.0)
    assert ((margin - z).abs() <= 2 * U * z.abs()).all()
    assert ((g_lp[:P] - want).abs() <= 2 * U * want.abs()).all()
    assert torch.equal(g_lp[P:], -g_lp[:P])
    assert abs(loss.item() - torch.log1p(x).mean().item()) <= 2 * U


# ------------------------------------------------------------ clipping

@pytest.mark.parametrize("kind", ["l2", "inf"])
@pytest.mark.parametrize("value,max_norm", [(3e38, 1.0), (3e38, 1e-3), (1e20, 1e-25), (1e30, 1e-12),
                                            (3e38, 1e-37), (1.0, 1e-30), (1.0, 1e-31)])
def test_clip_by_a_factor_below_the_range(kind, value, max_norm):
    # the factor (3e-33 to 1e-75 here) is no fp32 number, or one of few bits; its
    # rounding, the product's and the output's are half a step each
    import torch
    import hadamard_rank_linear_amd as h
    _say(f"clip of gradients of {value} to {max_norm}, {kind}")
    rng = np.random.default_rng(4)
    host = [torch.from_numpy(value * rng.uniform(0.1, 1.0, n)).to(dt)
            for n, dt in ((1000, torch.float32), (9, torch.bfloat16), (4099, torch.float32))]
    norm, want = o.clip_grad_norm([_np(v) for v in host], max_norm, kind == "inf")
    code = h.HLQ_NORM_L2 if kind == "l2" else h.HLQ_NORM_INF
    out = [torch.empty_like(v, device="cuda") for v in host]
    got = h.hlq_clip_grad_norm(own := [v.cuda() for v in host], max_norm, code, out=out)
    h.hlq_clip_grad_norm(own, max_norm, code)
    torch.cuda.synchronize()
    assert got.item() == pytest.approx(norm, rel=2.0 ** -33)
    for a, b, v in zip(out, own, want):
        half = torch.finfo(a.dtype).eps / 2
        # below the type's normal range steps do not shrink any more: one of those
        step = 2 * half * torch.finfo(a.dtype).smallest_normal
        assert (np.abs(_np(a) - v) <= (2 * U + half * (1 + 2 * U)) * np.abs(v) + step).all()
        assert torch.equal(a, b)
