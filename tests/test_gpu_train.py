"""The training step's operators on the GPU against their definitions in 64
bits (oracle/train_oracle.py), at the sizes, masks and layouts where they can
go wrong.

Tolerances, with u = 2^-24 the half step of fp32 and e the half step of the
output's type (2^-8 relative for bf16):
 - a sum of n fp32 terms, added k at a time by a thread and then over a tree,
   is off by at most (k + 12) u sum|terms|; no kernel gives a thread more than
   64 + n / 256 terms;
 - an exponential 2^(c d), d the logit above the maximum: c is rounded (u),
   d is (u), so is c d (u): 3 u |c d| ln 2 + 2 u relative;
 - each further operation: u.
"""
import math

import numpy as np
import pytest

import oracle.train_oracle as o

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}


def _torch():
    import torch
    return torch


def _h():
    import hadamard_rank_linear_amd as h
    return h


def _dt(name):
    t = _torch()
    return {"f32": t.float32, "bf16": t.bfloat16}[name]


def _round(name):
    return o.round_bf16 if name == "bf16" else o.round_f32


def _say(msg):
    print(f"\n[gpu-case] {msg}", flush=True)


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _dev(v, name, offset=0):
    """v on the GPU, contiguous, starting ``offset`` elements into its storage."""
    torch = _torch()
    v = torch.as_tensor(v)
    buf = torch.full((v.numel() + offset + 32,), float("nan"), dtype=_dt(name), device="cuda")
    out = buf[offset:offset + v.numel()].view(v.shape)
    out.copy_(v)
    return out


def _within(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    tol = np.broadcast_to(tol, want.shape)
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want)
    bad = ~((off <= tol) | (got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at "
                           f"{np.argwhere(bad)[0]}: {got[bad][0]} for {want[bad][0]} "
                           f"(tolerance {tol[bad][0]})")


def _terms(n):
    return 64 + n / 256 + 12


# ------------------------------------------------------------ layer norm

NORM_SHAPES = [(1, 1), (1, 8), (3, 7), (2, 64), (65, 100), (5, 129), (7, 257), (33, 768), (17, 770),
               (2, 1000), (9, 1536), (3, 2048), (1, 4096), (5, 5001), (3, 8192), (2, 16384),
               (3, 16385), (2, 40003)]


def _norm_case(T, C, name, param, seed, shift=0.3):
    torch = _torch()
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x = r(T, C) * torch.exp(0.5 * r(C)) + shift
    return dict(x=x.to(_dt(name)), residual=(0.5 * r(T, C)).to(_dt(name)),
                weight=(1 + 0.1 * r(C)).to(_dt(param)), bias=(0.1 * r(C)).to(_dt(param)),
                g_y=(1e-3 * r(T, C)).to(_dt(name)), g_h=(1e-3 * r(T, C)).to(_dt(name)))


def _check_norm_forward(s, name, residual, bias, offset, eps=1e-5, param="f32"):
    h = _h()
    T, C = s["x"].shape
    args = {k: _dev(s[k], name, offset) for k in ("x", "residual")}
    w, b = _dev(s["weight"], param, offset), _dev(s["bias"], param, offset)
    y, hh, mean, rstd = h.hlq_layer_norm_forward(args["x"], w, b if bias else None, eps,
                                                 residual=args["residual"] if residual else None)
    _torch().cuda.synchronize()
    oy, oh, om, orr = o.layer_norm_forward(_np(s["x"]), _np(s["weight"]),
                                           _np(s["bias"]) if bias else None, eps,
                                           _np(s["residual"]) if residual else None, _round(name))
    assert np.array_equal(_np(hh), oh)          # one rounding of an exact sum
    k = _terms(C) * U
    e_mean = k * np.abs(oh).mean(-1)
    _within(_np(mean), om, e_mean + U * np.abs(om), "mean")
    # the variance: its sum, the squares, and (error of the mean)^2
    var = 1.0 / orr ** 2
    rel = 0.5 * ((k + 4 * U) + (2 * e_mean * np.abs(oh - om[:, None]).mean(-1) * k + e_mean ** 2) /
                 var) + 3 * U
    _within(_np(rstd), orr, rel * orr, "rstd")
    d = np.abs(oh - om[:, None]) * orr[:, None] * np.abs(_np(s["weight"]))
    tol = d * (rel[:, None] + 4 * U) + (e_mean * orr)[:, None] * np.abs(_np(s["weight"])) + \
        2 * U * np.abs(oy) + HALF[name] * np.abs(oy)
    _within(_np(y), oy, tol * 1.01 + 1e-38, "y")


@pytest.mark.parametrize("name,param", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                        ("f32", "bf16")])
@pytest.mark.parametrize("T,C", NORM_SHAPES)
def test_layer_norm_forward(T, C, name, param):
    _say(f"norm forward T={T} C={C} {name} {param}")
    s = _norm_case(T, C, name, param, 1000 * T + C)
    _check_norm_forward(s, name, True, True, 0, param=param)
    _check_norm_forward(s, name, False, False, 1, param=param)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_layer_norm_of_far_and_flat_rows(name):
    _say(f"norm of rows far from zero and of constant rows, {name}")
    torch = _torch()
    s = _norm_case(4, 771, name, "f32", 5, shift=300.0)
    s["x"][1] = 7.0                      # variance 0
    s["residual"][1] = 0.0
    s["x"][2] = 0.0
    s["residual"][2] = 0.0
    _check_norm_forward(s, name, True, True, 3)
    h = _h()
    y, _, mean, rstd = h.hlq_layer_norm_forward(_dev(s["x"], name), _dev(s["weight"], "f32"), None,
                                                1e-5)
    assert (y[1:3] == 0).all() and mean[1] == 7 and mean[2] == 0
    assert torch.allclose(rstd[1:3], torch.full((2,), 1e-5 ** -0.5, device="cuda"))


def _check_norm_backward(s, name, with_g_h, bias, offset, param="f32"):
    h = _h()
    T, C = s["x"].shape
    x, w = _np(s["x"]), _np(s["weight"])
    _, oh, om, orr = o.layer_norm_forward(x, w, None, 1e-5)
    mean, rstd = (_dev(v.astype(np.float32), "f32") for v in (om, orr))
    om, orr = _np(mean), _np(rstd)
    gy, gh = _np(s["g_y"]), _np(s["g_h"])
    got = h.hlq_layer_norm_backward(_dev(s["g_y"], name, offset), _dev(s["x"], name, offset), mean,
                                    rstd, _dev(s["weight"], param, offset),
                                    g_h=_dev(s["g_h"], name, offset) if with_g_h else None,
                                    with_bias=bias)
    _torch().cuda.synchronize()
    o_x, o_w, o_b = o.layer_norm_backward(gy, oh, om, orr, w, gh if with_g_h else None)
    n = np.abs(oh - om[:, None]) * orr[:, None]
    a = np.abs(gy * w)
    k = (_terms(C) + 6) * U
    tol = orr[:, None] * (6 * U * a + k * a.mean(-1)[:, None] +
                          n * (k + 6 * U) * (a * n).mean(-1)[:, None]) + 3 * U * np.abs(o_x)
    if with_g_h:
        tol = tol + U * np.abs(gh)
    _within(_np(got[0]), o_x, tol + HALF[name] * (np.abs(o_x) + tol) + 1e-38, "g_x")
    # column sums: at most every row in one accumulator
    kt = (T + 16) * U
    tol_w = (kt + 4 * U) * (np.abs(gy) * n).sum(0)
    _within(_np(got[1]), o_w, tol_w + HALF[param] * (np.abs(o_w) + tol_w) + 1e-38, "g_weight")
    if bias:
        tol_b = kt * np.abs(gy).sum(0)
        _within(_np(got[2]), o_b, tol_b + HALF[param] * (np.abs(o_b) + tol_b) + 1e-38, "g_bias")
    else:
        assert got[2] is None


@pytest.mark.parametrize("name,param", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                        ("f32", "bf16")])
@pytest.mark.parametrize("T,C", NORM_SHAPES + [(1500, 24), (700, 96), (300, 1025)])
def test_layer_norm_backward(T, C, name, param):
    _say(f"norm backward T={T} C={C} {name} {param}")
    s = _norm_case(T, C, name, param, 2000 * T + C)
    _check_norm_backward(s, name, True, True, 0, param)
    _check_norm_backward(s, name, False, False, 1, param)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("T,C", [(70001, 9), (9000, 200), (6000, 600), (5001, 1000), (4500, 1030),
                                 (2100, 2050)])
def test_layer_norm_of_many_rows(T, C, name):
    """More rows than the launch's workgroups take at once, lanes past the last
    row and past a row's end."""
    _say(f"norm T={T} C={C} {name}")
    s = _norm_case(T, C, name, "f32", T + C)
    _check_norm_forward(s, name, True, True, 1)
    _check_norm_forward(s, name, False, False, 0)
    _check_norm_backward(s, name, True, True, 1)
    _check_norm_backward(s, name, False, False, 0)


@pytest.mark.parametrize("C", [8, 64, 770, 2048, 4100, 16384, 17001])
def test_layer_norm_backward_of_few_rows(C):
    # one workgroup's rounds, and one row more than they take
    for T in (1, 2, 3, 17, 33):
        _say(f"norm backward T={T} C={C}")
        s = _norm_case(T, C, "bf16", "bf16", T + C)
        _check_norm_backward(s, "bf16", False, T % 2 == 0, 0, "bf16")


def test_layer_norm_of_no_rows():
    torch, h = _torch(), _h()
    _say("norm of no rows")
    x, w = torch.empty((0, 24), device="cuda"), torch.ones(24, device="cuda")
    y, _, mean, rstd = h.hlq_layer_norm_forward(x, w)
    assert y.shape == (0, 24) and mean.shape == (0,)
    g_x, g_w, g_b = h.hlq_layer_norm_backward(x, x, mean, rstd, w)
    torch.cuda.synchronize()
    assert (g_w == 0).all() and (g_b == 0).all() and g_x.shape == (0, 24)


def test_layer_norm_repeats_bit_for_bit():
    torch, h = _torch(), _h()
    _say("norm backward twice")
    g = torch.Generator(device="cuda").manual_seed(3)
    x, gy = (torch.randn((4111, 768), generator=g, device="cuda") for _ in range(2))
    w = torch.ones(768, device="cuda")
    _, _, mean, rstd = h.hlq_layer_norm_forward(x, w)
    a = h.hlq_layer_norm_backward(gy, x, mean, rstd, w)
    b = h.hlq_layer_norm_backward(gy, x, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_layer_norm_backward_of_one_endless_row():
    # more columns than one launch of the fold takes; a single row's bias gradient is g_y itself
    torch, h = _torch(), _h()
    C = (1 << 26) + 5
    _say(f"layer norm backward T=1 C={C}")
    g_y = torch.randn(1, C, device="cuda").bfloat16()
    x, w = torch.randn(1, C, device="cuda").bfloat16(), torch.ones(C, device="cuda").bfloat16()
    one = torch.ones(1, device="cuda")
    _, g_w, g_b = h.hlq_layer_norm_backward(g_y, x, 0 * one, one, w)
    torch.cuda.synchronize()
    assert torch.equal(g_b, g_y[0]) and torch.equal(g_w, (g_y[0].float() * x[0].float()).bfloat16())


# ------------------------------------------------------------ log probabilities

LOGIT_SHAPES = [(1, 1), (3, 2), (5, 7), (2, 513), (17, 1000), (4, 4099), (3, 32003), (2, 65536),
                (2, 65541), (2, 128256), (1, 140001)]


def _logits(T, V, name, seed, banned=0.1):
    torch = _torch()
    g = torch.Generator().manual_seed(seed)
    x = 2.5 * torch.randn((T, V), generator=g)
    t = torch.randint(0, V, (T,), generator=g)
    x[torch.arange(T), t] += 8.0
    drop = torch.rand((T, V), generator=g) < banned
    drop[torch.arange(T), t] = False
    x[drop] = -math.inf
    return x.to(_dt(name)), t


def _logit_errors(x, t, scale):
    """(absolute error of logprob, relative error of s) by rows, for finite
    rows: every exponential's error, weighted by what it adds to s."""
    T, V = x.shape
    e_lp, e_s = np.zeros(T), np.zeros(T)
    for i in range(T):
        m = x[i].max()
        if not np.isfinite(m):
            continue
        z = scale * (x[i] - m)
        e = np.exp(z)
        live = np.isfinite(z)
        rel = np.where(live, 3 * U * np.abs(np.where(live, z, 0.0)) + 2 * U, 0.0)
        e_s[i] = (e * rel).sum() / e.sum() + (_terms(V) + 8) * U + 3 * U
        zt = z[t[i]] if 0 <= t[i] < V else 0.0
        e_lp[i] = e_s[i] + U * abs((zt if np.isfinite(zt) else 0.0) - math.log(e.sum()))
    return e_lp, e_s


def _gradient_tolerance(x, t, g, e_s, scale, name, want):
    tol = np.zeros(x.shape)
    for i in range(len(x)):
        m = x[i].max()
        if not 0 <= t[i] < x.shape[1] or not np.isfinite(m):
            continue
        z = scale * (x[i] - m)
        e = np.exp(z)
        p = e / e.sum()
        z = np.where(np.isfinite(z), np.abs(z), 0.0)
        tol[i] = abs(scale * g[i]) * p * (3 * U * z + e_s[i] + 8 * U)
        tol[i, t[i]] += 4 * U * abs(scale * g[i])
    # an exponential below 2^-126 may vanish
    tol = tol + np.abs(scale * g)[:, None] * 2.0 ** -125
    return tol + HALF[name] * (np.abs(want) + tol) + 1e-37


def _check_logprob(x, t, name, scale, offset=0, pitch=0):
    torch, h = _torch(), _h()
    T, V = x.shape
    dx = _dev(torch.cat([x, x.new_zeros((T, pitch))], 1), name, offset)[:, :V]
    dt = t.cuda()
    lp, stats = h.hlq_token_logprob_forward(dx, dt, scale)
    torch.cuda.synchronize()
    xn, tn = _np(x), t.numpy()
    olp, ost = o.token_logprob(xn, tn, scale)
    e_lp, e_s = _logit_errors(xn, tn, scale)
    _within(_np(stats)[:, 0], ost[:, 0], 0.0, "maximum")
    _within(_np(stats)[:, 1], ost[:, 1], e_s * np.abs(ost[:, 1]), "sum")
    with np.errstate(invalid="ignore"):
        _within(_np(lp), olp, e_lp + U * np.abs(np.nan_to_num(olp)), "logprob")
    g = np.random.default_rng(T + V).normal(size=T).astype(np.float32)
    g[T // 2] = 0.0
    out = torch.full((T, V + pitch), float("nan"), dtype=_dt(name), device="cuda")
    g_x = h.hlq_token_logprob_backward(torch.from_numpy(g).cuda(), dx, dt, stats, scale,
                                       g_x=out[:, :V])
    torch.cuda.synchronize()
    want = o.token_logprob_backward(g.astype(np.float64), xn, tn, scale)
    _within(_np(g_x), want, _gradient_tolerance(xn, tn, g, e_s, scale, name, want), "g_x")
    assert pitch == 0 or torch.isnan(out[:, V:]).all()      # nothing written past a row


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", LOGIT_SHAPES)
def test_token_logprob(T, V, name):
    _say(f"logprob T={T} V={V} {name}")
    x, t = _logits(T, V, name, T * 7 + V)
    _check_logprob(x, t, name, 1.0)
    if T > 1:
        t[T - 1] = -100
    _check_logprob(x, t, name, 1.0 / 0.7, offset=1, pitch=3)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 4099, 131072])
def test_token_logprob_masks(V, name):
    _say(f"logprob masks V={V} {name}")
    torch = _torch()
    low = torch.finfo(_dt(name)).min
    x, t = _logits(8, V, name, V, banned=0.5)
    x[0] = -math.inf                          # nothing allowed
    x[1] = low                                # all of the type's lowest value: uniform
    x[2, 1:] = low                            # one live logit
    t[2] = 0
    x[3] = -math.inf                          # one live logit, and it is far below zero
    x[3, V - 1], t[3] = low, V - 1
    x[4, t[4]] = -math.inf                    # the target itself is banned
    x[5], t[5] = math.nan, -100               # ignored, whatever the row holds
    x[6], t[6] = math.inf, V                  # out of range
    x[7] = torch.finfo(_dt(name)).max         # the highest value
    _check_logprob(x, t, name, 1.0)
    x[1, 0], x[2, V - 1] = math.nan, math.inf
    h = _h()
    lp, _ = h.hlq_token_logprob_forward(x.cuda(), t.cuda())
    assert torch.isnan(lp[1:3]).all() and not torch.isnan(lp[3:]).any()


def test_token_logprob_far_rows():
    """Rows whose elements lie past 2^31 in the buffer."""
    torch, h = _torch(), _h()
    ld = (1 << 30) + 5
    _say(f"logprob at pitch {ld}")
    V = 1003
    buf = torch.empty((3 * ld,), dtype=torch.bfloat16, device="cuda")
    x, t = _logits(3, V, "bf16", 11)
    view = torch.as_strided(buf, (3, V), (ld, 1))
    view.copy_(x.cuda())
    lp, stats = h.hlq_token_logprob_forward(view, t.cuda())
    lp2, stats2 = h.hlq_token_logprob_forward(x.cuda(), t.cuda())
    assert torch.equal(lp, lp2) and torch.equal(stats, stats2)
    g = torch.ones(3, device="cuda")
    want = h.hlq_token_logprob_backward(g, x.cuda(), t.cuda(), stats)
    got = h.hlq_token_logprob_backward(g, x.cuda(), t.cuda(), stats, g_x=view)
    assert torch.equal(got, want)


# ------------------------------------------------------------ policy loss

def _policy_inputs(x, t, scale, seed, zero=0.2):
    rng = np.random.default_rng(seed)
    T = len(t)
    lp = o.token_logprob(_np(x), t.numpy(), scale)[0]
    f = lambda v: np.asarray(v, np.float32)
    return dict(old=f(lp + 0.2 * rng.normal(size=T)), adv=f(rng.normal(size=T)),
                w=f(rng.uniform(0.5, 1.5, size=T) * (rng.uniform(size=T) >= zero) / T),
                ref=f(lp + 0.3 * rng.normal(size=T)))


def _clear_of_the_border(lp, s, lo, hi, margin):
    """Moves old log probabilities whose ratio lies within the error of a clip
    bound, where either side is right."""
    for t in range(len(lp)):
        for b in (math.log(1 - lo) if lo < 1 else -math.inf, math.log(1 + hi)):
            if abs(lp[t] - float(s["old"][t]) - b) < margin:
                s["old"][t] += np.float32(4 * margin)


def _check_policy(x, t, name, scale, kl, weighted, seed, offset=0, pitch=0, lo=0.2, hi=0.28):
    torch, h = _torch(), _h()
    T, V = x.shape
    s = _policy_inputs(x, t, scale, seed)
    xn, tn = _np(x), t.numpy()
    live = (tn >= 0) & (tn < V)
    olp = o.token_logprob(xn, tn, scale)[0]
    e_lp, e_s = _logit_errors(xn, tn, scale)
    _clear_of_the_border(olp, s, lo, hi, 1e-3)
    w = s["w"] if weighted else None
    counts = live & ((s["w"] != 0) if weighted else True)
    osums, og = o.policy_loss(olp, s["old"], s["adv"], w, s["ref"], lo, hi, kl, counts)
    c = lambda v: torch.from_numpy(v).cuda()
    dx = _dev(torch.cat([x, x.new_zeros((T, pitch))], 1), name, offset)[:, :V]
    out = torch.full((T, V + pitch), float("nan"), dtype=_dt(name), device="cuda")
    sums, lp, g_x = h.hlq_policy_loss_logits(
        dx, t.cuda(), c(s["old"]), c(s["adv"]), c(s["w"]) if weighted else None,
        ref_logprob=c(s["ref"]) if kl else None, scale=scale, clip_low=lo, clip_high=hi, kl_coef=kl,
        g_x=out[:, :V])
    torch.cuda.synchronize()
    want_lp = np.where(counts, olp, 0.0)
    _within(_np(lp), want_lp, np.where(counts, e_lp + U * np.abs(want_lp), 0.0), "logprob")
    # the ratio and exp(d) move by the log probability's error, in proportion
    ratio = np.exp(np.where(counts, olp - s["old"], 0.0))
    away = np.exp(np.where(counts, s["ref"] - olp, 0.0))
    ws = np.abs(s["w"].astype(np.float64)) if weighted else np.ones(T)
    move = ws * counts * 1.01 * e_lp
    e_g = move * (ratio * np.abs(s["adv"]) + kl * away)
    tol = np.array([(move * (ratio * np.abs(s["adv"]) + kl * np.abs(away - 1))).sum(),
                    (move * np.abs(away - 1)).sum(), 0.0])
    _within(_np(sums), osums, tol * 1.01 + 2 * U * np.abs(osums) + 1e-12, "sums")
    want = o.token_logprob_backward(og, xn, tn, scale)
    g_tol = _gradient_tolerance(xn, tn, og, e_s, scale, name, want)
    for i in np.flatnonzero(counts):
        g_tol[i] += (1 + HALF[name]) * np.abs(want[i]) * (e_g[i] / max(abs(og[i]), 1e-30) + 2 * U)
    _within(_np(g_x), want, g_tol, "g_x")
    assert pitch == 0 or torch.isnan(out[:, V:]).all()
    # the same loss from the log probabilities
    sums2, g_lp = h.hlq_policy_loss(lp, c(s["old"]), c(s["adv"]),
                                    c(np.where(counts, s["w"] if weighted else 1.0, 0.0)
                                      .astype(np.float32)),
                                    c(s["ref"]) if kl else None, lo, hi, kl)
    torch.cuda.synchronize()
    once = U * np.abs(want_lp) * ws * counts           # the log probabilities' rounding
    tol2 = tol + np.array([(once * (ratio * np.abs(s["adv"]) + kl * np.abs(away - 1))).sum(),
                           (once * np.abs(away - 1)).sum(), 0.0])
    _within(_np(sums2), osums, tol2 * 1.01 + 2 * U * np.abs(osums) + 1e-12,
            "sums from log probabilities")
    _within(_np(g_lp), og, e_g + (4 + np.abs(olp)) * U * ws *
            (ratio * np.abs(s["adv"]) + kl * away) * 1.01, "g_logprob")


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", LOGIT_SHAPES + [(300, 600), (1030, 77)])
def test_policy_loss(T, V, name):
    _say(f"policy T={T} V={V} {name}")
    x, t = _logits(T, V, name, T * 3 + V)
    if T > 2:
        t[1] = -100
    _check_policy(x, t, name, 1.0, 0.05, True, T + V)
    _check_policy(x, t, name, 1.25, 0.0, False, T + V + 1, offset=1, pitch=1)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(300, 2100), (300, 4099), (260, 4801), (257, 9001), (257, 17003)])
def test_logits_of_more_rows_than_units(T, V, name):
    # other threads per row than for the few rows above
    _say(f"logits T={T} V={V} {name}")
    x, t = _logits(T, V, name, T + V)
    t[2] = -100
    _check_logprob(x, t, name, 0.9, offset=1)
    _check_policy(x, t, name, 1.0, 0.05, True, T + V, offset=3)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(5, 3), (40, 1001), (300, 4099), (3, 65541), (2, 140001)])
def test_logits_gradient_in_place(T, V, name):
    # the gradient may take the place of the logits: the same bits
    torch, h = _torch(), _h()
    _say(f"gradient in place T={T} V={V} {name}")
    x, t = _logits(T, V, name, T + V)
    t[1] = -100
    x, t = _dev(x, name, 1), t.cuda()
    lp, stats = h.hlq_token_logprob_forward(x, t)
    adv = torch.ones(T, device="cuda") - 2.0 * (torch.arange(T, device="cuda") % 2)
    for f in (lambda v, g: h.hlq_token_logprob_backward(adv, v, t, stats, g_x=g),
              lambda v, g: h.hlq_policy_loss_logits(v, t, lp, adv, g_x=g)[2]):
        want = f(x, None)
        own = _dev(x.cpu(), name, 1)
        got = f(own, own)
        torch.cuda.synchronize()
        assert got.data_ptr() == own.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_logits_past_the_cache_equal_their_parts(name):
    """Logits of more than 96 MB take non-temporal accesses; parts of them,
    with as many threads per row, do not: the same bits."""
    torch, h = _torch(), _h()
    T, V = 1203, 50257
    _say(f"T={T} V={V} {name}")
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((T, V), generator=g, device="cuda").mul_(2.5).to(_dt(name))
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    old = torch.randn(T, generator=g, device="cuda") - 12.0
    adv = torch.randn(T, generator=g, device="cuda")
    whole = h.hlq_token_logprob_forward(x, t) + h.hlq_policy_loss_logits(x, t, old, adv)[1:]
    for a in range(0, T, 401):
        b = a + 401
        part = h.hlq_token_logprob_forward(x[a:b], t[a:b]) + \
            h.hlq_policy_loss_logits(x[a:b], t[a:b], old[a:b], adv[a:b])[1:]
        assert all(torch.equal(p, w[a:b]) for p, w in zip(part, whole))


def test_policy_loss_of_masked_tokens():
    torch, h = _torch(), _h()
    _say("policy: masked tokens hold anything")
    x, t = _logits(6, 100, "f32", 4)
    bad = [math.nan, math.inf, -math.inf]
    x[0], x[1] = math.nan, math.inf
    old, adv, w, ref = torch.zeros(6), torch.ones(6), torch.tensor([0., 0., 0., 1., 1., 1.]), \
        torch.zeros(6)
    for v in (old, adv, ref):
        v[:3] = torch.tensor(bad)
    t[5] = -1
    x[5] = math.nan
    sums, lp, g_x = h.hlq_policy_loss_logits(x.cuda(), t.cuda(), old.cuda(), adv.cuda(), w.cuda(),
                                             ref.cuda(), kl_coef=0.1)
    torch.cuda.synchronize()
    assert torch.isfinite(sums).all() and torch.isfinite(lp).all()
    assert (g_x[[0, 1, 2, 5]] == 0).all() and (lp[[0, 1, 2, 5]] == 0).all()
    assert torch.isfinite(g_x).all() and (g_x[3:5] != 0).any()
    lp[:3] = torch.tensor(bad)
    sums2, g = h.hlq_policy_loss(lp, old.cuda(), adv.cuda(), w.cuda(), ref.cuda(), kl_coef=0.1)
    torch.cuda.synchronize()
    assert torch.isfinite(sums2).all() and (g[:3] == 0).all() and torch.isfinite(g).all()


def test_policy_loss_of_no_tokens():
    torch, h = _torch(), _h()
    _say("policy of no tokens")
    e = torch.empty(0, device="cuda")
    sums, lp, g_x = h.hlq_policy_loss_logits(torch.empty((0, 9), device="cuda"),
                                             torch.empty(0, dtype=torch.int64, device="cuda"), e, e)
    sums2, g = h.hlq_policy_loss(e, e, e)
    torch.cuda.synchronize()
    assert (sums == 0).all() and (sums2 == 0).all() and g_x.shape == (0, 9)


# ------------------------------------------------------------ preference loss

@pytest.mark.parametrize("T,P", [(2, 1), (4, 1), (301, 2), (500, 7), (3000, 1), (8190, 32),
                                 (20000, 3), (1500, 600)])
@pytest.mark.parametrize("mean", [False, True])
def test_preference_loss(T, P, mean):
    torch, h = _torch(), _h()
    _say(f"preference T={T} P={P} mean={mean}")
    rng = np.random.default_rng(T + P)
    lp, ref = (rng.normal(size=T).astype(np.float32) - 2 for _ in range(2))
    w = (rng.uniform(0, 2, size=T) * (rng.uniform(size=T) > 0.3)).astype(np.float32)
    start = np.concatenate([[0], np.sort(rng.integers(0, T + 1, 2 * P - 1)), [T]])
    c = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()
    for r, ww, e, off in ((ref, w, 0.1, 1), (None, None, 0.0, 0)):
        dead = lp.copy()
        if ww is not None:
            dead[ww == 0] = np.nan                 # what a masked token holds does not matter
        pad = lambda v: None if v is None else _dev(v, "f32", off)
        loss, margin, g = h.hlq_preference_loss(pad(dead), c(start), 0.3, ref_logprob=pad(r),
                                                weight=pad(ww), label_smoothing=e,
                                                reduction=h.HLQ_MEAN if mean else h.HLQ_SUM)
        torch.cuda.synchronize()
        ol, om, og = o.preference_loss(lp.astype(np.float64), start, 0.3, r, ww, e, mean)
        # sums in fp64: what is left is the rounding of the outputs
        _within(_np(margin), om, 2 * U * np.abs(om) + 1e-10, "margin")
        _within(_np(loss), [ol], 2 * U * abs(ol) + 1e-10, "loss")
        _within(_np(g), og, 2 * U * np.abs(og) + 1e-14, "g_logprob")


def test_preference_loss_of_bad_bounds_stays_inside():
    torch, h = _torch(), _h()
    _say("preference: bounds outside the tokens are limited to them")
    lp = torch.full((10,), -1.0, device="cuda")
    for start in ([0, 3, 50], [-7, 5, 10], [0, 1 << 40, 10], [9, 4, 10]):
        loss, margin, g = h.hlq_preference_loss(lp, torch.tensor(start).cuda(), 0.1)
        torch.cuda.synchronize()
        assert torch.isfinite(loss).all() and torch.isfinite(margin).all()
    # no tokens at all: margins of zero
    e = torch.empty(0, device="cuda")
    loss, margin, g = h.hlq_preference_loss(e, torch.zeros(5, dtype=torch.int64, device="cuda"), 0.1)
    assert loss.item() == pytest.approx(math.log(2), rel=1e-6) and (margin == 0).all()


@pytest.mark.parametrize("pad", [5, 3000])
def test_preference_loss_of_a_padded_batch(pad):
    # tokens before the first and behind the last sequence: no part in the loss, gradient zero
    torch, h = _torch(), _h()
    _say(f"preference: {pad} tokens of no sequence on either side")
    g = torch.Generator(device="cuda").manual_seed(pad)
    lp = -torch.rand(40 + 2 * pad, generator=g, device="cuda")
    start = torch.tensor([0, 7, 20, 21, 40], device="cuda")
    inner = h.hlq_preference_loss(lp[pad:pad + 40], start, 0.3)
    h.hlq_preference_loss(torch.full_like(lp, -3.0), start * (lp.numel() // 40), 0.3)
    outer = h.hlq_preference_loss(lp, start + pad, 0.3)
    torch.cuda.synchronize()
    assert torch.equal(outer[0], inner[0]) and torch.equal(outer[1], inner[1])
    assert torch.equal(outer[2][pad:pad + 40], inner[2])
    assert (outer[2][:pad] == 0).all() and (outer[2][pad + 40:] == 0).all()


def test_preference_loss_of_far_margins():
    torch, h = _torch(), _h()
    _say("preference: margins far from zero")
    lp = torch.tensor([0.0, -4e4, -4e4, 0.0], device="cuda")
    start = torch.tensor([0, 1, 2, 3, 4]).cuda()        # margins +4e3 and -4e3
    loss, margin, g = h.hlq_preference_loss(lp, start, 0.1)
    torch.cuda.synchronize()
    assert margin.tolist() == [4000.0, -4000.0] and loss.item() == pytest.approx(2000.0)
    assert g.tolist() == pytest.approx([0.0, -0.05, 0.0, 0.05], abs=1e-9)


# ------------------------------------------------------------ clipping

def _grads(sizes, seed, types=("f32", "bf16")):
    torch = _torch()
    g = torch.Generator().manual_seed(seed)
    return [(1e-2 * torch.randn(n, generator=g)).to(_dt(types[i % len(types)]))
            for i, n in enumerate(sizes)]


CLIP_SIZES = [[1], [0, 5, 0], [3, 8191, 8192, 8193, 1], [100003, 7], [17] * 400,
              [70000, 1, 131075] * 5, [64 * k + k % 7 for k in range(161)]]


@pytest.mark.parametrize("sizes", CLIP_SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("kind", ["l2", "inf"])
@pytest.mark.parametrize("offset", [0, 1])
def test_clip_grad_norm(sizes, kind, offset):
    torch, h = _torch(), _h()
    _say(f"clip {len(sizes)} tensors, largest {max(sizes)}, {kind}, offset {offset}")
    host = _grads(sizes, len(sizes) + max(sizes))
    names = ["bf16" if v.dtype == torch.bfloat16 else "f32" for v in host]
    want, _ = o.clip_grad_norm([_np(v) for v in host], 1.0, kind == "inf")
    code = h.HLQ_NORM_L2 if kind == "l2" else h.HLQ_NORM_INF
    for max_norm in (0.37 * want, 3.0 * want, 0.0):
        _, outs = o.clip_grad_norm([_np(v) for v in host], max_norm, kind == "inf")
        dev = [_dev(v, n, offset) for v, n in zip(host, names)]
        out = [_dev(v, n, 1 - offset) for v, n in zip(host, names)]
        norm = h.hlq_clip_grad_norm(dev, max_norm, code, out=out)
        norm2 = h.hlq_clip_grad_norm(dev_in := [v.clone() for v in dev], max_norm, code)
        torch.cuda.synchronize()
        # exact squares in fp64, fewer than 2^20 additions of them
        assert abs(norm.item() - want) <= (2.0 ** -33 if kind == "l2" else 0.0) * want
        assert torch.equal(norm, norm2)
        for v, a, b, ref, n in zip(dev, out, dev_in, outs, names):
            if ref.size:
                tol = 3 * U * np.abs(ref)
                _within(_np(a), ref, tol + HALF[n] * (np.abs(ref) + tol) + 1e-38, "clipped")
            assert torch.equal(a, b)
            assert max_norm <= want or torch.equal(a, v)      # a factor of one changes nothing


@pytest.mark.parametrize("kind", [0, 1])
def test_clip_past_the_cache(kind):
    # more than 96 MB: non-temporal accesses, workgroups that take several chunks
    torch, h = _torch(), _h()
    _say(f"clip of 150 MB, kind {kind}")
    g = torch.Generator(device="cuda").manual_seed(7)
    v = [torch.randn(n, generator=g, device="cuda").mul_(1e-2).to(_dt(d))
         for n, d in ((30_000_001, "f32"), (7, "bf16"), (15_000_003, "bf16"), (5, "f32"))]
    d = [w.double() for w in v]
    want = sum((w * w).sum() for w in d).sqrt() if kind == 0 else max(w.abs().max() for w in d)
    norm = h.hlq_clip_grad_norm(v, 1e-3, kind)
    torch.cuda.synchronize()
    assert abs(norm.item() / want.item() - 1) < 1e-12      # 4.5e7 fp64 additions, in trees
    f = 1e-3 / (want + 1e-6)
    for got, w in zip(v, d):
        half = torch.finfo(got.dtype).eps / 2
        assert ((got.double() - w * f).abs() <= (w * f).abs() * (half + 2 * U)).all()


@pytest.mark.parametrize("kind", [0, 1])
def test_clip_of_infinities_and_nan(kind):
    torch, h = _torch(), _h()
    _say(f"clip: infinities and NaN, norm {kind}")
    a, b = torch.ones(5000, device="cuda"), torch.ones(300, dtype=torch.bfloat16, device="cuda")
    a[4999] = math.inf
    norm = h.hlq_clip_grad_norm([a, b], 1.0, kind)
    assert norm.item() == math.inf and torch.isnan(a[4999]) and (a[:4999] == 0).all()
    assert (b == 0).all()
    b[299] = math.nan
    norm = h.hlq_clip_grad_norm([torch.ones(9, device="cuda"), b], 1.0, kind)
    assert math.isnan(norm.item()) and torch.isnan(b).all()
    # squares that fp32 cannot hold
    big = [torch.full((4,), 3e38, device="cuda"), torch.full((4,), 1e-30, device="cuda")]
    assert h.hlq_clip_grad_norm(big[:1], math.inf).item() == pytest.approx(6e38, rel=1e-6)
    assert h.hlq_clip_grad_norm(big[1:], 1.0).item() == pytest.approx(2e-30, rel=1e-6)
    assert (big[0] == 3e38).all()


def test_clip_of_nothing_and_of_other_layouts():
    torch, h = _torch(), _h()
    _say("clip: no tensors, transposed and channels-last tensors")
    assert h.hlq_clip_grad_norm([], 1.0).item() == 0.0
    assert h.hlq_clip_grad_norm([torch.empty(0, device="cuda")], 1.0).item() == 0.0
    w = torch.randn(6, 10, device="cuda").t()
    c = torch.randn(2, 3, 4, 5, device="cuda").to(memory_format=torch.channels_last)
    want_w, want_c = w.clone(), c.clone()
    norm = h.hlq_clip_grad_norm([w, c], 0.5)
    ref = math.sqrt(float(want_w.double().square().sum() + want_c.double().square().sum()))
    assert norm.item() == pytest.approx(ref, rel=1e-9)
    assert torch.allclose(w, want_w * (0.5 / ref)) and torch.allclose(c, want_c * (0.5 / ref))
    with pytest.raises(ValueError, match="dense"):
        h.hlq_clip_grad_norm([torch.zeros(8, 8, device="cuda")[:, :4]], 1.0)
    with pytest.raises(ValueError, match="match"):
        h.hlq_clip_grad_norm([want_w], 1.0, out=[want_w.contiguous()])


# ------------------------------------------------------------ layouts, streams, graphs

def test_binding_refuses_layouts():
    torch, h = _torch(), _h()
    x, t = torch.zeros(6, 8, device="cuda"), torch.zeros(8, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        h.hlq_layer_norm_forward(torch.zeros(8, 6, device="cuda").t(), torch.ones(8, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        h.hlq_token_logprob_forward(x.t(), t)
    with pytest.raises(ValueError, match="overlap"):
        h.hlq_token_logprob_forward(x[:1].expand(8, 8), t)
    with pytest.raises(TypeError, match="dtype"):
        h.hlq_token_logprob_forward(x.half(), t[:6])
    with pytest.raises(h.HLQError):
        h.hlq_token_logprob_forward(x, t[:6], 0.0)


def _step(h, s):
    y, hh, mean, rstd = h.hlq_layer_norm_forward(s["x"], s["w"], s["b"], residual=s["r"])
    sums, lp, g_x = h.hlq_policy_loss_logits(y, s["t"], s["old"], s["adv"], scale=0.8)
    lp2, stats = h.hlq_token_logprob_forward(hh, s["t"])
    loss, margin, g = h.hlq_preference_loss(lp2, s["start"], 0.2, weight=s["wt"])
    g_h = h.hlq_token_logprob_backward(g, hh, s["t"], stats)
    grads = h.hlq_layer_norm_backward(g_x, hh, mean, rstd, s["w"], g_h=g_h)
    out = [_torch().empty_like(v) for v in grads]
    norm = h.hlq_clip_grad_norm(grads, 1e-3, out=out)
    return [y, hh, sums, lp, lp2, loss, margin, g, *grads, norm, *out]


def _step_inputs(seed):
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    T, C = 129, 1001
    return dict(x=r(T, C).bfloat16(), r=r(T, C).bfloat16(), w=1 + 0.1 * r(C), b=r(C),
                t=torch.randint(0, C, (T,), generator=g, device="cuda"), old=r(T) - 7, adv=r(T),
                start=torch.tensor([0, 30, 64, 100, T]).cuda(), wt=(r(T) > 0).float())


def test_graph_replays_match_eager():
    torch, h = _torch(), _h()
    _say("graph of all operators")
    s = _step_inputs(1)
    ref = [v.clone() for v in _step(h, s)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(h, s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(h, s)
    for rep in range(4):
        other = _step_inputs(10 + rep)
        for k in s:
            s[k].copy_(other[k])
        want = [v.clone() for v in _step(h, s)]
        for v in got:
            v.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (rep, i)
    assert not torch.equal(got[2], ref[2])


def test_calls_on_another_stream():
    torch, h = _torch(), _h()
    _say("calls on a stream that is not the current one")
    s = _step_inputs(2)
    y, _, mean, rstd = h.hlq_layer_norm_forward(s["x"], s["w"], s["b"])
    ref = h.hlq_layer_norm_backward(s["r"], s["x"], mean, rstd, s["w"])
    lp, stats = h.hlq_token_logprob_forward(s["x"], s["t"])
    norm = h.hlq_clip_grad_norm([v.clone() for v in ref], 1.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        a = h.hlq_layer_norm_forward(s["x"], s["w"], s["b"], stream=side)
        g = h.hlq_layer_norm_backward(s["r"], s["x"], a[2], a[3], s["w"], stream=side)
        q = h.hlq_token_logprob_forward(s["x"], s["t"], stream=side)
        # memory freed here must not be handed to the current stream's work while in use
        junk = [torch.full((1 << 16,), float("nan"), device="cuda") for _ in range(8)]
        n = h.hlq_clip_grad_norm(g, 1.0, out=[torch.empty_like(v) for v in g], stream=side)
        side.synchronize()
        assert torch.equal(a[0], y) and torch.equal(q[0], lp) and torch.equal(n, norm)
        assert all(torch.equal(u, v) for u, v in zip(g, ref))
        del junk
