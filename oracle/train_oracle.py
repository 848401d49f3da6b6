"""Plain numpy statement, in 64 bits, of the operators of a training step:
layer norm, token log probabilities, the policy and preference losses on them,
and gradient clipping.  One row, token or tensor at a time, from the formulas;
shares no code with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np

CLIP_EPS = 1e-6


def round_bf16(v):
    """float64 values rounded to nearest-even bf16, as float64 (by way of an
    fp32 rounded to odd, so that the value is rounded once)."""
    v = np.asarray(v, np.float64)
    f = v.astype(np.float32)
    up = np.nextafter(f, np.float32(np.inf))
    down = np.nextafter(f, np.float32(-np.inf))
    odd = (f.view(np.uint32) & 1) == 1
    g = np.where((f == v) | odd | ~np.isfinite(f), f, np.where(v > f, up, down)).astype(np.float32)
    b = g.view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(g), g, r).astype(np.float64)


def round_f32(v):
    return np.asarray(v, np.float64).astype(np.float32).astype(np.float64)


# ------------------------------------------------------------ layer norm

def layer_norm_forward(x, weight, bias=None, eps=1e-5, residual=None, rounding=None):
    """(y, h, mean, rstd); ``rounding`` rounds h = x + residual to x's type."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + residual
        if rounding is not None:
            h = rounding(h)
    mean = h.mean(-1)
    d = h - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(-1) + eps)
    y = d * rstd[:, None] * weight
    return (y if bias is None else y + bias), h, mean, rstd


def layer_norm_backward(g_y, h, mean, rstd, weight, g_h=None):
    """(g_x, g_weight, g_bias) given the row statistics."""
    g_x = np.empty(h.shape, np.float64)
    g_w, g_b = np.zeros(h.shape[1]), np.zeros(h.shape[1])
    for t in range(h.shape[0]):
        n = (h[t] - mean[t]) * rstd[t]
        u = g_y[t] * weight
        g_x[t] = rstd[t] * (u - u.mean() - n * (u * n).mean())
        g_w += g_y[t] * n
        g_b += g_y[t]
    return (g_x if g_h is None else g_x + g_h), g_w, g_b


# ------------------------------------------------------------ log probabilities

def token_logprob(logits, targets, scale=1.0):
    """(logprob [T], stats [T, 2])."""
    T, V = logits.shape
    lp, stats = np.zeros(T), np.zeros((T, 2))
    for t in range(T):
        if not 0 <= targets[t] < V:
            stats[t] = 0.0, 1.0
            continue
        x = logits[t].astype(np.float64)
        if np.isnan(x).any() or np.isposinf(x).any():
            lp[t], stats[t] = np.nan, (x.max(), np.nan)
            continue
        m = x.max()
        if m == -np.inf:
            lp[t], stats[t] = -np.inf, (m, 0.0)
            continue
        s = np.exp(scale * (x - m)).sum()
        lp[t], stats[t] = scale * (x[targets[t]] - m) - math.log(s), (m, s)
    return lp, stats


def token_logprob_backward(g_logprob, logits, targets, scale=1.0):
    """Gradient of the logits."""
    T, V = logits.shape
    out = np.zeros((T, V))
    for t in range(T):
        if g_logprob[t] == 0 or not 0 <= targets[t] < V:
            continue
        x = logits[t].astype(np.float64)
        m = x.max()
        if m == -np.inf:
            continue
        e = np.exp(scale * (x - m))
        d = -e / e.sum()
        d[targets[t]] += 1.0
        out[t][d != 0] = d[d != 0] * (scale * g_logprob[t])    # infinite ones: no inf * 0
    return out


# ------------------------------------------------------------ losses

def policy_loss(logprob, old, advantage, weight=None, ref=None, clip_low=0.2, clip_high=0.2,
                kl_coef=0.0, counts=None):
    """(sums [3], g_logprob [T]); ``counts`` False takes a token out."""
    sums, g = np.zeros(3), np.zeros(len(logprob))
    for t in range(len(logprob)):
        w = 1.0 if weight is None else float(weight[t])
        if w == 0 or (counts is not None and not counts[t]):
            continue
        with np.errstate(over="ignore"):
            r = float(np.exp(logprob[t] - old[t]))
        free = 0.0 if advantage[t] == 0 and r == math.inf else r * advantage[t]
        held = min(max(r, 1.0 - clip_low), 1.0 + clip_high) * advantage[t]
        kl, slope = 0.0, 0.0
        if kl_coef:
            d = float(ref[t]) - logprob[t]
            with np.errstate(over="ignore"):
                away = float(np.expm1(d))
            kl, slope = away - d if away < math.inf else away, -away
        sums += w * (kl_coef * kl - min(free, held)), w * kl, w if held < free else 0.0
        g[t] = w * (kl_coef * slope - (free if free <= held else 0.0))
    return sums, g


def _softplus(v):
    return max(v, 0.0) + math.log1p(math.exp(-abs(v)))


def preference_loss(logprob, start, beta, ref=None, weight=None, smoothing=0.0, mean=False):
    """(loss, margin [P], g_logprob [T])."""
    P, T = len(start) // 2, len(logprob)
    w = np.ones(T) if weight is None else np.asarray(weight, np.float64)
    score, share = np.zeros(2 * P), np.ones(2 * P)
    for q in range(2 * P):
        length = 0.0
        for t in range(start[q], start[q + 1]):
            if w[t] != 0:
                score[q] += w[t] * (logprob[t] - (0.0 if ref is None else ref[t]))
                length += w[t]
        if mean:
            share[q] = 1.0 / length if length > 0 else 0.0
    score *= share
    margin = beta * (score[:P] - score[P:])
    loss, g = 0.0, np.zeros(T)
    for p in range(P):
        z = margin[p]
        for part, v in ((1.0 - smoothing, -z), (smoothing, z)):
            loss += part * _softplus(v) / P if part else 0.0
        slope = beta / P * (math.exp(-_softplus(-z)) - 1.0 + smoothing)
        for q, sign in ((p, 1.0), (P + p, -1.0)):
            for t in range(start[q], start[q + 1]):
                if w[t] != 0:
                    g[t] = sign * slope * share[q] * w[t]
    return loss, margin, g


# ------------------------------------------------------------ clipping

def clip_grad_norm(grads, max_norm, inf_norm=False):
    """(norm, clipped gradients before their rounding)."""
    if inf_norm:
        norm = max([0.0] + [float(np.abs(g).max()) for g in grads if g.size])
    else:
        norm = math.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads))
    factor = min(1.0, max_norm / (norm + CLIP_EPS))
    return norm, [g.astype(np.float64) * factor for g in grads]
