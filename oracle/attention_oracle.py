"""Plain numpy statement, in 64 bits, of the attention block's operators:
attention over packed sequences with its backward pass, the relative position
bias by buckets, and counter-based dropout.  One sequence and head, or one
element, at a time, from the formulas; shares no code with the GPU path.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np


# ------------------------------------------------------------ position bias

def bucket(distance, buckets, max_distance, bidirectional):
    """The definition in whole numbers: with e exact buckets of n a side, a
    distance a >= e is at least k steps along the logarithm exactly when
    (a / e)^(n - e) >= (max_distance / e)^k."""
    n = buckets // 2 if bidirectional else buckets
    a = abs(distance) if bidirectional else max(-distance, 0)
    e = n // 2
    if a >= e:
        k, lhs, step = 0, Fraction(a, e) ** (n - e), Fraction(max_distance, e)
        while e + k < n - 1 and lhs >= step ** (k + 1):
            k += 1
        a = e + k
    return a + (n if bidirectional and distance > 0 else 0)


def bucket_table(lq, lk, buckets, max_distance, bidirectional):
    """[lq, lk] buckets of the pairs of one sequence."""
    line = {d: bucket(d, buckets, max_distance, bidirectional) for d in range(-lk + 1, lk + lq)}
    return np.array([[line[j - (i + lk - lq)] for j in range(lk)] for i in range(lq)],
                    np.int64).reshape(lq, lk)


# ------------------------------------------------------------ attention

def scores(q, k, scale, causal, bias=None, which=None):
    """(S [lq, lk], seen [lq, lk]) of one sequence and head; bias [buckets]."""
    lq, lk = len(q), len(k)
    s = np.zeros((lq, lk))
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(lq):
            s[i] = scale * (k * q[i]).sum(-1)
        if bias is not None:
            s = s + bias[which]
    at = np.arange(lq)[:, None] + lk - lq
    seen = np.arange(lk)[None, :] <= at if causal else np.ones((lq, lk), bool)
    return s, seen


def forward(q, k, v, scale, causal, bias=None, which=None):
    """(o [lq, D], lse [lq]) of one sequence and head; hidden keys do not enter."""
    s, seen = scores(q, k, scale, causal, bias, which)
    o, lse = np.zeros(q.shape), np.full(len(q), -np.inf)
    with np.errstate(invalid="ignore"):
        for i in range(len(q)):
            x, y = s[i, seen[i]], v[seen[i]]
            if not len(x) or (x == -np.inf).all():
                continue
            m = x.max()
            p = np.exp(x - m)
            total = p.sum()
            o[i] = (p[:, None] * y).sum(0) / total
            lse[i] = m + np.log(total)
    return o, lse


def backward(g_o, q, k, v, o, lse, scale, causal, bias=None, which=None):
    """(g_q, g_k, g_v, G [lq, lk]) of one sequence and head; rows of lse -inf
    have no probabilities."""
    s, seen = scores(q, k, scale, causal, bias, which)
    g_q, g_k, g_v = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    G = np.zeros(s.shape)
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(len(q)):
            at = seen[i]
            if lse[i] == -np.inf or not at.any():
                continue
            p = np.exp(s[i, at] - lse[i])
            d = p * ((v[at] * g_o[i]).sum(-1) - (g_o[i] * o[i]).sum())
            g_v[at] += p[:, None] * g_o[i]
            g_k[at] += scale * d[:, None] * q[i]
            g_q[i] = scale * (d[:, None] * k[at]).sum(0)
            G[i, at] = d
    return g_q, g_k, g_v, G


# ------------------------------------------------------------ dropout

def philox(block, site, step, key):
    """Four words of Philox 4x32 with seven rounds for the counter (block, site,
    step low, step high) and the key (low, high)."""
    low = 0xFFFFFFFF
    c = [block & low, site & low, step & low, step >> 32 & low]
    k = [key & low, key >> 32 & low]
    for _ in range(7):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [q >> 32 ^ c[1] ^ k[0], q & low, p >> 32 ^ c[3] ^ k[1], p & low]
        k = [k[0] + 0x9E3779B9 & low, k[1] + 0xBB67AE85 & low]
    return c


def random_bits(n, site, step, key, first=0):
    """16 bits for each of the elements first .. first + n - 1."""
    out, block, words = np.zeros(n, np.int64), -1, None
    for i in range(n):
        e = first + i
        if e // 8 != block:
            block = e // 8
            words = philox(block, site, step, key)
        out[i] = words[e % 8 // 2] >> 16 * (e % 2) & 0xFFFF
    return out


def dropout(x, p, seed, site=0, residual=None, first=0):
    """(y, kept) for elements first .. of a longer tensor."""
    limit = int(np.rint(p * 65536))
    kept = random_bits(len(x), site, seed[1], seed[0], first) >= limit
    y = np.zeros(len(x))
    if limit < 65536:
        y[kept] = np.asarray(x, np.float64)[kept] * (65536 / (65536 - limit))
    return (y if residual is None else residual + y), kept
