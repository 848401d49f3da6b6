"""Attention over packed sequences, its backward pass and the relative position
bias on the GPU against their definitions in 64 bits (oracle/attention_oracle.py),
at the sizes, bounds, masks and layouts where they can go wrong.

Tolerances, with u = 2^-24 the half step of fp32 and e that of the type (2^-8
relative for bf16, 0 for fp32, whose half step counts among the u):
 - a score: D products summed in fp32 in any order and scaled, (D + 4) u scale
   sum_d |q_d k_d|; with a bias 3 u |bias| more; 4 u |S| for powers of two;
 - a probability: relative, that of its score and of the row's maximum or lse,
   and 4 u for the exponential and the sum's factors;
 - each product's sum of n terms: n u sum|terms|, and e sum|terms| for the
   rounding of the probabilities or score gradients to the type; in the gradient of
   q, 2 n terms and e^2: what the rounding takes off is a second product, and only
   its rounding is lost;
 - an output: e of itself.
fp32 has nothing below TINY = 2^-126 (an exponential under it is zero, where the
definition in 64 bits still has 10^-73 at scores of hundreds): each probability and
each product may be off by that much besides.
"""
import numpy as np
import pytest

import oracle.attention_oracle as o
from oracle.train_oracle import round_bf16, round_f32

pytestmark = pytest.mark.gpu

U, TINY = 2.0 ** -24, 2.0 ** -126
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


def _say(msg):
    print(f"\n[gpu-case] {msg}", flush=True)


def _np(t):
    return t.detach().double().cpu().numpy()


def _round(v, name):
    return round_bf16(v) if name == "bf16" else round_f32(v)


def _within(got, want, tol, what):
    tol = np.broadcast_to(tol, want.shape)
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want)
        ok = (off <= tol) | (got == want) | (np.isnan(got) & np.isnan(want))
    assert ok.all(), (f"{what}: {(~ok).sum()} of {ok.size} off, first at {np.argwhere(~ok)[0]}: "
                      f"{got[~ok][0]} for {want[~ok][0]} (tolerance {tol[~ok][0]})")


def _place(v, name, layout):
    """v [T, heads, D] on the GPU: dense, a slice of wider rows, or heads first
    with every row one element off a 16-byte boundary."""
    torch = _torch()
    v = torch.as_tensor(v)
    T, H, D = v.shape
    nan = lambda *s: torch.full(s, float("nan"), dtype=_dt(name), device="cuda")
    out = {"dense": lambda: nan(T, H, D),
           "slice": lambda: nan(T, H + 3, D)[:, 2:2 + H],
           "odd": lambda: nan(H, T, D + 3).permute(1, 0, 2)[:, :, 1:1 + D]}[layout]()
    return out.copy_(v)


class Case:
    """Inputs of one call, rounded to the type, and the oracle's outputs with
    their tolerances."""

    def __init__(self, lens, heads, kv, D, dtype, causal=False, klens=None, buckets=0, reach=128,
                 both=None, gaps=(0, 0), layout="dense", scale=None, seed=0, table="f32", poison=None):
        rng = np.random.default_rng(seed + 1000 * D + sum(lens))
        self.lens, self.klens = list(lens), list(klens if klens is not None else lens)
        self.H, self.K, self.D, self.dtype, self.causal = heads, kv, D, dtype, causal
        self.buckets, self.reach = buckets, reach
        self.both = (not causal) if both is None else both
        self.scale = float(np.float32(scale or D ** -0.5))
        self.table, self.layout, self.split = table, layout, klens is not None
        a, b = gaps
        self.Tq = a + sum(self.lens) + b
        self.Tk = a + sum(self.klens) + b
        self.start = a + np.concatenate([[0], np.cumsum(self.lens)])
        self.start_k = a + np.concatenate([[0], np.cumsum(self.klens)])
        make = lambda T, h, s=1.0: _round(s * rng.normal(size=(T, h, D)), dtype)
        self.q, self.k, self.v = make(self.Tq, heads, 1.5), make(self.Tk, kv), make(self.Tk, kv)
        self.g = make(self.Tq, heads)
        self.bias = _round(rng.normal(size=(buckets, heads)), table) if buckets else None
        for x, n in ((self.q, self.Tq), (self.k, self.Tk), (self.v, self.Tk), (self.g, self.Tq)):
            x[:a] = np.nan                       # tokens of no sequence
            x[n - b:] = np.nan if b else x[n - b:]
        if poison:
            poison(self)

    def parts(self):
        for s in range(len(self.lens)):
            rows = slice(self.start[s], self.start[s + 1])
            cols = slice(self.start_k[s], self.start_k[s + 1])
            which = o.bucket_table(self.lens[s], self.klens[s], self.buckets, self.reach, self.both) \
                if self.buckets else None
            for h in range(self.H):
                yield rows, cols, h, h * self.K // self.H, which

    def score_error(self, q, k, h, which):
        err = (self.D + 4) * U * self.scale * (np.abs(q)[:, None] * np.abs(k)[None]).sum(-1)
        s, seen = o.scores(q, k, self.scale, self.causal,
                           None if which is None else self.bias[:, h], which)
        s = np.where(seen & np.isfinite(s), s, 0.0)
        if which is not None:
            b = np.where(np.isfinite(self.bias[:, h]), self.bias[:, h], 0.0)
            err = err + 3 * U * np.abs(b)[which]
        return np.where(seen, err + 4 * U * np.abs(s), 0.0), s, seen

    def forward(self):
        """(o, lse, tolerances of both)."""
        out, lse = np.zeros((self.Tq, self.H, self.D)), np.full((self.H, self.Tq), -np.inf)
        tol, ltol = np.zeros_like(out), np.zeros_like(lse)
        e = HALF[self.dtype]
        fin = lambda x: np.where(np.isfinite(x), np.abs(x), 0.0)
        with np.errstate(invalid="ignore", over="ignore"):
            for rows, cols, h, kv, which in self.parts():
                q, k, v = self.q[rows, h], self.k[cols, kv], self.v[cols, kv]
                bias = None if which is None else self.bias[:, h]
                out[rows, h], lse[h, rows] = o.forward(q, k, v, self.scale, self.causal, bias, which)
                if not len(q) or not len(k):
                    continue
                err, s, seen = self.score_error(q, k, h, which)
                worst = 2 * err.max(-1) + 8 * U
                p = np.where(seen, np.exp(s - lse[h, rows][:, None]), 0.0)
                p = np.where(np.isfinite(p), p, 0.0)
                mass = p @ fin(v)
                n = len(k)
                tol[rows, h] = (worst[:, None] + (n + 8) * U + e) * mass + (e + U) * np.abs(out[rows, h]) \
                    + TINY * (1 + fin(v).sum(0))
                ltol[h, rows] = worst + (n + 8) * U + 4 * U * np.abs(lse[h, rows])
        return out, lse, tol, ltol

    def backward(self, out, lse):
        """((g_q, g_k, g_v, g_bias), tolerances) for the o and lse that are given."""
        new = lambda T, h: np.zeros((T, h, self.D))
        g = [new(self.Tq, self.H), new(self.Tk, self.K), new(self.Tk, self.K),
             np.zeros((max(self.buckets, 1), self.H))]
        tol = [np.zeros_like(x) for x in g]
        e, et, sc = HALF[self.dtype], HALF[self.table], self.scale
        fin = lambda x: np.where(np.isfinite(x), np.abs(x), 0.0)
        for rows, cols, h, kv, which in self.parts():
            q, k, v, go = self.q[rows, h], self.k[cols, kv], self.v[cols, kv], self.g[rows, h]
            bias = None if which is None else self.bias[:, h]
            oo, ls = out[rows, h], lse[h, rows]
            gq, gk, gv, G = o.backward(go, q, k, v, oo, ls, sc, self.causal, bias, which)
            g[0][rows, h] += gq
            g[1][cols, kv] += gk
            g[2][cols, kv] += gv
            if not len(q) or not len(k):
                continue
            err, s, seen = self.score_error(q, k, h, which)
            live = np.where(np.isfinite(ls), ls, np.inf)[:, None]
            p = np.where(seen, np.exp(s - live), 0.0)
            perr = p * (err + 4 * U * np.abs(ls)[:, None].clip(max=1e30) + 8 * U)
            perr = np.where(np.isfinite(perr), perr, 0.0) + TINY
            dp, de = fin(go) @ fin(v).T, (fin(go) * fin(oo)).sum(-1)[:, None]
            diff = fin(G) / np.where(p > 0, p, 1.0)
            gerr = perr * (diff + 2 * U * (dp + de)) + p * (self.D + 4) * U * (dp + de) \
                + TINY * (1 + dp + de)
            G = fin(G)
            n, m = len(k), len(q) * (self.H // self.K)
            tol[0][rows, h] += sc * ((gerr + (e * e + (2 * n + 4) * U) * G) @ fin(k))
            tol[1][cols, kv] += sc * ((gerr + (e + (m + 4) * U) * G).T @ fin(q))
            tol[2][cols, kv] += (perr + (e + (m + 4) * U) * p).T @ fin(go)
            if which is not None:
                # blocks of 32 rows, the keys' blocks, the line and its fold
                adds = (len(q) + len(k) + 2 * self.reach + 300) * U
                for b in range(self.buckets):
                    at = which == b
                    g[3][b, h] += o_sum(G, at, self, rows, cols, h, kv, which, oo, ls)
                    tol[3][b, h] += (gerr[at] + adds * G[at]).sum()
        for i, half in ((0, e), (1, e), (2, e), (3, et)):
            tol[i] += (half + 2 * U) * np.abs(np.where(np.isfinite(g[i]), g[i], 0.0)) + TINY
        return g, tol

    def device(self):
        torch = _torch()
        up = lambda v: torch.as_tensor(v, device="cuda")
        d = dict(q=_place(self.q, self.dtype, self.layout), k=_place(self.k, self.dtype, self.layout),
                 v=_place(self.v, self.dtype, self.layout))
        kw = dict(start=up(self.start), start_k=up(self.start_k) if self.split else None,
                  causal=self.causal, scale=self.scale)
        if self.buckets:
            kw.update(bias=up(self.bias).to(_dt(self.table)), max_distance=self.reach,
                      bidirectional=self.both)
        return d, kw


def o_sum(G, at, case, rows, cols, h, kv, which, oo, ls):
    """Sum of the signed score gradients of one bucket."""
    if not hasattr(case, "_signed") or case._signed[0] != (rows.start, h):
        signed = o.backward(case.g[rows, h], case.q[rows, h], case.k[cols, kv], case.v[cols, kv], oo,
                            ls, case.scale, case.causal, case.bias[:, h], which)[3]
        case._signed = ((rows.start, h), signed)
    return case._signed[1][at].sum()


def _check(case, max_len=0, backward=True):
    """One forward and one backward call against the oracle; every output."""
    torch, h = _torch(), _h()
    d, kw = case.device()
    want, lse, tol, ltol = case.forward()
    got, gl = h.hlq_attention_forward(**d, **kw, max_len=max_len)
    _within(_np(gl), lse, ltol, "lse")
    _within(_np(got), want, tol, "o")
    if not backward:
        return
    # the backward pass from the definition's o and lse, stored in their types
    so, sl = _round(want, case.dtype), round_f32(lse)
    up = lambda v: torch.as_tensor(v, device="cuda")
    g, gt = case.backward(so, sl)
    grads = h.hlq_attention_backward(_place(case.g, case.dtype, case.layout), d["q"], d["k"], d["v"],
                                     _place(so, case.dtype, case.layout), up(sl).float(), **kw,
                                     max_len=max_len)
    for name, a, b, t in zip(("g_v", "g_k", "g_q"), grads[2::-1], g[2::-1], gt[2::-1]):
        _within(_np(a), b, t, name)
    if case.buckets:
        _within(_np(grads[3]), g[3], gt[3], "g_bias")
    else:
        assert grads[3] is None


# the smallest, block edges, odd lengths, an empty sequence
LENS = {"one": [1], "two": [1, 2], "edges": [31, 32, 33, 0, 1], "tile": [64, 65, 127],
        "tiles": [128, 129, 3], "long": [300]}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(dtype, lens, causal):
    _say(f"attention lengths {lens} {dtype} causal {causal}")
    _check(Case(LENS[lens], 2, 2, 64, dtype, causal))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 7, 8, 32, 33, 40, 72, 80, 96, 100, 127, 128])
def test_head_sizes(dtype, D):
    _say(f"attention head size {D} {dtype}")
    _check(Case([70, 19], 2, 1, D, dtype, causal=D % 2 == 0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["slice", "odd"])
@pytest.mark.parametrize("D", [17, 64, 128])
def test_layouts(dtype, layout, D):
    _say(f"attention layout {layout} D {D} {dtype}")
    _check(Case([40, 90], 3, 3, D, dtype, causal=True, layout=layout))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv", [(4, 1), (6, 2), (5, 5), (35, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_shared_heads(dtype, heads, kv, causal):
    _say(f"attention heads {heads}/{kv} {dtype} causal {causal}")
    _check(Case([5, 66], heads, kv, 32, dtype, causal))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,klens", [([1, 1, 1], [1, 300, 700]), ([2, 1], [0, 130]),
                                        ([7, 5], [3, 900]), ([40], [1500]), ([200, 3], [60, 0])])
@pytest.mark.parametrize("causal", [False, True])
def test_queries_against_a_cache(dtype, lens, klens, causal):
    """Fewer queries than keys (a cache), more (rows that see nothing), none."""
    _say(f"attention cache {lens} {klens} {dtype} causal {causal}")
    _check(Case(lens, 4, 2, 64, dtype, causal, klens=klens))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,D", [(8, 128), (1, 40)])
def test_shares_of_the_keys(dtype, heads, D):
    """Long caches are cut into shares, joined by a second launch: one query of
    each head (32 rows shared by the waves), and 50 (128 rows)."""
    h = _h()
    _say(f"attention shares {dtype} {heads} {D}")
    for n in (1, 50):
        case = Case([n, n, 0], heads, 1, D, dtype, True, klens=[2100, 77, 30], gaps=(3, 2))
        d, kw = case.device()
        _check(case, max_len=n, backward=False)
        _check(case, max_len=0, backward=False)
    assert h.lib_handle()  # the library was loaded


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("klens", [[9000, 1, 0, 2, 300, 129, 40, 128, 127, 1, 1, 65], [70001]])
def test_shares_of_unequal_sequences(dtype, klens):
    """Sequences far longer than the shares are made for, many shares without a key
    (whose part of the workspace holds NaN), more keys than 64 of the least shares."""
    torch, h = _torch(), _h()
    _say(f"attention shares of {len(klens)} sequences {dtype}")
    case = Case([1] * len(klens), 4, 2, 64, dtype, True, klens=klens)
    _check(case, max_len=1, backward=False)
    d, kw = case.device()
    want = h.hlq_attention_forward(**d, **kw, max_len=1)
    rows = case.H * sum(case.lens) * (case.D + 2) * 4      # one share's bytes
    ws = torch.full((64 * rows,), 255, dtype=torch.uint8, device="cuda")
    got = h.hlq_attention_forward(**d, **kw, max_len=1, workspace=ws)
    assert not bool((ws == 255).all())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_hint_with_keys_of_their_own(dtype):
    """The longest sequence's queries say nothing of its keys."""
    _say(f"attention hint, keys of their own {dtype}")
    _check(Case([3, 5, 1], 4, 2, 64, dtype, True, klens=[700, 30, 300]), max_len=5)
    _check(Case([40, 2], 2, 2, 40, dtype, False, klens=[9, 290], buckets=8, reach=20), max_len=40)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("max_len", [1, 33, 1 << 20])
def test_hint_does_not_matter(dtype, max_len):
    """A longest length that is wrong either way: sequences beyond it are looped
    over."""
    _say(f"attention hint {max_len} {dtype}")
    _check(Case([150, 2, 290, 0], 2, 1, 32, dtype, True, gaps=(1, 4)), max_len=max_len)
    _check(Case([150, 290], 2, 2, 32, dtype, False, buckets=8, reach=20), max_len=max_len)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gaps", [(0, 5), (9, 0), (70, 130)])
def test_tokens_of_no_sequence_get_zeros(dtype, gaps):
    """They hold NaN here; the oracle's outputs there are zeros, and lse -inf."""
    _say(f"attention gaps {gaps} {dtype}")
    _check(Case([20, 30], 2, 1, 32, dtype, True, gaps=gaps))
    _check(Case([20, 30], 2, 2, 32, dtype, False, gaps=gaps, buckets=4, reach=9))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_sequence_has_tokens(dtype):
    _say(f"attention of nothing {dtype}")
    _check(Case([0, 0], 2, 1, 32, dtype, True, gaps=(4, 3)))
    _check(Case([0], 2, 2, 32, dtype, False, buckets=4, reach=9))
    _check(Case([3, 2], 2, 2, 32, dtype, False, klens=[0, 0], buckets=4, reach=9))


BIAS = [(32, 128, True), (32, 128, False), (4, 3, True), (2, 2, False), (128, 1024, True), (16, 40, False)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("buckets,reach,both", BIAS)
@pytest.mark.parametrize("causal", [False, True])
def test_position_bias(dtype, buckets, reach, both, causal):
    """Tiles near the diagonal, beyond reach on either side, and across."""
    _say(f"position bias {buckets} {reach} {both} {dtype} causal {causal}")
    _check(Case([333, 1, 0, 64], 3, 3, 32, dtype, causal, buckets=buckets, reach=reach, both=both,
                table=dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [40, 64, 96, 128])
def test_position_bias_shared_heads(dtype, D):
    _say(f"position bias, shared heads, D {D} {dtype}")
    _check(Case([130, 45], 4, 2, D, dtype, True, buckets=32))
    _check(Case([1, 3], 4, 2, D, dtype, True, klens=[1100, 400], buckets=32), max_len=3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bias_of_minus_infinity_hides_a_bucket(dtype):
    """Bucket 0 of one head (the query itself and, one-sided, what lies behind) and
    every bucket of another: rows without keys."""
    _say(f"bias -inf {dtype}")

    def poison(c):
        c.bias[0, 0] = -np.inf
        c.bias[:, 1] = -np.inf
    case = Case([70, 5], 3, 3, 32, dtype, True, buckets=16, poison=poison)
    _check(case)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_hidden_tokens_do_not_reach_others(dtype, value):
    """The last tokens of a causal sequence hold infinities or NaN: no earlier
    query sees them, nor does any other sequence; gradients of earlier keys get
    nothing from queries that are finite, and those of the last tokens are what
    the formulas give."""
    torch, h = _torch(), _h()
    _say(f"hidden {value} {dtype}")
    n, bad = 100, 3

    def poison(c):
        for x in (c.k, c.v):
            x[c.start_k[1] - bad:c.start_k[1]] = value
    case = Case([n, 50], 2, 1, 64, dtype, True, poison=poison)
    d, kw = case.device()
    want, lse, tol, ltol = case.forward()
    got, gl = h.hlq_attention_forward(**d, **kw)
    ok = np.ones(case.Tq, bool)
    ok[n - bad:n] = False
    assert np.isfinite(want[ok]).all()
    _within(_np(gl)[:, ok], lse[:, ok], ltol[:, ok], "lse")
    _within(_np(got)[ok], want[ok], tol[ok], "o")
    so, sl = _round(np.where(np.isfinite(want), want, 0.0), case.dtype), round_f32(np.where(
        np.isfinite(lse), lse, 0.0))
    # upstream gradients of the rows that see them are zero or poisoned too; those
    # rows' queries are seen by no later key
    case.g[n - bad:n] = value
    grads = h.hlq_attention_backward(
        _place(case.g, dtype, "dense"), d["q"], d["k"], d["v"], _place(so, dtype, "dense"),
        torch.as_tensor(sl, device="cuda").float(), **kw)
    g, t = case.backward(so, sl)
    _within(_np(grads[0])[ok], g[0][ok], t[0][ok], "g_q")
    other = slice(n, n + 50)
    _within(_np(grads[1])[other], g[1][other], t[1][other], "g_k")
    _within(_np(grads[2])[other], g[2][other], t[2][other], "g_v")
    # keys that the poisoned queries see get NaN or infinities from them
    assert not np.isfinite(_np(grads[2])[:n - bad]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_poisoned_queries_do_not_reach_hidden_keys(dtype):
    """A query in the middle of a causal sequence is NaN: keys behind it are
    finite, keys up to it are not."""
    torch, h = _torch(), _h()
    _say(f"poisoned query {dtype}")

    def poison(c):
        c.q[37] = c.g[37] = np.nan
    case = Case([90], 1, 1, 64, dtype, True, poison=poison)
    d, kw = case.device()
    want, lse, tol, ltol = case.forward()
    rest = np.arange(90) != 37
    got, _ = h.hlq_attention_forward(**d, **kw)
    _within(_np(got)[rest], want[rest], tol[rest], "o")
    so, sl = _round(np.nan_to_num(want), dtype), round_f32(np.nan_to_num(lse))
    g, t = case.backward(so, sl)
    grads = h.hlq_attention_backward(
        _place(case.g, dtype, "dense"), d["q"], d["k"], d["v"], _place(so, dtype, "dense"),
        torch.as_tensor(sl, device="cuda").float(), **kw)
    for i in (1, 2):
        assert np.isnan(_np(grads[i])[:38]).all()
        _within(_np(grads[i])[38:], g[i][38:], t[i][38:], f"gradient {i}")
    _within(_np(grads[0])[rest], g[0][rest], t[0][rest], "g_q")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [40, 128])
def test_keys_with_a_common_part(dtype, D):
    """It cancels in the gradient of q, whose score gradients sum to zero; their
    rounding, times the common part, would be many times the result's."""
    _say(f"attention, keys with a common part, D {D} {dtype}")

    def shift(c):
        c.k = _round(c.k + 24.0, c.dtype)

    _check(Case([70, 150], 4, 2, D, dtype, True, poison=shift))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [2.0 ** -40, 30.0])
def test_scales(dtype, scale):
    """Scores of nothing, and scores of hundreds (one key takes the row)."""
    _say(f"scale {scale} {dtype}")
    _check(Case([50, 33], 2, 1, 32, dtype, True, scale=scale))


def test_offsets_past_32_bits():
    """Keys and values 4 MiB apart, 1100 of them: byte offsets up to 4.6e9."""
    torch, h = _torch(), _h()
    _say("attention offsets past 32 bits")
    n, step = 1100, 1 << 21
    big = torch.empty(n * step, dtype=torch.bfloat16, device="cuda")
    far = [big.as_strided((n, 1, 64), (step, 64, 1), i * 128) for i in (0, 1, 2, 3)]
    gen = torch.Generator(device="cuda").manual_seed(5)
    dense = [torch.randn((n, 1, 64), generator=gen, device="cuda").bfloat16() for _ in range(2)]
    for f, x in zip(far, dense):
        f.copy_(x)
    q = torch.randn((n, 1, 64), generator=gen, device="cuda").bfloat16()
    a = h.hlq_attention_forward(q, far[0], far[1], causal=True)
    b = h.hlq_attention_forward(q, *dense, causal=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    ga = h.hlq_attention_backward(q, q, far[0], far[1], *a, causal=True, g_k=far[2], g_v=far[3])
    gb = h.hlq_attention_backward(q, q, *dense, *b, causal=True)
    assert all(torch.equal(x, y) for x, y in zip(ga[:3], gb[:3]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_calls_repeat_bit_for_bit(dtype):
    torch, h = _torch(), _h()
    _say(f"attention repeats {dtype}")
    case = Case([200, 3, 130], 4, 2, 64, dtype, False, buckets=32)
    d, kw = case.device()
    g = _place(case.g, dtype, "dense")
    first = None
    for _ in range(4):
        y, lse = h.hlq_attention_forward(**d, **kw)
        got = (y, lse, *h.hlq_attention_backward(g, *d.values(), y, lse, **kw))
        first = first or [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_outputs_given_and_nothing_else_written():
    """Gradients into slices of one tensor; what lies between the slices stays."""
    torch, h = _torch(), _h()
    _say("attention outputs given")
    for D in (24, 64, 33):
        case = Case([77, 40], 4, 2, D, "bf16", True)
        d, kw = case.device()
        g = _place(case.g, "bf16", "dense")
        o_, lse = h.hlq_attention_forward(**d, **kw)
        box = torch.full((117, 12, D), 7.0, dtype=torch.bfloat16, device="cuda")
        y = box[:, 1:5]
        assert h.hlq_attention_forward(**d, **kw, o=y)[0] is not None
        assert torch.equal(y, o_) and (box[:, 0] == 7).all() and (box[:, 5:] == 7).all()
        box.fill_(7.0)
        out = dict(g_q=box[:, 0:4], g_k=box[:, 5:7], g_v=box[:, 9:11])
        got = h.hlq_attention_backward(g, *d.values(), o_, lse, **kw, **out)
        want = h.hlq_attention_backward(g, *d.values(), o_, lse, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
        assert all((box[:, i] == 7).all() for i in (4, 7, 8, 11))


def test_expanded_inputs():
    """A key and value that every token and head shares (strides of zero)."""
    torch, h = _torch(), _h()
    _say("attention expanded")
    q = torch.randn(40, 4, 32, device="cuda")
    k = torch.randn(32, device="cuda")
    far, near = k.expand(40, 2, 32), k.expand(40, 2, 32).contiguous()
    a = h.hlq_attention_forward(q, far, far)
    assert all(torch.equal(x, y) for x, y in zip(a, h.hlq_attention_forward(q, near, near)))
    ga = h.hlq_attention_backward(q, q, far, far, *a)
    gb = h.hlq_attention_backward(q, q, near, near, *a)
    assert all(torch.equal(x, y) for x, y in zip(ga[:3], gb[:3]))


def test_refusals_on_the_gpu():
    torch, h = _torch(), _h()
    _say("attention refusals")
    f = lambda *s, **k: torch.zeros(s, device="cuda", **k)
    q, k = f(6, 4, 8), f(6, 2, 8)
    start = torch.tensor([0, 2, 6], device="cuda")
    bad = [(dict(q=q.cpu(), k=k, v=k), ValueError), (dict(q=q, k=k.cpu(), v=k), ValueError),
           (dict(q=q, k=k, v=k.double()), TypeError), (dict(q=q.half(), k=k.half(), v=k.half()), TypeError),
           (dict(q=q, k=k, v=f(6, 2, 9)), ValueError), (dict(q=q, k=f(6, 2, 16)[:, :, ::2], v=k), ValueError),
           (dict(q=q, k=f(6, 3, 8), v=f(6, 3, 8)), h.HLQError), (dict(q=f(6, 4, 200), k=f(6, 2, 200),
                                                                     v=f(6, 2, 200)), h.HLQError),
           (dict(q=q, k=k, v=k, start=start.int()), TypeError), (dict(q=q, k=k, v=k, start=start[:1]), ValueError),
           (dict(q=q, k=k, v=k, start=start.cpu()), ValueError), (dict(q=q, k=k, v=k, start_k=start), ValueError),
           (dict(q=q, k=k, v=k, start=start, start_k=start[:2]), ValueError),
           (dict(q=q[:5], k=k, v=k, start=start), ValueError),
           (dict(q=q, k=k, v=k, bias=f(32, 3)), ValueError), (dict(q=q, k=k, v=k, bias=f(32)), ValueError),
           (dict(q=q, k=k, v=k, bias=f(32, 4, dtype=torch.float64)), TypeError),
           (dict(q=q, k=k, v=k, bias=f(31, 4)), h.HLQError), (dict(q=q, k=k, v=k, bias=f(0, 4)), ValueError),
           (dict(q=q, k=k, v=k, scale=0.0), h.HLQError), (dict(q=q, k=k, v=k, scale="a"), TypeError),
           (dict(q=q, k=k, v=k, max_len=-1), h.HLQError), (dict(q=q, k=k, v=k, o=f(6, 4, 9)), ValueError),
           (dict(q=q, k=k, v=k, o=f(6, 1, 8).expand(6, 4, 8)), h.HLQError),
           (dict(q=q, k=k, v=k, workspace=f(8)), TypeError), (dict(q=q, k=k, v=k, stream=3), TypeError)]
    for kw, error in bad:
        with pytest.raises(error):
            h.hlq_attention_forward(**kw)
    y, lse = h.hlq_attention_forward(q, k, k)
    for kw, error in [(dict(lse=lse.t()), ValueError), (dict(g_o=q[:, :2]), ValueError),
                      (dict(g_k=f(6, 4, 8)), ValueError), (dict(workspace=f(1, dtype=torch.uint8)), h.HLQError)]:
        args = dict(g_o=q, q=q, k=k, v=k, o=y, lse=lse)
        args.update(kw)
        with pytest.raises(error):
            h.hlq_attention_backward(**args)
    torch.cuda.synchronize()
