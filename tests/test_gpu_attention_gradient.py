"""Attention's backward pass after its own forward pass against the gradient itself, whose
D_i = sum_j P_ij g_o_i v_j belongs to the o that is not rounded.  The formula takes o as it
is stored, so that besides the tolerances against the formula
 - D_i is off by at most sum_d |g_o| times the tolerance of o (in bf16 mostly its rounding),
   and with it G_ij by P_ij of that, where what keys have in common no longer cancels;
 - P_ij is off by the relative tolerance of exp(lse_i)."""
import numpy as np
import pytest

from test_gpu_attention import Case, HALF, _h, _np, _place, _round, _say, _within

pytestmark = pytest.mark.gpu


def _rounded_o(case, tol, ltol):
    """What the errors of o and lse may add to the tolerances of g_q, g_k and g_v."""
    add = [np.zeros((case.Tq, case.H, case.D)), *(np.zeros((case.Tk, case.K, case.D)) for _ in range(2))]
    for rows, cols, h, kv, which in case.parts():
        q, k, v, go = case.q[rows, h], case.k[cols, kv], case.v[cols, kv], case.g[rows, h]
        if not len(q) or not len(k):
            continue
        _, s, seen = case.score_error(q, k, h, which)
        s = np.where(seen, s, -np.inf)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        dp = go @ v.T
        off = (np.abs(go) * tol[rows, h]).sum(-1, keepdims=True)
        moved = np.expm1(ltol[h, rows])[:, None] * p
        dG = moved * (np.abs(dp - (p * dp).sum(-1, keepdims=True)) + off) + p * off
        dG *= 1 + HALF[case.dtype] + 1e-6                       # rounded like G itself
        add[0][rows, h] += case.scale * dG @ np.abs(k)
        add[1][cols, kv] += case.scale * dG.T @ np.abs(q)
        add[2][cols, kv] += (1 + HALF[case.dtype] + 1e-6) * moved.T @ np.abs(go)
    return add


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,heads,kv", [(40, 4, 2), (64, 3, 3), (128, 4, 1)])
@pytest.mark.parametrize("common", [0.0, 24.0])
@pytest.mark.parametrize("causal", [False, True])
def test_against_the_gradient(dtype, D, heads, kv, common, causal):
    h = _h()
    _say(f"attention's gradient, keys with {common} in common, D {D} {dtype} causal {causal}")

    def shift(c):
        c.k = _round(c.k + common, c.dtype)
    case = Case([70, 150, 1], heads, kv, D, dtype, causal, poison=shift)
    d, kw = case.device()
    want, lse, tol, ltol = case.forward()
    o, sums = h.hlq_attention_forward(**d, **kw)
    grads = h.hlq_attention_backward(_place(case.g, dtype, "dense"), *d.values(), o, sums, **kw)
    g, t = case.backward(want, lse)                             # o not rounded: the gradient
    add = _rounded_o(case, tol, ltol)
    for name, got, ref, a, b in zip(("g_q", "g_k", "g_v"), grads, g, t, add):
        # its output's own rounding is relative to what it is, not to the gradient
        _within(_np(got), ref, a + (1 + HALF[dtype]) * b, name)
