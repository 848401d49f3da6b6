"""Attention of shared heads that are packed into neighbouring rows, and launches of
more items than workgroups, whose later items go by a loop."""
import numpy as np
import pytest

from test_gpu_attention import Case, HALF, U, _check, _dt, _h, _say, _torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv", [(4, 1), (8, 1), (16, 1), (32, 8)])
@pytest.mark.parametrize("D", [72, 96, 128])
def test_packed_heads(dtype, heads, kv, D):
    _say(f"packed heads {heads}/{kv}, D {D} {dtype}")
    _check(Case([5, 66], heads, kv, D, dtype, True))
    if heads == 4:
        _check(Case([5, 131], heads, kv, D, dtype, False))


def _pairs(q, k, v, g, lens, scale, causal, bias, dtype):
    """Outputs and tolerances for sequences of up to two tokens, in 64 bits: a token
    sees itself and, unless it is hidden, the other one.  q, g [T, H, D], k, v [T, K, D]
    (fp64), bias [buckets, H] of two buckets a side of one distance each.
    Returns ((o, lse, g_q, g_k, g_v, g_bias), tolerances) with o as the type stores it
    in the gradients."""
    torch = _torch()
    T, H, D = q.shape
    K = k.shape[1]
    e = HALF[dtype]
    at = torch.repeat_interleave(torch.arange(len(lens), device=q.device), lens)
    start = torch.cumsum(lens, 0) - lens
    i = torch.arange(T, device=q.device)
    first = i == start[at]
    two = lens[at] == 2
    other = torch.where(two, torch.where(first, i + 1, i - 1), i)
    sees = two & ~first if causal else two           # whether it sees the other one
    K2, V2 = (x.repeat_interleave(H // K, 1) for x in (k, v))
    keys = torch.stack([K2, K2[other]], 2)           # [T, H, 2, D]
    vals = torch.stack([V2, V2[other]], 2)
    S = scale * (q[:, :, None] * keys).sum(-1)
    err = (D + 4) * U * scale * (q[:, :, None] * keys).abs().sum(-1)
    if bias is not None:
        # buckets of distance 0, of the key behind (+1) and of the one before (-1)
        b = torch.stack([bias[0].expand(T, H),
                         torch.where(first[:, None], bias[3 if not causal else 0], bias[1])], 2)
        S, err = S + b, err + 3 * U * b.abs()
    err = err + 4 * U * S.abs()
    S[:, :, 1] = torch.where(sees[:, None], S[:, :, 1], float("-inf"))
    err[:, :, 1] = torch.where(sees[:, None], err[:, :, 1], 0.0)
    lse = torch.logsumexp(S, -1)
    P = torch.exp(S - lse[:, :, None])
    worst = 2 * err.max(-1).values + 8 * U
    o = (P[..., None] * vals).sum(2)
    to = (worst[..., None] + 10 * U + e) * (P[..., None] * vals.abs()).sum(2) + (e + U) * o.abs() + 1e-30
    tl = worst + 10 * U + 4 * U * lse.abs()
    so = o.to(_dt(dtype)).double()
    sl = lse.float().double()
    P = torch.exp(S - sl[:, :, None])
    perr = P * (err + 4 * U * sl.abs()[..., None] + 8 * U)
    dp = (g[:, :, None] * vals).sum(-1)
    delta = (g * so).sum(-1)[..., None]
    size = (g[:, :, None] * vals).abs().sum(-1) + (g * so).abs().sum(-1)[..., None]
    G = P * (dp - delta)
    gerr = perr * ((dp - delta).abs() + 2 * U * size) + P * (D + 4) * U * size
    m = 2 * (H // K)
    shared = lambda x: x.view(T, K, H // K, D).sum(2)

    def back(w, x):
        """What the queries leave at their keys: w [T, H, 2], x [T, H, D]."""
        y = w[:, :, :1] * x
        y.index_add_(0, other, w[:, :, 1:] * x)
        return shared(y)
    Ge, Pe = gerr + (e + (m + 4) * U) * G.abs(), perr + (e + (m + 4) * U) * P
    out = [o, lse.t(), scale * (G[..., None] * keys).sum(2), scale * back(G, q), back(P, g)]
    tol = [to, tl.t(), scale * ((gerr + (e * e + 8 * U) * G.abs())[..., None] * keys.abs()).sum(2),
           scale * back(Ge, q.abs()), back(Pe, g.abs())]
    if bias is not None:
        where = torch.zeros((4, T, H, 2), dtype=torch.bool, device=q.device)
        where[0, :, :, 0] = True
        for b, rows in (((3 if not causal else 0), first), (1, ~first)):
            where[b, :, :, 1] |= (sees & rows)[:, None]
        out.append((where * G).sum((1, 3)))
        # an item's sum in fp32: its two pairs a row, the line and its fold
        tol.append((where * (gerr + 308 * U * G.abs())).sum((1, 3)))
    for n in range(2, len(out)):
        half = e if n < 5 else 0.0
        tol[n] = tol[n] + (half + 2 * U) * out[n].abs() + 1e-30
    return out, tol, so, sl


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("max_len", [0, 40])     # tiles of 32, and of 128
@pytest.mark.parametrize("bias", [False, True])
def test_more_items_than_workgroups(dtype, max_len, bias):
    """2^18 sequences of up to two tokens, 8 items each (4 for the keys beside a bias): workgroups take a second item.  Every output is compared."""
    torch, h = _torch(), _h()
    _say(f"items beyond 2^20, {dtype} hint {max_len} bias {bias}")
    S, H, K, D, causal = (1 << 18) + 77, 16 if not bias else 8, 8 if not bias else 4, 8, not bias
    gen = torch.Generator(device="cuda").manual_seed(6)
    lens = torch.randint(0, 3, (S,), generator=gen, device="cuda")
    T = int(lens.sum())
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(_dt(dtype))
    q, k, v, g = r(T, H, D), r(T, K, D), r(T, K, D), r(T, H, D)
    table = torch.randn((4, H), generator=gen, device="cuda") if bias else None
    start = torch.cat([lens.new_zeros(1), lens.cumsum(0)])
    scale = float(np.float32(D ** -0.5))
    kw = dict(start=start, causal=causal, scale=scale, bias=table, max_distance=2, max_len=max_len)
    up = lambda t: None if t is None else t.double()
    want, tol, so, sl = _pairs(up(q), up(k), up(v), up(g), lens, scale, causal, up(table), dtype)
    o, lse = h.hlq_attention_forward(q, k, v, **kw)
    grads = h.hlq_attention_backward(g, q, k, v, so.to(_dt(dtype)), sl.t().contiguous().float(), **kw)
    names = ("o", "lse", "g_q", "g_k", "g_v", "g_bias")
    for name, got, w, t in zip(names, (o, lse, *grads), want, tol):
        off = (got.double() - w).abs()
        assert bool((off <= t).all()), (name, float((off - t).max()), int((off > t).sum()))
