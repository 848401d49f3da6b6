"""Attention's tiles of 128 rows (or keys) against the oracle.

Tiles of 128 are for calls that fill the GPU.  Most cases here get there by hundreds
of empty sequences beside a few that the oracle goes through, and each one first shows
by the size of a workspace that it does: that of a bias's gradient holds one line of
buckets for each sequence, head and tile."""
import ctypes

import numpy as np
import pytest

from oracle.train_oracle import round_f32
from test_gpu_attention import Case, _check, _h, _np, _place, _round, _say, _torch, _within

pytestmark = pytest.mark.gpu

LENS = [150, 2, 290, 0, 33, 64, 1, 129] + [0] * 300


def _tiles(total, sequences, heads, rows, dtype, D, causal):
    """Tiles of a sequence in a call with the hint `rows` on `total` rows a head."""
    from hadamard_rank_linear_amd.hlq import Attention
    # a bias in fp32 above 64 keeps small tiles for the gradient of q alone; the rule for
    # the rest sees no more of a head's size than whether its rows have up to 128 bytes
    small = D * (4 if dtype == "f32" else 2) <= 128
    a = Attention(queries=total, keys=total, sequences=sequences, max_len=rows, start_q=1 << 20,
                  start_k=1 << 20, bias=1 << 20, scale=1.0, dtype=1, heads=heads, kv_heads=heads,
                  head_dim=64 if small else 128, causal=causal, bias_dtype=0, buckets=2,
                  max_distance=2, bidirectional=0)
    size = _h().lib_handle().hlq_attention_backward_workspace_size(ctypes.byref(a))
    return (size - (total * heads * 4 + 15) // 16 * 16) // (sequences * heads * 2 * 4)


def _large(case, max_len):
    """All three kernels of the case take tiles of 128 rows."""
    S, shared = len(case.lens), 1 if case.buckets else case.H // case.K
    kind = (case.dtype, case.D, case.causal)
    want = lambda rows: (rows + 127) // 128
    keys = max_len or 2 * -(-case.Tk // S)
    if case.split:
        keys = 2 * -(-case.Tk // S)
    rows = (max_len or 2 * -(-case.Tq // S)) * shared
    assert rows > 32 and keys > 32
    assert _tiles(case.Tq * shared, S, case.H // shared, rows, *kind) == want(rows) < rows / 32
    assert _tiles(case.Tk, S, case.K, keys, *kind) == want(keys) < keys / 32


def _run(case, max_len=290):
    _large(case, max_len)
    _check(case, max_len=max_len)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [32, 40, 64, 96, 128, 33, 100])
@pytest.mark.parametrize("causal", [False, True])
def test_head_sizes(dtype, D, causal):
    _say(f"tiles of 128, D {D} {dtype} causal {causal}")
    _run(Case(LENS, 2, 2, D, dtype, causal))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_longer_than_the_hint(dtype, D, causal):
    """One tile a sequence, which loops over what lies behind it."""
    _say(f"tiles of 128 in a loop, D {D} {dtype} causal {causal}")
    _run(Case(LENS, 2, 2, D, dtype, causal), max_len=33)
    _run(Case(LENS, 2, 2, D, dtype, causal, buckets=8, reach=20), max_len=33)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [40, 64, 96, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_position_bias(dtype, D, causal):
    _say(f"tiles of 128 with a bias, D {D} {dtype} causal {causal}")
    _run(Case(LENS, 2, 2, D, dtype, causal, buckets=32, reach=90, table=dtype))
    _run(Case(LENS, 4, 2, D, dtype, causal, buckets=16, reach=40, both=not causal))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv", [(8, 2), (6, 2), (16, 2)])
@pytest.mark.parametrize("D", [32, 72, 128])
def test_shared_heads(dtype, heads, kv, D):
    _say(f"tiles of 128, heads {heads}/{kv}, D {D} {dtype}")
    _run(Case([70, 0, 150, 3] + [0] * 300, heads, kv, D, dtype, True), max_len=150)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["slice", "odd"])
@pytest.mark.parametrize("D", [17, 64, 128])
def test_layouts_and_tokens_of_no_sequence(dtype, layout, D):
    _say(f"tiles of 128, layout {layout}, D {D} {dtype}")
    _run(Case(LENS, 3, 3, D, dtype, True, layout=layout, gaps=(70, 130)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
def test_keys_of_their_own(dtype, causal):
    """More keys than queries, fewer (rows that see nothing), and none."""
    _say(f"tiles of 128, keys of their own {dtype} causal {causal}")
    rng = np.random.default_rng(3)
    lens, klens = rng.integers(0, 45, 44).tolist(), rng.integers(0, 70, 44).tolist()
    lens[:3], klens[:3] = [140, 60, 9], [20, 0, 300]
    _run(Case(lens, 6, 6, 128, dtype, causal, klens=klens), max_len=140)
    _run(Case(lens, 12, 12, 32, dtype, causal, klens=klens, buckets=8, reach=30), max_len=140)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
def test_without_a_hint(dtype, causal):
    """Real sequences enough, their length guessed from the mean."""
    _say(f"tiles of 128, no hint {dtype} causal {causal}")
    lens = np.random.default_rng(4).integers(2, 60, 66).tolist()
    _run(Case(lens, 8, 8, 64, dtype, causal), max_len=0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("D", [64, 128])
def test_hidden_tokens_do_not_reach_others(dtype, value, D):
    """The last tokens of a causal sequence hold infinities or NaN, upstream gradients
    among them; earlier queries, and other sequences, do not see them."""
    torch, h = _torch(), _h()
    _say(f"tiles of 128, hidden {value} D {D} {dtype}")
    n, bad = 200, 3

    def poison(c):
        for x in (c.k, c.v):
            x[n - bad:n] = value
    case = Case([n, 50] + [0] * 300, 2, 2, D, dtype, True, poison=poison)
    _large(case, n)
    d, kw = case.device()
    want, lse, tol, ltol = case.forward()
    got, gl = h.hlq_attention_forward(**d, **kw, max_len=n)
    ok = np.ones(case.Tq, bool)
    ok[n - bad:n] = False
    assert np.isfinite(want[ok]).all()
    _within(_np(gl)[:, ok], lse[:, ok], ltol[:, ok], "lse")
    _within(_np(got)[ok], want[ok], tol[ok], "o")
    so = _round(np.where(np.isfinite(want), want, 0.0), dtype)
    sl = round_f32(np.where(np.isfinite(lse), lse, 0.0))
    case.g[n - bad:n] = value
    grads = h.hlq_attention_backward(
        _place(case.g, dtype, "dense"), d["q"], d["k"], d["v"], _place(so, dtype, "dense"),
        torch.as_tensor(sl, device="cuda").float(), **kw, max_len=n)
    g, t = case.backward(so, sl)
    _within(_np(grads[0])[ok], g[0][ok], t[0][ok], "g_q")
    other = slice(n, n + 50)
    for i in (1, 2):
        _within(_np(grads[i])[other], g[i][other], t[i][other], f"gradient {i}")
    assert not np.isfinite(_np(grads[2])[:n - bad]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_calls_repeat_bit_for_bit(dtype):
    torch, h = _torch(), _h()
    _say(f"tiles of 128 repeat {dtype}")
    case = Case(LENS, 4, 2, 64, dtype, False, buckets=32)
    _large(case, 290)
    d, kw = case.device()
    g = _place(case.g, dtype, "dense")
    first = None
    for _ in range(4):
        y, lse = h.hlq_attention_forward(**d, **kw, max_len=290)
        got = (y, lse, *h.hlq_attention_backward(g, *d.values(), y, lse, **kw, max_len=290))
        first = first or [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(first, got))
