"""Attention of batches that are padded to a fixed number of tokens: what belongs to no
sequence gets zeros, by as many workgroups as the padding may need."""
import pytest

from test_attention_sizes import _sizes
from test_gpu_attention import _dt, _h, _say, _torch

pytestmark = pytest.mark.gpu


def _nan(torch, *shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 33, 64, 100, 128])
@pytest.mark.parametrize("before,behind", [(0, 6000), (5001, 0), (2000, 3003)])
def test_much_padding(dtype, D, before, behind):
    """The padding holds NaN, the outputs NaN before the call; the rest is as without
    padding, bit for bit."""
    torch, h = _torch(), _h()
    _say(f"attention padded by {before} and {behind}, D {D} {dtype}")
    t, H, K, n = _dt(dtype), 6, 3, 90
    T = before + n + behind
    gen = torch.Generator(device="cuda").manual_seed(D)
    full = lambda heads: _nan(torch, T, heads, D, dtype=t)
    q, k, v, g = full(H), full(K), full(K), full(H)
    mine = slice(before, before + n)
    for x in (q, k, v, g):
        x[mine] = torch.randn((n, x.shape[1], D), generator=gen, device="cuda").to(t)
    at = torch.tensor([0, 20, 20, n], device="cuda")
    kw = dict(causal=True, max_len=70)
    o, lse = h.hlq_attention_forward(q, k, v, at + before, o=full(H), **kw)
    grads = h.hlq_attention_backward(g, q, k, v, o, lse, at + before, g_q=full(H), g_k=full(K),
                                     g_v=full(K), **kw)
    cut = [x[mine].contiguous() for x in (q, k, v, g)]
    want, wl = h.hlq_attention_forward(*cut[:3], at, **kw)
    wg = h.hlq_attention_backward(cut[3], *cut[:3], want, wl, at, **kw)
    for got, ref in zip((o, *grads[:3]), (want, *wg[:3])):
        assert torch.equal(got[mine], ref)
        assert not got[:before].any() and not got[before + n:].any()
    assert torch.equal(lse[:, mine], wl)
    rest = torch.cat([lse[:, :before], lse[:, before + n:]], 1)
    assert bool((rest == float("-inf")).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padding_with_shares_of_the_keys(dtype):
    """Single tokens against long caches in a batch of many empty places."""
    torch, h = _torch(), _h()
    _say(f"attention padded, shares {dtype}")
    t, H, K, D, n, before, behind = _dt(dtype), 4, 1, 64, 3, 700, 2000
    T = before + n + behind
    gen = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(t)
    q = _nan(torch, T, H, D, dtype=t)
    q[before:before + n] = r(n, H, D)
    k, v = r(9000, K, D), r(9000, K, D)
    at = torch.arange(n + 1, device="cuda")
    keys = torch.tensor([0, 4000, 4001, 9000], device="cuda")
    assert _sizes(T, 9000, n, H, K, D, 1, dtype=dtype == "bf16")[0] > 0
    o, lse = h.hlq_attention_forward(q, k, v, at + before, keys, True, max_len=1,
                                     o=_nan(torch, T, H, D, dtype=t))
    want, wl = h.hlq_attention_forward(q[before:before + n].contiguous(), k, v, at, keys, True, max_len=1)
    mine = slice(before, before + n)
    # fewer shares may fit, whose sums are added up in another order: at most 64 shares, a
    # few roundings of 2^-24 each, and one of the type's in the output
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    top = float(v.abs().max())
    assert bool(((o[mine].double() - want.double()).abs() <= (2 * half + 9100 * 2.0 ** -24) * top).all())
    assert bool(((lse[:, mine] - wl).abs() <= 9100 * 2.0 ** -24).all())
    assert not o[:before].any() and not o[before + n:].any()
    rest = torch.cat([lse[:, :before], lse[:, before + n:]], 1)
    assert bool((rest == float("-inf")).all())
