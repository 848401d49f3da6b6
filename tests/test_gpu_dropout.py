"""Dropout with the residual addition on the GPU against its definition
(oracle/attention_oracle.py).  The mask has to be the generator's bit for bit; a
kept value is a product and a sum, each off by 2^-24 of its own size at most,
rounded once to the type (2^-8 relative for bf16); the factor 65536 / (65536 - t)
is rounded to fp32 (2^-24)."""
import numpy as np
import pytest

import oracle.attention_oracle as o
from oracle.train_oracle import round_bf16, round_f32

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}


def _say(msg):
    print(f"\n[gpu-case] {msg}", flush=True)


def _torch():
    import torch
    return torch


def _h():
    import hadamard_rank_linear_amd as h
    return h


def _dev(v, dtype, offset=0):
    """v on the GPU, ``offset`` elements into a storage of NaN."""
    torch = _torch()
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    buf = torch.full((len(v) + offset + 16,), float("nan"), dtype=t, device="cuda")
    out = buf[offset:offset + len(v)]
    return out.copy_(torch.as_tensor(v))


def _seed(key, step):
    return _torch().tensor([key, step], device="cuda")


def _np(t):
    return t.detach().double().cpu().numpy()


def _check(got, x, r, p, seed, site, dtype, first=0):
    want, kept = o.dropout(x, p, seed, site, r, first)
    tol = 4 * U * (np.abs(want) + (0 if r is None else np.abs(r))) + HALF[dtype] * np.abs(want)
    assert (np.abs(_np(got) - want) <= tol).all()
    if r is None:
        assert ((_np(got) != 0) == (kept & (x != 0))).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 3, 7, 8, 9, 63, 1000, 2048, 4099])
@pytest.mark.parametrize("residual", [False, True])
def test_sizes(dtype, n, residual):
    _say(f"dropout {n} {dtype} residual {residual}")
    h = _h()
    rng = np.random.default_rng(n)
    rnd = round_bf16 if dtype == "bf16" else round_f32
    x, r = rnd(rng.normal(size=n)), rnd(rng.normal(size=n)) if residual else None
    for offset in (0, 1):
        y = h.hlq_dropout_forward(_dev(x, dtype, offset), 0.3, _seed(77, n), site=5,
                                  residual=None if r is None else _dev(r, dtype, 3))
        _check(y, x, r, 0.3, (77, n), 5, dtype)


@pytest.mark.parametrize("p", [0.0, 2.0 ** -17, 2.0 ** -16, 0.1, 0.5, 1 - 2.0 ** -16, 1.0])
def test_probabilities(p):
    """2^-17 is a tie and goes to 0, the even one; 1 leaves the residual alone."""
    _say(f"dropout p {p}")
    h = _h()
    x = np.random.default_rng(1).normal(size=3001).astype(np.float32).astype(np.float64)
    _check(h.hlq_dropout_forward(_dev(x, "f32"), p, _seed(1, 2)), x, None, p, (1, 2), 0, "f32")
    y = h.hlq_dropout_forward(_dev(x, "f32"), p, _seed(1, 2), residual=_dev(x, "f32"))
    _check(y, x, x, p, (1, 2), 0, "f32")


@pytest.mark.parametrize("key,step,site", [(0, 0, 0), (-1, -1, 2 ** 32 - 1), (2 ** 62 + 5, 2 ** 40, 9),
                                           (-2 ** 63, 2 ** 63 - 1, 1)])
def test_keys_steps_and_sites(key, step, site):
    _say(f"dropout key {key} step {step} site {site}")
    x = np.ones(999)
    y = _h().hlq_dropout_forward(_dev(x, "f32"), 0.5, _seed(key, step), site=site)
    low = 2 ** 64 - 1
    _check(y, x, None, 0.5, (key & low, step & low), site, "f32")


def test_backward_draws_the_same_mask():
    torch, h = _torch(), _h()
    _say("dropout backward")
    x = torch.randn(20, 333, device="cuda") + 10.0
    seed = _seed(3, 4)
    y = h.hlq_dropout_forward(x, 0.2, seed, site=1)
    g = torch.ones_like(x)
    g_x = h.hlq_dropout_backward(g, 0.2, seed, site=1)
    assert torch.equal(g_x != 0, y != 0) and torch.equal(g_x * x, y)
    assert not torch.equal(h.hlq_dropout_backward(g, 0.2, seed, site=2) != 0, y != 0)
    seed[1] += 1
    assert not torch.equal(h.hlq_dropout_forward(x, 0.2, seed, site=1) != 0, y != 0)


def test_share_of_the_kept():
    """10^7 elements at p = 0.1 (t = 6554): the share kept is within five standard
    deviations, 5 sqrt(p (1 - p) / n) = 4.8e-4."""
    torch, h = _torch(), _h()
    _say("dropout share")
    x = torch.ones(10_000_000, dtype=torch.bfloat16, device="cuda")
    kept = (h.hlq_dropout_forward(x, 0.1, _seed(11, 0)) != 0).double().mean().item()
    assert abs(kept - (1 - 6554 / 65536)) < 4.8e-4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_dropped_values_do_not_matter(dtype):
    torch, h = _torch(), _h()
    _say(f"dropout of NaN {dtype}")
    kept = o.dropout(np.ones(500), 0.5, (8, 9), 0)[1]
    x = np.where(kept, 1.0, np.nan)
    x[kept.argmax()] = np.inf
    y = _np(h.hlq_dropout_forward(_dev(x, dtype), 0.5, _seed(8, 9)))
    assert (y[~kept] == 0).all() and y[kept.argmax()] == np.inf and (y[kept][1:] == 2).all()


def test_in_place():
    """The output in the place of x, of the residual, and of the gradient; rows
    that do not start at 16 bytes."""
    torch, h = _torch(), _h()
    _say("dropout in place")
    for n, offset in ((1001, 0), (1001, 1)):
        base = torch.randn(n, device="cuda").bfloat16()
        make = lambda: _dev(base.float().cpu(), "bf16", offset)
        want = h.hlq_dropout_forward(make(), 0.3, _seed(1, 1), residual=make())
        x, r = make(), make()
        assert h.hlq_dropout_forward(x, 0.3, _seed(1, 1), residual=r, y=x).data_ptr() == x.data_ptr()
        assert torch.equal(x, want) and torch.equal(r, base)
        x = make()
        h.hlq_dropout_forward(x, 0.3, _seed(1, 1), residual=r, y=r)
        assert torch.equal(r, want) and torch.equal(x, base)
        g = make()
        want = h.hlq_dropout_backward(g, 0.3, _seed(1, 1))
        h.hlq_dropout_backward(g, 0.3, _seed(1, 1), g_x=g)
        assert torch.equal(g, want)


def test_elements_past_32_bits():
    """2^32 + 20 elements: the last ones' block is 2^29 and above."""
    torch, h = _torch(), _h()
    _say("dropout past 2^32")
    n = (1 << 32) + 20
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    x[-40:] = 1.0
    y = h.hlq_dropout_forward(x, 0.5, _seed(4, 5), site=6, y=x)[-40:]
    want, _ = o.dropout(np.ones(40), 0.5, (4, 5), 6, first=n - 40)
    assert (_np(y) == want).all()


def test_refusals_on_the_gpu():
    torch, h = _torch(), _h()
    _say("dropout refusals")
    x, s = torch.zeros(8, 4, device="cuda"), _seed(1, 2)
    for kw, error in [(dict(p=1.5), h.HLQError), (dict(p=float("nan")), h.HLQError),
                      (dict(seed=s.cpu()), ValueError), (dict(seed=s.int()), TypeError),
                      (dict(residual=x[:4]), ValueError), (dict(residual=x.bfloat16()), TypeError),
                      (dict(x=x.t()), ValueError), (dict(x=x.double()), TypeError),
                      (dict(y=x.t().contiguous()), ValueError), (dict(stream=1), TypeError)]:
        a = dict(x=x, p=0.5, seed=s)
        a.update(kw)
        with pytest.raises(error):
            h.hlq_dropout_forward(**a)
    assert h.hlq_dropout_forward(x[:0], 0.5, s).shape == (0, 4)
    torch.cuda.synchronize()
