"""The autograd forms of the training step's operators, and the tuning example
that runs them together with the HLQ linear layer."""
import math

import numpy as np
import pytest

import oracle.train_oracle as o

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"\n[gpu-case] {msg}", flush=True)


def _leaf(g, *shape, scale=1.0):
    import torch
    return (scale * torch.randn(shape, generator=g, device="cuda")).requires_grad_()


def _gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def _np(t):
    return t.detach().double().cpu().numpy()


def test_layer_norm_module_gradients():
    """Against the oracle: fp32, so a few parts in 10^6 of the largest value
    (sums of 100 terms of the same size)."""
    import torch
    from hadamard_rank_linear_amd.autograd import HLQLayerNorm
    _say("layer norm module")
    g = _gen(1)
    norm = HLQLayerNorm(100, device="cuda")
    with torch.no_grad():
        norm.weight.add_(0.1 * torch.randn(100, generator=g, device="cuda"))
    x, r = _leaf(g, 3, 7, 100), _leaf(g, 3, 7, 100)
    gy, gh = (torch.randn(3, 7, 100, generator=g, device="cuda") for _ in range(2))
    y, h = norm(x, r)
    torch.autograd.backward([y, h], [gy, gh])
    flat = lambda t: _np(t).reshape(21, 100)
    _, oh, om, orr = o.layer_norm_forward(flat(x), _np(norm.weight), _np(norm.bias), 1e-5, flat(r),
                                          o.round_f32)
    g_x, g_w, g_b = o.layer_norm_backward(flat(gy), oh, om, orr, _np(norm.weight), flat(gh))
    for got, want in ((flat(x.grad), g_x), (flat(r.grad), g_x), (_np(norm.weight.grad), g_w),
                      (_np(norm.bias.grad), g_b)):
        assert np.abs(got - want).max() <= 4e-6 * max(1.0, np.abs(want).max())


def test_layer_norm_partial_graphs():
    import torch
    from hadamard_rank_linear_amd.autograd import hlq_layer_norm
    _say("layer norm: one of the outputs unused, inputs of other layouts")
    g = _gen(2)
    x, r, w = _leaf(g, 8, 20), _leaf(g, 8, 20), _leaf(g, 20)
    y, h = hlq_layer_norm(x, w, residual=r)
    h.sum().backward()
    assert (x.grad == 1).all() and (r.grad == 1).all() and w.grad is None
    x.grad = r.grad = None
    y, h = hlq_layer_norm(x, w, residual=r)
    y.square().sum().backward()
    assert torch.equal(x.grad, r.grad) and w.grad is not None
    t = _leaf(g, 20, 8)
    y1 = hlq_layer_norm(t.t(), w)                     # a transposed view
    y2 = hlq_layer_norm(t.detach().t().contiguous(), w)
    assert torch.equal(y1, y2)
    y1.square().sum().backward()
    assert t.grad.shape == (20, 8) and torch.isfinite(t.grad).all()
    with pytest.raises(RuntimeError):                 # gradients of gradients are refused
        z = hlq_layer_norm(x, w)
        gx, = torch.autograd.grad(z.sum(), x, create_graph=True)
        gx.sum().backward()


@pytest.mark.parametrize("kl", [0.0, 0.05])
def test_policy_loss_through_log_probabilities_equals_the_fused_call(kl):
    """Two routes to the same gradient: they share every exponential, and
    differ by the rounding of the log probability (2^-24 of up to 12, which
    moves a gradient by 10^-6 of itself) and of the product with the upstream
    gradient."""
    import torch
    import hadamard_rank_linear_amd as h
    from hadamard_rank_linear_amd.autograd import hlq_policy_loss, hlq_token_logprob
    _say(f"policy loss, two routes, kl {kl}")
    g = _gen(3)
    logits = _leaf(g, 33, 515, scale=2.0)
    t = torch.randint(0, 515, (33,), generator=g, device="cuda")
    t[3] = -100
    base = h.hlq_token_logprob_forward(logits.detach(), t, 0.9)[0]
    old = base + 0.2 * torch.randn(33, generator=g, device="cuda")
    adv = torch.randn(33, generator=g, device="cuda")
    ref = base + 0.1 * torch.randn(33, generator=g, device="cuda") if kl else None
    w = (t >= 0).float() / 32
    sums, lp, g_x = h.hlq_policy_loss_logits(logits.detach(), t, old, adv, w, ref, scale=0.9,
                                             kl_coef=kl)
    loss, est, clipped = hlq_policy_loss(hlq_token_logprob(logits, t, 0.9), old, adv, w, ref,
                                         kl_coef=kl)
    (2.0 * loss).backward()
    assert torch.allclose(loss, sums[0], rtol=4e-6, atol=4e-6)
    assert torch.allclose(est, sums[1], rtol=1e-4, atol=1e-6) and torch.allclose(clipped, sums[2])
    assert torch.equal(lp, base)
    assert (logits.grad - 2.0 * g_x).abs().max() <= 8e-6 * g_x.abs().max()
    assert (logits.grad[3] == 0).all() and not est.requires_grad


def test_preference_loss_gradient_by_differences():
    """Central differences of the oracle's loss in 64 bits along the library's
    gradient: the slope is the gradient's squared length.  The gradient is
    fp32 (10^-5 covers its rounding over 60 rows), the step's truncation
    10^-6."""
    import torch
    from hadamard_rank_linear_amd.autograd import hlq_preference_loss, hlq_token_logprob
    _say("preference loss, directional difference")
    g = _gen(4)
    T, V = 60, 130
    logits = _leaf(g, T, V)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    start = torch.tensor([0, 10, 31, 44, T], device="cuda")
    w = (torch.rand(T, generator=g, device="cuda") > 0.2).float()
    ref = -5.0 + torch.randn(T, generator=g, device="cuda")
    loss, margin = hlq_preference_loss(hlq_token_logprob(logits, t), start, 0.3, ref, w, 0.1)
    loss.backward()
    grad, x, tn = _np(logits.grad), _np(logits), t.cpu().numpy()

    def f(step):
        lp = o.token_logprob(x + step * grad, tn)[0]
        return o.preference_loss(lp, start.tolist(), 0.3, _np(ref), _np(w), 0.1)[0]

    assert abs(loss.item() - f(0.0)) <= 1e-6 * max(1.0, abs(f(0.0)))
    step = 1e-3 / np.abs(grad).max()
    slope = (f(step) - f(-step)) / (2 * step)
    assert slope == pytest.approx((grad ** 2).sum(), rel=2e-5)


def test_clip_of_parameters():
    import torch
    from hadamard_rank_linear_amd.autograd import HLQLayerNorm, HLQLinear, hlq_clip_grad_norm_
    _say("clip parameters")
    m = torch.nn.Sequential(HLQLayerNorm(64, device="cuda"),
                            HLQLinear(64, 48, device="cuda", dtype=torch.float32))
    m[0].bias.grad = torch.full((64,), 3.0, device="cuda")
    m[1].weight.grad = torch.full((48, 64), 1.0, device="cuda")
    norm = hlq_clip_grad_norm_(m.parameters(), 1.0)
    want = math.sqrt(64 * 9.0 + 48 * 64)
    assert norm.item() == pytest.approx(want, rel=1e-12)
    assert torch.allclose(m[1].weight.grad, torch.tensor(1.0 / want, device="cuda"))
    assert m[0].weight.grad is None


def test_tuning_example_learns():
    from hadamard_rank_linear_amd import tuning_study as ts
    _say("tuning example")
    a, b = ts.tune_preferences(steps=12)
    assert abs(a) < 1e-6 and b > 0.2, (a, b)       # the first step is the reference itself
    c, d = ts.tune_policy(steps=16)
    assert abs(c - 0.5) < 0.1 and d > c + 0.15, (c, d)
