"""Outputs that the caller supplies (in place of the logits, clipped gradients,
given buffers): autograd sees that they were written."""
import pytest

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"\n[gpu-case] {msg}", flush=True)


def test_every_supplied_output_counts_a_write():
    import torch
    import hadamard_rank_linear_amd as h
    _say("version counters of supplied outputs")
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, w, t = r(6, 40), r(40), torch.arange(6, device="cuda")
    buf = {k: torch.empty_like(x) for k in ("y", "h", "a", "b", "c", "d")}
    _, hh, mean, rstd = h.hlq_layer_norm_forward(x, w, residual=x, y=buf["y"], h=buf["h"])
    h.hlq_layer_norm_backward(x, hh, mean, rstd, w, g_x=buf["a"])
    lp, stats = h.hlq_token_logprob_forward(x, t)
    h.hlq_token_logprob_backward(lp, x, t, stats, g_x=buf["b"])
    h.hlq_policy_loss_logits(x, t, lp, lp, g_x=buf["c"])
    h.hlq_clip_grad_norm([x], 1.0, out=[buf["d"]])
    assert {k: v._version for k, v in buf.items()} == dict.fromkeys(buf, 1)
    assert x._version == w._version == t._version == 0 and lp._version == stats._version == 0
    h.hlq_clip_grad_norm([x, w], 1.0)
    assert x._version == w._version == 1
    with pytest.raises(h.HLQError):            # a refused call has written nothing
        h.hlq_token_logprob_backward(lp, x, t, stats, 0.0, g_x=buf["b"])
    assert buf["b"]._version == 1
    with torch.inference_mode():               # tensors without a counter
        z = torch.empty(6, 40, device="cuda")
    h.hlq_token_logprob_backward(lp, x, t, stats, g_x=z)
    assert torch.equal(z, h.hlq_token_logprob_backward(lp, x, t, stats))


@pytest.mark.parametrize("fused", [False, True])
def test_a_gradient_in_place_of_saved_logits_is_noticed(fused):
    import torch
    import hadamard_rank_linear_amd as h
    from hadamard_rank_linear_amd.autograd import hlq_token_logprob
    _say(f"backward of logits that a gradient has replaced, fused {fused}")
    x = torch.randn(5, 33, device="cuda", requires_grad=True)
    t = torch.arange(5, device="cuda")
    logits = 2.0 * x
    lp = hlq_token_logprob(logits, t)
    flat = logits.detach()
    if fused:
        h.hlq_policy_loss_logits(flat, t, lp.detach(), torch.ones(5, device="cuda"), g_x=flat)
    else:
        stats = h.hlq_token_logprob_forward(flat, t)[1]
        h.hlq_token_logprob_backward(lp.detach(), flat, t, stats, g_x=flat)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        lp.sum().backward()
