"""Attention outputs given in another operand's place: refused, and nothing is written."""
import pytest

from test_gpu_attention import _h, _say, _torch

pytestmark = pytest.mark.gpu


def test_outputs_in_operands_places():
    torch, h = _torch(), _h()
    _say("attention outputs in operands' places")
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, g = (torch.randn((40, 2, 32), generator=gen, device="cuda") for _ in range(4))
    keep = [t.clone() for t in (q, k, v, g)]
    for o in (k, v):
        with pytest.raises(h.HLQError):
            h.hlq_attention_forward(q, k, v, o=o)
    o, lse = h.hlq_attention_forward(q, k, v)
    one = torch.empty_like(q)
    for out in (dict(g_q=q), dict(g_q=g), dict(g_k=q), dict(g_v=g), dict(g_k=one, g_v=one),
                dict(g_q=one, g_k=one)):
        with pytest.raises(h.HLQError):
            h.hlq_attention_backward(g, q, k, v, o, lse, **out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(keep, (q, k, v, g)))
