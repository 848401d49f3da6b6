"""Attention outputs in another operand's place: no GPU, nothing is launched."""
import ctypes

import pytest

import hadamard_rank_linear_amd as h
from hadamard_rank_linear_amd.hlq import Attention, Tokens

VALUE = 11
BACKWARD = ("g_o", "q", "k", "v", "o", "g_q", "g_k", "g_v")


def _operands(names, same, **kw):
    """A call's shape and tensors at addresses of their own, but one at another's."""
    at = {n: (i + 1) << 24 for i, n in enumerate(BACKWARD)}
    at[same[0]] = at[same[1]]
    a = Attention(**{**dict(queries=64, keys=64, sequences=1, scale=0.1, dtype=0, heads=2, kv_heads=2,
                            head_dim=16), **kw})
    return a, [ctypes.byref(Tokens(at[n], 32, 16)) for n in names]


@pytest.mark.parametrize("same", [("o", "k"), ("o", "v")])
def test_forward_refuses(same):
    a, t = _operands(("q", "k", "v", "o"), same)
    assert h.lib_handle().hlq_attention_forward(ctypes.byref(a), *t, 1 << 20, 1 << 20, 1 << 40,
                                                None) == VALUE


@pytest.mark.parametrize("same", [
    ("g_q", "q"), ("g_q", "g_o"), ("g_q", "k"), ("g_q", "v"), ("g_q", "g_k"), ("g_q", "g_v"),
    ("g_k", "q"), ("g_k", "g_o"), ("g_k", "g_v"), ("g_v", "q"), ("g_v", "g_o")])
def test_backward_refuses(same):
    a, t = _operands(BACKWARD, same)
    assert h.lib_handle().hlq_attention_backward(ctypes.byref(a), *t[:5], 1 << 20, *t[5:], None,
                                                 1 << 20, 1 << 40, None) == VALUE


def test_tensors_without_tokens_have_no_place():
    """Nothing to launch, whatever their addresses."""
    a, t = _operands(BACKWARD, ("g_k", "g_v"), queries=0, keys=0)
    assert h.lib_handle().hlq_attention_backward(ctypes.byref(a), *t[:5], None, *t[5:], None, None, 0,
                                                 None) == 0
