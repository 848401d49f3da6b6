"""Refusals of the autograd forms of attention (no GPU, nothing is launched)."""
import pytest
import torch

from hadamard_rank_linear_amd.autograd import hlq_attention, hlq_packed_attention


@pytest.mark.parametrize("shape,heads", [((), 1), ((4,), 1), ((4, 3), 1), ((2, 4, 3, 8), 1), ((4, 3, 8), 0),
                                         ((4, 3, 8), -1), ((4, 3, 8), 3), ((4, 4, 8), 1)])
def test_packed_attention_refuses(shape, heads):
    with pytest.raises(ValueError):
        hlq_packed_attention(torch.zeros(shape), heads)


@pytest.mark.parametrize("shape", [(), (4,), (4, 3)])
def test_attention_refuses(shape):
    x = torch.zeros(shape)
    with pytest.raises(ValueError):
        hlq_attention(x, x, x)
