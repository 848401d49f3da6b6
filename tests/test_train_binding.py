"""The binding's conversion of arguments that are no tensors (no GPU: the calls
end before their tensors are looked at)."""
import pytest

import hadamard_rank_linear_amd as h


@pytest.mark.parametrize("wrong", [1 << 32, -(1 << 32), (1 << 32) + 1, 1 << 80])
def test_integers_out_of_range_are_refused(wrong):
    # their low 32 bits are those of a valid code
    import torch
    v, start = torch.zeros(4), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="reduction is out of range"):
        h.hlq_preference_loss(v, start, 0.1, reduction=wrong)
    with pytest.raises(ValueError, match="norm_kind is out of range"):
        h.hlq_clip_grad_norm([v], 1.0, wrong)


def test_a_flag_without_a_truth_value_is_refused():
    import torch
    x, v, w = torch.zeros(4, 8), torch.zeros(4), torch.zeros(8)
    with pytest.raises(RuntimeError, match="ambiguous"):
        h.hlq_layer_norm_backward(x, x, v, v, w, with_bias=torch.ones(2))
