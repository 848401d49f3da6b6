"""Column sums of the norm's backward pass over small integers: every sum is
exact in fp32, so a row that is lost, doubled or given to a wrong column shows
in the result, however many rows there are."""
import pytest

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"\n[gpu-case] {msg}", flush=True)


def _integers(T, C, dtype, seed, low, high):
    """Integers from low to high - 1 without zero."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(low, high, (T, C), generator=g, device="cuda", dtype=torch.int8)
    return v.masked_fill_(v == 0, 1).to(dtype)


def _sums(g_y, h):
    """(sum_t g_y h, sum_t g_y), a few rows at a time."""
    import torch
    w, b = (torch.zeros(g_y.shape[1], dtype=torch.float64, device="cuda") for _ in range(2))
    step = max(1, (1 << 25) // g_y.shape[1])
    for a in range(0, len(g_y), step):
        p, q = g_y[a:a + step].double(), h[a:a + step].double()
        w += (p * q).sum(0)
        b += p.sum(0)
    return w, b


def _check(T, C, dtype, seed):
    import torch
    import hadamard_rank_linear_amd as h
    # at most 3 * 3 * T: below 2^24, so no partial sum is rounded
    assert 9 * T < 1 << 24
    g_y, x = _integers(T, C, dtype, seed, 1, 4), _integers(T, C, dtype, seed + 1, -3, 4)
    zero, one = torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
    w, b = _sums(g_y, x)
    for with_bias in (True, False):
        _, g_w, g_b = h.hlq_layer_norm_backward(g_y, x, zero, one, torch.ones(C, device="cuda"),
                                                with_bias=with_bias)
        torch.cuda.synchronize()
        assert torch.equal(g_w.double(), w)
        assert g_b is None if not with_bias else torch.equal(g_b.double(), b)


@pytest.mark.parametrize("name", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,C", [(300001, 3), (70001, 9), (40007, 8), (33000, 33), (9000, 200),
                                 (6000, 600), (5001, 1000), (4500, 1030), (2100, 2050),
                                 (1501, 4099), (1030, 8200), (700, 16384), (515, 17001),
                                 (1000003, 16), (9001, 768)])
def test_column_sums_of_many_rows(T, C, name):
    import torch
    _say(f"column sums T={T} C={C} {name}")
    _check(T, C, getattr(torch, name), T + C)


def test_column_sums_of_more_columns_than_one_fold_takes():
    # 2^24 columns a launch of the fold; 33 rows leave two partials to fold
    import torch
    C = (1 << 24) + 1003
    _say(f"column sums T=33 C={C}")
    import hadamard_rank_linear_amd as h
    assert h.hlq_layer_norm_backward_workspace_size(33, C, h.HLQ_BF16) == 2 * 2 * 4 * C
    _check(33, C, torch.bfloat16, 5)
