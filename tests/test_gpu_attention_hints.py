"""Attention's results where the expected length is wrong, or right for few of the
sequences: rows beyond it are looped over, with shares of the keys too."""
import pytest

from test_attention_sizes import _sizes
from test_gpu_attention import Case, _check, _h, _say, _torch
from test_gpu_attention_tiles import _tiles

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
def test_shares_of_more_queries_than_expected(dtype, causal):
    _say(f"attention hint of 1 for 300 queries, shares, {dtype} causal {causal}")
    assert _sizes(302, 1330, 2, 2, 1, 32, 1, dtype=dtype == "bf16", causal=causal)[0] > 0
    _check(Case([300, 2], 2, 1, 32, dtype, causal, klens=[1300, 30]), max_len=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_sequence_without_bounds(dtype):
    """The hint is not looked at: the same launches, bit for bit."""
    torch, h = _torch(), _h()
    _say(f"attention hint without bounds {dtype}")
    case = Case([700], 4, 2, 64, dtype, True)
    d, kw = case.device()
    kw.update(start=None)
    want, lse = h.hlq_attention_forward(**d, **kw)
    grads = h.hlq_attention_backward(want, *d.values(), want, lse, **kw)
    for max_len in (1, 33, 1 << 30):
        got = h.hlq_attention_forward(**d, **kw, max_len=max_len)
        again = h.hlq_attention_backward(want, *d.values(), want, lse, **kw, max_len=max_len)
        assert torch.equal(got[0], want) and torch.equal(got[1], lse)
        assert all(torch.equal(a, b) for a, b in zip(again[:3], grads[:3]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
def test_one_long_sequence_among_many(dtype, bias):
    """Its 18 tiles are more than the launch has: one workgroup takes two."""
    _say(f"attention, one long sequence of 200, {dtype} bias {bias}")
    lens = [2300] + [0, 1] * 3 + [0] * 193
    assert _tiles(sum(lens), len(lens), 3, 2300, dtype, 8, not bias) == 17
    _check(Case(lens, 3, 3, 8, dtype, not bias, buckets=16 if bias else 0), max_len=2300)
