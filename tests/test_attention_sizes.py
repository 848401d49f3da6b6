"""Workspaces of attention against the length that the caller expects (no GPU, nothing
is launched): a hint that is wrong, or right for few of the sequences, makes a launch
slower, and must not ask for more memory than the tensors themselves."""
import ctypes

import numpy as np
import pytest

import hadamard_rank_linear_amd as h
from hadamard_rank_linear_amd.hlq import Attention

P = 1 << 20


def _sizes(queries, keys, sequences, heads, kv_heads, D, max_len, buckets=0, dtype=1, bounds=True,
           causal=1):
    own = P if bounds and keys != queries else None
    a = Attention(queries=queries, keys=keys, sequences=sequences, max_len=max_len,
                  start_q=P if bounds else None, start_k=own, bias=P if buckets else None, scale=0.1,
                  dtype=dtype, heads=heads, kv_heads=kv_heads, head_dim=D, causal=causal,
                  bias_dtype=0, buckets=buckets, max_distance=128, bidirectional=0)
    lib = h.lib_handle()
    return (lib.hlq_attention_forward_workspace_size(ctypes.byref(a)),
            lib.hlq_attention_backward_workspace_size(ctypes.byref(a)))


@pytest.mark.parametrize("tokens", [8192, 65536])
def test_a_sequence_without_bounds_is_as_long_as_it_is(tokens):
    for max_len in (0, 1, 33, tokens, 1 << 40):
        assert _sizes(tokens, tokens, 1, 32, 8, 128, max_len, bounds=False) == \
            _sizes(tokens, tokens, 1, 32, 8, 128, 0, bounds=False)
        assert _sizes(tokens, tokens, 1, 32, 8, 128, max_len, bounds=False)[0] == 0


def test_a_hint_that_is_too_short_asks_for_little():
    """At most 2^18 rows of D + 2 floats; one sequence of 65536 tokens took 70 GB."""
    assert _sizes(65536, 65536, 1, 32, 8, 128, 1)[0] <= (1 << 18) * 130 * 4
    rng = np.random.default_rng(1)
    for _ in range(2000):
        S, kv = int(2 ** rng.uniform(0, 12)), int(2 ** rng.integers(0, 5))
        heads, D = kv * int(2 ** rng.integers(0, 4)), int(rng.integers(1, 129))
        queries, keys = (S * int(2 ** rng.uniform(0, 10)) for _ in range(2))
        if max(queries, keys) * heads >= 1 << 30:
            continue
        size, _ = _sizes(queries, keys, S, heads, kv, D, int(2 ** rng.uniform(0, 8)))
        assert size <= (1 << 18) * (D + 2) * 4


@pytest.mark.parametrize("queries,keys,S,heads,kv,shares", [
    (8, 32700, 8, 32, 8, 16), (1, 65536, 1, 32, 8, 64), (4, 65536, 4, 8, 1, 64), (2, 8192, 2, 4, 2, 32)])
def test_a_true_hint_keeps_its_shares(queries, keys, S, heads, kv, shares):
    assert _sizes(queries, keys, S, heads, kv, 128, 1)[0] == shares * queries * heads * 130 * 4


def test_a_hint_for_one_of_many_sequences():
    """With a bias a line of buckets for each tile and head: at most 16 times as many as
    tiles of 32 there can be."""
    rng = np.random.default_rng(2)
    for _ in range(2000):
        S, heads = int(2 ** rng.uniform(0, 16)), int(rng.integers(1, 17))
        queries = S * int(2 ** rng.uniform(0, 8))
        if queries * heads >= 1 << 30:
            continue
        hint = int(2 ** rng.uniform(0, 41))
        _, size = _sizes(queries, queries, S, heads, heads, 64, hint, buckets=32)
        lines = (size - (queries * heads * 4 + 15) // 16 * 16) / (32 * 4)
        assert lines <= 16 * (queries / 32 + S) * heads
    # 2^20 tokens in 2^16 sequences, one of them long: 137 GB
    assert _sizes(1 << 20, 1 << 20, 1 << 16, 16, 16, 64, 1 << 20, buckets=32)[1] < 3e9


@pytest.mark.parametrize("queries,S,heads,hint,tiles", [
    (12608, 64, 12, 197, 2), (8192, 16, 12, 512, 4), (8190, 16, 12, 0, 8), (65536, 8, 16, 30000, 235),
    (65536, 1, 16, 0, 512)])
def test_a_true_hint_keeps_its_tiles(queries, S, heads, hint, tiles):
    _, size = _sizes(queries, queries, S, heads, heads, 64, hint, buckets=32, causal=0)
    assert size == queries * heads * 4 + tiles * S * heads * 32 * 4
