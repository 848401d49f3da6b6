"""Host-side checks of the attention block's operators (no GPU, nothing is
launched): refusals of the C ABI and of the binding, workspace sizes, buckets."""
import ctypes
import os
import subprocess
import sys

import pytest

import hadamard_rank_linear_amd as h
import oracle.attention_oracle as o
from hadamard_rank_linear_amd.hlq import Attention, Tokens

P = 1 << 20          # a fake, aligned address: every call below must refuse before a launch
NAN, INF = float("nan"), float("inf")
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, VALUE = 1, 2, 6, 7, 9, 11


def _shape(**kw):
    a = dict(queries=64, keys=64, sequences=2, max_len=0, start_q=P, start_k=P, bias=P, scale=0.1,
             dtype=0, heads=4, kv_heads=2, head_dim=16, causal=1, bias_dtype=0, buckets=32,
             max_distance=128, bidirectional=0)
    a.update({k: v for k, v in kw.items() if k in a})
    return Attention(**a)


def _tokens(kw, name, heads, d=16):
    return Tokens(kw.get(name, P), kw.get(name + "_t", heads * d), kw.get(name + "_h", d))


def _forward(**kw):
    a = _shape(**kw)
    t = [_tokens(kw, n, a.kv_heads if n in "kv" else a.heads) for n in "qkvo"]
    return h.lib_handle().hlq_attention_forward(
        ctypes.byref(a) if kw.get("a", 1) else None,
        *(ctypes.byref(x) if kw.get(n + "_ref", 1) else None for n, x in zip("qkvo", t)),
        kw.get("lse", P), kw.get("ws", P), kw.get("bytes", 1 << 40), None)


def _backward(**kw):
    a = _shape(**kw)
    names = ("g_o", "q", "k", "v", "o", "g_q", "g_k", "g_v")
    t = {n: _tokens(kw, n, a.kv_heads if n[-1] in "kv" else a.heads) for n in names}
    r = {n: ctypes.byref(x) if kw.get(n + "_ref", 1) else None for n, x in t.items()}
    return h.lib_handle().hlq_attention_backward(
        ctypes.byref(a) if kw.get("a", 1) else None, *(r[n] for n in names[:5]), kw.get("lse", P),
        *(r[n] for n in names[5:]), kw.get("g_bias", P), kw.get("ws", P), kw.get("bytes", 1 << 40),
        None)


SHARED = [
    (dict(a=0), NULL), (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(o=None), NULL), (dict(lse=None), NULL), (dict(q_ref=0), NULL), (dict(o_ref=0), NULL),
    (dict(dtype=2), DTYPE), (dict(bias_dtype=-1), DTYPE),
    (dict(queries=-1), SHAPE), (dict(keys=-1), SHAPE), (dict(sequences=0), SHAPE),
    (dict(heads=0), SHAPE), (dict(kv_heads=0), SHAPE), (dict(kv_heads=3), SHAPE),
    (dict(head_dim=0), SHAPE), (dict(head_dim=129), SHAPE), (dict(max_len=-1), SHAPE),
    (dict(queries=1 << 28), SHAPE), (dict(keys=1 << 28), SHAPE), (dict(sequences=1 << 30), SHAPE),
    (dict(heads=1 << 16), SHAPE),
    (dict(start_q=None), SHAPE),                               # two sequences need their bounds
    (dict(start_q=None, sequences=1), SHAPE),                  # bounds of the keys alone
    (dict(start_k=None, keys=63), SHAPE),
    (dict(scale=0.0), VALUE), (dict(scale=-1.0), VALUE), (dict(scale=NAN), VALUE),
    (dict(scale=INF), VALUE), (dict(scale=2.0 ** -65), VALUE),
    (dict(buckets=1), VALUE), (dict(buckets=129), VALUE), (dict(buckets=0), VALUE),
    (dict(buckets=33, bidirectional=1), VALUE), (dict(buckets=2, bidirectional=1), VALUE),
    (dict(max_distance=16), VALUE), (dict(max_distance=1025), VALUE), (dict(max_distance=-5), VALUE),
    (dict(bias=P + 2), ALIGN), (dict(start_q=P + 4), ALIGN), (dict(start_k=P + 4), ALIGN),
    (dict(q=P + 2), ALIGN), (dict(v=P + 1, dtype=1), ALIGN), (dict(lse=P + 2), ALIGN),
    (dict(ws=P + 8), ALIGN), (dict(q_t=-1), SHAPE), (dict(k_h=1 << 40), SHAPE)]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(o=P + 2), ALIGN), (dict(o_h=15), SHAPE), (dict(o_t=63), SHAPE), (dict(o_t=0), SHAPE),
    (dict(o_h=0), SHAPE), (dict(o_t=16, o_h=1000), SHAPE),
    # two sequences of 4096 keys against one query each: the keys are shared out
    (dict(queries=2, keys=8192, ws=None), WORKSPACE), (dict(queries=2, keys=8192, bytes=64), WORKSPACE)])
def test_attention_forward_refuses(kw, status):
    assert _forward(**kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(g_o=None), NULL), (dict(g_q=None), NULL), (dict(g_k=None), NULL), (dict(g_v_ref=0), NULL),
    (dict(g_bias=None), NULL), (dict(bias=None), NULL),        # a gradient of no table
    (dict(g_bias=P + 2), ALIGN), (dict(g_v=P + 2), ALIGN), (dict(g_k_h=8), SHAPE),
    (dict(g_q_t=32), SHAPE), (dict(ws=None), WORKSPACE), (dict(bytes=1023), WORKSPACE)])
def test_attention_backward_refuses(kw, status):
    assert _backward(**kw) == status


@pytest.mark.parametrize("name", ["q", "k", "v", "g_o"])
def test_attention_refuses_tokens_too_far_apart(name):
    for far in (1 << 22, 1 << 40):
        assert _backward(**{name + "_t": far}) == SHAPE
        if name != "g_o":
            assert _forward(**{name + "_t": far}) == SHAPE
    # just near enough: the next thing to refuse is the workspace
    assert _backward(ws=None, **{name + "_t": (1 << 22) - 1}) == WORKSPACE


def test_attention_stride_of_a_single_token_or_head_is_not_looked_at():
    one = dict(queries=1, keys=1, sequences=1, start_k=None, ws=None)
    far = {n + "_t": 1 << 45 for n in ("g_o", "q", "k", "v", "o", "g_q", "g_k", "g_v")}
    assert _backward(**one, **far) == WORKSPACE
    far = {n + "_h": 1 << 45 for n in ("g_o", "q", "k", "v", "o", "g_q", "g_k", "g_v")}
    assert _backward(**{**one, "heads": 1, "kv_heads": 1}, **far) == WORKSPACE


def test_attention_workspace_sizes():
    fwd = lambda **kw: h.lib_handle().hlq_attention_forward_workspace_size(ctypes.byref(_shape(**kw)))
    bwd = lambda **kw: h.lib_handle().hlq_attention_backward_workspace_size(ctypes.byref(_shape(**kw)))
    assert fwd(head_dim=0) == 0 and bwd(dtype=5) == 0
    assert fwd(queries=1 << 16, keys=1 << 16, bias=None) == 0      # rows enough to fill the GPU
    # one share's sums, and its maximum and sum, for every query and head at least twice
    need = fwd(queries=2, keys=8192)
    assert need % (2 * 4 * (16 + 2) * 4) == 0 and need >= 2 * (2 * 4 * (16 + 2) * 4)
    assert bwd(bias=None) >= 64 * 4 * 4 and bwd() > bwd(bias=None)


@pytest.mark.parametrize("buckets,reach,both", [(32, 128, True), (32, 128, False), (16, 128, True),
                                                (2, 2, False), (4, 7, True), (128, 1024, True),
                                                (128, 1024, False), (5, 1000, False), (9, 5, False)])
def test_relative_bucket(buckets, reach, both):
    for d in list(range(-reach - 3, reach + 4)) + [-2 ** 31, 2 ** 31 - 1]:
        assert h.hlq_relative_bucket(d, buckets, reach, both) == o.bucket(d, buckets, reach, both)


@pytest.mark.parametrize("args", [(1, 128, False), (2, 128, True), (33, 128, True), (129, 128, False),
                                  (32, 8, True), (32, 1025, True), (-4, 10, False)])
def test_relative_bucket_refuses(args):
    with pytest.raises(ValueError):
        h.hlq_relative_bucket(1, *args)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), NULL), (dict(y=None), NULL), (dict(seed=None), NULL), (dict(dt=2), DTYPE),
    (dict(n=-1), SHAPE), (dict(n=1 << 35), SHAPE), (dict(p=-0.1), VALUE), (dict(p=1.1), VALUE),
    (dict(p=NAN), VALUE), (dict(x=P + 2), ALIGN), (dict(r=P + 1, dt=1), ALIGN),
    (dict(y=P + 2), ALIGN), (dict(seed=P + 4), ALIGN)])
def test_dropout_refuses(kw, status):
    a = dict(x=P, r=P, dt=0, n=9, p=0.1, seed=P, site=0, y=P)
    a.update(kw)
    lib = h.lib_handle()
    assert lib.hlq_dropout_forward(a["x"], a["r"], a["dt"], a["n"], a["p"], a["seed"], a["site"],
                                   a["y"], None) == status
    if "r" not in kw:
        assert lib.hlq_dropout_backward(a["x"], a["dt"], a["n"], a["p"], a["seed"], a["site"],
                                        a["y"], None) == status


def test_empty_calls_do_nothing():
    lib = h.lib_handle()
    assert lib.hlq_dropout_forward(None, None, 0, 0, 0.5, P, 0, None, None) == 0
    assert _forward(queries=0, keys=0, start_k=None, q=None, k=None, v=None, o=None, lse=None) == 0
    assert _backward(queries=0, keys=0, bias=None, g_bias=None, start_k=None, lse=None,
                     **{n: None for n in ("g_o", "q", "k", "v", "o", "g_q", "g_k", "g_v")}) == 0


def _cpu(*shape, dtype="float32"):
    import torch
    return torch.zeros(shape, dtype=getattr(torch, dtype))


@pytest.mark.parametrize("kw,error", [
    (dict(q=3), TypeError), (dict(q=(4, 8)), ValueError), (dict(k=(5, 8)), ValueError),
    (dict(), ValueError)])                                      # well formed, but on the CPU
def test_binding_refuses(kw, error):
    make = lambda s: _cpu(*s) if isinstance(s, tuple) else s
    q, k = make(kw.get("q", (4, 2, 8))), make(kw.get("k", (4, 1, 8)))
    with pytest.raises(error):
        h.hlq_attention_forward(q, k, k)


@pytest.mark.parametrize("kw,error", [
    (dict(p="x"), TypeError), (dict(site=-1), ValueError), (dict(site=1 << 32), ValueError),
    (dict(site=0.5), TypeError), (dict(seed=_cpu(2)), TypeError), (dict(seed=None), TypeError),
    (dict(seed=_cpu(3, dtype="int64")), ValueError), (dict(residual=_cpu(4)), ValueError),
    (dict(residual=_cpu(5, dtype="float64")), TypeError), (dict(), ValueError)])
def test_dropout_binding_refuses(kw, error):
    a = dict(p=0.1, seed=_cpu(2, dtype="int64"))
    a.update(kw)
    with pytest.raises(error):
        h.hlq_dropout_forward(_cpu(5), **a)


def test_one_hip_runtime_whatever_is_imported_first():
    """torch brings a HIP runtime of its own; the library loaded before it would bind
    another one, and no call would work in either."""
    code = ("import hadamard_rank_linear_amd as h; h.lib_handle(); import torch\n"
            "print(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "1", out
