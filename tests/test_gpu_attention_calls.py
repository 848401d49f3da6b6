"""Attention calls that the documentation allows and the other tests do not make: no bounds
with keys of another number, the farthest strides, tables of another type, hundreds of
heads on one, one workspace for two captured graphs."""
import pytest

from test_gpu_attention import Case, _check, _dt, _h, _say, _torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("queries,keys", [(5, 700), (700, 5), (3, 0), (1, 2000)])
@pytest.mark.parametrize("bias", [False, True])
def test_no_bounds_and_keys_of_another_number(dtype, queries, keys, bias):
    """As with the bounds of one sequence, bit for bit."""
    torch, h = _torch(), _h()
    _say(f"attention without bounds {queries} {keys} {dtype} bias {bias}")
    case = Case([queries], 4, 2, 40, dtype, True, klens=[keys], buckets=16 if bias else 0, reach=50)
    d, kw = case.device()
    g = torch.ones_like(d["q"])
    want = h.hlq_attention_forward(**d, **kw, max_len=queries)
    wg = h.hlq_attention_backward(g, *d.values(), *want, **kw, max_len=queries)
    kw.update(start=None, start_k=None)
    got = h.hlq_attention_forward(**d, **kw)
    gg = h.hlq_attention_backward(g, *d.values(), *got, **kw)
    same = lambda a, b: (a is None and b is None) or torch.equal(a, b)
    assert all(same(a, b) for a, b in zip(got, want))
    assert all(same(a, b) for a, b in zip(gg, wg))


@pytest.mark.parametrize("dtype,D", [("f32", 128), ("bf16", 128), ("f32", 64), ("bf16", 40)])
@pytest.mark.parametrize("less", [8, 1])
def test_farthest_tokens(dtype, D, less):
    """Tokens 2^22 elements apart but for 8, and for 1 (rows off a 16-byte boundary); heads
    further apart than all tokens."""
    torch, h = _torch(), _h()
    _say(f"attention of far tokens, D {D} {dtype} 2^22 - {less}")
    n, step = 300, (1 << 22) - less
    reach = n * step
    big = torch.empty(2 * reach + 4096, dtype=_dt(dtype), device="cuda")
    far = lambda heads, i: big.as_strided((n, heads, D), (step, reach, 1), i * 136)
    q, k, v, g, g_q, g_k, g_v, o = (far(heads, i) for i, heads in enumerate((2, 1, 1, 2, 2, 1, 1, 2)))
    gen = torch.Generator(device="cuda").manual_seed(9)
    dense = [torch.randn(t.shape, generator=gen, device="cuda").to(_dt(dtype)) for t in (q, k, v, g)]
    for f, x in zip((q, k, v, g), dense):
        f.copy_(x)
    start = torch.tensor([0, 100, n], device="cuda")
    a = h.hlq_attention_forward(q, k, v, start, causal=True, o=o)
    b = h.hlq_attention_forward(*dense[:3], start, causal=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    ga = h.hlq_attention_backward(g, q, k, v, *a, start, causal=True, g_q=g_q, g_k=g_k, g_v=g_v)
    gb = h.hlq_attention_backward(dense[3], *dense[:3], *b, start, causal=True)
    assert torch.equal(ga[0], gb[0])
    # heads that are too far apart for 32-bit offsets are not packed, which adds up the same
    # terms of the gradients of k and v, two heads of 200 rows at most, in another order
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    q, k, v, g = (t.double() for t in dense)
    for low, high in ((0, 100), (100, n)):
        rows = slice(low, high)
        tol_k = tol_v = 0.0
        for head in (0, 1):
            hidden = torch.ones((high - low,) * 2, dtype=torch.bool, device="cuda").triu(1)
            P = ((q[rows, head] @ k[rows, 0].T) * D ** -0.5).masked_fill(hidden, float("-inf")).softmax(-1)
            dp = g[rows, head] @ v[rows, 0].T
            # |G| with twice its parts covers what the types round off
            G = P * (dp.abs() + (P * dp).sum(-1, keepdim=True).abs() + 1.0)
            tol_k = tol_k + D ** -0.5 * G.T @ q[rows, head].abs()
            tol_v = tol_v + 1.02 * P.T @ g[rows, head].abs()
        for x, y, t in ((ga[1], gb[1], tol_k), (ga[2], gb[2], tol_v)):
            x, y = x[rows, 0].double(), y[rows, 0].double()
            assert bool(((x - y).abs() <= 2 * 401 * 2.0 ** -24 * t + half * (x.abs() + y.abs())).all())


@pytest.mark.parametrize("dtype,table", [("f32", "bf16"), ("bf16", "f32")])
def test_table_of_another_type(dtype, table):
    _say(f"attention {dtype}, table {table}")
    _check(Case([90, 40], 2, 2, 64, dtype, False, buckets=16, reach=30, table=table))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv", [(256, 1), (130, 2)])
def test_hundreds_of_heads(dtype, heads, kv):
    _say(f"attention of {heads} heads on {kv} {dtype}")
    _check(Case([3, 20], heads, kv, 16, dtype, True))


def test_one_workspace_for_two_graphs():
    """Two captured graphs that write the same workspace, replayed one after the other: each
    is done with it before the next."""
    torch, h = _torch(), _h()
    _say("attention graphs on one workspace")
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()
    at, keys = torch.arange(3, device="cuda"), torch.tensor([0, 3000, 4000], device="cuda")
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    sets = [(r(2, 8, 64), r(4000, 2, 64), r(4000, 2, 64)) for _ in range(2)]
    bias = torch.randn((8, 8), generator=gen, device="cuda")
    where = torch.tensor([0, 700, 4000], device="cuda")

    def run(s):
        o, lse = h.hlq_attention_forward(*s, at, keys, True, max_len=1, workspace=ws)
        big = s[1].repeat(1, 4, 1)
        p = h.hlq_attention_forward(big, s[1], s[2], where, bias=bias, max_distance=9)
        g = h.hlq_attention_backward(big, big, s[1], s[2], *p, where, bias=bias, max_distance=9, workspace=ws)
        return [o, lse, *p, *g]
    want = [[t.clone() for t in run(s)] for s in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run(s))
        graphs.append(graph)
    for rep in range(3):
        for out in outs:
            for t in out:
                t.fill_(float("nan"))
        ws.fill_(255)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for out, ref in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, ref)), rep


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
def test_bounds_beyond_the_tokens(dtype, bias):
    """They are limited to the tokens there are."""
    torch, h = _torch(), _h()
    _say(f"attention, bounds beyond the tokens, {dtype} bias {bias}")
    case = Case([90], 4, 2, 40, dtype, True, buckets=16 if bias else 0, reach=50)
    d, kw = case.device()
    g = torch.ones_like(d["q"])
    far, near = [-(1 << 62), -3, 20, 80, 91, 1 << 40, 2 ** 63 - 1], [0, 0, 20, 80, 90, 90, 90]
    got = []
    for at in (far, near):
        kw["start"] = torch.tensor(at, device="cuda")
        o, lse = h.hlq_attention_forward(**d, **kw)
        got.append((o, lse, *h.hlq_attention_backward(g, *d.values(), o, lse, **kw)))
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("table", ["f32", "bf16"])
def test_lowest_values_hide_a_bucket(dtype, table):
    """A table that masks with its type's lowest value: as with -inf, bit for bit; bucket 0 of
    one head, every bucket of another."""
    torch, h = _torch(), _h()
    _say(f"attention, lowest values in a table, {dtype} {table}")
    case = Case([70, 5], 3, 3, 32, dtype, True, buckets=16, reach=40, table=table)
    d, kw = case.device()
    g = torch.ones_like(d["q"])
    got = []
    for low in (float("-inf"), torch.finfo(_dt(table)).min):
        kw["bias"][0, 0] = low
        kw["bias"][:, 1] = low
        o, lse = h.hlq_attention_forward(**d, **kw)
        got.append((o, lse, *h.hlq_attention_backward(g, *d.values(), o, lse, **kw)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert not got[1][0][:, 1].any() and bool((got[1][1][1] == float("-inf")).all())
