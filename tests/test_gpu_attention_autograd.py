"""The attention block's operators as a program uses them: autograd forms against
differences and against the calls they make, a block that runs them together with
the HLQ linear layer and the layer norm, other streams, and captured graphs."""
import numpy as np
import pytest

import oracle.attention_oracle as o

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _say(msg):
    print(f"\n[gpu-case] {msg}", flush=True)


def _gen(seed):
    return _torch().Generator(device="cuda").manual_seed(seed)


def _leaf(g, *shape, scale=1.0):
    torch = _torch()
    return (scale * torch.randn(shape, generator=g, device="cuda")).requires_grad_()


def _np(t):
    return t.detach().double().cpu().numpy()


def test_gradients_by_differences():
    """Central differences of the oracle's loss in 64 bits along the library's
    gradient: the slope is the gradient's squared length.  The gradient is fp32,
    its o rounded to fp32 (10^-5 covers the sums over 40 keys), the step's
    truncation 10^-6."""
    torch = _torch()
    from hadamard_rank_linear_amd.autograd import hlq_attention
    _say("attention, directional difference")
    g = _gen(1)
    q, k, v = _leaf(g, 40, 4, 24), _leaf(g, 40, 2, 24), _leaf(g, 40, 2, 24)
    bias = _leaf(g, 8, 4)
    start = torch.tensor([0, 11, 40], device="cuda")
    g_o = torch.randn((40, 4, 24), generator=g, device="cuda")
    out = hlq_attention(q, k, v, start, causal=False, scale=0.2, bias=bias, max_distance=9)
    out.backward(g_o)
    x = [_np(t) for t in (q, k, v, bias)]
    grad = [_np(t.grad) for t in (q, k, v, bias)]
    go = _np(g_o)

    def loss(step):
        a, b, c, t = (p + step * d for p, d in zip(x, grad))
        total = 0.0
        for s0, s1 in ((0, 11), (11, 40)):
            which = o.bucket_table(s1 - s0, s1 - s0, 8, 9, True)
            for h in range(4):
                y, _ = o.forward(a[s0:s1, h], b[s0:s1, h // 2], c[s0:s1, h // 2], 0.2, False, t[:, h], which)
                total += (y * go[s0:s1, h]).sum()
        return total

    step = 1e-4 / max(np.abs(d).max() for d in grad)
    slope = (loss(step) - loss(-step)) / (2 * step)
    assert slope == pytest.approx(sum((d ** 2).sum() for d in grad), rel=2e-5)


def test_packed_form_equals_the_slices():
    torch = _torch()
    from hadamard_rank_linear_amd.autograd import hlq_attention, hlq_packed_attention
    _say("packed attention")
    g = _gen(2)
    a = _leaf(g, 70, 8, 32)
    b = a.detach().clone().requires_grad_()
    start = torch.tensor([0, 30, 70], device="cuda")
    g_o = torch.randn((70, 4, 32), generator=g, device="cuda")
    y = hlq_packed_attention(a, 4, start, causal=True)
    z = hlq_attention(*b.split((4, 2, 2), 1), start, causal=True)
    y.backward(g_o)
    z.backward(g_o)
    assert torch.equal(y, z) and torch.equal(a.grad, b.grad)
    with pytest.raises(ValueError):
        hlq_packed_attention(a, 5, start)
    # upstream gradients of other layouts: expanded, transposed
    for make in (lambda: y2.sum(), lambda: (y2.transpose(1, 2) * w).sum()):
        c = a.detach().clone().requires_grad_()
        w = torch.randn((70, 32, 4), generator=g, device="cuda")
        y2 = hlq_packed_attention(c, 4, start, causal=True)
        make().backward()
        assert torch.isfinite(c.grad).all()
    with pytest.raises(RuntimeError):                 # gradients of gradients are refused
        c = a.detach().clone().requires_grad_()
        gx, = torch.autograd.grad(hlq_packed_attention(c, 4).sum(), c, create_graph=True)
        gx.sum().backward()


def test_other_layouts_of_leaves():
    torch = _torch()
    from hadamard_rank_linear_amd.autograd import hlq_attention
    _say("attention of transposed leaves")
    g = _gen(3)
    q, k, v = (_leaf(g, 32, 2, 33) for _ in range(3))
    turn = lambda t: t.permute(2, 1, 0)
    y = hlq_attention(turn(q), turn(k), turn(v), causal=True)
    want = hlq_attention(*(turn(t).detach().contiguous() for t in (q, k, v)), causal=True)
    assert torch.equal(y, want)
    y.square().sum().backward()
    assert all(t.grad.shape == (32, 2, 33) and torch.isfinite(t.grad).all() for t in (q, k, v))


def test_dropout_form():
    torch = _torch()
    import hadamard_rank_linear_amd as h
    from hadamard_rank_linear_amd.autograd import HLQDropout, hlq_dropout
    _say("dropout form")
    g = _gen(4)
    x, r = _leaf(g, 30, 50), _leaf(g, 30, 50)
    seed = torch.tensor([5, 6], device="cuda")
    y = hlq_dropout(x, 0.25, seed, 7, r)
    g_y = torch.randn((30, 50), generator=g, device="cuda")
    y.backward(g_y)
    assert torch.equal(r.grad, g_y)
    assert torch.equal(x.grad, h.hlq_dropout_backward(g_y, 0.25, seed, 7))
    layer = HLQDropout(0.5, site=3)
    assert torch.equal(layer(x, seed), h.hlq_dropout_forward(x.detach(), 0.5, seed, 3))
    layer.eval()
    assert layer(x, seed) is x and torch.equal(layer(x, seed, r), r + x)
    # a seed that has moved on before the backward pass raises instead of another mask
    y = hlq_dropout(x, 0.25, seed, 7)
    seed[1] += 1
    with pytest.raises(RuntimeError):
        y.sum().backward()


def _block(dtype, seed=0):
    torch = _torch()
    from hadamard_rank_linear_amd.autograd import HLQDropout, HLQLayerNorm, HLQSelfAttention
    torch.manual_seed(seed)

    class Block(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.norm = HLQLayerNorm(64, device="cuda")
            self.attention = HLQSelfAttention(64, 4, 2, causal=True, buckets=8, max_distance=16,
                                              device="cuda", dtype=dtype)
            self.drop = HLQDropout(0.1, site=2)
            self.last = HLQLayerNorm(64, device="cuda")

        def forward(self, x, seed, start):
            x = self.drop(self.attention(self.norm(x), start, max_len=40), seed, residual=x)
            return self.last(x)

    block = Block()
    with torch.no_grad():
        block.attention.bias.normal_()
    return block


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_a_block_of_them(dtype):
    """Norm, qkv layer, attention with bias, output layer, dropout with the residual
    addition, norm: the same numbers as the calls one by one, gradients in every
    parameter, bit for bit again."""
    torch = _torch()
    import hadamard_rank_linear_amd as h
    _say(f"a block {dtype}")
    t = getattr(torch, dtype)
    block, g = _block(t), _gen(5)
    x = torch.randn((64, 64), generator=g, device="cuda").to(t)
    start, seed = torch.tensor([0, 24, 64], device="cuda"), torch.tensor([3, 0], device="cuda")
    a = x.clone().requires_grad_()
    y = block(a, seed, start)
    y.float().square().sum().backward()
    n = h.hlq_layer_norm_forward(x, block.norm.weight.detach(), block.norm.bias.detach())[0]
    w, u = block.attention.qkv.weight.detach(), block.attention.out.weight.detach()
    lin = (lambda p, m: h.hlq_linear_forward(p, m)[0]) if t == torch.bfloat16 else \
        (lambda p, m: p @ m.t())
    qkv = lin(n, w).view(64, 8, 16)
    o_ = h.hlq_attention_forward(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], start, causal=True, max_len=40,
                                 bias=block.attention.bias.detach(), max_distance=16)[0]
    x2 = h.hlq_dropout_forward(lin(o_.view(64, 64), u), 0.1, seed, 2, x)
    want = h.hlq_layer_norm_forward(x2, block.last.weight.detach(), block.last.bias.detach())[0]
    assert torch.equal(y, want)
    grads = {k: p.grad.clone() for k, p in block.named_parameters()}
    assert all(torch.isfinite(v).all() and (v != 0).any() for v in grads.values()), grads
    for p in block.parameters():
        p.grad = None
    b = x.clone().requires_grad_()
    block(b, seed, start).float().square().sum().backward()
    assert torch.equal(a.grad, b.grad)
    assert all(torch.equal(p.grad, grads[k]) for k, p in block.named_parameters())


def _inputs():
    torch = _torch()
    g = _gen(6)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    return dict(q=r(1000, 4, 64), k=r(1000, 2, 64), v=r(1000, 2, 64), g=r(1000, 4, 64),
                bias=torch.randn((32, 4), generator=g, device="cuda"),
                start=torch.tensor([0, 300, 307, 1000], device="cuda"),
                one=r(3, 4, 64), at=torch.tensor([0, 1, 2, 3], device="cuda"),
                seed=torch.tensor([1, 2], device="cuda"))


def _run(s, stream=None):
    """Every operator once: 16 tensors."""
    import hadamard_rank_linear_amd as h
    kw = dict(start=s["start"], stream=stream)
    o1, l1 = h.hlq_attention_forward(s["q"], s["k"], s["v"], causal=True, **kw)
    o2, l2 = h.hlq_attention_forward(s["q"], s["k"], s["v"], bias=s["bias"], **kw)
    o3, l3 = h.hlq_attention_forward(s["one"], s["k"], s["v"], s["at"], s["start"], causal=True,
                                     max_len=1, stream=stream)     # shares of the keys, joined
    g1 = h.hlq_attention_backward(s["g"], s["q"], s["k"], s["v"], o1, l1, causal=True, **kw)[:3]
    g2 = h.hlq_attention_backward(s["g"], s["q"], s["k"], s["v"], o2, l2, bias=s["bias"], **kw)
    d = h.hlq_dropout_forward(s["q"], 0.2, s["seed"], 1, s["g"], stream=stream)
    e = h.hlq_dropout_backward(s["g"], 0.2, s["seed"], 1, stream=stream)
    return [o1, l1, o2, l2, o3, l3, *g1, *g2, d, e]


def test_given_stream_beside_queued_work():
    """What the calls allocate belongs to the given stream: work that is queued on
    the current one, and tensors freed there, do not meet it."""
    torch = _torch()
    _say("attention on a given stream")
    s = _inputs()
    want = [t.clone() for t in _run(s)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a = torch.ones((4096, 4096), dtype=torch.bfloat16, device="cuda")
        for _ in range(10):
            a = torch.mm(a, a).mul_(0)
        junk = [torch.full_like(t, 7.0) for t in want]
        del junk                                     # freed, its fills still queued
        got = _run(s, side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_two_streams_at_once():
    """Calls on two streams of the same inputs, each with its own workspaces."""
    torch = _torch()
    _say("attention on two streams")
    s = _inputs()
    want = [t.clone() for t in _run(s)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(_run(s))
    torch.cuda.synchronize()
    for tensors in got:
        assert all(torch.equal(x, y) for x, y in zip(tensors, want))


def test_stream_of_another_device_or_kind_is_refused():
    import hadamard_rank_linear_amd as h
    _say("attention stream refusal")
    s = _inputs()
    with pytest.raises(TypeError):
        h.hlq_dropout_forward(s["q"], 0.1, s["seed"], stream=_torch().cuda.Event())


def test_graphs_replay_and_share_nothing():
    """Two captured graphs of the same calls, replayed in turn with eager work
    between: every replay equals the eager result; moving the seed on inside the
    graph gives each replay the next step's mask."""
    torch = _torch()
    import hadamard_rank_linear_amd as h
    _say("attention in graphs")
    s = _inputs()
    want = [t.clone() for t in _run(s)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run(s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    step = torch.tensor([9, 0], device="cuda")
    x = torch.ones(5000, device="cuda")
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(_run(s))
            outs[-1].append(h.hlq_dropout_forward(x, 0.5, step))
            step[1:] += 1
        graphs.append(graph)
    at = 0
    for rep in range(3):
        for graph, out in zip(graphs, outs):
            for t in out:
                t.fill_(float("nan"))
            junk = torch.randn(1 << 20, device="cuda").sum()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.isfinite(junk)
            assert all(torch.equal(a, b) for a, b in zip(out, want)), rep
            mask = h.hlq_dropout_forward(x, 0.5, torch.tensor([9, at], device="cuda"))
            assert torch.equal(out[-1], mask), (rep, at)
            at += 1


def test_training_step_in_a_graph():
    """A block's forward and backward pass captured once and replayed: gradients as
    in eager mode, bit for bit."""
    torch = _torch()
    _say("a block's step in a graph")
    block, g = _block(torch.bfloat16), _gen(8)
    x = torch.randn((64, 64), generator=g, device="cuda").bfloat16()
    start, seed = torch.tensor([0, 24, 64], device="cuda"), torch.tensor([3, 0], device="cuda")
    g_y = torch.randn((64, 64), generator=g, device="cuda").bfloat16()

    def step():
        return torch.autograd.grad(block(x, seed, start), list(block.parameters()), g_y)

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for rep in range(3):
        for t in got:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), rep


def test_written_buffers_count_as_written():
    """A buffer that a call writes is an in-place write to autograd."""
    torch = _torch()
    import hadamard_rank_linear_amd as h
    _say("written buffers")
    s = _inputs()
    w = torch.randn((1000, 4, 64), device="cuda").bfloat16().requires_grad_()
    box = torch.zeros_like(s["q"])
    y = (w * box).sum()
    h.hlq_attention_forward(s["q"], s["k"], s["v"], o=box)
    with pytest.raises(RuntimeError):
        y.backward()


def test_example_runs_with_attention():
    import hadamard_rank_linear_amd.tuning_study as ts
    _say("tuning example with attention")
    a = ts.tune_preferences(steps=2, pairs=4, heads=4)
    b = ts.tune_policy(steps=2, tokens=256, heads=4)
    assert all(np.isfinite(v) for v in a + b)
