"""Host-side checks of the training step's operators (no GPU, nothing is
launched): refusals of the C ABI and of the binding, workspace sizes."""
import ctypes

import pytest

import hadamard_rank_linear_amd as h

P = 1 << 20          # a fake, aligned address: every call below must refuse before a launch
NAN, INF = float("nan"), float("inf")
NULL, SHAPE, MODE, DTYPE, ALIGN, WORKSPACE, VALUE = 1, 2, 5, 6, 7, 9, 11


def _call(name, order, defaults, kw):
    args = dict(defaults, **kw)
    return getattr(h.lib_handle(), name)(*(args[k] for k in order.split()))


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), NULL), (dict(y=None), NULL), (dict(weight=None), NULL), (dict(mean=None), NULL),
    (dict(h=None), NULL),                      # a residual without its sum, and the reverse
    (dict(residual=None), NULL),
    (dict(dt=2), DTYPE), (dict(pdt=-1), DTYPE), (dict(T=-1), SHAPE), (dict(C=0), SHAPE),
    (dict(T=1 << 31), SHAPE), (dict(C=1 << 31), SHAPE), (dict(eps=-1.0), VALUE),
    (dict(eps=NAN), VALUE), (dict(eps=INF), VALUE),
    (dict(x=P + 2), ALIGN), (dict(x=P + 1, dt=1), ALIGN), (dict(rstd=P + 2), ALIGN),
    (dict(weight=P + 2), ALIGN)])
def test_layer_norm_forward_refuses(kw, status):
    assert _call("hlq_layer_norm_forward",
                 "x residual dt weight bias pdt T C eps y h mean rstd stream",
                 dict(x=P, residual=P, dt=0, weight=P, bias=P, pdt=0, T=4, C=8, eps=1e-5, y=P, h=P,
                      mean=P, rstd=P, stream=None), kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(gy=None), NULL), (dict(gx=None), NULL), (dict(gw=None), NULL), (dict(rstd=None), NULL),
    (dict(dt=7), DTYPE), (dict(C=0), SHAPE), (dict(T=-3), SHAPE), (dict(gy=P + 2), ALIGN),
    (dict(gw=P + 2), ALIGN), (dict(ws=P + 4), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(bytes=8), WORKSPACE)])
def test_layer_norm_backward_refuses(kw, status):
    assert _call("hlq_layer_norm_backward",
                 "gy h gh dt mean rstd weight pdt T C gx gw gb ws bytes stream",
                 dict(gy=P, h=P, gh=P, dt=0, mean=P, rstd=P, weight=P, pdt=0, T=4, C=8, gx=P, gw=P,
                      gb=P, ws=P, bytes=1 << 40, stream=None), kw) == status


LOGITS = [(dict(x=None), NULL), (dict(t=None), NULL), (dict(dt=3), DTYPE), (dict(ld=7), SHAPE),
          (dict(V=0, ld=0), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE),
          (dict(scale=0.0), VALUE), (dict(scale=-1.0), VALUE), (dict(scale=NAN), VALUE),
          (dict(scale=INF), VALUE), (dict(x=P + 2), ALIGN), (dict(t=P + 4), ALIGN)]


@pytest.mark.parametrize("kw,status", LOGITS + [(dict(lp=None), NULL), (dict(st=P + 2), ALIGN)])
def test_token_logprob_forward_refuses(kw, status):
    assert _call("hlq_token_logprob_forward", "x dt ld t T V scale lp st stream",
                 dict(x=P, dt=0, ld=8, t=P, T=4, V=8, scale=1.0, lp=P, st=P, stream=None),
                 kw) == status


@pytest.mark.parametrize("kw,status", LOGITS + [
    (dict(g=None), NULL), (dict(st=None), NULL), (dict(gx=None), NULL), (dict(gld=7), SHAPE),
    (dict(gx=P + 2), ALIGN)])
def test_token_logprob_backward_refuses(kw, status):
    assert _call("hlq_token_logprob_backward", "g x dt ld t st T V scale gx gld stream",
                 dict(g=P, x=P, dt=0, ld=8, t=P, st=P, T=4, V=8, scale=1.0, gx=P, gld=8,
                      stream=None), kw) == status


POLICY = [(dict(old=None), NULL), (dict(adv=None), NULL), (dict(sums=None), NULL),
          (dict(ref=None), NULL),                       # a KL term without its reference
          (dict(kl=0.0), NULL),                         # a reference that nothing reads
          (dict(lo=-0.1), VALUE), (dict(lo=1.5), VALUE), (dict(hi=NAN), VALUE),
          (dict(kl=-1.0), VALUE), (dict(kl=INF), VALUE), (dict(ws=None), WORKSPACE),
          (dict(bytes=95), WORKSPACE), (dict(ws=P + 8), ALIGN), (dict(w=P + 1), ALIGN)]


@pytest.mark.parametrize("kw,status", POLICY + [(dict(lp=None), NULL), (dict(g=None), NULL),
                                                (dict(T=-1), SHAPE)])
def test_policy_loss_refuses(kw, status):
    assert _call("hlq_policy_loss", "lp old adv w ref T lo hi kl sums g ws bytes stream",
                 dict(lp=P, old=P, adv=P, w=P, ref=P, T=4, lo=0.2, hi=0.2, kl=0.1, sums=P, g=P, ws=P,
                      bytes=1 << 30, stream=None), kw) == status


@pytest.mark.parametrize("kw,status", LOGITS + POLICY + [(dict(lp=None), NULL),
                                                         (dict(gx=None), NULL),
                                                         (dict(gld=3), SHAPE)])
def test_policy_loss_logits_refuses(kw, status):
    assert _call("hlq_policy_loss_logits",
                 "x dt ld t old adv w ref T V scale lo hi kl sums lp gx gld ws bytes stream",
                 dict(x=P, dt=0, ld=8, t=P, old=P, adv=P, w=P, ref=P, T=4, V=8, scale=1.0, lo=0.2,
                      hi=0.2, kl=0.1, sums=P, lp=P, gx=P, gld=8, ws=P, bytes=1 << 30, stream=None),
                 kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(lp=None), NULL), (dict(start=None), NULL), (dict(loss=None), NULL), (dict(margin=None), NULL),
    (dict(g=None), NULL), (dict(P=0), SHAPE), (dict(P=1 << 24), SHAPE), (dict(T=-1), SHAPE),
    (dict(beta=0.0), VALUE), (dict(beta=NAN), VALUE), (dict(e=1.5), VALUE), (dict(e=-0.1), VALUE),
    (dict(red=2), MODE), (dict(start=P + 4), ALIGN), (dict(ref=P + 2), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(bytes=15), WORKSPACE)])
def test_preference_loss_refuses(kw, status):
    assert _call("hlq_preference_loss",
                 "lp ref w start P T beta e red loss margin g ws bytes stream",
                 dict(lp=P, ref=P, w=P, start=P, P=2, T=9, beta=0.1, e=0.0, red=0, loss=P, margin=P,
                      g=P, ws=P, bytes=1 << 30, stream=None), kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(grads=None), NULL), (dict(grad1=0), NULL), (dict(out1=0), NULL), (dict(norm=None), NULL),
    (dict(sizes=None), NULL), (dict(dtypes=None), NULL), (dict(count=-1), SHAPE),
    (dict(size1=-4), SHAPE), (dict(size1=1 << 40), SHAPE), (dict(dtype1=2), DTYPE),
    (dict(grad1=P + 2), ALIGN), (dict(out1=P + 1, dtype1=1), ALIGN), (dict(norm=P + 4), ALIGN),
    (dict(max_norm=-1.0), VALUE), (dict(max_norm=NAN), VALUE), (dict(kind=2), MODE),
    (dict(ws=None), WORKSPACE), (dict(bytes=8), WORKSPACE)])
def test_clip_grad_norm_refuses(kw, status):
    a = dict(grad1=P, out1=P, size1=100, dtype1=0, max_norm=1.0, kind=0, norm=P, ws=P,
             bytes=1 << 30, count=2)
    a.update(kw)
    VP, I64, I32 = ctypes.c_void_p * 2, ctypes.c_int64 * 2, ctypes.c_int * 2
    lists = dict(grads=VP(P, a["grad1"]), outs=VP(P, a["out1"]), sizes=I64(7, a["size1"]),
                 dtypes=I32(1, a["dtype1"]))
    for k in ("grads", "sizes", "dtypes"):
        if k in kw:
            lists[k] = None
    assert h.lib_handle().hlq_clip_grad_norm(
        lists["grads"], lists["outs"], lists["sizes"], lists["dtypes"], a["count"], a["max_norm"],
        a["kind"], a["norm"], a["ws"], a["bytes"], None) == status


def test_empty_calls_need_no_pointers():
    # nothing to do: accepted with NULL operands, and nothing is launched
    lib = h.lib_handle()
    assert lib.hlq_layer_norm_forward(None, None, 0, P, None, 0, 0, 8, 1e-5, None, None, None, None,
                                      None) == 0
    assert lib.hlq_token_logprob_forward(None, 0, 8, None, 0, 8, 1.0, None, None, None) == 0
    assert lib.hlq_token_logprob_backward(None, None, 0, 8, None, None, 0, 8, 1.0, None, 8,
                                          None) == 0


def test_workspace_sizes():
    assert h.hlq_layer_norm_backward_workspace_size(0, 8) == 0
    assert h.hlq_layer_norm_backward_workspace_size(-1, 8) == 0
    assert h.hlq_layer_norm_backward_workspace_size(4, 0) == 0
    for T, C in ((1, 1), (7, 768), (65536, 64), (100000, 16384), (3, 100000)):
        for dt in (h.HLQ_F32, h.HLQ_BF16):
            size = h.hlq_layer_norm_backward_workspace_size(T, C, dt)
            assert size >= 8 * C and size % (8 * C) == 0
            assert size <= 8 * C * T                    # never more parts than rows
    assert h.hlq_policy_loss_workspace_size(5) >= 5 * 24 and h.hlq_policy_loss_workspace_size(0) == 0
    assert h.hlq_preference_loss_workspace_size(3) >= 24
    assert h.hlq_clip_grad_norm_workspace_size([]) == 0
    assert h.hlq_clip_grad_norm_workspace_size([0, 0]) == 0
    assert h.hlq_clip_grad_norm_workspace_size([1]) >= 8
    assert h.hlq_clip_grad_norm_workspace_size([5, -1]) == 0
    assert h.hlq_clip_grad_norm_workspace_size([3 << 30]) >= 8


def test_binding_refuses():
    import torch
    x, w = torch.zeros(4, 8), torch.zeros(8)
    t, v = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        h.hlq_layer_norm_forward(x, w)
    with pytest.raises(ValueError, match="weight"):
        h.hlq_layer_norm_forward(x, torch.zeros(4))
    with pytest.raises(TypeError, match="bias"):
        h.hlq_layer_norm_forward(x, w, torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="residual"):
        h.hlq_layer_norm_forward(x, w, residual=x.bfloat16())
    with pytest.raises(ValueError, match="no residual"):
        h.hlq_layer_norm_forward(x, w, h=x)
    with pytest.raises(ValueError, match="g_y"):
        h.hlq_layer_norm_backward(x[:2], x, v, v, w)
    with pytest.raises(ValueError, match="mean"):
        h.hlq_layer_norm_backward(x, x, v[:2], v, w)
    with pytest.raises(ValueError, match="GPU"):
        h.hlq_token_logprob_forward(x, t)
    with pytest.raises(ValueError, match="2-D"):
        h.hlq_token_logprob_forward(v, t)
    with pytest.raises(ValueError, match="GPU"):
        h.hlq_policy_loss(v, v, v)
    with pytest.raises(ValueError, match="advantage"):
        h.hlq_policy_loss(v, v, v[:3])
    with pytest.raises(ValueError, match="expected|cpu"):
        h.hlq_clip_grad_norm([v], 1.0)
    with pytest.raises(ValueError, match="outputs"):
        h.hlq_clip_grad_norm([v], 1.0, out=[])
