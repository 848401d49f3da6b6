"""Calls with ``stream=`` beside work that is still queued on the current
stream, and tensors that are dropped while they are in use.

The allocator hands a block that was freed on a stream to the next request of
that stream at once, while the work that used it may still be queued.  So what
a call writes on a given stream must not come from the current one's pool, and
what it reads must not go back there before the given stream is done."""
import math

import pytest

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _say(msg):
    print(f"\n[gpu-case] {msg}", flush=True)


def _busy():
    """Some 20 ms of work on the current stream."""
    torch = _torch()
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device="cuda")
    for _ in range(20):
        torch.mm(a, a)


def _train_inputs():
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    T, C = 700, 1500
    return dict(x=r(T, C), r=r(T, C), w=1 + 0.1 * r(C), b=r(C), g=r(T), old=r(T) - 7, adv=r(T),
                mean=0.1 * r(T), rstd=1 + 0.1 * r(T).abs(), lp=-r(T).abs(),
                t=torch.randint(0, C, (T,), generator=g, device="cuda"),
                stats=torch.stack([r(T) + 5, 2 + r(T).abs()], 1).contiguous(),
                start=torch.tensor([0, 100, 350, 500, T], device="cuda"))


def _train_calls():
    import hadamard_rank_linear_amd as h

    def outs(s, st):                           # the caller's own tensors, of the stream that writes
        with _torch().cuda.stream(st):
            return [_torch().empty_like(s["x"])]

    return {
        "norm_forward": (_train_inputs, lambda s, st: h.hlq_layer_norm_forward(
            s["x"], s["w"], s["b"], residual=s["r"], stream=st)),
        "norm_backward": (_train_inputs, lambda s, st: h.hlq_layer_norm_backward(
            s["r"], s["x"], s["mean"], s["rstd"], s["w"], stream=st)),
        "score": (_train_inputs, lambda s, st: h.hlq_token_logprob_forward(s["x"], s["t"],
                                                                           stream=st)),
        "gradient": (_train_inputs, lambda s, st: [h.hlq_token_logprob_backward(
            s["g"], s["x"], s["t"], s["stats"], stream=st)]),
        "policy": (_train_inputs, lambda s, st: h.hlq_policy_loss(s["lp"], s["old"], s["adv"],
                                                                  stream=st)),
        "policy_logits": (_train_inputs, lambda s, st: h.hlq_policy_loss_logits(
            s["x"], s["t"], s["old"], s["adv"], stream=st)),
        "preference": (_train_inputs, lambda s, st: h.hlq_preference_loss(
            s["lp"], s["start"], 0.3, stream=st)),
        "clip": (_train_inputs, lambda s, st: (lambda o: [h.hlq_clip_grad_norm(
            [s["x"]], 0.5, out=o, stream=st), *o])(outs(s, st))),
    }


def _linear_inputs():
    import hadamard_rank_linear_amd as h
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    x = r(1024, 512)
    codes, scales = h.hlq_compress_act(x)
    return dict(x=x, gy=r(1024, 256), w=r(256, 512), codes=codes, scales=scales)


def _conv_inputs():
    import hadamard_rank_linear_amd as h
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    codes, scales = h.hlq_compress_act(r(512, 32))       # 2 images of 16 x 16, 32 channels
    return dict(gy=r(512, 64), w=r(64, 9 * 32), codes=codes, scales=scales)


def _linear_calls():
    import hadamard_rank_linear_amd as h
    four = lambda s: (s["gy"], s["codes"], s["scales"], s["w"])
    return {
        "compress": (_linear_inputs, lambda s, st: h.hlq_compress_act(s["x"], stream=st)),
        "linear_forward": (_linear_inputs, lambda s, st: h.hlq_linear_forward(
            s["x"], s["w"], stream=st)),
        "linear_backward": (_linear_inputs, lambda s, st: h.hlq_linear_backward(
            *four(s), 16, 8, stream=st)),
        "linear_backward_noalloc": (_linear_inputs, lambda s, st: h.hlq_linear_backward_noalloc(
            *four(s), 16, 8, stream=st)),
        "ablation": (_linear_inputs, lambda s, st: h.hlq_linear_backward_ablation(
            *four(s), 16, 8, h.HLQ_VAR_HQ4, h.HLQ_VAR_HLA8_INT, stream=st)),
        "lqs": (_linear_inputs, lambda s, st: [h.hlq_lqs_accumulate(*four(s), 16, 8, stream=st)]),
        "conv_backward": (_conv_inputs, lambda s, st: h.hlq_conv_backward(
            *four(s), 2, 16, 16, 32, 3, 3, 1, 1, 16, 8, stream=st)),
    }


def _calls():
    return {**_train_calls(), **_linear_calls()}


NAMES = ["compress", "linear_forward", "linear_backward", "linear_backward_noalloc", "ablation",
         "lqs", "conv_backward",
         "norm_forward", "norm_backward", "score", "gradient", "policy", "policy_logits",
         "preference", "clip"]


def _same(got, want, what):
    torch = _torch()
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), f"{what}: output {i}"


def _spoil(shape, dtype):
    torch = _torch()
    return torch.empty(shape, dtype=dtype, device="cuda").fill_(
        float("nan") if dtype.is_floating_point else 7)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_apart_from_queued_work(name):
    torch = _torch()
    _say(f"{name}: outputs beside queued work of the current stream")
    inputs, call = _calls()[name]
    s = inputs()
    want = [v.clone() for v in call(s, None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the outputs' sizes and small ones, written late and freed at once
    blocks = [torch.empty_like(v) for v in want] + \
        [torch.empty(n, dtype=torch.uint8, device="cuda") for n in [256] * 32 + [1 << 15] * 8]
    _busy()
    for v in blocks:
        v.fill_(float("nan") if v.is_floating_point() else 255)
    del v, blocks
    got = call(s, side)
    _same(got, want, name)


@pytest.mark.parametrize("name", NAMES)
def test_inputs_dropped_while_in_use(name):
    torch = _torch()
    _say(f"{name}: inputs dropped before the given stream reads them")
    inputs, call = _calls()[name]
    s = inputs()
    want = [v.clone() for v in call(s, None)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _busy()                                # its own warm-up
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _busy()
    got = call(s, side)
    shapes = [(v.shape, v.dtype) for v in s.values()]
    del s
    junk = [_spoil(*v) for v in shapes]
    _same(got, want, name)
    del junk


@pytest.mark.parametrize("name", NAMES)
def test_outputs_dropped_while_in_use(name):
    torch = _torch()
    _say(f"{name}: outputs dropped while the current stream reads them")
    inputs, call = _calls()[name]
    s = inputs()
    want = [v.clone() for v in call(s, None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(s, side)
    if name == "clip":                         # the clipped tensors are the caller's own
        got, want = got[:1], want[:1]
    torch.cuda.current_stream().wait_stream(side)
    _busy()
    kept = [v.clone() for v in got]
    with torch.cuda.stream(side):
        del got
        junk = [_spoil(v.shape, v.dtype) for v in want]
    _same(kept, want, name)
    del junk


def test_the_given_stream_is_current_and_no_longer():
    torch = _torch()
    import hadamard_rank_linear_amd as h
    _say("streams: refusals, and the current stream after a call")
    x, w = torch.randn(8, 64, device="cuda"), torch.ones(64, device="cuda")
    before = torch.cuda.current_stream()
    side = torch.cuda.Stream()
    side.wait_stream(before)
    y = h.hlq_layer_norm_forward(x, w, stream=side)[0]
    assert torch.cuda.current_stream() == before
    with torch.cuda.stream(side):
        z = h.hlq_layer_norm_forward(x, w, stream=side)[0]
        before.wait_stream(side)
        u = h.hlq_layer_norm_forward(x, w, stream=before)[0]
        assert torch.cuda.current_stream() == side
    torch.cuda.synchronize()
    assert torch.equal(y, z) and torch.equal(y, u)
    for wrong in (0, "side", side.cuda_stream):
        with pytest.raises((TypeError, AttributeError)):
            h.hlq_layer_norm_forward(x, w, stream=wrong)
    with pytest.raises(h.HLQError):            # a refused call leaves the stream as it was
        h.hlq_layer_norm_forward(x, w, eps=math.nan, stream=side)
    assert torch.cuda.current_stream() == before


def test_streams_of_other_makes():
    # an object that only names its handle, as the linear layer's entry points take it
    torch = _torch()
    import types

    import hadamard_rank_linear_amd as h
    _say("linear layer on a stream that is no torch object")
    s = _linear_inputs()
    want = h.hlq_compress_act(s["x"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = h.hlq_compress_act(s["x"], stream=types.SimpleNamespace(cuda_stream=side.cuda_stream))
    _same(got, want, "compress")
