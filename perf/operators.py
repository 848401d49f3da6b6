"""Cases, inputs and plain forms of the operators around the HLQ linear layer
in a training step: layer norm, token log probabilities with the policy and
preference losses on them, and the clipping of gradients by their global norm.

``run`` computes a case in elementary torch operations while ``own`` is false,
and through the calls of ``hadamard_rank_linear_amd`` when it is true.
``exact`` gives the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
CLIP_EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the norm of one new token in a decoder of width 4096, with the residual add
        dict(name="norm_one_token", op="norm_forward", rows=1, cols=4096, dtype="bf16",
             param="bf16", residual=True, bias=True),
        # ViT-B's tokens at batch 64, in front of the qkv layer, residual add fused
        dict(name="norm_vitb", op="norm_forward", rows=12608, cols=768, dtype="bf16",
             param="f32", residual=True, bias=True),
        # its backward, with the gradient that comes along the residual stream
        dict(name="norm_backward_vitb", op="norm_backward", rows=12608, cols=768, dtype="bf16",
             param="f32", residual=True, bias=True),
        # a wide 32-bit norm over an odd count of tokens, weight alone
        dict(name="norm_backward_wide", op="norm_backward", rows=16383, cols=4096, dtype="f32",
             param="f32", residual=False, bias=False),
        # scoring the last tokens of a few requests; an odd vocabulary
        dict(name="score_few", op="score", rows=3, vocab=32003, dtype="bf16", scale=1.0,
             banned=0.0, ignored=0.0),
        # scoring a batch under the old or the reference policy, padded vocabulary masked with
        # -inf, prompt tokens ignored
        dict(name="score_batch", op="score", rows=4096, vocab=128256, dtype="bf16", scale=1.0,
             banned=0.01, ignored=0.1),
        # a policy update over sampled answers (temperature 0.7), prompts masked
        dict(name="policy_large", op="policy", rows=2048, vocab=128256, dtype="bf16", scale=1.0 / 0.7,
             clip_low=0.2, clip_high=0.28, kl=0.02, prompt=0.2, banned=0.0),
        # 32-bit logits of an odd vocabulary, no KL term, every token counts
        dict(name="policy_odd_f32", op="policy", rows=1023, vocab=48003, dtype="f32", scale=1.0,
             clip_low=0.2, clip_high=0.2, kl=0.0, prompt=0.0, banned=0.0),
        # two short pairs: a step of preference tuning at its smallest
        dict(name="preference_small", op="preference", rows=301, vocab=4099, pairs=2, dtype="f32",
             beta=0.1, smoothing=0.0, mean=False, prompt=0.3),
        # thirty-two ragged pairs, packed
        dict(name="preference_batch", op="preference", rows=8190, vocab=32000, pairs=32,
             dtype="bf16", beta=0.1, smoothing=0.1, mean=False, prompt=0.3),
        # 146 gradients of a small model: launch-bound
        dict(name="clip_small", op="clip", layers=12, hidden=63, inner=257, vocab=1001,
             dtype="f32", norm="l2", clips=True),
        # eight decoder layers, bf16 matrices and 32-bit norm parameters
        dict(name="clip_large", op="clip", layers=8, hidden=4096, inner=14336, vocab=32000,
             dtype="bf16", norm="l2", clips=True),
    ]


def _log(rng, lo, hi):
    """An integer from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "score", "policy", "preference", "clip"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("norm_forward", "norm_backward"):
        cols = _log(rng, 8, 16384)
        if rng.random() < 0.5:
            cols = max(8, cols // 64 * 64)
        rows = _log(rng, 1, min(65536, (1 << 26) // cols))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, param=rng.choice(["f32", dtype]),
                    residual=rng.random() < 0.5, bias=rng.random() < 0.7)
    if op == "clip":
        hidden = _log(rng, 32, 4096)
        inner = hidden * rng.randint(2, 4) + rng.randint(0, 3)
        layer = 4 * hidden * hidden + 2 * hidden * inner
        layers = _log(rng, 1, max(1, min(32, (1 << 31) // SIZE[dtype] // layer)))
        return dict(op=op, layers=layers, hidden=hidden, inner=inner, vocab=_log(rng, 100, 32000),
                    dtype=dtype, norm=rng.choice(["l2", "l2", "inf"]), clips=rng.random() < 0.75)
    vocab = _log(rng, 512, 131072)
    if rng.random() < 0.5:
        vocab = vocab // 128 * 128
    most = (1 << 28) // SIZE[dtype] * 2 // vocab
    case = dict(op=op, vocab=vocab, dtype=dtype)
    if op == "score":
        case.update(rows=_log(rng, 1, min(8192, most)), scale=rng.choice([1.0, 1.0, 1.25, 0.5]),
                    banned=rng.choice([0.0, 0.02]), ignored=rng.choice([0.0, 0.2]))
    elif op == "policy":
        case.update(rows=_log(rng, 1, min(8192, most)), scale=rng.choice([1.0, 1.0, 1.25]),
                    clip_low=0.2, clip_high=rng.choice([0.2, 0.28]), kl=rng.choice([0.0, 0.05]),
                    prompt=rng.choice([0.0, 0.25, 0.5]), banned=rng.choice([0.0, 0.02]))
    else:
        pairs = _log(rng, 1, 64)
        case.update(rows=_log(rng, 4 * pairs, max(4 * pairs, min(8192, most))), pairs=pairs,
                    beta=rng.choice([0.1, 0.5]), smoothing=rng.choice([0.0, 0.1]),
                    mean=rng.random() < 0.3, prompt=rng.choice([0.0, 0.3]))
    return case


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _norm_inputs(case, g):
    """Activations with an offset and a spread per channel, as a residual
    stream has them; upstream gradients with a heavy tail."""
    T, C, dt, pt = case["rows"], case["cols"], DTYPES[case["dtype"]], DTYPES[case["param"]]
    spread, offset = torch.exp(0.5 * _randn(g, C)), 0.3 * _randn(g, C)
    s = dict(case=case, weight=(1.0 + 0.1 * _randn(g, C)).to(pt),
             bias=(0.1 * _randn(g, C)).to(pt) if case["bias"] else None, eps=1e-5)
    x = (_randn(g, T, C) * spread + offset).to(dt)
    if case["op"] == "norm_forward":
        s.update(x=x, residual=(0.5 * _randn(g, T, C)).to(dt) if case["residual"] else None)
        return s
    x32 = x.float()
    mean = x32.mean(-1)
    var = (x32 - mean[:, None]).square().mean(-1)
    s.update(h=x, mean=mean, rstd=torch.rsqrt(var + s["eps"]),
             g_y=(1e-3 * _randn(g, T, C) * torch.exp(0.5 * _randn(g, T, C))).to(dt),
             g_h=(1e-3 * _randn(g, T, C)).to(dt) if case["residual"] else None)
    return s


def _logit_inputs(case, g):
    """Logits as a head gives them: a spread of 2.5, the chosen token raised
    by up to 10; a share of the vocabulary's end banned by -inf."""
    T, V, dt = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    live = V - int(V * case.get("banned", 0.0))
    targets = torch.randint(0, live, (T,), generator=g, device="cuda")
    logits = _randn(g, T, V).mul_(2.5)
    logits[torch.arange(T, device="cuda"), targets] += 10.0 * _rand(g, T)
    if live < V:
        logits[:, live:] = -math.inf
    return logits.to(dt), targets


def _plain_logprob(logits, targets, scale):
    """Log probability of each target in 64 bits, from 32-bit exponentials,
    and each row's (maximum, sum of exponentials above it); ignored targets
    give 0 and (0, 1)."""
    T, V = logits.shape
    lp = torch.empty(T, dtype=torch.float64, device=logits.device)
    stats = torch.empty((T, 2), dtype=torch.float32, device=logits.device)
    step = max(1, (1 << 27) // V)
    for a in range(0, T, step):
        x = logits[a:a + step].float()
        m = x.amax(-1, keepdim=True)
        total = torch.exp((x - m) * scale).sum(-1, dtype=torch.float64)
        at = targets[a:a + step].clamp(0, V - 1)[:, None]
        lp[a:a + step] = (x.gather(1, at) - m)[:, 0].double() * scale - torch.log(total)
        stats[a:a + step, 0], stats[a:a + step, 1] = m[:, 0], total.float()
    live = (targets >= 0) & (targets < V)
    none = torch.tensor([0.0, 1.0], device=logits.device)
    return torch.where(live, lp, torch.zeros_like(lp)), torch.where(live[:, None], stats, none)


def _shapes(case):
    """Gradient shapes of a decoder: an embedding, a last norm, and twelve
    parameters a layer."""
    h, i = case["hidden"], case["inner"]
    per_layer = [(h,), (h,), (h, h), (h,), (h, h), (h, h), (h, h), (h,), (h,), (h,), (i, h), (h, i)]
    return [(case["vocab"], h), (h,)] + per_layer * case["layers"]


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op in ("norm_forward", "norm_backward"):
        return _norm_inputs(case, g)
    if op == "clip":
        mat = DTYPES[case["dtype"]]
        grads = []
        for shape in _shapes(case):
            v = torch.randn(shape, generator=g, device="cuda",
                            dtype=mat if len(shape) > 1 else torch.float32)
            grads.append(v.mul_(1e-3))
        n = sum(v.numel() for v in grads)
        # the clipped gradients are views of one flat buffer a type, packed as a bucket packs them
        flat = {t: torch.empty(sum(v.numel() for v in grads if v.dtype == t), dtype=t, device="cuda")
                for t in dict.fromkeys(v.dtype for v in grads)}
        used, out = dict.fromkeys(flat, 0), []
        for v in grads:
            a = used[v.dtype]
            out.append(flat[v.dtype][a:a + v.numel()].view(v.shape))
            used[v.dtype] = a + v.numel()
        # the norm is close to 1e-3 sqrt(n), the largest magnitude below 1e-2
        size = 1e-3 * (math.sqrt(n) if case["norm"] == "l2" else 1.0)
        return dict(case=case, grads=grads, out=out, flat=list(flat.values()),
                    max_norm=0.3 * size if case["clips"] else 20.0 * size)
    logits, targets = _logit_inputs(case, g)
    T = case["rows"]
    s = dict(case=case, logits=logits, targets=targets)
    if op == "score":
        targets[_rand(g, T) < case["ignored"]] = -100
        return s
    lp = _plain_logprob(logits, targets, case.get("scale", 1.0))[0]
    s["ref"] = (lp + 0.2 * _randn(g, T)).float()
    if op == "policy":
        # the first tokens of the packed batch are the prompts; the weights sum to one
        live = torch.arange(T, device="cuda") >= int(T * case["prompt"])
        s.update(old=(lp + 0.1 * _randn(g, T)).float(), advantage=_randn(g, T),
                 weight=live.float() / max(1, T - int(T * case["prompt"])))
        return s
    # ragged sequences, chosen ones first; each starts with an ignored prompt
    cuts = np.sort(np.random.default_rng(seed).integers(0, T + 1, 2 * case["pairs"] - 1))
    start = np.concatenate([[0], cuts, [T]]).astype(np.int64)
    for a, b in zip(start[:-1], start[1:]):
        targets[a:a + int((b - a) * case["prompt"])] = -100
    s["start"] = torch.from_numpy(start).cuda()
    s["weight"] = (targets >= 0).float()
    return s


# ---------------------------------------------------------------- plain forms

def _plain_norm_forward(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = (h + s["residual"].float()).to(s["x"].dtype)
    h32 = h.float()
    mean = h32.mean(-1, keepdim=True)
    d = h32 - mean
    rstd = torch.rsqrt((d * d).mean(-1, keepdim=True) + s["eps"])
    y = d * rstd * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = y.to(s["x"].dtype)
    if s["residual"] is not None:
        return y, h, mean[:, 0], rstd[:, 0]
    return y, mean[:, 0], rstd[:, 0]


def _plain_norm_backward(s):
    g, h, w = s["g_y"].float(), s["h"].float(), s["weight"]
    rstd = s["rstd"][:, None]
    xh = (h - s["mean"][:, None]) * rstd
    u = g * w.float()
    g_x = rstd * (u - u.mean(-1, keepdim=True) - xh * (u * xh).mean(-1, keepdim=True))
    if s["g_h"] is not None:
        g_x = g_x + s["g_h"].float()
    g_w = (g * xh).sum(0, dtype=torch.float64).to(w.dtype)
    if s["bias"] is None:
        return g_x.to(s["h"].dtype), g_w
    return g_x.to(s["h"].dtype), g_w, g.sum(0, dtype=torch.float64).to(w.dtype)


def _plain_logit_gradient(logits, targets, stats, g_lp, scale):
    """g_lp scale ([v = target] - softmax), rows with g_lp = 0 all zero."""
    T, V = logits.shape
    out = torch.empty_like(logits)
    step = max(1, (1 << 27) // V)
    for a in range(0, T, step):
        x, g = logits[a:a + step].float(), g_lp[a:a + step]
        at = targets[a:a + step].clamp(0, V - 1)[:, None]
        d = -torch.exp((x - stats[a:a + step, :1]) * scale) / stats[a:a + step, 1:]
        d.scatter_add_(1, at, torch.ones_like(at, dtype=torch.float32))
        d = d * (g * scale)[:, None]
        out[a:a + step] = torch.where((g == 0)[:, None], torch.zeros_like(d), d).to(logits.dtype)
    return out


def _plain_policy(s):
    c = s["case"]
    lp, stats = _plain_logprob(s["logits"], s["targets"], c["scale"])
    w, A = s["weight"].double(), s["advantage"].double()
    live = w != 0
    ratio = torch.exp(lp - s["old"].double())
    free = ratio * A
    clipped = torch.minimum(torch.maximum(ratio, torch.full_like(ratio, 1.0 - c["clip_low"])),
                            torch.full_like(ratio, 1.0 + c["clip_high"])) * A
    d = s["ref"].double() - lp
    kl = torch.exp(d) - d - 1.0 if c["kl"] else torch.zeros_like(d)
    zero = torch.zeros_like(lp)
    loss = torch.where(live, w * (c["kl"] * kl - torch.minimum(free, clipped)), zero).sum()
    cut = torch.where(live & (clipped < free), w, zero).sum()
    sums = torch.stack([loss, torch.where(live, w * kl, zero).sum(), cut]).float()
    g = torch.where(free <= clipped, -free, zero)
    if c["kl"]:
        g = g + c["kl"] * (1.0 - torch.exp(d))
    g = torch.where(live, w * g, zero).float()
    lp = torch.where(live, lp, zero)
    g_x = _plain_logit_gradient(s["logits"], s["targets"], stats, g, c["scale"])
    return sums, lp.float(), g_x


def _plain_preference(s):
    c = s["case"]
    lp, stats = _plain_logprob(s["logits"], s["targets"], 1.0)
    w, P = s["weight"].double(), c["pairs"]
    diff = w * (lp.float().double() - s["ref"].double())
    edge = torch.zeros(len(diff) + 1, dtype=torch.float64, device=diff.device)
    edge[1:] = diff.cumsum(0)
    wide = torch.zeros_like(edge)
    wide[1:] = w.cumsum(0)
    a, b = s["start"][:-1], s["start"][1:]
    total, length = edge[b] - edge[a], wide[b] - wide[a]
    part = torch.where(length > 0, 1.0 / length, torch.zeros_like(length)) if c["mean"] \
        else torch.ones_like(length)
    z = c["beta"] * ((total * part)[:P] - (total * part)[P:])
    e = c["smoothing"]
    up, down = torch.log1p(torch.exp(-z.abs())) + torch.relu(-z), \
        torch.log1p(torch.exp(-z.abs())) + torch.relu(z)
    loss = ((1.0 - e) * up + e * down).mean()
    p = 1.0 / (1.0 + torch.exp(-z))
    g_z = c["beta"] / P * ((1.0 - e) * (p - 1.0) + e * p)
    g_seq = torch.cat([g_z, -g_z]) * part
    seq = torch.searchsorted(s["start"][1:].contiguous(),
                             torch.arange(len(w), device=w.device), right=True)
    g_lp = (w * g_seq[seq]).float()
    g_x = _plain_logit_gradient(s["logits"], s["targets"], stats, g_lp, 1.0)
    return loss.float().reshape(1), z.float(), g_x


def _plain_clip(s):
    if s["case"]["norm"] == "l2":
        norm = torch.stack([(v.double() * v.double()).sum() for v in s["grads"]]).sum().sqrt()
    else:
        norm = torch.stack([v.float().abs().max() for v in s["grads"]]).max().double()
    coef = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0).float()
    for v, o in zip(s["grads"], s["out"]):
        o.copy_(v.float() * coef)
    return norm.reshape(1), *s["flat"]


def _plain(s):
    op = s["case"]["op"]
    if op == "norm_forward":
        return _plain_norm_forward(s)
    if op == "norm_backward":
        return _plain_norm_backward(s)
    if op == "score":
        lp, stats = _plain_logprob(s["logits"], s["targets"], s["case"]["scale"])
        return lp.float(), stats
    if op == "policy":
        return _plain_policy(s)
    if op == "preference":
        return _plain_preference(s)
    return _plain_clip(s)


# ---------------------------------------------------------------- the framework's calls

def _framework(s):
    import hadamard_rank_linear_amd as h
    c = s["case"]
    op = c["op"]
    if op == "norm_forward":
        y, total, mean, rstd = h.hlq_layer_norm_forward(s["x"], s["weight"], s["bias"], s["eps"],
                                                        residual=s["residual"])
        return (y, mean, rstd) if s["residual"] is None else (y, total, mean, rstd)
    if op == "norm_backward":
        g_x, g_w, g_b = h.hlq_layer_norm_backward(s["g_y"], s["h"], s["mean"], s["rstd"],
                                                  s["weight"], g_h=s["g_h"],
                                                  with_bias=s["bias"] is not None)
        return (g_x, g_w) if s["bias"] is None else (g_x, g_w, g_b)
    if op == "score":
        return h.hlq_token_logprob_forward(s["logits"], s["targets"], c["scale"])
    if op == "policy":
        return h.hlq_policy_loss_logits(s["logits"], s["targets"], s["old"], s["advantage"],
                                        s["weight"], ref_logprob=s["ref"] if c["kl"] else None,
                                        scale=c["scale"], clip_low=c["clip_low"],
                                        clip_high=c["clip_high"], kl_coef=c["kl"])
    if op == "preference":
        lp, stats = h.hlq_token_logprob_forward(s["logits"], s["targets"])
        loss, margin, g_lp = h.hlq_preference_loss(
            lp, s["start"], c["beta"], ref_logprob=s["ref"], weight=s["weight"],
            label_smoothing=c["smoothing"], reduction=h.HLQ_MEAN if c["mean"] else h.HLQ_SUM)
        return loss, margin, h.hlq_token_logprob_backward(g_lp, s["logits"], s["targets"], stats)
    norm = h.hlq_clip_grad_norm(s["grads"], s["max_norm"],
                                h.HLQ_NORM_L2 if c["norm"] == "l2" else h.HLQ_NORM_INF,
                                out=s["out"])
    return norm, *s["flat"]


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------- in 64 bits

def _exact_norm(s):
    op, C = s["case"]["op"], s["case"]["cols"]
    w = s["weight"].double().requires_grad_()
    b = None if s["bias"] is None else s["bias"].double().requires_grad_()
    if op == "norm_forward":
        h = s["x"].double()
        if s["residual"] is not None:
            h = h + s["residual"].double()
        out_h = h
        h = h.float().to(s["x"].dtype).double()    # the stored sum is what gets normalised
        with torch.no_grad():
            y = torch.nn.functional.layer_norm(h, (C,), w, b, s["eps"])
        var, mean = torch.var_mean(h, -1, correction=0)
        stats = (mean, 1.0 / torch.sqrt(var + s["eps"]))
        return (y, *stats) if s["residual"] is None else (y, out_h, *stats)
    h = s["h"].double().requires_grad_()
    y = torch.nn.functional.layer_norm(h, (C,), w, b, s["eps"])
    grads = torch.autograd.grad(y, [h, w] + ([] if b is None else [b]), s["g_y"].double())
    g_x = grads[0] if s["g_h"] is None else grads[0] + s["g_h"].double()
    return (g_x, *grads[1:])


def _exact_rows(s, scale, g_lp=None):
    """Log probabilities, (maximum, sum) by rows and, with g_lp, the logits' gradient."""
    logits, targets = s["logits"], s["targets"]
    T, V = logits.shape
    lps, stats = [], []
    g_x = None if g_lp is None else torch.zeros((T, V), dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // V)
    for a in range(0, T, step):
        x = logits[a:a + step].double()
        t = targets[a:a + step]
        live = (t >= 0) & (t < V)
        lse = torch.logsumexp(scale * x, -1)
        lp = scale * x.gather(1, t.clamp(0, V - 1)[:, None])[:, 0] - lse
        lps.append(lp.masked_fill(~live, 0.0))
        m = x.amax(-1)
        row = torch.stack([m, torch.exp(lse - scale * m)], -1)
        stats.append(torch.where(live[:, None], row, row.new_tensor([0.0, 1.0])))
        if g_lp is not None:
            part = torch.softmax(scale * x, -1).neg_()
            part[torch.arange(len(t), device="cuda"), t.clamp(0, V - 1)] += 1.0
            part *= scale * g_lp[a:a + step, None]
            part[g_lp[a:a + step] == 0] = 0.0
            g_x[a:a + step] = part
    return torch.cat(lps), torch.cat(stats), g_x


def _exact_policy(s):
    c = s["case"]
    lp, _, _ = _exact_rows(s, c["scale"])
    live = s["weight"] != 0
    q = lp[live].clone().requires_grad_()
    w, A = s["weight"][live].double(), s["advantage"][live].double()
    ratio = torch.exp(q - s["old"][live].double())
    bounded = torch.clamp(ratio, 1.0 - c["clip_low"], 1.0 + c["clip_high"])
    surrogate = torch.where(bounded * A < ratio * A, bounded.detach() * A, ratio * A)
    away = s["ref"][live].double() - q
    kl = torch.expm1(away) - away if c["kl"] else torch.zeros_like(q)
    loss = (w * (c["kl"] * kl - surrogate)).sum()
    g = torch.zeros_like(lp)
    g[live] = torch.autograd.grad(loss, q)[0]
    stats = torch.stack([loss.detach(), (w * kl).sum().detach(),
                         w[bounded * A < ratio * A].sum()])
    g_x = _exact_rows(s, c["scale"], g)[2]
    return stats, torch.where(live, lp, torch.zeros_like(lp)), g_x


def _exact_preference(s):
    c, P = s["case"], s["case"]["pairs"]
    lp, _, _ = _exact_rows(s, 1.0)
    q = lp.clone().requires_grad_()
    gain = s["weight"].double() * (q - s["ref"].double())
    start = s["start"].tolist()
    score = []
    for a, b in zip(start[:-1], start[1:]):
        total = gain[a:b].sum()
        length = float(s["weight"][a:b].sum()) if c["mean"] else 1.0
        score.append(total / length if length else total)
    score = torch.stack(score)
    margin = c["beta"] * (score[:P] - score[P:])
    ls = torch.nn.functional.logsigmoid
    loss = -((1.0 - c["smoothing"]) * ls(margin) + c["smoothing"] * ls(-margin)).mean()
    g = torch.autograd.grad(loss, q)[0]
    return loss.detach().reshape(1), margin.detach(), _exact_rows(s, 1.0, g)[2]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm_forward", "norm_backward"):
        return _exact_norm(s)
    if op == "score":
        return _exact_rows(s, case["scale"])[:2]
    if op == "policy":
        return _exact_policy(s)
    if op == "preference":
        return _exact_preference(s)
    if case["norm"] == "l2":
        norm = math.sqrt(sum(float(torch.dot(d, d)) for d in
                             (v.double().flatten() for v in s["grads"])))
    else:
        norm = max(float(v.abs().max()) for v in s["grads"])
    coef = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
    types = dict.fromkeys(v.dtype for v in s["grads"])
    return (torch.tensor([norm], dtype=torch.float64, device="cuda"),
            *(torch.cat([v.double().flatten() for v in s["grads"] if v.dtype == t]) * coef
              for t in types))


# ---------------------------------------------------------------- the work

def work(case):
    op, es = case["op"], SIZE[case["dtype"]]
    if op in ("norm_forward", "norm_backward"):
        n, C, ps = case["rows"] * case["cols"], case["cols"], SIZE[case["param"]]
        params = (2 if case["bias"] else 1) * C * ps
        if op == "norm_forward":
            return dict(bytes=n * es * (4 if case["residual"] else 2) + 8 * case["rows"] + params,
                        flops=9 * n)
        return dict(bytes=n * es * (4 if case["residual"] else 3) + 8 * case["rows"] + C * ps
                    + params, flops=14 * n)
    if op == "clip":
        sizes = [(math.prod(s), es if len(s) > 1 else 4) for s in _shapes(case)]
        return dict(bytes=sum(2 * n * e for n, e in sizes), flops=sum(3 * n for n, _ in sizes))
    T, V = case["rows"], case["vocab"]
    live = T - int(T * case.get("prompt", case.get("ignored", 0.0)))
    if op == "score":
        return dict(bytes=live * V * es + 20 * T, flops=5 * live * V)
    # one read of the rows that count, one write of every row's gradient
    return dict(bytes=(live + T) * V * es + 28 * T, flops=9 * live * V)
