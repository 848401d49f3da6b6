"""PyTorch autograd wrapper: a linear layer y = x . w^T whose backward is the
HLQ/HOT backward of libhlq.so.

"HOT: Hadamard-based Optimized Training" (scime.ai summary, "Approach"): the
stored activation is compressed at forward time (activation buffer
compression), and the backward runs Hadamard quantization on g_x and Hadamard
low-rank approximation plus INT8 on g_w.  The forward product itself is
unchanged by the method; what this wrapper keeps for the backward is the ACBP
form of x (INT4 codes + one fp32 scale per token) instead of x, and its
backward is one ``hlq_linear_backward`` call.  For bf16 x and w with I a
multiple of 32 the forward is one ``hlq_linear_forward`` launch (the bf16
MFMA product with the codes of x emitted by the same launch); otherwise
torch's matmul and ``hlq_compress_act``.  Leading dimensions of x are
flattened into tokens.  No bias (its gradient is not part of the method).

Around it, the operators of a training step in the same form: the layer norm
with its residual addition (:class:`HLQLayerNorm`), token log probabilities,
the policy and preference losses on them, and the clipping of gradients; and
those of an attention block: attention over packed sequences with a relative
position bias (:class:`HLQSelfAttention` between two HLQ linear layers), and
dropout with the residual addition (:class:`HLQDropout`).
"""
from __future__ import annotations

import torch

from . import hlq


class HLQLinearFunction(torch.autograd.Function):
    """y = x . w^T; backward by ``hlq_linear_backward`` on the ACBP codes of x."""

    @staticmethod
    def forward(ctx, x, w, block, rank, gx_mode, gw_mode, reduction):
        if x.shape[-1] != w.shape[1]:
            raise ValueError("x [..., I] and w [O, I] disagree on I")
        x2 = x.reshape(-1, x.shape[-1]).contiguous()
        if x2.dtype == torch.bfloat16 and w.dtype == torch.bfloat16 and x2.shape[1] % 32 == 0:
            y, codes, scales = hlq.hlq_linear_forward(x2, w.contiguous())
        else:
            y = x2 @ w.t()
            codes, scales = hlq.hlq_compress_act(x2)
        ctx.save_for_backward(codes, scales, w)
        ctx.cfg = (block, rank, gx_mode, gw_mode, reduction)
        ctx.x_shape, ctx.x_dtype = x.shape, x.dtype
        return y.reshape(*x.shape[:-1], w.shape[0])

    @staticmethod
    def backward(ctx, g_y):
        codes, scales, w = ctx.saved_tensors
        block, rank, gx_mode, gw_mode, reduction = ctx.cfg
        gy2 = g_y.reshape(-1, g_y.shape[-1])
        if gy2.dtype != w.dtype:
            gy2 = gy2.to(w.dtype)
        gy2 = gy2.contiguous()
        g_x, g_w = hlq.hlq_linear_backward(gy2, codes, scales, w.contiguous(), block, rank,
                                           gx_mode, gw_mode, reduction)
        g_x = g_x.reshape(ctx.x_shape).to(ctx.x_dtype) if ctx.needs_input_grad[0] else None
        g_w = g_w.to(w.dtype) if ctx.needs_input_grad[1] else None
        return g_x, g_w, None, None, None, None, None


def hlq_linear(x, w, block, rank, gx_mode=hlq.HLQ_PER_TOKEN, gw_mode=hlq.HLQ_PER_TOKEN,
               reduction=hlq.HLQ_SUM):
    """Functional form of :class:`HLQLinear`."""
    return HLQLinearFunction.apply(x, w, block, rank, gx_mode, gw_mode, reduction)


class HLQLinear(torch.nn.Module):
    """Bias-free linear layer (weight [out_features, in_features]) trained with
    the HLQ/HOT backward.  ``block`` and ``rank`` are the Hadamard block and the
    low-rank r of the g_w path; the token count of every batch must be a
    multiple of ``block``, and out_features too."""

    def __init__(self, in_features, out_features, block=16, rank=8,
                 gx_mode=hlq.HLQ_PER_TOKEN, gw_mode=hlq.HLQ_PER_TOKEN, reduction=hlq.HLQ_SUM,
                 device=None, dtype=None):
        super().__init__()
        self.weight = torch.nn.Parameter(
            torch.empty((out_features, in_features), device=device, dtype=dtype))
        torch.nn.init.kaiming_uniform_(self.weight, a=5 ** 0.5)
        self.block, self.rank = block, rank
        self.gx_mode, self.gw_mode, self.reduction = gx_mode, gw_mode, reduction

    def forward(self, x):
        return hlq_linear(x, self.weight, self.block, self.rank, self.gx_mode, self.gw_mode,
                          self.reduction)

    def extra_repr(self):
        return (f"in_features={self.weight.shape[1]}, out_features={self.weight.shape[0]}, "
                f"block={self.block}, rank={self.rank}, gx_mode={self.gx_mode}, "
                f"gw_mode={self.gw_mode}")


class HLQLayerNormFunction(torch.autograd.Function):
    """(y, h): h = x + residual, y its layer norm; both have gradients."""

    @staticmethod
    def forward(ctx, x, residual, weight, bias, eps):
        ctx.set_materialize_grads(False)
        y, h, mean, rstd = hlq.hlq_layer_norm_forward(
            x.contiguous(), weight.contiguous(), None if bias is None else bias.contiguous(), eps,
            residual=None if residual is None else residual.contiguous())
        ctx.save_for_backward(h, mean, rstd, weight)
        ctx.with_bias, ctx.with_residual = bias is not None, residual is not None
        return (y, h) if residual is not None else y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_y, g_h=None):
        h, mean, rstd, weight = ctx.saved_tensors
        if g_y is None:  # only h was used
            return g_h, g_h, None, None, None
        g_x, g_w, g_b = hlq.hlq_layer_norm_backward(
            g_y.contiguous(), h, mean, rstd, weight.contiguous(),
            g_h=None if g_h is None else g_h.contiguous(), with_bias=ctx.with_bias)
        return g_x, (g_x if ctx.with_residual else None), g_w, g_b, None


def hlq_layer_norm(x, weight, bias=None, eps=1e-5, residual=None):
    """Layer norm over the last dimension; with ``residual`` returns (y, h), h
    = x + residual being what the residual stream carries on."""
    return HLQLayerNormFunction.apply(x, residual, weight, bias, eps)


class HLQLayerNorm(torch.nn.Module):
    """Layer norm of the last dimension (fp32 parameters unless ``dtype`` says
    otherwise); called with a residual it returns (norm of the sum, sum)."""

    def __init__(self, features, eps=1e-5, bias=True, device=None, dtype=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(features, device=device, dtype=dtype)) \
            if bias else None

    def forward(self, x, residual=None):
        return hlq_layer_norm(x, self.weight, self.bias, self.eps, residual)

    def extra_repr(self):
        return f"features={self.weight.shape[0]}, eps={self.eps}, bias={self.bias is not None}"


class HLQTokenLogprobFunction(torch.autograd.Function):
    """Log probabilities [T] of targets under logits [T, V]."""

    @staticmethod
    def forward(ctx, logits, targets, scale):
        logprob, stats = hlq.hlq_token_logprob_forward(logits, targets, scale)
        ctx.save_for_backward(logits, targets, stats)
        ctx.scale = scale
        return logprob

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_logprob):
        logits, targets, stats = ctx.saved_tensors
        return hlq.hlq_token_logprob_backward(g_logprob.contiguous(), logits, targets, stats,
                                              ctx.scale), None, None


def hlq_token_logprob(logits, targets, scale=1.0):
    """Differentiable log probability of each target (fp32 [T]), 0 for targets
    outside [0, V), which the losses below count unless their weight is 0."""
    return HLQTokenLogprobFunction.apply(logits, targets, scale)


class HLQPolicyLossFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logprob, old_logprob, advantage, weight, ref_logprob, clip_low, clip_high,
                kl_coef):
        sums, g = hlq.hlq_policy_loss(logprob.contiguous(), old_logprob, advantage, weight,
                                      ref_logprob, clip_low, clip_high, kl_coef)
        ctx.save_for_backward(g)
        loss, kl, clipped = (v.clone() for v in sums.unbind())
        ctx.mark_non_differentiable(kl, clipped)
        return loss, kl, clipped

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_loss, _g_kl, _g_clipped):
        return ctx.saved_tensors[0] * g_loss, *(None,) * 7


def hlq_policy_loss(logprob, old_logprob, advantage, weight=None, ref_logprob=None, clip_low=0.2,
                    clip_high=0.2, kl_coef=0.0):
    """(loss, weighted KL estimate, weight of the clipped tokens), the loss
    differentiable in ``logprob``.  ``hlq.hlq_policy_loss_logits`` gives the
    loss and the gradient of the logits in one pass, for
    ``logits.backward(g_x)``."""
    return HLQPolicyLossFunction.apply(logprob, old_logprob, advantage, weight, ref_logprob,
                                       clip_low, clip_high, kl_coef)


class HLQPreferenceLossFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logprob, start, beta, ref_logprob, weight, label_smoothing, reduction):
        loss, margin, g = hlq.hlq_preference_loss(logprob.contiguous(), start, beta, ref_logprob,
                                                  weight, label_smoothing, reduction)
        ctx.save_for_backward(g)
        ctx.mark_non_differentiable(margin)
        return loss.reshape(()), margin

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_loss, _g_margin):
        return ctx.saved_tensors[0] * g_loss, *(None,) * 6


def hlq_preference_loss(logprob, start, beta, ref_logprob=None, weight=None, label_smoothing=0.0,
                        reduction=hlq.HLQ_SUM):
    """(loss, margin [P]), the loss differentiable in ``logprob``."""
    return HLQPreferenceLossFunction.apply(logprob, start, beta, ref_logprob, weight,
                                           label_smoothing, reduction)


def hlq_clip_grad_norm_(parameters, max_norm, norm_kind=hlq.HLQ_NORM_L2):
    """Clips the gradients of ``parameters`` in place by their global norm;
    returns the norm (float64 [1], on the GPU).  Parameters without a gradient
    are left out."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    return hlq.hlq_clip_grad_norm([p.grad for p in parameters if p.grad is not None], max_norm,
                                  norm_kind)


def _rows_dense(t):
    return t if t.dim() == 0 or t.shape[-1] <= 1 or t.stride(-1) == 1 else t.contiguous()


class HLQAttentionFunction(torch.autograd.Function):
    """Attention over packed sequences; gradients of q, k, v and the bias table."""

    @staticmethod
    def forward(ctx, q, k, v, start, start_k, bias, causal, scale, max_distance, bidirectional,
                max_len):
        q, k, v = _rows_dense(q), _rows_dense(k), _rows_dense(v)
        bias = None if bias is None else bias.contiguous()
        ctx.kw = dict(causal=causal, scale=scale, max_distance=max_distance,
                      bidirectional=bidirectional, max_len=max_len)
        o, lse = hlq.hlq_attention_forward(q, k, v, start, start_k, bias=bias, **ctx.kw)
        ctx.save_for_backward(q, k, v, o, lse, start, start_k, bias)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_o):
        q, k, v, o, lse, start, start_k, bias = ctx.saved_tensors
        g_q, g_k, g_v, g_bias = hlq.hlq_attention_backward(
            _rows_dense(g_o), q, k, v, o, lse, start, start_k, bias=bias, **ctx.kw)
        return g_q, g_k, g_v, None, None, g_bias, *(None,) * 5


def hlq_attention(q, k, v, start=None, start_k=None, causal=False, scale=None, bias=None,
                  max_distance=128, bidirectional=None, max_len=0):
    """Differentiable :func:`hlq.hlq_attention_forward`: o [queries, heads, D]."""
    return HLQAttentionFunction.apply(q, k, v, start, start_k, bias, causal, scale, max_distance,
                                      bidirectional, max_len)


class HLQPackedAttentionFunction(torch.autograd.Function):
    """Self-attention on what a qkv layer writes, [tokens, heads + 2 kv_heads, D];
    the gradient comes as one tensor, no sum of slices' gradients."""

    @staticmethod
    def forward(ctx, qkv, heads, start, bias, causal, scale, max_distance, bidirectional, max_len):
        kv = (qkv.shape[1] - heads) // 2 if qkv.dim() == 3 else 0
        if heads < 1 or kv < 1 or qkv.shape[1] != heads + 2 * kv:
            raise ValueError("qkv must be [tokens, heads + 2 kv_heads, D]")
        qkv = _rows_dense(qkv)
        bias = None if bias is None else bias.contiguous()
        ctx.cuts = (heads, kv, kv)
        ctx.kw = dict(causal=causal, scale=scale, max_distance=max_distance,
                      bidirectional=bidirectional, max_len=max_len)
        o, lse = hlq.hlq_attention_forward(*qkv.split(ctx.cuts, 1), start, bias=bias, **ctx.kw)
        ctx.save_for_backward(qkv, o, lse, start, bias)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_o):
        qkv, o, lse, start, bias = ctx.saved_tensors
        g_qkv = torch.empty(qkv.shape, dtype=qkv.dtype, device=qkv.device)
        g_q, g_k, g_v = g_qkv.split(ctx.cuts, 1)
        g_bias = hlq.hlq_attention_backward(
            _rows_dense(g_o), *qkv.split(ctx.cuts, 1), o, lse, start, bias=bias, **ctx.kw, g_q=g_q,
            g_k=g_k, g_v=g_v)[3]
        return g_qkv, None, None, g_bias, *(None,) * 5


def hlq_packed_attention(qkv, heads, start=None, causal=False, scale=None, bias=None,
                         max_distance=128, bidirectional=None, max_len=0):
    """Differentiable self-attention on the slices of ``qkv`` [tokens, heads + 2
    kv_heads, D]: o [tokens, heads, D]."""
    return HLQPackedAttentionFunction.apply(qkv, heads, start, bias, causal, scale, max_distance,
                                            bidirectional, max_len)


class HLQSelfAttention(torch.nn.Module):
    """Self-attention over packed sequences between two :class:`HLQLinear` layers:
    x [tokens, features] -> [tokens, features].  ``buckets`` of a learned
    relative position bias (0: none).  The token count has to suit the linear
    layers (a multiple of ``block``); sequences end where ``start`` says."""

    def __init__(self, features, heads, kv_heads=None, causal=False, buckets=0, max_distance=128,
                 block=16, rank=8, device=None, dtype=None):
        super().__init__()
        kv_heads = heads if kv_heads is None else kv_heads
        if features % heads or heads % kv_heads:
            raise ValueError("features must be a multiple of heads, heads of kv_heads")
        self.heads, self.kv_heads, self.dim = heads, kv_heads, features // heads
        self.causal, self.max_distance = causal, max_distance
        self.qkv = HLQLinear(features, (heads + 2 * kv_heads) * self.dim, block, rank, device=device,
                             dtype=dtype)
        self.out = HLQLinear(features, features, block, rank, device=device, dtype=dtype)
        self.bias = torch.nn.Parameter(torch.zeros((buckets, heads), device=device)) \
            if buckets else None

    def forward(self, x, start=None, max_len=0):
        qkv = self.qkv(x).view(x.shape[0], self.heads + 2 * self.kv_heads, self.dim)
        o = hlq_packed_attention(qkv, self.heads, start, self.causal, bias=self.bias,
                                 max_distance=self.max_distance, max_len=max_len)
        return self.out(o.view(x.shape[0], -1))

    def extra_repr(self):
        return (f"heads={self.heads}, kv_heads={self.kv_heads}, dim={self.dim}, "
                f"causal={self.causal}, buckets={0 if self.bias is None else len(self.bias)}")


class HLQDropoutFunction(torch.autograd.Function):
    """residual + dropout(x); the backward pass draws the mask again."""

    @staticmethod
    def forward(ctx, x, residual, p, seed, site):
        ctx.p, ctx.site, ctx.with_residual = p, site, residual is not None
        ctx.save_for_backward(seed)
        return hlq.hlq_dropout_forward(x.contiguous(), p, seed, site,
                                       None if residual is None else residual.contiguous())

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_y):
        seed, = ctx.saved_tensors
        g_x = hlq.hlq_dropout_backward(g_y.contiguous(), ctx.p, seed, ctx.site) \
            if ctx.needs_input_grad[0] else None
        return g_x, (g_y if ctx.with_residual else None), None, None, None


def hlq_dropout(x, p, seed, site=0, residual=None):
    """residual + dropout(x).  ``seed`` (int64 [2] on the GPU) must not move on
    before the backward pass has drawn the mask again: autograd raises if it was
    changed in place."""
    return HLQDropoutFunction.apply(x, residual, p, seed, site)


class HLQDropout(torch.nn.Module):
    """Dropout in front of a residual addition: called with (x, seed, residual).
    ``site`` tells the places of a model apart that share a seed.  In evaluation
    nothing is dropped."""

    def __init__(self, p=0.1, site=0):
        super().__init__()
        self.p, self.site = p, site

    def forward(self, x, seed, residual=None):
        if self.training:
            return hlq_dropout(x, self.p, seed, self.site, residual)
        return x if residual is None else residual + x

    def extra_repr(self):
        return f"p={self.p}, site={self.site}"
