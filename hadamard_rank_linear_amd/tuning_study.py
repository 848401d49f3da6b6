"""Preference tuning and policy updates of a small model whose linear layers
train with the HLQ/HOT backward, with every operator of the step from this
library: ``python -m hadamard_rank_linear_amd.tuning_study``.

The model predicts a token from the one before it: embedding, one MLP block
with its layer norm and residual addition, a last norm and a head.  With
``--heads`` an attention block comes before the MLP's: causal attention within
each sequence with a relative position bias, and dropout in front of the residual
addition.  Synthetic tasks with a known direction:

- preference: in each pair the chosen sequence counts up by one, the rejected
  one is random; the mean margin over the reference model has to grow;
- policy: tokens are sampled, an even token earns 1; the mean reward has to
  grow.  The loss and the gradient of the logits come from one call.
"""
from __future__ import annotations

import argparse

import torch

from . import hlq
from .autograd import (HLQDropout, HLQLayerNorm, HLQLinear, HLQSelfAttention, hlq_clip_grad_norm_,
                       hlq_preference_loss, hlq_token_logprob)


class TokenModel(torch.nn.Module):
    """Logits [T, vocab] of the next token for tokens [T] (T a multiple of 16).
    With ``heads``, packed sequences of the bounds ``start``; ``seed`` moves on by
    one step after each batch."""

    def __init__(self, vocab=512, width=256, inner=512, device="cuda", dtype=torch.bfloat16,
                 heads=0, dropout=0.1):
        super().__init__()
        self.embed = torch.nn.Parameter(
            torch.randn(vocab, width, device=device).mul_(0.5).to(dtype))
        self.norm = HLQLayerNorm(width, device=device)
        self.up = HLQLinear(width, inner, device=device, dtype=dtype)
        self.down = HLQLinear(inner, width, device=device, dtype=dtype)
        self.last = HLQLayerNorm(width, device=device)
        self.head = HLQLinear(width, vocab, device=device, dtype=dtype)
        self.attention = None
        if heads:
            self.first = HLQLayerNorm(width, device=device)
            self.attention = HLQSelfAttention(width, heads, max(1, heads // 2), causal=True,
                                              buckets=16, max_distance=64, device=device, dtype=dtype)
            self.drop = HLQDropout(dropout, site=1)
            self.register_buffer("seed", torch.tensor([1234, 0], device=device))

    def forward(self, tokens, start=None):
        x = self.embed[tokens]
        if self.attention is not None:
            x = self.drop(self.attention(self.first(x), start), self.seed, residual=x)
        f = self.down(torch.nn.functional.gelu(self.up(self.norm(x))))
        y, _ = self.last(f, residual=x)
        return self.head(y)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def preference_pairs(pairs, length, vocab, seed):
    """(inputs [T], targets [T], start [2P + 1]): P counting sequences, then P
    random ones, ``length`` tokens each; the first target of each is ignored
    as its prompt."""
    g = _generator(seed)
    first = torch.randint(0, vocab, (pairs, 1), generator=g, device="cuda")
    chosen = (first + torch.arange(length + 1, device="cuda")) % vocab
    rejected = torch.randint(0, vocab, (pairs, length + 1), generator=g, device="cuda")
    rejected[:, :1] = first
    rows = torch.cat([chosen, rejected])
    targets = rows[:, 1:].clone()
    targets[:, 0] = -100
    start = torch.arange(2 * pairs + 1, device="cuda") * length
    return rows[:, :-1].reshape(-1), targets.reshape(-1), start


def _update(model, lr, max_norm):
    norm = hlq_clip_grad_norm_(model.parameters(), max_norm)
    with torch.no_grad():
        for p in model.parameters():
            if p.grad is not None:
                p.add_(p.grad, alpha=-lr)
                p.grad = None
    return norm


def _next_masks(model):
    """Once per batch, whose updates are compared with its rollout under one mask."""
    if model.attention is not None:
        model.seed[1] += 1


def tune_preferences(steps=20, pairs=16, length=32, vocab=512, lr=0.2, beta=0.1, seed=0, log=None,
                     heads=0):
    """Mean margin before and after ``steps`` steps of preference tuning."""
    torch.manual_seed(seed)
    model = TokenModel(vocab, heads=heads)
    margins = []
    for step in range(steps):
        inputs, targets, start = preference_pairs(pairs, length, vocab, seed)
        logits = model(inputs, start)
        logprob = hlq_token_logprob(logits, targets)
        if step == 0:
            ref = logprob.detach().clone()
        loss, margin = hlq_preference_loss(logprob, start, beta, ref,
                                           weight=(targets >= 0).float())
        loss.backward()
        norm = _update(model, lr, max_norm=1.0)
        _next_masks(model)
        margins.append(margin.mean())
        if log:
            log(f"preference step {step:3d} loss {loss.item():.4f} margin "
                f"{margins[-1].item():+.4f} gradient norm {norm.item():.3f}")
    return margins[0].item(), margins[-1].item()


def tune_policy(steps=20, tokens=1024, vocab=512, lr=0.5, updates=2, seed=0, log=None, heads=0):
    """Mean reward of the first and of the last batch of ``steps``.  With
    ``heads`` the tokens are sequences of 16."""
    torch.manual_seed(seed)
    g = _generator(seed)
    model = TokenModel(vocab, heads=heads)
    start = torch.arange(tokens // 16 + 1, device="cuda") * 16
    rewards = []
    for step in range(steps):
        inputs = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        with torch.no_grad():
            logits = model(inputs, start)
            actions = torch.multinomial(torch.softmax(logits.float(), -1), 1, generator=g)[:, 0]
            old = hlq.hlq_token_logprob_forward(logits, actions)[0]
        reward = (actions % 2 == 0).float()
        advantage = (reward - reward.mean()) / (reward.std() + 1e-6)
        weight = torch.full_like(reward, 1.0 / tokens)
        for _ in range(updates):
            logits = model(inputs, start)
            sums, _, g_x = hlq.hlq_policy_loss_logits(logits.detach(), actions, old, advantage,
                                                      weight, ref_logprob=old, clip_high=0.28,
                                                      kl_coef=0.01)
            logits.backward(g_x)
            norm = _update(model, lr, max_norm=1.0)
        _next_masks(model)
        rewards.append(reward.mean())
        if log:
            log(f"policy step {step:3d} loss {sums[0].item():+.4f} KL {sums[1].item():.5f} clipped "
                f"{sums[2].item():.3f} reward {rewards[-1].item():.3f} gradient norm "
                f"{norm.item():.3f}")
    return rewards[0].item(), rewards[-1].item()


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--seed", type=int, default=0)
    p.add_argument("--heads", type=int, default=0, help="query heads of an attention block (0: none)")
    args = p.parse_args()
    say = lambda m: print(m, flush=True)
    a, b = tune_preferences(args.steps, seed=args.seed, log=say, heads=args.heads)
    c, d = tune_policy(args.steps, seed=args.seed, log=say, heads=args.heads)
    say(f"mean margin {a:+.4f} -> {b:+.4f}, mean reward {c:.3f} -> {d:.3f}")


if __name__ == "__main__":
    main()
