"""Cases, inputs and plain forms of the attention block's operators in a training
step: attention over packed sequences with its backward pass, the learned
relative position bias in its scores, and dropout in front of the residual
addition.

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


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one new token for each of eight requests against their caches
        dict(name="attention_one_token", op="attention", queries=8, keys=32700, seqs=8, ragged=True,
             heads=32, kv_heads=8, dim=128, dtype="bf16", causal=True, buckets=0),
        # ViT-B at batch 64: 197 tokens an image, packed
        dict(name="attention_vitb", op="attention", queries=12608, keys=0, seqs=64, ragged=False,
             heads=12, kv_heads=12, dim=64, dtype="bf16", causal=False, buckets=0),
        # one long sequence of a decoder with shared key and value heads
        dict(name="attention_long", op="attention", queries=8192, keys=0, seqs=1, ragged=False,
             heads=32, kv_heads=8, dim=128, dtype="bf16", causal=True, buckets=0),
        # a few ragged sequences in 32 bits, an odd head size
        dict(name="attention_odd_f32", op="attention", queries=1001, keys=0, seqs=5, ragged=True,
             heads=6, kv_heads=2, dim=72, dtype="f32", causal=True, buckets=0),
        # the backward pass of ViT-B's attention
        dict(name="attention_backward_vitb", op="attention_backward", queries=12608, keys=0, seqs=64,
             ragged=False, heads=12, kv_heads=12, dim=64, dtype="bf16", causal=False, buckets=0),
        # a step over ragged sequences packed into one batch of a decoder
        dict(name="attention_backward_ragged", op="attention_backward", queries=8192, keys=0, seqs=6,
             ragged=True, heads=32, kv_heads=8, dim=128, dtype="bf16", causal=True, buckets=0),
        # a small model in 32 bits, an odd head size
        dict(name="attention_backward_odd_f32", op="attention_backward", queries=777, keys=0, seqs=3,
             ragged=True, heads=5, kv_heads=5, dim=40, dtype="f32", causal=False, buckets=0),
        # an encoder's scores with the bias of 32 buckets, 16 texts of 512 tokens
        dict(name="bias_encoder", op="attention", queries=8192, keys=0, seqs=16, ragged=False,
             heads=12, kv_heads=12, dim=64, dtype="bf16", causal=False, buckets=32),
        # its backward pass over ragged texts, with the bias table's gradient
        dict(name="bias_backward_ragged", op="attention_backward", queries=8190, keys=0, seqs=16,
             ragged=True, heads=12, kv_heads=12, dim=64, dtype="bf16", causal=False, buckets=32),
        # a short activation of odd size: latency
        dict(name="dropout_small", op="dropout", count=4099, dtype="f32", p=0.1, residual=True),
        # what a block adds to ViT-B's residual stream at batch 64
        dict(name="dropout_vitb", op="dropout", count=12608 * 768, dtype="bf16", p=0.1, residual=True),
        # the gradient behind a decoder's wide activation
        dict(name="dropout_backward_wide", op="dropout_backward", count=8192 * 14336, dtype="bf16",
             p=0.25, residual=False),
    ]


def _log(rng, lo, hi):
    """An integer from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention_backward", "attention_backward", "dropout",
                     "dropout_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("dropout"):
        return dict(op=op, count=_log(rng, 1000, 8192 * 14336 // SIZE[dtype] * 2 - 1000), dtype=dtype,
                    p=rng.choice([0.05, 0.1, 0.5]),
                    residual=op == "dropout" and rng.random() < 0.7)
    kv_heads = rng.choice([1, 2, 4, 8, 12])
    dim = rng.choice([32, 64, 64, 128, 128, rng.randint(9, 128)])
    buckets = rng.choice([0, 0, 32, 16])
    heads = kv_heads * rng.choice([1, 1, 2, 4])
    seqs = _log(rng, 1, 48)
    # as many queries as keep the products of one pass below the largest listed case's
    most = 2.0e11 if dtype == "bf16" else 1.2e10
    if op == "attention" and rng.random() < 0.3:
        keys = _log(rng, 64 * seqs, 65536)
        return dict(op=op, queries=seqs * rng.choice([1, 1, 2, 5]), keys=keys, seqs=seqs, ragged=True,
                    heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, causal=True,
                    buckets=buckets)
    longest = int(math.sqrt(most * seqs / (4 * (heads * dim) * 3)))
    queries = _log(rng, 5 * seqs, max(5 * seqs, min(12608, longest)))
    return dict(op=op, queries=queries, keys=0, seqs=seqs, ragged=True, heads=heads,
                kv_heads=kv_heads, dim=dim, dtype=dtype, causal=rng.random() < 0.5, buckets=buckets)


def _lengths(case):
    """(queries, keys) of each sequence: equal ones, or ragged ones with a
    single token and, where there are more than four, an empty sequence."""
    Q, S = case["queries"], case["seqs"]
    r = np.random.default_rng(Q * 1009 + case["keys"] * 31 + S)

    def split(total, least):
        share = r.dirichlet(np.full(S, 4.0))
        n = np.floor(share * (total - least * S)).astype(np.int64) + least
        n[-1] += total - n.sum()
        return n

    if case["keys"]:  # new tokens against a cache: as many queries in each
        return np.full(S, Q // S), split(case["keys"], Q // S)
    if not case["ragged"]:
        return np.full(S, Q // S), np.full(S, Q // S)
    n = split(Q, 1)
    if S > 2:
        n[0] += n[1] - 1
        n[1] = 1
    if S > 4:
        n[2] += n[3]
        n[3] = 0
    return n, n


# ---------------------------------------------------------------- the inputs

REACH = 128   # distance from which the bias stays the same


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _bounds(n):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int64)).cuda()


def prepare(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    if case["op"].startswith("dropout"):
        x = _randn(g, case["count"]).to(dt)
        return dict(case=case, x=x,
                    residual=_randn(g, case["count"]).to(dt) if case["residual"] else None,
                    seed=torch.tensor([seed * 7919 + 12345, seed % 1000], device="cuda"))
    H, K, D = case["heads"], case["kv_heads"], case["dim"]
    nq, nk = _lengths(case)
    Tq, Tk = int(nq.sum()), int(nk.sum())
    s = dict(case=case, lengths=(nq.tolist(), nk.tolist()), start=_bounds(nq),
             longest=int(nq.max()), scale=1.0 / math.sqrt(D),
             bias=(0.5 * _randn(g, case["buckets"], H)) if case["buckets"] else None)
    # queries and keys share a direction, so that some scores stand out; q, k and v are
    # slices of what the qkv layer gives, or the new token's and the cache's
    if case["keys"]:
        q, kv = _randn(g, Tq, H, D), _randn(g, Tk, 2 * K, D)
        s.update(q=(1.5 * q).to(dt), start_k=_bounds(nk))
        kv = kv.to(dt)
        s.update(k=kv[:, :K], v=kv[:, K:])
        return s
    qkv = _randn(g, Tq, H + 2 * K, D)
    common = _randn(g, 1, 1, D)
    qkv[:, :H + K] += 0.7 * common * torch.randn((Tq, 1, 1), generator=g, device="cuda")
    qkv = qkv.to(dt)
    s.update(qkv=qkv, q=qkv[:, :H], k=qkv[:, H:H + K], v=qkv[:, H + K:], start_k=None)
    if case["op"] == "attention_backward":
        o, s["lse"] = _plain_forward(s)
        s["o"] = o
        s["g_o"] = (1e-2 * _randn(g, Tq, H, D)).to(dt)
    return s


# ---------------------------------------------------------------- plain forms

def _edges(side):
    """First distance of each bucket of one side (``side`` buckets, half of
    them exact, the rest spread over the logarithm up to REACH), from the
    borders' powers in whole numbers."""
    e = side // 2
    m, first = side - e, list(range(e))
    for step in range(m):
        n = e
        while n ** m * e ** step < REACH ** step * e ** m:
            n += 1
        first.append(n)
    return first


def _bucket(rel, buckets, causal):
    """Bucket of key position minus query position; one side when causal."""
    side = buckets if causal else buckets // 2
    far = -rel if causal else rel.abs()
    first = torch.tensor(_edges(side), device=rel.device)
    at = torch.searchsorted(first, far.clamp(min=0).contiguous(), right=True) - 1
    return at if causal else at + side * (rel > 0)


def _runs(s):
    """(first query, first key, count, queries, keys) of neighbouring sequences
    of equal lengths."""
    nq, nk = s["lengths"]
    a = b = i = 0
    while i < len(nq):
        n = 1
        while i + n < len(nq) and nq[i + n] == nq[i] and nk[i + n] == nk[i]:
            n += 1
        yield a, b, n, nq[i], nk[i]
        a, b, i = a + n * nq[i], b + n * nk[i], i + n


def _parts(s):
    """Pieces of the batch whose scores fit 2^27 values: ((rows, first query),
    (keys, first key), sequences, queries, keys, heads h0 .. h1)."""
    H = s["case"]["heads"]
    group = H // s["case"]["kv_heads"]
    for a, b, n, lq, lk in _runs(s):
        if not lq or not lk:
            continue
        per = max(1, (1 << 27) // (lq * lk * group))       # (sequence, kv head) pairs at once
        step = max(1, min(n, per // s["case"]["kv_heads"]))
        heads = H if per >= s["case"]["kv_heads"] else max(1, per) * group
        for i in range(0, n, step):
            c = min(step, n - i)
            for h0 in range(0, H, heads):
                yield a + i * lq, b + i * lk, c, lq, lk, h0, min(H, h0 + heads)


def _rows(t, first, n, length, h0, h1):
    """[n, heads, length, D] in 32 bits."""
    part = t[first:first + n * length, h0:h1].float()
    return part.reshape(n, length, h1 - h0, -1).permute(0, 2, 1, 3).contiguous()


def _packed(t):
    return t.permute(0, 2, 1, 3).reshape(-1, t.shape[1], t.shape[3])


def _plain_scores(s, q, k, lq, lk, h0, h1):
    """Scores in 32 bits, -inf where a key is hidden, and the bias's buckets."""
    x = (q @ k.transpose(-1, -2)) * s["scale"]
    rel = torch.arange(lk, device="cuda")[None, :] - \
        (torch.arange(lq, device="cuda")[:, None] + (lk - lq))
    bucket = None
    if s["bias"] is not None:
        line = torch.arange(-(lk - 1), lk + lq, device="cuda")
        bucket = _bucket(line, s["case"]["buckets"], s["case"]["causal"])
        x = x + s["bias"][:, h0:h1].float().t()[:, bucket[rel + lk - 1]]
    if s["case"]["causal"]:
        x = x.masked_fill(rel > 0, -math.inf)
    return x, bucket


def _plain_forward(s):
    c = s["case"]
    H, group = c["heads"], c["heads"] // c["kv_heads"]
    T, D = s["q"].shape[0], c["dim"]
    o = torch.zeros((T, H, D), dtype=s["q"].dtype, device="cuda")
    lse = torch.full((H, T), -math.inf, device="cuda")
    for a, b, n, lq, lk, h0, h1 in _parts(s):
        q = _rows(s["q"], a, n, lq, h0, h1)
        k, v = (_rows(s[x], b, n, lk, h0 // group, h1 // group).repeat_interleave(group, 1)
                for x in "kv")
        x, _ = _plain_scores(s, q, k, lq, lk, h0, h1)
        m = x.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = torch.exp(x - m)
        total = p.sum(-1, keepdim=True)
        y = (p @ v) / torch.where(total == 0, torch.ones_like(total), total)
        o[a:a + n * lq, h0:h1] = _packed(y).to(o.dtype)
        lse[h0:h1, a:a + n * lq] = (m + torch.log(total))[..., 0].permute(1, 0, 2) \
            .reshape(h1 - h0, -1)
    return o, lse


def _plain_backward(s):
    c = s["case"]
    H, K, D = c["heads"], c["kv_heads"], c["dim"]
    group, T = H // K, s["q"].shape[0]
    g_qkv = torch.zeros((T, H + 2 * K, D), dtype=s["q"].dtype, device="cuda")
    g_bias = torch.zeros((H, c["buckets"]), dtype=torch.float64, device="cuda")
    for a, b, n, lq, lk, h0, h1 in _parts(s):
        k0, k1 = h0 // group, h1 // group
        q, o, g_o = (_rows(s[x], a, n, lq, h0, h1) for x in ("q", "o", "g_o"))
        k, v = (_rows(s[x], b, n, lk, k0, k1).repeat_interleave(group, 1) for x in "kv")
        x, bucket = _plain_scores(s, q, k, lq, lk, h0, h1)
        lse = s["lse"][h0:h1, a:a + n * lq].reshape(h1 - h0, n, lq).permute(1, 0, 2)
        p = torch.exp(x - lse[..., None])
        d = p * (g_o @ v.transpose(-1, -2) - (g_o * o).sum(-1, keepdim=True))
        shared = lambda t: t.reshape(n, k1 - k0, group, lk, D).sum(2)
        g_qkv[a:a + n * lq, h0:h1] = _packed((d @ k) * s["scale"]).to(g_qkv.dtype)
        g_qkv[b:b + n * lk, H + k0:H + k1] = \
            _packed(shared(d.transpose(-1, -2) @ q) * s["scale"]).to(g_qkv.dtype)
        g_qkv[b:b + n * lk, H + K + k0:H + K + k1] = \
            _packed(shared(p.transpose(-1, -2) @ g_o)).to(g_qkv.dtype)
        if bucket is not None:
            # row i of the reversed queries moved right by i: equal distances share a column
            wide = torch.nn.functional.pad(d.sum(0).flip(1), (0, lq))
            wide = wide.reshape(h1 - h0, -1)[:, :lq * (lk + lq - 1)]
            line = wide.reshape(h1 - h0, lq, lk + lq - 1).sum(1, dtype=torch.float64)
            # column c: distance c - (lq - 1) - (lk - lq) = c - (lk - 1)
            which = bucket[:lk + lq - 1]
            one = which[:, None] == torch.arange(c["buckets"], device="cuda")
            g_bias[h0:h1] += (line[:, :, None] * one).sum(1)
    return (g_qkv,) if s["bias"] is None else (g_qkv, g_bias.t().to(s["bias"].dtype))


def _plain_random(count, seed, site):
    """16 random bits for each element: Philox 4x32 of seven rounds (Salmon,
    Moraes, Dror, Shaw 2011) of the counter (block of eight elements, site,
    step) under the key."""
    n = (count + 7) // 8
    low = 0xFFFFFFFF
    key, step = seed[0], seed[1]
    c = [torch.arange(n, device="cuda"), torch.full((n,), site, device="cuda"),
         (step & low).expand(n), ((step >> 32) & low).expand(n)]
    k0, k1 = key & low, (key >> 32) & low
    for _ in range(7):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57    # the low 64 bits of each product
        c = [((q >> 32) & low) ^ c[1] ^ k0, q & low, ((p >> 32) & low) ^ c[3] ^ k1, p & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack(c, 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:count]


def _plain_dropout(s):
    c = s["case"]
    out = torch.empty_like(s["x"])
    limit = round(c["p"] * 65536)
    r = _plain_random(c["count"], s["seed"], 3)
    y = torch.where(r >= limit, s["x"].float() * (65536 / (65536 - limit)), torch.zeros((), device="cuda"))
    if s["residual"] is not None:
        y = s["residual"].float() + y
    return out.copy_(y)


def _plain(s):
    op = s["case"]["op"]
    if op == "attention":
        return _plain_forward(s)
    if op == "attention_backward":
        return _plain_backward(s)
    return _plain_dropout(s)


# ---------------------------------------------------------------- the framework's calls

def _framework(s):
    import hadamard_rank_linear_amd as h
    c = s["case"]
    op = c["op"]
    if op == "dropout":
        return h.hlq_dropout_forward(s["x"], c["p"], s["seed"], site=3, residual=s["residual"])
    if op == "dropout_backward":
        return h.hlq_dropout_backward(s["x"], c["p"], s["seed"], site=3)
    bias = {} if s["bias"] is None else dict(bias=s["bias"], max_distance=REACH,
                                             bidirectional=not c["causal"])
    if op == "attention":
        return h.hlq_attention_forward(s["q"], s["k"], s["v"], s["start"], s["start_k"],
                                       causal=c["causal"], scale=s["scale"], max_len=s["longest"],
                                       **bias)
    H, K = c["heads"], c["kv_heads"]
    g_qkv = torch.empty_like(s["qkv"])
    g_bias = h.hlq_attention_backward(s["g_o"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["start"],
                                      s["start_k"], causal=c["causal"], scale=s["scale"],
                                      max_len=s["longest"], g_q=g_qkv[:, :H], g_k=g_qkv[:, H:H + K],
                                      g_v=g_qkv[:, H + K:], **bias)[3]
    return (g_qkv,) if s["bias"] is None else (g_qkv, g_bias)


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------- in 64 bits

def _exact_bucket(d, buckets, one_sided):
    """The definition, for one distance."""
    side = buckets if one_sided else buckets // 2
    n = max(-d, 0) if one_sided else abs(d)
    e = side // 2
    if n >= e:
        share = math.log(n / e) / math.log(REACH / e)
        # 1e-9: distances whose share is a whole number belong to the bucket they begin
        n = min(side - 1, e + math.floor((side - e) * share + 1e-9))
    return n + (side if not one_sided and d > 0 else 0)


def _exact_attention(s):
    c = s["case"]
    H, K, B = c["heads"], c["kv_heads"], c["buckets"]
    backward = c["op"] == "attention_backward"
    T, TK = s["q"].shape[0], s["k"].shape[0]
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")
    o, lse = new(T, H, c["dim"]), torch.full((H, T), -math.inf, dtype=torch.float64, device="cuda")
    g_q, g_k, g_v = new(T, H, c["dim"]), new(TK, K, c["dim"]), new(TK, K, c["dim"])
    g_bias = new(max(B, 1), H)
    i0 = j0 = 0
    for lq, lk in zip(*s["lengths"]):
        rows, cols = slice(i0, i0 + lq), slice(j0, j0 + lk)
        i0, j0 = i0 + lq, j0 + lk
        if not lq or not lk:
            continue
        at = torch.arange(lq, device="cuda") + lk - lq
        hidden = torch.arange(lk, device="cuda") > at[:, None] if c["causal"] else None
        if B:
            # distances of every row from the last key down: a window that slides over the line
            line = torch.tensor([_exact_bucket(d, B, c["causal"]) for d in range(-lk + 1, lk + lq)],
                                device="cuda")
            which = line.unfold(0, lk, 1)[:lq].flip(0)     # row i: distances j - at_i
        for h in range(H):
            q, k, v = (x.double() for x in (s["q"][rows, h], s["k"][cols, h * K // H],
                                            s["v"][cols, h * K // H]))
            x = torch.addmm(s["bias"].double()[which, h] if B else q.new_zeros(()), q, k.t(),
                            alpha=s["scale"])
            if hidden is not None:
                x[hidden] = -math.inf
            if not backward:
                lse[h, rows] = torch.logsumexp(x, -1)
                o[rows, h] = torch.nan_to_num(torch.softmax(x, -1)) @ v
                continue
            p = (x - s["lse"][h, rows].double()[:, None]).exp_()
            g = s["g_o"][rows, h].double()
            g_v[cols, h * K // H] += p.t() @ g
            p *= torch.addmm(-(g * s["o"][rows, h].double()).sum(1, keepdim=True), g, v.t())
            g_q[rows, h] = s["scale"] * (p @ k)
            g_k[cols, h * K // H] += s["scale"] * (p.t() @ q)
            if B:
                for b in range(B):
                    g_bias[b, h] += p[which == b].sum()
    if not backward:
        return o, lse
    return (torch.cat([g_q, g_k, g_v], 1), *([g_bias] if B else []))


def _exact_random(count, key, step, site):
    """The generator in unsigned 64-bit arithmetic of the host."""
    u = lambda v: np.uint64(v & 0xFFFFFFFF)
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    n = (count + 7) // 8
    a = np.arange(n, dtype=np.uint64)
    b, c, d = (np.full(n, u(w)) for w in (site, step, step >> 32))
    x, y = key & 0xFFFFFFFF, key >> 32 & 0xFFFFFFFF
    for r in range(7):
        left, right = a * np.uint64(0xD2511F53), c * np.uint64(0xCD9E8D57)
        a, b, c, d = ((right >> half) ^ b ^ u(x + r * 0x9E3779B9), right & low,
                      (left >> half) ^ d ^ u(y + r * 0xBB67AE85), left & low)
    out = np.empty((n, 4, 2), np.uint16)
    for i, w in enumerate((a, b, c, d)):
        out[:, i, 0], out[:, i, 1] = w & np.uint64(0xFFFF), w >> np.uint64(16)
    return out.reshape(-1)[:count]


def exact(case, seed):
    s = prepare(case, seed)
    if not case["op"].startswith("dropout"):
        return _exact_attention(s)
    key, step = s["seed"].tolist()
    limit = round(case["p"] * 65536)
    keep = torch.from_numpy(_exact_random(case["count"], key, step, 3) >= limit).cuda()
    y = s["x"].double() * keep / (1.0 - limit / 65536.0)
    return y if s["residual"] is None else y + s["residual"].double()


# ---------------------------------------------------------------- the work

def work(case):
    es = SIZE[case["dtype"]]
    if case["op"].startswith("dropout"):
        return dict(bytes=case["count"] * es * (3 if case["residual"] else 2),
                    flops=3 * case["count"])
    nq, nk = _lengths(case)
    H, K, D = case["heads"], case["kv_heads"], case["dim"]
    # visible pairs: all of them, or for the last lq of lk positions what lies before
    hidden = nq * (nq - 1) // 2 if case["causal"] else 0
    pairs = int((nq * nk - hidden).sum())
    q, kv = int(nq.sum()) * H * D * es, int(nk.sum()) * K * D * es
    lse, table = 4 * H * int(nq.sum()), 4 * case["buckets"] * H
    if case["op"] == "attention":
        return dict(bytes=2 * q + 2 * kv + lse + table, flops=4 * D * H * pairs)
    # q, o, g_o and k, v read, their gradients written
    return dict(bytes=4 * q + 4 * kv + lse + 2 * table, flops=10 * D * H * pairs)
