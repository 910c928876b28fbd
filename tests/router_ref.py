"""The router, its balance losses and its gradient in 64 bits, from the
definitions in include/ep_router.h, on the CPU (torch.float64, one token or
one sequence at a time where that is the plain way to say it)."""
from __future__ import annotations

import math

import torch

F32_MAX = torch.finfo(torch.float32).max


def clean(logits: torch.Tensor) -> torch.Tensor:
    l = logits.double()
    l = torch.where(torch.isnan(l), torch.full_like(l, -math.inf), l)
    return l.clamp(max=F32_MAX)


def scores(l: torch.Tensor, sigmoid: bool) -> torch.Tensor:
    """s of cleaned logits; closed experts 0."""
    closed = torch.isneginf(l)
    if sigmoid:
        s = torch.sigmoid(torch.where(closed, torch.zeros_like(l), l))
    else:
        s = torch.softmax(torch.where(closed.all(dim=1, keepdim=True), torch.zeros_like(l), l), dim=1)
    return torch.where(closed, torch.zeros_like(s), s)


def topk(logits, K, sigmoid=False, bias=None, groups=1, topk_groups=1, group_top=1, normalize=True, scale=1.0,
         mask=None):
    l = clean(logits)
    T, E = l.shape
    s = scores(l, sigmoid)
    c = l.clone() if bias is None and groups == 1 else s + (0 if bias is None else bias.double())
    c[torch.isneginf(l) | torch.isnan(c)] = -math.inf
    idx = torch.full((T, K), -1, dtype=torch.int64)
    w = torch.zeros((T, K), dtype=torch.float64)
    per = E // groups
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        row = c[t].tolist()
        if groups > 1:
            value = []
            for g in range(groups):
                best = sorted((v for v in row[g * per:(g + 1) * per] if v > -math.inf), reverse=True)[:group_top]
                value.append(sum(best) if best else -math.inf)
            keep = sorted(range(groups), key=lambda g: (-value[g], g))[:topk_groups]
            row = [v if e // per in keep else -math.inf for e, v in enumerate(row)]
        order = [e for e in sorted(range(E), key=lambda e: (-row[e], e)) if row[e] > -math.inf][:K]
        idx[t, :len(order)] = torch.tensor(order, dtype=torch.int64)
        if order:
            lo = l[t, order]
            if normalize and sigmoid:  # ratios of sigmoids, without underflow
                ls = torch.nn.functional.logsigmoid(lo)
                w[t, :len(order)] = torch.softmax(ls, dim=0)
            elif normalize:
                w[t, :len(order)] = torch.softmax(lo, dim=0)
            else:
                w[t, :len(order)] = s[t, order]
    return idx, w * scale


def spans(T, offsets):
    return [(0, T)] if offsets is None else [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]


def shares(l, sigmoid):
    """q: the scores over their sum; 0 for a row with nothing open."""
    if not sigmoid:
        return scores(l, False)
    closed = torch.isneginf(l)
    ls = torch.nn.functional.logsigmoid(torch.where(closed, torch.zeros_like(l), l))
    ls = torch.where(closed, torch.full_like(ls, -math.inf), ls)
    dead = closed.all(dim=1, keepdim=True)
    q = torch.softmax(torch.where(dead, torch.zeros_like(ls), ls), dim=1)
    return torch.where(closed, torch.zeros_like(q), q)


def balance(logits, idx, K, sigmoid=False, mask=None, offsets=None):
    """losses [S, 2], counts [S, E], seq_tokens [S], mean_scores [S, E]."""
    l = clean(logits)
    T, E = l.shape
    live = ~torch.isneginf(l).all(dim=1)
    if mask is not None:
        live &= mask.bool()
    q = shares(l, sigmoid)
    lse = torch.logsumexp(l, dim=1)
    losses, counts, tokens, means = [], [], [], []
    for a, b in spans(T, offsets):
        at = [t for t in range(a, b) if live[t]]
        n = len(at)
        count = torch.zeros(E, dtype=torch.int64)
        for t in at:
            for e in idx[t].tolist():
                if 0 <= e < E:
                    count[e] += 1
        mean = q[at].sum(dim=0) / n if n else torch.zeros(E, dtype=torch.float64)
        counts.append(count)
        tokens.append(n)
        means.append(mean)
        z = (lse[at] ** 2).sum() / n if n else torch.zeros((), dtype=torch.float64)
        bal = (count.double() * mean).sum() * E / (K * n) if n else torch.zeros((), dtype=torch.float64)
        losses.append(torch.stack([bal, z]))
    return torch.stack(losses), torch.stack(counts), torch.tensor(tokens), torch.stack(means)


def objective(l, logits, idx, K, sigmoid, normalize, scale, d_w, d_losses, mask, offsets):
    """The scalar whose gradient the backward pass returns, as a function of the
    open logits l (float64, of the shape of logits; closed places ignored)."""
    closed = torch.isneginf(clean(logits))
    l = torch.where(closed, torch.full_like(l, -math.inf), l)
    T, E = l.shape
    live = ~closed.all(dim=1)
    if mask is not None:
        live &= mask.bool()
    total = torch.zeros((), dtype=torch.float64)
    if d_w is not None:
        safe = torch.where(closed, torch.zeros_like(l), l)
        for t in range(T):
            slots = [k for k in range(K) if live[t] and 0 <= int(idx[t, k]) < E and not closed[t, int(idx[t, k])]]
            if not slots:
                continue
            at = idx[t, slots]
            if normalize:
                w = torch.softmax(torch.nn.functional.logsigmoid(safe[t, at]) if sigmoid else safe[t, at], dim=0)
            elif sigmoid:
                w = torch.sigmoid(safe[t, at])
            else:
                w = torch.exp(safe[t, at] - torch.logsumexp(l[t][~closed[t]], dim=0))
            total = total + scale * (w * d_w[t, slots].double()).sum()
    if d_losses is not None:
        _, counts, _, _ = balance(logits, idx, K, sigmoid, mask, offsets)
        for s, (a, b) in enumerate(spans(T, offsets)):
            at = [t for t in range(a, b) if live[t]]
            n = len(at)
            for t in at:
                o = ~closed[t]
                lo = l[t][o]
                q = torch.softmax(torch.nn.functional.logsigmoid(lo) if sigmoid else lo, dim=0)
                total = total + d_losses[s, 0].double() * E / (K * n) * (counts[s][o].double() * q).sum() / n
                total = total + d_losses[s, 1].double() * torch.logsumexp(lo, dim=0) ** 2 / n
    return total


def backward(logits, idx, K, sigmoid=False, normalize=True, scale=1.0, d_w=None, d_losses=None, mask=None,
             offsets=None):
    l = clean(logits)
    x = torch.where(torch.isneginf(l), torch.zeros_like(l), l).requires_grad_(True)
    total = objective(x, logits, idx, K, sigmoid, normalize, scale, d_w, d_losses, mask, offsets)
    if not total.requires_grad:
        return torch.zeros_like(l)
    return torch.autograd.grad(total, x)[0]
