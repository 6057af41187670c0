"""Plain CPU oracle for layers of experts and for log probabilities: routing with
its plan, the products of experts from packed weights, their weighted sum, norms of
query and key heads, log probabilities with entropy and top tokens.

TEST INFRASTRUCTURE ONLY, like qlin_oracle: nothing in the product path imports it,
and it shares no code with the CUDA library.  Everything is float64.
"""

from __future__ import annotations

import numpy as np


def route(logits, top_k, scoring="softmax", bias=None, groups=1, top_groups=1,
          group_score="max", renormalise=True, scale=1.0):
    """One row: (experts, weights, margin).  margin: the least difference between two
    choices or groups on which the result depends (infinity: none)."""
    x = np.array(logits, np.float64)
    x[np.isnan(x)] = -np.inf
    ok = x > -np.inf
    n = x.size
    experts, weights = np.full(top_k, -1), np.zeros(top_k)
    if not ok.any():
        return experts, weights, np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.where(x == x.max(), 1.0, np.exp(x - x.max()))
        e = np.where(ok, e, 0.0)
        score = e / e.sum() if scoring == "softmax" else 1 / (1 + np.exp(-x))
    part = score if scoring == "sigmoid" else e
    choice = x if bias is None else score + np.asarray(bias, np.float64)
    margin = np.inf

    def order(v):
        return np.argsort(-v, kind="stable")

    def gap(v, k):
        """The least difference between neighbours among the k + 1 first of a sorted v."""
        v = v[: k + 1]
        v = v[np.isfinite(v)]
        d = -np.diff(v)
        return d[d > 0].min() if (d > 0).any() else np.inf

    if groups > 1:
        size = n // groups
        values = []
        for g in range(groups):
            at = slice(g * size, (g + 1) * size)
            two = group_score == "top2"
            v = np.sort((part if two and bias is None else choice)[at][ok[at]])[::-1]
            values.append(-np.inf if not v.size else v[0] if not two or v.size < 2
                          else v[0] + v[1])
        values = np.array(values)
        best = order(values)
        if top_groups < groups:
            a, b = values[best[top_groups - 1]], values[best[top_groups]]
            if a > b:
                margin = min(margin, a - b)
        kept = np.zeros(groups, bool)
        kept[best[:top_groups]] = True
        ok = ok & np.repeat(kept, size)
    choice = np.where(ok, choice, -np.inf)
    best = order(choice)
    margin = min(margin, gap(choice[best], top_k))
    for j in range(min(top_k, int(ok.sum()))):
        experts[j], weights[j] = best[j], score[best[j]]
    if renormalise and weights.sum() > 0:
        weights = weights / weights.sum()
    return experts, weights * scale, margin


def plan(experts, n_experts):
    """order and offsets of experts [T, top_k]."""
    flat = np.where(experts < 0, n_experts, experts).reshape(-1)
    order = np.argsort(flat, kind="stable")
    offsets = np.array([(flat < e).sum() for e in range(n_experts + 1)])
    return order, offsets


def combine(y, experts, weights, add=None):
    """(out, sum of magnitudes) of y [T, top_k, N]."""
    there = (experts >= 0)[..., None]
    part = np.where(there, np.where(there, y, 0) * weights[..., None], 0)
    out, size = part.sum(1), np.abs(part).sum(1)
    return (out, size) if add is None else (out + add, size + np.abs(add))


def head_norm(x, weight, eps):
    """x [.., D] normed."""
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def logprobs(logits, token, top):
    """One row: (logprob, entropy, top tokens, their log probabilities)."""
    x = np.array(logits, np.float64)
    x[np.isnan(x)] = -np.inf
    most = x.max()
    tokens, values = np.full(top, -1), np.full(top, -np.inf)
    if most == -np.inf:
        return -np.inf, 0.0, tokens, values
    with np.errstate(invalid="ignore"):
        d = np.where(x == most, 0.0, x - most)
    z = np.exp(d).sum()
    lp = d - np.log(z)
    p = np.exp(lp)
    entropy = -(p[p > 0] * lp[p > 0]).sum()
    best = np.argsort(-x, kind="stable")[:top]
    best = best[x[best] > -np.inf]
    tokens[: best.size], values[: best.size] = best, lp[best]
    return (lp[token] if 0 <= token < x.size else -np.inf), entropy, tokens, values
