"""Routing of tokens to experts, token by token in float64 (test infrastructure).

    s = softmax(l) or sigmoid(l);  r = s + bias;  selection by r (by l without a bias), equal ones by index,
    within the topk_group groups of largest value (the sum of a group's group_top largest r);
    w = scale * s[ids] (/ sum s[ids]).

The pages name mixture-of-experts models without their router's arithmetic ("ExLlamaV3 & EXL3 Deep Dive",
Section 4); this is the common form. An expert whose logit or bias is -inf is not available; slots without an
expert get id -1 and weight 0; a token whose scores have no order (NaN, +inf under softmax, a bias of NaN or
+inf) gets ids 0 .. top_k - 1 and NaN weights.

Pins (tests/test_oracle_route.py): hand-worked scores and selections; a brute-force selection over all subsets.
"""
from __future__ import annotations

import math

import numpy as np


def scores(logits, sigmoid: bool):
    l = [float(v) for v in logits]
    if sigmoid:
        return [0.0 if v == -math.inf else (1.0 / (1.0 + math.exp(-v)) if v > -700 else math.exp(v)) for v in l]
    top = max(l)
    if top == -math.inf:
        return [0.0] * len(l)
    e = [math.exp(v - top) for v in l]
    z = math.fsum(e)
    return [v / z for v in e]


def route_token(logits, top_k, bias=None, sigmoid=False, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0):
    l = [float(v) for v in logits]
    b = [0.0] * len(l) if bias is None else [float(v) for v in bias]
    if any(math.isnan(v) for v in l + b) or math.inf in b or (not sigmoid and math.inf in l):
        return list(range(top_k)), [math.nan] * top_k
    s = scores(l, sigmoid)
    there = [i for i in range(len(l)) if l[i] != -math.inf and b[i] != -math.inf]
    ranked = {i: s[i] + b[i] for i in there}
    if n_group > 1:
        size = len(l) // n_group
        value = {}
        for g in range(n_group):
            inside = sorted((ranked[i] for i in there if i // size == g), reverse=True)
            if inside:
                value[g] = inside[0] if group_top == 1 or len(inside) == 1 else inside[0] + inside[1]
        kept = sorted(value, key=lambda g: (-value[g], g))[:topk_group]
        there = [i for i in there if i // size in kept]
    key = (lambda i: (-l[i], i)) if bias is None else (lambda i: (-ranked[i], i))
    ids = sorted(there, key=key)[:top_k]
    w = [s[i] for i in ids]
    if renormalize:
        z = math.fsum(w)
        w = [v / z if z > 0 else 0.0 for v in w]
    w = [v * scale for v in w]
    return ids + [-1] * (top_k - len(ids)), w + [0.0] * (top_k - len(w))


def route(logits, top_k, **kw):
    """(ids int32 [tokens, top_k], weights float64 [tokens, top_k])."""
    rows = [route_token(r, top_k, **kw) for r in np.asarray(logits, np.float64)]
    return np.array([r[0] for r in rows], np.int32), np.array([r[1] for r in rows], np.float64)


def group(sel, experts: int):
    """(offsets int32 [experts + 1], order int32 [pairs]): pairs by expert, ids outside [0, experts) last."""
    lists = [[] for _ in range(experts + 1)]
    for p, e in enumerate(np.asarray(sel).reshape(-1).tolist()):
        lists[e if 0 <= e < experts else experts].append(p)
    offsets = np.cumsum([0] + [len(v) for v in lists[:-1]])
    return offsets.astype(np.int32), np.array([p for v in lists for p in v], np.int32)
