"""Routing and the sum of a token's experts in Python and numpy float64, token by
token from the definitions, independent of the library."""
import math

import numpy as np


def scores(x, score):
    """p of one row of float64 logits; 0 where x = -inf."""
    p = np.zeros(len(x))
    there = [i for i in range(len(x)) if x[i] != -math.inf]
    with np.errstate(invalid="ignore", over="ignore"):
        if score == "sigmoid":
            for i in there:
                p[i] = 1 / (1 + np.exp(-x[i]))
        elif there:
            e = np.exp(x[there] - np.max(x[there]))
            p[there] = e / e.sum()
    return p


def largest(values, n):
    """Indices of the n largest, the lowest of equal ones first, NaN above all, -inf never."""
    order = sorted((i for i in range(len(values)) if values[i] != -math.inf),
                   key=lambda i: (0, 0, i) if math.isnan(values[i]) else (1, -values[i], i))
    return order[:n]


def route(logits, top, score="softmax", bias=None, groups=1, top_groups=None, group_top=2, renormalise=True, scale=1.0):
    T, E = logits.shape
    top_groups = groups if top_groups is None else top_groups
    experts, weights = np.full((T, top), -1, np.int32), np.zeros((T, top))
    for t in range(T):
        x = logits[t].astype(np.float64)
        p = scores(x, score)
        if bias is None and (top_groups == groups or group_top == 1):
            c = x.copy()
        else:
            c = np.where(x == -math.inf, -math.inf, p + (0.0 if bias is None else bias.astype(np.float64)))
        if top_groups < groups:
            size = E // groups
            g = np.full(groups, -math.inf)
            for j in range(groups):
                best = largest(c[j * size:(j + 1) * size], group_top)
                if best:
                    g[j] = sum(c[j * size + i] for i in best)
            kept = largest(g, top_groups)
            for e in range(E):
                if e // size not in kept:
                    c[e] = -math.inf
        for k, e in enumerate(largest(c, top)):
            experts[t, k], weights[t, k] = e, p[e]
        if renormalise:
            total = weights[t].sum()
            weights[t] = weights[t] / (total if total != 0 else 1)
    return experts, weights * scale, *lists(experts, E)


def lists(experts, E):
    """(rows, offsets, places) of the experts."""
    T, top = experts.shape
    rows, places, offsets = np.full(T * top, -1, np.int32), np.full((T, top), -1, np.int32), np.zeros(E + 1, np.int32)
    at = 0
    for e in range(E):
        for t in range(T):
            for k in range(top):
                if experts[t, k] == e:
                    rows[at], places[t, k] = t, at
                    at += 1
        offsets[e + 1] = at
    return rows, offsets, places


def route_gradient(dweights, logits, experts, score="softmax", renormalise=True, scale=1.0):
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        p = scores(logits[t].astype(np.float64), score)
        at = [k for k in range(experts.shape[1]) if experts[t, k] >= 0]
        e, g = experts[t, at], scale * dweights[t, at].astype(np.float64)
        dp = np.zeros(E)
        if renormalise:
            S = p[e].sum()
            dp[e] = (g - (g * p[e]).sum() / S) / S if S != 0 else 0
        else:
            dp[e] = g
        out[t] = p * (dp - (p * dp).sum()) if score == "softmax" else p * (1 - p) * dp
    return out


def combine(y, places, weights=None, residual=None):
    """(out, sum of magnitudes) in float64."""
    T, top = places.shape
    out = np.zeros((T, y.shape[1])) if residual is None else residual.astype(np.float64).copy()
    size = np.abs(out)
    for t in range(T):
        for k in range(top):
            if 0 <= places[t, k] < len(y):
                v = (1.0 if weights is None else float(weights[t, k])) * y[places[t, k]].astype(np.float64)
                out[t] += v
                size[t] += np.abs(v)
    return out, size
