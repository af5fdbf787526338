"""Definitions, in fp64, of the scored router with its gradient, of products of
rows with an MXFP4 matrix, and of the experts' combine with its gradients.

TEST INFRASTRUCTURE ONLY: nothing in the product path may import this module.
Written token by token; sizes in tests are small.
"""
from __future__ import annotations

import numpy as np

from .operators import mxfp4_values

F32_MAX = float(np.finfo(np.float32).max)


def scores(row: np.ndarray, score: str) -> np.ndarray:
    """Scores of one token's logits; 0 where masked (-inf, NaN)."""
    l = np.asarray(row, np.float64)
    open_ = ~(np.isnan(l) | (l == -np.inf))
    l = np.minimum(np.where(open_, l, 0.0), F32_MAX)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(open_, 1.0 / (1.0 + np.exp(-l)), 0.0)
    if not open_.any():
        return np.zeros_like(l)
    with np.errstate(under="ignore"):
        e = np.where(open_, np.exp(l - l[open_].max()), 0.0)
    return e / e.sum()


def selected_weights(row, ids, score: str, renormalize: bool, scale: float) -> np.ndarray:
    """Weights of the given ids; renormalised ones from the logits' differences,
    so that no score underflows."""
    l = np.asarray(row, np.float64)
    live = np.array([0 <= i < len(l) and l[i] > -np.inf for i in ids])
    x = np.minimum(np.where(live, l[np.where(live, ids, 0)], 0.0), F32_MAX)
    if not renormalize:
        return np.where(live, scale * scores(l, score)[np.where(live, ids, 0)], 0.0)
    if not live.any():
        return np.zeros(len(ids))
    with np.errstate(under="ignore", over="ignore"):
        log_s = x if score == "softmax" else np.minimum(x, 0.0) - np.log1p(np.exp(-np.abs(x)))
        e = np.where(live, np.exp(log_s - log_s[live].max()), 0.0)
    return scale * e / e.sum()


def router_select(logits, k, score="softmax", bias=None, num_groups=1, group_limit=1, group_top=1, renormalize=True,
                  scale=1.0):
    """(ids [T, k] int32, weights [T, k])."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    per = E // num_groups
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        l = np.minimum(logits[t], F32_MAX)
        s = scores(l, score)
        b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
        able = [e for e in range(E) if l[e] > -np.inf and b[e] > -np.inf]
        value = {e: (l[e] if bias is None else s[e] + b[e]) for e in able}
        grades = []
        for g in range(num_groups):
            best = sorted((value[e] if bias is not None or group_top == 1 else s[e] for e in able if e // per == g),
                          reverse=True)
            grades.append(sum(best[:group_top]) if best else -np.inf)
        stay = sorted(range(num_groups), key=lambda g: (-grades[g], g))[:group_limit]
        order = sorted((e for e in able if e // per in stay), key=lambda e: (-value[e], e))[:k]
        ids[t, :len(order)] = order
        weights[t] = selected_weights(l, ids[t], score, renormalize, scale)
    return ids, weights


def router_select_backward(dweights, logits, ids, score="softmax", renormalize=True, scale=1.0):
    """dlogits [T, E] from the Jacobian of selected_weights, slot by slot."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        l, i = logits[t], np.asarray(ids[t])
        live = [s for s in range(len(i)) if 0 <= i[s] < E and l[i[s]] > -np.inf]
        if not live:
            continue
        s = scores(l, score)
        w = selected_weights(l, i, score, renormalize, 1.0)
        g = scale * np.asarray(dweights[t], np.float64)
        x = np.minimum(np.where(l > -np.inf, l, 0.0), F32_MAX)
        with np.errstate(under="ignore"):
            one_less = np.where(x < 0, 1.0, np.exp(-np.abs(x))) / (1.0 + np.exp(-np.abs(x)))   # 1 - sigmoid
        for a in live:
            if score == "sigmoid" and not renormalize:
                out[t, i[a]] += g[a] * s[i[a]] * one_less[i[a]]
            elif renormalize:   # dw_a/dl_b = w_a (delta_ab - w_b) [times 1 - s_b]
                for b in live:
                    out[t, i[b]] += g[a] * w[a] * ((a == b) - w[b]) * (one_less[i[b]] if score == "sigmoid" else 1.0)
            else:               # dw_a/dl_e = s_a (delta - s_e)
                out[t] -= g[a] * s[i[a]] * s
                out[t, i[a]] += g[a] * s[i[a]]
    return out


def mxfp4_linear(x, codes, scales, gate=False):
    y = np.asarray(x, np.float64) @ mxfp4_values(codes, scales).T
    if not gate:
        return y
    g, u = np.split(y, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def expert_combine(y, rowpos, weights=None):
    y = np.asarray(y, np.float64)
    out = np.zeros((len(rowpos), y.shape[1]))
    for t, row in enumerate(rowpos):
        for s, r in enumerate(row):
            if 0 <= r < len(y):
                out[t] += (1.0 if weights is None else float(weights[t][s])) * y[r]
    return out


def expert_combine_backward(dout, y, rowpos, perm, weights, dy):
    """(dy with the rows that perm and rowpos give one another replaced, dweights)."""
    dout, y = np.asarray(dout, np.float64), np.asarray(y, np.float64)
    gy, gw = np.array(dy, dtype=np.float64), np.zeros(np.shape(rowpos))
    k = np.shape(rowpos)[1]
    for t, row in enumerate(rowpos):
        for s, r in enumerate(row):
            if not 0 <= r < len(y):
                continue
            gw[t, s] = dout[t] @ y[r]
            if perm[r] == t * k + s:
                gy[r] = (1.0 if weights is None else float(weights[t][s])) * dout[t]
    return gy, gw
