"""The router's choice by scores and its gradient, in float64, one token at a
time from the definitions (no GPU code shared)."""
from __future__ import annotations

import numpy as np

BF16_LOWEST = -3.3895313892515355e38


def _row_scores(z, score):
    """Scores of one row; experts that take no part have none (NaN)."""
    on = z > BF16_LOWEST                      # (False for NaN)
    s = np.full(z.shape, np.nan)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            s[on] = 1.0 / (1.0 + np.exp(-z[on]))
    elif on.any():
        m = z[on].max()
        with np.errstate(invalid="ignore"):
            ex = np.where(z[on] == m, 1.0, np.exp(z[on] - m))
        s[on] = ex / ex.sum()
    return s


def _order(values):
    """Indices by decreasing value, the lower index of equals first."""
    return sorted(range(len(values)), key=lambda i: (-values[i], i))


def router_select(logits, k, score="softmax", bias=None, groups=1, top_groups=None, best=1,
                  renorm=True, scale=1.0):
    """(topk_idx int32 [T, k], probs float64 [T, k])."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    n = E // groups
    top_groups = groups if top_groups is None else top_groups
    idx = np.full((T, k), -1, np.int32)
    probs = np.zeros((T, k))
    for t in range(T):
        s = _row_scores(logits[t], score)
        c = s if bias is None else s + np.asarray(bias, np.float64)
        c = np.where(np.isnan(c), -np.inf, c)
        if bias is None and best == 1:        # the scores' order is the logits', where they underflow too
            c = np.where(c > -np.inf, logits[t], -np.inf)
        if top_groups < groups:
            gs = []
            for g in range(groups):
                top = sorted(c[g * n:(g + 1) * n], reverse=True)[:best]
                some = [v for v in top if v > -np.inf]
                gs.append(sum(some) if some else -np.inf)
            keep = set(_order(gs)[:top_groups])
            c = np.array([c[e] if e // n in keep else -np.inf for e in range(E)])
        if bias is None:
            c = np.where(c > -np.inf, logits[t], -np.inf)
        picks = [e for e in _order(c) if c[e] > -np.inf][:k]
        if not picks:
            continue
        if renorm and score == "softmax":     # the softmax's own sum cancels
            z = logits[t, picks]
            with np.errstate(invalid="ignore"):
                w = np.where(z == z.max(), 1.0, np.exp(z - z.max()))
            w = w / w.sum()
        else:
            w = s[picks]
            if renorm:
                w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        idx[t, :len(picks)] = picks
        probs[t, :len(picks)] = scale * w
    return idx, probs


def router_select_bwd(logits, topk_idx, dprobs, score="softmax", renorm=True, scale=1.0):
    """dlogits [T, E] by the chain rule from the scores of the chosen experts
    (distinct ids of experts that take part)."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        s = np.nan_to_num(_row_scores(logits[t], score))
        e = [int(i) for i in topk_idx[t] if 0 <= i < E]
        dw = scale * np.array([float(dprobs[t, j]) for j, i in enumerate(topk_idx[t]) if 0 <= i < E])
        ds = np.zeros(E)
        if e:
            q = s[e]
            tot = q.sum()
            if renorm and tot > 0:
                dw = dw / tot - (dw * q).sum() / tot ** 2
            ds[e] = dw
        out[t] = ds * s * (1 - s) if score == "sigmoid" else s * (ds - (ds * s).sum())
    return out
