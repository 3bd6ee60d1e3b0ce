"""Oracle: the operators around the expert MLP - the router's losses, the
product with bias, activation and residual, activations kept in 8 bits.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  float64 numpy, written
from the definitions; the gated activations and the MX block rule are those
of ``moe.py`` and ``mx.py``.
"""
from __future__ import annotations

import numpy as np

from .moe import act_backward, act_forward, dphi, grouped_gemm, grouped_wgrad, phi
from .mx import e4m3_decode, mx_quantize_rows

__all__ = ["router_loss", "router_loss_bwd", "linear_act", "linear_dact", "linear_fwd",
           "linear_bwd", "checkpoint_pack", "checkpoint_unpack"]


# ---------------------------------------------------------------------------
# router losses ([TE] "용량 기반 MoE와 드롭리스 MoE": a dropless layer has no
# capacity that bounds an expert's load; the load-balance and z losses are
# the common training terms)
# ---------------------------------------------------------------------------

LOWEST = -3.3895313892515355e38     # bf16's lowest finite value


def _softmax(logits):
    """P [T, E] and lse [T]; a row with nothing above bf16's lowest value (a
    mask of -inf or of a type's lowest) is empty: P = 0 and lse = -inf."""
    z = np.asarray(logits, np.float64)
    m = z.max(axis=1)
    z = np.where((m <= LOWEST)[:, None], -np.inf, z)
    m = np.where(m <= LOWEST, -np.inf, m)
    safe = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        e = np.where(np.isneginf(z), 0.0, np.exp(z - safe[:, None]))
        tot = e.sum(axis=1)
        lse = safe + np.log(tot)
        P = np.where(tot[:, None] == 0.0, 0.0, e / np.where(tot == 0.0, 1.0, tot)[:, None])
    return P, lse


def _segments(T, seg):
    seg = [0, T] if seg is None else [int(v) for v in seg]
    owner = np.full(T, -1)
    for s in range(len(seg) - 1):
        owner[seg[s]:seg[s + 1]] = s
    return len(seg) - 1, owner


def router_loss(logits, topk_idx, seg_offsets=None, token_mask=None):
    """loss [2] (balance, z), counts [S, E], lse [T], n_valid [S]: see
    ``moe_router_loss``.  Balance E/(kN) sum_s 1/N_s sum_e c_se sum_t P_te;
    z the mean squared log-partition of the valid tokens."""
    T, E = np.shape(logits)
    k = np.shape(topk_idx)[1]
    P, lse = _softmax(logits)
    S, owner = _segments(T, seg_offsets)
    valid = (owner >= 0) & ~np.isneginf(lse)
    if token_mask is not None:
        valid &= np.asarray(token_mask) != 0
    counts = np.zeros((S, E), np.int64)
    n_valid = np.zeros(S, np.int64)
    bal = 0.0
    N = int(valid.sum())
    for s in range(S):
        rows = np.nonzero(valid & (owner == s))[0]
        n_valid[s] = len(rows)
        for t in rows:
            for e in np.asarray(topk_idx)[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        if len(rows):
            bal += float((counts[s] * P[rows].sum(axis=0)).sum()) / len(rows)
    loss = np.array([E * bal / (k * N), float((lse[valid] ** 2).sum()) / N]) if N else np.zeros(2)
    return {"loss": loss, "counts": counts, "lse": lse, "n_valid": n_valid}


def router_loss_bwd(logits, topk_idx, dloss, probs=None, dprobs=None, seg_offsets=None,
                    token_mask=None):
    """dlogits [T, E] of dloss . loss (counts held constant) and, with probs
    and dprobs, of the softmax over the selected logits ([Sonic] "역전파 계산
    그래프 재작성하기": dS reaches the router)."""
    T, E = np.shape(logits)
    idx = np.asarray(topk_idx)
    k = idx.shape[1]
    f = router_loss(logits, topk_idx, seg_offsets, token_mask)
    P, lse = _softmax(logits)
    S, owner = _segments(T, seg_offsets)
    N = int(f["n_valid"].sum())
    d = np.zeros((T, E))
    for t in range(T):
        s = owner[t]
        ok = s >= 0 and not np.isneginf(lse[t]) and (token_mask is None or token_mask[t] != 0)
        if ok:
            w = dloss[0] * E * f["counts"][s] / (k * N * f["n_valid"][s])
            d[t] = P[t] * (w - (P[t] * w).sum() + 2.0 * dloss[1] * lse[t] / N)
        if probs is not None:
            p, dp = np.asarray(probs, np.float64)[t], np.asarray(dprobs, np.float64)[t]
            on = (idx[t] >= 0) & (idx[t] < E)
            mean = (p * dp)[on].sum()
            for j in np.nonzero(on)[0]:
                d[t, idx[t, j]] += p[j] * (dp[j] - mean)
    return d


# ---------------------------------------------------------------------------
# product with bias, activation and residual ([TE] "최적화 1: grouped GEMM";
# [CuTe] "핵심 아이디어 / 구조 / 동작 방식": the output's work in the epilogue)
# ---------------------------------------------------------------------------

_GATED = ("swiglu", "geglu")
_AS_GATE = {"silu": "swiglu", "gelu": "geglu"}


def linear_act(z, act: str):
    """act(z): the gated ones halve the columns ([CuTe] "핵심 아이디어")."""
    z = np.asarray(z, np.float64)
    if act in _GATED or act == "srelu":
        return act_forward(z, act)
    if act == "relu":
        return np.maximum(z, 0.0)
    return phi(z, _AS_GATE[act]) if act in _AS_GATE else z


def linear_dact(z, g, act: str):
    """dz from the gradient g of act(z) ([CuTe] "GroupGemm + dActivation")."""
    z, g = np.asarray(z, np.float64), np.asarray(g, np.float64)
    if act in _GATED or act == "srelu":
        return act_backward(z, g, act)
    if act == "relu":
        return np.where(z > 0, g, 0.0)
    return g * dphi(z, _AS_GATE[act]) if act in _AS_GATE else g


def linear_fwd(a, offsets, B, act="none", bias=None, residual=None, b_layout="kn"):
    """(out, z) in float64; rows outside every expert NaN."""
    z = grouped_gemm(a, offsets, B, b_layout, round_out=False)
    if bias is not None:
        for e in range(len(offsets) - 1):
            z[offsets[e]:offsets[e + 1]] += np.asarray(bias, np.float64)[e]
    out = linear_act(z, act)
    if residual is not None:
        out = out + np.asarray(residual, np.float64)
    return out, z


def linear_bwd(dout, a, offsets, B, act="none", z=None, b_layout="kn"):
    """(dz, da, dB, dbias) in float64, nothing rounded."""
    dout = np.asarray(dout, np.float64)
    dz = dout if act == "none" else linear_dact(z, dout, act)
    da = grouped_gemm(dz, offsets, B, "nk" if b_layout == "kn" else "kn", round_out=False)
    dB = (grouped_wgrad(a, dz, offsets, False) if b_layout == "kn"
          else grouped_wgrad(dz, a, offsets, False))
    E = len(offsets) - 1
    dbias = np.stack([dz[offsets[e]:offsets[e + 1]].sum(axis=0) for e in range(E)])
    return dz, da, dB, dbias


# ---------------------------------------------------------------------------
# activations in 8 bits (OCP MX v1.0 block rule along rows)
# ---------------------------------------------------------------------------

def checkpoint_pack(x):
    """codes [rows, cols], scale bytes [rows, cols/32] (OCP MX v1.0)."""
    return mx_quantize_rows(x)


def checkpoint_unpack(q, s):
    """The values that codes and scales stand for."""
    v = e4m3_decode(np.asarray(q)).reshape(q.shape[0], -1, 32)
    return (v * np.ldexp(1.0, np.asarray(s, np.int64) - 127)[..., None]).reshape(q.shape)
