"""The operators around the expert FFN in fp64 -- test infrastructure only: residual addition and
RMS norm, the dense product with its epilogue, scored routing.  Plain definitions, row by row."""
from __future__ import annotations

import math

import numpy as np

from . import formats as F


# ------------------------------------------------------------------ residual + RMS norm
def bf16_round(v) -> np.ndarray:
    """fp32 -> the nearest bf16 value (ties to even), as fp32."""
    u = np.ascontiguousarray(v, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint32) << 16
    return u.view(np.float32)


def add_rmsnorm(x, residual, weight, eps: float, residual_bf16: bool):
    """x, residual (or None): fp32 arrays [T][H] (bf16 inputs as the values they stand for); weight
    [H].  Returns (s, y): s fp32 as stored (the fp32 sum, rounded to bf16 if the residual is bf16),
    y fp64, unrounded."""
    s = np.asarray(x, dtype=np.float32)
    if residual is not None:
        s = s + np.asarray(residual, dtype=np.float32)
        if residual_bf16:
            s = bf16_round(s)
    d = s.astype(np.float64)
    y = d * np.asarray(weight, dtype=np.float64) / np.sqrt((d * d).mean(axis=1, keepdims=True) + eps)
    return s, y


# ------------------------------------------------------------------ dense product
def act(a, name: str):
    a = np.asarray(a, dtype=np.float64)
    if name == "relu":
        return np.maximum(a, 0.0)
    if name == "gelu":
        # 0.5 a (1 + tanh u) = a / (1 + exp(-2u)), without the cancellation for negative u
        u = math.sqrt(2.0 / math.pi) * (a + 0.044715 * a**3)
        with np.errstate(over="ignore"):
            return a / (1.0 + np.exp(-2.0 * u))
    if name == "silu":
        with np.errstate(over="ignore"):
            return a / (1.0 + np.exp(-a))
    if name == "swiglu":
        n = a.shape[1] // 2
        return act(a[:, :n], "silu") * a[:, n:]
    assert name == "none"
    return a


def linear(x, w, bias=None, act_name: str = "none", residual=None):
    """x [T][K], w [N][K] as values; fp64 throughout."""
    a = np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
    if bias is not None:
        a = a + np.asarray(bias, dtype=np.float64)
    a = act(a, act_name)
    return a if residual is None else a + np.asarray(residual, dtype=np.float64)


def mxfp8_values(elems, scales):
    return F.dequant_fp8(elems, scales)


# ------------------------------------------------------------------ scored routing
def scores(logits, score: str):
    lg = np.asarray(logits, dtype=np.float32).astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-lg))
        z = np.exp(lg - lg.max(axis=1, keepdims=True))
        return z / z.sum(axis=1, keepdims=True)


def route_scored(logits, k: int, score: str, bias=None, n_group: int = 1, topk_group: int = 1, group_top: int = 1,
                 renormalize: bool = False, scale: float = 1.0):
    """ids int32 [T][k] and gates fp64 [T][k], one token at a time."""
    lg = np.asarray(logits, dtype=np.float32).astype(np.float64)
    T, E = lg.shape
    gs = E // n_group
    p = scores(logits, score)
    ids, gates = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        with np.errstate(invalid="ignore"):
            c = p[t] if bias is None else p[t] + np.asarray(bias, dtype=np.float32).astype(np.float64)
            live = c > -np.inf
        order = lg[t] if bias is None else c
        groups = []
        for g in range(n_group):
            best = sorted((c[e] for e in range(g * gs, (g + 1) * gs) if live[e]), reverse=True)[:group_top]
            groups.append((-sum(best) if best else np.inf, g))
        kept = {g for _, g in sorted(groups)[:topk_group]}
        cand = [(0, -(order[e] + 0.0), e) if live[e] else (1, 0.0, e) for e in range(E) if e // gs in kept]
        chosen = [e for _, _, e in sorted(cand)[:k]]
        ids[t] = chosen
        gt = np.array([p[t][e] if live[e] else 0.0 for e in chosen])
        if renormalize:
            gt = gt / gt.sum() if gt.sum() > 0 else np.zeros(k)
        gates[t] = gt * scale
    return ids, gates
