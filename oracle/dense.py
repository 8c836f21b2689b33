"""The dense feed-forward operators beside the routed experts in fp64 -- test infrastructure only: FP8 with a
scale per block of 128 and products of it, the gated projection, and the gradients of both."""
from __future__ import annotations

import math

import numpy as np

from . import block as B
from . import formats as F


def up(n: int, by: int = 128) -> int:
    return -(-n // by)


# ------------------------------------------------------------------ FP8 blocks of 128
def spread(scales, by: int, rows: int, K: int) -> np.ndarray:
    """A scale for each value from one per block of by x 128."""
    return np.repeat(np.repeat(np.asarray(scales), by, axis=0)[:rows], 128, axis=1)[:, :K]


def fp8_quantize(x, by: int):
    """x fp32 [rows][K] -> (e4m3fn bytes, fp32 scales): scale = max|x| / 448, element = x / scale, both quotients
    fp32.  Finite values and NaN, infinities; a NaN element is byte 0x7F."""
    x = np.asarray(x, dtype=np.float32)
    rows, K = x.shape
    pad = np.zeros((up(rows, by) * by, up(K) * 128), dtype=np.float32)
    pad[:rows, :K] = np.abs(x)
    top = pad.reshape(-1, by, up(K), 128).max(axis=(1, 3))  # NaN if there is one
    with np.errstate(all="ignore"):
        scales = (top / np.float32(448)).astype(np.float32)
        s = spread(scales, by, rows, K)
        v = np.where(s == 0, np.float32(0), x / s).astype(np.float32)
    nan = np.isnan(v)
    q = F.e4m3fn_encode(np.where(nan, 0, np.clip(v, -448, 448)).astype(np.float64))
    return np.where(nan, 0x7F, q).astype(np.uint8), scales


def fp8_values(q, scales, by: int, gated: bool = False) -> np.ndarray:
    """The values of such a matrix in fp64; gated: two of them, one behind the other."""
    q = np.asarray(q)
    if gated:
        h, b = q.shape[0] // 2, scales.shape[0] // 2
        return np.concatenate([fp8_values(q[:h], scales[:b], by), fp8_values(q[h:], scales[b:], by)])
    return F.e4m3fn_value(q) * spread(np.asarray(scales, dtype=np.float64), by, *q.shape)


# ------------------------------------------------------------------ gated projection and gradients
def glu(x, w, act_name: str):
    """(h, a): a = x W^T, its first half the gate's."""
    a = np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
    n = a.shape[1] // 2
    return B.act(a[:, :n], act_name) * a[:, n:], a


def slope(g, act_name: str) -> np.ndarray:
    """act'(g); relu'(0) = 0."""
    g = np.asarray(g, dtype=np.float64)
    if act_name == "none":
        return np.ones_like(g)
    if act_name == "relu":
        return (g > 0).astype(np.float64)
    # a p(z) with p the logistic function: silu z = g, gelu z = 2 sqrt(2/pi) (g + 0.044715 g^3)
    c = 2.0 * math.sqrt(2.0 / math.pi)
    z, dz = (g, 1.0) if act_name == "silu" else (c * (g + 0.044715 * g**3), c * (1 + 3 * 0.044715 * g * g))
    with np.errstate(over="ignore"):
        p, q = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))
    return p + g * p * q * dz


def glu_grad(dh, a, act_name: str) -> np.ndarray:
    """The gradient of the pre-activations a [T][2I] from dh [T][I]."""
    dh, a = np.asarray(dh, dtype=np.float64), np.asarray(a, dtype=np.float64)
    n = dh.shape[1]
    g, u = a[:, :n], a[:, n:]
    return np.concatenate([dh * u * slope(g, act_name), dh * B.act(g, act_name)], axis=1)


def linear_grad(dy, x, w):
    """(dx, dw) of y = x W^T."""
    dy, x, w = (np.asarray(v, dtype=np.float64) for v in (dy, x, w))
    return dy @ w, dy.T @ x
