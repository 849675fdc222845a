"""CPU reference of the operators around the adapters, in 64 bits (test
infrastructure only): MX4 values and products, the block norm, sampling.
Arrays are numpy; bf16 enters as float64 holding bf16 values."""
from __future__ import annotations

import math

import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TABLE = np.concatenate([MAGNITUDES, -MAGNITUDES])


def mx4_quantize(x: np.ndarray):
    """Codes [M, K] and scale bytes [M, K/32] of x's rows: every magnitude is compared, the nearest wins, and of
    two equally near ones the even code."""
    v = x.astype(np.float64).reshape(x.shape[0], -1, BLOCK)
    amax = np.max(np.abs(v), axis=-1)
    bad = ~np.isfinite(amax)
    safe = np.where(bad | (amax == 0), 1.0, amax)
    e = np.floor(np.log2(safe)).astype(np.int64)
    e = np.where(np.exp2(e.astype(np.float64)) > safe, e - 1, e)        # log2 may round up to the next power
    e = np.where(np.exp2(e.astype(np.float64) + 1) <= safe, e + 1, e)
    e = np.clip(np.where(amax == 0, -127, e - 2), -127, 127)
    r = np.abs(np.where(bad[..., None], 0.0, v)) / np.exp2(e.astype(np.float64))[..., None]
    d = np.abs(r[..., None] - MAGNITUDES)
    near = d == d.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    code = np.where(bad[..., None], 0, code | (np.signbit(v) << 3))
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def mx4_pack(code: np.ndarray) -> np.ndarray:
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def mx4_unpack(q: np.ndarray) -> np.ndarray:
    return np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)


def mx4_values(code: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """The float64 values of codes [M, K] and scale bytes [M, K/32] (255: NaN)."""
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127.0))
    return (TABLE[code].reshape(code.shape[0], -1, BLOCK) * s[..., None]).reshape(code.shape)


def norm(v, kind: str, w, b, eps: float):
    """(norm(v), the reciprocal root it used, the centred v)."""
    if kind == "none":
        return v, np.ones(v.shape[:-1] + (1,)), v
    c = v - v.mean(-1, keepdims=True) if kind == "layer" else v
    rs = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    out = c * rs
    if w is not None:
        out = out * w
    if b is not None:
        out = out + b
    return out, rs, c


def weights(logits: np.ndarray, temperature: float) -> np.ndarray:
    """The whole-number weights of one row (exp in 64 bits, rounded to a multiple of 2^-31)."""
    l = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    m = l.max()
    if m == -np.inf:
        return np.zeros(l.shape, dtype=np.int64)
    with np.errstate(invalid="ignore", over="ignore"):
        z = np.where(l == m, 0.0, (l - m) / temperature)
    return np.rint(2.0 ** 31 * np.exp(z)).astype(np.int64)


def kept_weights(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0) -> np.ndarray:
    """One row's weights after top-k, top-p and min-p, zero where a token is not kept."""
    l = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    V = l.shape[0]
    greedy = not temperature > 0
    w = weights(logits, 1.0 if greedy else temperature)
    if not w.any():
        return w
    order = np.argsort(-l, kind="stable")
    n = 1 if greedy else (top_k if 0 < top_k < V else V)
    order = order[:n]
    if not greedy and top_p < 1.0:
        before = np.cumsum(w[order]) - w[order]
        mass = max(math.ceil(float(np.float32(top_p)) * float(w[order].sum())), 1)
        order = order[before < mass]
    if not greedy and min_p > 0:
        order = order[w[order] >= min(math.ceil(float(np.float32(min_p)) * 2.0 ** 31), 2 ** 31)]
    kept = np.zeros_like(w)
    kept[order] = w[order]
    return kept


def draw(kept: np.ndarray, u: float) -> int:
    """The token a random number u picks from kept weights, -1 if nothing is kept."""
    total = int(kept.sum())
    if total == 0:
        return -1
    t = min(int(math.floor(float(np.float32(u)) * total)), total - 1)
    return int(np.searchsorted(np.cumsum(kept), max(t, 0), side="right"))
