"""CPU reference of the verification of drafted tokens (test infrastructure only), by its definition on the whole-number
weights of oracle/step.py."""
from __future__ import annotations

import math

import numpy as np

from oracle.step import draw, kept_weights

UNIT = 2.0 ** 40


def probabilities(kept: np.ndarray) -> np.ndarray:
    """P of one row's kept weights, as float64 whole numbers."""
    total = int(kept.sum())
    return np.rint(kept.astype(np.float64) * (UNIT / total)) if total else np.zeros(kept.shape)


def verify(target, draft, drafted, u, settings):
    """One sequence: target [n + 1, V], draft [n, V] or None, drafted [n], u [n + 1], settings of kept_weights.
    (tokens [n + 1], accepted, logprobs [n + 1])."""
    n, V = len(drafted), target.shape[1]
    tokens, logprobs = [], []
    source = None
    for j in range(n + 1):
        w = kept_weights(target[j], *settings)
        x = int(drafted[j]) if j < n else -1
        if not 0 <= x < V:
            source = w
            break
        P = probabilities(w)
        Q = probabilities(kept_weights(draft[j], *settings)) if draft is not None else np.where(np.arange(V) == x, UNIT, 0.0)
        if (float(np.float32(u[j])) if u[j] > 0 else 0.0) * Q[x] < P[x]:
            tokens.append(x)
            logprobs.append(math.log(w[x] / w.sum()))
            continue
        source = np.maximum(P - Q, 0.0).astype(np.int64)
        if not source.any():
            source = w
        break
    token = draw(source, u[n])
    accepted = len(tokens)
    tokens.append(token)
    logprobs.append(math.log(w[token] / w.sum()) if token >= 0 else -math.inf)
    pad = n - accepted
    return tokens + [-1] * pad, accepted, logprobs + [-math.inf] * pad
