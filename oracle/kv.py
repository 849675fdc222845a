"""CPU reference of the paged 8-bit cache (test infrastructure only): its codes
and scales, appending, attention in 64 bits.  Arrays are numpy; bf16 enters as
float64 holding bf16 values."""
from __future__ import annotations

import numpy as np

BLOCK = 16


def _code_values():
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        out[c] = np.nan if c & 127 == 127 else -v if c & 128 else v
    return out


VALUES = _code_values()
_POSITIVE = VALUES[:127]                                        # 0 .. 448, rising


def encode(x: np.ndarray) -> np.ndarray:
    """Codes of float64 values: the nearest, of two equally near ones the even code; past 448 the largest."""
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = code | (np.signbit(x).astype(np.int64) << 7)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def scale_byte(amax: float) -> int:
    b = 27
    while b < 246 and amax > 448.0 * 2.0 ** (b - 127):
        b += 1
    return b


def head_norm(x, w, eps, dtype):
    """RMS norm over the last axis, every operation rounded to dtype, the squares summed in 64 bits."""
    x = x.astype(dtype)
    if w is None:
        return x
    mean = (np.square(x.astype(np.float64)).sum(-1, keepdims=True) / x.shape[-1]).astype(dtype)
    inv = dtype(1) / np.sqrt(mean + dtype(eps))
    return x * inv * w.astype(dtype)


def rotate(x, row, pairs):
    """Rotate x [..., D] by a table row [rope_dim] (NaN where the position has none)."""
    R = row.shape[-1]
    h = R // 2
    c, s = row[..., :h], row[..., h:]
    ia, ib = (np.arange(0, R, 2), np.arange(1, R, 2)) if pairs else (np.arange(h), np.arange(h, R))
    out = x.copy()
    a, b = x[..., ia], x[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = b * c + a * s
    return out


def step_rows(table, seq_lens, cu, T, page_size, n_pages):
    """Per row of a step: (sequence, position, page or -1), None for rows of no sequence."""
    rows = [None] * T
    for b in range(len(seq_lens)):
        first, end = int(cu[b]), int(cu[b + 1])
        for i in range(first, end):
            pos = int(seq_lens[b]) - (end - i)
            j = pos // page_size
            page = int(table[b, j]) if 0 <= j < table.shape[1] else -1
            rows[i] = (b, pos, page if 0 <= page < n_pages else -1)
    return rows


def append(cache, k, v, table, seq_lens, cu, page_size):
    """Appends rows k, v [T, H, D] (any float type, normed and rotated) to cache (dict of codes k, v and scales ks, vs,
    changed in place), block by block."""
    n_pages, H = cache["ks"].shape[:2]
    rows = step_rows(table, seq_lens, cu, k.shape[0], page_size, n_pages)
    blocks = {}
    for i, r in enumerate(rows):
        if r is not None and r[1] >= 0 and r[2] >= 0:
            blocks.setdefault((r[2], r[1] % page_size // BLOCK), []).append((r[1] % BLOCK, i))
    for (page, w), new in blocks.items():
        first = new[0][0]
        ids = [i for _, i in new]
        for h in range(H):
            for name, x in (("k", k), ("v", v)):
                x = x[ids, h].astype(np.float64)
                finite = np.abs(x[np.isfinite(x)])
                b = scale_byte(finite.max() if finite.size else 0.0)
                scales = cache[name + "s"]
                codes = cache["k"][page, h, w * BLOCK:(w + 1) * BLOCK] if name == "k" else cache["v"][page, h, w].T
                if first > 0:
                    old = int(scales[page, h, w])
                    b = max(b, old)
                    if b > old:
                        codes[:first] = encode(VALUES[codes[:first]] * 2.0 ** max(old - b, -120))
                scales[page, h, w] = b
                codes[first:first + len(new)] = encode(np.clip(x, -1e200, 1e200) * 2.0 ** (127 - b))


def sequence(cache, table, b, n, page_size):
    """Values (keys, values [n, H, D]) and whether its tokens are there."""
    n_pages, H = cache["ks"].shape[:2]
    D = cache["k"].shape[-1]
    k, v, there = np.zeros((n, H, D)), np.zeros((n, H, D)), np.zeros(n, dtype=bool)
    for p in range(n):
        j = p // page_size
        page = int(table[b, j]) if j < table.shape[1] else -1
        if not 0 <= page < n_pages:
            continue
        there[p] = True
        w, t = p % page_size // BLOCK, p % BLOCK
        k[p] = VALUES[cache["k"][page, :, p % page_size]] * np.exp2(cache["ks"][page, :, w, None].astype(float) - 127)
        v[p] = VALUES[cache["v"][page, :, w, :, t]] * np.exp2(cache["vs"][page, :, w, None].astype(float) - 127)
    return k, v, there


def attention(q, cache, table, seq_lens, cu, page_size, scale, causal=True, window=0, max_len=None):
    """(out, lse, bound of out, bound of lse) for q [T, Hq, D]; rows of no sequence NaN.

    The bounds follow the arithmetic: a logit of products exact in fp32 accumulators is off by at most
    (D + 8) 2^-24 scale sum|q k| (its terms' sums, the scale, the shift under the maximum, exp2's argument), which is
    also the relative error of its p, next to 2^-21 from exp2 and the rescaling; the p are rounded to bf16 (half a step,
    2^-8) before the product, whose sums add n 2^-24, as the sum of p does; the output is rounded by half a step."""
    T, Hq, D = q.shape
    H = cache["ks"].shape[1]
    out, lse = np.full(q.shape, np.nan), np.full((T, Hq), np.nan)
    tol, ltol = np.zeros(q.shape), np.zeros((T, Hq))
    for b in range(len(seq_lens)):
        n = int(seq_lens[b])
        first, end = int(cu[b]), int(cu[b + 1])
        if end <= first:
            continue
        k, v, there = sequence(cache, table, b, n, page_size)
        for i in range(first, end):
            pos = n - (end - i)
            j = np.arange(n)
            seen = there & (j < (n if max_len is None else max_len))
            if causal:
                seen &= j <= pos
            if window:
                seen &= j > pos - window
            for h in range(Hq):
                kh, vh = k[seen, h * H // Hq], v[seen, h * H // Hq]
                if not seen.any():
                    out[i, h], lse[i, h] = 0.0, -np.inf
                    continue
                s = scale * (kh @ q[i, h])
                top = s.max()
                e = np.exp(s - top)
                p = e / e.sum()
                out[i, h] = p @ vh
                lse[i, h] = top + np.log(e.sum())
                m = seen.sum()
                ds = (D + 8) * 2.0 ** -24 * scale * np.max(np.abs(kh) @ np.abs(q[i, h])) + 2.0 ** -21 + m * 2.0 ** -24
                tol[i, h] = (p @ np.abs(vh)) * (2.0 ** -8 + 2 * ds) + np.abs(out[i, h]) * 2.0 ** -8 + 1e-30
                ltol[i, h] = ds + 2.0 ** -22 * (1 + abs(lse[i, h]))
    return out, lse, tol, ltol
