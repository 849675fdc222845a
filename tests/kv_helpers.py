"""Plumbing of the paged cache's tests: pools, batches and their way to the GPU."""
from __future__ import annotations

import numpy as np

import deterministic_split_lora_amd as dsl
from oracle import bf16_to_f64, kv
from synth import normal_bf16, rng_for
from tests.helpers import bf16_to_gpu, torch


class Batch:
    """Sequences (new tokens, tokens with them) on shuffled pages of a pool whose codes are NaN and whose scales are
    anything until something is appended."""

    def __init__(self, lengths, page_size, heads, D, seed=0, spare=2, extra_pages=1, start=0, rows_behind=0):
        rng = rng_for(seed, "kv-batch")
        self.lengths, self.P, self.H, self.D, self.seed = lengths, page_size, heads, D, seed
        pages = [(n + page_size - 1) // page_size for _, n in lengths]
        self.n_pages = sum(pages) + spare
        order = rng.permutation(self.n_pages).astype(np.int32)
        width = max(pages + [1]) + extra_pages
        self.table = np.full((len(lengths), width), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.lens = np.array([n for _, n in lengths], dtype=np.int32)
        self.cu = (start + np.cumsum([0] + [m for m, _ in lengths])).astype(np.int32)
        self.T = int(self.cu[-1]) + rows_behind
        shape = (self.n_pages, heads, page_size)
        self.cache = {
            "k": rng.choice(np.array([0x7F, 0xFF], dtype=np.uint8), (*shape, D)),
            "v": rng.choice(np.array([0x7F, 0xFF], dtype=np.uint8), (*shape[:2], page_size // 16, D, 16)),
            "ks": rng.integers(0, 256, (*shape[:2], page_size // 16)).astype(np.uint8),
            "vs": rng.integers(0, 256, (*shape[:2], page_size // 16)).astype(np.uint8)}

    def fill(self, std=1.0):
        """Puts tokens into every sequence, through the reference."""
        whole = Batch.__new__(Batch)
        cu = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32)
        total = int(cu[-1])
        if total:
            k = bf16_to_f64(normal_bf16((total, self.H, self.D), std, self.seed, "kv-k"))
            v = bf16_to_f64(normal_bf16((total, self.H, self.D), std, self.seed, "kv-v"))
            del whole
            kv.append(self.cache, k, v, self.table, self.lens, cu, self.P)
        return self

    def gpu(self, pad=0):
        """The batch as a KvCache; pad: bytes between pages."""
        t = torch()

        def pages(a):
            n = a[0].size
            buf = t.full((self.n_pages, n + pad), 0xEE, dtype=t.uint8, device="cuda")
            buf[:, :n] = t.from_numpy(np.ascontiguousarray(a).reshape(self.n_pages, n)).cuda()
            strides, s = [], 1
            for d in reversed(a.shape[1:]):
                strides.append(s)
                s *= d
            return buf.as_strided(a.shape, (n + pad, *reversed(strides)))
        c = self.cache
        return dsl.KvCache(pages(c["k"]), pages(c["v"]), pages(c["ks"]), pages(c["vs"]), ints(self.table),
                           ints(self.lens), ints(self.cu))

    def same(self, g):
        """Asserts that the GPU's cache holds what the reference's does (any code of a NaN)."""
        for name, t in (("ks", g.k_scales), ("vs", g.v_scales), ("k", g.k), ("v", g.v)):
            a, b = t.cpu().numpy(), self.cache[name]
            if name in ("k", "v"):
                a, b = np.where(a & 127 == 127, 127, a), np.where(b & 127 == 127, 127, b)
            bad = np.argwhere(a != b)
            assert bad.size == 0, f"{name}: {len(bad)} differ, first at {bad[0].tolist()}: {a[tuple(bad[0])]} for {b[tuple(bad[0])]}"


def ints(a):
    t = torch()
    return t.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def heads_bf16(T, heads, D, std, seed, name):
    """(values in 64 bits [T, heads, D], the same on the GPU)."""
    bits = normal_bf16((T, heads, D), std, seed, name)
    return bf16_to_f64(bits), bf16_to_gpu(bits)


def attend(q, g, max_new, out=None, lse=True, max_len=None, chunk=0, **kw):
    """lora_kv_attention with its workspace: (out, lse)."""
    t = torch()
    T, Hq, D = q.shape
    out = t.full((T, Hq, D), 7.0, dtype=t.bfloat16, device="cuda") if out is None else out
    lse = t.full((T, Hq), 7.0, dtype=t.float32, device="cuda") if lse else None
    n = max_len if max_len is not None else g.page_table.shape[1] * g.k.shape[2]
    need = dsl.lora_kv_attention_workspace_bytes(T, Hq, g.k.shape[1], D, max_new, n, chunk)
    ws = t.full((need,), 0xFF, dtype=t.uint8, device="cuda") if need else None       # NaN, if any of it is read
    dsl.lora_kv_attention(q, g, out, max_new, max_len=max_len, chunk=chunk, lse=lse, workspace=ws, **kw)
    return out, lse
