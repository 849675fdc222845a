"""Verification of drafted tokens on the GPU against the definition (oracle/verify.py): tokens and counts exactly, for
random numbers far enough from where a rounding of exp could decide."""
import math

import numpy as np
import pytest

import deterministic_split_lora_amd as dsl
from oracle import verify as ref
from oracle.step import kept_weights, weights
from synth import rng_for
from tests.helpers import gpu_available, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def logits_gpu(l, bf16, pad=0):
    """(GPU tensor of a wider row stride, the values it holds in 64 bits)."""
    t = torch()
    v = t.from_numpy(np.ascontiguousarray(l, dtype=np.float32)).to(t.bfloat16 if bf16 else t.float32)
    g = t.full((v.shape[0], v.shape[1] + pad), 99.0, dtype=v.dtype, device="cuda")[:, :v.shape[1]]
    g.copy_(v)
    return g, v.double().numpy()


def run(target, draft, drafted, u, settings=None, stream=None):
    t = torch()
    drafted = np.asarray(drafted, dtype=np.int32)
    B, n = drafted.shape
    kw = {}
    for name, v in zip(("temperature", "top_k", "top_p", "min_p"), settings or ()):
        kw[name] = t.from_numpy(np.asarray(v, dtype=np.int32 if name == "top_k" else np.float32)).cuda()
    tokens = t.full((B, n + 1), -7, dtype=t.int32, device="cuda")
    accepted = t.full((B,), -7, dtype=t.int32, device="cuda")
    lp = t.full((B, n + 1), math.nan, dtype=t.float32, device="cuda")
    ws = t.full((dsl.lora_verify_workspace_bytes(B, n),), 0xFF, dtype=t.uint8, device="cuda")
    dsl.lora_verify(target, t.from_numpy(drafted).cuda(), t.from_numpy(np.asarray(u, dtype=np.float32)).cuda(), tokens,
                    accepted, ws, draft_logits=draft, logprobs=lp, **kw)
    t.cuda.synchronize()
    return tokens.cpu().numpy(), accepted.cpu().numpy(), lp.cpu().numpy()


def far_top_p(rows, T, k, rng):
    """A top_p whose border is no nearer than 2^-19 of the weight to an element's edge, for every row."""
    for _ in range(200):
        p = float(np.float32(0.3 + 0.69 * rng.random()))
        for r in rows:
            w = np.sort(kept_weights(r, T, k))[::-1]
            c = np.cumsum(w[w > 0]) / max(int(w.sum()), 1)
            if len(c) > 1 and np.abs(c - p).min() < 2.0 ** -19:
                break
        else:
            return p
    return 1.0


def far_min_p(rows, T, rng):
    """A min_p that is no nearer than 2^-20 to a weight, for every row."""
    for _ in range(200):
        m = float(np.float32(0.2 * rng.random()))
        if all(np.abs(weights(r, T) / 2.0 ** 31 / m - 1).min() > 2.0 ** -20 for r in rows):
            return m
    return 0.0


def choose(target, draft, drafted, settings, rng):
    """Random numbers for one sequence that decide each test and the draw far from their borders: sums of P and Q are
    within 2^-22 of exact, a drawn token's share is 2^-17 of all at least and its middle 2^-18 from either end."""
    n, V = len(drafted), target.shape[1]
    u = np.full(n + 1, 0.5)
    source = None
    for j in range(n + 1):
        w = kept_weights(target[j], *settings)
        x = int(drafted[j]) if j < n else -1
        if not 0 <= x < V:
            source = w / max(int(w.sum()), 1)
            break
        P = ref.probabilities(w) / ref.UNIT
        Q = ref.probabilities(kept_weights(draft[j], *settings)) / ref.UNIT if draft is not None \
            else np.where(np.arange(V) == x, 1.0, 0.0)
        ratio = P[x] / Q[x] if Q[x] > 0 else (2.0 if P[x] > 0 else 0.0)
        if ratio >= 1.001:
            u[j] = 0.999 * rng.random()
        elif ratio <= 0.0 or (ratio < 0.95 and rng.random() < 0.4):
            u[j] = (ratio + 1.0) / 2
            source = np.maximum(P - Q, 0.0)
            break
        else:
            u[j] = min(ratio, 0.999) / 2
    if source.sum() == 0:                                       # a masked row, or nothing left over
        return u
    c, wide = np.cumsum(source), np.flatnonzero(source > 2.0 ** -17)
    wide = wide if wide.size else np.array([int(source.argmax())])
    i = int(rng.choice(wide))
    u[n] = (c[i] - source[i] / 2) / c[-1]
    return u


def compare(target, draft, values, dvalues, drafted, u, settings):
    B, n = drafted.shape
    tokens, accepted, lp = run(target, draft, drafted, u, settings)
    for i in range(B):
        s = [v[i] for v in settings]
        want = ref.verify(values[i * (n + 1):(i + 1) * (n + 1)], None if draft is None else dvalues[i * n:(i + 1) * n],
                          drafted[i], u[i].astype(np.float32), s)
        assert tokens[i].tolist() == want[0], f"sequence {i} {s}"
        assert accepted[i] == want[1]
        # weights within 2^-22 of exact, one division, one logarithm in fp32
        w = np.array(want[2])
        some = np.isfinite(w)
        assert np.array_equal(some, np.isfinite(lp[i]))
        assert np.all(np.abs(lp[i][some] - w[some]) <= 2.0 ** -20 + 2.0 ** -22 * np.abs(w[some]))
    return accepted


@pytest.mark.parametrize("with_draft", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V,n", [(1, 2), (2, 3), (5, 1), (64, 4), (1000, 5), (4096, 2), (4097, 4), (32000, 3), (128259, 2)])
def test_verify(V, n, bf16, with_draft):
    rng = rng_for(V, f"verify{bf16}{with_draft}")
    B = 12 if V < 10000 else 8
    l = rng.standard_normal((B * (n + 1), V)) * 2.5
    target, values = logits_gpu(l, bf16, pad=3)
    near = l.reshape(B, n + 1, V)[:, :n].reshape(B * n, V) + 0.7 * rng.standard_normal((B * n, V))
    draft, dvalues = logits_gpu(near, bf16, pad=1) if with_draft else (None, None)
    T = np.where(np.arange(B) % 6 == 5, 0.0, 0.5 + rng.random(B)).astype(np.float32)
    k = np.where(np.arange(B) % 2 == 0, rng.integers(1, 60, B), 0).astype(np.int32)
    p, m = np.ones(B, np.float32), np.zeros(B, np.float32)
    drafted, u = np.zeros((B, n), np.int32), np.zeros((B, n + 1))
    for i in range(B):
        tv = values[i * (n + 1):(i + 1) * (n + 1)]
        dv = dvalues[i * n:(i + 1) * n] if with_draft else None
        rows = list(tv) + (list(dv) if with_draft else [])
        if i % 3 == 1:
            p[i] = far_top_p(rows, T[i], k[i], rng)
        if i % 4 == 2 and T[i] > 0:
            m[i] = far_min_p(rows, T[i], rng)
        s = [T[i], k[i], p[i], m[i]]
        for j in range(n):
            w = kept_weights(dv[j] if with_draft else tv[j], *s).astype(np.float64)
            # a likely token of the draft, now and then any token at all
            drafted[i, j] = rng.integers(0, V) if rng.random() < 0.15 else rng.choice(V, p=(w ** 1.5) / (w ** 1.5).sum())
        if i % 5 == 4:
            drafted[i, rng.integers(0, n)] = [-1, V, -2 ** 31, 2 ** 31 - 1][i % 4]
        u[i] = choose(tv, dv, drafted[i], s, rng)
    accepted = compare(target, draft, values, dvalues, drafted, u, [T, k, p, m])
    if V >= 64:
        assert 0 < accepted.sum() < B * n


def test_by_hand():
    """p = (1/2, 1/4, 1/4), q = (1/4, 1/2, 1/4): token 1 is kept below u = 1/2, else token 0 stands for it; token 0 is
    always kept; a draft that is never proposed by q is kept; ends of the drafts; a masked target."""
    p, q = np.log([2.0, 1.0, 1.0]), np.log([1.0, 2.0, 1.0])
    target, _ = logits_gpu(np.tile(p, (12, 1)), False)
    draft, _ = logits_gpu(np.tile(q, (6, 1)), False)
    drafted = [[1], [1], [0], [2], [-1], [3]]
    u = [[0.49, 0.1], [0.51, 0.9], [0.999, 0.6], [0.999, 0.9], [0.0, 0.6], [0.0, 0.1]]
    tokens, accepted, lp = run(target, draft, drafted, u)
    assert tokens.tolist() == [[1, 0], [0, -1], [0, 1], [2, 2], [1, -1], [0, -1]]
    assert accepted.tolist() == [1, 0, 1, 1, 0, 0]
    assert np.allclose(lp[0], np.log([0.25, 0.5])) and np.isneginf(lp[1, 1])
    # of certainty: kept below p, else any token but it
    tokens, accepted, _ = run(target[:8], None, drafted[:4], [[0.24, 0.1], [0.26, 0.6], [0.51, 0.4], [0.9, 0.7]])
    assert tokens.tolist() == [[1, 0], [0, -1], [1, -1], [1, -1]]
    masked, _ = logits_gpu(np.where(np.arange(4)[:, None] % 4 == 1, -np.inf, np.tile(p, (4, 1))), False)
    tokens, accepted, lp = run(masked, None, [[0], [0]], [[0.1, 0.2], [0.1, 0.9]])
    assert tokens.tolist() == [[0, -1], [0, 2]] and accepted.tolist() == [1, 1]
    assert np.isneginf(lp[0, 1])


@pytest.mark.parametrize("bf16", [False, True])
def test_without_drafts_it_is_a_draw(bf16):
    """n = 0, rows of every way through the sampling (large top-k, ties, flat rows, masks, infinite maxima), and ends at
    once: the tokens and log-probabilities of lora_sample, bit for bit."""
    t = torch()
    V, B = 20011, 24
    rng = rng_for(5, "draws")
    l = rng.standard_normal((B, V)) * 2.0
    l[3], l[4, ::2], l[5, 7] = 0.0, -np.inf, np.inf
    l[6, [5, 900]] = np.inf
    l[7] = -np.inf
    l[8] = np.round(l[8])
    l[9, :] = np.linspace(9, -9, V)
    l[10, 5] = np.nan
    g, _ = logits_gpu(l, bf16, pad=5)
    T = np.where(np.arange(B) % 7 == 6, 0.0, 0.3 + rng.random(B) * 2).astype(np.float32)
    T[11], T[12] = 1e38, np.nan
    k = np.where(np.arange(B) % 3 == 0, [1, 40, 700, 3000, 20010, 20011] * 4, 0).astype(np.int32)
    p = np.where(np.arange(B) % 4 == 1, 0.9, 1.0).astype(np.float32)
    m = np.where(np.arange(B) % 5 == 2, 0.01, 0.0).astype(np.float32)
    u = rng.random((B, 2)).astype(np.float32)
    s = [t.from_numpy(a).cuda() for a in (T, k, p, m)]
    want, lp = t.empty(B, dtype=t.int32, device="cuda"), t.empty(B, device="cuda")
    dsl.lora_sample(g, t.from_numpy(u[:, 1].copy()).cuda(), want, *s, logprobs=lp)
    tokens, accepted, got = run(g, None, np.zeros((B, 0)), u[:, 1:], [T, k, p, m])
    assert tokens[:, 0].tolist() == want.tolist() and not accepted.any()
    assert np.array_equal(got[:, 0].view(np.int32), lp.cpu().numpy().view(np.int32))
    twice = g.repeat_interleave(2, 0)
    tokens, accepted, got = run(twice, None, np.full((B, 1), -1), u, [T, k, p, m])
    assert tokens[:, 0].tolist() == want.tolist() and not accepted.any() and (tokens[:, 1] == -1).all()


@pytest.mark.parametrize("with_draft", [False, True])
def test_tokens_have_the_targets_distribution(with_draft):
    """Counts of the first token over many sequences against p: 5 standard deviations (a chance of 6e-7 a token)."""
    V, B = 8, 60000
    rng = rng_for(7, f"law{with_draft}")
    p, q = rng.standard_normal(V), rng.standard_normal(V)
    target, _ = logits_gpu(np.tile(p, (2 * B, 1)), False)
    draft, _ = logits_gpu(np.tile(q, (B, 1)), False)
    pq = [np.exp(x) / np.exp(x).sum() for x in (p, q)]
    drafted = rng.choice(V, (B, 1), p=pq[1])
    tokens, accepted, _ = run(target, draft if with_draft else None, drafted, rng.random((B, 2)))
    # without draft probabilities the drafts are certain: given x, its successor is x with p(x), else p without x
    count = np.bincount(tokens[:, 0], minlength=V)
    want = pq[0]
    assert np.all(np.abs(count - B * want) <= 5 * np.sqrt(B * want * (1 - want)))
    second = tokens[accepted == 1, 1]
    n = len(second)
    assert np.all(np.abs(np.bincount(second, minlength=V) - n * pq[0]) <= 5 * np.sqrt(n * pq[0] * (1 - pq[0])))


def test_many_drafts_and_the_batch_does_not_matter():
    V, n, B = 300, 63, 5
    rng = rng_for(8, "many")
    l = rng.standard_normal((B * (n + 1), V))
    target, values = logits_gpu(l, False)
    drafted = values.reshape(B, n + 1, V)[:, :n].argmax(-1).astype(np.int32)
    u = np.full((B, n + 1), 0.3)
    u[:, :n] = 0.0
    u[1, 40] = 0.9999
    u[2, 62] = 0.9999
    drafted[3, 50] = -1
    T, k, p, m = np.full(B, 0.8, np.float32), np.full(B, 5, np.int32), np.ones(B, np.float32), np.zeros(B, np.float32)
    accepted = compare(target, None, values, None, drafted, u, [T, k, p, m])
    assert accepted.tolist() == [63, 40, 62, 50, 63]
    whole = run(target, None, drafted, u, [T, k, p, m])
    one = run(target[64:128], None, drafted[1:2], u[1:2], [T[1:2], k[1:2], p[1:2], m[1:2]])
    for a, b in zip(whole, one):
        assert np.array_equal(a[1:2], b)


def test_random_numbers_at_the_ends():
    """u of 0, below 0, NaN, 1 and above: a test is passed or not, a drawn token always has weight."""
    p = np.log([0.5, 0.25, 0.25])
    u = [[0.0, 0.0], [-1.0, -1.0], [np.nan, np.nan], [1.0, 1.0], [7.0, 7.0], [0.4999999, 0.9999999]]
    target, _ = logits_gpu(np.tile(p, (12, 1)), False)
    tokens, accepted, _ = run(target, None, [[0]] * 6, u)
    assert accepted.tolist() == [1, 1, 1, 0, 0, 1]
    assert tokens.tolist() == [[0, 0], [0, 0], [0, 0], [2, -1], [2, -1], [0, 2]]


def test_captured_into_a_graph_and_on_another_stream():
    t = torch()
    V, n, B = 5000, 3, 4
    rng = rng_for(9, "graph")
    target, _ = logits_gpu(rng.standard_normal((B * (n + 1), V)), True)
    draft, _ = logits_gpu(rng.standard_normal((B * n, V)), True)
    drafted = t.zeros(B, n, dtype=t.int32, device="cuda")
    u = t.zeros(B, n + 1, device="cuda")
    ws = t.empty(dsl.lora_verify_workspace_bytes(B, n), dtype=t.uint8, device="cuda")
    tokens, accepted = t.empty(B, n + 1, dtype=t.int32, device="cuda"), t.empty(B, dtype=t.int32, device="cuda")
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    dsl.lora_verify(target, drafted, u, tokens, accepted, ws, draft_logits=draft, stream=s)
    s.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        dsl.lora_verify(target, drafted, u, tokens, accepted, ws, draft_logits=draft)
    for i in range(12):
        target.copy_(t.from_numpy(rng.standard_normal((B * (n + 1), V)) * 3))
        draft.copy_(target.view(B, n + 1, V)[:, :n].reshape(B * n, V) + 0.5)
        drafted.copy_(draft.view(B, n, V).argmax(-1))
        u.copy_(t.from_numpy(rng.random((B, n + 1))))
        graph.replay()
        got = tokens.clone(), accepted.clone()
        want = run(target, draft, drafted.cpu().numpy(), u.cpu().numpy())
        assert got[0].tolist() == want[0].tolist() and got[1].tolist() == want[1].tolist()
