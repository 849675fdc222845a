"""Attention over the paged 8-bit cache on the GPU against the formula in 64 bits (oracle/kv.py, whose bounds follow the
arithmetic), and what must not matter to it: the batch, other tokens, what the pool holds elsewhere."""
import numpy as np
import pytest

import deterministic_split_lora_amd as dsl
from oracle import bf16_to_f64, kv
from tests.helpers import bf16_from_gpu, gpu_available, torch
from tests.kv_helpers import Batch, attend, heads_bf16, ints

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def check(batch, q, got, what="", scale=None, **kw):
    out, lse, tol, ltol = kv.attention(q, batch.cache, batch.table, batch.lens, batch.cu, batch.P,
                                       batch.D ** -0.5 if scale is None else np.float32(scale), **kw)
    rows = np.zeros(q.shape[0], dtype=bool)
    for b in range(len(batch.lens)):
        rows[batch.cu[b]:batch.cu[b + 1]] = True
    o, l = bf16_to_f64(bf16_from_gpu(got[0])), got[1].double().cpu().numpy()
    assert np.all(o[~rows] == 7.0) and np.all(l[~rows] == 7.0), "rows of no sequence were written"
    assert np.array_equal(np.isnan(o[rows]), np.isnan(out[rows])), f"{what}: NaN elsewhere"
    fine = rows[:, None, None] & ~np.isnan(out)
    err, tol = np.abs(o - out)[fine], tol[fine]
    assert np.all(err[tol == 0] == 0), f"{what}: rows that see nothing"
    worst = np.max(err[tol > 0] / tol[tol > 0], initial=0.0)
    assert worst <= 1.0, f"{what}: output beyond its bound by {worst:.3g}"
    empty = np.isneginf(lse)
    assert np.array_equal(empty[rows], np.isneginf(l[rows])), f"{what}: empty rows"
    fine = rows[:, None] & ~empty & ~np.isnan(lse)
    assert np.all(np.abs(l[fine] - lse[fine]) <= ltol[fine]), f"{what}: lse"
    return worst


CASES = [  # D, Hq, H, page, [(new, tokens)]
    (128, 8, 2, 64, [(1, 1), (1, 63), (1, 64), (1, 65), (1, 300), (1, 1100)]),
    (128, 4, 4, 16, [(1, 17), (1, 16), (1, 700)]),
    (64, 8, 1, 32, [(1, 257), (1, 513), (1, 5)]),
    (256, 5, 1, 16, [(1, 129), (1, 640)]),
    (128, 64, 2, 128, [(1, 90), (1, 400)]),                     # 32 rows of one token: two tiles
    (128, 8, 2, 16, [(4, 4), (3, 40), (1, 300), (4, 611)]),
    (64, 7, 1, 64, [(5, 100), (9, 333), (1, 64)]),
    (256, 4, 2, 64, [(6, 77), (8, 290)]),
    (128, 8, 2, 64, [(40, 40), (33, 180), (1, 70), (129, 300)]),
    (64, 3, 1, 16, [(130, 130), (47, 500)]),
    (256, 4, 2, 32, [(40, 64), (35, 300)]),
    (128, 5, 5, 32, [(200, 200), (1, 9), (0, 30), (65, 65)]),
]


@pytest.mark.parametrize("D,Hq,H,P,lengths", CASES)
@pytest.mark.parametrize("chunk", [0, 256, 1 << 20])
def test_attention(D, Hq, H, P, lengths, chunk):
    batch = Batch(lengths, P, H, D, seed=1, start=2, rows_behind=3).fill()
    q, qg = heads_bf16(batch.T, Hq, D, 1.5, 2, "q")
    got = attend(qg, batch.gpu(pad=48), max(n for n, _ in lengths), chunk=chunk)
    check(batch, q, got)


@pytest.mark.parametrize("window", [1, 16, 50, 64, 257, 5000])
@pytest.mark.parametrize("lengths", [[(1, 400), (1, 3), (1, 64)], [(5, 300), (3, 60)], [(70, 310), (1, 80), (33, 33)]])
def test_window(window, lengths):
    batch = Batch(lengths, 16, 2, 64, seed=3).fill()
    q, qg = heads_bf16(batch.T, 8, 64, 1.0, 4, "q")
    for chunk in (0, 256):
        got = attend(qg, batch.gpu(), max(n for n, _ in lengths), window=window, chunk=chunk)
        check(batch, q, got, window=window)


@pytest.mark.parametrize("lengths", [[(1, 300), (4, 90)], [(60, 70), (2, 200)]])
def test_every_key(lengths):
    """Not causal: every query sees the whole sequence; a scale of the caller's; fewer keys than there are."""
    batch = Batch(lengths, 32, 1, 128, seed=3).fill()
    q, qg = heads_bf16(batch.T, 4, 128, 1.0, 4, "q")
    got = attend(qg, batch.gpu(), max(n for n, _ in lengths), causal=False, scale=0.3)
    check(batch, q, got, scale=0.3, causal=False)
    got = attend(qg, batch.gpu(), max(n for n, _ in lengths), max_len=77)
    check(batch, q, got, max_len=77)


@pytest.mark.parametrize("lengths", [[(1, 200), (1, 100)], [(6, 200), (6, 100)], [(50, 200), (40, 100)]])
def test_missing_pages_and_empty_rows(lengths):
    """Pages that are not there are seen by nobody; rows that see nothing are 0 and -inf; more new tokens than tokens."""
    batch = Batch(lengths + [(2, 30), (3, 2), (1, 0)], 16, 2, 64, seed=5, rows_behind=2).fill()
    batch.table[0, 3] = -1
    batch.table[0, 7] = batch.n_pages
    batch.table[1, 0] = 2 ** 31 - 1
    batch.table[2, :] = -7
    q, qg = heads_bf16(batch.T, 4, 64, 1.0, 4, "q")
    for chunk in (0, 256):
        got = attend(qg, batch.gpu(), max(n for n, _ in lengths), chunk=chunk)
        check(batch, q, got)
        check(batch, q, attend(qg, batch.gpu(), max(n for n, _ in lengths), chunk=chunk, window=40), window=40)


@pytest.mark.parametrize("new,Hq", [(1, 4), (3, 8), (40, 4)])
def test_nan_reaches_only_who_sees_it(new, Hq):
    """NaN codes in keys and values: rows that see the token get them, others and other heads do not."""
    batch = Batch([(new, 150), (new, 150)], 16, 2, 64, seed=6).fill()
    q, qg = heads_bf16(batch.T, Hq, 64, 1.0, 4, "q")

    def spoil(b, p, h, name, d):
        page, at = int(batch.table[b, p // 16]), p % 16
        if name == "k":
            batch.cache["k"][page, h, at, d] = 0xFF
        else:
            batch.cache["v"][page, h, 0, d, at] = 0x7F
    spoil(0, 149, 0, "v", 3)                                    # the last token: only the last query sees it
    spoil(0, 148, 1, "k", 60)
    spoil(1, 20, 1, "v", 63)                                    # behind the window below
    got = attend(qg, batch.gpu(), new, chunk=256)
    check(batch, q, got)
    got = attend(qg, batch.gpu(), new, window=100)
    check(batch, q, got, window=100)


def test_far_scales_and_large_logits():
    """Blocks whose scales lie far apart; logits of several hundred, where one key takes all; equal logits."""
    batch = Batch([(1, 100), (20, 100)], 16, 1, 64, seed=6).fill()
    batch.cache["ks"][:, :, :] = np.where(np.arange(batch.n_pages)[:, None, None] % 3 == 0, 131, 118)
    batch.cache["vs"][:, :, :] = np.where(np.arange(batch.n_pages)[:, None, None] % 2 == 0, 30, 140)
    for std in (0.0, 1.0, 30.0):
        q, qg = heads_bf16(batch.T, 4, 64, std, 4, "q")
        check(batch, q, attend(qg, batch.gpu(), 20), what=str(std))


def test_strides_streams_and_no_lse():
    t = torch()
    batch = Batch([(3, 40), (1, 90)], 32, 2, 128, seed=6).fill()
    T, Hq, D = batch.T, 4, 128
    qkv, qkvg = heads_bf16(T, Hq + 4, D, 1.0, 4, "q")
    wide = t.full((T + 1, Hq + 1, D), 7.0, dtype=t.bfloat16, device="cuda")
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    g = batch.gpu()
    attend(qkvg[:, :Hq], g, 3, out=wide[:T, :Hq], lse=False, stream=s)
    s.synchronize()
    want, _ = attend(qkvg[:, :Hq].contiguous(), g, 3)
    assert t.equal(wide[:T, :Hq], want)
    assert bool((wide[T] == 7.0).all()) and bool((wide[:, Hq] == 7.0).all())
    check(batch, qkv[:, :Hq], attend(qkvg[:, :Hq], g, 3))


@pytest.mark.parametrize("new", [1, 2, 5, 50])
@pytest.mark.parametrize("chunk", [256, 1 << 20])
def test_bits_do_not_depend_on_the_batch(new, chunk):
    """One sequence alone, and among others of other lengths on other pages."""
    t = torch()
    G = 8
    alone = Batch([(new, 700)], 16, 2, 64, seed=2).fill()
    many = Batch([(1, 60), (new, 700), (new, 1300), (1, 5)], 16, 2, 64, seed=3).fill()
    for p in range(44):
        for name in ("k", "v", "ks", "vs"):
            many.cache[name][many.table[1, p]] = alone.cache[name][alone.table[0, p]]
    q, qg = heads_bf16(many.T, 2 * G, 64, 1.0, 4, "q")
    a, al = attend(qg[1:1 + new], alone.gpu(), new, chunk=chunk)
    b, bl = attend(qg, many.gpu(), new, chunk=chunk)
    assert t.equal(a.view(t.int16), b[1:1 + new].view(t.int16)) and t.equal(al, bl[1:1 + new])


def test_chunks_by_the_rule():
    """The rule's chunk is a multiple of the unit, and naming it gives the same bits as leaving it out."""
    t = torch()
    batch = Batch([(1, 3000)], 64, 1, 64, seed=2).fill()
    q, qg = heads_bf16(1, 4, 64, 1.0, 4, "q")
    g = batch.gpu()
    n = g.page_table.shape[1] * 64
    chunk = dsl.lora_kv_attention_chunk(1, 4, 1, 64, n)
    assert chunk % 256 == 0 and 0 < chunk < n
    assert t.equal(attend(qg, g, 1)[0], attend(qg, g, 1, chunk=chunk)[0])


def test_many_sequences():
    """More sequences than a wave has lanes."""
    batch = Batch([(1, 1 + 5 * b % 90) for b in range(200)], 16, 1, 64, seed=2).fill()
    q, qg = heads_bf16(batch.T, 2, 64, 1.0, 4, "q")
    check(batch, q, attend(qg, batch.gpu(), 1))


def test_tables_that_make_no_sense():
    """Offsets that fall or lie outside the rows, lengths below zero or past the pages: the calls end, and the sequence
    whose entries are sound gets what it gets among sound ones."""
    t = torch()
    batch = Batch([(2, 10), (2, 20), (2, 30)], 16, 1, 64, seed=5).fill()
    g = batch.gpu()
    q, qg = heads_bf16(6, 2, 64, 1.0, 4, "q")
    for new in (1, 10, 100):
        want, _ = attend(qg, g, new)
        for cu, lens, sound in (([0, 9, 2, 6], [10, 20, 30], None), ([-5, 2, 4, 6], [10, 20, 30], 2),
                                ([0, 2, 4, 600], [10, 20, 30], 0), ([0, 2, 4, 6], [-10, 2 ** 31 - 1, 30], 2)):
            out, _ = attend(qg, g._replace(cu_tokens=ints(cu), seq_lens=ints(lens)), new)
            if sound is not None:
                rows = slice(2 * sound, 2 * sound + 2)
                assert t.equal(out[rows], want[rows])


def test_captured_into_a_graph():
    """A decode step (append, then attention) captured once and replayed with other lengths, pages and inputs; eager work
    and other graphs' calls between the replays."""
    t = torch()
    H, Hq, D, P, B = 2, 8, 64, 16, 3
    batch = Batch([(1, 400)] * B, P, H, D, seed=2)
    batch.lens[:] = 0
    g = batch.gpu()
    x = t.zeros(B, Hq + 2 * H, D, dtype=t.bfloat16, device="cuda")
    q = t.zeros(B, Hq, D, dtype=t.bfloat16, device="cuda")
    out = t.zeros(B, Hq, D, dtype=t.bfloat16, device="cuda")
    ws = t.empty(dsl.lora_kv_attention_workspace_bytes(B, Hq, H, D, 1, 400), dtype=t.uint8, device="cuda")
    assert ws.numel() > 0

    def step():
        dsl.lora_kv_append(x[:, Hq:Hq + H], x[:, Hq + H:], g, q=x[:, :Hq], q_out=q)
        dsl.lora_kv_attention(q, g, out, 1, max_len=400, workspace=ws)
    step()
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step()
    twin = g._replace(**{n: getattr(g, n).clone() for n in ("k", "v", "k_scales", "v_scales")})
    ws2, out2, q2 = t.empty_like(ws), t.empty_like(out), t.empty_like(q)
    for n in range(1, 400):
        x.copy_(heads_bf16(B, Hq + 2 * H, D, 1.0, n, "x")[1])
        g.seq_lens.copy_(t.tensor([n, max(1, n - 13), (n + 1) // 2], dtype=t.int32))
        graph.replay()
        dsl.lora_kv_append(x[:, Hq:Hq + H], x[:, Hq + H:], twin, q=x[:, :Hq], q_out=q2)
        dsl.lora_kv_attention(q2, twin, out2, 1, max_len=400, workspace=ws2)
        if n % 57 == 0 or n > 397:
            t.cuda.synchronize()
            assert t.equal(out.view(t.int16), out2.view(t.int16)), n
    assert t.equal(g.k, twin.k) and t.equal(g.v, twin.v)
