"""Appending to the paged 8-bit cache on the GPU against the CPU reference (oracle/kv.py): codes, scales and queries bit
for bit where every operation rounds alike, and within the bounds of the formula in 64 bits."""
import numpy as np
import pytest

import deterministic_split_lora_amd as dsl
from oracle import bf16_to_f64, kv
from synth import normal_bf16
from tests.helpers import bf16_from_gpu, bf16_to_gpu, f32_to_gpu, gpu_available, torch
from tests.kv_helpers import Batch, heads_bf16

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

EPS = 1e-6


def rope_table(n, dim):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, dim, 2) / dim)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def ready(x, w, rope, rows, pairs, dtype=np.float32):
    """Normed and rotated heads of a step's rows, in dtype."""
    y = kv.head_norm(x, w, EPS, dtype)
    if rope is None:
        return y
    out = y.copy()
    for i, r in enumerate(rows):
        if r is not None:
            row = rope[r[1]] if 0 <= r[1] < rope.shape[0] else np.full(rope.shape[1], np.nan)
            out[i] = kv.rotate(y[i], row.astype(dtype), pairs)
    return out


def bf16_round(x):
    """Bits of fp32 values rounded to bf16, ties to even."""
    u = x.astype(np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def run(batch, g, Hq, norm, rope, pairs, seed, in_place=False, std=1.0):
    """One append on both sides; checks the queries, returns nothing: the caches are compared by the caller."""
    t = torch()
    T, H, D = batch.T, batch.H, batch.D
    x, xg = heads_bf16(T, Hq + 2 * H, D, std, seed, "qkv")
    wq = normal_bf16((D,), 1.0, seed, "wq") if norm else None
    wk = normal_bf16((D,), 1.0, seed, "wk") if norm else None
    f = lambda w: None if w is None else bf16_to_f64(w)  # noqa: E731
    q_out = xg[:, :Hq] if in_place else t.full((T, Hq, D), 7.0, dtype=t.bfloat16, device="cuda")
    before = bf16_from_gpu(q_out)
    dsl.lora_kv_append(xg[:, Hq:Hq + H], xg[:, Hq + H:], g, q=xg[:, :Hq], q_out=q_out,
                       q_norm=None if wq is None else bf16_to_gpu(wq), k_norm=None if wk is None else bf16_to_gpu(wk),
                       rope=None if rope is None else f32_to_gpu(rope), pairs=pairs, eps=EPS)
    t.cuda.synchronize()
    rows = kv.step_rows(batch.table, batch.lens, batch.cu, T, batch.P, batch.n_pages)
    k = ready(x[:, Hq:Hq + H], f(wk), rope, rows, pairs)
    kv.append(batch.cache, k, x[:, Hq + H:], batch.table, batch.lens, batch.cu, batch.P)
    want = bf16_round(ready(x[:, :Hq], f(wq), rope, rows, pairs))
    got = bf16_from_gpu(q_out)
    for i, r in enumerate(rows):
        if r is None:
            assert np.array_equal(got[i], before[i]), f"row {i} of no sequence was written"
        else:
            assert np.array_equal(got[i], want[i]), f"queries of row {i}"
    # against the formula in 64 bits: rounding to bf16 (half a step), and of fp32 operations 2^-20 of the pair
    exact = ready(x[:, :Hq], f(wq), rope, rows, pairs, np.float64)
    size = np.abs(exact) + (np.abs(exact).max(-1, keepdims=True) if rope is not None else 0)
    for i, r in enumerate(rows):
        if r is not None:
            err = np.abs(bf16_to_f64(got[i]) - exact[i])
            nan = np.isnan(exact[i])                            # a position outside the table
            assert np.array_equal(np.isnan(err), nan)
            assert np.all((err <= np.abs(exact[i]) * 2.0 ** -8 + size[i] * 2.0 ** -20) | nan)
    return x


@pytest.mark.parametrize("D,Hq,H,P", [(128, 8, 2, 64), (64, 3, 3, 16), (256, 4, 1, 32), (128, 32, 8, 128), (64, 7, 1, 1024)])
@pytest.mark.parametrize("norm,rope_dim,pairs", [(False, 0, False), (True, 1, False), (True, 1, True), (False, 2, False),
                                                 (False, 2, True)])
def test_append_in_steps(D, Hq, H, P, norm, rope_dim, pairs):
    """Prompts in chunks that end inside a block, then single tokens whose values grow and shrink; a sequence that is taken
    back to an earlier token and goes on from there."""
    rope = rope_table(400, D // rope_dim // 16 * 16) if rope_dim else None
    steps = [[(21, 21), (21, 21), (1, 1), (0, 0)], [(11, 32), (6, 16), (39, 40), (3, 3)],
             [(1, 33), (34, 50), (7, 47), (0, 3)], [(1, 34), (1, 51), (1, 48), (16, 19)],
             [(1, 35), (1, 52), (1, 49), (1, 20)]]
    batch = None
    for step, lengths in enumerate(steps):
        nxt = Batch([(m, max(steps[i][b][1] for i in range(5))) for b, (m, _) in enumerate(lengths)], P, H, D, seed=1)
        nxt.lens = np.array([n for _, n in lengths], dtype=np.int32)
        if batch is not None:
            nxt.cache = batch.cache
        batch = nxt
        g = batch.gpu(pad=16 * (step % 2))
        run(batch, g, Hq, norm, rope, pairs, seed=step, in_place=step % 2 == 1, std=[1.0, 0.5, 3.0, 0.1, 40.0][step])
        batch.same(g)


def test_large_batch_and_long_prompt():
    """More sequences than a wave has lanes, and a prompt of several hundred blocks next to single tokens."""
    lengths = [(1, 1 + 7 * b % 45) for b in range(150)] + [(3000, 3005)] + [(2, 2)] * 3
    batch = Batch(lengths, 32, 2, 64, seed=3, start=5, rows_behind=9).fill()
    g = batch.gpu()
    run(batch, g, 4, True, rope_table(3005, 64), False, seed=5)
    batch.same(g)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [[1] * 9, [0, 3, 0, 1, 2, 0, 0, 2, 1], [9] + [0] * 8, [0, 0, 40] + [0] * 37])
def test_as_many_tokens_as_sequences(D, new):
    """A step of single tokens, and others that only count as many: sequences without any, with blocks of several."""
    lengths = [(n, n + 13 * b % 40) for b, n in enumerate(new)]
    batch = Batch(lengths, 16, 2, D, seed=3).fill()
    g = batch.gpu(pad=16)
    assert batch.T == len(new)
    run(batch, g, 3, True, rope_table(100, D), True, seed=5)
    batch.same(g)


def test_columns_of_a_wider_table():
    """The page table as a view of a wider one."""
    t = torch()
    batch = Batch([(3, 40), (2, 33)], 16, 1, 64, seed=4).fill()
    wide = t.full((2, 10), 7 << 20, dtype=t.int32, device="cuda")
    wide[:, 2:2 + batch.table.shape[1]] = t.from_numpy(batch.table).cuda()
    g = batch.gpu()
    g = g._replace(page_table=wide[:, 2:2 + batch.table.shape[1]])
    run(batch, g, 1, False, None, False, seed=5)
    batch.same(g)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_codes_are_the_nearest(D):
    """Values of one block against the formula in 64 bits: half a step of the code, the scale the least that fits."""
    batch = Batch([(16, 16), (5, 5), (16, 16)], 16, 1, D, seed=9)
    g = batch.gpu()
    k, kg = heads_bf16(37, 1, D, 3.0, 4, "k")
    v, vg = heads_bf16(37, 1, D, 0.01, 5, "v")
    dsl.lora_kv_append(kg, vg, g)
    torch().cuda.synchronize()
    batch.cache = {n: a.cpu().numpy() for n, a in (("k", g.k), ("v", g.v), ("ks", g.k_scales), ("vs", g.v_scales))}
    for b, (n, first) in enumerate(((16, 0), (5, 16), (16, 21))):
        gk, gv, _ = kv.sequence(batch.cache, batch.table, b, n, 16)
        for got, x in ((gk, k[first:first + n]), (gv, v[first:first + n])):
            top = np.abs(x).max()
            scale = 2.0 ** np.ceil(np.log2(top / 448.0))
            step = np.maximum(2.0 ** (np.floor(np.log2(np.abs(x) / scale + 1e-300)) - 3), 2.0 ** -9) * scale
            assert np.all(np.abs(got - x) <= step / 2)


def test_unusual_values():
    """NaN, infinities, zeros, the largest and the smallest values, blocks of nothing finite."""
    t = torch()
    D, P = 64, 32
    rows = []
    for fill in (0.0, np.nan, np.inf, -np.inf, 3.3895314e38, 1e-38, 448.0, 449.0, 2.0 ** -120):
        x = np.zeros((16, 1, D))
        x[3, 0, 5] = fill
        x[4, 0, 6] = 1.5 if fill != 1e-38 else 0.0
        rows.append(x)
        y = np.full((16, 1, D), fill)
        rows.append(y)
    x = np.concatenate(rows)
    xg = t.from_numpy(x.astype(np.float32)).cuda().to(t.bfloat16)
    x = xg.double().cpu().numpy()
    batch = Batch([(16, 16)] * (len(x) // 16), P, 1, D, seed=2)
    g = batch.gpu()
    dsl.lora_kv_append(xg, xg, g)
    t.cuda.synchronize()
    kv.append(batch.cache, x, x, batch.table, batch.lens, batch.cu, P)
    batch.same(g)


def test_growing_scale_rounds_the_earlier_codes():
    """A block whose later tokens are larger and larger: codes that turn subnormal, then zero."""
    t = torch()
    batch = Batch([(1, 16)], 16, 1, 64, seed=6)
    g = batch.gpu()
    for p in range(16):
        batch.lens[:] = p + 1
        g.seq_lens.fill_(p + 1)
        x, xg = heads_bf16(1, 1, 64, 2.0 ** (2 * p - 8 if p % 3 else -8), p, "grow")
        dsl.lora_kv_append(xg, xg, g)
        kv.append(batch.cache, x, x, batch.table, batch.lens, batch.cu, 16)
    t.cuda.synchronize()
    batch.same(g)


def test_what_is_not_there_stays():
    """Missing pages, positions before the start and past the table, rows of no sequence, sequences without new tokens."""
    t = torch()
    batch = Batch([(40, 40), (3, 3), (0, 20), (5, 2), (2, 0), (4, 70)], 16, 2, 64, seed=8, start=3, rows_behind=4).fill()
    batch.table[0, 1] = -1
    batch.table[1, 0] = batch.n_pages
    batch.table[5, 4] = 1 << 30
    g = batch.gpu()
    short = rope_table(30, 64)                                  # positions 30 .. rotate by NaN
    run(batch, g, 2, False, short, False, seed=1)
    batch.same(g)
    assert np.isnan(kv.VALUES[batch.cache["k"]]).any()
    narrow = g._replace(page_table=g.page_table[:, :1].contiguous())
    nar = Batch.__new__(Batch)
    nar.__dict__.update(batch.__dict__)
    nar.table = batch.table[:, :1].copy()
    run(nar, narrow, 2, False, None, False, seed=2)             # pages behind the table's width are not there
    nar.same(narrow)


def test_tables_that_make_no_sense_write_nothing_outside():
    """Offsets that fall or lie outside the rows, lengths below zero: the call ends, rows of sound sequences are right."""
    t = torch()
    batch = Batch([(2, 10), (2, 20), (2, 30)], 16, 1, 64, seed=5).fill()
    g = batch.gpu(pad=32)
    for cu, lens in (([0, 9, 2, 6], [10, 20, 30]), ([-5, 2, 4, 6], [10, 20, 30]), ([0, 2, 4, 600], [10, 20, 30]),
                     ([0, 2, 4, 6], [-10, 2 ** 31 - 1, 30])):
        g.cu_tokens.copy_(t.tensor(cu, dtype=t.int32))
        g.seq_lens.copy_(t.tensor(lens, dtype=t.int32))
        x, xg = heads_bf16(6, 3, 64, 1.0, 1, "x")
        out = t.empty(6, 1, 64, dtype=t.bfloat16, device="cuda")
        dsl.lora_kv_append(xg[:, 1:2], xg[:, 2:], g, q=xg[:, :1], q_out=out)
    t.cuda.synchronize()
    for a in (g.k, g.v):
        whole = a.as_strided((batch.n_pages, a.stride(0)), (a.stride(0), 1))
        assert bool((whole[:-1, a[0].numel():] == 0xEE).all())


def test_no_queries_no_tokens_and_another_stream():
    t = torch()
    batch = Batch([(3, 7), (1, 33)], 16, 2, 128, seed=4).fill()
    g = batch.gpu()
    x, xg = heads_bf16(4, 4, 128, 1.0, 1, "x")
    dsl.lora_kv_append(xg[:0, :2], xg[:0, 2:], g)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    dsl.lora_kv_append(xg[:, :2], xg[:, 2:], g, stream=s)
    s.synchronize()
    kv.append(batch.cache, x[:, :2], x[:, 2:], batch.table, batch.lens, batch.cu, 16)
    batch.same(g)


def test_bits_do_not_depend_on_the_batch():
    """A sequence appended alone and among others."""
    t = torch()
    x, xg = heads_bf16(50, 3, 64, 1.0, 1, "x")
    rope = f32_to_gpu(rope_table(64, 64))
    codes = []
    for lengths, at in (([(20, 23)], 0), ([(7, 9), (20, 23), (23, 40)], 7)):
        batch = Batch(lengths, 16, 1, 64, seed=2).fill()
        b = 0 if at == 0 else 1
        g = batch.gpu()
        # the sequence's earlier tokens alike on both sides
        for p in range(2):
            page = int(batch.table[b, p])
            g.k[page].fill_(0x30), g.v[page].fill_(0x31), g.k_scales[page].fill_(127), g.v_scales[page].fill_(126)
        rows = xg[:20] if at == 0 else t.cat([xg[20:27], xg[:20], xg[27:]])
        out = t.empty(rows.shape[0], 1, 64, dtype=t.bfloat16, device="cuda")
        dsl.lora_kv_append(rows[:, 1:2], rows[:, 2:], g, q=rows[:, :1], q_out=out, rope=rope)
        t.cuda.synchronize()
        pages = [int(batch.table[b, p]) for p in range(2)]
        codes.append([g.k[pages].cpu(), g.v[pages].cpu(), g.k_scales[pages].cpu(), g.v_scales[pages].cpu(),
                      out[at:at + 20].cpu()])
    for a, b in zip(*codes):
        assert t.equal(a, b)
