"""Attention over the paged 8-bit cache at its edges: every kernel variant (rows of a key head that the waves split, two
tiles of them, many) with windows, pages that are not there, blocks that were never written and values that are NaN."""
import numpy as np
import pytest

import deterministic_split_lora_amd as dsl
from oracle import bf16_to_f64, kv
from synth import rng_for
from tests.helpers import bf16_from_gpu, gpu_available, torch
from tests.kv_helpers import Batch, attend, heads_bf16, ints
from tests.test_gpu_kv_append import bf16_round, ready, rope_table
from tests.test_gpu_kv_attention import check

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

NEW = [1, 5, 40]                                                # with 8 rows a token: 8, 40 and 320 rows of a key head


def bits(t):
    return t.view(torch().int16 if t.dtype == torch().bfloat16 else torch().int32)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("P", [16, 64, 128])
@pytest.mark.parametrize("new", NEW)
def test_blocks_before_the_window_may_hold_anything(D, P, new):
    """Codes and scales of blocks that no query of the step sees any more: NaN, the largest, scales that are none."""
    t = torch()
    window = 10
    batch = Batch([(new, 150), (new, 107)], P, 1, D, seed=3).fill()
    q, qg = heads_bf16(batch.T, 8, D, 1.0, 4, "q")
    want, wlse = attend(qg, batch.gpu(), new, window=window)
    for scale in (0, 247, 254, 255):
        for code in (0x7E, 0xFE, 0x7F):
            for b, n in ((0, 150), (1, 107)):
                for block in range((n - new - window + 1) // 16):
                    page, w = batch.table[b, block * 16 // P], block * 16 % P // 16
                    batch.cache["ks"][page, :, w] = batch.cache["vs"][page, :, w] = scale
                    batch.cache["k"][page, :, w * 16:(w + 1) * 16] = code
                    batch.cache["v"][page, :, w] = code
            out, lse = attend(qg, batch.gpu(), new, window=window)
            assert not bool(t.isnan(out).any()), (scale, code)
            assert t.equal(bits(out), bits(want)) and t.equal(bits(lse), bits(wlse)), (scale, code)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", NEW)
def test_weights_keep_eleven_bits(D, new):
    """The bounds of oracle/kv.py with 2^-11 in the place of 2^-8 for the p (fp16, half a step), and for what is below
    2^-29 of the largest half a step of 2^-39 of it, times codes up to 448, for every key: 448 2^-40 < 2^-31."""
    batch = Batch([(new, 60), (new, 45)], 16, 1, D, seed=7).fill()
    q, qg = heads_bf16(batch.T, 8, D, 1.0, 4, "q")
    args = (batch.table, batch.lens, batch.cu, 16, D ** -0.5)
    out, _, tol, _ = kv.attention(q, batch.cache, *args)
    size = kv.attention(q, dict(batch.cache, v=batch.cache["v"] & 127), *args)[0]       # sums of p |v|
    used = batch.cache["vs"][batch.table[batch.table >= 0]].max()
    tol = tol - size * (2.0 ** -8 - 2.0 ** -11) + 60 * 2.0 ** (int(used) - 127 - 31)
    for chunk in (0, 256):
        got = bf16_to_f64(bf16_from_gpu(attend(qg, batch.gpu(), new, chunk=chunk)[0]))
        assert np.all(np.abs(got - out) <= tol), np.max(np.abs(got - out) / tol)


@pytest.mark.parametrize("new", NEW)
def test_largest_values_and_zeros(new):
    """Values at the top of bf16, whose sums would pass the largest float; a long run of zeros, whose scale is the least."""
    t = torch()
    batch = Batch([(new, 20000), (new, 300)], 128, 1, 64, seed=7)
    batch.cache["k"][:] = 0
    batch.cache["ks"][:] = 127
    batch.cache["v"][:], batch.cache["vs"][:] = 0, 27
    for page in batch.table[1][batch.table[1] >= 0]:
        batch.cache["v"][page], batch.cache["vs"][page] = 0x7E, 246
    q, qg = heads_bf16(batch.T, 8, 64, 1.0, 4, "q")
    for chunk in (0, 1 << 20):
        out, lse = attend(qg, batch.gpu(), new, chunk=chunk)
        o = bf16_to_f64(bf16_from_gpu(out))
        assert not o[:new].any()
        assert np.all(np.abs(o[new:] / 2.0 ** 127 - 1.75) <= 1.75 * 2.0 ** -8)
        # sums of equal numbers in fp32, and the size of what the scale's exponent adds to the logarithm
        want = np.log(np.concatenate([np.arange(20000 - new, 20000), np.arange(300 - new, 300)]) + 1.0)
        assert np.all(np.abs(lse.double().cpu().numpy() - want[:, None]) <= 2.0 ** -16)


@pytest.mark.parametrize("new", NEW)
def test_the_longest_chunk(new):
    """A chunk past every length, up to the largest number, is one chunk of the whole."""
    t = torch()
    batch = Batch([(new, 700), (new, 90)], 16, 1, 64, seed=7).fill()
    q, qg = heads_bf16(batch.T, 8, 64, 1.0, 4, "q")
    want, wlse = attend(qg, batch.gpu(), new, chunk=768)
    for chunk in (1 << 31, (1 << 63) - 256):
        out, lse = attend(qg, batch.gpu(), new, chunk=chunk)
        assert t.equal(bits(out), bits(want)) and t.equal(bits(lse), bits(wlse))


def test_a_step_without_tokens():
    """Every argument of a step given, and no row in any of them."""
    t = torch()
    batch = Batch([(0, 20), (0, 5)], 16, 2, 64, seed=7).fill()
    g = batch.gpu()
    x = t.empty(0, 8, 64, dtype=t.bfloat16, device="cuda")
    norm = t.ones(64, dtype=t.bfloat16, device="cuda")
    rope = t.zeros(30, 64, device="cuda")
    out = t.empty(0, 4, 64, dtype=t.bfloat16, device="cuda")
    dsl.lora_kv_append(x[:, 4:6], x[:, 6:], g, q=x[:, :4], q_out=out, q_norm=norm, k_norm=norm, rope=rope)
    dsl.lora_kv_attention(out, g, t.empty_like(out), 1, max_len=20, lse=t.empty(0, 4, device="cuda"))
    t.cuda.synchronize()
    batch.same(g)


def test_a_rotation_table_without_rows_is_refused():
    t = torch()
    g = Batch([(2, 20)], 16, 2, 64, seed=7).fill().gpu()
    x = t.zeros(2, 4, 64, dtype=t.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="rope"):
        dsl.lora_kv_append(x[:, :2], x[:, 2:], g, rope=t.empty(0, 64, device="cuda"))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_drafts_that_are_taken_back(D):
    """A prompt, a token with drafts behind it of which one has values 200 times as large, and tokens that go on from the
    accepted one: the same as the reference, whose byte stays raised."""
    batch = Batch([(1, 40), (1, 40)], 32, 2, D, seed=7)
    g = None
    plain = None
    for i, (new, lens) in enumerate([((20, 4), (20, 4)), ((3, 4), (23, 8)), ((1, 2), (22, 7)), ((1, 1), (23, 8))]):
        batch.lens = np.array(lens, dtype=np.int32)
        batch.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        batch.T = int(batch.cu[-1])
        x, xg = heads_bf16(batch.T, 4, D, 1.0, i, "x")
        if i == 1:
            plain = batch.cache["ks"][batch.table[:, 0]].copy(), batch.cache["vs"][batch.table[:, 0]].copy()
            scale = np.ones(batch.T)
            scale[[2, 5]] = 256.0                               # drafts: the second of the one, the second of the other
            x = x * scale[:, None, None]
            xg = (xg.float() * torch().from_numpy(scale).float().cuda()[:, None, None]).to(torch().bfloat16)
        g = batch.gpu()
        dsl.lora_kv_append(xg[:, :2], xg[:, 2:], g)
        torch().cuda.synchronize()
        kv.append(batch.cache, x[:, :2], x[:, 2:], batch.table, batch.lens, batch.cu, 32)
        batch.same(g)
    for name, old in zip(("ks", "vs"), plain):
        now = batch.cache[name][batch.table[:, 0]]
        assert np.all(now[0, :, 1] > old[0, :, 1] + 5) and np.all(now[1, :, 0] > old[1, :, 0] + 5)


def any_values(batch, seed):
    """Codes that are no NaN, and scales within a factor of 2^8."""
    rng = rng_for(seed, "kv-any")
    c = batch.cache
    for name in ("k", "v"):
        c[name][:] = rng.integers(0, 127, c[name].shape) | rng.integers(0, 2, c[name].shape) << 7
    for name in ("ks", "vs"):
        c[name][:] = rng.integers(113, 122, c[name].shape)
    return batch


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,longest", [(1, 2), (2, 2), (1, 8), (3, 8), (5, 8), (1, 100), (20, 100)])
@pytest.mark.parametrize("chunk", [512, 2048])
def test_bits_with_a_named_chunk(D, new, longest, chunk):
    """A sequence alone, with the sizes it has, and beside one twenty times as long and one with more new tokens: the same
    bits where the chunk is named and the longest run of new tokens times 8 rows lies in the same class."""
    t = torch()
    alone = any_values(Batch([(new, 700)], 64, 1, D, seed=2), 2)
    many = any_values(Batch([(longest, 800), (1, 14000), (new, 700), (1, 1)], 64, 1, D, seed=3), 3)
    at = longest + 1
    for p in range(11):
        for name in ("k", "v", "ks", "vs"):
            many.cache[name][many.table[2, p]] = alone.cache[name][alone.table[0, p]]
    q, qg = heads_bf16(many.T, 8, D, 1.0, 4, "q")
    least = {2: new, 8: max(new, 3), 100: max(new, 9)}[longest]             # of the class
    a, al = attend(qg[at:at + new], alone.gpu(), least, max_len=700, chunk=chunk)
    b, bl = attend(qg, many.gpu(), longest, chunk=chunk)
    assert t.equal(bits(a), bits(b[at:at + new])) and t.equal(bits(al), bits(bl[at:at + new]))
    assert not bool(t.isnan(b).any())


SIZES = [(D, P) for D in (64, 128, 256) for P in (16, 64, 128)]


def ragged(new, P, D):
    """Two sequences of these new tokens, one whose pages are all missing, more new tokens than tokens, no token."""
    return Batch([(new, 200), (new, 100), (2, 30), (3, 2), (1, 0)], P, 2, D, seed=5, rows_behind=2).fill()


@pytest.mark.parametrize("D,P", SIZES)
@pytest.mark.parametrize("new", NEW[:2] + [20])
def test_pages_that_are_not_there(D, P, new):
    batch = ragged(new, P, D)
    batch.table[0, 100 // P] = -1
    batch.table[0, 199 // P] = batch.n_pages                    # the newest tokens
    batch.table[1, 0] = 2 ** 31 - 1                             # of the second, at pages of 128, everything
    batch.table[2, :] = -7
    q, qg = heads_bf16(batch.T, 16, D, 1.0, 4, "q")
    g = batch.gpu()
    check(batch, q, attend(qg, g, new))
    check(batch, q, attend(qg, g, new, window=40, chunk=256), window=40)
    check(batch, q, attend(qg, g, new, causal=False), causal=False)


@pytest.mark.parametrize("D,P", SIZES)
@pytest.mark.parametrize("new", NEW[:2] + [20])
def test_nan_codes(D, P, new):
    """Values and keys that are NaN, in columns from one end of the head to the other."""
    batch = ragged(new, P, D)

    def spoil(b, p, h, name, d):
        page, at = int(batch.table[b, p // P]), p % P
        if name == "k":
            batch.cache["k"][page, h, at, d] = 0xFF
        else:
            batch.cache["v"][page, h, at // 16, d, at % 16] = 0x7F
    for d in (0, D // 2 + 5, D - 1):
        spoil(0, 199, 0, "v", d)                                # the last token: only the last query sees it
    spoil(0, 200 - (new + 1) // 2, 0, "v", D // 2 - 3)          # one among the new ones
    spoil(0, 198, 1, "k", D - 1)
    spoil(1, 20, 1, "v", D - 2)                                 # behind the window below
    spoil(1, 21, 0, "k", 3)
    spoil(1, 70, 1, "v", 1)
    q, qg = heads_bf16(batch.T, 16, D, 1.0, 4, "q")
    g = batch.gpu()
    check(batch, q, attend(qg, g, new))
    check(batch, q, attend(qg, g, new, window=40, chunk=256), window=40)
    check(batch, q, attend(qg, g, new, causal=False), causal=False)


TABLES = [  # offsets, lengths, the sequences whose entries are sound (none: their order is not)
    ([0, 9, 2, 6], [10, 20, 30], []), ([6, 4, 2, 0], [10, 20, 30], []), ([-5, 2, 4, 6], [10, 20, 30], [1, 2]),
    ([0, 2, 4, 600], [10, 20, 30], [0, 1]), ([0, 2, 4, 6], [-10, 2 ** 31 - 1, 30], [2]),
    ([0, 2, 4, 6], [2 ** 31 - 1, 20, -2 ** 31], [1])]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cu,lens,sound", TABLES)
def test_append_with_tables_that_make_no_sense(D, cu, lens, sound):
    """Sound sequences get what they get among sound ones; nothing else is written, in the pool, between its pages or
    around the queries."""
    t = torch()
    batch = Batch([(2, 10), (2, 20), (2, 30)], 16, 1, D, seed=5).fill()
    g = batch.gpu(pad=32)
    g = g._replace(cu_tokens=ints(cu), seq_lens=ints(lens))
    x, xg = heads_bf16(6, 5, D, 1.0, 1, "x")
    w = heads_bf16(1, 1, D, 1.0, 2, "w")
    rope = rope_table(40, D)
    around = t.full((8, 4, D), 7.0, dtype=t.bfloat16, device="cuda")
    dsl.lora_kv_append(xg[:, 3:4], xg[:, 4:], g, q=xg[:, :3], q_out=around[1:7, :3], q_norm=w[1].view(-1),
                       k_norm=w[1].view(-1), rope=t.from_numpy(rope).cuda())
    t.cuda.synchronize()
    assert bool((around[[0, 7]] == 7.0).all()) and bool((around[:, 3] == 7.0).all())
    for a in (g.k, g.v, g.k_scales, g.v_scales):
        whole = a.as_strided((batch.n_pages, a.stride(0)), (a.stride(0), 1))
        assert bool((whole[:, a[0].numel():] == 0xEE).all())
    out = around[1:7, :3].float().cpu().numpy()
    for b in sound:
        rows = range(cu[b], cu[b + 1])
        at = [(b, lens[b] - (cu[b + 1] - i), 0) for i in rows]
        part = x[list(rows)]
        k = ready(part[:, 3:4], w[0][0, 0], rope, at, False)
        kv.append(batch.cache, k, part[:, 4:], batch.table[[b]], [lens[b]], [0, 2], 16)
        want = bf16_to_f64(bf16_round(ready(part[:, :3], w[0][0, 0], rope, at, False)))
        assert np.array_equal(out[list(rows)], want)
    if sound:
        batch.same(g)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 5, 40])
@pytest.mark.parametrize("cu,lens,sound", TABLES)
def test_attention_with_tables_that_make_no_sense(D, new, cu, lens, sound):
    t = torch()
    batch = Batch([(2, 10), (2, 20), (2, 30)], 16, 1, D, seed=5).fill()
    g = batch.gpu()
    q, qg = heads_bf16(6, 8, D, 1.0, 4, "q")
    want, wlse = attend(qg, g, new)
    bad = g._replace(cu_tokens=ints(cu), seq_lens=ints(lens))
    for chunk in (0, 256):
        around = t.full((8, 9, D), 7.0, dtype=t.bfloat16, device="cuda")
        out, lse = attend(qg, bad, new, out=around[1:7, :8], max_len=700, chunk=chunk)
        assert bool((around[[0, 7]] == 7.0).all()) and bool((around[:, 8] == 7.0).all())
        for b in sound:
            rows = slice(cu[b], cu[b + 1])
            assert t.equal(bits(out[rows].contiguous()), bits(want[rows])) and t.equal(bits(lse[rows]), bits(wlse[rows]))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_step_in_two_calls(D):
    """A prompt's tokens and single ones over parts of the batch's tables, each call with its own sizes: every row is
    served, by the call whose sequences it belongs to."""
    t = torch()
    batch = Batch([(30, 90), (1, 40), (1, 130), (1, 7)], 16, 1, D, seed=5, start=1, rows_behind=2).fill()
    q, qg = heads_bf16(batch.T, 8, D, 1.0, 4, "q")
    g = batch.gpu()
    first = g._replace(page_table=g.page_table[:1], seq_lens=g.seq_lens[:1], cu_tokens=g.cu_tokens[:2])
    rest = g._replace(page_table=g.page_table[1:], seq_lens=g.seq_lens[1:], cu_tokens=g.cu_tokens[1:])
    out, lse = attend(qg, first, 30, max_len=90)
    more, mlse = attend(qg, rest, 1, max_len=130)
    assert bool((out[31:] == 7.0).all()) and bool((more[:31] == 7.0).all())
    rows = t.arange(batch.T, device="cuda") >= 31
    check(batch, q, (t.where(rows[:, None, None], more, out), t.where(rows[:, None], mlse, lse)))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", NEW)
def test_weights_far_below_the_largest(D, new):
    """A column in which the key of the largest weight has 0: what is left is the second's, with half a step of 2^-40
    of the largest weight; 2^-8 is the output's half step, and 2^-10 holds the weight's own, 2^-11, and the fp32 ones."""
    n = max(new, 2)
    for logit, code in ((-1.0, 0xB8), (-18.0, 0xD9), (-22.0, 0xDB), (-24.0, 0xDC), (-26.0, 0xDD)):
        assert kv.VALUES[code] == logit
        batch = Batch([(new, n)], 64, 1, D, seed=5)
        c, page = batch.cache, batch.table[0, 0]
        c["k"][page], c["v"][page], c["ks"][page], c["vs"][page] = 0, 0, 127, 110
        c["k"][page, 0, 1, 0] = code
        c["k"][page, 0, 2:, 0] = 0xF7                           # -240: nothing of the others
        c["v"][page, 0, 0, 0, 0] = 0x7E                         # 448, in the first column the first token's
        c["v"][page, 0, 0, D - 1, 1] = 0x7E                     # in the last one the second's
        q = torch().zeros(new, 8, D, dtype=torch().bfloat16, device="cuda")
        q[:, :, 0] = 1.0
        out = bf16_to_f64(bf16_from_gpu(attend(q, batch.gpu(), new, scale=1.0)[0]))[1 if new > 1 else 0:]
        w, one = np.exp(logit), 448.0 * 2.0 ** -17
        first, last = one / (1 + w), one * w / (1 + w)
        assert np.all(np.abs(out[:, :, 0] - first) <= first * (2.0 ** -8 + 2.0 ** -10))
        assert np.all(np.abs(out[:, :, D - 1] - last) <= last * (2.0 ** -8 + 2.0 ** -10) + one * 2.0 ** -40), (logit, out[0, 0, D - 1], last)
        assert not out[:, :, 1:D - 1].any()
