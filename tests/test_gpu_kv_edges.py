"""Attention over the paged 8-bit cache at its edges: every kernel variant (rows of a key head that the waves split, two
tiles of them, many) with windows, pages that are not there, blocks that were never written and values that are NaN."""
import numpy as np
import pytest

import deterministic_split_lora_amd as dsl
from oracle import bf16_to_f64, kv
from synth import rng_for
from tests.helpers import bf16_from_gpu, gpu_available, torch
from tests.kv_helpers import Batch, attend, heads_bf16

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
