"""MX4 products through every schedule, with scales read by 16 bytes and by 4, against the 64-bit reference: whole and
ragged chunks, chunks that start inside a scale word, pitches that are no multiple of 16."""
import numpy as np
import pytest

import deterministic_split_lora_amd as dsl
from oracle import step
from tests.helpers import bf16_from_gpu, gpu_available, torch
from tests.test_gpu_step import Product, check_padding, f64, padded, quantized

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

POISON = 0xFF                                # a workspace of NaN


def product(p, S, rows=slice(None), y=None):
    """(y, whether the workspace was written, i.e. the chunks were split over workgroups)."""
    t = torch()
    x = p.xg[rows]
    M = x.shape[0]
    y = t.full((M, p.N), float("nan"), dtype=t.bfloat16, device="cuda") if y is None else y
    n = dsl.lora_mx4_linear_workspace_bytes(M, p.K, p.N, S)
    ws = t.full((n,), POISON, dtype=t.uint8, device="cuda") if n else None
    if p.mx:
        dsl.lora_mx4_linear_q(x, p.xs[rows], p.wq, p.ws, y, S, ws)
    else:
        dsl.lora_mx4_linear(x, p.wq, p.ws, y, S, ws)
    t.cuda.synchronize()
    return y, bool(n) and bool((ws != POISON).any())


def narrow_scales(p):
    """The same scales at a pitch that is no multiple of 16, so that they are read 4 bytes at a time."""
    t = torch()

    def copy(s):
        pitch = s.shape[1] + (4 if s.shape[1] % 16 == 0 else 0)
        out = t.full((s.shape[0], pitch), 0xEE, dtype=t.uint8, device="cuda")
        out[:, :s.shape[1]] = s
        return out
    p.ws = copy(p.ws)
    if p.mx:
        p.xs = copy(p.xs)
    return p


# M, K, N, split_k: the chunks go to workgroups of their own, for x of either kind
SPLIT = [
    (200, 5120, 2568, 4),                    # whole chunks, scales by 16 bytes
    (300, 8448, 2056, 2),                    # whole chunks, scale rows of 264 bytes
    (200, 8256, 2568, 2),                    # chunks of 129 blocks
    (130, 8832, 2056, 4),                    # chunks of 69 blocks: they start at every place of a word
    (65, 8704, 2568, 16),                    # chunks of 17 blocks
]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("M,K,N,S", SPLIT)
def test_split_schedule(M, K, N, S, mx):
    p = Product(M, K, N, 17 * M + K, mx).gpu()
    buf, y = padded(M, N)
    _, split = product(p, S, y=y)
    assert split, "this size is meant for the split schedule"
    check_padding(buf, M, N)
    p.check(f64(y), S)
    # the same rows in a batch of two, which the few-rows kernel takes, and from scales read the other way
    part, split = product(p, S, rows=slice(M - 2, M))
    assert not split
    assert np.array_equal(bf16_from_gpu(part), bf16_from_gpu(y)[M - 2:])
    again, split = product(narrow_scales(p), S)
    assert split and np.array_equal(bf16_from_gpu(again), bf16_from_gpu(y))


# all chunks in one workgroup: small, middle and large tiles, whole and ragged
TILES = [(1300, 416, 6144, 1), (1300, 288, 6144, 1), (1300, 512, 6144, 1), (2048, 288, 4096, 1), (2048, 1024, 4096, 1),
         (1100, 704, 6144, 2), (1100, 512, 6144, 2), (1800, 512, 4104, 4), (520, 320, 1032, 1), (260, 192, 3208, 2)]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("M,K,N,S", TILES)
def test_tiles_with_scales_read_by_4_and_by_16(M, K, N, S, mx):
    p = Product(M, K, N, 13 * M + K, mx).gpu()
    buf, y = padded(M, N)
    product(p, S, y=y)
    check_padding(buf, M, N)
    p.check(f64(y), S)
    narrow, _ = product(narrow_scales(p), S)
    assert np.array_equal(bf16_from_gpu(narrow), bf16_from_gpu(y))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("M,K,N,S", [(17, 1024, 520, 8), (20, 2048, 512, 8), (24, 4096, 1024, 4), (32, 8192, 264, 16),
                                     (29, 512, 136, 1), (31, 1024, 72, 2), (40, 4096, 512, 8), (50, 2048, 264, 4)])
def test_few_rows_of_whole_chunks(M, K, N, S, mx):
    p = Product(M, K, N, 19 * M + K, mx).gpu()
    buf, y = padded(M, N)
    product(p, S, y=y)
    check_padding(buf, M, N)
    p.check(f64(y), S)
    for a, b in [(0, 1), (3, 16), (M - 9, M)]:
        part, _ = product(p, S, rows=slice(a, b))
        assert np.array_equal(bf16_from_gpu(part), bf16_from_gpu(y)[a:b])


def test_quantised_x_against_its_values_with_a_workspace():
    """Quantised x and the bf16 values it stands for, at a size whose chunks are split: both within the bound of the same
    exact product."""
    t = torch()
    M, K, N, S = 130, 4096, 2056, 4
    p = Product(M, K, N, 3, False).gpu()
    q, s, code, sc = quantized(p.xg, M, K)
    v = t.empty(M, K, dtype=t.bfloat16, device="cuda")
    dsl.lora_mx4_dequantize(q, s, v)
    n = dsl.lora_mx4_linear_workspace_bytes(M, K, N, S)
    assert n > 0
    p.x = f64(v)
    for call in (lambda y, ws: dsl.lora_mx4_linear_q(q, s, p.wq, p.ws, y, S, ws),
                 lambda y, ws: dsl.lora_mx4_linear(v, p.wq, p.ws, y, S, ws)):
        ws = t.full((n,), POISON, dtype=t.uint8, device="cuda")
        y = t.full((M, N), float("nan"), dtype=t.bfloat16, device="cuda")
        call(y, ws)
        t.cuda.synchronize()
        p.check(f64(y), S)


@pytest.mark.parametrize("M", [3, 300])
def test_largest_scales(M):
    """With MX4 x, W's values enter exactly whatever their scale.  With bf16 x they do up to the scale byte 252, the largest
    that quantisation writes; beyond it a value past bf16's range is infinite, as from lora_mx4_dequantize."""
    t = torch()
    K, N = 128, 136
    codes = np.tile(np.arange(1, 8, dtype=np.uint8), K)[:K]
    p = Product(M, K, N, 9, True)
    p.wc = np.tile(codes, (N, 1))
    p.wc[1::2] |= 8
    p.wsc[:] = 252
    p.wsc[10:12] = 253
    p.wsc[20:22] = 254
    p.wc[22:24] = 2                                            # 1.0: 2^127 is finite
    p.wsc[22:24] = 254
    p.w = step.mx4_values(p.wc, p.wsc)
    p.xc = np.full((M, K), 3, dtype=np.uint8)                  # 1.5, positive: no sum cancels
    p.xsc[:] = 100
    p.x = step.mx4_values(p.xc, p.xsc)
    p.gpu()
    p.check(f64(product(p, 1)[0]), 1)

    x, deq = t.empty(M, K, dtype=t.bfloat16, device="cuda"), t.empty(N, K, dtype=t.bfloat16, device="cuda")
    dsl.lora_mx4_dequantize(p.xg, p.xs, x)
    dsl.lora_mx4_dequantize(p.wq, p.ws, deq)
    p.xg, p.mx = x, False
    got = f64(product(p, 1)[0])
    inf = np.isinf(f64(deq)).any(1)
    assert np.flatnonzero(inf).tolist() == [10, 11, 20, 21]
    assert np.array_equal(got[:, inf], np.tile(np.where(np.arange(N)[inf] % 2, -np.inf, np.inf), (M, 1)))
    e = p.x @ p.w.T
    tol = 2.0 ** -8 * np.abs(e) + (128 + 2) * 2.0 ** -23 * (np.abs(p.x) @ np.abs(p.w).T)
    assert np.all(np.abs(got - e)[:, ~inf] <= tol[:, ~inf])


def test_quantisation_writes_no_scale_past_252():
    """Of every finite bf16 magnitude."""
    t = torch()
    v = np.arange(0x7F80, dtype=np.uint16)
    x = t.from_numpy(np.repeat(v[:, None], 32, 1).view(np.int16)).cuda().view(t.bfloat16)
    _, _, _, scales = quantized(x, v.size, 32)
    assert scales.max() == 252
