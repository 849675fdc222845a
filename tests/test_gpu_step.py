"""The operators around the adapters on the GPU, through the C ABI, against the
64-bit CPU reference (oracle/step.py): MX4 conversion bit for bit, products and
norms within bounds derived from their arithmetic, drawn tokens exactly."""
import numpy as np
import pytest

import deterministic_split_lora_amd as dsl
from oracle import bf16_to_f64, step
from synth import normal_bf16, rng_for
from tests.helpers import bf16_from_gpu, bf16_to_gpu, f32_bits, f32_to_gpu, gpu_available, torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

SENTINEL = 0x7E5A                       # a bf16 pattern that no result here has


def u8_to_gpu(a):
    return torch().from_numpy(np.ascontiguousarray(a, dtype=np.uint8)).cuda()


def scale_rows(M, K):
    """A scales buffer of M rows with the stride the library asks for, filled with 0xEE."""
    return torch().full((M, (K // 32 + 3) // 4 * 4), 0xEE, dtype=torch().uint8, device="cuda")


def padded(M, N, pad=16):
    """A bf16 buffer [M + 1, N + pad] of sentinels and its view [M, N]."""
    t = torch()
    buf = t.full((M + 1, N + pad), SENTINEL, dtype=t.int16, device="cuda")
    return buf, buf.view(t.bfloat16)[:M, :N]


def check_padding(buf, M, N):
    b = buf.cpu().numpy().view(np.uint16)
    assert np.all(b[M:] == SENTINEL) and np.all(b[:, N:] == SENTINEL), "wrote outside the output"


def f64(t):
    return bf16_to_f64(bf16_from_gpu(t))


# ---------------------------------------------------------------------------
# MX4 conversion
# ---------------------------------------------------------------------------
def all_bf16_blocks():
    """Every finite bf16 value, in blocks with companions that set the scale: [n, 64] bits, one value per block at
    different places, the block's largest magnitude up to 2^4 times it."""
    v = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    v = v[(v & 0x7F80) != 0x7F80]
    top = ((v & 0x7FFF) >> 7).astype(np.int64)
    rows = []
    for up in (0, 1, 2, 3, 4):
        b = np.zeros((v.size, 32), dtype=np.uint16)
        b[:, 7] = (np.minimum(top + up, 254) << 7).astype(np.uint16) | 0x8000
        b[:, 19] = v
        b[:, 31] = v ^ 0x8000
        rows.append(b)
    b = np.concatenate(rows)
    return b[: b.shape[0] // 2 * 2].reshape(-1, 64)


def quantized(xg, M, K):
    t = torch()
    q = t.full((M, K // 2), 0xEE, dtype=t.uint8, device="cuda")
    s = scale_rows(M, K)
    dsl.lora_mx4_quantize(xg, q, s)
    t.cuda.synchronize()
    sc = s.cpu().numpy()
    assert np.all(sc[:, K // 32:] == 0xEE), "wrote past the scales"
    return q, s, step.mx4_unpack(q.cpu().numpy()), sc[:, :K // 32]


def test_quantize_every_bf16_value():
    bits = all_bf16_blocks()
    M, K = bits.shape
    q, s, code, sc = quantized(bf16_to_gpu(bits), M, K)
    ref_c, ref_s = step.mx4_quantize(bf16_to_f64(bits))
    assert np.array_equal(sc, ref_s)
    assert np.array_equal(code, ref_c)


@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (5, 2048), (2, 2080), (33, 4096), (7, 14336), (130, 416)])
def test_quantize_and_dequantize(M, K):
    t = torch()
    bits = normal_bf16((M, K), 3.0, 11 * M + K, "x")
    bits[0, :32] = 0
    if K > 32:
        bits[M - 1, K - 1] = 0x7F80                            # an infinity in the last block
        bits[M // 2, 33] = 0x7FC1 if M > 1 else bits[M // 2, 33]
    x, xv = padded(M, K)
    xv.copy_(bf16_to_gpu(bits))
    q, s, code, sc = quantized(xv, M, K)
    ref_c, ref_s = step.mx4_quantize(bf16_to_f64(bits))
    assert np.array_equal(sc, ref_s) and np.array_equal(code, ref_c)
    buf, out = padded(M, K)
    dsl.lora_mx4_dequantize(q, s, out)
    t.cuda.synchronize()
    check_padding(buf, M, K)
    assert np.array_equal(f64(out), step.mx4_values(ref_c, ref_s), equal_nan=True)


def test_dequantize_every_scale():
    t = torch()
    sc = np.arange(256, dtype=np.uint8).reshape(16, 16)
    code = np.tile(np.arange(16, dtype=np.uint8), (16, 32))
    q, s = u8_to_gpu(step.mx4_pack(code)), u8_to_gpu(sc)
    out = t.empty(16, 512, dtype=t.bfloat16, device="cuda")
    dsl.lora_mx4_dequantize(q, s, out)
    v = step.mx4_values(code, sc)
    big = np.abs(v) >= 2.0 ** 128                              # past the largest bf16: infinite
    want = np.where(big, np.copysign(np.inf, v), v)
    assert np.array_equal(f64(out), want, equal_nan=True)


def test_more_rows_than_one_launch_holds():
    """Past 2^20 workgroups a wave (a workgroup of the norm) takes further rows."""
    t = torch()
    M, K = (1 << 22) + 4099, 32
    few = normal_bf16((4099, K), 1.0, 3, "x")
    x = bf16_to_gpu(few).repeat(M // 4099 + 1, 1)[:M].contiguous()
    q, s = t.empty(M, 16, dtype=t.uint8, device="cuda"), t.zeros(M, 4, dtype=t.uint8, device="cuda")
    dsl.lora_mx4_quantize(x, q, s)
    code, sc = step.mx4_quantize(bf16_to_f64(few))
    want_q, want_s = u8_to_gpu(step.mx4_pack(code)), u8_to_gpu(sc)
    out = t.empty_like(x)
    dsl.lora_mx4_dequantize(q, s, out)
    small = t.empty(4099, K, dtype=t.bfloat16, device="cuda")
    dsl.lora_mx4_dequantize(q[:4099], s[:4099], small)
    for a in range(0, M - 4099, 4099 * 97):
        assert t.equal(q[a:a + 4099], want_q) and t.equal(s[a:a + 4099, :1], want_s)
        assert t.equal(out[a:a + 4099].view(t.int16), small.view(t.int16))
    tail = M // 4099 * 4099
    assert t.equal(q[tail:], want_q[:M - tail]) and t.equal(out[tail:].view(t.int16), small[:M - tail].view(t.int16))
    r, n = t.empty_like(x), t.empty_like(x)
    dsl.lora_block_norm(x, r, y=out, post="rms", pre="layer", x_out=n)
    r1, n1 = t.empty_like(small), t.empty_like(small)
    dsl.lora_block_norm(x[:4099], r1, y=small, post="rms", pre="layer", x_out=n1)
    for a in list(range(0, M - 4099, 4099 * 97)) + [tail]:
        b = min(a + 4099, M)
        assert t.equal(r[a:b].view(t.int16), r1[:b - a].view(t.int16))
        assert t.equal(n[a:b].view(t.int16), n1[:b - a].view(t.int16))


def test_conversions_of_no_rows():
    t = torch()
    x = t.empty(0, 64, dtype=t.bfloat16, device="cuda")
    dsl.lora_mx4_quantize(x, t.empty(0, 32, dtype=t.uint8, device="cuda"), t.empty(0, 4, dtype=t.uint8, device="cuda"))


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
class Product:
    """Inputs of one product and its exact value.

    Tolerance: x's and W's values are exact and so are their products in fp32 (8 x 2 significant bits).  A chunk is a
    chain of steps; a step adds at most 128 products to the accumulator and its own additions may truncate, so each
    of the at most 128 + steps + split_k additions that a product passes through is off by at most 2^-23 of the sum of
    magnitudes.  The last rounding is within 2^-9 of the value; 2^-8 leaves room for it to fall the other way."""

    def __init__(self, M, K, N, seed, mx):
        r = rng_for(seed, "product")
        self.M, self.K, self.N, self.mx = M, K, N, mx
        self.wc = r.integers(0, 16, (N, K)).astype(np.uint8)
        self.wsc = r.integers(118, 125, (N, K // 32)).astype(np.uint8)
        self.w = step.mx4_values(self.wc, self.wsc)
        if mx:
            self.xc = r.integers(0, 16, (M, K)).astype(np.uint8)
            self.xsc = r.integers(122, 130, (M, K // 32)).astype(np.uint8)
            self.x = step.mx4_values(self.xc, self.xsc)
        else:
            self.xbits = normal_bf16((M, K), 2.0, seed, "x")
            self.x = bf16_to_f64(self.xbits)

    def gpu(self):
        def scales(a):
            s = scale_rows(a.shape[0], self.K)
            s[:, :self.K // 32] = u8_to_gpu(a)
            return s
        self.wq, self.ws = u8_to_gpu(step.mx4_pack(self.wc)), scales(self.wsc)
        if self.mx:
            self.xg, self.xs = u8_to_gpu(step.mx4_pack(self.xc)), scales(self.xsc)
        else:
            self.xg, self.xs = bf16_to_gpu(self.xbits), None
        return self

    def run(self, S, rows=None, y=None, stream=None):
        t = torch()
        x = self.xg if rows is None else self.xg[rows]
        M = x.shape[0]
        y = t.full((M, self.N), float("nan"), dtype=t.bfloat16, device="cuda") if y is None else y
        n = dsl.lora_mx4_linear_workspace_bytes(M, self.K, self.N, S)
        ws = t.full((n,), 0xFF, dtype=t.uint8, device="cuda") if n else None
        if self.mx:
            xs = self.xs if rows is None else self.xs[rows]
            dsl.lora_mx4_linear_q(x, xs, self.wq, self.ws, y, S, ws, stream=stream)
        else:
            dsl.lora_mx4_linear(x, self.wq, self.ws, y, S, ws, stream=stream)
        t.cuda.synchronize()
        return y

    def check(self, got, S, rows=slice(None)):
        x = self.x[rows]
        e = x @ self.w.T
        depth = 128 + (self.K // S + 127) // 128 + S
        tol = 2.0 ** -8 * np.abs(e) + depth * 2.0 ** -23 * (np.abs(x) @ np.abs(self.w).T)
        err = np.abs(got - e)
        assert np.all(err <= tol), f"worst {np.max(err / np.maximum(tol, 1e-300)):.3g} of the bound"


SIZES = [  # M, K, N, split_k
    (1, 32, 8, 1), (1, 512, 16, 16), (1, 4096, 6144, 8), (2, 160, 40, 1), (5, 320, 24, 2), (15, 1024, 520, 8),
    (16, 2048, 256, 4), (17, 96, 72, 1), (31, 768, 136, 8), (33, 1152, 264, 4), (48, 512, 1000, 2), (63, 256, 64, 8),
    (64, 14336, 128, 8), (65, 1024, 328, 1), (97, 640, 136, 4), (128, 2048, 512, 8), (129, 512, 776, 16),
    (200, 4096, 384, 4), (255, 1024, 264, 1), (256, 288, 1032, 1), (257, 1536, 520, 2), (300, 544, 136, 1),
    (511, 2048, 248, 8), (513, 192, 2056, 1), (1030, 1024, 1288, 1), (1100, 352, 776, 1), (700, 1056, 2304, 1),
    (1025, 768, 2056, 4), (1100, 256, 6144, 1), (1100, 256, 6144, 2), (1100, 320, 6144, 2), (1300, 416, 6144, 1),
    (1300, 512, 6144, 1), (33, 2048, 1024, 16), (48, 3584, 512, 16), (64, 8192, 40, 1), (1, 16384, 24, 2),
]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("M,K,N,S", SIZES)
def test_product(M, K, N, S, mx):
    p = Product(M, K, N, 31 * M + K + N, mx).gpu()
    buf, y = padded(M, N)
    got = f64(p.run(S, y=y))
    check_padding(buf, M, N)
    p.check(got, S)
    again = bf16_from_gpu(p.run(S))
    assert np.array_equal(again, bf16_from_gpu(y)), "two runs differ"


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("K,N,S", [(1024, 520, 8), (2048, 2056, 1), (960, 1032, 2), (4096, 264, 16), (1536, 3080, 4)])
def test_product_rows_do_not_depend_on_the_batch(K, N, S, mx):
    """A row's bits are the same in batches of every size, so through every kernel and schedule."""
    M = 1300
    p = Product(M, K, N, K + N + S, mx).gpu()
    whole = bf16_from_gpu(p.run(S))
    for a, b in [(0, 1), (7, 23), (100, 133), (64, 128), (1, 66), (256, 384), (40, 341), (3, 600), (150, 1250)]:
        part = bf16_from_gpu(p.run(S, rows=slice(a, b)))
        assert np.array_equal(part, whole[a:b]), f"rows {a}..{b}"


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("M,S", [(3, 4), (70, 1), (300, 1), (300, 4)])
def test_product_not_finite_and_extreme_scales(M, S, mx):
    """A NaN block of W makes its column NaN and no other, one of x its row; the smallest and large scales keep their
    value; an all-zero row and column give exact zeros."""
    K, N = 512, 264
    p = Product(M, K, N, 5, mx)
    p.wsc[9, 3] = 255
    p.wc[21] = 0
    p.wsc[40] = 0                                              # 2^-127
    p.wsc[41] = 200
    p.w = step.mx4_values(p.wc, p.wsc)
    if mx:
        p.xsc[M - 1, K // 32 - 1] = 255
        p.xc[1] = 8                                            # minus zero
        p.x = step.mx4_values(p.xc, p.xsc)
    else:
        p.xbits[M - 1, K - 1] = 0x7FC0
        p.xbits[1] = 0x8000
        p.x = bf16_to_f64(p.xbits)
    got = f64(p.gpu().run(S))
    e = p.x @ p.w.T
    assert np.array_equal(np.isnan(got), np.isnan(e))
    fine = ~np.isnan(e)
    with np.errstate(invalid="ignore"):
        tol = 2.0 ** -8 * np.abs(e) + (128 + K // 128 + S) * 2.0 ** -23 * (np.abs(p.x) @ np.abs(p.w).T) + 2.0 ** -126
    assert np.all(np.abs(got - e)[fine] <= tol[fine])
    assert not got[fine[:, 21], 21].any() and not got[1, fine[1]].any()


def test_product_strided_operands():
    """Rows with padding on every side; what lies between them is poison."""
    t = torch()
    M, K, N, S = 70, 288, 136, 1
    p = Product(M, K, N, 77, False).gpu()
    plain = bf16_from_gpu(p.run(S))
    nan = t.full((M, K + 24), float("nan"), dtype=t.bfloat16, device="cuda")
    nan[:, 8:8 + K] = p.xg
    p.xg = nan[:, 8:8 + K]
    wq = t.full((N, K // 2 + 48), 0x77, dtype=t.uint8, device="cuda")
    wq[:, 16:16 + K // 2] = p.wq
    p.wq = wq[:, 16:16 + K // 2]
    ws = t.full((N, 24), 0xFF, dtype=t.uint8, device="cuda")
    ws[:, 4:4 + K // 32] = p.ws[:, :K // 32]
    p.ws = ws[:, 4:4 + K // 32]
    assert np.array_equal(bf16_from_gpu(p.run(S)), plain)


def test_product_agrees_with_its_parts():
    """Quantised x through lora_mx4_linear_q against its values through lora_mx4_linear: the same exact operands, so
    both are within the bound of the same exact result."""
    t = torch()
    M, K, N, S = 40, 1024, 264, 4
    p = Product(M, K, N, 3, False).gpu()
    q, s, code, sc = quantized(p.xg, M, K)
    v = t.empty(M, K, dtype=t.bfloat16, device="cuda")
    dsl.lora_mx4_dequantize(q, s, v)
    a, b = t.empty(M, N, dtype=t.bfloat16, device="cuda"), t.empty(M, N, dtype=t.bfloat16, device="cuda")
    dsl.lora_mx4_linear_q(q, s, p.wq, p.ws, a, S, None) if not dsl.lora_mx4_linear_workspace_bytes(M, K, N, S) else None
    dsl.lora_mx4_linear(v, p.wq, p.ws, b, S, None)
    p.x = step.mx4_values(code, sc)
    p.check(f64(a), S)
    p.check(f64(b), S)


def test_product_past_32_bit_offsets():
    """y beyond 2^31 elements: the last rows land where they belong."""
    t = torch()
    M, K, N = 70000, 32, 32776
    p = Product(256, K, N, 8, False).gpu()
    x = p.xg.repeat((M + 255) // 256, 1)[:M]
    y = t.empty(M, N, dtype=t.bfloat16, device="cuda")
    dsl.lora_mx4_linear(x, p.wq, p.ws, y, 1)
    small = p.run(1)
    for a in (0, 65280, 69888 - 256):
        assert t.equal(y[a:a + 256].view(t.int16), small.view(t.int16))
    assert t.equal(y[69888:].view(t.int16), small[:M - 69888].view(t.int16))


# ---------------------------------------------------------------------------
# block norm
# ---------------------------------------------------------------------------
def norm_case(M, C, post, pre, gate, seed, bias=True):
    f = lambda name, shape, std, mean=0.0: normal_bf16(shape, std, seed, name) if not mean else _shift(  # noqa: E731
        normal_bf16(shape, std, seed, name), mean)
    c = {"y": f("y", (M, C), 2.0), "r": f("r", (M, C), 3.0)}
    for side, kind in (("post", post), ("pre", pre)):
        c[side + "_w"] = None if kind == "none" else f(side + "w", (C,), 0.3, 1.0)
        c[side + "_b"] = f(side + "b", (C,), 0.3) if kind != "none" and bias else None
    rows = {"none": 0, "channel": 1, "token": M, "group": (M + 2) // 3}[gate]
    c["gate"] = f("gate", (rows, C), 0.7) if rows else None
    return c


def _shift(bits, mean):
    t = torch()
    v = t.from_numpy(bf16_to_f64(bits) + mean).to(t.bfloat16)
    return v.view(t.int16).numpy().view(np.uint16).copy()


def run_norm(c, post, pre, rs, eps, group=None, inplace=False):
    t = torch()
    g = {k: None if v is None else bf16_to_gpu(v) for k, v in c.items()}
    M, C = c["r"].shape
    bufs = []
    if inplace:
        r_out, x_out = g["r"], g["y"] if pre != "none" else None
    else:
        b1, r_out = padded(M, C)
        b2, x_out = padded(M, C, 24)
        bufs, x_out = [b1, b2], x_out if pre != "none" else None
    dsl.lora_block_norm(g["r"], r_out, y=g["y"], post=post, post_w=g["post_w"], post_b=g["post_b"], gate=g["gate"],
                        gate_group=group, res_scale=rs, pre=pre, pre_w=g["pre_w"], pre_b=g["pre_b"], x_out=x_out,
                        eps=eps)
    t.cuda.synchronize()
    for b in bufs:
        check_padding(b, M, C)
    return bf16_from_gpu(r_out), None if x_out is None else bf16_from_gpu(x_out)


def check_norm(c, post, pre, rs, eps, group, r_bits, x_bits):
    """Bounds.  A row sum passes each element through fewer than 32 + 6 + 16 additions (a thread's own, the wave's
    butterfly, the waves), so a mean or mean square is within 64 2^-24 of its magnitudes' mean, and its square root
    within half of that; with the handful of multiplications after it, D = 96 units of 2^-24 of the magnitudes cover
    every fp32 value.  The pre-norm sees r' off by E and passes that on.  Rounding to bf16 adds 2^-8 at most."""
    D = 96 * 2.0 ** -24
    v = {k: None if a is None else bf16_to_f64(a) for k, a in c.items()}
    M, C = v["r"].shape
    zero = np.zeros((M, C))
    t, tol = zero, zero
    if v["y"] is not None:
        t, irs, cen = step.norm(v["y"], post, v["post_w"], v["post_b"], eps)
        w = 1.0 if v["post_w"] is None else np.abs(v["post_w"])
        b = 0.0 if v["post_b"] is None else np.abs(v["post_b"])
        mean_abs = np.abs(v["y"]).mean(-1, keepdims=True)
        # a layer norm's centred value is off by D mean|y|, which reaches the variance as well
        off = D * (np.abs(v["y"]) + mean_abs) if post == "layer" else D * np.abs(v["y"])
        tol = (off + np.abs(cen) * irs * off.max(-1, keepdims=True) * (post == "layer")) * irs * w + D * b
        if v["gate"] is not None:
            gt = v["gate"][np.arange(M) // group]
            t, tol = t * gt, tol * np.abs(gt) + D * np.abs(t * gt)
    r = rs * v["r"] + t
    E = tol + D * (np.abs(rs * v["r"]) + np.abs(t))
    got = bf16_to_f64(r_bits)
    assert np.all(np.abs(got - r) <= E + 2.0 ** -8 * np.abs(r)), "r' beyond its bound"
    if x_bits is None:
        return
    x, irs, cen = step.norm(r, pre, v["pre_w"], v["pre_b"], eps)
    w = 1.0 if v["pre_w"] is None else np.abs(v["pre_w"])
    b = 0.0 if v["pre_b"] is None else np.abs(v["pre_b"])
    layer = pre == "layer"
    off = E + (E.max(-1, keepdims=True) + D * np.abs(r).mean(-1, keepdims=True)) * layer + D * (np.abs(r) + np.abs(cen))
    tol = (off + np.abs(cen) * irs * off.max(-1, keepdims=True)) * irs * w + D * b
    assert np.all(np.abs(bf16_to_f64(x_bits) - x) <= tol + 2.0 ** -8 * np.abs(x)), "x beyond its bound"


@pytest.mark.parametrize("post,pre,gate", [("rms", "rms", "channel"), ("layer", "layer", "token"),
                                           ("none", "rms", "none"), ("rms", "none", "group"),
                                           ("none", "layer", "token"), ("layer", "rms", "none"),
                                           ("none", "none", "channel")])
@pytest.mark.parametrize("M,C", [(1, 8), (3, 64), (2, 504), (5, 512), (4, 520), (7, 2048), (3, 2056), (2, 4096),
                                 (5, 8192), (2, 8200), (1, 16384), (2, 16392), (1, 32768), (300, 1024)])
def test_block_norm(M, C, post, pre, gate):
    c = norm_case(M, C, post, pre, gate, 7 * M + C)
    group = {"channel": M, "group": 3}.get(gate, 1)
    r, x = run_norm(c, post, pre, 0.75, 1e-5, group if c["gate"] is not None else None)
    check_norm(c, post, pre, 0.75, 1e-5, group, r, x)
    r2, x2 = run_norm(c, post, pre, 0.75, 1e-5, group if c["gate"] is not None else None, inplace=True)
    assert np.array_equal(r, r2) and (x is None or np.array_equal(x, x2)), "in place differs"


def test_block_norm_without_block_output():
    c = norm_case(9, 1000, "none", "layer", "none", 4, bias=False)
    c["y"] = None
    r, x = run_norm(c, "none", "layer", 1.0, 1e-6)
    check_norm(c, "none", "layer", 1.0, 1e-6, 1, r, x)
    assert np.array_equal(r, c["r"]), "a residual of scale 1 has to pass unchanged"


def test_block_norm_zero_rows_and_no_weights():
    c = norm_case(4, 256, "rms", "rms", "none", 2, bias=False)
    c["y"][1] = 0
    c["r"][1] = 0
    c["post_w"] = c["pre_w"] = None
    r, x = run_norm(c, "rms", "rms", 1.0, 1e-5)
    check_norm(c, "rms", "rms", 1.0, 1e-5, 1, r, x)
    assert not bf16_to_f64(r)[1].any() and not bf16_to_f64(x)[1].any()


@pytest.mark.parametrize("C", [256, 1536, 4096, 9000])
def test_block_norm_rows_do_not_depend_on_the_batch(C):
    c = norm_case(700, C, "rms", "layer", "token", C)
    r, x = run_norm(c, "rms", "layer", 1.25, 1e-5)
    for a, b in [(0, 1), (13, 14), (5, 40), (699, 700), (100, 612)]:
        part = {k: (v[a:b] if v is not None and v.ndim == 2 else v) for k, v in c.items()}
        pr, px = run_norm(part, "rms", "layer", 1.25, 1e-5)
        assert np.array_equal(pr, r[a:b]) and np.array_equal(px, x[a:b])


# ---------------------------------------------------------------------------
# sampling
# ---------------------------------------------------------------------------
def gpu_logits(l, bf16, pad=0):
    """The logits on the GPU (rows `pad` elements apart from contiguous) and the values they hold."""
    t = torch()
    v = t.from_numpy(np.ascontiguousarray(l, dtype=np.float32))
    v = v.to(t.bfloat16) if bf16 else v
    g = t.full((l.shape[0], l.shape[1] + pad), 50.0, dtype=v.dtype, device="cuda")[:, :l.shape[1]]
    g.copy_(v)
    return g, v.to(t.float64).numpy()


def run_sample(g, u, **kw):
    t = torch()
    B = g.shape[0]
    tokens = t.full((B,), -7, dtype=t.int32, device="cuda")
    logprobs = t.full((B,), float("nan"), dtype=t.float32, device="cuda")
    f = {k: (t.as_tensor(np.asarray(v, dtype=np.int32 if k == "top_k" else np.float32)).cuda()) for k, v in kw.items()}
    dsl.lora_sample(g, f32_to_gpu(np.asarray(u, dtype=np.float32)), tokens, logprobs=logprobs, **f)
    t.cuda.synchronize()
    return tokens.cpu().numpy(), logprobs.cpu().numpy()


def steady(kept, rng):
    """A random number in the middle of a kept token's share, for tokens whose share is wide enough that neither the
    rounding of exp nor that of the number itself can move it to a neighbour: the weights are within 2^-22 of exact,
    so sums are too; a share of 2^-18 has its middle 2^-19 from either end."""
    total = kept.sum()
    wide = np.flatnonzero(kept > total * 2.0 ** -18)
    i = int(rng.choice(wide))
    return i, (np.cumsum(kept)[i] - kept[i] / 2) / total


def safe_p(w_sorted, n):
    """A top_p that keeps n tokens of these sorted weights, as far as possible from keeping one more or less."""
    c = np.cumsum(w_sorted) / w_sorted.sum()
    return float((c[n - 1] + (c[n - 2] if n > 1 else 0.0)) / 2)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [1, 2, 63, 64, 65, 1000, 1023, 4097, 32000, 50021, 128259])
def test_sample_settings(V, bf16):
    """Rows with every combination of settings against the reference."""
    rng = rng_for(V, "sample")
    B = 24
    l = rng.standard_normal((B, V)) * 3.0
    l[:, rng.integers(0, V, max(1, V // 10))] = -np.inf
    l[:, 0] = 1.0
    g, val = gpu_logits(l, bf16, pad=3)
    T = np.where(np.arange(B) % 6 == 5, 0.0, 0.5 + rng.random(B)).astype(np.float32)
    k = np.where(np.arange(B) % 2 == 0, rng.integers(1, 100, B), 0).astype(np.int32)
    p, m, u, want, lp = np.ones(B, np.float32), np.zeros(B, np.float32), np.zeros(B, np.float32), [], []
    for i in range(B):
        base = step.kept_weights(val[i], T[i], k[i])
        n = np.count_nonzero(base)
        if i % 3 == 1 and n > 1:
            keep = int(rng.integers(1, min(n, 200)))
            p[i] = safe_p(np.sort(base[base > 0])[::-1], keep)
        if i % 4 >= 2 and n > 1:
            s = np.sort(base[base > 0])[::-1]
            j = int(rng.integers(1, min(n, 300)))
            m[i] = (s[j] + s[j - 1]) / 2 / 2.0 ** 31 if s[j - 1] > s[j] * (1 + 2.0 ** -12) else 0.0
        kept = step.kept_weights(val[i], T[i], k[i], p[i], m[i])
        tok, u[i] = steady(kept, rng)
        want.append(tok)
        lp.append(np.log(kept[tok] / kept.sum()))
    tokens, logprobs = run_sample(g, u, temperature=T, top_k=k, top_p=p, min_p=m)
    assert tokens.tolist() == want
    # weights within 2^-22 of exact, one division, one logarithm in fp32: 2^-20 absolute and 2^-22 relative
    assert np.all(np.abs(logprobs - lp) <= 2.0 ** -20 + 2.0 ** -22 * np.abs(lp))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [7, 5000, 40000, 131072])
def test_sample_ties(V, bf16):
    """Equal logits have equal whole weights, so everything is exact: the lowest indices are kept."""
    l = np.zeros((8, V))
    l[6:, :] = -1.0
    l[6:, V // 2:V // 2 + 3] = 2.0
    g, _ = gpu_logits(l, bf16)
    k = np.array([5, 0, 0, 1, V, V + 9, 2, 0], np.int32)
    p = np.array([1, 0.5, 0, 1, 1, 2, 1, 0.3], np.float32)
    u = np.array([0.99, 0.999999, 0.7, 0.5, 0.5, 0.25, 0.75, 0.0], np.float32)
    tokens, logprobs = run_sample(g, u, top_k=k, top_p=p)
    k0 = min(5, V)
    half = int(np.ceil(0.5 * V))
    third = step.kept_weights(l[7], 1.0, 0, 0.3)
    assert tokens.tolist() == [k0 - 1, min(int(np.float32(0.999999) * np.float64(half)), half - 1), 0, 0,
                               int(0.5 * V), int(0.25 * V), V // 2 + 1, step.draw(third, 0.0)]
    assert logprobs[3] == 0.0 and logprobs[2] == 0.0
    assert abs(logprobs[0] + np.log(k0)) < 1e-6


@pytest.mark.parametrize("bf16", [False, True])
def test_sample_edges(bf16):
    """Masked rows, a single token left, NaN, infinities, random numbers at and past the ends, odd settings."""
    V, ninf, nan = 300, -np.inf, np.nan
    l = np.zeros((14, V))
    l[0] = ninf                                                # nothing left
    l[1] = ninf
    l[1, 299] = -3.0e38                                        # one token, near the type's lowest value
    l[2] = nan
    l[3, :] = nan
    l[3, 17] = 1.0
    l[4, [5, 200]] = np.inf                                    # infinite logits share the weight
    l[5] = -3.0e38                                             # a mask of the lowest value everywhere
    l[6, 100] = 80.0                                           # everything else weighs nothing
    tokens, logprobs = run_sample(
        gpu_logits(l, bf16)[0],
        [0.5, 0.5, 0.5, 0.5, 0.75, 0.0, 0.999, 1.0, 7.0, -1.0, nan, 0.5, 0.5, 0.5],
        temperature=[1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, nan, -2, np.inf],
        top_k=[0, 3, 3, 3, 0, 1, 0, 0, -5, 0, 0, 0, 0, 0],
        top_p=[1, 0.5, 0.5, 0.5, 1, 1, 0.9, nan, -1, 1, 1, 1, 1, 1],
        min_p=[0, 0, 0, 0.5, 0, 0, 0, nan, 0, 0, 2.0, 0, 0, 0])
    assert tokens.tolist() == [-1, 299, -1, 17, 200, 0, 100, V - 1, 0, 0, 0, 0, 0, 150]
    assert np.array_equal(np.isneginf(logprobs), np.isin(np.arange(14), [0, 2]))
    assert logprobs[1] == 0.0 and logprobs[6] == 0.0 and abs(logprobs[4] - np.log(0.5)) < 1e-6


@pytest.mark.parametrize("bf16", [False, True])
def test_sample_rows_of_every_path(bf16):
    """top-k past what is gathered in one list, cuts near the smallest weights, logits from one end of the type to the
    other, bins with more elements than their list holds."""
    rng = rng_for(77, "paths")
    V = 60000
    rows, kw = [], dict(temperature=[], top_k=[], top_p=[], min_p=[])

    def add(l, T=1.0, k=0, p=1.0, m=0.0):
        rows.append(l)
        for name, v in zip(kw, (T, k, p, m)):
            kw[name].append(v)

    base = rng.standard_normal(V) * 2.0
    add(base, k=1024)
    add(base, k=1025)
    add(base, k=20000)
    add(base, k=59999)
    add(base, m=1e-9, T=0.25)
    add(base, m=2.0 ** -31)
    add(base, m=0.9)
    wide = base.copy()
    wide[:3] = [3.0e38, -3.0e38, -3.3e38]
    add(wide, k=2)
    add(wide, T=1e38)
    add(wide, T=1e-39)                                         # its inverse is infinite
    near = 1.0 + 2.0 ** -6 * rng.integers(0, 4, V)             # four values, all in few bins
    add(near, k=30000)
    few = base.copy()
    few[rng.permutation(V)[:V - 40]] = -np.inf                 # forty tokens left
    add(few, k=50)
    add(few, k=39, T=2.0)
    g, val = gpu_logits(np.stack(rows), bf16, pad=1)
    want, u = [], []
    for i in range(len(rows)):
        kept = step.kept_weights(val[i], np.float32(kw["temperature"][i]), kw["top_k"][i], kw["top_p"][i], kw["min_p"][i])
        if kw["temperature"][i] < 1e-38:                       # the maximum's elements share the weight
            kept = (val[i] == val[i].max()).astype(np.int64) << 31
        tok, x = steady(kept, rng)
        want.append(tok)
        u.append(x)
    tokens, _ = run_sample(g, u, **kw)
    assert tokens.tolist() == want


def test_sample_largest_vocabulary():
    V = 1 << 22
    l = rng_for(5, "large").standard_normal((1, V)) * 3.0
    g, val = gpu_logits(l, False)
    for kw in (dict(), dict(temperature=[0.8], top_k=[7])):
        kept = step.kept_weights(val[0], kw.get("temperature", [1.0])[0], kw.get("top_k", [0])[0])
        tok, u = steady(kept, rng_for(6, "u"))
        tokens, _ = run_sample(g, [u], **kw)
        assert tokens[0] == tok


def test_sample_large_ties_with_top_p():
    """Thousands of equal logits below a few large ones: the threshold falls inside the tie."""
    V = 100000
    l = np.full((3, V), 1.0)
    l[:, 999:99999:1000] = 5.0
    g, val = gpu_logits(l, True)
    for i, n in enumerate((50, 2000, 60000)):
        w = step.weights(val[i], 1.0)
        p = np.float32(safe_p(np.sort(w)[::-1], n))
        kept = step.kept_weights(val[i], 1.0, 0, p)
        u = 0.9999
        tokens, _ = run_sample(g[i:i + 1], [u], top_p=[p])
        share = np.cumsum(kept) / kept.sum()
        # the tied weights are off by the same 2^-22 at most: the place in the sum moves by no more than that
        lo, hi = np.searchsorted(share, u - 2.0 ** -21), np.searchsorted(share, u + 2.0 ** -21)
        assert lo <= tokens[0] <= hi and kept[tokens[0]] > 0


def test_sample_rows_do_not_depend_on_the_batch():
    rng = rng_for(3, "batch")
    B, V = 300, 9001
    g, _ = gpu_logits(rng.standard_normal((B, V)) * 2, False)
    u = rng.random(B).astype(np.float32)
    kw = dict(top_k=rng.integers(0, 50, B).astype(np.int32), top_p=rng.random(B).astype(np.float32),
              temperature=(0.3 + rng.random(B)).astype(np.float32))
    tokens, lp = run_sample(g, u, **kw)
    for a, b in [(0, 1), (7, 8), (20, 95), (299, 300)]:
        t2, lp2 = run_sample(g[a:b], u[a:b], **{k: v[a:b] for k, v in kw.items()})
        assert np.array_equal(t2, tokens[a:b]) and np.array_equal(lp2.view(np.int32), lp[a:b].view(np.int32))


def test_sample_follows_the_distribution():
    """Even random numbers hit each token as often as its share says: the draw is an inverse of the kept sum."""
    V, B = 40, 4000
    l = rng_for(9, "dist").standard_normal(V)
    g, val = gpu_logits(np.tile(l, (B, 1)), False)
    tokens, _ = run_sample(g, (np.arange(B) + 0.5) / B, top_p=np.full(B, 0.8))
    kept = step.kept_weights(val[0], 1.0, 0, 0.8)
    # a share of s B points falls on between floor(s B) and ceil(s B) + 1 of them
    assert np.all(np.abs(np.bincount(tokens, minlength=V) - B * kept / kept.sum()) <= 1.0 + 1e-3)


# ---------------------------------------------------------------------------
# streams, graphs, refusals
# ---------------------------------------------------------------------------
def test_operators_on_another_stream_and_in_a_graph():
    """All of them captured in one graph on a side stream; each replay, after new inputs, against the eager calls."""
    t = torch()
    M, K, N, S = 96, 1024, 1032, 4
    p = Product(M, K, N, 12, False).gpu()
    pn = {k: None if v is None else bf16_to_gpu(v) for k, v in norm_case(M, K, "rms", "rms", "channel", 5).items()}
    q, s = t.empty(M, K // 2, dtype=t.uint8, device="cuda"), scale_rows(M, K)
    n = dsl.lora_mx4_linear_workspace_bytes(M, K, N, S)
    ws = t.empty(max(n, 16), dtype=t.uint8, device="cuda")
    u = t.rand(M, device="cuda")

    def outputs():
        return dict(r=t.zeros(M, K, dtype=t.bfloat16, device="cuda"), x=t.zeros(M, K, dtype=t.bfloat16, device="cuda"),
                    a=t.zeros(M, N, dtype=t.bfloat16, device="cuda"), b=t.zeros(M, N, dtype=t.bfloat16, device="cuda"),
                    tok=t.zeros(M, dtype=t.int32, device="cuda"), lp=t.zeros(M, device="cuda"))

    def call(o):
        dsl.lora_block_norm(pn["r"], o["r"], y=pn["y"], post="rms", post_w=pn["post_w"], post_b=pn["post_b"],
                            gate=pn["gate"], res_scale=0.5, pre="rms", pre_w=pn["pre_w"], pre_b=pn["pre_b"],
                            x_out=o["x"])
        dsl.lora_mx4_quantize(o["x"], q, s)
        dsl.lora_mx4_linear(o["x"], p.wq, p.ws, o["a"], S, ws)
        dsl.lora_mx4_linear_q(q, s, p.wq, p.ws, o["b"], S, ws)
        dsl.lora_sample(o["a"], u, o["tok"], top_k=t_k, top_p=t_p, logprobs=o["lp"])

    t_k = t.full((M,), 40, dtype=t.int32, device="cuda")
    t_p = t.full((M,), 0.9, device="cuda")
    side, captured = t.cuda.Stream(), outputs()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        call(captured)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=side):
        call(captured)
    for i in range(4):
        pn["y"].copy_(t.randn(M, K, device="cuda") * (i + 1))
        u.copy_(t.rand(M, device="cuda"))
        eager = outputs()
        call(eager)
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        for k in eager:
            assert t.equal(eager[k].view(t.uint8), captured[k].view(t.uint8)), f"replay {i}: {k}"


def test_example_runs():
    import examples.adapted_step as example
    report = example.main(["--layers", "2", "--tokens", "5"])
    assert report["tokens"] == report["reference_tokens"]
    assert report["worst"] < 0.05


def test_binding_refuses():
    t = torch()
    x, w = t.zeros(4, 64, dtype=t.bfloat16, device="cuda"), t.zeros(8, 32, dtype=t.uint8, device="cuda")
    s, y = t.zeros(8, 4, dtype=t.uint8, device="cuda"), t.zeros(4, 8, dtype=t.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        dsl.lora_mx4_linear(x.float(), w, s, y, 1)
    with pytest.raises(ValueError):
        dsl.lora_mx4_linear(x, w[:4], s[:4], y, 1)
    with pytest.raises(ValueError):
        dsl.lora_mx4_linear(x, w, s[:, :1], y, 1)
    with pytest.raises(ValueError):
        dsl.lora_mx4_linear(x.cpu(), w, s, y, 1)
    with pytest.raises(dsl.LoraError):
        dsl.lora_mx4_linear(x, w, s, y, 4)                      # 64 is no multiple of 32 * 4
    with pytest.raises(dsl.LoraError):
        dsl.lora_block_norm(x, t.empty_like(x), pre="rms")      # no x_out
    with pytest.raises(ValueError):
        dsl.lora_block_norm(x, t.empty_like(x), y=x[:2])
    with pytest.raises(ValueError):
        dsl.lora_block_norm(x, t.empty_like(x), y=x, gate=x[:2], gate_group=1)
    with pytest.raises(KeyError):
        dsl.lora_block_norm(x, t.empty_like(x), pre="group", x_out=t.empty_like(x))
    u, tok = t.zeros(4, device="cuda"), t.zeros(4, dtype=t.int32, device="cuda")
    with pytest.raises(TypeError):
        dsl.lora_sample(x.half(), u, tok)
    with pytest.raises(TypeError):
        dsl.lora_sample(x, u, tok.long())
    with pytest.raises(ValueError):
        dsl.lora_sample(x, u[:3], tok)
    with pytest.raises(ValueError):
        dsl.lora_sample(x, t.zeros(8, device="cuda")[::2], tok)
