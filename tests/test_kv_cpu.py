"""The paged cache and the verification of drafts on the host: argument checks (every call below carries a defect that the
host catches, or has nothing to do, so the fake addresses are never followed), workspace sizes, and the CPU references' own
pins."""
import ctypes
import math

import numpy as np
import pytest

import deterministic_split_lora_amd as dsl
from deterministic_split_lora_amd import _binding as B
from oracle import kv, step
from oracle import verify as ref

FAKE = 0x100000
MIS = 0x100002


class Cache(ctypes.Structure):
    """lora_kv_cache of include/lora_det.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scales", "v_scales")] + \
               [(n, ctypes.c_int64) for n in ("ld_k", "ld_v", "ld_ks", "ld_vs", "n_pages")] + \
               [(n, ctypes.c_int32) for n in ("page_size", "heads", "head_dim")] + \
               [("page_table", ctypes.c_void_p), ("ld_table", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("seq_lens", ctypes.c_void_p), ("cu_tokens", ctypes.c_void_p), ("n_seqs", ctypes.c_int64)]


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scales=FAKE, v_scales=FAKE, ld_k=2 * 64 * 128, ld_v=2 * 64 * 128, ld_ks=8, ld_vs=8,
             n_pages=10, page_size=64, heads=2, head_dim=128, page_table=FAKE, ld_table=20, max_pages=20, seq_lens=FAKE,
             cu_tokens=FAKE, n_seqs=3)
    a.update(kw)
    return Cache(**a)


CACHE_REFUSALS = [
    (dict(n_seqs=-1), B.LORA_ERR_SHAPE), (dict(n_seqs=65537), B.LORA_ERR_SHAPE), (dict(n_pages=0), B.LORA_ERR_SHAPE),
    (dict(n_pages=1 << 31), B.LORA_ERR_SHAPE), (dict(max_pages=0), B.LORA_ERR_SHAPE), (dict(ld_table=19), B.LORA_ERR_SHAPE),
    (dict(head_dim=96), B.LORA_ERR_UNSUPPORTED), (dict(head_dim=0), B.LORA_ERR_UNSUPPORTED),
    (dict(page_size=8), B.LORA_ERR_UNSUPPORTED), (dict(page_size=48), B.LORA_ERR_UNSUPPORTED),
    (dict(page_size=65536), B.LORA_ERR_UNSUPPORTED),
    (dict(k=None), B.LORA_ERR_NULL), (dict(v=None), B.LORA_ERR_NULL), (dict(k_scales=None), B.LORA_ERR_NULL),
    (dict(v_scales=None), B.LORA_ERR_NULL), (dict(page_table=None), B.LORA_ERR_NULL),
    (dict(seq_lens=None), B.LORA_ERR_NULL), (dict(cu_tokens=None), B.LORA_ERR_NULL),
    (dict(ld_k=2 * 64 * 128 - 16), B.LORA_ERR_SHAPE), (dict(ld_v=2 * 64 * 128 - 16), B.LORA_ERR_SHAPE),
    (dict(ld_ks=7), B.LORA_ERR_SHAPE), (dict(ld_vs=7), B.LORA_ERR_SHAPE),
    (dict(k=MIS), B.LORA_ERR_ALIGN), (dict(v=MIS), B.LORA_ERR_ALIGN), (dict(ld_k=2 * 64 * 128 + 8), B.LORA_ERR_ALIGN),
    (dict(ld_v=2 * 64 * 128 + 4), B.LORA_ERR_ALIGN), (dict(page_table=MIS), B.LORA_ERR_ALIGN),
    (dict(seq_lens=MIS), B.LORA_ERR_ALIGN), (dict(cu_tokens=MIS), B.LORA_ERR_ALIGN),
    (dict(n_seqs=0, k=None), B.LORA_OK),
]


def append(c=None, **kw):
    a = dict(q=FAKE, ld_q=1536, q_out=FAKE, ld_qo=1024, q_heads=8, k=FAKE, ld_k=1536, v=FAKE, ld_v=1536, T=4, q_norm=FAKE,
             k_norm=FAKE, eps=1e-6, rope=FAKE, ld_rope=128, rope_rows=100, rope_dim=128, pairs=0)
    a.update(kw)
    c = cache() if c is None else c
    f = dsl.lib().lora_kv_append
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    return f(ctypes.byref(c) if c else None, vp(a["q"]), i64(a["ld_q"]), vp(a["q_out"]), i64(a["ld_qo"]), i32(a["q_heads"]),
             vp(a["k"]), i64(a["ld_k"]), vp(a["v"]), i64(a["ld_v"]), i64(a["T"]), vp(a["q_norm"]), vp(a["k_norm"]),
             ctypes.c_float(a["eps"]), vp(a["rope"]), i64(a["ld_rope"]), i64(a["rope_rows"]), i32(a["rope_dim"]),
             i32(a["pairs"]), None)


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_append_refuses_caches(kw, status):
    assert append(cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), B.LORA_ERR_SHAPE), (dict(T=1 << 31), B.LORA_ERR_SHAPE), (dict(T=(1 << 31) - 1), B.LORA_ERR_SHAPE),
    (dict(q_heads=0), B.LORA_ERR_SHAPE), (dict(q_heads=65537), B.LORA_ERR_SHAPE),
    (dict(pairs=2), B.LORA_ERR_UNSUPPORTED), (dict(rope_dim=8), B.LORA_ERR_UNSUPPORTED),
    (dict(rope_dim=24), B.LORA_ERR_UNSUPPORTED), (dict(rope_dim=144), B.LORA_ERR_UNSUPPORTED),
    (dict(q=None), B.LORA_ERR_UNSUPPORTED), (dict(q_out=None), B.LORA_ERR_UNSUPPORTED),
    (dict(q=None, q_out=None), B.LORA_ERR_UNSUPPORTED),          # a norm for queries that are not there
    (dict(k=None), B.LORA_ERR_NULL), (dict(v=None), B.LORA_ERR_NULL),
    (dict(ld_k=248), B.LORA_ERR_SHAPE), (dict(ld_v=248), B.LORA_ERR_SHAPE), (dict(ld_q=1016), B.LORA_ERR_SHAPE),
    (dict(ld_qo=1016), B.LORA_ERR_SHAPE), (dict(ld_rope=124), B.LORA_ERR_SHAPE), (dict(rope_rows=-1), B.LORA_ERR_SHAPE),
    (dict(q=MIS), B.LORA_ERR_ALIGN), (dict(q_out=MIS), B.LORA_ERR_ALIGN), (dict(k=MIS), B.LORA_ERR_ALIGN),
    (dict(v=MIS), B.LORA_ERR_ALIGN), (dict(q_norm=MIS), B.LORA_ERR_ALIGN), (dict(k_norm=MIS), B.LORA_ERR_ALIGN),
    (dict(rope=MIS), B.LORA_ERR_ALIGN), (dict(ld_k=1540), B.LORA_ERR_ALIGN), (dict(ld_v=1532), B.LORA_ERR_ALIGN),
    (dict(ld_q=1540), B.LORA_ERR_ALIGN), (dict(ld_qo=1028), B.LORA_ERR_ALIGN), (dict(ld_rope=130), B.LORA_ERR_ALIGN),
    (dict(T=0, k=None, v=None, q=None, q_out=None, q_norm=None), B.LORA_OK),
])
def test_append_refusals(kw, status):
    assert append(**kw) == status


def test_no_cache_is_refused():
    assert append(False) == B.LORA_ERR_NULL and attention(False) == B.LORA_ERR_NULL


def attention(c=None, **kw):
    a = dict(q=FAKE, ld_q=1024, out=FAKE, ld_out=1024, lse=FAKE, ld_lse=8, T=4, q_heads=8, max_new=1, max_len=1280, scale=0.1,
             causal=1, window=0, chunk=256, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    c = cache() if c is None else c
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    return dsl.lib().lora_kv_attention(
        ctypes.byref(c) if c else None, vp(a["q"]), i64(a["ld_q"]), vp(a["out"]), i64(a["ld_out"]), vp(a["lse"]),
        i64(a["ld_lse"]), i64(a["T"]), i32(a["q_heads"]), i64(a["max_new"]), i64(a["max_len"]), ctypes.c_float(a["scale"]),
        i32(a["causal"]), i64(a["window"]), i64(a["chunk"]), vp(a["ws"]), ctypes.c_size_t(a["wsb"]), None)


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_attention_refuses_caches(kw, status):
    assert attention(cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), B.LORA_ERR_SHAPE), (dict(T=1 << 28, ld_q=1 << 20), B.LORA_ERR_SHAPE), (dict(q_heads=1), B.LORA_ERR_SHAPE),
    (dict(q_heads=7), B.LORA_ERR_UNSUPPORTED), (dict(max_new=0), B.LORA_ERR_SHAPE), (dict(max_new=1 << 40), B.LORA_ERR_SHAPE),
    (dict(max_len=0), B.LORA_ERR_SHAPE), (dict(max_len=(1 << 30) + 1), B.LORA_ERR_UNSUPPORTED),
    (dict(chunk=-256), B.LORA_ERR_SHAPE), (dict(chunk=100), B.LORA_ERR_UNSUPPORTED),
    (dict(window=-1), B.LORA_ERR_SHAPE), (dict(window=1 << 31), B.LORA_ERR_SHAPE),
    (dict(window=5, causal=0), B.LORA_ERR_UNSUPPORTED), (dict(causal=2), B.LORA_ERR_UNSUPPORTED),
    (dict(scale=0.0), B.LORA_ERR_UNSUPPORTED), (dict(scale=-1.0), B.LORA_ERR_UNSUPPORTED),
    (dict(scale=math.inf), B.LORA_ERR_UNSUPPORTED), (dict(scale=math.nan), B.LORA_ERR_UNSUPPORTED),
    (dict(q=None), B.LORA_ERR_NULL), (dict(out=None), B.LORA_ERR_NULL), (dict(ws=None), B.LORA_ERR_NULL),
    (dict(ld_q=1016), B.LORA_ERR_SHAPE), (dict(ld_out=1016), B.LORA_ERR_SHAPE), (dict(ld_lse=7), B.LORA_ERR_SHAPE),
    (dict(q=MIS), B.LORA_ERR_ALIGN), (dict(out=MIS), B.LORA_ERR_ALIGN), (dict(lse=MIS), B.LORA_ERR_ALIGN),
    (dict(ws=MIS), B.LORA_ERR_ALIGN), (dict(ld_q=1028), B.LORA_ERR_ALIGN), (dict(ld_out=1028), B.LORA_ERR_ALIGN),
    (dict(wsb=0), B.LORA_ERR_WORKSPACE), (dict(T=0, q=None, out=None), B.LORA_OK),
])
def test_attention_refusals(kw, status):
    assert attention(**kw) == status


def test_attention_launches_that_are_too_large_are_refused():
    many = cache(max_pages=1 << 24, ld_table=1 << 24, n_seqs=60000)
    assert attention(many, max_len=1 << 30, T=60000) == B.LORA_ERR_SHAPE
    assert dsl.lora_kv_attention_workspace_bytes(1 << 27, 8, 2, 128, 1, 1 << 30, 256) == 0


def test_attention_workspace():
    size = dsl.lora_kv_attention_workspace_bytes
    assert size(4, 8, 2, 128, 1, 1280, 1280) == 0 and size(4, 8, 2, 128, 1, 1280, 2560) == 0    # one chunk
    assert size(0, 8, 2, 128, 1, 1280, 256) == 0 and size(4, 8, 3, 128, 1, 1280, 256) == 0
    n = size(4, 8, 2, 128, 1, 1280, 256)
    assert n >= 5 * 4 * 8 * (128 + 2) * 4
    assert attention(wsb=n - 1) == B.LORA_ERR_WORKSPACE
    # fewer pages than the length asked for never take more
    for max_len in (300, 1280, 5000, 16640, 100000):
        need = size(4, 8, 2, 128, 1, max_len, 0)
        for pages in (1, 4, 5, 20, 260, 2000):
            st = attention(cache(max_pages=pages, ld_table=pages), max_len=max_len, chunk=0, wsb=need, q=MIS)
            assert st == B.LORA_ERR_ALIGN
            if need:
                c = cache(max_pages=pages, ld_table=pages, n_seqs=60000)
                assert attention(c, max_len=max_len, chunk=0, wsb=need, ws=FAKE, T=0) == B.LORA_OK


def test_attention_chunk_rule():
    rule = dsl.lora_kv_attention_chunk
    assert rule(0, 8, 2, 128, 100) == 0 and rule(1, 7, 2, 128, 100) == 0 and rule(1, 8, 2, 128, 0) == 0 and rule(1, 8, 2, 96, 9) == 0
    for max_new, Hq, H, n in [(1, 32, 8, 100), (1, 32, 8, 131072), (5, 32, 8, 6000), (512, 32, 8, 32768), (8192, 64, 8, 8192),
                              (1, 8, 1, 1 << 30), (1 << 20, 8, 8, 1 << 20)]:
        c = rule(max_new, Hq, H, 128, n)
        assert c > 0 and c % 256 == 0


def verify(**kw):
    a = dict(t=FAKE, ld_t=100, d=FAKE, ld_d=100, type=0, B=4, n=2, V=100, drafted=FAKE, u=FAKE, T=FAKE, k=FAKE, p=FAKE, m=FAKE,
             tokens=FAKE, accepted=FAKE, lp=FAKE, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    return dsl.lib().lora_verify(vp(a["t"]), i64(a["ld_t"]), vp(a["d"]), i64(a["ld_d"]), ctypes.c_int32(a["type"]), i64(a["B"]),
                                 i64(a["n"]), i64(a["V"]), vp(a["drafted"]), vp(a["u"]), vp(a["T"]), vp(a["k"]), vp(a["p"]),
                                 vp(a["m"]), vp(a["tokens"]), vp(a["accepted"]), vp(a["lp"]), vp(a["ws"]),
                                 ctypes.c_size_t(a["wsb"]), None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), B.LORA_ERR_SHAPE), (dict(n=-1), B.LORA_ERR_SHAPE), (dict(V=0), B.LORA_ERR_SHAPE),
    (dict(B=1 << 21), B.LORA_ERR_SHAPE), (dict(B=1 << 17, n=1, V=1 << 22, ld_t=1 << 22, ld_d=1 << 22), B.LORA_ERR_SHAPE),
    (dict(n=64), B.LORA_ERR_UNSUPPORTED), (dict(V=(1 << 22) + 1), B.LORA_ERR_UNSUPPORTED), (dict(type=2), B.LORA_ERR_UNSUPPORTED),
    (dict(t=None), B.LORA_ERR_NULL), (dict(u=None), B.LORA_ERR_NULL), (dict(drafted=None), B.LORA_ERR_NULL),
    (dict(tokens=None), B.LORA_ERR_NULL), (dict(accepted=None), B.LORA_ERR_NULL), (dict(ws=None), B.LORA_ERR_NULL),
    (dict(ld_t=99), B.LORA_ERR_SHAPE), (dict(ld_d=99), B.LORA_ERR_SHAPE),
    (dict(t=0x100001), B.LORA_ERR_ALIGN), (dict(type=1, t=MIS), B.LORA_ERR_ALIGN), (dict(type=1, d=MIS), B.LORA_ERR_ALIGN),
    (dict(drafted=MIS), B.LORA_ERR_ALIGN), (dict(u=MIS), B.LORA_ERR_ALIGN), (dict(lp=MIS), B.LORA_ERR_ALIGN),
    (dict(ws=0x100008), B.LORA_ERR_ALIGN), (dict(wsb=16), B.LORA_ERR_WORKSPACE), (dict(B=0, t=None, ws=None), B.LORA_OK),
])
def test_verify_refusals(kw, status):
    assert verify(**kw) == status


def test_verify_workspace():
    size = dsl.lora_verify_workspace_bytes
    assert size(0, 3) == 0 and size(4, -1) == 0 and size(4, 64) == 0 and size(1 << 21, 1) == 0
    assert verify(wsb=size(4, 2) - 1) == B.LORA_ERR_WORKSPACE
    assert size(5, 2) > size(4, 2) and size(4, 3) > size(4, 2)


def test_binding_refuses_what_does_not_fit():
    """On the CPU every tensor is refused before anything else of it is looked at."""
    import torch
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    c = dsl.KvCache(*[torch.zeros(1, dtype=torch.uint8)] * 7)
    with pytest.raises(ValueError, match="GPU tensor"):
        dsl.lora_kv_append(x, x, c)
    with pytest.raises(TypeError, match="KvCache"):
        dsl.lora_kv_attention(x, (1, 2), x, 1)
    with pytest.raises(TypeError, match="cache.k must be a tensor"):
        dsl.lora_kv_attention(x, dsl.KvCache(*[None] * 7), x, 1)
    with pytest.raises(ValueError, match="GPU tensor"):
        dsl.lora_verify(x, torch.zeros(4, 2, dtype=torch.int32), None, None, None, None)


# ---------------------------------------------------------------------------
# the references' own pins (values worked out by hand)
# ---------------------------------------------------------------------------
def test_reference_codes_by_hand():
    x = np.array([0.0, 1.0, -1.0, 1.0625, 1.1875, 448.0, 464.0, 1e9, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, -2.0 ** -11, 0.0146])
    # 1.0625 lies between 1 and 1.125: the even 1; 1.1875 between 1.125 and 1.25: the even 1.25; half the least: 0
    want = [0, 0x38, 0xB8, 0x38, 0x3A, 0x7E, 0x7E, 0x7E, 1, 0, 2, 0x80, 7]
    assert kv.encode(x).tolist() == want
    assert kv.VALUES[0x38] == 1.0 and kv.VALUES[0x7E] == 448.0 and np.isnan(kv.VALUES[0xFF]) and kv.VALUES[8] == 2.0 ** -6
    codes = np.arange(256)
    codes = codes[codes & 127 != 127]
    assert np.array_equal(kv.encode(kv.VALUES[codes]), codes)
    assert [kv.scale_byte(a) for a in (0.0, 448.0, 449.0, 224.0, 1.75, 3.4e38)] == [27, 127, 128, 126, 119, 246]


def test_reference_append_and_attention_by_hand():
    D = 64
    c = {"k": np.full((2, 1, 16, D), 0x7F, np.uint8), "v": np.full((2, 1, 1, D, 16), 0x7F, np.uint8),
         "ks": np.full((2, 1, 1), 200, np.uint8), "vs": np.full((2, 1, 1), 200, np.uint8)}
    table = np.array([[1]], dtype=np.int32)
    k, v = np.zeros((1, 1, D)), np.zeros((1, 1, D))
    k[0, 0, 0], v[0, 0, :2] = 1.0, [2.0, 448.0]
    kv.append(c, k, v, table, [1], [0, 1], 16)
    assert c["vs"][1, 0, 0] == 127 and c["v"][1, 0, 0, :2, 0].tolist() == [0x40, 0x7E] and c["ks"][0, 0, 0] == 200
    k[0, 0, 0], v[0, 0, :2] = 1.0, [4.0, 896.0]
    kv.append(c, k, v, table, [2], [0, 1], 16)
    assert c["vs"][1, 0, 0] == 128 and c["v"][1, 0, 0, :2, :2].tolist() == [[0x38, 0x40], [0x76, 0x7E]]
    q = np.zeros((1, 1, D))
    out, lse, _, _ = kv.attention(q, c, table, [2], [0, 1], 16, 1.0)
    assert out[0, 0, :2].tolist() == [3.0, 672.0] and abs(lse[0, 0] - math.log(2)) < 1e-12
    out, lse, _, _ = kv.attention(q, c, table, [2], [0, 1], 16, 1.0, window=1)
    assert out[0, 0, 0] == 4.0 and lse[0, 0] == 0.0
    out, lse, _, _ = kv.attention(q, c, np.array([[-1]]), [2], [0, 1], 16, 1.0)
    assert not out.any() and np.isneginf(lse).all()


def test_reference_verification_by_hand():
    p, q = np.log([[2.0, 1.0, 1.0]] * 2), np.log([[1.0, 2.0, 1.0]])
    plain = (1.0, 0, 1.0, 0.0)
    assert ref.probabilities(step.kept_weights(p[0])).tolist() == [2.0 ** 39, 2.0 ** 38, 2.0 ** 38]
    assert ref.verify(p, q, [1], [0.49, 0.1], plain)[:2] == ([1, 0], 1)
    assert ref.verify(p, q, [1], [0.51, 0.9], plain)[:2] == ([0, -1], 0)
    assert ref.verify(p, None, [1], [0.26, 0.7], plain)[:2] == ([2, -1], 0)
    assert ref.verify(p, None, [-1], [0.0, 0.6], plain)[:2] == ([1, -1], 0)
    assert ref.verify(p, None, [0], [0.9, 0.0], (0.0, 0, 1.0, 0.0))[:2] == ([0, 0], 1)
