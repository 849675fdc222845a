"""The operators around the adapters on the host: argument checks (every call
below carries a defect that the host catches, or has nothing to do, so the
fake addresses are never followed), workspace sizes, and the CPU reference's
own pins."""
import numpy as np
import pytest

import deterministic_split_lora_amd as dsl
from deterministic_split_lora_amd import _binding as B
from oracle import step

FAKE = 0x100000
MIS = 0x100002


def quantize(fn="lora_mx4_quantize", **kw):
    a = dict(x=FAKE, ld_x=256, q=FAKE, ld_q=128, s=FAKE, ld_s=8, M=4, K=256)
    a.update(kw)
    if fn == "lora_mx4_quantize":
        return dsl.lib().lora_mx4_quantize(a["x"], a["ld_x"], a["q"], a["ld_q"], a["s"], a["ld_s"], a["M"], a["K"], None)
    return dsl.lib().lora_mx4_dequantize(a["q"], a["ld_q"], a["s"], a["ld_s"], a["x"], a["ld_x"], a["M"], a["K"], None)


@pytest.mark.parametrize("fn", ["lora_mx4_quantize", "lora_mx4_dequantize"])
@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), B.LORA_ERR_SHAPE), (dict(K=0), B.LORA_ERR_SHAPE), (dict(K=1 << 31), B.LORA_ERR_SHAPE),
    (dict(M=(1 << 31) - 1, K=1 << 20, ld_x=1 << 20), B.LORA_ERR_SHAPE),
    (dict(K=40), B.LORA_ERR_UNSUPPORTED),
    (dict(x=None), B.LORA_ERR_NULL), (dict(q=None), B.LORA_ERR_NULL), (dict(s=None), B.LORA_ERR_NULL),
    (dict(ld_x=248), B.LORA_ERR_SHAPE), (dict(ld_q=112), B.LORA_ERR_SHAPE), (dict(ld_s=4), B.LORA_ERR_SHAPE),
    (dict(x=MIS), B.LORA_ERR_ALIGN), (dict(q=MIS), B.LORA_ERR_ALIGN), (dict(s=MIS), B.LORA_ERR_ALIGN),
    (dict(ld_x=260), B.LORA_ERR_ALIGN), (dict(ld_q=136), B.LORA_ERR_ALIGN), (dict(ld_s=9), B.LORA_ERR_ALIGN),
    (dict(M=0, x=None, q=None, s=None), B.LORA_OK),
])
def test_mx4_conversion_refusals(fn, kw, status):
    assert quantize(fn, **kw) == status


def linear(mx=False, **kw):
    a = dict(x=FAKE, ld_x=(256 if mx else 512), xs=FAKE, ld_xs=16, wq=FAKE, ld_wq=256, ws=FAKE, ld_ws=16, y=FAKE,
             ld_y=64, M=4, K=512, N=64, S=4, wsp=FAKE, wspb=1 << 40)
    a.update(kw)
    L = dsl.lib()
    if mx:
        return L.lora_mx4_linear_q(a["x"], a["ld_x"], a["xs"], a["ld_xs"], a["wq"], a["ld_wq"], a["ws"], a["ld_ws"],
                                   a["y"], a["ld_y"], a["M"], a["K"], a["N"], a["S"], a["wsp"], a["wspb"], None)
    return L.lora_mx4_linear(a["x"], a["ld_x"], a["wq"], a["ld_wq"], a["ws"], a["ld_ws"], a["y"], a["ld_y"], a["M"],
                             a["K"], a["N"], a["S"], a["wsp"], a["wspb"], None)


LINEAR_REFUSALS = [
    (dict(M=-1), B.LORA_ERR_SHAPE), (dict(N=-8), B.LORA_ERR_SHAPE), (dict(K=0), B.LORA_ERR_SHAPE),
    (dict(M=(1 << 31) - 1), B.LORA_ERR_SHAPE), (dict(N=(1 << 25) + 8, ld_y=1 << 26), B.LORA_ERR_SHAPE),
    (dict(M=64 * 65535, N=1 << 14, ld_y=1 << 14), B.LORA_ERR_SHAPE),
    (dict(ld_wq=(1 << 23) + 16), B.LORA_ERR_UNSUPPORTED), (dict(ld_ws=(1 << 23) + 4), B.LORA_ERR_UNSUPPORTED),
    (dict(ld_x=(1 << 23) + 16), B.LORA_ERR_UNSUPPORTED),
    (dict(S=3), B.LORA_ERR_UNSUPPORTED), (dict(S=32), B.LORA_ERR_UNSUPPORTED), (dict(S=0), B.LORA_ERR_UNSUPPORTED),
    (dict(K=96, S=2), B.LORA_ERR_UNSUPPORTED), (dict(N=60), B.LORA_ERR_UNSUPPORTED),
    (dict(x=None), B.LORA_ERR_NULL), (dict(wq=None), B.LORA_ERR_NULL), (dict(ws=None), B.LORA_ERR_NULL),
    (dict(y=None), B.LORA_ERR_NULL),
    (dict(ld_x=248), B.LORA_ERR_SHAPE), (dict(ld_wq=240), B.LORA_ERR_SHAPE), (dict(ld_ws=12), B.LORA_ERR_SHAPE),
    (dict(ld_y=56), B.LORA_ERR_SHAPE),
    (dict(x=MIS), B.LORA_ERR_ALIGN), (dict(wq=MIS), B.LORA_ERR_ALIGN), (dict(ws=MIS), B.LORA_ERR_ALIGN),
    (dict(y=MIS), B.LORA_ERR_ALIGN), (dict(wsp=MIS), B.LORA_ERR_ALIGN), (dict(ld_x=517), B.LORA_ERR_ALIGN),
    (dict(ld_wq=264), B.LORA_ERR_ALIGN), (dict(ld_ws=17), B.LORA_ERR_ALIGN), (dict(ld_y=68), B.LORA_ERR_ALIGN),
    (dict(M=0, x=None), B.LORA_OK), (dict(N=0, wq=None), B.LORA_OK),
]


@pytest.mark.parametrize("kw,status", LINEAR_REFUSALS)
def test_linear_refusals(kw, status):
    assert linear(**kw) == status


@pytest.mark.parametrize("kw,status", LINEAR_REFUSALS + [
    (dict(xs=None), B.LORA_ERR_NULL), (dict(xs=MIS), B.LORA_ERR_ALIGN), (dict(ld_xs=12), B.LORA_ERR_SHAPE),
    (dict(ld_xs=18), B.LORA_ERR_ALIGN)])
def test_linear_q_refusals(kw, status):
    assert linear(True, **kw) == status


def test_linear_workspace_is_checked():
    assert dsl.lora_mx4_linear_workspace_bytes(-1, 512, 64, 4) == 0
    assert dsl.lora_mx4_linear_workspace_bytes(4, 512, 64, 3) == 0
    assert dsl.lora_mx4_linear_workspace_bytes(0, 512, 64, 4) == 0
    assert dsl.lora_mx4_linear_workspace_bytes(4096, 4096, 4096, 1) == 0       # one chunk: nothing to join
    for M, K, N, S in [(200, 4096, 6144, 4), (128, 8192, 1024, 8), (300, 2048, 512, 16)]:
        n = dsl.lora_mx4_linear_workspace_bytes(M, K, N, S)
        if n:                                  # the larger need of the two products: one byte less is refused by one
            kw = dict(M=M, K=K, N=N, S=S, ld_wq=K // 2, ld_ws=K // 32, ld_y=N, wsp=None, wspb=0)
            assert linear(ld_x=K, **kw) == B.LORA_ERR_WORKSPACE


def norm(**kw):
    a = dict(y=FAKE, ld_y=64, post=1, post_w=FAKE, post_b=None, gate=FAKE, ld_gate=64, group=1, r=FAKE, ld_r=64,
             rs=1.0, r_out=FAKE, ld_ro=64, pre=1, pre_w=FAKE, pre_b=None, x_out=FAKE, ld_xo=64, M=4, C=64, eps=1e-5)
    a.update(kw)
    return dsl.lib().lora_block_norm(a["y"], a["ld_y"], a["post"], a["post_w"], a["post_b"], a["gate"], a["ld_gate"],
                                     a["group"], a["r"], a["ld_r"], a["rs"], a["r_out"], a["ld_ro"], a["pre"],
                                     a["pre_w"], a["pre_b"], a["x_out"], a["ld_xo"], a["M"], a["C"], a["eps"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), B.LORA_ERR_SHAPE), (dict(C=-8), B.LORA_ERR_SHAPE),
    (dict(C=0), B.LORA_ERR_UNSUPPORTED), (dict(C=60), B.LORA_ERR_UNSUPPORTED), (dict(C=32776), B.LORA_ERR_UNSUPPORTED),
    (dict(post=3), B.LORA_ERR_UNSUPPORTED), (dict(pre=-1), B.LORA_ERR_UNSUPPORTED),
    (dict(r=None), B.LORA_ERR_NULL), (dict(r_out=None), B.LORA_ERR_NULL), (dict(x_out=None), B.LORA_ERR_NULL),
    (dict(y=None), B.LORA_ERR_NULL), (dict(pre=0, pre_w=None), B.LORA_ERR_UNSUPPORTED),
    (dict(post=0), B.LORA_ERR_UNSUPPORTED), (dict(y=None, post=0, post_w=None), B.LORA_ERR_UNSUPPORTED),
    (dict(ld_y=56), B.LORA_ERR_SHAPE), (dict(ld_r=56), B.LORA_ERR_SHAPE), (dict(ld_ro=56), B.LORA_ERR_SHAPE),
    (dict(ld_xo=56), B.LORA_ERR_SHAPE), (dict(ld_gate=56), B.LORA_ERR_SHAPE), (dict(group=0), B.LORA_ERR_SHAPE),
    (dict(y=MIS), B.LORA_ERR_ALIGN), (dict(r=MIS), B.LORA_ERR_ALIGN), (dict(r_out=MIS), B.LORA_ERR_ALIGN),
    (dict(x_out=MIS), B.LORA_ERR_ALIGN), (dict(gate=MIS), B.LORA_ERR_ALIGN), (dict(post_w=MIS), B.LORA_ERR_ALIGN),
    (dict(pre_w=MIS), B.LORA_ERR_ALIGN), (dict(pre_b=MIS), B.LORA_ERR_ALIGN), (dict(ld_y=68), B.LORA_ERR_ALIGN),
    (dict(ld_gate=68), B.LORA_ERR_ALIGN), (dict(M=0, r=None), B.LORA_OK),
])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


def sample(**kw):
    a = dict(logits=FAKE, type=0, ld=100, B=4, V=100, t=FAKE, k=FAKE, p=FAKE, m=FAKE, u=FAKE, tok=FAKE, lp=FAKE)
    a.update(kw)
    return dsl.lib().lora_sample(a["logits"], a["type"], a["ld"], a["B"], a["V"], a["t"], a["k"], a["p"], a["m"],
                                 a["u"], a["tok"], a["lp"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), B.LORA_ERR_SHAPE), (dict(B=(1 << 21) + 1), B.LORA_ERR_SHAPE), (dict(V=0), B.LORA_ERR_SHAPE), (dict(ld=99), B.LORA_ERR_SHAPE),
    (dict(V=(1 << 22) + 1, ld=1 << 23), B.LORA_ERR_UNSUPPORTED), (dict(type=2), B.LORA_ERR_UNSUPPORTED),
    (dict(logits=None), B.LORA_ERR_NULL), (dict(u=None), B.LORA_ERR_NULL), (dict(tok=None), B.LORA_ERR_NULL),
    (dict(logits=FAKE + 1), B.LORA_ERR_ALIGN), (dict(logits=MIS, type=1), B.LORA_ERR_ALIGN),
    (dict(t=MIS), B.LORA_ERR_ALIGN), (dict(k=MIS), B.LORA_ERR_ALIGN), (dict(u=MIS), B.LORA_ERR_ALIGN),
    (dict(tok=MIS), B.LORA_ERR_ALIGN), (dict(lp=MIS), B.LORA_ERR_ALIGN), (dict(B=0, logits=None), B.LORA_OK),
])
def test_sample_refusals(kw, status):
    assert sample(**kw) == status


def test_compiled_binding_refuses_host_tensors():
    import torch
    x, q, s = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(
        2, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU tensor"):
        dsl.lora_mx4_quantize(x, q, s)
    with pytest.raises(TypeError):
        dsl.lora_mx4_quantize(x.float(), q, s)
    with pytest.raises(TypeError):
        dsl.lora_sample(None, None, None)


# ---------------------------------------------------------------------------
# the reference's own pins (values worked out by hand)
# ---------------------------------------------------------------------------
def test_reference_quantisation_by_hand():
    x = np.zeros((1, 64))
    x[0, :12] = [6.0, 0.25, 0.75, -1.25, 1.75, 2.5, 3.5, 5.0, -0.2, 0.3, 7.9, -0.0]
    x[0, 32:35] = [2.0 ** -130, -2.0 ** -126, 2.0 ** -128]
    code, s = step.mx4_quantize(x)
    assert s.tolist() == [[127, 0]]
    # ties go to the even code: .25 -> 0, .75 -> 1 (2), 1.25 -> 1 (2), 1.75 -> 2 (4), 2.5 -> 2 (4), 3.5 -> 4 (6), 5 -> 4 (6)
    assert code[0, :12].tolist() == [7, 0, 2, 8 + 2, 4, 4, 6, 6, 8, 1, 7, 8]
    # 2^-126 = 2 2^-127 and 2^-128 = 0.5 2^-127; 2^-130 is an eighth of a unit: 0
    assert code[0, 32:35].tolist() == [0, 8 + 4, 1]
    assert step.mx4_values(code, s)[0, 33] == -2.0 ** -126
    x[0, 5] = np.inf
    code, s = step.mx4_quantize(x)
    assert s[0, 0] == 255 and np.isnan(step.mx4_values(code, s)[0, :32]).all() and not code[0, :32].any()
    q = step.mx4_pack(np.arange(16, dtype=np.uint8).reshape(1, 16))
    assert q.tolist() == [[0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]]
    assert step.mx4_unpack(q).tolist() == [list(range(16))]


def test_reference_sampling_by_hand():
    l = np.log(np.array([1.0, 4.0, 2.0, 1.0]))                 # weights 1/4, 1, 1/2, 1/4 of the largest
    w = step.weights(l, 1.0)
    assert abs(w / 2.0 ** 31 - [0.25, 1, 0.5, 0.25]).max() < 1e-9
    assert np.flatnonzero(step.kept_weights(l, top_k=3)).tolist() == [0, 1, 2]       # the tie goes to index 0
    assert np.flatnonzero(step.kept_weights(l, top_p=0.45)).tolist() == [1]          # 1 of 2 >= 0.45
    assert np.flatnonzero(step.kept_weights(l, top_p=0.6)).tolist() == [1, 2]
    assert np.flatnonzero(step.kept_weights(l, min_p=0.4)).tolist() == [1, 2]
    assert np.flatnonzero(step.kept_weights(l, top_p=0.0)).tolist() == [1]
    assert np.flatnonzero(step.kept_weights(l, temperature=0.0)).tolist() == [1]
    k = step.kept_weights(l)
    assert [step.draw(k, u) for u in (0.0, 0.12, 0.13, 0.62, 0.63, 0.87, 0.88, 0.999)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert step.draw(step.kept_weights(np.full(3, -np.inf)), 0.5) == -1
