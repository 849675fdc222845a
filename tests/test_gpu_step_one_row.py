"""Matrices of one row, whose stride(0) says nothing: 0, a transposed column's 1, or their width where it is odd."""
import numpy as np
import pytest

import deterministic_split_lora_amd as dsl
from tests.helpers import gpu_available, torch
from tests.test_gpu_step import Product

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def one_rows(v):
    """[1, n] views of a vector with strides 0, 1 and n."""
    return [v.as_strided((1, v.numel()), (0, 1)), v.view(-1, 1).t(), v.view(1, -1)]


def test_norm_and_gate_of_one_row():
    t = torch()
    C = 200
    r, y, gate = (t.randn(C, device="cuda").to(t.bfloat16) for _ in range(3))
    outs = []
    for rv, yv, gv in zip(one_rows(r), one_rows(y), one_rows(gate)):
        ro, xo = (one_rows(t.empty(C, dtype=t.bfloat16, device="cuda"))[len(outs)] for _ in range(2))
        dsl.lora_block_norm(rv, ro, y=yv, post="rms", gate=gv, pre="layer", x_out=xo)
        outs.append((ro.clone(), xo.clone()))
    for ro, xo in outs[:2]:
        assert t.equal(ro, outs[2][0]) and t.equal(xo, outs[2][1])


@pytest.mark.parametrize("mx", [False, True])
def test_product_of_one_row(mx):
    t = torch()
    K, N = 1056, 72
    p = Product(1, K, N, 4, mx).gpu()
    want = p.run(1)
    for i in range(3):
        x = one_rows(p.xg[0])[i]
        y = one_rows(t.empty(N, dtype=t.bfloat16, device="cuda"))[i]
        if mx:
            dsl.lora_mx4_linear_q(x, one_rows(p.xs[0, :K // 32])[i], p.wq, p.ws, y, 1)
        else:
            dsl.lora_mx4_linear(x, p.wq, p.ws, y, 1)
        assert np.array_equal(y.view(t.int16).cpu().numpy(), want.view(t.int16).cpu().numpy())
        if not mx:
            q, s = (one_rows(t.full((n,), 7, dtype=t.uint8, device="cuda"))[i] for n in (K // 2, K // 32))
            back = one_rows(t.empty(K, dtype=t.bfloat16, device="cuda"))[i]
            dsl.lora_mx4_quantize(x, q, s)
            dsl.lora_mx4_dequantize(q, s, back)
            q1, s1 = t.empty(1, K // 2, dtype=t.uint8, device="cuda"), t.empty(1, 36, dtype=t.uint8, device="cuda")
            dsl.lora_mx4_quantize(p.xg, q1, s1)
            assert t.equal(q, q1) and t.equal(s, s1[:, :K // 32])


def test_sample_of_one_row():
    t = torch()
    l = t.randn(1001, device="cuda")
    u = t.full((1,), 0.3, device="cuda")
    got = []
    for v in one_rows(l):
        tok = t.empty(1, dtype=t.int32, device="cuda")
        dsl.lora_sample(v, u, tok)
        got.append(int(tok))
    assert got[0] == got[1] == got[2]
