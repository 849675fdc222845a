"""The paged cache's operators and the verification together, as a step of a model uses them."""
import numpy as np
import pytest

import deterministic_split_lora_amd as dsl
from oracle import bf16_to_f64, kv
from tests.helpers import bf16_from_gpu, gpu_available, torch
from tests.kv_helpers import Batch, attend, heads_bf16

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def test_example_runs():
    import examples.drafted_step as example
    report = example.main([])
    # the first draft is the model's likeliest token and its random number 0, so it is always accepted
    assert all(1 <= n <= 3 for n in report["accepted"])
    for got, drafted, n in zip(report["tokens"], report["drafted"], report["accepted"]):
        assert got[:n] == drafted[:n] and got[n] >= 0 and all(t == -1 for t in got[n + 1:])
    # activations are rounded to bf16 (half a step, 2^-8) about seven times a layer, the P and the adapters' h once more
    assert report["worst"] < 0.1


@pytest.mark.parametrize("Hq,H,D,P", [(8, 2, 128, 32), (6, 6, 64, 16), (4, 1, 256, 64)])
def test_prompt_then_tokens(Hq, H, D, P):
    """A prompt in two chunks, then single tokens and drafts: every step's attention against the formula on the reference's
    cache, which is appended to alike."""
    lens = [0, 0, 0]
    top = 220
    batch = Batch([(1, top)] * 3, P, H, D, seed=7)
    g = None
    for i, new in enumerate(([70, 3, 17], [90, 64, 16], [1, 1, 1], [1, 1, 1], [4, 2, 5], [1, 0, 1])):
        lens = [a + b for a, b in zip(lens, new)]
        batch.lens = np.array(lens, dtype=np.int32)
        batch.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        batch.T = int(batch.cu[-1])
        g = batch.gpu()
        x, xg = heads_bf16(batch.T, Hq + 2 * H, D, 1.0, i, "x")
        q = torch().empty(batch.T, Hq, D, dtype=torch().bfloat16, device="cuda")
        dsl.lora_kv_append(xg[:, Hq:Hq + H], xg[:, Hq + H:], g, q=xg[:, :Hq], q_out=q)
        kv.append(batch.cache, x[:, Hq:Hq + H], x[:, Hq + H:], batch.table, batch.lens, batch.cu, P)
        got, _ = attend(q, g, max(new))
        out, _, tol, _ = kv.attention(x[:, :Hq], batch.cache, batch.table, batch.lens, batch.cu, P, D ** -0.5)
        assert np.all(np.abs(bf16_to_f64(bf16_from_gpu(got)) - out) <= tol), f"step {i}"
        batch.same(g)


def test_drafted_tokens_get_the_bits_of_single_ones():
    """Up to 16 rows of a key head, a token's attention does not depend on how many tokens its step has."""
    t = torch()
    batch = Batch([(4, 700), (4, 333)], 16, 2, 64, seed=2).fill()
    q, qg = heads_bf16(8, 8, 64, 1.0, 4, "q")
    whole, lse = attend(qg, batch.gpu(), 4, chunk=256)
    for i in range(4):
        one = Batch([(1, 700 - 3 + i), (1, 333 - 3 + i)], 16, 2, 64, seed=2)
        one.cache, one.table, one.n_pages = batch.cache, batch.table, batch.n_pages
        out, l = attend(qg[[i, 4 + i]], one.gpu(), 1, chunk=256)
        assert t.equal(out.view(t.int16), whole[[i, 4 + i]].view(t.int16)) and t.equal(l, lse[[i, 4 + i]])


def test_the_longest_hint_is_only_a_hint():
    """More new tokens than max_new says, and fewer: every row is served."""
    batch = Batch([(9, 90), (40, 300), (1, 20)], 16, 1, 128, seed=2).fill()
    q, qg = heads_bf16(50, 5, 128, 1.0, 4, "q")
    out, _, tol, _ = kv.attention(q, batch.cache, batch.table, batch.lens, batch.cu, 16, 128 ** -0.5)
    for hint in (1, 3, 10, 40, 1000):
        for chunk in (0, 256):
            got, _ = attend(qg, batch.gpu(), hint, chunk=chunk)
            assert np.all(np.abs(bf16_to_f64(bf16_from_gpu(got)) - out) <= tol), hint


def test_binding_refuses():
    t = torch()
    batch = Batch([(2, 20)], 16, 2, 64, seed=1).fill()
    g = batch.gpu()
    x, xg = heads_bf16(2, 8, 64, 1.0, 1, "x")
    q, out = xg[:, :4], t.empty(2, 4, 64, dtype=t.bfloat16, device="cuda")
    for bad in (g._replace(v=g.v[:1]), g._replace(k_scales=g.k_scales[:, :1]), g._replace(page_table=g.page_table.long()),
                g._replace(seq_lens=g.seq_lens[:0]), g._replace(cu_tokens=g.cu_tokens[:1]), g._replace(k=g.k[..., :32]),
                g._replace(k=g.k.transpose(1, 2)), g._replace(k=g.k.cpu()), g._replace(k=g.k.to(t.int32))):
        with pytest.raises((ValueError, TypeError)):
            dsl.lora_kv_attention(q, bad, out, 2)
        with pytest.raises((ValueError, TypeError)):
            dsl.lora_kv_append(xg[:, 4:6], xg[:, 6:], bad)
    for call in (lambda: dsl.lora_kv_attention(q.float(), g, out, 2), lambda: dsl.lora_kv_attention(q, g, out[:1], 2),
                 lambda: dsl.lora_kv_attention(q[..., :32], g, out, 2), lambda: dsl.lora_kv_attention(q[:, :2], g, out, 2),
                 lambda: dsl.lora_kv_attention(q, g, out, 2, lse=t.empty(4, 2, device="cuda")),
                 lambda: dsl.lora_kv_append(xg[:, 4:5], xg[:, 6:7], g), lambda: dsl.lora_kv_append(xg[:, 4:6], xg[:1, 6:], g),
                 lambda: dsl.lora_kv_append(xg[:, 4:6], xg[:, 6:], g, q=q), lambda: dsl.lora_kv_append(
                     xg[:, 4:6], xg[:, 6:], g, k_norm=t.ones(32, dtype=t.bfloat16, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(dsl.LoraError):
        dsl.lora_kv_attention(q, g, out, 2, window=3, causal=False)
    with pytest.raises(dsl.LoraError):
        dsl.lora_kv_attention(q, g, out, 2, max_len=512, chunk=100)
    with pytest.raises(dsl.LoraError):
        dsl.lora_kv_attention(xg[:, :3], g, t.empty(2, 3, 64, dtype=t.bfloat16, device="cuda"), 2)
    l, d = t.zeros(6, 50, device="cuda"), t.zeros(2, 2, dtype=t.int32, device="cuda")
    u, tok, acc = t.zeros(2, 3, device="cuda"), t.zeros(2, 3, dtype=t.int32, device="cuda"), t.zeros(2, dtype=t.int32, device="cuda")
    ws = t.empty(dsl.lora_verify_workspace_bytes(2, 2), dtype=t.uint8, device="cuda")
    dsl.lora_verify(l, d, u, tok, acc, ws)
    for call in (lambda: dsl.lora_verify(l[:5], d, u, tok, acc, ws), lambda: dsl.lora_verify(l, d, u[:, :2], tok, acc, ws),
                 lambda: dsl.lora_verify(l, d, u, tok[:1], acc, ws), lambda: dsl.lora_verify(l.half(), d, u, tok, acc, ws),
                 lambda: dsl.lora_verify(l, d, u, tok, acc, ws, draft_logits=l[:4].to(t.bfloat16)),
                 lambda: dsl.lora_verify(l, d, u, tok, acc, ws, draft_logits=l[:4, :40]),
                 lambda: dsl.lora_verify(l, d.t().contiguous().t(), u, tok, acc, ws)):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(dsl.LoraError):
        dsl.lora_verify(l, d, u, tok, acc, ws[:16])
