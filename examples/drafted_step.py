"""A prompt and a step with drafted tokens of an adapted attention model, on this library's operators alone.

A small random model: per layer the fused QKV projection (MX4 weight, the adapter's LoRA term on top), the append of keys and
values to the paged 8-bit cache with the norms and the rotation, attention over it, the output projection and the normed
residual step; then a projection to the vocabulary.  Each sequence takes its prompt, then a step with its last token and
drafted ones, which are verified against the model's own distributions.

    python examples/drafted_step.py [--prompts 37 5 90] [--drafts 3] [--layers 2] [--hidden 512] [--vocab 4000]

Prints what was accepted and drawn, and how far the step's logits are from float32 over the same cache.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import deterministic_split_lora_amd as dsl  # noqa: E402
from examples.adapted_step import EPS, SPLIT_K, Mx4Weight  # noqa: E402

HEADS, KV_HEADS, D, PAGE, RANK = 8, 2, 64, 32, 16


def make_model(layers, hidden, vocab, gen):
    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

    def weight(rows, cols):
        return Mx4Weight(normal(rows, cols, std=1.0 / math.sqrt(cols)))

    qkv = (HEADS + 2 * KV_HEADS) * D
    return {"embed": normal(vocab, hidden), "head": weight(vocab, hidden), "final_norm": 1.0 + normal(hidden, std=0.1),
            "layers": [{"qkv": weight(qkv, hidden), "o": weight(hidden, HEADS * D),
                        "A": normal(RANK, hidden, std=1.0 / math.sqrt(hidden)), "B": normal(qkv, RANK, std=0.1),
                        "q_norm": 1.0 + normal(D, std=0.1), "k_norm": 1.0 + normal(D, std=0.1),
                        "pre": 1.0 + normal(hidden, std=0.1)} for _ in range(layers)]}


def make_caches(layers, lengths):
    """A cache of each layer over the same pages: room for these many tokens a sequence."""
    pages = [(n + PAGE - 1) // PAGE for n in lengths]
    table = torch.full((len(lengths), max(pages)), -1, dtype=torch.int32)
    order = torch.randperm(sum(pages), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    for b, n in enumerate(pages):
        table[b, :n] = order[sum(pages[:b]):sum(pages[:b]) + n]
    shape = (sum(pages), KV_HEADS)
    zeros = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    lens = torch.zeros(len(lengths), dtype=torch.int32, device="cuda")
    starts = torch.zeros(len(lengths) + 1, dtype=torch.int32, device="cuda")
    return [dsl.KvCache(zeros(*shape, PAGE, D), zeros(*shape, PAGE // 16, D, 16), zeros(*shape, PAGE // 16),
                        zeros(*shape, PAGE // 16), table.cuda(), lens, starts) for _ in range(layers)]


def rope_table(n):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    return torch.cat((a.cos(), a.sin()), 1).float().cuda()


def step(model, caches, tokens, new, lengths, rope):
    """Logits of all new tokens (new[b] of sequence b, lengths[b] tokens with them), whose keys and values are appended."""
    T, hidden, vocab = tokens.numel(), model["embed"].shape[1], model["head"].q.shape[0]
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    caches[0].seq_lens.copy_(torch.tensor(lengths, dtype=torch.int32))
    caches[0].cu_tokens.copy_(torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32))
    width = (HEADS + 2 * KV_HEADS) * D
    r = model["embed"][tokens.long()]
    x, y, qkv = torch.empty(T, hidden, **bf16), torch.empty(T, hidden, **bf16), torch.empty(T, width, **bf16)
    q, att, logits = torch.empty(T, HEADS, D, **bf16), torch.empty(T, HEADS, D, **bf16), torch.empty(T, vocab, **bf16)
    sizes = ((hidden, width), (HEADS * D, hidden), (hidden, vocab))
    need = max(dsl.lora_mx4_linear_workspace_bytes(T, k, n, SPLIT_K) for k, n in sizes)
    base_ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    lora_ws = torch.empty(dsl.lora_shrink_expand_workspace_bytes(T, RANK, SPLIT_K), dtype=torch.uint8, device="cuda")
    need = dsl.lora_kv_attention_workspace_bytes(T, HEADS, KV_HEADS, D, max(new), max(lengths))
    att_ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    dsl.lora_block_norm(r, r, pre="rms", pre_w=model["layers"][0]["pre"], x_out=x, eps=EPS)
    for i, (layer, cache) in enumerate(zip(model["layers"], caches)):
        layer["qkv"](x, qkv, base_ws)
        dsl.lora_shrink_expand(x, layer["A"], layer["B"], qkv, lora_ws, SPLIT_K)
        heads = qkv.view(T, -1, D)
        dsl.lora_kv_append(heads[:, HEADS:HEADS + KV_HEADS], heads[:, HEADS + KV_HEADS:], cache, q=heads[:, :HEADS], q_out=q,
                           q_norm=layer["q_norm"], k_norm=layer["k_norm"], rope=rope)
        dsl.lora_kv_attention(q, cache, att, max_new=max(new), max_len=max(lengths), workspace=att_ws)
        layer["o"](att.view(T, -1), y, base_ws)
        nxt = model["layers"][i + 1]["pre"] if i + 1 < len(model["layers"]) else model["final_norm"]
        dsl.lora_block_norm(r, r, y=y, pre="rms", pre_w=nxt, x_out=x, eps=EPS)
    model["head"](x, logits, base_ws)
    return logits


def reference(model, caches, tokens, new, lengths, rope):
    """The logits in float32, with the same quantised weights and what the caches hold."""
    def rms(v, w):
        return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w.float()

    def turn(v, c, s):
        a, b = v[..., :D // 2], v[..., D // 2:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    pos = torch.cat([torch.arange(n - m, n) for m, n in zip(new, lengths)]).cuda()
    c, s = rope[pos][:, None, :D // 2], rope[pos][:, None, D // 2:]
    r = model["embed"][tokens.long()].float()
    x = rms(r, model["layers"][0]["pre"])
    for i, (layer, cache) in enumerate(zip(model["layers"], caches)):
        qkv = x @ layer["qkv"].values.float().t() + (x @ layer["A"].float().t()) @ layer["B"].float().t()
        q = turn(rms(qkv.view(len(pos), -1, D)[:, :HEADS], layer["q_norm"]), c, s)
        out, at = torch.empty(len(pos), HEADS, D, device="cuda"), 0
        for b, (m, n) in enumerate(zip(new, lengths)):
            page = cache.page_table[b, :(n + PAGE - 1) // PAGE].long()
            scale = lambda t: torch.exp2(t[page].float() - 127)[..., None, None]  # noqa: E731
            k = cache.k.view(torch.float8_e4m3fn)[page].float().view(len(page), KV_HEADS, -1, 16, D) * scale(cache.k_scales)
            v = cache.v.view(torch.float8_e4m3fn)[page].float().transpose(-1, -2) * scale(cache.v_scales)
            k, v = (t.transpose(0, 1).reshape(KV_HEADS, -1, D)[:, :n].repeat_interleave(HEADS // KV_HEADS, 0) for t in (k, v))
            l = q[at:at + m].transpose(0, 1) @ k.transpose(1, 2).contiguous() / math.sqrt(D)
            hidden = torch.arange(n, device="cuda") > torch.arange(n - m, n, device="cuda")[:, None]
            out[at:at + m] = (torch.softmax(l.masked_fill(hidden, -math.inf), -1) @ v).transpose(0, 1)
            at += m
        r = r + out.flatten(1) @ layer["o"].values.float().t()
        x = rms(r, model["layers"][i + 1]["pre"] if i + 1 < len(model["layers"]) else model["final_norm"])
    return x @ model["head"].values.float().t()


def run(a):
    gen = torch.Generator(device="cuda").manual_seed(0)
    model = make_model(a.layers, a.hidden, a.vocab, gen)
    B, n = len(a.prompts), a.drafts
    caches = make_caches(a.layers, [p + n + 1 for p in a.prompts])
    rope = rope_table(max(a.prompts) + n + 1)
    tokens = torch.randint(0, a.vocab, (sum(a.prompts),), generator=gen, device="cuda")
    step(model, caches, tokens, a.prompts, a.prompts, rope)
    # each sequence's next token and its drafts, as a lookup table proposes them
    line = torch.randint(0, a.vocab, (B, n + 1), generator=gen, device="cuda", dtype=torch.int32)
    lengths = [p + n + 1 for p in a.prompts]
    first = step(model, caches, line.flatten(), [n + 1] * B, lengths, rope)
    # each first draft is what the model itself would say (the drafts behind a token reach its logits only through the
    # scale that their block of 16 tokens shares)
    own = first.view(B, n + 1, -1)[:, :n].float().argmax(-1).to(torch.int32)
    line[:, 1:2] = own[:, :1]
    logits = step(model, caches, line.flatten(), [n + 1] * B, lengths, rope)
    u = torch.rand(B, n + 1, generator=gen, device="cuda")
    u[:, 0] = 0.0
    out = torch.empty(B, n + 1, dtype=torch.int32, device="cuda")
    accepted = torch.empty(B, dtype=torch.int32, device="cuda")
    logprobs = torch.empty(B, n + 1, device="cuda")
    ws = torch.empty(dsl.lora_verify_workspace_bytes(B, n), dtype=torch.uint8, device="cuda")
    settings = {"temperature": torch.full((B,), 0.8, device="cuda"), "top_p": torch.full((B,), 0.95, device="cuda")}
    dsl.lora_verify(logits, line[:, 1:].contiguous(), u, out, accepted, ws, logprobs=logprobs, **settings)
    torch.cuda.synchronize()
    want = reference(model, caches, line.flatten(), [n + 1] * B, lengths, rope)
    worst = float((logits.float() - want).abs().max() / want.square().mean().sqrt())
    return {"drafted": line[:, 1:].tolist(), "tokens": out.tolist(), "accepted": accepted.tolist(), "logits": logits,
            "worst": worst}


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--prompts", type=int, nargs="+", default=[37, 5, 90])
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=4000)
    a = ap.parse_args(argv)
    report = run(a)
    again = run(a)
    assert torch.equal(report["logits"], again["logits"]) and report["tokens"] == again["tokens"], "two runs differ"
    print("drafted ", report["drafted"])
    print("accepted", report["accepted"])
    print("tokens  ", report["tokens"])
    print("largest difference of a logit from float32, in units of the logits' size: %.4f" % report["worst"])
    return report


if __name__ == "__main__":
    main()
