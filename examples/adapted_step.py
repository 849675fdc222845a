"""One decode step of an adapted model, on this library's operators alone.

A small random model: per layer a projection whose frozen weight is held in MX4
(4.25 bits a value), the LoRA term of each token's own adapter, and the gated,
normed residual step between layers; then a projection to the vocabulary and a
draw of every token's successor with its own settings.

    python examples/adapted_step.py [--tokens 8] [--layers 4] [--hidden 1024] [--vocab 8000] [--adapters 3]

Prints the drawn tokens and how far the step is from the same step in float32.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import deterministic_split_lora_amd as dsl  # noqa: E402

SPLIT_K = 4
EPS = 1e-5


class Mx4Weight:
    """A weight [N, K], quantised once, and the values it then stands for."""

    def __init__(self, w: torch.Tensor):
        N, K = w.shape
        self.q = torch.empty(N, K // 2, dtype=torch.uint8, device=w.device)
        self.scales = torch.empty(N, (K // 32 + 3) // 4 * 4, dtype=torch.uint8, device=w.device)
        self.values = torch.empty_like(w)
        dsl.lora_mx4_quantize(w, self.q, self.scales)
        dsl.lora_mx4_dequantize(self.q, self.scales, self.values)

    def __call__(self, x, y, workspace):
        dsl.lora_mx4_linear(x, self.q, self.scales, y, SPLIT_K, workspace)


def make_model(layers, hidden, vocab, adapters, rank, gen):
    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

    model = {"layers": [], "head": Mx4Weight(normal(vocab, hidden, std=1.0 / math.sqrt(hidden))),
             "final_norm": 1.0 + normal(hidden, std=0.1)}
    for _ in range(layers):
        model["layers"].append({
            "w": Mx4Weight(normal(hidden, hidden, std=1.0 / math.sqrt(hidden))),
            "A": [normal(rank, hidden, std=1.0 / math.sqrt(hidden)) for _ in range(adapters)],
            "B": [normal(hidden, rank, std=1.0 / math.sqrt(rank)) for _ in range(adapters)],
            "post": 1.0 + normal(hidden, std=0.1), "pre": 1.0 + normal(hidden, std=0.1),
            "gate": normal(1, hidden, std=0.5)})
    return model


def step(model, r, ids, rank, u, settings):
    """Hidden states r [M, hidden] and adapter ids to (tokens, log-probabilities, logits, hidden states)."""
    M, hidden = r.shape
    layers, adapters = model["layers"], len(model["layers"][0]["A"])
    vocab = model["head"].q.shape[0]
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    plan = torch.empty(dsl.lora_sgmv_plan_bytes(M), dtype=torch.uint8, device="cuda")
    dsl.lora_sgmv_plan(ids, adapters, plan)                    # once for all layers
    ranks = torch.full((adapters,), rank, dtype=torch.int32, device="cuda")
    lora_ws = torch.empty(dsl.lora_sgmv_workspace_bytes(M, rank, SPLIT_K), dtype=torch.uint8, device="cuda")
    need = max(dsl.lora_mx4_linear_workspace_bytes(M, hidden, n, SPLIT_K) for n in (hidden, vocab))
    base_ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None

    x, y, r = torch.empty(M, hidden, **bf16), torch.empty(M, hidden, **bf16), r.clone()
    logits = torch.empty(M, vocab, **bf16)
    dsl.lora_block_norm(r, r, pre="rms", pre_w=layers[0]["pre"], x_out=x, eps=EPS)     # before the first layer
    for i, layer in enumerate(layers):
        layer["w"](x, y, base_ws)
        pointers = [torch.tensor([t.data_ptr() for t in layer[n]], dtype=torch.int64, device="cuda") for n in "AB"]
        dsl.lora_sgmv_shrink_expand(x, pointers[0], hidden, pointers[1], ranks, None, None, ids, adapters, plan, y,
                                    rank, SPLIT_K, lora_ws)
        nxt = layers[i + 1]["pre"] if i + 1 < len(layers) else model["final_norm"]
        dsl.lora_block_norm(r, r, y=y, post="rms", post_w=layer["post"], gate=layer["gate"], res_scale=0.9, pre="rms",
                            pre_w=nxt, x_out=x, eps=EPS)
    model["head"](x, logits, base_ws)
    tokens = torch.empty(M, dtype=torch.int32, device="cuda")
    logprobs = torch.empty(M, dtype=torch.float32, device="cuda")
    dsl.lora_sample(logits, u, tokens, logprobs=logprobs, **settings)
    return tokens, logprobs, logits, r


def reference(model, r, ids):
    """The logits in float32, with the same quantised weights."""
    def rms(v, w):
        return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w.float()

    r = r.float()
    layers = model["layers"]
    x = rms(r, layers[0]["pre"])
    for i, layer in enumerate(layers):
        y = x @ layer["w"].values.float().t()
        for a in range(len(layer["A"])):
            rows = (ids == a).unsqueeze(-1)
            y = y + rows * ((x @ layer["A"][a].float().t()) @ layer["B"][a].float().t())
        r = 0.9 * r + layer["gate"].float() * rms(y, layer["post"])
        x = rms(r, layers[i + 1]["pre"] if i + 1 < len(layers) else model["final_norm"])
    return x @ model["head"].values.float().t()


def drawn_by(logits, u, settings):
    """The tokens that the definition draws from given logits (double precision)."""
    out = []
    for i, l in enumerate(logits.double()):
        T, k, p = (float(settings[n][i]) for n in ("temperature", "top_k", "top_p"))
        if T <= 0:
            out.append(int(l.argmax()))
            continue
        w = torch.exp((l - l.max()) / T)
        order = torch.argsort(l, descending=True, stable=True)
        order = order[:int(k)] if k > 0 else order
        c = torch.cumsum(w[order], 0)
        kept = order[(c - w[order]) < p * c[-1]].sort().values if p < 1 else order.sort().values
        c = torch.cumsum(w[kept], 0)
        out.append(int(kept[min(int((c <= float(u[i]) * c[-1]).sum()), kept.numel() - 1)]))
    return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=8000)
    ap.add_argument("--adapters", type=int, default=3)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(0)
    rank, M = 16, a.tokens
    model = make_model(a.layers, a.hidden, a.vocab, a.adapters, rank, gen)
    r = torch.randn(M, a.hidden, generator=gen, device="cuda").to(torch.bfloat16)
    ids = (torch.arange(M, device="cuda") % (a.adapters + 1) - 1).to(torch.int32)      # -1: no adapter
    u = torch.rand(M, generator=gen, device="cuda")
    settings = {"temperature": torch.linspace(0.0, 1.2, M, device="cuda"),
                "top_k": 20 * (torch.arange(M, device="cuda", dtype=torch.int32) % 3),
                "top_p": torch.full((M,), 0.9, device="cuda")}
    tokens, logprobs, logits, _ = step(model, r, ids, rank, u, settings)
    again = step(model, r, ids, rank, u, settings)
    alone = step(model, r[:1], ids[:1], rank, u[:1], {k: v[:1] for k, v in settings.items()})
    torch.cuda.synchronize()
    assert torch.equal(again[2], logits) and torch.equal(again[0], tokens), "two runs differ"
    assert torch.equal(alone[2], logits[:1]), "a token's logits depend on its batch"
    want = reference(model, r, ids)
    worst = float((logits.float() - want).abs().max() / want.square().mean().sqrt())
    report = {"tokens": tokens.tolist(), "reference_tokens": drawn_by(logits.cpu(), u.cpu(), settings), "worst": worst}
    print("tokens        ", report["tokens"])
    print("log-probability", ["%.3f" % v for v in logprobs.tolist()])
    print("largest difference of a logit from float32, in units of the logits' size: %.4f" % worst)
    return report


if __name__ == "__main__":
    main()
