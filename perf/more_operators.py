"""What the attention of an adapted step, and its drafted tokens, are measured on.

Between the fused QKV product and the output product a step appends its keys and values to a paged cache (with the norms
of queries and keys and the position rotation on the way) and attends over that cache.  The cache holds 8 bits a value
(E4M3) with a power-of-two scale for every block of 16 tokens and head.  After the last layer, tokens that a draft
proposed are verified against the model's own probabilities.

Where ``own`` is false everything is computed in its plain form: elementary torch operations in 32 bits (64 where a sum
decides how a value is rounded), rounded once at the end.  Where it is true the library's entry points are called.
"""
import math

import torch

own = False

BLOCK = 16                                                    # tokens that share a scale
E4M3_MAX = 448.0
MIN_EXPONENT = -100                                           # of a scale
ONE = 2147483648.0                                            # fixed-point weight of a row's largest logit (2^31)
UNIT = 1099511627776.0                                        # fixed-point probability of 1 (2^40)
EPS = 1e-6


# ----------------------------------------------------------------------------
# the cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one user's decode step: all latency
        {"name": "append_decode_1", "op": "append", "seqs": 1, "new": 1, "context": 517, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 64, "norm": False, "pairs": False},
        # an odd serving batch, every sequence at another length, queries and keys normed
        {"name": "append_decode_251", "op": "append", "seqs": 251, "new": 1, "context": 300, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 32, "norm": True, "pairs": False},
        # three prompts of different lengths, each begun by an earlier chunk
        {"name": "append_prefill", "op": "append", "seqs": 3, "new": 4099, "context": 4200, "Hq": 64, "Hkv": 8,
         "D": 128, "page": 64, "norm": True, "pairs": True},
        # one user's decode step in a short context: all latency
        {"name": "attend_decode_1", "op": "attend", "seqs": 1, "new": 1, "context": 1025, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "window": 0},
        # the same user far into a document: the work of one sequence over the whole chip
        {"name": "attend_decode_1_long", "op": "attend", "seqs": 1, "new": 1, "context": 131071, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "window": 0},
        # a serving batch, every sequence at another length: the cache's bytes
        {"name": "attend_decode_61", "op": "attend", "seqs": 61, "new": 1, "context": 16384, "Hq": 64, "Hkv": 8,
         "D": 128, "page": 32, "window": 0},
        # drafted tokens of a batch, verified together, small heads, a layer that looks back a limited way
        {"name": "attend_draft_32", "op": "attend", "seqs": 32, "new": 5, "context": 6000, "Hq": 32, "Hkv": 8,
         "D": 64, "page": 16, "window": 4096},
        # a chunk of a long prompt against what came before
        {"name": "attend_chunk", "op": "attend", "seqs": 1, "new": 512, "context": 32768, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "window": 0},
        # whole prompts, ragged: the largest in operations
        {"name": "attend_prefill", "op": "attend", "seqs": 2, "new": 8191, "context": 8191, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "window": 0},
        # one user's drafts from a lookup table (no draft probabilities), small vocabulary
        {"name": "verify_1", "op": "verify", "seqs": 1, "drafts": 4, "V": 32000, "dtype": "bf16", "draft": False},
        # a serving batch with a draft model, large odd vocabulary, each request with its own settings
        {"name": "verify_32", "op": "verify", "seqs": 32, "drafts": 4, "V": 128259, "dtype": "fp32", "draft": True},
        # a batch with drafts from lookup tables, no cuts asked for by most
        {"name": "verify_64", "op": "verify", "seqs": 64, "drafts": 3, "V": 50257, "dtype": "bf16", "draft": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "append", "attend", "attend", "attend", "attend", "verify", "verify"))
    if op == "verify":
        V, n = _log_int(rng, 1000, 160000), rng.randint(1, 8)
        draft = rng.random() < 0.5
        return {"op": op, "seqs": max(1, min(_log_int(rng, 1, 64), 32_000_000 // (V * (2 * n + 1)))), "drafts": n,
                "V": V, "dtype": rng.choice(("bf16", "fp32")), "draft": draft}
    D = rng.choice((64, 128, 128, 256))
    Hkv = rng.choice((1, 2, 4, 8))
    Hq = Hkv * rng.choice((1, 2, 4, 5, 7, 8))
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        seqs = _log_int(rng, 1, 200)
        new = _log_int(rng, 1, max(1, min(4000, 6000 // seqs))) if rng.random() < 0.5 else rng.randint(1, 4)
        return {"op": op, "seqs": seqs, "new": new, "context": new + rng.randint(0, 300), "Hq": Hq, "Hkv": Hkv,
                "D": D, "page": page, "norm": rng.random() < 0.5, "pairs": rng.random() < 0.5}
    kind = rng.choice(("decode", "decode", "draft", "chunk"))
    window = rng.choice((0, 0, 0, _log_int(rng, 100, 5000)))
    if kind == "chunk":
        new = _log_int(rng, 17, 4000)
        context = new + rng.choice((0, _log_int(rng, 1, 16000)))
        seqs = max(1, min(rng.randint(1, 4), 60_000_000 // (new * context)))
    else:
        new = 1 if kind == "decode" else rng.randint(2, 8)
        context = new + _log_int(rng, 1, 60000)
        seqs = max(1, min(_log_int(rng, 1, 200), 300_000_000 // (context * Hkv * D)))
    return {"op": op, "seqs": seqs, "new": new, "context": context, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
            "window": window}


def _lengths(case):
    """(new tokens, tokens with them) of every sequence: the first is the longest, the others fall off."""
    out = []
    for b in range(case["seqs"]):
        f = 1.0 - 0.75 * b / case["seqs"]
        new = max(1, int(case["new"] * f))
        out.append((new, max(new, int(case["context"] * f))))
    return out


def work(case):
    if case["op"] == "verify":
        rows = case["seqs"] * (case["drafts"] * (2 if case["draft"] else 1) + 1)
        return {"bytes": rows * case["V"] * (2 if case["dtype"] == "bf16" else 4), "flops": 0}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    T = sum(n for n, _ in _lengths(case))
    if case["op"] == "append":
        return {"bytes": T * D * (2 * (Hq + 2 * Hkv) + 2 * Hq + 2 * Hkv) + T * D * 4, "flops": 0}
    pairs, keys = 0, 0
    for new, n in _lengths(case):
        w = case["window"] or n
        first = n - new                                        # position of the first query
        full = max(0, min(n, w - 1) - first)                   # queries whose window reaches past the start
        pairs += full * first + full * (full + 1) // 2 + (new - full) * w
        keys += min(n, new - 1 + w)
    return {"bytes": 2 * Hkv * D * keys + keys // BLOCK * 2 * Hkv + 4 * T * Hq * D, "flops": 4 * Hq * D * pairs}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _normal(gen, *shape, dtype=torch.bfloat16, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def _fill_cache(s, gen):
    """A pool of pages whose blocks hold values as an earlier step left them: keys with a few large channels."""
    n, H, P, D = s["n_pages"], s["Hkv"], s["page"], s["D"]
    large = torch.exp(0.4 * torch.randn(D, generator=gen, device="cuda"))
    large[torch.randint(0, D, (max(1, D // 32),), generator=gen, device="cuda")] *= 4.0
    k = torch.empty(n, H, P // BLOCK, BLOCK, D, dtype=torch.uint8, device="cuda")
    v = torch.empty(n, H, P // BLOCK, D, BLOCK, dtype=torch.uint8, device="cuda")
    ks = torch.empty(n, H, P // BLOCK, dtype=torch.uint8, device="cuda")
    vs = torch.empty(n, H, P // BLOCK, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (H * P * D))
    for a in range(0, n, step):
        m = min(step, n - a)
        for codes, scales, c in ((k, ks, large), (v, vs, large.new_ones(D, 1))):
            x = torch.randn(m, *codes.shape[1:], generator=gen, device="cuda") * c
            e = _exponent(x.abs().amax((-1, -2)))
            codes[a:a + m] = _encode(x, e[..., None, None]).view(torch.uint8)
            scales[a:a + m] = e + 127
    s["k"], s["v"] = k.view(n, H, P, D), v
    s["k_scales"], s["v_scales"] = ks, vs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "verify":
        return _prepare_verify(s, gen)
    lengths = _lengths(case)
    Hq, Hkv, D, P = case["Hq"], case["Hkv"], case["D"], case["page"]
    s["lengths"], T = lengths, sum(n for n, _ in lengths)
    # what a scheduler hands over: which pages a sequence has, its length, where its new tokens lie in the batch
    pages = [(n + P - 1) // P for _, n in lengths]
    s["n_pages"] = sum(pages) + 3
    order = torch.randperm(s["n_pages"], generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s["seq_lens"] = torch.tensor([n for _, n in lengths], dtype=torch.int32, device="cuda")
    starts = [0]
    for new, _ in lengths:
        starts.append(starts[-1] + new)
    s["starts"] = starts
    s["cu_tokens"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["max_new"], s["max_len"] = max(n for n, _ in lengths), max(n for _, n in lengths)
    _fill_cache(s, gen)
    if case["op"] == "attend":
        # logits of a spread of about 1.5 to 2 at a scale of 1 / sqrt(D)
        s["q"] = _normal(gen, T, Hq, D)
        s["out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(T, Hq, dtype=torch.float32, device="cuda")
        return s
    s["qkv"] = _normal(gen, T, Hq + 2 * Hkv, D, scale=1.5)     # the fused projection's output
    s["q_norm"] = 1.0 + _normal(gen, D, scale=0.25) if case["norm"] else None
    s["k_norm"] = 1.0 + _normal(gen, D, scale=0.25) if case["norm"] else None
    position = torch.arange(s["max_len"], device="cuda", dtype=torch.float64)
    angle = position[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    s["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float()
    s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    # for the plain form: of every new token its position, its block of the pool and its place in it; of every block
    # that is written, the tokens of it that are there already
    device, blocks, kept = "cuda", {}, []
    pos, block = [], []
    pages_of = table.tolist()
    for b, (new, n) in enumerate(lengths):
        for p in range(n - new, n):
            key = pages_of[b][p // P] * (P // BLOCK) + p % P // BLOCK
            if key not in blocks:
                blocks[key] = len(kept)
                kept.append(p % BLOCK)
            pos.append(p)
            block.append(blocks[key])
    s["pos"] = torch.tensor(pos, device=device)
    s["block"] = torch.tensor(block, device=device)
    s["blocks"] = torch.tensor(list(blocks), device=device)
    s["kept"] = torch.tensor(kept, device=device)
    return s


def _prepare_verify(s, gen):
    B, n, V = s["seqs"], s["drafts"], s["V"]
    dt = torch.bfloat16 if s["dtype"] == "bf16" else torch.float32
    rand = lambda *shape: torch.rand(*shape, generator=gen, device="cuda")  # noqa: E731
    base = _normal(gen, B * (n + 1), V, dtype=torch.float32, scale=2.5)
    s["target"] = base.to(dt)
    # the draft model is nearly right; its tokens come from the head of its distribution
    near = (base.view(B, n + 1, V)[:, :n].reshape(B * n, V) + _normal(gen, B * n, V, dtype=torch.float32, scale=0.7)).to(dt)
    top, ids = near.float().topk(min(V, 20), dim=-1)
    pick = (top - torch.log(-torch.log(rand(*top.shape).clamp(1e-6, 1 - 1e-6)))).argmax(-1, keepdim=True)
    s["drafted"] = ids.gather(-1, pick).view(B, n).to(torch.int32)
    s["near"] = near if s["draft"] else None
    # requests differ: greedy ones, some with top-k, some with top-p, some with min-p, some with none of them
    s["temperature"] = torch.where(rand(B) < 0.1, torch.zeros(B, device="cuda"), 0.5 + rand(B))
    k = torch.randint(20, 200, (B,), generator=gen, device="cuda", dtype=torch.int32)
    s["top_k"] = torch.where(rand(B) < 0.4, k, torch.zeros_like(k))
    s["top_p"] = torch.where(rand(B) < 0.5, 0.7 + 0.29 * rand(B), torch.ones(B, device="cuda"))
    s["min_p"] = torch.where(rand(B) < 0.3, 0.05 * rand(B), torch.zeros(B, device="cuda"))
    s["u"] = rand(B, n + 1)
    s["tokens"] = torch.empty(B, n + 1, dtype=torch.int32, device="cuda")
    s["accepted"] = torch.empty(B, dtype=torch.int32, device="cuda")
    s["logprobs"] = torch.empty(B, n + 1, dtype=torch.float32, device="cuda")
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import deterministic_split_lora_amd as dsl
    if s["op"] == "verify":
        if "workspace" not in s:
            need = dsl.lora_verify_workspace_bytes(s["seqs"], s["drafts"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        dsl.lora_verify(s["target"], s["drafted"], s["u"], s["tokens"], s["accepted"], s["workspace"],
                        draft_logits=s["near"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                        min_p=s["min_p"], logprobs=s["logprobs"])
        return {"tokens": s["tokens"], "accepted": s["accepted"], "logprobs": s["logprobs"]}
    if "cache" not in s:
        s["cache"] = dsl.KvCache(s["k"], s["v"], s["k_scales"], s["v_scales"], s["table"], s["seq_lens"], s["cu_tokens"])
    Hq, Hkv = s["Hq"], s["Hkv"]
    if s["op"] == "append":
        qkv = s["qkv"]
        dsl.lora_kv_append(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], s["cache"], q=qkv[:, :Hq], q_out=s["q_out"],
                           q_norm=s["q_norm"], k_norm=s["k_norm"], rope=s["rope"], pairs=s["pairs"], eps=EPS)
        return _appended(s)
    if "workspace" not in s:
        need = dsl.lora_kv_attention_workspace_bytes(s["q"].shape[0], Hq, Hkv, s["D"], s["max_new"], s["max_len"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    dsl.lora_kv_attention(s["q"], s["cache"], s["out"], max_new=s["max_new"], max_len=s["max_len"],
                          window=s["window"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _appended(s):
    codes, scales = torch.float8_e4m3fn, torch.float8_e8m0fnu
    return {"q": s["q_out"], "k": s["k"].view(codes), "v": s["v"].view(codes), "k_scales": s["k_scales"].view(scales),
            "v_scales": s["v_scales"].view(scales)}


# ---- the cache's numbers ----
def _power(e):
    """2^e for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The least e >= MIN_EXPONENT with amax 2^-e <= 448 = 1.75 2^8, for finite amax >= 0."""
    bits = amax.view(torch.int32)
    e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    return e.clamp_(min=MIN_EXPONENT)


def _encode(x, e):
    return (x * _power(-e)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


# ---- append ----
def _rotate(x, cos, sin, pairs):
    h = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :h], x[..., h:])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    return torch.stack((lo, hi), -1).flatten(-2) if pairs else torch.cat((lo, hi), -1)


def _head_norm(x, w):
    x = x.float()
    if w is None:
        return x
    mean = ((x.double() * x.double()).sum(-1, keepdim=True) / x.shape[-1]).float()
    return x * (1.0 / torch.sqrt(mean + EPS)) * w.float()


def _append_plain(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    rows = s["rope"][s["pos"]]
    cos, sin = rows[:, None, :D // 2], rows[:, None, D // 2:]
    qkv = s["qkv"]
    s["q_out"].copy_(_rotate(_head_norm(qkv[:, :Hq], s["q_norm"]), cos, sin, s["pairs"]))
    k = _rotate(_head_norm(qkv[:, Hq:Hq + Hkv], s["k_norm"]), cos, sin, s["pairs"])
    v = qkv[:, Hq + Hkv:].float()
    per = s["page"] // BLOCK
    page, within = s["blocks"] // per, s["blocks"] % per       # of the blocks that are written
    place = s["pos"] % BLOCK
    for x, codes, scales, by_token in ((k, s["k"].view(-1, Hkv, per, BLOCK, D), s["k_scales"], True),
                                       (v, s["v"], s["v_scales"], False)):
        amax = torch.zeros(len(s["blocks"]), Hkv, device=x.device)
        amax.scatter_reduce_(0, s["block"][:, None].expand(-1, Hkv), x.abs().amax(-1), "amax")
        e = _exponent(amax)
        old = scales[page, :, within].to(torch.int32) - 127
        live = (s["kept"] > 0)[:, None]
        e = torch.where(live, torch.maximum(e, old), e)
        c = codes[page, :, within]                             # [blocks, Hkv, 16, D] or [blocks, Hkv, D, 16]
        c = c if by_token else c.transpose(-1, -2)
        again = _encode(c.view(torch.float8_e4m3fn).float(), (e - old)[..., None, None].clamp(0, 120)).view(torch.uint8)
        earlier = (torch.arange(BLOCK, device=x.device) < s["kept"][:, None])[:, None, :, None]
        c = torch.where(earlier, again, c)
        c[s["block"], :, place] = _encode(x, e[s["block"]][..., None]).view(torch.uint8)
        codes[page, :, within] = c if by_token else c.transpose(-1, -2)
        scales[page, :, within] = (e + 127).to(torch.uint8)
    return _appended(s)


# ---- attention ----
def _sequence(s, b):
    """Keys and values [Hkv, len, D] of a sequence, in 32 bits."""
    P, D, Hkv, n = s["page"], s["D"], s["Hkv"], s["lengths"][b][1]
    pages = s["table"][b, :(n + P - 1) // P].long()
    k = s["k"][pages].view(torch.float8_e4m3fn).float().view(-1, Hkv, P // BLOCK, BLOCK, D)
    k = k * _power(s["k_scales"][pages].to(torch.int32) - 127)[..., None, None]
    v = s["v"][pages].view(torch.float8_e4m3fn).float().transpose(-1, -2)
    v = v * _power(s["v_scales"][pages].to(torch.int32) - 127)[..., None, None]
    return tuple(t.transpose(0, 1).reshape(Hkv, -1, D)[:, :n] for t in (k, v))


def _attend_plain(s):
    Hkv, D, w = s["Hkv"], s["D"], s["window"]
    G = s["Hq"] // Hkv
    for b, (new, n) in enumerate(s["lengths"]):
        k, v = _sequence(s, b)
        kt = k.transpose(1, 2).contiguous()
        step = max(1, (1 << 28) // (n * G * Hkv))
        for a in range(0, new, step):
            m = min(step, new - a)
            t = s["starts"][b] + a
            q = s["q"][t:t + m].float().view(m, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, m * G, D)
            l = (q @ kt).mul_(1.0 / math.sqrt(D)).view(Hkv, m, G, n)
            p = torch.arange(n - new + a, n - new + a + m, device=l.device)[:, None]
            j = torch.arange(n, device=l.device)[None, :]
            out = (j > p) | (j <= p - w) if w else j > p
            l.masked_fill_(out[None, :, None, :], -math.inf)
            top = l.amax(-1, keepdim=True)
            l.sub_(top).exp_()
            total = l.sum(-1, keepdim=True)
            o = (l.view(Hkv, m * G, n) @ v).view(Hkv, m, G, D) / total
            s["out"][t:t + m].view(m, Hkv, G, D).copy_(o.permute(1, 0, 2, 3))
            s["lse"][t:t + m].view(m, Hkv, G).copy_((top + total.log()).squeeze(-1).permute(1, 0, 2))
    return {"out": s["out"], "lse": s["lse"]}


# ---- verification ----
def _weights(logits, T, top_k, top_p, min_p):
    """Whole-number weights of the kept tokens of every row, in the vocabulary's order, and their sums."""
    order_l, order = torch.sort(logits.float(), dim=-1, descending=True, stable=True)
    B, V = order_l.shape
    T, k, p = T.unsqueeze(-1), top_k.unsqueeze(-1), top_p.unsqueeze(-1)
    greedy = T <= 0
    z = (order_l - order_l[:, :1]) * (1.0 / torch.where(greedy, torch.ones_like(T), T))
    w = torch.round(torch.exp(z) * ONE).to(torch.int64)
    rank = torch.arange(V, device=w.device).expand(B, V)
    keep = (rank < torch.where(k <= 0, V, k)) & (~greedy | (rank == 0))
    w = w * keep
    before = torch.cumsum(w, -1) - w
    mass = torch.ceil(p.double() * w.sum(-1, keepdim=True).double()).to(torch.int64).clamp(min=1)
    keep = keep & ((p >= 1) | (before < mass))
    floor = torch.ceil(min_p.double().clamp(0, 1) * ONE).to(torch.int64).unsqueeze(-1)
    w = w * (keep & (greedy | (w >= floor)))
    w = torch.zeros_like(w).scatter_(-1, order, w)
    return w, w.sum(-1, keepdim=True)


def _verify_plain(s):
    B, n, V = s["seqs"], s["drafts"], s["V"]
    per = lambda t, m: t.repeat_interleave(m)  # noqa: E731
    cuts = (s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    w, W = _weights(s["target"], *(per(t, n + 1) for t in cuts))
    P = torch.round(w.double() / W.double() * UNIT).view(B, n + 1, V)
    x = s["drafted"].long()
    if s["near"] is not None:
        v, U = _weights(s["near"], *(per(t, n) for t in cuts))
        Q = torch.round(v.double() / U.double() * UNIT).view(B, n, V)
    else:
        Q = torch.zeros(B, n, V, dtype=torch.float64, device=w.device).scatter_(-1, x.unsqueeze(-1), UNIT)
    u = s["u"].double()
    px, qx = P[:, :n].gather(-1, x.unsqueeze(-1)).squeeze(-1), Q.gather(-1, x.unsqueeze(-1)).squeeze(-1)
    ok = u[:, :n] * qx < px
    accepted = ok.to(torch.int64).cumprod(-1).sum(-1)
    row = torch.arange(B, device=w.device)
    w, W = w.view(B, n + 1, V), W.view(B, n + 1)
    rest = (P[row, accepted] - Q[row, accepted.clamp(max=n - 1)]).clamp(min=0).to(torch.int64)
    rest = torch.where(((accepted < n) & (rest.sum(-1) > 0)).unsqueeze(-1), rest, w[row, accepted])
    total = rest.sum(-1, keepdim=True)
    t = torch.floor(u[:, n:] * total.double()).to(torch.int64)
    token = (torch.cumsum(rest, -1) <= t).sum(-1)
    place = torch.arange(n + 1, device=w.device)[None, :]
    a = accepted.unsqueeze(-1)
    tokens = torch.where(place < a, torch.cat((x, x[:, :1]), 1), torch.where(place == a, token.unsqueeze(-1), -1))
    of = w.gather(-1, tokens.clamp(min=0).unsqueeze(-1)).squeeze(-1)
    logprobs = torch.log((of.double() / W.double()).float()).masked_fill(tokens < 0, -math.inf)
    return {"tokens": tokens.to(torch.int32), "accepted": accepted.to(torch.int32), "logprobs": logprobs}


def _run_plain(s):
    return {"append": _append_plain, "attend": _attend_plain, "verify": _verify_plain}[s["op"]](s)


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def _exact_e4m3(v):
    """Nearest value with four significant bits, an exponent of at least -6, ties to even, at most 448."""
    _, ex = torch.frexp(v)                                     # |v| = m 2^ex with m in [1/2, 1)
    unit = torch.exp2((ex - 4).clamp(min=-9).double())
    return (torch.round(v / unit) * unit).clamp(-448.0, 448.0)


def _exact_append(s):
    Hq, Hkv, D, P = s["Hq"], s["Hkv"], s["D"], s["page"]
    position = torch.cat([torch.arange(n - new, n) for new, n in s["lengths"]]).cuda()
    x = s["qkv"].double()
    for heads, weight in ((slice(0, Hq), s["q_norm"]), (slice(Hq, Hq + Hkv), s["k_norm"])):
        if weight is not None:
            part = x[:, heads]
            x[:, heads] = part / torch.sqrt(part.square().mean(-1, keepdim=True) + EPS) * weight.double()
    table = s["rope"].double()[position]
    turn = torch.complex(table[:, :D // 2], table[:, D // 2:]).unsqueeze(1)
    part = x[:, :Hq + Hkv]
    if s["pairs"]:
        z = torch.complex(part[..., 0::2].contiguous(), part[..., 1::2].contiguous()) * turn
        x[:, :Hq + Hkv] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(part[..., :D // 2].contiguous(), part[..., D // 2:].contiguous()) * turn
        x[:, :Hq + Hkv] = torch.cat((z.real, z.imag), -1)
    out = {"q": x[:, :Hq].clone()}
    tables = s["table"].tolist()
    for name, values in (("k", x[:, Hq:Hq + Hkv]), ("v", x[:, Hq + Hkv:])):
        codes = s[name].view(torch.float8_e4m3fn).double()
        codes = codes.view(-1, Hkv, P // BLOCK, BLOCK, D) if name == "k" else codes.transpose(-1, -2).contiguous()
        scale = torch.exp2(s[name + "_scales"].double() - 127)
        for b, (new, n) in enumerate(s["lengths"]):            # block by block of every sequence
            p = n - new
            while p < n:
                end = min(n, (p // BLOCK + 1) * BLOCK)
                page, block, first = tables[b][p // P], p % P // BLOCK, p % BLOCK
                t = s["starts"][b] + p - (n - new)
                fresh = values[t:t + end - p].transpose(0, 1)  # [Hkv, tokens, D]
                need = torch.exp2(torch.ceil(torch.log2(fresh.abs().amax((1, 2)) / 448.0)).clamp(min=MIN_EXPONENT))
                had = scale[page, :, block]
                to = torch.maximum(need, had) if first else need
                target = codes[page, :, block]
                target[:, :first] = _exact_e4m3(target[:, :first] * (had / to)[:, None, None])
                target[:, first:first + end - p] = _exact_e4m3(fresh / to[:, None, None])
                scale[page, :, block] = to
                p = end
        out[name] = codes.view(s[name].shape) if name == "k" else codes.transpose(-1, -2).contiguous()
        out[name + "_scales"] = scale
    return out


def _exact_attend(s):
    D, P, Hkv = s["D"], s["page"], s["Hkv"]
    G = s["Hq"] // Hkv
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    for b, (new, n) in enumerate(s["lengths"]):
        at = torch.arange(n, device="cuda")
        page, slot = s["table"][b].long()[at // P], at % P
        for h in range(Hkv):
            scale = torch.exp2(s["k_scales"][page, h, slot // BLOCK].double() - 127).unsqueeze(-1)
            k = s["k"][page, h, slot].view(torch.float8_e4m3fn).double() * scale
            scale = torch.exp2(s["v_scales"][page, h, slot // BLOCK].double() - 127).unsqueeze(-1)
            v = s["v"][page, h, slot // BLOCK, :, slot % BLOCK].view(torch.float8_e4m3fn).double() * scale
            for g in range(G):
                head = h * G + g
                for a in range(0, new, 4096):
                    t0, m = s["starts"][b] + a, min(4096, new - a)
                    logits = torch.matmul(s["q"][t0:t0 + m, head].double(), k.t()) / D ** 0.5
                    past = (n - new + a + torch.arange(m, device="cuda")).unsqueeze(-1) - at
                    seen = past >= 0
                    if s["window"]:
                        seen &= past < s["window"]
                    logits = torch.where(seen, logits, torch.full_like(logits, -math.inf))
                    z = torch.logsumexp(logits, -1)
                    lse[t0:t0 + m, head] = z
                    out[t0:t0 + m, head] = torch.exp(logits - z.unsqueeze(-1)) @ v
    return {"out": out, "lse": lse}


def _exact_distribution(l, T, k, p, m):
    """Probabilities of one row in 64 bits, from the definition."""
    q = torch.zeros_like(l)
    if T <= 0:
        q[(l == l.max()).nonzero()[0]] = 1.0
        return q
    e = torch.exp((l - l.max()) / T)
    order = torch.argsort(l, descending=True, stable=True)
    order = order[:k] if k > 0 else order
    if p < 1:
        c = torch.cumsum(e[order], 0)
        order = order[(c - e[order]) < p * c[-1]]
    order = order[e[order] >= m]
    q[order] = e[order] / e[order].sum()
    return q


def _exact_verify(s):
    B, n = s["seqs"], s["drafts"]
    logprobs = torch.full((B, n + 1), -math.inf, dtype=torch.float64)
    settings = [s[name].tolist() for name in ("temperature", "top_k", "top_p", "min_p")]
    u, drafted = s["u"].double().tolist(), s["drafted"].tolist()
    for i in range(B):                                         # one request at a time
        cuts = [c[i] for c in settings]
        for j in range(n + 1):
            p = _exact_distribution(s["target"][i * (n + 1) + j].double(), *cuts)
            rest = p
            if j < n:
                x = drafted[i][j]
                if s["near"] is not None:
                    q = _exact_distribution(s["near"][i * n + j].double(), *cuts)
                else:
                    q = torch.zeros_like(p)
                    q[x] = 1.0
                if u[i][j] * float(q[x]) < float(p[x]):
                    logprobs[i, j] = math.log(float(p[x]))
                    continue
                rest = (p - q).clamp(min=0.0)
            c = torch.cumsum(rest, 0)
            token = min(int((c <= u[i][n] * c[-1]).sum()), c.numel() - 1)
            logprobs[i, j] = torch.log(p[token])
            break
    return {"tokens": None, "accepted": None, "logprobs": logprobs}


def exact(case, seed):
    return {"append": _exact_append, "attend": _exact_attend, "verify": _exact_verify}[case["op"]](prepare(case, seed))
