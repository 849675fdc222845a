"""What the operators of one adapted decode or prefill step are measured on.

A program that serves LoRA adapters calls, besides the adapters' shrink and expand: the frozen base layer's product with
weights held in microscaled 4 bits (MX4: E2M1 elements, one power-of-two scale for 32 of them along the reduced
dimension), the norm / gate / residual step between two blocks, and the draw of the next token.

Where ``own`` is false everything is computed in its plain form: elementary torch operations in 32 bits, rounded once at
the end.  Where it is true the library's entry points are called.
"""
import math

import torch

own = False

BLOCK = 32                                                    # elements of one MX4 scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)               # values of the codes 0..7; bit 3 is the sign
ONE = 2147483648.0                                            # fixed-point weight of a row's largest logit (2^31)
EPS = 1e-5


# ----------------------------------------------------------------------------
# the cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # activations of a decode batch, quantised before an MX4 x MX4 product: all latency
        {"name": "quantize_32", "op": "quantize", "M": 32, "K": 4096},
        # a checkpoint's MLP weight, quantised when it is loaded, its row count ragged as after a vocabulary-sized split
        {"name": "quantize_weight", "op": "quantize", "M": 4099, "K": 14336},
        # one user's decode step through the fused QKV projection: the smallest product
        {"name": "linear_decode_1", "op": "linear", "M": 1, "K": 4096, "N": 6144, "split_k": 8},
        # decode batch one past a full tile, MLP down projection: long reduction
        {"name": "linear_decode_33", "op": "linear", "M": 33, "K": 14336, "N": 4096, "split_k": 8},
        # a short prompt, neither tile-aligned rows nor enough of them to fill the chip
        {"name": "linear_prompt_200", "op": "linear", "M": 200, "K": 4096, "N": 6144, "split_k": 4},
        # chunked prefill through the MLP up projection
        {"name": "linear_prefill", "op": "linear", "M": 4096, "K": 4096, "N": 14336, "split_k": 1},
        # decode batch with activations in 4 bits too (quantised within the call)
        {"name": "linear_q_decode_16", "op": "linear_q", "M": 16, "K": 8192, "N": 8192, "split_k": 8},
        # prefill of a wide layer with both operands in 4 bits: the largest matrix product
        {"name": "linear_q_prefill", "op": "linear_q", "M": 4096, "K": 8192, "N": 28672, "split_k": 1},
        # one token between two blocks: post-norm, channel gate, scaled residual, pre-norm
        {"name": "norm_1", "op": "norm", "M": 1, "C": 8192, "post": "rms", "pre": "rms", "gate": "channel"},
        # a prefill chunk with a gate for every token
        {"name": "norm_prefill", "op": "norm", "M": 4096, "C": 8192, "post": "rms", "pre": "rms", "gate": "token"},
        # one user's next token from a small vocabulary
        {"name": "sample_1", "op": "sample", "B": 1, "V": 32000, "dtype": "bf16"},
        # a full serving batch, large odd vocabulary, each row with its own settings
        {"name": "sample_256", "op": "sample", "B": 256, "V": 128259, "dtype": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "linear", "linear", "linear_q", "linear_q", "norm", "norm", "sample", "sample"))
    if op == "quantize":
        K = 32 * _log_int(rng, 8, 512)
        return {"op": op, "M": min(_log_int(rng, 1, 16384), 60_000_000 // K), "K": K}
    if op in ("linear", "linear_q"):
        M = _log_int(rng, 1, 4096)
        S = rng.choice((4, 8, 16) if M <= 64 else (1, 2, 4, 8))
        return {"op": op, "M": M, "K": 32 * S * max(1, _log_int(rng, 512, 14336 if M < 1024 else 8192) // (32 * S)),
                "N": 8 * _log_int(rng, 64, 3584 if M < 1024 else 1792), "split_k": S}
    if op == "norm":
        C = 8 * _log_int(rng, 32, 2048)
        return {"op": op, "M": min(_log_int(rng, 1, 16384), 33_000_000 // C), "C": C,
                "post": rng.choice(("none", "rms", "rms", "layer")), "pre": rng.choice(("rms", "rms", "layer")),
                "gate": rng.choice(("none", "channel", "token"))}
    V = _log_int(rng, 1000, 160000)
    return {"op": op, "B": min(_log_int(rng, 1, 512), 32_000_000 // V), "V": V, "dtype": rng.choice(("bf16", "fp32"))}


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": 4 * n, "flops": 0}
    if op in ("linear", "linear_q"):
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * M * K + N * K // 2 + N * K // BLOCK + 2 * M * N, "flops": 2 * M * K * N}
    if op == "norm":
        n = case["M"] * case["C"]
        gate = {"none": 0, "channel": case["C"], "token": n}[case["gate"]]
        return {"bytes": 2 * (4 * n + gate), "flops": 0}
    return {"bytes": case["B"] * case["V"] * (2 if case["dtype"] == "bf16" else 4), "flops": 0}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _normal(gen, *shape, dtype=torch.bfloat16, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def _activations(gen, M, K):
    """Hidden states: channels of different sizes, a few of them large."""
    c = torch.exp(0.5 * torch.randn(K, generator=gen, device="cuda"))
    c[torch.randint(0, K, (max(1, K // 512),), generator=gen, device="cuda")] *= 8.0
    return (torch.randn(M, K, generator=gen, device="cuda") * c).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], dict(case)
    if op == "quantize":
        M, K = case["M"], case["K"]
        s["x"] = _activations(gen, M, K)
        s["q"] = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(M, _scale_stride(K), dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    elif op in ("linear", "linear_q"):
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = _activations(gen, M, K)
        s["wq"] = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
        s["ws"] = torch.zeros(N, _scale_stride(K), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // K)
        for a in range(0, N, step):                            # a weight is quantised once, in slices of its rows
            w = _normal(gen, min(step, N - a), K, dtype=torch.float32, scale=1.0 / math.sqrt(K))
            code, e = _quantize(w)
            s["wq"][a:a + step] = code[:, 0::2] | (code[:, 1::2] << 4)
            s["ws"][a:a + step, :K // BLOCK] = e + 127
        s["y"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        if op == "linear_q":
            s["xq"] = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
            s["xs"] = torch.empty(M, _scale_stride(K), dtype=torch.uint8, device="cuda")
    elif op == "norm":
        M, C = case["M"], case["C"]
        s["y"] = _activations(gen, M, C)
        s["r"] = _normal(gen, M, C, scale=3.0)
        s["res_scale"] = 0.875
        for side in ("post", "pre"):
            kind = case[side]
            s[side + "_w"] = None if kind == "none" else 1.0 + _normal(gen, C, scale=0.25)
            s[side + "_b"] = _normal(gen, C, scale=0.25) if kind == "layer" else None
        g = case["gate"]
        s["gate"] = None if g == "none" else _normal(gen, M if g == "token" else 1, C, scale=0.5)
        s["r_out"] = torch.empty(M, C, dtype=torch.bfloat16, device="cuda")
        s["x_out"] = torch.empty(M, C, dtype=torch.bfloat16, device="cuda")
    else:
        B, V = case["B"], case["V"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["logits"] = _normal(gen, B, V, dtype=dt, scale=2.5)
        rand = lambda: torch.rand(B, generator=gen, device="cuda")  # noqa: E731
        # requests differ: greedy ones, some with top-k, some with top-p, some with min-p, some with none of them
        s["temperature"] = torch.where(rand() < 0.1, torch.zeros(B, device="cuda"), 0.5 + rand())
        k = torch.randint(1, 200, (B,), generator=gen, device="cuda", dtype=torch.int32)
        s["top_k"] = torch.where(rand() < 0.5, k, torch.zeros_like(k))
        s["top_p"] = torch.where(rand() < 0.6, 0.5 + 0.49 * rand(), torch.ones(B, device="cuda"))
        s["min_p"] = torch.where(rand() < 0.4, 0.1 * rand(), torch.zeros(B, device="cuda"))
        s["u"] = rand()
        s["tokens"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["logprobs"] = torch.empty(B, dtype=torch.float32, device="cuda")
    return s


def _scale_stride(K):
    return (K // BLOCK + 3) // 4 * 4


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import deterministic_split_lora_amd as dsl
    op = s["op"]
    if op == "quantize":
        dsl.lora_mx4_quantize(s["x"], s["q"], s["scales"])
        dsl.lora_mx4_dequantize(s["q"], s["scales"], s["out"])
        return s["out"]
    if op in ("linear", "linear_q"):
        if "workspace" not in s:
            n = dsl.lora_mx4_linear_workspace_bytes(s["M"], s["K"], s["N"], s["split_k"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        if op == "linear":
            dsl.lora_mx4_linear(s["x"], s["wq"], s["ws"], s["y"], s["split_k"], s["workspace"])
        else:
            dsl.lora_mx4_quantize(s["x"], s["xq"], s["xs"])
            dsl.lora_mx4_linear_q(s["xq"], s["xs"], s["wq"], s["ws"], s["y"], s["split_k"], s["workspace"])
        return s["y"]
    if op == "norm":
        dsl.lora_block_norm(s["r"], s["r_out"], y=s["y"], post=s["post"], post_w=s["post_w"], post_b=s["post_b"],
                            gate=s["gate"], res_scale=s["res_scale"], pre=s["pre"], pre_w=s["pre_w"],
                            pre_b=s["pre_b"], x_out=s["x_out"], eps=EPS)
        return {"r": s["r_out"], "x": s["x_out"]}
    dsl.lora_sample(s["logits"], s["u"], s["tokens"], temperature=s["temperature"], top_k=s["top_k"],
                    top_p=s["top_p"], min_p=s["min_p"], logprobs=s["logprobs"])
    return {"tokens": s["tokens"], "logprobs": s["logprobs"]}


def _quantize(x):
    """Codes (uint8, sign in bit 3) and scale exponents of x's rows, blocks of 32."""
    v = x.float().view(x.shape[0], -1, BLOCK)
    amax = v.abs().amax(-1)
    e = (((amax.view(torch.int32) >> 23) & 255) - 129).clamp_(-127, 127)
    r = v.abs() * ((127 - e) << 23).view(torch.float32).unsqueeze(-1)
    code = (r > 0.25).to(torch.uint8)                          # nearest value, ties to the even code
    code += r >= 0.75
    code += r > 1.25
    code += r >= 1.75
    code += r > 2.5
    code += r >= 3.5
    code += r > 5.0
    code |= (v < 0).to(torch.uint8) << 3
    return code.view(x.shape), e


def _values(code, e):
    """The fp32 values that codes and scale exponents stand for."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=code.device)
    v = table[code.to(torch.int32)].view(code.shape[0], -1, BLOCK)
    return (v * ((e + 127) << 23).view(torch.float32).unsqueeze(-1)).view(code.shape)


def _weight(s):
    code = torch.stack((s["wq"] & 15, s["wq"] >> 4), -1).view(s["N"], s["K"])
    return _values(code, s["ws"][:, :s["K"] // BLOCK].to(torch.int32) - 127)


def _norm(v, kind, w, b):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w.to(v.dtype)
    return v if b is None else v + b.to(v.dtype)


def _run_plain(s):
    op = s["op"]
    if op == "quantize":
        return _values(*_quantize(s["x"])).to(torch.bfloat16)
    if op in ("linear", "linear_q"):
        x = s["x"].float() if op == "linear" else _values(*_quantize(s["x"]))
        return (x @ _weight(s).t()).to(torch.bfloat16)
    if op == "norm":
        t = _norm(s["y"].float(), s["post"], s["post_w"], s["post_b"])
        if s["gate"] is not None:
            t = t * s["gate"].float()
        r = s["res_scale"] * s["r"].float() + t
        x = _norm(r, s["pre"], s["pre_w"], s["pre_b"])
        return {"r": r.to(torch.bfloat16), "x": x.to(torch.bfloat16)}
    return _sample_plain(s)


def _sample_plain(s):
    """Weights are whole numbers, so that every sum is exact and ties and thresholds are the same in any order."""
    logits = s["logits"].float()
    B, V = logits.shape
    order_l, order = torch.sort(logits, dim=-1, descending=True, stable=True)
    T = s["temperature"].unsqueeze(-1)
    greedy = T <= 0
    z = (order_l - order_l[:, :1]) * (1.0 / torch.where(greedy, torch.ones_like(T), T))
    w = torch.round(torch.exp(z) * ONE).to(torch.int64)
    rank = torch.arange(V, device=w.device).expand(B, V)
    k = s["top_k"].unsqueeze(-1)
    keep = (rank < torch.where(k <= 0, V, k)) & (~greedy | (rank == 0))
    w = w * keep
    before = torch.cumsum(w, -1) - w
    p = s["top_p"].unsqueeze(-1)
    mass = torch.ceil(p.double() * w.sum(-1, keepdim=True).double()).to(torch.int64).clamp(min=1)
    keep = keep & ((p >= 1) | (before < mass))
    floor = torch.ceil(s["min_p"].double().clamp(0, 1) * ONE).to(torch.int64).unsqueeze(-1)
    w = w * (keep & (w >= floor))
    w = torch.zeros_like(w).scatter_(-1, order, w)             # back to the order of the vocabulary
    total = w.sum(-1, keepdim=True)
    t = torch.floor(s["u"].double().unsqueeze(-1) * total.double()).to(torch.int64)
    token = (torch.cumsum(w, -1) <= t).sum(-1, keepdim=True)
    logprob = torch.log((w.gather(-1, token).double() / total.double()).float())
    return {"tokens": token.squeeze(-1).to(torch.int32), "logprobs": logprob.squeeze(-1)}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def _exact_mx4(x):
    """Values of x after quantisation, from the definition: nearest representable value of each block, ties to the even
    code.  The candidates are compared by their distance."""
    v = x.double().view(x.shape[0], -1, BLOCK)
    _, ex = torch.frexp(v.abs().amax(-1, keepdim=True))        # amax = m 2^ex with m in [1/2, 1)
    scale = ((ex.long() + (1023 - 3)) << 52).view(torch.float64)
    r = v.abs() / scale
    best = torch.zeros_like(r)
    gap = r.clone()                                            # distance to the value 0
    for c in (2, 4, 6, 1, 3, 5, 7):                            # even codes first: an odd one has to be strictly nearer
        d = (r - E2M1[c]).abs()
        near = d < gap
        best = torch.where(near, torch.full_like(best, E2M1[c]), best)
        gap = torch.where(near, d, gap)
    return (torch.copysign(best, v) * scale).view(x.shape)


def _exact_norm(v, kind, w, b):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.sum(-1, keepdim=True) / v.shape[-1]
    v = v / torch.sqrt(v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS) * w.double()
    return v if b is None else v + b.double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return torch.cat([_exact_mx4(p) for p in s["x"].split(1024)])
    if op in ("linear", "linear_q"):
        x = s["x"].double() if op == "linear" else _exact_mx4(s["x"])
        lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
        cols = []
        for wq, ws in zip(s["wq"].split(4096), s["ws"].split(4096)):
            w = torch.empty(wq.shape[0], case["K"], dtype=torch.float64, device="cuda")
            w[:, 0::2] = lut[(wq & 15).long()]
            w[:, 1::2] = lut[(wq >> 4).long()]
            e = ws[:, :case["K"] // BLOCK].double() - 127
            cols.append(x @ (w.view(-1, case["K"] // BLOCK, BLOCK) * torch.exp2(e).unsqueeze(-1)).view(w.shape).t())
        return torch.cat(cols, 1)
    if op == "norm":
        t = _exact_norm(s["y"].double(), case["post"], s["post_w"], s["post_b"])
        if s["gate"] is not None:
            t = t * s["gate"].double()
        r = s["res_scale"] * s["r"].double() + t
        return {"r": r, "x": _exact_norm(r, case["pre"], s["pre_w"], s["pre_b"])}
    logprobs = torch.empty(case["B"], dtype=torch.float64)
    rows = s["logits"].double()
    T, k, p, m, u = (s[n].double().tolist() for n in ("temperature", "top_k", "top_p", "min_p", "u"))
    for i in range(case["B"]):                                 # one request at a time, from the definition
        l = rows[i]
        if T[i] <= 0:
            logprobs[i] = 0.0
            continue
        q = torch.exp((l - l.max()) / T[i])
        order = torch.argsort(l, descending=True, stable=True)
        order = order[:int(k[i])] if k[i] > 0 else order
        if p[i] < 1:
            c = torch.cumsum(q[order], 0)
            order = order[(c - q[order]) < p[i] * c[-1]]
        order = order[q[order] >= m[i]]
        kept = order.sort().values
        c = torch.cumsum(q[kept], 0)
        j = min(int((c <= u[i] * c[-1]).sum()), kept.numel() - 1)
        logprobs[i] = torch.log(q[kept[j]] / c[-1])
    return {"tokens": None, "logprobs": logprobs}
