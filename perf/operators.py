"""Measured cases of the 4-bit microscaled (MXFP4) linear layers and of the mixture-of-experts layer.

Four operators, each with a plain form in elementary torch operations (32-bit
arithmetic, one rounding at the end) and the library's own call:

  quantize  values -> MXFP4 codes and scales, and back to BF16 values
  linear    Y = X W^T, X in BF16, W in MXFP4 (weight-only)
  linear_mx the same with X quantized to MXFP4 within the call (both operands 4-bit)
  moe       router softmax and top-k, gate and up projections, silu(gate) * up,
            down projection, weighted sum over the chosen experts; expert weights
            in the 8-bit affine format or in MXFP4

MXFP4: blocks of 32 consecutive values of a row share one scale byte s, worth
2^(s - 127); every value is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign (bit
3), two codes to a byte, the even element in the low half.  Quantizing a block
with largest magnitude a: s - 127 = floor(log2 a) - 2 (not below -127), each
value divided by the scale and rounded to the nearest code, ties to the even
code, magnitudes above 6 to 6.
8-bit affine: w = q * scale + bias, one BF16 scale and bias per group of a row.
"""
import math

import torch

own = False  # False: the plain forms; True: this repository's kernels

MX_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # one decoding step's activations of a small batch: a call of a few microseconds, f32 from the step before
        {"name": "quantize_16x4096_f32", "op": "quantize", "rows": 16, "k": 4096, "dtype": "f32"},
        # a whole gate/up weight on loading a checkpoint
        {"name": "quantize_14336x4096", "op": "quantize", "rows": 14336, "k": 4096, "dtype": "bf16"},
        # decode of one token: the q or o projection, latency counts
        {"name": "linear_m1_4096x4096", "op": "linear", "m": 1, "n": 4096, "k": 4096},
        # decode of one token: the largest down projection
        {"name": "linear_m1_8192x28672", "op": "linear", "m": 1, "n": 8192, "k": 28672},
        # decode of a batch of 16 sequences: the down projection
        {"name": "linear_m16_4096x14336", "op": "linear", "m": 16, "n": 4096, "k": 14336},
        # prefill of a prompt: the gate or up projection
        {"name": "linear_m512_14336x4096", "op": "linear", "m": 512, "n": 14336, "k": 4096},
        # a few sequences, both operands in 4 bits
        {"name": "linear_mx_m8_4096x14336", "op": "linear_mx", "m": 8, "n": 4096, "k": 14336},
        # prefill of a long prompt, both operands in 4 bits
        {"name": "linear_mx_m2048_14336x4096", "op": "linear_mx", "m": 2048, "n": 14336, "k": 4096},
        # one token through many small 4-bit experts: the smallest layer call
        {"name": "moe_mxfp4_t1_64x1024x2048_top8", "op": "moe", "fmt": "mxfp4", "gs": 32, "tokens": 1, "experts": 64,
         "topk": 8, "inner": 1024, "hidden": 2048, "renorm": True, "logits": "f32", "masked": False},
        # one token through eight large 8-bit experts
        {"name": "moe_int8_t1_8x14336x4096_top2", "op": "moe", "fmt": "int8", "gs": 64, "tokens": 1, "experts": 8,
         "topk": 2, "inner": 14336, "hidden": 4096, "renorm": True, "logits": "f32", "masked": False},
        # an odd few tokens through many small 8-bit experts, BF16 logits (ties), some experts masked out
        {"name": "moe_int8_t13_64x1024x2048_top6", "op": "moe", "fmt": "int8", "gs": 128, "tokens": 13, "experts": 64,
         "topk": 6, "inner": 1024, "hidden": 2048, "renorm": False, "logits": "bf16", "masked": True},
        # a decode batch through eight large 4-bit experts: every expert has several tokens
        {"name": "moe_mxfp4_t37_8x14336x4096_top2", "op": "moe", "fmt": "mxfp4", "gs": 32, "tokens": 37, "experts": 8,
         "topk": 2, "inner": 14336, "hidden": 4096, "renorm": True, "logits": "f32", "masked": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "linear", "linear_mx", "moe"))
    if op == "quantize":
        k = 32 * _log(rng, 4, 896)
        return {"op": op, "rows": max(1, min(_log(rng, 1, 28672), 14336 * 4096 // k)), "k": k,
                "dtype": rng.choice(("bf16", "f32"))}
    if op in ("linear", "linear_mx"):
        k = 32 * _log(rng, 8, 896)
        n = min(_log(rng, 100, 28672), 8192 * 28672 // k)
        m = rng.choice((1, _log(rng, 1, 2048)))
        most = 512 if op == "linear" else 2048
        return {"op": op, "m": max(1, min(m, most * 14336 * 4096 // (n * k))), "n": n, "k": k}
    fmt = rng.choice(("int8", "mxfp4"))
    gs = rng.choice((32, 64, 128)) if fmt == "int8" else 32
    experts = rng.choice((4, 6, 8, 16, 32, 60, 64, 128))
    hidden = gs * max(1, _log(rng, 512, 4096) // gs)
    inner = gs * max(1, min(_log(rng, 256, 14336), 8 * 14336 * 4096 // (experts * hidden)) // gs)
    return {"op": op, "fmt": fmt, "gs": gs, "tokens": rng.choice((1, _log(rng, 1, 64))), "experts": experts,
            "topk": min(experts, rng.choice((1, 2, 4, 6, 8))), "inner": inner, "hidden": hidden,
            "renorm": rng.random() < 0.5, "logits": rng.choice(("f32", "bf16")), "masked": rng.random() < 0.5}


# ---- inputs -----------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, rows, k, dtype=torch.bfloat16):
    """Normalized hidden states: N(0, 1) with a few strong channels."""
    x = torch.randn(rows, k, generator=g, device="cuda")
    strong = 1.0 + 15.0 * (torch.rand(k, generator=g, device="cuda") < 0.01)
    return (x * strong).to(dtype)


def _mx_weight(g, n, k):
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(117, 122, (n, k // 32), generator=g, device="cuda", dtype=torch.uint8)
    return {"codes": codes, "scales": scales}


def _int8_weight(g, n, k, gs):
    """8-bit affine: uniform codes, biases near -128 scale, as the repository's synthetic weights, at a checkpoint's size of values."""
    codes = torch.randint(0, 256, (n, k), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(n, k // gs, generator=g, device="cuda") * 2e-4 + 1e-4).bfloat16()
    b = (-128.0 * s.float() * (1.0 + 0.1 * (torch.rand(n, k // gs, generator=g, device="cuda") - 0.5))).bfloat16()
    return {"packed": codes.view(torch.int32), "scales": s, "biases": b, "gs": gs}


def _weight(g, case, n, k):
    return _mx_weight(g, n, k) if case["fmt"] == "mxfp4" else _int8_weight(g, n, k, case["gs"])


def _handle(w):
    """The weight object that a program keeps after loading its checkpoint (it borrows the tensors)."""
    from weight_only_quantized_int8_amd import Int8Weight, Mxfp4Weight
    return Mxfp4Weight(w["codes"], w["scales"]) if "codes" in w else Int8Weight(w["packed"], w["scales"], w["biases"], w["gs"])


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "quantize":
        s["x"] = _activations(g, case["rows"], case["k"], torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["x"][case["rows"] // 2, :32] = 0  # a block with nothing in it
    elif case["op"] in ("linear", "linear_mx"):
        s["w"] = _mx_weight(g, case["n"], case["k"])
        s["x"] = _activations(g, case["m"], case["k"])
    else:
        e, t, i, h = case["experts"], case["tokens"], case["inner"], case["hidden"]
        s["gate"], s["up"], s["down"] = _weight(g, case, e * i, h), _weight(g, case, e * i, h), _weight(g, case, e * h, i)
        s["x"] = torch.randn(t, h, generator=g, device="cuda").bfloat16()
        logits = 1.5 * torch.randn(t, e, generator=g, device="cuda")
        if case["masked"]:
            logits[torch.rand(t, e, generator=g, device="cuda") < 0.2] = -math.inf
            if t > 4:
                logits[t // 2] = -math.inf  # a token that no expert may take
        s["route"] = logits.bfloat16() if case["logits"] == "bf16" else logits
    if own:
        for name in ("w", "gate", "up", "down"):
            if name in s:
                s[name] = _handle(s[name])
    return s


# ---- the plain forms --------------------------------------------------------------------------

def _mx_values(codes, scales):
    """[..., K/2] code bytes and [..., K/32] scale bytes -> f32 [..., K]."""
    table = torch.tensor(MX_VALUES + tuple(-v for v in MX_VALUES), device=codes.device)
    q = torch.stack((codes & 15, codes >> 4), -1).reshape(*scales.shape, 32)
    return (table[q.int()] * torch.exp2(scales.float() - 127.0).unsqueeze(-1)).reshape(*scales.shape[:-1], -1)


def _mx_rounded(x):
    """f32 [..., K] -> the values that its MXFP4 codes and scales stand for."""
    v = x.reshape(*x.shape[:-1], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    e = torch.frexp(top).exponent - 3  # floor(log2 top) - 2
    scale = torch.exp2(torch.where(top > 0, e, -127).clamp(min=-127).float())
    v = v / scale
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
    return ((torch.round(v / step) * step).clamp(-6.0, 6.0) * scale).reshape(x.shape)


def _plain_weight(w, pick=None, experts=1):
    """f32 [experts, N, K] of a stacked weight, or [len(pick), N, K] of the picked experts."""
    def of(t):
        t = t.reshape(experts, t.shape[0] // experts, t.shape[1])
        return t if pick is None else t[pick]
    if "codes" in w:
        return _mx_values(of(w["codes"]), of(w["scales"]))
    s, b = of(w["scales"]).float(), of(w["biases"]).float()
    q = of(w["packed"].view(torch.uint8)).float().reshape(*s.shape, w["gs"])
    return (q * s.unsqueeze(-1) + b.unsqueeze(-1)).reshape(*s.shape[:-1], -1)


def _plain_moe(s):
    t, e, k = s["tokens"], s["experts"], s["topk"]
    logits = s["route"].float()
    top = logits.amax(-1, keepdim=True)
    p = torch.where(logits > -math.inf, torch.exp(logits - top), 0.0)
    order = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]  # ties: the lowest expert first
    chosen = p.gather(1, order)
    total = (chosen if s["renorm"] else p).sum(-1, keepdim=True)
    weight = torch.where(total > 0, chosen / total, 0.0)
    x = s["x"].float()
    if t * k <= e:  # few slots: the chosen experts' weights alone
        ids = order.reshape(-1)
        xs = x.repeat_interleave(k, 0).unsqueeze(-1)
        gate, up = _plain_weight(s["gate"], ids, e) @ xs, _plain_weight(s["up"], ids, e) @ xs
        y = _plain_weight(s["down"], ids, e) @ (gate / (1.0 + torch.exp(-gate)) * up)
        y = (y.reshape(t, k, -1) * weight.unsqueeze(-1)).sum(1)
    else:  # every expert on every token, weighted
        by = torch.zeros(t, e, device=x.device).scatter(1, order, weight)
        gate = torch.matmul(x, _plain_weight(s["gate"], None, e).transpose(1, 2))
        up = torch.matmul(x, _plain_weight(s["up"], None, e).transpose(1, 2))
        y = torch.matmul(gate / (1.0 + torch.exp(-gate)) * up, _plain_weight(s["down"], None, e).transpose(1, 2))
        y = (y * by.t().unsqueeze(-1)).sum(0)
    return y.bfloat16()


def _plain(s):
    if s["op"] == "quantize":
        return _mx_rounded(s["x"].float()).bfloat16()
    if s["op"] == "moe":
        return _plain_moe(s)
    x = s["x"].float()
    if s["op"] == "linear_mx":
        x = _mx_rounded(x)
    return (x @ _mx_values(s["w"]["codes"], s["w"]["scales"]).t()).bfloat16()


# ---- one pass ---------------------------------------------------------------------------------

def run(state):
    s = state
    if not own:
        return _plain(s)
    from weight_only_quantized_int8_amd import Mxfp4Weight, moe_layer
    if s["op"] == "quantize":
        return Mxfp4Weight.quantize(s["x"]).dequantize_to()
    if s["op"] == "linear":
        return s["w"].gemm(s["x"])
    if s["op"] == "linear_mx":
        return s["w"].gemm_mx(Mxfp4Weight.quantize(s["x"]))
    return moe_layer(s["gate"], s["up"], s["down"], s["experts"], s["x"], s["route"], s["topk"],
                     renormalize=s["renorm"])


# ---- what a pass cannot do without ------------------------------------------------------------

def work(case):
    mx = 0.5 + 1.0 / 32.0  # bytes a value in MXFP4
    if case["op"] == "quantize":
        v = case["rows"] * case["k"]
        return {"bytes": v * ((2 if case["dtype"] == "bf16" else 4) + 2 * mx + 2), "flops": 4.0 * v}
    if case["op"] in ("linear", "linear_mx"):
        m, n, k = case["m"], case["n"], case["k"]
        more = 2 * m * k * mx if case["op"] == "linear_mx" else 0.0  # the codes in between
        return {"bytes": n * k * mx + 2 * m * k + 2 * m * n + more, "flops": 2.0 * m * n * k}
    t, e, k, i, h = (case[n] for n in ("tokens", "experts", "topk", "inner", "hidden"))
    named = e * (1.0 - (1.0 - k / e) ** t)  # experts that any token names, for even routing
    per = mx if case["fmt"] == "mxfp4" else 1.0 + 4.0 / case["gs"]
    return {"bytes": named * 3 * i * h * per + 4 * t * h + 4 * t * e, "flops": 6.0 * t * k * i * h}


# ---- the definition in 64 bits ----------------------------------------------------------------

def _exact_mx(w):
    """float64 [N, K]: 2^(scale - 127) times sign * magnitude, from the code's bits: exponent e = bits 2..1, mantissa b = bit 0."""
    c, n = w["codes"], w["codes"].shape[0]
    out = torch.empty(n, 2 * c.shape[1], dtype=torch.float64, device=c.device)
    for half in range(2):
        q = ((c >> (4 * half)) & 15).to(torch.int32)
        e, b, sign = (q >> 1) & 3, (q & 1).double(), 1.0 - 2.0 * (q >> 3).double()
        out[:, half::2] = sign * torch.where(e == 0, 0.5 * b, (1.0 + 0.5 * b) * torch.pow(2.0, (e - 1).double()))
    return out * torch.pow(2.0, w["scales"].double() - 127.0).repeat_interleave(32, 1)


def _exact_weight(w, lo, hi):
    if "codes" in w:
        return _exact_mx({"codes": w["codes"][lo:hi], "scales": w["scales"][lo:hi]})
    q = w["packed"][lo:hi].view(torch.uint8).double()
    return q * w["scales"][lo:hi].double().repeat_interleave(w["gs"], 1) + w["biases"][lo:hi].double().repeat_interleave(w["gs"], 1)


def _exact_rounded(x):
    x = x.double()
    a = x.reshape(-1, 32).abs()
    top = a.max(1).values
    s = torch.where(top > 0, torch.floor(torch.log2(top)), torch.full_like(top, -125.0))
    s = torch.where(torch.pow(2.0, s) > top, s - 1, torch.where(torch.pow(2.0, s + 1) <= top, s + 1, s))
    unit = torch.pow(2.0, torch.clamp(torch.where(top > 0, s, torch.full_like(s, -125.0)) - 2, min=-127.0)).unsqueeze(1)
    a = a / unit
    got = torch.zeros_like(a)
    # the code above begins at the midpoint, which itself goes to the even one of the two codes
    for c in range(1, 8):
        mid = (MX_VALUES[c - 1] + MX_VALUES[c]) / 2
        got = torch.where(a >= mid if c % 2 == 0 else a > mid, torch.full_like(a, MX_VALUES[c]), got)
    return (got * unit).reshape(x.shape) * torch.sign(x)


def _exact_moe(s):
    logits, x = s["route"].double().cpu(), s["x"].double()
    e, i, h = s["experts"], s["inner"], s["hidden"]
    r = torch.zeros(s["tokens"], e, dtype=torch.float64)
    for t, row in enumerate(logits.tolist()):
        if max(row) == -math.inf:
            continue
        z = [math.exp(v - max(row)) for v in row]
        best = sorted(range(e), key=lambda j: (-row[j], j))[:s["topk"]]
        total = sum(z[j] for j in best) if s["renorm"] else sum(z)
        for j in best:
            r[t, j] = z[j] / total
    r = r.to(x.device)
    y = torch.zeros(s["tokens"], h, dtype=torch.float64, device=x.device)
    for j in range(e):
        on = torch.nonzero(r[:, j] > 0).flatten()
        if on.numel() == 0:
            continue
        gate = x[on] @ _exact_weight(s["gate"], j * i, (j + 1) * i).t()
        up = x[on] @ _exact_weight(s["up"], j * i, (j + 1) * i).t()
        out = (gate * torch.sigmoid(gate) * up) @ _exact_weight(s["down"], j * h, (j + 1) * h).t()
        y[on] += r[on, j].unsqueeze(1) * out
    return y


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "quantize":
        return _exact_rounded(s["x"])
    if case["op"] == "moe":
        return _exact_moe(s)
    x = _exact_rounded(s["x"]) if case["op"] == "linear_mx" else s["x"].double()
    return x @ _exact_mx(s["w"]).t()
