"""Measured cases of low-rank adapters beside a shared projection, of the routing to experts, and of an expert layer from such a routing.

Three operators, each with a plain form in elementary torch operations (32-bit
arithmetic, 64-bit where scores are compared, one rounding at the end) and the
library's own call:

  lora    rows of many requests, each through its own request's adapter:
          y[t] = base[t] + scale[e] * B[e] (A[e] x[t]) with e = ids[t], base[t] alone
          for ids[t] = -1; up to three projections that share x (q, k and v)
  route   scores s = softmax(l) or sigmoid(l); choice by c = s + bias (c orders as l
          without bias and groups); groups of experts scored by their largest c or
          the sum of their two largest, the best topk_groups stay; the topk largest c
          in them, ties to the lowest index; weights s, divided by their sum where
          renormalized, times a factor.  Experts at -inf are never taken: the slots
          that are left over hold id -1 and weight 0
  experts route, then silu(gate) * up and down projections of the chosen experts and
          their weighted sum; expert weights in the 8-bit affine format or in MXFP4

MXFP4: blocks of 32 values of a row share a scale byte worth 2^(s - 127); each is
one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign (bit 3), the even element in the low
half of a byte.  8-bit affine: w = q * scale + bias by groups of a row.
"""
import math

import torch

own = False  # False: the plain forms; True: this repository's kernels

MX_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ------------------------------------------------------------------------------------
# lora: m rows, the first `decode` of them single tokens with an adapter each, the rest `prompts` runs of one adapter each;
# `pool` adapters of rank `rank` (where `mixed`, of ranks from 8 up to it), projections k -> n, n2, n3 (0: none).

def listed():
    return [
        # one token of one request, the o projection: latency counts
        {"name": "lora_m1_4096x4096_r16", "op": "lora", "m": 1, "decode": 1, "prompts": 0, "pool": 8, "rank": 16, "mixed": False,
         "k": 4096, "n": 4096, "n2": 0, "n3": 0, "base": True},
        # a decode batch through q, k and v, adapters of different ranks
        {"name": "lora_m33_qkv_4096_r32_mixed", "op": "lora", "m": 33, "decode": 33, "prompts": 0, "pool": 40, "rank": 32, "mixed": True,
         "k": 4096, "n": 4096, "n2": 1024, "n3": 1024, "base": True},
        # a large decode batch, the down projection
        {"name": "lora_m200_4096x14336_r64", "op": "lora", "m": 200, "decode": 200, "prompts": 0, "pool": 60, "rank": 64, "mixed": False,
         "k": 14336, "n": 4096, "n2": 0, "n3": 0, "base": True},
        # a prompt's chunk next to a decode batch, gate and up, without a base
        {"name": "lora_m549_gate_up_14336x4096_r16", "op": "lora", "m": 549, "decode": 37, "prompts": 1, "pool": 16, "rank": 16,
         "mixed": False, "k": 4096, "n": 14336, "n2": 14336, "n3": 0, "base": False},
        # a few prompts next to a decode batch, the down projection, adapters of different ranks
        {"name": "lora_m2109_4096x14336_r64_mixed", "op": "lora", "m": 2109, "decode": 61, "prompts": 3, "pool": 24, "rank": 64,
         "mixed": True, "k": 14336, "n": 4096, "n2": 0, "n3": 0, "base": True},
        # several long prompts, the gate or up projection
        {"name": "lora_m8192_14336x4096_r64", "op": "lora", "m": 8192, "decode": 0, "prompts": 5, "pool": 12, "rank": 64, "mixed": False,
         "k": 4096, "n": 14336, "n2": 0, "n3": 0, "base": True},
        # one token, the smallest routing: a call of a few microseconds
        {"name": "route_t1_64_top6", "op": "route", "tokens": 1, "experts": 64, "topk": 6, "scoring": "softmax", "bias": False, "groups": 1,
         "topk_groups": 1, "group_score": "max", "renorm": True, "scale": 1.0, "logits": "f32", "masked": False},
        # a decode batch, BF16 logits (ties), some experts masked out
        {"name": "route_t131_60_top4_bf16", "op": "route", "tokens": 131, "experts": 60, "topk": 4, "scoring": "softmax", "bias": False,
         "groups": 1, "topk_groups": 1, "group_score": "max", "renorm": False, "scale": 1.0, "logits": "bf16", "masked": True},
        # a decode batch, sigmoid scores with a bias for balance, groups
        {"name": "route_t64_256_sigmoid_8groups", "op": "route", "tokens": 64, "experts": 256, "topk": 8, "scoring": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "group_score": "top2", "renorm": True, "scale": 2.5, "logits": "f32", "masked": False},
        # the prompts of a large batch, the same
        {"name": "route_t16384_256_sigmoid_8groups", "op": "route", "tokens": 16384, "experts": 256, "topk": 8, "scoring": "sigmoid",
         "bias": True, "groups": 8, "topk_groups": 4, "group_score": "top2", "renorm": True, "scale": 2.5, "logits": "f32", "masked": False},
        # one token through small 4-bit experts chosen by groups
        {"name": "experts_mxfp4_t1_64x1024x2048_top8", "op": "experts", "fmt": "mxfp4", "gs": 32, "inner": 1024, "hidden": 2048, "tokens": 1,
         "experts": 64, "topk": 8, "scoring": "sigmoid", "bias": True, "groups": 8, "topk_groups": 4, "group_score": "top2",
         "renorm": True, "scale": 2.5, "logits": "f32", "masked": False},
        # a decode batch through small 8-bit experts, softmax scores with a bias, some experts masked out
        {"name": "experts_int8_t29_64x1024x2048_top6", "op": "experts", "fmt": "int8", "gs": 64, "inner": 1024, "hidden": 2048, "tokens": 29,
         "experts": 64, "topk": 6, "scoring": "softmax", "bias": True, "groups": 4, "topk_groups": 2, "group_score": "max",
         "renorm": False, "scale": 16.0, "logits": "f32", "masked": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_lora(rng):
    rank = rng.choice((8, 16, 24, 32, 64, 128))
    k = 32 * _log(rng, 16, 448)
    n, n2, n3 = _log(rng, 200, 14336), 0, 0
    if rng.random() < 0.3:
        n2 = _log(rng, 200, n)
        n3 = n2 if rng.random() < 0.5 else 0
    outs = 1 + (n2 > 0) + (n3 > 0)
    pool = max(1, min(_log(rng, 1, 64), 100_000_000 // (rank * (outs * k + n + n2 + n3))))
    most = 8192 * (14336 + 4096) * 64 // ((n + n2 + n3 + outs * k) * max(rank, 64))
    kind = rng.choice(("decode", "decode", "mix", "prompts"))
    if kind == "decode":
        m = decode = min(most, _log(rng, 1, 256))
        prompts = 0
    else:
        decode = 0 if kind == "prompts" else min(most, _log(rng, 1, 64))
        m = max(decode + 1, min(most, decode + _log(rng, 17, 8192)))
        prompts = min(m - decode, rng.randint(1, 6))
    return {"op": "lora", "m": m, "decode": decode, "prompts": prompts, "pool": pool, "rank": rank,
            "mixed": rng.random() < 0.3, "k": k, "n": n, "n2": n2, "n3": n3, "base": rng.random() < 0.8}


def _draw_route(rng, most_tokens):
    size, groups = rng.choice(((64, 1), (60, 1), (60, 6), (8, 1), (16, 4), (128, 1), (128, 8), (160, 8), (256, 8), (512, 16)))
    return {"tokens": rng.choice((1, _log(rng, 2, 64), _log(rng, 2, most_tokens))), "experts": size, "topk": rng.choice((1, 2, 4, 6, 8)),
            "scoring": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.6, "groups": groups,
            "topk_groups": max(1, groups // 2), "group_score": rng.choice(("max", "top2")), "renorm": rng.random() < 0.6,
            "scale": rng.choice((1.0, 2.5)), "logits": rng.choice(("f32", "bf16")), "masked": rng.random() < 0.4}


def draw(rng):
    op = rng.choice(("lora", "lora", "route", "experts"))
    if op == "lora":
        return _draw_lora(rng)
    if op == "route":
        return {"op": op, **_draw_route(rng, 8192)}
    case = {"op": op, **_draw_route(rng, 48)}
    fmt = rng.choice(("int8", "mxfp4"))
    gs = rng.choice((32, 64, 128)) if fmt == "int8" else 32
    hidden = gs * max(1, _log(rng, 512, 4096) // gs)
    inner = gs * max(1, min(_log(rng, 256, 4096), 64 * 1024 * 2048 // (case["experts"] * hidden)) // gs)
    case["topk"] = min(case["topk"], 6)
    return {**case, "fmt": fmt, "gs": gs, "hidden": hidden, "inner": inner}


# ---- inputs -----------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _outs(case):
    return [n for n in (case["n"], case["n2"], case["n3"]) if n]


def _ranks(case):
    """The adapters' own ranks, 8 .. rank."""
    r = case["rank"]
    return [max(8, r >> (i % 3)) // 8 * 8 if case["mixed"] else r for i in range(case["pool"])]


def _lora_inputs(g, case, s):
    m, k, r, pool = case["m"], case["k"], case["rank"], case["pool"]
    # normalized hidden states: N(0, 1) with a few strong channels
    s["x"] = (_randn(g, m, k) * (1.0 + 15.0 * (_rand(g, k) < 0.01))).bfloat16()
    ids = torch.randint(0, pool, (m,), generator=g, device="cuda", dtype=torch.int32)
    ids[1:max(case["decode"], 1)][_rand(g, max(case["decode"], 1) - 1) < 0.1] = -1  # requests without an adapter
    # the plan of the batch, as a server has it on the host: the prompts' first and last rows; their adapters by their number
    s["runs"], at = [], case["decode"]
    for i in range(case["prompts"]):
        end = at + (m - at) // (case["prompts"] - i)
        e = (7 * i + m) % pool
        ids[at:end] = e
        s["runs"].append((at, end, e))
        at = end
    s["ids"] = ids
    ranks = _ranks(case)
    s["ranks"] = torch.tensor(ranks, dtype=torch.int32, device="cuda") if case["mixed"] else None
    live = torch.arange(r, device="cuda").unsqueeze(0) < torch.tensor(ranks, device="cuda").unsqueeze(1)  # [pool, r]
    s["stacks"] = []
    for n in _outs(case):
        a = (_randn(g, pool, r, k) * k ** -0.5 * live.unsqueeze(2)).bfloat16()
        b = (_randn(g, pool, n, r) * 0.2 * live.unsqueeze(1)).bfloat16()
        s["stacks"].append({"a": a, "b": b, "scales": 0.5 + _rand(g, pool)})
    if case["base"]:  # the fused projection's output, cut by columns
        s["base"] = list(torch.split(_randn(g, m, sum(_outs(case))).bfloat16(), _outs(case), dim=1))
    else:
        s["base"] = None


def _route_inputs(g, case, s):
    t, e = case["tokens"], case["experts"]
    logits = 1.5 * _randn(g, t, e)
    if case["masked"]:
        logits[_rand(g, t, e) < 0.2] = -math.inf
        if t > 4:
            logits[t // 2] = -math.inf  # a token that no expert may take
    s["route"] = logits.bfloat16() if case["logits"] == "bf16" else logits
    s["choice_bias"] = 0.05 * _randn(g, e) if case["bias"] else None


def _weight(g, case, n, k):
    if case["fmt"] == "mxfp4":
        return {"codes": torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8),
                "scales": torch.randint(117, 122, (n, k // 32), generator=g, device="cuda", dtype=torch.uint8)}
    codes = torch.randint(0, 256, (n, k), generator=g, device="cuda", dtype=torch.uint8)
    scales = (_rand(g, n, k // case["gs"]) * 2e-4 + 1e-4).bfloat16()
    biases = (-128.0 * scales.float() * (1.0 + 0.1 * (_rand(g, n, k // case["gs"]) - 0.5))).bfloat16()
    return {"packed": codes.view(torch.int32), "scales": scales, "biases": biases, "gs": case["gs"]}


def _handles(s):
    """The objects that a program keeps after loading its checkpoint (they borrow the tensors)."""
    from weight_only_quantized_int8_amd import Int8Weight, LoraAdapters, Mxfp4Weight
    if s["op"] == "lora":
        s["adapters"] = [LoraAdapters(t["a"], t["b"], t["scales"], s["ranks"]) for t in s["stacks"]]
    if s["op"] == "experts":
        for name in ("gate", "up", "down"):
            w = s[name]
            s[name] = Mxfp4Weight(w["codes"], w["scales"]) if "codes" in w else \
                Int8Weight(w["packed"], w["scales"], w["biases"], w["gs"])


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    s["choice_bias"] = None
    if case["op"] == "lora":
        _lora_inputs(g, case, s)
    else:
        _route_inputs(g, case, s)
    if case["op"] == "experts":
        e, i, h = case["experts"], case["inner"], case["hidden"]
        s["gate"], s["up"], s["down"] = _weight(g, case, e * i, h), _weight(g, case, e * i, h), _weight(g, case, e * h, i)
        s["x"] = _randn(g, case["tokens"], h).bfloat16()
    if own:
        _handles(s)
    return s


# ---- the plain forms --------------------------------------------------------------------------

def _plain_lora(s):
    x, ids, d = s["x"].float(), s["ids"], s["decode"]
    outs = []
    for i, t in enumerate(s["stacks"]):
        delta = torch.empty(s["m"], t["b"].shape[1], device=x.device)
        if d:  # single rows: their adapters gathered
            e = ids[:d].clamp(min=0).long()
            u = torch.matmul(t["a"][e].float(), x[:d].unsqueeze(2))
            one = torch.matmul(t["b"][e].float(), u).squeeze(2) * t["scales"][e].unsqueeze(1)
            delta[:d] = torch.where(ids[:d].unsqueeze(1) >= 0, one, 0.0)
        for lo, hi, e in s["runs"]:
            delta[lo:hi] = ((x[lo:hi] @ t["a"][e].float().t()) @ t["b"][e].float().t()) * t["scales"][e]
        outs.append((delta + s["base"][i].float() if s["base"] else delta).bfloat16())
    return outs


def _plain_route(s):
    """ids int32 and weights f32 [tokens, topk]."""
    t, e, k, groups = s["tokens"], s["experts"], s["topk"], s["groups"]
    l = s["route"].double()
    if s["scoring"] == "softmax":
        p = torch.exp(l - l.amax(-1, keepdim=True))
        p = torch.where(l > -math.inf, p, 0.0)
        score = torch.where(l > -math.inf, p / p.sum(-1, keepdim=True), 0.0)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    c = l
    if s["choice_bias"] is not None or groups > 1:
        c = score if s["choice_bias"] is None else score + s["choice_bias"].double()
        c = torch.where(l > -math.inf, c, -math.inf)
    if groups > 1:
        by = c.reshape(t, groups, e // groups)
        if s["group_score"] == "max":
            of = by.amax(-1)
        else:  # of a group with one expert left, that one; with none, -inf
            two = torch.topk(by, 2, dim=-1).values
            of = torch.where(two[..., 1] > -math.inf, two.sum(-1), two[..., 0])
        best = torch.sort(of, dim=-1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        keep = torch.zeros(t, groups, dtype=torch.bool, device=l.device).scatter(1, best, True)
        c = torch.where(keep.unsqueeze(2), by, -math.inf).reshape(t, e)
    top = torch.sort(c, dim=-1, descending=True, stable=True)
    have = top.values[:, :k] > -math.inf
    ids = torch.where(have, top.indices[:, :k], -1)
    w = torch.where(have, score.gather(1, top.indices[:, :k]), 0.0)
    if s["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return ids.int(), (w * s["scale"]).float()


def _plain_weight(w, pick, experts):
    """f32 [experts, N, K] of a stacked weight, or [len(pick), N, K] of the picked experts."""
    def of(t):
        t = t.reshape(experts, t.shape[0] // experts, t.shape[1])
        return t if pick is None else t[pick]
    if "codes" in w:
        codes, scales = of(w["codes"]), of(w["scales"])
        table = torch.tensor(MX_VALUES + tuple(-v for v in MX_VALUES), device=codes.device)
        q = torch.stack((codes & 15, codes >> 4), -1).reshape(*scales.shape, 32)
        return (table[q.int()] * torch.exp2(scales.float() - 127.0).unsqueeze(-1)).reshape(*scales.shape[:-1], -1)
    scales, biases = of(w["scales"]).float(), of(w["biases"]).float()
    q = of(w["packed"].view(torch.uint8)).float().reshape(*scales.shape, w["gs"])
    return (q * scales.unsqueeze(-1) + biases.unsqueeze(-1)).reshape(*scales.shape[:-1], -1)


def _plain_experts(s):
    ids, weights = _plain_route(s)
    t, e, k = s["tokens"], s["experts"], s["topk"]
    x = s["x"].float()
    if t * k <= e:  # few slots: the chosen experts' weights alone
        pick = ids.clamp(min=0).reshape(-1).long()
        xs = x.repeat_interleave(k, 0).unsqueeze(-1)
        gate, up = _plain_weight(s["gate"], pick, e) @ xs, _plain_weight(s["up"], pick, e) @ xs
        y = _plain_weight(s["down"], pick, e) @ (gate / (1.0 + torch.exp(-gate)) * up)
        y = (y.reshape(t, k, -1) * weights.unsqueeze(-1)).sum(1)
    else:  # every expert on every token, weighted
        by = torch.zeros(t, e, device=x.device).scatter_add(1, ids.clamp(min=0).long(), weights)
        gate = torch.matmul(x, _plain_weight(s["gate"], None, e).transpose(1, 2))
        up = torch.matmul(x, _plain_weight(s["up"], None, e).transpose(1, 2))
        y = torch.matmul(gate / (1.0 + torch.exp(-gate)) * up, _plain_weight(s["down"], None, e).transpose(1, 2))
        y = (y * by.t().unsqueeze(-1)).sum(0)
    return {"ids": ids, "weights": weights, "y": y.bfloat16()}


# ---- one pass ---------------------------------------------------------------------------------

def run(state):
    s = state
    if not own:
        return {"lora": _plain_lora, "route": _plain_route, "experts": _plain_experts}[s["op"]](s)
    from weight_only_quantized_int8_amd import lora_add, moe_layer_routed, moe_route
    if s["op"] == "lora":
        return lora_add(s["adapters"], s["x"], s["ids"], s["base"])
    ids, weights = moe_route(s["route"], s["topk"], scoring=s["scoring"], bias=s["choice_bias"], groups=s["groups"],
                             topk_groups=s["topk_groups"], group_score=s["group_score"], renormalize=s["renorm"],
                             routed_scale=s["scale"])
    if s["op"] == "route":
        return ids, weights
    y = moe_layer_routed(s["gate"], s["up"], s["down"], s["experts"], s["x"], ids, weights)
    return {"ids": ids, "weights": weights, "y": y}


# ---- what a pass cannot do without ------------------------------------------------------------

def work(case):
    if case["op"] == "lora":
        m, k, n, outs = case["m"], case["k"], sum(_outs(case)), len(_outs(case))
        pool, rank = case["pool"], sum(_ranks(case)) / case["pool"]
        named = pool * (1.0 - (1.0 - 1.0 / pool) ** (0.9 * case["decode"]))  # adapters that any row names
        named = min(float(pool), named + min(pool, case["prompts"]))
        rows = m - 0.1 * max(0, case["decode"] - 1)
        return {"bytes": 2 * m * k + named * rank * 2 * (outs * k + n) + 2 * m * n * (2 if case["base"] else 1) + 4 * m,
                "flops": 2.0 * rows * rank * (outs * k + n)}
    t, e, topk = case["tokens"], case["experts"], case["topk"]
    route = {"bytes": t * e * (4 if case["logits"] == "f32" else 2) + 8 * t * topk, "flops": 6.0 * t * e}
    if case["op"] == "route":
        return route
    i, h = case["inner"], case["hidden"]
    named = e * (1.0 - (1.0 - topk / e) ** t)  # experts that any token names, for even routing
    per = 0.5 + 1.0 / 32.0 if case["fmt"] == "mxfp4" else 1.0 + 4.0 / case["gs"]
    return {"bytes": route["bytes"] + named * 3 * i * h * per + 4 * t * h, "flops": route["flops"] + 6.0 * t * topk * i * h}


# ---- the definition in 64 bits ----------------------------------------------------------------

def _exact_lora(s):
    outs = []
    rows_of = {}
    for row, e in enumerate(s["ids"].tolist()):
        rows_of.setdefault(e, []).append(row)
    for i, t in enumerate(s["stacks"]):
        n = t["b"].shape[1]
        y = s["base"][i].double().clone() if s["base"] else torch.zeros(s["m"], n, dtype=torch.float64, device=s["x"].device)
        for e, rows in rows_of.items():
            if e < 0:
                continue
            at = torch.tensor(rows, device=y.device)
            u = s["x"][at].double() @ t["a"][e].double().t()
            y[at] += float(t["scales"][e]) * (u @ t["b"][e].double().t())
        outs.append(y)
    return outs


def _exact_route(s):
    """Token by token, on the host: lists of ids and weights."""
    e, k, groups = s["experts"], s["topk"], s["groups"]
    size = e // groups
    bias = s["choice_bias"].double().tolist() if s["choice_bias"] is not None else [0.0] * e
    plain = s["choice_bias"] is None and groups == 1
    ids, weights = [], []
    for row in s["route"].double().tolist():
        free = [j for j in range(e) if row[j] > -math.inf]
        if s["scoring"] == "sigmoid":
            score = {j: 1.0 / (1.0 + math.exp(-row[j])) for j in free}
        else:
            z = {j: math.exp(row[j] - max(row)) for j in free}
            total = math.fsum(z.values())
            score = {j: z[j] / total for j in free}
        c = {j: row[j] if plain else score[j] + bias[j] for j in free}
        if groups > 1:
            members = [sorted((c[j] for j in free if j // size == g), reverse=True) for g in range(groups)]
            of = {g: sum(v[:2]) if s["group_score"] == "top2" else v[0] for g, v in enumerate(members) if v}
            stay = set(sorted(of, key=lambda g: (-of[g], g))[:s["topk_groups"]])
            free = [j for j in free if j // size in stay]
        best = sorted(free, key=lambda j: (-c[j], j))[:k]
        w = [score[j] for j in best]
        if s["renorm"] and sum(w) > 0:
            w = [v / math.fsum(w) for v in w]
        ids.append(best + [-1] * (k - len(best)))
        weights.append([v * s["scale"] for v in w] + [0.0] * (k - len(best)))
    return torch.tensor(ids, dtype=torch.int32), torch.tensor(weights, dtype=torch.float64)


def _exact_weight(w, lo, hi):
    """float64 rows lo .. hi - 1."""
    if "packed" in w:
        wide = [w[n][lo:hi].double().repeat_interleave(w["gs"], 1) for n in ("scales", "biases")]
        return w["packed"][lo:hi].view(torch.uint8).double() * wide[0] + wide[1]
    c = w["codes"][lo:hi]
    out = torch.empty(hi - lo, 2 * c.shape[1], dtype=torch.float64, device=c.device)
    for half in range(2):  # exponent: bits 2..1, mantissa: bit 0
        q = ((c >> (4 * half)) & 15).to(torch.int32)
        exp, frac, sign = (q >> 1) & 3, (q & 1).double(), 1.0 - 2.0 * (q >> 3).double()
        out[:, half::2] = sign * torch.where(exp == 0, 0.5 * frac, (1.0 + 0.5 * frac) * torch.pow(2.0, (exp - 1).double()))
    return out * torch.pow(2.0, w["scales"][lo:hi].double() - 127.0).repeat_interleave(32, 1)


def _exact_experts(s):
    ids, weights = _exact_route(s)
    x, i, h = s["x"].double(), s["inner"], s["hidden"]
    y = torch.zeros(s["tokens"], h, dtype=torch.float64, device=x.device)
    for e in range(s["experts"]):
        at = torch.nonzero(ids == e)
        if at.shape[0] == 0:
            continue
        rows = at[:, 0].to(x.device)
        gate = x[rows] @ _exact_weight(s["gate"], e * i, (e + 1) * i).t()
        up = x[rows] @ _exact_weight(s["up"], e * i, (e + 1) * i).t()
        out = (gate * torch.sigmoid(gate) * up) @ _exact_weight(s["down"], e * h, (e + 1) * h).t()
        y[rows] += weights[at[:, 0], at[:, 1]].to(x.device).unsqueeze(1) * out
    return {"ids": ids.to(x.device), "weights": weights.to(x.device), "y": y}


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "lora":
        return _exact_lora(s)
    if case["op"] == "experts":
        return _exact_experts(s)
    ids, weights = _exact_route(s)
    return ids.to(s["route"].device), weights.to(s["route"].device)
