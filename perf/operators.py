"""Cases of the serving-step operators, each in its plain form and as a call of the library.

Four operators of one decoder layer served in NVFP4:

  route      the experts of every token and their weights, from router logits
  moe        a whole mixture-of-experts layer (gate, up, SiLU * up, down, weighted sum) for a few tokens
             with bf16 activations and NVFP4 expert weights
  lora_down  d = x @ A[adapter]^T, the low-rank input product of many requests' adapters
  gemm_lora  a shared NVFP4 projection with every request's d @ B[adapter]^T and a bias added

`listed()` gives named cases, `draw()` more of the same ranges, `prepare()` the tensors a program holds,
`run()` one pass, `work()` the bytes and operations of a pass, `exact()` the outputs in 64 bits.
"""
import math

import torch

own = False

FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
SOFTMAX, SOFTMAX_SELECTED, SIGMOID = 0, 1, 2


# ---- cases ------------------------------------------------------------------------------------------


def listed():
    return [
        # the router of one decode step of a small batch
        {"name": "route_decode", "op": "route", "t": 32, "experts": 128, "topk": 8, "weighting": SOFTMAX_SELECTED,
         "bf16": False, "masked": 0},
        # the router over a prefill chunk, bf16 logits, a few experts switched off
        {"name": "route_prefill", "op": "route", "t": 8192, "experts": 256, "topk": 8, "weighting": SOFTMAX,
         "bf16": True, "masked": 5},
        # one token of a model with many narrow experts: latency
        {"name": "moe_one_token", "op": "moe", "t": 1, "experts": 128, "topk": 8, "k": 2048, "n": 768, "padded": 0},
        # a small ragged call: odd numbers of tokens and experts, two padded tokens
        {"name": "moe_ragged", "op": "moe", "t": 7, "experts": 5, "topk": 3, "k": 320, "n": 192, "padded": 2},
        # the routed experts at the repository's own sizes, a small decode batch
        {"name": "moe_wide_experts", "op": "moe", "t": 8, "experts": 16, "topk": 2, "k": 5120, "n": 8192, "padded": 0},
        # the largest batch: every expert has several tokens
        {"name": "moe_full_batch", "op": "moe", "t": 64, "experts": 64, "topk": 6, "k": 2048, "n": 1408, "padded": 0},
        # decode: every row another request, most with an adapter of their own
        {"name": "lora_down_decode", "op": "lora_down", "m": 48, "k": 5120, "r": 16, "adapters": 40, "run": 1},
        # a chunk of prefill rows, long runs of one request
        {"name": "lora_down_prefill", "op": "lora_down", "m": 4096, "k": 5120, "r": 64, "adapters": 8, "run": 700},
        # one row, one adapter: latency
        {"name": "gemm_lora_one_row", "op": "gemm_lora", "m": 1, "n": 5120, "k": 5120, "r": 16, "adapters": 4, "run": 1,
         "bias": False},
        {"name": "gemm_lora_decode", "op": "gemm_lora", "m": 48, "n": 7168, "k": 5120, "r": 16, "adapters": 40, "run": 1,
         "bias": True},
        # prefill rows of several requests beside decode rows: ragged m, runs that end inside a tile
        {"name": "gemm_lora_prefill", "op": "gemm_lora", "m": 2011, "n": 8192, "k": 5120, "r": 32, "adapters": 12,
         "run": 300, "bias": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log_multiple(rng, lo, hi, of):
    return min(hi, max(of, (_log(rng, lo, hi) + of // 2) // of * of))


def draw(rng):
    op = rng.choice(("route", "moe", "moe", "lora_down", "gemm_lora", "gemm_lora"))
    if op == "route":
        experts = _log(rng, 2, 512)
        return {"op": op, "t": _log(rng, 1, 8192), "experts": experts, "topk": rng.randint(1, min(16, experts)),
                "weighting": rng.randint(0, 2), "bf16": rng.random() < 0.5,
                "masked": rng.randint(0, min(6, experts - 1))}
    if op == "moe":
        k, n = _log_multiple(rng, 128, 5120, 64), _log_multiple(rng, 128, 8192, 64)
        experts = _log(rng, 2, min(128, max(2, (1 << 29) // (k * n))))
        t = _log(rng, 1, 64)
        return {"op": op, "t": t, "experts": experts, "topk": rng.randint(1, min(8, experts)), "k": k, "n": n,
                "padded": rng.randint(0, t // 4)}
    m = _log(rng, 1, 4096) if op == "lora_down" else _log(rng, 1, 2048)
    case = {"op": op, "m": m, "k": _log_multiple(rng, 128, 5120, 64), "r": 8 * _log(rng, 1, 16),
            "adapters": _log(rng, 1, 48), "run": _log(rng, 1, max(1, m))}
    if op == "gemm_lora":
        case["n"] = _log_multiple(rng, 64, 8192, 8)
        case["bias"] = rng.random() < 0.5
    return case


# ---- inputs -----------------------------------------------------------------------------------------


def _generator(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + salt) & 0x7FFFFFFFFFFF)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _swizzle(scales):
    """[rows, blocks] scale bytes -> the 128x4 layout: 512-byte chunks of 128 rows x 4 blocks."""
    rows, blocks = scales.shape
    rp, bp = -(-rows // 128) * 128, -(-blocks // 4) * 4
    full = torch.zeros((rp, bp), dtype=torch.uint8, device="cuda")
    full[:rows, :blocks] = scales
    return full.view(rp // 128, 4, 32, bp // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _quantize(w):
    """fp32 [rows, k] -> packed e2m1 codes, swizzled ue4m3 block scales, amax: NVFP4 as the quantizer makes it."""
    rows, k = w.shape
    amax = w.abs().max()
    gsf = 2688.0 / amax
    blocks = w.view(rows, k // 16, 16)
    s8 = (blocks.abs().amax(-1) / 6.0 * gsf).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()
    y = blocks * torch.where(s > 0, gsf / s, torch.zeros_like(s))[..., None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    codes = (torch.bucketize(y.abs(), edges) + 8 * (y < 0)).to(torch.uint8).view(rows, k)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), _swizzle(s8.view(torch.uint8)), amax


def _expert_weights(g, experts, rows, k):
    """Weights ~ N(0, 0.02), another spread for each expert: codes, scales and amax stacked over the experts."""
    made = [_quantize(_normal(g, rows, k) * (0.02 * (0.75 + 0.5 * (e % 5) / 4))) for e in range(experts)]
    return torch.stack([q for q, _, _ in made]), torch.stack([s for _, s, _ in made]), torch.stack([a for _, _, a in made])


def _adapters(g, m, adapters, run):
    """One adapter index a row in runs of about `run` rows (a request's rows are adjacent); about one run in six has none (-1)."""
    runs = -(-m // run) + 1
    ids = torch.randint(0, adapters, (runs,), generator=g, device="cuda", dtype=torch.int32)
    ids = torch.where(torch.rand(runs, generator=g, device="cuda") < 1 / 6, torch.full_like(ids, -1), ids)
    start = torch.randint(0, run, (1,), generator=g, device="cuda")
    return ids[(torch.arange(m, device="cuda") + start) // run].contiguous()


def _activations(g, m, k):
    """N(0, 1) with some channels that are much larger, as hidden states have."""
    x = _normal(g, m, k)
    loud = torch.rand(k, generator=g, device="cuda") < 0.002
    return torch.where(loud[None, :], x * 30.0, x)


def prepare(case, seed):
    c, op = case, case["op"]
    g = _generator(seed, 11)
    s = {"case": dict(c), "op": op}
    if op == "route":
        logits = _normal(g, c["t"], c["experts"]) * 1.5
        if c["masked"]:
            off = torch.rand(c["t"], c["experts"], generator=g, device="cuda").argsort(-1)[:, : c["masked"]]
            logits.scatter_(1, off, float("-inf"))
        s["logits"] = logits.to(torch.bfloat16) if c["bf16"] else logits
    elif op == "moe":
        t, E, topk, k, n = c["t"], c["experts"], c["topk"], c["k"], c["n"]
        s["x"] = _activations(g, t, k).to(torch.bfloat16)
        # some experts are asked for more often than others
        score = _normal(g, t, E) + 0.5 * _normal(g, 1, E)
        top = score.topk(topk, dim=-1)
        s["ids"] = top.indices.to(torch.int32).contiguous()
        s["weights"] = torch.softmax(top.values, dim=-1).contiguous()
        if c["padded"]:
            s["ids"][t - c["padded"]:] = -1
        s["gate"], s["gate_sf"], s["gate_amax"] = _expert_weights(g, E, n, k)
        s["up"], s["up_sf"], s["up_amax"] = _expert_weights(g, E, n, k)
        s["down"], s["down_sf"], s["down_amax"] = _expert_weights(g, E, k, n)
    elif op == "lora_down":
        s["x"] = _activations(g, c["m"], c["k"]).to(torch.bfloat16)
        s["w"] = (_normal(g, c["adapters"], c["r"], c["k"]) / math.sqrt(c["k"])).to(torch.bfloat16)
        s["adapter"] = _adapters(g, c["m"], c["adapters"], c["run"])
    else:
        s["a"], s["a_sf"], amax_a = _quantize(_activations(g, c["m"], c["k"]))
        s["b"], s["b_sf"], amax_b = _quantize(_normal(g, c["n"], c["k"]) * 0.02)
        s["alpha"] = (amax_a.double() * amax_b.double() / 2688.0 ** 2).float().view(1)
        s["d"] = _normal(g, c["m"], c["r"]).to(torch.bfloat16)
        s["l1"] = (_normal(g, c["adapters"], c["n"], c["r"]) * (0.4 / math.sqrt(c["r"]))).to(torch.bfloat16)
        s["adapter"] = _adapters(g, c["m"], c["adapters"], c["run"])
        s["bias"] = (_normal(g, c["n"]) * 0.1).to(torch.bfloat16) if c["bias"] else None
    return s


# ---- one pass ---------------------------------------------------------------------------------------


def _unswizzle(sf, rows, blocks):
    rp, bp = -(-rows // 128) * 128, -(-blocks // 4) * 4
    full = sf.view(*sf.shape[:-1], rp // 128, bp // 4, 32, 4, 4)
    d = full.dim()
    return full.permute(*range(d - 5), d - 5, d - 2, d - 3, d - 4, d - 1).reshape(*sf.shape[:-1], rp, bp)[..., :rows, :blocks]


def _dequantize(q, sf):
    """Packed codes [..., rows, k/2] and swizzled scales [..., bytes] -> fp32 values [..., rows, k]."""
    rows, half = q.shape[-2:]
    pairs = torch.tensor([[FP4[b & 15], FP4[b >> 4]] for b in range(256)], device=q.device)[q.int()]
    scales = _unswizzle(sf, rows, half // 8).view(torch.float8_e4m3fn).float()
    return (pairs.view(*q.shape[:-1], half // 8, 16) * scales[..., None]).view(*q.shape[:-1], 2 * half)


def _route(logits, topk, weighting):
    x = logits.float()
    x = torch.where(x.isnan(), torch.full_like(x, float("-inf")), x).clamp(max=torch.finfo(torch.float32).max)
    order = x.sort(dim=-1, descending=True, stable=True)
    best, ids = order.values[:, :topk], order.indices[:, :topk].to(torch.int32)
    fine = best > float("-inf")
    if weighting == SIGMOID:
        w = 1.0 / (1.0 + torch.exp(-best))
    else:
        e = torch.exp(best - best[:, :1])
        total = torch.where(fine, e, torch.zeros_like(e)) if weighting == SOFTMAX_SELECTED else torch.exp(x - best[:, :1])
        w = e / total.sum(-1, keepdim=True)
    return torch.where(fine, ids, torch.full_like(ids, -1)), torch.where(fine, w, torch.zeros_like(w))


def _moe(s):
    E, t = s["gate"].shape[0], s["x"].shape[0]
    x = s["x"].float()
    ids = s["ids"].long()
    fine = (ids >= 0) & (ids < E)
    share = torch.zeros((t, E), device=x.device)
    share.scatter_add_(1, torch.where(fine, ids, 0), torch.where(fine, s["weights"], 0.0))
    g = torch.matmul(x, _dequantize(s["gate"], s["gate_sf"]).transpose(1, 2)) * (s["gate_amax"] / 2688.0)[:, None, None]
    u = torch.matmul(x, _dequantize(s["up"], s["up_sf"]).transpose(1, 2)) * (s["up_amax"] / 2688.0)[:, None, None]
    h = g / (1.0 + torch.exp(-g)) * u
    y = torch.matmul(h, _dequantize(s["down"], s["down_sf"]).transpose(1, 2)) * (s["down_amax"] / 2688.0)[:, None, None]
    return (y * share.t()[:, :, None]).sum(0).to(torch.bfloat16)


def _lora_down(x, w, adapter):
    A, r, k = w.shape
    every = torch.matmul(x.float(), w.float().view(A * r, k).t()).view(-1, A, r)
    fine = (adapter >= 0) & (adapter < A)
    at = torch.where(fine, adapter, 0).long()[:, None, None].expand(-1, 1, r)
    return torch.where(fine[:, None], every.gather(1, at)[:, 0], 0.0).to(torch.bfloat16)


def _gemm_lora(s):
    A, n, r = s["l1"].shape
    out = torch.matmul(_dequantize(s["a"], s["a_sf"]), _dequantize(s["b"], s["b_sf"]).t()) * s["alpha"]
    hot = (s["adapter"][:, None] == torch.arange(A, device=out.device)[None, :]).float()
    spread = (hot[:, :, None] * s["d"].float()[:, None, :]).view(-1, A * r)
    out = out + torch.matmul(spread, s["l1"].float().transpose(1, 2).reshape(A * r, n))
    if s["bias"] is not None:
        out = out + s["bias"].float()
    return out.to(torch.bfloat16)


def run(state):
    s, op = state, state["op"]
    if own:
        import nvfp4_block_scaled_16_b200 as nv
        if op == "route":
            return nv.nvfp4_moe_route(s["logits"], s["case"]["topk"], s["case"]["weighting"])
        if op == "moe":
            return nv.nvfp4_moe_few_tokens(s["x"], s["ids"], s["weights"], s["gate"], s["up"], s["down"], s["gate_sf"],
                                           s["up_sf"], s["down_sf"], s["gate_amax"], s["up_amax"], s["down_amax"])
        if op == "lora_down":
            return nv.nvfp4_lora_down_batched(s["x"], s["w"], s["adapter"])
        return nv.nvfp4_gemm_lora_batched(s["a"], s["b"], s["a_sf"], s["b_sf"], s["alpha"], s["d"], s["l1"],
                                          s["adapter"], bias=s["bias"])
    if op == "route":
        return _route(s["logits"], s["case"]["topk"], s["case"]["weighting"])
    if op == "moe":
        return _moe(s)
    if op == "lora_down":
        return _lora_down(s["x"], s["w"], s["adapter"])
    return _gemm_lora(s)


# ---- what a pass cannot do without ------------------------------------------------------------------


def _fp4_bytes(rows, k):
    return rows * k / 2 + rows * k / 16


def _distinct(things, asked):
    """Expected number of distinct ones among `asked` picks of `things`."""
    return things * (1.0 - (1.0 - 1.0 / things) ** asked)


def work(case):
    c, op = case, case["op"]
    if op == "route":
        return {"bytes": c["t"] * (c["experts"] * (2 if c["bf16"] else 4) + 8 * c["topk"]), "flops": 2.0 * c["t"] * c["experts"]}
    if op == "moe":
        t, k, n = c["t"] - c["padded"], c["k"], c["n"]
        hit = min(c["experts"], max(c["topk"], c["experts"] * (1.0 - (1.0 - c["topk"] / c["experts"]) ** t)))
        return {"bytes": hit * (2 * _fp4_bytes(n, k) + _fp4_bytes(k, n)) + 4 * c["t"] * k + 8 * c["t"] * c["topk"],
                "flops": 2.0 * t * c["topk"] * 3 * n * k}
    used = _distinct(c["adapters"], max(1.0, c["m"] / c["run"] * 5 / 6))
    if op == "lora_down":
        return {"bytes": 2.0 * c["m"] * (c["k"] + c["r"]) + 4 * c["m"] + 2.0 * used * c["r"] * c["k"],
                "flops": 2.0 * c["m"] * c["k"] * c["r"]}
    return {"bytes": _fp4_bytes(c["m"], c["k"]) + _fp4_bytes(c["n"], c["k"]) + 2.0 * c["m"] * (c["n"] + c["r"]) + 4 * c["m"]
            + 2.0 * used * c["n"] * c["r"], "flops": 2.0 * c["m"] * c["n"] * (c["k"] + c["r"])}


# ---- the definitions in 64 bits ---------------------------------------------------------------------


def _values64(q, sf):
    """One matrix's values code by code: sign, exponent and mantissa of e2m1, the scale of row r and block b at its chunk's place."""
    rows, half = q.shape
    codes = torch.stack((q & 15, q >> 4), -1).view(rows, 2 * half).long()
    exponent, odd = (codes >> 1) & 3, (codes & 1).double()
    size = torch.where(exponent == 0, 0.5 * odd, (1.0 + 0.5 * odd) * 2.0 ** (exponent - 1).double())
    value = torch.where(codes >= 8, -size, size)
    r = torch.arange(rows, device=q.device)[:, None]
    b = torch.arange(half // 8, device=q.device)[None, :]
    groups = -(-(half // 8) // 4)
    byte = sf[((r // 128) * groups + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4].long()
    e, f = byte >> 3, (byte & 7).double()
    scale = torch.where(e == 0, f / 8 * 2.0 ** -6, (1.0 + f / 8) * 2.0 ** (e - 7).double())
    return value * scale.repeat_interleave(16, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "route":
        x, topk = s["logits"].double(), case["topk"]
        x[x.isnan()] = float("-inf")
        ids = torch.full((case["t"], topk), -1, dtype=torch.int32, device="cuda")
        w = torch.zeros((case["t"], topk), dtype=torch.float64, device="cuda")
        left = x.clone()
        top = x.max(-1, keepdim=True).values
        for j in range(topk):
            best = left.max(-1, keepdim=True).values
            at = (left == best).double().argmax(-1)  # the first of equals
            ok = best[:, 0] > float("-inf")
            ids[:, j] = torch.where(ok, at.int(), -1)
            value = torch.sigmoid(best[:, 0]) if case["weighting"] == SIGMOID else torch.exp(best - top)[:, 0]
            w[:, j] = torch.where(ok, value, 0.0)
            left.scatter_(1, at[:, None], float("-inf"))
        if case["weighting"] != SIGMOID:
            total = torch.exp(x - top).sum(-1) if case["weighting"] == SOFTMAX else w.sum(-1)
            w = torch.where(w > 0, w / total[:, None], 0.0)
        return ids, w
    if op == "moe":
        x, out = s["x"].double(), torch.zeros(case["t"], case["k"], dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            at, slot = (s["ids"] == e).nonzero(as_tuple=True)
            if not at.numel():
                continue
            g = x[at] @ _values64(s["gate"][e], s["gate_sf"][e]).t() * (s["gate_amax"][e].double() / 2688)
            u = x[at] @ _values64(s["up"][e], s["up_sf"][e]).t() * (s["up_amax"][e].double() / 2688)
            y = (g * torch.sigmoid(g) * u) @ _values64(s["down"][e], s["down_sf"][e]).t() * (s["down_amax"][e].double() / 2688)
            out.index_add_(0, at, y * s["weights"][at, slot].double()[:, None])
        return out
    if op == "lora_down":
        d = torch.zeros(case["m"], case["r"], dtype=torch.float64, device="cuda")
        for a in range(case["adapters"]):
            at = (s["adapter"] == a).nonzero()[:, 0]
            d[at] = s["x"][at].double() @ s["w"][a].double().t()
        return d
    out = _values64(s["a"], s["a_sf"]) @ _values64(s["b"], s["b_sf"]).t() * s["alpha"].double()
    for a in range(case["adapters"]):
        at = (s["adapter"] == a).nonzero()[:, 0]
        out[at] += s["d"][at].double() @ s["l1"][a].double().t()
    return out + s["bias"].double() if s["bias"] is not None else out
