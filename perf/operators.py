"""The operators around an adapted mixture-of-experts layer, and what is measured of them.

route    routing logits -> the chosen experts and their weights
group    (token, choice) pairs sorted by expert: offsets, gather and scatter indices, adapter slots
quantise rows -> 4-bit elements with a scale for each 32 (MXFP4), optionally gathered or after SwiGLU, and back
linear   product of MXFP4 rows with an MXFP4 weight (a base projection)
experts  the same over rows sorted by expert, each block with its expert's weight
combine  weighted sum of each token's expert rows
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token decoding through the routed layer (128 experts, top-8): latency
        dict(name="route one token", op="route", T=1, E=128, k=8, score="softmax", bias=False, G=1, g=1, pair=False,
             renorm=True, scale=1.0, dtype="bf16"),
        # a long prompt, many experts, balance bias, groups: the whole selection
        dict(name="route prompt", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, G=8, g=4, pair=True,
             renorm=True, scale=2.5, dtype="bf16"),
        # a decode batch of 37 requests
        dict(name="group decode", op="group", T=37, E=128, k=8, slots=4, pad=0.0),
        # a padded prefill batch: tokens behind the requests' ends chose nothing
        dict(name="group prompt", op="group", T=16384, E=256, k=8, slots=16, pad=0.05),
        # the hidden states of a decode batch before a base projection
        dict(name="quantise decode", op="quantise", rows=37, F=4096, gather=0, silu=False, dtype="bf16"),
        # each of 2048 tokens copied to its 8 experts' blocks, bf16 for the adapters and 4 bits for the product
        dict(name="quantise gathered", op="quantise", rows=16384, F=2048, gather=8, silu=False, dtype="bf16"),
        # one token through a fused gate and up projection
        dict(name="linear one token", op="linear", rows=1, K=4096, N=28672, dtype="bf16"),
        # a prompt through it
        dict(name="linear prompt", op="linear", rows=8192, K=4096, N=28672, dtype="bf16"),
        # a decode batch through the experts' gate and up: mostly one or two rows an expert
        dict(name="experts decode", op="experts", T=32, k=8, E=128, K=2048, N=1536, dtype="bf16"),
        # a prompt through the same experts, ragged blocks from a few rows to a thousand
        dict(name="experts prompt", op="experts", T=2048, k=8, E=128, K=2048, N=1536, dtype="bf16"),
        # a decode batch back from its experts
        dict(name="combine decode", op="combine", T=37, k=8, F=2048, residual=False, dtype="bf16"),
        # a prompt, with the residual stream added
        dict(name="combine prompt", op="combine", T=8192, k=8, F=2048, residual=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "group", "quantise", "linear", "experts", "combine"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256, 384, 512])
        k = rng.randint(1, min(E, 10))
        T = _log(rng, 1, 4194304 // E)
        G, g = 1, 1
        if E % 8 == 0 and rng.random() < 0.5:
            G = rng.choice([2, 4, 8])
            g = rng.randint(-(-k * G // E), G)
        return dict(op=op, T=T, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, G=G, g=g,
                    pair=E // G > 1 and rng.random() < 0.5, renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 1.0, 2.5]), dtype=dtype)
    if op == "group":
        k = rng.randint(1, 8)
        return dict(op=op, T=_log(rng, 1, 131072 // k), E=rng.choice([8, 60, 64, 128, 256, 512]), k=k,
                    slots=rng.choice([1, 4, 16, 64]), pad=rng.choice([0.0, 0.0, 0.1]))
    if op == "quantise":
        F = 32 * _log(rng, 2, 448)
        rows = _log(rng, 1, 33554432 // F)
        return dict(op=op, rows=rows, F=F, gather=rng.choice([0, 0, 1, 8]), silu=rng.random() < 0.3, dtype=dtype)
    if op == "linear":
        K, N = 32 * _log(rng, 4, 448), 8 * _log(rng, 16, 3584)
        return dict(op=op, rows=_log(rng, 1, max(1, min(8192, 400_000_000_000 // (K * N)))), K=K, N=N, dtype=dtype)
    if op == "experts":
        K, N = 32 * _log(rng, 4, 128), 8 * _log(rng, 8, 512)
        E = rng.choice([8, 16, 60, 64, 128])
        while E * K * N > 420_000_000:
            N = 8 * (N // 16)
        k = rng.randint(1, min(8, E))
        return dict(op=op, T=_log(rng, 1, 16384 // k), k=k, E=E, K=K, N=N, dtype=dtype)
    F = 8 * _log(rng, 8, 1024)
    k = rng.randint(1, 8)
    return dict(op=op, T=_log(rng, 1, max(1, 134217728 // (F * k))), k=k, F=F, residual=rng.random() < 0.5, dtype=dtype)


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------

def _randn(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * std


def _popularity(E):
    """How often each expert is asked for: a few are hot, most are not."""
    p = 1.0 / (torch.arange(E, dtype=torch.float64) + 0.1 * E + 1)
    return p / p.sum()


def _choices(gen, T, E, k):
    """k distinct experts for each token, with that popularity, which expert has which rank by chance."""
    order = torch.randperm(E, generator=gen, device="cuda")
    logp = _popularity(E).log().to("cuda", torch.float32)[order]
    noise = torch.rand(T, E, generator=gen, device="cuda").clamp_min(1e-20)
    return torch.topk(logp - (-noise.log()).log(), k, dim=1).indices.to(torch.int32)


def _quantise(x):
    """Codes [rows, F / 2] (two elements a byte, the first in the low bits) and scales [rows, F / 32] (exponent + 127)."""
    v = x.float().unflatten(-1, (-1, 32))
    top = v.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
    a = torch.ldexp(v.abs(), -e)
    code = sum((a > m) if i % 2 == 0 else (a >= m) for i, m in [(0, 0.25), (1, 0.75), (2, 1.25), (3, 1.75), (4, 2.5),
                                                                (5, 3.5), (6, 5.0)])
    code = (code + 8 * torch.signbit(v)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, (e + 127).squeeze(-1).to(torch.uint8)


def _values(codes, scales):
    """What codes and scales stand for, in fp32."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2).unflatten(-1, (-1, 32))
    return torch.ldexp(v, (scales.int() - 127).unsqueeze(-1)).flatten(-2)


def _weight(gen, E, N, K):
    """An MXFP4 weight [E, N, K], as a checkpoint holds it."""
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, N, K // 32, dtype=torch.uint8, device="cuda")
    some = max(1, (1 << 25) // (N * K))
    for e in range(0, E, some):
        n = min(some, E - e)
        codes[e:e + n], scales[e:e + n] = _quantise(_randn(gen, n, N, K, std=K ** -0.5))
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)
    c, op, s = case, case["op"], dict(case=case)
    dtype = TYPES[c.get("dtype", "bf16")]
    i32 = dict(dtype=torch.int32, device="cuda")
    if op == "route":
        # logits of a trained router: a token's spread is a few units, experts differ in their mean
        s["logits"] = (_randn(gen, c["T"], c["E"], std=1.5) + _randn(gen, c["E"])).to(dtype)
        s["bias"] = _randn(gen, c["E"], std=0.1) if c["bias"] else None
        s["ids"] = torch.empty(c["T"], c["k"], **i32)
        s["weights"] = torch.empty(c["T"], c["k"], device="cuda")
    elif op == "group":
        s["ids"] = _choices(gen, c["T"], c["E"], c["k"])
        dead = int(c["T"] * c["pad"])
        if dead:
            s["ids"][c["T"] - dead:] = -1
        s["slot"] = torch.randint(-1, c["slots"], (c["T"],), generator=gen, device="cuda").to(torch.int32)
        rows = c["T"] * c["k"]
        s["offsets"] = torch.empty(c["E"] + 1, **i32)
        s["row_token"], s["pair_row"], s["row_slot"] = (torch.full((rows,), -1, **i32) for _ in range(3))
    elif op == "quantise":
        n = -(-c["rows"] // c["gather"]) if c["gather"] else c["rows"]
        s["x"] = _randn(gen, n, c["F"] * (2 if c["silu"] else 1)).to(dtype)
        s["index"] = None
        s["rows_out"] = torch.empty(c["rows"], c["F"], dtype=dtype, device="cuda") if c["gather"] or c["silu"] else None
        if c["gather"]:
            s["index"] = (torch.randperm(n * c["gather"], generator=gen, device="cuda")[:c["rows"]]
                          // c["gather"]).to(torch.int32)
        s["codes"] = torch.empty(c["rows"], c["F"] // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(c["rows"], c["F"] // 32, dtype=torch.uint8, device="cuda")
        s["values"] = torch.empty(c["rows"], c["F"], dtype=torch.bfloat16, device="cuda")
    elif op in ("linear", "experts"):
        rows = c["rows"] if op == "linear" else c["T"] * c["k"]
        s["x_codes"], s["x_scales"] = _quantise(_randn(gen, rows, c["K"]))
        s["w_codes"], s["w_scales"] = _weight(gen, c.get("E", 1), c["N"], c["K"])
        s["y"] = torch.empty(rows, c["N"], dtype=dtype, device="cuda")
        if op == "experts":
            count = torch.bincount(_choices(gen, c["T"], c["E"], c["k"]).flatten().long(), minlength=c["E"])
            s["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
            s["most"] = int(count.max())  # the plain form's room for an expert
    else:
        s["y"] = _randn(gen, c["T"] * c["k"], c["F"]).to(dtype)
        s["pair_row"] = torch.randperm(c["T"] * c["k"], generator=gen, device="cuda").to(torch.int32).view(-1, c["k"])
        s["weights"] = torch.softmax(_randn(gen, c["T"], c["k"]), -1)
        s["residual"] = _randn(gen, c["T"], c["F"]).to(dtype) if c["residual"] else None
        s["out"] = torch.empty(c["T"], c["F"], dtype=dtype, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s, s["case"])


def _best(c, k):
    """Indices of the k largest, ties to the lowest index."""
    return torch.sort(c, dim=-1, descending=True, stable=True).indices[..., :k]


def _route(s, c):
    x = s["logits"].double()  # the choice between scores next to each other
    if c["score"] == "softmax":
        p = (x - x.amax(-1, keepdim=True)).exp()
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1 / (1 + (-x).exp())
    key = p if s["bias"] is None else p + s["bias"].double()
    if c["G"] > 1:
        key = key.unflatten(-1, (c["G"], -1))
        high = key.amax(-1)
        if c["pair"]:
            high = high + torch.sort(key, dim=-1, descending=True).values[..., 1]
        kept = torch.zeros_like(high, dtype=torch.bool).scatter(-1, _best(high, c["g"]), True)
        key = torch.where(kept.unsqueeze(-1), key, -math.inf).flatten(-2)
    ids = _best(key, c["k"])
    w = p.gather(-1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _group(s, c):
    ids = s["ids"].flatten().long()
    rows = ids.numel()
    ids = torch.where(ids < 0, c["E"], ids)
    order = torch.sort(ids, stable=True).indices
    count = torch.zeros(c["E"] + 1, dtype=torch.int64, device=ids.device).scatter_add(0, ids, torch.ones_like(ids))
    offsets = torch.cat([count.new_zeros(1), count[:c["E"]].cumsum(0)])
    live = torch.arange(rows, device=ids.device) < offsets[-1]
    token = order // c["k"]
    pair_row = torch.empty_like(order)
    pair_row[order] = torch.where(live, torch.arange(rows, device=ids.device), -1)
    return (offsets.to(torch.int32), torch.where(live, token, -1).to(torch.int32), pair_row.to(torch.int32),
            torch.where(live, s["slot"].long()[token], -1).to(torch.int32))


def _rounded(x, dtype):
    """`x` in 64 bits, rounded once: what the step through 32 bits drops goes into their last bit."""
    f = x.float()
    back = f.double()
    bits = f.view(torch.int32) - (back.abs() > x.abs()).int()
    return torch.where(back != x, bits | 1, bits).view(torch.float32).to(dtype) if dtype != torch.float32 else f


def _quantise_rows(s, c):
    x = s["x"]
    if s["index"] is not None:
        x = x[s["index"].long()]
    if c["silu"]:
        gate, up = x[:, :c["F"]].double(), x[:, c["F"]:].double()  # it is rounded next to its borders
        x = _rounded(gate / (1 + (-gate).exp()) * up, x.dtype)
    return x if s["rows_out"] is not None else None, _values(*_quantise(x)).to(torch.bfloat16)


def _linear(s, c):
    x, w = _values(s["x_codes"], s["x_scales"]), _values(s["w_codes"][0], s["w_scales"][0])
    return (x @ w.T).to(s["y"].dtype)


def _experts(s, c):
    at = torch.arange(len(s["x_codes"]), device="cuda")
    expert = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    place = at - s["offsets"].long()[expert]
    x = torch.zeros(c["E"], s["most"], c["K"], device="cuda")
    x[expert, place] = _values(s["x_codes"], s["x_scales"])
    return torch.bmm(x, _values(s["w_codes"], s["w_scales"]).mT)[expert, place].to(s["y"].dtype)


def _combine(s, c):
    out = (s["y"].float()[s["pair_row"].long()] * s["weights"].unsqueeze(-1)).sum(1)
    return (out if s["residual"] is None else s["residual"].float() + out).to(s["out"].dtype)


_plain = {"route": _route, "group": _group, "quantise": _quantise_rows, "linear": _linear, "experts": _experts,
          "combine": _combine}


def _own_route(s, c):
    from adapter_lora_serving_b200 import lora as L
    L.lora_route_experts(s["logits"], s["bias"], s["ids"], s["weights"], c["T"], c["E"], c["k"],
                         score=L.LORA_SCORE_SOFTMAX if c["score"] == "softmax" else L.LORA_SCORE_SIGMOID,
                         num_groups=c["G"], top_groups=c["g"],
                         group_score=L.LORA_GROUP_TOP_PAIR if c["pair"] else L.LORA_GROUP_MAX,
                         renormalize=c["renorm"], scale=c["scale"])
    return s["ids"], s["weights"]


def _own_group(s, c):
    from adapter_lora_serving_b200 import lora as L
    L.lora_group_experts(s["ids"], s["slot"], s["offsets"], s["row_token"], s["pair_row"], s["row_slot"], c["T"],
                         c["k"], c["E"])
    return s["offsets"], s["row_token"], s["pair_row"], s["row_slot"]


def _own_quantise(s, c):
    from adapter_lora_serving_b200 import lora as L
    L.lora_mx_quantize(s["x"], s["codes"], s["scales"], c["rows"], c["F"], row_index=s["index"],
                       activation=L.LORA_ACT_SILU_MUL if c["silu"] else L.LORA_ACT_NONE, rows_out=s["rows_out"])
    L.lora_mx_dequantize(s["codes"], s["scales"], s["values"], c["rows"], c["F"])
    return s["rows_out"], s["values"]


def _own_linear(s, c):
    from adapter_lora_serving_b200 import lora as L
    L.lora_mx_linear(s["x_codes"], s["x_scales"], s["w_codes"], s["w_scales"], s["y"], c["rows"], c["K"], c["N"])
    return s["y"]


def _own_experts(s, c):
    from adapter_lora_serving_b200 import lora as L
    L.lora_mx_expert_linear(s["x_codes"], s["x_scales"], s["w_codes"], s["w_scales"], s["offsets"], s["y"],
                            c["T"] * c["k"], c["K"], c["N"], c["E"])
    return s["y"]


def _own_combine(s, c):
    from adapter_lora_serving_b200 import lora as L
    L.lora_combine_experts(s["y"], s["pair_row"], s["weights"], s["residual"], s["out"], c["T"], c["k"],
                           c["T"] * c["k"], c["F"])
    return s["out"]


_own = {"route": _own_route, "group": _own_group, "quantise": _own_quantise, "linear": _own_linear,
        "experts": _own_experts, "combine": _own_combine}


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without, and its exact result
# ---------------------------------------------------------------------------------------------------------------------

def work(case):
    c, op = case, case["op"]
    size = 4 if c.get("dtype") == "f32" else 2
    if op == "route":
        return {"bytes": c["T"] * c["E"] * size + 4 * c["E"] * c["bias"] + 8 * c["T"] * c["k"], "flops": 0}
    if op == "group":
        return {"bytes": 4 * (c["T"] * (4 * c["k"] + 1) + c["E"] + 1), "flops": 0}
    if op == "quantise":
        # the values come back from the codes, so the codes and scales are written and read
        n = -(-c["rows"] // c["gather"]) if c["gather"] else c["rows"]
        kept = size if c["gather"] or c["silu"] else 0
        return {"bytes": n * c["F"] * size * (2 if c["silu"] else 1) + 4 * c["rows"] * (c["gather"] > 0)
                + c["rows"] * c["F"] * (2 * (1 / 2 + 1 / 32) + 2 + kept), "flops": 0}
    if op in ("linear", "experts"):
        rows, weights = c.get("rows", c.get("T", 0) * c.get("k", 0)), 1.0
        if op == "experts":  # those that some row is sent to
            weights = float((1 - (1 - (c["k"] * _popularity(c["E"])).clamp_max(1)) ** c["T"]).sum())
        return {"bytes": (rows + weights * c["N"]) * c["K"] * (1 / 2 + 1 / 32) + rows * c["N"] * size,
                "flops": 2 * rows * c["N"] * c["K"]}
    return {"bytes": c["T"] * c["F"] * size * (c["k"] + 1 + c["residual"]) + 8 * c["T"] * c["k"], "flops": 0}


def _decode(codes, scales):
    """Sign, exponent and fraction of each element, and its block's exponent, in 64 bits."""
    at = torch.arange(2 * codes.shape[-1], device=codes.device)
    b = (codes[..., at // 2] >> (4 * (at % 2)).to(torch.uint8) & 15).long()
    e, m = b >> 1 & 3, (b & 1).double()
    v = torch.where(e > 0, (1 + m / 2) * 2.0 ** (e - 1).double(), m / 2) * (1 - 2 * (b >> 3).double())
    return v * 2.0 ** (scales.double() - 127).repeat_interleave(32, -1)


def _nearest(x):
    """`x` in 64 bits as MXFP4 holds it: the nearest of the elements' values, in even steps where two are as near."""
    v = x.unflatten(-1, (-1, 32))
    top = v.abs().amax(-1, keepdim=True)
    unit = 2.0 ** (torch.floor(torch.log2(top.clamp_min(2.0 ** -125))) - 2)
    a = (v / unit).abs().clamp_max(6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step * unit * torch.sign(v)).flatten(-2)


def exact(case, seed):
    c, op, s = case, case["op"], prepare(case, seed)
    if op == "route":
        x = s["logits"].double()
        p = torch.sigmoid(x) if c["score"] == "sigmoid" else (x - torch.logsumexp(x, -1, keepdim=True)).exp()
        key = p + (0 if s["bias"] is None else s["bias"].double())
        if c["G"] > 1:
            n = c["E"] // c["G"]
            high = torch.topk(key.view(-1, c["G"], n), 2 if c["pair"] else 1).values.sum(-1)
            out = torch.argsort(torch.argsort(-high, dim=-1, stable=True), dim=-1) >= c["g"]
            key = key.masked_fill(out.repeat_interleave(n, -1), -math.inf)
        ids = torch.argsort(-key, dim=-1, stable=True)[:, :c["k"]]
        w = torch.take_along_dim(p, ids, -1)
        return ids.to(torch.int32), (w / w.sum(-1, keepdim=True) if c["renorm"] else w) * c["scale"]
    if op == "group":
        return None
    if op == "quantise":
        x = s["x"].double()
        x = x[s["index"].long()] if s["index"] is not None else x
        if c["silu"]:
            x = x[:, :c["F"]] * torch.sigmoid(x[:, :c["F"]]) * x[:, c["F"]:]
        held = x
        if c["silu"]:  # rounded to the type that holds it, to the nearest of its steps
            kept = torch.finfo(s["x"].dtype)
            step = 2.0 ** torch.floor(torch.log2(x.abs().clamp_min(kept.smallest_normal))) * kept.eps
            held = torch.round(x / step) * step
        return x if s["rows_out"] is not None else None, _nearest(held)
    if op == "linear":
        return _decode(s["x_codes"], s["x_scales"]) @ _decode(s["w_codes"][0], s["w_scales"][0]).T
    if op == "experts":
        y = torch.empty(len(s["y"]), c["N"], dtype=torch.float64, device="cuda")
        at = s["offsets"].tolist()
        for e in range(c["E"]):
            if at[e] < at[e + 1]:
                x = _decode(s["x_codes"][at[e]:at[e + 1]], s["x_scales"][at[e]:at[e + 1]])
                y[at[e]:at[e + 1]] = x @ _decode(s["w_codes"][e], s["w_scales"][e]).T
        return y
    out = torch.zeros(c["T"], c["F"], dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        out += s["weights"][:, j:j + 1].double() * s["y"][s["pair_row"][:, j].long()].double()
    return out if s["residual"] is None else out + s["residual"].double()
