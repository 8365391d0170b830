"""Measured cases of four operators of the routed-MoE library: routing from logits with expert groups, the dense
8-bit integer product, and the grouped gate/up and down projections with 8-bit integer experts.

Each case has a plain form (elementary torch operations, ``own`` false) and the library's call (``own`` true).
Sizes are the layer's workloads (H = 7168, I = 2048, E = 256, top_k = 16; 8 to 2048 tokens) and ranges around them.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step: 8 sequences, 256 experts in 8 groups of which 4 stay, a balance bias on the scores
        _route("route_decode_m8", 8, 8, 32, 4, 8, "sigmoid", "top2", True, 2.5, True, "fp32"),
        # the prefill workload's routing from a gate that leaves bf16 logits (ties), groups by their best expert
        _route("route_prefill_m2048_bf16", 2048, 8, 32, 3, 16, "softmax", "max", False, 1.0, False, "bf16"),
        # a long prompt batch, no power of two of tokens
        _route("route_m32767", 32767, 8, 32, 4, 8, "sigmoid", "top2", True, 2.5, True, "fp32"),
        # the up projection of a shared expert for one token
        _linear("linear_m1", 1, 2048, 7168, "bf16", 0),
        # odd sizes throughout, rows of x taken out of a wider buffer, fp32 results
        _linear("linear_m1000_ragged", 1000, 4099, 1777, "fp32", 24),
        # a full-width projection of a long prompt
        _linear("linear_m8192", 8192, 7168, 7168, "bf16", 0),
        # gate/up of the decode, batch and skewed prefill workloads
        _experts("up_decode_m8", "up", 8, 7168, 2048, 256, 16, 16, 0.0),
        _experts("up_batch_m512", "up", 512, 7168, 2048, 256, 16, 64, 0.0),
        _experts("up_prefill_m2048_zipf", "up", 2048, 7168, 2048, 256, 16, 128, 0.44),
        # down for one token, for the 1000-token decode batch and for the skewed prefill
        _experts("down_decode_m1", "down", 1, 7168, 2048, 256, 16, 16, 0.0),
        _experts("down_m1000", "down", 1000, 7168, 2048, 256, 16, 16, 0.0),
        _experts("down_prefill_m2048_zipf", "down", 2048, 7168, 2048, 256, 16, 128, 0.44),
    ]


def _route(name, M, groups, group_size, keep, K, scoring, group_score, bias, scale, renorm, logits):
    return dict(name=name, op="route", M=M, groups=groups, group_size=group_size, keep=keep, K=K, scoring=scoring,
                group_score=group_score, bias=bias, scale=scale, renorm=renorm, logits=logits)


def _linear(name, M, N, K, out, pad):
    return dict(name=name, op="linear", M=M, N=N, K=K, out=out, pad=pad)


def _experts(name, op, M, H, I, E, K, B, skew):
    return dict(name=name, op=op, M=M, H=H, I=I, E=E, K=K, B=B, skew=skew)


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "linear", "up", "down"])
    if op == "route":
        groups = rng.choice([1, 2, 4, 8, 16, 5])
        group_size = _log(rng, 2, 1024 // groups)
        keep = rng.randint(1, groups)
        c = _route("", _log(rng, 1, 32767), groups, group_size, keep, rng.randint(1, min(32, keep * group_size)),
                   rng.choice(["sigmoid", "softmax"]), rng.choice(["top2", "max"]), rng.random() < 0.7,
                   rng.choice([1.0, 2.5]), rng.random() < 0.5, rng.choice(["fp32", "bf16"]))
    elif op == "linear":
        c = _linear("", _log(rng, 1, 8192), _log(rng, 16, 7168), _log(rng, 32, 7168), rng.choice(["bf16", "fp32"]),
                    rng.choice([0, 1, 8, 40]))
    else:
        E = _log(rng, 1, 256)
        c = _experts("", op, _log(rng, 1, 2048), 256 * rng.randint(1, 28), 128 * rng.randint(1, 16), E,
                     rng.randint(1, min(E, 16)), rng.choice([16, 32, 64, 128]), rng.choice([0.0, 0.44]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return {"route": _prepare_route, "linear": _prepare_linear, "up": _prepare_experts,
            "down": _prepare_experts}[case["op"]](case, g)


def _randn(g, *size):
    return torch.randn(*size, generator=g, device=DEV)


def _prepare_route(c, g):
    E = c["groups"] * c["group_size"]
    z = _randn(g, c["M"], E)  # x . w_router with w_router ~ N(0, 1/H)
    return dict(case=c, logits=z.to(torch.bfloat16) if c["logits"] == "bf16" else z,
                bias=0.05 * _randn(g, E) if c["bias"] else None)


def _codes(g, rows, cols, pitch):
    """int8 codes of N(0, 1) rows whose largest magnitude is about 4, in rows of `pitch` bytes, and their scales."""
    codes = torch.zeros(rows, pitch, dtype=torch.int8, device=DEV)
    step = max(1, (1 << 27) // pitch)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        codes[r:r + n, :cols] = (32.0 * _randn(g, n, cols)).round_().clamp_(-127, 127).to(torch.int8)
    scales = (1.0 + 0.1 * torch.rand(rows, generator=g, device=DEV)) / (32.0 * math.sqrt(cols))
    return codes[:, :cols], scales


def _prepare_linear(c, g):
    x = _randn(g, c["M"], c["K"] + c["pad"]).to(torch.bfloat16)[:, :c["K"]]
    codes, scales = _codes(g, c["N"], c["K"], (c["K"] + 15) // 16 * 16)
    return dict(case=c, x=x, codes=codes, scales=scales)


def _plan(ids, E, B):
    """The expert-major plan of the routed ids: every expert's slots in ascending order, padded to B rows; and, for
    the real rows in that order, their plan row, slot, expert and place within the expert."""
    M, K = ids.shape
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat, minlength=E)
    padded = (counts + B - 1) // B * B
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    slot = torch.argsort(flat, stable=True)
    expert = flat[slot]
    place = torch.arange(M * K, device=DEV) - (counts.cumsum(0) - counts)[expert]
    row = offsets[:-1][expert] + place
    cap = M * K + E * (B - 1)
    sorted_ids = torch.full((cap,), M * K, dtype=torch.int32, device=DEV)
    sorted_ids[row] = slot.int()
    block_expert = torch.zeros(cap // B + 1, dtype=torch.int32, device=DEV)
    of_block = torch.repeat_interleave(torch.arange(E, device=DEV), padded // B)
    block_expert[:of_block.numel()] = of_block.int()
    plan = dict(sorted_ids=sorted_ids, block_expert=block_expert, expert_counts=counts.int(),
                expert_offsets=offsets.int(), num_tokens_post_padded=offsets[-1:].int())
    return plan, dict(row=row, slot=slot, expert=expert, place=place, most=int(counts.max()), cap=cap)


def _prepare_experts(c, g):
    M, H, I, E, K = (c[k] for k in ("M", "H", "I", "E", "K"))
    rank = torch.randperm(E, generator=g, device=DEV).float() + 1.0
    ids = (_randn(g, M, E) - c["skew"] * torch.log(rank)).topk(K, dim=1).indices
    plan, rows = _plan(ids, E, c["B"])
    s = dict(case=c, plan=plan, rows=rows)
    if c["op"] == "up":
        s["x"] = _randn(g, M, H).to(torch.bfloat16)
        for w in ("gate", "up"):
            codes, scales = _codes(g, E * I, H, H)
            s[w], s[w + "_scales"] = codes.view(E, I, H), scales.view(E, I)
        s["h"] = torch.zeros(rows["cap"], I, dtype=torch.bfloat16, device=DEV)
    else:
        # h = silu(gate) * up of unit-variance projections; the plan's padding rows hold no numbers
        s["h"] = torch.full((rows["cap"], I), float("nan"), dtype=torch.bfloat16, device=DEV)
        a, b = _randn(g, M * K, I), _randn(g, M * K, I)
        s["h"][rows["row"]] = (a / (1.0 + torch.exp(-a)) * b).to(torch.bfloat16)
        codes, scales = _codes(g, E * H, I, I)
        s["down"], s["down_scales"] = codes.view(E, H, I), scales.view(E, H)
        s["y"] = torch.zeros(M * K, H, dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return {"route": _run_route, "linear": _run_linear, "up": _run_up, "down": _run_down}[state["case"]["op"]](state)


def _run_route(s):
    c = s["case"]
    if own:
        import prefill_sigmoid_top_b200 as moe
        return moe.route_logits(s["logits"], s["bias"], c["K"], n_group=c["groups"], topk_group=c["keep"],
                                group_score=moe.GROUP_TOP2 if c["group_score"] == "top2" else moe.GROUP_MAX,
                                scoring=moe.SCORE_SIGMOID if c["scoring"] == "sigmoid" else moe.SCORE_SOFTMAX,
                                renormalize=c["renorm"], routed_scale=c["scale"])
    # in 64 bits: the choice between two experts next to each other is a matter of the last bits
    z = s["logits"].double()
    if c["scoring"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-z))
    else:
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    key = p if s["bias"] is None else p + s["bias"].double()
    by_group = key.view(c["M"], c["groups"], c["group_size"])
    of_group = by_group.amax(2) if c["group_score"] == "max" else by_group.topk(2, dim=2).values.sum(2)
    kept = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
    out = torch.ones(c["M"], c["groups"], dtype=torch.bool, device=z.device).scatter_(1, kept, False)
    key = by_group.masked_fill(out[:, :, None], -math.inf).view(c["M"], -1)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["K"]]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.int(), (w * c["scale"]).float()


def _quantize(x):
    """Codes rint(127 x / amax) (ties to even; 127 x is exact in 32 bits) and scales amax / 127 of each row."""
    x = x.float()
    amax = x.abs().amax(1, keepdim=True)
    return torch.round(127.0 * x / amax.clamp_min(1e-30)), amax / 127.0


def _run_linear(s):
    out = torch.bfloat16 if s["case"]["out"] == "bf16" else torch.float32
    if own:
        import prefill_sigmoid_top_b200 as moe
        return moe.linear_int8(s["x"], s["codes"], s["scales"], out_dtype=out)
    xq, sx = _quantize(s["x"])
    return ((xq @ s["codes"].float().t()) * sx * s["scales"]).to(out)


def _product(s, xq, codes, scales):
    """The real plan rows' product with their expert's codes [E, n, k], times the channels' scales."""
    r = s["rows"]
    if xq.shape[0] <= codes.shape[0]:  # few rows: each with its expert's matrix
        y = torch.bmm(codes[r["expert"]].float(), xq[:, :, None]).squeeze(2)
    else:  # the experts' rows side by side, padded to the longest
        side = xq.new_zeros(codes.shape[0], r["most"], xq.shape[1])
        side[r["expert"], r["place"]] = xq
        y = torch.bmm(side, codes.float().transpose(1, 2))[r["expert"], r["place"]]
    return y * scales[r["expert"]]


def _shape(c):
    import prefill_sigmoid_top_b200 as moe
    return moe.Shape(c["M"], c["H"], c["I"], c["E"], c["K"], c["B"])


def _run_up(s):
    if own:
        import prefill_sigmoid_top_b200 as moe
        w = moe.Int8Weights(gate=s["gate"], up=s["up"], gate_scales=s["gate_scales"], up_scales=s["up_scales"])
        return moe.grouped_up_swiglu_int8(s["x"], w, s["plan"], _shape(s["case"]), h=s["h"])
    xq, sx = _quantize(s["x"])
    token = s["rows"]["slot"] // s["case"]["K"]
    xq, sx = xq[token], sx[token]
    gate = _product(s, xq, s["gate"], s["gate_scales"]) * sx
    up = _product(s, xq, s["up"], s["up_scales"]) * sx
    s["h"][s["rows"]["row"]] = (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16)
    return s["h"]


def _run_down(s):
    if own:
        import prefill_sigmoid_top_b200 as moe
        w = moe.Int8Weights(down=s["down"], down_scales=s["down_scales"])
        return moe.grouped_down_int8(s["h"], w, s["plan"], _shape(s["case"]), y=s["y"])
    hq, sh = _quantize(s["h"][s["rows"]["row"]])
    s["y"][s["rows"]["slot"]] = (_product(s, hq, s["down"], s["down_scales"]) * sh).to(torch.bfloat16)
    return s["y"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "route":
        E = c["groups"] * c["group_size"]
        return {"bytes": c["M"] * E * (4 if c["logits"] == "fp32" else 2) + 4 * E + 8 * c["M"] * c["K"],
                "flops": 8 * c["M"] * E}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": 2 * M * K + N * K + 4 * N + M * N * (2 if c["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    M, H, I, E, K = (c[k] for k in ("M", "H", "I", "E", "K"))
    used = E * (1.0 - (1.0 - K / E) ** M)  # experts that get a token, of evenly spread ones
    if c["op"] == "up":
        return {"bytes": used * 2 * I * (H + 4) + 2 * M * H + 2 * M * K * I, "flops": 4 * M * K * H * I}
    return {"bytes": used * H * (I + 4) + 2 * M * K * I + 2 * M * K * H, "flops": 2 * M * K * H * I}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "linear": _exact_linear, "up": _exact_up, "down": _exact_down}[case["op"]](s)


def _exact_route(s):
    c = s["case"]
    z = s["logits"].double()
    p = torch.softmax(z, 1) if c["scoring"] == "softmax" else torch.sigmoid(z)
    key = (p + s["bias"].double()) if s["bias"] is not None else p.clone()
    M, E = key.shape
    lowest = torch.arange(E, device=key.device)
    group = lowest // c["group_size"]
    scores = []
    for g in range(c["groups"]):
        best = torch.sort(key[:, group == g], dim=1).values
        scores.append(best[:, -1] if c["group_score"] == "max" else best[:, -1] + best[:, -2])
    scores = torch.stack(scores, 1)
    allowed = torch.zeros(M, E, dtype=torch.bool, device=key.device)
    for _ in range(c["keep"]):
        g = scores.argmax(1)  # the first of equal ones
        g = (scores == scores.gather(1, g[:, None])).int().argmax(1)
        scores[torch.arange(M, device=key.device), g] = -math.inf
        allowed |= group[None, :] == g[:, None]
    key[~allowed] = -math.inf
    ids = []
    for _ in range(c["K"]):
        e = (key == key.amax(1, keepdim=True)).int().argmax(1)
        ids.append(e)
        key[torch.arange(M, device=key.device), e] = -math.inf
    ids = torch.stack(ids, 1)
    w = torch.gather(p, 1, ids) * c["scale"]
    return ids.int(), w * (c["scale"] / w.sum(1, keepdim=True)) if c["renorm"] else w


def _values64(x):
    """The 64-bit values that the rows' 8-bit codes stand for."""
    x = x.double()
    top = x.abs().max(dim=1, keepdim=True).values
    return torch.where(top > 0, torch.round(x * 127 / top) * (top / 127), torch.zeros_like(x))


def _exact_linear(s):
    return _values64(s["x"]) @ (s["codes"].double() * s["scales"].double()[:, None]).T


def _exact_experts(s, x, names):
    """Per expert and weight: (plan rows, slots, [values of the rows . the expert's values^T])."""
    plan, K = s["plan"], s["case"]["K"]
    counts, offsets = plan["expert_counts"].tolist(), plan["expert_offsets"].tolist()
    for e, n in enumerate(counts):
        if n:
            rows = slice(offsets[e], offsets[e] + n)
            slots = plan["sorted_ids"][rows].long()
            a = x[slots // K] if s["case"]["op"] == "up" else _values64(x[rows])
            yield rows, slots, [a @ (s[w][e].double() * s[w + "_scales"][e].double()[:, None]).T for w in names]


def _exact_up(s):
    h = torch.zeros(s["h"].shape, dtype=torch.float64, device=s["h"].device)
    for rows, _, (gate, up) in _exact_experts(s, _values64(s["x"]), ("gate", "up")):
        h[rows] = gate * torch.sigmoid(gate) * up
    return h


def _exact_down(s):
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=s["y"].device)
    for _, slots, (v,) in _exact_experts(s, s["h"], ("down",)):
        y[slots] = v
    return y
