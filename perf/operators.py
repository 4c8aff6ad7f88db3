"""What the operators of a mixture-of-experts layer cost: the residual's addition with the RMS norm (bf16 or
8-bit output), the routing to experts with its plan, and the experts' products with the combine.

Each case is one operator at one size. `run` computes it with plain torch operations in 32 bits, or, with
`own` set, with this package's entry points on the same data.
"""
import math

import torch

own = False

EPS = 1e-5
DEV = "cuda"


# ------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # --- residual + norm
        # a decode step after the AllReduce: fp32 rows + bf16 residual -> the 8-bit operand of a projection
        {"name": "norm_decode_fp8", "op": "norm", "rows": 16, "cols": 8192, "x": "fp32", "residual": True, "out": "fp8"},
        # a prefill step of 4096 tokens, bf16 throughout
        {"name": "norm_prefill_bf16", "op": "norm", "rows": 4096, "cols": 8192, "x": "bf16", "residual": True,
         "out": "bf16"},
        # the rows an AllToAll delivered (a ragged count), without a residual, to 8 bits
        {"name": "norm_ragged_fp8", "op": "norm", "rows": 4951, "cols": 7168, "x": "bf16", "residual": False,
         "out": "fp8"},
        # --- routing and its plan
        # a decode batch, few experts, all of them on this rank
        {"name": "route_decode", "op": "route", "tokens": 16, "experts": 64, "k": 2, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "logits": "fp32", "ranks": 1, "masked": 0},
        # the tokens of eight ranks of 4096, sigmoid scores with a balance bias, 4 of 8 groups, this rank holding 1/8
        {"name": "route_prefill", "op": "route", "tokens": 32768, "experts": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "logits": "fp32", "ranks": 8, "masked": 0},
        # ragged tokens, an expert count that is no power of two, bf16 logits (many ties), disabled experts and padding
        {"name": "route_ragged", "op": "route", "tokens": 4951, "experts": 60, "k": 4, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "logits": "bf16", "ranks": 1, "masked": 3},
        # --- the experts' products; "up" is the gated first product, "down" the second with the combine
        # a decode batch of 16: four rows an expert, bound by the weights
        {"name": "up_decode_bf16", "op": "up", "tokens": 16, "experts": 8, "k": 2, "hidden": 8192, "inner": 3584,
         "dtype": "bf16", "ranks": 1},
        # a prefill of 5120 tokens
        {"name": "up_prefill_bf16", "op": "up", "tokens": 5120, "experts": 8, "k": 2, "hidden": 8192, "inner": 3584,
         "dtype": "bf16", "ranks": 1},
        # the largest: 8192 tokens in 8 bits
        {"name": "up_prefill_fp8", "op": "up", "tokens": 8192, "experts": 8, "k": 2, "hidden": 8192, "inner": 3584,
         "dtype": "fp8", "ranks": 1},
        # a single decode step in 8 bits, back to the hidden width and combined
        {"name": "down_decode_fp8", "op": "down", "tokens": 16, "experts": 8, "k": 2, "hidden": 8192, "inner": 3584,
         "dtype": "fp8", "ranks": 1},
        # a prefill of 5120 tokens, second product and combine
        {"name": "down_prefill_bf16", "op": "down", "tokens": 5120, "experts": 8, "k": 2, "hidden": 8192,
         "inner": 3584, "dtype": "bf16", "ranks": 1},
        # many small experts, odd widths, half of the choices on another rank
        {"name": "down_ragged_bf16", "op": "down", "tokens": 777, "experts": 30, "k": 4, "hidden": 1032, "inner": 1000,
         "dtype": "bf16", "ranks": 2},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "route", "up", "down"])
    if op == "norm":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "cols": 8 * _log_int(rng, 8, 1280),
                "x": rng.choice(["bf16", "bf16", "fp32"]), "residual": rng.random() < 0.7,
                "out": rng.choice(["bf16", "fp8"])}
    if op == "route":
        score = rng.choice(["softmax", "sigmoid"])
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _log_int(rng, 8 if groups == 1 else 4, 384 // groups)
        experts = groups * size
        top_groups = rng.randint(1, groups)
        return {"op": op, "tokens": _log_int(rng, 1, 32768), "experts": experts,
                "k": rng.randint(1, min(8, top_groups * size)), "score": score, "bias": score == "sigmoid",
                "groups": groups, "top_groups": top_groups, "logits": rng.choice(["fp32", "bf16"]),
                "ranks": rng.choice([1, 2]) if experts % 2 == 0 else 1, "masked": rng.choice([0, 0, 2])}
    dtype = rng.choice(["bf16", "fp8"])
    step = 16 if dtype == "fp8" else 8
    experts = _log_int(rng, 2, 64)
    # widths whose weights stay below those of the listed cases
    hidden = step * _log_int(rng, 16, 8192 // step)
    most = min(3584, 8 * 8192 * 3584 // (experts * hidden))
    inner = step * _log_int(rng, 8, max(9, most // step))
    tokens = _log_int(rng, 1, 8192)
    k = rng.randint(1, min(4, experts))
    while tokens * k > 16384 or tokens * k * hidden * inner > 16384 * 8192 * 3584:
        tokens = max(1, tokens // 2)
    return {"op": op, "tokens": tokens, "experts": experts, "k": k, "hidden": hidden, "inner": inner, "dtype": dtype,
            "ranks": rng.choice([1, 1, 2])}


# ------------------------------------------------------------------------------------------ the inputs

def _choices(case, g):
    """Which experts each token takes: k different ones, some experts more popular than others."""
    total = case["experts"] * case["ranks"]
    liking = torch.randn(case["tokens"], total, generator=g, device=DEV) + 0.5 * torch.randn(total, generator=g, device=DEV)
    return torch.topk(liking, case["k"], dim=1).indices


def _sorted_by_expert(ids, first, n_local):
    """The plan of a routing: offsets, slot -> token, (token, choice) -> slot."""
    tokens, k = ids.shape
    local = ids.reshape(-1).long() - first
    bucket = torch.where((local >= 0) & (local < n_local) & (ids.reshape(-1) >= 0), local, n_local)
    order = torch.sort(bucket, stable=True).indices
    held = bucket[order] < n_local
    place = torch.arange(tokens * k, device=ids.device)
    slot_token = torch.where(held, order // k, -1)
    token_slot = torch.empty_like(place)
    token_slot[order] = torch.where(held, place, -1)
    counts = (bucket[:, None] == torch.arange(n_local, device=ids.device)).sum(0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=ids.device), counts.cumsum(0)])
    return offsets.int(), slot_token.int(), token_slot.reshape(tokens, k).int()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        x = torch.randn(rows, cols, generator=g, device=DEV)
        x[:, :: max(1, cols // 8)] *= 20.0  # a few channels far above the others, as hidden states have
        s["x_in"] = x if case["x"] == "fp32" else x.bfloat16()
        s["r_in"] = torch.randn(rows, cols, generator=g, device=DEV).bfloat16() if case["residual"] else None
        s["w"] = (1 + 0.1 * torch.randn(cols, generator=g, device=DEV)).bfloat16()
        s["out_q"] = torch.empty(rows, cols, dtype=torch.float8_e4m3fn if case["out"] == "fp8" else torch.bfloat16, device=DEV)
        s["scales"] = torch.empty(rows, device=DEV) if case["out"] == "fp8" else None
        s["r_out"] = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV) if case["residual"] else None
        return s
    if case["op"] == "route":
        tokens, experts, k = case["tokens"], case["experts"], case["k"]
        x = 1.5 * torch.randn(tokens, experts, generator=g, device=DEV) + 0.5 * torch.randn(experts, generator=g, device=DEV)
        if case["masked"]:
            x[:, 1 :: max(2, experts // case["masked"])] = -math.inf  # disabled experts
            x[tokens - tokens // 50 :] = -math.inf  # padding at the end of the batch
        s["x_in"] = x if case["logits"] == "fp32" else x.bfloat16()
        s["b_in"] = 0.1 * torch.randn(experts, generator=g, device=DEV) if case["bias"] else None
        s["n_local"] = experts // case["ranks"]
        s["first"] = (case["ranks"] // 2) * s["n_local"]
        s["ids"] = torch.empty(tokens, k, dtype=torch.int32, device=DEV)
        s["wts"] = torch.empty(tokens, k, device=DEV)
        s["offsets"] = torch.empty(s["n_local"] + 1, dtype=torch.int32, device=DEV)
        s["slot_token"] = torch.empty(tokens * k, dtype=torch.int32, device=DEV)
        s["token_slot"] = torch.empty(tokens, k, dtype=torch.int32, device=DEV)
        # the plan's scratch: a count for each 1024 (token, choice) pairs and expert
        s["scratch"] = torch.empty((tokens * k // 1024 + 1) * (s["n_local"] + 1), dtype=torch.int32, device=DEV)
        return s
    tokens, k, experts = case["tokens"], case["k"], case["experts"]
    up = case["op"] == "up"
    kk, nn = (case["hidden"], 2 * case["inner"]) if up else (case["inner"], case["hidden"])
    ids = _choices(case, g)
    s["offsets"], s["slot_token"], s["token_slot"] = _sorted_by_expert(ids, 0, experts)
    counts = s["offsets"].diff()
    s["most"] = max(1, int(counts.max()))  # rows of the fullest expert: the plain form's padding
    wts = torch.rand(tokens, k, generator=g, device=DEV) + 0.1
    s["wts"] = wts / wts.sum(1, keepdim=True)
    rows = tokens if up else tokens * k
    a = torch.randn(rows, kk, generator=g, device=DEV)
    if case["dtype"] == "fp8":
        a_scale = a.abs().amax(1) / 448
        s["a"], s["a_scale"] = (a / a_scale[:, None]).to(torch.float8_e4m3fn), a_scale
        s["b"] = torch.empty(experts, kk, nn, dtype=torch.float8_e4m3fn, device=DEV)
        for e in range(experts):
            s["b"][e] = (100 * torch.randn(kk, nn, generator=g, device=DEV)).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s["b_scale"] = 2e-4 * (0.5 + torch.rand(experts, nn, generator=g, device=DEV))
    else:
        s["a"], s["a_scale"], s["b_scale"] = a.bfloat16(), None, None
        s["b"] = torch.empty(experts, kk, nn, dtype=torch.bfloat16, device=DEV)
        for e in range(experts):
            s["b"][e] = (0.02 * torch.randn(kk, nn, generator=g, device=DEV)).bfloat16()
    s["out"] = torch.zeros(tokens * k, nn // 2 if up else nn, dtype=torch.bfloat16, device=DEV)
    s["sum"] = None if up else torch.empty(tokens, nn, dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------------------------------ the plain form

def _norm(s):
    x = s["x_in"].float()
    if s["r_in"] is not None:
        x = x + s["r_in"].float()
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["w"].float()
    got = {"residual": x.bfloat16()} if s["r_in"] is not None else {}
    if s["out"] == "bf16":
        return {**got, "out": y.bfloat16()}
    scale = y.abs().amax(1) / 448
    scale = torch.where(scale > 0, scale, 1.0)
    return {**got, "out": (y / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), "scales": scale}


def _route(s):
    x = s["x_in"].float()
    tokens, experts = x.shape
    k, groups = s["k"], s["groups"]
    open_ = x > -math.inf
    if s["score"] == "softmax":
        top = x.amax(1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
        p = torch.exp(x - top)
        p = p / p.sum(1, keepdim=True).clamp_min(1e-30)
        key = x
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
        key = p
    if s["b_in"] is not None:
        key = key + s["b_in"]
    key = torch.where(open_, key, -math.inf)
    if groups > 1:
        grouped = key.reshape(tokens, groups, experts // groups)
        best = torch.sort(grouped, dim=2, descending=True).values
        score = best[:, :, 0]
        if s["score"] == "sigmoid":
            score = score + torch.where(best[:, :, 1] > -math.inf, best[:, :, 1], 0.0)
        kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, : s["top_groups"]]
        stays = (kept[:, :, None] == torch.arange(groups, device=x.device)).any(1)
        key = torch.where(stays.repeat_interleave(experts // groups, 1), key, -math.inf)
    value, ids = torch.sort(key, dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    chosen = value > -math.inf
    w = torch.where(chosen, p.gather(1, ids), 0.0)
    w = w / torch.where(chosen[:, :1], w.sum(1, keepdim=True), 1.0)
    ids = torch.where(chosen, ids, -1).int()
    offsets, slot_token, token_slot = _sorted_by_expert(ids, s["first"], s["n_local"])
    return {"ids": ids, "weights": w, "offsets": offsets, "slot_token": slot_token, "token_slot": token_slot}


def _padded(s):
    """The slots of each expert side by side, padded to the fullest: [experts, most] slot numbers and which are real."""
    lane = torch.arange(s["most"], device=DEV)
    counts = s["offsets"].diff()
    real = lane < counts[:, None]
    return torch.where(real, s["offsets"][:-1, None] + lane, 0).long(), real


def _experts(s, wide=torch.float32):
    """The experts' product of every slot, in `wide` precision: [slots, columns], zero where no expert is."""
    slot, real = _padded(s)
    row = s["slot_token"].long()[slot].clamp_min(0) if s["op"] == "up" else slot
    a, b = s["a"].to(wide), s["b"].to(wide)
    if s["a_scale"] is not None:
        a, b = a * s["a_scale"].to(wide)[:, None], b * s["b_scale"].to(wide)[:, None, :]
    y = torch.bmm(a[row], b)
    if s["op"] == "up":
        gate, up = y[:, :, : s["inner"]], y[:, :, s["inner"] :]
        y = gate / (1 + torch.exp(-gate)) * up
    flat = torch.zeros(s["slot_token"].numel(), y.shape[2], dtype=wide, device=DEV)
    flat[slot[real]] = y[real]
    return flat


def _combined(s, y):
    at = s["token_slot"].long()
    w = torch.where(at >= 0, s["wts"].to(y.dtype), 0.0)
    return (y[at.clamp_min(0)] * w[:, :, None]).sum(1)


# ------------------------------------------------------------------------------------------ one pass

_handle = None


def _own(s):
    from allgather_gemm_persistent_amd import binding as B
    global _handle
    if _handle is None:
        _handle = B.agg_ctx_create(0)
    c, stream = _handle, torch.cuda.current_stream()
    if s["op"] == "norm":
        B.rms_norm(c, s["rows"], s["cols"], s["x_in"], s["w"], s["out_q"], residual=s["r_in"], residual_out=s["r_out"],
                   eps=EPS, scales=s["scales"], stream=stream)
        got = {"residual": s["r_out"]} if s["r_out"] is not None else {}
        return {**got, "out": s["out_q"]} | ({"scales": s["scales"]} if s["scales"] is not None else {})
    if s["op"] == "route":
        B.moe_route(c, s["tokens"], s["experts"], s["k"], s["x_in"], s["ids"], s["wts"], score=s["score"],
                    bias=s["b_in"], groups=s["groups"], top_groups=s["top_groups"], stream=stream)
        B.moe_plan(c, s["tokens"], s["k"], s["ids"], s["first"], s["n_local"], s["offsets"], s["slot_token"],
                   s["token_slot"], s["scratch"], stream=stream)
        return {"ids": s["ids"], "weights": s["wts"], "offsets": s["offsets"], "slot_token": s["slot_token"],
                "token_slot": s["token_slot"]}
    slots = s["tokens"] * s["k"]
    if s["op"] == "up":
        B.moe_gemm(c, slots, s["experts"], s["inner"], s["hidden"], s["dtype"], s["a"], s["b"], s["offsets"], s["out"],
                   gated=True, slot_token=s["slot_token"], a_scale=s["a_scale"], b_scale=s["b_scale"], stream=stream)
        return s["out"]
    B.moe_gemm(c, slots, s["experts"], s["hidden"], s["inner"], s["dtype"], s["a"], s["b"], s["offsets"], s["out"],
               a_scale=s["a_scale"], b_scale=s["b_scale"], stream=stream)
    B.moe_combine(c, s["tokens"], s["k"], s["hidden"], slots, s["out"], s["token_slot"], s["wts"], s["sum"], stream=stream)
    return s["sum"]


def run(state):
    if own:
        return _own(state)
    if state["op"] == "norm":
        return _norm(state)
    if state["op"] == "route":
        return _route(state)
    y = _experts(state)
    return y.bfloat16() if state["op"] == "up" else _combined(state, y).bfloat16()


# ------------------------------------------------------------------------------------------ what it has to move

def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        each = (4 if case["x"] == "fp32" else 2) + (4 if case["residual"] else 0) + (1 if case["out"] == "fp8" else 2)
        return {"bytes": n * each + 2 * case["cols"] + (4 * case["rows"] if case["out"] == "fp8" else 0), "flops": 6 * n}
    if case["op"] == "route":
        n = case["tokens"] * case["experts"]
        pairs = case["tokens"] * case["k"]
        return {"bytes": n * (4 if case["logits"] == "fp32" else 2) + 16 * pairs, "flops": 4 * n}
    pairs = case["tokens"] * case["k"]
    held = max(1, pairs // case["ranks"])  # choices that fall on this rank, on average
    touched = case["experts"] * (1 - (1 - 1 / (case["experts"] * case["ranks"])) ** pairs)
    up = case["op"] == "up"
    kk, nn = (case["hidden"], 2 * case["inner"]) if up else (case["inner"], case["hidden"])
    size = 1 if case["dtype"] == "fp8" else 2
    rows = case["tokens"] if up else held
    written = held * (nn // 2) * 2 if up else case["tokens"] * nn * 2
    return {"bytes": int(max(1.0, touched) * kk * nn * size + rows * kk * size + written), "flops": 2 * held * kk * nn}


# ------------------------------------------------------------------------------------------ the same in 64 bits

def _exact_norm(s):
    x = s["x_in"].double() + (0 if s["r_in"] is None else s["r_in"].double())
    rms = (x.pow(2).sum(1) / x.shape[1] + EPS).sqrt()
    y = x / rms[:, None] * s["w"].double()
    got = {"residual": x} if s["r_in"] is not None else {}
    if s["out"] == "bf16":
        return {**got, "out": y}
    scale = y.abs().max(1).values / 448
    scale[scale == 0] = 1
    return {**got, "out": y / scale[:, None], "scales": scale}


def _exact_route(s):
    x = s["x_in"].double()
    experts, k = x.shape[1], s["k"]
    if s["score"] == "softmax":
        p = torch.nan_to_num(torch.softmax(x, 1), nan=0.0)
    else:
        p = torch.sigmoid(x)
    key = (x if s["score"] == "softmax" else p) + (0 if s["b_in"] is None else s["b_in"].double())
    key = key.masked_fill(x == -math.inf, -math.inf)
    if s["groups"] > 1:
        size = experts // s["groups"]
        best = key.view(-1, s["groups"], size).topk(min(2, size), dim=2).values
        best[:, :, 1:][best[:, :, 1:] == -math.inf] = 0
        score = best.sum(2) if s["score"] == "sigmoid" else best[:, :, 0]
        # of equal groups the first: the score is compared with an index behind it
        rank = torch.argsort(score, dim=1, descending=True, stable=True).argsort(1)
        key = key.masked_fill((rank >= s["top_groups"]).repeat_interleave(size, 1), -math.inf)
    ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :k]
    w = p.gather(1, ids).masked_fill(key.gather(1, ids) == -math.inf, 0)
    total = w.sum(1, keepdim=True)
    return {"ids": None, "weights": w / total.masked_fill(total == 0, 1), "offsets": None, "slot_token": None,
            "token_slot": None}


def _exact_experts(s):
    """Expert by expert, its rows alone."""
    up = s["op"] == "up"
    bounds = s["offsets"].tolist()
    y = torch.zeros(s["slot_token"].numel(), s["inner"] if up else s["hidden"], dtype=torch.float64, device=DEV)
    for e in range(s["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        row = s["slot_token"][lo:hi].long() if up else torch.arange(lo, hi, device=DEV)
        a, b = s["a"][row].double(), s["b"][e].double()
        if s["a_scale"] is not None:
            a, b = a * s["a_scale"][row].double()[:, None], b * s["b_scale"][e].double()
        z = a @ b
        y[lo:hi] = z[:, : s["inner"]] * torch.sigmoid(z[:, : s["inner"]]) * z[:, s["inner"] :] if up else z
    if up:
        return y
    out = torch.zeros(s["tokens"], s["hidden"], dtype=torch.float64, device=DEV)
    for j in range(s["k"]):
        at = s["token_slot"][:, j].long()
        has = at >= 0
        out[has] += s["wts"][has, j].double()[:, None] * y[at[has]]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "up": _exact_experts, "down": _exact_experts}[case["op"]](s)
