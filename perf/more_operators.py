"""What the operators of an attention layer's decode step cost: the projections with their epilogue (bias,
activation, residual), the rotation of the queries and keys with the write of keys and values into a paged cache
(bf16, or 8 bits with a scale for each token and head), the attention of one new token a sequence over that cache,
and the cache's rows read back.

Each case is one operator at one size. `run` computes it with plain torch operations in 32 bits, or, with
`own` set, with this package's entry points on the same data.
"""
import math

import torch

own = False

DEV = "cuda"
FP8 = torch.float8_e4m3fn
ROPE_BASE = 10000.0


# ------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # --- rotation and write into the cache
        # a decode step of 16 sequences: one token each, bound by the launch
        {"name": "write_decode_bf16", "op": "write", "tokens": 16, "padded": 0, "seqs": 16, "context": 8192,
         "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 16, "cache": "bf16", "heads_first": False, "rope": 128,
         "pairs": False},
        # a prefill of 8192 tokens of four sequences into an 8-bit cache, the batch's last rows padding
        {"name": "write_prefill_fp8", "op": "write", "tokens": 8192, "padded": 37, "seqs": 4, "context": 16384,
         "q_heads": 64, "kv_heads": 8, "dim": 128, "page": 64, "cache": "fp8", "heads_first": True, "rope": 128,
         "pairs": False},
        # --- the cache's rows read back
        # a prefix of a ragged length from an 8-bit cache, for a prefill that continues it
        {"name": "read_prefix_fp8", "op": "read", "tokens": 4951, "padded": 7, "seqs": 3, "context": 2048,
         "kv_heads": 8, "dim": 128, "page": 16, "cache": "fp8", "heads_first": False, "out": "bf16"},
        # long contexts of 64-wide heads
        {"name": "read_long_bf16", "op": "read", "tokens": 65536, "padded": 0, "seqs": 4, "context": 16384,
         "kv_heads": 8, "dim": 64, "page": 64, "cache": "bf16", "heads_first": True, "out": "bf16"},
        # --- attention of one new token
        # the smallest: one sequence, one rank's share of the heads, bound by latency
        {"name": "attn_one_sequence", "op": "attn", "rows": 1, "context": 500, "ragged": False, "q_heads": 8,
         "kv_heads": 1, "dim": 128, "page": 16, "cache": "bf16", "heads_first": False, "window": 0, "out": "bf16",
         "lse": False},
        # a decode batch of grouped heads, lengths spread from a few tokens to 8192
        {"name": "attn_decode_bf16", "op": "attn", "rows": 16, "context": 8192, "ragged": True, "q_heads": 64,
         "kv_heads": 8, "dim": 128, "page": 16, "cache": "bf16", "heads_first": False, "window": 0, "out": "bf16",
         "lse": False},
        # the largest: four sequences of 131072 tokens in 8 bits
        {"name": "attn_long_fp8", "op": "attn", "rows": 4, "context": 131072, "ragged": False, "q_heads": 64,
         "kv_heads": 8, "dim": 128, "page": 64, "cache": "fp8", "heads_first": True, "window": 0, "out": "bf16",
         "lse": False},
        # one head of keys for each head of queries, 80 wide, a sliding window, fp32 with the logarithms of the sums:
        # what ranks that hold parts of a context join
        {"name": "attn_window_ragged", "op": "attn", "rows": 61, "context": 4000, "ragged": True, "q_heads": 20,
         "kv_heads": 20, "dim": 80, "page": 48, "cache": "bf16", "heads_first": False, "window": 1000, "out": "fp32",
         "lse": True},
        # --- products with an epilogue
        # the query, key and value projection of a decode batch with its bias, bound by the weight
        {"name": "linear_decode_bf16", "op": "linear", "m": 16, "k": 8192, "n": 10240, "dtype": "bf16", "bias": True,
         "act": "none", "residual": "none", "out": "bf16"},
        # an output projection of 128 tokens in 8 bits, added to the residual stream
        {"name": "linear_decode_fp8", "op": "linear", "m": 128, "k": 8192, "n": 8192, "dtype": "fp8", "bias": False,
         "act": "none", "residual": "bf16", "out": "bf16"},
        # the same projection of a prefill of 4096 tokens
        {"name": "linear_prefill_bf16", "op": "linear", "m": 4096, "k": 8192, "n": 8192, "dtype": "bf16",
         "bias": False, "act": "none", "residual": "bf16", "out": "bf16"},
        # ragged sizes, the first product of a small feed-forward layer
        {"name": "linear_ragged_gelu", "op": "linear", "m": 777, "k": 1032, "n": 1000, "dtype": "bf16", "bias": True,
         "act": "gelu", "residual": "none", "out": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "linear"])
    if op == "linear":
        dtype = rng.choice(["bf16", "bf16", "fp8"])
        step = 16 if dtype == "fp8" else 8
        m, k = _log_int(rng, 1, 8192), step * _log_int(rng, 8, 8192 // step)
        most = min(10240, 8 * 8192 * 8192 // k, 4096 * 8192 * 8192 // (m * k))
        n = step * _log_int(rng, 4, max(5, most // step))
        return {"op": op, "m": m, "k": k, "n": n, "dtype": dtype, "bias": rng.random() < 0.5,
                "act": rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"]),
                "residual": rng.choice(["none", "bf16", "fp32"]),
                "out": "bf16" if dtype == "fp8" else rng.choice(["bf16", "bf16", "fp32"])}
    dim = rng.choice([64, 64, 80, 96, 112, 128, 128, 128, 192, 256])
    paged = {"dim": dim, "page": 16 * rng.choice([1, 1, 2, 3, 4, 8]), "cache": rng.choice(["bf16", "fp8"]),
             "heads_first": rng.random() < 0.5}
    kv_heads = rng.choice([1, 2, 4, 5, 8, 8, 16])
    if op == "attn":
        rows, context = _log_int(rng, 1, 128), _log_int(rng, 1, 131072)
        while rows * context * kv_heads * dim > 4 * 131072 * 8 * 128:
            context = max(1, context // 2)
        return {"op": op, "rows": rows, "context": context, "ragged": rng.random() < 0.7,
                "q_heads": kv_heads * rng.choice([1, 1, 2, 4, 5, 7, 8, 8, 12, 16, 24]), "kv_heads": kv_heads, **paged,
                "window": rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]), "out": rng.choice(["bf16", "bf16", "fp32"]),
                "lse": rng.random() < 0.3}
    tokens, seqs = _log_int(rng, 1, 8192 if op == "write" else 65536), _log_int(rng, 1, 64)
    seqs = min(seqs, tokens)
    each = -(-tokens // seqs)
    case = {"op": op, "tokens": tokens, "padded": rng.choice([0, 0, tokens // 20]), "seqs": seqs,
            "context": each + min(_log_int(rng, 1, 4096), 32768 // seqs)}
    if op == "read":
        while tokens * kv_heads * dim > 65536 * 8 * 64:
            kv_heads = max(1, kv_heads // 2)
            dim = dim if kv_heads > 1 else 64
        paged["dim"] = dim
        return {**case, "kv_heads": kv_heads, **paged, "out": rng.choice(["bf16", "fp32"])}
    q_heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
    while tokens * q_heads * dim > 8192 * 64 * 128 or q_heads > 64:
        q_heads, kv_heads = max(1, q_heads // 2), max(1, kv_heads // 2)
        q_heads = q_heads // kv_heads * kv_heads
    return {**case, "q_heads": q_heads, "kv_heads": kv_heads, **paged, "rope": rng.choice([0, dim, dim, dim // 32 * 16]),
            "pairs": rng.random() < 0.3}


# ------------------------------------------------------------------------------------------ the inputs

def _pool(case, pages, g):
    """A cache's keys or values and their scales, its pages lying as the case says."""
    h, p, d = case["kv_heads"], case["page"], case["dim"]
    shape = (pages, h, p, d) if case["heads_first"] else (pages, p, h, d)
    fp8 = case["cache"] == "fp8"
    x = torch.empty(shape, dtype=FP8 if fp8 else torch.bfloat16, device=DEV)
    piece = max(1, (1 << 26) // (h * p * d))  # (made in pieces, in 32 bits)
    for a in range(0, pages, piece):
        y = torch.randn((min(pages, a + piece) - a, *shape[1:]), generator=g, device=DEV)
        x[a : a + piece] = (y * 100).clamp_(-448, 448).to(FP8) if fp8 else y.bfloat16()
    scale = 0.01 * (0.5 + torch.rand(pages, h, p, generator=g, device=DEV)) if fp8 else None
    return (x.permute(0, 2, 1, 3) if case["heads_first"] else x), scale


def _table(case, lengths, g):
    """Pages for sequences of these lengths, in no order, and how many the pool has: a few to spare, or, where it is
    itself an output, as many as full sequences take."""
    p = case["page"]
    held = [-(-n // p) for n in lengths]
    total, width = sum(held) if case["op"] == "attn" else len(lengths) * -(-case["context"] // p), max(1, max(held))
    order = torch.randperm(total + 3, generator=g, device=DEV).int()
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(held):
        table[i, :n] = order[at : at + n]
        at += n
    return table, total + 3


def _placed(case, g):
    """Sequences and positions of the tokens: runs of neighbours that end where their sequence does."""
    tokens, seqs, context = case["tokens"], case["seqs"], case["context"]
    runs = [tokens // seqs + (i < tokens % seqs) for i in range(seqs)]
    spare = torch.rand(seqs, generator=g, device=DEV).tolist()
    lengths = [r + int(s * (context - r + 1)) for r, s in zip(runs, spare)]
    seq = torch.cat([torch.full((r,), i, dtype=torch.int32) for i, r in enumerate(runs)])
    pos = torch.cat([torch.arange(n - r, n, dtype=torch.int32) for r, n in zip(runs, lengths)])
    if case["padded"]:
        pos[tokens - case["padded"] :] = -1
    return seq.to(DEV), pos.to(DEV), lengths


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case)
    rand = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        if case["dtype"] == "fp8":
            a = rand(m, k)
            s["a_scale"] = a.abs().amax(1) / 448
            s["a"] = (a / s["a_scale"][:, None]).to(FP8)
            s["b"] = (100 * rand(k, n)).clamp_(-448, 448).to(FP8)
            s["b_scale"] = 2e-4 * (0.5 + torch.rand(n, generator=g, device=DEV))
        else:
            s["a"], s["a_scale"], s["b_scale"] = rand(m, k).bfloat16(), None, None
            s["b"] = (rand(k, n) / k ** 0.5).bfloat16()
        s["bias_in"] = rand(n).bfloat16() if case["bias"] else None
        types = {"bf16": torch.bfloat16, "fp32": torch.float32}
        s["r_in"] = None if case["residual"] == "none" else rand(m, n).to(types[case["residual"]])
        s["y"] = torch.empty(m, n, dtype=types[case["out"]], device=DEV)
        return s
    h, d, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "attn":
        rows, most = case["rows"], case["context"]
        if case["ragged"]:  # lengths spread over their logarithm, the longest the context; of many rows one is empty
            u = torch.rand(rows, generator=g, device=DEV).tolist()
            lengths = [min(most, max(1, int(math.exp(x * math.log(most + 0.5))))) for x in u]
            lengths[rows // 2] = most
            if rows > 8:
                lengths[3] = 0
        else:
            lengths = [most] * rows
        s["table"], pages = _table(case, lengths, g)
        (s["k"], s["k_scale"]), (s["v"], s["v_scale"]) = _pool(case, pages, g), _pool(case, pages, g)
        # what no sequence holds is memory that nobody wrote
        free = torch.ones(pages, page, dtype=torch.bool, device=DEV)
        for i, n in enumerate(lengths):
            t = torch.arange(n, device=DEV)
            free[s["table"][i].long()[t // page], t % page] = False
        for x in (s["k"], s["v"]):
            bits = x.view(torch.uint8 if case["cache"] == "fp8" else torch.int16)
            bits[free] = 0x7F if case["cache"] == "fp8" else 0x7FC0
        order = torch.randperm(rows, generator=g, device=DEV)  # a batch in another order than the table's
        s["row_seq"] = order.int()
        s["lens"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)[order]
        s["q"] = (1.5 * rand(rows, case["q_heads"] * d)).bfloat16()
        s["y"] = torch.empty(rows, case["q_heads"] * d, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32,
                             device=DEV)
        s["sums"] = torch.empty(rows, case["q_heads"], device=DEV) if case["lse"] else None
        s["longest"] = max(1, max(lengths))
    else:
        s["seq"], s["pos"], lengths = _placed(case, g)
        s["table"], pages = _table(case, lengths, g)
        (s["k"], s["k_scale"]), (s["v"], s["v_scale"]) = _pool(case, pages, g), _pool(case, pages, g)
        if case["op"] == "read":
            to = torch.bfloat16 if case["out"] == "bf16" else torch.float32
            s["k_rows"], s["v_rows"] = (torch.empty(case["tokens"], h * d, dtype=to, device=DEV) for _ in range(2))
        else:
            # the projection's rows: queries, keys and values side by side
            qd = case["q_heads"] * d
            rows = rand(case["tokens"], qd + 2 * h * d)
            rows[:, qd :: max(1, d // 4)] *= 8.0  # a few channels far above the others, as keys have
            rows = rows.bfloat16()
            s["q_in"], s["k_in"], s["v_in"] = rows[:, :qd], rows[:, qd : qd + h * d], rows[:, qd + h * d :]
            s["q_out"] = torch.zeros(case["tokens"], qd, dtype=torch.bfloat16, device=DEV)
            s["angles"] = None
            if case["rope"]:  # cosines, then sines, of every position
                half = case["rope"] // 2
                rate = ROPE_BASE ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
                turn = torch.arange(max(lengths), dtype=torch.float64, device=DEV)[:, None] * rate
                s["angles"] = torch.cat([turn.cos(), turn.sin()], 1).float()
    return s


# ------------------------------------------------------------------------------------------ the plain form

def _activated(act, x):
    if act == "relu":
        return x.clamp_min(0)
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh((2 / math.pi) ** 0.5 * (x + 0.044715 * x * x * x)))
    return x


def _linear(s):
    y = s["a"].float() @ s["b"].float()
    if s["a_scale"] is not None:
        y = y * s["a_scale"][:, None] * s["b_scale"]
    if s["bias_in"] is not None:
        y = y + s["bias_in"].float()
    y = _activated(s["act"], y)
    if s["r_in"] is not None:
        y = y + s["r_in"].float()
    return y.to(s["y"].dtype)


def _rotated(s, x, heads, n):
    """The first n rows of x by heads, rotated, in 32 bits."""
    x = x[:n].float().reshape(n, heads, s["dim"])
    r = s["rope"]
    if not r:
        return x
    turn = s["angles"][s["pos"][:n].long()][:, None]
    c, w = turn[..., : r // 2], turn[..., r // 2 :]
    first, second = (x[..., 0:r:2], x[..., 1:r:2]) if s["pairs"] else (x[..., : r // 2], x[..., r // 2 : r])
    a, b = first * c - second * w, second * c + first * w
    both = torch.stack([a, b], -1).reshape(n, heads, r) if s["pairs"] else torch.cat([a, b], -1)
    return torch.cat([both, x[..., r:]], -1)


def _stored(pool, scales, y, page, off):
    """y's rows at their places in the cache."""
    if scales is None:
        pool[page, off] = y.bfloat16()
        return
    scale = y.abs().amax(-1) / 448
    scale = torch.where(scale > 0, scale, 1.0)
    pool.view(torch.uint8)[page, off] = (y / scale[..., None]).clamp(-448, 448).to(FP8).view(torch.uint8)
    scales[page, :, off] = scale


def _places(s, n):
    pos = s["pos"][:n].long()
    return s["table"][s["seq"][:n].long(), pos // s["page"]].long(), pos % s["page"]


def _write(s):
    n, h = s["tokens"] - s["padded"], s["kv_heads"]
    page, off = _places(s, n)
    s["q_out"][:n] = _rotated(s, s["q_in"], s["q_heads"], n).reshape(n, -1).bfloat16()
    _stored(s["k"], s["k_scale"], _rotated(s, s["k_in"], h, n), page, off)
    _stored(s["v"], s["v_scale"], s["v_in"][:n].float().reshape(n, h, s["dim"]), page, off)
    return _written(s)


def _written(s):
    got = {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    return got if s["k_scale"] is None else {**got, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _read_pool(pool, scales, page, off):
    x = pool[page, off].float()
    return x if scales is None else x * scales[page, :, off][..., None]


def _read(s):
    n, h, d = s["tokens"] - s["padded"], s["kv_heads"], s["dim"]
    page, off = _places(s, n)
    got = {}
    for name in ("k", "v"):
        x = _read_pool(s[name], s[name + "_scale"], page, off).reshape(n, h * d)
        got[name] = torch.cat([x, x.new_zeros(s["padded"], h * d)]).to(s["k_rows"].dtype)
    return got


def _attn(s):
    rows, h, d, most = s["rows"], s["kv_heads"], s["dim"], s["longest"]
    t = torch.arange(most, device=DEV)
    ends = s["lens"].long()[:, None]
    valid = (t < ends) & ((t >= ends - s["window"]) if s["window"] else (t >= 0))
    page = s["table"][s["row_seq"].long()][:, t // s["page"]].long().clamp_min(0)
    off = (t % s["page"]).expand_as(page)
    k, v = (torch.where(valid[:, :, None, None], _read_pool(s[x], s[x + "_scale"], page, off), 0.0) for x in "kv")
    q = s["q"].float().reshape(rows, h, s["q_heads"] // h, d) * d ** -0.5
    score = q @ k.permute(0, 2, 3, 1)
    score = torch.where(valid[:, None, None, :], score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    y = (p @ v.transpose(1, 2)) / total.clamp_min(1e-30)
    got = {"out": y.reshape(rows, -1).to(s["y"].dtype)}
    if s["lse"]:
        got["lse"] = torch.where(total > 0, top + torch.log(total), -math.inf).reshape(rows, -1)
    return got


# ------------------------------------------------------------------------------------------ one pass

_handle = None


def _own(s):
    from allgather_gemm_persistent_amd import binding as B
    global _handle
    if _handle is None:
        _handle = B.agg_ctx_create(0)
    c, stream = _handle, torch.cuda.current_stream()
    if s["op"] == "linear":
        B.linear(c, s["m"], s["n"], s["k"], s["dtype"], s["a"], s["b"], s["y"], a_scale=s["a_scale"],
                 b_scale=s["b_scale"], bias=s["bias_in"], act=s["act"], residual=s["r_in"], stream=stream)
        return s["y"]
    cache = s.get("cache_handle")
    if cache is None:  # made once for a cache, as a program keeps it
        cache = s["cache_handle"] = B.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if s["op"] == "write":
        B.kv_write(c, cache, s["tokens"], s["k_in"], s["v_in"], s["pos"], s["table"], token_seq=s["seq"], q=s["q_in"],
                   q_out=s["q_out"], rope=s["angles"], rope_pairs=s["pairs"], stream=stream)
        return _written(s)
    if s["op"] == "read":
        B.kv_read(c, cache, s["tokens"], s["pos"], s["table"], s["k_rows"], s["v_rows"], token_seq=s["seq"],
                  stream=stream)
        return {"k": s["k_rows"], "v": s["v_rows"]}
    B.paged_attn(c, cache, s["rows"], s["q"], s["lens"], s["table"], s["y"], scale=s["dim"] ** -0.5,
                 row_seq=s["row_seq"], window=s["window"], lse=s["sums"], stream=stream)
    return {"out": s["y"]} | ({"lse": s["sums"]} if s["lse"] else {})


def run(state):
    if own:
        return _own(state)
    return {"linear": _linear, "write": _write, "read": _read, "attn": _attn}[state["op"]](state)


# ------------------------------------------------------------------------------------------ what it has to move

def _lengths_sum(case):
    """Cached tokens of all rows, on average where they are ragged."""
    most = case["context"]
    mean = most if not case["ragged"] or most < 2 else (most - 1) / math.log(most)
    total = most + (case["rows"] - 1) * mean
    return min(total, case["rows"] * case["window"]) if case["window"] else total


def work(case):
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        size = 1 if case["dtype"] == "fp8" else 2
        per = {"none": 0, "bf16": 2, "fp32": 4}
        return {"bytes": (m * k + k * n) * size + m * n * (per[case["out"]] + per[case["residual"]]) +
                         (2 * n if case["bias"] else 0) + (4 * (m + n) if size == 1 else 0),
                "flops": 2 * m * n * k}
    h, d = case["kv_heads"], case["dim"]
    held = 2 * h * (d * 2 if case["cache"] == "bf16" else d + 4)  # a token's keys and values in the cache
    if case["op"] == "attn":
        tokens = _lengths_sum(case)
        rows = case["rows"] * case["q_heads"]
        out = d * (2 if case["out"] == "bf16" else 4) + (4 if case["lse"] else 0)
        return {"bytes": int(tokens * (held + 4 / case["page"]) + rows * (2 * d + out)),
                "flops": int(4 * tokens * case["q_heads"] * d)}
    n = case["tokens"] - case["padded"]
    if case["op"] == "read":
        each = 2 * h * d * (2 if case["out"] == "bf16" else 4)
        return {"bytes": n * (held + 12) + case["tokens"] * each, "flops": 2 * n * h * d if case["cache"] == "fp8" else 0}
    q = case["q_heads"] * d
    return {"bytes": n * (4 * q + 4 * h * d + held + 12) + 4 * min(n, case["context"]) * case["rope"],
            "flops": n * (3 * (case["q_heads"] + h) * case["rope"] + 4 * h * d)}


# ------------------------------------------------------------------------------------------ the same in 64 bits

def _exact_linear(s):
    y = torch.mm(s["a"].double(), s["b"].double())
    if s["a_scale"] is not None:
        y = s["a_scale"].double().unsqueeze(1) * y * s["b_scale"].double().unsqueeze(0)
    if s["bias_in"] is not None:
        y += s["bias_in"].double()
    f = torch.nn.functional
    y = {"none": lambda x: x, "relu": torch.relu, "silu": f.silu, "gelu": f.gelu,
         "gelu_tanh": lambda x: f.gelu(x, approximate="tanh")}[s["act"]](y)
    return y if s["r_in"] is None else y + s["r_in"].double()


def _turned(s, x, heads):
    """The rotation as a complex product."""
    n = s["tokens"] - s["padded"]
    x = x[:n].double().reshape(n, heads, s["dim"]).clone()
    r = s["rope"]
    if r:
        turn = s["angles"][s["pos"][:n].long()].double()
        turn = torch.complex(turn[:, : r // 2], turn[:, r // 2 :])[:, None]
        if s["pairs"]:
            z = torch.view_as_complex(x[..., :r].reshape(n, heads, r // 2, 2).contiguous()) * turn
            x[..., :r] = torch.view_as_real(z).reshape(n, heads, r)
        else:
            z = torch.complex(x[..., : r // 2], x[..., r // 2 : r]) * turn
            x[..., : r // 2], x[..., r // 2 : r] = z.real, z.imag
    return x


def _exact_write(s):
    n, h, d = s["tokens"] - s["padded"], s["kv_heads"], s["dim"]
    seq, pos = s["seq"][:n].tolist(), s["pos"][:n].tolist()
    table = s["table"].tolist()
    page = torch.tensor([table[a][p // s["page"]] for a, p in zip(seq, pos)], device=DEV)
    off = torch.tensor([p % s["page"] for p in pos], device=DEV)
    q = s["q_out"].double()
    q[:n] = _turned(s, s["q_in"], s["q_heads"]).reshape(n, -1)
    got = {"q": q}
    for name, y in (("k", _turned(s, s["k_in"], h)), ("v", s["v_in"][:n].double().reshape(n, h, d))):
        if s["k_scale"] is None:
            got[name] = s[name].double()
            got[name][page, off] = y
        else:
            scale = y.abs().max(-1).values / 448
            scale[scale == 0] = 1
            got[name] = s[name].double()
            got[name][page, off] = (y / scale[..., None]).clamp(-448, 448).to(FP8).double()
            got[name + "_scale"] = s[name + "_scale"].double()
            got[name + "_scale"][page, :, off] = scale
    return got


def _exact_read(s):
    h, d, page = s["kv_heads"], s["dim"], s["page"]
    got = {}
    for name in ("k", "v"):
        out = torch.zeros(s["tokens"], h, d, dtype=torch.float64, device=DEV)
        for i in range(s["table"].shape[0]):
            mine = (s["seq"] == i) & (s["pos"] >= 0)
            pages = s["table"][i][s["table"][i] >= 0].long()
            if not bool(mine.any()):
                continue
            rows = s[name][pages].double()
            if s["k_scale"] is not None:
                rows = rows * s[name + "_scale"][pages].double().transpose(1, 2)[..., None]
            out[mine] = rows.reshape(-1, h, d)[s["pos"][mine].long()]
        got[name] = out.reshape(s["tokens"], h * d)
    return got


def _exact_attn(s):
    rows, h, d = s["rows"], s["kv_heads"], s["dim"]
    out = torch.zeros(rows, s["q_heads"], d, dtype=torch.float64, device=DEV)
    sums = torch.full((rows, s["q_heads"]), -math.inf, dtype=torch.float64, device=DEV)
    for r, (seq, n) in enumerate(zip(s["row_seq"].tolist(), s["lens"].tolist())):
        if not n:
            continue
        first = max(0, n - s["window"]) if s["window"] else 0
        pages = s["table"][seq, : -(-n // s["page"])].long()
        k, v = (s[x][pages].reshape(-1, h, d)[first:n].double() for x in "kv")
        if s["k_scale"] is not None:
            k, v = (x * s[name][pages].transpose(1, 2).reshape(-1, h)[first:n].double()[..., None]
                    for x, name in ((k, "k_scale"), (v, "v_scale")))
        q = s["q"][r].double().reshape(h, -1, d)
        score = torch.bmm(q, k.permute(1, 2, 0).contiguous()) / d ** 0.5
        sums[r] = torch.logsumexp(score, -1).reshape(-1)
        out[r] = torch.bmm(torch.softmax(score, -1), v.transpose(0, 1).contiguous()).reshape(-1, d)
    got = {"out": out.reshape(rows, -1)}
    return {**got, "lse": sums} if s["lse"] else got


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "write": _exact_write, "read": _exact_read, "attn": _exact_attn}[case["op"]](s)
