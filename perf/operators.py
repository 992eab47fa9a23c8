"""Workloads of the mixture-of-experts operators: the router, the quantized expert products and the combine.

Each case is one call.  With ``own`` false, ``run`` computes the operator in elementary torch operations in fp32;
with ``own`` true it calls the library.  The routed rows of a batch of T tokens with k experts each are sorted by
expert: expert e owns rows offsets[e] .. offsets[e+1], and ``rows[p]`` is the token of sorted row p.

  route    logits [T, E] -> ids, weights, offsets, rows, slots (top-k softmax and the grouping by expert)
  w4a16    y[p] = W_e x[rows[p]], W_e packed INT4 with fp16 scales and 4-bit zeros per group, x fp16 or bf16
  w8a8     the same from INT8 codes with a scale per token and per output channel, optionally SwiGLU on top
  fp8      the same from E4M3 codes
  combine  out[t] = sum_j weights[t, j] * y[slots[t, j]]
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the router of one decode step: 32 sequences, 64 experts of which each takes 8
        {"name": "route_step", "op": "route", "tokens": 32, "experts": 64, "top_k": 8, "dtype": "fp32",
         "renorm": True, "off": 0},
        # the router of a long prompt; some experts are switched off and padded tokens have none at all
        {"name": "route_prefill", "op": "route", "tokens": 16384, "experts": 128, "top_k": 8, "dtype": "bf16",
         "renorm": False, "off": 9},
        # one sequence's decode step through the gate and up projections of two of eight 14336-wide experts
        {"name": "w4_token", "op": "w4a16", "dtype": "fp16", "tokens": 1, "top_k": 2, "experts": 8, "n": 28672,
         "k": 4096, "group": 128, "gather": True, "skew": 0.0},
        # a decode batch over many small experts: about three rows each, several experts empty
        {"name": "w4_step", "op": "w4a16", "dtype": "bf16", "tokens": 48, "top_k": 4, "experts": 64, "n": 4096,
         "k": 2048, "group": 64, "gather": True, "skew": 0.7},
        # a chunk of a prompt through the down projection: rows already sorted, odd and uneven counts
        {"name": "w4_ragged", "op": "w4a16", "dtype": "fp16", "tokens": 777, "top_k": 2, "experts": 8, "n": 4096,
         "k": 14336, "group": 128, "gather": False, "skew": 0.8},
        # a whole prompt batch
        {"name": "w4_prefill", "op": "w4a16", "dtype": "bf16", "tokens": 4096, "top_k": 4, "experts": 32, "n": 4096,
         "k": 4096, "group": 128, "gather": True, "skew": 0.3},
        # a decode batch through the INT8 down projection
        {"name": "w8_step", "op": "w8a8", "tokens": 16, "top_k": 2, "experts": 8, "n": 4096, "k": 14336,
         "gather": False, "swiglu": False, "skew": 0.3},
        # a prompt batch through INT8 gate and up projections with SwiGLU
        {"name": "w8_prefill", "op": "w8a8", "tokens": 4096, "top_k": 4, "experts": 32, "n": 4096, "k": 4096,
         "gather": True, "swiglu": True, "skew": 0.3},
        # odd sizes and very uneven experts
        {"name": "fp8_odd", "op": "fp8", "tokens": 301, "top_k": 3, "experts": 20, "n": 1000, "k": 1360,
         "gather": True, "swiglu": True, "skew": 1.5},
        # a prompt batch in FP8, half the experts' rows more than the tile width
        {"name": "fp8_prefill", "op": "fp8", "tokens": 8192, "top_k": 2, "experts": 16, "n": 4096, "k": 4096,
         "gather": True, "swiglu": False, "skew": 0.5},
        # the weighted sum at the end of a small decode step
        {"name": "combine_step", "op": "combine", "dtype": "fp16", "tokens": 8, "top_k": 2, "n": 4096},
        # the weighted sum of a prompt batch
        {"name": "combine_prefill", "op": "combine", "dtype": "bf16", "tokens": 8192, "top_k": 8, "n": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_ROW_PRODUCTS = 16384 * 4096 * 4096  # rows * n * k of the largest listed product
MOST_WEIGHTS = 8 * 28672 * 4096          # experts * n * k of the largest listed weights


def draw(rng):
    op = rng.choice(["route", "w4a16", "w4a16", "w8a8", "w8a8", "fp8", "combine"])
    if op == "route":
        experts = rng.choice([8, 16, 60, 64, 96, 128])
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts, "top_k": rng.randint(1, min(8, experts)),
                "dtype": rng.choice(["fp32", "fp16", "bf16"]), "renorm": rng.random() < 0.5,
                "off": rng.choice([0, 0, 1, experts // 8])}
    if op == "combine":
        dtype, top_k, n = rng.choice(["fp16", "bf16"]), rng.randint(1, 8), _log(rng, 500, 8192)
        return {"op": op, "dtype": dtype, "tokens": min(_log(rng, 1, 8192), 8192 * 8 * 4096 // (top_k * n)),
                "top_k": top_k, "n": n}
    while True:
        experts = _log(rng, 4, 128)
        top_k = rng.randint(1, min(8, experts))
        tokens = _log(rng, 1, 8192)
        n = 2 * _log(rng, 128, 14336)
        case = {"op": op, "tokens": tokens, "top_k": top_k, "experts": experts, "n": n,
                "gather": rng.random() < 0.6, "skew": rng.choice([0.0, 0.3, 0.8, 1.5])}
        if op == "w4a16":
            case["dtype"] = rng.choice(["fp16", "bf16"])
            case["group"] = rng.choice([32, 64, 128, 128, 256])
            case["k"] = case["group"] * max(1, _log(rng, 512, 14336) // case["group"])
        else:
            case["k"] = 16 * _log(rng, 16, 896)
            case["swiglu"] = rng.random() < 0.5
        rows = tokens * top_k
        if rows * n * case["k"] <= MOST_ROW_PRODUCTS and experts * n * case["k"] <= MOST_WEIGHTS and rows <= 16384:
            return case


# ---------------------------------------------------------------------------------------------------- inputs
def _assignment(g, tokens, experts, top_k, skew):
    """ids [T, k]: distinct experts per token, some experts more popular than others."""
    pop = torch.randn(experts, device="cuda", generator=g) * skew
    noise = -torch.log(-torch.log(torch.rand(tokens, experts, device="cuda", generator=g).clamp(1e-9, 1 - 1e-7)))
    return torch.topk(pop + noise, top_k, dim=1).indices


def _activations(g, shape):
    """N(0, 1) with one channel in a hundred fifty times larger."""
    x = torch.randn(shape, device="cuda", generator=g)
    x[:, torch.randperm(shape[1], device="cuda", generator=g)[: shape[1] // 100]] *= 50.0
    return x


def _words(g, shape, a, b, c):
    """int32 words of eight 4-bit codes; code = (r1 & a) + (r2 & b) + (r3 & c) per nibble, which never carries."""
    def bits(mask):
        r = torch.randint(-(1 << 31), 1 << 31, shape, device="cuda", dtype=torch.int32, generator=g)
        return r & torch.tensor(mask * 0x11111111, device="cuda", dtype=torch.int32)
    return bits(a) + bits(b) + bits(c)


def _logits(case, g):
    x = torch.randn(case["tokens"], case["experts"], device="cuda", generator=g) * 2.0
    if case["off"]:
        x[:, torch.randperm(case["experts"], device="cuda", generator=g)[: case["off"]]] = -math.inf
        x[torch.rand(case["tokens"], device="cuda", generator=g) < 0.05] = -math.inf  # padded tokens
    return x.to(DTYPES[case["dtype"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "route":
        s["logits"] = _logits(case, g)
        return s
    tokens, top_k = case["tokens"], case["top_k"]
    if case["op"] == "combine":
        rows = tokens * top_k
        s["y"] = torch.randn(rows, case["n"], device="cuda", generator=g).to(DTYPES[case["dtype"]])
        s["weights"] = torch.softmax(torch.randn(tokens, top_k, device="cuda", generator=g), dim=1)
        slots = torch.randperm(rows, device="cuda", generator=g).to(torch.int32).view(tokens, top_k)
        s["slots"] = torch.where(torch.rand(tokens, top_k, device="cuda", generator=g) < 0.02, -1, slots).to(torch.int32)
        return s

    experts, n, k = case["experts"], case["n"], case["k"]
    ids = _assignment(g, tokens, experts, top_k, case["skew"]).reshape(-1)
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=experts)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["rows"] = (order // top_k).to(torch.int32) if case["gather"] else None
    s["most"] = int(counts.max())
    held = tokens if case["gather"] else tokens * top_k
    if case["op"] == "w4a16":
        groups = k // case["group"]
        s["x"] = _activations(g, (held, k)).to(DTYPES[case["dtype"]])
        s["qweight"] = _words(g, (experts, n, k // 8), 7, 7, 1)                # 0 .. 15, mean 7.5
        s["scales"] = torch.exp(torch.randn(experts, n, groups, device="cuda", generator=g) * 0.3 - 5.0).half()
        s["qzeros"] = _words(g, (experts, n, (groups + 7) // 8), 3, 3, 1) + 0x44444444  # 4 .. 11
        if groups % 8:
            s["qzeros"][..., -1] &= (1 << (4 * (groups % 8))) - 1              # unused nibbles are zero
    else:
        x = _activations(g, (held, k)) * (0.4 if case["op"] == "w8a8" else 1.0)
        s["sx"] = torch.exp(torch.randn(held, device="cuda", generator=g) * 0.2 - 3.0)
        s["sw"] = torch.exp(torch.randn(experts, n, device="cuda", generator=g) * 0.3 - 8.0)
        w = torch.randn(experts, n, k, device="cuda", generator=g, dtype=torch.float16)
        if case["op"] == "w8a8":
            s["xq"] = (x * 6).round().clamp(-127, 127).to(torch.int8)
            s["wq"] = w.mul_(32).round_().clamp_(-127, 127).to(torch.int8)
        else:
            s["xq"] = (x * 6).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s["wq"] = w.mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return s


# ---------------------------------------------------------------------------------------------------- plain forms
def _route(s):
    logits, top_k = s["logits"].float(), s["top_k"]
    tokens, experts = logits.shape
    key = torch.where(logits > -math.inf, logits, -math.inf)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    rest = torch.exp(key - top[:, :1])
    top, ids = top[:, :top_k], ids[:, :top_k]
    taken = top > -math.inf
    e = torch.where(taken, torch.exp(top - top[:, :1]), 0.0)
    total = e.sum(1, keepdim=True) if s["renorm"] else torch.where(key > -math.inf, rest, 0.0).sum(1, keepdim=True)
    weights = torch.where(taken, e / total, 0.0)
    ids = torch.where(taken, ids, -1)
    flat = torch.where(ids < 0, experts, ids).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.zeros(experts + 1, dtype=torch.int64, device="cuda").scatter_add_(0, flat, torch.ones_like(flat))
    ends = counts.cumsum(0)
    offsets = torch.cat([ends.new_zeros(1), ends[:experts]])
    place = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device="cuda"))
    rows = torch.where(torch.arange(order.numel(), device="cuda") < offsets[-1], order // top_k, -1)
    slots = torch.where(ids < 0, -1, place.view(tokens, top_k))
    return ids.to(torch.int32), weights, offsets.to(torch.int32), rows.to(torch.int32), slots.to(torch.int32)


def _unpack(words, count):
    """[..., count] codes of int32 words of eight 4-bit codes, lowest bits first."""
    shifts = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    return ((words.unsqueeze(-1) >> shifts) & 15).flatten(-2)[..., :count]


def _grouped(s, x, w, sx, sw):
    """Every expert's rows padded to the longest, one batched product, the scales, and the rows put back."""
    offsets, experts = s["offsets"].long(), s["experts"]
    total = s["tokens"] * s["top_k"]
    place = offsets[:-1, None] + torch.arange(s["most"], device="cuda")
    inside = place < offsets[1:, None]
    place = place.clamp(max=total - 1)
    src = s["rows"].long()[place] if s["rows"] is not None else place
    y = torch.bmm(x[src], w.transpose(1, 2))
    if sx is not None:
        y = y * sx[src].unsqueeze(-1) * sw.unsqueeze(1)
    if s.get("swiglu"):
        gate, up = y.chunk(2, dim=2)
        y = gate / (1.0 + torch.exp(-gate)) * up
    out = torch.zeros(total + 1, y.shape[2], device="cuda")
    out.index_copy_(0, torch.where(inside, place, total).reshape(-1), y.reshape(experts * s["most"], -1))
    return out[:total]


def _w4a16(s):
    n, k, group = s["n"], s["k"], s["group"]
    codes = _unpack(s["qweight"], k).float().view(s["experts"], n, k // group, group)
    zeros = _unpack(s["qzeros"], k // group).float().unsqueeze(-1)
    w = ((codes - zeros) * s["scales"].float().unsqueeze(-1)).view(s["experts"], n, k)
    return _grouped(s, s["x"].float(), w, None, None).to(s["x"].dtype)


def _combine(s):
    slots = s["slots"].long()
    y = s["y"].float()[slots.clamp(min=0)]
    y = torch.where(slots.unsqueeze(-1) >= 0, y, 0.0)
    return (y * s["weights"].unsqueeze(-1)).sum(1).to(s["y"].dtype)


def run(s):
    op = s["op"]
    if own:
        import bit_gemv_gemm_group_b200 as wq
        if op == "route":
            return wq.moe_route(s["logits"], s["top_k"], renormalize=s["renorm"])
        if op == "w4a16":
            return wq.grouped_gemm_w4a16(s["x"], s["qweight"], s["scales"], s["qzeros"], s["offsets"], s["rows"],
                                         group_size=s["group"])
        if op == "w8a8":
            return wq.grouped_gemm_w8a8(s["xq"], s["sx"], s["wq"], s["sw"], s["offsets"], s["rows"],
                                        swiglu=s["swiglu"])
        if op == "fp8":
            return wq.grouped_gemm_fp8(s["xq"], s["sx"], s["wq"], s["sw"], s["offsets"], s["rows"],
                                       swiglu=s["swiglu"])
        return wq.moe_combine(s["y"], s["weights"], s["slots"])
    if op == "route":
        return _route(s)
    if op == "w4a16":
        return _w4a16(s)
    if op == "w8a8":
        return _grouped(s, s["xq"].float(), s["wq"].float(), s["sx"], s["sw"]).half()
    if op == "fp8":
        e4m3 = torch.float8_e4m3fn
        return _grouped(s, s["xq"].view(e4m3).float(), s["wq"].view(e4m3).float(), s["sx"], s["sw"]).half()
    return _combine(s)


# ---------------------------------------------------------------------------------------------------- work
def work(case):
    t, k = case["tokens"], case["top_k"]
    rows = t * k
    if case["op"] == "route":
        e = case["experts"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": t * e * size + rows * 16 + 4 * (e + 1), "flops": t * e * (k + 4)}
    n = case["n"]
    if case["op"] == "combine":
        return {"bytes": 2 * rows * n + 2 * t * n + 8 * rows, "flops": 2 * rows * n}
    depth = case["k"]
    used = case["experts"] * (1 - (1 - k / case["experts"]) ** t)  # experts with rows, if all are equally popular
    held = t if case["gather"] else rows
    if case["op"] == "w4a16":
        size, weight = 2, 0.5 + 2.5 / case["group"]
        scales = 0
    else:
        size, weight = 1, 1.0
        scales = 4 * held + 4 * used * n
    out = n // 2 if case.get("swiglu") else n
    return {"bytes": used * n * depth * weight + held * depth * size + scales + 2 * rows * out + 4 * rows,
            "flops": 2.0 * rows * n * depth}


# ---------------------------------------------------------------------------------------------------- 64 bits
def _exact_nibbles(words, count):
    """Codes through the bytes of the words: the low and the high half of each byte in turn."""
    b = words.contiguous().view(torch.uint8)
    return torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)[..., :count].double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        x = s["logits"].double()
        best = torch.topk(x, case["top_k"], dim=1).values   # values only: which of equal ones does not matter here
        high = x.amax(1, keepdim=True)
        base = best if case["renorm"] else x
        logsum = high + torch.log(torch.exp(base - high).sum(1, keepdim=True))
        weights = torch.nan_to_num(torch.exp(best - logsum), nan=0.0)
        return None, weights, None, None, None
    if op == "combine":
        rows = torch.cat([s["y"].double(), torch.zeros(1, case["n"], dtype=torch.float64, device="cuda")])
        out = torch.zeros(case["tokens"], case["n"], dtype=torch.float64, device="cuda")
        for j in range(case["top_k"]):
            out += s["weights"][:, j, None].double() * rows[s["slots"][:, j].long()]  # -1 is the row of zeros
        return out
    bounds = s["offsets"].tolist()
    parts = []
    for e, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
        if lo == hi:
            continue
        src = s["rows"][lo:hi].long() if s["rows"] is not None else slice(lo, hi)
        if op == "w4a16":
            codes = _exact_nibbles(s["qweight"][e], case["k"])
            zeros = _exact_nibbles(s["qzeros"][e], case["k"] // case["group"]).repeat_interleave(case["group"], dim=1)
            w = (codes - zeros) * s["scales"][e].double().repeat_interleave(case["group"], dim=1)
            y = s["x"][src].double() @ w.T
        else:
            x, w = s["xq"][src], s["wq"][e]
            if op == "fp8":
                x, w = x.view(torch.float8_e4m3fn), w.view(torch.float8_e4m3fn)
            y = (s["sx"][src].double()[:, None] * x.double()) @ (s["sw"][e].double()[:, None] * w.double()).T
        if case.get("swiglu"):
            half = case["n"] // 2
            y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
        parts.append(y)
    return torch.cat(parts)
