"""The routed-expert operators as they are measured: routing, the expert-sorted
rows, microscaled 4-bit quantisation, the products over it and the weighted
sum back to tokens.

A case names one operator and its sizes. prepare() draws what a serving step
has in hand, run() is one call of the operator: in elementary torch operations
where `own` is false, through adapter_lora_serving_amd where it is true.

Microscaled 4-bit floating point (MXFP4): a row of K values is held as K / 32
blocks of 32. A block has one scale 2^(byte - 127) (byte 255: not a number)
and 32 codes of 4 bits: a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6. The even
element of a pair is the low half of its byte. Scale rows are padded with zero
bytes to a multiple of four.
"""
import math

import torch

own = False

DEV = "cuda:0"
MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
LARGEST = 8192 * 28672 * 4096   # multiplications of the largest listed product
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the router of one request's next token: 64 experts, the two best
        dict(name="route_token", op="route", T=1, E=64, k=2, dtype="bf16", scores="softmax",
             bias=False, groups=1, top_groups=1, group_score="max", masked=False),
        # a prefill batch over 256 experts in 8 groups, of which 4 are open to a token
        dict(name="route_prefill", op="route", T=8192, E=256, k=8, dtype="f32", scores="sigmoid",
             bias=True, groups=8, top_groups=4, group_score="sum2", masked=False),
        # the decode step of 256 requests over 8 experts, top-2
        dict(name="rows_decode", op="rows", T=256, k=2, E=8, slots=32, dead=0.0),
        # the same for a prefill batch over 256 experts, top-8, with some choices dropped
        dict(name="rows_prefill", op="rows", T=8192, k=8, E=256, slots=128, dead=0.01),
        # activations of a few decode tokens before a projection
        dict(name="quantize_decode", op="quantize", form="plain", M=7, K=4096, dtype="bf16"),
        # the activation of a prefill batch's gate/up product, quantised for the down product
        dict(name="quantize_silu_prefill", op="quantize", form="silu_mul", M=8192, K=14336,
             dtype="bf16"),
        # the fused q/k/v projection of one token: a weight read from end to end
        dict(name="linear_token", op="linear", M=1, N=6144, K=4096, out="bf16"),
        # the fused gate/up projection of a prefill batch: the largest dense product
        dict(name="linear_prefill", op="linear", M=8192, N=28672, K=4096, out="bf16"),
        # gate/up of 8 experts for a decode step: every expert's weight, few rows each
        dict(name="experts_decode", op="experts", rows=512, E=8, N=28672, K=4096, out="bf16"),
        # down of 8 experts for a prefill batch of 8192 tokens, top-2
        dict(name="experts_prefill", op="experts", rows=16384, E=8, N=4096, K=14336, out="bf16"),
        # two experts' rows of each decode token back to the token
        dict(name="combine_decode", op="combine", T=256, k=2, H=4096, dtype="bf16", add=False,
             dead=0.0),
        # eight experts' rows of each prefill token, added to the residual
        dict(name="combine_prefill", op="combine", T=8192, k=8, H=4096, dtype="bf16", add=True,
             dead=0.01),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "rows", "quantize", "linear", "experts", "combine"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * max(_log(rng, 8, 512) // groups, 1)
        top_groups = rng.randint(1, groups)
        return dict(op=op, T=_log(rng, 1, 8192), E=E,
                    k=rng.randint(1, min(16, E // groups * top_groups)),
                    dtype=rng.choice(["bf16", "f32"]), scores=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                    group_score=rng.choice(["max", "sum2"]), masked=rng.random() < 0.3)
    if op == "rows":
        E = _log(rng, 4, 512)
        return dict(op=op, T=_log(rng, 1, 8192), k=rng.randint(1, min(8, E)), E=E,
                    slots=rng.randint(1, 128), dead=rng.choice([0.0, 0.02, 0.3]))
    if op == "quantize":
        return dict(op=op, form=rng.choice(["plain", "rows", "silu_mul"]), M=_log(rng, 1, 8192),
                    K=32 * _log(rng, 1, 448), dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "combine":
        return dict(op=op, T=_log(rng, 1, 8192), k=rng.randint(1, 8), H=8 * _log(rng, 8, 512),
                    dtype=rng.choice(["bf16", "bf16", "f32"]) if rng.random() < 0.5 else "bf16",
                    add=rng.random() < 0.5, dead=rng.choice([0.0, 0.02]))
    N, K = _log(rng, 64, 28672), 32 * _log(rng, 4, 448)
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, max(1, min(8192, LARGEST // (N * K)))), N=N, K=K,
                    out=rng.choice(["bf16", "bf16", "f32"]))
    E = min(_log(rng, 2, 64), max(1, 8 * 28672 * 4096 // (N * K)))
    return dict(op=op, rows=_log(rng, 1, max(1, min(16384, LARGEST // (N * K)))), E=E, N=N, K=K,
                out=rng.choice(["bf16", "bf16", "f32"]))


# ---- inputs ---------------------------------------------------------------

def _activations(g, rows, K):
    """Rows whose channels differ in size, as the inputs of a projection do."""
    x = torch.randn(rows, K, device=DEV, generator=g)
    return x * torch.exp(0.5 * torch.randn(K, device=DEV, generator=g))


def _held(x):
    """x (f32) in MXFP4: codes [.., K / 2] and padded scale bytes, uint8."""
    mag, sign, byte = _blocks(x)
    code = torch.where(mag < 2, 2 * mag, torch.where(mag < 4, mag + 2, mag / 2 + 4)).to(torch.uint8)
    code = (code + 8 * sign.to(torch.uint8)).flatten(-2)
    scales = byte.to(torch.uint8)
    pad = -scales.shape[-1] % 4
    return code[..., 0::2] + 16 * code[..., 1::2], torch.nn.functional.pad(scales, (0, pad))


def _held_weight(g, N, K):
    return _held(torch.randn(N, K, device=DEV, generator=g) / math.sqrt(K))


def _bounds(g, rows, E):
    """Bounds of the experts' rows: uneven loads, some experts idle in small batches."""
    load = torch.exp(0.5 * torch.randn(E, device=DEV, generator=g))
    ids = torch.multinomial(load, rows, replacement=True, generator=g)
    counts = torch.bincount(ids, minlength=E)
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c = dict(case)
    op = c["op"]
    s = dict(case=c)
    if op == "route":
        x = 1.5 * torch.randn(c["T"], c["E"], device=DEV, generator=g)
        if c["masked"]:   # experts that a token may not take
            x[torch.rand(x.shape, device=DEV, generator=g) < 0.1] = -math.inf
        s["logits"] = x.to(DTYPES[c["dtype"]])
        s["bias"] = 0.05 * torch.randn(c["E"], device=DEV, generator=g) if c["bias"] else None
    elif op == "rows":
        T, k, E = c["T"], c["k"], c["E"]
        load = torch.exp(0.5 * torch.randn(E, device=DEV, generator=g))
        ids = torch.multinomial(load.expand(T, E), k, generator=g)
        ids[torch.rand(T, k, device=DEV, generator=g) < c["dead"]] = -1
        s["ids"] = ids.to(torch.int32)
        s["token_slot"] = torch.randint(-1, c["slots"], (T,), device=DEV, generator=g,
                                        dtype=torch.int32)
    elif op == "quantize":
        M, K = c["M"], c["K"]
        tokens = max(1, M // 2) if c["form"] == "rows" else M
        x = _activations(g, tokens, 2 * K if c["form"] == "silu_mul" else K)
        s["x"] = x.to(DTYPES[c["dtype"]])
        if c["form"] == "rows":   # the token of every expert-sorted row
            s["row_token"] = torch.randint(0, tokens, (M,), device=DEV, generator=g,
                                           dtype=torch.int32)
    elif op == "linear":
        s["x"] = _held(_activations(g, c["M"], c["K"]))
        s["w"] = _held_weight(g, c["N"], c["K"])
    elif op == "experts":
        s["x"] = _held(_activations(g, c["rows"], c["K"]))
        w = [_held_weight(g, c["N"], c["K"]) for _ in range(c["E"])]
        s["w"] = tuple(torch.stack(p) for p in zip(*w))
        s["offsets"] = _bounds(g, c["rows"], c["E"])
    else:
        T, k, H = c["T"], c["k"], c["H"]
        dtype = DTYPES[c["dtype"]]
        s["rows"] = torch.randn(T * k, H, device=DEV, generator=g).to(dtype)
        pos = torch.randperm(T * k, device=DEV, generator=g).reshape(T, k)
        pos[torch.rand(T, k, device=DEV, generator=g) < c["dead"]] = -1
        s["positions"] = pos.to(torch.int32)
        w = torch.rand(T, k, device=DEV, generator=g) + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        s["residual"] = torch.randn(T, H, device=DEV, generator=g).to(dtype) if c["add"] else None
    return s


# ---- the operators in elementary operations -------------------------------

def _blocks(x):
    """Magnitudes [.., K / 32, 32], signs and scale bytes of x (f32)."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    byte = (torch.frexp(top).exponent.to(torch.int32) + 124).clamp(0, 254)
    byte = torch.where(top == 0, torch.zeros_like(byte), byte)
    a = b.abs() * torch.exp2((127 - byte).float()).unsqueeze(-1)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp(max=6.0), b < 0, byte


def _rounded(x):
    """x (f32) as MXFP4 holds it."""
    mag, sign, byte = _blocks(x)
    return (torch.where(sign, -mag, mag) * torch.exp2((byte - 127).float()).unsqueeze(-1)).flatten(-2)


def _values(held):
    """The f32 values that codes and scale bytes stand for."""
    codes, scales = held
    pair = torch.tensor(MAGNITUDES + [-v for v in MAGNITUDES], device=codes.device)
    pair = torch.stack([pair.repeat(16), pair.repeat_interleave(16)], 1)
    v = pair[codes.int()].flatten(-2).unflatten(-1, (-1, 32))
    return (v * torch.exp2(scales[..., :v.shape[-2]].float() - 127).unsqueeze(-1)).flatten(-2)


def _route(s, c):
    x = s["logits"].float()
    shut = torch.isnan(x) | (x == -math.inf)
    x = x.clamp(max=torch.finfo(torch.float32).max)
    if c["scores"] == "softmax":
        top = x.masked_fill(shut, -math.inf).amax(1, keepdim=True)
        e = torch.exp(x - top).masked_fill(shut, 0.0)
        # summed in 64 bits: a score, and with it the choice between near
        # experts, does not go by the order of the sum
        score = e / e.double().sum(1, keepdim=True).float()
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    choice = score if s["bias"] is None else score + s["bias"]
    choice = choice.masked_fill(shut | torch.isnan(choice), -math.inf)
    if c["top_groups"] < c["groups"]:
        by = choice.unflatten(1, (c["groups"], -1))
        best = by.sort(2, descending=True).values[:, :, :2 if c["group_score"] == "sum2" else 1]
        worth = best.masked_fill(best == -math.inf, 0.0).sum(2)
        worth = worth.masked_fill(best[:, :, 0] == -math.inf, -math.inf)
        rank = worth.sort(dim=1, descending=True, stable=True).indices.sort(1).indices
        choice = by.masked_fill((rank >= c["top_groups"]).unsqueeze(2), -math.inf).flatten(1)
    order = choice.sort(dim=1, descending=True, stable=True)
    ids = order.indices[:, :c["k"]]
    none = order.values[:, :c["k"]] == -math.inf
    w = score.gather(1, ids).masked_fill(none, 0.0)
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return dict(ids=ids.masked_fill(none, -1).to(torch.int32), weights=w)


def _rows(s, c):
    k, E = c["k"], c["E"]
    ids = s["ids"].flatten().long()
    live = (ids >= 0) & (ids < E)
    key = torch.where(live, ids, torch.full_like(ids, E))
    order = key.sort(stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    token = order // k
    slot = torch.where(live[order], s["token_slot"][token], -1)
    return dict(row_token=token.to(torch.int32),
                positions=torch.where(live, place, -1).to(torch.int32).unflatten(0, (-1, k)),
                offsets=offsets.to(torch.int32), row_slot=slot.to(torch.int32))


def _experts(s, c):
    """One batched product over the experts, each padded to the longest one's rows."""
    counts = s["offsets"].long().diff()
    longest = int(counts.max())
    expert = torch.repeat_interleave(torch.arange(c["E"], device=counts.device), counts)
    at = torch.arange(c["rows"], device=counts.device) - s["offsets"].long()[expert]
    x = torch.zeros(c["E"], longest, c["K"], device=counts.device)
    x[expert, at] = _values(s["x"])
    return torch.bmm(x, _values(s["w"]).transpose(1, 2))[expert, at]


def _plain(s, c):
    op = c["op"]
    if op == "route":
        return _route(s, c)
    if op == "rows":
        return _rows(s, c)
    if op == "quantize":
        x = s["x"]
        if c["form"] == "plain":
            return dict(values=_rounded(x.float()).to(x.dtype))
        if c["form"] == "rows":
            rows = x[s["row_token"].long()]
        else:
            gate, up = x.float().chunk(2, 1)
            rows = (gate / (1.0 + torch.exp(-gate)) * up).to(x.dtype)
        return dict(rows=rows, values=_rounded(rows.float()).to(x.dtype))
    if op == "linear":
        return dict(y=(_values(s["x"]) @ _values(s["w"]).t()).to(DTYPES[c["out"]]))
    if op == "experts":
        return dict(y=_experts(s, c).to(DTYPES[c["out"]]))
    pos = s["positions"].long()
    w = s["weights"].masked_fill(pos < 0, 0.0)
    y = (s["rows"][pos.clamp(min=0)].float() * w.unsqueeze(2)).sum(1)
    if c["add"]:
        y = y + s["residual"].float()
    return dict(y=y.to(s["rows"].dtype))


# ---- the framework's calls ------------------------------------------------

def _own(s, c):
    import adapter_lora_serving_amd as L
    op = c["op"]
    if op == "route":
        r = L.route_experts(s["logits"], c["k"], scores=c["scores"], bias=s["bias"],
                            groups=c["groups"], top_groups=c["top_groups"],
                            group_score=c["group_score"])
        return dict(ids=r.ids, weights=r.weights)
    if op == "rows":
        r = L.expert_rows(s["ids"], c["E"], s["token_slot"])
        return dict(row_token=r.row_token, positions=r.positions, offsets=r.offsets,
                    row_slot=r.row_slot)
    if op == "quantize":
        x = s["x"]
        if c["form"] == "plain":
            return dict(values=L.dequantize_mxfp4(L.quantize_mxfp4(x), x.dtype))
        if c["form"] == "rows":
            rows, held = L.gather_quantize_mxfp4(x, s["row_token"])
        else:
            rows, held = L.silu_mul_quantize_mxfp4(x)
        return dict(rows=rows, values=L.dequantize_mxfp4(held, x.dtype))
    if op == "linear":
        return dict(y=L.mxfp4_linear(L.MXFP4(*s["x"]), L.MXFP4(*s["w"]), dtype=DTYPES[c["out"]]))
    if op == "experts":
        return dict(y=L.mxfp4_expert_linear(L.MXFP4(*s["x"]), L.MXFP4(*s["w"]), s["offsets"],
                                            dtype=DTYPES[c["out"]]))
    return dict(y=L.combine_experts(s["rows"], s["positions"], s["weights"],
                                    residual=s["residual"]))


def run(state):
    return (_own if own else _plain)(state, state["case"])


# ---- what a pass cannot do without ----------------------------------------

def _bytes_held(rows, K):
    return rows * (K // 2 + K // 32)


def work(case):
    c, op = case, case["op"]
    if op == "route":
        e = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=c["T"] * c["E"] * e + 4 * c["E"] * c["bias"] + 8 * c["T"] * c["k"],
                    flops=4 * c["T"] * c["E"])
    if op == "rows":
        n = c["T"] * c["k"]
        return dict(bytes=4 * (n + c["T"] + 3 * n + c["E"] + 1), flops=0)
    if op == "quantize":
        M, K, e = c["M"], c["K"], 2 if c["dtype"] == "bf16" else 4
        read = {"plain": M, "rows": max(1, M // 2), "silu_mul": 2 * M}[c["form"]] * K * e
        rows = 0 if c["form"] == "plain" else M * K * e
        # codes and scales are written, then read back for the values
        return dict(bytes=read + rows + 2 * _bytes_held(M, K) + M * K * e
                    + 4 * M * (c["form"] == "rows"), flops=4 * M * K)
    if op in ("linear", "experts"):
        rows = c["M"] if op == "linear" else c["rows"]
        weights = c["N"] * (1 if op == "linear" else min(c["E"], rows))
        return dict(bytes=_bytes_held(rows, c["K"]) + _bytes_held(weights, c["K"])
                    + rows * c["N"] * (2 if c["out"] == "bf16" else 4)
                    + (4 * (c["E"] + 1) if op == "experts" else 0),
                    flops=2 * rows * c["N"] * c["K"])
    n, e = c["T"] * c["k"], 2 if c["dtype"] == "bf16" else 4
    return dict(bytes=n * (c["H"] * e + 8) + c["T"] * c["H"] * e * (2 if c["add"] else 1),
                flops=2 * n * c["H"])


# ---- the definitions in 64 bits -------------------------------------------

def _exact_route(s, c):
    x = s["logits"].double()
    open_ = ~(torch.isnan(x) | torch.isneginf(x))
    x = torch.where(open_, x, -math.inf)
    score = torch.sigmoid(x) if c["scores"] == "sigmoid" else torch.softmax(x, 1).nan_to_num(0.0)
    choice = score + (0.0 if s["bias"] is None else s["bias"].double())
    choice = torch.where(open_, choice, -math.inf)
    T, E, G = c["T"], c["E"], c["groups"]
    if c["top_groups"] < G:
        worth = choice.view(T, G, E // G).topk(min(2, E // G), 2).values
        worth = worth if c["group_score"] == "sum2" else worth[..., :1]
        worth = torch.where(worth[..., 0] == -math.inf, -math.inf,
                            worth.clamp(min=-1e9).masked_fill(worth == -math.inf, 0.0).sum(2))
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        keep.scatter_(1, worth.argsort(dim=1, descending=True, stable=True)[:, :c["top_groups"]], True)
        choice = torch.where(keep.repeat_interleave(E // G, 1), choice, -math.inf)
    at = choice.argsort(dim=1, descending=True, stable=True)[:, :c["k"]]
    w = torch.where(choice.gather(1, at) == -math.inf, 0.0, score.gather(1, at))
    return dict(ids=None, weights=(w / w.sum(1, keepdim=True)).nan_to_num(0.0))


def _exact_rounded(x):
    """Nearest value of each block's grid by its definition, ties to the even code."""
    b = x.view(x.shape[0], -1, 32)
    top = b.abs().amax(2)
    scale = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, 1.0))) - 2).clamp(min=2.0**-127)
    a = (b / scale.unsqueeze(2)).abs()
    grid = torch.tensor(MAGNITUDES, device=x.device, dtype=torch.float64)
    near = torch.zeros_like(a)
    for i in range(1, 8):   # past the midpoint, or on it where the upper code is even
        mid = (grid[i - 1] + grid[i]) / 2
        near = torch.where((a > mid) | ((a == mid) & (i % 2 == 0)), grid[i], near)
    return (near * scale.unsqueeze(2) * b.sign()).view_as(x)


def _exact_values(held):
    codes, scales = held[0].to(torch.int16), held[1]
    v = torch.stack([codes % 16, codes // 16], -1).flatten(-2)
    m = v % 8
    mag = torch.where(m < 2, m * 0.5, (1 + (m % 2) * 0.5) * torch.exp2((m // 2 - 1).double()))
    scale = torch.exp2(scales.double() - 127).repeat_interleave(32, -1)[..., :v.shape[-1]]
    return torch.where(v >= 8, -mag, mag).double() * scale


def exact(case, seed):
    s, c = prepare(case, seed), case
    op = c["op"]
    if op == "route":
        return _exact_route(s, c)
    if op == "rows":
        return None
    if op == "quantize":
        x = s["x"].double()
        if c["form"] == "plain":
            return dict(values=_exact_rounded(x))
        if c["form"] == "rows":
            rows = x[s["row_token"].long()]
            return dict(rows=rows, values=_exact_rounded(rows))
        gate, up = x[:, :c["K"]], x[:, c["K"]:]
        rows = gate * torch.sigmoid(gate) * up
        return dict(rows=rows, values=_exact_rounded(rows.to(s["x"].dtype).double()))
    if op == "linear":
        return dict(y=torch.mm(_exact_values(s["x"]), _exact_values(s["w"]).t()))
    if op == "experts":
        y = torch.empty(c["rows"], c["N"], device=DEV, dtype=torch.float64)
        at = s["offsets"].tolist()
        for e in range(c["E"]):
            if at[e + 1] > at[e]:
                part = slice(at[e], at[e + 1])
                y[part] = _exact_values([p[part] for p in s["x"]]) @ _exact_values([p[e] for p in s["w"]]).t()
        return dict(y=y)
    w, pos = s["weights"].double(), s["positions"].long()
    y = torch.zeros(c["T"], c["H"], device=DEV, dtype=torch.float64)
    for j in range(c["k"]):
        y += torch.where(pos[:, j] >= 0, w[:, j], 0.0).unsqueeze(1) * s["rows"][pos[:, j].clamp(min=0)].double()
    return dict(y=y if s["residual"] is None else y + s["residual"].double())
