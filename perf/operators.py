"""The operators around 4-bit experts, as cases that can be timed: the top-k router, MXFP4
quantisation, the grouped MXFP4 product and the whole MXFP4 expert layer.

``run`` computes each in its plain form (elementary torch operations in 32 bits) or, where
``own`` is set, through the framework's entry points.  ``exact`` is the definition in 64 bits.

MXFP4: elements are e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte, the
even one in the low nibble; every 32 consecutive elements share one e8m0 scale byte b, worth
2^(b - 127); b = 255 is NaN.
"""
import math

import torch

own = False

# ------------------------------------------------------------------------------------ cases
# Sizes are those of the repository's own workloads: decode / decode16 (K 7168, I 2048, 256 or 16
# experts, top 8) and prefill (K 4096, I 1408, 64 experts, top 6), and odd ones between them.


def listed():
    return [
        # the router of one decoded token: latency alone
        {"name": "route one token", "op": "route", "M": 1, "E": 256, "topK": 8, "type": "f32", "score": "softmax", "masked": 0.0},
        # the router of a prefill batch, logits left in binary16 by the gate product, a tenth of the experts masked
        {"name": "route prefill", "op": "route", "M": 8192, "E": 64, "topK": 6, "type": "f16", "score": "softmax", "masked": 0.1},
        # many requests' prompts at once, sigmoid scores, whole rows masked now and then (padding tokens)
        {"name": "route many", "op": "route", "M": 65521, "E": 256, "topK": 8, "type": "f32", "score": "sigmoid", "masked": 0.02},
        # one token's activations quantised and read back
        {"name": "quant one token", "op": "quant", "M": 1, "D": 7168, "type": "f16"},
        # one expert stack's bf16 weights quantised at load time and read back to look at the error
        {"name": "quant weights", "op": "quant", "M": 90112, "D": 4096, "type": "bf16"},
        # a ragged handful of rows per expert, a depth that ends inside a 256-deep tile (GMM2 of prefill's model)
        {"name": "product odd", "op": "product", "M": 101, "D": 1408, "N": 4096, "E": 8, "topK": 2, "skew": 0.5},
        # GMM1 of a decode batch: the weights of every expert stream past four rows each
        {"name": "product decode", "op": "product", "M": 128, "D": 7168, "N": 4096, "E": 256, "topK": 8, "skew": 0.0},
        # GMM1 of a prefill batch: bound by the tensor cores
        {"name": "product prefill", "op": "product", "M": 8192, "D": 4096, "N": 2816, "E": 64, "topK": 6, "skew": 0.0},
        # the layer for one decoded token
        {"name": "layer one token", "op": "layer", "M": 1, "K": 7168, "I": 2048, "E": 256, "topK": 8, "skew": 0.0},
        # eight concurrent requests on few experts
        {"name": "layer 8 tokens", "op": "layer", "M": 8, "K": 7168, "I": 2048, "E": 16, "topK": 8, "skew": 0.3},
        # an odd number of requests, some routes dropped
        {"name": "layer 29 tokens", "op": "layer", "M": 29, "K": 4096, "I": 1408, "E": 64, "topK": 6, "skew": 0.5},
        # the layer over a prefill batch
        {"name": "layer prefill", "op": "layer", "M": 8192, "K": 4096, "I": 1408, "E": 64, "topK": 6, "skew": 0.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "quant", "product", "layer"])
    if op == "route":
        E = _log_int(rng, 8, 512)
        return {"op": op, "M": _log_int(rng, 1, 65521 * 256 // max(E, 256)), "E": E, "topK": rng.randint(1, min(E, 10)),
                "type": rng.choice(["f32", "f16", "bf16"]), "score": rng.choice(["softmax", "sigmoid"]), "masked": rng.choice([0.0, 0.05, 0.3])}
    if op == "quant":
        return {"op": op, "M": _log_int(rng, 1, 40000), "D": 64 * rng.randint(1, 128), "type": rng.choice(["f32", "f16", "bf16"])}
    skew = rng.choice([0.0, 0.5, 1.2])
    if op == "product":
        E = _log_int(rng, 1, 64)
        return {"op": op, "M": _log_int(rng, 1, 4096), "D": 64 * rng.randint(2, 64), "N": 128 * rng.randint(1, 22), "E": E, "topK": rng.randint(1, min(E, 8)), "skew": skew}
    E = _log_int(rng, 1, 64)
    return {"op": op, "M": _log_int(rng, 1, rng.choice([64, 2048])), "K": 128 * rng.randint(1, 32), "I": 64 * rng.randint(1, 22), "E": E, "topK": rng.randint(1, min(E, 8)), "skew": skew}


# ------------------------------------------------------------------------------------ MXFP4, plainly
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E2M1 = E2M1 + [-v for v in E2M1]


def _tables(device):
    """Values of a code byte's two elements, [256][2], and of a scale byte, [256]."""
    pair = torch.tensor([[E2M1[b & 15], E2M1[b >> 4]] for b in range(256)], dtype=torch.float32, device=device)
    scale = torch.tensor([2.0 ** (b - 127) for b in range(255)] + [math.nan], dtype=torch.float64).to(torch.float32).to(device)
    return pair, scale


def _quantise(x, tables):
    """Code indexes 0..15 [..., D] (uint8) and scale bytes [..., D / 32] (uint8) of x [..., D]."""
    b = x.to(torch.float32).unflatten(-1, (-1, 32))
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    a = b.abs().amax(-1)
    e = (torch.frexp(a).exponent - 3).clamp(-127, 127)
    e = torch.where(a > 0, e, torch.full_like(e, -127))
    y = (b * tables[1][127 - e][..., None]).abs()  # 2^-e, exactly
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = torch.where(torch.signbit(b), code | 8, code)
    return code.flatten(-2), torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)


def _values(code, scale, tables):
    """The values that codes (indexes) and scale bytes stand for, in 32 bits."""
    one = tables[0][:16, 0]
    return (one[code.int()].unflatten(-1, (-1, 32)) * tables[1][scale.int()][..., None]).flatten(-2)


def _unpack(packed, scale, tables):
    """The same of packed code bytes [..., D / 2]."""
    v = torch.nn.functional.embedding(packed.int(), tables[0]).flatten(-2)
    return v.unflatten(-1, (-1, 32)).mul_(tables[1][scale.int()][..., None]).flatten(-2)


# ------------------------------------------------------------------------------------ inputs
def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(M, D, g, dtype):
    """Hidden states: each token has its own size, some channels are much larger than the rest."""
    x = torch.randn(M, D, device="cuda", generator=g)
    x *= torch.exp(0.3 * torch.randn(M, 1, device="cuda", generator=g))
    x *= torch.where(torch.rand(1, D, device="cuda", generator=g) < 0.01, 8.0, 1.0)
    return x.to(dtype)


def _weights(E, N, D, g, tables):
    """MXFP4 weights of N(0, 1 / D) channels as rows: codes [E][N][D / 2], scales [E][N][D / 32].
    The channels are taken from a pool of quantised rows: made quickly, and every value is a real one."""
    rows = min(E * N, 8192)
    w = torch.randn(rows, D, device="cuda", generator=g) / math.sqrt(D)
    code, scale = _quantise(w * torch.exp(0.2 * torch.randn(rows, 1, device="cuda", generator=g)), tables)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    at = torch.randint(0, rows, (E * N,), device="cuda", generator=g)
    return packed[at].view(E, N, D // 2), scale[at].view(E, N, D // 32)


def _blocks(codes, scales, gate_up):
    """The framework's layout of MXFP4 weights, made once when they are loaded: per expert, per 128
    channels, per 256-deep step one block of 17408 bytes.  Its first 16 KiB are the channels' 128-byte
    code rows, the 16-byte chunk c of row r at chunk c ^ (r % 8); then, for each half of the step,
    128 words of four scale bytes.  gate_up: a block's channels are 32 gate, 32 up, 32 gate, 32 up."""
    E, N, half = codes.shape
    KB = (half + 127) // 128
    if gate_up:
        order = torch.arange(N, device=codes.device).view(2, N // 64, 32).transpose(0, 1).reshape(-1)
        codes, scales = codes[:, order], scales[:, order]
    c = torch.nn.functional.pad(codes, (0, KB * 128 - half)).view(E, N // 128, 16, 8, KB, 8, 16)
    s = torch.nn.functional.pad(scales, (0, KB * 8 - scales.shape[-1])).view(E, N // 128, 128, KB, 2, 4)
    out = torch.empty(E, N // 128, KB, 17408, dtype=torch.uint8, device=codes.device)
    r = torch.arange(8, device=codes.device)[:, None]
    c = c.permute(0, 1, 4, 2, 3, 5, 6)[:, :, :, :, r, r ^ r.T]  # [E][NB][KB][16][8 rows][8 chunks][16]
    out[..., :16384] = c.reshape(E, N // 128, KB, 16384)
    out[..., 16384:] = s.permute(0, 1, 3, 4, 2, 5).reshape(E, N // 128, KB, 1024)
    return out


def _routing(M, E, topK, skew, g):
    """Distinct experts per token (a share of popular ones where skew > 0) and softmax weights."""
    logits = -skew * torch.log(1 + torch.randperm(E, device="cuda", generator=g).float())[None].expand(M, E)
    noise = -torch.log(-torch.log(torch.rand(M, E, device="cuda", generator=g).clamp(1e-20, 1 - 1e-7)))
    idx = torch.topk(logits + noise, topK, dim=1).indices.int()
    probs = torch.softmax(torch.randn(M, topK, device="cuda", generator=g), dim=1)
    return idx.contiguous(), probs.contiguous()


def _sorted_routes(idx, E):
    """The route tables of idx [M][topK] (every id valid): expanded_row_idx [R], cumsum [E]."""
    order = torch.sort(idx.reshape(-1), stable=True).indices
    rows = torch.empty_like(order, dtype=torch.int32)
    rows[order] = torch.arange(order.numel(), device="cuda", dtype=torch.int32)
    return rows, torch.cumsum(torch.bincount(idx.reshape(-1), minlength=E), 0).int()


def prepare(case, seed):
    c, g = dict(case), _rng(seed)
    s = {"case": c}
    if c["op"] == "route":
        x = 2.0 * torch.randn(c["M"], c["E"], device="cuda", generator=g)
        if c["masked"]:
            x[:, torch.rand(c["E"], device="cuda", generator=g) < c["masked"]] = -math.inf
            x[torch.rand(c["M"], device="cuda", generator=g) < c["masked"] / 10] = -math.inf
        s["logits"] = x.to(TYPES[c["type"]])
        s["expert_idx"] = torch.empty(c["M"], c["topK"], dtype=torch.int32, device="cuda")
        s["probs"] = torch.empty(c["M"], c["topK"], dtype=torch.float32, device="cuda")
        return s
    s["tables"] = _tables("cuda")
    if c["op"] == "quant":
        s["x"] = _activations(c["M"], c["D"], g, TYPES[c["type"]])
        s["out"] = torch.empty_like(s["x"])
        rows, D = c["M"], c["D"]
    elif c["op"] == "product":
        s["x"] = _activations(c["M"], c["D"], g, torch.float16)
        s["w"], s["ws"] = _weights(c["E"], c["N"], c["D"], g, s["tables"])
        s["w_blocks"] = _blocks(s["w"], s["ws"], False)
        idx, _ = _routing(c["M"], c["E"], c["topK"], c["skew"], g)
        s["rows"], s["cumsum"] = _sorted_routes(idx, c["E"])
        s["cap"] = int(torch.bincount(idx.reshape(-1), minlength=c["E"]).max())
        s["c"] = torch.empty(c["M"] * c["topK"], c["N"], dtype=torch.float16, device="cuda")
        rows, D = c["M"] * c["topK"], c["D"]
    else:
        s["x"] = _activations(c["M"], c["K"], g, torch.float16)
        s["w1"], s["w1s"] = _weights(c["E"], 2 * c["I"], c["K"], g, s["tables"])
        s["w2"], s["w2s"] = _weights(c["E"], c["K"], c["I"], g, s["tables"])
        s["w1_blocks"], s["w2_blocks"] = _blocks(s["w1"], s["w1s"], True), _blocks(s["w2"], s["w2s"], False)
        s["expert_idx"], s["probs"] = _routing(c["M"], c["E"], c["topK"], c["skew"], g)
        s["cap"] = int(torch.bincount(s["expert_idx"].reshape(-1), minlength=c["E"]).max())  # enough for the fullest expert
        if c["skew"]:  # requests that hit their expert's capacity: the route is dropped
            s["expert_idx"][torch.rand(c["M"], c["topK"], device="cuda", generator=g) < 0.03] = -1
        s["out"] = torch.empty(c["M"], c["K"], dtype=torch.float16, device="cuda")
        return s
    s["codes"] = torch.empty(rows, D // 2, dtype=torch.uint8, device="cuda")
    s["scales"] = torch.empty((D + 127) // 128, (rows + 3) // 4 * 4, dtype=torch.int32, device="cuda")  # words of four scale bytes, one plane per 128 of depth
    return s


# ------------------------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


def _run_own(s, c):
    import moe_expert_layer_gb300 as moe
    if c["op"] == "route":
        moe.moe_route_topk(s["logits"], s["expert_idx"], s["probs"], scoring=moe.SCORE_SIGMOID if c["score"] == "sigmoid" else moe.SCORE_SOFTMAX)
        return {"expert_idx": s["expert_idx"], "probs": s["probs"]}
    if c["op"] == "quant":
        moe.moe_mxfp4_quant(s["x"], s["codes"], s["scales"])
        moe.moe_mxfp4_dequant(s["codes"], s["scales"], s["out"])
        return s["out"]
    if c["op"] == "product":
        if "workspace" not in s:
            s["workspace"] = torch.empty(moe.moe_mxfp4_gmm_workspace_size(c["M"] * c["topK"], c["E"], c["N"], c["D"]), dtype=torch.uint8, device="cuda")
        moe.moe_mxfp4_quant(s["x"], s["codes"], s["scales"], row_map=s["rows"], copies=c["topK"])
        moe.moe_mxfp4_gmm(s["codes"], s["scales"], s["cumsum"], s["w_blocks"], s["c"], s["workspace"])
        return s["c"]
    if "workspace" not in s:
        s["dims"] = moe.dims(c["M"], c["K"], c["I"], c["E"], c["topK"])
        s["workspace"] = torch.empty(moe.moe_mxfp4_layer_workspace_size(s["dims"]), dtype=torch.uint8, device="cuda")
    moe.moe_mxfp4_layer_fwd(s["dims"], s["x"], s["expert_idx"], s["probs"], s["w1_blocks"], s["w2_blocks"], s["out"], s["workspace"])
    return s["out"]


def _run_plain(s, c):
    if c["op"] == "route":
        return _route_plain(s["logits"].float(), c["topK"], c["score"])
    if c["op"] == "quant":
        return _values(*_quantise(s["x"], s["tables"]), s["tables"]).to(s["x"].dtype)
    if c["op"] == "product":
        x = _values(*_quantise(s["x"], s["tables"]), s["tables"])
        token = torch.empty_like(s["rows"])
        token[s["rows"].long()] = torch.arange(s["rows"].numel(), device="cuda", dtype=torch.int32) // c["topK"]
        return _grouped_plain(x, token, s["cumsum"], s["cap"], _unpack(s["w"], s["ws"], s["tables"])).half()
    return _layer_plain(s, c)


def _route_plain(x, topK, score):
    masked = torch.isnan(x) | (x == -math.inf)
    x = torch.where(masked, torch.full_like(x, -math.inf), x.clamp(max=torch.finfo(torch.float32).max))
    top = torch.sort(x, dim=1, descending=True, stable=True)
    l, idx = top.values[:, :topK], top.indices[:, :topK].int()
    if score == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:  # over the whole row, though the sum cancels when the chosen are made to sum to one
        big = torch.where(masked.all(1, keepdim=True), torch.zeros_like(l[:, :1]), l[:, :1])
        p = torch.exp(l - big) / torch.exp(x - big).sum(1, keepdim=True)
    none = l == -math.inf
    p = torch.where(none, torch.zeros_like(p), p)
    total = p.sum(1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    return {"expert_idx": torch.where(none, torch.full_like(idx, -1), idx), "probs": p}


def _grouped_plain(x, token, cumsum, cap, w):
    """x [T][D] by the rows' experts: row d is x[token[d]], its expert by cumsum (rows past the last
    expert's come back with any values); w [E][N][D]; cap: rows of the fullest expert."""
    first = torch.cat([torch.zeros_like(cumsum[:1]), cumsum[:-1]])
    at = first[:, None] + torch.arange(cap, device="cuda", dtype=torch.int32)[None]
    inside = at < cumsum[:, None]
    xe = x[token[torch.where(inside, at, torch.zeros_like(at)).long()].long()]
    y = torch.bmm(xe, w.transpose(1, 2))
    row = torch.arange(token.numel(), device="cuda", dtype=torch.int32)
    e = torch.searchsorted(cumsum, row, right=True).clamp(max=cumsum.numel() - 1)
    return y[e, (row - first[e]).clamp(max=cap - 1).long()]


def _layer_plain(s, c):
    M, I, E, topK, t = c["M"], c["I"], c["E"], c["topK"], s["tables"]
    x = _values(*_quantise(s["x"], t), t)
    ei = s["expert_idx"].reshape(-1)
    kept, e = ei >= 0, ei.clamp(min=0).long()
    token = torch.arange(M * topK, device="cuda", dtype=torch.int32) // topK
    if M * topK <= E or M == 1:  # each route reads its expert's weights
        gu = torch.bmm(_unpack(s["w1"][e], s["w1s"][e], t), x[token.long()][:, :, None])[:, :, 0]
    else:  # each expert's routes together
        group = torch.where(kept, e, torch.full_like(e, E))  # dropped routes come last
        order = torch.sort(group, stable=True).indices
        cumsum = torch.cumsum(torch.bincount(group, minlength=E + 1), 0)[:E].int()
        gu = torch.empty(M * topK, 2 * I, device="cuda")
        gu[order] = _grouped_plain(x, token[order], cumsum, s["cap"], _unpack(s["w1"], s["w1s"], t))
    g, u = gu[:, :I], gu[:, I:]
    h = _values(*_quantise(g / (1.0 + torch.exp(-g)) * u, t), t)
    if M * topK <= E or M == 1:
        y = torch.bmm(_unpack(s["w2"][e], s["w2s"][e], t), h[:, :, None])[:, :, 0]
    else:
        y = torch.empty(M * topK, c["K"], device="cuda")
        y[order] = _grouped_plain(h, order.int(), cumsum, s["cap"], _unpack(s["w2"], s["w2s"], t))
    y = torch.where(kept[:, None], y, torch.zeros_like(y)) * s["probs"].reshape(-1, 1)
    return y.view(M, topK, -1).sum(1).half()


# ------------------------------------------------------------------------------------ work
def _active(M, E, topK):
    """Experts that M tokens reach, about, at topK distinct ones each."""
    return E * (1.0 - (1.0 - topK / E) ** M)


def work(case):
    c, size = case, {"f32": 4, "f16": 2, "bf16": 2}
    if c["op"] == "route":
        return {"bytes": c["M"] * (c["E"] * size[c["type"]] + 8 * c["topK"]), "flops": 4 * c["M"] * c["E"]}
    if c["op"] == "quant":  # x in; codes, scales and values out
        return {"bytes": c["M"] * c["D"] * (2 * size[c["type"]] + 17 / 32), "flops": 3 * c["M"] * c["D"]}
    R = c["M"] * c["topK"]
    if c["op"] == "product":
        w = _active(c["M"], c["E"], c["topK"]) * c["N"] * c["D"] * 17 / 32
        return {"bytes": w + 2 * c["M"] * c["D"] + 2 * R * c["N"], "flops": 2 * R * c["N"] * c["D"]}
    w = _active(c["M"], c["E"], c["topK"]) * 3 * c["K"] * c["I"] * 17 / 32
    return {"bytes": w + 4 * c["M"] * c["K"] + 8 * R, "flops": 6 * R * c["K"] * c["I"]}


# ------------------------------------------------------------------------------------ 64 bits
def _mx64(x):
    """The value that each element of x (64 bits) has after MXFP4: the nearest multiple of its binade's
    step, ties to the even multiple, at most 6, times the block's power of two."""
    b = x.unflatten(-1, (-1, 32))
    a = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a))))
    e = torch.where(torch.pow(2.0, e) > a, e - 1, e)
    e = torch.where(torch.pow(2.0, e + 1) <= a, e + 1, e)
    unit = torch.pow(2.0, (e - 2).clamp(-127, 127))
    y = b / unit
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0)).double()
    v = (torch.round(y / step) * step).clamp(-6, 6) * unit
    return torch.where(a > 0, v, torch.zeros_like(v)).flatten(-2)


def _w64(codes, scales):
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)[n]
    return (v.unflatten(-1, (-1, 32)) * torch.pow(2.0, scales.double() - 127)[..., None]).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "route":
        x, topK = s["logits"].double(), c["topK"]
        idx = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :topK]
        l = torch.gather(x, 1, idx)
        if c["score"] == "sigmoid":
            p = torch.sigmoid(l)
        else:
            p = torch.softmax(torch.where(torch.isinf(x).all(1, keepdim=True), torch.zeros_like(x), x), 1).gather(1, idx)
        none = torch.isinf(l)
        p = torch.where(none, torch.zeros_like(p), p)
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
        return {"expert_idx": torch.where(none, torch.full_like(idx, -1), idx).int(), "probs": p}
    if c["op"] == "quant":
        return _mx64(s["x"].double())
    topK, x = c["topK"], _mx64(s["x"].double())
    if c["op"] == "product":
        out = torch.empty(c["M"] * topK, c["N"], dtype=torch.float64, device="cuda")
        route = torch.sort(s["rows"].long()).indices  # the route at each row
        start = 0
        for e, end in enumerate(s["cumsum"].tolist()):
            if end > start:
                out[start:end] = x[route[start:end] // topK] @ _w64(s["w"][e], s["ws"][e]).T
            start = end
        return out
    out = torch.zeros(c["M"], c["K"], dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        t, j = torch.nonzero(s["expert_idx"] == e, as_tuple=True)
        if t.numel():
            gu = x[t] @ _w64(s["w1"][e], s["w1s"][e]).T
            g, u = gu[:, :c["I"]], gu[:, c["I"]:]
            y = _mx64(g * torch.sigmoid(g) * u) @ _w64(s["w2"][e], s["w2s"][e]).T
            out.index_add_(0, t, y * s["probs"][t, j].double()[:, None])
    return out
