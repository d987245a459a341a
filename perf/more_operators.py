"""The operators of 16-bit experts, as cases that can be timed: products grouped by expert and their
gradients, SwiGLU and its gradient, the dispatch and combine of rows with their gradients, and the
low-rank adapters of many requests.

``run`` computes each in its plain form (elementary torch operations in 32 bits) or, where ``own`` is
set, through the framework's entry points.  ``exact`` is the definition in 64 bits.

Rows are expert-major: those of expert e are cumsum[e - 1] .. cumsum[e] - 1; rows from cumsum[E - 1] on
belong to no expert and are left as they were (zeros here).
"""
import math

import torch

own = False

# ------------------------------------------------------------------------------------ cases
# Sizes are those of the repository's own workloads: decode / decode16 (K 7168, I 2048, 256 or 16
# experts, top 8) and prefill (K 4096, I 1408, 64 experts, top 6), and odd ones between them.


def listed():
    return [
        # GMM1 of one decoded token on unquantised experts: eight experts' weights stream past a row each
        {"name": "product one token", "op": "product", "M": 1, "D": 7168, "N": 4096, "E": 16, "topK": 8, "skew": 0.0, "dropped": 0.0, "type": "f16"},
        # a ragged handful of rows per expert, some routes dropped, sizes that end inside every tile
        {"name": "product odd", "op": "product", "M": 101, "D": 1400, "N": 4104, "E": 8, "topK": 2, "skew": 0.5, "dropped": 0.05, "type": "f16"},
        # GMM1 of a decode batch: the weights of every expert
        {"name": "product decode", "op": "product", "M": 128, "D": 7168, "N": 4096, "E": 256, "topK": 8, "skew": 0.0, "dropped": 0.0, "type": "bf16"},
        # GMM1 of a prefill or training batch: bound by the tensor cores
        {"name": "product prefill", "op": "product", "M": 8192, "D": 4096, "N": 2816, "E": 64, "topK": 6, "skew": 0.0, "dropped": 0.0, "type": "bf16"},
        # both gradients of a small fine-tuning batch on a few experts, one of them often without rows
        {"name": "gradients odd", "op": "gradients", "M": 301, "D": 1024, "N": 1416, "E": 8, "topK": 2, "skew": 1.2, "dropped": 0.05, "type": "f16", "master": False},
        # both gradients of GMM2 of a training batch, the weights' in 32 bits as an optimizer keeps them
        {"name": "gradients training", "op": "gradients", "M": 8192, "D": 1408, "N": 4096, "E": 64, "topK": 6, "skew": 0.0, "dropped": 0.0, "type": "bf16", "master": True},
        # the activation between the products of a decode batch, forwards and backwards
        {"name": "swiglu decode", "op": "swiglu", "R": 1024, "I": 2048, "dropped": 0.0, "type": "bf16"},
        # the same of a training batch
        {"name": "swiglu training", "op": "swiglu", "R": 49152, "I": 1408, "dropped": 0.02, "type": "bf16"},
        # a few tokens to their experts' rows and back, with the gradients
        {"name": "combine few", "op": "combine", "M": 61, "D": 7168, "topK": 8, "E": 16, "dropped": 0.05, "type": "f16"},
        # the same of a training batch
        {"name": "combine training", "op": "combine", "M": 8192, "D": 4096, "topK": 6, "E": 64, "dropped": 0.02, "type": "bf16"},
        # a decode batch of requests that each brought an adapter, beside a projection they share
        {"name": "adapters decode", "op": "adapters", "M": 128, "D": 7168, "N": 4096, "rank": 16, "L": 100, "bare": 0.1, "prompt": 1, "type": "bf16"},
        # prompts of many requests, a few adapters of a larger rank
        {"name": "adapters prefill", "op": "adapters", "M": 8192, "D": 4096, "N": 4096, "rank": 64, "L": 24, "bare": 0.1, "prompt": 256, "type": "f16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "gradients", "swiglu", "combine", "adapters"])
    case = {"op": op, "type": rng.choice(["f16", "bf16"])}
    if op in ("product", "gradients"):
        E = _log_int(rng, 1, 64)
        case.update(M=_log_int(rng, 1, 4096), D=8 * _log_int(rng, 8, 512), N=8 * _log_int(rng, 8, 352), E=E, topK=rng.randint(1, min(E, 8)),
                    skew=rng.choice([0.0, 0.5, 1.2]), dropped=rng.choice([0.0, 0.05]))
        if op == "gradients":
            case["master"] = rng.random() < 0.5
    elif op == "swiglu":
        case.update(R=_log_int(rng, 1, 32768), I=8 * _log_int(rng, 8, 256), dropped=rng.choice([0.0, 0.05, 0.5]))
    elif op == "combine":
        E = _log_int(rng, 1, 128)
        case.update(M=_log_int(rng, 1, 4096), D=8 * _log_int(rng, 8, 896), topK=rng.randint(1, min(E, 10)), E=E, dropped=rng.choice([0.0, 0.05, 0.5]))
    else:
        case.update(M=_log_int(rng, 1, 4096), D=8 * _log_int(rng, 8, 896), N=8 * _log_int(rng, 8, 512), rank=8 * rng.randint(1, 16), L=_log_int(rng, 1, 128),
                    bare=rng.choice([0.0, 0.1, 0.5]), prompt=rng.choice([1, 1, 40, 300]))
    return case


# ------------------------------------------------------------------------------------ inputs
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(M, D, g, dtype, size=1.0):
    """Hidden states: each row has its own size, some channels are much larger than the rest."""
    x = torch.randn(M, D, device="cuda", generator=g)
    x *= size * torch.exp(0.3 * torch.randn(M, 1, device="cuda", generator=g))
    x *= torch.where(torch.rand(1, D, device="cuda", generator=g) < 0.01, 8.0, 1.0)
    return x.to(dtype)


def _weights(E, N, D, g, dtype, fan):
    """Weights of N(0, 1 / fan)."""
    w = torch.randn(E, N, D, device="cuda", generator=g, dtype=dtype)
    return w.mul_(1.0 / math.sqrt(fan))


def _routing(M, E, topK, skew, dropped, g):
    """Distinct experts per token (a share of popular ones where skew > 0), -1 where a route hit its
    expert's capacity, and softmax weights."""
    logits = -skew * torch.log(1 + torch.randperm(E, device="cuda", generator=g).float())[None].expand(M, E)
    noise = -torch.log(-torch.log(torch.rand(M, E, device="cuda", generator=g).clamp(1e-20, 1 - 1e-7)))
    idx = torch.topk(logits + noise, topK, dim=1).indices.int()
    idx = torch.where(torch.rand(M, topK, device="cuda", generator=g) < dropped, torch.full_like(idx, -1), idx)
    probs = torch.softmax(torch.randn(M, topK, device="cuda", generator=g), dim=1)
    return idx.contiguous(), probs.contiguous()


def _sorted_routes(idx, E):
    """The tables of idx (any shape): the route at each row, the row of each route (-1: dropped), cumsum [E]."""
    flat = idx.reshape(-1)
    group = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.sort(group, stable=True).indices
    rows = torch.empty_like(order, dtype=torch.int32)
    rows[order] = torch.arange(order.numel(), device="cuda", dtype=torch.int32)
    cumsum = torch.cumsum(torch.bincount(group, minlength=E + 1), 0)[:E].int()
    return order.int(), torch.where(flat < 0, torch.full_like(rows, -1), rows), cumsum


def prepare(case, seed):
    c, g = dict(case), _rng(seed)
    t = TYPES[c["type"]]
    s = {"case": c}
    if c["op"] in ("product", "gradients"):
        idx, _ = _routing(c["M"], c["E"], c["topK"], c["skew"], c["dropped"], g)
        route, _, s["cumsum"] = _sorted_routes(idx, c["E"])
        s["ends"] = s["cumsum"].tolist()
        s["a"] = _activations(c["M"], c["D"], g, t)[route.long() // c["topK"]]
        s["w"] = _weights(c["E"], c["N"], c["D"], g, t, c["D"])
        R = c["M"] * c["topK"]
        if c["op"] == "product":
            s["c"] = torch.zeros(R, c["N"], dtype=t, device="cuda")
        else:
            s["dc"] = _activations(R, c["N"], g, t, 0.02)
            s["da"] = torch.zeros(R, c["D"], dtype=t, device="cuda")
            s["dw"] = torch.zeros(c["E"], c["N"], c["D"], dtype=torch.float32 if c["master"] else t, device="cuda")
    elif c["op"] == "swiglu":
        R, I = c["R"], c["I"]
        s["gu"], s["dh"] = _activations(R, 2 * I, g, t, 1.5), _activations(R, I, g, t, 0.05)
        # 64 experts of about the same size, the rows of dropped routes behind theirs
        valid = R - int(c["dropped"] * R)
        s["cumsum"] = torch.arange(1, 65, device="cuda").mul(valid).div(64, rounding_mode="floor").int()
        s["valid"] = valid
        s["h"], s["dgu"] = torch.zeros(R, I, dtype=t, device="cuda"), torch.zeros(R, 2 * I, dtype=t, device="cuda")
    elif c["op"] == "combine":
        M, D, topK = c["M"], c["D"], c["topK"]
        idx, s["probs"] = _routing(M, c["E"], topK, 0.0, c["dropped"], g)
        _, s["row_map"], _ = _sorted_routes(idx, c["E"])
        s["x"], s["dout"] = _activations(M, D, g, t), _activations(M, D, g, t, 0.05)
        s["y"] = _activations(M * topK, D, g, t)
        s["a"], s["dy"] = torch.zeros(M * topK, D, dtype=t, device="cuda"), torch.zeros(M * topK, D, dtype=t, device="cuda")
        s["out"], s["dprobs"] = torch.zeros(M, D, dtype=t, device="cuda"), torch.zeros(M, topK, device="cuda")
    else:
        M, D, N, r, L = c["M"], c["D"], c["N"], c["rank"], c["L"]
        per = torch.randint(0, L, ((M + c["prompt"] - 1) // c["prompt"],), device="cuda", generator=g, dtype=torch.int32)
        per = torch.where(torch.rand(per.numel(), device="cuda", generator=g) < c["bare"], torch.full_like(per, -1), per)
        idx = per.repeat_interleave(c["prompt"])[:M].contiguous()
        s["adapter"] = idx
        s["route"], _, s["cumsum"] = _sorted_routes(idx, L)
        s["ends"] = s["cumsum"].tolist()
        s["x"], s["base"] = _activations(M, D, g, t), _activations(M, N, g, t)
        s["a"] = _weights(L, r, D, g, t, D)
        s["b"] = _weights(L, N, r, g, t, 4 * r)
        s["scales"] = 0.5 + torch.rand(L, device="cuda", generator=g)
        s["out"] = torch.zeros(M, N, dtype=t, device="cuda")
    return s


# ------------------------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


def _run_own(s, c):
    import moe_expert_layer_gb300 as moe
    if c["op"] in ("product", "gradients"):
        if "workspace" not in s:
            s["workspace"] = torch.empty(moe.moe_gmm16_workspace_size(s["a"].shape[0], c["E"], c["N"], c["D"]), dtype=torch.uint8, device="cuda")
        if c["op"] == "product":
            moe.moe_gmm16(s["a"], s["cumsum"], s["w"], s["c"], s["workspace"])
            return s["c"]
        moe.moe_gmm16_input_grad(s["dc"], s["cumsum"], s["w"], s["da"], s["workspace"])
        moe.moe_gmm16_weight_grad(s["dc"], s["a"], s["cumsum"], s["dw"], s["workspace"])
        return {"da": s["da"], "dw": s["dw"]}
    if c["op"] == "swiglu":
        moe.moe_swiglu16(s["gu"], s["cumsum"], s["h"])
        moe.moe_swiglu16_grad(s["dh"], s["gu"], s["cumsum"], s["dgu"])
        return {"h": s["h"], "dgu": s["dgu"]}
    if c["op"] == "combine":
        moe.moe_dispatch16(s["x"], s["row_map"], s["a"], copies=c["topK"])
        moe.moe_combine16(s["y"], s["row_map"], s["probs"], s["out"], copies=c["topK"])
        moe.moe_combine16_grad(s["dout"], s["y"], s["row_map"], s["probs"], s["dy"], s["dprobs"], copies=c["topK"])
        return {"a": s["a"], "out": s["out"], "dy": s["dy"], "dprobs": s["dprobs"]}
    if "workspace" not in s:
        s["workspace"] = torch.empty(moe.moe_lora16_workspace_size(c["M"], c["N"], c["D"], c["rank"]), dtype=torch.uint8, device="cuda")
    moe.moe_lora16(s["x"], s["route"], s["cumsum"], s["a"], s["b"], s["base"], s["out"], s["workspace"], scales=s["scales"])
    return s["out"]


def _groups(ends):
    """(expert, first row, last row + 1) of the experts that have rows."""
    start = 0
    for e, end in enumerate(ends):
        if end > start:
            yield e, start, end
        start = end


def _run_plain(s, c):
    t = TYPES[c["type"]]
    if c["op"] == "product":
        out = torch.zeros(s["a"].shape[0], c["N"], dtype=t, device="cuda")
        for e, lo, hi in _groups(s["ends"]):
            out[lo:hi] = (s["a"][lo:hi].float() @ s["w"][e].float().T).to(t)
        return out
    if c["op"] == "gradients":
        da = torch.zeros_like(s["da"])
        dw = torch.zeros_like(s["dw"])
        for e, lo, hi in _groups(s["ends"]):
            dc = s["dc"][lo:hi].float()
            da[lo:hi] = (dc @ s["w"][e].float()).to(t)
            dw[e] = (dc.T @ s["a"][lo:hi].float()).to(dw.dtype)
        return {"da": da, "dw": dw}
    if c["op"] == "swiglu":
        n, I = s["valid"], c["I"]
        h, dgu = torch.zeros_like(s["h"]), torch.zeros_like(s["dgu"])
        g, u, dh = s["gu"][:n, :I].float(), s["gu"][:n, I:].float(), s["dh"][:n].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        h[:n] = (g * sig * u).to(t)
        dgu[:n, :I] = (dh * u * sig * (1.0 + g * (1.0 - sig))).to(t)
        dgu[:n, I:] = (dh * g * sig).to(t)
        return {"h": h, "dgu": dgu}
    if c["op"] == "combine":
        M, D, topK = c["M"], c["D"], c["topK"]
        row = s["row_map"].view(M, topK)
        a, dy = torch.zeros_like(s["a"]), torch.zeros_like(s["dy"])
        out = torch.zeros(M, D, device="cuda")
        dprobs = torch.zeros(M, topK, device="cuda")
        dout = s["dout"].float()
        for j in range(topK):
            here = torch.nonzero(row[:, j] >= 0)[:, 0]
            r, p = row[here, j].long(), s["probs"][here, j, None]
            a[r] = s["x"][here]
            y = s["y"][r].float()
            out[here] += p * y
            dy[r] = (p * dout[here]).to(t)
            dprobs[here, j] = (dout[here] * y).sum(1)
        return {"a": a, "out": out.to(t), "dy": dy, "dprobs": dprobs}
    out = s["base"].clone()
    for l, lo, hi in _groups(s["ends"]):
        token = s["route"][lo:hi].long()
        v = s["x"][token].float() @ s["a"][l].float().T
        out[token] = (s["base"][token].float() + s["scales"][l] * (v @ s["b"][l].float().T)).to(t)
    return out


# ------------------------------------------------------------------------------------ work
def _active(M, E, topK):
    """Experts that M tokens reach, about, at topK distinct ones each."""
    return E * (1.0 - (1.0 - topK / E) ** M)


def work(case):
    c = case
    if c["op"] in ("product", "gradients"):
        R, ND = c["M"] * c["topK"] * (1.0 - c["dropped"]), c["N"] * c["D"]
        w, rows = 2 * _active(c["M"], c["E"], c["topK"]) * ND, 2 * R * (c["N"] + c["D"])
        if c["op"] == "product":
            return {"bytes": w + rows, "flops": 2 * R * ND}
        return {"bytes": w + rows + 2 * R * c["D"] + (4 if c["master"] else 2) * c["E"] * ND, "flops": 4 * R * ND}
    if c["op"] == "swiglu":  # gu, dh in; h, dgu out
        n = c["R"] * (1.0 - c["dropped"]) * c["I"]
        return {"bytes": 2 * n * 6, "flops": 24 * n}
    if c["op"] == "combine":  # x, y, dout in; a, out, dy out
        R = c["M"] * c["topK"] * (1.0 - c["dropped"])
        return {"bytes": 2 * c["D"] * (3 * c["M"] + 3 * R) + 12 * R, "flops": 5 * R * c["D"]}
    M, r = c["M"] * (1.0 - c["bare"]), c["rank"]
    live = min(c["L"], _active(max(1, M / c["prompt"]), c["L"], 1))
    return {"bytes": 2 * (M * c["D"] + 2 * c["M"] * c["N"] + live * r * (c["D"] + c["N"])), "flops": 2 * M * r * (c["D"] + c["N"])}


# ------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "product":
        out = torch.zeros(s["c"].shape, dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            rows = slice(s["ends"][e - 1] if e else 0, s["ends"][e])
            out[rows] = torch.einsum("dk,nk->dn", s["a"][rows].double(), s["w"][e].double())
        return out
    if c["op"] == "gradients":
        da = torch.zeros(s["da"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(s["dw"].shape, dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            rows = slice(s["ends"][e - 1] if e else 0, s["ends"][e])
            dc = s["dc"][rows].double()
            da[rows] = torch.einsum("dn,nk->dk", dc, s["w"][e].double())
            dw[e] = torch.einsum("dn,dk->nk", dc, s["a"][rows].double())
        return {"da": da, "dw": dw}
    if c["op"] == "swiglu":
        x, dh = s["gu"].double(), s["dh"].double()
        g, u = x[:, :c["I"]], x[:, c["I"]:]
        sig = torch.special.expit(g)
        dg = u * dh * (sig + g * sig * torch.special.expit(-g))
        keep = (torch.arange(c["R"], device="cuda") < s["cumsum"][-1])[:, None].double()
        return {"h": g * sig * u * keep, "dgu": torch.cat([dg, dh * g * sig], 1) * keep}
    if c["op"] == "combine":
        M, topK = c["M"], c["topK"]
        token = torch.arange(M * topK, device="cuda") // topK
        kept = torch.nonzero(s["row_map"] >= 0)[:, 0]
        row, token = s["row_map"][kept].long(), token[kept]
        p = s["probs"].double().reshape(-1)[kept]
        a, dy = (torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        dprobs = torch.zeros(M * topK, dtype=torch.float64, device="cuda")
        y, dout = s["y"].double()[row], s["dout"].double()[token]
        a[row] = s["x"].double()[token]
        out.index_add_(0, token, y * p[:, None])
        dy[row] = dout * p[:, None]
        dprobs[kept] = torch.einsum("rd,rd->r", dout, y)
        return {"a": a, "out": out, "dy": dy, "dprobs": dprobs.view(M, topK)}
    out = s["base"].double()
    for l in range(c["L"]):
        token = torch.nonzero(s["adapter"] == l)[:, 0]
        if token.numel():
            v = torch.einsum("td,rd->tr", s["x"][token].double(), s["a"][l].double())
            out[token] += s["scales"][l].double() * torch.einsum("tr,nr->tn", v, s["b"][l].double())
    return out
