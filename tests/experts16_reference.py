"""The operators of 16-bit experts in 64 bits, plainly, for the tests: elementary torch operations
on the inputs' device, no code of the library."""
import torch


def groups(ends):
    """(expert, first row, last row + 1) of every expert; entries of `ends` are the inclusive prefix."""
    start = 0
    for e, end in enumerate(ends):
        yield e, start, max(start, end)
        start = max(start, end)


def product(a, ends, w):
    """c [R][N]; rows of no expert are 0."""
    c = torch.zeros(a.shape[0], w.shape[1], dtype=torch.float64, device=a.device)
    for e, lo, hi in groups(ends):
        c[lo:hi] = a[lo:hi].double() @ w[e].double().T
    return c


def input_grad(dc, ends, w):
    da = torch.zeros(dc.shape[0], w.shape[2], dtype=torch.float64, device=dc.device)
    for e, lo, hi in groups(ends):
        da[lo:hi] = dc[lo:hi].double() @ w[e].double()
    return da


def weight_grad(dc, a, ends):
    dw = torch.zeros(len(ends), dc.shape[1], a.shape[1], dtype=torch.float64, device=a.device)
    for e, lo, hi in groups(ends):
        dw[e] = dc[lo:hi].double().T @ a[lo:hi].double()
    return dw


def swiglu(gu):
    g, u = gu.double().chunk(2, 1)
    return g * torch.sigmoid(g) * u


def swiglu_grad(dh, gu):
    g, u = gu.double().chunk(2, 1)
    s, dh = torch.sigmoid(g), dh.double()
    return torch.cat([dh * u * s * (1 + g * torch.sigmoid(-g)), dh * g * s], 1)


def combine(y, row_map, probs):
    """out [M][D] from y [rows][D], row_map [M][copies] (entries outside [0, rows) skipped)."""
    kept = (row_map >= 0) & (row_map < y.shape[0])
    v = y.double()[row_map.clamp(0, y.shape[0] - 1).long()] * (1.0 if probs is None else probs.double()[..., None])
    return torch.where(kept[..., None], v, torch.zeros_like(v)).sum(1)


def combine_grad(dout, y, row_map, probs):
    """dy [rows][D] (0 where no entry names the row), dprobs [M][copies]."""
    kept = (row_map >= 0) & (row_map < y.shape[0])
    t, j = kept.nonzero(as_tuple=True)
    row = row_map[t, j].long()
    dy = torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    dy[row] = probs[t, j].double()[:, None] * dout[t].double()
    dprobs = torch.zeros(row_map.shape, dtype=torch.float64, device=y.device)
    dprobs[t, j] = (dout[t].double() * y[row].double()).sum(1)
    return dy, dprobs


def lora(x, adapter, a, b, scales, base):
    out = base.double()
    for l in range(a.shape[0]):
        t = (adapter == l).nonzero()[:, 0]
        v = x[t].double() @ a[l].double().T
        out[t] += (1.0 if scales is None else scales[l].double()) * (v @ b[l].double().T)
    return out


def tables(idx, n):
    """Of expert (or adapter) ids of any shape, sorted stably, ids outside [0, n) last: the route at each row, the
    row of each route (-1 where it has none) and the inclusive prefix of the counts."""
    flat = idx.reshape(-1).long()
    group = torch.where((flat < 0) | (flat >= n), torch.full_like(flat, n), flat)
    route = torch.sort(group, stable=True).indices
    row = torch.empty_like(route)
    row[route] = torch.arange(route.numel(), device=idx.device)
    row = torch.where(group == n, torch.full_like(row, -1), row)
    cumsum = torch.cumsum(torch.bincount(group, minlength=n + 1), 0)[:n]
    return route.int(), row.int(), cumsum.int()


def half_step(t, v):
    """What rounding the values v to type t may move them by: half a step, relative, or half the smallest
    subnormal."""
    f = torch.finfo(t)
    return v.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def rounded(v, t):
    """64-bit values rounded to nearest even once, saturating in binary16."""
    if t == torch.float16:
        v = v.clamp(-65504.0, 65504.0)
    if t == torch.bfloat16:  # by hand: a conversion through fp32 would round twice
        m, e = torch.frexp(v)
        step = torch.ldexp(torch.ones_like(v), (e - 8).clamp(min=-133))
        return (torch.round(v / step) * step).to(t)
    return v.to(t)
