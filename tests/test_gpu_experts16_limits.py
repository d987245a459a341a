"""The operators of 16-bit experts at the ends of their documented sizes, and from several host threads."""
import threading

import pytest

import experts16_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_expert_layer_gb300 as moe
    from test_gpu_experts16 import F32, ints, marked, prefix, rng, space
    from test_gpu_experts16_use import Step, same

F16, BF16 = torch.float16, torch.bfloat16
MOST = (1 << 24) - 1  # rows
SIDE = 65536          # channels


def sampled(n):
    return torch.tensor([0, 1, 63, 64, n // 3, n // 2, n - 65, n - 2, n - 1], device="cuda")


@pytest.mark.parametrize("counts", [[MOST], [5, MOST - 12, 0, 7]])
def test_products_of_most_rows(counts):
    g, N, D, E = rng(1), 72, 64, len(counts)
    a, dc, w = ints((MOST, D), F16, g, 2), ints((MOST, N), F16, g, 1), ints((E, N, D), F16, g, 2)
    cumsum, ws = prefix(counts), space(MOST, E, N, D)
    c, da = marked((MOST, N), F16), marked((MOST, D), F16)
    moe.moe_gmm16(a, cumsum, w, c, ws)
    moe.moe_gmm16_input_grad(dc, cumsum, w, da, ws)
    assert moe.moe_workspace_status(ws) == 0
    ends = cumsum.tolist()
    for lo in range(0, MOST, 1 << 20):
        hi = min(MOST, lo + (1 << 20))
        part = [min(max(e - lo, 0), hi - lo) for e in ends]
        assert torch.equal(c[lo:hi].double(), ref.product(a[lo:hi], part, w))
        assert torch.equal(da[lo:hi].double(), ref.input_grad(dc[lo:hi], part, w))


def test_row_operators_of_most_rows():
    g, D, t = rng(2), 8, BF16
    x, y = ints((MOST, D), t, g), ints((MOST, D), t, g)
    row_map = torch.randperm(MOST, device="cuda", generator=g).int()
    dropped = torch.rand(MOST, device="cuda", generator=g) < 0.1
    row_map = torch.where(dropped, -1, row_map).int()
    kept = (~dropped).nonzero()[:, 0]
    row = row_map[kept].long()
    out = marked((MOST, D), t)
    moe.moe_dispatch16(x, row_map, out)
    want = marked((MOST, D), t)
    want[row] = x[kept]
    assert torch.equal(out, want)
    moe.moe_combine16(y, row_map, None, out)
    want.zero_()
    want[kept] = y[row]
    assert torch.equal(out, want)
    probs, dprobs, dy = torch.full((MOST,), 2.0, device="cuda"), marked((MOST,), F32), marked((MOST, D), t)
    moe.moe_combine16_grad(x, y, row_map, probs, dy, dprobs)
    want.fill_(-7)
    want[row] = 2 * x[kept]
    assert torch.equal(dy, want)
    want_p = torch.zeros(MOST, device="cuda")
    want_p[kept] = (x[kept].float() * y[row].float()).sum(1)
    assert torch.equal(dprobs, want_p)
    gu, cumsum, h = ints((MOST, 16), t, g), prefix([3, MOST - 5]), marked((MOST, 8), t)
    dgu, h2, dh = marked((MOST, 16), t), marked((MOST, 8), t), y
    moe.moe_swiglu16(gu, cumsum, h)
    moe.moe_swiglu16_grad(dh, gu, cumsum, dgu, h2)
    assert torch.equal(h, h2) and (h[-2:] == -7).all() and (dgu[-2:] == -7).all()
    at = sampled(MOST - 2)
    for got, want in ((h[at], ref.swiglu(gu[at])), (dgu[at], ref.swiglu_grad(dh[at], gu[at]))):
        assert ((got.double() - want).abs() <= want.abs() * 2.0 ** -15 + 2.0 ** -17 + ref.half_step(t, want)).all()


def test_adapters_of_most_tokens():
    g, D, N, r = rng(3), 64, 72, 8
    x, base = ints((MOST, D), F16, g, 1), ints((MOST, N), F16, g, 4)
    a, b = ints((2, r, D), F16, g, 1), ints((2, N, r), F16, g, 1)
    adapter = torch.arange(MOST, device="cuda") % 3  # the third has none
    route = torch.cat([torch.arange(k, MOST, 3, device="cuda") for k in range(3)]).int()
    cumsum = prefix([(adapter == 0).sum().item(), (adapter == 1).sum().item()])
    ws = torch.empty(moe.moe_lora16_workspace_size(MOST, N, D, r), dtype=torch.uint8, device="cuda")
    out = marked((MOST, N), F16)
    moe.moe_lora16(x, route, cumsum, a, b, base, out, ws)
    for lo in range(0, MOST, 1 << 20):
        s = slice(lo, min(MOST, lo + (1 << 20)))
        assert torch.equal(out[s].double(), ref.lora(x[s], adapter[s], a, b, None, base[s]))


def test_products_of_most_channels():
    """65536 x 65536 weights of one expert, three rows."""
    g, R = rng(4), 3
    w = torch.zeros((1, SIDE, SIDE), dtype=BF16, device="cuda")
    at = torch.randint(0, SIDE, (2, 20000), device="cuda", generator=g)
    at[:, 0], at[:, 1], at[:, 2] = 0, SIDE - 1, torch.tensor([SIDE - 1, 0], device="cuda")
    w[0, at[0], at[1]] = ints((20000,), BF16, g, 2)
    rows = ints((R, SIDE), BF16, g, 2)
    cumsum, ws = prefix([R]), space(R, 1, SIDE, SIDE)
    c, da = marked((R, SIDE), BF16), marked((R, SIDE), BF16)
    moe.moe_gmm16(rows, cumsum, w, c, ws)
    moe.moe_gmm16_input_grad(rows, cumsum, w, da, ws)
    sparse = w[0, at[0], at[1]].double()
    pairs = torch.unique(at[0] * SIDE + at[1], return_inverse=True)[1]
    once = torch.zeros(pairs.max() + 1, dtype=torch.long, device="cuda").scatter_(0, pairs, torch.arange(20000, device="cuda"))
    n, k, v = at[0][once], at[1][once], sparse[once]
    want_c, want_da = (torch.zeros((R, SIDE), dtype=torch.float64, device="cuda") for _ in range(2))
    want_c.index_add_(1, n, rows[:, k].double() * v)
    want_da.index_add_(1, k, rows[:, n].double() * v)
    assert torch.equal(c.double(), want_c) and torch.equal(da.double(), want_da)
    moe.moe_gmm16_weight_grad(rows, rows, cumsum, w, ws)
    for lo in range(0, SIDE, 8192):
        want = rows[:, lo:lo + 8192].float().T @ rows.float()
        assert torch.equal(w[0, lo:lo + 8192], want.to(BF16))
    assert moe.moe_workspace_status(ws) == 0


def test_from_several_host_threads():
    """Steps of their own on streams of their own, from threads that start at once."""
    sizes = [(1, 256, 64, 4, 2), (40, 384, 128, 8, 3), (700, 512, 256, 6, 2), (3000, 512, 512, 2, 2)]
    steps = [Step(i, *s) for i, s in enumerate(sizes)]
    for s in steps:
        s.run(wait=True)
    want = [s.results() for s in steps]
    torch.cuda.synchronize()
    gate, errors = threading.Barrier(len(steps)), []

    def work(s, w):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait()
                for _ in range(20):
                    s.run()
                    assert same(s.results(), w)
                    assert moe.moe_workspace_status(s.ws) == 0
        except Exception as e:  # seen by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(steps, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
