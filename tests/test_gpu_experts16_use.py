"""The operators of 16-bit experts as programs call them: captured and replayed, on several streams at
once, one right behind the other, repeatedly, and past 32-bit offsets."""
import os
import subprocess
import sys

import pytest

import experts16_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_expert_layer_gb300 as moe
    from test_gpu_experts16 import F32, ints, normal, prefix, rng, space
    from test_gpu_mxfp4_waits import narrow_stream  # noqa: F401  (a fixture)

F16, BF16 = torch.float16, torch.bfloat16


class Step:
    """One training step of a layer with adapters, on its own buffers: every operator behind the other."""

    def __init__(self, seed, M, K, I, E, topK, t=BF16):
        g = rng(seed)
        self.M, self.topK, R = M, topK, M * topK
        self.x, self.dout = normal((M, K), t, g), normal((M, K), t, g)
        self.w1, self.w2 = normal((E, 2 * I, K), t, g, K ** -0.5), normal((E, K, I), t, g, I ** -0.5)
        idx = torch.stack([torch.randperm(E, device="cuda", generator=g)[:topK] for _ in range(M)]).int()
        idx[torch.rand(idx.shape, device="cuda", generator=g) < 0.05] = -1
        self.probs = torch.rand(M, topK, device="cuda", generator=g)
        _, self.rows, self.cumsum = ref.tables(idx, E)
        self.route, _, self.lcum = ref.tables(torch.randint(-1, 3, (M,), device="cuda", generator=g), 3)
        self.la, self.lb = normal((3, 16, K), t, g, K ** -0.5), normal((3, K, 16), t, g)
        z = lambda *s: torch.zeros(s, dtype=t, device="cuda")
        self.a, self.gu, self.h, self.y, self.out, self.out2 = z(R, K), z(R, 2 * I), z(R, I), z(R, K), z(M, K), z(M, K)
        self.dy, self.dh, self.dgu, self.da, self.dx = z(R, K), z(R, I), z(R, 2 * I), z(R, K), z(M, K)
        self.dprobs = torch.zeros(M, topK, device="cuda")
        self.dw1, self.dw2 = torch.zeros(w1_shape(E, I, K), device="cuda"), z(E, K, I)
        self.ws = torch.empty(max(moe.moe_gmm16_workspace_size(R, E, 2 * I, K), moe.moe_gmm16_workspace_size(R, E, K, I)),
                              dtype=torch.uint8, device="cuda")
        self.lws = torch.empty(moe.moe_lora16_workspace_size(M, K, K, 16), dtype=torch.uint8, device="cuda")

    def calls(self):
        s, k = self, self.topK
        return [
            lambda: moe.moe_dispatch16(s.x, s.rows, s.a, copies=k),
            lambda: moe.moe_gmm16(s.a, s.cumsum, s.w1, s.gu, s.ws),
            lambda: moe.moe_swiglu16(s.gu, s.cumsum, s.h),
            lambda: moe.moe_gmm16(s.h, s.cumsum, s.w2, s.y, s.ws),
            lambda: moe.moe_combine16(s.y, s.rows, s.probs, s.out, copies=k),
            lambda: moe.moe_lora16(s.x, s.route, s.lcum, s.la, s.lb, s.out, s.out2, s.lws),
            lambda: moe.moe_combine16_grad(s.dout, s.y, s.rows, s.probs, s.dy, s.dprobs, copies=k),
            lambda: moe.moe_gmm16_input_grad(s.dy, s.cumsum, s.w2, s.dh, s.ws),
            lambda: moe.moe_gmm16_weight_grad(s.dy, s.h, s.cumsum, s.dw2, s.ws),
            lambda: moe.moe_swiglu16_grad(s.dh, s.gu, s.cumsum, s.dgu),
            lambda: moe.moe_gmm16_input_grad(s.dgu, s.cumsum, s.w1, s.da, s.ws),
            lambda: moe.moe_gmm16_weight_grad(s.dgu, s.a, s.cumsum, s.dw1, s.ws, accumulate=True),
            lambda: moe.moe_combine16(s.da, s.rows, None, s.dx, copies=k),
        ]

    def run(self, wait=False):
        self.dw1.zero_()
        for c in self.calls():
            c()
            if wait:
                torch.cuda.synchronize()

    def results(self):
        return [v.clone() for v in (self.out, self.out2, self.dprobs, self.dw1, self.dw2, self.dx)]


def w1_shape(E, I, K):
    return (E, 2 * I, K)


# the last two: rows and pieces of many tokens, and weight gradients whose rows are divided, or in parts
SIZES = [(1, 256, 64, 4, 2), (40, 384, 128, 8, 3), (700, 512, 256, 6, 2), (3000, 512, 512, 2, 2), (4000, 1024, 512, 8, 2)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("sizes", SIZES)
def test_calls_right_behind_one_another_and_repeatedly(sizes):
    """Kernels start while the one before still runs: a step waited for call by call, and forty without."""
    s = Step(1, *sizes)
    s.run(wait=True)
    want = s.results()
    for _ in range(40):
        s.out.zero_(), s.dx.zero_(), s.y.zero_(), s.da.zero_()
        s.run()
        assert same(s.results(), want)
    assert moe.moe_workspace_status(s.ws) == 0


@pytest.mark.parametrize("sizes", SIZES)
def test_captured_and_replayed(sizes):
    """A graph of the whole step gives what the calls give, again when its inputs have changed, beside a second graph
    with its own buffers on another stream."""
    a, b = Step(1, *sizes), Step(2, *sizes)
    other = Step(3, *sizes)
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, stream in zip((a, b), streams):
        s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            s.run()
        graphs.append(g)
    want = []
    for s in (a, b):
        s.run(wait=True)
        want.append(s.results())
    for s in (a, b):
        for v in (s.out, s.out2, s.dprobs, s.dw1, s.dw2, s.dx):
            v.fill_(5)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    assert same(a.results(), want[0]) and same(b.results(), want[1])
    for n in ("x", "dout", "w1", "w2", "rows", "cumsum", "probs", "la", "lb", "route", "lcum"):
        getattr(a, n).copy_(getattr(other, n))
    other.run(wait=True)
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert same(a.results(), other.results())


def test_on_several_streams_at_once():
    """Steps of different sizes on streams of two priorities, none ordered with another."""
    steps = [Step(i, *SIZES[i % 5]) for i in range(6)]
    for s in steps:
        s.run(wait=True)
    want = [s.results() for s in steps]
    streams = [torch.cuda.Stream(priority=p) for p in (0, -1, 0, -1, 0, -1)]
    torch.cuda.synchronize()
    for _ in range(15):
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.run()
    torch.cuda.synchronize()
    assert all(same(s.results(), w) for s, w in zip(steps, want))
    for s in steps:
        assert moe.moe_workspace_status(s.ws) == 0


@pytest.mark.parametrize("rows,E,N,D", [(20, 9, 2568, 4104), (3, 1, 4096, 4096), (100, 3, 512, 2048)])
def test_products_repeat_to_the_bit(rows, E, N, D):
    """Sums that a cluster divides are added in the same order every time."""
    g, R = rng(5), rows * E
    a, w = normal((R, D), BF16, g), normal((E, N, D), BF16, g)
    cumsum, ws = prefix([rows] * E), space(R, E, N, D)
    first = torch.empty((R, N), dtype=BF16, device="cuda")
    moe.moe_gmm16(a, cumsum, w, first, ws)
    for _ in range(20):
        again = torch.zeros_like(first)
        moe.moe_gmm16(a, cumsum, w, again, ws)
        assert torch.equal(again, first)


@pytest.mark.parametrize("rows,E,N,D", [(3000, 1, 512, 520), (2000, 3, 200, 264), (1500, 16, 1024, 512), (100, 8, 512, 512)])
def test_weight_gradients_repeat_to_the_bit(rows, E, N, D):
    """Sums over parts, and over a cluster that divides the rows, are added in the same order every time."""
    g, R = rng(6), rows * E
    a, dc = normal((R, D), BF16, g), normal((R, N), BF16, g)
    cumsum, ws = prefix([rows] * E), space(R, E, N, D)
    first = torch.empty((E, N, D), device="cuda")
    moe.moe_gmm16_weight_grad(dc, a, cumsum, first, ws)
    for _ in range(20):
        again = torch.zeros_like(first)
        moe.moe_gmm16_weight_grad(dc, a, cumsum, again, ws)
        assert torch.equal(again, first)


def test_rows_past_32_bit_offsets():
    """300,000 rows of 8192: 2.46e9 elements, the last rows included, through every operator."""
    g, R, D, N = rng(2), 300_000, 8192, 64
    at = torch.tensor([0, 1, 149_999, 150_000, 262_144, R - 1], device="cuda")
    small = ints((1000, D), F16, g, 1)
    a = small.repeat(R // 1000, 1)
    w = ints((2, N, D), F16, g, 1)
    w *= (torch.arange(D, device="cuda") % 8 == 0)
    cumsum, ws = prefix([150_000, 150_000]), space(R, 2, N, D)
    c = torch.empty((R, N), dtype=F16, device="cuda")
    moe.moe_gmm16(a, cumsum, w, c, ws)
    for r in at.tolist():
        assert torch.equal(c[r].double(), a[r].double() @ w[r // 150_000].double().T)
    da = torch.empty_like(a)
    dc = ints((R, N), F16, g, 1)
    moe.moe_gmm16_input_grad(dc, cumsum, w, da, ws)
    for r in at.tolist():
        assert torch.equal(da[r].double(), dc[r].double() @ w[r // 150_000].double())
    dw = torch.empty((2, N, D), device="cuda")
    moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, ws)
    last = dc[150_000:].double().T @ a[150_000:, :16].double()
    assert torch.equal(dw[1, :, :16], last.float())
    del dc, c

    row_map = torch.randperm(R, device="cuda", generator=g).int()
    moe.moe_dispatch16(a, row_map, da)
    assert torch.equal(da[row_map[at].long()], a[at])
    out = torch.empty_like(a)
    moe.moe_combine16(da, row_map, None, out)
    assert torch.equal(out[at], a[at]) and torch.equal(out[-1000:], a[-1000:])
    probs, dprobs = torch.full((R,), 2.0, device="cuda"), torch.empty(R, device="cuda")
    moe.moe_combine16_grad(a, da, row_map, probs, out, dprobs)
    assert torch.equal(out[row_map[at].long()], 2 * a[at])
    assert torch.equal(dprobs[at].double(), (a[at].double() ** 2).sum(1))

    h = torch.empty((R, D // 2), dtype=F16, device="cuda")
    moe.moe_swiglu16(a, cumsum, h)
    want = ref.swiglu(a[at])
    assert ((h[at].double() - want).abs() <= want.abs() * 2.0 ** -15 + ref.half_step(F16, want)).all()
    moe.moe_swiglu16_grad(h, a, cumsum, out)
    want = ref.swiglu_grad(h[at], a[at])
    assert ((out[at].double() - want).abs() <= want.abs() * 2.0 ** -14 + ref.half_step(F16, want) + 2.0 ** -19).all()
    del h

    route, _, lcum = ref.tables(torch.arange(R, device="cuda") % 3, 2)  # a third of the rows without an adapter
    la, lb = ints((2, 8, D), F16, g, 1), ints((2, D, 8), F16, g, 1)
    la *= (torch.arange(D, device="cuda") % 64 == 0)
    lws = torch.empty(moe.moe_lora16_workspace_size(R, D, D, 8), dtype=torch.uint8, device="cuda")
    moe.moe_lora16(a, route, lcum, la, lb, a, out, lws)
    for r in at.tolist():
        v = a[r].double()
        assert torch.equal(out[r].double(), v if r % 3 == 2 else v + lb[r % 3].double() @ (la[r % 3].double() @ v))


def test_weights_past_32_bit_offsets():
    """64 experts of 8192 x 8192: 4.3e9 elements."""
    g, E, N, D = rng(3), 64, 8192, 8192
    w = ints((1, N, D), BF16, g, 1).repeat(E, 1, 1)
    w[E - 1] = -w[E - 1]
    a, dc = ints((E, D), BF16, g, 1), ints((E, N), BF16, g, 1)
    a *= (torch.arange(D, device="cuda") % 64 == 0)
    dc *= (torch.arange(N, device="cuda") % 64 == 0)
    cumsum, ws = prefix([1] * E), space(E, E, N, D)
    c, da = torch.empty((E, N), dtype=BF16, device="cuda"), torch.empty((E, D), dtype=BF16, device="cuda")
    moe.moe_gmm16(a, cumsum, w, c, ws)
    moe.moe_gmm16_input_grad(dc, cumsum, w, da, ws)
    for e in (0, 31, 32, 63):
        assert torch.equal(c[e].double(), a[e].double() @ w[e].double().T)
        assert torch.equal(da[e].double(), dc[e].double() @ w[e].double())
    moe.moe_gmm16_weight_grad(dc, a, cumsum, w, ws)
    for e in (0, 31, 32, 63):
        assert torch.equal(w[e], dc[e][:, None] * a[e][None])


def test_most_experts():
    """1023 experts, most of them empty."""
    g, E, N, D = rng(4), 1023, 136, 72
    counts = [0] * E
    for i, n in ((0, 3), (500, 40), (501, 1), (1021, 7), (1022, 70)):
        counts[i] = n
    cumsum, R = prefix(counts), sum(counts)
    ends = cumsum.tolist()
    a, dc, w = ints((R, D), F16, g), ints((R, N), F16, g, 2), ints((E, N, D), F16, g, 2)
    ws, c, dw = space(R, E, N, D), torch.empty((R, N), dtype=F16, device="cuda"), torch.empty((E, N, D), device="cuda")
    moe.moe_gmm16(a, cumsum, w, c, ws)
    assert torch.equal(c, ref.rounded(ref.product(a, ends, w), F16))
    moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, ws)
    assert torch.equal(dw, ref.weight_grad(dc, a, ends).float())
    x, base = ints((R, D), F16, g, 1), ints((R, N), F16, g, 9)
    adapter = torch.tensor([1022, 0, -1, 511] * R, device="cuda")[:R]
    route, _, lcum = ref.tables(adapter, E)
    la, lb = ints((E, 8, D), F16, g, 1), ints((E, N, 8), F16, g, 1)
    out = torch.empty_like(base)
    lws = torch.empty(moe.moe_lora16_workspace_size(R, N, D, 8), dtype=torch.uint8, device="cuda")
    moe.moe_lora16(x, route, lcum, la, lb, base, out, lws)
    assert torch.equal(out, ref.rounded(ref.lora(x, adapter, la, lb, None, base), F16))


def test_adapter_workspace_of_a_larger_batch():
    """A workspace of 9000 tokens serves one, and the tables' ids outside the batch are skipped."""
    g, D, N, r = rng(6), 264, 520, 72
    lws = torch.empty(moe.moe_lora16_workspace_size(9000, N, D, r), dtype=torch.uint8, device="cuda")
    a, b = ints((3, r, D), BF16, g, 1), ints((3, N, r), BF16, g, 1)
    for M in (1, 17, 600, 9000):
        x, base = ints((M, D), BF16, g, 1), ints((M, N), BF16, g, 3)
        x *= (torch.arange(D, device="cuda") % 16 == 0)
        adapter = torch.randint(0, 3, (M,), device="cuda", generator=g)
        route, _, cumsum = ref.tables(adapter, 3)
        out = torch.empty_like(base)
        moe.moe_lora16(x, route, cumsum, a, b, base, out, lws)
        want = ref.rounded(ref.lora(x, adapter, a, b, None, base), BF16)
        assert torch.equal(out, want)
        if M > 1:
            bad = route.clone()
            bad[0], bad[-1] = M + 5, -3
            out.fill_(-1)
            moe.moe_lora16(x, bad, cumsum, a, b, base, out, lws)
            skipped = route[[0, -1]].long()
            keep = torch.ones(M, dtype=torch.bool, device="cuda")
            keep[skipped] = False
            assert torch.equal(out[keep], want[keep]) and (out[skipped] == -1).all()


def test_tensors_elsewhere_are_refused():
    a, w = torch.zeros(4, 64, dtype=F16, device="cuda"), torch.zeros(1, 64, 64, dtype=F16, device="cuda")
    cumsum, ws = prefix([4]), space(4, 1, 64, 64)
    for bad in ("a", "w", "c", "cumsum", "workspace"):
        args = dict(a=a, cumsum=cumsum, w=w, c=torch.zeros_like(a), workspace=ws)
        args[bad] = args[bad].cpu()
        with pytest.raises(ValueError, match="device"):
            moe.moe_gmm16(**args)


@pytest.mark.parametrize("rows,E,N,D", [(3, 2, 4096, 4096), (60, 8, 512, 512), (600, 3, 1024, 512), (2000, 4, 1024, 512), (3000, 1, 512, 512)])
def test_on_a_part_of_the_device(narrow_stream, rows, E, N, D):  # noqa: F811
    """On a stream that may use fewer SMs than the device has, products and adapters give what they give on all of it."""
    g, R = rng(8), rows * E
    a, dc, w = ints((R, D), BF16, g, 2), ints((R, N), BF16, g, 1), ints((E, N, D), BF16, g, 1)
    cumsum, ws = prefix([rows] * E), space(R, E, N, D)
    la, lb = ints((E, 8, D), BF16, g, 1), ints((E, N, 8), BF16, g, 1)
    route = torch.arange(R, device="cuda").int()
    lws = torch.empty(moe.moe_lora16_workspace_size(R, N, D, 8), dtype=torch.uint8, device="cuda")
    got = []
    for stream in (None, narrow_stream):
        c, da, out = (torch.zeros(s, dtype=BF16, device="cuda") for s in ((R, N), (R, D), (R, N)))
        dw = torch.zeros((E, N, D), device="cuda")
        torch.cuda.synchronize()
        moe.moe_gmm16(a, cumsum, w, c, ws, stream=stream)
        moe.moe_gmm16_input_grad(dc, cumsum, w, da, ws, stream=stream)
        moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, ws, stream=stream)
        moe.moe_lora16(a, route, cumsum, la, lb, c, out, lws, stream=stream)
        torch.cuda.synchronize()
        assert moe.moe_workspace_status(ws) == 0
        got.append([c, da, dw, out])
    assert same(*got)


def test_first_calls_may_be_captured():
    """In a process of its own: nothing has run before the capture, whose replay gives what the calls give."""
    code = """
import torch
from test_gpu_experts16_use import Step, same
s = Step(1, 3000, 512, 512, 2, 2)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    s.run()
g.replay()
torch.cuda.synchronize()
got = s.results()
s.run(wait=True)
assert same(got, s.results())
"""
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
