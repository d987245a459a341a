"""The operators of 16-bit experts against their definitions in 64 bits (experts16_reference.py).

Integers small enough that every partial sum is exact in fp32 have to come out as their exact sum,
rounded once: sizes, tiles and ragged ends are tested this way, to the bit.  Real values are held to
a bound of the roundings: a sum of n products of 16-bit values, exact in fp32 each, is off by at most
n 2^-23 of the sum of their magnitudes in any order and also where the hardware truncates, and its
one rounding by half a step."""
import pytest

import experts16_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_expert_layer_gb300 as moe

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("t", [F16, BF16], ids=["f16", "bf16"])
MARK = -7.0  # what outputs hold before


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(shape, t, g, most=4):
    return torch.randint(-most, most + 1, shape, device="cuda", generator=g).to(t)


def normal(shape, t, g, size=1.0):
    return (size * torch.randn(shape, device="cuda", generator=g)).to(t)


def marked(shape, t):
    return torch.full(shape, MARK, dtype=t, device="cuda")


def space(R, E, N, D):
    return torch.full((moe.moe_gmm16_workspace_size(R, E, N, D),), 0xA5, dtype=torch.uint8, device="cuda")


def prefix(counts):
    return torch.tensor(counts, device="cuda").cumsum(0).int()


# every size around tiles: rows of an expert 0, 1, a few, one tile and one more or less, several
CASES = [
    ([1], 0, 8, 8), ([1], 0, 4096, 1024), ([0], 3, 64, 64), ([0, 5, 0], 1, 136, 72), ([3, 0, 0, 1, 7], 0, 64, 200),
    ([16] * 3, 2, 128, 64), ([17, 15, 33], 0, 264, 72), ([31, 32, 1, 0], 5, 120, 1000), ([64], 0, 512, 4096),
    ([255, 256, 257], 1, 256, 264), ([100, 0, 129, 500], 0, 520, 136), ([1000], 24, 1416, 520), ([2049, 3], 0, 248, 256),
    # few items, whose reduction a cluster divides: one round of them, several, odd depths, many rows
    ([2], 0, 136, 4104), ([3, 0, 5, 1, 2, 40, 1, 4, 7, 2], 3, 2568, 4104), ([30] * 4, 1, 2048, 2056), ([100, 90, 128, 1, 129] * 2, 0, 2824, 2312),
    ([250], 6, 1032, 4096), ([70, 3], 0, 4096, 1024),
    ([1, 2, 3] * 30, 0, 200, 128), ([0] * 60 + [40], 9, 1032, 640), ([511, 1], 0, 16, 2056), ([192, 193, 191, 224], 0, 384, 64),
]


@TYPES
@pytest.mark.parametrize("counts,behind,N,D", CASES)
def test_products_of_integers_are_exact(counts, behind, N, D, t):
    """All three products, exactly; rows behind the last expert hold NaN and keep what they held."""
    g, R, E = rng(N + D), sum(counts) + behind, len(counts)
    if R == 0:
        R = 1
    cumsum = prefix(counts)
    ends, n = cumsum.tolist(), sum(counts)
    a, dc, w = ints((R, D), t, g), ints((R, N), t, g, 2), ints((E, N, D), t, g, 2)
    a[n:], dc[n:] = float("nan"), float("nan")
    ws = space(R, E, N, D)

    c = marked((R, N), t)
    moe.moe_gmm16(a, cumsum, w, c, ws)
    assert moe.moe_workspace_status(ws) == 0
    assert torch.equal(c[:n], ref.rounded(ref.product(a, ends, w), t)[:n])
    assert (c[n:] == MARK).all()

    da = marked((R, D), t)
    moe.moe_gmm16_input_grad(dc, cumsum, w, da, ws)
    assert torch.equal(da[:n], ref.rounded(ref.input_grad(dc, ends, w), t)[:n])
    assert (da[n:] == MARK).all()

    want = ref.weight_grad(dc, a, ends)
    for out in (t, F32):
        dw = marked((E, N, D), out)
        moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, ws)
        assert torch.equal(dw, ref.rounded(want, out))
    start = ints((E, N, D), F32, g, 1000)
    dw = start.clone()
    moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, ws, accumulate=True)
    assert torch.equal(dw, (start.double() + want).float())
    assert moe.moe_workspace_status(ws) == 0


def close(got, want, sums, n, t):
    """Within n 2^-23 of the sums of magnitudes and a rounding."""
    tol = sums * (n * 2.0 ** -23)
    tol = tol + ref.half_step(t, want.abs() + tol)
    err = (got.double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()


@TYPES
@pytest.mark.parametrize("counts,N,D", [([37, 0, 300, 5], 328, 456), ([700, 1], 256, 192), ([1] * 20, 512, 264)])
def test_products_of_real_values(counts, N, D, t):
    g, R, E = rng(R_ := sum(counts)), R_, len(counts)
    cumsum = prefix(counts)
    ends = cumsum.tolist()
    a, dc, w = normal((R, D), t, g), normal((R, N), t, g, 1e-3), normal((E, N, D), t, g, D ** -0.5)
    ws = space(R, E, N, D)
    c, da, dw = marked((R, N), t), marked((R, D), t), marked((E, N, D), F32)
    moe.moe_gmm16(a, cumsum, w, c, ws)
    moe.moe_gmm16_input_grad(dc, cumsum, w, da, ws)
    moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, ws)
    close(c, ref.product(a, ends, w), ref.product(a.abs(), ends, w.abs()), D, t)
    close(da, ref.input_grad(dc, ends, w), ref.input_grad(dc.abs(), ends, w.abs()), N, t)
    close(dw, ref.weight_grad(dc, a, ends), ref.weight_grad(dc.abs(), a.abs(), ends), max(counts), F32)


@TYPES
@pytest.mark.parametrize(
    "counts,behind,N,D",
    [([0, 769, 1537, 3, 2304, 768, 1600, 0, 833], 5, 264, 328), ([769], 0, 8, 8), ([64 * 300 + 1, 50], 0, 136, 96),
     # several items of several parts to every pair of the device, short ones between them
     ([800, 20, 1700, 768] * 15, 3, 512, 512), ([900] * 80, 0, 512, 256)],
)
def test_weight_gradients_of_many_rows_are_exact(counts, behind, N, D, t):
    """Sums in several parts (in fp32, of experts with more than 768 or 512 rows), written and added."""
    g, R, E = rng(N + D), sum(counts) + behind, len(counts)
    cumsum, n = prefix(counts), sum(counts)
    a, dc, ws = ints((R, D), t, g), ints((R, N), t, g, 2), space(R, E, N, D)
    a[n:], dc[n:] = float("nan"), float("nan")
    want = ref.weight_grad(dc, a, cumsum.tolist())
    for out in (t, F32):
        dw = marked((E, N, D), out)
        moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, ws)
        assert torch.equal(dw, ref.rounded(want, out))
    start = ints((E, N, D), F32, g, 1000)
    dw = start.clone()
    moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, ws, accumulate=True)
    assert torch.equal(dw, (start.double() + want).float())
    assert moe.moe_workspace_status(ws) == 0


@TYPES
def test_long_weight_gradients_keep_fp32(t):
    """Sums of 70000 positive products, where bits dropped one way would add up: an fp32 gradient is made of
    parts of up to 768 rows (binary16: 512; n 2^-23 each, as above), added at half a step of the sum so far each."""
    g, counts, N, D = rng(3), [100, 70000], 72, 136
    cumsum, R = prefix(counts), sum(counts)
    a, dc = (torch.rand((R, k), device="cuda", generator=g).add(0.5).to(t) for k in (D, N))
    dw = marked((2, N, D), F32)
    moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, space(R, 2, N, D))
    want = ref.weight_grad(dc, a, cumsum.tolist())
    part = 768 if t == BF16 else 512
    close(dw, want, want, part + (70000 // part + 1) / 2, F32)


@TYPES
@pytest.mark.parametrize("E", [2, 40])
def test_gradients_against_differences(t, E):
    """The gradients of <dc, c(a, w)>: c is linear in a and in w, so the definition's differences along
    integer directions are exact, and so are the gradients' products with them."""
    g, N, D = rng(E), 72, 136
    counts = [3, 40] * (E // 2)
    cumsum, R = prefix(counts), sum(counts)
    ends = cumsum.tolist()
    a, dc, w = ints((R, D), t, g, 2), ints((R, N), t, g, 1), ints((E, N, D), t, g, 1)
    da, dw, ws = marked((R, D), t), marked((E, N, D), F32), space(R, E, N, D)
    moe.moe_gmm16_input_grad(dc, cumsum, w, da, ws)
    moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, ws)
    va, vw = ints((R, D), t, g, 1), ints((E, N, D), t, g, 1)
    loss = lambda x, y: (dc.double() * ref.product(x, ends, y)).sum()
    assert loss(a + va, w) - loss(a, w) == (da.double() * va.double()).sum()
    assert loss(a, w + vw) - loss(a, w) == (dw.double() * vw.double()).sum()


@TYPES
def test_products_keep_infinities_and_nan_to_their_rows(t):
    """A row that is not finite spoils itself alone (and its expert's weight gradient), whatever tile it
    shares with its neighbours; weights that are not finite spoil their channel."""
    g, counts, N, D = rng(7), [5, 30, 70, 1], 136, 200
    cumsum, R, E = prefix(counts), sum(counts), len(counts)
    ends = cumsum.tolist()
    a, dc, w = ints((R, D), t, g), ints((R, N), t, g), ints((E, N, D), t, g)
    ws = space(R, E, N, D)
    want_c, want_da, want_dw = ref.product(a, ends, w), ref.input_grad(dc, ends, w), ref.weight_grad(dc, a, ends)
    for row, e in ((4, 0), (5, 1), (34, 1), (35, 2), (105, 3)):
        for bad in (float("nan"), float("inf")):
            a2, dc2 = a.clone(), dc.clone()
            a2[row], dc2[row] = bad, bad
            c, da, dw = marked((R, N), t), marked((R, D), t), marked((E, N, D), F32)
            moe.moe_gmm16(a2, cumsum, w, c, ws)
            moe.moe_gmm16_input_grad(dc2, cumsum, w, da, ws)
            moe.moe_gmm16_weight_grad(dc2, a2, cumsum, dw, ws)
            other = [r for r in range(R) if r != row]
            assert torch.equal(c[other], ref.rounded(want_c, t)[other])
            assert torch.equal(da[other], ref.rounded(want_da, t)[other])
            if bad != bad:
                assert c[row].isnan().all() and da[row].isnan().all() and dw[e].isnan().all()
            rest = [x for x in range(E) if x != e]
            assert torch.equal(dw[rest], want_dw[rest].float())
    w2 = w.clone()
    w2[2, 77] = float("nan")
    c = marked((R, N), t)
    moe.moe_gmm16(a, cumsum, w2, c, ws)
    spoiled = c.isnan()
    assert spoiled[35:105, 77].all() and spoiled.sum() == 70


def test_outputs_past_their_type():
    """binary16 saturates, a NaN stays one; bfloat16 goes to infinity; both signs."""
    for t, big, want in ((F16, 256.0, 65504.0), (BF16, 2.0 ** 100, float("inf"))):
        a, w = torch.full((40, 64), big, dtype=t, device="cuda"), torch.full((1, 64, 64), big, dtype=t, device="cuda")
        w[0, 32:] = -big
        cumsum, ws = prefix([40]), space(40, 1, 64, 64)
        c, dw = marked((40, 64), t), marked((1, 64, 64), t)
        moe.moe_gmm16(a, cumsum, w, c, ws)
        assert (c[:, :32] == want).all() and (c[:, 32:] == -want).all()
        moe.moe_gmm16_weight_grad(a, a, cumsum, dw, ws)
        assert (dw == want).all()


@TYPES
def test_prefix_entries_are_held_to_the_rows(t):
    """Entries below 0 and above R: the rows between are the expert's."""
    g, R, N, D = rng(3), 20, 64, 64
    a, w = ints((R, D), t, g), ints((3, N, D), t, g)
    ws, c = space(R, 3, N, D), marked((R, N), t)
    moe.moe_gmm16(a, torch.tensor([-5, 7, 1000], dtype=torch.int32, device="cuda"), w, c, ws)
    assert torch.equal(c, ref.rounded(ref.product(a, [0, 7, 20], w), t))


# ------------------------------------------------------------------------------ SwiGLU
def gate_values(R, I, t, g):
    """Gates over all of fp32's exponential and past it, up values of every size."""
    gu = normal((R, 2 * I), t, g, 2.0)
    special = torch.tensor([0.0, -0.0, 1e-3, -1.2784645, 20, -20, 79, -79.5, -80, -80.5, -85, -88, -95, -104, 120, -130],
                           device="cuda")
    gu[0, :I] = special.repeat((I + 15) // 16)[:I].to(t)
    if t == BF16:
        gu[0, I:] *= 2.0 ** 60
    return gu


@TYPES
@pytest.mark.parametrize("R,I,behind", [(1, 8, 0), (5, 200, 2), (300, 1408, 7), (1025, 64, 0), (4, 32768, 1),
                                        (3000, 1000, 5), (40000, 64, 9), (77, 32768, 2)])
def test_swiglu_and_gradient(R, I, behind, t):
    """exp's relative error is 2^-22 |g| + 2^-22, a division's and each product's 2^-22: 2^-15 covers |g| up
    to 120; the slope 1 + g (1 - s) is off by 2^-22 (1 + |g|) absolutely, where it passes through zero."""
    g = rng(R + I)
    gu, dh = gate_values(R + behind, I, t, g), normal((R + behind, I), t, g, 0.1)
    gu[R:], dh[R:] = float("nan"), float("nan")
    cumsum = torch.tensor([0, R // 2, R // 2, R], dtype=torch.int32, device="cuda")
    h, h2, dgu = marked((R + behind, I), t), marked((R + behind, I), t), marked((R + behind, 2 * I), t)
    moe.moe_swiglu16(gu, cumsum, h)
    moe.moe_swiglu16_grad(dh, gu, cumsum, dgu, h2)
    want, want_d = ref.swiglu(gu[:R]), ref.swiglu_grad(dh[:R], gu[:R])
    err = (h[:R].double() - want).abs()
    assert (err <= want.abs() * 2.0 ** -15 + ref.half_step(t, want) * 1.001 + 2.0 ** -140).all()
    assert torch.equal(h, h2) or (h[:R] == h2[:R]).all()
    gate, up = gu[:R].double().chunk(2, 1)
    slack = (dh[:R].double() * up).abs() * torch.sigmoid(gate) * (1 + gate.abs()) * 2.0 ** -21
    slack = torch.cat([slack, torch.zeros_like(slack)], 1)
    err = (dgu[:R].double() - want_d).abs()
    assert (err <= want_d.abs() * 2.0 ** -15 + slack + ref.half_step(t, want_d) * 1.001 + 2.0 ** -140).all()
    for o in (h, h2, dgu):
        assert (o[R:] == MARK).all()
    # in place: dgu over gu, h over dh
    moe.moe_swiglu16_grad(dh, gu, cumsum, gu, dh)
    assert torch.equal(gu[:R], dgu[:R]) and torch.equal(dh[:R], h[:R])


def test_swiglu_gradient_against_differences():
    """Central differences of the definition, step 2^-10: their error is of third order, 2^-20 / 6 of a third
    derivative below 1 in magnitude times u dh."""
    g = rng(11)
    gu, dh = normal((40, 128), BF16, g), normal((40, 64), BF16, g)
    dgu, cumsum = marked((40, 128), BF16), prefix([40])
    moe.moe_swiglu16_grad(dh, gu, cumsum, dgu)
    e = 2.0 ** -10
    for half in (0, 1):
        step = torch.zeros(128, dtype=torch.float64, device="cuda")
        step[64 * half:64 * half + 64] = e
        d = dh.double() * (ref.swiglu(gu.double() + step) - ref.swiglu(gu.double() - step)) / (2 * e)
        scale = (dh.double() * (gu[:, 64:].double().abs() + 1)).abs()
        assert ((dgu[:, 64 * half:64 * half + 64].double() - d).abs() <= scale * 2.0 ** -20 + ref.half_step(BF16, d) * 1.01).all()


# ------------------------------------------------------------------------------ dispatch, combine
def maps(M, copies, rows, g, dropped=0.2):
    """Distinct rows for the entries, some of them out of range."""
    m = torch.randperm(max(rows, M * copies), device="cuda", generator=g)[:M * copies].int().view(M, copies)
    out = torch.where(torch.rand(M, copies, device="cuda", generator=g) < 0.5, -1, rows + 5).int()
    bad = (torch.rand(M, copies, device="cuda", generator=g) < dropped) | (m >= rows)
    return torch.where(bad, out, m)


MAPS = pytest.mark.parametrize("M,copies,rows,D", [(1, 1, 1, 8), (1, 8, 8, 7168), (3, 2, 9, 200), (61, 8, 488, 1032),
                                                   (300, 6, 1700, 264), (7, 33, 300, 72), (2, 300, 600, 16), (1000, 1, 1000, 65536 // 64),
                                                   # many tokens: whole and partial pieces, more threads than pieces, ninth routes
                                                   (2000, 3, 5000, 520), (230, 8, 1840, 4104), (20000, 2, 30000, 64), (130, 5, 600, 65536),
                                                   (9000, 1, 9000, 136), (2000, 9, 17000, 520), (700, 16, 9000, 2056), (2000, 17, 30000, 520)])


@TYPES
@MAPS
def test_dispatch_combine_and_gradients(M, copies, rows, D, t):
    g = rng(M * copies + D)
    row_map, probs = maps(M, copies, rows, g), torch.rand(M, copies, device="cuda", generator=g)
    kept = (row_map >= 0) & (row_map < rows)
    named = torch.zeros(rows, dtype=torch.bool, device="cuda")
    named[row_map[kept].long()] = True
    x, y, dout = normal((M, D), t, g), normal((rows, D), t, g), normal((M, D), t, g, 0.1)
    y[~named] = float("nan")

    a = marked((rows, D), t)
    moe.moe_dispatch16(x, row_map, a, copies=copies)
    tok = kept.nonzero()[:, 0]
    assert torch.equal(a[row_map[kept].long()], x[tok]) and (a[~named] == MARK).all()

    for p in (probs, None):
        out = marked((M, D), t)
        moe.moe_combine16(y, row_map, p, out, copies=copies)
        close(out, ref.combine(y, row_map, p), ref.combine(y.abs(), row_map, p), copies, t)

    dy, dprobs = marked((rows, D), t), marked((M, copies), F32)
    moe.moe_combine16_grad(dout, y, row_map, probs, dy, dprobs, copies=copies)
    want_dy, want_dp = ref.combine_grad(dout, y, row_map, probs)
    close(dy[named], want_dy[named], want_dy[named].abs(), 1, t)
    assert (dy[~named] == MARK).all()
    close(dprobs, want_dp, ref.combine_grad(dout.abs(), y.abs(), row_map, probs)[1], D, F32)
    assert (dprobs[~kept] == 0).all()
    moe.moe_combine16_grad(dout, y, row_map, probs, y, dprobs, copies=copies)  # in place
    assert torch.equal(y[named], dy[named]) and y[~named].isnan().all()


@TYPES
def test_combine_takes_a_row_twice_and_dispatch_a_token_once(t):
    y = torch.arange(24, device="cuda").view(3, 8).to(t)
    row_map = torch.tensor([[1, 1, 1], [0, 2, 0]], dtype=torch.int32, device="cuda")
    out = marked((2, 8), t)
    moe.moe_combine16(y, row_map, None, out, copies=3)
    assert torch.equal(out[0], 3 * y[1]) and torch.equal(out[1], 2 * y[0] + y[2])
    a = marked((3, 8), t)
    moe.moe_dispatch16(y[:1], torch.tensor([[2, 2]], dtype=torch.int32, device="cuda"), a, copies=2)
    assert torch.equal(a[2], y[0]) and (a[:2] == MARK).all()


# ------------------------------------------------------------------------------ adapters
def lora_call(x, adapter, a, b, scales, base, out):
    (M, D), (L, r, _), N = x.shape, a.shape, b.shape[1]
    route, _, cumsum = ref.tables(adapter, L)
    ws = torch.full((moe.moe_lora16_workspace_size(M, N, D, r),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_lora16(x, route, cumsum, a, b, base, out, ws, scales=scales)


LORA = pytest.mark.parametrize("M,D,N,r,L,prompt", [
    (1, 8, 8, 8, 1, 1), (1, 4096, 4096, 16, 3, 1), (5, 264, 72, 24, 4, 1), (33, 1000, 520, 8, 2, 33), (128, 512, 1032, 16, 100, 1),
    (130, 72, 264, 64, 1, 130), (300, 328, 200, 128, 5, 70), (700, 136, 136, 40, 3, 300), (64, 7168, 128, 32, 64, 1), (9, 64, 16392, 104, 2, 4)])


def adapters_of(M, L, prompt, g):
    per = torch.randint(-1, L, ((M + prompt - 1) // prompt,), device="cuda", generator=g).int()
    return per.repeat_interleave(prompt)[:M].contiguous()


@TYPES
@LORA
def test_adapters_of_integers_are_exact(M, D, N, r, L, prompt, t):
    """Sparse integers: the rank values stay below 2^8 and the output's terms below 2^16, exact throughout."""
    g = rng(M + D + r)
    adapter = adapters_of(M, L, prompt, g)
    x, a, b = ints((M, D), t, g, 1), ints((L, r, D), t, g, 1), ints((L, N, r), t, g, 1)
    x *= (torch.arange(D, device="cuda") % max(1, D // 64) == 0)
    base = ints((M, N), t, g, 100)
    scales = 2.0 ** torch.randint(-1, 2, (L,), device="cuda", generator=g).float()
    for s in (scales, None):
        out = marked((M, N), t)
        lora_call(x, adapter, a, b, s, base, out)
        want = ref.rounded(ref.lora(x, adapter, a, b, s, base), t)
        assert torch.equal(out, want)
    own = base.clone()
    lora_call(x, adapter, a, b, None, own, own)  # in place
    assert torch.equal(own, want)


@TYPES
@LORA
def test_adapters_of_real_values(M, D, N, r, L, prompt, t):
    """The rank values: D 2^-23 of their sums of magnitudes, then 2^-16 of the token's largest (16 significant
    bits); the second sum r 2^-23, scale and base two roundings of 2^-24, the output half a step."""
    g = rng(M + N)
    adapter = adapters_of(M, L, prompt, g)
    x, base = normal((M, D), t, g), normal((M, N), t, g)
    a, b = normal((L, r, D), t, g, D ** -0.5), normal((L, N, r), t, g, r ** -0.5)
    scales = 0.5 + torch.rand(L, device="cuda", generator=g)
    out = marked((M, N), t)
    lora_call(x, adapter, a, b, scales, base, out)
    want = ref.lora(x, adapter, a, b, scales, base)
    tol = torch.zeros_like(want)
    for l in range(L):
        k = (adapter == l).nonzero()[:, 0]
        if len(k):
            v, size = x[k].double() @ a[l].double().T, x[k].double().abs() @ a[l].double().abs().T
            dv = size * D * 2.0 ** -23
            dv = dv + 2.0 ** -16 * (v.abs() + dv).amax(1, keepdim=True)
            tol[k] = scales[l].double() * ((dv + (v.abs() + dv) * r * 2.0 ** -23) @ b[l].double().abs().T)
    tol += 2.0 ** -22 * (want.abs() + base.double().abs())
    tol += ref.half_step(t, want.abs() + tol)
    err = (out.double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()
    bare = (adapter < 0) | (adapter >= L)
    assert torch.equal(out[bare], base[bare])


@TYPES
def test_adapters_keep_infinities_and_large_values(t):
    """Rank values far outside the type (the sums are fp32) come back through small weights; a token that is not
    finite spoils itself alone."""
    M, D, N, r = 20, 256, 64, 16
    x, a = torch.full((M, D), 200.0, dtype=t, device="cuda"), torch.full((2, r, D), 200.0, dtype=t, device="cuda")
    b = torch.full((2, N, r), 2.0 ** -20, dtype=t, device="cuda")
    base = torch.zeros((M, N), dtype=t, device="cuda")
    adapter = torch.arange(M, device="cuda").int() % 2
    out = marked((M, N), t)
    lora_call(x, adapter, a, b, None, base, out)
    want = ref.lora(x, adapter, a, b, None, base)  # 200 * 200 * 256 * 16 / 2^20 = 156.25
    assert ((out.double() - want).abs() <= want * 2.0 ** -15 + ref.half_step(t, want)).all()
    x[6] = float("inf")
    lora_call(x, adapter, a, b, None, base, out)
    assert (out[6] == (65504.0 if t == F16 else float("inf"))).all()
    x[6], x[7] = float("nan"), 0.0
    lora_call(x, adapter, a, b, None, base, out)
    assert out[6].isnan().all() and (out[7] == 0).all() and torch.isfinite(out[[i for i in range(M) if i != 6]]).all()


# ------------------------------------------------------------------------------ together
@TYPES
@pytest.mark.parametrize("M,K,I,E,topK,adapters", [(1, 128, 64, 4, 2, 1), (70, 256, 192, 8, 3, 3), (400, 384, 128, 16, 4, 5)])
def test_layer_forwards_and_backwards(M, K, I, E, topK, adapters, t):
    """Router, sort, dispatch, products, an adapter of each request on the first one, SwiGLU, combine, and back: each
    stage against its definition on the very inputs it got, and the gradients together against 64-bit ones.  Every
    stage rounds once, half a step e: the norm of the gradients, behind at most 9 roundings that each spread as the
    values themselves do, is held to 16 e."""
    g = rng(M)
    x, w1, w2 = normal((M, K), t, g), normal((E, 2 * I, K), t, g, K ** -0.5), normal((E, K, I), t, g, I ** -0.5)
    la, lb = normal((adapters, 8, K), t, g, K ** -0.5), normal((adapters, 2 * I, 8), t, g, 0.2)
    idx, probs = torch.empty((M, topK), dtype=torch.int32, device="cuda"), torch.empty((M, topK), device="cuda")
    moe.moe_route_topk(normal((M, E), F32, g), idx, probs)
    idx[0, 0] = -1  # a dropped route
    d, R = moe.dims(M, K, I, E, topK), M * topK
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
    src, rows, tpe, cumsum = i32(R), i32(R), i32(E), i32(E)
    sort_ws = torch.empty(max(1, moe.moe_route_sort_workspace_size(d)), dtype=torch.uint8, device="cuda")
    moe.moe_route_sort(d, idx, src, rows, tpe, cumsum, sort_ws)
    ends, n, row_map = cumsum.tolist(), int(cumsum[-1]), rows.view(M, topK)
    # the adapters of the rows: token t's is t % adapters; the rows sorted by it
    of_row = torch.where(torch.arange(R, device="cuda") < n, (src // topK) % adapters, -1).int()
    route, _, lcum = ref.tables(of_row, adapters)
    new = lambda *s: torch.zeros(s, dtype=t, device="cuda")
    a, gu, gu2, h, y, out = new(R, K), new(R, 2 * I), new(R, 2 * I), new(R, I), new(R, K), new(M, K)
    ws = space(R, E, 2 * I, K)
    lws = torch.empty(moe.moe_lora16_workspace_size(R, 2 * I, K, 8), dtype=torch.uint8, device="cuda")
    moe.moe_dispatch16(x, rows, a, copies=topK)
    moe.moe_gmm16(a, cumsum, w1, gu, ws)
    moe.moe_lora16(a, route, lcum, la, lb, gu, gu2, lws)
    moe.moe_swiglu16(gu2, cumsum, h)
    moe.moe_gmm16(h, cumsum, w2, y, ws)
    moe.moe_combine16(y, rows, probs, out, copies=topK)
    close(gu[:n], ref.product(a, ends, w1)[:n], ref.product(a.abs(), ends, w1.abs())[:n], K, t)
    close(y[:n], ref.product(h, ends, w2)[:n], ref.product(h.abs(), ends, w2.abs())[:n], I, t)
    close(out, ref.combine(y, row_map, probs), ref.combine(y.abs(), row_map, probs), topK, t)

    dout = normal((M, K), t, g)
    dy, dprobs, dh, dgu, da, dx = new(R, K), torch.empty_like(probs), new(R, I), new(R, 2 * I), new(R, K), new(M, K)
    dw1, dw2 = torch.empty(w1.shape, device="cuda"), torch.empty(w2.shape, device="cuda")
    moe.moe_combine16_grad(dout, y, rows, probs, dy, dprobs, copies=topK)
    moe.moe_gmm16_input_grad(dy, cumsum, w2, dh, ws)
    moe.moe_gmm16_weight_grad(dy, h, cumsum, dw2, ws)
    moe.moe_swiglu16_grad(dh, gu2, cumsum, dgu)
    moe.moe_gmm16_input_grad(dgu, cumsum, w1, da, ws)
    moe.moe_gmm16_weight_grad(dgu, a, cumsum, dw1, ws)
    dlb = torch.zeros_like(la)  # the adapters' own input gradient goes through their two products
    back = torch.zeros_like(da)
    moe.moe_lora16(dgu, route, lcum, lb.transpose(1, 2).contiguous(), la.transpose(1, 2).contiguous(), da, back, lws2(R, K, 2 * I))
    moe.moe_combine16(back, rows, None, dx, copies=topK)
    assert moe.moe_workspace_status(ws) == 0 and dlb.sum() == 0

    # the same in 64 bits, by autograd of the definition
    leaves = [v.double().requires_grad_() for v in (x, w1, w2, probs)]
    x64, w164, w264, p64 = leaves
    kept = (idx.reshape(-1) >= 0).nonzero()[:, 0]
    tok, e = kept // topK, idx.reshape(-1)[kept].long()
    xr, ad = x64[tok], (tok % adapters)
    pre = torch.einsum("rk,rnk->rn", xr, w164[e]) + torch.einsum("rnq,rq->rn", lb.double()[ad], torch.einsum("rqk,rk->rq", la.double()[ad], xr))
    hid = torch.nn.functional.silu(pre[:, :I]) * pre[:, I:]
    yy = torch.einsum("ri,rki->rk", hid, w264[e])
    o64 = torch.zeros(M, K, dtype=torch.float64, device="cuda").index_add(0, tok, yy * p64.reshape(-1)[kept][:, None])
    (o64 * dout.double()).sum().backward()
    e16 = 16 * torch.finfo(t).eps / 2
    for got, want in ((out, o64), (dx, x64.grad), (dw1, w164.grad), (dw2, w264.grad), (dprobs, p64.grad)):
        want = want.detach()
        assert (got.double() - want).norm() <= e16 * want.norm()


def lws2(M, N, D):
    return torch.empty(moe.moe_lora16_workspace_size(M, N, D, 8), dtype=torch.uint8, device="cuda")
