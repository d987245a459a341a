"""How far the sums of 16-bit experts' products are from 64 bits, where they are long.

The tensor cores add 16 products a step to an fp32 sum and drop what lies below its last place, two units of it at
most, always towards zero: n products of one sign lose up to n / 16 steps of 2^-22 of the sum so far, which is half of
the whole on average: 2^-27 n of the sum.  A part of a weight gradient's sum has up to 4096 (binary16) or 32768 (bfloat16)
rows in 16 bits, 512 or 768 in fp32.  Parts are added in fp32 (half a step each at most), and the whole is rounded once
where it is stored."""
import pytest

import experts16_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_expert_layer_gb300 as moe
    from test_gpu_experts16 import marked, rng, space

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
CHUNK = 1 << 18


def filled(R, C, t, g, positive):
    """Values of one sign around 2^-6, or normal ones, made in pieces."""
    x = torch.empty((R, C), dtype=t, device="cuda")
    for lo in range(0, R, CHUNK):
        v = x[lo:lo + CHUNK]
        r = torch.rand(v.shape, device="cuda", generator=g).add_(0.5) if positive else torch.randn(v.shape, device="cuda", generator=g)
        v.copy_(r.mul_(2.0 ** -6))
    return x


def corner64(dc, a, n, d):
    """Channels 0 .. n - 1 and columns 0 .. d - 1 of dc^T a."""
    w = torch.zeros(n, d, dtype=torch.float64, device="cuda")
    for lo in range(0, dc.shape[0], CHUNK):
        w += dc[lo:lo + CHUNK, :n].double().T @ a[lo:lo + CHUNK, :d].double()
    return w


# rows of one expert among E, channels, columns; the other experts have none.  Experts without rows make the blocks
# many and the rows few on average: pairs of CTAs take a block and all of its rows.  With one expert of
# few blocks clusters divide the rows.
PAIRS = [(76, 300_000, 256, 256), (1, 40_000, 4096, 4096)]
DIVIDED = [(1, 300_000, 72, 136), (1, 1_200_000, 256, 256)]


def gradient(E, R, N, D, t, out, positive):
    g = rng(R)
    a, dc, dw, ws = filled(R, D, t, g, positive), filled(R, N, t, g, positive), marked((E, N, D), out), space(R, E, N, D)
    cumsum = torch.zeros(E, dtype=torch.int32, device="cuda")
    cumsum[E // 2:] = R
    moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, ws)
    assert moe.moe_workspace_status(ws) == 0
    assert (dw[:E // 2] == 0).all() and (dw[E // 2 + 1:] == 0).all()
    return dw[E // 2], dc, a


def check16(E, R, N, D, t):
    """Half a step of rounding, what a part drops, and half an fp32 step for each part."""
    dw, dc, a = gradient(E, R, N, D, t, t, True)
    want = corner64(dc, a, min(N, 64), min(D, 64))
    err = (dw[:min(N, 64), :min(D, 64)].double() - want).abs()
    part = 4096 if t == F16 else 32768
    tol = ref.half_step(t, want) + want * (part * 2.0 ** -27 + (R / part + 1) * 2.0 ** -24)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("E,R,N,D", PAIRS + DIVIDED)
def test_long_16_bit_weight_gradients_of_binary16(E, R, N, D):
    check16(E, R, N, D, F16)


# bfloat16's half step is eight times as long, and so are the sums that would show what is dropped
@pytest.mark.parametrize("E,R,N,D", [(76, 4_000_000, 256, 256), (1, 10_000_000, 256, 256)])
def test_long_16_bit_weight_gradients_of_bfloat16(E, R, N, D):
    check16(E, R, N, D, BF16)


def test_most_rows():
    """2^24 - 1 rows, of both types."""
    for t in (F16, BF16):
        check16(1, (1 << 24) - 1, 64, 72, t)


@pytest.mark.parametrize("t", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("E,N,D", [(76, 200, 264), (3, 1032, 2056)])
def test_long_16_bit_weight_gradients_of_integers_are_exact(E, N, D, t):
    """Parts of every length beside short experts and empty ones, ragged channels and columns, exactly: integers whose
    sums fp32 holds, stored in 16 bits."""
    g, n = rng(E + N), 4096 if t == F16 else 32768
    lengths = [0, n, n + 1, 3, 2 * n + 100, 0, 64, 3 * n - 17, 16]
    counts = [lengths[i % 9] if E < 9 or i < 9 else i % 5 for i in range(E)]
    if E < 9:
        counts = [2 * n + 100, n + 1, 3 * n - 17]
    R = sum(counts) + 5
    cumsum = torch.tensor(counts, device="cuda").cumsum(0).int()
    small = lambda k, m: torch.randint(-m, m + 1, (R, k), device="cuda", generator=g).to(t)
    a, dc, dw, ws = small(D, 2), small(N, 1), marked((E, N, D), t), space(R, E, N, D)
    a[R - 5:], dc[R - 5:] = float("nan"), float("nan")
    moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, ws)
    assert moe.moe_workspace_status(ws) == 0
    assert torch.equal(dw, ref.rounded(ref.weight_grad(dc, a, cumsum.tolist()), t))


@pytest.mark.parametrize("positive", [True, False], ids=["one sign", "normal"])
@pytest.mark.parametrize("t", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("E,R,N,D", PAIRS + DIVIDED)
def test_long_fp32_weight_gradients(E, R, N, D, t, positive):
    """By the norm: what a part drops, and half an fp32 step for every second part.  One accumulator for all of
    the rows (for a fourth of them where clusters divide them), off by 6e-9 (one sign) and 1e-9 (normal values) of the
    sum to a product as measured, would be off by 20 times and 5 times as much at least."""
    dw, dc, a = gradient(E, R, N, D, t, F32, positive)
    n, d = min(N, 64), min(D, 64)
    want = corner64(dc, a, n, d)
    part = 512 if t == F16 else 768
    share = R if (E, R, N, D) in PAIRS else R / 4
    tol = part * 2.0 ** -27 + (share / part / 2 + 4) * 2.0 ** -24
    assert tol <= share * (6e-9 / 20 if positive else 1e-9 / 5), "the test would not tell"
    assert (dw[:n, :d].double() - want).norm() <= tol * want.norm()


@pytest.mark.parametrize("t", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("R", [1, 16, 128, 2048])
@pytest.mark.parametrize("depth", [8192, 65536])
def test_deep_products_of_one_sign(R, depth, t):
    """Products and gradients for the rows, whose sums are never in parts: half a step and 2^-27 of a sum's
    magnitudes to a product."""
    g, other = rng(R), 256
    rows, ws = filled(R, depth, t, g, True), space(R, 1, other, depth)
    cumsum = torch.tensor([R], dtype=torch.int32, device="cuda")
    c = marked((R, other), t)
    w = filled(other, depth, t, g, True)
    moe.moe_gmm16(rows, cumsum, w[None], c, ws)
    da = marked((R, other), t)
    wt = w.T.contiguous()
    moe.moe_gmm16_input_grad(rows, cumsum, wt[None], da, space(R, 1, depth, other))
    want = rows.double() @ w.double().T
    tol = ref.half_step(t, want) + want * depth * 2.0 ** -27
    for got in (c, da):
        err = (got.double() - want).abs()
        assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("t", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("N,D", [(264, 520), (136, 72)])
def test_long_experts_among_many_short_ones(N, D, t):
    """Few rows to an expert on average, one or two with several parts all the same: exactly, written and added."""
    g, E = rng(N), 200
    counts = [(3 * i) % 7 for i in range(E)]
    for i, n in ((7, 9000), (8, 0), (9, 4097)) if t == F16 else ((7, 33000), (8, 0), (9, 1537)):
        counts[i] = n
    cumsum, R = torch.tensor(counts, device="cuda").cumsum(0).int(), sum(counts) + 3
    assert 4096 < R <= 192 * E
    values = lambda k, m: torch.randint(-m, m + 1, (R, k), device="cuda", generator=g).to(t)
    a, dc, ws = values(D, 2), values(N, 1), space(R, E, N, D)
    a[R - 3:], dc[R - 3:] = float("nan"), float("nan")
    want = ref.weight_grad(dc, a, cumsum.tolist())
    for out in (t, F32):
        dw = marked((E, N, D), out)
        moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, ws)
        assert torch.equal(dw, ref.rounded(want, out))
    start = torch.randint(-1000, 1000, (E, N, D), device="cuda", generator=g).float()
    dw = start.clone()
    moe.moe_gmm16_weight_grad(dc, a, cumsum, dw, ws, accumulate=True)
    assert torch.equal(dw, (start.double() + want).float())
    assert moe.moe_workspace_status(ws) == 0
