"""Low-rank adapters at the ends of their numbers, and as programs call them: for both forms, few tokens to an adapter and
many (more than 16)."""
import pytest

import experts16_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_expert_layer_gb300 as moe
    from test_gpu_experts16 import lora_call, marked

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("t", [F16, BF16], ids=["f16", "bf16"])
RANKS = pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 56, 64, 72, 104, 128])
TOKENS = pytest.mark.parametrize("M", [16, 40, 200])


@TYPES
@RANKS
@TOKENS
def test_infinite_tokens_give_infinities(M, r, t):
    """All weights positive: a token with an infinite element is infinite in every channel (binary16: saturated), one
    with two of different signs NaN, and the others stay what they are."""
    D, N = 136, 72
    x, base = torch.ones((M, D), dtype=t, device="cuda"), torch.zeros((M, N), dtype=t, device="cuda")
    a, b = torch.ones((1, r, D), dtype=t, device="cuda"), torch.full((1, N, r), 2.0 ** -8, dtype=t, device="cuda")
    adapter = torch.zeros(M, dtype=torch.int32, device="cuda")
    x[3, 5], x[8, D - 1], x[10, 0], x[10, 77] = float("inf"), -float("inf"), float("inf"), -float("inf")
    out = marked((M, N), t)
    lora_call(x, adapter, a, b, None, base, out)
    most = 65504.0 if t == F16 else float("inf")
    assert (out[3] == most).all() and (out[8] == -most).all() and out[10].isnan().all()
    rest = [i for i in range(M) if i not in (3, 8, 10)]
    assert torch.equal(out[rest], ref.rounded(ref.lora(x[rest], adapter[rest], a, b, None, base[rest]), t))


@pytest.mark.parametrize("rank_value,weight", [(-120, 127), (-30, 127), (0, 120), (120, -120), (127, -127), (100, -126), (-126, 100)])
@pytest.mark.parametrize("r", [8, 64, 128])
@pytest.mark.parametrize("M", [16, 40])
def test_bfloat16_weights_and_rank_values_at_their_ends(M, r, rank_value, weight):
    """Rank values and weights far apart, whose products are ordinary numbers: powers of two, exact (with signs that
    leave r / 4 of the products, so that no sum on the way leaves fp32)."""
    D, N = 64, 72
    lo = rank_value // 2
    x, a = torch.full((M, D), 2.0 ** lo, dtype=BF16, device="cuda"), torch.zeros((1, r, D), dtype=BF16, device="cuda")
    a[..., 7] = 2.0 ** (rank_value - lo)
    b = torch.full((1, N, r), 2.0 ** min(weight, 127), dtype=BF16, device="cuda")
    b[..., 3::4], b[..., 2::4] = -b[..., 3::4], 0.0
    base, out = torch.zeros((M, N), dtype=BF16, device="cuda"), marked((M, N), BF16)
    lora_call(x, torch.zeros(M, dtype=torch.int32, device="cuda"), a, b, None, base, out)
    assert (out.double() == r / 4 * 2.0 ** (rank_value + weight)).all()


def sorted_by_library(adapter, L):
    """Tables of moe_route_sort, one adapter to a token."""
    M = adapter.numel()
    d = moe.dims(M, 128, 64, L, 1)
    route, row, count, cumsum = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (M, M, L, L))
    ws = torch.empty(max(1, moe.moe_route_sort_workspace_size(d)), dtype=torch.uint8, device="cuda")
    moe.moe_route_sort(d, adapter, route, row, count, cumsum, ws)
    return route, row, cumsum


def adapters_of(M, L, g):
    """Ids of adapters, and others that name none."""
    adapter = torch.randint(0, L, (M,), device="cuda", generator=g).int()
    other = torch.tensor([-1, L, L + 3, -(1 << 31), (1 << 31) - 1], device="cuda").int()
    none = torch.rand(M, device="cuda", generator=g) < 0.2
    return torch.where(none, other[torch.arange(M, device="cuda") % 5], adapter).contiguous()


@TYPES
@pytest.mark.parametrize("M,L", [(1, 1), (2, 3), (40, 1), (130, 100), (3000, 5), (20000, 1023), (70000, 24)])
def test_adapters_on_the_tables_of_the_route_sort(M, L, t):
    """The tables that moe_route_sort makes of the tokens' adapters give what tables made otherwise give, to the bit:
    tokens whose id names no adapter are sorted behind the others and get their base."""
    g = torch.Generator(device="cuda").manual_seed(M + L)
    D, N, r = 136, 72, 24
    adapter = adapters_of(M, L, g)
    normal = lambda *s: torch.randn(s, device="cuda", generator=g).to(t)
    x, a, b, base = normal(M, D), normal(L, r, D) * D ** -0.5, normal(L, N, r), normal(M, N)
    scales = torch.rand(L, device="cuda", generator=g)
    want, out = marked((M, N), t), marked((M, N), t)
    lora_call(x, adapter, a, b, scales, base, want)
    route, _, cumsum = sorted_by_library(adapter, L)
    ws = torch.empty(moe.moe_lora16_workspace_size(M, N, D, r), dtype=torch.uint8, device="cuda")
    moe.moe_lora16(x, route, cumsum, a, b, base, out, ws, scales=scales)
    assert torch.equal(out, want)
    bare = (adapter < 0) | (adapter >= L)
    assert torch.equal(out[bare], base[bare]) and (M < 40 or not torch.equal(out, base))


@TYPES
@pytest.mark.parametrize("M,L", [(5, 2), (300, 4), (2500, 70)])
def test_gradients_of_adapters_by_the_products(M, L, t):
    """The gradients of a and b are those of two products grouped by adapter, on the rows sorted by it; against
    autograd in 64 bits.  Rank values and their gradients round once each, and so do the results: within
    four half steps of the norm."""
    g = torch.Generator(device="cuda").manual_seed(M)
    D, N, r = 264, 136, 16
    adapter = adapters_of(M, L, g)
    normal = lambda *s: torch.randn(s, device="cuda", generator=g).to(t)
    x, a, b, dout = normal(M, D), normal(L, r, D) * D ** -0.5, normal(L, N, r), normal(M, N)
    _, row, cumsum = sorted_by_library(adapter, L)
    ws = torch.empty(moe.moe_gmm16_workspace_size(M, L, max(N, r), max(D, r)), dtype=torch.uint8, device="cuda")
    new = lambda *s: marked(s, t)
    xs, ds, v, dv, da, db = new(M, D), new(M, N), new(M, r), new(M, r), marked(a.shape, F32), marked(b.shape, F32)
    moe.moe_dispatch16(x, row, xs)
    moe.moe_dispatch16(dout, row, ds)
    moe.moe_gmm16(xs, cumsum, a, v, ws)
    moe.moe_gmm16_weight_grad(ds, v, cumsum, db, ws)
    moe.moe_gmm16_input_grad(ds, cumsum, b, dv, ws)
    moe.moe_gmm16_weight_grad(dv, xs, cumsum, da, ws)
    a64, b64 = a.double().requires_grad_(), b.double().requires_grad_()
    has = ((adapter >= 0) & (adapter < L)).nonzero()[:, 0]
    l = adapter[has].long()
    y = torch.einsum("tnr,tr->tn", b64[l], torch.einsum("trd,td->tr", a64[l], x[has].double()))
    (y * dout[has].double()).sum().backward()
    e = 4 * torch.finfo(t).eps / 2
    for got, want in ((da, a64.grad), (db, b64.grad)):
        assert (got.double() - want).norm() <= e * want.norm()
