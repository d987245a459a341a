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
