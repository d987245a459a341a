"""The grouped MXFP4 product's hand-overs between its warps and CTAs, and the expert sizes at which
it goes from one tile and one kernel to the next."""
import numpy as np
import pytest

import mx_reference as mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_expert_layer_gb300 as moe
    import test_gpu_mxfp4 as base
    from gpu_util import dev, empty, host
    from test_gpu_mxfp4 import make_rows, make_weights


@pytest.mark.parametrize("counts,N,D", [([260, 240], 384, 1024), ([700, 3, 100], 256, 2016), ([40, 0, 33, 60], 640, 512)])
def test_pair_uses_both_halves_scale_words(counts, N, D):
    """CTA pairs, with new scales of rows and channels in every call: all elements are 1, so a sum is 32
    times a sum of powers of two, and exact; a scale word of an earlier call, or one out of order,
    shows in it."""
    E, R = len(counts), sum(counts)
    assert R / E > 32
    gen = torch.Generator(device="cuda").manual_seed(R)
    cum = dev(np.cumsum(counts).astype(np.int32))
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(counts, device="cuda"))
    planes, pitch, blocks = (D + 127) // 128, (R + 3) // 4 * 4, D // 32
    codes = torch.full((R, D // 2), 0x22, dtype=torch.uint8, device="cuda")
    w_codes = torch.full((E, N, D // 2), 0x22, dtype=torch.uint8, device="cuda")
    w = empty((moe.moe_mxfp4_weights_bytes(E, N, D),), torch.uint8)
    ws = empty(moe.moe_mxfp4_gmm_workspace_size(R, E, N, D), torch.uint8)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(60):
        sa = torch.randint(0, 2, (R, blocks), generator=gen, device="cuda")
        sw = torch.randint(0, 2, (E, N, blocks), generator=gen, device="cuda")
        words = torch.full((planes, pitch, 4), 0xAA, dtype=torch.uint8, device="cuda")
        padded = torch.nn.functional.pad(sa + 127, (0, planes * 4 - blocks)).to(torch.uint8)
        words[:, :R] = padded.view(R, planes, 4).transpose(0, 1)
        moe.moe_mxfp4_pack_weights(w_codes, (sw + 127).to(torch.uint8), w)
        c = torch.zeros((R, N), dtype=torch.float16, device="cuda")
        moe.moe_mxfp4_gmm(codes, words.view(torch.int32).view(-1), cum, w, c, ws)
        want = 32 * torch.bmm((1 << sa).double()[:, None], (1 << sw).double()[expert].transpose(1, 2))[:, 0]
        wrong += (c.double() != want).sum()
    assert wrong.item() == 0 and moe.moe_workspace_status(ws) == 0


@pytest.mark.parametrize("rows", [1, 9, 40])
def test_swiglu_of_very_negative_gates(rows):
    """h = g / (1 + exp(-g)) u where exp(-g) is near fp32's end and past it, but h, with u large, is far
    from MXFP4's: gates from -70 to -165, one to a scaled block, whose sums are exact (whole numbers)."""
    rng = np.random.default_rng(rows)
    gates = np.array([-70, -79, -80, -81, -86, -87, -88, -89, -90, -95, -103, -104, -120, -140, -160, -165], np.float64)
    I, D = 32 * len(gates), 32
    code, scale = np.zeros((1, 2 * I, D), np.uint8), np.full((1, 2 * I, 1), 127, np.uint8)
    for b, g in enumerate(gates):  # -6 as often as it fits, and the rest
        sixes, rest = divmod(int(-g), 6)
        code[0, 32 * b:32 * b + 32, :sixes] = 15
        code[0, 32 * b:32 * b + 32, sixes] = 8 + [0, 2, 4, 5, 6, 7][rest] if rest < 5 else 14
        if rest == 5:
            code[0, 32 * b:32 * b + 32, sixes + 1] = 10
    code[0, I:, 0] = rng.integers(1, 16, I)
    code[0, I:, 0][code[0, I:, 0] == 8] = 3
    scale[0, I:] = 127 + 110  # u: up to 6 2^110
    wv = mx.values(code, scale)
    g, u = wv[0, :I].sum(-1)[None].repeat(rows, 0), wv[0, I:].sum(-1)[None].repeat(rows, 0)
    assert np.array_equal(g[0, ::32], gates)
    w = empty((moe.moe_mxfp4_weights_bytes(1, 2 * I, D),), torch.uint8)
    moe.moe_mxfp4_pack_weights(dev(mx.pack(code)), dev(scale), w, True)
    a = np.full((rows, D), 2, np.uint8)  # ones
    words = dev(mx.scale_planes(np.full((rows, 1), 127, np.uint8)).view(np.int32))
    hc = empty((rows, I // 2), torch.uint8)
    hs = empty((moe.moe_mxfp4_scale_words(rows, I),), torch.int32)
    ws = empty(moe.moe_mxfp4_gmm_workspace_size(rows, 1, 2 * I, D), torch.uint8)
    moe.moe_mxfp4_gmm_swiglu(dev(mx.pack(a)), words, dev(np.array([rows], np.int32)), w, hc, hs, ws)
    h, eh = mx.silu_mul(g, u, np.zeros_like(g), np.zeros_like(u))
    least, most, s0, s1 = mx.quantise_interval(h, eh)
    assert s0.min() > 0
    planes = host(hs).view(np.uint32).reshape((I + 127) // 128, -1)
    s = np.ascontiguousarray(planes[:, :rows].T).view(np.uint8).reshape(rows, -1)[:, :I // 32]
    v = np.abs(mx.values(np.stack([host(hc) & 15, host(hc) >> 4], -1).reshape(rows, I), s))
    assert (s >= s0).all() and (s <= s1).all()
    assert (v >= least).all() and (v <= most).all()


# experts of more than 32 rows where the average is less: single CTAs with several tiles for an expert,
# of sizes around the tile's, behind experts that end on any row
SKEWED = [([100, 0, 1, 3, 0, 0, 37, 5], 256, 288), ([100, 0, 1, 3, 0, 0, 37, 5], 384, 64), ([33, 0, 31], 128, 160),
          ([1, 64, 0, 0, 0], 128, 512), ([2, 65, 3, 0, 0, 0], 640, 256), ([200] + [0] * 9 + [1], 256, 1408),
          ([3, 97, 0, 0, 96, 5, 0, 34, 2, 0], 256, 224)]


@pytest.mark.parametrize("counts,N,D", SKEWED)
def test_gmm_of_skewed_experts(counts, N, D):
    assert (sum(counts) + 5) / len(counts) <= 32 < max(counts)
    base.test_gmm(counts, N, D)


@pytest.mark.parametrize("counts,N,D", SKEWED)
def test_gmm_swiglu_of_skewed_experts(counts, N, D):
    assert (sum(counts) + 3) / len(counts) <= 32 < max(counts)
    base.test_gmm_swiglu(counts, N // 2, D)


@pytest.mark.parametrize("counts", [[64, 65, 66], [192, 1, 193, 383], [31, 193, 0, 0, 200], [385, 0, 7]])
@pytest.mark.parametrize("N,D", [(128, 96), (384, 320)])
def test_gmm_of_pairs_around_their_tiles(counts, N, D):
    assert sum(counts) / len(counts) > 32
    base.test_gmm(counts, N, D)
    base.test_gmm_swiglu(counts, N // 2, D)


@pytest.mark.parametrize("R,E", [(20, 2), (200, 2), (500, 3)])
def test_nan_rows_and_channels_stay_alone(R, E):
    """A NaN block of a row makes the row's sums NaN, one of a channel the channel's, on single CTAs and on
    pairs; prefix entries outside 0 .. R are held there."""
    rng = np.random.default_rng(R)
    N, D = 256, 384
    codes, scales, a = make_rows(rng, R, D)
    bad_row = R - 9
    planes = host(scales).copy()
    planes.view(np.uint8).reshape(D // 128, -1, 4)[1, bad_row, 2] = 255
    code = rng.integers(0, 16, (E, N, D), dtype=np.uint8)
    scale = rng.integers(115, 128, (E, N, D // 32)).astype(np.uint8)
    scale[E - 1, 77, 5] = 255
    w = empty((moe.moe_mxfp4_weights_bytes(E, N, D),), torch.uint8)
    moe.moe_mxfp4_pack_weights(dev(mx.pack(code)), dev(scale), w)
    wv = mx.values(code, scale)[E - 1]
    cum = np.array([-5, 1 << 30] if E == 2 else [-1, -7, 1 << 30], np.int32)
    c = torch.full((R, N), 7.0, dtype=torch.float16, device="cuda")
    ws = empty(moe.moe_mxfp4_gmm_workspace_size(R, E, N, D), torch.uint8)
    moe.moe_mxfp4_gmm(codes, dev(planes), dev(cum), w, c, ws)
    assert moe.moe_workspace_status(ws) == 0
    got, n = host(c).astype(np.float64), np.arange(N) != 77
    assert np.isnan(got[bad_row]).all() and np.isnan(got[:, 77]).all() and np.isnan(got).sum() == R + N - 1
    keep = np.arange(R) != bad_row
    ref, err = a[keep] @ wv[n].T, mx.sum_error(a[keep], wv[n])
    assert (np.abs(got[keep][:, n] - ref.clip(-65504, 65504)) <= err + mx.f16_error(np.abs(ref) + err)).all()


@pytest.mark.parametrize("counts,N,D", [([3, 2], 128, 16384), ([50, 40], 128, 16384), ([1, 0, 1] * 341, 128, 64), ([2], 16384, 32)])
def test_gmm_at_the_ends_of_its_ranges(counts, N, D):
    base.test_gmm(counts, N, D)
    base.test_gmm_swiglu(counts, N // 2, D)
