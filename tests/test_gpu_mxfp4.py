"""The router, MXFP4 quantisation, the grouped MXFP4 product and the MXFP4 layer against the
64-bit reference (mx_reference.py), whose error bounds are the tolerances."""
import numpy as np
import pytest

import mx_reference as mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_expert_layer_gb300 as moe
    from gpu_util import dev, empty, host

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def typed(x, kind):
    """float64 numpy -> device tensor of the type, and its values in 64 bits."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DTYPES[kind])
    return t.cuda(), t.double().numpy()


# ------------------------------------------------------------------------------ router
def run_route(logits, topK, **kw):
    M = logits.shape[0]
    idx, probs = empty((M, topK), torch.int32), empty((M, topK), torch.float32)
    idx.fill_(-7)
    probs.fill_(-7)
    moe.moe_route_topk(logits, idx, probs, **kw)
    return host(idx), host(probs).astype(np.float64)


def check_route(got, ref, E, same_idx=True):
    """Weights: exp's argument is off by 2^-24 of up to 2^7, the sums of up to E / 32 + 5 additions
    and the divisions by 2^-23 each; 2^-17 of the value covers them, and the smallest normal."""
    idx, probs = got
    if same_idx:
        assert np.array_equal(idx, ref[0])
        tol = np.abs(ref[1]) * (2.0 ** -17 + (E / 32 + 16) * 2.0 ** -23) + 2.0 ** -120
        assert (np.abs(probs - ref[1]) <= tol).all()


@pytest.mark.parametrize("M,E,topK,kind", [
    (1, 1, 1, "f32"), (1, 256, 8, "f32"), (3, 5, 5, "f16"), (33, 33, 4, "bf16"), (129, 257, 8, "f32"),
    (64, 1023, 16, "f16"), (2, 1023, 1023, "f32"), (500, 64, 6, "f16"), (7, 31, 31, "f32"), (70001, 8, 2, "f32")])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_matches_the_definition(M, E, topK, kind, sigmoid):
    rng = np.random.default_rng(M * E + topK)
    logits, l = typed(3.0 * rng.standard_normal((M, E)), kind)
    for renormalise, scale in ((True, 1.0), (False, 2.5)):
        got = run_route(logits, topK, scoring=int(sigmoid), renormalise=renormalise, scale=scale)
        check_route(got, mx.route(l, topK, sigmoid, renormalise, scale), E)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_masks_ties_and_infinities(kind, sigmoid):
    """Ties take the lower expert, signed zeros tie, masked experts (-inf, NaN) are never chosen, the
    type's lowest value is not a mask, +inf is the largest finite value, a fully masked row has no route."""
    low = {"f32": -3.4e38, "f16": -65504.0, "bf16": -3.38e38}[kind]
    rows = [[1.0] * 6, [0.0, -0.0, 0.0, -0.0, 0.0, -1.0], [-np.inf] * 6, [np.nan] * 6,
            [-np.inf, 2.0, np.nan, -np.inf, 1.0, -np.inf], [low] * 6, [low, 3.0, low, low, low, low],
            [np.inf, 1.0, 2.0, np.inf, -np.inf, 0.0], [-np.inf] * 5 + [low], [np.nan, np.inf] + [-np.inf] * 4,
            [100.0, -100.0, 50.0, 100.0, 0.0, -50.0]]
    logits, l = typed(np.array(rows), kind)
    for renormalise in (True, False):
        got = run_route(logits, 3, scoring=int(sigmoid), renormalise=renormalise)
        ref = mx.route(np.where(np.isposinf(l), 3.402823466e38, l), 3, sigmoid, renormalise, 1.0)
        assert np.isfinite(got[1]).all()
        check_route(got, ref, 6)
        assert (got[0][2:4] == -1).all() and (got[1][2:4] == 0).all()


def test_route_takes_any_row_stride_and_bias():
    rng = np.random.default_rng(5)
    wide, w = typed(rng.standard_normal((37, 90)), "f16")
    for lo, E in ((0, 64), (0, 90), (8, 61)):  # 16-byte aligned starts, rows 180 bytes apart
        check_route(run_route(wide[:, lo:lo + E], 6), mx.route(w[:, lo:lo + E], 6, False, True, 1.0), E)
    bias = rng.standard_normal(64) * 0.3
    b = dev(bias.astype(np.float32))
    for sigmoid in (False, True):
        idx, probs = run_route(wide[:, :64], 6, scoring=int(sigmoid), bias=b)
        _, _, key, p = mx.route(w[:, :64], 6, sigmoid, True, 1.0, bias.astype(np.float32).astype(np.float64))
        chosen = np.take_along_axis(key, idx, 1)
        assert (np.diff(chosen, axis=1) <= 1e-6).all()   # keys are fp32 sums of terms of size 1
        rest = key.copy()
        np.put_along_axis(rest, idx.astype(np.int64), -np.inf, 1)
        assert (rest.max(1) <= chosen[:, -1] + 1e-6).all()
        pw = np.take_along_axis(p, idx, 1)
        assert np.allclose(probs, pw / pw.sum(1, keepdims=True), rtol=2.0 ** -16, atol=0)


# ------------------------------------------------------------------------------ quantisation
def quant_device(x, rows=None, row_map=None, copies=1):
    M, D = x.shape
    rows = M if rows is None else rows
    codes = torch.full((rows, D // 2), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full(((D + 127) // 128, (rows + 3) // 4 * 4), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    moe.moe_mxfp4_quant(x, codes, scales, row_map=row_map, copies=copies)
    return codes, scales


def awkward(rng, M, D):
    """Magnitudes over the whole range, ties, zero blocks, powers of two and their neighbours."""
    x = rng.standard_normal((M, D)) * np.exp2(rng.integers(-24, 12, (M, 1)))
    b = x.reshape(M, -1, 32)
    pick = rng.random(b.shape[:2])
    b[pick < 0.1] = 0.0
    ties = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, -0.25, -5.0], b.shape) * 0.5
    ties[..., 0] = 2.0
    return np.where((pick > 0.9)[..., None], ties, b).reshape(M, D)


@pytest.mark.parametrize("M,D", [(1, 32), (1, 7168), (3, 64), (5, 160), (130, 1408), (1000, 256), (2, 16384)])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_quant_bits_and_back(M, D, kind):
    rng = np.random.default_rng(M + D)
    x, v = typed(awkward(rng, M, D), kind)
    codes, scales = quant_device(x)
    c, s = mx.quantise(v)
    assert np.array_equal(host(codes) & 0x77, mx.pack(c) & 0x77)  # magnitudes
    got = np.stack([host(codes) & 15, host(codes) >> 4], -1).reshape(M, D)
    assert np.array_equal(mx.E2M1[got], mx.E2M1[c])               # and signs, but for zero
    assert np.array_equal(host(scales).view(np.uint32)[:, :M], mx.scale_planes(s)[:, :M])
    for back in ("f32", "f16", "bf16"):
        out = empty((M, D), DTYPES[back])
        moe.moe_mxfp4_dequant(codes, scales, out)
        want = torch.from_numpy(mx.values(c, s).clip(-65504, 65504) if back == "f16" else mx.values(c, s))
        assert torch.equal(out.cpu(), want.to(DTYPES[back]))


def test_quant_extremes():
    """fp32's subnormals and largest values; a block with an infinity or a NaN is NaN, its neighbours are not."""
    x = np.zeros((4, 128), np.float32)
    x[0, :4] = [1e-45, -1e-40, 2.0 ** -126, 0.0]
    x[1, :4] = [3.4e38, -3e38, 1e30, 1.0]
    x[2, 5], x[2, 32:64] = np.inf, 1.0
    x[3, 64], x[3, 70], x[3, 96:] = np.nan, 3.0, -2.0
    codes, scales = quant_device(dev(x))
    c, s = mx.quantise(x.astype(np.float64))
    out = empty((4, 128), torch.float32)
    moe.moe_mxfp4_dequant(codes, scales, out)
    want = mx.values(c, s)
    assert np.array_equal(host(out).astype(np.float64), want, equal_nan=True)
    assert np.isnan(want[2, :32]).all() and np.isnan(want[3, 64:96]).all() and np.isnan(want).sum() == 64


def test_quant_dispatches_rows_and_strides():
    rng = np.random.default_rng(8)
    M, D, copies = 41, 96, 3
    wide, w = typed(rng.standard_normal((M, 200)), "bf16")
    x, v = wide[:, 8:8 + D], w[:, 8:8 + D]
    place = rng.permutation(M * copies + 10)[:M * copies].astype(np.int32)  # some rows are named by none
    place[rng.random(M * copies) < 0.2] = -1
    place[5], place[6] = M * copies + 10, 1 << 30
    rows = M * copies + 10
    codes, scales = quant_device(x, rows, dev(place), copies)
    c, s = mx.quantise(v)
    want_c = np.full((rows, D // 2), 0x5A, np.uint8)
    planes = np.full((1, (rows + 3) // 4 * 4), 0x5A5A5A5A, np.uint32)
    for t in range(M):
        for j in range(copies):
            d = place[t * copies + j]
            if 0 <= d < rows:
                want_c[d] = mx.pack(c)[t]
                planes[:, d] = mx.scale_planes(s)[:, t]
    got = host(codes)
    assert np.array_equal(got & 0x77, want_c & 0x77)
    assert np.array_equal(host(scales).view(np.uint32), planes)


@pytest.mark.parametrize("M,D,copies,kind", [(2500, 96, 2, "f16"), (3000, 1056, 3, "f32"), (2433, 288, 33, "bf16")])
def test_quant_dispatches_many_rows(M, D, copies, kind):
    """The warp-per-row form: every copy of a row equals the row quantised by itself, nothing else is written."""
    rng = np.random.default_rng(M)
    for extra in (0, 3):  # rows on 16-byte boundaries, and not
        wide, _ = typed(rng.standard_normal((M, D + extra)), kind)
        x = wide[:, :D]
        codes, scales = quant_device(x.contiguous())
        rows = M * copies + 7
        place = rng.permutation(rows)[:M * copies].astype(np.int32)
        place[rng.random(M * copies) < 0.1] = -1
        place[17] = rows
        got_c, got_s = quant_device(x, rows, dev(place), copies)
        want_c = np.full((rows, D // 2), 0x5A, np.uint8)
        want_s = np.full(tuple(got_s.shape), 0x5A5A5A5A, np.int32)
        at = np.nonzero((place >= 0) & (place < rows))[0]
        want_c[place[at]] = host(codes)[at // copies]
        want_s[:, place[at]] = host(scales)[:, at // copies]
        assert np.array_equal(host(got_c), want_c) and np.array_equal(host(got_s), want_s)


@pytest.mark.parametrize("E,N,D", [(1, 128, 32), (2, 256, 288), (3, 384, 1408), (1, 128, 256)])
@pytest.mark.parametrize("gate_up", [False, True])
def test_weight_blocks(E, N, D, gate_up):
    rng = np.random.default_rng(N + D)
    for kind in ("f16", "bf16", "f32"):
        w, v = typed(rng.standard_normal((E, N, D)) * 0.05, kind)
        c, s = mx.quantise(v)
        want = mx.blocks(c, s, gate_up).reshape(-1)
        out = torch.full((moe.moe_mxfp4_weights_bytes(E, N, D),), 0x5A, dtype=torch.uint8, device="cuda")
        moe.moe_mxfp4_pack_weights(dev(mx.pack(c)), dev(s), out, gate_up)
        assert np.array_equal(host(out), want)
        out.fill_(0x5A)
        moe.moe_mxfp4_quant_weights(w, out, gate_up)
        got = host(out).reshape(-1, 17408)
        ref = want.reshape(-1, 17408)
        assert np.array_equal(got[:, 16384:], ref[:, 16384:])
        assert np.array_equal(got[:, :16384] & 0x77, ref[:, :16384] & 0x77)


# ------------------------------------------------------------------------------ products
def make_weights(rng, E, N, D, gate_up):
    """Device blocks and values of random MXFP4 weights with spread-out scales and some zero blocks."""
    code = rng.integers(0, 16, (E, N, D), dtype=np.uint8)
    scale = rng.integers(115, 128, (E, N, D // 32)).astype(np.uint8)
    scale[rng.random(scale.shape) < 0.05] = 0
    b = torch.empty(moe.moe_mxfp4_weights_bytes(E, N, D), dtype=torch.uint8, device="cuda")
    moe.moe_mxfp4_pack_weights(dev(mx.pack(code)), dev(scale), b, gate_up)
    return b, mx.values(code, scale)


def make_rows(rng, R, D):
    x = rng.standard_normal((R, D)) * np.exp2(rng.integers(-6, 7, (R, D // 32)).repeat(32, 1))
    c, s = mx.quantise(x)
    return dev(mx.pack(c)), dev(mx.scale_planes(s).view(np.int32)), mx.values(c, s)


# (rows per expert, N, D): empty experts, single rows, tile edges, many rows, odd depths
GMMS = [([1], 128, 32), ([0, 3, 0, 1], 256, 64), ([8, 7, 9], 128, 256), ([5], 384, 288), ([31, 32, 33, 0, 64], 256, 512),
        ([130, 1, 255], 256, 192), ([300], 128, 1408), ([257, 511, 16], 384, 256), ([0, 0], 128, 128),
        ([1000, 2, 40], 640, 448), ([17] * 20, 128, 2048), ([1, 0, 2] * 30, 256, 7168)]


@pytest.mark.parametrize("counts,N,D", GMMS)
def test_gmm(counts, N, D):
    rng = np.random.default_rng(sum(counts) + N + D)
    E, used = len(counts), sum(counts)
    R = used + 5  # rows past the last expert's are dropped routes: not written
    cum = np.cumsum(counts).astype(np.int32)
    codes, scales, a = make_rows(rng, R, D)
    w, wv = make_weights(rng, E, N, D, False)
    c = torch.full((R, N), 7.0, dtype=torch.float16, device="cuda")
    ws = empty(moe.moe_mxfp4_gmm_workspace_size(R, E, N, D), torch.uint8)
    moe.moe_mxfp4_gmm(codes, scales, dev(cum), w, c, ws)
    assert moe.moe_workspace_status(ws) == 0
    got = host(c).astype(np.float64)
    assert (got[used:] == 7.0).all()
    for e in range(E):
        lo, hi = cum[e] - counts[e], cum[e]
        ref, err = a[lo:hi] @ wv[e].T, mx.sum_error(a[lo:hi], wv[e])
        over = np.abs(ref) > 65504
        assert (np.abs(got[lo:hi] - ref.clip(-65504, 65504)) <= err + mx.f16_error(np.abs(ref) + err))[~over].all()
        assert (np.abs(got[lo:hi])[over & (np.abs(ref) > 66000 + err)] == 65504).all()
    again = torch.full_like(c, 7.0)
    moe.moe_mxfp4_gmm(codes, scales, dev(cum), w, again, ws)
    assert torch.equal(c, again)


@pytest.mark.parametrize("counts,I,D", [([1], 64, 32), ([0, 3, 1], 128, 64), ([9, 8], 192, 288), ([33, 0, 100], 256, 512),
                                        ([300, 20], 64, 1024), ([1, 2] * 8, 448, 128), ([700], 704, 256)])
def test_gmm_swiglu(counts, I, D):
    rng = np.random.default_rng(sum(counts) + I + D)
    E, used = len(counts), sum(counts)
    R = used + 3
    cum = np.cumsum(counts).astype(np.int32)
    codes, scales, a = make_rows(rng, R, D)
    w, wv = make_weights(rng, E, 2 * I, D, True)
    hc = torch.full((R, I // 2), 0x5A, dtype=torch.uint8, device="cuda")
    hs = torch.full(((I + 127) // 128, (R + 3) // 4 * 4), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    ws = empty(moe.moe_mxfp4_gmm_workspace_size(R, E, 2 * I, D), torch.uint8)
    moe.moe_mxfp4_gmm_swiglu(codes, scales, dev(cum), w, hc, hs, ws)
    assert moe.moe_workspace_status(ws) == 0
    got_c = np.stack([host(hc) & 15, host(hc) >> 4], -1).reshape(R, I)
    planes = host(hs).view(np.uint32)
    got_s = np.ascontiguousarray(planes[:, :R].T).view(np.uint8).reshape(R, -1)
    assert (host(hc)[used:] == 0x5A).all() and (planes[:, used:R] == 0x5A5A5A5A).all()
    assert (got_s[:used, I // 32:] == 0).all()
    got = mx.values(got_c[:used], got_s[:used, :I // 32])
    for e in range(E):
        lo, hi = cum[e] - counts[e], cum[e]
        gu, err = a[lo:hi] @ wv[e].T, mx.sum_error(a[lo:hi], wv[e])
        h, eh = mx.silu_mul(gu[:, :I], gu[:, I:], err[:, :I], err[:, I:])
        least, most, s0, s1 = mx.quantise_interval(h, eh)
        v, s = got[lo:hi], got_s[lo:hi, :I // 32]
        assert (s >= s0).all() and (s <= s1).all()
        assert (np.abs(v) >= least).all() and (np.abs(v) <= most).all()
        assert ((np.sign(v) == np.sign(h)) | (v == 0) | (np.abs(h) <= eh)).all()


def test_gmm_holds_bad_prefixes_and_nan():
    """cumsum entries outside 0 .. R are held there; a NaN block makes its row's sums NaN, alone."""
    rng = np.random.default_rng(1)
    R, N, D = 20, 128, 128
    codes, scales, a = make_rows(rng, R, D)
    scales[0, 3] = 0x7F7FFF7F  # one block of row 3 is NaN
    w, wv = make_weights(rng, 2, N, D, False)
    c = torch.full((R, N), 7.0, dtype=torch.float16, device="cuda")
    ws = empty(moe.moe_mxfp4_gmm_workspace_size(R, 2, N, D), torch.uint8)
    moe.moe_mxfp4_gmm(codes, scales, dev(np.array([-5, 1 << 30], np.int32)), w, c, ws)
    got = host(c).astype(np.float64)
    assert np.isnan(got[3]).all() and np.isnan(got).sum() == N
    keep = np.arange(R) != 3
    ref = a[keep] @ wv[1].T
    err = mx.sum_error(a[keep], wv[1])
    assert (np.abs(got[keep] - ref.clip(-65504, 65504)) <= err + mx.f16_error(np.abs(ref) + err)).all()


# ------------------------------------------------------------------------------ layer
LAYERS = [  # M, K, I, E, topK
    (1, 128, 64, 1, 1), (1, 256, 256, 8, 2), (1, 1024, 192, 16, 8), (2, 512, 320, 4, 4), (7, 256, 64, 3, 2),
    (16, 256, 256, 8, 2), (29, 384, 128, 5, 3), (32, 256, 448, 2, 1), (33, 256, 128, 2, 2), (64, 128, 64, 8, 8),
    (90, 512, 192, 4, 2), (400, 256, 128, 3, 2), (3, 2048, 704, 4, 2)]


def layer_case(M, K, I, E, topK, seed, drop=0.15):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((M, K)) * np.exp2(rng.integers(-3, 3, (M, 1)))).astype(np.float16)
    ei = np.stack([rng.permutation(E)[:topK] for _ in range(M)]).astype(np.int32)
    ei[rng.random(ei.shape) < drop] = rng.choice([-1, E, 1 << 30])
    if M > 2:
        ei[1] = -1            # a token without a route
        ei[2] = ei[2, 0]      # one expert topK times
    probs = rng.standard_normal((M, topK)).astype(np.float32)
    w1, v1 = make_weights(rng, E, 2 * I, K, True)
    w2, v2 = make_weights(rng, E, K, I, False)
    return x, ei, probs, w1, v1 , w2, v2


def run_layer(x, ei, probs, w1, w2, I, E, ws=None, stream=None):
    (M, K), topK = x.shape, ei.shape[1]
    d = moe.dims(M, K, I, E, topK)
    if ws is None:
        ws = empty(moe.moe_mxfp4_layer_workspace_size(d), torch.uint8)
        ws.fill_(0xEE)
    out = empty((M, K), torch.float16)
    out.fill_(float("nan"))
    moe.moe_mxfp4_layer_fwd(d, x, ei, probs, w1, w2, out, ws, stream=stream)
    return out, ws


@pytest.mark.parametrize("M,K,I,E,topK", LAYERS)
def test_layer(M, K, I, E, topK):
    x, ei, probs, w1, v1, w2, v2 = layer_case(M, K, I, E, topK, M + K + I)
    x = (x * np.float16(2.0 ** -6)).astype(np.float16)  # keeps outputs inside binary16
    args = (dev(x), dev(ei), dev(probs), w1, w2, I, E)
    out, ws = run_layer(*args)
    assert moe.moe_workspace_status(ws) == 0
    ref, err = mx.layer(mx.values(*mx.quantise(x.astype(np.float64))), ei, probs, v1, v2)
    got = host(out).astype(np.float64)
    over = np.abs(ref) + err > 65504
    assert over.mean() < 0.5
    assert (np.abs(got - ref) <= err)[~over].all()
    if M > 2:
        assert (got[1] == 0).all()
    for _ in range(3):  # the same workspace, as it was left
        again, _ = run_layer(*args, ws=ws)
        assert torch.equal(out, again)


def test_layer_without_routes_and_with_nan():
    x, ei, probs, w1, v1, w2, v2 = layer_case(4, 256, 64, 4, 2, 3, drop=0.0)
    none = np.full_like(ei, -1)
    out, ws = run_layer(dev(x), dev(none), dev(probs), w1, w2, 64, 4)
    assert (host(out) == 0).all()
    x[3, 40] = np.nan
    x[0, 7] = np.inf
    ei[1] = -1
    out, ws = run_layer(dev(x), dev(ei), dev(probs), w1, w2, 64, 4)
    got = host(out)
    assert np.isnan(got[3]).all() and np.isnan(got[0]).all() and np.isfinite(got[1:3]).all()


def test_layer_on_another_stream_and_in_a_graph():
    x, ei, probs, w1, v1, w2, v2 = layer_case(5, 512, 128, 8, 2, 11)
    dx, de, dp = dev(x), dev(ei), dev(probs)
    want, ws = run_layer(dx, de, dp, w1, w2, 128, 8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out, _ = run_layer(dx, de, dp, w1, w2, 128, 8, ws=ws)
    s.synchronize()
    assert torch.equal(out, want)
    d = moe.dims(5, 512, 128, 8, 2)
    out.fill_(0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_mxfp4_layer_fwd(d, dx, de, dp, w1, w2, out, ws)
    for _ in range(3):
        out.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_route_then_layer():
    """The router's output is the layer's input, masked experts and padding tokens included."""
    rng = np.random.default_rng(21)
    M, K, I, E, topK = 9, 256, 128, 8, 3
    logits = rng.standard_normal((M, E)).astype(np.float32)
    logits[:, 5] = -np.inf
    logits[4] = -np.inf
    x, _, _, w1, v1, w2, v2 = layer_case(M, K, I, E, topK, 22)
    x = (x * np.float16(2.0 ** -6)).astype(np.float16)
    ei, pr = empty((M, topK), torch.int32), empty((M, topK), torch.float32)
    moe.moe_route_topk(dev(logits), ei, pr)
    out, _ = run_layer(dev(x), ei, pr, w1, w2, I, E)
    ref, err = mx.layer(mx.values(*mx.quantise(x.astype(np.float64))), host(ei), host(pr), v1, v2)
    got = host(out).astype(np.float64)
    assert (np.abs(got - ref) <= err).all() and (got[4] == 0).all()


@pytest.mark.parametrize("tiles,I", [(5, 1024), (19, 512), (12, 1024), (19, 1024), (24, 1024), (17, 1216)])
def test_few_tokens_share_of_the_device(tiles, I):
    """A few tokens' gate and up product in fewer units (64 channels of h x experts) than SMs, as many,
    between one and two of them each, twice as many, more: every way the kernel deals them out."""
    K, topK = 256, 1
    x, _, probs, w1, v1, w2, v2 = layer_case(tiles, K, I, tiles, topK, tiles + I)
    x = (x * np.float16(2.0 ** -6)).astype(np.float16)
    ei = np.random.default_rng(tiles).permutation(tiles).astype(np.int32)[:, None]
    args = (dev(x), dev(ei), dev(probs), w1, w2, I, tiles)
    out, ws = run_layer(*args)
    assert moe.moe_workspace_status(ws) == 0
    ref, err = mx.layer(mx.values(*mx.quantise(x.astype(np.float64))), ei, probs, v1, v2)
    over = np.abs(ref) + err > 65504
    assert (np.abs(host(out).astype(np.float64) - ref) <= err)[~over].all()


@pytest.mark.parametrize("M,K,I,E,topK", [(1, 2048, 1408, 16, 8), (9, 512, 1024, 16, 2), (30, 1024, 256, 4, 4),
                                          (200, 1024, 512, 2, 2)])
def test_layer_repeats_bit_for_bit(M, K, I, E, topK):
    """Whichever CTA finishes first, sums that meet are added in the same order."""
    x, ei, probs, w1, _, w2, _ = layer_case(M, K, I, E, topK, M + I)
    args = (dev(x), dev(ei), dev(probs), w1, w2, I, E)
    out, ws = run_layer(*args)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        again, _ = run_layer(*args, ws=ws)
        differ += (again.view(torch.int16) != out.view(torch.int16)).sum()
    assert differ.item() == 0 and moe.moe_workspace_status(ws) == 0


def test_example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_experts.py")
    spec = importlib.util.spec_from_file_location("mxfp4_experts", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # Each of the three products' factors is off by four bits' 2^-2 / sqrt(3) of its size at most, a
    # uniform error of half a step: x, W1, h, W2 independent, sqrt(4) * 0.145, and more through SwiGLU.
    for tokens in (1, 40):
        _, distance = example.run(tokens=tokens, hidden=512, intermediate=256, experts=8, topk=2, steps=2)
        assert 0.01 < distance < 0.5


def test_many_tokens_on_another_stream_and_in_a_graph():
    """The path of many tokens, whose launches overlap: the same bits on a second stream behind work of its
    own, from a CUDA graph, and with calls on two workspaces in flight at once."""
    M, K, I, E, topK = 150, 512, 128, 4, 2
    x, ei, probs, w1, _, w2, _ = layer_case(M, K, I, E, topK, 17)
    dx, de, dp = dev(x), dev(ei), dev(probs)
    want, ws = run_layer(dx, de, dp, w1, w2, I, E)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    late = torch.zeros_like(dx)
    with torch.cuda.stream(s):
        torch.cuda._sleep(1000000)
        late.copy_(dx)
        there, ws2 = run_layer(late, de, dp, w1, w2, I, E)
    here, _ = run_layer(dx, de, dp, w1, w2, I, E, ws=ws)
    s.synchronize()
    assert torch.equal(there, want) and torch.equal(here, want)
    d = moe.dims(M, K, I, E, topK)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        moe.moe_mxfp4_layer_fwd(d, dx, de, dp, w1, w2, out, ws)
        moe.moe_mxfp4_layer_fwd(d, dx, de, dp, w1, w2, out, ws2)
    for _ in range(5):
        out.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert moe.moe_workspace_status(ws) == 0 and moe.moe_workspace_status(ws2) == 0


def test_product_behind_the_quantisation_that_feeds_it():
    """Rows quantised and multiplied back to back with new rows each time: a product that began before
    its operands were written would use the call's before."""
    rng = np.random.default_rng(5)
    E, N, D, per = 3, 256, 1056, 40
    R = E * per
    cum = dev(np.arange(1, E + 1, dtype=np.int32) * per)
    w, _ = make_weights(rng, E, N, D, False)
    ws = empty(moe.moe_mxfp4_gmm_workspace_size(R, E, N, D), torch.uint8)
    codes, scales = empty((R, D // 2), torch.uint8), empty((moe.moe_mxfp4_scale_words(R, D),), torch.int32)
    xs = [torch.randn(R, D, device="cuda", dtype=torch.float16) for _ in range(8)]

    def product(x):
        c = empty((R, N), torch.float16)
        moe.moe_mxfp4_quant(x, codes, scales)
        moe.moe_mxfp4_gmm(codes, scales, cum, w, c, ws)
        return c

    alone = []
    for x in xs:
        alone.append(product(x))
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, [product(x) for x in xs]))


def test_offsets_past_32_bits():
    """Elements and bytes past 2^32: the last rows of large arrays are those of a call on them alone."""
    rows, D, last = 270000, 16384, 37  # 2^32 elements are 262144 rows
    x = torch.zeros(rows, D, dtype=torch.float16, device="cuda")
    x[-last:] = torch.randn(last, D, device="cuda", dtype=torch.float16)
    codes, scales = quant_device(x)
    want_codes, want_scales = quant_device(x[-last:].contiguous())
    planes = scales.view(D // 128, -1)[:, rows - last:rows]
    assert torch.equal(codes[-last:], want_codes)
    assert torch.equal(planes, want_scales.view(D // 128, -1)[:, :last])
    assert not codes[:-last].any() and not scales.view(D // 128, -1)[:, :rows - last].any()
    back = x.fill_(1.0)
    moe.moe_mxfp4_dequant(codes, scales, back)
    small = empty((last, D), torch.float16)
    moe.moe_mxfp4_dequant(want_codes, want_scales, small)
    assert torch.equal(back[-last:], small) and not back[:-last].any()
    del x, back, codes, scales

    R, N, D = 70004, 65536, 64  # 2^32 outputs are 65536 rows
    rng = np.random.default_rng(8)
    w, _ = make_weights(rng, 1, N, D, False)
    a = torch.randn(R, D, device="cuda", dtype=torch.float16)
    codes, scales = quant_device(a)
    few_codes, few_scales = quant_device(a[-last:].contiguous())
    ws = empty(moe.moe_mxfp4_gmm_workspace_size(R, 1, N, D), torch.uint8)
    c, want = empty((R, N), torch.float16), empty((last, N), torch.float16)
    moe.moe_mxfp4_gmm(codes, scales, dev(np.array([R], np.int32)), w, c, ws)
    moe.moe_mxfp4_gmm(few_codes, few_scales, dev(np.array([last], np.int32)), w, want, ws)
    assert torch.equal(c[-last:], want)


def test_router_and_layer_behind_the_work_that_feeds_them():
    """Logits and tokens written, routed and put through the layer without a pause, with new ones each
    time: a kernel that read before the one in front of it had written would use the call's before."""
    K, I, E, topK = 512, 128, 8, 2
    rng = np.random.default_rng(33)
    w1, _ = make_weights(rng, E, 2 * I, K, True)
    w2, _ = make_weights(rng, E, K, I, False)
    for M in (1, 6, 100):  # a few tokens, and many
        d = moe.dims(M, K, I, E, topK)
        ws = empty(moe.moe_mxfp4_layer_workspace_size(d), torch.uint8)
        logits, x = empty((M, E), torch.float32), empty((M, K), torch.float16)
        idx, probs = empty((M, topK), torch.int32), empty((M, topK), torch.float32)
        sets = [(torch.randn(M, E, device="cuda"), torch.randn(M, K, device="cuda").half() / 64) for _ in range(10)]

        def layer(s):
            out = empty((M, K), torch.float16)
            logits.copy_(s[0])
            x.copy_(s[1])
            moe.moe_route_topk(logits, idx, probs)
            moe.moe_mxfp4_layer_fwd(d, x, idx, probs, w1, w2, out, ws)
            return out

        alone = []
        for s in sets:
            alone.append(layer(s))
            torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone * 3, [layer(s) for s in sets * 3]))
        assert moe.moe_workspace_status(ws) == 0
