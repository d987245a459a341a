"""The MXFP4 layer where its paths could differ: a token's routes are weighted and added in 32 bits
whichever kernels a batch takes, and rounded to binary16 once."""
import numpy as np
import pytest

import mx_reference as mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_expert_layer_gb300 as moe
    import test_gpu_mxfp4 as base
    from gpu_util import dev, empty, host
    from test_gpu_mxfp4 import layer_case, make_weights, run_layer


def routes64(x, ei, w1, w2):
    """Every route's row of the down product, [M][topK][K], and how far fp32 sums and the codes of h
    that they may move can take it; 0 for routes that are dropped."""
    I, shape = w2.shape[2], ei.shape + (x.shape[1],)
    y, err = np.zeros(shape), np.zeros(shape)
    for t, j in zip(*np.nonzero((ei >= 0) & (ei < w1.shape[0]))):
        a, wu, wd = x[t:t + 1], w1[ei[t, j]], w2[ei[t, j]]
        gu, eg = a @ wu.T, mx.sum_error(a, wu)
        h, eh = mx.silu_mul(gu[:, :I], gu[:, I:], eg[:, :I], eg[:, I:])
        q = mx.values(*mx.quantise(h))
        lo, hi, _, _ = mx.quantise_interval(h, eh)
        y[t, j] = (q @ wd.T)[0]
        err[t, j] = (mx.sum_error(np.maximum(np.abs(q), hi), wd) + (hi - lo) @ np.abs(wd).T)[0]
    return y, err


def weighted(y, err, probs):
    """The layer's output and its bound: fp32 products and sums of up to 15 routes (2^-20 of their
    magnitudes), one rounding to binary16."""
    p = probs.astype(np.float64)[..., None]
    out, e = (p * y).sum(1), (np.abs(p) * (err + np.abs(y) * 2.0 ** -20)).sum(1)
    return out, e + mx.f16_error(np.abs(out) + e)


# few tokens; many, of few rows per expert; many, of more (CTA pairs)
SHAPES = [(32, 256, 128, 4, 2), (33, 256, 128, 4, 2), (90, 256, 128, 4, 2)]


@pytest.mark.parametrize("M,K,I,E,topK", SHAPES)
def test_routes_past_binary16(M, K, I, E, topK):
    """Rows of routes many times past 65504 whose weights bring the output back."""
    x, ei, probs, w1, v1, w2, v2 = layer_case(M, K, I, E, topK, 5)
    x = (x * np.float16(2.0 ** 4)).astype(np.float16)
    y, err = routes64(mx.values(*mx.quantise(x.astype(np.float64))), ei, v1, v2)
    probs = (probs * (20000.0 / np.abs(weighted(y, err, probs)[0]).max())).astype(np.float32)
    ref, bound = weighted(y, err, probs)
    assert (np.abs(y) > 4 * 65504.0).mean() > 0.02 and np.abs(ref).max() < 30000
    out, ws = run_layer(dev(x), dev(ei), dev(probs), w1, w2, I, E)
    assert moe.moe_workspace_status(ws) == 0
    assert (np.abs(host(out).astype(np.float64) - ref) <= bound).all()


@pytest.mark.parametrize("M,K,I,E,topK", SHAPES)
def test_routes_below_binary16(M, K, I, E, topK):
    """Rows of routes in and under binary16's subnormals whose weights bring the output up."""
    x, ei, probs, w1, v1, w2, v2 = layer_case(M, K, I, E, topK, 6)
    x = (x * np.float16(2.0 ** -12)).astype(np.float16)
    y, err = routes64(mx.values(*mx.quantise(x.astype(np.float64))), ei, v1, v2)
    probs = (probs * (100.0 / np.abs(weighted(y, err, probs)[0]).max())).astype(np.float32)
    ref, bound = weighted(y, err, probs)
    assert np.abs(y).max() < 2.0 ** -4
    out, ws = run_layer(dev(x), dev(ei), dev(probs), w1, w2, I, E)
    assert moe.moe_workspace_status(ws) == 0
    assert (np.abs(host(out).astype(np.float64) - ref) <= bound).all()


@pytest.mark.parametrize("M,K,I,E,topK", SHAPES)
def test_output_is_rounded_once(M, K, I, E, topK):
    """Routes that partly cancel: the rounding of their rows to binary16 would show in the sum."""
    x, ei, probs, w1, v1, w2, v2 = layer_case(M, K, I, E, topK, 7, drop=0.0)
    x = (x * np.float16(2.0 ** -6)).astype(np.float16)
    probs[:, 1] = -probs[:, 0]
    y, err = routes64(mx.values(*mx.quantise(x.astype(np.float64))), ei, v1, v2)
    ref, bound = weighted(y, err, probs)
    out, ws = run_layer(dev(x), dev(ei), dev(probs), w1, w2, I, E)
    over = np.abs(ref) + bound > 65504
    assert over.mean() < 0.5 and moe.moe_workspace_status(ws) == 0
    assert (np.abs(host(out).astype(np.float64) - ref) <= bound)[~over].all()


@pytest.mark.parametrize("M", [880, 960])
def test_combine_reads_the_rows_of_its_call(M):
    """On both sides of the batch up to which the weighted sum is launched beside the product whose rows
    it reads (912 blocks on 152 SMs, one per token here): with other tokens and routes in every call,
    a line read early is that of a call before."""
    K, I, E, topK = 1024, 64, 8, 2
    rng = np.random.default_rng(M)
    w1, _ = make_weights(rng, E, 2 * I, K, True)
    w2, _ = make_weights(rng, E, K, I, False)
    d = moe.dims(M, K, I, E, topK)
    ws = torch.full((moe.moe_mxfp4_layer_workspace_size(d),), 0xEE, dtype=torch.uint8, device="cuda")
    sets = [(torch.randn(M, K, device="cuda").half() / 64,
             torch.rand(M, E, device="cuda").topk(topK, 1).indices.int().contiguous(), torch.rand(M, topK, device="cuda"))
            for _ in range(8)]

    def layer(x, ei, probs):
        out = torch.empty((M, K), dtype=torch.float16, device="cuda")
        moe.moe_mxfp4_layer_fwd(d, x, ei, probs, w1, w2, out, ws)
        return out

    alone = []
    for s in sets:
        alone.append(layer(*s))
        torch.cuda.synchronize()
    for _ in range(10):
        outs = [layer(*s) for s in sets]
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))
    assert moe.moe_workspace_status(ws) == 0


@pytest.mark.parametrize("M,K,I,E,topK", [(128, 128, 64, 64, 6), (40, 256, 128, 16, 2), (200, 128, 192, 33, 3)])
@pytest.mark.parametrize("skew", [False, True])
def test_layer_of_many_tokens_on_many_experts(M, K, I, E, topK, skew):
    """Past the few-token path with up to 32 rows per expert on average; skewed: half of the tokens on one
    set of experts, which then have more."""
    x, ei, probs, w1, v1, w2, v2 = layer_case(M, K, I, E, topK, M + E)
    if skew:
        ei[::2] = np.arange(topK)
    x = (x * np.float16(2.0 ** -6)).astype(np.float16)
    y, err = routes64(mx.values(*mx.quantise(x.astype(np.float64))), ei, v1, v2)
    ref, bound = weighted(y, err, probs)
    assert M * topK / E <= 32 and (not skew or np.bincount(ei[(ei >= 0) & (ei < E)]).max() >= M // 2)
    out, ws = run_layer(dev(x), dev(ei), dev(probs), w1, w2, I, E)
    over = np.abs(ref) + bound > 65504
    assert over.mean() < 0.5 and moe.moe_workspace_status(ws) == 0
    assert (np.abs(host(out).astype(np.float64) - ref) <= bound)[~over].all()


def signed(codes, D):
    """Values of packed codes [..][D / 2], their signs with them."""
    c = host(codes)
    return mx.E2M1[np.stack([c & 15, c >> 4], -1).reshape(c.shape[:-1] + (D,))]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_signs_of_dispatched_rows_and_weights(kind):
    rng = np.random.default_rng(14)
    M, D, copies = 53, 160, 2
    x, v = base.typed(base.awkward(rng, M, D), kind)
    place = rng.permutation(M * copies).astype(np.int32)
    codes, _ = base.quant_device(x, M * copies, dev(place), copies)
    want = mx.E2M1[mx.quantise(v)[0]]
    assert np.array_equal(signed(codes, D)[place], want.repeat(copies, 0))
    for gate_up in (False, True):
        E, N, D = 2, 256, 288
        w, v = base.typed(base.awkward(rng, E * N, D).reshape(E, N, D), kind)
        c, s = mx.quantise(v)
        out = empty((moe.moe_mxfp4_weights_bytes(E, N, D),), torch.uint8)
        moe.moe_mxfp4_quant_weights(w, out, gate_up)
        got, ref = host(out).reshape(-1, 17408), mx.blocks(c, s, gate_up).reshape(-1, 17408)
        assert np.array_equal(got[:, 16384:], ref[:, 16384:])
        assert np.array_equal(mx.E2M1[got[:, :16384] & 15], mx.E2M1[ref[:, :16384] & 15])
        assert np.array_equal(mx.E2M1[got[:, :16384] >> 4], mx.E2M1[ref[:, :16384] >> 4])


@pytest.mark.parametrize("M,K,I,E,topK", [(4, 128, 64, 80, 64), (1, 256, 128, 256, 256), (32, 128, 64, 8, 8), (32, 128, 64, 9, 8),
                                          (2, 128, 64, 1023, 100), (40, 128, 64, 1023, 3), (3, 16384, 64, 3, 2),
                                          (2, 128, 8192, 3, 2), (50, 128, 8192, 2, 1)])
def test_layer_at_the_ends_of_its_ranges(M, K, I, E, topK):
    """As many routes and experts as there may be, the deepest products, and the few-token path's last sizes."""
    x, ei, probs, w1, v1, w2, v2 = layer_case(M, K, I, E, topK, M + I)
    x = (x * np.float16(2.0 ** -7)).astype(np.float16)
    y, err = routes64(mx.values(*mx.quantise(x.astype(np.float64))), ei, v1, v2)
    ref, bound = weighted(y, err, probs / 16)
    # more than 15 routes: every addition may drop 2^-24 of the magnitudes
    bound = bound + topK * 2.0 ** -24 * (np.abs(probs.astype(np.float64) / 16)[..., None] * np.abs(y)).sum(1)
    out, ws = run_layer(dev(x), dev(ei), dev((probs / 16).astype(np.float32)), w1, w2, I, E)
    over = np.abs(ref) + bound > 65504
    assert over.mean() < 0.5 and moe.moe_workspace_status(ws) == 0
    assert (np.abs(host(out).astype(np.float64) - ref) <= bound)[~over].all()
