"""The MXFP4 layer where its paths could differ: a token's routes are weighted and added in 32 bits
whichever kernels a batch takes, and rounded to binary16 once."""
import numpy as np
import pytest

import mx_reference as mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_expert_layer_gb300 as moe
    from gpu_util import dev, host
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
