"""Without a GPU: the tests' 64-bit MXFP4 reference against hand-worked values, the sizes and
refusals of the router's and the MXFP4 operators' entry points, and the binding's checks."""
import ctypes

import numpy as np
import pytest

import mx_reference as mx

A, U = 4096, 4096 + 8  # aligned to 256 bytes; to 8 only


@pytest.fixture(scope="module")
def lib():
    from moe_expert_layer_gb300 import build
    build.build()
    import moe_expert_layer_gb300 as moe
    return moe.load_library()


def test_reference_quantisation_by_hand():
    """a = 5: floor(log2 5) - 2 = 0, so elements are the e2m1 values themselves; ties go to the even code."""
    x = np.zeros((1, 64))
    x[0, :10] = [5.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -0.75, 0.2500001, -5.0]
    x[0, 32:35] = [7.9, 6.1, 2.0 ** -3]       # above 6: saturates
    code, scale = mx.quantise(x)
    assert scale.tolist() == [[127, 127]]
    assert mx.values(code, scale)[0, :10].tolist() == [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, -1.0, 0.5, -4.0]
    assert mx.values(code, scale)[0, 32:35].tolist() == [6.0, 6.0, 0.0]
    for a, b in ((0.0, 0), (1.0, 125), (2.0 ** -130, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (3.0e38, 252)):
        assert mx.scale_byte(np.array(a)) == b


def test_reference_interval_holds_the_value():
    rng = np.random.default_rng(3)
    h = rng.standard_normal((40, 64))
    err = np.full_like(h, 1e-3)
    lo, hi, s0, s1 = mx.quantise_interval(h, err)
    for sign in (-1, 0, 1):
        moved = h + sign * err * rng.random(h.shape)
        code, scale = mx.quantise(moved)
        v = np.abs(mx.values(code, scale))
        assert (v >= lo).all() and (v <= hi).all() and (scale >= s0).all() and (scale <= s1).all()


def test_sizes(lib):
    import moe_expert_layer_gb300 as moe
    assert moe.moe_mxfp4_scale_words(5, 160) == 2 * 8
    assert moe.moe_mxfp4_scale_words(1, 32) == 4
    for rows, D in ((0, 64), (1 << 24, 64), (4, 48), (4, 0), (4, 16416)):
        assert moe.moe_mxfp4_scale_words(rows, D) == 0
    assert moe.moe_mxfp4_weights_bytes(64, 2816, 4096) == 64 * 22 * 16 * 17408
    assert moe.moe_mxfp4_weights_bytes(1, 128, 288) == 2 * 17408
    for E, N, D in ((0, 128, 64), (1024, 128, 64), (1, 64, 64), (1, 192, 64), (1, 128, 40)):
        assert moe.moe_mxfp4_weights_bytes(E, N, D) == 0
        assert moe.moe_mxfp4_gmm_workspace_size(4, E, N, D) == 0
    assert moe.moe_mxfp4_gmm_workspace_size(4, 8, 128, 64) > 0
    assert moe.moe_mxfp4_gmm_workspace_size(0, 8, 128, 64) == 0
    assert moe.moe_mxfp4_layer_workspace_size(moe.dims(1, 256, 64, 4, 2)) > 0
    assert moe.moe_mxfp4_layer_workspace_size(moe.dims(1, 200, 64, 4, 2)) == 0


def test_refusals(lib):
    """Shape, NULL and alignment are refused on the host, in this order, before any device call."""
    import moe_expert_layer_gb300 as moe
    f32, none, score = moe.TYPE_F32, None, moe.SCORE_SOFTMAX

    def route(M=4, E=8, topK=2, l=A, type=f32, stride=8, bias=none, sc=score, i=A, p=A):
        return lib.moe_route_topk(M, E, topK, l, type, stride, bias, sc, 1, 1.0, i, p, none)
    for bad in (dict(M=0), dict(topK=0), dict(topK=9), dict(E=1024, stride=1024), dict(stride=7), dict(type=3),
                dict(type=-1), dict(sc=2), dict(M=1 << 23)):
        assert route(**bad) == -2, bad
    for k in ("l", "i", "p"):
        assert route(**{k: none}) == -1
        assert route(**{k: U}) == -3
    assert route(bias=U) == -3

    def quant(M=4, D=64, x=A, type=f32, stride=64, map=none, copies=1, rows=4, c=A, s=A):
        return lib.moe_mxfp4_quant(M, D, x, type, stride, map, copies, rows, c, s, none)
    for bad in (dict(M=0), dict(D=48), dict(D=16416, stride=16416), dict(stride=63), dict(type=9), dict(copies=0),
                dict(copies=2), dict(rows=5), dict(rows=0, map=A), dict(copies=1 << 22, map=A)):
        assert quant(**bad) == -2, bad
    assert quant(x=none) == -1 and quant(c=none) == -1 and quant(s=none) == -1
    assert quant(x=U) == -3 and quant(map=U, copies=2, rows=9) == -3 and quant(s=U) == -3

    assert lib.moe_mxfp4_dequant(4, 48, A, A, A, f32, none) == -2
    assert lib.moe_mxfp4_dequant(4, 64, A, A, A, 5, none) == -2
    assert lib.moe_mxfp4_dequant(4, 64, A, none, A, f32, none) == -1
    assert lib.moe_mxfp4_dequant(4, 64, A, A, U, f32, none) == -3
    assert lib.moe_mxfp4_quant_weights(1, 64, 64, 0, A, f32, A, none) == -2
    assert lib.moe_mxfp4_quant_weights(1, 128, 64, 0, A, 7, A, none) == -2
    assert lib.moe_mxfp4_quant_weights(1, 128, 64, 0, none, f32, A, none) == -1
    assert lib.moe_mxfp4_quant_weights(1, 128, 64, 0, A, f32, U, none) == -3
    assert lib.moe_mxfp4_pack_weights(1, 128, 60, 0, A, A, A, none) == -2
    assert lib.moe_mxfp4_pack_weights(1, 128, 64, 0, A, none, A, none) == -1
    assert lib.moe_mxfp4_pack_weights(1, 128, 64, 0, A, U, A, none) == -3

    ws = moe.moe_mxfp4_gmm_workspace_size(4, 8, 128, 64)
    assert lib.moe_mxfp4_gmm(4, 8, 130, 64, *[A] * 6, ws, none) == -2
    assert lib.moe_mxfp4_gmm_swiglu(4, 8, 96, 64, *[A] * 7, ws, none) == -2
    assert lib.moe_mxfp4_gmm_swiglu(4, 8, 8256, 64, *[A] * 7, ws, none) == -2
    for f, n, N in ((lib.moe_mxfp4_gmm, 6, 128), (lib.moe_mxfp4_gmm_swiglu, 7, 64)):
        for i in range(n):
            p = [A] * n
            p[i] = none
            assert f(4, 8, N, 64, *p, ws, none) == -1
            p[i] = U
            assert f(4, 8, N, 64, *p, ws, none) == -3
        assert f(4, 8, N, 64, *[A] * n, ws - 1, none) == -5

    d, bad = moe.dims(2, 256, 64, 4, 2), moe.dims(2, 256, 96, 4, 2)
    ws = moe.moe_mxfp4_layer_workspace_size(d)
    assert lib.moe_mxfp4_layer_fwd(None, *[A] * 7, ws, none) == -1
    assert lib.moe_mxfp4_layer_fwd(ctypes.byref(bad), *[A] * 7, ws, none) == -2
    for i in range(7):
        p = [A] * 7
        p[i] = none
        assert lib.moe_mxfp4_layer_fwd(ctypes.byref(d), *p, ws, none) == -1
        p[i] = U
        assert lib.moe_mxfp4_layer_fwd(ctypes.byref(d), *p, ws, none) == -3
    assert lib.moe_mxfp4_layer_fwd(ctypes.byref(d), *[A] * 7, ws - 1, none) == -5


def test_binding_checks_shapes_and_types(lib):
    """Sizes come from the tensors: too small, of another type or with rows that are not dense they
    are refused before the library is called."""
    import torch
    import moe_expert_layer_gb300 as moe
    logits = torch.zeros(4, 8)
    idx, probs = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        moe.moe_route_topk(logits.double(), idx, probs, stream=0)
    with pytest.raises(ValueError):
        moe.moe_route_topk(torch.zeros(8, 4).t(), idx, probs, stream=0)
    with pytest.raises(ValueError):
        moe.moe_route_topk(logits, idx.long(), probs, stream=0)
    with pytest.raises(ValueError):
        moe.moe_route_topk(logits, idx, probs[:3], stream=0)
    x = torch.zeros(4, 64, dtype=torch.float16)
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.moe_mxfp4_quant(x, codes, scales[:, :3].contiguous(), stream=0)
    with pytest.raises(ValueError):
        moe.moe_mxfp4_quant(x, codes[:, :31].contiguous(), scales, stream=0)
    with pytest.raises(ValueError):
        moe.moe_mxfp4_dequant(codes, scales, x.double(), stream=0)
    with pytest.raises(ValueError):
        moe.moe_mxfp4_quant_weights(torch.zeros(1, 128, 64), torch.zeros(17407, dtype=torch.uint8), stream=0)
    with pytest.raises(ValueError):
        moe.moe_mxfp4_gmm(codes, scales, torch.zeros(1, dtype=torch.int32), torch.zeros(17000, dtype=torch.uint8),
                          torch.zeros(4, 128, dtype=torch.float16), torch.zeros(256, dtype=torch.uint8), stream=0)
