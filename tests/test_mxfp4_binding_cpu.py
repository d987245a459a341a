"""Without a GPU: what the MXFP4 layer's sizes promise, and what its binding refuses."""
import pytest


@pytest.fixture(scope="module")
def moe():
    from moe_expert_layer_gb300 import build
    build.build()
    import moe_expert_layer_gb300
    moe_expert_layer_gb300.load_library()
    return moe_expert_layer_gb300


@pytest.mark.parametrize("K,I,E,topK", [(128, 64, 1, 1), (7168, 2048, 256, 8), (4096, 1408, 64, 6), (256, 64, 64, 40),
                                        (16384, 8192, 8, 8), (1024, 8192, 512, 300), (128, 64, 1023, 1023)])
def test_layer_workspace_never_shrinks(moe, K, I, E, topK):
    """A workspace made for the largest batch serves every smaller one."""
    tokens = [m for m in [*range(1, 300), 512, 1000, 4096, 8192, 65536] if m * topK < 1 << 24]
    sizes = [moe.moe_mxfp4_layer_workspace_size(moe.dims(m, K, I, E, topK)) for m in tokens]
    assert min(sizes) > 0
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def layer_arguments(moe):
    import torch
    d = moe.dims(4, 128, 64, 2, 2)
    return d, {"x": torch.zeros(4, 128, dtype=torch.float16), "expert_idx": torch.zeros(4, 2, dtype=torch.int32),
               "probs": torch.zeros(4, 2), "w1": torch.zeros(moe.moe_mxfp4_weights_bytes(2, 128, 128), dtype=torch.uint8),
               "w2": torch.zeros(moe.moe_mxfp4_weights_bytes(2, 128, 64), dtype=torch.uint8),
               "out": torch.zeros(4, 128, dtype=torch.float16),
               "workspace": torch.zeros(moe.moe_mxfp4_layer_workspace_size(d), dtype=torch.uint8)}


def test_layer_refuses_arrays_of_other_types_and_sizes(moe):
    """The indices of torch.topk are int64, and bfloat16 has binary16's size: both were read as what
    they are not.  Short arrays were read and written past their end."""
    import torch
    for name, bad in (("x", lambda t: t.bfloat16()), ("x", lambda t: t.float()), ("x", lambda t: t[:3]),
                      ("expert_idx", lambda t: t.long()), ("expert_idx", lambda t: t.float()),
                      ("expert_idx", lambda t: t[:, :1].contiguous()), ("probs", lambda t: t.half()),
                      ("probs", lambda t: t.int()), ("probs", lambda t: t[:3]), ("w1", lambda t: t[:-1]),
                      ("w2", lambda t: t[:-1]), ("out", lambda t: t.bfloat16()), ("out", lambda t: t[:3]),
                      ("out", lambda t: t.float())):
        d, a = layer_arguments(moe)
        a[name] = bad(a[name])
        with pytest.raises(ValueError, match=name):
            moe.moe_mxfp4_layer_fwd(d, **a, stream=0)
    d, a = layer_arguments(moe)
    a["x"] = torch.zeros(128, 4, dtype=torch.float16).t()
    with pytest.raises(ValueError):
        moe.moe_mxfp4_layer_fwd(d, **a, stream=0)


def test_layer_takes_what_it_took(moe):
    """Larger arrays, bits of binary16, weights of any type and raw pointers reach the library, which
    refuses on its own what it does: here a missing array."""
    import torch
    d, a = layer_arguments(moe)
    a["x"], a["out"] = torch.zeros(9, 128, dtype=torch.int16), 4096
    a["w1"] = a["w1"].view(torch.int32)
    a["probs"] = None
    with pytest.raises(moe.MoeError, match="NULL"):
        moe.moe_mxfp4_layer_fwd(d, **a, stream=0)


def test_operators_refuse_arrays_of_other_types(moe):
    import torch
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.int32)
    w = torch.zeros(moe.moe_mxfp4_weights_bytes(1, 128, 64), dtype=torch.uint8)
    ws, cumsum = torch.zeros(256, dtype=torch.uint8), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="c:"):
        moe.moe_mxfp4_gmm(codes, scales, cumsum, w, torch.zeros(4, 128, dtype=torch.bfloat16), ws, stream=0)
    with pytest.raises(ValueError, match="cumsum"):
        moe.moe_mxfp4_gmm(codes, scales, cumsum.float(), w, torch.zeros(4, 128, dtype=torch.float16), ws, stream=0)
    logits, idx, probs = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="expert_idx"):
        moe.moe_route_topk(logits, idx.float(), probs, stream=0)
    with pytest.raises(ValueError, match="probs"):
        moe.moe_route_topk(logits, idx, probs.int(), stream=0)
    with pytest.raises(ValueError, match="bias"):
        moe.moe_route_topk(logits, idx, probs, bias=torch.zeros(8, dtype=torch.int32), stream=0)
    with pytest.raises(ValueError, match="row_map"):
        moe.moe_mxfp4_quant(torch.zeros(4, 64), codes, scales, row_map=torch.zeros(4), stream=0)
