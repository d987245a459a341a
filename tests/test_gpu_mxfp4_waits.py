"""How the few-token MXFP4 layer's blocks wait for one another and for work: answers that have to
agree, and calls that share the device."""
import ctypes

import numpy as np
import pytest

import mx_reference as mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_expert_layer_gb300 as moe
    from gpu_util import dev, empty, host
    from test_gpu_mxfp4 import layer_case, make_weights
    from test_gpu_mxfp4_layer import routes64, weighted


def test_epilogue_warps_give_up_together():
    """A unit that arrives after one warp has seen the block give up is taken by none of them."""
    for _ in range(20):
        answers = torch.full((4,), -7, dtype=torch.int32, device="cuda")
        moe.moe_selftest_mxfp4_tickets(answers)
        assert answers.tolist() == [0, 0, 0, 0]


def layers(sizes, K, I, E, topK):
    """Few-token layers of the given numbers of tokens on the same experts, each with its own buffers:
    calls, and their outputs when they run alone."""
    rng = np.random.default_rng(sum(sizes))
    w1, _ = make_weights(rng, E, 2 * I, K, True)
    w2, _ = make_weights(rng, E, K, I, False)
    calls, alone = [], []
    for M in sizes:
        x, ei, probs = layer_inputs(rng, M, K, E, topK)
        d = moe.dims(M, K, I, E, topK)
        ws = empty(moe.moe_mxfp4_layer_workspace_size(d), torch.uint8)

        def call(out, d=d, x=x, ei=ei, probs=probs, ws=ws):
            moe.moe_mxfp4_layer_fwd(d, x, ei, probs, w1, w2, out, ws)
            return ws

        out = empty((M, K), torch.float16)
        call(out)
        torch.cuda.synchronize()
        calls.append(call)
        alone.append(out)
    return calls, alone


def layer_inputs(rng, M, K, E, topK):
    x = (rng.standard_normal((M, K)) / 64).astype(np.float16)
    ei = np.stack([rng.permutation(E)[:topK] for _ in range(M)]).astype(np.int32)
    return dev(x), dev(ei), dev(rng.random((M, topK)).astype(np.float32))


@pytest.mark.parametrize("priorities", [(0, 0), (0, -1), (0, 0, -1, -1)])
def test_few_token_layers_on_several_streams(priorities):
    """Layers whose kernels each want every SM, in flight on streams of the same and of different
    priorities, beside many small kernels: each gives what it gives alone, and none runs into its limit."""
    sizes = [3, 17, 1, 30][:len(priorities)]
    calls, alone = layers(sizes, 1024, 512, 16, 4)
    streams = [torch.cuda.Stream(priority=p) for p in priorities]
    outs = [[torch.zeros_like(a) for _ in range(40)] for a in alone]
    noise = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for i in range(40):
        for s, call, o in zip(streams, calls, outs):
            with torch.cuda.stream(s):
                call(o[i])
        noise.mul_(1.0)
    torch.cuda.synchronize()
    for call, o, want in zip(calls, outs, alone):
        assert all(torch.equal(out, want) for out in o)
        assert moe.moe_workspace_status(call(o[0])) == 0


def test_few_token_layers_beside_large_ones():
    """Few tokens on one stream, hundreds on two others, whose kernels hold every SM's shared memory and are
    launched ahead of what they wait for."""
    sizes = [2, 300, 25, 600]
    calls, alone = layers(sizes, 1024, 512, 16, 4)
    streams = [torch.cuda.Stream(priority=p) for p in (0, 0, -1, -1)]
    outs = [[torch.zeros_like(a) for _ in range(30)] for a in alone]
    torch.cuda.synchronize()
    for i in range(30):
        for s, call, o in zip(streams, calls, outs):
            with torch.cuda.stream(s):
                call(o[i])
    torch.cuda.synchronize()
    for call, o, want in zip(calls, outs, alone):
        assert all(torch.equal(out, want) for out in o)
        assert moe.moe_workspace_status(call(o[0])) == 0


class DevResource(ctypes.Structure):
    """CUdevResource of the driver API; of its union only the number of SMs is read."""
    _fields_ = [("type", ctypes.c_int), ("padding", ctypes.c_ubyte * 92), ("sm_count", ctypes.c_uint),
                ("rest", ctypes.c_ubyte * 44)]


@pytest.fixture
def narrow_stream():
    """A stream of a green context of this process with less than half of the device's SMs."""
    torch.zeros(1, device="cuda")
    cu = ctypes.CDLL("libcuda.so.1")
    whole, part, rest = DevResource(), DevResource(), DevResource()
    groups, desc, ctx, stream = ctypes.c_uint(1), ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    ref = ctypes.byref
    for rc in (cu.cuDeviceGetDevResource(0, ref(whole), 1),
               cu.cuDevSmResourceSplitByCount(ref(part), ref(groups), ref(whole), ref(rest), 0, 64),
               cu.cuDevResourceGenerateDesc(ref(desc), ref(part), 1), cu.cuGreenCtxCreate(ref(ctx), desc, 0, 1),
               cu.cuGreenCtxStreamCreate(ref(stream), ctx, 1, 0)):
        if rc:
            pytest.skip("green contexts: the driver answered %d" % rc)
    assert part.sm_count < whole.sm_count
    yield stream.value
    cu.cuStreamDestroy_v2(stream)
    cu.cuGreenCtxDestroy(ctx)


def test_few_token_layer_with_part_of_the_device(narrow_stream):
    """Where the blocks that wait for one another could not all run, the call takes the other path."""
    M, K, I, E, topK = 9, 512, 128, 4, 2
    x, ei, probs, w1, v1, w2, v2 = layer_case(M, K, I, E, topK, 12)
    x = (x * np.float16(2.0 ** -6)).astype(np.float16)
    y, err = routes64(mx.values(*mx.quantise(x.astype(np.float64))), ei, v1, v2)
    ref, bound = weighted(y, err, probs)
    d, dx, de, dp = moe.dims(M, K, I, E, topK), dev(x), dev(ei), dev(probs)
    ws = empty(moe.moe_mxfp4_layer_workspace_size(d), torch.uint8)
    out = torch.full((M, K), float("nan"), dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    moe.moe_mxfp4_layer_fwd(d, dx, de, dp, w1, w2, out, ws, stream=narrow_stream)
    torch.cuda.synchronize()
    assert moe.moe_workspace_status(ws) == 0
    over = np.abs(ref) + bound > 65504
    assert over.mean() < 0.5
    assert (np.abs(host(out).astype(np.float64) - ref) <= bound)[~over].all()


@pytest.mark.parametrize("M,K,I,E,topK", [(1, 2048, 1024, 16, 8), (8, 1024, 1024, 16, 4), (32, 512, 704, 8, 4)])
def test_h_is_that_of_the_call(M, K, I, E, topK):
    """The down product's rows come from other blocks of the kernel, through the workspace: with other
    tokens and routes in every call, a row read before its block had written it is that of a call before."""
    rng = np.random.default_rng(M + I)
    w1, _ = make_weights(rng, E, 2 * I, K, True)
    w2, _ = make_weights(rng, E, K, I, False)
    d = moe.dims(M, K, I, E, topK)
    ws = empty(moe.moe_mxfp4_layer_workspace_size(d), torch.uint8)
    sets = [layer_inputs(rng, M, K, E, topK) for _ in range(16)]

    def layer(x, ei, probs, workspace):
        out = empty((M, K), torch.float16)
        moe.moe_mxfp4_layer_fwd(d, x, ei, probs, w1, w2, out, workspace)
        return out

    alone = []
    for s in sets:
        alone.append(layer(*s, torch.full_like(ws, 0xEE)))
        torch.cuda.synchronize()
    for _ in range(10):
        outs = [layer(*s, ws) for s in sets]
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))
    assert moe.moe_workspace_status(ws) == 0
