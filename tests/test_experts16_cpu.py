"""Without a GPU: sizes and refusals of the 16-bit experts' entry points, and the binding's checks."""
import pytest

A, U = 4096, 4096 + 8  # aligned to 256 bytes; to 8 only
F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def moe():
    from moe_expert_layer_gb300 import build
    build.build()
    import moe_expert_layer_gb300
    moe_expert_layer_gb300.load_library()
    return moe_expert_layer_gb300


@pytest.fixture(scope="module")
def lib(moe):
    return moe.load_library()


def each_pointer(call, n, optional=()):
    """Every pointer missing is MOE_ERR_NULL (unless optional), every one misaligned MOE_ERR_ALIGN."""
    for i in range(n):
        p = [A] * n
        p[i] = None
        if i not in optional:
            assert call(p) == -1, i
        p[i] = U
        assert call(p) == -3, i


BAD_SIZES = [(0, 4, 64, 64), (1 << 24, 4, 64, 64), (8, 0, 64, 64), (8, 1024, 64, 64), (8, 4, 0, 64), (8, 4, 12, 64), (8, 4, 65544, 64),
             (8, 4, 64, 0), (8, 4, 64, 100), (8, 4, 64, 65544)]


def test_sizes(moe):
    assert moe.moe_gmm16_workspace_size(8, 4, 64, 64) > 0 and moe.moe_gmm16_workspace_size(1, 1, 65536, 65536) > 0
    for bad in BAD_SIZES:
        assert moe.moe_gmm16_workspace_size(*bad) == 0
    for bad in ((0, 64, 64, 16), (8, 60, 64, 16), (8, 64, 4, 16), (8, 64, 64, 0), (8, 64, 64, 12), (8, 64, 64, 136)):
        assert moe.moe_lora16_workspace_size(*bad) == 0


@pytest.mark.parametrize("N,D,rank", [(8, 8, 8), (4096, 4096, 16), (65536, 65536, 128), (4096, 7168, 64), (72, 65536, 24)])
def test_adapter_workspace_never_shrinks(moe, N, D, rank):
    """A workspace made for the largest batch serves every smaller one."""
    sizes = [moe.moe_lora16_workspace_size(m, N, D, rank) for m in [*range(1, 700), 1024, 5000, 65536, 1 << 20]]
    assert min(sizes) > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_product_refusals(lib, moe):
    ws = moe.moe_gmm16_workspace_size(8, 4, 64, 128)
    for f in (lib.moe_gmm16, lib.moe_gmm16_input_grad):
        for bad in BAD_SIZES:
            assert f(*bad, F16, *[A] * 5, ws, None) == -2
        for t in (F32, 3, -1):
            assert f(8, 4, 64, 128, t, *[A] * 5, ws, None) == -2
        each_pointer(lambda p: f(8, 4, 64, 128, BF16, *p, ws, None), 5)
        assert f(8, 4, 64, 128, F16, *[A] * 4, A + 16, ws, None) == -3
        assert f(8, 4, 64, 128, F16, *[A] * 5, ws - 1, None) == -5

    def grad(p=(A,) * 5, sizes=(8, 4, 64, 128), t=F16, out=F16, acc=0, n=ws):
        return lib.moe_gmm16_weight_grad(*sizes, t, *p[:4], out, acc, p[4], n, None)
    for bad in BAD_SIZES:
        assert grad(sizes=bad) == -2
    for bad in (dict(t=F32), dict(out=BF16), dict(out=5), dict(acc=1), dict(t=F32, out=F32)):
        assert grad(**bad) == -2, bad
    each_pointer(lambda p: grad(p), 5)
    assert grad(n=ws - 1) == -5


def test_row_operator_refusals(lib):
    for I in (0, 4, 12, 32776):
        assert lib.moe_swiglu16(8, 4, I, F16, A, A, A, None) == -2
        assert lib.moe_swiglu16_grad(8, 4, I, F16, A, A, A, A, A, None) == -2
    for R, E, t in ((0, 4, F16), (1 << 24, 4, F16), (8, 0, F16), (8, 1024, F16), (8, 4, F32), (8, 4, 7)):
        assert lib.moe_swiglu16(R, E, 64, t, A, A, A, None) == -2
        assert lib.moe_swiglu16_grad(R, E, 64, t, A, A, A, A, A, None) == -2
    each_pointer(lambda p: lib.moe_swiglu16(8, 4, 64, F16, *p, None), 3)
    each_pointer(lambda p: lib.moe_swiglu16_grad(8, 4, 64, F16, *p, None), 5, optional=(4,))
    for f, n, optional in ((lib.moe_dispatch16, 3, ()), (lib.moe_combine16, 4, (2,)), (lib.moe_combine16_grad, 6, ())):
        for bad in ((0, 64, 2, 8, F16), (8, 60, 2, 8, F16), (8, 65544, 2, 8, F16), (8, 64, 0, 8, F16), (8, 64, 2, 0, F16),
                    (8, 64, 2, 1 << 24, F16), (1 << 23, 64, 2, 8, F16), (8, 64, 2, 8, F32), (8, 64, 2, 8, 9)):
            assert f(*bad, *[A] * n, None) == -2, bad
        each_pointer(lambda p: f(8, 64, 2, 8, BF16, *p, None), n, optional)


def test_adapter_refusals(lib, moe):
    ws = moe.moe_lora16_workspace_size(8, 64, 128, 16)

    def call(p=(A,) * 9, M=8, N=64, D=128, r=16, L=4, t=F16, n=ws):
        return lib.moe_lora16(M, N, D, r, L, t, *p, n, None)
    for bad in (dict(M=0), dict(M=1 << 24), dict(N=60), dict(N=0), dict(D=4), dict(D=65544), dict(r=0), dict(r=12), dict(r=136),
                dict(L=0), dict(L=1024), dict(t=F32), dict(t=4)):
        assert call(**bad) == -2, bad
    each_pointer(lambda p: call(p), 9, optional=(5,))
    assert call((A,) * 8 + (A + 16,)) == -3
    assert call(n=ws - 1) == -5


def arguments(moe):
    """Of every entry point: its tensors by name, all right but for being on the CPU."""
    import torch
    h = lambda *s: torch.zeros(s, dtype=torch.float16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    ws = torch.zeros(max(moe.moe_gmm16_workspace_size(6, 3, 64, 72), moe.moe_lora16_workspace_size(6, 64, 72, 8)), dtype=torch.uint8)
    return {
        "moe_gmm16": dict(a=h(6, 72), cumsum=i32(3), w=h(3, 64, 72), c=h(6, 64), workspace=ws),
        "moe_gmm16_input_grad": dict(dc=h(6, 64), cumsum=i32(3), w=h(3, 64, 72), da=h(6, 72), workspace=ws),
        "moe_gmm16_weight_grad": dict(dc=h(6, 64), a=h(6, 72), cumsum=i32(3), dw=h(3, 64, 72), workspace=ws),
        "moe_swiglu16": dict(gu=h(6, 128), cumsum=i32(3), h=h(6, 64)),
        "moe_swiglu16_grad": dict(dh=h(6, 64), gu=h(6, 128), cumsum=i32(3), dgu=h(6, 128), h=h(6, 64)),
        "moe_dispatch16": dict(x=h(6, 72), row_map=i32(6), out=h(4, 72)),
        "moe_combine16": dict(y=h(4, 72), row_map=i32(6), probs=torch.zeros(6), out=h(6, 72)),
        "moe_combine16_grad": dict(dout=h(6, 72), y=h(4, 72), row_map=i32(6), probs=torch.zeros(6), dy=h(4, 72), dprobs=torch.zeros(6)),
        "moe_lora16": dict(x=h(6, 72), route=i32(6), cumsum=i32(3), a=h(3, 8, 72), b=h(3, 64, 8), base=h(6, 64), out=h(6, 64),
                           workspace=ws, scales=torch.zeros(3)),
    }


def test_binding_refuses_other_types_shapes_and_strides(moe):
    """Every tensor of every call: of another type, with a row or column fewer, with rows that are not dense,
    or not on the GPU, it is refused before the library is called."""
    import torch
    for name, args in arguments(moe).items():
        f = getattr(moe, name)
        with pytest.raises(ValueError):  # all right, but in the host's memory
            f(**args, stream=0)
        for k, v in args.items():
            if k == "workspace":
                continue
            bads = [v.long() if v.dtype == torch.int32 else v.double(), v[..., :-1].contiguous(), v.repeat_interleave(2, -1)[..., ::2]]
            if v.dtype == torch.float16:
                bads.append(v.bfloat16())
            if v.dim() > 1 and k not in ("x", "out", "a", "dc", "dout", "gu", "y", "dh", "c"):
                bads.append(v[:-1])
            for bad in bads:
                with pytest.raises(ValueError):
                    f(**{**args, k: bad}, stream=0)
    args = arguments(moe)["moe_gmm16_weight_grad"]
    with pytest.raises(ValueError):
        moe.moe_gmm16_weight_grad(**{**args, "dw": args["dw"].to(torch.int16)}, stream=0)


PTXAS = """ptxas info    : Compiling entry function '_ZN3moe12gmm16_kernelILNS_5Gmm16E2ELi256ELb1ELNS_4SumsE%dEEEvi' for 'sm_103a'
ptxas info    : Function properties for _ZN3moe12gmm16_kernelILNS_5Gmm16E2ELi256ELb1ELNS_4SumsE%dEEEvi
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 1 barriers, 1024 bytes smem
"""


def test_build_refuses_other_launch_registers():
    """Kernels whose warps hand registers over are built with the registers that they count on, or not at all."""
    from moe_expert_layer_gb300 import build
    log = lambda *kernels: "".join(PTXAS % (i, i, n) for i, n in kernels)
    build.check_registers("gmm16.cu", log((1, 116), (2, 168), (0, 117), (3, 168)))
    for bad in (((1, 168), (2, 168), (0, 117), (3, 160)), ((2, 128), (3, 168)), ((2, 168),), ((0, 168), (1, 168)), ()):
        with pytest.raises(RuntimeError, match="gmm16.cu"):
            build.check_registers("gmm16.cu", log(*bad))


def test_binding_refuses_other_numbers_of_dimensions(moe):
    """Every matrix and stack of matrices of every call, flattened or with a dimension more: refused as other shapes are."""
    for name, args in arguments(moe).items():
        f = getattr(moe, name)
        for k, v in args.items():
            if v.dim() > 1:
                for bad in (v.reshape(-1), v[None]):
                    with pytest.raises(ValueError):
                        f(**{**args, k: bad}, stream=0)
