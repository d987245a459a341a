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
