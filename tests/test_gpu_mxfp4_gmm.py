"""The grouped MXFP4 product's hand-overs between its warps and CTAs, and the expert sizes at which
it goes from one tile and one kernel to the next."""
import numpy as np
import pytest

import mx_reference as mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_expert_layer_gb300 as moe
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
