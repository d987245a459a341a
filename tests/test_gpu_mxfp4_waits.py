"""How the few-token MXFP4 layer's blocks wait for one another and for work: answers that have to
agree, and calls that share the device."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import moe_expert_layer_gb300 as moe


def test_epilogue_warps_give_up_together():
    """A unit that arrives after one warp has seen the block give up is taken by none of them."""
    for _ in range(20):
        answers = torch.full((4,), -7, dtype=torch.int32, device="cuda")
        moe.moe_selftest_mxfp4_tickets(answers)
        assert answers.tolist() == [0, 0, 0, 0]
