"""BlockRunner.update_bias takes the counts of a routing, not of none."""
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from tests.test_gpu_block import PATHS, _block

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_no_bias_step_before_a_routing():
    """The counts that it takes are those of a block_forward."""
    w = PATHS["stream_bf16"]
    bias = torch.zeros(w.E, device=DEV)
    b, par, x, dout = _block(w, w.T, 5, "sigmoid", True, bias=bias)
    with pytest.raises(B.MoeError, match="block_forward"):
        b.update_bias(0.01)
    torch.cuda.synchronize()
    assert (bias == 0).all()
    b.block_forward(x)
    b.update_bias(0.01)
    torch.cuda.synchronize()
    assert (bias != 0).any()
