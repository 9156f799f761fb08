"""GPU: one router workspace, made for the largest batch, serves every smaller one."""
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("E,most", [(160, 8192), (256, 8192), (512, 4096)])
def test_workspace_of_the_largest_batch(E, most):
    """Around the number of rows where the forward pass puts 16 experts into a lane: the same bits as with a
    workspace of the batch's own size."""
    say(f"[router-workspace] E={E} most={most}")
    R = B.make_router(E, 4)
    ws = B.router_workspace(R, most, DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(E)
    for T in (most, most - 1, most - 192, most // 2 + 1, 33, 1, 0, most):
        logits = torch.randn((T, E), generator=g, device=DEV)
        own, one = (B.router_forward(R, logits, B.alloc_router(R, T, DEV), w, status)
                    for w in (B.router_workspace(R, T, DEV), ws))
        torch.cuda.synchronize()
        for k in own:
            assert torch.equal(own[k], one[k]), (T, k)
    assert int(status.item()) == 0
