"""A choice belongs to routers of the experts that it was made for: its bias has one value for each."""
import pytest
import torch

from moe_expert_ffn_amd import binding as B


def _forward(R, C, T=4):
    x = torch.zeros(T, R.E)
    return B.router_forward(R, x, B.alloc_router(R, T, "cpu"), B.router_workspace(R, T, "cpu"),
                            torch.zeros(1, dtype=torch.int32), choice=C)


@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
@pytest.mark.parametrize("E", [64, 252])
def test_a_bias_of_fewer_experts_is_refused(E, groups, top):
    """It would be read past its end."""
    C = B.make_choice(B.make_router(E, 4), torch.zeros(E), groups, top)
    with pytest.raises(B.MoeError, match="bias"):
        _forward(B.make_router(256, 4), C)


def test_of_as_many_experts_it_serves():
    """Up to the device, which the next check asks for."""
    C = B.make_choice(B.make_router(256, 4), torch.zeros(256), 4, 2)
    with pytest.raises(B.MoeError, match="current device"):
        _forward(B.make_router(256, 8, score="sigmoid"), C)
    with pytest.raises(B.MoeError, match="current device"):
        _forward(B.make_router(256, 8), B.make_choice(B.make_router(64, 4), None, 4, 2))     # no bias: groups alone
