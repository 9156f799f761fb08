"""The scale of a list's gradients lies in none of them: it would be scaled while other workgroups read it."""
import pytest
import torch

from moe_expert_ffn_amd import binding as B

FULL = torch.zeros(4096)                       # one allocation, so that places next to each other are known


def _list():
    grads = [FULL[100:200], FULL[0:0], FULL[300:1300].view(10, 100), FULL[500:600], FULL[1400:1401]]
    ws = FULL[2048:2560].view(torch.uint8)
    return B.PreparedGrads(B.GradList(ws.data_ptr(), len(grads), 4, 0), ws, grads)


INSIDE = [100, 150, 199, 300, 500, 599, 600, 1299, 1400, 2048, 2559]
OUTSIDE = [0, 99, 200, 299, 1300, 1399, 1401, 2047, 2560, 4095]


@pytest.mark.parametrize("at", INSIDE)
def test_inside(at):
    p, one = _list(), FULL[at:at + 1]
    with pytest.raises(B.MoeError, match="scale: lies in"):
        B.grad_scale(p, one)


@pytest.mark.parametrize("at", OUTSIDE)
def test_beside(at):
    """Up to the device, which the next check asks for."""
    p, one = _list(), FULL[at:at + 1]
    with pytest.raises(B.MoeError, match="current device"):
        B.grad_scale(p, one)


def test_two_bytes_of_a_gradient():
    """A gradient that ends inside the scale's four bytes."""
    half = FULL.view(torch.bfloat16)
    p = B.PreparedGrads(B.GradList(4096, 1, 1, 1), torch.zeros(256, dtype=torch.uint8), [half[0:2001]])
    with pytest.raises(B.MoeError, match="lies in"):
        B.grad_scale(p, FULL[1000:1001])
    with pytest.raises(B.MoeError, match="current device"):
        B.grad_scale(p, FULL[1001:1002])


def test_a_list_of_nothing():
    p = B.PreparedGrads(B.GradList(4096, 0, 0, 1), torch.zeros(256, dtype=torch.uint8), [])
    with pytest.raises(B.MoeError, match="current device"):
        B.grad_scale(p, FULL[5:6])
