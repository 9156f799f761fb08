"""BlockRunner.optimizer_step's grad_scale as a number, as its documentation has it."""
import math

import pytest
import torch

from moe_expert_ffn_amd import binding as B
from tests.test_gpu_block import PATHS, _block

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _stepped(**kw):
    b, par, x, dout = _block(PATHS["small_f32"], 150, 3, "softmax", True)
    b.block_forward(x)
    b.block_backward(dout)
    b.make_optimizer()
    b.optimizer_step(1e-3, 1, **kw)
    torch.cuda.synchronize()
    return [t.clone() for t in (*par.values(), *b.state["m"], *b.state["v"])]


@pytest.mark.parametrize("number", [0.5, 1, 0.0, -2.0])
def test_a_number_is_the_tensor_of_it(number):
    want = _stepped(grad_scale=torch.tensor([float(number)], device=DEV))
    assert all(torch.equal(a, b) for a, b in zip(_stepped(grad_scale=number), want))


@pytest.mark.parametrize("max_norm", [None, 1.0])
def test_numbers_that_are_refused(max_norm):
    for bad in (math.nan, math.inf, -math.inf) + ((1e39, -1e39) if max_norm is None else ()):
        with pytest.raises(B.MoeError):
            _stepped(grad_scale=bad, max_norm=max_norm)
