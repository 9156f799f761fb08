"""GPU: what a BlockRunner may be given of its own buffers."""
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from moe_expert_ffn_amd.inputs import Workload, contiguous_owners
from moe_expert_ffn_amd.runner import BlockRunner
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
W = Workload("small_f32", "f32", "f32", T=150, k=3, E=6, d=256, d_ff=128, beta=16, P=2, s=1, kappas=(0,), cfg_id=23)


def _block(**kw):
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    rnd = lambda *s, scale=1.0: torch.randn(s, generator=g, device=DEV) * scale
    par = dict(w1=rnd(W.E, 2 * W.d_ff, W.d, scale=W.d ** -0.5), w2=rnd(W.E, W.d, W.d_ff, scale=W.d ** -0.5),
               w_router=rnd(W.E, W.d, scale=W.d ** -0.5), w_in=1 + 0.1 * rnd(W.d), w_out=1 + 0.1 * rnd(W.d))
    owner = torch.from_numpy(contiguous_owners(W.E, W.P))
    b = BlockRunner(**par, act_dtype=torch.float32, T=kw.pop("T", W.T), k=W.k, beta=W.beta, P=W.P, s=W.s, owner=owner,
                    with_backward=True, **kw)
    return b, rnd(W.T, W.d), rnd(W.T, W.d)


def test_a_forward_of_its_own_output_has_no_backward():
    """Two forwards in a row through the same runner: the outputs are those of a copy, and the backward pass, whose
    x the second call has overwritten, is refused instead of computed from it."""
    say("[block-buffers] out")
    b, x, dout = _block()
    copy = b.block_forward(x).clone()
    want = b.block_forward(copy).clone()
    ref = b.block_backward(dout).clone()
    out = b.block_forward(x)
    assert torch.equal(b.block_forward(out), want)
    for view in (out, out[:]):
        b.block_forward(view)
        with pytest.raises(B.MoeError, match="block_forward of an x"):
            b.block_backward(dout)
    b.block_forward(copy)
    assert torch.equal(b.block_backward(dout), ref)


def test_buffers_that_a_call_overwrites_are_refused():
    say("[block-buffers] refused")
    b, x, dout = _block()
    b.block_forward(x)
    ref = b.block_backward(dout).clone()
    for name in ("n", "y", "dy", "dn", "dx", "dx_block"):
        with pytest.raises(B.MoeError, match="overwrites"):
            b.block_forward(getattr(b, name))
    b.block_forward(x)
    for name in ("dy", "dn", "dx"):
        with pytest.raises(B.MoeError, match="overwrites"):
            b.block_backward(getattr(b, name))
    b.dx_block.copy_(dout)                              # in place: dx over the dout that it adds
    assert torch.equal(b.block_backward(b.dx_block), ref)


def test_block_takes_a_gate_of_features_only():
    """A gate per token went through where T <= d, into a gradient of d numbers."""
    say("[block-buffers] gate")
    one = lambda *n: torch.ones(n, device=DEV)
    for gate in (one(W.T, 1), one(1, W.d), one(W.d - 1), one()):
        with pytest.raises(B.MoeError, match="gate: expected"):
            _block(gate=gate)
    b, x, dout = _block(gate=one(W.d))
    b.block_forward(x)
    b.block_backward(dout)
    torch.cuda.synchronize()
    assert b.dgate.shape == (W.d,) and int(b.status.item()) == 0


def test_block_of_no_tokens():
    """Empty tensors share no memory, though all of them stand at address 0."""
    say("[block-buffers] empty")
    b, x, dout = _block(T=0)
    assert b.block_forward(x[:0]).shape == (0, W.d)
    assert b.block_backward(dout[:0]).shape == (0, W.d)
    assert b.block_forward(torch.empty((0, W.d), device=DEV)).shape == (0, W.d)
    assert b.block_backward(torch.empty((0, W.d), device=DEV)).shape == (0, W.d)
    torch.cuda.synchronize()
    assert int(b.status.item()) == 0
    for t in (b.dw1, b.dw2, b.dw_router, b.dw_in, b.dw_out):
        assert (t == 0).all()
