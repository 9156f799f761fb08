"""One expert a token (k = 1) on each path of the layer, forward and backward, against the dense oracle."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_amd.inputs import Workload
from oracle import ffn as offn
from tests.conftest import rel_l2
from tests.gpu_util import Case, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,w", [
    ("tiles_f32", Workload("tiles_f32", "f32", "f32", T=150, k=1, E=6, d=256, d_ff=128, beta=16, P=2, s=1, kappas=(0,), cfg_id=31)),
    ("tiles_bf16", Workload("tiles_bf16", "bf16", "bf16", T=300, k=1, E=4, d=256, d_ff=192, beta=32, P=2, s=1, kappas=(0,), cfg_id=32)),
    ("stream_bf16", Workload("stream_bf16", "bf16", "bf16", T=700, k=1, E=4, d=512, d_ff=256, beta=128, P=4, s=2, kappas=(0,), cfg_id=33))])
def test_top1(name, w):
    say(f"[top1] {name}")
    c = Case(w, 0, backward=True)
    r = c.runner
    r.step(c.x, c.gates, c.ids, dy=c.dy)
    torch.cuda.synchronize()
    assert c.status() == 0
    x, w1, w2, ids, gates = c.oracle_inputs()
    tol = 1e-5 if w.act == "f32" else 2e-2                 # the bars of the layer's other tests
    assert rel_l2(r.y.double().cpu().numpy(), offn.forward(x, w1, w2, ids, gates)) <= tol
    bw = offn.backward(x, w1, w2, ids, gates, c.dy.double().cpu().numpy())
    assert rel_l2(r.dx.double().cpu().numpy(), bw["dx"]) <= tol
    for got, ref in ((r.dw1, bw["dw1"]), (r.dw2, bw["dw2"])):
        assert rel_l2(got.double().cpu().numpy(), np.stack([ref[e] for e in range(w.E)])) <= tol
