"""GPU: the whole block (norm -> router -> layer -> norm, gradients, AdamW) at a workload's own size, each step against
the fp64 oracle on the tensors that the step before it stored."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from moe_expert_ffn_amd.inputs import WORKLOADS, contiguous_owners, make_layer
from moe_expert_ffn_amd.runner import BlockRunner
from oracle import adamw as oadam
from oracle import ffn as offn
from oracle import norm as onorm
from oracle import router as orouter
from tests.conftest import rel_l2
from tests.gpu_util import LazyWeights, say

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("score,masked", [("softmax", False), ("sigmoid", True)])
def test_block_of_the_training_workload(score, masked):
    w = WORKLOADS["qwen3_bf16_fwdbwd"]
    say(f"[block-workload] {w.name} {score} masked={masked}")
    T, d, E, bf = w.T, w.d, w.E, torch.bfloat16
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    rnd = lambda *s, scale=1.0: torch.randn(s, generator=g, device=DEV) * scale
    lay = make_layer(w, DEV)
    par = {"w_router": rnd(E, d, scale=d ** -0.5).to(bf), "w_in": (1 + 0.1 * rnd(d)).to(bf),
           "w_out": (1 + 0.1 * rnd(d)).to(bf), "gate": 0.5 + 0.2 * rnd(d)}
    b = BlockRunner(lay["w1"], lay["w2"], **par, act_dtype=bf, T=T, k=w.k, beta=w.beta, P=w.P, s=w.s,
                    owner=torch.from_numpy(contiguous_owners(E, w.P)), with_backward=True, score=score, alpha=0.8)
    x, dout = rnd(T, d).to(bf), rnd(T, d, scale=1.0 / T).to(bf)
    mask = None
    if masked:
        mask = torch.ones(T, dtype=torch.bool, device=DEV)
        mask[::9] = False
        x[~mask] = float("nan")
        dout[~mask] = 0
    dl = torch.tensor([0.02, 0.01], device=DEV)
    out = b.block_forward(x, mask)
    dx = b.block_backward(dout, dl)
    torch.cuda.synchronize()
    assert int(b.status.item()) == 0

    on = np.ones(T, bool) if mask is None else mask.cpu().numpy()
    X = np.where(on[:, None], _f64(x), 0.0)
    D, N, Y, L = _f64(dout), _f64(b.n), _f64(b.y), _f64(b.logits)
    ids, gates = b.routed["topk_ids"].cpu().numpy(), _f64(b.routed["gates"])
    P = {k: _f64(v) for k, v in par.items()}
    w1, w2 = LazyWeights(lay["w1"]), LazyWeights(lay["w2"])
    a = float(np.float32(0.8))
    some = np.flatnonzero(on)[np.linspace(0, on.sum() - 1, 24).astype(int)]
    errs = {}

    def near(name, got, want, tol):
        errs[name] = rel_l2(got, want)
        assert errs[name] <= tol, errs

    # a bf16 output of a 32-bit computation is off by half a step, 2^-8 of each value at most; the layer's products,
    # whose inner rows are bf16 too, by the bar of their own tests, 2e-2
    half = 2.0 ** -8
    _, n, s_in = onorm.norm_in(X, P["w_in"], 1e-6)
    near("n", N[on], n[on], half)
    near("logits", L[on], N[on] @ P["w_router"].T, half)
    f = orouter.forward(L, w.k, score == "sigmoid", True, mask=on)
    assert (ids == f["topk_ids"]).all() and (b.routed["counts"].cpu().numpy() == f["counts"]).all()
    assert int(b.routed["live"].item()) == f["live"] == on.sum()
    near("gates", gates, f["gates"], 1e-5)
    near("losses", _f64(b.routed["losses"]), f["losses"], 1e-5)
    near("y", Y[some], offn.forward(N, w1, w2, ids, gates, tokens=some), 2e-2)
    o, s_out = onorm.norm_out(Y, X, P["w_out"], 1e-6, P["gate"], a)
    near("out", _f64(out)[on], o[on], half)
    dy, dw_out, dgate = onorm.norm_out_backward(D[on], Y[on], P["w_out"], s_out[on], P["gate"], a)
    DY = _f64(b.dy)
    near("dy", DY[on], dy, half)
    near("dw_out", _f64(b.dw_out), dw_out, 1e-5)
    near("dgate", _f64(b.dgate), dgate, 1e-5)
    few = [int(np.argmax(f["counts"])), int(np.argmin(f["counts"]))]
    bw = offn.backward(N, w1, w2, ids, gates, DY, tokens=some, experts=few)
    near("dx of the layer", _f64(b.dx)[some], bw["dx"], 2e-2)
    for e in few:
        near(f"dw1[{e}]", _f64(b.dw1[e]), bw["dw1"][e], 2e-2)
        near(f"dw2[{e}]", _f64(b.dw2[e]), bw["dw2"][e], 2e-2)
    h = np.zeros((some.size, w.k))
    for i, t in enumerate(some):
        for j, e in enumerate(ids[t]):
            z = w1[e] @ N[t]
            h[i, j] = gates[t, j] * float(DY[t] @ (w2[e] @ (offn.silu(z[:w.d_ff]) * z[w.d_ff:])))
    H = _f64(b.dlogp)
    near("dlogp", H[some], h, 2e-2)
    assert (H[~on] == 0).all()
    G = _f64(b.dlogits)
    dlogits = orouter.backward(L[some], ids[some], H[some], f["counts"], f["live"], *dl.double().tolist(),
                               score == "sigmoid", True)
    near("dlogits", G[some], dlogits, half)
    assert (G[~on] == 0).all()
    near("dw_router", _f64(b.dw_router), G.T @ N, half)
    DN = _f64(b.dn)
    near("dn", DN[on], (_f64(b.dx) + G @ P["w_router"])[on], half)
    want, dw_in, _, _ = onorm.norm_in_backward(DN[on], X[on], P["w_in"], s_in[on], D[on])
    near("dx", _f64(dx)[on], want, half)
    near("dw_in", _f64(b.dw_in), dw_in, 1e-5)
    say("  " + " ".join(f"{k}={v:.1e}" for k, v in errs.items()))
    if masked:
        assert (N[~on] == 0).all() and (DY[~on] == 0).all() and (_f64(dx)[~on] == 0).all()
        assert out[~mask].isnan().all()

    # one step with 8-bit states, of one expert, the router and the gate; bf16 weights to a neighbour, 2^-7 of the value
    b.make_optimizer(8)
    before = [t[:, :7].clone() if t.dim() > 1 else t.clone() for t in (lay["w1"][few[0]], par["w_router"], par["gate"])]
    grads = [b.dw1[few[0]], b.dw_router, b.dgate]
    b.optimizer_step(1e-3, 1, weight_decay=0.0)
    torch.cuda.synchronize()
    for old, new, gr in zip(before, (lay["w1"][few[0]], par["w_router"], par["gate"]), grads):
        cut = (lambda t: t[:, :7]) if new.dim() > 1 else (lambda t: t)
        q = _f64(cut(gr))
        p, _, _ = oadam.step(_f64(old), q, 0 * q, 0 * q, 1, 1e-3, 0.9, 0.999, 1e-8, 0.0)
        step = 2.0 ** -7 * np.abs(p) if new.dtype == bf else 2.0 ** -20 * np.abs(p)
        assert (np.abs(_f64(cut(new)) - p) <= step + 1e-3 * 2.0 ** -18).all()
