"""The operators around the layer as a training step runs them: gate gradients out of the layer's
backward on each of its paths, and the whole block (norm -> router -> layer -> norm, its gradients,
AdamW) against the chained fp64 oracles."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from moe_expert_ffn_amd.inputs import WORKLOADS, Workload, contiguous_owners
from moe_expert_ffn_amd.runner import BlockRunner
from oracle import adamw as oadam
from oracle import ffn as offn
from oracle import norm as onorm
from oracle import router as orouter
from tests.conftest import rel_l2
from tests.gpu_util import Case, say

pytestmark = pytest.mark.gpu
DEV = "cuda"

PATHS = {
    "small_f32": Workload("small_f32", "f32", "f32", T=150, k=3, E=6, d=256, d_ff=128, beta=16, P=2,
                          s=1, kappas=(0,), cfg_id=23),
    "small_bf16": Workload("small_bf16", "bf16", "bf16", T=300, k=4, E=16, d=256, d_ff=192, beta=128,
                           P=4, s=2, kappas=(0,), cfg_id=21),
    "stream_bf16": Workload("stream_bf16", "bf16", "bf16", T=700, k=4, E=8, d=512, d_ff=256, beta=128,
                            P=8, s=4, kappas=(0,), cfg_id=24),
    "small_fp8": Workload("small_fp8", "bf16", "fp8", T=0, k=4, E=8, d=256, d_ff=128, beta=64, P=4, s=2,
                          kappas=(1,), rows=500, cfg_id=41),
    "stream_fp8": Workload("stream_fp8", "bf16", "fp8", T=0, k=4, E=8, d=512, d_ff=256, beta=128, P=4,
                           s=2, kappas=(1,), rows=900, cfg_id=42),
}


def _dlogp_oracle(c):
    """p <dy, W2 (SiLU(G) U)> of every routed row, 0 elsewhere, fp64."""
    x, w1, w2, ids, gates = c.oracle_inputs()
    dy = c.dy.double().cpu().numpy()
    out = np.zeros(ids.shape)
    F = c.w.d_ff
    for t, j in zip(*np.nonzero(ids >= 0)):
        z = w1[ids[t, j]] @ x[t]
        out[t, j] = gates[t, j] * float(dy[t] @ (w2[ids[t, j]] @ (offn.silu(z[:F]) * z[F:])))
    return out


@pytest.mark.parametrize("name,mode", [(n, "plain") for n in PATHS] + [("stream_bf16", "two_phase"),
                                                                       ("stream_fp8", "two_phase"),
                                                                       ("stream_fp8", "fp8_act")])
def test_gate_gradients_of_the_layer(name, mode):
    w = PATHS[name]
    say(f"[gates] {name} {mode}")
    c = Case(w, w.kappas[0], backward=True)
    r = c.runner
    r.two_phase, r.fp8_act = mode == "two_phase", mode == "fp8_act"
    r.step(c.x, c.gates, c.ids, dy=c.dy)
    torch.cuda.synchronize()
    ref = [t.clone() for t in (r.dx, r.dw1, r.dw2)]
    dlogp = torch.full(c.ids.shape, 9.0, device=DEV)
    r.backward(c.x, c.gates, c.dy, c.ids, dlogp=dlogp)
    torch.cuda.synchronize()
    assert c.status() == 0
    for a, b in zip((r.dx, r.dw1, r.dw2), ref):                   # nothing else changes
        assert torch.equal(a, b)
    got = dlogp.double().cpu().numpy()
    assert (got[c.ids_np < 0] == 0).all()
    # the bars of the layer's other gradients; quantized activations add 2^-4 a value over two
    # products, averaged over a row's terms
    tol = 1e-5 if w.act == "f32" else {"fp8_act": 6e-2}.get(mode, 2e-2)
    err = rel_l2(got, _dlogp_oracle(c))
    say(f"  dlogp={err:.3e}")
    assert err <= tol


def test_a_gate_of_zero_has_a_gradient_of_zero_in_log_form():
    w = PATHS["stream_bf16"]
    c = Case(w, 0, backward=True)
    c.gates[5, 1] = 0.0
    c.gates[6, :] = 0.0
    r = c.runner
    r.step(c.x, c.gates, c.ids, dy=c.dy)
    dlogp = torch.full(c.ids.shape, 9.0, device=DEV)
    r.backward(c.x, c.gates, c.dy, c.ids, dlogp=dlogp)
    torch.cuda.synchronize()
    assert float(dlogp[5, 1]) == 0 and (dlogp[6] == 0).all() and not dlogp.isnan().any()


def _block(w, T, seed, score, renorm, gate=True, state=None, **kw):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = torch.float32 if w.act == "f32" else torch.bfloat16
    rnd = lambda *s, scale=1.0: torch.randn(s, generator=g, device=DEV) * scale
    par = {"w1": rnd(w.E, 2 * w.d_ff, w.d, scale=w.d ** -0.5).to(dt),
           "w2": rnd(w.E, w.d, w.d_ff, scale=w.d ** -0.5).to(dt),
           "w_router": rnd(w.E, w.d, scale=w.d ** -0.5).to(dt),
           "w_in": (1 + 0.1 * rnd(w.d)).to(dt), "w_out": (1 + 0.1 * rnd(w.d)).to(dt),
           "gate": 0.5 + 0.2 * rnd(w.d) if gate else None}
    owner = torch.from_numpy(contiguous_owners(w.E, w.P))
    b = BlockRunner(**par, act_dtype=dt, T=T, k=w.k, beta=w.beta, P=w.P, s=w.s, owner=owner,
                    with_backward=True, score=score, renorm=renorm, alpha=0.8, **kw)
    return b, par, rnd(T, w.d).to(dt), rnd(T, w.d, scale=1.0 / T).to(dt)


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _chain(b, par, x, dout, mask, dl, sigmoid, renorm):
    """The block in fp64 from the same inputs; the routing's choice is the kernels' (a logit next to
    another may go either way in lower precision), checked on its own."""
    X, D = _f64(x), _f64(dout)
    P = {k: _f64(v) for k, v in par.items()}
    eps, a = 1e-6, float(np.float32(b.alpha))
    ids = b.routed["topk_ids"].cpu().numpy()
    _, n, s_in = onorm.norm_in(X, P["w_in"], eps)
    logits = n @ P["w_router"].T
    f = orouter.forward(logits, b.k, sigmoid, renorm, mask=mask)
    E = b.E
    gates = np.zeros(ids.shape)
    s = -np.logaddexp(0, -logits) if sigmoid else logits
    for t, j in zip(*np.nonzero(ids >= 0)):
        den = s[t][ids[t]] if renorm else s[t]
        lse = np.log(np.exp(den - den.max()).sum()) + den.max()
        gates[t, j] = np.exp(s[t, ids[t, j]] - (0 if sigmoid and not renorm else lse))
    y = offn.forward(n, P["w1"], P["w2"], ids, gates)
    out, s_out = onorm.norm_out(y, X, P["w_out"], eps, P["gate"], a)
    dy, dw_out, dgate = onorm.norm_out_backward(D, y, P["w_out"], s_out, P["gate"], a)
    bw = offn.backward(n, P["w1"], P["w2"], ids, gates, dy)
    dlogp = np.zeros(ids.shape)
    F = P["w2"].shape[2]
    for t, j in zip(*np.nonzero(ids >= 0)):
        e = ids[t, j]
        z = P["w1"][e] @ n[t]
        dlogp[t, j] = gates[t, j] * float(dy[t] @ (P["w2"][e] @ (offn.silu(z[:F]) * z[F:])))
    counts = np.bincount(ids[ids >= 0], minlength=E)
    live = int((ids >= 0).any(1).sum())
    dlogits = orouter.backward(logits, ids, dlogp, counts, live, *dl, sigmoid, renorm, mask)
    dn = bw["dx"] + dlogits @ P["w_router"]
    dx, dw_in, _, _ = onorm.norm_in_backward(dn, X, P["w_in"], s_in, D)
    stack = lambda k: np.stack([bw[k][e] for e in range(E)])
    return {"out": out, "losses": f["losses"], "dx_block": dx, "dw1": stack("dw1"), "dw2": stack("dw2"),
            "dw_router": dlogits.T @ n, "dw_in": dw_in, "dw_out": dw_out, "dgate": dgate}, logits


@pytest.mark.parametrize("name,score,renorm,masked", [
    ("small_f32", "softmax", True, False), ("small_f32", "sigmoid", True, True),
    ("small_f32", "softmax", False, True), ("small_f32", "sigmoid", False, False),
    ("small_bf16", "softmax", True, True), ("stream_bf16", "sigmoid", True, False)])
def test_block_forward_and_backward(name, score, renorm, masked):
    w = PATHS[name]
    say(f"[block] {name} {score} renorm={renorm} masked={masked}")
    b, par, x, dout = _block(w, w.T, 11, score, renorm)
    mask = None
    if masked:
        mask = torch.ones(w.T, dtype=torch.uint8, device=DEV)
        mask[::7] = 0
    dl = torch.tensor([0.02, 0.01], device=DEV)
    out = b.block_forward(x, mask)
    b.block_backward(dout, dl)
    torch.cuda.synchronize()
    assert int(b.status.item()) == 0
    m = None if mask is None else mask.cpu().numpy()
    ref, logits = _chain(b, par, x, dout, m, dl.double().tolist(), score == "sigmoid", renorm)
    if mask is not None:                                          # padding: the residual alone
        assert torch.equal(out[::7], x[::7]) and (b.routed["topk_ids"][::7] == -1).all()
    # every choice is within the logits' error of the k-th largest: half a bf16 step of |l| and of
    # its d products' rounding, or 32-bit sums of d terms
    ids = b.routed["topk_ids"].cpu().numpy()
    kth = np.sort(logits, 1)[:, -b.k]
    eps = 1e-5 if w.act == "f32" else 2.0 ** -6
    for t in range(w.T):
        if ids[t, 0] >= 0:
            assert (logits[t, ids[t]] >= kth[t] - eps * (1 + np.abs(kth[t]))).all()
    # the layer's own bars: 1e-5 in fp32 and 2e-2 in bf16, the router's and the first norm's
    # gradients pass two more bf16 tensors (dlogits, dn): 3e-2
    tol = 1e-5 if w.act == "f32" else 2e-2
    for key, val in ref.items():
        got = b.routed["losses"] if key == "losses" else getattr(b, key)
        err = rel_l2(_f64(got), val)
        say(f"  {key}={err:.2e}")
        assert err <= (tol if w.act == "f32" or key not in ("dw_router", "dx_block", "dw_in") else 3e-2), key


@pytest.mark.parametrize("name", ["small_f32", "small_bf16", "stream_bf16"])
def test_block_padding_holds_anything(name):
    """Padding rows of NaN: every weight's gradient, the losses and the other rows stay bit for bit."""
    w = PATHS[name]
    say(f"[block-padding] {name}")
    dl = torch.tensor([0.02, 0.01], device=DEV)
    mask = torch.ones(w.T, dtype=torch.bool, device=DEV)
    mask[::7] = False
    keys = ("out", "dx_block", "dw1", "dw2", "dw_router", "dw_in", "dw_out", "dgate")
    res = []
    for pad in (False, True):
        b, par, x, dout = _block(w, w.T, 11, "softmax", True)
        dout[~mask] = 0
        if pad:
            x[~mask] = float("nan")
        b.block_forward(x, mask)
        b.block_backward(dout, dl)
        torch.cuda.synchronize()
        assert int(b.status.item()) == 0
        res.append({k: getattr(b, k).clone() for k in keys} | {"losses": b.routed["losses"].clone()})
    clean, padded = res
    assert padded["out"][~mask].isnan().all() and not padded["dx_block"][~mask].any()
    for k in ("out", "dx_block"):
        assert torch.equal(padded[k][mask], clean[k][mask]), k
    for k in ("dw1", "dw2", "dw_router", "dw_in", "dw_out", "dgate", "losses"):
        assert torch.equal(padded[k], clean[k]), k


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("name", ["small_f32", "stream_bf16"])
def test_block_trains_and_its_step_replays(name, bits):
    """Three whole steps eager, then the same three as replays of a captured step, from the same
    start: weights and states bit for bit."""
    w = PATHS[name]
    say(f"[block-train] {name} bits={bits}")
    dl = torch.tensor([0.02, 0.01], device=DEV)
    hyper = dict(beta1=0.9, beta2=0.99, weight_decay=0.01, seed=3)

    def start():
        b, par, x, dout = _block(w, w.T, 12, "softmax", True)
        b.make_optimizer(bits)
        b.step_no = torch.ones(1, dtype=torch.int32, device=DEV)
        return b, par, x, dout

    def one(b, x, dout):
        b.block_forward(x)
        b.block_backward(dout, dl)
        b.optimizer_step(1e-3, b.step_no, **hyper)

    def everything(b, par):
        torch.cuda.synchronize()
        s = b.state
        ts = list(par.values()) + s["m"] + s["v"] + (s["m_scale"] or []) + (s["v_scale"] or [])
        return [t.clone() for t in ts]

    b, par, x, dout = start()
    first = everything(b, par)
    hist = []
    for t in range(1, 4):
        b.step_no.fill_(t)
        one(b, x, dout)
        hist.append(everything(b, par))
        if t == 1:                                                # the first step, against the oracle
            grads = [b.dw1, b.dw2, b.dw_router, b.dw_in, b.dw_out, b.dgate]
            for j, (p0, p1, g) in enumerate(zip(first, hist[0], grads)):
                G = _f64(g).reshape(-1)
                want, _, _ = oadam.step(_f64(p0).reshape(-1), G, 0 * G, 0 * G, 1, 1e-3, 0.9, 0.99, 1e-8, 0.01)
                got = _f64(p1).reshape(-1)
                half = 2.0 ** -7 if p1.dtype == torch.bfloat16 else 2.0 ** -20
                assert (np.abs(got - want) <= half * np.abs(want) + 1e-3 * 2.0 ** -18).all(), j
    assert int(b.status.item()) == 0
    assert not torch.equal(hist[0][0], hist[2][0])

    c, cpar, x, dout = start()
    one(c, x, dout)                                               # warm, then back to the start
    now = list(cpar.values()) + c.state["m"] + c.state["v"] + (c.state["m_scale"] or []) + \
        (c.state["v_scale"] or [])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(c, x, dout)
    for rep in range(2):
        for a, v in zip(now, first):
            a.copy_(v)
        for t in range(1, 4):
            c.step_no.fill_(t)
            graph.replay()
            torch.cuda.synchronize()
            for i, (a, v) in enumerate(zip(everything(c, cpar), hist[t - 1])):
                assert torch.equal(a, v), (rep, t, i)
        c.block_forward(x)                                        # eager work between the replays
    del graph


def test_forwards_in_a_row_leave_the_last_ones_gradients():
    """Forward passes without a backward between them (an evaluation), then a training step: the
    gradients are the last call's."""
    w = PATHS["stream_bf16"]
    say("[block-forwards]")
    b, par, x, dout = _block(w, w.T, 13, "softmax", True)
    b.block_forward(x)
    ref = [t.clone() for t in (b.block_backward(dout), b.dw1, b.dw_router)]
    other = torch.randn_like(x)
    for v in (other, x, other, other, x):
        b.block_forward(v)
    b.block_backward(dout)
    torch.cuda.synchronize()
    assert int(b.status.item()) == 0
    for a, c in zip((b.dx_block, b.dw1, b.dw_router), ref):
        assert torch.equal(a, c)


def test_block_refusals():
    w = PATHS["small_f32"]
    b, par, x, dout = _block(w, w.T, 1, "softmax", True)
    with pytest.raises(B.MoeError, match="make_optimizer"):
        b.optimizer_step(1e-3, 1)
    with pytest.raises(B.MoeError, match="8 or 32"):
        b.make_optimizer(16)
    with pytest.raises(B.MoeError, match="w_router"):
        BlockRunner(par["w1"], par["w2"], par["w_router"][:, :-1], par["w_in"], par["w_out"],
                    act_dtype=torch.float32, T=w.T, k=w.k, beta=w.beta, P=w.P, s=w.s,
                    owner=torch.from_numpy(contiguous_owners(w.E, w.P)))


def test_block_backward_needs_its_forward():
    w = PATHS["small_f32"]
    b, par, x, dout = _block(w, w.T, 1, "softmax", True)
    with pytest.raises(B.MoeError, match="block_forward"):
        b.block_backward(dout)
    only = BlockRunner(**par, act_dtype=torch.float32, T=w.T, k=w.k, beta=w.beta, P=w.P, s=w.s,
                       owner=torch.from_numpy(contiguous_owners(w.E, w.P)))
    only.block_forward(x)
    with pytest.raises(B.MoeError, match="block_forward"):
        only.block_backward(dout)
