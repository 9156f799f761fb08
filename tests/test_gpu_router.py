"""GPU parity of the router, its losses, its gradient and the gate gradients against the fp64 oracle.

Ids, counts and live rows are exact.  Tolerances, u = 2^-24: an exponential of l - max is off by
u |l - max| (its argument's rounding) and 2 u (the function), a sum of E terms in a lane's order and
a tree by (V + log2 64) u <= 22 u, so a probability or gate of a row of spread r by (r + 2 + 22 + 4) u
relative; with sigmoid scores the logarithm adds 4 u (|l| + 1) to the argument.  A sum over tokens
adds T / 256 + 16 roundings.  `_rel` holds this, doubled."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from oracle import router as orouter
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -9 * 2}      # half a step: eps / 2


def _rel(l):
    fin = np.abs(l[np.isfinite(l)])
    spread = 2 * (fin.max() if fin.size else 1.0)
    return 2 * (spread * 5 + 40) * U


def _logits(rng, T, E, dtype, pad=0, offset=0):
    full = torch.from_numpy((rng.standard_normal((T, E + pad)) * 2).astype(np.float32)).to(dtype).to(DEV)
    return full[:, offset:offset + E]


def _forward(R, logits, mask=None):
    T = logits.shape[0]
    out, ws = B.alloc_router(R, T, DEV), B.router_workspace(R, T, DEV)
    for t in out.values():
        t.fill_(-7)
    ws.fill_(0xAB)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.router_forward(R, logits, out, ws, st, mask=mask)
    torch.cuda.synchronize()
    return out, int(st.item())


def _check_forward(logits, k, score, renorm, scale=1.0, mask=None, lim=None):
    T, E = logits.shape
    R = B.make_router(E, k, logits.dtype, score, renorm, scale)
    out, st = _forward(R, logits, mask)
    l = logits.double().cpu().numpy()
    o = orouter.forward(l, k, score == "sigmoid", renorm, scale,
                        None if mask is None else mask.cpu().numpy())
    assert st == (B.DEV_BAD_LOGIT if o["bad"] else 0)
    np.testing.assert_array_equal(out["topk_ids"].cpu().numpy(), o["topk_ids"])
    np.testing.assert_array_equal(out["counts"].cpu().numpy(), o["counts"])
    assert int(out["live"].item()) == o["live"]
    rel = _rel(l)
    np.testing.assert_allclose(out["gates"].cpu().numpy(), o["gates"], rtol=rel, atol=1e-37)
    more = 2 * (T / 256 + 16) * U
    np.testing.assert_allclose(out["prob_sum"].cpu().numpy(), o["prob_sum"], rtol=rel + more, atol=1e-37)
    # the losses: products of these sums; lse carries u |lse| and the sum's relative error
    np.testing.assert_allclose(out["losses"].cpu().numpy(), o["losses"], rtol=2 * (rel + more),
                               atol=4 * rel * (1 + np.abs(o["losses"][1])))
    return R, out, o


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (16, 128, 8), (17, 64, 8), (100, 65, 3), (257, 128, 1),
          (33, 200, 9), (300, 256, 8), (65, 257, 32), (40, 512, 10), (70, 513, 16), (31, 1024, 32),
          (5000, 8, 2), (4200, 63, 4)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_router_forward_and_backward(T, E, k, dtype, score, renorm):
    say(f"[router] T={T} E={E} k={k} {dtype} {score} renorm={renorm}")
    rng = np.random.default_rng(T * 1000 + E)
    logits = _logits(rng, T, E, dtype)
    logits[torch.rand(logits.shape, device=DEV) < 0.02] = float("-inf")
    R, out, o = _check_forward(logits, k, score, renorm, 1.0 if score == "softmax" else 2.5)
    h = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).to(DEV)
    dl = torch.tensor([0.8, 0.05], device=DEV)
    _check_backward(R, logits, out, o, h, dl, score, renorm)


@pytest.mark.parametrize("T,E,k,dtype,score", [(8200, 256, 8, torch.bfloat16, "sigmoid"),
                                               (4100, 400, 5, torch.float32, "softmax"),
                                               (8300, 157, 12, torch.float32, "sigmoid"),
                                               (5000, 512, 32, torch.bfloat16, "softmax")])
def test_router_of_many_rows(T, E, k, dtype, score):
    """Enough rows for the forward pass that puts 16 experts into a lane."""
    say(f"[router-many] T={T} E={E} k={k} {dtype} {score}")
    rng = np.random.default_rng(T)
    logits = _logits(rng, T, E, dtype, pad=3, offset=1)
    logits[torch.rand(logits.shape, device=DEV) < 0.02] = float("-inf")
    mask = torch.from_numpy((rng.random(T) < 0.9).astype(np.uint8)).to(DEV)
    R, out, o = _check_forward(logits, k, score, True, 1.0, mask)
    _check_backward(R, logits, out, o, torch.randn((T, k), device=DEV), torch.tensor([0.8, 0.05], device=DEV),
                    score, True, mask)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [8, 60, 256, 1000])
def test_router_sigmoid_tops(E, dtype, renorm):
    """Rows whose largest logit lies around the bound up to which a sigmoid is made from e^(l - top),
    far from it on both sides, and with the others far below it."""
    say(f"[router-tops] E={E} {dtype} renorm={renorm}")
    rng = np.random.default_rng(E)
    tops = np.array([-60, -20, -16.25, -16, -15.75, -3, 0, 3, 15.75, 16, 16.25, 20, 60], dtype=np.float32)
    l = -np.abs(rng.standard_normal((6 * len(tops), E))).astype(np.float32)
    l *= np.repeat(np.array([0.5, 4, 12], dtype=np.float32), 2 * len(tops))[:, None]
    l[np.arange(len(l)), rng.integers(0, E, len(l))] = 0
    l += np.tile(tops, 6)[:, None]
    logits = torch.from_numpy(l).to(dtype).to(DEV)
    R, out, o = _check_forward(logits, min(E, 6), "sigmoid", renorm)
    _check_backward(R, logits, out, o, torch.randn((len(l), R.k), device=DEV),
                    torch.tensor([0.8, 0.05], device=DEV), "sigmoid", renorm)


def _check_backward(R, logits, out, o, h, dl, score, renorm, mask=None, dlogits=None):
    T, E = logits.shape
    if dlogits is None:
        dlogits = torch.full((T, E), 9.0, dtype=logits.dtype, device=DEV)
    l = logits.double().cpu().numpy()
    B.router_backward(R, logits, out, h, dl, dlogits, mask=mask)
    torch.cuda.synchronize()
    hn = np.zeros((T, R.k)) if h is None else h.double().cpu().numpy()
    db, dz = (0.0, 0.0) if dl is None else dl.double().tolist()
    m = None if mask is None else mask.cpu().numpy()
    ref = orouter.backward(l, o["topk_ids"], hn, o["counts"], o["live"], db, dz, score == "sigmoid",
                           renorm, m)
    got = dlogits.double().cpu().numpy()
    # terms of a row: sum |h|, the balance term max |g|, the z term
    n = max(o["live"], 1)
    lse = np.abs(np.where(np.isfinite(l), l, 0)).max() + np.log(E)
    size = (np.abs(np.where(o["topk_ids"] >= 0, hn, 0)).sum(1, keepdims=True) * (2 + R.k * U)
            + 2 * abs(db) * E / R.k / n / n * o["counts"].max(initial=0) + 2 * abs(dz) / n * lse)
    tol = (2 * _rel(l) + R.k * U) * size + HALF[logits.dtype] * np.abs(ref) * 1.01 + 1e-37
    assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())
    return dlogits


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,offset", [(3, 1), (8, 0), (8, 8), (1, 0)])
def test_router_strided_rows(dtype, pad, offset):
    say(f"[router-ld] {dtype} pad={pad} offset={offset}")
    rng = np.random.default_rng(5)
    T, E, k = 90, 128, 8
    logits = _logits(rng, T, E, dtype, pad, offset)
    R, out, o = _check_forward(logits, k, "softmax", True)
    wide = torch.full((T, E + 2 * pad), 5.0, dtype=dtype, device=DEV)
    dlogits = wide[:, pad:pad + E]
    h = torch.randn((T, k), device=DEV)
    _check_backward(R, logits, out, o, h, None, "softmax", True, dlogits=dlogits)
    assert (wide[:, :pad] == 5).all() and (wide[:, pad + E:] == 5).all()


@pytest.mark.parametrize("E", [8, 100, 256, 700])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_router_ties_extremes_and_masks(E, score, dtype):
    say(f"[router-odd] E={E} {score} {dtype}")
    inf, low = float("inf"), torch.finfo(dtype).min
    k = 4
    rows = [[0.0] * E,                                            # all equal: the lowest indexes
            [-0.0 if e % 2 else 0.0 for e in range(E)],           # -0 equals 0
            [-inf] * E,                                           # nothing left
            [-inf] * (E - 2) + [1.0, -inf],                       # one left
            [low] * (E - 1) + [2.0],                              # barred by the type's lowest value
            [float("nan")] + [0.0] * (E - 1),
            [0.0] * (E - 1) + [inf],
            [80.0] + [-80.0] * (E - 1),
            [-300.0 - e % 7 for e in range(E)]]                   # sigmoid underflows in 32 bits
    logits = torch.tensor(rows, dtype=dtype, device=DEV)
    mask = torch.ones(len(rows), dtype=torch.uint8, device=DEV)
    T = len(rows)
    for renorm in (True, False):
        for m in (None, mask, torch.tensor([1, 1, 1, 1, 0, 0, 0, 1, 0], dtype=torch.bool, device=DEV)):
            R = B.make_router(E, k, dtype, score, renorm)
            out, st = _forward(R, logits, m)
            l = logits.double().cpu().numpy()
            mn = None if m is None else m.cpu().numpy()
            with np.errstate(all="ignore"):
                o = orouter.forward(l, k, score == "sigmoid", renorm, 1.0, mn)
            assert st == (B.DEV_BAD_LOGIT if o["bad"] else 0)
            np.testing.assert_array_equal(out["topk_ids"].cpu().numpy(), o["topk_ids"])
            np.testing.assert_array_equal(out["counts"].cpu().numpy(), o["counts"])
            # |l| to 306 (`low` only enters as an exponential of 0): 5 * 612 + 40 roundings, doubled
            np.testing.assert_allclose(out["gates"].cpu().numpy(), o["gates"], rtol=6200 * U, atol=1e-37)
            np.testing.assert_allclose(out["prob_sum"].cpu().numpy(), o["prob_sum"], rtol=6200 * U,
                                       atol=1e-37)
            h = torch.ones((T, k), device=DEV)
            d = torch.full((T, E), 9.0, dtype=dtype, device=DEV)
            B.router_backward(R, logits, out, h, torch.tensor([0.5, 0.0], device=DEV), d, mask=m)
            torch.cuda.synchronize()
            with np.errstate(all="ignore"):
                ref = orouter.backward(l, o["topk_ids"], np.ones((T, k)), o["counts"], o["live"], 0.5,
                                       0.0, score == "sigmoid", renorm, mn)
            # h terms up to 2 k = 8, the same relative error, and half a step of the output's type
            np.testing.assert_allclose(d.double().cpu().numpy(), ref, rtol=HALF[dtype] * 1.01,
                                       atol=6200 * U * 16)


def test_router_nothing_routed_and_no_tokens():
    say("[router-none]")
    R = B.make_router(16, 2, torch.float32)
    for logits, mask in ((torch.randn(40, 16, device=DEV), torch.zeros(40, dtype=torch.uint8, device=DEV)),
                         (torch.empty(0, 16, device=DEV), None)):
        out, st = _forward(R, logits, mask)
        assert st == 0 and int(out["live"].item()) == 0
        assert (out["topk_ids"] == -1).all() and (out["gates"] == 0).all()
        assert (out["counts"] == 0).all() and (out["prob_sum"] == 0).all() and (out["losses"] == 0).all()
        d = torch.full(logits.shape, 3.0, device=DEV)
        h = torch.ones((logits.shape[0], 2), device=DEV)
        B.router_backward(R, logits, out, h, torch.ones(2, device=DEV), d, mask=mask)
        torch.cuda.synchronize()
        assert (d == 0).all()


def test_router_backward_in_place_without_gradients_of_losses_or_gates_and_foreign_ids():
    say("[router-bwd-odd]")
    rng = np.random.default_rng(8)
    T, E, k = 50, 96, 6
    logits = _logits(rng, T, E, torch.float32)
    R, out, o = _check_forward(logits, k, "softmax", False)
    h = torch.randn((T, k), device=DEV)
    ref = _check_backward(R, logits, out, o, h, None, "softmax", False)
    _check_backward(R, logits, out, o, None, torch.tensor([0.3, 0.2], device=DEV), "softmax", False)
    keep = logits.clone()
    B.router_backward(R, logits, out, h, None, logits)            # over the logits themselves
    torch.cuda.synchronize()
    assert torch.equal(logits, ref)
    # ids a caller edits: the same expert twice adds up, ids outside [0, E) are left out
    ids = out["topk_ids"]
    ids[0, 1] = ids[0, 0]
    ids[1, 0] = E
    ids[2, 3] = -5
    hn = h.clone()
    hn[1, 0] = float("nan")                                       # not read
    o["topk_ids"] = ids.cpu().numpy()
    d = torch.empty((T, E), device=DEV)
    B.router_backward(R, keep, out, hn, None, d)
    torch.cuda.synchronize()
    hn[1, 0] = 0.0
    want = orouter.backward(keep.double().cpu().numpy(), o["topk_ids"], hn.double().cpu().numpy(),
                            o["counts"], o["live"], 0.0, 0.0, False, False)
    np.testing.assert_allclose(d.cpu().numpy(), want, rtol=0, atol=1e-5)   # sum |h| <= 24, 40 roundings


def test_router_is_repeatable_on_a_side_stream_and_in_a_graph():
    say("[router-graph]")
    rng = np.random.default_rng(9)
    T, E, k = 3000, 128, 8
    logits = _logits(rng, T, E, torch.bfloat16)
    mask = torch.from_numpy((rng.random(T) < 0.9).astype(np.uint8)).to(DEV)
    R = B.make_router(E, k, torch.bfloat16)
    out, ws = B.alloc_router(R, T, DEV), B.router_workspace(R, T, DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    h, dl = torch.randn((T, k), device=DEV), torch.tensor([0.1, 0.01], device=DEV)
    d = torch.empty((T, E), dtype=torch.bfloat16, device=DEV)

    def both():
        B.router_forward(R, logits, out, ws, st, mask=mask)
        B.router_backward(R, logits, out, h, dl, d, mask=mask)

    def outs():
        torch.cuda.synchronize()
        return [t.clone() for t in (*out.values(), d)]

    both()
    ref = outs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    for a, b in zip(outs(), ref):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for rep in range(3):
        for t in (*out.values(), d):
            t.zero_()
        g.replay()
        for a, b in zip(outs(), ref):
            assert torch.equal(a, b), rep
        both()
    logits.copy_(_logits(rng, T, E, torch.bfloat16))
    both()
    ref = outs()
    g.replay()
    for a, b in zip(outs(), ref):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Rows far apart and far into their buffers: the last bytes lie beyond 2^32."""
    say("[router-far]")
    rng = np.random.default_rng(10)
    T, E, k, ld = 1100, 72, 4, 1 << 20
    logits = torch.empty((T, ld), dtype=torch.float32, device=DEV)[:, 5:5 + E]
    logits.copy_(_logits(rng, T, E, torch.float32))
    assert T * ld * 4 > 1 << 32
    R, out, o = _check_forward(logits, k, "softmax", True)
    dlogits = torch.empty((T, ld), dtype=torch.float32, device=DEV)[:, 3:3 + E]
    _check_backward(R, logits, out, o, torch.randn((T, k), device=DEV), None, "softmax", True, dlogits=dlogits)
    del logits, dlogits
    slots, d_ff = 600_000, 2048
    z = torch.empty((slots, 2 * d_ff), dtype=torch.bfloat16, device=DEV)
    dz = torch.empty_like(z)
    at = [0, slots // 2, slots - 1]
    for s in at:
        z[s].normal_()
        dz[s].normal_()
    got = torch.empty(3, device=DEV)
    B.gate_grad(z, dz, torch.tensor(at, dtype=torch.int32, device=DEV), got)
    torch.cuda.synchronize()
    for i, s in enumerate(at):
        u, du = z[s, d_ff:].double(), dz[s, d_ff:].double()
        assert abs(float(got[i]) - float(u @ du)) <= (d_ff / 16 + 8) * U * float(u.abs() @ du.abs())


def test_another_device_is_refused(monkeypatch):
    R = B.make_router(8, 2)
    x = torch.zeros((4, 8), device=DEV)
    out, ws = B.alloc_router(R, 4, DEV), B.router_workspace(R, 4, DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(B.MoeError, match="current device"):
        B.router_forward(R, x, out, ws, st)


# ---- gate gradients: a dot of d_ff products, summed by a lane in turn and a tree of 16:
# (d_ff / 16 + 4) roundings of partial sums below sum |z dz|
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,slots,d_ff", [(1, 1, 64), (7, 40, 64), (600, 700, 192), (513, 600, 768),
                                             (33, 50, 2048), (0, 5, 64), (4, 0, 64)])
def test_gate_grad(dtype, rows, slots, d_ff):
    say(f"[gate_grad] {dtype} rows={rows} slots={slots} d_ff={d_ff}")
    rng = np.random.default_rng(rows + d_ff)
    z = torch.from_numpy(rng.standard_normal((slots, 2 * d_ff)).astype(np.float32)).to(dtype).to(DEV)
    dz = torch.from_numpy(rng.standard_normal((slots, 2 * d_ff)).astype(np.float32)).to(dtype).to(DEV)
    r2s = rng.integers(-1, max(slots, 1), size=rows).astype(np.int32)
    if slots == 0:
        r2s[:] = 0
    if rows > 4:
        r2s[0], r2s[1], r2s[2], r2s[3] = slots, 2 ** 31 - 1, -2 ** 31, slots - 1
        z[:, :d_ff] = float("nan")                                # G is not read
    got = torch.full((rows,), 9.0, device=DEV)
    B.gate_grad(z, dz, torch.from_numpy(r2s).to(DEV), got)
    torch.cuda.synchronize()
    u, du = z[:, d_ff:].double().cpu().numpy(), dz[:, d_ff:].double().cpu().numpy()
    for i, s in enumerate(r2s):
        want = float(u[s] @ du[s]) if 0 <= s < slots else 0.0
        size = float(np.abs(u[s]) @ np.abs(du[s])) if 0 <= s < slots else 0.0
        assert abs(float(got[i]) - want) <= (d_ff / 16 + 8) * U * size, i
