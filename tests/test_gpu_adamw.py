"""GPU parity of AdamW over lists of tensors against the fp64 oracle.

Tolerances, u = 2^-24: m and v are two rounded products and a rounded sum (3 u of the terms'
magnitudes), p a rounded product, the update (some 12 roundings and two reciprocals of 1 u) and a
sum.  8-bit states: the code is the oracle's wherever the sum that is cut off lies further from a whole
number than the 32-bit arithmetic's error, 16 * 8 u for the quotient (q below 16) and 16 u for the
sum, taken as 2^-15; elsewhere the neighbouring code is right too."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from oracle import adamw as oadam
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
HY = dict(beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


def _lists(rng, sizes, pdt, gdt, bits, master=False, odd=False):
    def dev(a, dt=F32):
        t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
        t = t.to(dt) if t.dtype == F32 else t
        if not odd:
            return t
        full = torch.zeros(t.numel() + 3, dtype=t.dtype, device=DEV)     # a view off every alignment
        full[1:1 + t.numel()] = t
        return full[1:1 + t.numel()]

    normal = lambda n: rng.standard_normal(n).astype(np.float32)
    s = {"p": [], "g": [], "m": [], "v": [], "m_scale": None, "v_scale": None, "master": None}
    p32 = [normal(n) * 0.1 for n in sizes]
    s["p"] = [dev(p, pdt) for p in p32]
    s["g"] = [dev(normal(n) * 1e-2, gdt) for n in sizes]
    if master:
        s["master"] = [dev(p) for p in p32]
    if bits == 32:
        s["m"] = [dev(normal(n) * 1e-3) for n in sizes]
        s["v"] = [dev((normal(n) * 1e-2) ** 2) for n in sizes]
    else:
        blocks = [-(-n // 128) for n in sizes]
        codes = lambda n, sign: (rng.integers(0, 127, n) | (rng.integers(0, 2, n) * 128 * sign)).astype(np.uint8)
        s["m"] = [dev(codes(n, 1)) for n in sizes]
        s["v"] = [dev(codes(n, 0)) for n in sizes]
        s["m_scale"] = [dev((rng.random(b) * 1e-5).astype(np.float32)) for b in blocks]
        s["v_scale"] = [dev((rng.random(b) * 1e-4).astype(np.float32)) for b in blocks]
    return s


def _np(t):
    return t.double().cpu().numpy() if t.dtype != torch.uint8 else t.cpu().numpy()


def _snap(s):
    return {k: None if v is None else [_np(t) for t in v] for k, v in s.items()}


def _check(before, s, j, t, lr, bits, seed, grad_scale=1.0, beta1=0.9, beta2=0.999, eps=1e-8,
           weight_decay=0.1):
    b1, b2, c1, c2 = (float(np.float32(x)) for x in (beta1, beta2, 1 - beta1, 1 - beta2))
    src = before["p"][j] if before["master"] is None else before["master"][j]
    g = before["g"][j] * grad_scale
    n = src.size
    if bits == 32:
        m0, v0 = before["m"][j], before["v"][j]
    else:
        m0 = oadam.decode(before["m"][j], before["m_scale"][j])
        v0 = oadam.decode(before["v"][j], before["v_scale"][j]) ** 2
    p, m, v = oadam.step(src, g, m0, v0, t, lr, beta1, beta2, eps, weight_decay)
    em = 6 * U * (np.abs(b1 * m0) + np.abs(c1 * g)) + 1e-44
    ev = 8 * U * v + 1e-44
    upd = np.abs(lr * m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    eupd = 24 * U * upd + np.abs(lr / (1 - beta1 ** t)) * em / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    ep = 6 * U * np.abs(src) + eupd + 2 * U * np.abs(p)
    word = oadam.words(seed, t, j, n)
    pt = s["p"][j]
    got = _np(pt)
    if before["master"] is not None:
        full = _np(s["master"][j])
        assert (np.abs(full - p) <= ep).all()
        assert torch.equal(pt, s["master"][j].to(BF16))
    elif pt.dtype == F32:
        assert (np.abs(got - p) <= ep).all(), float((np.abs(got - p) / ep).max())
    else:
        step = np.exp2(np.floor(np.log2(np.abs(p) + ep + 1e-38)) - 7)
        assert (np.abs(got - p) <= step + ep).all()
        # the same neighbour as the oracle's, but where 32-bit errors move the cut
        want = oadam.random_bf16(p, word)
        frac = (p / step + ((((word * oadam.ROOT3) & 0xFFFFFFFF) >> 16) / 65536) * np.sign(p)) % 1
        near = np.minimum(frac, 1 - frac) < ep / step + 2.0 ** -14
        assert (got == want)[~near].all()
        assert n < 1000 or near.mean() < 0.1     # the comparison covers nearly all (a share of few says nothing)
    if bits == 32:
        assert (np.abs(_np(s["m"][j]) - m) <= em).all()
        assert (np.abs(_np(s["v"][j]) - v) <= ev).all()
        return
    for x, e, name, u16 in ((m, em, "m", word & 0xFFFF), (np.sqrt(v), None, "v", word >> 16)):
        codes, scales, dist = oadam.encode(x, u16)
        got_c, got_s = _np(s[name][j]), _np(s[name + "_scale"][j])
        tol_s = 16 * U * scales if name == "v" else None
        if tol_s is None:                                         # m may cancel: its largest term's error
            tol_s = 4 * U * scales + np.max(np.concatenate([e, np.zeros(-n % 128)]).reshape(-1, 128), 1) / 448
        assert (np.abs(got_s - scales) <= tol_s + 1e-44).all()
        # an error of e in x is e / scale / unit in the sum; unit >= 2^-9
        per = np.repeat(scales, 128)[:n]
        y = np.abs(x) / np.where(per > 0, per, 1)
        unit = np.exp2(np.clip(np.floor(np.log2(np.maximum(y, 2.0 ** -20))), -6, 8) - 3)
        rel = np.repeat(tol_s, 128)[:n] / np.where(per > 0, per, 1)
        err = ((e if e is not None else 16 * U * x) / np.where(per > 0, per, 1) + y * rel) / unit + 2.0 ** -15
        near = dist <= err
        assert (got_c == codes)[~near].all(), (name, int((got_c != codes)[~near].sum()))
        off = np.abs(oadam.decode(got_c, got_s) - x)
        assert (off <= per * unit * 2.01 + (e if e is not None else 16 * U * x)).all()


SIZES = [[1], [127], [128, 129], [0, 5, 0, 4096, 4097], [100000], [7] * 70, [20481, 3, 0, 8192]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("pdt,master", [(F32, False), (BF16, False), (BF16, True)])
@pytest.mark.parametrize("gdt", [F32, BF16])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("odd", [False, True])
def test_adamw_steps(sizes, pdt, master, gdt, bits, odd):
    say(f"[adamw] {len(sizes)} of {max(sizes)} {pdt} master={master} {gdt} bits={bits} odd={odd}")
    rng = np.random.default_rng(sum(sizes) + bits)
    s = _lists(rng, sizes, pdt, gdt, bits, master, odd)
    opt = B.make_adamw(**s)
    for t in (1, 2, 1000):
        before = _snap(s)
        B.adamw(opt, lr=1e-3, step=t, seed=77, **HY)
        torch.cuda.synchronize()
        for j in range(len(sizes)):
            _check(before, s, j, t, 1e-3, bits, 77)


def test_views_leave_their_neighbours_alone():
    say("[adamw-edges]")
    for bits in (32, 8):
        rng = np.random.default_rng(3)
        whole = _lists(rng, [1000], BF16, BF16, bits)
        cut = {k: None if v is None or "scale" in k else [t[9:900] for t in v] for k, v in whole.items()}
        if bits == 8:
            cut["m_scale"], cut["v_scale"] = [whole["m_scale"][0][:7]], [whole["v_scale"][0][:7]]
        before = _snap(whole)
        B.adamw(B.make_adamw(**cut), lr=1e-2, step=3, **HY)
        torch.cuda.synchronize()
        after = _snap(whole)
        for k in ("p", "m", "v"):
            a, b = after[k][0], before[k][0]
            assert (a[:9] == b[:9]).all() and (a[900:] == b[900:]).all() and (a[9:900] != b[9:900]).any()
        if bits == 8:
            assert (after["m_scale"][0][7:] == before["m_scale"][0][7:]).all()


def test_device_step_rate_and_grad_scale_in_a_replayed_graph():
    say("[adamw-graph]")
    for bits in (32, 8):
        rng = np.random.default_rng(4)
        sizes = [5000, 33]
        s = _lists(rng, sizes, BF16, F32, bits)
        opt = B.make_adamw(**s)
        step = torch.ones(1, dtype=torch.int32, device=DEV)
        lr, gs = torch.full((1,), 1e-3, device=DEV), torch.full((1,), 0.25, device=DEV)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.adamw(opt, lr=lr, step=step, seed=9, grad_scale=gs, **HY)
        for t in range(1, 5):
            step.fill_(t)
            lr.fill_(1e-3 / t)
            before = _snap(s)
            graph.replay()
            torch.cuda.synchronize()
            for j in range(len(sizes)):
                _check(before, s, j, t, float(np.float32(1e-3 / t)), bits, 9, 0.25)


@pytest.mark.parametrize("bits", [32, 8])
def test_values_that_are_not_finite_stay_in_their_element(bits):
    say(f"[adamw-odd] bits={bits}")
    n = 600
    rng = np.random.default_rng(6)
    a, b = _lists(rng, [n], F32, F32, bits), None
    b = {k: None if v is None else [t.clone() for t in v] for k, v in a.items()}
    for s in (a, b):
        s["g"][0][300] = 0.0
        s["g"][0][301] = 0.0
        s["m"][0][300:302] = 0
        s["v"][0][300:302] = 0
    b["g"][0][300] = float("nan")
    b["g"][0][301] = float("inf")
    for s in (a, b):
        B.adamw(B.make_adamw(**s), lr=1e-3, step=5, **HY)
    torch.cuda.synchronize()
    rest = torch.ones(n, dtype=torch.bool, device=DEV)
    rest[300:302] = False
    for k in ("p", "m", "v"):
        assert torch.equal(a[k][0][rest], b[k][0][rest]), k
    assert b["p"][0][300:302].isnan().all()
    if bits == 8:
        assert (b["m"][0][300:302] & 127 == 127).all() and torch.equal(a["m_scale"][0], b["m_scale"][0])
        assert (b["v"][0][300:302] & 127 == 127).all() and torch.equal(a["v_scale"][0], b["v_scale"][0])
    else:
        assert b["m"][0][300].isnan() and b["m"][0][301].isinf()


def test_eight_bit_states_follow_slow_changes():
    """A state rounded to nearest would stop where its change per step is below half a code step;
    rounded at random it follows on average.  One constant gradient for each element: after t
    steps m = g (1 - b1^t) and v = g^2 (1 - b2^t)."""
    say("[adamw-slow]")
    n, t = 1 << 16, 300
    rng = np.random.default_rng(7)
    g = torch.from_numpy(np.exp(rng.standard_normal(n)).astype(np.float32)).to(DEV)
    z8 = lambda: torch.zeros(n, dtype=torch.uint8, device=DEV)
    zs = lambda: torch.zeros(n // 128, device=DEV)
    s = {"p": [torch.zeros(n, device=DEV)], "g": [g], "m": [z8()], "v": [z8()], "m_scale": [zs()],
         "v_scale": [zs()]}
    opt = B.make_adamw(**s)
    for i in range(1, t + 1):
        B.adamw(opt, lr=0.0, step=i, seed=5, beta1=0.9, beta2=0.999)
    torch.cuda.synchronize()
    G = g.double().cpu().numpy()
    m = oadam.decode(_np(s["m"][0]), _np(s["m_scale"][0])) / G
    v = oadam.decode(_np(s["v"][0]), _np(s["v_scale"][0])) ** 2 / G ** 2 / (1 - 0.999 ** t)
    # m: noise of a code step (at most 1/8 of the value) a step, decaying by 0.9: at most
    # 1/8 / 2 / sqrt(1 - 0.81) = 0.15 an element, 0.0006 in the mean of 65536; five of them
    assert abs(m.mean() - 1) < 0.003
    # v: sqrt(v) is rounded at random without bias, its square gains the rounding's variance: each
    # step adds at most (step/2)^2 f with a fraction f of a code step; the sum over the steps is bounded
    # by the drift |d sqrt(v)| * step / 1, so v is high by at most 1/8 of itself, and not low
    assert -0.01 < v.mean() - 1 < 0.125


def test_elements_past_2_to_the_31():
    say("[adamw-far]")
    n, tail = (1 << 31) + 1000, 1000
    s = {"p": [torch.zeros(n, device=DEV)], "g": [torch.zeros(n, dtype=BF16, device=DEV)],
         "m": [torch.zeros(n, dtype=torch.uint8, device=DEV)], "v": [torch.zeros(n, dtype=torch.uint8, device=DEV)],
         "m_scale": [torch.zeros(-(-n // 128), device=DEV)], "v_scale": [torch.zeros(-(-n // 128), device=DEV)]}
    s["g"][0][-tail:] = torch.randn(tail, device=DEV).to(BF16)
    B.adamw(B.make_adamw(**s), lr=1e-3, step=1, seed=4, **HY)
    torch.cuda.synchronize()
    start = n - tail
    assert start % 128 == 0
    g = _np(s["g"][0][start:])
    p, m, v = oadam.step(0 * g, g, 0 * g, 0 * g, 1, 1e-3, 0.9, 0.999, 1e-8, 0.1)
    assert (np.abs(_np(s["p"][0][start:]) - p) <= 40 * U * np.abs(p)).all()
    word = oadam.words(4, 1, 0, tail, start)
    for x, name, u16 in ((m, "m", word & 0xFFFF), (np.sqrt(v), "v", word >> 16)):
        codes, scales, dist = oadam.encode(x, u16)
        got = _np(s[name][0][start:])
        # x in 32 bits is off by 8 u, 16 units of the sum that is cut: 16 * 16 u with the quotient's
        assert (got == codes)[dist > 2.0 ** -14].all() and (dist > 2.0 ** -14).mean() > 0.99
        np.testing.assert_allclose(_np(s[name + "_scale"][0][start // 128:]), scales, rtol=16 * U)
    assert (s["p"][0][:start:4097] == 0).all() and (s["m"][0][:start:4097] == 0).all()


def test_lists_that_are_empty_or_long():
    say("[adamw-long]")
    B.adamw(B.make_adamw([], [], [], []), lr=1.0, step=1)
    sizes = [((i * 37) % 400) for i in range(3000)]
    rng = np.random.default_rng(8)
    s = _lists(rng, sizes, F32, F32, 32)
    before = _snap(s)
    B.adamw(B.make_adamw(**s), lr=1e-3, step=2, **HY)
    torch.cuda.synchronize()
    for j in range(len(sizes)):
        _check(before, s, j, 2, 1e-3, 32, 0)


def test_refused_lists():
    say("[adamw-refused]")
    f = lambda n=64: torch.zeros(n, device=DEV)
    x = f()
    with pytest.raises(B.MoeError, match="invalid argument"):     # the same parameter twice
        B.make_adamw([x, x], [f(), f()], [f(), f()], [f(), f()])
    with pytest.raises(B.MoeError, match="invalid argument"):     # a state on top of the gradient
        B.make_adamw([f()], [x], [x], [f()])
    y = f(100)
    with pytest.raises(B.MoeError, match="invalid argument"):     # views that overlap
        B.make_adamw([y[:60], y[50:]], [f(60), f(50)], [f(60), f(50)], [f(60), f(50)])
    B.make_adamw([f(), f()], [x, x], [f(), f()], [f(), f()])      # a gradient may be shared
    with pytest.raises(B.MoeError, match="invalid argument"):     # master of an fp32 parameter
        B.make_adamw([f()], [f()], [f()], [f()], master=[f()])
    with pytest.raises(B.MoeError):
        B.make_adamw([f().half()], [f()], [f()], [f()])
    opt = B.make_adamw([f()], [f()], [f()], [f()])
    for bad in (dict(step=0), dict(step=1, beta1=1.0), dict(step=1, beta2=-0.1), dict(step=1, eps=0.0),
                dict(step=1, weight_decay=float("nan"))):
        with pytest.raises(B.MoeError, match="invalid argument"):
            B.adamw(opt, lr=1e-3, **bad)
    with pytest.raises(B.MoeError):
        B.adamw(opt, lr=float("inf"), step=1)
