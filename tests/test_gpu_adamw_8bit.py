"""GPU: 8-bit optimizer states over many steps, with gradients that lie far apart inside a block."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from oracle import adamw as oadam
from tests.adamw_cases import run_constant, run_normal, update_bound
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _updates(g_of, steps, beta2, check=None):
    """|update| / lr of every step [steps][n], from zero states; check(t, g, before, list) after each."""
    n, lr = g_of(1).size, 1e-3
    z8 = lambda: [torch.zeros(n, dtype=torch.uint8, device=DEV)]
    zs = lambda: [torch.zeros(n // 128, device=DEV)]
    s = {"p": [torch.zeros(n, device=DEV)], "g": [torch.zeros(n, device=DEV)], "m": z8(), "v": z8(),
         "m_scale": zs(), "v_scale": zs()}
    opt = B.make_adamw(**s)
    out = []
    for t in range(1, steps + 1):
        g = g_of(t)
        s["g"][0].copy_(torch.from_numpy(g))
        s["p"][0].zero_()                               # the update itself, without p's rounding
        before = {k: s[k][0].cpu().numpy() for k in ("m", "v", "m_scale", "v_scale")}
        B.adamw(opt, lr=lr, beta1=0.9, beta2=beta2, eps=1e-8, step=t, seed=5)
        torch.cuda.synchronize()
        out.append(np.abs(s["p"][0].double().cpu().numpy()) / lr)
        if check is not None:
            check(t, g, before, {k: s[k][0].cpu().numpy() for k in before})
    return np.stack(out)


@pytest.mark.parametrize("beta2", [0.95, 0.99, 0.999])
def test_updates_of_constant_gradients_are_bounded(beta2):
    say(f"[adamw-8bit] constant beta2={beta2}")
    g, ratio = run_constant()
    upd = _updates(lambda t: g, 60, beta2)
    assert (upd <= update_bound(ratio, 60, beta2)).all()


@pytest.mark.parametrize("beta2", [0.95, 0.99, 0.999])
def test_updates_of_noise_stay_near_those_of_32_bit_states(beta2):
    say(f"[adamw-8bit] noise beta2={beta2}")
    g_of, limit = run_normal(beta2)
    assert _updates(g_of, 100, beta2)[20:].max() <= limit


@pytest.mark.parametrize("beta2", [0.5, 0.99, 0.9999])
def test_codes_of_far_apart_states_are_the_definitions(beta2):
    """Every code of sqrt(v) at each step against the oracle's from the same states; 16 u for the quotient and 16
    for the sum that is cut, as in the tests of single steps: within 2^-15 of a whole number either code is right
    (u = 2^-24).  The limit of m carries some 6 u (two scales, a reciprocal, a sum); no code of m is as near to it."""
    say(f"[adamw-8bit] codes beta2={beta2}")
    g_of, _ = run_normal(beta2)
    low = [0, 0]
    b2, c2 = (float(np.float32(x)) for x in (beta2, 1 - beta2))

    def check(t, g, before, after):
        v0 = oadam.decode(before["v"], before["v_scale"]) ** 2
        root = np.sqrt(b2 * v0 + c2 * g * g)
        m = (after["m"], after["m_scale"].astype(np.float64))
        codes, scales, dist = oadam.encode(root, oadam.words(5, t, 0, g.size) >> 16, (*m, 0.9, beta2))
        under, most = oadam.under_m(*m, after["v_scale"].astype(np.float64), 0.9, beta2)
        mag = np.abs(oadam.decode(m[0], np.ones(m[1].size)))
        assert (np.abs(mag - most)[mag > 0] > 8 * 2.0 ** -24 * most[mag > 0]).all()
        # the error of sqrt(v) (8 u) and of the scale (16 u), in code steps of up to 16 a value
        near = dist <= 2.0 ** -15 + 24 * 16 * 2.0 ** -24
        assert (after["v"] == codes)[~near].all()
        assert (after["v"][under] > 0).all()
        np.testing.assert_allclose(after["v_scale"], scales, rtol=16 * 2.0 ** -24)
        low[0] += int((under & (codes == 1)).sum())
        low[1] += int(((codes == 0) & (root > 0)).sum())

    _updates(g_of, 12, beta2, check)
    assert low[0] > 1000 and low[1] > 1000               # both sides of the rule are there


def test_states_that_no_gradients_give_keep_their_codes():
    """Codes at random, m's far above what gradients give with a sqrt(v) of 0: rounded as they are, and the others."""
    say("[adamw-8bit] any codes")
    n = 1 << 20
    rng = np.random.default_rng(41)
    dev = lambda a: [torch.from_numpy(a).to(DEV)]
    for beta2, vs in ((0.99, 1e-3), (0.999, 1e-5), (0.5, 1e-3)):
        mc = (rng.integers(0, 127, n) | rng.integers(0, 2, n) << 7).astype(np.uint8)
        vc = (rng.integers(0, 127, n) * (rng.random(n) < 0.5)).astype(np.uint8)
        sc = [((rng.random(n // 128) + 0.5) * x / 448).astype(np.float32) for x in (1e-4, vs)]
        g = (rng.standard_normal(n) * 1e-8).astype(np.float32)       # sqrt(v) far below a step where its code was 0
        s = {"p": dev(np.zeros(n, np.float32)), "g": dev(g), "m": dev(mc), "v": dev(vc), "m_scale": dev(sc[0]),
             "v_scale": dev(sc[1])}
        B.adamw(B.make_adamw(**s), lr=1e-3, beta1=0.9, beta2=beta2, step=3, seed=8)
        torch.cuda.synchronize()
        b2, c2 = (float(np.float32(x)) for x in (beta2, 1 - beta2))
        root = np.sqrt(b2 * oadam.decode(vc, sc[1]) ** 2 + c2 * g.astype(np.float64) ** 2)
        m = (s["m"][0].cpu().numpy(), s["m_scale"][0].double().cpu().numpy())
        codes, _, dist = oadam.encode(root, oadam.words(8, 3, 0, n) >> 16, (*m, 0.9, beta2))
        _, most = oadam.under_m(*m, s["v_scale"][0].double().cpu().numpy(), 0.9, beta2)
        mag = np.abs(oadam.decode(m[0], np.ones(m[1].size)))
        near = (dist <= 2.0 ** -15 + 24 * 16 * 2.0 ** -24) | ((mag > 0) & (np.abs(mag - most) <= 8 * 2.0 ** -24 * most))
        got = s["v"][0].cpu().numpy()
        assert (got == codes)[~near].all() and near.mean() < 0.01
        assert ((codes == 0) & (mag > 0)).any() == (beta2 > 0.5) and ((codes == 1) & (root < 1e-8)).any()


@pytest.mark.parametrize("eps", [1e-8, 1e-25])
@pytest.mark.parametrize("bits", [32, 8])
def test_roots_of_tiny_and_subnormal_v(bits, eps):
    """One step from zero states with gradients whose v is near or below fp32's smallest normal number.  v is rounded
    to a multiple of 2^-149 (its two products and their sum: 1.5 steps), half of that relative to v in its root; 24
    roundings of 2^-24 for the rest."""
    say(f"[adamw-tiny] bits={bits} eps={eps}")
    u = 2.0 ** -24
    rng = np.random.default_rng(21)
    for G in (1e-13, 1e-17, 1e-18, 1e-19, 1e-20):
        n = 256
        g = (G * (1 + rng.random(n))).astype(np.float32).astype(np.float64)
        f = lambda: torch.zeros(n, device=DEV)
        b8 = lambda: torch.zeros(n, dtype=torch.uint8, device=DEV)
        s = {"p": [f()], "g": [torch.from_numpy(g.astype(np.float32)).to(DEV)], "m": [f()], "v": [f()]}
        if bits == 8:
            s.update(m=[b8()], v=[b8()], m_scale=[f()[:2]], v_scale=[f()[:2]])
        B.adamw(B.make_adamw(**s), lr=1e-3, beta1=0.9, beta2=0.99, eps=eps, step=1, seed=2)
        torch.cuda.synchronize()
        p, _, v = oadam.step(0 * g, g, 0 * g, 0 * g, 1, 1e-3, 0.9, 0.99, eps, 0.0)
        off = 24 * u + 0.75 * 2.0 ** -149 / v
        # g^2 is rounded in fp32 before its product with 1 - beta2
        off = off + 0.5 * 2.0 ** -149 / (g * g)
        got = s["p"][0].double().cpu().numpy()
        assert (np.abs(got - p) <= off * np.abs(p) + 2.0 ** -149).all(), G
        if bits == 8:                                    # v's code within its step, the scale within the error
            root = np.sqrt(v)
            top = root.reshape(-1, 128).max(1)
            scale = s["v_scale"][0].double().cpu().numpy()
            assert (np.abs(scale - top / 448) <= np.max(off) * top / 448 + 2.0 ** -149).all(), G
            back = oadam.decode(s["v"][0].cpu().numpy(), scale)
            assert (np.abs(back - root) <= root / 8 + np.max(off) * root * 2).all(), G


@pytest.mark.parametrize("bits", [32, 8])
def test_the_smallest_eps_leaves_what_has_no_gradient(bits):
    say(f"[adamw-eps] bits={bits}")
    n = 300
    f = lambda m=n: torch.zeros(m, device=DEV)
    b8 = lambda: torch.zeros(n, dtype=torch.uint8, device=DEV)
    s = {"p": [torch.randn(n, device=DEV)], "g": [f()], "m": [f()], "v": [f()]}
    if bits == 8:
        s.update(m=[b8()], v=[b8()], m_scale=[f(3)], v_scale=[f(3)])
    was = s["p"][0].clone()
    opt = B.make_adamw(**s)
    with pytest.raises(B.MoeError, match="invalid argument"):
        B.adamw(opt, lr=1e-3, eps=1e-40)
    for t in (1, 2):
        B.adamw(opt, lr=1e-3, eps=2.0 ** -126, step=t)
    torch.cuda.synchronize()
    assert torch.equal(s["p"][0], was)
