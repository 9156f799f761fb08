"""The oracles of the router, the norms and AdamW against closed forms and central differences."""
import numpy as np
import pytest

from oracle import adamw as oadam
from oracle import norm as onorm
from oracle import router as orouter


def _diff(f, x, h=1e-5):
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        hi = f()
        x[i] = keep - h
        lo = f()
        x[i] = keep
        out[i] = (hi - lo) / (2 * h)
    return out


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_is_the_objectives(sigmoid, renorm):
    rng = np.random.default_rng(3)
    l = rng.standard_normal((5, 7))
    l[1, 2] = -np.inf
    mask = np.array([1, 1, 0, 1, 1])
    f = orouter.forward(l, 3, sigmoid, renorm, mask=mask)
    h = rng.standard_normal((5, 3))
    args = (f["topk_ids"], h, f["counts"], f["live"], 0.7, 0.3, sigmoid, renorm, mask)
    got = orouter.backward(l, *args)
    with np.errstate(invalid="ignore"):
        want = _diff(lambda: orouter.objective(l, *args), l)
    want[1, 2] = 0.0
    np.testing.assert_allclose(got, want, atol=1e-8)
    assert (got[2] == 0).all()


def test_router_losses_of_even_routing():
    # the logits of token t favour expert t, all alike: c = 1, P sums to 1 for every expert
    E = 6
    l = np.eye(E) * 2.0
    f = orouter.forward(l, 1)
    assert f["losses"][0] == pytest.approx(1.0)
    lse = np.log(np.exp(2.0) + E - 1)
    assert f["losses"][1] == pytest.approx(lse * lse)
    assert f["gates"].tolist() == [[1.0]] * E


def test_router_ties_masks_and_empty_rows():
    ninf = -np.inf
    l = np.array([[0.0, -0.0, 0.0, -1.0], [ninf] * 4, [ninf, 3.0, ninf, ninf], [np.nan, 0, 0, 0],
                  [np.inf, 0, 0, 0], [1, 2, 3, 4]])
    f = orouter.forward(l, 2, mask=np.array([1, 1, 1, 1, 1, 0]))
    assert f["topk_ids"].tolist() == [[0, 1], [-1, -1], [1, -1], [-1, -1], [-1, -1], [-1, -1]]
    assert f["live"] == 2 and f["bad"]
    assert not orouter.forward(l, 2, mask=np.array([1, 1, 1, 0, 0, 1]))["bad"]
    assert f["gates"][2].tolist() == [1.0, 0.0]


@pytest.mark.parametrize("kind", [None, "token", "feature"])
def test_norm_gradients_are_differences(kind):
    rng = np.random.default_rng(4)
    T, d, eps, alpha = 3, 5, 1e-3, 0.6
    x, u, w = rng.standard_normal((T, d)), rng.standard_normal((T, d)), rng.standard_normal(d)
    g = {None: None, "token": rng.standard_normal((T, 1)), "feature": rng.standard_normal(d)}[kind]
    dn, dr = rng.standard_normal((T, d)), rng.standard_normal((T, d))

    def before():
        r, n, _ = onorm.norm_in(x, w, eps, u, g, alpha)
        return float((n * dn).sum() + (r * dr).sum())

    r, _, rstd = onorm.norm_in(x, w, eps, u, g, alpha)
    dx, dw, du, dg = onorm.norm_in_backward(dn, r, w, rstd, dr, u, g, alpha)
    for got, at in ((dx, x), (dw, w), (du, u)) + (() if g is None else ((dg, g),)):
        np.testing.assert_allclose(got, _diff(before, at), atol=1e-7)

    def after():
        return float((onorm.norm_out(u, x, w, eps, g, alpha)[0] * dn).sum())

    _, rstd = onorm.norm_out(u, x, w, eps, g, alpha)
    dy, dw, dg = onorm.norm_out_backward(dn, u, w, rstd, g, alpha)
    for got, at in ((dy, u), (dw, w)) + (() if g is None else ((dg, g),)):
        np.testing.assert_allclose(got, _diff(after, at), atol=1e-7)


def test_adamw_first_step_is_signed_learning_rate():
    g = np.array([3.0, -1e-3, 0.0])
    p, m, v = oadam.step(np.ones(3), g, np.zeros(3), np.zeros(3), 1, 0.1, 0.9, 0.999, 1e-12, 0.0)
    np.testing.assert_allclose(p, [0.9, 1.1, 1.0], rtol=1e-6)
    np.testing.assert_allclose(m, 0.1 * g)


def test_e4m3_rounding_is_unbiased_and_to_a_neighbour():
    rng = np.random.default_rng(5)
    x = np.full(128 * 512, 0.337)
    x[::128] = 1.0                                       # the scale: 1 / 448
    codes, scales, _ = oadam.encode(x, oadam.words(7, 1, 0, x.size) & 0xFFFF)
    back = oadam.decode(codes, scales)
    y = 0.337 * 448                                      # between 144 and 160: steps of 16
    rest = np.ones(x.size, bool)
    rest[::128] = False
    assert set(np.round(back[rest] * 448).astype(int)) == {144, 160}
    # a mean of n draws of a step of 16: standard error 16 * sqrt(f (1 - f) / n); five of them
    f = (y - 144) / 16
    assert abs(back[rest].mean() * 448 - y) < 5 * 16 * np.sqrt(f * (1 - f) / rest.sum())
    x = rng.standard_normal(1000) * np.exp(rng.standard_normal(1000) * 4)
    codes, scales, _ = oadam.encode(x, oadam.words(8, 2, 1, x.size) >> 16)
    back, per = oadam.decode(codes, scales), np.repeat(scales, 128)[:1000]
    step = np.exp2(np.maximum(np.floor(np.log2(np.abs(x) / per)), -6) - 3) * per
    assert (np.abs(back - x) <= step * (1 + 1e-9)).all()


def test_words_are_even():
    w = oadam.words(1234, 17, 3, 1 << 16)
    for part in (w & 0xFFFF, w >> 16, ((w * oadam.ROOT3) & 0xFFFFFFFF) >> 16):
        # 64 bins of 1024: a count's deviation is about 32 (random) -- six of them, twice over
        # for bins that are not independent
        assert (np.abs(np.bincount(part >> 10, minlength=64) - 1024) < 12 * 32).all()
        assert abs(np.corrcoef(part[1:], part[:-1])[0, 1]) < 6 / 256
