"""Pins of the 8-bit optimizer states' definition, on the oracle: updates stay bounded."""
import numpy as np
import pytest

from oracle import adamw as oadam
from tests.adamw_cases import run_constant, run_normal, update_bound


def _oracle_run(g_of, steps, beta1, beta2):
    """|update| of lr 1 at each step [steps][n], states as 8-bit codes, from zero."""
    n = g_of(1).size
    mc, vc = np.zeros(n, np.uint8), np.zeros(n, np.uint8)
    ms, vs = np.zeros(n // 128), np.zeros(n // 128)
    out = []
    for t in range(1, steps + 1):
        m0, v0 = oadam.decode(mc, ms), oadam.decode(vc, vs) ** 2
        upd, m, v = oadam.step(np.zeros(n), g_of(t), m0, v0, t, 1.0, beta1, beta2, 1e-8, 0.0)
        word = oadam.words(5, t, 0, n)
        mc, ms, _ = oadam.encode(m, word & 0xFFFF, root=False)
        vc, vs, _ = oadam.encode(np.sqrt(v), word >> 16, root=True)
        out.append(np.abs(upd))
    return np.stack(out)


@pytest.mark.parametrize("beta2", [0.95, 0.99, 0.999])
def test_updates_of_constant_gradients_are_bounded(beta2):
    g, ratio = run_constant()
    upd = _oracle_run(lambda t: g, 60, 0.9, beta2)
    assert (upd <= update_bound(ratio, 60, beta2)).all()


@pytest.mark.parametrize("beta2", [0.95, 0.99, 0.999])
def test_updates_of_noise_stay_near_those_of_32_bit_states(beta2):
    g_of, limit = run_normal(beta2)
    assert _oracle_run(g_of, 100, 0.9, beta2)[20:].max() <= limit


def test_a_root_is_zero_only_where_it_is_zero():
    x = np.zeros(256)
    x[0], x[1], x[2], x[128] = 1.0, 1e-12, 1e-30, 2.0 ** -101
    for u16 in (0, 65535):
        codes, scales, _ = oadam.encode(x, np.full(256, u16), root=True)
        assert (codes[:3] == [126, 1, 1]).all() and not codes[3:].any() and scales[1] == 0
    codes, _, _ = oadam.encode(x, np.zeros(256, dtype=np.int64), root=False)
    assert (codes[:3] == [126, 0, 0]).all()
