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
        mc, ms, _ = oadam.encode(m, word & 0xFFFF)
        vc, vs, _ = oadam.encode(np.sqrt(v), word >> 16, (mc, ms, beta1, beta2))
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


def test_where_a_root_keeps_a_step():
    """A code of 0 becomes 1 under an m of codes 1 to the limit, and nowhere else."""
    x = np.zeros(256)
    x[:8], x[128] = [1.0, 1e-12, 1e-12, 1e-12, 0.0, 1e-12, 1e-12, 0.5], 2.0 ** -101
    mc = np.zeros(256, np.uint8)
    mc[:8] = [0, 0, 1, 0x81, 0, 20, 0x7F, 3]
    mc[128:] = 1
    ms = np.array([1.0 / 448, 1e-38])
    none = np.zeros(256, dtype=np.int64)                     # random bits that never round a small value up
    plain, _, _ = oadam.encode(x, none)
    assert not plain[1:7].any()
    # limit 2 C / 512 + 5.7 / 512 in m's units: 10.4 steps at beta2 = 0.99, 80 at 0.9999 (code 20: 24 steps)
    codes, scales, _ = oadam.encode(x, none, (mc, ms, 0.9, 0.99))
    assert list(codes[:8]) == [126, 0, 1, 1, 0, 0, 0, plain[7]] and not codes[8:].any() and scales[1] == 0
    codes, _, _ = oadam.encode(x, none, (mc, ms, 0.9, 0.9999))
    assert codes[5] == 1
    codes, _, _ = oadam.encode(x, none, (mc, ms, 0.9, 0.5))          # beta1^2 >= beta2: no limit, but NaN's code
    assert codes[5] == 1 and codes[6] == 0
