"""Gradients whose magnitudes lie far apart inside the blocks of 128 elements that share a scale, and how large
an AdamW update of theirs may be with 8-bit states.  Shared by the oracle's and the GPU's tests."""
import numpy as np

STEP = 2.0 ** -9 / 448          # the smallest code step of a block, of its largest element: 4.4e-6


def run_constant():
    """One element of 1 in each block, the others at a ratio of 1e-7 to 1 of it; (gradients, ratios)."""
    rng = np.random.default_rng(11)
    ratio = np.exp(rng.uniform(np.log(1e-7), 0, 128 * 64))
    ratio[::128] = 1.0
    sign = np.where(rng.random(ratio.size) < 0.5, -1.0, 1.0)
    ratio = ratio.astype(np.float32).astype(np.float64)
    return ratio * sign, ratio


def update_bound(ratio, steps, beta2):
    """[steps][n] of |update| / lr for the same gradient at every step, from zero states.

    In units of the block's largest, whose code is always the last one and which follows m and sqrt(v) of a
    constant gradient without rounding, m and v after a step are weighted means of their last values and of
    the ratio r (of r^2).  Rounded to neighbours, m never leaves r's code cell upwards and sqrt(v) never
    downwards; under an m that is not 0 sqrt(v) is one step at least.  So the update's m is at most up(r) of the
    largest's m and its sqrt(v) at least sqrt(beta2) of down(r) of the largest's the step before:
      |update| <= up(r) / down(r) * sqrt((1 - beta2^t) / (beta2 (1 - beta2^(t - 1)))).
    Where m's code is 0 the update's m is 0.1 g, its v at least (1 - beta2) g^2:
      |update| <= 0.1 / (1 - 0.9^t) * sqrt((1 - beta2^t) / (1 - beta2)), which is 1 at t = 1.  2^-10 for 60 steps of 32-bit arithmetic: each state a few
    roundings (2^-24 each) a step."""
    cell = np.exp2(np.maximum(np.floor(np.log2(ratio * 448)), -6) - 3) / 448
    down = np.maximum(np.floor(ratio / cell * (1 - 1e-6)), 1) * cell
    up = np.ceil(ratio / cell * (1 + 1e-6)) * cell
    t = np.arange(1, steps + 1, dtype=np.float64)
    with np.errstate(divide="ignore"):
        grow = np.sqrt((1 - beta2 ** t) / (beta2 * (1 - beta2 ** (t - 1))))
        fresh = 0.1 / (1 - 0.9 ** t) * np.sqrt((1 - beta2 ** t) / (1 - beta2))
    bound = np.maximum((up / down)[None] * grow[:, None], fresh[:, None])
    bound[0] = 1.0
    return bound * (1 + 2.0 ** -10)


def run_normal(beta2):
    """Normal gradients of another sign and size at every step, the blocks' first element of scale 1, the others
    of 1e-4 to 1e-7; (gradients of step t, limit of |update| / lr after 20 steps).

    With exact states |update| <= sqrt(sum w_i^2 / u_i) of the weights w_i = 0.1 * 0.9^i of m and u_i = (1 - beta2)
    beta2^i of v, whatever the gradients (Cauchy-Schwarz; 1.2 at beta2 = 0.95, 7.3 at 0.999).  Rounded, an element
    of one code step has an m of up to some three steps (half a step's noise at each step, / sqrt(1 - 0.81), at
    five deviations) over a sqrt(v) of one: a few times that bound.  Ten times is the limit; an m of one step over
    the sqrt((1 - beta2) g^2) of a g below it is STEP / (sqrt(1 - beta2) 1e-7) = 200 and more."""
    i = np.arange(2000)
    w, u = 0.1 * 0.9 ** i, (1 - beta2) * beta2 ** i
    exact = np.sqrt((w[u > 0] ** 2 / u[u > 0]).sum())
    rng = np.random.default_rng(12)
    scale = np.exp(rng.uniform(np.log(1e-7), np.log(1e-4), 128 * 64))
    scale[::128] = 1.0

    def g_of(t):
        return (np.random.default_rng(1000 + t).standard_normal(scale.size) * scale).astype(np.float32).astype(np.float64)

    return g_of, 10 * exact
