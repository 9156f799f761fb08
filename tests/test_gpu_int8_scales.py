"""The int8 layer against its oracle more closely than by the worst roundings: an output is off by roundings to bf16,
which average, and by nothing that all outputs share.

u = 2^-8, half a step of bf16 at 1.  A rounding is off by u / sqrt(3) rms at most, of the value's power of two.  An
output has two, its contributions' and its own: sqrt(2 / 3) u = 0.82 u of the norm.  An A within fp32's roundings of a
border (2^-12 of them) moves by a step of 2 u, and a row's largest with all its codes: 2 u 2^-6 = 2^-13.  So u in all.

What all outputs share: <y, ref> / <ref, ref> - 1 is the mean of N independent errors, u sqrt(3 / N) for normal
outputs, 2^-14.7 at N = 2^15; six of those are 2^-12.  A scale of max / 128 instead of max / 127 would be 2^-7.

The two forms of the products have the same codes, whole sums and order of scales.  Their sigmoids may differ in the
last bits: an A moves where it is that near to a border, 2^-12.4 of them, 5% of the rows of 256 have one, whose outputs
move by 2^-7 / 16 of themselves, a bf16 step for one in 16: k 5% / 16, 0.6% of the outputs for two experts a token, by
a step of a contribution.  Taken as 2^-5 of them, and 2^-9 of the norm (2^-7 sqrt(2^-5) = 2^-9.5)."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_int8 import Layer8

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


# T, k, E, d, f, beta, P: few rows an expert, off the 256 grid (few and many rows), the 256 x 256 tiles
@pytest.mark.parametrize("T,k,E,d,f,beta,P", [(64, 8, 128, 512, 256, 16, 1), (60, 4, 64, 768, 320, 32, 2), (333, 3, 10, 384, 192, 32, 2),
                                              (600, 2, 4, 512, 256, 128, 1), (900, 3, 5, 768, 512, 300, 2), (1500, 2, 3, 256, 1344, 64, 1)])
def test_errors_are_roundings(T, k, E, d, f, beta, P):
    c = Layer8(T, k, E, d, f, beta, P, seed=T)
    assert T * d >= 1 << 15
    y, ref = c.run().double().cpu().numpy(), c.oracle()
    err = np.linalg.norm(y - ref) / np.linalg.norm(ref)
    shared = (y * ref).sum() / (ref * ref).sum() - 1
    say(f"[int8 scales] T={T} d={d} f={f}: {err:.2e}, shared {shared:.1e}")
    assert err <= U
    assert abs(shared) <= 2.0 ** -12


@pytest.mark.parametrize("seed", [1, 2])
def test_both_forms_agree_to_a_rounding(seed):
    """40 tokens of 16 experts by tiles of few rows, and among 900 by the 256 x 256 tiles."""
    large, small = (Layer8(T, 2, 16, 512, 256, 128, 1, seed=seed) for T in (900, 40))
    for n in ("w1", "w2", "s1", "s2"):
        small.dev[n].copy_(large.dev[n])
    for n in ("x", "ids", "gates"):
        small.dev[n].copy_(large.dev[n][:40])
    a, b = small.run().double(), large.run()[:40].double()
    moved, off = (a != b).double().mean().item(), ((a - b).norm() / b.norm()).item()
    say(f"[int8 forms] {moved:.2e} of the outputs differ, {off:.2e} of the norm")
    assert moved <= 2.0 ** -5 and off <= 2.0 ** -9
