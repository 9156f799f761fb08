"""The router's choice by values where equal experts stand before a larger one that 32 bits do not tell apart.

Scores of sigmoid logits around 20 differ by 10^-9 and less, those of neighbouring fp32 softmax logits by 10^-8: next
to nothing in 32 bits, where the lower index leads, and apart in 64.  Two of the lower logit first, then the higher one:
the last place (or the member that makes a group's value) is followed by its equal, and the expert that belongs there
comes behind both."""
import itertools

import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_choice import _check

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def _levels(score, dtype):
    """Three logits whose scores are near to each other, and one far below."""
    if score == "sigmoid":                                        # 2^-3 apart: bf16 numbers
        return [20.0, 20.125, 20.25], -5.0
    one = np.float32(1.0)
    up = np.nextafter(one, np.float32(2))
    return [float(one), float(up), float(np.nextafter(up, np.float32(2)))], -5.0


KINDS = [("sigmoid", F32), ("sigmoid", BF16), ("softmax", F32)]  # bf16 softmax scores that differ are far apart


@pytest.mark.parametrize("score,dtype", KINDS)
@pytest.mark.parametrize("E", [8, 64, 100, 256, 512, 600, 1024])
@pytest.mark.parametrize("k", [1, 2, 3, 7, 8])
def test_last_place_before_equals(score, dtype, E, k):
    say(f"[equals] {score} {dtype} E={E} k={k}")
    rng = np.random.default_rng(E * 10 + k)
    near, far = _levels(score, dtype)
    rows = []
    for same in range(1, 12):                                     # that many equals first, then a larger one
        row = np.full(E, far, dtype=np.float32)
        at = np.sort(rng.choice(E, min(same + 1, E), replace=False))
        row[at] = near[0]
        row[at[-1]] = near[1]
        rows.append(row)
        mixed = np.full(E, far, dtype=np.float32)
        at = rng.choice(E, min(E, 3 + same), replace=False)
        mixed[at] = rng.choice(near, len(at))
        rows.append(mixed)
    rows.append(rng.choice(near, E).astype(np.float32))
    logits = torch.from_numpy(np.stack(rows)).to(dtype).to(DEV)
    for bias in (torch.zeros(E, device=DEV), torch.full((E,), 0.25, device=DEV)):
        _check(logits, k, score, True, bias)


@pytest.mark.parametrize("score,dtype", KINDS)
@pytest.mark.parametrize("E,groups,top", [(64, 8, 4), (64, 2, 1), (100, 4, 2), (128, 4, 2), (256, 8, 4), (512, 16, 5), (1024, 8, 3)])
@pytest.mark.parametrize("rank", ["max", "top2"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_members_before_equals(score, dtype, E, groups, top, rank, with_bias):
    """Groups whose value is made by a member that its equal hides."""
    say(f"[equal members] {score} {dtype} E={E} groups={groups}/{top} {rank}")
    rng = np.random.default_rng(E + groups)
    near, far = _levels(score, dtype)
    size = E // groups
    rows = []
    for _ in range(12):
        row = np.full(E, far, dtype=np.float32)
        for g in range(groups):
            at = g * size + np.sort(rng.choice(size, 4, replace=False))
            kind = rng.integers(0, 4)
            if rank == "top2" and kind < 3:                       # one far above the others makes half of the value
                row[at[0]] = near[0]
            row[at[1:]] = [[near[0], near[0], near[1]], [near[0], near[0], near[0]], [near[0], near[1], near[1]],
                           [near[1], near[0], near[2]]][kind]
        rows.append(row)
    logits = torch.from_numpy(np.stack(rows)).to(dtype).to(DEV)
    bias = torch.full((E,), 0.25, device=DEV) if with_bias else None
    _check(logits, min(8, top * size), score, True, bias, groups, top, rank)


@pytest.mark.parametrize("score,dtype", KINDS)
@pytest.mark.parametrize("E,groups,top", [(16, 2, 1), (32, 4, 2), (64, 4, 1), (256, 8, 4), (12, 3, 1), (1024, 32, 5)])
@pytest.mark.parametrize("rank", ["max", "top2"])
def test_every_order_of_near_members(score, dtype, E, groups, top, rank):
    """Two to four members of a group on three near levels, in every order: the two that make its value may be a lower
    one and a higher one whose equal is left out."""
    say(f"[orders] {score} {dtype} E={E} groups={groups}/{top} {rank}")
    rng = np.random.default_rng(E + 7 * groups)
    near, far = _levels(score, dtype)
    size = E // groups
    orders = [o for n in (2, 3, 4) for o in itertools.product(near, repeat=n)]
    rows = []
    for o in orders:
        row = np.full(E, far, dtype=np.float32)
        for g in range(groups):
            members = o if g == 0 else orders[rng.integers(len(orders))]
            row[g * size + np.sort(rng.choice(size, len(members), replace=False))] = members
        rows.append(row)
    logits = torch.from_numpy(np.stack(rows)).to(dtype).to(DEV)
    _check(logits, min(3, top * size), score, True, None, groups, top, rank)
