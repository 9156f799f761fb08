"""Host-side checks of the router's choice by values: refusals before any device work, and pins of its oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from oracle import choice as ochoice
from oracle import router as orouter

P = ctypes.c_void_p(256)
ARG, UNSUP, WS = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE


def _call(router=None, null=False, ld=16, T=4, ids=P, ws=P, **kw):
    R = router or B.Router(16, 2, 0, 0, 1, 1.0)
    C = B.Choice(**{**dict(bias=256, groups=4, top_groups=2, group_score=1), **kw})
    return B.load().moe_router_forward_choice(ctypes.byref(R), None if null else ctypes.byref(C), P, ld, None, T, ids, P, P,
                                              P, P, P, P, ws, 1 << 20, None)


def test_choice_refusals():
    for bad in (dict(groups=0), dict(groups=-1), dict(groups=3), dict(groups=32), dict(top_groups=0), dict(top_groups=5),
                dict(group_score=2), dict(group_score=-1), dict(groups=16, top_groups=1)):      # k = 2 of one expert
        assert _call(**bad) == ARG, bad
    assert _call(null=True) == ARG and _call(ids=None) == ARG and _call(ld=15) == ARG and _call(T=-1) == ARG
    assert _call(ws=None) == WS
    assert _call(router=B.Router(128, 2, 0, 0, 1, 1.0), ld=128, groups=128, top_groups=64) == UNSUP
    assert _call(router=B.Router(2048, 2, 0, 0, 1, 1.0), ld=2048) == UNSUP
    R = B.make_router(16, 4)
    for kw in (dict(groups=3), dict(groups=4, top_groups=5), dict(groups=8, top_groups=1), dict(groups=0), dict(groups=4, top_groups=0)):
        with pytest.raises(B.MoeError, match="not supported"):
            B.make_choice(R, **kw)
    with pytest.raises(B.MoeError, match="group_score"):
        B.make_choice(R, group_score="mean")
    with pytest.raises(B.MoeError, match="bias"):
        B.make_choice(R, torch.zeros(15))
    with pytest.raises(B.MoeError, match="bias"):
        B.make_choice(R, torch.zeros(16, dtype=torch.float64))
    c = B.make_choice(R, torch.zeros(16), 4, 2)
    with pytest.raises(B.MoeError, match="current device"):
        x = torch.zeros(4, 16)
        B.router_forward(R, x, B.alloc_router(R, 4, "cpu"), B.router_workspace(R, 4, "cpu"),
                         torch.zeros(1, dtype=torch.int32), choice=c)


def test_bias_update_refusals():
    f = B.load().moe_router_bias_update
    assert f(P, 0, 0.1, P, None) == ARG and f(None, 4, 0.1, P, None) == ARG and f(P, 4, 0.1, None, None) == ARG
    assert f(P, 4, math.nan, P, None) == ARG and f(P, 4, math.inf, P, None) == ARG
    assert f(P, 1025, 0.1, P, None) == UNSUP
    with pytest.raises(B.MoeError, match="current device"):
        B.router_bias_update(torch.zeros(4), torch.zeros(4, dtype=torch.int32), 0.1)


def test_oracle_pins():
    row = np.log(np.array([0.1, 0.2, 0.3, 0.4]))
    assert ochoice.choose(row, 2, False) == [3, 2]
    assert ochoice.choose(row, 2, False, bias=np.array([0.5, 0, 0, 0])) == [0, 3]
    # groups (0.1 + 0.5, 0.2) and (0.3, 0.4): the best member chooses the first, two best the first (0.8 > 0.7)
    b = np.array([0.35, 0, 0, 0])
    assert ochoice.choose(row, 2, False, bias=b, groups=2, top_groups=1, two=False) == [0, 1]
    assert ochoice.choose(row, 2, False, bias=b, groups=2, top_groups=1, two=True) == [3, 2]
    assert ochoice.choose(np.zeros(6), 3, True, groups=3, top_groups=2) == [0, 1, 2]           # equals: the lowest
    low = np.array([0.0, -np.inf, -np.inf, -np.inf])
    assert ochoice.choose(low, 2, True, groups=2, top_groups=1) == [0]
    assert ochoice.choose(row, 2, False, bias=np.array([np.nan, 0, 0, -np.inf])) == [2, 1]


def test_oracle_without_bias_and_groups_is_the_routers():
    rng = np.random.default_rng(0)
    l = rng.standard_normal((20, 12))
    for sigmoid in (False, True):
        a, b = ochoice.forward(l, 3, sigmoid), orouter.forward(l, 3, sigmoid)
        for k in a:
            np.testing.assert_allclose(a[k], b[k], rtol=1e-14)


def test_bias_update_of_the_oracle():
    b = ochoice.bias_update(np.zeros(3, np.float32), [1, 2, 3], 0.5)
    assert b.tolist() == [0.5, 0.0, -0.5]
