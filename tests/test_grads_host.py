"""Host-side checks of the gradient norm: refusals that return before any device work, and its oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from oracle.grads import norm_and_scale

P = ctypes.c_void_p(256)
ARG, UNSUP, WS = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE


def _prepare(count=1, ws=P, n_ws=1 << 20, out=True, **kw):
    f = dict(g=4096, n=16, dtype=0)
    f.update(kw)
    arr = (B.GradTensor * 1)(B.GradTensor(**f))
    return B.load().moe_grad_prepare(arr, count, ctypes.byref(B.GradList()) if out else None, ws, n_ws, None)


def test_prepare_refusals():
    assert _prepare(count=-1) == ARG and _prepare(count=4097) == ARG and _prepare(out=False) == ARG
    assert _prepare(g=None) == ARG and _prepare(n=-1) == ARG
    assert _prepare(dtype=2) == ARG and _prepare(dtype=-1) == ARG
    assert _prepare(g=4098) == ARG and _prepare(g=4097, dtype=1) == ARG         # off the element's size
    assert _prepare(n=(1 << 43) + 1) == UNSUP
    assert _prepare(n=(1 << 24) * 8192) == UNSUP
    assert _prepare(ws=None) == WS and _prepare(ws=ctypes.c_void_p(8)) == WS and _prepare(n_ws=64) == WS
    assert B.load().moe_grad_prepare(None, 1, ctypes.byref(B.GradList()), P, 1 << 20, None) == ARG
    size = B.load().moe_grad_workspace_size
    assert size(-1) == 0 and size(4097) == 0 and 0 < size(0) <= size(1) <= size(4096)


def test_norm_and_scale_refusals():
    lib = B.load()
    L = B.GradList(256, 1, 1, 1)
    norm = lambda L=L, c=True, n=P, s=P, st=P, **kw: lib.moe_grad_norm(
        ctypes.byref(L) if L else None, ctypes.byref(B.Clip(**{**dict(max_norm=1.0, mult=1.0), **kw})) if c else None,
        n, s, st, None)
    assert norm(L=None) == ARG and norm(c=False) == ARG
    assert norm(n=None) == ARG and norm(s=None) == ARG and norm(st=None) == ARG
    for bad in (dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=math.nan), dict(mult=math.inf), dict(mult=math.nan)):
        assert norm(**bad) == ARG, bad
    assert norm(L=B.GradList(None, 1, 1, 1)) == ARG and norm(L=B.GradList(256, -1, 1, 1)) == ARG
    assert norm(L=B.GradList(256, 1, 1 << 24, 1)) == ARG
    assert lib.moe_grad_scale(None, P, None) == ARG and lib.moe_grad_scale(ctypes.byref(L), None, None) == ARG
    shared = B.GradList(256, 2, 2, 0)
    assert lib.moe_grad_scale(ctypes.byref(shared), P, None) == ARG


def test_binding_refusals():
    x = torch.zeros(8)
    with pytest.raises(B.MoeError, match="current device"):
        B.make_grads([x])
    with pytest.raises(B.MoeError, match="contiguous"):
        B.make_grads([torch.zeros(4, 4).t()])
    with pytest.raises(B.MoeError):
        B.make_grads([torch.zeros(4, dtype=torch.float16)])


def test_oracle():
    assert norm_and_scale([np.array([3.0]), np.array([4.0])], 10.0) == (5.0, 1.0)
    assert norm_and_scale([np.array([3.0]), np.array([4.0])], 2.5) == (5.0, 0.5)
    assert norm_and_scale([np.array([3.0]), np.array([4.0])], 2.5, -2.0) == (10.0, -0.5)
    assert norm_and_scale([], 1.0) == (0.0, 1.0)
    n, s = norm_and_scale([np.array([np.inf])], 1.0)
    assert n == math.inf and s == 0.0
    n, s = norm_and_scale([np.array([np.nan, 1.0])], 1.0)
    assert math.isnan(n) and math.isnan(s)
