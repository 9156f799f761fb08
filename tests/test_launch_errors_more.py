"""Host side, as tests/test_launch_errors.py: an error of any launch of the int8 layer, the router's choice by values,
the quantizer and the gradients' norm is reported.  Nothing reaches a GPU."""
import os
import subprocess
import sys

import pytest

from tests.test_launch_errors import ROOT, shim  # noqa: F401

RUN = r"""
import ctypes, sys
shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
from moe_expert_ffn_amd import binding as B
lib = B.load()
P = ctypes.c_void_p(256)
def layer(T, d, f):
    L = B.Layer(8, d, f, B.MOE_BF16, B.MOE_INT8, 256, 256, 256, 256)
    return lambda: lib.moe_forward(ctypes.byref(L), P, P, P, T, 2, 128, 4, P, P, P, P, P, P, None, P, P, 1 << 40, 0, None, None, None)
R, C = B.Router(64, 4, 0, 1, 1, 1.0), B.Choice(256, 8, 4, 1)
G = B.GradList(256, 1, 5, 1)
many = (B.GradTensor * 200)(*[B.GradTensor(4096 * (i + 1), 16, 0) for i in range(200)])
calls = {
    "few": (layer(5, 384, 192), 5), "wide": (layer(700, 512, 256), 5),
    "choice": (lambda: lib.moe_router_forward_choice(ctypes.byref(R), ctypes.byref(C), P, 64, None, 500, P, P, P, P, P, P, P, P,
                                                     1 << 30, None), 2),
    "bias": (lambda: lib.moe_router_bias_update(P, 64, 0.1, P, None), 1),
    "rows": (lambda: lib.moe_quantize_int8_rows(P, 64, 0, 5, 64, ctypes.c_void_p(1 << 16),
                                                ctypes.c_void_p(1 << 20), None), 1),
    "prepare": (lambda: lib.moe_grad_prepare(many, 200, ctypes.byref(B.GradList()), P, 1 << 20, None), 3),
    "norm": (lambda: lib.moe_grad_norm(ctypes.byref(G), ctypes.byref(B.Clip(1.0, 1.0, None)), P, P, P, None), 1),
    "scale": (lambda: lib.moe_grad_scale(ctypes.byref(G), P, None), 1)}
once, least = calls[sys.argv[3]]
shim.shim_start(0)
assert once() == B.MOE_OK, once()
n = shim.shim_seen()
assert n >= least, n
lost = []
for i in range(1, n + 1):
    shim.shim_start(i)
    if once() != B.MOE_ERR_HIP:
        lost.append(i)
assert not lost, f"launches {lost} of {n} failed unnoticed"
shim.shim_start(0)
assert once() == B.MOE_OK
"""


@pytest.mark.parametrize("call", ["few", "wide", "choice", "bias", "rows", "prepare", "norm", "scale"])
def test_failed_launches(shim, call):  # noqa: F811
    r = subprocess.run([sys.executable, "-c", RUN, shim, ROOT, call], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
