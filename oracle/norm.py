"""Oracle: norms before and after a block with gate and residual scale -- TEST INFRASTRUCTURE ONLY.

    before:  r = x + alpha g u,  n = w r / rms(r)
    after:   out = x + alpha g w y / rms(y)
rms(v) = sqrt(mean(v^2) + eps) over the features; g is None, [T, 1] or [d].
fp64; the gradients take the saved 1 / rms as given.
"""
from __future__ import annotations

import numpy as np


def _g(gate, alpha):
    return alpha if gate is None else alpha * gate


def norm_in(x, w, eps, u=None, gate=None, alpha=1.0):
    r = x if u is None else x + _g(gate, alpha) * u
    rstd = 1.0 / np.sqrt((r * r).mean(1) + eps)
    return r, w * r * rstd[:, None], rstd


def norm_out(y, x, w, eps, gate=None, alpha=1.0):
    rstd = 1.0 / np.sqrt((y * y).mean(1) + eps)
    return x + _g(gate, alpha) * w * y * rstd[:, None], rstd


def _through(dv, v, w, rstd):
    vh = v * rstd[:, None]
    a = dv * w
    return rstd[:, None] * (a - vh * (a * vh).mean(1, keepdims=True)), (dv * vh).sum(0)


def _gate_grad(each, gate):
    if gate is None:
        return None
    return each.sum(1, keepdims=True) if gate.ndim == 2 else each.sum(0)


def norm_in_backward(dn, r, w, rstd, dr=None, u=None, gate=None, alpha=1.0):
    dx, dw = _through(dn, r, w, rstd)
    if dr is not None:
        dx = dx + dr
    if u is None:
        return dx, dw, None, None
    return dx, dw, _g(gate, alpha) * dx, _gate_grad(alpha * u * dx, gate)


def norm_out_backward(dout, y, w, rstd, gate=None, alpha=1.0):
    dy, dw = _through(_g(gate, alpha) * dout, y, w, rstd)
    return dy, dw, _gate_grad(alpha * dout * w * y * rstd[:, None], gate)
