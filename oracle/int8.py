"""Oracle: 8-bit integer rows and the expert layer with int8 weights -- TEST INFRASTRUCTURE ONLY.

A row's scale is max|v| / 127 and its codes the nearest whole numbers to 127 v / max|v|, half to even (exact
rational arithmetic through whole numbers next to a half); rows below 2^-100 are zeros, rows that are not
finite have a scale of NaN and codes of 0.  The layer: x rows quantized, [G, U] from the codes' products and the
scales, A = SiLU(G) U rounded to bf16, quantized again, O likewise, gated and summed.  fp64 elsewhere."""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from oracle.ffn import _pairs_by_expert, round_bf16, silu


def quantize_rows(v):
    v = np.asarray(v, dtype=np.float64)
    codes, scales = np.zeros(v.shape, dtype=np.int8), np.zeros(len(v), dtype=np.float32)
    for r, row in enumerate(v):
        if not np.isfinite(row).all():
            scales[r] = np.nan
            continue
        amax = np.abs(row).max() if row.size else 0.0
        if amax < 2.0 ** -100:
            continue
        scales[r] = np.float32(amax) / np.float32(127)
        t = row / amax * 127.0
        c = np.rint(t)
        for i in np.nonzero(np.abs(np.abs(t - np.trunc(t)) - 0.5) < 1e-9)[0]:
            c[i] = round(Fraction(float(row[i])) * 127 / Fraction(float(amax)))     # half to even
        codes[r] = c
    return codes, scales


def forward(x, w1, s1, w2, s2, ids, gates):
    """y [T][d] of bf16 x; w1, w2 codes, s1 [E][2 d_ff], s2 [E][d]."""
    x = np.asarray(x, dtype=np.float64)
    F = w1.shape[1] // 2
    y = np.zeros(x.shape)
    cx, sx = quantize_rows(x)
    for e, (t, j) in _pairs_by_expert(np.asarray(ids), np.arange(len(x))).items():
        z = (cx[t].astype(np.float64) @ w1[e].astype(np.float64).T) * sx[t].astype(np.float64)[:, None] * \
            s1[e].astype(np.float64)
        with np.errstate(over="ignore"):
            a = round_bf16(silu(z[:, :F]) * z[:, F:])
        ca, sa = quantize_rows(a)
        o = (ca.astype(np.float64) @ w2[e].astype(np.float64).T) * sa.astype(np.float64)[:, None] * \
            s2[e].astype(np.float64)
        np.add.at(y, t, o * gates[t, j].astype(np.float64)[:, None])
    return y
