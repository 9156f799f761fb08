"""Oracle: AdamW with fp32 states or e4m3 states -- TEST INFRASTRUCTURE ONLY.

    m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2
    p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
in fp64.  8-bit states hold m and sqrt(v) in blocks of 128 as e4m3 codes times
a scale, the block's largest finite magnitude over 448, rounded up with the
probability of the part cut off, a sqrt(v) under an m that is not 0 to the code
1 at least; the random words are a hash of the seed, the step, the tensor's
place in its list and the element's index.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
GOLD, ROOT2, ROOT3 = 0x9E3779B9, 0x6A09E667, 0xBB67AE85
_M = 0xFFFFFFFF


def _mix(x):
    x = x ^ (x >> 16)
    x = (x * ROOT2) & _M
    return x ^ (x >> 15)


def words(seed, step, tensor, n, start=0):
    """Of elements start .. start + n."""
    key = _mix((seed + step * GOLD + tensor * ROOT3) & _M)
    i = np.arange(start, start + n, dtype=np.uint64)
    x = (i * np.uint64(GOLD) + np.uint64(key)) & np.uint64(_M)
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(ROOT2)) & np.uint64(_M)
    return (x ^ (x >> np.uint64(15))).astype(np.int64)


def step(p, g, m, v, t, lr, b1, b2, eps, wd):
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    with np.errstate(invalid="ignore"):
        p = p * (1 - lr * wd) - lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return p, m, v


def decode(codes, scales):
    c = np.asarray(codes).astype(np.int64)
    e, f = (c >> 3) & 15, c & 7
    mag = np.where(e > 0, np.ldexp(1.0 + f / 8.0, e - 7), f / 512.0)
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c & 128, -mag, mag) * np.repeat(np.asarray(scales, dtype=np.float64), BLOCK)[:c.size]


def block_tops(x):
    n = x.size
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    a = np.concatenate([a, np.zeros(-n % BLOCK)]).reshape(-1, BLOCK).max(1)
    return np.where(a < 2.0 ** -100, 0.0, a)


def under_m(m_codes, m_scales, v_scales, b1, b2):
    """Where a sqrt(v) of code 0 becomes 1: m's code is not 0 and no more than gradients give with a sqrt(v) below a
    code step, |m| <= C sqrt(v) by Cauchy-Schwarz (twice, for the rounding of larger codes), and five deviations of
    m's own rounding.  (Which of them, the limit in m's code units)."""
    C = (1 - b1) / np.sqrt((1 - b2) * (1 - b1 * b1 / b2)) if b1 * b1 < b2 else np.inf
    with np.errstate(divide="ignore", invalid="ignore"):
        most = 2 * C / 512 * (v_scales / m_scales) + 2.5 / np.sqrt(1 - b1 * b1) / 512
    most = np.minimum(np.where((v_scales > 0) & (m_scales > 0), most, 0.0), 480.0)      # above every code but NaN's
    most = np.repeat(most, BLOCK)[:m_codes.size]
    mag = np.abs(decode(m_codes, np.ones(m_scales.size)))
    return (mag > 0) & (mag <= most), most


def encode(x, u16, m=None):
    """(codes, scales, distance): distance of the sum that is cut to the next whole number, in code
    steps -- where it is within the arithmetic's error, the neighbouring code is right as well.
    m: of x = sqrt(v), (m's codes, m's scales, b1, b2).  Without it the codes of 0 of an x that has no negative
    element, which may be such roots, have a distance of 0: the code 1 may be right too."""
    top = block_tops(x)
    per = np.repeat(top, BLOCK)[:x.size]
    fin = np.isfinite(x)
    y = np.where(per > 0, np.abs(np.where(fin, x, 0.0)) * 448 / np.where(per > 0, per, 1.0), 0.0)
    ex = np.clip(np.floor(np.log2(np.maximum(y, 2.0 ** -20))), -6, 8).astype(np.int64)
    s = np.ldexp(y, 3 - ex) + (u16 + 0.5) / 65536
    code = np.minimum((ex + 6) * 8 + np.floor(s).astype(np.int64), 126)
    dist = np.abs(s - np.round(s))
    if m is not None:
        code = np.maximum(code, under_m(*m[:2], top / 448, *m[2:])[0])
    elif not (x < 0).any():
        dist = np.where((code == 0) & (y > 0), 0.0, dist)
    code = np.where(fin, code, 127) | np.where(x < 0, 128, 0)
    return code.astype(np.uint8), top / 448, dist


def random_bf16(p, word):
    """fp32 values rounded to bf16 at random by the high half of word * ROOT3."""
    b = np.asarray(p, dtype=np.float32).view(np.uint32).astype(np.int64)
    up = ((b + (((word * ROOT3) & _M) >> 16)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(p), up, p)
