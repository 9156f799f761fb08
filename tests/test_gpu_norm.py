"""GPU parity of the norms before and after a block, forward and backward, against the fp64 oracle.

Tolerances, u = 2^-24: a row's sum of squares is added by threads of at most 32 terms and a tree of
10 levels (42 u relative, half of it in 1/rms), rows are rounded once on the way out (half a step
of their type), r once more in 32 bits before it enters the norm.  A sum over a row of signed terms
is off by 42 u of the sum of their magnitudes, one over T tokens by T / 256 + 40 such steps."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from oracle import norm as onorm
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
EPS = 1e-6


def _rows(rng, T, d, dtype, pad=0, off=0, big=False):
    if big:                                                       # only the rows are written
        out = torch.empty((T, d + pad), dtype=dtype, device=DEV)[:, off:off + d]
        return out.copy_(_rows(rng, T, d, dtype))
    full = torch.from_numpy(rng.standard_normal((T, d + pad)).astype(np.float32)).to(dtype).to(DEV)
    return full[:, off:off + d]


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _gate(rng, kind, T, d):
    if kind == "none":
        return None
    g = rng.standard_normal((T, 1) if kind == "token" else d).astype(np.float32)
    g.reshape(-1)[:1] = 0.0                                       # a closed gate
    return torch.from_numpy(g).to(DEV)


def _close(name, got, ref, tol):
    got = _f64(got)
    worst = np.max(np.abs(got - ref) / (tol + 1e-37), initial=0.0)
    assert worst <= 1.0, f"{name}: {worst:.2f} times the tolerance"


SHAPES = [(1, 1), (3000, 2), (2100, 5), (1500, 9), (700, 17), (1025, 31), (1, 2048), (1, 7168), (2, 7), (5, 64), (3, 65), (9, 512), (4, 513), (17, 1000), (300, 1023),
          (1030, 128), (40, 2048), (21, 2056), (13, 4096), (6, 4104), (7, 7168), (5, 8200), (3, 16384),
          (2, 16381), (0, 64)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("dtype,wide", [(torch.float32, True), (torch.bfloat16, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("kind", ["none", "token", "feature"])
def test_norm_in(T, d, dtype, wide, kind):
    _norm_in(T, d, dtype, wide, kind)


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("dtype,wide", [(torch.float32, True), (torch.bfloat16, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("kind", ["none", "token", "feature"])
def test_norm_out(T, d, dtype, wide, kind):
    _norm_out(T, d, dtype, wide, kind)


def _norm_in(T, d, dtype, wide, kind, pad=0, off=0, residual=True, big=False):
    say(f"[norm_in] T={T} d={d} {dtype} w32={wide} gate={kind} pad={pad} residual={residual}")
    rng = np.random.default_rng(T * 17 + d)
    x, dn, dr = (_rows(rng, T, d, dtype, pad, off, big) for _ in range(3))
    u = _rows(rng, T, d, dtype, pad, off, big) if residual else None
    w = torch.from_numpy(rng.standard_normal(d).astype(np.float32)).to(DEV)
    w = w if wide else w.to(dtype)
    g, alpha, half = _gate(rng, kind, T, d) if residual else None, 0.7, HALF[dtype]
    new = lambda: _rows(rng, T, d, dtype, pad, off, big)
    n, r, rstd = new(), new() if residual else None, torch.full((T,), 9.0, device=DEV)
    B.norm_in(x, w, EPS, n, rstd, u=u, gate=g, alpha=alpha, r=r)
    torch.cuda.synchronize()
    a32 = float(np.float32(alpha))
    X, Un, W, G = _f64(x), _f64(u), _f64(w), _f64(g)
    R, N, S = onorm.norm_in(X, W, float(np.float32(EPS)), Un, G, a32)
    gu = 0.0 if u is None else np.abs((a32 if G is None else a32 * G) * Un)
    dR = 4 * U * (np.abs(X) + gu)                                 # r's own error in 32 bits
    # r's error reaches 1/rms as a mean of r dr / rms^2
    relS = 30 * U + np.abs(dR * R).mean(1) * S * S
    _close("rstd", rstd, S, relS * S)
    _close("n", n, N, np.abs(W) * S[:, None] * dR + np.abs(N) * (relS[:, None] + 6 * U + half * 1.01))
    if r is not None:
        _close("r", r, R, dR + half * 1.01 * np.abs(R))

    src = r if r is not None else x
    dx, du = new(), new() if residual else None
    dw = torch.full((d,), 9.0, device=DEV)
    dg = None if g is None else torch.full_like(g, 9.0)
    ws = B.norm_workspace(T, d, DEV)
    ws.fill_(0xAB)
    B.norm_in_backward(dn, src, w, rstd, dx, dw, ws, dr=dr if residual else None, u=u, gate=g,
                       alpha=alpha, du=du, dgate=dg)
    torch.cuda.synchronize()
    Rs, S, D = _f64(src), _f64(rstd), _f64(dn)
    DX, DW, DU, DG = onorm.norm_in_backward(D, Rs, W, S, _f64(dr) if residual else None, Un, G, a32)
    xh = np.abs(Rs) * S[:, None]
    a = np.abs(D * W)
    big = S[:, None] * (a + xh * (a * xh).mean(1, keepdims=True)) + (np.abs(_f64(dr)) if residual else 0)
    eDX = 56 * U * big
    _close("dx", dx, DX, eDX + half * 1.01 * np.abs(DX))
    many = (T / 256 + 40) * U
    _close("dw", dw, DW, many * (np.abs(D) * xh).sum(0))
    if residual:
        k = np.abs(a32 if G is None else a32 * G)
        _close("du", du, DU, k * (eDX + 4 * U * np.abs(DX)) + half * 1.01 * np.abs(DU))
    if g is not None:
        axis = dict(axis=1, keepdims=True) if kind == "token" else dict(axis=0)
        _close("dgate", dg, DG, a32 * (np.abs(Un) * (eDX + (many + 44 * U) * np.abs(DX))).sum(**axis))


def _norm_out(T, d, dtype, wide, kind, pad=0, off=0, big=False):
    say(f"[norm_out] T={T} d={d} {dtype} w32={wide} gate={kind} pad={pad}")
    rng = np.random.default_rng(T * 13 + d)
    y, x, do = (_rows(rng, T, d, dtype, pad, off, big) for _ in range(3))
    w = torch.from_numpy(rng.standard_normal(d).astype(np.float32)).to(DEV)
    w = w if wide else w.to(dtype)
    g, alpha, half = _gate(rng, kind, T, d), -1.3, HALF[dtype]
    new = lambda: _rows(rng, T, d, dtype, pad, off, big)
    out, rstd = new(), torch.full((T,), 9.0, device=DEV)
    B.norm_out(y, x, w, EPS, out, rstd, gate=g, alpha=alpha)
    torch.cuda.synchronize()
    a32 = float(np.float32(alpha))
    Y, X, W, G = _f64(y), _f64(x), _f64(w), _f64(g)
    O, S = onorm.norm_out(Y, X, W, float(np.float32(EPS)), G, a32)
    _close("rstd", rstd, S, 30 * U * S)
    _close("out", out, O, 38 * U * np.abs(O - X) + 2 * U * np.abs(O) + half * 1.01 * np.abs(O))

    dy, dw = new(), torch.full((d,), 9.0, device=DEV)
    dg = None if g is None else torch.full_like(g, 9.0)
    ws = B.norm_workspace(T, d, DEV)
    ws.fill_(0xAB)
    B.norm_out_backward(do, y, w, rstd, dy, dw, ws, gate=g, alpha=alpha, dgate=dg)
    torch.cuda.synchronize()
    S, D = _f64(rstd), _f64(do)
    DY, DW, DG = onorm.norm_out_backward(D, Y, W, S, G, a32)
    yh = np.abs(Y) * S[:, None]
    dv = np.abs(D * (a32 if G is None else a32 * G))
    a = dv * np.abs(W)
    big = S[:, None] * (a + yh * (a * yh).mean(1, keepdims=True))
    _close("dy", dy, DY, 56 * U * big + half * 1.01 * np.abs(DY))
    many = (T / 256 + 40) * U
    _close("dw", dw, DW, (many + 4 * U) * (dv * yh).sum(0))
    if g is not None:
        axis = dict(axis=1, keepdims=True) if kind == "token" else dict(axis=0)
        _close("dgate", dg, DG, (many + 48 * U) * abs(a32) * (np.abs(D * W) * yh).sum(**axis))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d,pad,off", [(33, 128, 8, 0), (33, 128, 8, 8), (33, 128, 3, 1), (9, 2048, 1, 1),
                                         (1, 64, 5, 3), (12, 7168, 16, 8)])
def test_norms_of_strided_rows(dtype, T, d, pad, off):
    _norm_in(T, d, dtype, False, "feature", pad, off)
    _norm_out(T, d, dtype, False, "token", pad, off)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_in_without_residual(dtype):
    for T, d in ((1, 1), (50, 2048), (700, 96), (3, 7168)):
        _norm_in(T, d, dtype, True, "none", residual=False)


def test_many_tokens():
    _norm_in(20011, 64, torch.bfloat16, False, "feature")
    _norm_out(9001, 512, torch.float32, True, "token")


def test_offsets_past_32_bits():
    """Rows far apart in buffers of more than 2^32 bytes."""
    say("[norm-far]")
    _norm_in(600, 129, torch.bfloat16, True, "feature", pad=4_000_000, off=7, big=True)
    _norm_out(600, 129, torch.bfloat16, True, "token", pad=4_000_000, off=7, big=True)


def test_zero_rows_and_rows_that_are_not_finite_stay_alone():
    say("[norm-odd]")
    T, d = 6, 256
    rng = np.random.default_rng(1)
    x, u = _rows(rng, T, d, torch.float32), _rows(rng, T, d, torch.float32)
    x[0] = 0
    u[0] = 0
    w = torch.ones(d, device=DEV)
    n, rstd = torch.empty_like(x), torch.empty(T, device=DEV)
    B.norm_in(x, w, EPS, n, rstd, u=u)
    clean = n.clone()
    x[2, 5] = float("nan")
    x[4, 7] = float("inf")
    B.norm_in(x, w, EPS, n, rstd, u=u)
    torch.cuda.synchronize()
    assert (n[0] == 0).all() and abs(float(rstd[0]) * EPS ** 0.5 - 1) < 1e-6
    assert n[2].isnan().all()
    for t in (0, 1, 3, 5):
        assert torch.equal(n[t], clean[t])
    ws, dw = B.norm_workspace(T, d, DEV), torch.empty(d, device=DEV)
    do = _rows(rng, T, d, torch.float32)
    B.norm_in(x.nan_to_num(0, 0), w, EPS, n, rstd)
    r = x.nan_to_num(0, 0)
    dx, dx2 = torch.empty_like(x), torch.empty_like(x)
    B.norm_in_backward(do, r, w, rstd, dx, dw, ws)
    do[3, 9] = float("nan")
    B.norm_in_backward(do, r, w, rstd, dx2, dw, ws)
    torch.cuda.synchronize()
    assert dx2[3].isnan().all() and dw[9].isnan() and not dw[:9].isnan().any()
    for t in (0, 1, 2, 4, 5):
        assert torch.equal(dx[t], dx2[t])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [3, 96, 509, 2047, 7168, 8199, 12001])
def test_norms_in_place_repeat_and_replay(dtype, d):
    say(f"[norm-inplace] {dtype} d={d}")
    T = 700
    rng = np.random.default_rng(d)
    x, u, do = (_rows(rng, T, d, dtype) for _ in range(3))
    w, g = torch.randn(d, device=DEV), torch.randn(d, device=DEV)
    n, r, dx, du, out, dy = (torch.empty_like(x) for _ in range(6))
    rstd, dw, dg = torch.empty(T, device=DEV), torch.empty(d, device=DEV), torch.empty(d, device=DEV)
    ws = B.norm_workspace(T, d, DEV)
    B.norm_in(x, w, EPS, n, rstd, u=u, gate=g, alpha=0.5, r=r)
    # r over x, n over u
    xa, ua, rs = x.clone(), u.clone(), torch.empty_like(rstd)
    B.norm_in(xa, w, EPS, ua, rs, u=ua, gate=g, alpha=0.5, r=xa)
    torch.cuda.synchronize()
    assert torch.equal(xa, r) and torch.equal(ua, n) and torch.equal(rs, rstd)
    B.norm_in_backward(do, r, w, rstd, dx, dw, ws, dr=do, u=u, gate=g, alpha=0.5, du=du, dgate=dg)
    da, ub, dw2, dg2 = do.clone(), u.clone(), torch.empty_like(dw), torch.empty_like(dg)
    B.norm_in_backward(da, r, w, rstd, da, dw2, ws, dr=do, u=ub, gate=g, alpha=0.5, du=ub, dgate=dg2)
    torch.cuda.synchronize()
    for a, b in ((da, dx), (ub, du), (dw2, dw), (dg2, dg)):
        assert torch.equal(a, b)

    def both():
        B.norm_out(u, x, w, EPS, out, rstd, gate=g, alpha=0.5)
        B.norm_out_backward(do, u, w, rstd, dy, dw, ws, gate=g, alpha=0.5, dgate=dg)

    def outs():
        torch.cuda.synchronize()
        return [t.clone() for t in (out, rstd, dy, dw, dg)]

    both()
    ref = outs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    for a, b in zip(outs(), ref):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for rep in range(3):
        for t in (out, rstd, dy, dw, dg):
            t.zero_()
        graph.replay()
        for a, b in zip(outs(), ref):
            assert torch.equal(a, b), rep
        both()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["none", "token", "feature"])
@pytest.mark.parametrize("T,d", [(1, 8), (50, 5), (700, 96), (37, 509), (300, 2047), (9, 8199), (5, 12001)])
def test_padding_rows_hold_anything(dtype, kind, T, d):
    """NaN in every input of the padding rows: they pass the stream alone, the other rows and the sums
    over tokens are, bit for bit, those of the same rows with zeros as padding."""
    say(f"[norm-padding] {dtype} gate={kind} T={T} d={d}")
    rng = np.random.default_rng(T + d)
    mask = torch.ones(T, dtype=torch.bool, device=DEV)
    mask[::3] = False
    x, u, do, dr = (_rows(rng, T, d, dtype) for _ in range(4))
    for t in (u, do):
        t[~mask] = 0
    fill = lambda t: t.masked_fill(~mask[:, None], float("nan"))
    g = _gate(rng, kind, T, d)
    gn = fill(g) if kind == "token" else g
    w = torch.randn(d, device=DEV)
    ws = B.norm_workspace(T, d, DEV)
    rows = lambda: torch.full_like(x, 7)
    vec = lambda n: torch.full((n,), 7.0, device=DEV)

    def all_of(x, u, do, dr, g, y, mask):
        n, r, dx, du, out, dy = (rows() for _ in range(6))
        s, s2, dw, dw2 = vec(T), vec(T), vec(d), vec(d)
        dg = dg2 = None
        if g is not None:
            dg, dg2 = torch.full_like(g, 7), torch.full_like(g, 7)
        B.norm_in(x, w, EPS, n, s, u=u, gate=g, alpha=0.7, r=r, mask=mask)
        B.norm_in_backward(do, r, w, s, dx, dw, ws, dr=dr, u=u, gate=g, alpha=0.7, du=du, dgate=dg,
                           mask=mask)
        B.norm_out(y, x, w, EPS, out, s2, gate=g, alpha=0.7, mask=mask)
        B.norm_out_backward(do, y, w, s2, dy, dw2, ws, gate=g, alpha=0.7, dgate=dg2, mask=mask)
        torch.cuda.synchronize()
        return dict(n=n, r=r, s=s, dx=dx, du=du, out=out, dy=dy, s2=s2, dw=dw, dw2=dw2, dg=dg, dg2=dg2)

    got = all_of(fill(x), fill(u), fill(do), dr, gn, fill(u), mask.to(torch.uint8))
    ref = all_of(x, u, do, dr, g, u, None)
    off = ~mask
    assert got["r"][off].isnan().all() and got["out"][off].isnan().all()      # x's own
    assert torch.equal(got["dx"][off], dr[off])
    for key in ("n", "du", "dy", "s", "s2"):
        assert not got[key][off].any(), key
    for key in ("n", "r", "s", "dx", "du", "out", "dy", "s2"):
        assert torch.equal(got[key][mask], ref[key][mask]), key
    # zeros add nothing to dw and dgate but to dgate before the block, which takes dr: u is 0 there
    for key in ("dw", "dw2", "dg", "dg2"):
        if ref[key] is not None:
            assert torch.equal(got[key], ref[key]), key


def test_padding_mask_is_checked():
    x, w, s = torch.zeros((4, 8), device=DEV), torch.ones(8, device=DEV), torch.zeros(4, device=DEV)
    for mask in (torch.ones(3, dtype=torch.uint8, device=DEV), torch.ones(4, device=DEV),
                 torch.ones(4, dtype=torch.uint8)):
        with pytest.raises(B.MoeError):
            B.norm_in(x, w, EPS, x.clone(), s, mask=mask)
        with pytest.raises(B.MoeError):
            B.norm_out_backward(x, x, w, s, x.clone(), w.clone(), B.norm_workspace(4, 8, DEV), mask=mask)
