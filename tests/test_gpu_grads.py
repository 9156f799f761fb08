"""GPU parity of the gradient norm and of clipping against the 64-bit oracle.

Tolerances, u = 2^-24: the sum is made in 64 bits, where 2^32 terms lose at most 2^-20 of u, so norm and
scale are one rounding from the oracle's: u, taken as 1.001 u (below 2^-126, where fp32's numbers are 2^-149
apart, half of that: 2^-150; from 2^128 - 2^103 on, half a step above its largest number, the rounding is
infinity).  A scaled element is the rounded product of
the element and the scale as returned: the same bits."""
import math

import numpy as np
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from oracle.grads import norm_and_scale
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 1.001 * 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def _grads(sizes, kinds, seed=0, off=0, size=1e-3):
    gen = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        full = (torch.randn(n + off, generator=gen) * size).to(kinds[i % len(kinds)]).to(DEV)
        out.append(full[off:])
    return out


def _norm(grads, max_norm=1.0, mult=1.0, prepared=None):
    p = B.make_grads(grads) if prepared is None else prepared
    norm, scale = torch.full((1,), -7.0, device=DEV), torch.full((1,), -7.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.grad_norm(p, max_norm, norm, scale, status, mult)
    return p, norm, scale, status


def _close(got, want):
    got = float(got)
    want = math.inf if want >= 2.0 ** 128 - 2.0 ** 103 else want
    if math.isnan(want):
        assert math.isnan(got)
    elif math.isinf(want) or want == 0:
        assert got == want
    else:
        assert abs(got - want) <= max(U * abs(want), 2.0 ** -150), (got, want)


def _check(grads, max_norm=1.0, mult=1.0, bad=0):
    say(f"grads {len(grads)} max {max_norm} mult {mult}")
    before = [g.clone() for g in grads]
    m = float(mult) if not isinstance(mult, torch.Tensor) else float(mult.item())
    want = norm_and_scale([g.double().cpu().numpy() for g in before], max_norm, m)
    p, norm, scale, status = _norm(grads, max_norm, mult)
    _close(norm, want[0])
    _close(scale, want[1])
    assert int(status) == bad
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(grads, before))
    B.grad_scale(p, scale)
    for a, b in zip(grads, before):
        ref = b if float(scale) == 1.0 else (b.float() * scale).to(b.dtype)
        both = torch.isnan(a) & torch.isnan(ref)
        assert torch.equal(a.masked_fill(both, 0.0), ref.masked_fill(both, 0.0))
    return want


@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [8191, 8192, 8193], [3, 100_003, 1, 0, 8192 * 7], [16384 * 2000 + 5],
                                   [1 + 37 * i % 1000 for i in range(300)]])
@pytest.mark.parametrize("kinds", [(F32,), (BF16,), (F32, BF16)])
@pytest.mark.parametrize("off", [0, 1])
def test_parity(sizes, kinds, off):
    _check(_grads(sizes, kinds, off=off), max_norm=1e-3)
    _check(_grads(sizes, kinds, off=off), max_norm=1e9)


def test_the_most_tensors():
    _check(_grads([1 + i % 7 for i in range(4096)], (F32, BF16)), max_norm=0.01)
    with pytest.raises(B.MoeError):
        B.make_grads(_grads([1] * 4097, (F32,)))


def test_no_gradients():
    assert _check([]) == (0.0, 1.0)
    assert _check(_grads([0, 0], (F32,)), mult=0.5) == (0.0, 0.5)


@pytest.mark.parametrize("size", [1e-30, 1e-42, 1e30, 3e38])
def test_squares_that_32_bits_do_not_hold(size):
    g = _grads([5000, 70], (F32,), size=1.0)
    for t in g:
        t.clamp_(-1, 1).mul_(size)
    _check(g, max_norm=size)
    _check(g, max_norm=math.inf)


def test_norm_beyond_32_bits():
    """norm infinite in fp32, the scale still right, and no bad gradient."""
    g = [torch.full((1 << 20,), 3e38, device=DEV)]
    want = _check(g, max_norm=1.0)
    assert want[0] < math.inf
    _, norm, _, status = _norm([torch.full((1 << 20,), 3e38, device=DEV)])
    assert float(norm) == math.inf and int(status) == 0


@pytest.mark.parametrize("mult", [0.0, -2.0, 0.25, 65536.0])
def test_mult(mult):
    for on_device in (False, True):
        m = torch.tensor([mult], device=DEV) if on_device else mult
        _check(_grads([1000, 77], (F32, BF16), size=1.0), max_norm=3.0, mult=m)


def test_one_rounding_below_and_at_the_limit():
    g = [torch.tensor([3.0, 4.0], device=DEV)]
    assert _check(g, max_norm=5.0) == (5.0, 1.0)
    _check(g, max_norm=float(np.nextafter(5.0, 0)))
    _check(g, max_norm=4.9999)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("kind", [F32, BF16])
def test_gradients_that_are_not_finite(value, kind):
    g = _grads([9000, 17], (kind,))
    g[1][16] = value
    _check(g, bad=B.DEV_BAD_GRAD)
    _check(g, max_norm=math.inf, bad=B.DEV_BAD_GRAD)


def test_shared_gradients():
    """A gradient listed twice counts twice; such a list is not scaled in place."""
    g = torch.randn(1000, device=DEV)
    p, norm, scale, _ = _norm([g, g, g[10:20]])
    want = math.sqrt(2 * float(g.double().square().sum()) + float(g[10:20].double().square().sum()))
    _close(norm, want)
    with pytest.raises(B.MoeError, match="argument"):
        B.grad_scale(p, scale)
    halves = [g[:500], g[500:]]
    p, _, scale, _ = _norm(halves)
    B.grad_scale(p, scale)                     # side by side is apart


def test_past_32_bit_offsets():
    n = (1 << 32) + 8195
    g = torch.ones(n, dtype=BF16, device=DEV)
    g[-1] = 65536.0
    p, norm, scale, _ = _norm([g], max_norm=1e9)
    _close(norm, math.sqrt(n - 1 + 65536.0 ** 2))
    scale.fill_(2.0)
    B.grad_scale(p, scale)
    assert float(g[-1]) == 131072.0 and float(g[-2]) == 2.0 and float(g[0]) == 2.0 and float(g[1 << 31]) == 2.0
    _, norm, _, _ = _norm([g], max_norm=1e9)
    _close(norm, 2 * math.sqrt(n - 1 + 65536.0 ** 2))


def test_same_bits_at_every_call_and_rows_around_untouched():
    full = torch.randn(100_000, device=DEV)
    g = [full[3:50_001], full[60_000:99_999]]
    before = full.clone()
    p, norm, scale, _ = _norm(g, max_norm=0.1)
    for _ in range(5):
        _, n2, s2, _ = _norm(g, max_norm=0.1, prepared=p)
        assert torch.equal(n2, norm) and torch.equal(s2, scale)
    B.grad_scale(p, scale)
    for a, b in ((0, 3), (50_001, 60_000), (99_999, 100_000)):
        assert torch.equal(full[a:b], before[a:b])
    assert not torch.equal(full[3:50_001], before[3:50_001])


def test_captured_and_on_another_stream():
    """A graph of the norm, the scaling and AdamW, replayed between eager calls on the same list."""
    g = _grads([5000, 20_001, 3], (F32,), size=1.0)
    start = [t.clone() for t in g]
    p = B.make_grads(g)
    norm, scale = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mult = torch.ones(1, device=DEV)

    def both():
        B.grad_norm(p, 0.5, norm, scale, status, mult)
        B.grad_scale(p, scale)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for turn in range(4):
        m = 1.0 + turn
        want = norm_and_scale([t.double().cpu().numpy() for t in start], 0.5, m)
        for eager in (False, True):
            for a, b in zip(g, start):
                a.copy_(b)
            mult.fill_(m)
            norm.zero_()
            both() if eager else graph.replay()
            torch.cuda.synchronize()
            _close(norm, want[0])
            _close(scale, want[1])
            assert all(torch.equal(a, b * scale) for a, b in zip(g, start))


def test_two_lists_on_two_streams():
    a, b = _grads([400_000], (F32,), 1), _grads([300_000], (BF16,), 2)
    want = [norm_and_scale([t.double().cpu().numpy() for t in x], 1.0)[0] for x in (a, b)]
    lists = [B.make_grads(x) for x in (a, b)]
    outs = [[torch.zeros(1, device=DEV) for _ in range(2)] for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, p, o in zip(streams, lists, outs):
            with torch.cuda.stream(s):
                B.grad_norm(p, 1.0, o[0], o[1], status)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        _close(o[0], w)


@pytest.mark.parametrize("grad_scale", [None, 0.5, "device"])
def test_block_step_clipped(grad_scale):
    """BlockRunner.optimizer_step with max_norm: the step of gradients scaled by the norm's factor."""
    from tests.test_gpu_block import PATHS, _block
    results = []
    for max_norm in (1e-2, None):
        b, par, x, dout = _block(PATHS["small_f32"], 150, 3, "softmax", True)
        b.block_forward(x)
        b.block_backward(dout)
        b.make_optimizer()
        gs = torch.tensor([0.5], device=DEV) if grad_scale == "device" else grad_scale
        m = 1.0 if grad_scale is None else 0.5
        g = [b.dw1, b.dw2, b.dw_router, b.dw_in, b.dw_out, b.dgate]
        want = norm_and_scale([t.double().cpu().numpy() for t in g], 1e-2, m)
        assert want[0] > 1e-2
        if max_norm is not None:
            b.optimizer_step(1e-3, 1, max_norm=max_norm, grad_scale=gs)
            _close(b.grad_norm, want[0])
        else:
            b.optimizer_step(1e-3, 1, grad_scale=torch.tensor([want[1]], dtype=F32, device=DEV))
        torch.cuda.synchronize()
        results.append([t.clone() for t in (*par.values(), *b.state["m"], *b.state["v"])])
    # the scales are the same to a rounding: m to 2 u, v to 4 u, p's update to 6 u and its own roundings
    for i, (a, b) in enumerate(zip(*results)):
        assert torch.allclose(a, b, rtol=2.0 ** -21, atol=2.0 ** -21 * 1e-3)
