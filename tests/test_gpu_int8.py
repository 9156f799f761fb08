"""GPU parity of int8 rows and of the expert layer with int8 weights against the oracle.

Rows: codes are those of the real numbers, scales one fp32 division (the same bits).  Layer, relative to the
output's norm: a contribution p O is stored in bf16 and their sum is rounded again, 2^-8 each at most; the
fp32 arithmetic of a product (sums are whole numbers, six roundings around them) moves an A that lies within
2^-21 of a bf16 rounding's border by a step, and a row's largest A with its scale by 2^-7, each for some
2^-12 of the values: 2^-9 covers them.  So 2^-7 + 2^-9."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from moe_expert_ffn_amd.inputs import contiguous_owners
from moe_expert_ffn_amd.runner import LayerRunner
from oracle import int8 as oi8
from tests.conftest import rel_l2
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
TOL = 2.0 ** -7 + 2.0 ** -9


def _rows(src, pad_codes=True):
    rows, cols = src.shape
    full = torch.full((rows * cols + 64,), 77, dtype=torch.int8, device=DEV)
    scales = torch.full((rows + 2,), -1.0, device=DEV)
    B.quantize_int8_rows(src, full[:rows * cols], scales[:rows])
    torch.cuda.synchronize()
    assert (full[rows * cols:] == 77).all() and (scales[rows:] == -1).all()
    return full[:rows * cols].reshape(rows, cols).cpu().numpy(), scales[:rows].cpu().numpy()


def _check_rows(src):
    codes, scales = _rows(src)
    c, s = oi8.quantize_rows(src.double().cpu().numpy())
    np.testing.assert_array_equal(scales, s)
    np.testing.assert_array_equal(codes, c)


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (70, 64), (33, 513), (20, 2048), (9, 2049), (6, 8192),
                                       (5, 8195), (3, 20011), (1, 131072), (2500, 130)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
def test_rows(rows, cols, dtype, pad, offset):
    say(f"[rows] {rows} x {cols} {dtype} pad {pad}")
    gen = torch.Generator(device=DEV)
    gen.manual_seed(rows * 7 + cols)
    full = torch.randn((rows, cols + pad), generator=gen, device=DEV).to(dtype)
    src = full[:, offset:offset + cols]
    src[::3] *= 100
    _check_rows(src)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [254, 600, 2100])
def test_halves(dtype, cols):
    """Values whose code lies on a half, a rounding above it and one below, for many largest values."""
    gen = np.random.default_rng(cols)
    rows = []
    for k in range(60):
        amax = float(torch.tensor(1 + gen.random()).to(dtype)) * 2.0 ** (k % 40 - 20)
        half = torch.tensor(amax * (gen.integers(0, 127, cols) + 0.5) / 127, dtype=torch.float64).to(dtype)
        bits = half.view(torch.int16 if dtype == BF16 else torch.int32)
        bits += torch.from_numpy(gen.integers(-1, 2, cols)).to(bits.dtype)
        half[gen.random(cols) < 0.1] = amax / 2                           # exactly 63.5
        row = half * torch.from_numpy(gen.integers(0, 2, cols) * 2 - 1).to(dtype)
        row = row.clamp(-amax, amax)
        row[k % cols] = amax
        rows.append(row)
    _check_rows(torch.stack(rows).to(DEV))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_extremes(dtype):
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    rows = [[0.0] * 9, [big, -big, big / 2, big / 254, 1.0, 0, 0, 0, 0], [tiny] * 9, [2.0 ** -100] + [2.0 ** -107] * 8,
            [2.0 ** -101] * 9, [float("inf")] + [1.0] * 8, [1.0] * 8 + [float("nan")], [-float("inf")] * 9,
            [2.0 ** 64] + [2.0 ** 57, 2.0 ** 56] * 4, [1e-30, -1e-30] * 4 + [0.5e-30]]
    _check_rows(torch.tensor(rows, dtype=dtype, device=DEV))
    _check_rows(torch.tensor([r * 300 for r in rows], dtype=dtype, device=DEV))


def test_no_rows_and_offsets_past_32_bits():
    B.quantize_int8_rows(torch.zeros((0, 8), device=DEV), torch.zeros(0, dtype=torch.int8, device=DEV),
                         torch.zeros(0, device=DEV))
    rows, cols = 66000, 33000                                     # 2.2 billion elements
    src = torch.zeros((rows, cols), dtype=BF16, device=DEV)
    src[-1, -3:] = torch.tensor([1.0, -2.0, 127.0], dtype=BF16, device=DEV)
    codes, scales = torch.empty((rows, cols), dtype=torch.int8, device=DEV), torch.empty(rows, device=DEV)
    B.quantize_int8_rows(src, codes, scales)
    assert codes[-1, -4:].tolist() == [0, 1, -2, 127] and float(scales[-1]) == 1.0 and float(scales[0]) == 0.0


class Layer8:
    def __init__(self, T, k, E, d, f, beta=16, P=1, routed=1.0, seed=0, s=1, experts=None):
        gen = torch.Generator().manual_seed(seed)
        self.x = (torch.randn((T, d), generator=gen) * (1 + 5 * (torch.rand(d, generator=gen) < 0.02))).to(BF16)
        pool = E if experts is None else experts
        ids = torch.stack([torch.randperm(pool, generator=gen)[:k] for _ in range(T)]) if T else torch.zeros((0, k))
        ids = ids.to(torch.int32)
        ids[torch.rand((T, k), generator=gen) >= routed] = -1
        self.ids, self.gates = ids, torch.rand((T, k), generator=gen)
        self.w1 = torch.randint(-127, 128, (E, 2 * f, d), generator=gen).to(torch.int8)
        self.w2 = torch.randint(-127, 128, (E, d, f), generator=gen).to(torch.int8)
        self.s1 = (torch.rand((E, 2 * f), generator=gen) + 0.5) / (73 * d ** 0.5)
        self.s2 = (torch.rand((E, d), generator=gen) + 0.5) / (73 * f ** 0.5)
        dev = {n: getattr(self, n).to(DEV) for n in ("x", "ids", "gates", "w1", "w2", "s1", "s2")}
        self.dev = dev
        self.r = LayerRunner(dev["w1"], dev["w2"], dev["s1"], dev["s2"], act_dtype=BF16, T=T, k=k, beta=beta, P=P, s=s,
                             owner=torch.from_numpy(contiguous_owners(E, P)))

    def run(self):
        self.r.ws.fill_(0xA5)
        self.r.y.fill_(-3.0)
        y = self.r.step(self.dev["x"], self.dev["gates"], self.dev["ids"]).clone()
        torch.cuda.synchronize()
        assert int(self.r.status) == 0
        return y

    def oracle(self):
        n = lambda t: t.double().numpy() if t.dtype != torch.int8 else t.numpy()
        return oi8.forward(n(self.x), n(self.w1), n(self.s1), n(self.w2), n(self.s2), self.ids.numpy(), n(self.gates))


# few rows an expert, sizes off the 256 grid, the 256 x 256 tiles; beta above and below the tiles
LAYERS = [(1, 1, 1, 128, 64, 16, 1), (1, 8, 16, 256, 256, 16, 1), (3, 2, 5, 384, 192, 1, 2), (17, 4, 8, 256, 64, 16, 4),
          (64, 8, 32, 512, 256, 16, 1), (150, 3, 6, 384, 192, 32, 2), (300, 2, 4, 128, 320, 50, 8), (333, 3, 10, 384, 192, 300, 2),
          (40, 2, 2, 512, 512, 128, 1), (700, 4, 8, 512, 256, 128, 8), (600, 2, 4, 256, 512, 16, 4), (900, 3, 5, 768, 256, 300, 2),
          (130, 1, 1, 256, 256, 128, 1), (257, 2, 3, 1024, 768, 50, 1), (3, 1, 2, 8320, 64, 16, 1), (20, 2, 3, 2176, 2112, 16, 2)]


@pytest.mark.parametrize("T,k,E,d,f,beta,P", LAYERS)
@pytest.mark.parametrize("routed", [1.0, 0.6])
def test_layer(T, k, E, d, f, beta, P, routed):
    say(f"[int8] T={T} k={k} E={E} d={d} f={f} beta={beta} P={P} routed={routed}")
    c = Layer8(T, k, E, d, f, beta, P, routed, seed=T + E)
    y = c.run()
    assert not y.isnan().any()
    ref = c.oracle()
    none = (c.ids < 0).all(1).numpy()
    assert (y.float().cpu().numpy()[none] == 0).all()
    err = rel_l2(y.double().cpu().numpy(), ref)
    say(f"  {err:.3e}")
    assert err <= TOL
    assert torch.equal(c.run(), y)                                # the same bits, whatever the workspace held


def test_layer_of_nothing():
    for T, routed in ((0, 1.0), (5, 0.0)):
        c = Layer8(T, 2, 4, 256, 256, routed=routed)
        y = c.run()
        assert y.shape == (T, 256) and (y == 0).all()


@pytest.mark.parametrize("T,E,f", [(40, 8, 192), (700, 4, 256)])
def test_rows_that_are_not_finite_stay_alone(T, E, f):
    """A token of NaN or infinities has a row of NaN; the others are those of the same batch without it, and a
    token's row does not depend on its place or the others."""
    c = Layer8(T, 2, E, 256, f, seed=3)
    ref = c.run()
    c.dev["x"][T // 2, 7] = float("nan")
    c.dev["x"][3, 0] = float("inf")
    y = c.run()
    bad = torch.zeros(T, dtype=torch.bool)
    bad[[3, T // 2]] = True
    assert y[bad].isnan().all()
    assert torch.equal(y[~bad], ref[~bad])


@pytest.mark.parametrize("T,P", [(700, 8), (30, 4)])
def test_result_does_not_depend_on_the_plan(T, P):
    c = Layer8(T, 4, 8, 512, 256, 32, P, seed=9, s=4, experts=5)
    y = c.run()
    for s in (0, 2):
        c.r.step(c.dev["x"], c.dev["gates"], c.dev["ids"], s=s)
        assert torch.equal(c.r.y, y)


def test_both_ways_agree():
    """The same tokens in a batch of few rows an expert and in a large one: codes and whole sums are the same, so
    only the order of scales differs."""
    c = Layer8(800, 2, 4, 512, 256, 128, 1, seed=5)
    y = c.run()
    small = Layer8(8, 2, 4, 512, 256, 128, 1, seed=5)
    for n in ("w1", "w2", "s1", "s2"):
        small.dev[n].copy_(c.dev[n])
    for n in ("x", "ids", "gates"):
        small.dev[n].copy_(c.dev[n][:8])
    assert rel_l2(small.run().double().cpu().numpy(), y[:8].double().cpu().numpy()) <= 2 * TOL


@pytest.mark.parametrize("T,E,d,f", [(4, 16, 256, 192), (600, 4, 512, 256)])
def test_captured_on_a_side_stream_and_replayed(T, E, d, f):
    c = Layer8(T, 2, E, d, f, 32, 2, seed=2)
    other = Layer8(T, 2, E, d, f, 32, 2, seed=8)
    want = [c.run(), None]
    step = lambda: c.r.step(c.dev["x"], c.dev["gates"], c.dev["ids"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert torch.equal(c.r.y, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kept = {n: c.dev[n].clone() for n in ("x", "ids", "gates")}
    for turn in range(4):
        src = kept if turn % 2 == 0 else {n: other.dev[n] for n in kept}
        for n in kept:
            c.dev[n].copy_(src[n])
        graph.replay()
        torch.cuda.synchronize()
        got = c.r.y.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, c.r.y)
        if turn % 2 == 0:
            assert torch.equal(got, want[0])


def test_weights_quantized_by_the_library():
    """A bf16 layer and the same layer with weights quantized by quantize_int8_rows: within the quantizations,
    some 2^-8 a value over three operands, averaged over the sums."""
    T, k, E, d, f = 300, 2, 4, 512, 256
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)
    w1, w2, x = (rnd(E, 2 * f, d) * d ** -0.5).to(BF16), (rnd(E, d, f) * f ** -0.5).to(BF16), rnd(T, d).to(BF16)
    ids = torch.stack([torch.randperm(E, device=DEV)[:k] for _ in range(T)]).to(torch.int32)
    gates = torch.rand((T, k), device=DEV)
    owner = torch.zeros(E, dtype=torch.int32)
    kw = dict(act_dtype=BF16, T=T, k=k, beta=64, P=1, s=0, owner=owner)
    ref = LayerRunner(w1, w2, **kw).step(x, gates, ids).double()
    q = []
    for w in (w1, w2):
        c, s = torch.empty(w.shape, dtype=torch.int8, device=DEV), torch.empty(w.shape[:2], device=DEV)
        B.quantize_int8_rows(w.reshape(-1, w.shape[2]), c, s)
        q.append((c, s))
    got = LayerRunner(q[0][0], q[1][0], q[0][1], q[1][1], **kw).step(x, gates, ids).double()
    torch.cuda.synchronize()
    # a code is off by half a step of max / 127 at most: rms 2^-8.8 of a row whose max is 3.5 deviations, in four operands
    assert rel_l2(got.cpu().numpy(), ref.cpu().numpy()) <= 2 * 3.5 / 127 / 12 ** 0.5 + 2 * TOL


def test_runner_refuses_a_backward_pass():
    c = Layer8(4, 2, 4, 256, 64)
    with pytest.raises(B.MoeError, match="backward"):
        LayerRunner(c.dev["w1"], c.dev["w2"], c.dev["s1"], c.dev["s2"], act_dtype=BF16, T=4, k=2, beta=16, P=1, s=1,
                    owner=torch.zeros(4, dtype=torch.int32), with_backward=True)


def test_block_forward_with_int8_experts():
    """Norm, router and int8 experts of a block that only answers."""
    from moe_expert_ffn_amd.runner import BlockRunner
    c = Layer8(50, 2, 8, 256, 256, seed=4)
    wr, one = (torch.randn(8, 256, device=DEV) / 16).to(BF16), torch.ones(256, dtype=BF16, device=DEV)
    b = BlockRunner(c.dev["w1"], c.dev["w2"], wr, one, one, None, c.dev["s1"], c.dev["s2"], act_dtype=BF16, T=50, k=2, beta=16,
                    P=1, s=1, owner=torch.zeros(8, dtype=torch.int32), groups=4, top_groups=2, score="sigmoid")
    b.block_forward(c.dev["x"])
    torch.cuda.synchronize()
    assert int(b.status) == 0
    n = lambda t: t.double().cpu().numpy() if t.dtype != torch.int8 else t.cpu().numpy()
    ref = oi8.forward(n(b.n), n(c.w1), n(c.s1), n(c.w2), n(c.s2), b.routed["topk_ids"].cpu().numpy(), n(b.routed["gates"]))
    assert rel_l2(n(b.y), ref) <= TOL
