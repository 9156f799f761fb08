"""GPU parity of the router's choice by values against the fp64 oracle.

Ids, counts and live rows are exact, also where values differ by less than 32 bits show.  Gates, sums and
losses have the tolerances of the choice by logits (tests/test_gpu_router.py)."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from oracle import choice as ochoice
from oracle import router as orouter
from tests.gpu_util import say
from tests.test_gpu_router import U, _check_backward, _logits, _rel

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def _forward(R, C, logits, mask=None, bufs=None):
    T = logits.shape[0]
    out, ws = bufs or (B.alloc_router(R, T, DEV), B.router_workspace(R, T, DEV))
    for t in out.values():
        t.fill_(-7)
    ws.fill_(0xAB)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.router_forward(R, logits, out, ws, st, mask=mask, choice=C)
    torch.cuda.synchronize()
    return out, int(st.item())


def _check(logits, k, score, renorm, bias=None, groups=1, top=1, rank="top2", scale=1.0, mask=None):
    T, E = logits.shape
    R = B.make_router(E, k, logits.dtype, score, renorm, scale)
    C = B.make_choice(R, bias, groups, top, rank)
    out, st = _forward(R, C, logits, mask)
    l = logits.double().cpu().numpy()
    o = ochoice.forward(l, k, score == "sigmoid", renorm, scale, None if mask is None else mask.cpu().numpy(),
                        bias=None if bias is None else bias.double().cpu().numpy(), groups=groups, top_groups=top,
                        two=rank == "top2")
    assert st == (B.DEV_BAD_LOGIT if o["bad"] else 0)
    np.testing.assert_array_equal(out["topk_ids"].cpu().numpy(), o["topk_ids"])
    np.testing.assert_array_equal(out["counts"].cpu().numpy(), o["counts"])
    assert int(out["live"].item()) == o["live"]
    rel = _rel(l)
    np.testing.assert_allclose(out["gates"].cpu().numpy(), o["gates"], rtol=rel, atol=1e-37)
    more = 2 * (T / 256 + 16) * U
    np.testing.assert_allclose(out["prob_sum"].cpu().numpy(), o["prob_sum"], rtol=rel + more, atol=1e-37)
    np.testing.assert_allclose(out["losses"].cpu().numpy(), o["losses"], rtol=2 * (rel + more),
                               atol=4 * rel * (1 + np.abs(o["losses"][1])))
    return R, C, out, o


# T, E, k, groups, open groups: aligned to lanes and not, one expert a group, the largest
SHAPES = [(1, 8, 2, 4, 2), (16, 256, 8, 8, 4), (17, 64, 8, 8, 3), (100, 60, 6, 4, 3), (33, 16, 4, 16, 5),
          (50, 65, 3, 5, 2), (40, 160, 6, 8, 3), (70, 512, 12, 16, 4), (20, 1024, 32, 64, 9), (31, 513, 16, 3, 1),
          (3000, 12, 2, 3, 2), (5, 1, 1, 1, 1), (300, 128, 8, 2, 1), (64, 128, 5, 64, 7), (25, 384, 8, 6, 6),
          (60, 256, 32, 4, 2), (45, 48, 3, 48, 4)]


@pytest.mark.parametrize("T,E,k,groups,top", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score,renorm,rank", [("softmax", True, "max"), ("softmax", False, "top2"),
                                               ("sigmoid", True, "top2"), ("sigmoid", False, "max")])
def test_choice_and_gradient(T, E, k, groups, top, dtype, score, renorm, rank):
    say(f"[choice] T={T} E={E} k={k} groups={groups}/{top} {dtype} {score} renorm={renorm} {rank}")
    rng = np.random.default_rng(T * 1000 + E + groups)
    logits = _logits(rng, T, E, dtype)
    logits[torch.rand(logits.shape, device=DEV) < 0.03] = float("-inf")
    for bias in (None, torch.from_numpy((rng.integers(-60, 61, E) * 0.001).astype(np.float32)).to(DEV)):
        scale = 1.0 if score == "softmax" else 2.5
        R, C, out, o = _check(logits, k, score, renorm, bias, groups, top, rank, scale)
    h = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).to(DEV)
    _check_backward(R, logits, out, o, h, torch.tensor([0.8, 0.05], device=DEV), score, renorm)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,offset", [(3, 1), (8, 8), (1, 0)])
def test_strided_rows_and_padding(dtype, pad, offset):
    rng = np.random.default_rng(5)
    T, E, k = 1100, 256, 8
    logits = _logits(rng, T, E, dtype, pad, offset)
    mask = torch.from_numpy((rng.random(T) < 0.8).astype(np.uint8)).to(DEV)
    logits[~mask.bool()] = float("nan")
    bias = torch.randn(E, device=DEV) * 0.1
    R, C, out, o = _check(logits, k, "sigmoid", True, bias, 8, 4, mask=mask)
    _check_backward(R, logits, out, o, torch.randn((T, k), device=DEV), None, "sigmoid", True, mask)
    bits = {n: t.clone() for n, t in out.items()}
    again, _ = _forward(R, C, logits, mask)
    for n in bits:                                                # the same call, the same bits
        assert torch.equal(again[n], bits[n]), n


@pytest.mark.parametrize("E,groups,top", [(64, 1, 1), (256, 8, 4), (60, 4, 2), (200, 40, 9), (1024, 32, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_that_32_bits_cannot_tell_apart(E, groups, top, score):
    """Biases that bring every value to within 32 bits' rounding of one number: the order is the 64-bit one."""
    for seed in range(12):
        rng = np.random.default_rng(seed)
        row = rng.standard_normal(E).astype(np.float32)
        l = row.astype(np.float64)
        s = 1 / (1 + np.exp(-l)) if score == "sigmoid" else np.exp(l - l.max()) / np.exp(l - l.max()).sum()
        level = 1.25 if seed % 2 else 0.01
        bias = (level - s).astype(np.float32)
        if seed % 3 == 0:                                         # some equal to the last bit, some far away
            row[E // 2:E // 2 + 3], bias[E // 2:E // 2 + 3] = row[0], bias[0]
            bias[1::7] += 0.5
        logits = torch.from_numpy(np.stack([row] * 3)).to(DEV)
        _check(logits, min(6, top * (E // groups)), score, True, torch.from_numpy(bias).to(DEV), groups, top,
               "top2" if seed % 4 < 2 else "max")


@pytest.mark.parametrize("E", [8, 64, 100, 256, 600])
@pytest.mark.parametrize("left", [1, 2, 3, 7, 8])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_next_to_each_other_with_few_to_choose(E, left, score):
    """Fewer experts left than places, their values within 32 bits' rounding: the other places are -1."""
    for seed in range(6):
        rng = np.random.default_rng(100 * left + seed)
        row = np.full(E, -np.inf, dtype=np.float32)
        at = rng.choice(E, left, replace=False)
        row[at] = rng.standard_normal(left).astype(np.float32)
        l = row[at].astype(np.float64)
        s = 1 / (1 + np.exp(-l)) if score == "sigmoid" else np.exp(l - l.max()) / np.exp(l - l.max()).sum()
        bias = np.zeros(E, dtype=np.float32)
        bias[at] = (1.25 - s).astype(np.float32)
        logits = torch.from_numpy(np.stack([row, row + np.float32(0.0), row])).to(DEV)
        groups = 1 if E % 4 else 4
        _check(logits, min(E, 8), score, True, torch.from_numpy(bias).to(DEV))
        _check(logits, min(E // groups, 8), score, False, torch.from_numpy(bias).to(DEV), groups, max(1, groups - 1))


@pytest.mark.parametrize("E,groups,top", [(64, 8, 4), (64, 2, 1), (128, 4, 2), (256, 8, 4), (60, 4, 2), (512, 16, 5), (1024, 8, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_that_32_bits_cannot_tell_apart(E, groups, top, score):
    """Groups whose values, of two members or one, lie within 32 bits' rounding of each other, members that do not;
    and with a third member next to the second."""
    for seed in range(16):
        rng = np.random.default_rng(seed)
        size = E // groups
        row = rng.standard_normal(E).astype(np.float32)
        l = row.astype(np.float64)
        s = 1 / (1 + np.exp(-l)) if score == "sigmoid" else np.exp(l - l.max()) / np.exp(l - l.max()).sum()
        bias = (-3 + 0.5 * rng.random(E)).astype(np.float32)
        rank = "top2" if seed % 2 else "max"
        for g in range(groups):
            a, b, c = g * size + rng.choice(size, 3, replace=False)
            first = 1.7 + 0.1 * rng.random() if rank == "top2" else 2.0
            bias[a] = np.float32(first - s[a])
            second = 3.0 - (s[a] + float(bias[a])) if rank == "top2" else 1.0 + 0.3 * rng.random()
            bias[b] = np.float32(second - s[b])
            if seed % 4 >= 2 and g % 2:
                bias[c] = np.float32(second - s[c])
        _check(torch.from_numpy(np.stack([row] * 3)).to(DEV), min(8, top * size), score, True, torch.from_numpy(bias).to(DEV),
               groups, top, rank)


@pytest.mark.parametrize("E,groups,top", [(8, 2, 1), (100, 4, 2), (256, 8, 4), (700, 7, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ties_extremes_and_masks(E, groups, top, score, dtype):
    inf, low = float("inf"), torch.finfo(dtype).min
    k = 4
    g = E // groups
    rows = [[0.0] * E,                                            # all equal: the lowest indexes
            [-0.0 if e % 2 else 0.0 for e in range(E)],
            [-inf] * E,                                           # nothing left
            [-inf] * (E - 2) + [1.0, -inf],                       # one left
            [-inf] * g + [0.5 if e % 3 else -inf for e in range(E - g)],    # a whole group barred
            [low] * (E - 1) + [2.0],
            [float("nan")] + [0.0] * (E - 1),
            [0.0] * (E - 1) + [inf],
            [20.0] + [-20.0] * (E - 1),
            [30.0 if e % g == 0 else -3.0 for e in range(E)]]     # one large in every group
    logits = torch.tensor(rows, dtype=dtype, device=DEV)
    tie = torch.zeros(E, device=DEV)
    odd = torch.linspace(-1, 1, E, device=DEV)
    odd[::5], odd[1::11], odd[2] = -inf, float("nan"), 3.0
    large = torch.full((E,), 1e30, device=DEV)                    # hides every score: ties
    masks = (None, torch.tensor([1] * 6 + [0] * 2 + [1] * 2, dtype=torch.bool, device=DEV))
    for bias in (None, tie, odd, large):
        for m in masks:
            for rank in ("max", "top2"):
                R = B.make_router(E, k, dtype, score, True)
                C = B.make_choice(R, bias, groups, top, rank)
                out, st = _forward(R, C, logits, m)
                mn = None if m is None else m.cpu().numpy()
                with np.errstate(all="ignore"):
                    o = ochoice.forward(logits.double().cpu().numpy(), k, score == "sigmoid", True, 1.0, mn,
                                        bias=None if bias is None else bias.double().cpu().numpy(), groups=groups,
                                        top_groups=top, two=rank == "top2")
                assert st == (B.DEV_BAD_LOGIT if o["bad"] else 0)
                np.testing.assert_array_equal(out["topk_ids"].cpu().numpy(), o["topk_ids"])
                np.testing.assert_array_equal(out["counts"].cpu().numpy(), o["counts"])
                # |l| to 30: 5 * 60 + 40 roundings, doubled
                np.testing.assert_allclose(out["gates"].cpu().numpy(), o["gates"], rtol=680 * U, atol=1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 128, 600])
def test_chosen_scores_of_next_to_nothing(score, E):
    """The experts that the bias chooses have scores that underflow beside the row's (softmax) or by themselves:
    their shares of each other, and their gradient, are still there."""
    rng = np.random.default_rng(E)
    l = rng.standard_normal((40, E)).astype(np.float32)
    l[:, :4] -= np.array([100, 95, 130, 60], dtype=np.float32)
    l[20:, 4:] += 200.0 if score == "softmax" else 0.0
    logits = torch.from_numpy(l).to(DEV)
    bias = torch.zeros(E, device=DEV)
    bias[:4] = 5.0
    R, _, out, o = _check(logits, 4, score, True, bias)
    assert (o["gates"].max(1) < 1).any() and (o["topk_ids"] < 4).all()
    _check_backward(R, logits, out, o, torch.randn((40, 4), device=DEV), torch.tensor([0.8, 0.05], device=DEV), score, True)


def test_trivial_choice_is_the_choice_by_logits():
    logits = _logits(np.random.default_rng(1), 500, 96, F32)
    R = B.make_router(96, 5)
    C = B.make_choice(R, None, 6)
    out, _ = _forward(R, C, logits)
    ref = B.alloc_router(R, 500, DEV)
    B.router_forward(R, logits, ref, B.router_workspace(R, 500, DEV), torch.zeros(1, dtype=torch.int32, device=DEV))
    for n in ref:
        assert torch.equal(out[n], ref[n])


def test_no_tokens():
    R = B.make_router(16, 2)
    out, st = _forward(R, B.make_choice(R, torch.zeros(16, device=DEV), 4, 2), torch.zeros((0, 16), device=DEV))
    assert st == 0 and int(out["live"]) == 0 and (out["counts"] == 0).all() and (out["losses"] == 0).all()


@pytest.mark.parametrize("E", [1, 5, 64, 128, 1000, 1024])
def test_bias_update(E):
    rng = np.random.default_rng(E)
    for counts in (rng.integers(0, 50, E), np.full(E, 7), np.zeros(E, int), rng.integers(0, 2 ** 31 - 1, E)):
        b = (rng.standard_normal(E) * 0.1).astype(np.float32)
        t = torch.from_numpy(b).to(DEV)
        B.router_bias_update(t, torch.from_numpy(counts.astype(np.int32)).to(DEV), 0.001)
        np.testing.assert_array_equal(t.cpu().numpy(), ochoice.bias_update(b, counts, 0.001))


def test_captured_steps_with_a_moving_bias():
    """Choice and balancing step in a graph, replayed between eager steps: the bias is read when they run."""
    rng = np.random.default_rng(2)
    T, E, k = 700, 64, 4
    logits = _logits(rng, T, E, F32)
    R = B.make_router(E, k, F32, "sigmoid")
    bias = torch.zeros(E, device=DEV)
    C = B.make_choice(R, bias, 8, 4)
    out, ws = B.alloc_router(R, T, DEV), B.router_workspace(R, T, DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        B.router_forward(R, logits, out, ws, status, choice=C)
        B.router_bias_update(bias, out["counts"], 0.01)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    bias.zero_()
    want, spread = np.zeros(E, np.float32), []
    for turn in range(6):
        o = ochoice.forward(logits.double().cpu().numpy(), k, True, bias=want.astype(np.float64), groups=8, top_groups=4)
        step() if turn % 2 else graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(out["topk_ids"].cpu().numpy(), o["topk_ids"])
        want = ochoice.bias_update(want, o["counts"], 0.01)
        np.testing.assert_array_equal(bias.cpu().numpy(), want)
        spread.append(o["counts"].max() - o["counts"].min())
    assert spread[-1] < spread[0]


def test_block_with_a_bias_and_groups():
    """BlockRunner chooses by values, its gradients follow that choice, and update_bias moves the bias."""
    from tests.test_gpu_block import PATHS, _block
    w = PATHS["stream_bf16"]
    bias = torch.linspace(-0.1, 0.1, w.E, device=DEV)
    b, par, x, dout = _block(w, w.T, 5, "sigmoid", True, bias=bias, groups=4, top_groups=3)
    b.block_forward(x)
    dl = torch.tensor([0.1, 0.01], device=DEV)
    b.block_backward(dout, dl)
    torch.cuda.synchronize()
    assert int(b.status) == 0
    l = b.logits.double().cpu().numpy()
    o = ochoice.forward(l, w.k, True, bias=bias.double().cpu().numpy(), groups=4, top_groups=3)
    np.testing.assert_array_equal(b.routed["topk_ids"].cpu().numpy(), o["topk_ids"])
    _check_backward(b.router, b.logits, b.routed, o, b.dlogp, dl, "sigmoid", True)
    want = ochoice.bias_update(bias.cpu().numpy(), o["counts"], 0.01)
    b.update_bias(0.01)
    np.testing.assert_array_equal(bias.cpu().numpy(), want)
    b, *_ = _block(w, w.T, 5, "sigmoid", True)
    with pytest.raises(B.MoeError, match="no bias"):
        b.update_bias(0.01)
