"""Cases for more operators around the expert layer: routing with a selection bias and expert groups, the global gradient
norm with clipping, and the expert layer with 8-bit integer weights.

`run` computes one operator in its plain form (elementary torch operations, in 32 bits, and in 64 where a choice, a long sum
or a code next to a border needs them), or, where `own` is true, through the framework's binding and runner.  `exact`
computes the same outputs from the definitions in 64 bits.  Shapes are the workloads' of moe_expert_ffn_amd/inputs.py
(Qwen3- and DeepSeek-V3-shaped layers) and generic small and ragged ones.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F32 = torch.float32
F64 = torch.float64
TINY = 2.0 ** -100             # rows whose magnitudes are all below are zeros in 8 bits


def listed():
    return [
        # routing of a small decode batch of a DeepSeek-V3-shaped model, 8 groups of 32 experts: latency alone
        {"name": "groups decode", "op": "choice", "T": 16, "E": 256, "k": 8, "groups": 8, "top": 4, "rank": "top2",
         "bias": True, "dtype": "bf16", "score": "sigmoid", "renorm": True, "pad": 0, "masked": 0.0},
        # the same over a large ragged training batch with padding
        {"name": "groups train", "op": "choice", "T": 65521, "E": 256, "k": 8, "groups": 8, "top": 4, "rank": "top2",
         "bias": True, "dtype": "bf16", "score": "sigmoid", "renorm": True, "pad": 0, "masked": 0.05},
        # groups that are no power of two, softmax scores, logits in 32 bits as a slice of wider rows
        {"name": "groups odd", "op": "choice", "T": 8192, "E": 60, "k": 6, "groups": 4, "top": 3, "rank": "max",
         "bias": True, "dtype": "f32", "score": "softmax", "renorm": False, "pad": 3, "masked": 0.1},
        # norm over the many small gradients of a model (norms, biases, routers)
        {"name": "norm many", "op": "grad_norm", "tensors": 160, "total": 1_000_003, "dtype": "f32"},
        # norm over the gradients of one Qwen3-shaped expert layer, in 32 bits as its backward pass writes them
        {"name": "norm layer", "op": "grad_norm", "tensors": 0, "total": 604_246_016, "dtype": "f32"},
        # gradients clipped in place for an optimizer of the user's own: a few ragged tensors of a dense part
        {"name": "clip ragged", "op": "clip", "tensors": 12, "total": 25_000_013, "dtype": "bf16"},
        # the same over many small tensors of both types
        {"name": "clip many", "op": "clip", "tensors": 60, "total": 1_000_003, "dtype": "mixed"},
        # one token of a Qwen3-shaped layer with 8-bit weights: the chosen experts' weights are read once
        {"name": "int8 token", "op": "int8", "T": 1, "k": 8, "E": 128, "d": 2048, "d_ff": 768, "beta": 16, "P": 1,
         "routed": 1.0},
        # a batch of 64 decoding sequences: a few rows for each expert
        {"name": "int8 batch", "op": "int8", "T": 64, "k": 8, "E": 128, "d": 2048, "d_ff": 768, "beta": 16, "P": 1,
         "routed": 1.0},
        # a prompt batch of the Qwen3-shaped layer
        {"name": "int8 prompt", "op": "int8", "T": 8192, "k": 8, "E": 128, "d": 2048, "d_ff": 768, "beta": 128, "P": 8,
         "routed": 1.0},
        # a DeepSeek-V3-shaped share of experts, some of the tokens' slots routed to other ranks
        {"name": "int8 share", "op": "int8", "T": 4096, "k": 8, "E": 32, "d": 7168, "d_ff": 2048, "beta": 128, "P": 8,
         "routed": 0.5},
        # a small ragged layer with odd widths
        {"name": "int8 odd", "op": "int8", "T": 333, "k": 3, "E": 10, "d": 384, "d_ff": 192, "beta": 32, "P": 2,
         "routed": 0.9},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["choice", "choice", "grad_norm", "clip", "int8", "int8"])
    if op == "choice":
        groups = rng.choice([1, 2, 3, 4, 5, 8, 16])
        E = groups * rng.choice([_log(rng, 1, 512 // groups), 512 // groups, max(1, 256 // groups), max(1, 64 // groups)])
        top = rng.randint(1, groups)
        return {"op": op, "T": _log(rng, 1, 65536 * 256 // max(E, 256)), "E": E,
                "k": rng.randint(1, min(top * (E // groups), 12)), "groups": groups, "top": top,
                "rank": rng.choice(["max", "top2"]), "bias": rng.random() < 0.75, "dtype": rng.choice(["f32", "bf16"]),
                "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.5,
                "pad": rng.choice([0, 0, 3, 8]), "masked": rng.choice([0.0, 0.1, 0.5])}
    if op in ("grad_norm", "clip"):
        tensors = _log(rng, 1, 200 if op == "grad_norm" else 60)
        return {"op": op, "tensors": tensors, "total": _log(rng, tensors * 4, 100_000_000),
                "dtype": rng.choice(["f32", "bf16", "mixed"])}
    E = _log(rng, 1, 128)
    k = rng.randint(1, min(E, 8))
    d, d_ff = 128 * _log(rng, 1, 56), 64 * _log(rng, 1, 32)
    E = max(k, min(E, 604_000_000 // (3 * d * d_ff)))
    return {"op": op, "T": _log(rng, 1, max(1, min(16384, 65536 * 2048 * 768 // (k * d * d_ff)))), "k": k, "E": E,
            "d": d, "d_ff": d_ff, "beta": rng.choice([16, 50, 128]), "P": rng.choice([1, 2, 8]), "routed": rng.choice([1.0, 0.9, 0.5])}


# ---------------------------------------------------------------- inputs

def _dtype(name):
    return F32 if name == "f32" else torch.bfloat16


def _sizes(case):
    """Element counts of the tensors: `total` in all, ragged; tensors = 0: an expert layer's (w1, w2, router, norms)."""
    n, total = case["tensors"], case["total"]
    if n == 0:
        E, d, d_ff = 128, 2048, 768
        return [E * 2 * d_ff * d, E * d * d_ff, E * d, d, d]
    r = random.Random(total * 31 + n)
    cut = sorted(r.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cut, cut + [total])]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"choice": _prepare_choice, "grad_norm": _prepare_grads, "clip": _prepare_grads,
         "int8": _prepare_int8}[case["op"]](case, gen)
    s["case"] = case
    if own:
        _handles(case, s)
    return s


def _prepare_choice(case, gen):
    T, E, dt = case["T"], case["E"], _dtype(case["dtype"])
    # a router's logits: a popularity of the experts beside the tokens' own part; some experts barred
    logits = torch.randn((T, E + case["pad"]), generator=gen, device=DEV) * 1.5
    logits += torch.randn((1, E + case["pad"]), generator=gen, device=DEV)
    logits[torch.rand(logits.shape, generator=gen, device=DEV) < 0.01] = -math.inf
    mask = None
    if case["masked"]:
        mask = torch.rand(T, generator=gen, device=DEV) >= case["masked"]
        logits[~mask] = math.nan                       # what padded rows hold is anything
        mask = mask.to(torch.uint8)
    bias = None
    if case["bias"]:                                   # what balancing steps of 0.001 have summed up to
        bias = torch.randint(-60, 61, (E,), generator=gen, device=DEV).float() * 0.001
    return {"logits": logits.to(dt)[:, :E], "mask": mask, "bias": bias,
            "scale": 2.5 if case["score"] == "sigmoid" else 1.0}


def _prepare_grads(case, gen):
    g = []
    for i, n in enumerate(_sizes(case)):
        dt = _dtype(("f32", "bf16")[i % 2] if case["dtype"] == "mixed" else case["dtype"])
        g.append(torch.randn(n, generator=gen, device=DEV).mul_(1e-3).to(dt))
    # below what the gradients have, so that clipping takes place
    return {"g": g, "max": 0.7e-3 * math.sqrt(case["total"]), "turn": 0}


def _prepare_int8(case, gen):
    T, k, E, d, f, dt = case["T"], case["k"], case["E"], case["d"], case["d_ff"], torch.bfloat16
    rand = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    logits = rand(T, E) + 0.5 * rand(1, E)
    chosen, ids = torch.topk(logits, k, dim=1)
    gates = torch.exp(chosen - chosen[:, :1])
    gates = gates / gates.sum(1, keepdim=True)
    if case["routed"] < 1:                             # the other slots' experts are elsewhere
        away = torch.rand((T, k), generator=gen, device=DEV) >= case["routed"]
        ids, gates = ids.masked_fill(away, -1), gates.masked_fill(away, 0.0)
    strong = 1 + 8 * (torch.rand(d, generator=gen, device=DEV) < 0.01)       # a few features are large
    s = {"x": (rand(T, d) * strong).to(dt), "ids": ids.to(torch.int32), "gates": gates.contiguous()}
    for name, rows, cols in (("w1", 2 * f, d), ("w2", d, f)):
        w = torch.empty((E, rows, cols), dtype=torch.int8, device=DEV)
        for e in range(E):
            w[e] = rand(rows, cols).mul_(32).round_().clamp_(-127, 127)
        s[name] = w
        s[name + "_scale"] = (torch.rand((E, rows), generator=gen, device=DEV) + 0.5) / (32 * math.sqrt(cols))
    # the rows of each expert, in the order of the tokens
    flat = s["ids"].reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat + 1, minlength=E + 1).tolist()
    s["rows"] = order[counts[0]:].split(counts[1:])
    return s


def _handles(case, s):
    """What a user's program keeps between calls of the framework: outputs, workspaces, prepared lists, the routing."""
    from moe_expert_ffn_amd import binding as B

    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if case["op"] == "choice":
        r = s["router"] = B.make_router(case["E"], case["k"], s["logits"].dtype, case["score"], case["renorm"],
                                        s["scale"])
        s["choice"] = B.make_choice(r, s["bias"], case["groups"], case["top"], case["rank"])
        s["out"] = B.alloc_router(r, case["T"], DEV)
        s["ws"] = B.router_workspace(r, case["T"], DEV)
    elif case["op"] in ("grad_norm", "clip"):
        s["list"] = B.make_grads(s["g"])
        s["norm"], s["scale"] = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    else:
        from moe_expert_ffn_amd.runner import LayerRunner

        owner = torch.arange(case["E"], dtype=torch.int32) * case["P"] // case["E"]
        s["runner"] = LayerRunner(s["w1"], s["w2"], s["w1_scale"], s["w2_scale"], act_dtype=s["x"].dtype, T=case["T"],
                                  k=case["k"], beta=case["beta"], P=case["P"], s=1, owner=owner)
        s["runner"].route(s["ids"])
        s["runner"].make_plan()


# ---------------------------------------------------------------- one pass

def run(s):
    return globals()[("_own_" if own else "_run_") + s["case"]["op"]](s)


def _own_choice(s):
    from moe_expert_ffn_amd import binding as B

    B.router_forward(s["router"], s["logits"], s["out"], s["ws"], s["status"], mask=s["mask"], choice=s["choice"])
    return {n: s["out"][n] for n in ("topk_ids", "gates", "counts", "prob_sum", "losses")}


def _own_grad_norm(s):
    from moe_expert_ffn_amd import binding as B

    B.grad_norm(s["list"], s["max"], s["norm"], s["scale"], s["status"])
    return {"norm": s["norm"], "scale": s["scale"]}


def _clip_turn(s):
    """Norm wanted and factor before it: clipped at every pass, up and down in turn, so that values keep their size."""
    s["turn"] ^= 1
    return s["max"] * (1.0 if s["turn"] else 0.5), 2.5


def _own_clip(s):
    from moe_expert_ffn_amd import binding as B

    most, mult = _clip_turn(s)
    B.grad_norm(s["list"], most, s["norm"], s["scale"], s["status"], mult=mult)
    B.grad_scale(s["list"], s["scale"])
    return {"g": s["g"], "norm": s["norm"], "scale": s["scale"]}


def _own_int8(s):
    return s["runner"].forward(s["x"], s["gates"], s["ids"])


# the plain forms

def _rows_in_use(l, mask):
    ok = ~(torch.isnan(l) | (l == math.inf)).any(1) & (l > -math.inf).any(1)
    return ok if mask is None else ok & (mask != 0)


def _first(v, n):
    """The n largest of each row, the lower index among equals, in descending order."""
    v, at = torch.sort(v, dim=1, descending=True, stable=True)
    return v[:, :n], at[:, :n]


def _choose(case, l, ok, bias):
    """ids [T][k], -1 where nothing is left.  Values are compared in 64 bits: two that differ by less than 32 bits show
    would otherwise be chosen by their rounding."""
    T, E, G = l.shape[0], case["E"], case["groups"]
    l64 = l.double()
    if case["score"] == "softmax":
        v = torch.exp(l64 - l64.amax(1, keepdim=True))
        v = v / v.sum(1, keepdim=True)
    else:
        v = 1 / (1 + torch.exp(-l64))
    if bias is not None:
        v = v + bias.double()
    v = torch.where(l > -math.inf, v, -math.inf)
    if case["top"] < G:
        each = v.reshape(T, G, E // G).sort(dim=2, descending=True).values
        worth = each[:, :, 0]
        if case["rank"] == "top2" and E // G > 1:
            worth = worth + torch.where(each[:, :, 1] > -math.inf, each[:, :, 1], 0.0)
        _, at = _first(worth, case["top"])
        allowed = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, at, True)
        v = torch.where(allowed.repeat_interleave(E // G, 1), v, -math.inf)
    best, ids = _first(v, case["k"])
    return torch.where((best > -math.inf) & ok[:, None], ids, -1)


def _run_choice(s):
    case, E, k = s["case"], s["case"]["E"], s["case"]["k"]
    l = s["logits"].float()
    ok = _rows_in_use(l, s["mask"])
    l = torch.where(ok[:, None], l, 0.0)               # rows that are not routed: any numbers, left out below
    ids = _choose(case, l, ok, s["bias"])
    there = ids >= 0
    ls = l if case["score"] == "softmax" else l.clamp(max=0) - torch.log1p(torch.exp(-l.abs()))
    e = torch.exp(ls - ls.amax(1, keepdim=True))
    P = e / e.sum(1, keepdim=True) * ok[:, None]
    chosen = ls.gather(1, ids.clamp(min=0))
    if case["renorm"]:
        chosen = torch.where(there, chosen, -math.inf)
        best = chosen.amax(1, keepdim=True)
        g = torch.exp(chosen - torch.where(best > -math.inf, best, 0.0))
        gates = g / torch.where(there.any(1, keepdim=True), g.sum(1, keepdim=True), 1.0)
    elif case["score"] == "softmax":
        gates = P.gather(1, ids.clamp(min=0)) * there
    else:
        gates = torch.exp(chosen) * there
    n = ok.sum()
    hits = torch.zeros(E + 1, dtype=torch.int32, device=l.device)
    hits.scatter_add_(0, (ids + 1).reshape(-1), torch.ones(ids.numel(), dtype=torch.int32, device=l.device))
    counts, prob_sum = hits[1:], P.sum(0)
    top = l.amax(1)
    lse = top + torch.log(torch.exp(l - top[:, None]).sum(1))
    many = n.clamp(min=1).float()
    balance = (counts * prob_sum).sum() * (E / k) / many / many
    return {"topk_ids": ids.to(torch.int32), "gates": gates * s["scale"], "counts": counts, "prob_sum": prob_sum,
            "losses": torch.stack([balance, (lse * lse * ok).sum() / many])}


def _norm_and_scale(s, most, mult):
    total = torch.zeros((), dtype=F64, device=DEV)
    for g in s["g"]:
        g = g.double()
        total = total + (g * g).sum()
    norm = mult * torch.sqrt(total)
    scale = mult * torch.where(norm > most, most / norm, 1.0)
    return norm.float().reshape(1), scale.float().reshape(1)


def _run_grad_norm(s):
    norm, scale = _norm_and_scale(s, s["max"], 1.0)
    return {"norm": norm, "scale": scale}


def _run_clip(s):
    norm, scale = _norm_and_scale(s, *_clip_turn(s))
    for g in s["g"]:
        g.copy_(g.float() * scale)
    return {"g": s["g"], "norm": norm, "scale": scale}


def _to_int8(x):
    """Codes (as 32-bit numbers) and scales of rows: round(127 x / max|x|), half to even, in 64 bits, so that a value
    next to half a step has its code from its own value and not from a rounding."""
    amax = x.abs().amax(1, keepdim=True)
    amax = torch.where(amax < TINY, 0.0, amax)
    codes = torch.round(x.double() * 127 / torch.where(amax > 0, amax, 1.0).double()) * (amax > 0)
    return codes.float(), amax / 127


def _run_int8(s):
    case, x = s["case"], s["x"]
    f = case["d_ff"]
    cx, sx = _to_int8(x.float())
    flat = torch.zeros((case["T"] * case["k"], case["d"]), device=DEV)
    for e, rows in enumerate(s["rows"]):
        if rows.numel() == 0:
            continue
        t = rows // case["k"]
        z = (cx[t] @ s["w1"][e].float().t()) * sx[t] * s["w1_scale"][e]
        g, u = z[:, :f], z[:, f:]
        a = (g / (1 + torch.exp(-g)) * u).to(x.dtype).float()      # the activations' type is a part of the definition
        ca, sa = _to_int8(a)
        o = (ca @ s["w2"][e].float().t()) * sa * s["w2_scale"][e]
        flat[rows] = o * s["gates"].reshape(-1)[rows, None]
    return flat.reshape(case["T"], case["k"], -1).sum(1).to(x.dtype)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, s)


def _largest(v):
    """Index of each row's largest entry, the lowest of several, and the entry."""
    m = v.max(1, keepdim=True).values
    at = torch.arange(v.shape[1], device=v.device).expand_as(v)
    return torch.where(v == m, at, v.shape[1]).min(1).values.clamp(max=v.shape[1] - 1), m[:, 0]


def _exact_choice(case, s):
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    l = s["logits"].double()
    use = ~(l.isnan() | l.isposinf()).any(1) & ~l.isneginf().all(1)
    if s["mask"] is not None:
        use &= s["mask"].bool()
    l = l.masked_fill(~use[:, None], 1.0)
    score = l.softmax(1) if case["score"] == "softmax" else l.sigmoid()
    v = score.clone() if s["bias"] is None else score + s["bias"].double()
    v[l.isneginf()] = -math.inf
    parts = v.view(T, G, E // G)
    worth = torch.empty((T, G), dtype=F64, device=l.device)
    for g in range(G):
        part = parts[:, g].clone()
        at, first = _largest(part)
        part.scatter_(1, at[:, None], -math.inf)
        second = part.amax(1)
        worth[:, g] = first if case["rank"] == "max" else first + second.masked_fill(second.isneginf(), 0.0)
    closed = torch.ones((T, G), dtype=torch.bool, device=l.device)
    for _ in range(case["top"]):
        at, _ = _largest(worth)
        closed.scatter_(1, at[:, None], False)
        worth.scatter_(1, at[:, None], -math.inf)
    v = parts.masked_fill(closed[:, :, None], -math.inf).reshape(T, E)
    ids = torch.full((T, k), -1, dtype=torch.int64, device=l.device)
    for j in range(k):
        at, best = _largest(v)
        ids[:, j] = torch.where(best.isneginf() | ~use, -1, at)
        v.scatter_(1, at[:, None], -math.inf)
    taken = ids >= 0
    picked = score.gather(1, ids.clamp(min=0)) * taken
    gates = picked / picked.sum(1, keepdim=True).masked_fill(~taken.any(1, keepdim=True), 1.0) if case["renorm"] else picked
    share = score / score.sum(1, keepdim=True) * use[:, None]
    counts = torch.bincount(ids[taken], minlength=E)
    n = max(int(use.sum()), 1)
    prob = share.sum(0)
    z = l.logsumexp(1)[use].square().sum() / n
    return {"topk_ids": ids.to(torch.int32), "gates": gates * s["scale"], "counts": counts.to(torch.int32),
            "prob_sum": prob, "losses": torch.stack([E * (counts * prob).sum() / (k * n * n), z])}


def _exact_grad_norm(case, s):
    norm = math.sqrt(sum(float(g.double().pow(2).sum()) for g in s["g"]))
    scale = s["max"] / norm if norm > s["max"] else 1.0
    return {"norm": torch.tensor([norm], dtype=F64), "scale": torch.tensor([scale], dtype=F64)}


def _exact_clip(case, s):
    norm = 2.5 * math.sqrt(sum(float(g.double().pow(2).sum()) for g in s["g"]))
    scale = 2.5 * min(1.0, s["max"] / norm)
    return {"g": [g.double() * scale for g in s["g"]], "norm": torch.tensor([norm], dtype=F64),
            "scale": torch.tensor([scale], dtype=F64)}


def _codes(v):
    """Nearest whole numbers to 127 v / max|v| of 64-bit rows, half to even, and the steps."""
    step = v.abs().max(1).values / 127
    step = step.masked_fill(step * 127 < TINY, 0.0)[:, None]
    return torch.where(step > 0, (v / step.masked_fill(step == 0, 1.0)).round(), 0.0), step


def _exact_int8(case, s):
    T, k, f = case["T"], case["k"], case["d_ff"]
    y = torch.zeros((T, case["d"]), dtype=F64, device=DEV)
    ids = s["ids"]
    for e in range(case["E"]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        codes, step = _codes(s["x"][t].double())
        z = torch.mm(codes, s["w1"][e].double().t()) * (step * s["w1_scale"][e].double())
        a = torch.nn.functional.silu(z[:, :f]) * z[:, f:]
        codes, step = _codes(a.to(s["x"].dtype).double())
        o = torch.mm(codes, s["w2"][e].double().t()) * (step * s["w2_scale"][e].double())
        y.index_add_(0, t, o * s["gates"][t, j].double()[:, None])
    return y


# ---------------------------------------------------------------- the least work

def work(case):
    op = case["op"]
    if op == "choice":
        T, E, k = case["T"], case["E"], case["k"]
        b = 4 if case["dtype"] == "f32" else 2
        return {"bytes": T * E * b + (T if case["masked"] else 0) + (4 * E if case["bias"] else 0) + 8 * T * k + 8 * E + 8,
                "flops": 12 * T * E}
    if op in ("grad_norm", "clip"):
        b = {"f32": 4, "bf16": 2, "mixed": 3}[case["dtype"]] * case["total"]
        return {"bytes": 2 * b + 8, "flops": 3 * case["total"]} if op == "clip" else {"bytes": b + 8,
                                                                                      "flops": 2 * case["total"]}
    T, k, E, d, f = case["T"], case["k"], case["E"], case["d"], case["d_ff"]
    rows = T * k * case["routed"]
    used = min(E * (1 - (1 - k * case["routed"] / E) ** T), rows)            # experts with a row, on average
    return {"bytes": used * (3 * d * f + 8 * f + 4 * d) + 4 * T * d + 8 * T * k, "flops": 6 * rows * d * f}
