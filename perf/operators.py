"""Cases for the operators around the expert layer: router and balance loss, gate gradient, block norms, AdamW.

`run` computes one operator in its plain form (elementary torch operations in 32 bits), or, where `own` is true, through
the framework's binding.  `exact` computes the same outputs from the definitions in 64 bits.  Shapes are the workloads'
of moe_expert_ffn_amd/inputs.py (OLMoE-, Qwen3- and DeepSeek-V3-shaped layers) and generic small and ragged ones.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F32 = torch.float32
BLOCK = 128                    # elements that share one scale of an 8-bit optimizer state
MASK32 = 0xFFFFFFFF
# odd 32-bit constants of the rounding's random words: the fractional parts of the golden ratio, sqrt(2) and sqrt(3)
GOLD, ROOT2, ROOT3 = 0x9E3779B9, 0x6A09E667, 0xBB67AE85
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.99, 1e-8, 0.1
NORM_EPS = 1e-6


def listed():
    return [
        # the router of a small decode batch on a Qwen3-shaped layer: latency alone
        {"name": "router decode", "op": "router", "T": 16, "E": 128, "k": 8, "dtype": "bf16", "score": "softmax",
         "renorm": True, "pad": 0, "masked": 0.0},
        # the router of a training batch, its sequences padded, logits in 32 bits and as a slice of wider rows
        {"name": "router train", "op": "router", "T": 8192, "E": 128, "k": 8, "dtype": "f32", "score": "softmax",
         "renorm": True, "pad": 8, "masked": 0.1},
        # gradients of the OLMoE-shaped router (gates not renormalised)
        {"name": "router bwd", "op": "router_bwd", "T": 4096, "E": 64, "k": 8, "dtype": "f32", "score": "softmax",
         "renorm": False, "pad": 0, "masked": 0.0},
        # gradients of a DeepSeek-V3-shaped router over a large ragged batch, sigmoid scores
        {"name": "router bwd large", "op": "router_bwd", "T": 65521, "E": 256, "k": 8, "dtype": "bf16",
         "score": "sigmoid", "renorm": True, "pad": 0, "masked": 0.05},
        # gate gradients of a small 32-bit layer
        {"name": "gates small", "op": "gate_grad", "T": 257, "k": 2, "d_ff": 64, "dtype": "f32", "routed": 0.9},
        # gate gradients of the Qwen3-shaped training batch
        {"name": "gates train", "op": "gate_grad", "T": 8192, "k": 8, "d_ff": 768, "dtype": "bf16", "routed": 1.0},
        # residual update and norm before the block, one token of a DeepSeek-V3-shaped model: latency alone
        {"name": "norm in token", "op": "norm_in", "T": 1, "d": 7168, "dtype": "bf16", "gate": "feature",
         "residual": True, "pad": 0},
        # its gradients on a ragged training batch
        {"name": "norm in bwd", "op": "norm_in_bwd", "T": 4099, "d": 7168, "dtype": "bf16", "gate": "feature",
         "residual": True, "pad": 0},
        # norm of the block's output with a gate per token, added to the residual: Qwen3-shaped batch
        {"name": "norm out", "op": "norm_out", "T": 8192, "d": 2048, "dtype": "bf16", "gate": "token",
         "residual": True, "pad": 0},
        # its gradients in 32 bits with an odd width
        {"name": "norm out bwd", "op": "norm_out_bwd", "T": 1000, "d": 1023, "dtype": "f32", "gate": "token",
         "residual": True, "pad": 1},
        # the many small tensors of a model (norms, biases, routers), 32-bit states
        {"name": "adamw many", "op": "adamw", "tensors": 160, "total": 1_000_003, "p": "f32", "g": "f32", "bits": 32},
        # one Qwen3-shaped expert layer: bf16 weights, the layer's 32-bit gradients, 8-bit states
        {"name": "adamw layer", "op": "adamw", "tensors": 0, "total": 604_246_016, "p": "bf16", "g": "f32", "bits": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "router_bwd", "gate_grad", "norm_in", "norm_in_bwd", "norm_out", "norm_out_bwd",
                     "adamw"])
    dt = rng.choice(["f32", "bf16"])
    if op in ("router", "router_bwd"):
        E = rng.choice([_log(rng, 4, 512), 8, 64, 128, 256])
        return {"op": op, "T": _log(rng, 1, 65536 * 256 // max(E, 256)), "E": E, "k": rng.randint(1, min(E, 12)),
                "dtype": dt, "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.5,
                "pad": rng.choice([0, 0, 3, 8]), "masked": rng.choice([0.0, 0.1, 0.5])}
    if op == "gate_grad":
        d_ff = 64 * _log(rng, 1, 32)
        k = rng.randint(1, 10)
        return {"op": op, "T": _log(rng, 1, max(1, 50_000_000 // (d_ff * k))), "k": k, "d_ff": d_ff, "dtype": dt,
                "routed": rng.choice([1.0, 0.5])}
    if op == "adamw":
        tensors = _log(rng, 1, 200)
        return {"op": op, "tensors": tensors, "total": _log(rng, tensors * 4, 100_000_000),
                "p": rng.choice(["f32", "bf16", "master"]), "g": dt, "bits": rng.choice([8, 32])}
    d = rng.choice([_log(rng, 1, 8192), 8 * _log(rng, 8, 1024)])
    return {"op": op, "T": _log(rng, 1, max(1, 29_000_000 // d)), "d": d, "dtype": dt,
            "gate": rng.choice(["none", "token", "feature"]), "residual": rng.random() < 0.75,
            "pad": rng.choice([0, 0, 1, 8])}


# ---------------------------------------------------------------- inputs

def _dtype(name):
    return F32 if name == "f32" else torch.bfloat16


def _wide(T, n, pad, dtype, gen, scale=1.0):
    """[T][n] normal values as a slice of rows of n + pad."""
    full = torch.randn((T, n + pad), generator=gen, device=DEV) * scale
    return full.to(dtype)[:, :n]


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
    s = globals()["_prepare_" + case["op"].replace("_bwd", "")](case, gen)
    s["case"] = case
    s["seed"] = seed & MASK32
    if own:
        _handles(case, s)
    return s


def _prepare_router(case, gen):
    T, E, k, dt = case["T"], case["E"], case["k"], _dtype(case["dtype"])
    # a router's logits: a popularity of the experts beside the tokens' own part; some experts barred
    logits = torch.randn((T, E + case["pad"]), generator=gen, device=DEV) * 1.5
    logits += torch.randn((1, E + case["pad"]), generator=gen, device=DEV)
    logits[torch.rand(logits.shape, generator=gen, device=DEV) < 0.01] = -math.inf
    mask = None
    if case["masked"]:
        mask = (torch.rand(T, generator=gen, device=DEV) >= case["masked"])
        logits[~mask] = math.nan                       # what padded rows hold is anything
        mask = mask.to(torch.uint8)
    s = {"logits": logits.to(dt)[:, :E], "mask": mask, "scale": 2.5 if case["score"] == "sigmoid" else 1.0}
    if case["op"] == "router_bwd":
        f = _router_plain(case, s["logits"], mask, s["scale"])
        s["fwd"] = f
        s["dlogp"] = torch.randn((T, k), generator=gen, device=DEV) * (0.1 / T)
        s["dlosses"] = torch.tensor([0.01, 0.001], device=DEV)
    return s


def _prepare_gate_grad(case, gen):
    T, k, f, dt = case["T"], case["k"], case["d_ff"], _dtype(case["dtype"])
    rows = T * k
    slots = rows + rows // 8 + 1                       # blocks are padded
    z = torch.randn((slots, 2 * f), generator=gen, device=DEV).to(dt)
    dz = (torch.randn((slots, 2 * f), generator=gen, device=DEV) * 1e-3).to(dt)
    # rows of one expert lie together in the order of their tokens, whose k slots are far apart
    slot = torch.randperm(slots, generator=gen, device=DEV)[:rows].to(torch.int32)
    if case["routed"] < 1:
        slot[torch.rand(rows, generator=gen, device=DEV) >= case["routed"]] = -1
    return {"z": z, "dz": dz, "slot": slot.reshape(T, k)}


def _prepare_norm(case, gen):
    T, d, dt, pad = case["T"], case["d"], _dtype(case["dtype"]), case["pad"]
    s = {"x": _wide(T, d, pad, dt, gen, 2.0), "u": _wide(T, d, pad, dt, gen),
         "w": (1 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(dt), "alpha": 0.7, "gate": None}
    if case["gate"] == "token":
        s["gate"] = torch.rand((T, 1), generator=gen, device=DEV)
    elif case["gate"] == "feature":
        s["gate"] = 0.5 + 0.3 * torch.randn(d, generator=gen, device=DEV)
    s["residual"] = case["residual"]
    if "bwd" in case["op"]:
        s["do"] = _wide(T, d, pad, dt, gen, 0.1)
        s["dr"] = _wide(T, d, pad, dt, gen, 0.1)
        src = s["x"] if "norm_in" in case["op"] else s["u"]
        s["rstd"] = (src.float().square().mean(1) + NORM_EPS).rsqrt()
    return s


_prepare_norm_in = _prepare_norm_out = _prepare_norm


def _prepare_adamw(case, gen):
    sizes = _sizes(case)
    rand = lambda n: torch.randn(n, generator=gen, device=DEV)  # noqa: E731
    p = [rand(n).mul_(0.02) for n in sizes]
    s = {"p": [x if case["p"] == "f32" else x.to(torch.bfloat16) for x in p],
         "master": p if case["p"] == "master" else None,
         "g": [rand(n).mul_(1e-3).to(_dtype(case["g"])) for n in sizes], "step": 100}
    if case["bits"] == 32:
        s["m"] = [rand(n).mul_(1e-4) for n in sizes]
        s["v"] = [rand(n).mul_(1e-3).square_() for n in sizes]
        s["ms"] = s["vs"] = None
    else:                                              # any finite codes, scales of gradients' sizes
        blocks = [-(-n // BLOCK) for n in sizes]
        byte = lambda n, hi: torch.randint(0, hi, (n,), generator=gen, device=DEV, dtype=torch.uint8)  # noqa: E731
        s["m"] = [byte(n, 126) | (byte(n, 2) << 7) for n in sizes]
        s["v"] = [byte(n, 126) for n in sizes]
        s["ms"] = [torch.rand(b, generator=gen, device=DEV).add_(0.5).mul_(3e-4 / 448) for b in blocks]
        s["vs"] = [torch.rand(b, generator=gen, device=DEV).add_(0.5).mul_(3e-3 / 448) for b in blocks]
    return s


def _handles(case, s):
    """What a user's program keeps between calls of the framework: outputs, workspaces, the optimizer's list."""
    from moe_expert_ffn_amd import binding as B

    op = case["op"]
    if op.startswith("router"):
        r = s["router"] = B.make_router(case["E"], case["k"], s["logits"].dtype, case["score"], case["renorm"],
                                        s["scale"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if op == "router":
            s["out"] = B.alloc_router(r, case["T"], DEV)
            s["ws"] = B.router_workspace(r, case["T"], DEV)
        else:
            s["dlogits"] = torch.empty(s["logits"].shape, dtype=s["logits"].dtype, device=DEV)
    elif op == "gate_grad":
        s["dlogp"] = torch.empty(s["slot"].shape, dtype=F32, device=DEV)
    elif op.startswith("norm"):
        T, d = s["x"].shape
        new = lambda: torch.empty((T, d), dtype=s["x"].dtype, device=DEV)  # noqa: E731
        s["a"], s["b"] = new(), new()
        if op.endswith("_bwd"):
            s["dw"] = torch.empty(d, dtype=F32, device=DEV)
            s["dgate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
            s["ws"] = B.norm_workspace(T, d, DEV)
        else:
            s["rstd"] = torch.empty(T, dtype=F32, device=DEV)
    else:
        s["list"] = B.make_adamw(s["p"], s["g"], s["m"], s["v"], m_scale=s["ms"], v_scale=s["vs"], master=s["master"])


# ---------------------------------------------------------------- one pass

def run(s):
    return globals()[("_own_" if own else "_run_") + s["case"]["op"]](s)


def _own_router(s):
    from moe_expert_ffn_amd import binding as B

    B.router_forward(s["router"], s["logits"], s["out"], s["ws"], s["status"], mask=s["mask"])
    return {n: s["out"][n] for n in ("topk_ids", "gates", "counts", "prob_sum", "losses")}


def _own_router_bwd(s):
    from moe_expert_ffn_amd import binding as B

    B.router_backward(s["router"], s["logits"], s["fwd"], s["dlogp"], s["dlosses"], s["dlogits"], mask=s["mask"])
    return s["dlogits"]


def _own_gate_grad(s):
    from moe_expert_ffn_amd import binding as B

    return B.gate_grad(s["z"], s["dz"], s["slot"], s["dlogp"])


def _own_norm_in(s):
    from moe_expert_ffn_amd import binding as B

    if not s["residual"]:
        B.norm_in(s["x"], s["w"], NORM_EPS, s["a"], s["rstd"])
        return {"n": s["a"], "rstd": s["rstd"]}
    B.norm_in(s["x"], s["w"], NORM_EPS, s["a"], s["rstd"], u=s["u"], gate=s["gate"], alpha=s["alpha"], r=s["b"])
    return {"n": s["a"], "rstd": s["rstd"], "r": s["b"]}


def _own_norm_in_bwd(s):
    from moe_expert_ffn_amd import binding as B

    if not s["residual"]:
        B.norm_in_backward(s["do"], s["x"], s["w"], s["rstd"], s["a"], s["dw"], s["ws"])
        return {"dx": s["a"], "dw": s["dw"]}
    B.norm_in_backward(s["do"], s["x"], s["w"], s["rstd"], s["a"], s["dw"], s["ws"], dr=s["dr"], u=s["u"],
                       gate=s["gate"], alpha=s["alpha"], du=s["b"], dgate=s["dgate"])
    return {"dx": s["a"], "dw": s["dw"], "du": s["b"], "dgate": s["dgate"]}


def _own_norm_out(s):
    from moe_expert_ffn_amd import binding as B

    B.norm_out(s["u"], s["x"], s["w"], NORM_EPS, s["a"], s["rstd"], gate=s["gate"], alpha=s["alpha"])
    return {"out": s["a"], "rstd": s["rstd"]}


def _own_norm_out_bwd(s):
    from moe_expert_ffn_amd import binding as B

    B.norm_out_backward(s["do"], s["u"], s["w"], s["rstd"], s["a"], s["dw"], s["ws"], gate=s["gate"],
                        alpha=s["alpha"], dgate=s["dgate"])
    return {"dy": s["a"], "dw": s["dw"], "dgate": s["dgate"]}


def _own_adamw(s):
    from moe_expert_ffn_amd import binding as B

    s["step"] += 1
    B.adamw(s["list"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY, step=s["step"], seed=s["seed"])
    return _adamw_outputs(s)


# the plain forms

def _scores(case, l):
    """The router's log scores: the logits, or log sigma of them."""
    return l if case["score"] == "softmax" else l.clamp(max=0) - torch.log1p(torch.exp(-l.abs()))


def _live(logits, mask):
    l = logits.float() + 0.0
    ok = ~(torch.isnan(l) | (l == math.inf)).any(1) & (l > -math.inf).any(1)
    if mask is not None:
        ok &= mask != 0
    return torch.where(ok[:, None], l, -math.inf), ok


def _shares(ls, ok):
    """softmax of the rows that are live, zeros in the others; the rows' maxima"""
    top = torch.where(ok, ls.amax(1), 0.0)[:, None]
    e = torch.exp(ls - top)
    return e / torch.where(ok, e.sum(1), 1.0)[:, None], top


def _router_plain(case, logits, mask, scale):
    E, k = case["E"], case["k"]
    l, ok = _live(logits, mask)
    ls = _scores(case, l)
    # one whole number per logit, ordered as the logits are and by the lower index among equals
    bits = l.view(torch.int32).long()
    key = (torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) << 32) + (E - 1 - torch.arange(E, device=l.device))
    ids = E - 1 - (torch.topk(key, k, dim=1).values & MASK32)
    chosen = l.gather(1, ids)
    ids = torch.where(chosen > -math.inf, ids, -1)
    P, top = _shares(ls, ok)
    sel = torch.exp(ls.gather(1, ids.clamp(min=0)) - top) * (ids >= 0)
    if case["renorm"]:
        gates = sel / torch.where(ok, sel.sum(1), 1.0)[:, None]
    elif case["score"] == "softmax":
        gates = P.gather(1, ids.clamp(min=0)) * (ids >= 0)
    else:
        gates = sel * torch.exp(top)
    n = ok.sum()
    hits = torch.zeros(E + 1, dtype=torch.int32, device=l.device)
    hits.scatter_add_(0, (ids + 1).reshape(-1), torch.ones(ids.numel(), dtype=torch.int32, device=l.device))
    counts, prob_sum = hits[1:], P.sum(0)
    lse = _lse(l, ok)
    many = n.clamp(min=1).float()
    balance = (counts * prob_sum).sum() * (E / k) / many / many
    return {"topk_ids": ids.to(torch.int32), "gates": gates * scale, "counts": counts, "prob_sum": prob_sum,
            "live": n.to(torch.int32).reshape(1), "losses": torch.stack([balance, (lse * lse).sum() / many])}


def _lse(l, ok):
    top = torch.where(ok, l.amax(1), 0.0)
    return torch.where(ok, top + torch.log(torch.exp(l - top[:, None]).sum(1).clamp(min=1e-30)), 0.0)


def _run_router(s):
    f = _router_plain(s["case"], s["logits"], s["mask"], s["scale"])
    return {n: f[n] for n in ("topk_ids", "gates", "counts", "prob_sum", "losses")}


def _run_router_bwd(s):
    case, f = s["case"], s["fwd"]
    E, k = case["E"], case["k"]
    l, ok = _live(s["logits"], s["mask"])
    P, _ = _shares(_scores(case, l), ok)
    ids = f["topk_ids"].long()
    there = ids >= 0
    h = torch.where(there, s["dlogp"], 0.0)
    at = torch.where(there, ids, E)
    zeros = torch.zeros((l.shape[0], E + 1), device=l.device)
    dls = zeros.scatter_add(1, at, h)[:, :E]
    if case["renorm"]:
        q = P * zeros.scatter(1, at, 1.0)[:, :E]
        total = q.sum(1, keepdim=True)
        dls = dls - q / torch.where(total > 0, total, 1.0) * h.sum(1, keepdim=True)
    elif case["score"] == "softmax":
        dls = dls - P * h.sum(1, keepdim=True)
    many = f["live"].clamp(min=1).float()
    g = f["counts"] * (s["dlosses"][0] * (E / k) / many / many)
    dls = dls + P * (g - (P * g).sum(1, keepdim=True))
    if case["score"] == "softmax":
        dl = dls + P * (s["dlosses"][1] * 2 / many * _lse(l, ok))[:, None]
    else:
        away = torch.exp(-l.clamp(min=0)) / (1 + torch.exp(-l.abs()))     # sigma(-l)
        share, _ = _shares(l, ok)
        dl = dls * away + share * (s["dlosses"][1] * 2 / many * _lse(l, ok))[:, None]
    return torch.where(ok[:, None], dl, 0.0).to(s["logits"].dtype)


def _run_gate_grad(s):
    f, slot = s["case"]["d_ff"], s["slot"].reshape(-1)
    at = slot.clamp(min=0).long()
    dot = (s["z"][:, f:][at].float() * s["dz"][:, f:][at].float()).sum(1)
    return torch.where(slot >= 0, dot, 0.0).reshape(s["slot"].shape)


def _scaled(s, v):
    return v * s["alpha"] if s["gate"] is None else v * (s["gate"] * s["alpha"])


def _run_norm_in(s):
    dt, r = s["x"].dtype, s["x"].float()
    if s["residual"]:
        r = r + _scaled(s, s["u"].float())
    rstd = (r.square().mean(1) + NORM_EPS).rsqrt()
    out = {"n": (r * rstd[:, None] * s["w"].float()).to(dt), "rstd": rstd}
    return {**out, "r": r.to(dt)} if s["residual"] else out


def _norm_grad(do, x, w, rstd):
    """gradients of w * x * rstd(x): of x, and of w summed over the rows"""
    xhat = x * rstd[:, None]
    dx = do * w
    return (dx - xhat * (dx * xhat).mean(1, keepdim=True)) * rstd[:, None], (do * xhat).sum(0)


def _gate_sum(s, v):
    """gradient of the gate from its elementwise one"""
    if s["gate"] is None:
        return None
    return s["alpha"] * (v.sum(1, keepdim=True) if s["gate"].dim() == 2 else v.sum(0))


def _run_norm_in_bwd(s):
    dt = s["x"].dtype
    dx, dw = _norm_grad(s["do"].float(), s["x"].float(), s["w"].float(), s["rstd"])
    if not s["residual"]:
        return {"dx": dx.to(dt), "dw": dw}
    dx = dx + s["dr"].float()
    return {"dx": dx.to(dt), "dw": dw, "du": _scaled(s, dx).to(dt), "dgate": _gate_sum(s, s["u"].float() * dx)}


def _run_norm_out(s):
    y = s["u"].float()
    rstd = (y.square().mean(1) + NORM_EPS).rsqrt()
    out = s["x"].float() + _scaled(s, y * rstd[:, None] * s["w"].float())
    return {"out": out.to(s["x"].dtype), "rstd": rstd}


def _run_norm_out_bwd(s):
    do, y, w = s["do"].float(), s["u"].float(), s["w"].float()
    dy, dw = _norm_grad(_scaled(s, do), y, w, s["rstd"])
    return {"dy": dy.to(s["u"].dtype), "dw": dw, "dgate": _gate_sum(s, do * (y * s["rstd"][:, None] * w))}


def _words(seed, step, sizes, dev):
    """A random 32-bit word (in 64) for every element of every tensor: a hash of the seed, the step, the tensor's
    place in the list and the element's index."""
    key = [_mix((seed + step * GOLD + i * ROOT3) & MASK32) for i in range(len(sizes))]
    return torch.cat([_mix_t((torch.arange(n, device=dev) * GOLD + k) & MASK32) for n, k in zip(sizes, key)])


def _mix(x):
    x ^= x >> 16
    x = (x * ROOT2) & MASK32
    return x ^ (x >> 15)


def _mix_t(x):
    x = ((x ^ (x >> 16)) * ROOT2) & MASK32
    return x ^ (x >> 15)


def _blocks(x, sizes):
    """the tensors end to end, each filled up to whole blocks: [blocks][BLOCK]"""
    parts = [torch.nn.functional.pad(t, (0, -t.numel() % BLOCK)) for t in x.split(sizes)]
    return torch.cat(parts).reshape(-1, BLOCK)


def _flat(x, sizes):
    """back from _blocks: the tensors end to end"""
    whole = [n + -n % BLOCK for n in sizes]
    return torch.cat([t[:n] for t, n in zip(x.reshape(-1).split(whole), sizes)])


def _to_e4m3(x, u16, sizes):
    """e4m3 codes and 32-bit scales of blocks, rounded up or down at random: up with the probability of the part cut
    off.  Values that are not finite become the NaN code and do not enter the scale."""
    b, u = _blocks(x, sizes), _blocks(u16, sizes)
    finite = torch.isfinite(b)
    amax = torch.where(finite, b.abs(), 0.0).amax(1, keepdim=True)
    amax = torch.where(amax < 2.0 ** -100, 0.0, amax)
    y = b.abs() * torch.where(amax > 0, 448 / amax, 0.0)
    ex = ((y.view(torch.int32) >> 23) - 127).clamp(-6, 8)
    q = torch.floor(y * torch.exp2((3 - ex).float()) + (u.float() + 0.5) * 2.0 ** -16)
    code = ((ex + 6) * 8 + q.nan_to_num().to(torch.int32)).clamp(max=126)
    code = torch.where(finite, code, 127) | torch.where(b < 0, 128, 0)
    return _flat(code.to(torch.uint8), sizes), (amax * (1 / 448)).reshape(-1)


def _from_e4m3(codes, scales, sizes):
    v = _blocks(torch.cat(codes).view(torch.float8_e4m3fn).float(), sizes)
    return _flat(v * torch.cat(scales)[:, None], sizes)


def _store(to, x):
    sizes = [t.numel() for t in to]
    [t.copy_(v) for t, v in zip(to, x.split(sizes))]


def _store_e4m3(to, scales, x, u16, sizes):
    codes, amax = _to_e4m3(x, u16, sizes)
    _store(to, codes)
    _store(scales, amax)


def _run_adamw(s):
    case = s["case"]
    sizes = [t.numel() for t in s["p"]]
    s["step"] += 1
    t = s["step"]
    p = torch.cat(s["p"] if s["master"] is None else s["master"]).float()
    g = torch.cat(s["g"]).float()
    if case["bits"] == 32:
        m, v = torch.cat(s["m"]), torch.cat(s["v"])
    else:
        m, v = _from_e4m3(s["m"], s["ms"], sizes), _from_e4m3(s["v"], s["vs"], sizes).square()
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    p = p * (1 - LR * DECAY) - LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    word = _words(s["seed"], t, sizes, p.device) if case["bits"] == 8 or case["p"] == "bf16" else None
    if case["p"] == "bf16":                            # no 32-bit copy: rounded at random, or small steps are lost
        up = (p.view(torch.int32) + (((word * ROOT3) & MASK32) >> 16).to(torch.int32)) & -65536
        _store(s["p"], torch.where(torch.isfinite(p), up.view(F32), p))
    else:
        _store(s["p"], p)
        if s["master"] is not None:
            _store(s["master"], p)
    if case["bits"] == 32:
        _store(s["m"], m)
        _store(s["v"], v)
    else:
        _store_e4m3(s["m"], s["ms"], m, word & 0xFFFF, sizes)
        _store_e4m3(s["v"], s["vs"], v.sqrt(), word >> 16, sizes)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    """Parameters and states after the step, end to end (the many small ones) or as they are."""
    join = (lambda x: [torch.cat(x)]) if len(s["p"]) > 8 else list
    value = (lambda x: x) if s["ms"] is None else (lambda x: [t.view(torch.float8_e4m3fn) for t in x])
    out = {"p": join(s["p"]), "m": value(join(s["m"])), "v": value(join(s["v"]))}
    if s["ms"] is not None:
        out["ms"], out["vs"] = join(s["ms"]), join(s["vs"])
    if s["master"] is not None:
        out["master"] = join(s["master"])
    return out


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](case, s)


def _exact_rows(case, s):
    """64-bit logits, log scores, the rows in use"""
    l = s["logits"].double()
    use = torch.isfinite(l).any(1) & ~l.isnan().any(1) & ~l.isposinf().any(1)
    if s["mask"] is not None:
        use = use & s["mask"].bool()
    l = l.masked_fill(~use[:, None], 0.0)              # a row that is not in use: any numbers, left out below
    return l, (l if case["score"] == "softmax" else -torch.log1p(torch.exp(-l))), use


def _exact_router(case, s):
    l, ls, use = _exact_rows(case, s)
    E, k = case["E"], case["k"]
    ids = l.sort(dim=1, descending=True, stable=True).indices[:, :k]
    good = use[:, None] & (l.gather(1, ids) > -math.inf)
    P = (ls - ls.logsumexp(1, keepdim=True)).exp() * use[:, None]
    sc = ls.gather(1, ids).exp() * good
    if case["renorm"]:
        gates = sc / sc.sum(1, keepdim=True).masked_fill(~use[:, None], 1.0)
    else:
        gates = P.gather(1, ids) * good if case["score"] == "softmax" else sc
    n = max(int(use.sum()), 1)
    counts = torch.stack([((ids == e) & good).sum() for e in range(E)])
    prob = P.sum(0)
    z = (l.logsumexp(1).square() * use).sum() / n
    return {"topk_ids": torch.where(good, ids, -1).to(torch.int32), "gates": gates * s["scale"],
            "counts": counts.to(torch.int32), "prob_sum": prob,
            "losses": torch.stack([E / k * (counts * prob).sum() / n / n, z])}


def _exact_router_bwd(case, s):
    """By the chain rule through autograd in 64 bits of sum h log p + the two losses."""
    l, _, use = _exact_rows(case, s)
    f = s["fwd"]
    ids, E = f["topk_ids"].long(), case["E"]
    low = l == -math.inf
    x = l.masked_fill(low, -1e30).requires_grad_()
    ls = x if case["score"] == "softmax" else torch.nn.functional.logsigmoid(x)
    picked = ls.gather(1, ids.clamp(min=0)).masked_fill(ids < 0, -1e30)
    logP = ls - ls.logsumexp(1, keepdim=True)
    if case["renorm"]:
        logp = picked - picked.logsumexp(1, keepdim=True)
    else:
        logp = logP.gather(1, ids.clamp(min=0)) if case["score"] == "softmax" else picked
    n = max(int(f["live"]), 1)
    on = (ids >= 0) & use[:, None]
    loss = (logp.masked_fill(~on, 0.0) * s["dlogp"].double()).sum()
    prob = (logP.exp() * use[:, None]).sum(0)
    d0, d1 = s["dlosses"].double().tolist()
    loss = loss + d0 * E / case["k"] * (f["counts"] * prob).sum() / n / n
    loss = loss + d1 * (x.logsumexp(1).square() * use).sum() / n
    loss.backward()
    return x.grad.masked_fill(low | ~use[:, None], 0.0)


def _exact_gate_grad(case, s):
    f = case["d_ff"]
    rows = torch.bmm(s["z"][:, None, f:].double(), s["dz"][:, f:, None].double().contiguous()).reshape(-1)
    slot = s["slot"].long()
    return torch.where(slot < 0, 0.0, rows[slot.clamp(min=0)])


def _exact_gate(s):
    return s["alpha"] if s["gate"] is None else s["alpha"] * s["gate"].double()


def _exact_norm_in(case, s):
    r = s["x"].double()
    if s["residual"]:
        r = r + _exact_gate(s) * s["u"].double()
    rms = (r.pow(2).sum(1) / case["d"] + NORM_EPS).sqrt()
    out = {"n": r / rms[:, None] * s["w"].double(), "rstd": 1 / rms}
    return {**out, "r": r} if s["residual"] else out


def _exact_norm_out(case, s):
    y = s["u"].double()
    rms = (y.pow(2).sum(1) / case["d"] + NORM_EPS).sqrt()
    return {"out": s["x"].double() + _exact_gate(s) * s["w"].double() * y / rms[:, None], "rstd": 1 / rms}


def _exact_norm_in_bwd(case, s):
    """Row by row: the Jacobian of x / rms(x) is (I - xhat xhat^T / d) / rms, with the saved 1 / rms."""
    r, c = s["x"].double(), s["rstd"].double()[:, None]
    a = s["do"].double() * s["w"].double()
    dx = a * c - r * c.pow(3) * (a * r).sum(1, keepdim=True) / case["d"]
    dw = (s["do"].double() * r * c).sum(0)
    if not s["residual"]:
        return {"dx": dx, "dw": dw}
    dx = dx + s["dr"].double()
    dg = s["u"].double() * dx * s["alpha"]
    dg = None if s["gate"] is None else dg.sum(1, keepdim=True) if case["gate"] == "token" else dg.sum(0)
    return {"dx": dx, "dw": dw, "du": dx * _exact_gate(s), "dgate": dg}


def _exact_norm_out_bwd(case, s):
    y, c, do = s["u"].double(), s["rstd"].double()[:, None], s["do"].double()
    w, g = s["w"].double(), _exact_gate(s)
    a = do * g * w
    dy = a * c - y * c.pow(3) * (a * y).sum(1, keepdim=True) / case["d"]
    each = s["alpha"] * do * w * y * c
    dg = None if s["gate"] is None else each.sum(1, keepdim=True) if case["gate"] == "token" else each.sum(0)
    return {"dy": dy, "dw": (do * g * y * c).sum(0), "dgate": dg}


def _exact_adamw(case, s):
    t = s["step"] + 1
    out = {"p": [], "m": [], "v": [], "ms": [], "vs": [], "master": []}
    for i, p in enumerate(s["p"] if s["master"] is None else s["master"]):
        g, n = s["g"][i].double(), p.numel()
        at = torch.arange(n, device=p.device)
        if case["bits"] == 32:
            m, v = s["m"][i].double(), s["v"][i].double()
        else:
            m = s["m"][i].view(torch.float8_e4m3fn).double() * s["ms"][i].double()[at // BLOCK]
            v = (s["v"][i].view(torch.float8_e4m3fn).double() * s["vs"][i].double()[at // BLOCK]).square()
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g * g
        new = p.double() * (1 - LR * DECAY) - LR * m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
        del g
        out["p"].append(new)
        out["master"].append(new)
        if case["bits"] == 32:
            out["m"].append(m)
            out["v"].append(v)
            continue
        word = (at * GOLD + _mix((s["seed"] + t * GOLD + i * ROOT3) & MASK32)) & MASK32
        word = ((word ^ (word >> 16)) * ROOT2) & MASK32
        word = word ^ (word >> 15)
        for x, name, u in ((m, "m", word % 65536), (v.sqrt(), "v", word // 65536)):
            blocks = -(-n // BLOCK)
            top = torch.zeros(blocks, dtype=torch.float64, device=p.device)
            top = top.scatter_reduce_(0, at // BLOCK, x.abs(), "amax")
            y = x.abs() * (448 / top.clamp(min=1e-300))[at // BLOCK]
            unit = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
            cell = torch.floor(y / unit + (u.double() + 0.5) / 65536) * unit
            out[name].append(torch.copysign(cell.clamp(max=448.0), x))
            out[name + "s"].append(top / 448)
    if s["master"] is None:
        del out["master"]
    if case["bits"] == 32:
        del out["ms"], out["vs"]
    return {k: [torch.cat(v)] if len(s["p"]) > 8 else v for k, v in out.items()}


# ---------------------------------------------------------------- the least work

def work(case):
    op = case["op"]
    b = 4 if case.get("dtype", "f32") == "f32" else 2
    if op in ("router", "router_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        mask = T if case["masked"] else 0
        if op == "router":
            return {"bytes": T * E * b + mask + 8 * T * k + 8 * E + 8, "flops": 8 * T * E}
        return {"bytes": 2 * T * E * b + mask + 8 * T * k + 4 * E + 12, "flops": 20 * T * E}
    if op == "gate_grad":
        rows = case["T"] * case["k"]
        used = rows * case["routed"]
        return {"bytes": 2 * used * case["d_ff"] * b + 8 * rows, "flops": 2 * used * case["d_ff"]}
    if op == "adamw":
        p = {"f32": 8, "bf16": 4, "master": 10}[case["p"]]
        per = p + (4 if case["g"] == "f32" else 2) + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)
        return {"bytes": per * case["total"], "flops": 16 * case["total"]}
    T, d = case["T"], case["d"]
    gate = {"none": 0, "token": 4 * T, "feature": 4 * d}[case["gate"]]
    if op == "norm_in":
        full = case["residual"]
        return {"bytes": (4 if full else 2) * T * d * b + d * b + 4 * T + (gate if full else 0), "flops": 6 * T * d}
    if op == "norm_in_bwd":
        full = case["residual"]
        return {"bytes": (6 if full else 3) * T * d * b + d * b + 4 * d + 4 * T + (2 * gate if full else 0),
                "flops": 12 * T * d}
    if op == "norm_out":
        return {"bytes": 3 * T * d * b + d * b + 4 * T + gate, "flops": 6 * T * d}
    return {"bytes": 3 * T * d * b + d * b + 4 * d + 4 * T + 2 * gate, "flops": 12 * T * d}
