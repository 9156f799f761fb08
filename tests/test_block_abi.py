"""Host-side checks of the operators around the layer: refusals that return before any device work."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from moe_expert_ffn_amd import binding as B

P = ctypes.c_void_p(256)
ARG, UNSUP, WS = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE


def _router(E=16, k=2, dtype=0, score=0, renorm=1, scale=1.0):
    return B.Router(E, k, dtype, score, renorm, scale)


def _fwd(R, logits=P, ld=16, T=4, ids=P, gates=P, ws=P, n=1 << 20, losses=P):
    return B.load().moe_router_forward(ctypes.byref(R), logits, ld, None, T, ids, gates, P, P, P, losses, P,
                                       ws, n, None)


def test_router_refusals():
    for bad in (dict(E=0), dict(k=0), dict(k=17), dict(dtype=2), dict(score=2), dict(score=-1),
                dict(scale=float("inf")), dict(scale=float("nan"))):
        assert _fwd(_router(**bad)) == ARG, bad
        assert B.load().moe_router_workspace_size(ctypes.byref(_router(**bad)), 4) == 0
    assert _fwd(_router(), ld=15) == ARG
    assert _fwd(_router(), T=-1) == ARG
    assert _fwd(_router(E=1025), ld=1025) == UNSUP
    assert _fwd(_router(E=64, k=33), ld=64) == UNSUP
    assert _fwd(_router(), T=1 << 30) == UNSUP
    for name in ("logits", "ids", "gates", "losses"):
        assert _fwd(_router(), **{name: None}) == ARG, name
    assert _fwd(_router(), ws=None) == WS
    assert _fwd(_router(), ws=ctypes.c_void_p(8)) == WS
    assert _fwd(_router(), n=64) == WS
    bwd = lambda R, ld=16, T=4, ids=P, out=P, ld_out=16: B.load().moe_router_backward(
        ctypes.byref(R), P, ld, None, T, ids, P, P, P, P, out, ld_out, None)
    assert bwd(_router(), ld_out=15) == ARG
    assert bwd(_router(), ids=None) == ARG
    assert bwd(_router(), out=None) == ARG
    assert bwd(_router(E=0)) == ARG
    with pytest.raises(B.MoeError, match="not supported"):
        B.make_router(16, 17)
    with pytest.raises(B.MoeError, match="score"):
        B.make_router(16, 2, score="linear")
    with pytest.raises(B.MoeError, match="element type"):
        B.make_router(16, 2, torch.float16)


def test_gate_grad_refusals():
    f = B.load().moe_gate_grad
    assert f(P, P, 0, P, -1, 4, 64, P, None) == ARG
    assert f(P, P, 0, P, 4, -1, 64, P, None) == ARG
    assert f(P, P, 2, P, 4, 4, 64, P, None) == ARG
    assert f(P, P, 0, P, 4, 4, 0, P, None) == ARG
    assert f(P, P, 0, P, 4, 4, 96, P, None) == UNSUP
    assert f(None, P, 0, P, 4, 4, 64, P, None) == ARG
    assert f(P, P, 0, None, 4, 4, 64, P, None) == ARG
    L = B.Layer(8, 128, 64, 0, 0, 16, 32, None, None)
    assert B.load().moe_backward_gates(ctypes.byref(L), P, P, P, P, P, 4, 2, 16, 4, 1, *([P] * 9), None, P, P,
                                       1 << 30, 0, None, None, None) == ARG
    assert B.load().moe_backward_gates(ctypes.byref(L), P, P, P, P, P, 4, 2, 16, 3, 1, *([P] * 9), P, P, P,
                                       1 << 30, 0, None, None, None) == UNSUP


def _norm(T=4, d=8, dtype=0, w_dtype=0, kind=0, alpha=1.0, eps=1e-6, w=256, gate=None):
    return B.Norm(T, d, dtype, w_dtype, kind, alpha, eps, w, gate)


def test_norm_refusals():
    lib = B.load()
    nin = lambda N, x=P, ldx=8, u=P, ldu=8, r=P, ldr=8, n=P, ldn=8, s=P: lib.moe_norm_in(
        ctypes.byref(N), x, ldx, u, ldu, r, ldr, n, ldn, s, None)
    nout = lambda N, y=P, ldy=8, x=P, ldx=8, o=P, ldo=8, s=P: lib.moe_norm_out(
        ctypes.byref(N), y, ldy, x, ldx, o, ldo, s, None)
    inb = lambda N, u=P, du=P, dg=None, ws=P, n=1 << 24, dw=P, ld=8: lib.moe_norm_in_backward(
        ctypes.byref(N), P, ld, P, 8, P, 8, u, 8, P, P, 8, du, 8, dw, dg, ws, n, None)
    outb = lambda N, dg=None, ws=P, n=1 << 24, dw=P, ld=8: lib.moe_norm_out_backward(
        ctypes.byref(N), P, ld, P, 8, P, P, 8, dw, dg, ws, n, None)
    for bad in (dict(d=0), dict(T=-1), dict(dtype=2), dict(kind=3), dict(kind=-1), dict(eps=0.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(alpha=float("nan")), dict(w=None),
                dict(kind=1), dict(kind=0, gate=256)):
        for f in (nin, nout, inb, outb):
            assert f(_norm(**bad)) == ARG, (bad, f)
    for f in (nin, nout, inb, outb):
        assert f(_norm(dtype=0, w_dtype=1)) == UNSUP
    assert nin(_norm(d=16385), ldx=20000) == UNSUP
    for name in ("x", "n", "s"):
        assert nin(_norm(), **{name: None}) == ARG
    for name in ("ldx", "ldu", "ldr", "ldn"):
        assert nin(_norm(), **{name: 7}) == ARG
    for name in ("y", "x", "o", "s"):
        assert nout(_norm(), **{name: None}) == ARG
    for name in ("ldx", "ldy", "ldo"):
        assert nout(_norm(), **{name: 7}) == ARG
    gate = dict(kind=2, gate=256)
    assert nin(_norm(**gate), u=None) == ARG                      # a gate of nothing
    assert inb(_norm(**gate), dg=None) == ARG
    assert outb(_norm(**gate), dg=None) == ARG
    assert inb(_norm(), dg=P) == ARG and outb(_norm(), dg=P) == ARG
    assert inb(_norm(), u=None) == ARG and inb(_norm(), du=None) == ARG
    assert inb(_norm(), dw=None) == ARG and outb(_norm(), dw=None) == ARG
    assert inb(_norm(), ld=7) == ARG and outb(_norm(), ld=7) == ARG
    assert inb(_norm(), ws=None) == WS and outb(_norm(), n=16) == WS
    assert lib.moe_norm_workspace_size(-1, 8) == 0 and lib.moe_norm_workspace_size(4, 0) == 0
    assert lib.moe_norm_workspace_size(4, 16385) == 0


def test_adamw_refusals():
    lib = B.load()

    def prepare(count=1, bits=32, ws=P, n=1 << 20, **kw):
        f = dict(p=4096, master=None, g=8192, m=12288, v=16384, m_scale=None, v_scale=None, n=16, p_dtype=0,
                 g_dtype=0)
        f.update(kw)
        arr = (B.AdamwTensor * 1)(B.AdamwTensor(**f))
        return lib.moe_adamw_prepare(arr, count, bits, ctypes.byref(B.AdamwList()), ws, n, None)

    assert prepare(count=-1) == ARG and prepare(count=4097) == ARG
    assert prepare(bits=16) == UNSUP
    for name in ("p", "g", "m", "v"):
        assert prepare(**{name: None}) == ARG, name
        assert prepare(**{name: 4098}) == ARG, name               # off its element size
    assert prepare(p_dtype=2) == ARG and prepare(g_dtype=3) == ARG
    assert prepare(bits=8) == ARG                                 # no scales
    assert prepare(master=20480) == ARG                           # of an fp32 parameter
    assert prepare(m=4096 + 32) == ARG                            # inside p
    assert prepare(g=4096) == ARG                                 # the gradient on p
    assert prepare(ws=None) == WS and prepare(ws=ctypes.c_void_p(8)) == WS
    arr = (B.AdamwTensor * 1)(B.AdamwTensor(n=-1))
    assert lib.moe_adamw_prepare(arr, 1, 32, ctypes.byref(B.AdamwList()), P, 1 << 20, None) == ARG
    arr = (B.AdamwTensor * 1)(B.AdamwTensor(p=4096, g=8192, m=12288, v=16384, n=(1 << 43) + 1))
    assert lib.moe_adamw_prepare(arr, 1, 32, ctypes.byref(B.AdamwList()), P, 1 << 20, None) == UNSUP
    arr = (B.AdamwTensor * 1)(B.AdamwTensor(p=1 << 50, g=1 << 51, m=1 << 52, v=1 << 53, n=(1 << 24) * 2048))
    assert lib.moe_adamw_prepare(arr, 1, 32, ctypes.byref(B.AdamwList()), P, 1 << 20, None) == UNSUP
    assert lib.moe_adamw_prepare(None, 1, 32, ctypes.byref(B.AdamwList()), P, 1 << 20, None) == ARG
    assert lib.moe_adamw_workspace_size(-1) == 0 and lib.moe_adamw_workspace_size(4097) == 0
    L = B.AdamwList(256, 1, 32, 0)
    ok = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1)
    for bad in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=float("nan")), dict(eps=0.0),
                dict(eps=float("inf")), dict(lr=float("nan")), dict(weight_decay=float("inf")), dict(step=0)):
        assert lib.moe_adamw(ctypes.byref(L), ctypes.byref(B.AdamwHyper(**{**ok, **bad})), None) == ARG, bad
    assert lib.moe_adamw(None, ctypes.byref(B.AdamwHyper(**ok)), None) == ARG
    assert lib.moe_adamw(ctypes.byref(B.AdamwList(None, 1, 32, 5)), ctypes.byref(B.AdamwHyper(**ok)), None) == ARG
    assert lib.moe_adamw(ctypes.byref(B.AdamwList(256, 1, 16, 5)), ctypes.byref(B.AdamwHyper(**ok)), None) == ARG


def test_binding_takes_device_tensors_only():
    """Buffers in host memory are refused by name before any pointer is taken."""
    x = torch.zeros(4, 8)
    R = B.make_router(8, 2)
    with pytest.raises(B.MoeError, match="current device"):
        B.router_forward(R, x, B.alloc_router(R, 4, "cpu"), B.router_workspace(R, 4, "cpu"),
                         torch.zeros(1, dtype=torch.int32))
    with pytest.raises(B.MoeError, match="current device"):
        B.norm_in(x, torch.ones(8), 1e-6, x.clone(), torch.zeros(4))
    with pytest.raises(B.MoeError, match="current device"):
        B.norm_out(x, x, torch.ones(8), 1e-6, x.clone(), torch.zeros(4))
    with pytest.raises(B.MoeError, match="current device"):
        B.gate_grad(x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(4))
    with pytest.raises(B.MoeError, match="current device"):
        B.make_adamw([x], [x], [x], [x])


@pytest.mark.parametrize("make,why", [
    (lambda: torch.zeros(8, 4).t(), "strides"), (lambda: torch.zeros(1, 8).expand(4, 8), "strides"),
    (lambda: torch.zeros(4, 9), "expected"), (lambda: torch.zeros(32), "expected"),
    (lambda: torch.zeros(4, 8).double(), "expected")])
def test_rows_that_are_no_rows(make, why):
    with pytest.raises(B.MoeError, match=why):
        B._rows(make(), 4, 8, torch.float32, "x")


def test_row_strides():
    t = torch.zeros(6, 20)
    assert B._rows(t[:, 3:11], 6, 8, torch.float32, "x") == 20
    assert B._rows(t[2:3, :8], 1, 8, torch.float32, "x") == 20
    assert B._rows(torch.zeros(8).as_strided((1, 8), (3, 1)), 1, 8, torch.float32, "x") == 8
    assert B._rows(t[::2, :8], 3, 8, torch.float32, "x") == 40
    assert B._rows(torch.zeros(0, 8), 0, 8, torch.float32, "x") == 8
    assert B._rows(torch.zeros(5, 1), 5, 1, torch.float32, "x") == 1


@pytest.mark.parametrize("E", [1, 16, 64, 65, 128, 129, 160, 256, 257, 384, 512, 513, 1024])
def test_router_workspace_serves_every_smaller_batch(E):
    size = lambda T: B.load().moe_router_workspace_size(ctypes.byref(_router(E=E, k=1)), T)
    Ts = sorted({max(0, b + o) for b in [0] + [1 << i for i in range(23)] for o in range(-9, 10)})
    sizes = [size(T) for T in Ts]
    assert all(s > 0 for s in sizes)
    assert sizes == sorted(sizes), next((Ts[i], sizes[i - 1], sizes[i]) for i in range(1, len(Ts)) if sizes[i] < sizes[i - 1])


def test_norm_workspace_serves_every_smaller_batch():
    Ts = sorted({max(0, b + o) for b in [0] + [1 << i for i in range(23)] for o in (-2, -1, 0, 1, 2)})
    for d in (1, 7, 64, 1023, 4096, 16384):
        sizes = [B.load().moe_norm_workspace_size(T, d) for T in Ts]
        assert sizes == sorted(sizes) and sizes[0] > 0


def test_adamw_numbers_that_fp32_does_not_hold():
    L = B.AdamwList(256, 1, 32, 0)
    ok = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1)
    rc = lambda **kw: B.load().moe_adamw(ctypes.byref(L), ctypes.byref(B.AdamwHyper(**{**ok, **kw})), None)
    for bad in (dict(eps=1e-46), dict(eps=1e-38), dict(eps=1e39), dict(lr=1e39), dict(lr=-1e39),
                dict(weight_decay=1e39), dict(eps=-1e-8)):
        assert rc(**bad) == ARG, bad
    for good in (dict(), dict(eps=2.0 ** -126), dict(lr=0.0), dict(lr=-1e-3), dict(lr=1e38), dict(weight_decay=1e38)):
        assert rc(**good) == B.MOE_OK, good


@pytest.mark.parametrize("make,T,cols", [
    (lambda: torch.empty((2 ** 32 + 5, 1), device="meta"), 2 ** 32 + 5, 1),              # 5 rows in 32 bits
    (lambda: torch.empty((2 ** 31, 2), device="meta"), 2 ** 31, 2),
    (lambda: torch.empty((1, 2 ** 32 + 8), device="meta"), 1, 2 ** 32 + 8),
    (lambda: torch.empty_strided((3, 8), (2 ** 32 + 8, 1), device="meta"), 3, 8),        # rows 8 apart
    (lambda: torch.empty_strided((2 ** 32 + 5, 1), (1, 2), device="meta"), 2 ** 32 + 5, 1)])
def test_sizes_beyond_32_bits_are_refused(make, T, cols):
    with pytest.raises(B.MoeError, match="32-bit"):
        B._rows(make(), T, cols, torch.float32, "x")


def test_numbers_beyond_32_bits_are_refused():
    R = _router()
    for call in (lambda: B.router_workspace(R, 2 ** 32 + 5, "cpu"), lambda: B.norm_workspace(2 ** 32 + 5, 8, "cpu"),
                 lambda: B.norm_workspace(5, 2 ** 32 + 8, "cpu"), lambda: B.make_router(2 ** 32 + 16, 2),
                 lambda: B.make_router(16, 2 ** 32 + 2)):
        with pytest.raises(B.MoeError, match="32-bit"):
            call()
    big = torch.empty_strided((3, 8), (2 ** 31 - 1, 1), device="meta")
    assert B._rows(big, 3, 8, torch.float32, "x") == 2 ** 31 - 1
    one = torch.empty_strided((1, 8), (2 ** 40, 1), device="meta")       # one row has no stride
    assert B._rows(one, 1, 8, torch.float32, "x") == 8


def test_the_library_has_no_allocator():
    """No entry point allocates memory, the host's neither: the library imports nothing that could."""
    B.load()
    r = subprocess.run(["nm", "-D", "--undefined-only", os.path.join(os.path.dirname(B.__file__), "libmoe_ffn.so")],
                       capture_output=True, text=True, check=True)
    names = {line.split()[-1].split("@")[0] for line in r.stdout.splitlines()}
    bad = {n for n in names if n.startswith(("malloc", "calloc", "realloc", "posix_memalign", "_Zn", "hipMalloc", "hipHostMalloc",
                                             "hipFree", "hipStreamSynchronize", "hipDeviceSynchronize", "hipMemset"))}
    assert not bad and "hipLaunchKernel" in names


def test_adamw_lists_that_share_memory():
    """Every pair of buffers of a list's first and last tensor, whole or by the last four bytes."""
    sizes = {"p": 2, "master": 4, "g": 2, "m": 1, "v": 1, "m_scale": 4, "v_scale": 4}     # bytes of an element
    n, far = 256, 1 << 20
    count = {k: n if "scale" not in k else n // 128 for k in sizes}

    def rc(moved, onto, by, total):
        arr = (B.AdamwTensor * total)()
        for i in range(total):
            for j, k in enumerate(sizes):
                setattr(arr[i], k, far * (7 * i + j + 1))
            arr[i].n, arr[i].p_dtype, arr[i].g_dtype = n, B.MOE_BF16, B.MOE_BF16
        setattr(arr[0], moved, getattr(arr[total - 1], onto) + by)
        return B.load().moe_adamw_prepare(arr, total, 8, ctypes.byref(B.AdamwList()), P, 1 << 30, None)

    for total in (2, 33):
        for a in sizes:
            for b in sizes:
                end = count[b] * sizes[b]
                if a == b == "g":
                    continue                                     # gradients may be shared
                assert rc(a, b, end - 4, total) == ARG, (a, b)
                assert rc(a, b, 0, total) == ARG, (a, b)


def test_router_kernels_are_those_that_calls_reach():
    """Lanes and experts a lane of the compiled variants: 16 experts in fewer than 64 lanes only forward."""
    B.load()
    with open(os.path.join(os.path.dirname(B.__file__), "libmoe_ffn.so"), "rb") as f:
        data = f.read()                                           # the kernels' names stand in their code objects
    shapes = {"k_router": set(), "k_router_bwd": set()}
    for name, lanes, each in re.findall(rb"\d+(k_router|k_router_bwd)I[ft]Li(\d+)ELi(\d+)E", data):
        shapes[name.decode()].add((int(lanes), int(each)))
    both = {(8, 8), (16, 8), (32, 8), (64, 8), (64, 16)}
    assert shapes["k_router_bwd"] == both and shapes["k_router"] == both | {(16, 16), (32, 16)}
