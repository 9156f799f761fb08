"""Host-side checks of the int8 rows and layers: refusals before any device work, and pins of their oracle."""
import ctypes

import numpy as np
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from oracle import int8 as oi8

P = ctypes.c_void_p(256)
ARG, UNSUP, WS = B.MOE_ERR_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE


def test_quantizer_refusals():
    q = lambda src=P, ld=8, dt=0, rows=4, cols=8, codes=P, scales=P: B.load().moe_quantize_int8_rows(
        src, ld, dt, rows, cols, codes, scales, None)
    assert q(rows=-1) == ARG and q(cols=0) == ARG and q(ld=7) == ARG and q(dt=2) == ARG and q(dt=-1) == ARG
    assert q(src=None) == ARG and q(codes=None) == ARG and q(scales=None) == ARG
    x = torch.zeros(4, 8)
    with pytest.raises(B.MoeError, match="current device"):
        B.quantize_int8_rows(x, torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4))


def test_quantizer_refuses_shared_memory_and_rows_past_32_bits():
    """Rows are taken in any order: codes over a row that is still to be read would be its own input."""
    def q(src, codes, scales, cols=64, ld=64, dt=B.MOE_BF16):
        return B.load().moe_quantize_int8_rows(ctypes.c_void_p(src), ld, dt, 4, cols, ctypes.c_void_p(codes),
                                               ctypes.c_void_p(scales), None)
    at = 1 << 20                                  # src is 4 rows of 128 bytes there
    assert q(at, at, 1 << 22) == ARG and q(at, at + 511, 1 << 22) == ARG and q(at, at - 255, 1 << 22) == ARG
    assert q(at, 1 << 22, at + 508) == ARG and q(at, 1 << 22, at - 12) == ARG
    assert q(at, 1 << 22, (1 << 22) + 252) == ARG and q(at, 1 << 22, (1 << 22) - 12) == ARG
    assert q(at, 1 << 45, 1 << 46, cols=(1 << 30) + 1, ld=(1 << 30) + 1) == UNSUP


def _layer(E=8, d=256, f=128, act=B.MOE_BF16, s1=256, s2=256):
    return B.Layer(E, d, f, act, B.MOE_INT8, 256, 256, s1, s2)


def _forward(L, z=None, flags=0, ws=P, n=1 << 40):
    return B.load().moe_forward(ctypes.byref(L), P, P, P, 40, 2, 16, 2, P, P, P, P, P, P, z, P, ws, n, flags, None, None, None)


def test_layer_refusals():
    assert _forward(_layer(s1=None)) == ARG and _forward(_layer(s2=None)) == ARG
    assert _forward(_layer(), z=P) == ARG                                        # nothing to save for a backward pass
    assert _forward(_layer(), flags=1) == ARG and _forward(_layer(), flags=2) == ARG
    assert _forward(_layer(act=B.MOE_F32)) == UNSUP
    assert _forward(_layer(d=192)) == UNSUP and _forward(_layer(f=96)) == UNSUP and _forward(_layer(E=513)) == UNSUP
    assert _forward(_layer(d=131072 + 128, f=64)) == UNSUP and _forward(_layer(f=131072 + 64, d=128)) == UNSUP
    assert _forward(_layer(), ws=None) == WS and _forward(_layer(), n=4096) == WS
    for i, at in ((5, 264), (6, 264), (7, 258), (8, 257)):                       # weights off 16 bytes, scales off 4
        f = [8, 256, 128, B.MOE_BF16, B.MOE_INT8, 256, 256, 256, 256]
        f[i] = at
        assert _forward(B.Layer(*f)) == ARG, i
    L = _layer()
    assert B.load().moe_backward(ctypes.byref(L), P, P, P, P, P, 40, 2, 16, 2, 1, *([P] * 9), P, P, 1 << 40, 0, None, None,
                                 None) == UNSUP
    size = lambda back: B.load().moe_workspace_size(ctypes.byref(L), 40, 2, 16, 2, 1, back)
    assert size(0) > 0 and size(1) == 0
    assert _forward(B.Layer(8, 256, 128, B.MOE_BF16, 4, 256, 256, 256, 256)) == ARG


@pytest.mark.parametrize("beta", [1, 16, 50, 128, 300])
@pytest.mark.parametrize("d,f", [(256, 256), (2048, 768), (384, 192)])
def test_workspace_serves_every_smaller_batch(beta, d, f):
    L = _layer(E=32, d=d, f=f)
    size = lambda T: B.load().moe_workspace_size(ctypes.byref(L), T, 4, beta, 8, 0, 0)
    Ts = sorted({max(0, b + o) for b in [0, 128] + [1 << i for i in range(13)] for o in range(-3, 4)})
    sizes = [size(T) for T in Ts]
    assert all(sizes) and sizes == sorted(sizes)


def test_binding_refusals():
    class Fake:
        is_cuda, device = True, torch.device("cuda", 0)

        def __init__(self, dtype, *shape):
            self.dtype, self.shape = dtype, torch.Size(shape)

        def is_contiguous(self):
            return True

        def dim(self):
            return len(self.shape)

        def numel(self):
            return self.shape.numel()

        def data_ptr(self):
            return 256

    w1, w2 = Fake(torch.int8, 4, 256, 128), Fake(torch.int8, 4, 128, 128)
    s = lambda n: Fake(torch.float32, n)
    assert B.make_layer(w1, w2, s(1024), s(512)).w_dtype == B.MOE_INT8
    for bad in ((None, s(512)), (s(1024), None), (s(1023), s(512)), (s(1024), s(511)), (Fake(torch.float64, 1024), s(512))):
        with pytest.raises(B.MoeError):
            B.make_layer(w1, w2, *bad)
    with pytest.raises(B.MoeError, match="bfloat16"):
        B.make_layer(w1, w2, s(1024), s(512), torch.float32)


def test_oracle_pins():
    c, s = oi8.quantize_rows([[1.0, 0.5, -0.5, 0.25, 0.0], [0, 0, 0, 0, 0], [127, 1.5, 2.5, -3.5, -127],
                              [np.inf, 1, 1, 1, 1], [1, np.nan, 1, 1, 1], [2.0 ** -101] * 5])
    assert c.tolist() == [[127, 64, -64, 32, 0], [0] * 5, [127, 2, 2, -4, -127], [0] * 5, [0] * 5, [0] * 5]
    assert s[0] == np.float32(1) / np.float32(127) and s[1] == 0 and s[2] == 1 and np.isnan(s[3:5]).all() and s[5] == 0
    # one expert, exact numbers: x = (127, 0), G = 127 * 2, U = 127 * 1 at scale 1
    w1 = np.zeros((1, 2, 2), np.int8)
    w1[0, 0], w1[0, 1] = (2, 0), (1, 0)
    y = oi8.forward([[127.0, 0.0]], w1, np.full((1, 2), 2.0 ** -7), np.full((1, 2, 1), 100, np.int8), np.ones((1, 2)),
                    np.array([[0]]), np.array([[0.5]]))
    g, u = 254 / 128, 127 / 128
    a = float(torch.tensor(g / (1 + np.exp(-g)) * u).bfloat16())
    np.testing.assert_allclose(y, [[0.5 * 100 * 127 * float(np.float32(a) / np.float32(127))] * 2], rtol=1e-12)
