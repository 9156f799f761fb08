"""Host side: an error of any launch inside a call of several is reported.

A small library stands in for the HIP calls that the launches make: the launch of a given number fails, with
an error that stays until it is read, as HIP's does.  Nothing reaches a GPU."""
import os
import subprocess
import sys

import pytest

SHIM = r"""
static int fail_at, seen, last;
void shim_start(int n) { fail_at = n; seen = 0; last = 0; }
int shim_seen(void) { return seen; }
int hipLaunchKernel(const void* f) { if (++seen == fail_at) { last = 1; return 1; } return 0; }
int hipGetLastError(void) { int e = last; last = 0; return e; }
int __hipPushCallConfiguration(void) { return 0; }
int __hipPopCallConfiguration(void) { return 0; }
int hipFuncSetAttribute(void) { return 0; }
int hipGetDevice(int* d) { *d = 0; return 0; }
int hipDeviceGetAttribute(int* v, int a, int d) { *v = 256; return 0; }
int hipOccupancyMaxActiveBlocksPerMultiprocessor(int* v) { *v = 1; return 0; }
"""

RUN = r"""
import ctypes, sys
shim = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
from moe_expert_ffn_amd import binding as B
lib = B.load()
P = ctypes.c_void_p(256)
act, w, flags, d, dff, call = *map(int, sys.argv[3:8]), sys.argv[8]
scale = 256 if w == B.MOE_FP8_E4M3 else None
L = B.Layer(8, d, dff, act, w, 256, 256, scale, scale)
sizes = (300, 2, 128, 4, 1)
def once():
    if call == "forward":
        return lib.moe_forward(ctypes.byref(L), P, P, P, *sizes[:4], P, P, P, P, P, P, P, P, P, 1 << 40, flags,
                               None, None, None)
    f, more = (lib.moe_backward, []) if call == "backward" else (lib.moe_backward_gates, [P])
    return f(ctypes.byref(L), P, P, P, P, P, *sizes, *([P] * 9), *more, P, P, 1 << 40, flags, None, None, None)
shim.shim_start(0)
assert once() == B.MOE_OK, once()
n = shim.shim_seen()
assert n >= 3, n
lost = []
for i in range(1, n + 1):
    shim.shim_start(i)
    if once() != B.MOE_ERR_HIP:
        lost.append(i)
assert not lost, f"launches {lost} of {n} failed unnoticed"
shim.shim_start(0)
assert once() == B.MOE_OK
print("launches", n)
"""

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16, FP8 = 0, 1, 2


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    at = tmp_path_factory.mktemp("shim")
    (at / "shim.c").write_text(SHIM)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(at / "shim.so"), str(at / "shim.c")], check=True)
    return str(at / "shim.so")


def _every_launch(shim, call, act, w, flags, d=512, dff=256):
    r = subprocess.run([sys.executable, "-c", RUN, shim, ROOT, *map(str, (act, w, flags, d, dff)), call],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("call", ["backward", "backward_gates"])
@pytest.mark.parametrize("act,w,flags", [(F32, F32, 0), (BF16, BF16, 0), (BF16, BF16, 1)])
def test_failed_launches_of_the_backward_pass(shim, call, act, w, flags):
    _every_launch(shim, call, act, w, flags)


@pytest.mark.parametrize("call,flags,d,dff", [
    ("forward", 0, 512, 256), ("forward", 2, 512, 256), ("forward", 0, 384, 128),
    ("backward", 0, 512, 256), ("backward", 2, 512, 256), ("backward_gates", 0, 512, 256),
    ("backward_gates", 2, 512, 256), ("backward_gates", 0, 256, 128), ("backward", 0, 384, 128)])
def test_failed_launches_of_e4m3_layers(shim, call, flags, d, dff):
    """Their quantizers are launches of the same calls."""
    _every_launch(shim, call, BF16, FP8, flags, d, dff)
