"""The operators in a second context of the device: the kernels' attributes and the address of the
error word belong to a context, and what was kept of the first one's must not be used in it.
In a child process, through the C ABI and the driver's API alone."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = r"""
import ctypes, sys
from expert_routed_ffn_gb300 import capi

cuda = ctypes.CDLL("libcuda.so.1")
lib = capi.load()


def cu(name, *args):
    r = getattr(cuda, name)(*args)
    assert r == 0, (name, r)


def buffer(data):
    p = ctypes.c_uint64()
    cu("cuMemAlloc_v2", ctypes.byref(p), ctypes.c_size_t(len(data)))
    cu("cuMemcpyHtoD_v2", p, data, ctypes.c_size_t(len(data)))
    return p


def context(offsets_first):
    ROWS, E, N, K = 48, 2, 64, 128
    one = b"\x80\x3f"  # bf16 1.0
    X, W, dY = buffer(one * (ROWS * K)), buffer(one * (E * N * K)), buffer(one * (ROWS * N))
    Y, dW = buffer(bytes(4 * ROWS * N)), buffer(bytes(4 * E * N * K))
    mx = [buffer(b"\x22" * n) for n in (ROWS * K // 2, E * N * K // 2)]  # E2M1 1.0 twice
    ms = [buffer(b"\x7f" * n) for n in (ROWS * K // 32, E * N * K // 32)]

    def ints(*v):
        return buffer(b"".join(x.to_bytes(4, "little", signed=True) for x in v))

    good, bad = ints(0, 20, 48), ints(0, 49, 48)

    def run(offs):
        for st in (lib.moe_grouped_forward(X.value, W.value, offs.value, ROWS, E, N, K, 1, Y.value, None),
                   lib.moe_grouped_wgrad(dY.value, X.value, offs.value, ROWS, E, N, K, 1, 0, dW.value, None),
                   lib.moe_mx_grouped_forward(mx[0].value, ms[0].value, mx[1].value, ms[1].value, offs.value, ROWS, E, N, K,
                                              1, Y.value, None)):
            assert st == 0, lib.moe_last_error()
        return lib.moe_operators_status()

    def floats(p, n):
        host = (ctypes.c_float * n)()
        cu("cuMemcpyDtoH_v2", host, p, ctypes.c_size_t(4 * n))
        return host[:]

    for offs in ((good, bad, good) if offsets_first else (bad, good)):
        assert run(offs) == (0 if offs is good else capi.MOE_ERR_DEVICE_CHECK), lib.moe_last_error()
    assert set(floats(Y, ROWS * N)) == {float(K)}
    assert floats(dW, E * N * K) == [20.0] * (N * K) + [28.0] * (N * K)


cu("cuInit", 0)
first, second = ctypes.c_void_p(), ctypes.c_void_p()
cu("cuDevicePrimaryCtxRetain", ctypes.byref(first), 0)
cu("cuCtxSetCurrent", first)
context(True)
cu("cuCtxCreate_v2", ctypes.byref(second), 0, 0)  # and makes it the current one
context(False)
cu("cuCtxSetCurrent", first)
context(True)
cu("cuCtxDestroy_v2", second)
cu("cuCtxCreate_v2", ctypes.byref(second), 0, 0)  # a new one, perhaps where the other was
context(False)
cu("cuCtxDestroy_v2", second)
cu("cuCtxSetCurrent", first)
context(True)
print("contexts ok")
"""


def test_second_context():
    from expert_routed_ffn_gb300 import build, capi
    build.build()
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=240, cwd=capi.ROOT,
                       env={**os.environ, "PYTHONPATH": capi.ROOT})
    assert r.returncode == 0 and "contexts ok" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])
