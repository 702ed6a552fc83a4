"""The calls over the cache in two CUDA contexts of one process, the device's primary one and an engine's own, and
behind a reset of the process's device state."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = r"""
import ctypes as C, math, sys
import numpy as np
import speculative_decoding_verification_token_gb300 as sv
cu = C.CDLL("libcuda.so.1")
def ok(code):
    assert code == 0, code
ok(cu.cuInit(0))
dev, first, second = C.c_int(), C.c_void_p(), C.c_void_p()
ok(cu.cuDeviceGet(C.byref(dev), 0))
ok(cu.cuDevicePrimaryCtxRetain(C.byref(first), dev))
ok(cu.cuCtxCreate_v2(C.byref(second), C.c_uint(0), dev))
L = sv.lib()

def up(a):
    a = np.ascontiguousarray(a)
    p = C.c_void_p()
    ok(cu.cuMemAlloc_v2(C.byref(p), C.c_size_t(max(a.nbytes, 16))))
    ok(cu.cuMemcpyHtoD_v2(p, a.ctypes.data_as(C.c_void_p), C.c_size_t(a.nbytes)))
    return p

def down(p, like):
    ok(cu.cuMemcpyDtoH_v2(like.ctypes.data_as(C.c_void_p), p, C.c_size_t(like.nbytes)))
    return like

def attend(heads, columns):
    rows, kv, D, page, pages, ctx = 2, 2, 64, 16, 2, 20
    i32, u16 = np.int32, np.uint16
    table = np.full((1, columns), -7, i32)
    table[0, :2] = 1, 0
    q = np.full((rows, heads, D), 0x3F80, u16)          # ones
    k = np.zeros((pages, page, kv, D), u16)
    v = np.full((pages, page, kv, D), 0x4040, u16)      # threes
    need = L.spec_tree_attention_workspace_bytes(1, 1, 1, heads, kv, D)
    out, lse, st = np.zeros_like(q), np.zeros((rows, heads), np.float32), np.full(1, 9, i32)
    d = [up(x) for x in (q, np.zeros(1, np.int64), np.ones(1, i32), np.full(1, ctx, i32), table, k, v, out, lse, st,
                         np.zeros(need, np.uint8))]
    code = L.spec_tree_attention(d[0], heads * D, D, rows, heads, kv, D, 0.125, d[1], d[2], 1, 1, None, 1, d[3], d[4],
                                 columns, columns, d[5], d[6], pages, page, page * kv * D, kv * D, D, d[7], heads * D,
                                 D, d[8], heads, d[9], d[10], need, None)
    assert code == 0, (code, heads, columns)
    ok(cu.cuCtxSynchronize())
    assert down(d[9], st)[0] == 0
    assert (down(d[7], out) == 0x4040).all()
    z = down(d[8], lse)
    assert np.allclose(z[0], math.log(ctx + 1), rtol=1e-6) and np.allclose(z[1], math.log(ctx + 2), rtol=1e-6)

for ctx in (first, second, first, second):
    ok(cu.cuCtxSetCurrent(ctx))
    for heads, columns in ((8, 2), (32, 2), (64, 2), (8, 1100), (128, 2)):
        attend(heads, columns)
print("both contexts")
# the process ends its own primary context and begins another
ok(cu.cuCtxSetCurrent(first))
ok(C.CDLL("libcudart.so.13").cudaDeviceReset())
ok(cu.cuDevicePrimaryCtxRetain(C.byref(first), dev))
ok(cu.cuCtxSetCurrent(first))
for heads, columns in ((8, 2), (32, 2), (64, 2), (8, 1100), (128, 2)):
    attend(heads, columns)
print("a new context")
"""


def test_attention_in_contexts():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", CHILD], cwd=root, env={**os.environ, "PYTHONPATH": root},
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "a new context" in run.stdout, run.stdout + run.stderr
