"""The experts' products after cudaDeviceReset: the shared-memory limits and the
number of resident block pairs are kept per CUDA context, so calls in the next
context set them again.  In a child process, through the C ABI and the CUDA
runtime only (PyTorch's allocator does not survive a reset); small integers as
operands make every sum exact."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import ctypes, os, sys
import numpy as np
lib = ctypes.CDLL(os.path.join(sys.argv[1], "combine_moe_route_topk_gb300", "libmoe_route.so"))
lib.moe_last_error.restype = ctypes.c_char_p
rt = ctypes.CDLL(next(l.split()[-1] for l in open("/proc/self/maps") if "libcudart.so" in l))
P, i32 = ctypes.c_void_p, ctypes.c_int

class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("N", "T", "E", "R", "H", "x", "y", "z")] + [("cap", ctypes.c_int64)]

rows, K, F, E = 50, 128, 136, 2
d = ctypes.byref(Dims(1, rows, E, 1, 8, 0, 1, 0, rows))  # f32 results

def put(a):
    p = P()
    assert rt.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(a.nbytes)) == 0
    assert rt.cudaMemcpy(p, a.ctypes.data_as(P), ctypes.c_size_t(a.nbytes), 1) == 0
    return p

def get(p, shape, dtype):
    a = np.empty(shape, dtype)
    assert rt.cudaDeviceSynchronize() == 0
    assert rt.cudaMemcpy(a.ctypes.data_as(P), p, ctypes.c_size_t(a.nbytes), 2) == 0
    return a

def bf16(a):  # exact for small integers
    return (a.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)

def ok(rc):
    assert rc == 0, (rc, lib.moe_last_error())

rng = np.random.default_rng(3)
x, w, dy = (rng.integers(-3, 4, s) for s in ((rows, K), (E, F, K), (rows, F)))
off = np.array([0, 20, rows], np.int32)
e = np.repeat([0, 1], [20, 30])

def round_():
    zero = lambda n: put(np.zeros(n, np.uint8))
    px, pw, pdy, po = put(bf16(x)), put(bf16(w)), put(bf16(dy)), put(off)
    y, dx, dw, y8 = zero(rows * F * 4), zero(rows * K * 2), zero(E * F * K * 4), zero(rows * F * 4)
    ok(lib.moe_expert_gemm(d, i32(K), i32(F), i32(0), px, pw, po, y, None, None))
    ok(lib.moe_expert_gemm_dgrad(d, i32(K), i32(F), pdy, pw, po, dx, None))
    ok(lib.moe_expert_gemm_wgrad(d, i32(K), i32(F), pdy, px, po, dw, i32(1), None))
    # e4m3: 1.0 is 0x38
    q = lambda a: np.where(a > 0, 0x38, np.where(a < 0, 0xB8, 0)).astype(np.uint8)
    one = lambda n: put(np.ones(n, np.float32))
    ok(lib.moe_expert_gemm_fp8(d, i32(K), i32(F), i32(0), put(q(x)), one(rows), put(q(w)), one(E * 2), po, y8, None, None))
    np.testing.assert_array_equal(get(y, (rows, F), np.float32), np.einsum("pk,pfk->pf", x, w[e]))
    np.testing.assert_array_equal(get(y8, (rows, F), np.float32), np.einsum("pk,pfk->pf", np.sign(x), np.sign(w)[e]))
    np.testing.assert_array_equal(get(dw, (E, F, K), np.float32),
                                  np.stack([dy[e == i].T @ x[e == i] for i in range(E)]))
    got = (get(dx, (rows, K), np.uint16).astype(np.uint32) << 16).view(np.float32)
    want = np.einsum("pf,pfk->pk", dy, w[e])
    assert (np.abs(got - want) <= np.abs(want) / 256).all()  # one rounding to bf16

round_()
assert rt.cudaDeviceReset() == 0
round_()
print("RESET_OK")
'''


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_moe_route_topk_gb300 import _build
    _build.build()


def test_expert_calls_after_a_device_reset():
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True, timeout=300)
    assert "RESET_OK" in r.stdout, r.stdout + r.stderr
