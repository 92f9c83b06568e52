"""The product with 4-bit weights after cudaDeviceReset: shared-memory limits and the number of resident clusters are
kept per CUDA context, so calls in the next context set them again.  In a child process, through the C ABI and the CUDA
runtime only (PyTorch's allocator does not survive a reset); small integers as operands make every sum exact."""
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

def round_(rows, K, F):  # one matrix, f32 results
    rng = np.random.default_rng(rows)
    d = ctypes.byref(Dims(1, rows, 1, 1, 8, 0, 1, 0, rows))
    x, q = rng.integers(-3, 4, (rows, K)), rng.integers(-8, 8, (F, K))
    words = np.zeros((F, K // 8), np.uint32)
    for i in range(8):
        words |= (q[:, i::8] & 15).astype(np.uint32) << np.uint32(4 * (i // 2) + 16 * (i % 2))
    bf16 = (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    y = put(np.zeros((rows, F), np.float32))
    rc = lib.moe_expert_gemm_w4(d, i32(K), i32(F), i32(0), i32(64), put(bf16), put(words),
                                put(np.full((K // 64, F), 0x38, np.uint8)), put(np.ones(F, np.float32)),
                                put(np.array([0, rows], np.int32)), y, None)
    assert rc == 0, lib.moe_last_error()
    np.testing.assert_array_equal(get(y, (rows, F), np.float32), x @ q.T)

def all_():
    round_(3, 512, 136)      # few rows
    round_(60, 1024, 136)    # blocks that share a reduction, in fours
    round_(60, 512, 136)     # in twos
    round_(700, 64, 136)     # large tiles

all_()
assert rt.cudaDeviceReset() == 0
all_()
print("RESET_OK")
'''


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_moe_route_topk_gb300 import _build
    _build.build()


def test_calls_after_a_device_reset():
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True, timeout=300)
    assert "RESET_OK" in r.stdout, r.stdout + r.stderr
