"""Every kernel of the product with 4-bit weights after cudaDeviceReset: limits of shared memory and the number of resident
clusters are kept per CUDA context, so calls in the next context set them again.  In a child process, through the C ABI
and the CUDA runtime only (PyTorch's allocator does not survive a reset); small integers as operands make every sum exact."""
import subprocess
import sys

import pytest
import torch

import combine_moe_route_topk_gb300 as moe
from conftest import ROOT
from w4_form import form

pytestmark = pytest.mark.gpu

# rows, K, F of one matrix with f32 results, and the form
CASES = [(3, 512, 136, (8, 1)), (64, 1024, 4864, (64, 4)), (128, 512, 4096, (64, 2)), (256, 256, 4096, (64, 1)),
         (700, 256, 4096, (128, 1))]

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

def product(rows, K, F):
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
    np.testing.assert_array_equal(get(y, (rows, F), np.float32), x.astype(np.float64) @ q.T.astype(np.float64))

cases = eval(sys.argv[2])
for c in cases:
    product(*c)
assert rt.cudaDeviceReset() == 0
for c in cases[::-1]:
    product(*c)
print("RESET_OK")
'''


def test_every_form_after_a_device_reset():
    from combine_moe_route_topk_gb300 import _build
    _build.build()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for rows, K, F, want in CASES:
        assert form(moe.make_dims(1, rows, 1, 1, 8, cap_rows=rows), K, F, False, True, sms) == want
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, repr([c[:3] for c in CASES])], capture_output=True, text=True, timeout=300)
    assert "RESET_OK" in r.stdout, r.stdout + r.stderr
