"""Which of its kernels the product with 4-bit weights takes a batch with: the library's own rule (w4_rule.cuh), compiled
for the host, so that a test can tell what its sizes reach and fails when the rule no longer leads there."""
from __future__ import annotations

import ctypes
import functools
import os
import subprocess
import tempfile

from combine_moe_route_topk_gb300 import _build

SOURCE = """
#include "w4_rule.cuh"
extern "C" void w4_form_of(int E, int N, long long T, int R, long long cap, int K, int F, int gated, int f32, int sms, int *out) {
    const long long nt = T * N;
    const moe::ExpertRows r{nullptr, E, E / N, cap, cap * N, nt < cap ? nt : cap, nt * R};
    const moe::W4Form f = moe::w4_form(r, K, F, gated, f32, sms);
    out[0] = f.tokens, out[1] = f.split;
}
"""


@functools.cache
def _rule():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "rule.cu"), os.path.join(d, "rule.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run([_build.nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-shared", "-o", so, src], check=True, capture_output=True)
        lib = ctypes.CDLL(so)
    i, q = ctypes.c_int, ctypes.c_longlong
    lib.w4_form_of.argtypes = [i, i, q, i, q, i, i, i, i, i, ctypes.POINTER(i)]
    return lib.w4_form_of


def form(dims, K, F, gated, f32, sms):
    """(most tokens of a tile, blocks that share a reduction) for a batch with cap_rows given."""
    out = (ctypes.c_int * 2)()
    _rule()(dims.E, dims.N, dims.T, dims.R, dims.cap_rows, K, F, int(gated), int(f32), sms, out)
    return tuple(out)


# Small batches that reach each kernel on a GPU of 152 SMs: rows per expert, K, F of a linear product (a gated one has half),
# group, and the form.  f32 results are in parts of 512 and have tiles of 128 tokens where bf16 ones have 160.
FORMS = {
    "few": ([3, 0, 12, 1], 544, 272, 32, (8, 1)),
    "split in fours": ([40, 0, 22], 1152, 1040, 128, (64, 4)),
    "split in twos": ([40, 0, 22], 544, 1296, 32, (64, 2)),
    "tiles of 64": ([40, 0, 40, 33, 20], 224, 1296, 32, (64, 1)),
    "large tiles": ([161, 0, 320, 129, 1], 544, 1552, 32, (160, 1)),
}


def expected(name, f32):
    tokens, split = FORMS[name][4]
    return (128 if tokens == 160 and f32 else tokens), split
