"""A host thread whose first use of CUDA is a call of the library, on tensors and a stream of another one."""
import threading

import pytest
import torch

import combine_moe_route_topk_gb300 as moe
from expert_ref import Batch, quantise

pytestmark = pytest.mark.gpu
LINEAR, SWIGLU = moe.MOE_EXPERT_LINEAR, moe.MOE_EXPERT_SWIGLU


def _products(b, K, F):
    d, off = b.dims(), b.offsets
    x, dy, w = b.randn(b.rows, K), b.randn(b.rows, F), b.randn(b.E, F, K)
    xq, xs = quantise(x)
    wq, ws = torch.zeros(b.E, F, K, dtype=torch.uint8, device="cuda"), torch.ones(b.E, F // 128, K // 128, device="cuda")
    return {
        "linear": (lambda y, s=None: moe.expert_gemm(d, K, F, LINEAR, x, w, off, y, stream=s), b.out(F, torch.bfloat16)),
        "gated": (lambda y, s=None: moe.expert_gemm(d, K, F // 2, SWIGLU, x, w, off, y, stream=s), b.out(F // 2, torch.bfloat16)),
        "dgrad": (lambda y, s=None: moe.expert_gemm_dgrad(d, K, F, dy, w, off, y, stream=s), b.out(K, torch.bfloat16)),
        "wgrad": (lambda y, s=None: moe.expert_gemm_wgrad(d, K, F, dy, x, off, y, stream=s), torch.zeros(b.E, F, K, device="cuda")),
        "fp8": (lambda y, s=None: moe.expert_gemm_fp8(d, K, F, LINEAR, xq, xs, wq, ws, off, y, stream=s), b.out(F, torch.bfloat16)),
    }


@pytest.mark.parametrize("name", ["linear", "gated", "dgrad", "wgrad", "fp8"])
def test_first_call_of_a_thread(name):
    from combine_moe_route_topk_gb300 import _build
    _build.build()
    call, y = _products(Batch(1, [40, 3], 64), 256, 256)[name]
    stream = torch.cuda.current_stream().cuda_stream
    start = y.clone()
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            call(y, stream)
        except BaseException as e:  # reported by the test's own thread
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    got = y.clone()
    y.copy_(start)
    call(y)
    assert torch.equal(got, y)
