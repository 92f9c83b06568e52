"""The bounded waits of the experts' products where nothing ever arrives: a wait
gives up after its limit, the block's other warps leave theirs when they see
it, draining a ring ends too, the error word tells the host once, and the
context stays usable.  A small program over the kernels' own header, with
barriers that nothing arrives at and limits of a few polls (a failing poll is
suspended for some microseconds)."""
import subprocess

import pytest

from combine_moe_route_topk_gb300 import _build

pytestmark = pytest.mark.gpu

PROGRAM = r'''
#include <stdio.h>
#include "tc_ops.cuh"
using namespace moe;

// out: warp 0's and warp 1's results, the block's word, and what a wait for an arrival gives
__global__ void waits(long long polls, int *out) {
    __shared__ __align__(8) unsigned long long never, once, ring[3];
    __shared__ int gave_up;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        mb_init(smem_u32(&never), 1);
        mb_init(smem_u32(&once), 1);
        for (int i = 0; i < 3; ++i) mb_init(smem_u32(&ring[i]), 1);
        gave_up = 0;
        mb_init_fence();
        mb_arrive(smem_u32(&once));
    }
    __syncthreads();
    if (warp == 0) {
        const bool there = mb_wait_warp(smem_u32(&once), 0, &gave_up, polls);
        const int before = gave_up;
        const bool ok = mb_wait_warp(smem_u32(&never), 0, &gave_up, polls);
        if (lane == 0) out[0] = ok, out[2] = before, out[3] = there;
    } else if (warp == 1) {  // its own limit is seconds: it leaves with the other
        const bool ok = mb_wait_warp(smem_u32(&never), 0, &gave_up);
        if (lane == 0) out[1] = ok;
    } else {
        Ring<3> r;
        for (int i = 0; i < 4; ++i) r.next();  // four loads were issued, and none landed
        drain_ring(smem_u32(ring), r, polls);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        out[4] = gave_up;
        if (gave_up) record_timeout();
    }
}

int main() {
    int *d, h[5], err = -1;
    if (cudaMalloc(&d, sizeof(h)) != cudaSuccess) return 1;
    for (int round = 0; round < 2; ++round) {
        cudaMemset(d, 0xff, sizeof(h));
        cudaEvent_t a, b;
        cudaEventCreate(&a), cudaEventCreate(&b);
        cudaEventRecord(a);
        waits<<<1, 96>>>(64, d);
        cudaEventRecord(b);
        if (cudaMemcpy(h, d, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess) return 2;
        float ms;
        cudaEventElapsedTime(&ms, a, b);
        printf("%d %d %d %d %d %.3f", h[0], h[1], h[2], h[3], h[4], ms);
        for (int i = 0; i < 2; ++i) {  // told once
            if (take_tc_error(&err) != cudaSuccess) return 3;
            printf(" %d", err);
        }
        printf("\n");
    }
}
'''


def test_waits_for_what_never_arrives_give_up(tmp_path):
    src = tmp_path / "waits.cu"
    src.write_text(PROGRAM)
    subprocess.run([_build.nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-o", str(tmp_path / "waits"), str(src)], check=True,
                   capture_output=True)
    r = subprocess.run([str(tmp_path / "waits")], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout + r.stderr
    lines = r.stdout.splitlines()
    assert len(lines) == 2  # the second round runs in the same context
    for line in lines:
        first, second, before, there, gave_up, ms, *errors = line.split()
        assert (first, second) == ("0", "0") and gave_up == "1"
        assert there == "1" and before == "0"
        assert float(ms) < 1000  # warp 1's own limit is 2^20 polls, seconds
        assert errors == ["-5", "0"]  # MOE_ERR_TIMEOUT, then nothing
