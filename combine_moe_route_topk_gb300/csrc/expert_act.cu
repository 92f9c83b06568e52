// Gradient of the experts' gated activation h = silu(g) u, on the rows that
// hold a token: with s = 1 / (1 + exp(-g)),
//   dg = dh u s (1 + g (1 - s)),  du = dh g s.
// Five values move per feature (g, u, dh in, dg, du out): bound by HBM.  A
// block takes whole rows, a thread eight features at a time (16-byte
// accesses); sums and products in f32, one rounding to bf16.
#include <cuda_bf16.h>

#include "expert_internal.cuh"
#include "mem_ops.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kActThreads = 256;
// Blocks per SM that the registers are for: 65536 rows of F = 2048 in four ranks
// take 205 us with 6, 212 with 5, 224 with 7 or 8, which spill.
constexpr int kActResident = 6;
constexpr int kActBlocks = 24;  // per SM at most: of these rows' time 8 cost 9 % more, 128 3 % more, 24 to 64 are alike

__device__ __forceinline__ float lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// The factors with s come first: s (1 + g (1 - s)) is at most 1.1 and |g s| at most
// |g|, and both are 0 where g is the type's lowest value; dh g or dh u could pass
// the range before s = 0 takes it back (infinity times 0).
__device__ __forceinline__ void grad(float g, float u, float dh, float *dg, float *du) {
    const float s = 1.f / (1.f + expf(-g));
    *dg = s * (1.f + g * (1.f - s)) * u * dh;
    *du = g * s * dh;
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Rows of rank d that hold a token: [d cap, d cap + rows(d)).  They are dealt
// out to blocks (and the thread rows of a block) round robin over all ranks, by
// a table of the ranks' first rows among them.  (With every thread row going
// through the ranks, a load for each, 16384 rows of F = 2048 in 32 ranks took
// 76 us instead of 56.)
template <bool kRanks>  // more than one
__global__ void __launch_bounds__(kActThreads, kActResident)
swiglu_grad_kernel(const int32_t *__restrict__ offsets, int N, int L, int64_t cap, int nvec, const uint4 *__restrict__ pre,
                   const uint4 *__restrict__ dh, uint4 *__restrict__ dpre) {
    extern __shared__ int s_first[];  // [N + 1]
    grid_dependency_wait();
    grid_launch_dependents();
    auto rows = [&](int d) {
        const int64_t n = (int64_t)__ldg(offsets + (d + 1) * L) - __ldg(offsets + d * L);
        return (int)(n < 0 ? 0 : (n < cap ? n : cap));
    };
    int all;
    if constexpr (!kRanks) {  // 0.3 us less than the table
        all = rows(0);
    } else {
        const int tid = threadIdx.y * blockDim.x + threadIdx.x;
        if (tid < 32) {
            const int per = (N + 31) / 32, d0 = tid * per, d1 = min(N, d0 + per);
            int sum = 0;
            for (int d = d0; d < d1; ++d) {
                s_first[d] = sum;  // within the lane's ranks
                sum += rows(d);
            }
            int before = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, before, o);
                if (tid >= o) before += v;
            }
            if (tid == 31) s_first[N] = before;
            before -= sum;
            for (int d = d0; d < d1; ++d) s_first[d] += before;
        }
        __syncthreads();
        all = s_first[N];
    }
    const int step = gridDim.x * blockDim.y;
    int d = 0;
    for (int64_t at = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; at < all; at += step) {
        for (int end = kRanks ? N : 1; end - d > 1;) {
            const int mid = (d + end) / 2;
            if (s_first[mid] <= at) d = mid;
            else end = mid;
        }
        const int64_t row = d * cap + (kRanks ? at - s_first[d] : at);
        const uint4 *g = pre + row * 2 * nvec, *u = g + nvec, *h = dh + row * nvec;
        uint4 *o = dpre + row * 2 * nvec;
        for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
            const uint4 gv = ld_stream(g + c), uv = ld_stream(u + c), hv = ld_stream(h + c);
            const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w}, uw[4] = {uv.x, uv.y, uv.z, uv.w},
                           hw[4] = {hv.x, hv.y, hv.z, hv.w};
            uint32_t dg[4], du[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float a0, a1, b0, b1;
                grad(lo(gw[i]), lo(uw[i]), lo(hw[i]), &a0, &b0);
                grad(hi(gw[i]), hi(uw[i]), hi(hw[i]), &a1, &b1);
                dg[i] = bf16x2(a0, a1);
                du[i] = bf16x2(b0, b1);
            }
            o[c] = make_uint4(dg[0], dg[1], dg[2], dg[3]);
            o[nvec + c] = make_uint4(du[0], du[1], du[2], du[3]);
        }
    }
}

}  // namespace

cudaError_t launch_expert_swiglu_grad(const ExpertRows &r, int N, int64_t pairs, int F, const void *pre, const void *dh,
                                      void *dpre, cudaStream_t stream) {
    const int nvec = F / 8;
    int tx = 32;
    while (tx < nvec && tx < kActThreads) tx *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(tx, kActThreads / tx);
    cfg.dynamicSmemBytes = (N + 1) * sizeof(int);
    const int64_t rows = pairs < r.rows_total ? pairs : r.rows_total;
    const int64_t blocks = (rows + cfg.blockDim.y - 1) / cfg.blockDim.y, most = (int64_t)sm_count() * kActBlocks;
    cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, N > 1 ? swiglu_grad_kernel<true> : swiglu_grad_kernel<false>, r.offsets, N, r.L, r.cap, nvec,
                              reinterpret_cast<const uint4 *>(pre), reinterpret_cast<const uint4 *>(dh),
                              reinterpret_cast<uint4 *>(dpre));
}

}  // namespace moe
