// Gradients of combine and of the dispatch pack.
//
//   combine   out[g] = sum_k w[g][k] y[p],  p = pos[g][k]:
//             dy[p] = w[g][k] dout[g],  dw[g][k] = <dout[g], y[p]>
//   dispatch  packed[p] = x[g]:  dx[g] = add[g] + sum_k dpacked[p]
//
// Both are streams of whole rows, ordered by token: a token's row of dout is
// read once for all its pairs, and what is summed (dw, dx) is summed inside
// one block, in a fixed order.
#include "grad_internal.cuh"
#include "mem_ops.cuh"
#include "pdl.cuh"
#include "vec_traits.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// The token's pairs that have a row, in k order, by the block's first warp:
// s_p their rows, s_k their places k.  Returns (after a barrier) their number.
__device__ __forceinline__ int gather_pairs(const int32_t *__restrict__ pos, int64_t g, int R, int64_t rows_total,
                                            int *s_p, int *s_k, int *s_n) {
    const int tid = threadIdx.x;
    if (tid < 32) {
        const int p = tid < R ? __ldg(pos + g * R + tid) : -1;
        const bool in = p >= 0 && (int64_t)p < rows_total;
        const unsigned m = __ballot_sync(0xffffffffu, in);
        if (in) {
            const int j = __popc(m & ((1u << tid) - 1u));
            s_p[j] = p;
            s_k[j] = tid;
        }
        if (tid == 0) *s_n = __popc(m);
    }
    __syncthreads();
    return *s_n;
}

// ---- combine ----------------------------------------------------------------

// Pairs whose rows a thread loads together.
constexpr int kPairs = 8;
// Vectors of a row that go into one f32 sum per thread before the block adds
// its threads' sums up and the total in 64 bits: 32 vectors a thread.
constexpr int kChunk = 32 * kThreads;

template <int kBf16>
struct Pair;
template <>
struct Pair<1> {
    __device__ __forceinline__ static float dot(float a, const uint4 &x, const uint4 &y) {
        const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16), a);
            a = fmaf(__uint_as_float(u[i] & 0xffff0000u), __uint_as_float(v[i] & 0xffff0000u), a);
        }
        return a;
    }
};
template <>
struct Pair<0> {
    __device__ __forceinline__ static float dot(float a, const uint4 &x, const uint4 &y) {
        a = fmaf(__uint_as_float(x.x), __uint_as_float(y.x), a);
        a = fmaf(__uint_as_float(x.y), __uint_as_float(y.y), a);
        a = fmaf(__uint_as_float(x.z), __uint_as_float(y.z), a);
        return fmaf(__uint_as_float(x.w), __uint_as_float(y.w), a);
    }
};

template <int kBf16>
__global__ void __launch_bounds__(kThreads)
combine_grad_kernel(const uint4 *__restrict__ dout, const uint4 *__restrict__ y, const int32_t *__restrict__ pos,
                    const float *__restrict__ topk_w, int64_t NT, int R, int nvec, int64_t rows_total,
                    uint4 *__restrict__ dy, float *__restrict__ dtopk_w) {
    using VT = Vec<kBf16>;
    __shared__ int s_p[32], s_k[32], s_n;
    __shared__ float s_w[32], s_sum[kWarps][kPairs];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    grid_dependency_wait();  // every input comes from earlier kernels
    grid_launch_dependents();
    for (int64_t g = blockIdx.x; g < NT; g += gridDim.x) {
        if (tid < 32 && tid < R) {
            s_w[tid] = __ldg(topk_w + g * R + tid);
            dtopk_w[g * R + tid] = 0.f;  // stays where there is no row
        }
        const int n = gather_pairs(pos, g, R, rows_total, s_p, s_k, &s_n);
        for (int j0 = 0; j0 < n; j0 += kPairs) {
            double total = 0.0;  // thread j < kPairs: of pair j0 + j
            for (int c1 = 0; c1 < nvec; c1 += kChunk) {
                float acc[kPairs];
#pragma unroll
                for (int j = 0; j < kPairs; ++j) acc[j] = 0.f;
                const int end = min(nvec, c1 + kChunk);
                for (int c = c1 + tid; c < end; c += kThreads) {
                    uint4 v[kPairs];
#pragma unroll
                    for (int j = 0; j < kPairs; ++j)
                        v[j] = j0 + j < n ? ld_stream(y + (int64_t)s_p[j0 + j] * nvec + c) : make_uint4(0u, 0u, 0u, 0u);
                    const uint4 d = __ldg(dout + g * nvec + c);
#pragma unroll
                    for (int j = 0; j < kPairs; ++j) {
                        if (j0 + j < n) {
                            acc[j] = Pair<kBf16>::dot(acc[j], d, v[j]);
                            float o[VT::kElems];
#pragma unroll
                            for (int i = 0; i < VT::kElems; ++i) o[i] = 0.f;
                            VT::fma(o, s_w[s_k[j0 + j]], d);
                            dy[(int64_t)s_p[j0 + j] * nvec + c] = VT::pack(o);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
                    if (lane == 0) s_sum[warp][j] = acc[j];
                }
                __syncthreads();
                if (tid < kPairs) {
#pragma unroll
                    for (int i = 0; i < kWarps; ++i) total += s_sum[i][tid];
                }
                __syncthreads();
            }
            if (tid < kPairs && j0 + tid < n) dtopk_w[g * R + s_k[j0 + tid]] = (float)total;
        }
        __syncthreads();  // the tables are rewritten for the next token
    }
}

// ---- dispatch -----------------------------------------------------------------

constexpr int kU = 2;   // vectors of dx per thread
constexpr int kKB = 4;  // rows loaded together

template <int kBf16>
__global__ void __launch_bounds__(kThreads, 8)
dispatch_grad_kernel(const uint4 *__restrict__ dpacked, const int32_t *__restrict__ pos, const uint4 *add, int64_t NT,
                     int R, int nvec, int64_t rows_total, uint4 *dx) {
    using VT = Vec<kBf16>;
    constexpr int EL = VT::kElems;
    __shared__ int s_p[32], s_k[32], s_n;
    const int tid = threadIdx.x;
    grid_dependency_wait();
    grid_launch_dependents();
    for (int64_t g = blockIdx.x; g < NT; g += gridDim.x) {
        const int n = gather_pairs(pos, g, R, rows_total, s_p, s_k, &s_n);
        for (int c0 = tid; c0 < nvec; c0 += kThreads * kU) {
            float acc[kU][EL];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int c = c0 + u * kThreads;
#pragma unroll
                for (int i = 0; i < EL; ++i) acc[u][i] = 0.f;
                if (add != nullptr && c < nvec) VT::add(acc[u], add[g * nvec + c]);  // read before dx, where it is the same
            }
            for (int j0 = 0; j0 < n; j0 += kKB) {
                uint4 v[kKB][kU];
#pragma unroll
                for (int jj = 0; jj < kKB; ++jj)
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        const int c = c0 + u * kThreads;
                        v[jj][u] = (j0 + jj < n && c < nvec) ? ld_stream(dpacked + (int64_t)s_p[j0 + jj] * nvec + c)
                                                             : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                for (int jj = 0; jj < kKB; ++jj)
#pragma unroll
                    for (int u = 0; u < kU; ++u) VT::add(acc[u], v[jj][u]);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int c = c0 + u * kThreads;
                if (c < nvec) dx[g * nvec + c] = VT::pack(acc[u]);
            }
        }
        __syncthreads();
    }
}

// One block of kThreads per token (the hardware schedules them).
struct Launch {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    Launch(int64_t NT, cudaStream_t stream) {
        attr[0] = pdl_attribute();
        cfg.gridDim = dim3((unsigned)(NT < 0x7fffffff ? NT : 0x7fffffff));
        cfg.blockDim = dim3(kThreads);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    Launch(const Launch &) = delete;
};

int row_vectors(int H, int dtype) { return (int)((int64_t)H * (dtype == MOE_BF16 ? 2 : 4) / 16); }

}  // namespace

cudaError_t launch_combine_grad(const void *dout, const void *y, int y_dtype, const int32_t *pos, const float *topk_w,
                                int64_t NT, int R, int H, int64_t rows_total, void *dy, float *dtopk_w,
                                cudaStream_t stream) {
    Launch l(NT, stream);
    auto kern = y_dtype == MOE_BF16 ? combine_grad_kernel<1> : combine_grad_kernel<0>;
    return cudaLaunchKernelEx(&l.cfg, kern, static_cast<const uint4 *>(dout), static_cast<const uint4 *>(y), pos, topk_w,
                              NT, R, row_vectors(H, y_dtype), rows_total, static_cast<uint4 *>(dy), dtopk_w);
}

cudaError_t launch_dispatch_grad(const void *dpacked, int x_dtype, const int32_t *pos, const void *add, int64_t NT,
                                 int R, int H, int64_t rows_total, void *dx, cudaStream_t stream) {
    Launch l(NT, stream);
    auto kern = x_dtype == MOE_BF16 ? dispatch_grad_kernel<1> : dispatch_grad_kernel<0>;
    return cudaLaunchKernelEx(&l.cfg, kern, static_cast<const uint4 *>(dpacked), pos, static_cast<const uint4 *>(add), NT,
                              R, row_vectors(H, x_dtype), rows_total, static_cast<uint4 *>(dx));
}

}  // namespace moe
