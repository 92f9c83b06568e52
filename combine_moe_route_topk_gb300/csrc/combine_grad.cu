// Gradients of combine and of the dispatch pack.
//
//   combine   out[g] = sum_k w[g][k] y[p],  p = pos[g][k]:
//             dy[p] = w[g][k] dout[g],  dw[g][k] = <dout[g], y[p]>
//   dispatch  packed[p] = x[g]:  dx[g] = add[g] + sum_k dpacked[p]
//
// Both are streams of whole rows, ordered by token: a token's row of dout is
// read once for all its pairs (by rows of y it would be read R times, or wait
// in L2 for a pair that comes much later), and what is summed (dw, dx) is
// summed inside one block or warp, in a fixed order, without atomics.  HBM
// bounds them: 65536 pairs of 8192 tokens, rows of 4096 bf16 172 us (1.14 GB,
// 0.98 of what a copy reaches), dispatch's 65536 rows of 7168 with a first
// summand 171 us (1.18 GB, 1.01).
#include "grad_internal.cuh"
#include "mem_ops.cuh"
#include "pdl.cuh"
#include "vec_traits.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;

// The threads that share a token: the whole block, or a warp where rows are short.
template <int kGroup>
__device__ __forceinline__ void group_sync() {
    if constexpr (kGroup == 32) __syncwarp();
    else __syncthreads();
}

// What a group knows of its token: its pairs that have a row, in k order.
struct Pairs {
    int row[32], k[32], n;  // rows, places k, number
};

// Fills it, by the group's first warp, and syncs the group.
template <int kGroup>
__device__ __forceinline__ int gather_pairs(const int32_t *__restrict__ pos, int64_t g, int R, int64_t rows_total,
                                            Pairs &s) {
    const int t = threadIdx.x % kGroup;
    if (t < 32) {
        const int p = t < R ? __ldg(pos + g * R + t) : -1;
        const bool in = p >= 0 && (int64_t)p < rows_total;
        const unsigned m = __ballot_sync(0xffffffffu, in);
        if (in) {
            const int j = __popc(m & ((1u << t) - 1u));
            s.row[j] = p;
            s.k[j] = t;
        }
        if (t == 0) s.n = __popc(m);
    }
    group_sync<kGroup>();
    return s.n;
}

// ---- combine ----------------------------------------------------------------

// Vectors of a row that go into one f32 sum per thread before the group adds
// its threads' sums up and the total in 64 bits: 32 vectors a thread.
constexpr int kRun = 32;

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

// kPairs: pairs whose rows a thread loads together, kU vectors of each.  Eight
// loads a thread are under way: with 8 x 1 for all, 16384 tokens of 1, 2 and
// 4 rows of 4096 bf16 took 99, 125 and 186 us, with 4 x 2 82, 110 and 180; eight rows
// 171 and 174.  In warps, 65536 tokens of two rows of 1024: 2 x 2 100, 4 x 1 111, 8 x 1
// 152; of four 180, 180, 213.
template <int kBf16, int kGroup, int kPairs, int kU>
__global__ void __launch_bounds__(kThreads)
combine_grad_kernel(const uint4 *__restrict__ dout, const uint4 *__restrict__ y, const int32_t *__restrict__ pos,
                    const float *__restrict__ topk_w, int64_t NT, int R, int nvec, int64_t rows_total,
                    uint4 *__restrict__ dy, float *__restrict__ dtopk_w) {
    using VT = Vec<kBf16>;
    constexpr int kGroups = kThreads / kGroup, kWarps = kGroup / 32, kChunk = kRun * kGroup;
    __shared__ Pairs s_pairs[kGroups];
    __shared__ float s_w[kGroups][32], s_sum[kGroups][kWarps][kPairs];
    const int which = threadIdx.x / kGroup, t = threadIdx.x % kGroup, warp = t / 32, lane = t % 32;
    Pairs &s = s_pairs[which];
    grid_dependency_wait();  // every input comes from earlier kernels
    grid_launch_dependents();
    for (int64_t g = (int64_t)blockIdx.x * kGroups + which; g < NT; g += (int64_t)gridDim.x * kGroups) {
        if (t < R) {  // R <= 32
            s_w[which][t] = __ldg(topk_w + g * R + t);
            dtopk_w[g * R + t] = 0.f;  // stays where there is no row
        }
        const int n = gather_pairs<kGroup>(pos, g, R, rows_total, s);
        for (int j0 = 0; j0 < n; j0 += kPairs) {
            double total = 0.0;  // thread j < kPairs: of pair j0 + j
            for (int c1 = 0; c1 < nvec; c1 += kChunk) {
                float acc[kPairs];
#pragma unroll
                for (int j = 0; j < kPairs; ++j) acc[j] = 0.f;
                const int end = min(nvec, c1 + kChunk);
                for (int c = c1 + t; c < end; c += kGroup * kU) {
                    uint4 v[kU][kPairs], d[kU];
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        const int cu = c + u * kGroup;
#pragma unroll
                        for (int j = 0; j < kPairs; ++j)
                            v[u][j] = cu < end && j0 + j < n ? ld_stream(y + (int64_t)s.row[j0 + j] * nvec + cu)
                                                             : make_uint4(0u, 0u, 0u, 0u);
                        d[u] = cu < end ? __ldg(dout + g * nvec + cu) : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        const int cu = c + u * kGroup;
                        if (cu >= end) break;
#pragma unroll
                        for (int j = 0; j < kPairs; ++j) {
                            if (j0 + j < n) {
                                acc[j] = Pair<kBf16>::dot(acc[j], d[u], v[u][j]);
                                float o[VT::kElems];
#pragma unroll
                                for (int i = 0; i < VT::kElems; ++i) o[i] = 0.f;
                                VT::fma(o, s_w[which][s.k[j0 + j]], d[u]);
                                dy[(int64_t)s.row[j0 + j] * nvec + cu] = VT::pack(o);
                            }
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
                    if (lane == 0) s_sum[which][warp][j] = acc[j];
                }
                group_sync<kGroup>();
                if (t < kPairs) {
#pragma unroll
                    for (int i = 0; i < kWarps; ++i) total += s_sum[which][i][t];
                }
                group_sync<kGroup>();
            }
            if (t < kPairs && j0 + t < n) dtopk_w[g * R + s.k[j0 + t]] = (float)total;
        }
        group_sync<kGroup>();  // the tables are rewritten for the next token
    }
}

// ---- dispatch -----------------------------------------------------------------

constexpr int kVecs = 2;  // vectors of dx per thread
constexpr int kLoads = 4;  // rows loaded together

template <int kBf16, int kGroup>
__global__ void __launch_bounds__(kThreads, 8)
dispatch_grad_kernel(const uint4 *__restrict__ dpacked, const int32_t *__restrict__ pos, const uint4 *add, int64_t NT,
                     int R, int nvec, int64_t rows_total, uint4 *dx) {
    using VT = Vec<kBf16>;
    constexpr int EL = VT::kElems, kGroups = kThreads / kGroup;
    __shared__ Pairs s_pairs[kGroups];
    const int which = threadIdx.x / kGroup, t = threadIdx.x % kGroup;
    Pairs &s = s_pairs[which];
    grid_dependency_wait();
    grid_launch_dependents();
    for (int64_t g = (int64_t)blockIdx.x * kGroups + which; g < NT; g += (int64_t)gridDim.x * kGroups) {
        const int n = gather_pairs<kGroup>(pos, g, R, rows_total, s);
        for (int c0 = t; c0 < nvec; c0 += kGroup * kVecs) {
            float acc[kVecs][EL];
#pragma unroll
            for (int u = 0; u < kVecs; ++u) {
                const int c = c0 + u * kGroup;
#pragma unroll
                for (int i = 0; i < EL; ++i) acc[u][i] = 0.f;
                if (add != nullptr && c < nvec) VT::add(acc[u], add[g * nvec + c]);  // read before dx, where it is the same
            }
            for (int j0 = 0; j0 < n; j0 += kLoads) {
                uint4 v[kLoads][kVecs];
#pragma unroll
                for (int jj = 0; jj < kLoads; ++jj)
#pragma unroll
                    for (int u = 0; u < kVecs; ++u) {
                        const int c = c0 + u * kGroup;
                        v[jj][u] = (j0 + jj < n && c < nvec) ? ld_stream(dpacked + (int64_t)s.row[j0 + jj] * nvec + c)
                                                             : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                for (int jj = 0; jj < kLoads; ++jj)
#pragma unroll
                    for (int u = 0; u < kVecs; ++u) VT::add(acc[u], v[jj][u]);
            }
#pragma unroll
            for (int u = 0; u < kVecs; ++u) {
                const int c = c0 + u * kGroup;
                if (c < nvec) dx[g * nvec + c] = VT::pack(acc[u]);
            }
        }
        group_sync<kGroup>();
    }
}

struct Launch {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    Launch(int64_t blocks, cudaStream_t stream) {
        attr[0] = pdl_attribute();
        cfg.gridDim = dim3((unsigned)(blocks < 0x7fffffff ? blocks : 0x7fffffff));
        cfg.blockDim = dim3(kThreads);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    Launch(const Launch &) = delete;
};

int row_vectors(int H, int dtype) { return (int)((int64_t)H * (dtype == MOE_BF16 ? 2 : 4) / 16); }
// A token is a warp's where its rows have little together and there are many of them, else a block's.
// A block costs 3.6 ns a token whatever it reads (positions, rows and sums wait for one
// another, and an SM has few blocks); a warp reads less at once.  Warps : blocks, us,
// combine's gradient in bf16, R rows of H: 65536 tokens 2 x 512 61 : 226, 4 x 1024 180 : 252, 2 x 2048 196 :
// 307, 32768 of 4 x 2048 182 : 186, 16384 of 8 x 2048 182 : 169; 4096 tokens 8 x 512 10 : 15, 8 x 1024 19 : 21;
// 2048 of them 7.4 : 8.3 and 12 : 11; 1024 6.3 : 4.8 and 10 : 6.5, 2 x 512 3.2 : 3.8; 256 4.2 : 3.8 (8 x 256) and 2.6 :
// 3.4 (2 x 256).  Dispatch's turns over at the same places (65536 tokens 4 x 1024 98 : 133, 16384 of 8 x 2048 90 : 88).
bool token_per_warp(int64_t NT, int R, int nvec) {
    const int64_t vectors = (int64_t)R * nvec;
    return vectors <= 1024 && vectors * 4 <= NT;
}
int64_t token_blocks(int64_t NT, bool warps) { return warps ? (NT + kThreads / 32 - 1) / (kThreads / 32) : NT; }

}  // namespace

cudaError_t launch_combine_grad(const void *dout, const void *y, int y_dtype, const int32_t *pos, const float *topk_w,
                                int64_t NT, int R, int H, int64_t rows_total, void *dy, float *dtopk_w,
                                cudaStream_t stream) {
    const int nvec = row_vectors(H, y_dtype);
    const bool warps = token_per_warp(NT, R, nvec);
    Launch l(token_blocks(NT, warps), stream);
    auto launch = [&](auto kern) {
        return cudaLaunchKernelEx(&l.cfg, kern, static_cast<const uint4 *>(dout), static_cast<const uint4 *>(y), pos,
                                  topk_w, NT, R, nvec, rows_total, static_cast<uint4 *>(dy), dtopk_w);
    };
    const bool bf16 = y_dtype == MOE_BF16;
    if (warps && R <= 2) return bf16 ? launch(combine_grad_kernel<1, 32, 2, 2>) : launch(combine_grad_kernel<0, 32, 2, 2>);
    if (warps) return bf16 ? launch(combine_grad_kernel<1, 32, 4, 1>) : launch(combine_grad_kernel<0, 32, 4, 1>);
    if (R <= 4) return bf16 ? launch(combine_grad_kernel<1, kThreads, 4, 2>) : launch(combine_grad_kernel<0, kThreads, 4, 2>);
    return bf16 ? launch(combine_grad_kernel<1, kThreads, 8, 1>) : launch(combine_grad_kernel<0, kThreads, 8, 1>);
}

cudaError_t launch_dispatch_grad(const void *dpacked, int x_dtype, const int32_t *pos, const void *add, int64_t NT,
                                 int R, int H, int64_t rows_total, void *dx, cudaStream_t stream) {
    const int nvec = row_vectors(H, x_dtype);
    const bool warps = token_per_warp(NT, R, nvec);
    Launch l(token_blocks(NT, warps), stream);
    auto launch = [&](auto kern) {
        return cudaLaunchKernelEx(&l.cfg, kern, static_cast<const uint4 *>(dpacked), pos, static_cast<const uint4 *>(add),
                                  NT, R, nvec, rows_total, static_cast<uint4 *>(dx));
    };
    if (warps) return x_dtype == MOE_BF16 ? launch(dispatch_grad_kernel<1, 32>) : launch(dispatch_grad_kernel<0, 32>);
    return x_dtype == MOE_BF16 ? launch(dispatch_grad_kernel<1, kThreads>) : launch(dispatch_grad_kernel<0, kThreads>);
}

}  // namespace moe
