// Gradient of the router's weights with respect to its logits, and the sum over
// the tokens that a bias gets.
//
// With h the gradient of the weights w and d = sum_k h_k w_k:
//   softmax                dz_e = p_e (h_e - d): every logit is read
//   softmax, renormalised  the weights are a softmax of the chosen logits alone,
//                          so dz_e = w_k (h_k - d) and no logit is read
//   sigmoid                ds/dz = s (1 - s), 1 - s = 1 / (1 + exp(z)) without
//                          cancellation; renormalised, the other chosen scores
//                          take d off: dz_e = w_k (1 - s_e) (h_k - d)
// All but the first have at most R entries a row: the warp writes the row's
// zeros, then (ordered by __syncwarp) its lanes k < R write their entries, both
// into lines that are still in L2.
#include <math.h>

#include "grad_internal.cuh"
#include "mem_ops.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;  // 8 tokens per block
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
// Sum over the lanes of each aligned run of P.
template <int P>
__device__ __forceinline__ float run_sum(float v) {
#pragma unroll
    for (int o = P / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// What lane k of a run of P >= R lanes knows of its token's k-th expert.
struct Choice {
    int e;       // -1: no part
    float w, h;  // weight and its gradient, 0 without a part
    float d;     // sum of h w over the token
};
template <int P>
__device__ __forceinline__ Choice load_choice(const int32_t *__restrict__ idx, const float *__restrict__ w,
                                              const float *__restrict__ dw, int64_t g, bool inside, int E, int R, int k) {
    Choice c{-1, 0.f, 0.f, 0.f};
    if (inside && k < R) {
        const int e = __ldg(idx + g * R + k);
        const float wk = __ldg(w + g * R + k), hk = __ldg(dw + g * R + k);
        if (e >= 0 && e < E) c.e = e, c.w = wk, c.h = hk;
    }
    c.d = run_sum<P>(c.h * c.w);
    return c;
}

// Sum of v over the lanes of a run that name the same expert, in every one of
// them, in lane order; without repeated experts (as the router chooses them) v
// itself.
template <int P>
__device__ __forceinline__ float sum_same(int e, float v, int lane) {
    const unsigned alike = __match_any_sync(kFull, e < 0 ? -1 - lane : e * 32 + lane / P);
    if (__any_sync(kFull, (alike & (alike - 1)) != 0)) {
        float s = 0.f;
        for (int k = 0; k < 32; ++k) {
            const float o = __shfl_sync(kFull, v, k);
            if ((alike >> k) & 1u) s += o;
        }
        v = s;
    }
    return v;
}

// Entries at the chosen experts only.  A warp takes 32 / P tokens at once, P the
// power of two that holds their R experts: its loads are whole lines and it
// has 32 gathers of logits under way (65536 tokens, 8 of 256 experts, sigmoid
// renormalised: 18.7 to 19.4 us; with a token a warp 27.5).  HBM bounds that: call
// after call (no cache flushed) 67 MB of zeros and entries are written and 51 MB
// read, 6 of them ids, weights and gradients and 44 the 524288 gathered logits, 85
// bytes each; a copy of these 118 MB would take 17.4 us.  Without gathers
// (softmax, renormalised) it writes the same and takes 13 us.
template <int P, bool kVec4>
__global__ void __launch_bounds__(kThreads)
route_grad_chosen_kernel(const float *__restrict__ logits, const float *__restrict__ bias, int64_t NT, int E, int R,
                         int sigmoid, int renormalize, const int32_t *__restrict__ idx, const float *__restrict__ w,
                         const float *__restrict__ dw, float *__restrict__ dlogits) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t first = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * (32 / P);
    if (first >= NT) return;  // uniform per warp
    const int64_t g = first + lane / P;
    const Choice c = load_choice<P>(idx, w, dw, g, g < NT, E, R, lane % P);
    float z = 0.f;
    if (sigmoid && c.e >= 0) {
        z = __ldg(logits + g * E + c.e);
        if (bias != nullptr) z = __fadd_rn(z, __ldg(bias + c.e));
    }
    const int64_t end = (min(first + 32 / P, NT) - first) * E;  // the tokens' rows are one run of memory
    float *rows = dlogits + first * E;
    if (kVec4) {
        for (int64_t i = lane * 4; i < end; i += 128) *reinterpret_cast<float4 *>(rows + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
        for (int64_t i = lane; i < end; i += 32) rows[i] = 0.f;
    }
    float at = c.w * (renormalize ? c.h - c.d : c.h);
    if (sigmoid) at = at / (1.0f + expf(z));
    at = sum_same<P>(c.e, at, lane);
    __syncwarp();
    if (c.e >= 0) dlogits[g * E + c.e] = at;
}

// Softmax over all experts: lane l holds J of them, four in a row at a time.  A
// token's logits are read once (its chosen ones again, from L1); the row is
// written as if nothing had been chosen, then the chosen entries.
// 65536 tokens of 256 experts 27.7 us, 31 with a bias; a copy of its 140 MB would
// take 20.7.  Instructions and a warp's one chain bound it: 341 instructions a
// token fill 76 % of the issue slots, and nothing of the next token is under way
// while the maximum and the sum go round the warp.  25734 of 38 experts take 11.7
// from HBM (a copy: 1.3): of a lane's four places there one or two hold a logit.
template <int J, bool kVec4>
__global__ void __launch_bounds__(kThreads)
route_grad_softmax_kernel(const float *__restrict__ logits, const float *__restrict__ bias, int64_t NT, int E, int R,
                          const int32_t *__restrict__ idx, const float *__restrict__ w, const float *__restrict__ dw,
                          float *__restrict__ dlogits) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t g = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (g >= NT) return;  // uniform per warp
    const float *row = logits + g * E;
    constexpr int kRun = kVec4 ? 4 : 1;
    auto expert = [&](int j) { return (j / kRun * 32 + lane) * kRun + j % kRun; };
    float z[J];
#pragma unroll
    for (int j = 0; j < J; j += kRun) {
        const int e = expert(j);
        if constexpr (kVec4) {
            const float4 v = e < E ? __ldg(reinterpret_cast<const float4 *>(row + e))
                                   : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            z[j] = v.x, z[j + 1] = v.y, z[j + 2] = v.z, z[j + 3] = v.w;
        } else {
            z[j] = e < E ? __ldg(row + e) : -INFINITY;
        }
    }
    const Choice c = load_choice<32>(idx, w, dw, g, true, E, R, lane);
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if (bias != nullptr && expert(j) < E) z[j] = __fadd_rn(z[j], __ldg(bias + expert(j)));
        top = fmaxf(top, z[j]);
    }
    top = warp_max(top);
    bool none = top == -INFINITY;  // nothing to choose from: zeros
    if (none) {  // uniform; the maximum passes NaN by, whose softmax is NaN
        bool nan = false;
#pragma unroll
        for (int j = 0; j < J; ++j) nan |= isnan(z[j]);
        none = !__any_sync(kFull, nan);
    }
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        z[j] = expf(__fsub_rn(z[j], top));
        sum += expert(j) < E ? z[j] : 0.f;
    }
    sum = run_sum<32>(sum);
    const float scale = none ? 0.f : 1.0f / sum, d = none ? 0.f : c.d;
    float *out = dlogits + g * E;
#pragma unroll
    for (int j = 0; j < J; j += kRun) {
        const int e = expert(j);
        if (e >= E) continue;
        if constexpr (kVec4) {
            float4 v = make_float4(z[j], z[j + 1], z[j + 2], z[j + 3]);
            v.x = none ? 0.f : -(v.x * scale * d), v.y = none ? 0.f : -(v.y * scale * d);
            v.z = none ? 0.f : -(v.z * scale * d), v.w = none ? 0.f : -(v.w * scale * d);
            *reinterpret_cast<float4 *>(out + e) = v;
        } else {
            out[e] = none ? 0.f : -(z[j] * scale * d);
        }
    }
    const float h = sum_same<32>(c.e, c.h, lane);
    __syncwarp();
    if (c.e >= 0 && !none) {
        float zc = __ldg(row + c.e);
        if (bias != nullptr) zc = __fadd_rn(zc, __ldg(bias + c.e));
        out[c.e] = expf(__fsub_rn(zc, top)) * scale * (h - d);
    }
}

// ---- bias ------------------------------------------------------------------

// dbias[e] = sum over the tokens of dlogits[g][e], which the kernel before has
// just written.  A cluster of kCluster blocks takes `width` columns, a 32nd of
// them but whole sectors, so that up to 256 blocks read; a block's threads take
// one column each of kSumThreads / width rows at a time.  A thread adds kRunRows
// values in f32 and those sums with what they round off; so does the block its
// threads' in a tree, and the first block the others' in their order.  No
// atomics: the same call gives the same bits.  Gradient and sum, us: 4101 tokens of 93
// experts 7.2 (the gradient alone 3.3), 25734 of 38 16.7 (10.2), 65536 of 256 53 (31).  The
// sum alone then reads 67 MB, half of them still in L2, in 22 us, at half of HBM's rate:
// a thread's additions of 16 values are one chain, and its next 16 loads are
// issued behind them, so that little is under way during the additions
// (loads are half of what the warps wait for).  With 1024 threads 8.9, 16.3, 65, 256 7.3, 19.6,
// 81; in clusters of four 7.7, 20, 85; by a 16th of the columns 7.2, 16.8, 62; 64-bit sums and
// 1024 threads 11.1, 18.4, 69.
constexpr int kCluster = 8;
constexpr int kSumThreads = 512;
constexpr int kRunRows = 16;

// A sum of f32 numbers and what its roundings took off (Knuth's two-sum): as good
// as 48 bits, where the GPU has few 64-bit units.
struct Sum2 {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float s = __fadd_rn(hi, v), t = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(v, t)));
        hi = s;
    }
    __device__ __forceinline__ void add(float vhi, float vlo) {
        add(vhi);
        lo = __fadd_rn(lo, vlo);
    }
    __device__ __forceinline__ float value() const {  // lo is NaN where hi is infinite
        return isfinite(hi) ? __fadd_rn(hi, lo) : hi;
    }
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSumThreads)
column_sum_kernel(const float *__restrict__ d, int64_t NT, int E, int width, float *__restrict__ dbias) {
    __shared__ float2 part[kSumThreads];
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int lanes = kSumThreads / width;  // rows at a time
    const int c = threadIdx.x % width, lane = threadIdx.x / width, e = (int)(blockIdx.x / kCluster) * width + c;
    grid_dependency_wait();  // d comes from the kernel before
    grid_launch_dependents();
    Sum2 sum;
    if (e < E && lane < lanes) {
        const int64_t step = (int64_t)kCluster * lanes;
        for (int64_t g = (int64_t)rank * lanes + lane; g < NT; g += step * kRunRows) {
            float v[kRunRows], run = 0.f;
#pragma unroll
            for (int i = 0; i < kRunRows; ++i) {
                const int64_t r = g + i * step;
                v[i] = r < NT ? __ldg(d + r * E + e) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kRunRows; ++i) run += v[i];
            sum.add(run);
        }
    }
    part[threadIdx.x] = make_float2(sum.hi, sum.lo);
    __syncthreads();
    for (int n = lanes; n > 1;) {
        const int half = (n + 1) / 2;
        if (lane < n - half) {
            const float2 o = part[threadIdx.x + half * width];
            sum.add(o.x, o.y);
            part[threadIdx.x] = make_float2(sum.hi, sum.lo);
        }
        __syncthreads();
        n = half;
    }
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    if (rank == 0 && lane == 0) {
        Sum2 t;
        const uint32_t here = (uint32_t)__cvta_generic_to_shared(&part[c]);
#pragma unroll
        for (int i = 0; i < kCluster; ++i) {
            uint32_t there;
            float2 v;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(i));
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(there) : "memory");
            t.add(v.x, v.y);
        }
        if (e < E) dbias[e] = t.value();
    }
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");  // the sums are read
}

struct Launch {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    Launch(int64_t blocks, cudaStream_t stream, int threads = kThreads) {
        attr[0] = pdl_attribute();
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(threads);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    Launch(const Launch &) = delete;
};

}  // namespace

cudaError_t launch_route_grad(const float *logits, const float *bias, int64_t NT, int E, int R, int score_fn,
                              int renormalize, const int32_t *topk_idx, const float *topk_w, const float *dtopk_w,
                              float *dlogits, float *dbias, cudaStream_t stream) {
    const bool softmax = (score_fn & ~MOE_BIAS_SELECT_ONLY) == MOE_SOFTMAX;
    if (score_fn & MOE_BIAS_SELECT_ONLY) bias = nullptr;  // the scores are the raw logits'
    auto at16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    auto blocks = [&](int tokens) { return (NT + tokens * kWarps - 1) / (tokens * kWarps); };
    cudaError_t e = cudaErrorInvalidValue;
    if (softmax && !renormalize) {
        const bool vec = E % 4 == 0 && at16(logits) && at16(dlogits);
        Launch l(blocks(1), stream);
        auto launch = [&](auto kern) {
            return cudaLaunchKernelEx(&l.cfg, kern, logits, bias, NT, E, R, topk_idx, topk_w, dtopk_w, dlogits);
        };
#define MOE_CASE(J) E <= 32 * J ? launch(vec ? route_grad_softmax_kernel<J, true> : route_grad_softmax_kernel<J, false>)
        e = MOE_CASE(4) : MOE_CASE(8) : MOE_CASE(16) : launch(vec ? route_grad_softmax_kernel<32, true> : route_grad_softmax_kernel<32, false>);
#undef MOE_CASE
    } else {
        const bool vec = E % 4 == 0 && at16(dlogits);
        auto launch = [&](int tokens, auto kern) {
            Launch l(blocks(tokens), stream);
            return cudaLaunchKernelEx(&l.cfg, kern, logits, bias, NT, E, R, softmax ? 0 : 1, renormalize, topk_idx, topk_w,
                                      dtopk_w, dlogits);
        };
#define MOE_CASE(P) R <= P ? launch(32 / P, vec ? route_grad_chosen_kernel<P, true> : route_grad_chosen_kernel<P, false>)
        e = MOE_CASE(2) : MOE_CASE(4) : MOE_CASE(8) : MOE_CASE(16) : launch(1, vec ? route_grad_chosen_kernel<32, true> : route_grad_chosen_kernel<32, false>);
#undef MOE_CASE
    }
    if (e != cudaSuccess || dbias == nullptr) return e;
    const int width = ((E + 31) / 32 + 7) / 8 * 8;  // whole sectors of a row where E is a multiple of 8
    Launch s((E + width - 1) / width * kCluster, stream, kSumThreads);
    return cudaLaunchKernelEx(&s.cfg, column_sum_kernel, static_cast<const float *>(dlogits), NT, E, width, dbias);
}

}  // namespace moe
