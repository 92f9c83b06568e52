// C entry points of libmoe_route.so: argument validation on the host, then
// one launcher per step.  See include/moe_route.h for the contract.
#include <stdarg.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <cuda.h>  // types only: the driver calls are fetched at run time

#include "expert_internal.cuh"
#include "expert_w4_internal.cuh"
#include "grad_internal.cuh"
#include "moe_internal.cuh"

namespace moe {

bool encode_map(CUtensorMap *m, int fp8, int rank, const void *base, const uint64_t *dims, const uint64_t *strides,
                const uint32_t *box);  // declared for the kernels in tc_ops.cuh

namespace {
thread_local char g_err[512] = "";
}

int set_error(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return code;
}

namespace {
// Driver functions fetched through the runtime (no link against libcuda).
typedef CUresult (*CtxGetCurrentFn)(CUcontext *);
typedef CUresult (*CtxGetIdFn)(CUcontext, unsigned long long *);
struct CtxFns {
    CtxGetCurrentFn get_current = nullptr;
    CtxGetIdFn get_id = nullptr;
    CtxFns() {
        cudaDriverEntryPointQueryResult q;
        void *f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            get_current = reinterpret_cast<CtxGetCurrentFn>(f);
        f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_id = reinterpret_cast<CtxGetIdFn>(f);
        cudaGetLastError();
    }
};
}  // namespace

unsigned long long context_key() {
    static const CtxFns fns;  // initialised once, thread-safe
    if (fns.get_current == nullptr || fns.get_id == nullptr) return 0;
    CUcontext ctx = nullptr;
    if (fns.get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr) return 0;
    unsigned long long id = 0;
    if (fns.get_id(ctx, &id) != CUDA_SUCCESS) return 0;
    return id + 1;  // never 0 for a real context
}

// Tensor maps of the experts' products.
bool encode_map(CUtensorMap *m, int fp8, int rank, const void *base, const uint64_t *dims, const uint64_t *strides,
                const uint32_t *box) {
    typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const EncodeFn encode = [] {  // initialised once, thread-safe
        cudaDriverEntryPointQueryResult q;
        void *f = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess || q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    if (encode == nullptr) return false;
    cuuint64_t d[5], st[4];
    cuuint32_t b[5], one[5] = {1, 1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        if (i + 1 < rank) st[i] = strides[i];
    }
    auto call = [&] {
        return encode(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
                      const_cast<void *>(base), d, st, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = call();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {
        // the calling thread's first use of CUDA: the driver wants a current
        // context, which the runtime would bind at the launch only
        int dev = 0;
        if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = call();
    }
    return r == CUDA_SUCCESS;
}

int sm_count() {
    static thread_local int dev_cached = -1, sms = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev != dev_cached) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) sms = 0;
        dev_cached = dev;
    }
    return sms;
}

int64_t l2_bytes() {
    static thread_local int dev_cached = -1, l2 = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev != dev_cached) {
        if (cudaDeviceGetAttribute(&l2, cudaDevAttrL2CacheSize, dev) != cudaSuccess) l2 = 0;
        dev_cached = dev;
    }
    return l2;
}

namespace {

constexpr int64_t kI32Max = 2147483647;

struct Derived {
    int64_t NT, cap, rows_total, pairs, x_row_bytes, y_row_bytes;
    int scales_per_row;
};

int elem_bytes(int dtype) {
    switch (dtype) {
        case MOE_BF16: return 2;
        case MOE_F32: return 4;
        case MOE_FP8E4M3_BLK128: return 1;
        default: return 0;
    }
}

// Validates dims and fills the derived sizes.  `what` names the caller.
int check_dims(const MoeDims *d, Derived *out, const char *what) {
    g_err[0] = '\0';
    if (d == nullptr) return set_error(MOE_ERR_INVALID_ARG, "%s: dims is NULL", what);
    if (d->N < 1 || d->T < 0 || d->E < 1 || d->R < 1 || d->H < 1)
        return set_error(MOE_ERR_INVALID_ARG, "%s: need N>=1, T>=0, E>=1, R>=1, H>=1 (got N=%d T=%d E=%d R=%d H=%d)",
                         what, d->N, d->T, d->E, d->R, d->H);
    if (d->E % d->N != 0)
        return set_error(MOE_ERR_INVALID_ARG, "%s: E=%d is not a multiple of N=%d", what, d->E, d->N);
    if (d->R > d->E)
        return set_error(MOE_ERR_INVALID_ARG, "%s: R=%d exceeds E=%d", what, d->R, d->E);
    if (d->E > 1024 || d->R > 32)
        return set_error(MOE_ERR_UNSUPPORTED, "%s: this build supports E<=1024 and R<=32 (got E=%d R=%d)",
                         what, d->E, d->R);
    if (d->reserved != 0) return set_error(MOE_ERR_INVALID_ARG, "%s: dims.reserved must be 0", what);
    if (elem_bytes(d->x_dtype) == 0)
        return set_error(MOE_ERR_INVALID_ARG, "%s: unknown x_dtype %d", what, d->x_dtype);
    if (d->y_dtype != MOE_BF16 && d->y_dtype != MOE_F32)
        return set_error(MOE_ERR_INVALID_ARG, "%s: y_dtype must be MOE_BF16 or MOE_F32 (got %d)", what,
                         d->y_dtype);
    if (d->H % 8 != 0)
        return set_error(MOE_ERR_INVALID_ARG, "%s: H=%d must be a multiple of 8", what, d->H);
    if (d->H > (1 << 24))  // keeps per-row vector counts and in-row indices in 32 bits
        return set_error(MOE_ERR_UNSUPPORTED, "%s: this build supports H <= 2^24 (got H=%d)", what, d->H);
    if (d->x_dtype == MOE_FP8E4M3_BLK128 && d->H % 128 != 0)
        return set_error(MOE_ERR_INVALID_ARG, "%s: fp8 rows need H %% 128 == 0 (got H=%d)", what, d->H);
    if (d->cap_rows < 0) return set_error(MOE_ERR_INVALID_ARG, "%s: cap_rows < 0", what);
    Derived v;
    v.NT = (int64_t)d->N * d->T;
    const int64_t L = d->E / d->N;
    const int64_t bound = v.NT * (d->R > L ? d->R : L);
    v.cap = d->cap_rows > 0 ? d->cap_rows : bound;
    if (v.cap < 1) v.cap = 1;  // T == 0: keep the region arithmetic well defined
    v.pairs = v.NT * d->R;
    v.rows_total = (int64_t)d->N * v.cap;
    if (v.pairs > kI32Max || v.rows_total > kI32Max || v.NT > kI32Max - 65536)
        return set_error(MOE_ERR_UNSUPPORTED,
                         "%s: N*T*R=%lld and N*cap=%lld must stay below 2^31 (32-bit row indices)",
                         what, (long long)v.pairs, (long long)v.rows_total);
    v.x_row_bytes = (int64_t)d->H * elem_bytes(d->x_dtype);
    v.y_row_bytes = (int64_t)d->H * elem_bytes(d->y_dtype);
    v.scales_per_row = d->x_dtype == MOE_FP8E4M3_BLK128 ? d->H / 128 : 0;
    if (out) *out = v;
    return MOE_OK;
}

// Pack kernel choice: the register-path kernel by default (the faster of
// the two on GB300 at R = 8); the environment variable MOE_PACK_KERNEL=bulk
// selects bulk copies through shared memory (read once per process).
bool use_bulk_pack() {
    static const bool bulk = [] {
        const char *v = getenv("MOE_PACK_KERNEL");
        return v && strcmp(v, "bulk") == 0;
    }();
    return bulk;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int cuda_result(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return MOE_OK;
    return set_error(MOE_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Checks of the experts' products: dims, the product's own sizes and act.
// `gated`: the matrices have 2F rows; `elem`: bytes of an operand's element.
int check_expert(const MoeDims *dims, int K, int F, bool gated, int elem, const int32_t *offsets, Derived *v,
                 ExpertRows *r, const char *what) {
    int rc = check_dims(dims, v, what);
    if (rc != MOE_OK) return rc;
    if (K < 8 || F < 8 || K % 8 != 0 || F % 8 != 0)
        return set_error(MOE_ERR_INVALID_ARG, "%s: K=%d and F=%d must be positive multiples of 8", what, K, F);
    if (K > (1 << 24) || F > (1 << 24))
        return set_error(MOE_ERR_UNSUPPORTED, "%s: this build supports K, F <= 2^24 (got K=%d F=%d)", what, K, F);
    if (v->rows_total > kI32Max - 65536)  // a block's last load begins up to a tile behind the last row
        return set_error(MOE_ERR_UNSUPPORTED, "%s: N*cap=%lld must stay below 2^31 - 65536", what, (long long)v->rows_total);
    const int64_t wide = gated ? 2 * (int64_t)F : F;
    if (wide * K * elem >= (int64_t)1 << 40)  // the stride of a tensor map
        return set_error(MOE_ERR_UNSUPPORTED, "%s: a matrix of %lld x %d must stay below 2^40 bytes", what,
                         (long long)wide, K);
    const int64_t big = wide > K ? wide : K;
    if ((v->pairs / 128 + dims->E) * ((big + 127) / 128) > kI32Max - 65536 ||
        (int64_t)dims->E * ((wide + 127) / 128) * (((int64_t)K + 127) / 128) > kI32Max - 65536)
        return set_error(MOE_ERR_UNSUPPORTED, "%s: too many tiles (N*T*R=%lld, E=%d, K=%d, F=%d)", what,
                         (long long)v->pairs, dims->E, K, F);
    if (!offsets || !aligned(offsets, 4))
        return set_error(MOE_ERR_INVALID_ARG, "%s: expert_offsets must be a 4-byte aligned pointer", what);
    // a token takes an expert once, and what does not fit the region is dropped
    *r = ExpertRows{offsets, dims->E, dims->E / dims->N, v->cap, v->rows_total, v->NT < v->cap ? v->NT : v->cap,
                    v->pairs};
    return MOE_OK;
}

bool bad_block_pointers(const void *a, const void *b, const void *c, const char *what, int *rc) {
    if (!a || !b || !c) {
        *rc = set_error(MOE_ERR_INVALID_ARG, "%s: a required pointer is NULL", what);
        return true;
    }
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(c, 16)) {
        *rc = set_error(MOE_ERR_INVALID_ARG, "%s: rows, matrices and results must be 16-byte aligned", what);
        return true;
    }
    return false;
}

// An array that a call reads or writes.
struct Span {
    const void *p;
    int64_t bytes;
};
bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}
Span offsets_span(const ExpertRows &r) { return {r.offsets, ((int64_t)r.E + 1) * 4}; }
// The kernels read their inputs by blocks, in no order: results in the same
// memory are refused.
template <int kIn>
bool overlap_any(const Span &out, const Span (&in)[kIn], const char *what, int *rc) {
    for (const Span &i : in)
        if (overlap(out, i)) {
            *rc = set_error(MOE_ERR_INVALID_ARG, "%s: a result overlaps another array of the call", what);
            return true;
        }
    return false;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_version(void) { return MOE_VERSION; }

const char *moe_last_error(void) { return g_err; }

int moe_buffer_sizes(const MoeDims *dims, MoeSizes *out) {
    Derived v;
    int rc = check_dims(dims, &v, "moe_buffer_sizes");
    if (rc != MOE_OK) return rc;
    if (out == nullptr) return set_error(MOE_ERR_INVALID_ARG, "moe_buffer_sizes: out is NULL");
    const int64_t N = dims->N, E = dims->E, H = dims->H;
    const int64_t L = E / N;
    memset(out, 0, sizeof(*out));
    out->bound_rows = v.NT * (dims->R > L ? dims->R : L);
    out->cap_rows = v.cap;
    out->total_pairs = v.pairs;
    out->logits_bytes = v.NT * E * 4;
    out->topk_idx_bytes = v.pairs * 4;
    out->topk_w_bytes = v.pairs * 4;
    out->pos_bytes = v.pairs * 4;
    out->expert_counts_bytes = E * 4;
    out->expert_offsets_bytes = (E + 1) * 4;
    out->rank_counts_bytes = N * 4;
    out->rank_offsets_bytes = (N + 1) * 4;
    out->send_counts_bytes = N * N * 4;
    out->x_bytes = v.NT * v.x_row_bytes;
    out->x_scales_bytes = v.NT * v.scales_per_row * 4;
    out->packed_x_bytes = v.rows_total * v.x_row_bytes;
    out->packed_scales_bytes = v.rows_total * v.scales_per_row * 4;
    out->packed_src_bytes = v.rows_total * 4;
    out->y_bytes = v.rows_total * v.y_row_bytes;
    out->out_bytes = v.NT * v.y_row_bytes;
    out->status_bytes = 4;
    out->partial_slots = dims->R < N ? dims->R : N;
    out->partial_bytes = v.NT * out->partial_slots * v.y_row_bytes;
    out->slot_rank_bytes = v.NT * out->partial_slots * 4;
    out->fused_workspace_bytes = fused_workspace_bytes(dims->N, dims->T, dims->E);
    (void)H;
    return MOE_OK;
}

static bool valid_score_fn(int score_fn) {
    const int fn = score_fn & ~MOE_BIAS_SELECT_ONLY;
    return fn == MOE_SOFTMAX || fn == MOE_SIGMOID;
}

int moe_route_topk(const MoeDims *dims, const float *logits, const float *bias, int score_fn,
                   int renormalize, int32_t *topk_idx, float *topk_w, void *stream) {
    Derived v;
    int rc = check_dims(dims, &v, "moe_route_topk");
    if (rc != MOE_OK) return rc;
    if (!valid_score_fn(score_fn))
        return set_error(MOE_ERR_INVALID_ARG, "moe_route_topk: unknown score_fn %d", score_fn);
    if (v.NT == 0) return MOE_OK;
    if (!logits || !topk_idx || !topk_w)
        return set_error(MOE_ERR_INVALID_ARG, "moe_route_topk: logits, topk_idx and topk_w must be non-NULL");
    if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4) || (bias && !aligned(bias, 4)))
        return set_error(MOE_ERR_INVALID_ARG, "moe_route_topk: pointers must be 4-byte aligned");
    return cuda_result(launch_route_topk(logits, bias, v.NT, dims->E, dims->R, score_fn, renormalize ? 1 : 0,
                                         topk_idx, topk_w, (cudaStream_t)stream),
                       "moe_route_topk");
}

int moe_dispatch_count(const MoeDims *dims, const int32_t *topk_idx, int32_t *expert_counts,
                       int32_t *expert_offsets, int32_t *rank_counts, int32_t *rank_offsets,
                       int32_t *send_counts, int32_t *pos, int32_t *status, void *stream) {
    Derived v;
    int rc = check_dims(dims, &v, "moe_dispatch_count");
    if (rc != MOE_OK) return rc;
    if (!expert_counts || !expert_offsets || !rank_counts || !rank_offsets || !send_counts || !status ||
        (v.NT > 0 && (!topk_idx || !pos)))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_count: a required pointer is NULL");
    const void *ptrs[] = {topk_idx, expert_counts, expert_offsets, rank_counts, rank_offsets,
                          send_counts, pos, status};
    for (const void *p : ptrs)
        if (p && !aligned(p, 4))
            return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_count: pointers must be 4-byte aligned");
    cudaError_t e = launch_dispatch_count(topk_idx, dims->N, dims->T, dims->E, dims->R, v.cap,
                                          expert_counts, expert_offsets, rank_counts, rank_offsets,
                                          send_counts, pos, status, (cudaStream_t)stream);
    if (e == cudaErrorNotSupported)
        return set_error(MOE_ERR_UNSUPPORTED,
                         "moe_dispatch_count: the device cannot schedule a thread-block cluster of this kernel");
    return cuda_result(e, "moe_dispatch_count");
}

int moe_dispatch_pack(const MoeDims *dims, const void *x, const float *x_scales, const int32_t *pos,
                      void *packed_x, float *packed_scales, int32_t *packed_src, void *stream) {
    Derived v;
    int rc = check_dims(dims, &v, "moe_dispatch_pack");
    if (rc != MOE_OK) return rc;
    if (v.NT == 0) return MOE_OK;
    const bool fp8 = dims->x_dtype == MOE_FP8E4M3_BLK128;
    if (!x || !pos || !packed_x || !packed_src || (fp8 && (!x_scales || !packed_scales)))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_pack: a required pointer is NULL");
    if (!aligned(x, 16) || !aligned(packed_x, 16))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_pack: x and packed_x must be 16-byte aligned");
    if (!aligned(pos, 4) || !aligned(packed_src, 4) || (fp8 && (!aligned(x_scales, 4) || !aligned(packed_scales, 4))))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_pack: index and scale pointers must be 4-byte aligned");
    if (use_bulk_pack() && pack_bulk_stages(v.x_row_bytes) > 0)
        return cuda_result(launch_dispatch_pack_bulk(x, fp8 ? x_scales : nullptr, pos, v.NT, dims->R,
                                                     v.x_row_bytes, v.scales_per_row, v.rows_total, packed_x,
                                                     fp8 ? packed_scales : nullptr, packed_src,
                                                     (cudaStream_t)stream),
                           "moe_dispatch_pack");
    return cuda_result(launch_dispatch_pack(x, fp8 ? x_scales : nullptr, pos, v.NT, dims->R, v.x_row_bytes,
                                            v.scales_per_row, v.rows_total, packed_x,
                                            fp8 ? packed_scales : nullptr, packed_src,
                                            (cudaStream_t)stream),
                       "moe_dispatch_pack");
}

int moe_dispatch_pack_quant(const MoeDims *dims, const void *x, const int32_t *pos, void *packed_q,
                            float *packed_scales, int32_t *packed_src, void *stream) {
    Derived v;
    int rc = check_dims(dims, &v, "moe_dispatch_pack_quant");
    if (rc != MOE_OK) return rc;
    if (dims->x_dtype != MOE_BF16)
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_pack_quant: x_dtype must be MOE_BF16 (the rows it reads)");
    if (dims->H % 128 != 0)
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_pack_quant: H=%d must be a multiple of 128", dims->H);
    if (v.NT == 0) return MOE_OK;
    if (!x || !pos || !packed_q || !packed_scales || !packed_src)
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_pack_quant: a required pointer is NULL");
    if (!aligned(x, 16) || !aligned(packed_q, 16))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_pack_quant: x and packed_q must be 16-byte aligned");
    if (!aligned(pos, 4) || !aligned(packed_scales, 4) || !aligned(packed_src, 4))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_pack_quant: pos, packed_scales and packed_src must be 4-byte aligned");
    return cuda_result(launch_dispatch_pack_quant(x, pos, v.NT, dims->R, dims->H, v.rows_total, packed_q,
                                                  packed_scales, packed_src, (cudaStream_t)stream),
                       "moe_dispatch_pack_quant");
}

int moe_combine(const MoeDims *dims, const void *y, const int32_t *pos, const float *topk_w, void *out,
                void *stream) {
    Derived v;
    int rc = check_dims(dims, &v, "moe_combine");
    if (rc != MOE_OK) return rc;
    if (v.NT == 0) return MOE_OK;
    if (!y || !pos || !topk_w || !out)
        return set_error(MOE_ERR_INVALID_ARG, "moe_combine: a required pointer is NULL");
    if (!aligned(y, 16) || !aligned(out, 16))
        return set_error(MOE_ERR_INVALID_ARG, "moe_combine: y and out must be 16-byte aligned");
    if (!aligned(pos, 4) || !aligned(topk_w, 4))
        return set_error(MOE_ERR_INVALID_ARG, "moe_combine: pos and topk_w must be 4-byte aligned");
    return cuda_result(launch_combine(y, dims->y_dtype, pos, topk_w, v.NT, dims->R, dims->H, v.rows_total,
                                      out, (cudaStream_t)stream),
                       "moe_combine");
}

int moe_dispatch_pack_rank(const MoeDims *dims, int rank, const void *x, const float *x_scales,
                           const int32_t *pos, void *packed_x, float *packed_scales,
                           int32_t *packed_src, void *stream) {
    Derived v;
    int rc = check_dims(dims, &v, "moe_dispatch_pack_rank");
    if (rc != MOE_OK) return rc;
    if (rank < 0 || rank >= dims->N)
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_pack_rank: rank %d outside [0, %d)", rank, dims->N);
    if (v.NT == 0) return MOE_OK;
    const bool fp8 = dims->x_dtype == MOE_FP8E4M3_BLK128;
    if (!x || !pos || !packed_x || !packed_src || (fp8 && (!x_scales || !packed_scales)))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_pack_rank: a required pointer is NULL");
    if (!aligned(x, 16) || !aligned(packed_x, 16))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_pack_rank: x and packed_x must be 16-byte aligned");
    if (!aligned(pos, 4) || !aligned(packed_src, 4) || (fp8 && (!aligned(x_scales, 4) || !aligned(packed_scales, 4))))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_pack_rank: index and scale pointers must be 4-byte aligned");
    return cuda_result(launch_pack_rank(x, fp8 ? x_scales : nullptr, pos, v.NT, dims->R, v.x_row_bytes,
                                        v.scales_per_row, (int64_t)rank * v.cap, (int64_t)(rank + 1) * v.cap,
                                        packed_x, fp8 ? packed_scales : nullptr, packed_src,
                                        (cudaStream_t)stream),
                       "moe_dispatch_pack_rank");
}

int moe_combine_rank(const MoeDims *dims, int rank, const void *y, const int32_t *pos,
                     const float *topk_w, void *out, void *stream) {
    Derived v;
    int rc = check_dims(dims, &v, "moe_combine_rank");
    if (rc != MOE_OK) return rc;
    if (rank < 0 || rank >= dims->N)
        return set_error(MOE_ERR_INVALID_ARG, "moe_combine_rank: rank %d outside [0, %d)", rank, dims->N);
    if (v.NT == 0) return MOE_OK;
    if (!y || !pos || !topk_w || !out)
        return set_error(MOE_ERR_INVALID_ARG, "moe_combine_rank: a required pointer is NULL");
    if (!aligned(y, 16) || !aligned(out, 16))
        return set_error(MOE_ERR_INVALID_ARG, "moe_combine_rank: y and out must be 16-byte aligned");
    if (!aligned(pos, 4) || !aligned(topk_w, 4))
        return set_error(MOE_ERR_INVALID_ARG, "moe_combine_rank: pos and topk_w must be 4-byte aligned");
    return cuda_result(launch_combine_rank(y, dims->y_dtype, pos, topk_w, v.NT, dims->R, dims->H,
                                           (int64_t)rank * v.cap, (int64_t)(rank + 1) * v.cap, out,
                                           (cudaStream_t)stream),
                       "moe_combine_rank");
}

int moe_combine_partials(const MoeDims *dims, const void *y, const int32_t *pos,
                         const float *topk_w, void *partial, int32_t *slot_rank, void *stream) {
    Derived v;
    int rc = check_dims(dims, &v, "moe_combine_partials");
    if (rc != MOE_OK) return rc;
    if (v.NT == 0) return MOE_OK;
    if (!y || !pos || !topk_w || !partial || !slot_rank)
        return set_error(MOE_ERR_INVALID_ARG, "moe_combine_partials: a required pointer is NULL");
    if (!aligned(y, 16) || !aligned(partial, 16))
        return set_error(MOE_ERR_INVALID_ARG, "moe_combine_partials: y and partial must be 16-byte aligned");
    if (!aligned(pos, 4) || !aligned(topk_w, 4) || !aligned(slot_rank, 4))
        return set_error(MOE_ERR_INVALID_ARG, "moe_combine_partials: pos, topk_w and slot_rank must be 4-byte aligned");
    const int P = dims->R < dims->N ? dims->R : dims->N;
    return cuda_result(launch_combine_partials(y, dims->y_dtype, pos, topk_w, v.NT, dims->R, dims->H, v.cap,
                                               v.rows_total, P, partial, slot_rank, (cudaStream_t)stream),
                       "moe_combine_partials");
}

int moe_combine_reduce_partials(const MoeDims *dims, const void *partial, const int32_t *slot_rank,
                                void *out, void *stream) {
    Derived v;
    int rc = check_dims(dims, &v, "moe_combine_reduce_partials");
    if (rc != MOE_OK) return rc;
    if (v.NT == 0) return MOE_OK;
    if (!partial || !slot_rank || !out)
        return set_error(MOE_ERR_INVALID_ARG, "moe_combine_reduce_partials: a required pointer is NULL");
    if (!aligned(partial, 16) || !aligned(out, 16) || !aligned(slot_rank, 4))
        return set_error(MOE_ERR_INVALID_ARG, "moe_combine_reduce_partials: misaligned pointer");
    const int P = dims->R < dims->N ? dims->R : dims->N;
    return cuda_result(launch_reduce_partials(partial, dims->y_dtype, slot_rank, v.NT, P, dims->H, out,
                                              (cudaStream_t)stream),
                       "moe_combine_reduce_partials");
}

int moe_dispatch_fused(const MoeDims *dims, const float *logits, const float *bias, int score_fn,
                       int renormalize, const void *x, const float *x_scales, int32_t *topk_idx,
                       float *topk_w, int32_t *expert_counts, int32_t *expert_offsets,
                       int32_t *rank_counts, int32_t *rank_offsets, int32_t *send_counts, int32_t *pos,
                       int32_t *status, void *packed_x, float *packed_scales, int32_t *packed_src,
                       void *workspace, void *stream) {
    Derived v;
    int rc = check_dims(dims, &v, "moe_dispatch_fused");
    if (rc != MOE_OK) return rc;
    if (!valid_score_fn(score_fn))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_fused: unknown score_fn %d", score_fn);
    const char *why = fused_unsupported(dims->N, dims->T, dims->E, dims->R, v.x_row_bytes);
    if (why[0] != '\0')
        return set_error(MOE_ERR_UNSUPPORTED, "moe_dispatch_fused: %s; use the separate calls", why);
    const bool fp8 = dims->x_dtype == MOE_FP8E4M3_BLK128;
    // an empty batch touches no workspace (its size is 0 there): NULL is fine
    if (!expert_counts || !expert_offsets || !rank_counts || !rank_offsets || !send_counts || !status ||
        (!workspace && v.NT > 0))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_fused: a required pointer is NULL");
    if (v.NT > 0 && (!logits || !x || !topk_idx || !topk_w || !pos || !packed_x || !packed_src ||
                     (fp8 && (!x_scales || !packed_scales))))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_fused: a required pointer is NULL");
    if ((x && !aligned(x, 16)) || (packed_x && !aligned(packed_x, 16)) || (workspace && !aligned(workspace, 16)))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_fused: x, packed_x and workspace must be 16-byte aligned");
    const void *ptrs4[] = {logits, bias, topk_idx, topk_w, expert_counts, expert_offsets, rank_counts,
                           rank_offsets, send_counts, pos, status, packed_src, x_scales, packed_scales};
    for (const void *p : ptrs4)
        if (p && !aligned(p, 4))
            return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_fused: pointers must be 4-byte aligned");
    cudaError_t e = launch_dispatch_fused(logits, bias, score_fn, renormalize ? 1 : 0, x, fp8 ? x_scales : nullptr,
                                          dims->N, dims->T, dims->E, dims->R, v.x_row_bytes, v.scales_per_row,
                                          v.cap, topk_idx, topk_w, expert_counts, expert_offsets, rank_counts,
                                          rank_offsets, send_counts, pos, status, packed_x,
                                          fp8 ? packed_scales : nullptr, packed_src, workspace,
                                          (cudaStream_t)stream);
    if (e == cudaErrorNotSupported)
        return set_error(MOE_ERR_UNSUPPORTED, "moe_dispatch_fused: the device cannot run this batch fused "
                                              "(thread-block cluster unavailable)");
    return cuda_result(e, "moe_dispatch_fused");
}

int moe_dispatch_fused_quant(const MoeDims *dims, const float *logits, const float *bias, int score_fn,
                             int renormalize, const void *x, int32_t *topk_idx, float *topk_w,
                             int32_t *expert_counts, int32_t *expert_offsets, int32_t *rank_counts,
                             int32_t *rank_offsets, int32_t *send_counts, int32_t *pos, int32_t *status,
                             void *packed_q, float *packed_scales, int32_t *packed_src, void *workspace,
                             void *stream) {
    Derived v;
    int rc = check_dims(dims, &v, "moe_dispatch_fused_quant");
    if (rc != MOE_OK) return rc;
    if (!valid_score_fn(score_fn))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_fused_quant: unknown score_fn %d", score_fn);
    if (dims->x_dtype != MOE_BF16)
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_fused_quant: x_dtype must be MOE_BF16 (the rows it reads)");
    if (dims->H % 128 != 0)
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_fused_quant: H=%d must be a multiple of 128", dims->H);
    const char *why = fused_quant_unsupported(dims->N, dims->T, dims->E, dims->R);
    if (why[0] != '\0')
        return set_error(MOE_ERR_UNSUPPORTED, "moe_dispatch_fused_quant: %s; use the separate calls", why);
    // an empty batch touches no workspace (its size is 0 there): NULL is fine
    if (!expert_counts || !expert_offsets || !rank_counts || !rank_offsets || !send_counts || !status ||
        (!workspace && v.NT > 0))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_fused_quant: a required pointer is NULL");
    if (v.NT > 0 && (!logits || !x || !topk_idx || !topk_w || !pos || !packed_q || !packed_scales || !packed_src))
        return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_fused_quant: a required pointer is NULL");
    if ((x && !aligned(x, 16)) || (packed_q && !aligned(packed_q, 16)) || (workspace && !aligned(workspace, 16)))
        return set_error(MOE_ERR_INVALID_ARG,
                         "moe_dispatch_fused_quant: x, packed_q and workspace must be 16-byte aligned");
    const void *ptrs4[] = {logits, bias, topk_idx, topk_w, expert_counts, expert_offsets, rank_counts,
                           rank_offsets, send_counts, pos, status, packed_scales, packed_src};
    for (const void *p : ptrs4)
        if (p && !aligned(p, 4))
            return set_error(MOE_ERR_INVALID_ARG, "moe_dispatch_fused_quant: pointers must be 4-byte aligned");
    return cuda_result(launch_dispatch_fused_quant(logits, bias, score_fn, renormalize ? 1 : 0, x, dims->N, dims->T,
                                                   dims->E, dims->R, dims->H, v.cap, topk_idx, topk_w,
                                                   expert_counts, expert_offsets, rank_counts, rank_offsets,
                                                   send_counts, pos, status, packed_q, packed_scales, packed_src,
                                                   workspace, (cudaStream_t)stream),
                       "moe_dispatch_fused_quant");
}

int moe_dispatch_fused_static(const MoeDims *dims, const float *logits, const float *bias, int score_fn,
                              int renormalize, const void *x, const float *x_scales, int32_t *topk_idx,
                              float *topk_w, int32_t *expert_counts, int32_t *expert_offsets,
                              int32_t *rank_counts, int32_t *rank_offsets, int32_t *send_counts,
                              int32_t *pos, int32_t *status, void *packed_x, float *packed_scales,
                              int32_t *packed_src, void *stream) {
    Derived v;
    int rc = check_dims(dims, &v, "moe_dispatch_fused_static");
    if (rc != MOE_OK) return rc;
    const char *why = fused_unsupported(dims->N, dims->T, dims->E, dims->R, v.x_row_bytes);
    if (why[0] != '\0')
        return set_error(MOE_ERR_UNSUPPORTED, "moe_dispatch_fused_static: %s; use the separate calls", why);
    const int64_t need = fused_workspace_bytes(dims->N, dims->T, dims->E);
    if (v.NT > 0 && need > fused_static_scratch_bytes())  // an empty batch uses no scratch
        return set_error(MOE_ERR_UNSUPPORTED,
                         "moe_dispatch_fused_static: N=%d T=%d E=%d needs %lld bytes of scratch; the library's "
                         "static array holds %lld", dims->N, dims->T, dims->E, (long long)need,
                         (long long)fused_static_scratch_bytes());
    void *scratch = nullptr;
    cudaError_t e = fused_static_scratch(&scratch);
    if (e != cudaSuccess) return cuda_result(e, "moe_dispatch_fused_static: scratch address");
    return moe_dispatch_fused(dims, logits, bias, score_fn, renormalize, x, x_scales, topk_idx, topk_w,
                              expert_counts, expert_offsets, rank_counts, rank_offsets, send_counts, pos,
                              status, packed_x, packed_scales, packed_src, scratch, stream);
}

int moe_expert_gemm(const MoeDims *dims, int K, int F, int act, const void *x, const void *w,
                    const int32_t *expert_offsets, void *y, void *pre, void *stream) {
    const char *what = "moe_expert_gemm";
    Derived v;
    ExpertRows r;
    int rc = check_expert(dims, K, F, act == MOE_EXPERT_SWIGLU, 2, expert_offsets, &v, &r, what);
    if (rc != MOE_OK) return rc;
    if (act != MOE_EXPERT_LINEAR && act != MOE_EXPERT_SWIGLU)
        return set_error(MOE_ERR_INVALID_ARG, "%s: unknown act %d", what, act);
    if (act == MOE_EXPERT_LINEAR && pre)
        return set_error(MOE_ERR_INVALID_ARG, "%s: pre is an output of MOE_EXPERT_SWIGLU only", what);
    if (v.NT == 0) return MOE_OK;
    if (bad_block_pointers(x, w, y, what, &rc) || (pre && bad_block_pointers(pre, pre, pre, what, &rc))) return rc;
    const int64_t wide = (act == MOE_EXPERT_SWIGLU ? 2 : 1) * (int64_t)F;
    const int64_t y_elem = act == MOE_EXPERT_LINEAR && dims->y_dtype == MOE_F32 ? 4 : 2;
    const Span out = {y, v.rows_total * F * y_elem}, kept = {pre, v.rows_total * wide * 2};
    const Span in[] = {{x, v.rows_total * K * 2}, {w, dims->E * wide * K * 2}, offsets_span(r)};
    const Span with_y[] = {in[0], in[1], in[2], out};
    if (overlap_any(out, in, what, &rc) || overlap_any(kept, with_y, what, &rc)) return rc;
    return cuda_result(launch_expert_gemm(r, K, F, act == MOE_EXPERT_SWIGLU, x, w, y, dims->y_dtype == MOE_F32, pre,
                                          (cudaStream_t)stream),
                       what);
}

int moe_expert_gemm_dgrad(const MoeDims *dims, int K, int F, const void *dy, const void *w,
                          const int32_t *expert_offsets, void *dx, void *stream) {
    const char *what = "moe_expert_gemm_dgrad";
    Derived v;
    ExpertRows r;
    int rc = check_expert(dims, K, F, false, 2, expert_offsets, &v, &r, what);
    if (rc != MOE_OK) return rc;
    if (v.NT == 0) return MOE_OK;
    if (bad_block_pointers(dy, w, dx, what, &rc)) return rc;
    const Span in[] = {{dy, v.rows_total * F * 2}, {w, (int64_t)dims->E * F * K * 2}, offsets_span(r)};
    if (overlap_any({dx, v.rows_total * K * 2}, in, what, &rc)) return rc;
    return cuda_result(launch_expert_dgrad(r, K, F, dy, w, dx, (cudaStream_t)stream), what);
}

int moe_expert_gemm_wgrad(const MoeDims *dims, int K, int F, const void *dy, const void *x,
                          const int32_t *expert_offsets, void *dw, int dw_dtype, void *stream) {
    const char *what = "moe_expert_gemm_wgrad";
    Derived v;
    ExpertRows r;
    int rc = check_expert(dims, K, F, false, 2, expert_offsets, &v, &r, what);
    if (rc != MOE_OK) return rc;
    if (dw_dtype != MOE_BF16 && dw_dtype != MOE_F32)
        return set_error(MOE_ERR_INVALID_ARG, "%s: dw_dtype must be MOE_BF16 or MOE_F32 (got %d)", what, dw_dtype);
    const Span out = {dw, (int64_t)dims->E * F * K * (dw_dtype == MOE_F32 ? 4 : 2)};
    if (v.NT == 0) {  // no rows anywhere: every sum is empty
        const Span in[] = {offsets_span(r)};
        if (bad_block_pointers(dw, dw, dw, what, &rc) || overlap_any(out, in, what, &rc)) return rc;
        return cuda_result(cudaMemsetAsync(dw, 0, (size_t)out.bytes, (cudaStream_t)stream), what);
    }
    if (bad_block_pointers(dy, x, dw, what, &rc)) return rc;
    const Span in[] = {{dy, v.rows_total * F * 2}, {x, v.rows_total * K * 2}, offsets_span(r)};
    if (overlap_any(out, in, what, &rc)) return rc;
    return cuda_result(launch_expert_wgrad(r, K, F, dy, x, dw, dw_dtype == MOE_F32, (cudaStream_t)stream), what);
}

int moe_expert_swiglu_grad(const MoeDims *dims, int F, const void *pre, const void *dh,
                           const int32_t *expert_offsets, void *dpre, void *stream) {
    const char *what = "moe_expert_swiglu_grad";
    Derived v;
    ExpertRows r;
    int rc = check_expert(dims, 8, F, false, 2, expert_offsets, &v, &r, what);
    if (rc != MOE_OK) return rc;
    if (v.NT == 0) return MOE_OK;
    if (bad_block_pointers(pre, dh, dpre, what, &rc)) return rc;
    const Span in[] = {{pre, v.rows_total * F * 4}, {dh, v.rows_total * F * 2}, offsets_span(r)};
    if (overlap_any({dpre, v.rows_total * F * 4}, in, what, &rc)) return rc;
    return cuda_result(launch_expert_swiglu_grad(r, dims->N, v.pairs, F, pre, dh, dpre, (cudaStream_t)stream), what);
}

int moe_expert_gemm_fp8(const MoeDims *dims, int K, int F, int act, const void *xq, const float *x_scales,
                        const void *wq, const float *w_scales, const int32_t *expert_offsets, void *y,
                        float *y_scales, void *stream) {
    const char *what = "moe_expert_gemm_fp8";
    Derived v;
    ExpertRows r;
    const bool gated = act == MOE_EXPERT_SWIGLU;
    int rc = check_expert(dims, K, F, gated, 1, expert_offsets, &v, &r, what);
    if (rc != MOE_OK) return rc;
    if (act != MOE_EXPERT_LINEAR && !gated) return set_error(MOE_ERR_INVALID_ARG, "%s: unknown act %d", what, act);
    if (K % 128 != 0 || (gated && F % 128 != 0))
        return set_error(MOE_ERR_INVALID_ARG, "%s: K=%d, and F=%d of the gated product, must be multiples of 128",
                         what, K, F);
    if (!gated && y_scales)
        return set_error(MOE_ERR_INVALID_ARG, "%s: y_scales is an output of MOE_EXPERT_SWIGLU only", what);
    if (v.NT == 0) return MOE_OK;
    if (bad_block_pointers(xq, wq, y, what, &rc)) return rc;
    if (!x_scales || !w_scales || (gated && !y_scales))
        return set_error(MOE_ERR_INVALID_ARG, "%s: a required pointer is NULL", what);
    if (!aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(y_scales, 4))
        return set_error(MOE_ERR_INVALID_ARG, "%s: scales must be 4-byte aligned", what);
    const int64_t wide = (gated ? 2 : 1) * (int64_t)F, blocks = K / 128;
    const Span out = {y, v.rows_total * F * (gated ? 1 : dims->y_dtype == MOE_F32 ? 4 : 2)};
    const Span in[] = {{xq, v.rows_total * K},
                       {x_scales, v.rows_total * blocks * 4},
                       {wq, dims->E * wide * K},
                       {w_scales, dims->E * ((wide + 127) / 128) * blocks * 4},
                       offsets_span(r)};
    const Span with_y[] = {in[0], in[1], in[2], in[3], in[4], out};
    if (overlap_any(out, in, what, &rc) || overlap_any({y_scales, v.rows_total * (F / 128) * 4}, with_y, what, &rc))
        return rc;
    return cuda_result(launch_expert_gemm_fp8(r, K, F, gated, xq, x_scales, wq, w_scales, y, dims->y_dtype == MOE_F32,
                                              y_scales, (cudaStream_t)stream),
                       what);
}

int moe_expert_gemm_w4(const MoeDims *dims, int K, int F, int act, int group, const void *x, const int32_t *wq,
                       const void *group_scales, const float *row_scales, const int32_t *expert_offsets, void *y,
                       void *stream) {
    const char *what = "moe_expert_gemm_w4";
    Derived v;
    ExpertRows r;
    const bool gated = act == MOE_EXPERT_SWIGLU;
    int rc = check_expert(dims, K, F, gated, 1, expert_offsets, &v, &r, what);
    if (rc != MOE_OK) return rc;
    if (act != MOE_EXPERT_LINEAR && !gated) return set_error(MOE_ERR_INVALID_ARG, "%s: unknown act %d", what, act);
    if (group != 32 && group != 64 && group != 128)
        return set_error(MOE_ERR_INVALID_ARG, "%s: group must be 32, 64 or 128 (got %d)", what, group);
    if (K % group != 0)
        return set_error(MOE_ERR_INVALID_ARG, "%s: K=%d must be a multiple of group=%d", what, K, group);
    if (v.NT == 0) return MOE_OK;
    if (bad_block_pointers(x, wq, y, what, &rc)) return rc;
    if (!group_scales || !row_scales) return set_error(MOE_ERR_INVALID_ARG, "%s: a required pointer is NULL", what);
    if (!aligned(group_scales, 8) || !aligned(row_scales, 4))  // groups' scales are copied by eight
        return set_error(MOE_ERR_INVALID_ARG, "%s: group_scales must be 8-byte, row_scales 4-byte aligned", what);
    const int64_t wide = (gated ? 2 : 1) * (int64_t)F;
    const Span out = {y, v.rows_total * F * (!gated && dims->y_dtype == MOE_F32 ? 4 : 2)};
    const Span in[] = {{x, v.rows_total * K * 2},
                       {wq, dims->E * wide * (K / 2)},
                       {group_scales, dims->E * wide * (K / group)},
                       {row_scales, dims->E * wide * 4},
                       offsets_span(r)};
    if (overlap_any(out, in, what, &rc)) return rc;
    return cuda_result(launch_expert_gemm_w4(r, K, F, gated, group, x, wq, group_scales, row_scales, y,
                                             dims->y_dtype == MOE_F32, (cudaStream_t)stream),
                       what);
}

int moe_combine_grad(const MoeDims *dims, const void *dout, const void *y, const int32_t *pos, const float *topk_w,
                     void *dy, float *dtopk_w, void *stream) {
    const char *what = "moe_combine_grad";
    Derived v;
    int rc = check_dims(dims, &v, what);
    if (rc != MOE_OK) return rc;
    if (v.NT == 0) return MOE_OK;
    if (!dout || !y || !pos || !topk_w || !dy || !dtopk_w)
        return set_error(MOE_ERR_INVALID_ARG, "%s: a required pointer is NULL", what);
    if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16))
        return set_error(MOE_ERR_INVALID_ARG, "%s: dout, y and dy must be 16-byte aligned", what);
    if (!aligned(pos, 4) || !aligned(topk_w, 4) || !aligned(dtopk_w, 4))
        return set_error(MOE_ERR_INVALID_ARG, "%s: pos, topk_w and dtopk_w must be 4-byte aligned", what);
    const Span rows = {dy, v.rows_total * v.y_row_bytes}, weights = {dtopk_w, v.pairs * 4};
    const Span in[] = {{dout, v.NT * v.y_row_bytes}, {y, rows.bytes}, {pos, v.pairs * 4}, {topk_w, v.pairs * 4}};
    const Span with_rows[] = {in[0], in[1], in[2], in[3], rows};
    if (overlap_any(rows, in, what, &rc) || overlap_any(weights, with_rows, what, &rc)) return rc;
    return cuda_result(launch_combine_grad(dout, y, dims->y_dtype, pos, topk_w, v.NT, dims->R, dims->H, v.rows_total, dy,
                                           dtopk_w, (cudaStream_t)stream),
                       what);
}

int moe_dispatch_grad(const MoeDims *dims, const void *dpacked, const int32_t *pos, const void *add, void *dx,
                      void *stream) {
    const char *what = "moe_dispatch_grad";
    Derived v;
    int rc = check_dims(dims, &v, what);
    if (rc != MOE_OK) return rc;
    if (dims->x_dtype != MOE_BF16 && dims->x_dtype != MOE_F32)
        return set_error(MOE_ERR_INVALID_ARG, "%s: x_dtype must be MOE_BF16 or MOE_F32 (got %d)", what, dims->x_dtype);
    if (v.NT == 0) return MOE_OK;
    if (!dpacked || !pos || !dx) return set_error(MOE_ERR_INVALID_ARG, "%s: a required pointer is NULL", what);
    if (!aligned(dpacked, 16) || !aligned(add, 16) || !aligned(dx, 16))
        return set_error(MOE_ERR_INVALID_ARG, "%s: dpacked, add and dx must be 16-byte aligned", what);
    if (!aligned(pos, 4)) return set_error(MOE_ERR_INVALID_ARG, "%s: pos must be 4-byte aligned", what);
    const Span out = {dx, v.NT * v.x_row_bytes};
    const Span in[] = {{dpacked, v.rows_total * v.x_row_bytes}, {pos, v.pairs * 4}, {add == dx ? nullptr : add, out.bytes}};
    if (overlap_any(out, in, what, &rc)) return rc;
    return cuda_result(launch_dispatch_grad(dpacked, dims->x_dtype, pos, add, v.NT, dims->R, dims->H, v.rows_total, dx,
                                            (cudaStream_t)stream),
                       what);
}

int moe_route_grad(const MoeDims *dims, const float *logits, const float *bias, int score_fn, int renormalize,
                   const int32_t *topk_idx, const float *topk_w, const float *dtopk_w, float *dlogits, float *dbias,
                   void *stream) {
    const char *what = "moe_route_grad";
    Derived v;
    int rc = check_dims(dims, &v, what);
    if (rc != MOE_OK) return rc;
    if (!valid_score_fn(score_fn)) return set_error(MOE_ERR_INVALID_ARG, "%s: unknown score_fn %d", what, score_fn);
    if ((score_fn & MOE_BIAS_SELECT_ONLY) && dbias)
        return set_error(MOE_ERR_INVALID_ARG, "%s: a bias for the selection alone has no gradient: dbias must be NULL", what);
    if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4) ||
        !aligned(dtopk_w, 4) || !aligned(dlogits, 4) || !aligned(dbias, 4))
        return set_error(MOE_ERR_INVALID_ARG, "%s: pointers must be 4-byte aligned", what);
    if (v.NT == 0)  // no tokens: an empty sum
        return dbias ? cuda_result(cudaMemsetAsync(dbias, 0, (size_t)dims->E * 4, (cudaStream_t)stream), what) : MOE_OK;
    if (!logits || !topk_idx || !topk_w || !dtopk_w || !dlogits)
        return set_error(MOE_ERR_INVALID_ARG, "%s: a required pointer is NULL", what);
    const int64_t all = v.NT * dims->E * 4;
    const Span out = {dlogits, all}, sums = {dbias, (int64_t)dims->E * 4};
    const Span in[] = {{logits, all}, {bias, sums.bytes}, {topk_idx, v.pairs * 4}, {topk_w, v.pairs * 4}, {dtopk_w, v.pairs * 4}};
    const Span with_out[] = {in[0], in[1], in[2], in[3], in[4], out};
    if (overlap_any(out, in, what, &rc) || overlap_any(sums, with_out, what, &rc)) return rc;
    return cuda_result(launch_route_grad(logits, bias, v.NT, dims->E, dims->R, score_fn, renormalize ? 1 : 0, topk_idx,
                                         topk_w, dtopk_w, dlogits, dbias, (cudaStream_t)stream),
                       what);
}

int moe_selftest_bounded_wait(int32_t *status, int64_t polls, void *stream) {
    g_err[0] = '\0';
    if (!status || !aligned(status, 4))
        return set_error(MOE_ERR_INVALID_ARG, "moe_selftest_bounded_wait: status must be a 4-byte aligned pointer");
    if (polls < 1 || polls > ((int64_t)1 << 20))
        return set_error(MOE_ERR_INVALID_ARG, "moe_selftest_bounded_wait: polls %lld outside [1, 2^20]",
                         (long long)polls);
    return cuda_result(launch_selftest_wait(status, (long long)polls, (cudaStream_t)stream),
                       "moe_selftest_bounded_wait");
}

int moe_take_device_error(void *stream) {
    g_err[0] = '\0';
    int err = 0;
    cudaError_t e = take_device_error(&err, (cudaStream_t)stream);
    cudaError_t (*const more[])(int *) = {take_expert_gemm_error, take_expert_wgrad_error, take_expert_fp8_error,
                                        take_expert_w4_error, take_expert_w4_few_error};
    for (auto take : more) {  // the stream has been waited for
        int one = 0;
        if (e == cudaSuccess) e = take(&one);
        if (err == 0) err = one;
    }
    if (e != cudaSuccess) return cuda_result(e, "moe_take_device_error");
    return err;
}

int moe_read_status(const int32_t *status, void *stream) {
    g_err[0] = '\0';
    if (!status) return set_error(MOE_ERR_INVALID_ARG, "moe_read_status: status is NULL");
    cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_result(e, "moe_read_status");
    int32_t host = 0;
    e = cudaMemcpy(&host, status, sizeof(host), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_result(e, "moe_read_status");
    return host;
}

}  // extern "C"
