// 4-bit codes to bf16, and what the kernels of the experts' product with
// 4-bit weights share besides.
//
// A nibble of two's complement with its top bit flipped is q + 8; put under the
// exponent of 128 it is the bf16 number 128 + (q + 8); and (128 + q + 8) s - 136 s
// in one multiply-add is q s exactly: q has at most four bits and the e4m3 scale
// s four, so q s fits bf16's eight, and so does 136 s = 17 * 8 s.  The elements of
// a word lie so that a shift and one logic operation give two of them in the
// halves of a register: 11 instructions for eight weights.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "tc_ops.cuh"

namespace moe {

// A group's scale, twice, and what takes the codes' offset off.
struct W4Scale {
    __nv_bfloat162 s, minus;
    __device__ __forceinline__ void set(float f) {
        s = __floats2bfloat162_rn(f, f);
        minus = __hmul2(s, __floats2bfloat162_rn(-136.f, -136.f));
    }
};
// Of two e4m3 codes, which are exact in bf16.  (One by one they took seven
// instructions each, a twelfth of all: 32 of 64 experts, 7168 x 4096 each, one token 103.6 us
// against 100.7.)
struct W4Scales {
    W4Scale first, second;
    __device__ __forceinline__ explicit W4Scales(uint32_t codes) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        first.set(f.x);
        second.set(f.y);
    }
};

// The constant of dequant8, from a register: as a literal next to the mask, which is
// one too, it cost an instruction for every pair.
__device__ __forceinline__ uint32_t w4_magic() {
    uint32_t r;
    asm volatile("mov.b32 %0, 0x43084308;" : "=r"(r));
    return r;
}

// The eight elements of a word, two a register, in their order.
__device__ __forceinline__ void dequant8(uint32_t word, const W4Scale &w, uint32_t magic, uint32_t *out) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t bits;  // (word >> 4 j) & 0x000f000f ^ magic
        asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(bits) : "r"(word >> (4 * j)), "r"(0x000f000fu), "r"(magic));
        const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&bits), w.s, w.minus);
        out[j] = *reinterpret_cast<const uint32_t *>(&v);
    }
}

// Which lane of a warp tells a barrier that the warp has read what it loaded from
// shared memory: lane 0, or 31 where every lane's `loaded` (a word of each of its
// loads, combined) is one certain number.  An arrival right behind the loads
// does not wait for them: in 8192 rows of 64 experts thousands of results were
// wrong, made of the next stage's bytes.  This one cannot be issued before the
// vote, nor the vote before every lane has its words; and as a vote orders no
// memory, __syncwarp puts every lane's loads before the arrival, which releases.
// (Behind the vote it cost more: one token of 8 of 64 experts 32.9 us, 32.4 so
// and without it; 32 tokens of 64 experts 203, 202 and 201.)
__device__ __forceinline__ int reader_lane(uint32_t loaded) {
    __syncwarp();
    return __all_sync(0xffffffffu, loaded == 0x9e3779b9u) ? 31 : 0;
}

// `kBytes` from global to shared memory without a register; `bytes` of them are read, the others are zeros.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(bytes) : "memory");
}
// Arrives on `bar` (whose count includes it) once this thread's copies so far are done.
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ uint32_t ld_shared8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_shared32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, int rank) {  // the same place in another block of the cluster
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// The two halves of cluster_sync.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// Stores into another block of the cluster (addr and bar from at_rank, of one block) and counts the 16 bytes at `bar`
// when they are there: nothing to wait for here.  (Plain stores, a fence and an arrival took the one that
// gives 2000 cycles, the one that gets some 3000 more.)
__device__ __forceinline__ void st_async128(uint32_t addr, const float4 &v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1, int c2,
                                            int c3, int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], "
        "[%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}

// The map of matrices of 4-bit codes, boxes of 256 elements (a line of 128 bytes)
// by `rows` rows; of a gated product's, blocks of 8 gate rows and the up rows of
// the same 8 features follow one another.
inline bool encode_w4(CUtensorMap *m, const void *wq, int E, int K, int F, int gated, int rows) {
    const uint64_t line = (uint64_t)K / 2, f = (uint64_t)F, e = (uint64_t)E;
    if (gated) {
        const uint64_t dims[5] = {line, 8, 2, f / 8, e}, strides[4] = {line, line * f, line * 8, line * f * 2};
        const uint32_t box[5] = {128, 8, 2, (uint32_t)rows / 16, 1};
        return encode_map(m, 1, 5, wq, dims, strides, box);
    }
    const uint64_t dims[3] = {line, f, e}, strides[2] = {line, line * f};
    const uint32_t box[3] = {128, (uint32_t)rows, 1};
    return encode_map(m, 1, 3, wq, dims, strides, box);
}

}  // namespace moe
