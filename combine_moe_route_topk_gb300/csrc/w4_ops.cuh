// 4-bit codes to bf16, shared by the kernels of the experts' product with
// 4-bit weights.
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

namespace moe {

// A group's scale, twice, and what takes the codes' offset off.
struct W4Scale {
    __nv_bfloat162 s, minus;
    __device__ __forceinline__ explicit W4Scale(uint32_t code) {  // e4m3; exact in bf16
        const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3);
        const float f = __half2float(__half(h));
        s = __floats2bfloat162_rn(f, f);
        minus = __hmul2(s, __floats2bfloat162_rn(-136.f, -136.f));
    }
};

// The eight elements of a word, two a register, in their order.
__device__ __forceinline__ void dequant8(uint32_t word, const W4Scale &w, uint32_t *out) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t bits = ((word >> (4 * j)) & 0x000f000fu) ^ 0x43084308u;
        const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&bits), w.s, w.minus);
        out[j] = *reinterpret_cast<const uint32_t *>(&v);
    }
}

}  // namespace moe
