// block_dev.cuh -- device helpers of the block-scaled FP8 operators.
#pragma once

#include <cstdint>

#include "block.h"

namespace moe {
namespace {

// A block's scale: its largest magnitude over 448, the largest E4M3 magnitude,
// as one product with the binary32 reciprocal.  (The quotient of the largest
// magnitude by its scale is 448 to within an ulp or two, so its code is 448.)
__device__ __forceinline__ float block_scale(float amax) { return __fmul_rn(amax, 1.0f / 448.0f); }

// Two E4M3 codes (lo in the low byte): round to nearest even, saturate.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// max(m, |v|) that keeps a NaN: a block with a NaN gets a NaN scale, and the
// product's rows that use it are NaN, as in a product of unquantised values.
__device__ __forceinline__ float amax_nan(float m, float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
    return r;
}

// Codes of four values over the scale s of their block (s == 0: zeros).
__device__ __forceinline__ uint32_t e4m3_quot4(float a, float b, float c, float d, float s) {
    if (s == 0.f) return 0u;
    return e4m3_pair(__fdiv_rn(a, s), __fdiv_rn(b, s)) | (e4m3_pair(__fdiv_rn(c, s), __fdiv_rn(d, s)) << 16);
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Two bf16 (lo in the low half) of two binary32 values, each rounded to nearest even.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// h = g / (1 + exp(-g)) * u.  The exponential and the quotient are the fast
// forms (about 2 ulp each): h is rounded to a 4-bit significand next, and a
// code that such an error moves lies as close to its neighbour as to h.
__device__ __forceinline__ float silu_mul(float g, float u) {
    return __fdividef(g, 1.0f + __expf(-g)) * u;
}

// Two binary32 values in one 64-bit register, and the packed multiply-add on
// them (two rounded FMAs in one instruction: twice the rate of fma.rn.f32).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ void fma2(f32x2& acc, f32x2 a, f32x2 b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}

}  // namespace
}  // namespace moe
