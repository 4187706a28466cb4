// block_dev.cuh -- device helpers of the block-scaled FP8 operators.
#pragma once

#include <cstdint>

#include "block.h"

namespace moe {
namespace {

// A block's scale: its largest magnitude over 448, the largest E4M3 magnitude,
// as one product with the binary32 reciprocal.  (For a normal scale the quotient
// of the largest magnitude by it is 448 to within an ulp or two, and its code 448;
// a subnormal one is coarser, and codes saturate or stay below.)
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

// e4m3_quot4 of N values, mostly without divisions.  A product with the
// rounded reciprocal of s is within 2^-22 of the rounded quotient, relatively,
// so the quotient lies between the products with the reciprocal 2^-22 lower
// and higher; where both round to the same codes, those are the quotients'.
// Elsewhere (a quotient next to a midpoint of two codes) and for scales whose
// reciprocal could overflow, be 0 or NaN, the divisions decide.  Worth it where a
// thread has a row's 64 codes to form and nothing else to wait for, at the end of
// the gate/up product: layer of 8192 tokens 522 us, 539 with divisions.  Where the
// row's loads leave the time, divisions are not slower: quant8 in the linear layer,
// 1 x 4096 x 4096 8.2 us with these products and 7.7 with divisions, 64 x 4096 x
// 4096 10.5 and 10.3, 4096 x 16 x 8192 50.5 and 49.3.
struct BlockQuot {
    float s, lo, hi;
    bool in_range;
    __device__ __forceinline__ explicit BlockQuot(float scale) : s(scale) {
        const float inv = __frcp_rn(s);
        lo = inv * (1.0f - 0x1p-22f);
        hi = inv * (1.0f + 0x1p-22f);
        in_range = s >= 0x1p-100f && s <= 0x1p100f;
    }
    template <int N>
    __device__ __forceinline__ void codes(const float (&f)[N], uint32_t (&c)[N / 4]) const {
        bool sure = in_range;
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float* v = f + 4 * i;
            c[i] = e4m3_pair(v[0] * lo, v[1] * lo) | (e4m3_pair(v[2] * lo, v[3] * lo) << 16);
            sure = sure && c[i] == (e4m3_pair(v[0] * hi, v[1] * hi) | (e4m3_pair(v[2] * hi, v[3] * hi) << 16));
        }
        if (sure) return;
#pragma unroll
        for (int i = 0; i < N / 4; ++i) c[i] = e4m3_quot4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3], s);
    }
};

// Codes of 8 values a lane, 16 lanes a block; s receives the block's scale.
// Every lane of the warp calls it.
__device__ __forceinline__ uint2 quant8(const float (&f)[8], float& s) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = amax_nan(amax, f[i]);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) amax = amax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    s = block_scale(amax);
    return make_uint2(e4m3_quot4(f[0], f[1], f[2], f[3], s), e4m3_quot4(f[4], f[5], f[6], f[7], s));
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

// h = g / (1 + exp(-g)) * u within 6 * 2^-23, by exp(-|g|), which does not pass
// binary32's range (where it is subnormal, |g| above 87.3, half of 2^-149 in it
// adds to that): expf to 2 ulp over its whole range, the fast quotient by 1 to 2
// to 2 ulp.  The fast exponential's error grows with its argument (2 + 1.17 |g|
// ulp) and so moved codes of h for far negative gates, and the fast quotient by
// 1 + exp(-g) gave 0 for gates below -87.3.  Layer of 8192 tokens: 546 us with both,
// 547 with expf, the same in this form; 636 with a rounded quotient besides (the other
// layers' form).
__device__ __forceinline__ float silu_mul(float g, float u) {
    const float t = expf(-fabsf(g));
    return __fdividef(g < 0.f ? __fmul_rn(g, t) : g, 1.0f + t) * u;
}

// Two binary32 values in one 64-bit register, and the packed multiply-add on
// them (two rounded FMAs).
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

// One tcgen05 MMA, kind::f8f6f4, both operands from shared memory: D[M x N]
// (+)= A[M x 32] * B[N x 32]^T, E4M3 (operand format 0) into fp32.
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

}  // namespace
}  // namespace moe
