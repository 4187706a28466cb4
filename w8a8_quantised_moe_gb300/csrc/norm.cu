// norm.cu -- the norms around a block, with its gate and residual scale:
//
//   b  = branch * rsqrt(mean(branch^2) + eps) * post_w   (post_w given, else b = branch)
//   r  = x + scale * gate * b                            (branch given, else r = x)
//   n  = r * rsqrt(mean(r^2) + eps) * pre_w              (pre_w given)
//
// with r and n each rounded once, from binary32; n is formed from the
// unrounded r.  One pass: a row's x and branch are read once into registers,
// both sums are taken from there, r and n are written.  Bound by HBM for many
// rows (x, branch in, r, n out), by one row's latency for one token.
//
// G warps hold a row, two 8-channel vectors a lane (H <= 512 G), so a CTA of 8
// warps takes 8 / G rows, and a CTA of G warps one row above 8.
#include "block.h"
#include "block_dev.cuh"

namespace moe {
namespace {

constexpr int kNormVec = 2;  // 8-channel vectors per lane

// Sum over the G warps of this warp's row (two words of shared memory a
// warp: `which` separates the two sums of a row, so one barrier each is
// enough).  Every warp of the CTA calls it.
__device__ __forceinline__ float row_sum(float v, int G, float* red, int which) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (G == 1) return v;
    if (lane == 0) red[which * 32 + warp] = v;
    __syncthreads();
    const float* r = red + which * 32 + warp / G * G;
    v = r[0];
    for (int i = 1; i < G; ++i) v += r[i];
    return v;
}

template <bool F32, GateForm GATE>
__global__ void __launch_bounds__(1024) norm_residual_kernel(const NormArgs a, int G) {
    __shared__ float red[64];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rows_cta = (int)(blockDim.x >> 5) / G;
    const int64_t t = (int64_t)blockIdx.x * rows_cta + warp / G;
    const bool live = t < a.T;
    const int H = a.H, nv = H / 8;
    const size_t row = live ? (size_t)t * H : 0;
    const int v0 = (warp % G) * 32 + lane;  // this lane's vectors: v0, v0 + 32 G
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

    float r[kNormVec][8];
    uint4 bv[kNormVec];
#pragma unroll
    for (int i = 0; i < kNormVec; ++i) {
        const int v = v0 + i * 32 * G;
        const bool in = live && v < nv;
        if (F32) {
            const float4* x = reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + row) + 2 * v;
            const float4 lo = in ? x[0] : make_float4(0.f, 0.f, 0.f, 0.f), hi = in ? x[1] : lo;
            r[i][0] = lo.x, r[i][1] = lo.y, r[i][2] = lo.z, r[i][3] = lo.w;
            r[i][4] = hi.x, r[i][5] = hi.y, r[i][6] = hi.z, r[i][7] = hi.w;
        } else {
            bf16x8_to_f32(in ? reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + row)[v] : zero, r[i]);
        }
        bv[i] = (in && a.branch) ? reinterpret_cast<const uint4*>(a.branch + row)[v] : zero;
    }
    if (a.branch) {
        float mul = a.scale;
        if (GATE == GateForm::Token) mul *= live ? __uint_as_float((uint32_t)a.gate[t] << 16) : 0.f;
        if (a.post_w) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < kNormVec; ++i) {
                float b[8];
                bf16x8_to_f32(bv[i], b);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(b[j], b[j], ss);
            }
            ss = row_sum(ss, G, red, 0);
            mul *= rsqrtf(ss / (float)H + a.eps);
        }
#pragma unroll
        for (int i = 0; i < kNormVec; ++i) {
            const int v = v0 + i * 32 * G;
            if (!live || v >= nv) continue;
            float b[8];
            bf16x8_to_f32(bv[i], b);
            if (a.post_w) {
                float w[8];
                bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(a.post_w) + v), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) b[j] *= w[j];
            }
            if (GATE == GateForm::Channel || GATE == GateForm::Element) {
                float w[8];
                bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(a.gate + (GATE == GateForm::Element ? row : 0)) + v), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) b[j] *= w[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] = fmaf(mul, b[j], r[i][j]);
            if (F32) {
                float4* out = reinterpret_cast<float4*>(static_cast<float*>(a.x_out) + row) + 2 * v;
                out[0] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
                out[1] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
            } else {
                reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.x_out) + row)[v] =
                    make_uint4(bf16_pair(r[i][0], r[i][1]), bf16_pair(r[i][2], r[i][3]), bf16_pair(r[i][4], r[i][5]),
                               bf16_pair(r[i][6], r[i][7]));
            }
        }
    }
    if (a.pre_w) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < kNormVec; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(r[i][j], r[i][j], ss);
        ss = row_sum(ss, G, red, 1);
        const float inv = rsqrtf(ss / (float)H + a.eps);
#pragma unroll
        for (int i = 0; i < kNormVec; ++i) {
            const int v = v0 + i * 32 * G;
            if (!live || v >= nv) continue;
            float w[8];
            bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(a.pre_w) + v), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] *= r[i][j] * inv;
            reinterpret_cast<uint4*>(a.n_out + row)[v] =
                make_uint4(bf16_pair(w[0], w[1]), bf16_pair(w[2], w[3]), bf16_pair(w[4], w[5]), bf16_pair(w[6], w[7]));
        }
    }
}

template <bool F32>
cudaError_t launch_norm(const NormArgs& a, GateForm gate, cudaStream_t st) {
    int G = 1;
    while (a.H > 512 * G) G *= 2;
    const int warps = G < 8 ? 8 : G, rows = warps / G;
    const dim3 grid((unsigned)((a.T + rows - 1) / rows)), block(32 * warps);
    switch (gate) {
        case GateForm::None: return launch_kernel(norm_residual_kernel<F32, GateForm::None>, grid, block, 0, st, false, a, G);
        case GateForm::Channel: return launch_kernel(norm_residual_kernel<F32, GateForm::Channel>, grid, block, 0, st, false, a, G);
        case GateForm::Token: return launch_kernel(norm_residual_kernel<F32, GateForm::Token>, grid, block, 0, st, false, a, G);
        case GateForm::Element: return launch_kernel(norm_residual_kernel<F32, GateForm::Element>, grid, block, 0, st, false, a, G);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_norm_residual(const NormArgs& a, bool fp32_residual, GateForm gate, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    return fp32_residual ? launch_norm<true>(a, gate, st) : launch_norm<false>(a, gate, st);
}

}  // namespace moe
