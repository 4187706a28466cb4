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
// G warps hold a row, one or two 8-channel vectors a lane; a CTA is one row of up
// to 32 warps, or 8 / G rows of G <= 4.  Rows are not kept waiting in registers
// for more rows: a persistent loop that loads its next row ahead spilled and
// took 98 us at 8192 x 4096 (46 as it is: 5.9 TB/s, 0.86 of the copy's rate).
#include "block.h"
#include "block_dev.cuh"

namespace moe {
namespace {

// Sum over the G warps of this warp's row.  Every warp of the CTA calls it;
// red: 32 words that no call within the last barrier used.
__device__ __forceinline__ float row_sum(float v, int G, float* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (G == 1) return v;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    // the G sums, added in the same tree by every lane
    v = lane < G ? red[warp / G * G + lane] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ void mul_bf16x8(float (&f)[8], const uint4& w) {
    float v[8];
    bf16x8_to_f32(w, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= v[j];
}

// V vectors a lane; MAXW: the CTA's warps.  Registers are held to what 1536
// threads an SM leave (two vectors) or 2048 (one).
template <bool F32, GateForm GATE, int V, int MAXW>
__global__ void __launch_bounds__(32 * MAXW, (V == 1 ? 64 : 48) / MAXW) norm_residual_kernel(const NormArgs a, int G) {
    __shared__ float red[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int H = a.H, step = 32 * G;
    const int v0 = (warp % G) * 32 + lane;  // this lane's vectors: v0, v0 + step
    const int64_t t = (int64_t)blockIdx.x * ((blockDim.x >> 5) / G) + warp / G;
    const bool live = t < a.T;
    const size_t row = live ? (size_t)t * H : 0;
    const float inv_h = 1.0f / (float)H;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    pdl_wait();
    pdl_trigger();

    float r[V][8];
    uint4 bv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = v0 + i * step;
        const bool in = live && v * 8 < H;
        if (F32) {
            const float4* x = reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + row) + 2 * v;
            const float4 none = make_float4(0.f, 0.f, 0.f, 0.f), lo = in ? x[0] : none, hi = in ? x[1] : none;
            r[i][0] = lo.x, r[i][1] = lo.y, r[i][2] = lo.z, r[i][3] = lo.w;
            r[i][4] = hi.x, r[i][5] = hi.y, r[i][6] = hi.z, r[i][7] = hi.w;
        } else {
            bf16x8_to_f32(in ? reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + row)[v] : zero, r[i]);
        }
        bv[i] = in && a.branch ? reinterpret_cast<const uint4*>(a.branch + row)[v] : zero;
    }
    if (a.branch) {
        float mul = a.scale;
        if (GATE == GateForm::Token && live) mul *= __uint_as_float((uint32_t)a.gate[t] << 16);
        if (a.post_w) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float b[8];
                bf16x8_to_f32(bv[i], b);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(b[j], b[j], ss);
            }
            ss = row_sum(ss, G, red[0]);
            mul *= rsqrtf(fmaf(ss, inv_h, a.eps));
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = v0 + i * step;
            if (!live || v * 8 >= H) continue;
            float b[8];
            bf16x8_to_f32(bv[i], b);
            if (a.post_w) mul_bf16x8(b, __ldg(reinterpret_cast<const uint4*>(a.post_w) + v));
            if (GATE == GateForm::Channel) mul_bf16x8(b, __ldg(reinterpret_cast<const uint4*>(a.gate) + v));
            if (GATE == GateForm::Element) mul_bf16x8(b, reinterpret_cast<const uint4*>(a.gate + row)[v]);
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
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(r[i][j], r[i][j], ss);
        ss = row_sum(ss, G, red[1]);
        const float inv = rsqrtf(fmaf(ss, inv_h, a.eps));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = v0 + i * step;
            if (!live || v * 8 >= H) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] *= inv;
            mul_bf16x8(r[i], __ldg(reinterpret_cast<const uint4*>(a.pre_w) + v));
            reinterpret_cast<uint4*>(a.n_out + row)[v] =
                make_uint4(bf16_pair(r[i][0], r[i][1]), bf16_pair(r[i][2], r[i][3]), bf16_pair(r[i][4], r[i][5]),
                           bf16_pair(r[i][6], r[i][7]));
        }
    }
}

template <bool F32, GateForm GATE>
cudaError_t launch_norm_form(const NormArgs& a, cudaStream_t st) {
    // One vector a lane where the whole call then fits the GPU at once (64 warps an
    // SM), two elsewhere (half the threads, each with twice the bytes in flight).
    // Measured, one vector / two: 1 x 4096 2.2 / 2.5 us, 1003 x 2056 fp32 6.5 / 6.8,
    // 8192 x 4096 51 / 46, 4096 x 7168 51 / 40.
    const int vecs = a.H / 8, warps1 = (vecs + 31) / 32;
    const int V = warps1 <= 32 && a.T * warps1 <= 64 * (int64_t)num_sms() ? 1 : 2;
    int G = (vecs + 32 * V - 1) / (32 * V);
    if (G == 3) G = 4;  // up to 4 warps a row: 8 / G rows a CTA
    const int rows = G <= 4 ? 8 / G : 1, warps = rows * G;
    const dim3 grid((unsigned)((a.T + rows - 1) / rows)), block(32 * warps);
    const bool pdl = pdl_default();
    if (V == 2) {
        if (warps <= 8) return launch_kernel(norm_residual_kernel<F32, GATE, 2, 8>, grid, block, 0, st, pdl, a, G);
        if (warps <= 16) return launch_kernel(norm_residual_kernel<F32, GATE, 2, 16>, grid, block, 0, st, pdl, a, G);
        return launch_kernel(norm_residual_kernel<F32, GATE, 2, 32>, grid, block, 0, st, pdl, a, G);
    }
    if (warps <= 8) return launch_kernel(norm_residual_kernel<F32, GATE, 1, 8>, grid, block, 0, st, pdl, a, G);
    if (warps <= 16) return launch_kernel(norm_residual_kernel<F32, GATE, 1, 16>, grid, block, 0, st, pdl, a, G);
    return launch_kernel(norm_residual_kernel<F32, GATE, 1, 32>, grid, block, 0, st, pdl, a, G);
}

template <bool F32>
cudaError_t launch_norm(const NormArgs& a, GateForm gate, cudaStream_t st) {
    switch (gate) {
        case GateForm::None: return launch_norm_form<F32, GateForm::None>(a, st);
        case GateForm::Channel: return launch_norm_form<F32, GateForm::Channel>(a, st);
        case GateForm::Token: return launch_norm_form<F32, GateForm::Token>(a, st);
        case GateForm::Element: return launch_norm_form<F32, GateForm::Element>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_norm_residual(const NormArgs& a, bool fp32_residual, GateForm gate, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    return fp32_residual ? launch_norm<true>(a, gate, st) : launch_norm<false>(a, gate, st);
}

}  // namespace moe
