// block.cu -- quantisers of the block-scaled FP8 operators.
//
// A block's scale is s = amax * (1/448) (one binary32 product with the rounded
// reciprocal) and its codes are the E4M3 values nearest to the binary32
// quotients x / s, ties to the even mantissa, saturated at +-448; a block of
// zeros has s = 0 and codes 0.
// Activations: a block is 128 channels of one row, so a row needs no
// reduction across its blocks.  Weights: a block is 128 x 128.

#include "block.h"
#include "block_dev.cuh"

namespace moe {
namespace {

// One CTA of 256 threads per 128 x 128 weight block, held in registers (16
// float4 a thread): one read of the fp32 weights, one write of the codes.
__global__ void __launch_bounds__(256) quantize_weights_block_kernel(const float* __restrict__ w, int64_t n_blocks,
                                                                     int rows, int K, uint8_t* __restrict__ q,
                                                                     float* __restrict__ s_out) {
    __shared__ float red[8];
    const int nb = blocks_of(rows), kb = blocks_of(K);
    const int c4 = threadIdx.x & 31, r0 = threadIdx.x >> 5;  // this thread's float4 column and first row
    for (int64_t b = blockIdx.x; b < n_blocks; b += gridDim.x) {
        const int64_t g = b / ((int64_t)nb * kb);
        const int rb = (int)(b / kb % nb), cb = (int)(b % kb);
        const int col = cb * kBlk + c4 * 4;
        const size_t base = ((size_t)g * rows + (size_t)rb * kBlk) * K + col;
        float4 v[16];
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = r0 + 8 * i;
            v[i] = (rb * kBlk + r < rows && col < K) ? __ldcs(reinterpret_cast<const float4*>(w + base + (size_t)r * K))
                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
            amax = amax_nan(amax_nan(amax_nan(amax_nan(amax, v[i].x), v[i].y), v[i].z), v[i].w);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) amax = amax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        __syncthreads();  // red of the previous block has been read
        if (c4 == 0) red[r0] = amax;
        __syncthreads();
        amax = red[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) amax = amax_nan(amax, red[i]);
        const float s = block_scale(amax);
        if (threadIdx.x == 0) s_out[b] = s;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = r0 + 8 * i;
            if (rb * kBlk + r < rows && col < K)
                *reinterpret_cast<uint32_t*>(q + base + (size_t)r * K) =
                    e4m3_quot4(v[i].x, v[i].y, v[i].z, v[i].w, s);
        }
    }
}

// A warp per (row, 256 V channels): V vectors of 8 channels a lane, all in
// flight; lanes 0-15 and 16-31 hold a block of a vector each.  SLOTS: the row
// is a token whose codes go to its k slots.
template <bool SLOTS, int V>
__global__ void __launch_bounds__(256) quantize_rows_block_kernel(
    const uint16_t* __restrict__ x, int M, int K, uint8_t* __restrict__ q, float* __restrict__ s_out,
    const int32_t* __restrict__ topk_ids, const int32_t* __restrict__ rank, const int32_t* __restrict__ base, int E,
    int k, int32_t* __restrict__ slot_of, int* __restrict__ error) {
    const int lane = threadIdx.x & 31;
    const int kb = blocks_of(K), parts = (kb + 2 * V - 1) / (2 * V);
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int r = (int)(item / parts), part = (int)(item - (int64_t)r * parts);
    const int col = part * 256 * V + lane * 8;
    pdl_wait();
    pdl_trigger();
    if (r >= M) return;
    uint4 v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = col + i * 256;
        v[i] = c < K ? *reinterpret_cast<const uint4*>(x + (size_t)r * K + c) : make_uint4(0u, 0u, 0u, 0u);
    }
    int my_slot = r;
    if (SLOTS && lane < k) {
        const int e = topk_ids[(size_t)r * k + lane];
        my_slot = in_range(e, 0, E, error) ? base[(size_t)(r / kRouterTokens) * E + e] + rank[(size_t)r * k + lane]
                                           : -1;  // -1: out of range (checked build), its writes skipped
        if (my_slot >= 0 && !in_range(my_slot, 0, (long long)M * k, error)) my_slot = -1;
        if (part == 0) slot_of[(size_t)r * k + lane] = my_slot;
    }
    const int n = SLOTS ? k : 1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = col + i * 256;
        float f[8], s;
        bf16x8_to_f32(v[i], f);
        const uint2 code = quant8(f, s);
        for (int j = 0; j < n; ++j) {
            const int row = SLOTS ? __shfl_sync(0xffffffffu, my_slot, j) : r;
            if (c < K && (!kChecked || row >= 0)) {
                *reinterpret_cast<uint2*>(q + (size_t)row * K + c) = code;
                if ((lane & 15) == 0) s_out[(size_t)row * kb + c / kBlk] = s;
            }
        }
    }
}

// Four vectors a lane where that still leaves work for every SM, else one.
template <bool SLOTS, typename... Args>
cudaError_t launch_quantize_rows(cudaStream_t st, bool pdl, const uint16_t* x, int M, int K, Args... args) {
    const int v4 = (blocks_of(K) + 7) / 8, v1 = (blocks_of(K) + 1) / 2;
    const bool wide = (int64_t)M * v4 >= 32LL * num_sms();
    const int64_t items = (int64_t)M * (wide ? v4 : v1);
    const dim3 grid((unsigned)((items + 7) / 8)), block(256);
    return wide ? launch_kernel(quantize_rows_block_kernel<SLOTS, 4>, grid, block, 0, st, pdl, x, M, K, args...)
                : launch_kernel(quantize_rows_block_kernel<SLOTS, 1>, grid, block, 0, st, pdl, x, M, K, args...);
}

}  // namespace

cudaError_t launch_quantize_weights_block(const float* w, int64_t groups, int rows, int K, uint8_t* q, float* s,
                                          cudaStream_t st) {
    const int64_t n = groups * blocks_of(rows) * blocks_of(K);
    if (n == 0) return cudaSuccess;
    const int64_t cap = (int64_t)num_sms() * 8;
    return launch_kernel(quantize_weights_block_kernel, dim3((unsigned)(n < cap ? n : cap)), dim3(256), 0, st, false,
                         w, n, rows, K, q, s);
}

cudaError_t launch_quantize_block(const uint16_t* x, int M, int K, uint8_t* q, float* s, cudaStream_t st, bool pdl) {
    if (M == 0) return cudaSuccess;
    return launch_quantize_rows<false>(st, pdl, x, M, K, q, s, nullptr, nullptr, nullptr, 0, 1, nullptr, nullptr);
}

cudaError_t launch_permute_quant_block(const uint16_t* x, const int32_t* topk_ids, const int32_t* rank,
                                       const int32_t* base, int T, int H, int E, int k, int32_t* slot_of,
                                       uint8_t* q, float* s, int* error, cudaStream_t st, bool pdl) {
    if (T == 0) return cudaSuccess;
    return launch_quantize_rows<true>(st, pdl, x, T, H, q, s, topk_ids, rank, base, E, k, slot_of, error);
}

}  // namespace moe
