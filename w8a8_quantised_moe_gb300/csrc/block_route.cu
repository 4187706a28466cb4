// block_route.cu -- routing and quantisation for a handful of tokens in one
// launch: the first of the three launches of the block-scaled layer for few
// tokens (the expert products in gemm_block_few.cu are the others).
//
// One token's layer is a chain of latencies, so it takes few links.  The products
// need no permutation: with at most kFewSlots (token, choice) pairs every pair's
// row fits one tile's columns, and a tile writes the pairs of its expert.  What is
// left is
//   1  partial logits: CTA s, rows [s hs, (s + 1) hs) of the fp32 router weights,
//      all tokens, read once over ~128 SMs; a cluster of eight CTAs adds its
//      slices up through distributed shared memory, in order;
//   2  the tokens' codes and scales, a half warp per 128 channels;
//   3  the CTA that finishes last (a ticket) sums the clusters in order, adds the
//      bias, and selects the top-k, a warp per token.  (Summing every slice there
//      instead took 8 us for 8 tokens of 64 experts.)
#include "block.h"
#include "block_dev.cuh"
#include "ptx.cuh"
#include "router_small.cuh"

namespace moe {
namespace {

constexpr int kRfThreads = 256;
constexpr int kRfCluster = 8;

// EPT: 32 EPT >= E experts, the smallest of 1, 2, 4, 8.
template <int EPT>
__global__ void __cluster_dims__(kRfCluster, 1, 1) __launch_bounds__(kRfThreads)
    block_route_few_kernel(const BlockRouteArgs a) {
    constexpr int EP = 32 * EPT, HG = kRfThreads / EP;  // expert columns, groups of rows
    __shared__ float red[HG > 1 ? HG : 1][kFewTokens][EP];
    __shared__ float xs[kRouterMaxSliceRows][kFewTokens];
    __shared__ float part[kFewTokens * EP];
    __shared__ unsigned int last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();

    // codes of the tokens: half warp i takes block i of T x (H / 128)
    const int kb = a.H / kBlk, l16 = tid & 15;
    for (int i0 = ((int)blockIdx.x * (kRfThreads / 16) + (tid >> 4)) & ~1; i0 < a.T * kb; i0 += gridDim.x * (kRfThreads / 16)) {
        const int i = i0 + (tid >> 4 & 1);
        const bool in = i < a.T * kb;
        const size_t at = (size_t)(in ? i : 0) * kBlk + l16 * 8;
        float f[8], s;
        bf16x8_to_f32(*reinterpret_cast<const uint4*>(a.x + at), f);
        const uint2 c = quant8(f, s);
        if (in) {
            *reinterpret_cast<uint2*>(a.q + at) = c;
            if (l16 == 0) a.s[i] = s;
        }
    }
    if (blockIdx.x == 0)
        for (int i = tid; i < a.n_done; i += kRfThreads) a.done[i] = 0u;

    // partial logits of this slice
    const int h0 = blockIdx.x * a.hs, hs = max(0, min(a.hs, a.H - h0));
    const int e = tid % EP, hg = tid / EP;
    for (int i = tid; i < hs * kFewTokens; i += kRfThreads) {
        const int r = i / kFewTokens, t = i % kFewTokens;
        xs[r][t] = t < a.T ? __uint_as_float((uint32_t)a.x[(size_t)t * a.H + h0 + r] << 16) : 0.f;
    }
    __syncthreads();
    float acc[kFewTokens] = {};
    if (e < a.E) {
#pragma unroll 8
        for (int r = hg; r < hs; r += HG) {
            const float w = __ldg(a.Wr + (size_t)(h0 + r) * a.E + e);
#pragma unroll
            for (int t = 0; t < kFewTokens; ++t) acc[t] = fmaf(xs[r][t], w, acc[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < kFewTokens; ++t) red[hg][t][e] = acc[t];
    __syncthreads();
    for (int i = tid; i < a.T * EP; i += kRfThreads) {
        const int t = i / EP, c = i % EP;
        float v = red[0][t][c];
#pragma unroll
        for (int g = 1; g < HG; ++g) v += red[g][t][c];
        part[i] = v;
    }
    cluster_sync_all();
    const int pairs = a.T * EP, rank = (int)cluster_ctarank();
    for (int i = rank * kRfThreads + tid; i < pairs; i += kRfCluster * kRfThreads) {
        float v[kRfCluster];
#pragma unroll
        for (int r = 0; r < kRfCluster; ++r)
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[r]) : "r"(cluster_addr(part + i, r)) : "memory");
#pragma unroll
        for (int r = 1; r < kRfCluster; ++r) v[0] += v[r];
        a.P[(size_t)(blockIdx.x / kRfCluster) * pairs + i] = v[0];
    }
    cluster_sync_all();  // the cluster's sums are written; no CTA leaves while another reads its part
    if (rank != 0) return;
    if (tid == 0) {
        __threadfence();
        last = atomicAdd(a.ticket, 1u) == gridDim.x / kRfCluster - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();

    const int n = (int)gridDim.x / kRfCluster;
    for (int i = tid; i < pairs; i += kRfThreads) {
        float v = 0.f;
#pragma unroll 16
        for (int s = 0; s < n; ++s) v += __ldcg(a.P + (size_t)s * pairs + i);
        part[i] = v;
    }
    __syncthreads();
    if (warp < a.T) {
        float v[1][EPT], my_w[1];
        int my_e[1];
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const int c = lane + 32 * i;
            const float l = part[warp * EP + c];
            v[0][i] = c < a.E && a.bias != nullptr ? l + __ldg(a.bias + c) : l;
        }
        const bool nan = warp_topk<EPT, 1>(v, a.E, a.k, lane, my_e, my_w);
        if (lane < a.k) {
            a.topk_ids[warp * a.k + lane] = my_e[0];
            a.topk_w[warp * a.k + lane] = my_w[0];
        }
        if (nan && lane == 0) atomicOr(a.error, kErrDevice);
    }
    if (tid == 0) *a.ticket = 0u;
}

}  // namespace

namespace {
int route_rows(int H) { return ((H + kRouterMaxSlicesFew - 1) / kRouterMaxSlicesFew + 7) / 8 * 8; }
int route_ctas(int H) {
    const int hs = route_rows(H), slices = (H + hs - 1) / hs;
    return (slices + kRfCluster - 1) / kRfCluster * kRfCluster;
}
}  // namespace

size_t block_route_scratch(int64_t T, int64_t H, int64_t E) {
    const int64_t cols = E <= 32 ? 32 : E <= 64 ? 64 : E <= 128 ? 128 : 256;
    return (size_t)route_ctas((int)H) / kRfCluster * T * cols * 4;
}

bool block_few_tokens(int64_t T, int64_t E, int64_t k) {
    return T <= kFewTokens && T * k <= kFewSlots && T * ((E + 31) / 32 * 32) <= 512;
}

cudaError_t launch_block_route_few(BlockRouteArgs a, cudaStream_t st, bool pdl) {
    a.hs = route_rows(a.H);
    const dim3 grid((unsigned)route_ctas(a.H)), block(kRfThreads);
    if (a.E <= 32) return launch_kernel(block_route_few_kernel<1>, grid, block, 0, st, pdl, a);
    if (a.E <= 64) return launch_kernel(block_route_few_kernel<2>, grid, block, 0, st, pdl, a);
    if (a.E <= 128) return launch_kernel(block_route_few_kernel<4>, grid, block, 0, st, pdl, a);
    return launch_kernel(block_route_few_kernel<8>, grid, block, 0, st, pdl, a);
}

}  // namespace moe
