// block.h -- declarations of the block-scaled FP8 operators (block.cu,
// gemm_block.cu) and of the norms around a block (norm.cu).
//
// Block scales: activations carry one binary32 scale per row and 128 input
// channels, weights one per 128 output x 128 input channels.  A scale is
// amax / 448 of its block (block_scale); the last block of a dimension may be shorter.
#pragma once

#include "internal.h"

namespace moe {

constexpr int kBlk = 128;  // channels that share a scale
__host__ __device__ constexpr int blocks_of(int n) { return (n + kBlk - 1) / kBlk; }

// What a block-scaled product writes.
enum class BlockEpi : int {
    GateUp = 0,  // h = silu(gate) * up, requantised: E4M3 codes and a scale per row and 128 channels
    F32 = 1,     // binary32 rows (second expert product)
    BF16 = 2     // bf16 rows (linear layer)
};

struct BlockGemmArgs {
    const uint8_t* act;      // E4M3 activation rows [total_rows][K]
    const float* act_scale;  // [total_rows][blocks_of(K)]
    const uint8_t* w;        // E4M3 weights [n_groups * w_rows][K]
    const float* w_scale;    // [n_groups][blocks_of(w_rows)][blocks_of(K)]
    int K;                   // multiple of 16
    int w_rows;              // weight rows per group (2I, H or N; a multiple of 16, of 128 with several groups)
    int up_offset;           // GateUp: row offset of the up half (I, a multiple of 128)
    int n_groups;
    int total_rows;          // activation rows
    const int32_t* offsets;  // [n_groups + 1] first row of each group, or nullptr: one group
    void* out;               // F32 / BF16: [total_rows][w_rows]
    uint8_t* q_out;          // GateUp: codes [total_rows][up_offset]
    float* s_out;            // GateUp: scales [total_rows][up_offset / 128]
    int* error;              // sticky device error word
    uint64_t timeout_ns;
    int stall;               // test hook (MOE_INJECT=stall)
    // few tokens only (ids != nullptr; offsets unused): total_rows activation
    // rows, all of them in every tile
    const int32_t* ids;      // [T][k] experts
    const float* topk_w;     // [T][k] (F32)
    int T, k;
    unsigned int* done;      // [column blocks] finished experts, zero before the launch (F32)
    uint16_t* y;             // bf16 [T][w_rows] (F32): the combine
};

// Tensor-core product, groups of many rows (gemm_block.cu).
cudaError_t launch_block_gemm(BlockEpi epi, const BlockGemmArgs& args, cudaStream_t st, bool pdl);
// The same for groups of a few rows (gemm_block_few.cu), GateUp and F32; reads
// the offsets before its wait for the previous kernel, which must have waited
// for the kernel that wrote them.
bool block_gemm_few_wanted(const BlockGemmArgs& args);
cudaError_t launch_block_gemm_few(BlockEpi epi, const BlockGemmArgs& args, cudaStream_t st, bool pdl);

// The linear layer for few rows (linear_block_few.cu): g as for
// launch_block_gemm with BlockEpi::BF16 and one group.  Where
// block_linear_few_fused, x is quantised in the launch and g.act is not read.
bool block_linear_few_fused(int M);
bool block_linear_few_supported(int M, int N, int K);
cudaError_t launch_block_linear_few(const BlockGemmArgs& g, const uint16_t* x, cudaStream_t st, bool pdl);

// Few tokens (block_route.cu): the layer in three launches, without a
// permutation.  Rows of q_out, out and the scales that go with them are then
// slots t k + j, and every tile's columns are all tokens (first product) or all
// slots (second).
constexpr int kFewTokens = 8, kFewSlots = 32;
constexpr int kRouterMaxSlicesFew = 128;   // slices of the router's rows, at most
constexpr int kRouterMaxSliceRows = 128;   // rows of one (H <= 16384)
bool block_few_tokens(int64_t T, int64_t E, int64_t k);
size_t block_route_scratch(int64_t T, int64_t H, int64_t E);  // bytes of P
struct BlockRouteArgs {
    const uint16_t* x;       // bf16 [T][H]
    const float *Wr, *bias;  // fp32 [H][E]; [E] or nullptr
    int T, H, E, k, hs;      // hs: set by the launch
    float* P;                // sums of the clusters [n][T][E rounded up to 32, 64, 128 or 256]
    uint8_t* q;              // codes [T][H]
    float* s;                // scales [T][H / 128]
    int32_t* topk_ids;       // [T][k]
    float* topk_w;           // [T][k]
    unsigned int* done;      // [n_done], cleared for the second product
    int n_done;
    unsigned int* ticket;    // zero between calls
    int* error;
};
cudaError_t launch_block_route_few(BlockRouteArgs a, cudaStream_t st, bool pdl);

// Weights fp32 [groups][rows][K] to E4M3 codes and scales per 128 x 128 block.
cudaError_t launch_quantize_weights_block(const float* w, int64_t groups, int rows, int K, uint8_t* q, float* s,
                                          cudaStream_t st);
// Rows of bf16 x [M][K] to codes [M][K] and scales [M][blocks_of(K)].
cudaError_t launch_quantize_block(const uint16_t* x, int M, int K, uint8_t* q, float* s, cudaStream_t st, bool pdl);
// The same for the layer: each token's row written to its k slots, the slots
// found from the router's chunk ranks and bases.
cudaError_t launch_permute_quant_block(const uint16_t* x, const int32_t* topk_ids, const int32_t* rank,
                                       const int32_t* base, int T, int H, int E, int k, int32_t* slot_of,
                                       uint8_t* q, float* s, int* error, cudaStream_t st, bool pdl);

// Shape of the gate of norm_residual.
enum class GateForm : int { None = 0, Channel = 1, Token = 2, Element = 3 };

struct NormArgs {
    const void* x;           // residual [T][H], bf16 or fp32
    const uint16_t* branch;  // bf16 [T][H] or nullptr
    const uint16_t* post_w;  // bf16 [H] or nullptr: the branch is taken as it is
    const uint16_t* gate;    // bf16 [H], [T] or [T][H] (GateForm), or nullptr
    const uint16_t* pre_w;   // bf16 [H] or nullptr: no second norm
    void* x_out;             // [T][H] as x (unused without a branch)
    uint16_t* n_out;         // bf16 [T][H] (unused without pre_w)
    int64_t T;
    int H;
    float scale, eps;
};
cudaError_t launch_norm_residual(const NormArgs& a, bool fp32_residual, GateForm gate, cudaStream_t st);

}  // namespace moe
