// kv.h -- declarations of the paged 8-bit key/value cache: appending to it
// (kv_append.cu) and attention over it (kv_attend_few.cu, kv_attend.cu).
//
// These kernels may start while the kernel before them on the stream still writes what they read
// (an append its queries, codes and scales): every load is a coherent one, none goes by the
// read-only path, whose data must not change while a kernel lives.
//
// A block of the cache is the tokens of one page and head: E4M3 codes [page][dim]
// and one binary32 scale, for keys and for values.
#pragma once

#include "internal.h"
#include "kv_plan.h"

namespace moe {

struct KvCache {
    uint8_t *k, *v;          // [n_pages][heads][page][dim], page_stride bytes from page to page
    float *k_scale, *v_scale;  // [n_pages][heads], scale_stride values from page to page
    int64_t page_stride, scale_stride;
    int n_pages, heads, page, dim;
    int page_bits;  // page = 1 << page_bits
};

struct KvAppendArgs {
    KvCache c;
    KvBatch bt;
    const uint16_t *k, *v, *q;  // bf16 rows of heads * dim (q: q_heads * dim) or nullptr (q)
    int64_t k_stride, v_stride, q_stride;
    int q_heads;
    const float* rope;  // [rope_rows][rope_dim]: cosines, then sines
    int rope_rows, rope_dim, interleaved;
    uint16_t* q_out;    // [T][q_heads][dim]
    int* error;
    // set by the launch
    int q_tokens;       // tokens of a block that turns queries
    int store_blocks, task_blocks;
    bool by_token;      // how a page of new tokens finds its slot (kv_plan.h)
};
cudaError_t launch_kv_append(KvAppendArgs a, cudaStream_t st, bool pdl);

struct KvAttendArgs {
    KvCache c;
    KvBatch bt;
    KvShape sh;
    const uint16_t* q;  // bf16 [T][q_heads][dim], q_stride elements from token to token
    int64_t q_stride;
    int q_heads;
    float scale;
    uint16_t* out;      // bf16 [T][q_heads][dim]
    float* lse;         // [T][q_heads] or nullptr
    int* error;
    uint64_t timeout_ns;
    int stall;          // test hook (MOE_INJECT=stall)
    // workspace
    int2* info;         // [T][q_heads]: where a row's parts are (kv_dev.cuh)
    float* part_o;      // [slots][rows][dim]
    float2* part_ml;    // [slots][rows]
    int slots;          // two a CTA of the grid; set by the launch
};
// Row tiles of 8 or 16 rows on warp-level MMAs: few rows a sequence and key head.
constexpr int kKvFewTokens = 128, kKvFewWarps = 4;
int64_t kv_few_part_rows();
cudaError_t launch_kv_attend_few(KvAttendArgs a, cudaStream_t st, bool pdl);

// Row tiles of 256 rows on tcgen05 (kv_attend.cu): many rows.
constexpr int kKvRows = 256;
int kv_tc_ctas();
cudaError_t launch_kv_attend(KvAttendArgs a, cudaStream_t st, bool pdl);

// Joins the parts of rows whose units several CTAs had.
cudaError_t launch_kv_join(const KvAttendArgs& a, cudaStream_t st, bool pdl);

}  // namespace moe
