// api_kv.cu -- the C entry points of the paged 8-bit key/value cache
// (include/moe_w8a8.h): argument checks, workspace layout and launches.
#include <initializer_list>

#include "api_common.h"
#include "kv.h"

using namespace moe;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 20;   // new tokens, sequences
constexpr int64_t kMaxKeys = int64_t(1) << 30;   // tokens of a sequence that a page table can name

bool heads_ok(int64_t Hkv, int64_t D) { return Hkv >= 1 && Hkv <= 256 && (D == 64 || D == 128); }
bool cache_shape_ok(const moe_w8a8_kv_cache_t& c) {
    return heads_ok(c.heads, c.dim) && (c.page == 16 || c.page == 32 || c.page == 64 || c.page == 128) &&
           c.n_pages >= 0 && c.n_pages <= INT32_MAX && c.page_stride >= c.heads * c.page * c.dim &&
           c.page_stride % 16 == 0 && c.page_stride < (int64_t(1) << 40) && c.scale_stride >= c.heads &&
           c.scale_stride < (int64_t(1) << 40);
}
bool batch_shape_ok(const moe_w8a8_kv_batch_t& b, const moe_w8a8_kv_cache_t& c) {
    return b.B >= 0 && b.B <= kMaxRows && b.T >= 0 && b.T <= kMaxRows && b.max_pages >= 0 &&
           b.max_pages <= kMaxKeys / c.page && b.table_stride >= b.max_pages && b.table_stride < (int64_t(1) << 40);
}
bool row_stride_ok(int64_t stride, int64_t heads, int64_t D) {
    return stride >= heads * D && stride % 8 == 0 && stride < (int64_t(1) << 40);
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether T contiguous rows of `width` bf16 values at `out` share bytes with T rows of `w` at
// `in`, `stride` values from one to the next (stride >= w).
bool rows_meet(const uint16_t* out, int64_t width, const uint16_t* in, int64_t w, int64_t stride, int64_t T) {
    const uint64_t o = reinterpret_cast<uintptr_t>(out), i = reinterpret_cast<uintptr_t>(in);
    const uint64_t end = o + 2 * (uint64_t)(T * width), row = 2 * (uint64_t)w, step = 2 * (uint64_t)stride;
    const uint64_t n = i + row > o ? 0 : (o - i - row) / step + 1;  // the first row that ends behind `o`
    return n < (uint64_t)T && i + n * step < end;
}

bool bad_ptrs(std::initializer_list<const void*> by16, std::initializer_list<const void*> by4) {
    for (const void* p : by16)
        if (p == nullptr || !aligned16(p)) return true;
    for (const void* p : by4)
        if (p == nullptr || !aligned4(p)) return true;
    return injected(kInjectBadPtr);
}

KvCache cache_of(const moe_w8a8_kv_cache_t& c) {
    const int bits = c.page == 16 ? 4 : c.page == 32 ? 5 : c.page == 64 ? 6 : 7;
    return {c.k,           c.v,          c.k_scale,    c.v_scale,   c.page_stride, c.scale_stride,
            (int)c.n_pages, (int)c.heads, (int)c.page, (int)c.dim, bits};
}
KvBatch batch_of(const moe_w8a8_kv_batch_t& b) {
    return {b.q_start, b.lengths, b.page_table, b.table_stride, (int)b.B, (int)b.T, (int)b.max_pages};
}

struct AttendLayout {
    size_t info, part_ml, part_o, total;
};
// Rows (new token, query head of a key head) that B sequences have on average, beyond which
// row tiles of 256 are taken.  32 sequences of 4096 keys, 4 key heads, us in tiles of 8 or 16
// and of 256, with 128 channels: 16 rows 50 / 91, 32 rows 74 / 91, 48 rows 104 / 92, 64 rows
// 130 / 94; with 64: 35 / 67, 55 / 68, 79 / 69, 98 / 68.  2 of 32768: 16 rows 37 / 46, 32 rows
// 45 / 46, 64 rows 71 / 46; with 64: 30 / 41, 36 / 41, 55 / 40.
// The average is the batch's, sequences without new tokens counted, and all of it takes one form:
// batches whose sequences differ pay for it (63 single tokens with a chunk of 256, which by
// themselves take 97 and 39 us: 234; a prompt of 8192 tokens in a batch of 1024 places, the
// others empty: 5028, in tiles of 256 518).
constexpr int64_t kManyRows = 32;
bool many_rows(int64_t B, int64_t T, int64_t group) { return T * group > kManyRows * B; }

AttendLayout attend_layout(int64_t T, int64_t Hq, int64_t Hkv, int64_t D) {
    AttendLayout L{};
    // room for the form with many rows where a batch of up to T tokens can take it
    const int64_t few = kv_few_part_rows(), many = 2 * (int64_t)kv_tc_ctas() * kKvRows;
    const int64_t part_rows = many_rows(1, T, Hq / Hkv) && many > few ? many : few;
    L.info = 256;
    L.part_ml = L.info + align256((size_t)T * Hq * 8);
    L.part_o = L.part_ml + align256((size_t)part_rows * 8);
    L.total = L.part_o + align256((size_t)part_rows * D * 4);
    return L;
}
bool attend_shape_ok(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D) {
    return B >= 0 && B <= kMaxRows && T >= 0 && T <= kMaxRows && heads_ok(Hkv, D) && Hq >= Hkv && Hq % Hkv == 0 &&
           Hq <= 1024 && T * Hq <= INT32_MAX;
}

}  // namespace

extern "C" {

moe_status_t moe_w8a8_kv_append(const moe_w8a8_kv_cache_t* cache, const moe_w8a8_kv_batch_t* batch,
                                const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                                const uint16_t* q, int64_t q_stride, int64_t q_heads, const float* rope,
                                int64_t rope_rows, int64_t rope_dim, int interleaved, uint16_t* q_out,
                                void* workspace, size_t workspace_bytes, void* stream) {
    if (cache == nullptr || batch == nullptr) return MOE_ERR_INVALID_ARG;
    const int64_t D = cache->dim;
    if (!cache_shape_ok(*cache) || !batch_shape_ok(*batch, *cache) || !row_stride_ok(k_stride, cache->heads, D) ||
        !row_stride_ok(v_stride, cache->heads, D))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (q != nullptr && (q_heads < 1 || q_heads > 1024 || !row_stride_ok(q_stride, q_heads, D)))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (rope_dim < 0 || rope_dim > D || rope_dim % 16 || rope_rows < 0 || rope_rows > INT32_MAX)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if ((rope == nullptr) != (rope_dim == 0)) return MOE_ERR_INVALID_ARG;
    if (batch->B == 0 || batch->T == 0) return MOE_OK;
    if (bad_ptrs({k, v, cache->k, cache->v, q != nullptr ? q : k, q != nullptr ? q_out : k,
                  rope != nullptr ? static_cast<const void*>(rope) : k, workspace},
                 {cache->k_scale, cache->v_scale, batch->q_start, batch->lengths, batch->page_table}))
        return MOE_ERR_INVALID_ARG;
    if (q != nullptr && q_out == q && q_stride != q_heads * D) return MOE_ERR_INVALID_ARG;  // in place: contiguous
    const int64_t T = batch->T, width = q_heads * D, kv = cache->heads * D;
    if (q != nullptr && q_out != q &&
        (rows_meet(q_out, width, q, width, q_stride, T) || rows_meet(q_out, width, k, kv, k_stride, T) ||
         rows_meet(q_out, width, v, kv, v_stride, T)))
        return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < 256 || injected(kInjectWsShort)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    KvAppendArgs a{};
    a.c = cache_of(*cache);
    a.bt = batch_of(*batch);
    a.k = k;
    a.v = v;
    a.q = q;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_stride = q_stride;
    a.q_heads = (int)q_heads;
    a.rope = rope;
    a.rope_rows = (int)rope_rows;
    a.rope_dim = (int)rope_dim;
    a.interleaved = interleaved;
    a.q_out = q_out;
    a.error = at<int>(workspace, 0);
    return from_cuda(launch_kv_append(a, static_cast<cudaStream_t>(stream), pdl_default()));
}

size_t moe_w8a8_kv_attention_workspace_size(int64_t B, int64_t T, int64_t q_heads, int64_t kv_heads, int64_t dim) {
    return attend_shape_ok(B, T, q_heads, kv_heads, dim) ? attend_layout(T, q_heads, kv_heads, dim).total : 0;
}

moe_status_t moe_w8a8_kv_attention(const moe_w8a8_kv_cache_t* cache, const moe_w8a8_kv_batch_t* batch,
                                   const uint16_t* q, int64_t q_stride, int64_t q_heads, float scale, int64_t window,
                                   uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (cache == nullptr || batch == nullptr) return MOE_ERR_INVALID_ARG;
    const int64_t D = cache->dim, B = batch->B, T = batch->T;
    if (!cache_shape_ok(*cache) || !batch_shape_ok(*batch, *cache) ||
        !attend_shape_ok(B, T, q_heads, cache->heads, D) || !row_stride_ok(q_stride, q_heads, D))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!(scale > 0.f) || scale > 1e30f || window < 0) return MOE_ERR_INVALID_ARG;
    if (B == 0 || T == 0) return MOE_OK;
    if (bad_ptrs({q, out, cache->k, cache->v, workspace},
                 {cache->k_scale, cache->v_scale, batch->q_start, batch->lengths, batch->page_table}) ||
        rows_meet(out, q_heads * D, q, q_heads * D, q_stride, T) || !aligned4(lse) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return MOE_ERR_INVALID_ARG;
    const AttendLayout L = attend_layout(T, q_heads, cache->heads, D);
    if (workspace_bytes < L.total || injected(kInjectWsShort)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    KvAttendArgs a{};
    a.c = cache_of(*cache);
    a.bt = batch_of(*batch);
    a.sh.group = (int)(q_heads / cache->heads);
    a.sh.window = window > kMaxKeys ? 0 : (int)window;  // longer than any sequence: none
    a.sh.page = (int)cache->page;
    a.q = q;
    a.q_stride = q_stride;
    a.q_heads = (int)q_heads;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.error = at<int>(workspace, 0);
    a.timeout_ns = current_timeout_ns();
    a.stall = injected(kInjectStall) ? 1 : 0;
    a.info = at<int2>(workspace, L.info);
    a.part_ml = at<float2>(workspace, L.part_ml);
    a.part_o = at<float>(workspace, L.part_o);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return from_cuda(many_rows(B, T, a.sh.group) ? launch_kv_attend(a, st, pdl_default())
                                                 : launch_kv_attend_few(a, st, pdl_default()));
}

}  // extern "C"
