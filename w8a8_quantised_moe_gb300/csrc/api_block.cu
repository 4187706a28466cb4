// api_block.cu -- the C entry points of the block-scaled FP8 operators and of
// the norms around a block (include/moe_w8a8.h): argument checks, workspace
// layout and launch sequences.
#include <initializer_list>

#include "api_common.h"
#include "block.h"

using namespace moe;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 20;
constexpr int64_t kMaxLinDim = 65536;

struct BlockLinLayout {
    size_t err, q_x, s_x, total;
};
BlockLinLayout block_lin_layout(int64_t M, int64_t K) {
    BlockLinLayout L{};
    L.err = 0;
    L.q_x = 256;
    L.s_x = L.q_x + align256((size_t)M * K);
    L.total = L.s_x + align256((size_t)M * blocks_of((int)K) * 4);
    return L;
}

bool lin_shape_ok(int64_t M, int64_t N, int64_t K) {
    return M >= 0 && M <= kMaxTokens && N >= 16 && N <= kMaxLinDim && N % 16 == 0 && K >= 16 && K <= kMaxLinDim &&
           K % 16 == 0;
}

// Router and routing regions as the layer's other forms (FwdLayout); codes of
// one byte, a scale per slot and 128 channels.
struct BlockFwdLayout {
    size_t err, counts, wsplit, logits, topk_ids, topk_w, rank, hist, offsets, slot_of, q_x, s_x, q_h, s_h, o, done,
        total;
};
BlockFwdLayout block_fwd_layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k) {
    BlockFwdLayout L{};
    const int64_t S = T * k, nchunk = (T + kRouterTokens - 1) / kRouterTokens;
    const RouterPlan rp = router_plan(T, H, E);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    L.err = take(256);
    L.counts = take(2 * 4);
    L.wsplit = take((size_t)3 * rp.E_pad * H * 2);
    int64_t t_few = T < kFewTokens ? T : kFewTokens;  // the most tokens, up to T, of the form for a few
    while (t_few > 0 && !block_few_tokens(t_few, E, k)) --t_few;
    const size_t few = block_route_scratch(t_few, H, E), logits = router_scratch(T, H, E);
    L.logits = take(logits > few ? logits : few);
    L.topk_ids = take(S * 4);
    L.topk_w = take(S * 4);
    L.rank = take(S * 4);
    L.hist = take(nchunk * E * 4);
    L.offsets = take((E + 1) * 4);
    L.slot_of = take(S * 4);
    L.q_x = take(S * H);
    L.s_x = take(S * (H / kBlk) * 4);
    L.q_h = take(S * I);
    L.s_h = take(S * (I / kBlk) * 4);
    L.o = take(S * H * 4);
    L.done = take((H + 255) / 256 * 4);
    L.total = off;
    return L;
}

// One of them null or misaligned (or faked so by the test hook).
bool bad_ptrs(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (p == nullptr || !aligned16(p)) return true;
    return injected(kInjectBadPtr);
}
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

}  // namespace

extern "C" {

moe_status_t moe_w8a8_fp8_block_quantize_weights(const float* w, int64_t groups, int64_t rows, int64_t K,
                                                 uint8_t* w_q, float* w_scale, void* stream) {
    if (groups < 0 || groups > kMaxTokens || rows < 16 || rows > kMaxLinDim || rows % 16 || K < 16 ||
        K > kMaxLinDim || K % 16)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (groups == 0) return MOE_OK;
    if (bad_ptrs({w, w_q, w_scale})) return MOE_ERR_INVALID_ARG;
    return from_cuda(launch_quantize_weights_block(w, groups, (int)rows, (int)K, w_q, w_scale,
                                                   static_cast<cudaStream_t>(stream)));
}

size_t moe_w8a8_fp8_block_linear_workspace_size(int64_t M, int64_t N, int64_t K) {
    return lin_shape_ok(M, N, K) ? block_lin_layout(M, K).total : 0;
}

moe_status_t moe_w8a8_fp8_block_linear(const uint16_t* x, const uint8_t* w_q, const float* w_scale, int64_t M,
                                       int64_t N, int64_t K, uint16_t* y, void* workspace, size_t workspace_bytes,
                                       void* stream) {
    if (!lin_shape_ok(M, N, K)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (M == 0) return MOE_OK;
    if (bad_ptrs({x, w_q, w_scale, y, workspace}) || !aligned256(workspace)) return MOE_ERR_INVALID_ARG;
    const BlockLinLayout L = block_lin_layout(M, K);
    if (workspace_bytes < L.total || injected(kInjectWsShort)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (gemm_path_forced()) return MOE_ERR_NOT_IMPLEMENTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool pdl = pdl_default();
    uint8_t* q_x = at<uint8_t>(workspace, L.q_x);
    float* s_x = at<float>(workspace, L.s_x);
    BlockGemmArgs g{};
    g.act = q_x;
    g.act_scale = s_x;
    g.w = w_q;
    g.w_scale = w_scale;
    g.K = (int)K;
    g.w_rows = (int)N;
    g.n_groups = 1;
    g.total_rows = (int)M;
    g.out = y;
    g.error = at<int>(workspace, L.err);
    g.timeout_ns = current_timeout_ns();
    g.stall = injected(kInjectStall) ? 1 : 0;
    const bool few = block_linear_few_supported((int)M, (int)N, (int)K);
    if (!few || !block_linear_few_fused((int)M)) {
        const cudaError_t e = launch_quantize_block(x, (int)M, (int)K, q_x, s_x, st, pdl);
        if (e != cudaSuccess) return from_cuda(e);
    }
    return from_cuda(few ? launch_block_linear_few(g, x, st, pdl) : launch_block_gemm(BlockEpi::BF16, g, st, pdl));
}

size_t moe_w8a8_fp8_block_workspace_size(int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k) {
    return moe_shape_ok(T, H, I, E, top_k) ? block_fwd_layout(T, H, I, E, top_k).total : 0;
}

moe_status_t moe_w8a8_fp8_block_forward(const uint16_t* x, const float* router_w, const float* router_bias,
                                        const uint8_t* w13_q, const float* w13_scale, const uint8_t* w2_q,
                                        const float* w2_scale, int64_t T, int64_t H, int64_t I, int64_t E,
                                        int64_t top_k, uint16_t* y, void* workspace, size_t workspace_bytes,
                                        void* stream) {
    if (!moe_shape_ok(T, H, I, E, top_k)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (bad_ptrs({x, router_w, w13_q, w13_scale, w2_q, w2_scale, y, workspace}) || !aligned16(router_bias) ||
        !aligned256(workspace))
        return MOE_ERR_INVALID_ARG;
    const BlockFwdLayout L = block_fwd_layout(T, H, I, E, top_k);
    if (workspace_bytes < L.total || injected(kInjectWsShort)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (gemm_path_forced()) return MOE_ERR_NOT_IMPLEMENTED;

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool pdl = pdl_default();  // every launch but the first of launch_router
    const int S = (int)(T * top_k), nchunk = (int)((T + kRouterTokens - 1) / kRouterTokens);
    int* err = at<int>(workspace, L.err);
    int32_t* hist = at<int32_t>(workspace, L.hist);
    int32_t* offsets = at<int32_t>(workspace, L.offsets);
    int32_t* counts = at<int32_t>(workspace, L.counts);
    const uint64_t timeout = current_timeout_ns();

    BlockGemmArgs g{};
    g.n_groups = (int)E;
    g.error = err;
    g.timeout_ns = timeout;
    g.stall = injected(kInjectStall) ? 1 : 0;
    auto first_product = [&](int rows) {
        g.act = at<uint8_t>(workspace, L.q_x);
        g.act_scale = at<float>(workspace, L.s_x);
        g.w = w13_q;
        g.w_scale = w13_scale;
        g.K = (int)H;
        g.w_rows = (int)(2 * I);
        g.up_offset = (int)I;
        g.total_rows = rows;
        g.q_out = at<uint8_t>(workspace, L.q_h);
        g.s_out = at<float>(workspace, L.s_h);
    };
    auto second_product = [&] {
        g.act = at<uint8_t>(workspace, L.q_h);
        g.act_scale = at<float>(workspace, L.s_h);
        g.w = w2_q;
        g.w_scale = w2_scale;
        g.K = (int)I;
        g.w_rows = (int)H;
        g.up_offset = 0;
        g.total_rows = S;
        g.out = at<float>(workspace, L.o);
    };
    cudaError_t e;
    if (block_few_tokens(T, E, top_k)) {  // three launches
        BlockRouteArgs r{};
        r.x = x;
        r.Wr = router_w;
        r.bias = router_bias;
        r.T = (int)T;
        r.H = (int)H;
        r.E = (int)E;
        r.k = (int)top_k;
        r.P = at<float>(workspace, L.logits);
        r.q = at<uint8_t>(workspace, L.q_x);
        r.s = at<float>(workspace, L.s_x);
        r.topk_ids = at<int32_t>(workspace, L.topk_ids);
        r.topk_w = at<float>(workspace, L.topk_w);
        r.done = at<unsigned int>(workspace, L.done);
        r.n_done = (int)((H + 255) / 256);
        r.ticket = at<unsigned int>(workspace, L.err + kTicketOffset);
        r.error = err;
        if ((e = launch_block_route_few(r, st, pdl)) != cudaSuccess) return from_cuda(e);
        g.ids = r.topk_ids;
        g.topk_w = r.topk_w;
        g.T = (int)T;
        g.k = (int)top_k;
        g.done = r.done;
        g.y = y;
        first_product((int)T);
        if ((e = launch_block_gemm_few(BlockEpi::GateUp, g, st, pdl)) != cudaSuccess) return from_cuda(e);
        second_product();
        return from_cuda(launch_block_gemm_few(BlockEpi::F32, g, st, pdl));
    }
    e = launch_router(x, router_w, router_bias, (int)T, (int)H, (int)E, (int)top_k,
                                  at<uint16_t>(workspace, L.wsplit), at<float>(workspace, L.logits),
                                  at<int32_t>(workspace, L.topk_ids), at<float>(workspace, L.topk_w),
                                  at<int32_t>(workspace, L.rank), hist, offsets, counts,
                                  at<unsigned int>(workspace, L.err + kTicketOffset), err, timeout, st, pdl);
    if (e != cudaSuccess) return from_cuda(e);
    if (!router_plan(T, H, E).small && (e = launch_scan(hist, nchunk, (int)E, offsets, counts, st, pdl)) != cudaSuccess)
        return from_cuda(e);
    e = launch_permute_quant_block(x, at<int32_t>(workspace, L.topk_ids), at<int32_t>(workspace, L.rank), hist,
                                   (int)T, (int)H, (int)E, (int)top_k, at<int32_t>(workspace, L.slot_of),
                                   at<uint8_t>(workspace, L.q_x), at<float>(workspace, L.s_x), err, st, pdl);
    if (e != cudaSuccess) return from_cuda(e);

    g.offsets = offsets;
    first_product(S);
    auto product = [&](BlockEpi epi) {
        return block_gemm_few_wanted(g) ? launch_block_gemm_few(epi, g, st, pdl) : launch_block_gemm(epi, g, st, pdl);
    };
    if ((e = product(BlockEpi::GateUp)) != cudaSuccess) return from_cuda(e);

    second_product();
    if ((e = product(BlockEpi::F32)) != cudaSuccess) return from_cuda(e);
    return from_cuda(launch_combine(at<float>(workspace, L.o), at<int32_t>(workspace, L.slot_of),
                                    at<float>(workspace, L.topk_w), (int)T, (int)H, (int)top_k, y, err, st, pdl));
}

moe_status_t moe_w8a8_norm_residual(const void* x, int x_fp32, const uint16_t* branch, const uint16_t* post_w,
                                    const uint16_t* gate, int gate_form, float scale, const uint16_t* pre_w,
                                    float eps, int64_t T, int64_t H, void* x_out, uint16_t* n_out, void* stream) {
    if (T < 0 || T > kMaxTokens || H < 8 || H > 16384 || H % 8) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (gate_form < 0 || gate_form > 3 || (branch == nullptr && pre_w == nullptr) ||
        (branch == nullptr && (post_w != nullptr || gate_form != 0)) || !(eps >= 0.f))
        return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (bad_ptrs({x, branch != nullptr ? x_out : x, pre_w != nullptr ? n_out : x, gate_form != 0 ? gate : x}) ||
        !aligned16(branch) || !aligned16(post_w) || !aligned16(gate) || !aligned16(pre_w))
        return MOE_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = x;
    a.branch = branch;
    a.post_w = post_w;
    a.gate = gate;
    a.pre_w = pre_w;
    a.x_out = x_out;
    a.n_out = n_out;
    a.T = T;
    a.H = (int)H;
    a.scale = scale;
    a.eps = eps;
    return from_cuda(launch_norm_residual(a, x_fp32 != 0, static_cast<GateForm>(gate_form),
                                          static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
