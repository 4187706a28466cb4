// kv_dev.cuh -- device helpers of the paged 8-bit key/value cache.
#pragma once

#include "kv.h"

namespace moe {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMinScale = 0x1p-64f;  // the least scale of a block

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two E4M3 codes (in the low half) as two fp16 values, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}
// The same for the upper two of four codes.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2_hi(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}

__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A block's scale where it is finite, else NaN.
__device__ __forceinline__ float finite_scale(float s) { return fabsf(s) < INFINITY ? s : __uint_as_float(0x7fffffffu); }
// A value block's scale as the attention uses it: the exponent that the weights
// take up, log2(scale), and 1 / scale, by which the sum of the weights is put right.
// A scale of 0 stands for a block that is not seen.  What is not finite counts as NaN: with an
// infinite addend a hidden score of -inf would become NaN.
__device__ __forceinline__ void value_scale(float s, float& lg, float& inv) {
    if (s == 0.f) {
        lg = -INFINITY;
        inv = 0.f;
    } else {
        if (s < kMinScale) s = kMinScale;
        s = finite_scale(s);
        lg = log2f(s);
        inv = __frcp_rn(s);
    }
}

// Whether page id `id` is the cache's; one that is not is reported.
__device__ __forceinline__ bool kv_page_ok(const KvCache& c, int id, int* error) {
    if ((unsigned)id < (unsigned)c.n_pages) return true;
    atomicOr(error, kErrDevice);
    return false;
}

// Sum over the block of THREADS of `mine`, and of the threads before this one;
// red: THREADS / 32 values of shared memory.  Every thread calls it.
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t mine, int64_t& before, int64_t* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t v = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    if (lane == 31) red[warp] = v;
    __syncthreads();
    int64_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const int64_t x = red[w];
        if (w < warp) base += x;
        all += x;
    }
    __syncthreads();
    before = base + v - mine;
    return all;
}

// What a CTA does of the batch's units: [u0, u1) of U, dealt to `ctas`, from `at` on.
struct KvWork {
    int64_t U, u0, u1, base;  // base: number of the first unit of sequence b
    int ctas, b;
    KvPlace at;
};
// Every thread of the block calls it; `work` is shared memory.  Each thread counts
// the units of consecutive sequences; the one whose the CTA's first unit is names the
// sequence, in which every thread looks at row tiles of its own.
template <int THREADS>
__device__ __forceinline__ void kv_find_work(const KvAttendArgs& a, int most_ctas, int least_units, KvWork* work,
                                             int64_t* red) {
    const int per = (a.bt.B + THREADS - 1) / THREADS;
    const int b0 = kv_min((int)threadIdx.x * per, a.bt.B), b1 = kv_min(b0 + per, a.bt.B);
    int64_t mine = 0, before;
    for (int b = b0; b < b1; ++b) mine += kv_seq_units(kv_seq(a.bt, b, a.sh.page), a.sh) * a.c.heads;
    const int64_t U = block_scan<THREADS>(mine, before, red);
    const int ctas = kv_ctas(U, most_ctas, least_units), cta = blockIdx.x;
    const int64_t u0 = cta < ctas ? kv_deal(U, ctas, cta) : U, u1 = cta < ctas ? kv_deal(U, ctas, cta + 1) : U;
    if (threadIdx.x == 0) {
        work->U = U;
        work->u0 = u0;
        work->u1 = u1;
        work->ctas = ctas;
    }
    if (u0 < u1 && u0 >= before && u0 < before + mine) {
        int b = b0;
        for (; b < b1 - 1; ++b) {
            const int64_t units = kv_seq_units(kv_seq(a.bt, b, a.sh.page), a.sh) * a.c.heads;
            if (u0 < before + units) break;
            before += units;
        }
        work->b = b;
        work->base = before;
    }
    __syncthreads();
    if (u0 >= u1) return;
    KvPlace p;
    p.b = work->b;
    p.s = kv_seq(a.bt, p.b, a.sh.page);
    const int64_t per_head = kv_seq_units(p.s, a.sh);
    p.head = (int)kv_quotient(u0 - work->base, per_head);
    const int64_t head_base = work->base + p.head * per_head;
    for (int rt = threadIdx.x, tiles = kv_row_tiles(p.s, a.sh); rt < tiles; rt += THREADS)
        if (kv_enter_if(p, a.sh, rt, u0 - head_base, head_base)) {
            work->at = p;
            break;
        }
    __syncthreads();
}

// Where the parts of a row tile's results are.  A CTA has at most two row tiles
// that it shares with others, its first and its last: parts 2 c and 2 c + 1.  A
// row's info: x the slot of its first part (the later ones are the first of the CTAs
// that follow), y the parts * 256 + its row in the tile; one part: the row is done.
struct KvParts {
    int slot, parts;  // of this CTA's part; parts of the row tile
    bool leader;      // this CTA has the row tile's first unit
};
__device__ __forceinline__ KvParts kv_parts(const KvWork& w, const KvPlace& p, bool first_segment) {
    KvParts r;
    const int c0 = kv_owner(w.U, w.ctas, p.base), c1 = kv_owner(w.U, w.ctas, p.base + (p.end - p.first) - 1);
    r.parts = c1 - c0 + 1;
    r.leader = c0 == (int)blockIdx.x;
    r.slot = 2 * (int)blockIdx.x + (first_segment ? 0 : 1);
    return r;
}

}  // namespace
}  // namespace moe
