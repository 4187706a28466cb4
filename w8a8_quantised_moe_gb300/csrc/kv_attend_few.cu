// kv_attend_few.cu -- attention over the paged 8-bit cache for few rows a sequence
// and key head (decoding), and the joining of partial results.
//
//   s_j = scale sk(j) <q, k_j>,  o = sum_j 2^(l_j - m) v_j / sum_j 2^(s'_j - m),
//   s'_j = s_j log2(e),  l_j = s'_j + log2 sv(j),  m the running maximum of l
//
// with k, v the E4M3 codes and sk, sv the scales of their blocks.  The values' scale
// is taken up by the weight's exponent, so that the products see the codes alone; the
// denominator divides it out again (exactly where it is a power of two).
//
// Bound by HBM: every cached byte is used by at most 16 rows.  A warp has 16 keys at
// a time and all their channels: m16n8k16 MMAs with fp16 operands, rows = the queries
// (head, token) of one key head.  E4M3 is exact in fp16; a query row is scaled by a
// power of two to 2^8 <= max < 2^9, so that fp16 holds its bf16 values exactly but for
// those 2^25 times smaller than the largest; weights are rounded to fp16 (11 bits, with
// 6 bits of headroom below and 8 above the maximum that is corrected lazily).  Warp-level
// MMAs rather than tcgen05: 16 rows of a 128-row tile are all that a decode step has,
// and the codes can go from their registers into the operands without a detour through
// shared memory as fp16.
//
// The order of channels inside a product, and of keys, is free; it is chosen so that a
// lane reads 16 bytes of a row at a time, for keys (its B operand: 4 channels of one
// key per word) and values (4 channels of 4 keys, paired by byte permutes), without
// bank conflicts: place(row, chunk) = chunk ^ (row & 7), lane's keys as in key_row().
//
// Work: the batch's units of 64 keys (16 a warp) are dealt to the CTAs in equal runs,
// whatever the lengths of the sequences (kv_plan.h); a run that starts or ends inside
// a row tile leaves its part in the workspace, and kv_join_kernel adds the parts in
// their order.  Copies run ahead over the borders of row tiles.
#include <mutex>

#include "block_dev.cuh"
#include "kv_dev.cuh"

namespace moe {
namespace {

constexpr int kFewThreads = 32 * kKvFewWarps;
constexpr int kFewKeys = 16;      // keys of a copy: they lie in one page
constexpr int kFewStep = 2;       // copies of a warp's step
constexpr int kFewStages = 6;     // copies under way or in use
constexpr int kFewLeast = 2;      // units of a CTA, at least (where there are that many)
constexpr float kHeadroom = 8.f;  // the maximum may lag behind by this much (base 2)
constexpr float kWeightBits = 6.f;  // weights are 2^6 at the maximum

// Row of the warp's 16 keys that is column n of MMA column tile j.
__device__ __forceinline__ int key_row(int j, int n) {
    const int t = n >> 1, b = n & 1;
    return 8 * j + (((t >> 1) ^ b) << 2 | (t & 1) << 1 | b);
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
struct Few {
    static constexpr int kChunks = D / 16;                    // 16-byte pieces of a row
    static constexpr int kHalf = kFewKeys * D;                // bytes of a step's keys (or values)
    static constexpr int kStage = 2 * kHalf + 16;             // and the two scales
    static constexpr int kRing = kFewStages * kStage;         // a warp's
    static constexpr int kOffO = kKvFewWarps * kRing;         // [16][D] binary32
    static constexpr int kOffMl = kOffO + 16 * D * 4;         // [warps][16] maxima, sums
    static constexpr int kOffWork = kOffMl + kKvFewWarps * 16 * 8;
    static constexpr int kSmem = kOffWork + (int)sizeof(KvWork);
    static_assert(kOffWork % 16 == 0 && kStage % 16 == 0, "alignment");
    __device__ static __forceinline__ int place(int row, int chunk) {
        return row * D + ((D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3)) << 4);
    }
    // 16-byte piece of a binary32 row of sums
    __device__ static __forceinline__ int place_o(int row, int c) {
        const int f = D == 128 ? ((c >> 3) << 1) | (row & 1) : (c >> 3) | (row & 1) << 1;
        return row * D * 4 + ((c ^ f) << 4);
    }
};

// The steps of a CTA's run, as one warp copies them, 16 keys at a time: the page of the
// next copy is looked up a copy ahead.
template <int D>
struct FewCopies {
    KvPlace at;
    int64_t left;  // copies
    int id, half;
    __device__ __forceinline__ int key0() const {
        return at.unit * kKvFewTokens + ((int)(threadIdx.x >> 5) * kFewStep + half) * kFewKeys;
    }
    __device__ __forceinline__ void look_up(const KvAttendArgs& a) {
        const int k0 = key0();
        id = k0 < at.s.len ? __ldg(a.bt.page_table + at.b * a.bt.table_stride + (k0 >> a.c.page_bits)) : -1;
    }
    __device__ __forceinline__ void start(const KvAttendArgs& a, const KvWork& w) {
        at = w.at;
        left = (w.u1 - w.u0) * kFewStep;
        half = 0;
        if (left > 0) look_up(a);
    }
    // Copies 16 keys, their values and the two scales to `stage`; what is not there
    // (behind the sequence, another's page) becomes 0, its scales too.
    __device__ __forceinline__ void issue(const KvAttendArgs& a, uint8_t* stage) {
        if (left > 0) {
            const int lane = threadIdx.x & 31, k0 = key0(), there_are = at.s.len - k0;
            const bool there = there_are > 0 && kv_page_ok(a.c, id, a.error);
            constexpr int kPer = 32 / Few<D>::kChunks;  // rows of an instruction
            const int c = lane % Few<D>::kChunks, row = lane / Few<D>::kChunks;
            const int64_t off =
                there ? id * a.c.page_stride + (((int64_t)at.head << a.c.page_bits) + (k0 & (a.c.page - 1)) + row) * D + c * 16
                      : 0;
            const uint8_t *k = a.c.k + off, *v = a.c.v + off;
#pragma unroll
            for (int i = 0; i < kFewKeys / kPer; ++i) {
                const bool valid = there && i * kPer + row < there_are;
                uint8_t* dst = stage + Few<D>::place(i * kPer + row, c);
                cp_async16_zfill(dst, k + (valid ? i * kPer * D : 0), valid);
                cp_async16_zfill(dst + Few<D>::kHalf, v + (valid ? i * kPer * D : 0), valid);
            }
            if (lane < 2) {
                const float* s = (lane == 0 ? a.c.k_scale : a.c.v_scale) + (there ? id * a.c.scale_stride + at.head : 0);
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(static_cast<uint32_t>(
                                 __cvta_generic_to_shared(stage + 2 * Few<D>::kHalf + 4 * lane))),
                             "l"(s), "r"(there ? 4 : 0)
                             : "memory");
            }
            if (--left > 0) {
                if (++half == kFewStep) {
                    half = 0;
                    kv_next(at, a.bt, a.sh, a.c.heads);
                }
                look_up(a);
            }
        }
        cp_async_commit();
    }
};

// A warp's part of a row tile: lane (g, t) = (lane / 4, lane % 4) has rows g and g + 8.
template <int D>
struct FewRows {
    static constexpr int kSteps = D / 16, kTiles = D / 8;
    uint32_t q[kSteps][4];
    float o[kTiles][4], m[2], l[2], factor[2];
    int pos[2], pos_min, pos_max;

    // Query rows of the row tile to fp16, the sums to 0.
    __device__ __forceinline__ void start(const KvAttendArgs& a, const KvPlace& p) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int rows = p.s.n * a.sh.group, r0 = p.rt * kKvFewRows;
        const int last = kv_min(r0 + kKvFewRows, rows) - 1;
        pos_min = p.s.len - p.s.n + r0 / a.sh.group;
        pos_max = p.s.len - p.s.n + last / a.sh.group;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = kv_min(r0 + g + 8 * h, last);  // rows behind the last repeat it
            const int tok = r / a.sh.group;
            pos[h] = p.s.len - p.s.n + tok;
            const uint16_t* row =
                a.q + (int64_t)(p.s.q0 + tok) * a.q_stride + (p.head * a.sh.group + r % a.sh.group) * D;
            uint2 w[kSteps];
            uint32_t top = 0;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                w[s] = __ldg(reinterpret_cast<const uint2*>(row + (s >> 2) * 64 + 16 * t + 4 * (s & 3)));
                // magnitudes of bf16 pairs, compared as whole numbers
                top = __vmaxu2(top, __vmaxu2(w[s].x & 0x7fff7fffu, w[s].y & 0x7fff7fffu));
            }
            top = max(top & 0xffffu, top >> 16);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^-e: e = the exponent of the largest magnitude less 8 (no scaling where it is not finite)
            int e = (int)(top >> 7) - 127 - 8;
            if (top >= 0x7f80u) e = 0;
            if (e < -120) e = -120;
            const float down = __uint_as_float((uint32_t)(127 - e) << 23);
            factor[h] = __fmul_rn(__fmul_rn(a.scale, kLog2e), __uint_as_float((uint32_t)(127 + e) << 23));
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                q[s][h] = f16_pair(bf16_lo(w[s].x) * down, bf16_hi(w[s].x) * down);
                q[s][2 + h] = f16_pair(bf16_lo(w[s].y) * down, bf16_hi(w[s].y) * down);
            }
            m[h] = -INFINITY;
            l[h] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    }

    // One step: 32 keys from k0 on, 16 at each of stage[0] and stage[1].
    __device__ __forceinline__ void step(const KvAttendArgs& a, const uint8_t* const (&stage)[kFewStep], int k0) {
        constexpr int J = 2 * kFewStep;  // column tiles of 8 keys
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        float s[J][4];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            uint4 k4[J];
#pragma unroll
            for (int j = 0; j < J; ++j)
                k4[j] = *reinterpret_cast<const uint4*>(stage[j >> 1] + Few<D>::place(key_row(j & 1, g), 4 * c + t));
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < J; ++j) {  // the column tiles' chains side by side
                    const uint32_t w = i == 0 ? k4[j].x : i == 1 ? k4[j].y : i == 2 ? k4[j].z : k4[j].w;
                    mma16816(s[j], q[4 * c + i], e4m3x2_to_f16x2(w), e4m3x2_to_f16x2_hi(w));
                }
        }
        float inv[kFewStep];
        bool gone = false;
#pragma unroll
        for (int h = 0; h < kFewStep; ++h) {
            const float2 sc = *reinterpret_cast<const float2*>(stage[h] + 2 * Few<D>::kHalf);
            float lg;
            value_scale(sc.y, lg, inv[h]);
            gone = gone || sc.y == 0.f;
            const float f[2] = {sc.x * factor[0], sc.x * factor[1]};
#pragma unroll
            for (int j = 2 * h; j < 2 * h + 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[j][i] = fmaf(s[j][i], f[i >> 1], lg);
        }
        const int window = a.sh.window;
        if (k0 + kFewStep * kFewKeys - 1 > pos_min || (window > 0 && k0 <= pos_max - window) || gone) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const bool none = inv[j >> 1] == 0.f;  // a block that is not there
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = k0 + (j >> 1) * kFewKeys + key_row(j & 1, 2 * t + (i & 1)), p = pos[i >> 1];
                    if (key > p || (window > 0 && key <= p - window) || none) s[j][i] = -INFINITY;
                }
            }
        }
        float top[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            top[h] = fmaxf(s[0][2 * h], s[0][2 * h + 1]);
#pragma unroll
            for (int j = 1; j < J; ++j) top[h] = fmaxf(top[h], fmaxf(s[j][2 * h], s[j][2 * h + 1]));
        }
        if (__any_sync(0xffffffffu, top[0] > m[0] + kHeadroom || top[1] > m[1] + kHeadroom)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v = fmaxf(top[h], m[h]);
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                v = v > m[h] + kHeadroom ? v : m[h];  // row by row: no row's bits depend on another's
                const float down = m[h] == v ? 1.f : ex2(m[h] - v);
                m[h] = v;
                l[h] *= down;
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    o[i][2 * h] *= down;
                    o[i][2 * h + 1] *= down;
                }
            }
        }
        uint32_t p[kFewStep][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float base = m[h] == -INFINITY ? 0.f : m[h] - kWeightBits;
#pragma unroll
            for (int b = 0; b < kFewStep; ++b) {
                float w[4], sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = ex2(s[2 * b + (i >> 1)][2 * h + (i & 1)] - base);
                    sum += w[i];
                }
                if (sum != 0.f) l[h] = fmaf(sum, inv[b], l[h]);  // unseen keys leave a block's NaN scale alone
                p[b][h] = f16_pair(w[0], w[1]);
                p[b][2 + h] = f16_pair(w[2], w[3]);
            }
        }
#pragma unroll
        for (int b = 0; b < kFewStep; ++b) {
            const uint8_t* values = stage[b] + Few<D>::kHalf;
            uint32_t v[4][kTiles / 4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = key_row(i >> 1, 2 * t + (i & 1));
                if (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4*>(values + Few<D>::place(row, g));
                    v[i][0] = x.x, v[i][1] = x.y, v[i][2 % (kTiles / 4)] = x.z, v[i][3 % (kTiles / 4)] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(values + Few<D>::place(row, g >> 1) + (g & 1) * 8);
                    v[i][0] = x.x, v[i][1] = x.y;
                }
            }
#pragma unroll
            for (int w = 0; w < kTiles / 4; ++w) {
                const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5140), a1 = __byte_perm(v[0][w], v[1][w], 0x7362);
                const uint32_t b0 = __byte_perm(v[2][w], v[3][w], 0x5140), b1 = __byte_perm(v[2][w], v[3][w], 0x7362);
                mma16816(o[4 * w], p[b], e4m3x2_to_f16x2(a0), e4m3x2_to_f16x2(b0));
                mma16816(o[4 * w + 1], p[b], e4m3x2_to_f16x2_hi(a0), e4m3x2_to_f16x2_hi(b0));
                mma16816(o[4 * w + 2], p[b], e4m3x2_to_f16x2(a1), e4m3x2_to_f16x2(b1));
                mma16816(o[4 * w + 3], p[b], e4m3x2_to_f16x2_hi(a1), e4m3x2_to_f16x2_hi(b1));
            }
        }
    }
};

// One output row's 4 channels from `c` on, and its log sum.
__device__ __forceinline__ void write_out4(const KvAttendArgs& a, int64_t row, int D, int c, const float4& o, float m,
                                           float l) {
    const float inv = l == 0.f ? 0.f : __fdiv_rn(1.f, l);
    *reinterpret_cast<uint2*>(a.out + row * D + c) =
        make_uint2(bf16_pair(o.x * inv, o.y * inv), bf16_pair(o.z * inv, o.w * inv));
    if (c == 0 && a.lse != nullptr) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D>
__global__ void __launch_bounds__(kFewThreads, 2) kv_attend_few_kernel(const KvAttendArgs a) {
    using F = Few<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* ring = smem + warp * F::kRing;
    float* ml = reinterpret_cast<float*>(smem + F::kOffMl);  // maxima [warps][16], sums [warps][16]
    KvWork* work = reinterpret_cast<KvWork*>(smem + F::kOffWork);
    pdl_wait();
    pdl_trigger();
    kv_find_work<kFewThreads>(a, gridDim.x, kFewLeast, work, reinterpret_cast<int64_t*>(ml));
    const int64_t units = work->u1 - work->u0;
    if (units <= 0) return;

    FewCopies<D> copies;
    copies.start(a, *work);
#pragma unroll
    for (int i = 0; i < kFewStages - kFewStep; ++i) copies.issue(a, ring + i * F::kStage);
    KvPlace at = work->at;
    FewRows<D> rows;
    rows.start(a, at);
    bool first_segment = true;
    int stage = 0;  // of the step, and of the copies asked for next
    auto next_stage = [](int st) { return st + kFewStep == kFewStages ? 0 : st + kFewStep; };
    int ahead = kFewStages - kFewStep;
    for (int64_t u = 0; u < units; ++u) {
#pragma unroll
        for (int i = 0; i < kFewStep; ++i) copies.issue(a, ring + (ahead + i) * F::kStage);
        ahead = next_stage(ahead);
        cp_async_wait<kFewStages - kFewStep>();
        __syncwarp();
        const uint8_t* const in[kFewStep] = {ring + stage * F::kStage, ring + (stage + 1) * F::kStage};
        rows.step(a, in, at.unit * kKvFewTokens + warp * kFewStep * kFewKeys);
        __syncwarp();  // the stages may be written again
        stage = next_stage(stage);
        if (at.unit + 1 == at.end || u + 1 == units) {
            // the end of the row tile, or of the CTA's run in it: the warps' sums together
            const KvParts parts = kv_parts(*work, at, first_segment);
            const int g = lane >> 2, t = lane & 3;
            uint8_t* sums = smem + F::kOffO;
            __syncthreads();  // the previous row tile's have been read
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float l = rows.l[h];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                if (t == 0) {
                    ml[warp * 16 + g + 8 * h] = rows.m[h];
                    ml[kKvFewWarps * 16 + warp * 16 + g + 8 * h] = l;
                }
            }
            __syncthreads();
            float f[2];  // what brings this warp's sums to the largest maximum
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float m = ml[g + 8 * h];
#pragma unroll
                for (int w = 1; w < kKvFewWarps; ++w) m = fmaxf(m, ml[w * 16 + g + 8 * h]);
                f[h] = rows.m[h] == m ? 1.f : ex2(rows.m[h] - m);
            }
            // one warp after the other, so that one row tile's room is enough
#pragma unroll 1
            for (int w = 0; w < kKvFewWarps; ++w) {
                if (w == warp) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        // lane's channels D/4 t ..: tile i's two columns are D/8 apart
#pragma unroll
                        for (int col = 0; col < 2; ++col)
#pragma unroll
                            for (int i = 0; i < D / 8; i += 4) {
                                float4* at4 = reinterpret_cast<float4*>(
                                    sums + F::place_o(g + 8 * h, (D / 4 * t + D / 8 * col + i) / 4));
                                float4 x = w == 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : *at4;
                                x.x = fmaf(f[h], rows.o[i][2 * h + col], x.x);
                                x.y = fmaf(f[h], rows.o[i + 1][2 * h + col], x.y);
                                x.z = fmaf(f[h], rows.o[i + 2][2 * h + col], x.z);
                                x.w = fmaf(f[h], rows.o[i + 3][2 * h + col], x.w);
                                *at4 = x;
                            }
                }
                __syncthreads();
            }
            // 8 threads a row
            const int row = threadIdx.x >> 3, all = at.s.n * a.sh.group, r = at.rt * kKvFewRows + row;
            float m = ml[row], l = 0.f;
#pragma unroll
            for (int w = 1; w < kKvFewWarps; ++w) m = fmaxf(m, ml[w * 16 + row]);
#pragma unroll
            for (int w = 0; w < kKvFewWarps; ++w) {
                const float mw = ml[w * 16 + row];
                l = fmaf(mw == m ? 1.f : ex2(mw - m), ml[kKvFewWarps * 16 + w * 16 + row], l);
            }
            // undo the weights' 2^6 (a row that has seen nothing has m = -inf, l = 0)
            const float down = 0x1p-6f;
            l *= down;
            if (r < all) {
                const int tok = r / a.sh.group;
                const int64_t out_row = (int64_t)(at.s.q0 + tok) * a.q_heads + at.head * a.sh.group + r % a.sh.group;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const int c = i * 8 + (threadIdx.x & 7);
                    float4 o = *reinterpret_cast<const float4*>(sums + F::place_o(row, c));
                    o = make_float4(o.x * down, o.y * down, o.z * down, o.w * down);
                    if (parts.parts == 1)
                        write_out4(a, out_row, D, c * 4, o, m, l);
                    else
                        *reinterpret_cast<float4*>(a.part_o + ((size_t)parts.slot * kKvFewRows + row) * D + c * 4) = o;
                }
                if ((threadIdx.x & 7) == 0) {
                    if (parts.parts > 1) a.part_ml[(size_t)parts.slot * kKvFewRows + row] = make_float2(m, l);
                    if (parts.leader) a.info[out_row] = make_int2(parts.slot, parts.parts * 256 + row);
                }
            }
            first_segment = false;
            if (u + 1 < units) {
                kv_next(at, a.bt, a.sh, a.c.heads);
                rows.start(a, at);
            }
        } else {
            ++at.unit;
        }
    }
    cp_async_wait<0>();
}

// Rows with several parts: their sum, each part's weights brought to the largest
// maximum, in the parts' order.  A warp a row at a time, rows dealt in turn.
template <int D>
__global__ void __launch_bounds__(256) kv_join_kernel(const KvAttendArgs a, int per_warp) {
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t all = (int64_t)a.bt.T * a.q_heads;
    pdl_wait();
    pdl_trigger();
    const int64_t lo = (int64_t)kv_clamp(a.bt.q_start[0], 0, a.bt.T) * a.q_heads;
    int64_t hi = lo;  // the rows of sequences are [lo, hi)
    hi = (int64_t)kv_max(kv_clamp(a.bt.q_start[a.bt.B], 0, a.bt.T), (int)(lo / a.q_heads)) * a.q_heads;
    for (int64_t r0 = warp * per_warp; r0 < kv_min64(warp * per_warp + per_warp, all); ++r0) {
        if (r0 < lo || r0 >= hi) continue;
        const int2 info = a.info[r0];
        const int parts = info.y >> 8, row = info.y & 255, c0 = info.x >> 1;
        if (parts <= 1) continue;
        auto slot = [&](int i) { return (size_t)(i == 0 ? info.x : 2 * (c0 + i)) * a.sh.rows + row; };
        float m = -INFINITY, l = 0.f;
        for (int i = lane; i < parts; i += 32) m = fmaxf(m, a.part_ml[slot(i)].x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < parts; i0 += 32) {  // a lane a part's maximum and sum, then the parts' rows
            const int some = kv_min(32, parts - i0);
            float f = 0.f;
            if (lane < some) {
                const float2 x = a.part_ml[slot(i0 + lane)];
                f = x.x == m ? 1.f : ex2(x.x - m);
                l = fmaf(f, x.y, l);
            }
#pragma unroll 8
            for (int i = 0; i < some; ++i) {
                const float fi = __shfl_sync(0xffffffffu, f, i);
                if (lane * 4 < D) {
                    const float4 v = *reinterpret_cast<const float4*>(a.part_o + slot(i0 + i) * D + lane * 4);
                    o.x = fmaf(fi, v.x, o.x);
                    o.y = fmaf(fi, v.y, o.y);
                    o.z = fmaf(fi, v.z, o.z);
                    o.w = fmaf(fi, v.w, o.w);
                }
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        if (lane * 4 < D) write_out4(a, r0, D, lane * 4, o, m, l);
    }
}

template <int D>
cudaError_t launch_few(const KvAttendArgs& a, cudaStream_t st, bool pdl) {
    auto kern = kv_attend_few_kernel<D>;
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [&] {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<D>::kSmem);
    });
    if (err != cudaSuccess) return err;
    return launch_kernel(kern, dim3(kv_few_ctas()), dim3(kFewThreads), Few<D>::kSmem, st, pdl, a);
}

}  // namespace

int kv_few_ctas() { return 2 * num_sms(); }

cudaError_t launch_kv_attend_few(KvAttendArgs a, cudaStream_t st, bool pdl) {
    a.sh.rows = kKvFewRows;
    a.sh.tokens = kKvFewTokens;
    a.sh.extra = 0;
    const cudaError_t e = a.c.dim == 64 ? launch_few<64>(a, st, pdl) : launch_few<128>(a, st, pdl);
    return e != cudaSuccess ? e : launch_kv_join(a, st, pdl);
}

cudaError_t launch_kv_join(const KvAttendArgs& a, cudaStream_t st, bool pdl) {
    const int64_t rows = (int64_t)a.bt.T * a.q_heads;
    // a row a warp until the GPU has its 64 warps an SM
    const int64_t per = rows / (64 * (int64_t)num_sms()) + 1;
    const dim3 grid((unsigned)((rows + 8 * per - 1) / (8 * per)));
    return a.c.dim == 64 ? launch_kernel(kv_join_kernel<64>, grid, dim3(256), 0, st, pdl, a, (int)per)
                         : launch_kernel(kv_join_kernel<128>, grid, dim3(256), 0, st, pdl, a, (int)per);
}

}  // namespace moe
