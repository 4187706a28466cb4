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
// Bound by HBM: every cached byte is used by a few rows only.  A warp has 32 keys at a
// time and all their channels, in m16n8k16 MMAs with fp16 operands whose M are the keys
// and then the values' channels, N the rows (head, token) of one key head:
//   S^T = K Q^T,  O^T += V^T P^T
// so that 8 rows fill an MMA, the codes are converted once for all rows, and a row costs
// no more registers than it has to.  (Rows as M: 16 of them, three quarters empty where 4
// heads share a key head, with twice the MMAs, exponentials and registers.)  P^T is S^T's
// 8 x 8 blocks transposed, one movmatrix each.
// E4M3 is exact in fp16; a query row is scaled by a power of two to 2^8 <= max < 2^9, so
// that fp16 holds its bf16 values exactly but for those 2^25 times smaller than the largest;
// weights are rounded to fp16 (11 bits, with 6 bits of headroom below and 8 above the maximum
// that is corrected lazily).  Warp-level MMAs rather than tcgen05: a decode step has a few
// rows of a 128-row tile, and the codes can go from their registers into the operands
// without a detour through shared memory as fp16.
//
// The order of channels inside a product, and of keys, is free; it is chosen so that a
// lane reads 16 bytes of a row at a time, for keys (4 channels of one key per word) and
// values (4 channels of 4 keys, paired by byte permutes), without bank conflicts:
// place(row, chunk) = chunk ^ (row & 7), lane's keys as in key_row().
//
// What it measured, 64 sequences of 2048 to 8192 keys, 32 heads on 8 of 128 channels, one token
// each (684 MB): 124 to 130 us, 0.78 to 0.81 of the copy's rate; 2 of 131072 keys, 56 heads on 8
// (537 MB): 105 to 110 us.  With rows as the MMAs' M: 154 and 111; 16 keys a step: 153 and 122;
// 6 copies in the ring and 2 CTAs an SM: 138 and 102.  Bound by the memory's rate and, near it,
// by instructions (about 500 a warp and 32 keys: conversions 190 of them).  With 16 rows
// (two n-tiles) a warp has 245 registers and an SM two CTAs: 32 sequences of 4096 keys with
// 16 rows each take 50 us (135 MB), which 3 CTAs of 168 registers (66) and one copy a step
// (55 to 60) did not improve.
//
// Work: the batch's units of 128 keys (32 a warp) are dealt to the CTAs in equal runs,
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
constexpr int kFewStages = 4;     // copies under way or in use
// Units of a CTA, at least (where there are that many): more CTAs end sooner but have more parts
// to join.  1 / 2 / 4 / 8, from graphs: a token on 4096 keys 19.4 / 15.7 / 15.4 / 19.6 us, 13
// with a window of 500 11.2 / 14.5 / 16.6 / 24.0.
constexpr int kFewLeast = 2;
constexpr float kHeadroom = 8.f;  // the maximum may lag behind by this much (base 2)
constexpr float kWeightBits = 6.f;  // weights are 2^6 at the maximum

// Row of the warp's 16 keys that is column n of MMA column tile j.
__device__ __forceinline__ int key_row(int j, int n) {
    const int t = n >> 1, b = n & 1;
    return 8 * j + (((t >> 1) ^ b) << 2 | (t & 1) << 1 | b);
}

// The 8 x 8 block of fp16 whose row lane / 4 this lane has two elements of, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D channels, NR n-tiles of 8 rows.
template <int D, int NR>
struct Few {
    static constexpr int kRows = 8 * NR;                      // of a row tile
    static constexpr int kHalf = kFewKeys * D;                // bytes of a copy's keys (or values)
    static constexpr int kStage = 2 * kHalf + 16;             // and the two scales
    static constexpr int kRing = kFewStages * kStage;         // a warp's
    static constexpr int kOffO = kKvFewWarps * kRing;         // [rows][D] binary32
    static constexpr int kOffMl = kOffO + kRows * D * 4;      // [warps][rows] maxima, then sums
    static constexpr int kOffWork = kOffMl + kKvFewWarps * kRows * 8;
    static constexpr int kSmem = kOffWork + (int)sizeof(KvWork);
    static constexpr int kCtas = NR == 1 ? 3 : 2;             // on an SM
    static_assert(kOffWork % 16 == 0 && kStage % 16 == 0 && kCtas * (kSmem + 1024) <= 233472, "shared memory");
    __device__ static __forceinline__ int place(int row, int chunk) {
        return row * D + ((D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3)) << 4);
    }
};

// The steps of a CTA's run, as one warp copies them, 16 keys at a time: the page of the
// next copy is looked up a copy ahead.  WINDOW: the call has a window; a kernel of its own, as
// the first seen key costs the others 5 % of a batch with drafted tokens (registers).
template <int D, bool WINDOW>
struct FewCopies {
    using F = Few<D, 1>;  // (a copy is the same for any rows)
    static constexpr int kChunks = D / 16;  // 16-byte pieces of a row
    KvPlace at;
    int64_t left;  // copies
    int id, half;
    int seen;  // the row tile's first seen key
    __device__ __forceinline__ int key0() const {
        return at.unit * kKvFewTokens + ((int)(threadIdx.x >> 5) * kFewStep + half) * kFewKeys;
    }
    __device__ __forceinline__ void look_up(const KvAttendArgs& a) {
        const int k0 = key0();
        id = k0 < at.s.len ? a.bt.page_table[at.b * a.bt.table_stride + (k0 >> a.c.page_bits)] : -1;
    }
    __device__ __forceinline__ void start(const KvAttendArgs& a, const KvWork& w) {
        at = w.at;
        seen = WINDOW ? kv_first_key(at.s, a.sh, at.rt) : 0;
        left = (w.u1 - w.u0) * kFewStep;
        half = 0;
        if (left > 0) look_up(a);
    }
    // Copies 16 keys, their values and the two scales to `stage`; what is not there
    // (behind the sequence, another's page, before the window) becomes 0, its scales too; so do
    // the values before the window in a page that reaches into it: a weight of 0 does not undo a NaN.
    __device__ __forceinline__ void issue(const KvAttendArgs& a, uint8_t* stage) {
        if (left > 0) {
            const int lane = threadIdx.x & 31, k0 = key0(), there_are = at.s.len - k0;
            const bool there = there_are > 0 && (!WINDOW || k0 + kFewKeys > seen) && kv_page_ok(a.c, id, a.error);
            constexpr int kPer = 32 / kChunks;  // rows of an instruction
            const int c = lane % kChunks, row = lane / kChunks;
            const int64_t off =
                there ? id * a.c.page_stride + (((int64_t)at.head << a.c.page_bits) + (k0 & (a.c.page - 1)) + row) * D + c * 16
                      : 0;
            const uint8_t *k = a.c.k + off, *v = a.c.v + off;
            if (there && there_are >= kFewKeys && (!WINDOW || k0 >= seen)) {
#pragma unroll
                for (int i = 0; i < kFewKeys / kPer; ++i) {
                    uint8_t* dst = stage + F::place(i * kPer + row, c);
                    cp_async16(dst, k + i * kPer * D);
                    cp_async16(dst + F::kHalf, v + i * kPer * D);
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < kFewKeys / kPer; ++i) {
                    const bool valid = there && i * kPer + row < there_are;
                    uint8_t* dst = stage + F::place(i * kPer + row, c);
                    cp_async16_zfill(dst, k + (valid ? i * kPer * D : 0), valid);
                    const bool value = valid && (!WINDOW || k0 + i * kPer + row >= seen);
                    cp_async16_zfill(dst + F::kHalf, v + (value ? i * kPer * D : 0), value);
                }
            }
            if (lane < 2) {
                const float* s = (lane == 0 ? a.c.k_scale : a.c.v_scale) + (there ? id * a.c.scale_stride + at.head : 0);
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(static_cast<uint32_t>(
                                 __cvta_generic_to_shared(stage + 2 * F::kHalf + 4 * lane))),
                             "l"(s), "r"(there ? 4 : 0)
                             : "memory");
            }
            if (--left > 0) {
                if (++half == kFewStep) {
                    half = 0;
                    kv_next(at, a.bt, a.sh, a.c.heads);
                    if (WINDOW && at.unit == at.first) seen = kv_first_key(at.s, a.sh, at.rt);
                }
                look_up(a);
            }
        }
        cp_async_commit();
    }
};

// A warp's part of a row tile: lane (g, t) = (lane / 4, lane % 4) has, of every n-tile, the
// rows 2 t and 2 t + 1 (index h) and of their sums the channels [D/8 g, D/8 g + D/8).
template <int D, int NR>
struct FewRows {
    using F = Few<D, NR>;
    static constexpr int kSteps = D / 16, kTiles = D / 16;
    uint32_t q[NR][kSteps][2];
    float o[NR][kTiles][4], m[NR][2], l[NR][2], factor[NR][2];
    int pos[NR][2], pos_min, pos_max;

    // Query rows of the row tile to fp16, the sums to 0.
    __device__ __forceinline__ void start(const KvAttendArgs& a, const KvPlace& p) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int rows = p.s.n * a.sh.group, r0 = p.rt * F::kRows;
        const int last = kv_min(r0 + F::kRows, rows) - 1;
        pos_min = p.s.len - p.s.n + r0 / a.sh.group;
        pos_max = p.s.len - p.s.n + last / a.sh.group;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int r = kv_min(r0 + 8 * n + g, last);  // rows behind the last repeat it
            const int tok = r / a.sh.group, at = p.s.len - p.s.n + tok;
            const uint16_t* row =
                a.q + (int64_t)(p.s.q0 + tok) * a.q_stride + (p.head * a.sh.group + r - tok * a.sh.group) * D;
            uint2 w[kSteps];
            uint32_t top = 0;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                w[s] = *reinterpret_cast<const uint2*>(row + (s >> 2) * 64 + 16 * t + 4 * (s & 3));
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
            const float f = __fmul_rn(__fmul_rn(a.scale, kLog2e), __uint_as_float((uint32_t)(127 + e) << 23));
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                q[n][s][0] = f16_pair(bf16_lo(w[s].x) * down, bf16_hi(w[s].x) * down);
                q[n][s][1] = f16_pair(bf16_lo(w[s].y) * down, bf16_hi(w[s].y) * down);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // row 2 t + h is lane group 2 t + h's
                factor[n][h] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + h));
                pos[n][h] = __shfl_sync(0xffffffffu, at, 4 * (2 * t + h));
                m[n][h] = -INFINITY;
                l[n][h] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
        }
    }

    // One step: 32 keys from k0 on, 16 at each of stage[0] and stage[1].
    __device__ __forceinline__ void step(const KvAttendArgs& a, const uint8_t* const (&stage)[kFewStep], int k0) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        // scores [16 keys][n-tile]: of the keys key_row(0, g) (elements 0, 1) and key_row(1, g) (2, 3)
        // with the rows 2 t, 2 t + 1
        float s[kFewStep][NR][4];
#pragma unroll
        for (int b = 0; b < kFewStep; ++b)
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[b][n][i] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            uint4 k4[kFewStep][2];
#pragma unroll
            for (int b = 0; b < kFewStep; ++b)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    k4[b][j] = *reinterpret_cast<const uint4*>(stage[b] + F::place(key_row(j, g), 4 * c + t));
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int b = 0; b < kFewStep; ++b) {  // the chains of sums side by side
                    auto word = [&](const uint4& v) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; };
                    const uint32_t x = word(k4[b][0]), y = word(k4[b][1]);
                    const uint32_t key[4] = {e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(y), e4m3x2_to_f16x2_hi(x),
                                             e4m3x2_to_f16x2_hi(y)};
#pragma unroll
                    for (int n = 0; n < NR; ++n) mma16816(s[b][n], key, q[n][4 * c + i][0], q[n][4 * c + i][1]);
                }
        }
        float inv[kFewStep];
        bool gone = false;
#pragma unroll
        for (int b = 0; b < kFewStep; ++b) {
            const float2 sc = *reinterpret_cast<const float2*>(stage[b] + 2 * F::kHalf);
            float lg;
            const float key = finite_scale(sc.x);
            value_scale(sc.y, lg, inv[b]);
            gone = gone || sc.y == 0.f;
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[b][n][i] = fmaf(s[b][n][i], key * factor[n][i & 1], lg);
        }
        const int window = a.sh.window;
        if (k0 + kFewStep * kFewKeys - 1 > pos_min || (window > 0 && k0 <= pos_max - window) || gone) {
#pragma unroll
            for (int b = 0; b < kFewStep; ++b) {
                const bool none = inv[b] == 0.f;  // a block that is not there
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = k0 + b * kFewKeys + key_row(i >> 1, g), p = pos[n][i & 1];
                        if (key > p || (window > 0 && key <= p - window) || none) s[b][n][i] = -INFINITY;
                    }
            }
        }
        bool behind = false;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float top = fmaxf(fmaxf(s[0][n][h], s[0][n][h + 2]), fmaxf(s[1][n][h], s[1][n][h + 2]));
                behind = behind || top > m[n][h] + kHeadroom;
            }
        if (__any_sync(0xffffffffu, behind)) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v = fmaxf(fmaxf(s[0][n][h], s[0][n][h + 2]), fmaxf(s[1][n][h], s[1][n][h + 2]));
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
                    v = v > m[n][h] + kHeadroom ? v : m[n][h];  // row by row: no row's bits depend on another's
                    const float down = m[n][h] == v ? 1.f : ex2(m[n][h] - v);
                    m[n][h] = v;
                    l[n][h] *= down;
#pragma unroll
                    for (int i = 0; i < kTiles; ++i) {
                        o[n][i][h] *= down;
                        o[n][i][h + 2] *= down;
                    }
                }
        }
        uint32_t p[kFewStep][NR][2];  // weights as the products' operand
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            float base[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) base[h] = m[n][h] == -INFINITY ? 0.f : m[n][h] - kWeightBits;
#pragma unroll
            for (int b = 0; b < kFewStep; ++b) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = ex2(s[b][n][i] - base[i & 1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float sum = w[h] + w[h + 2];
                    if (sum != 0.f) l[n][h] = fmaf(sum, inv[b], l[n][h]);  // unseen keys leave a block's NaN scale alone
                }
                p[b][n][0] = transposed(f16_pair(w[0], w[1]));
                p[b][n][1] = transposed(f16_pair(w[2], w[3]));
            }
        }
#pragma unroll
        for (int b = 0; b < kFewStep; ++b) {
            const uint8_t* values = stage[b] + F::kHalf;
            uint32_t v[4][D / 32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = key_row(i >> 1, 2 * t + (i & 1));
                if (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4*>(values + F::place(row, g));
                    v[i][0] = x.x, v[i][1] = x.y, v[i][2 % (D / 32)] = x.z, v[i][3 % (D / 32)] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(values + F::place(row, g >> 1) + (g & 1) * 8);
                    v[i][0] = x.x, v[i][1] = x.y;
                }
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w)
#pragma unroll
                for (int half = 0; half < 2; ++half) {  // channels 4 w + 2 half and the next of this lane's
                    const uint32_t sel = half ? 0x7362 : 0x5140;
                    const uint32_t x = __byte_perm(v[0][w], v[1][w], sel), y = __byte_perm(v[2][w], v[3][w], sel);
                    const uint32_t value[4] = {e4m3x2_to_f16x2(x), e4m3x2_to_f16x2_hi(x), e4m3x2_to_f16x2(y),
                                               e4m3x2_to_f16x2_hi(y)};
#pragma unroll
                    for (int n = 0; n < NR; ++n) mma16816(o[n][2 * w + half], value, p[b][n][0], p[b][n][1]);
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

template <int D, int NR, bool WINDOW>
__global__ void __launch_bounds__(kFewThreads, Few<D, NR>::kCtas) kv_attend_few_kernel(const KvAttendArgs a) {
    using F = Few<D, NR>;
    constexpr int kRows = F::kRows;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* ring = smem + warp * F::kRing;
    float* ml = reinterpret_cast<float*>(smem + F::kOffMl);  // maxima [warps][rows], sums [warps][rows]
    KvWork* work = reinterpret_cast<KvWork*>(smem + F::kOffWork);
    pdl_wait();
    pdl_trigger();
    kv_find_work<kFewThreads>(a, gridDim.x, kFewLeast, work, reinterpret_cast<int64_t*>(ml));
    const int64_t units = work->u1 - work->u0;
    if (units <= 0) return;

    FewCopies<D, WINDOW> copies;
    copies.start(a, *work);
#pragma unroll
    for (int i = 0; i < kFewStages - kFewStep; ++i) copies.issue(a, ring + i * F::kStage);
    KvPlace at = work->at;
    FewRows<D, NR> rows;
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
            float* sums = reinterpret_cast<float*>(smem + F::kOffO);
            __syncthreads();  // the previous row tile's have been read
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float l = rows.l[n][h];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
                    if (g == 0) {
                        ml[warp * kRows + 8 * n + 2 * t + h] = rows.m[n][h];
                        ml[(kKvFewWarps + warp) * kRows + 8 * n + 2 * t + h] = l;
                    }
                }
            __syncthreads();
            // one warp after the other, so that one row tile's room is enough
#pragma unroll 1
            for (int w = 0; w < kKvFewWarps; ++w) {
                if (w == warp) {
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int row = 8 * n + 2 * t + h;
                            float m = ml[row];  // the largest maximum
#pragma unroll
                            for (int k = 1; k < kKvFewWarps; ++k) m = fmaxf(m, ml[k * kRows + row]);
                            const float f = rows.m[n][h] == m ? 1.f : ex2(rows.m[n][h] - m);
                            float4* at4 = reinterpret_cast<float4*>(sums + row * D) + D / 32 * g;
#pragma unroll
                            for (int i = 0; i < D / 32; ++i) {  // tiles 2 i, 2 i + 1: four channels
                                const int c = (i + g + t) % (D / 32);  // spread over the banks
                                float4 x = w == 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : at4[c];
                                float v[4];
#pragma unroll
                                for (int k = 0; k < D / 32; ++k)
                                    if (k == c) {
                                        v[0] = rows.o[n][2 * k][h], v[1] = rows.o[n][2 * k][h + 2];
                                        v[2] = rows.o[n][2 * k + 1][h], v[3] = rows.o[n][2 * k + 1][h + 2];
                                    }
                                x.x = fmaf(f, v[0], x.x);
                                x.y = fmaf(f, v[1], x.y);
                                x.z = fmaf(f, v[2], x.z);
                                x.w = fmaf(f, v[3], x.w);
                                at4[c] = x;
                            }
                        }
                }
                __syncthreads();
            }
            // 128 / rows threads a row
            constexpr int kPer = kFewThreads / kRows;
            const int row = threadIdx.x / kPer, all = at.s.n * a.sh.group, r = at.rt * kRows + row;
            float m = ml[row], l = 0.f;
#pragma unroll
            for (int w = 1; w < kKvFewWarps; ++w) m = fmaxf(m, ml[w * kRows + row]);
#pragma unroll
            for (int w = 0; w < kKvFewWarps; ++w) {
                const float mw = ml[w * kRows + row];
                l = fmaf(mw == m ? 1.f : ex2(mw - m), ml[(kKvFewWarps + w) * kRows + row], l);
            }
            // undo the weights' 2^6 (a row that has seen nothing has m = -inf, l = 0)
            const float down = 0x1p-6f;
            l *= down;
            if (r < all) {
                const int tok = r / a.sh.group;
                const int64_t out_row = (int64_t)(at.s.q0 + tok) * a.q_heads + at.head * a.sh.group + r - tok * a.sh.group;
#pragma unroll
                for (int i = 0; i < D / 4 / kPer; ++i) {
                    const int c = i * kPer + threadIdx.x % kPer;
                    float4 o = *(reinterpret_cast<const float4*>(sums + row * D) + c);
                    o = make_float4(o.x * down, o.y * down, o.z * down, o.w * down);
                    if (parts.parts == 1)
                        write_out4(a, out_row, D, c * 4, o, m, l);
                    else
                        *reinterpret_cast<float4*>(a.part_o + ((size_t)parts.slot * kRows + row) * D + c * 4) = o;
                }
                if (threadIdx.x % kPer == 0) {
                    if (parts.parts > 1) a.part_ml[(size_t)parts.slot * kRows + row] = make_float2(m, l);
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
// maximum, in the parts' order.  A warp has `per_warp` rows, up to 32, far apart, as the
// rows to join stand in clusters: it reads their infos at once and then joins those that need
// it one after the other, a lane 4 channels.  (Behind a prompt of 8192 tokens 15 us; with
// neighbouring rows 38, with the infos read one by one 65.)
template <int D>
__global__ void __launch_bounds__(256) kv_join_kernel(const KvAttendArgs a, int per_warp) {
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t warps = (int64_t)gridDim.x * 8, mine = warp + lane * warps;
    pdl_wait();
    pdl_trigger();
    const int first = a.bt.q_start[0], end = a.bt.q_start[a.bt.B];
    int2 info = make_int2(0, 0);
    if (lane < per_warp && mine < (int64_t)a.bt.T * a.q_heads) {
        info = a.info[mine];
        // the rows of sequences; others' info is an earlier call's
        const int token = (int)((uint32_t)mine / (uint32_t)a.q_heads);
        const int parts = info.y >> 8, c0 = info.x >> 1;
        // (a row tile given up after a timeout may have left anything)
        if (token < first || token >= end || parts <= 1 || (unsigned)info.x >= (unsigned)a.slots || parts > a.slots ||
            2 * (c0 + parts - 1) >= a.slots || (info.y & 255) >= a.sh.rows)
            info.y = 0;
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, info.y != 0); todo != 0; todo &= todo - 1) {
        const int which = __ffs(todo) - 1;
        const int x = __shfl_sync(0xffffffffu, info.x, which), y = __shfl_sync(0xffffffffu, info.y, which);
        const int parts = y >> 8, row = y & 255, c0 = x >> 1;
        auto slot = [&](int i) { return (size_t)(i == 0 ? x : 2 * (c0 + i)) * a.sh.rows + row; };
        const bool has = lane * 4 < D;
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kFew = 4;
        float4 v[kFew];  // the first parts' channels, asked for with their maxima
#pragma unroll
        for (int i = 0; i < kFew; ++i)
            v[i] = has && i < parts ? *reinterpret_cast<const float4*>(a.part_o + slot(i) * D + lane * 4) : o;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < parts) ml = a.part_ml[slot(lane)];
        m = ml.x;
        for (int i = lane + 32; i < parts; i += 32) m = fmaxf(m, a.part_ml[slot(i)].x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        auto add = [&](float f, const float4& u) {
            o.x = fmaf(f, u.x, o.x);
            o.y = fmaf(f, u.y, o.y);
            o.z = fmaf(f, u.z, o.z);
            o.w = fmaf(f, u.w, o.w);
        };
        for (int i0 = 0; i0 < parts; i0 += 32) {  // a lane a part's maximum and sum, then the parts' rows
            const int some = kv_min(32, parts - i0);
            if (i0 > 0 && lane < some) ml = a.part_ml[slot(i0 + lane)];
            float f = 0.f;
            if (lane < some) {
                f = ml.x == m ? 1.f : ex2(ml.x - m);
                l = fmaf(f, ml.y, l);
            }
            int i = 0;
            if (i0 == 0) {
#pragma unroll
                for (; i < kFew; ++i) {
                    const float fi = __shfl_sync(0xffffffffu, f, i);
                    if (i < parts) add(fi, v[i]);
                }
            }
#pragma unroll 8
            for (; i < some; ++i) {
                const float fi = __shfl_sync(0xffffffffu, f, i);
                if (has) add(fi, *reinterpret_cast<const float4*>(a.part_o + slot(i0 + i) * D + lane * 4));
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        if (has) write_out4(a, warp + which * warps, D, lane * 4, o, m, l);
    }
}

template <int D, int NR, bool WINDOW>
cudaError_t launch_few_kernel(KvAttendArgs& a, cudaStream_t st, bool pdl) {
    using F = Few<D, NR>;
    auto kern = kv_attend_few_kernel<D, NR, WINDOW>;
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [&] {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem);
    });
    if (err != cudaSuccess) return err;
    a.sh.rows = F::kRows;
    a.slots = 2 * F::kCtas * num_sms();
    return launch_kernel(kern, dim3(F::kCtas * num_sms()), dim3(kFewThreads), F::kSmem, st, pdl, a);
}
template <int D, int NR>
cudaError_t launch_few(KvAttendArgs& a, cudaStream_t st, bool pdl) {
    return a.sh.window > 0 ? launch_few_kernel<D, NR, true>(a, st, pdl) : launch_few_kernel<D, NR, false>(a, st, pdl);
}

}  // namespace

// Rows of the parts that a grid of either form leaves, at most two a CTA (for any D).
int64_t kv_few_part_rows() {
    constexpr int k8 = Few<128, 1>::kCtas * Few<128, 1>::kRows, k16 = Few<128, 2>::kCtas * Few<128, 2>::kRows;
    static_assert(k8 == Few<64, 1>::kCtas * Few<64, 1>::kRows && k16 == Few<64, 2>::kCtas * Few<64, 2>::kRows, "rows");
    return 2 * (int64_t)num_sms() * (k8 > k16 ? k8 : k16);
}

cudaError_t launch_kv_attend_few(KvAttendArgs a, cudaStream_t st, bool pdl) {
    a.sh.tokens = kKvFewTokens;
    a.sh.extra = 0;
    // 8 rows a row tile where sequences and key heads have up to 8 on average, 16 elsewhere.
    const bool eight = (int64_t)a.bt.T * a.sh.group <= 8 * (int64_t)a.bt.B;
    const bool d64 = a.c.dim == 64;
    const cudaError_t e = eight ? (d64 ? launch_few<64, 1>(a, st, pdl) : launch_few<128, 1>(a, st, pdl))
                                : (d64 ? launch_few<64, 2>(a, st, pdl) : launch_few<128, 2>(a, st, pdl));
    return e != cudaSuccess ? e : launch_kv_join(a, st, pdl);
}

cudaError_t launch_kv_join(const KvAttendArgs& a, cudaStream_t st, bool pdl) {
    const int64_t rows = (int64_t)a.bt.T * a.q_heads;
    // a row a warp until the GPU has its 64 warps an SM
    int64_t per = 1;
    while (per < 32 && rows > per * 64 * (int64_t)num_sms()) per *= 2;
    const dim3 grid((unsigned)((rows + 8 * per - 1) / (8 * per)));
    return a.c.dim == 64 ? launch_kernel(kv_join_kernel<64>, grid, dim3(256), 0, st, pdl, a, (int)per)
                         : launch_kernel(kv_join_kernel<128>, grid, dim3(256), 0, st, pdl, a, (int)per);
}

}  // namespace moe
