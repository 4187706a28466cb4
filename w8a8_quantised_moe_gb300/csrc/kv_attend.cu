// kv_attend.cu -- attention over the paged 8-bit cache for many rows a sequence and
// key head (prompts, chunks of them, drafted tokens), on the tcgen05 tensor cores.
// The mathematics is that of kv_attend_few.cu.
//
// A CTA has 256 rows (query token, head of the group) of one key head as two tiles of
// 128, each an MMA's M, and 128 keys a step:
//   S = Q1 K^T + Q2 K^T   kind::f8f6f4 on the cache's codes as they are.  A bf16 query
//       channel has 8 significant bits, two E4M3 values of 4: Q1 = E4M3(q), Q2 =
//       E4M3(q - Q1), the row scaled to 128 <= max < 256, is q but for what lies below
//       2^-17 of the row's largest channel.  Both parts at twice the fp16 rate cost
//       what one fp16 product would, and the keys need no conversion.
//   O += P V              kind::f16: weights in fp16 (11 bits) from tensor memory,
//       values converted to fp16 (exact).  E4M3 pairs would not do here: weights
//       below 2^-18 of the largest would be lost, and long contexts are made of them.
//   warps 0-7, 8-15  softmax of one tile each, two threads a row: scores from tensor memory,
//                    weights back in their place; the maximum is corrected only when it
//                    rises by more than 2^8, by the same threads
//   warps 16-19      values: codes from global memory to fp16 in shared memory, keys'
//                    and values' scales
//   warp 20          keys: TMA, a box a page; reports pages that are not the cache's
//   warps 21, 22     MMA issuers, a tile each (21 also holds the tensor memory)
// Work is dealt as in kv_attend_few.cu, a row tile counting kTcExtra steps more than it has.
// Waits on mbarriers are bounded (ptx.cuh); the two warps of a row group meet at a hardware
// barrier, which neither leaves alone (TcRow).
//
// What bounds it: a step of both tiles is 2560 clocks of MMAs (of which the scores' halves of
// 64 keys read shared memory for 768, 512 with 128 keys) and takes about 4100 (1024 new
// tokens, 32 heads on 8, 16384 keys: 105 steps a CTA in 255 us).  The tensor pipe is active
// for half of that, and 60 % of the issue slots are taken: 2600 instructions a scheduler and
// step, of which the weights themselves (multiply-add, exponential, sum, packing) are 620, the
// maxima 110, the values' conversion 340 and the rest what a call, a wait and a barrier cost.
// A prompt of 8192 tokens, 32 heads on 8 of 128 channels: 555 to 562 us (0.55 TFLOP of scores
// and weighted values: 0.53 of the measured bf16 rate); without the softmax the same
// loop takes two thirds of it.  768 threads leave 80 registers each, of which the compiler
// spills 160 to 190 bytes a thread: one more value held in the values' warps costs a prompt up to
// 7 %.
//
// Measured on the way, that prompt and the case of 1024 new tokens (us): all 128 scores of a
// row in registers, unrolled: 1530 (warps waited for instructions; 64-bit sums over row tiles
// one by one at the start); short loops 857; MMAs issued under a predicate 828; scores a half
// ahead of the softmax 759 and 240, by one warp a row group (two: the same by themselves, 610
// against 665 once the deal counted what a row tile costs); barriers asked with a time for
// which the thread may be suspended, 252 against 277.  Slower: a warp for both tiles' MMAs; a
// row group's two warps with a half of the step each and no scores ahead, 757 and 339; the
// weights before the maximum, 742 and 309; more registers for the softmax by setmaxnreg, one
// unrolled pass over the scores (no change); pages prefetched to L2 (a chunk of 64 tokens on
// 131072 keys 148 against 154, the others no change).
#include <mutex>

#include "block_dev.cuh"
#include "block_tiles.cuh"
#include "kv_dev.cuh"

namespace moe {
namespace {

constexpr int kTcThreads = 768;
constexpr int kTcValues0 = 16, kTcKeys0 = 20, kTcProducts0 = 21;  // first warps of the roles behind the softmax's 16
constexpr int kTcTile = 128;      // rows of a tile, keys of a step
constexpr int kTcHalf = 64;       // keys of half a step, whose scores are one of a tile's two buffers
constexpr int kTcKS = 2, kTcVS = 2;  // stages of keys, of values (three of keys: the same times)
// What beginning and ending a row tile costs, in steps, for the deal.  A prompt of 8192
// tokens, 0 / 2 / 4 / 6 / 8: 809 / 706 / 590 / 581 / 593 us with 128 channels (before the join was
// made faster), 519 / 439 / 437 / 447 / 453 with 64 (the CTAs with a head's first row tiles have up
// to 29 of them).
constexpr int kTcExtra = 6;
constexpr float kTcHeadroom = 8.f, kTcWeightBits = 6.f;  // as in kv_attend_few.cu
constexpr uint32_t kTcCols = 512;

template <int D>
struct Tc {
    static constexpr int kPiece = kTcTile * D;        // bytes of a tile's rows in E4M3 (Q1, Q2; keys)
    static constexpr int kValues = kTcTile * D * 2;   // of a step's values in fp16
    static constexpr int kOffK = 4 * kPiece;          // after Q [tile][part]
    static constexpr int kOffV = kOffK + kTcKS * kPiece;
    static constexpr int kOffScales = kOffV + kTcVS * kValues;  // [stage][8 groups of 16 keys] (key, log2 value, 1 / value)
    static constexpr int kOffStage = kOffScales + kTcVS * 8 * 16;  // 2 KB a softmax warp
    static constexpr int kOffShared = kOffStage + 16 * 2048;       // [use][tile][row][part], what a row's two threads tell each other
    static constexpr int kOffBars = kOffShared + 3 * 2 * kTcTile * 8;
    // q_full[2] k_full[KS] k_empty[KS] v_full[VS] v_empty[VS] s_full[2][2] p_full[2][2] pv_done[2][2] teardown[2] stall
    static constexpr int kNumBars = 2 + 2 * kTcKS + 2 * kTcVS + 12 + 3;
    static constexpr int kOffWork = (kOffBars + kNumBars * 8 + 15) / 16 * 16;
    static constexpr int kOffMisc = (kOffWork + (int)sizeof(KvWork) + 15) / 16 * 16;
    static constexpr int kUsed = kOffMisc + 64 + kTcThreads / 32 * 8;
    // more than half an SM's, so that the one CTA that holds the tensor memory is alone there
    static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
    static_assert(kSmem <= 232448, "shared memory budget");
    // place of a 16-byte piece in a swizzled E4M3 tile (128-byte swizzle, 64-byte where rows are 64 bytes)
    __device__ static __forceinline__ int place(int row, int c) {
        return row * D + ((D == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3)) << 4);
    }
    __device__ static __forceinline__ uint64_t desc(uint32_t saddr) {
        if (D == 128) return smem_desc_sw128(saddr);
        uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
        d |= static_cast<uint64_t>(1) << 16;
        d |= static_cast<uint64_t>(512 >> 4) << 32;  // 8 rows x 64 B
        d |= static_cast<uint64_t>(1) << 46;
        d |= static_cast<uint64_t>(4) << 61;  // 64-byte swizzle
        return d;
    }
    // Values: channels contiguous ("MN-major"), 64 of them a 128-byte row, 8 keys a
    // 1024-byte group; the next group of keys follows, the next 64 channels are 16 KB on.
    __device__ static __forceinline__ uint64_t desc_values(uint32_t saddr) {
        uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
        d |= static_cast<uint64_t>((kTcTile * 128) >> 4) << 16;
        d |= static_cast<uint64_t>(1024 >> 4) << 32;
        d |= static_cast<uint64_t>(1) << 46;
        d |= static_cast<uint64_t>(2) << 61;
        return d;
    }
    __device__ static __forceinline__ int place_value(int key, int c) {  // c: 8 channels
        return (c >> 3) * (kTcTile * 128) + (key >> 3) * 1024 + (key & 7) * 128 + (((c & 7) ^ (key & 7)) << 4);
    }
};

struct TcBars {
    uint64_t *q_full, *k_full, *k_empty, *v_full, *v_empty, *s_full, *p_full, *pv_done, *teardown, *stall;
    __device__ __forceinline__ explicit TcBars(uint8_t* at) {
        uint64_t* b = reinterpret_cast<uint64_t*>(at);
        q_full = b;
        k_full = q_full + 2;
        k_empty = k_full + kTcKS;
        v_full = k_empty + kTcKS;
        v_empty = v_full + kTcVS;
        s_full = v_empty + kTcVS;
        p_full = s_full + 4;
        pv_done = p_full + 4;
        teardown = pv_done + 4;
        stall = teardown + 2;
    }
};

// warp_wait (gemm_common.cuh) for warps that share their schedulers with busy ones: a thread
// that waits is suspended for up to 20 us at a time, where the plain test came back some five
// times a wait and took a third of the issue slots.
__device__ __forceinline__ bool tc_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, const WaitCtl& ctl) {
    if (__all_sync(0xffffffffu, tc_test(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        if (__all_sync(0xffffffffu, tc_test(bar, parity))) return true;
        int give_up = 0;
        if ((threadIdx.x & 31) == 0) {
            if (*ctl.abort) {
                give_up = 1;
            } else if (global_timer_ns() - t0 > ctl.timeout_ns) {
                give_up_timeout(ctl);
                give_up = 1;
            }
        }
        if (__shfl_sync(0xffffffffu, give_up, 0)) return false;
    }
}

// A CTA's run, cut at the borders of row tiles; every role walks through it.
struct TcWalk {
    KvPlace at;
    int64_t end;  // of the run
    int n;        // steps here; 0: no more
    bool first;
    __device__ __forceinline__ explicit TcWalk(const KvWork& w) : at(w.at), end(w.u1), first(true) { count(); }
    __device__ __forceinline__ void count() {
        const int64_t left = end - (at.base + (at.unit - at.first));
        n = left <= 0 ? 0 : left < at.end - at.unit ? (int)left : at.end - at.unit;
    }
    __device__ __forceinline__ bool more() const { return n > 0; }
    __device__ __forceinline__ bool whole() const { return n == at.end - at.first; }  // the row tile is this CTA's alone
    __device__ __forceinline__ void next(const KvAttendArgs& a) {
        first = false;
        if (end <= at.base + (at.end - at.first)) {  // the run ends with this row tile, or in it
            n = 0;
        } else {
            at.unit = at.end - 1;
            kv_next(at, a.bt, a.sh, a.c.heads);
            count();
        }
    }
    // tiles of the row tile that have rows
    __device__ __forceinline__ int tiles(const KvAttendArgs& a) const {
        return at.s.n * a.sh.group - at.rt * a.sh.rows > kTcTile ? 2 : 1;
    }
};

// Rows r0 .. r0 + 31 of a sequence and key head: their token and query head, by one division
// and a product (x / group = x * ceil(2^21 / group) / 2^21 for x < 2^11, group <= 2^10).
struct TcRows {
    const KvAttendArgs& a;
    const KvPlace& p;
    int r0, tok0, rest0;
    uint32_t inverse;
    __device__ __forceinline__ TcRows(const KvAttendArgs& args, const KvPlace& place, int row)
        : a(args), p(place), r0(row), tok0(row / args.sh.group), rest0(row - row / args.sh.group * args.sh.group),
          inverse(((1u << 21) + args.sh.group - 1) / args.sh.group) {}
    __device__ __forceinline__ int token(int i) const { return tok0 + (int)(((uint32_t)(rest0 + i) * inverse) >> 21); }
    __device__ __forceinline__ int64_t row(int i, int64_t tokens, int heads) const {  // tokens: from one to the next
        const int more = (int)(((uint32_t)(rest0 + i) * inverse) >> 21);
        return (p.s.q0 + tok0 + more) * tokens + (int64_t)(p.head * a.sh.group + rest0 + i - more * a.sh.group) * heads;
    }
    __device__ __forceinline__ int64_t q_row(int i) const { return row(i, a.q_stride, a.c.dim); }
    __device__ __forceinline__ int64_t out_row(int i) const { return row(i, a.q_heads, 1); }
};

// A ring's stage and phase.
struct TcRing {
    uint32_t stage = 0, phase = 0;
    __device__ __forceinline__ void step(uint32_t n) {
        if (++stage == n) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

// Pages of 16-key groups: group i of the step that begins at key k0; -1: none there.
__device__ __forceinline__ int tc_page(const KvAttendArgs& a, const KvPlace& p, int k0, int i) {
    const int k = k0 + 16 * i;
    return k < p.s.len ? a.bt.page_table[p.b * a.bt.table_stride + (k >> a.c.page_bits)] : -1;
}

// max of three
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Waits for the warp's tensor-memory loads; no use of the registers moves above it.
__device__ __forceinline__ void tc_wait_ld_16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])::"memory");
}
__device__ __forceinline__ void tc_wait_ld_32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
// Each thread of the warp writes 16 consecutive columns of its lane.
__device__ __forceinline__ void tc_st_16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// a * b + c on pairs
__device__ __forceinline__ f32x2 fma2_of(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// ------------------------------------------------------------------ softmax
// Barrier of the two warps of a row group, and the OR of their conditions.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pair_any(int id, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// A thread of the softmax: row `row` of tile t's 128, keys [32 part, 32 part + 32) of every
// half, channels [D/2 part, D/2 part + D/2) of queries and output.  Two warps share 32 rows
// (and the tensor memory's lanes): a warp alone is a chain of latencies, and with one warp
// a row group the softmax of a half took 1250 clocks where its exponentials need 256.
// Their barriers are not bounded, so neither leaves the other: a warp whose wait gave up
// goes on, and both return at the next pair_any.
template <int D>
struct TcRow {
    static constexpr int kCols = D / 2;  // channels of a part
    float m, l, factor;
    int pos, pos_first, pos_last;  // position; those of the warp's first and last row
    bool valid;

    // The warp's 32 rows x its channels of the queries, as two E4M3 parts in shared memory.
    // Lanes side by side load a row; its largest magnitude is that of both warps.
    __device__ __forceinline__ void start(const KvAttendArgs& a, const KvPlace& p, int t, int row, int part,
                                          uint8_t* q_tile, uint32_t* shared, int pair) {
        constexpr int kLanes = kCols / 8, kRows = 32 / kLanes, kLoads = 32 / kRows;  // lanes of a row, rows of a load
        const int lane = threadIdx.x & 31, group = a.sh.group, rows = p.s.n * group;
        const TcRows of(a, p, p.rt * a.sh.rows + t * kTcTile + (row & ~31));  // the warp's rows
        const int r0 = of.r0, c = p.s.len - p.s.n;
        auto source = [&](int i) {
            const int rr = i * kRows + lane / kLanes;
            const uint16_t* src = a.q + of.q_row(rr) + part * kCols + lane % kLanes * 8;
            return r0 + rr < rows ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
        };
        uint4 w[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) w[i] = source(i);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            // magnitudes of bf16 pairs, compared as whole numbers
            uint32_t x = __vmaxu2(__vmaxu2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu),
                                  __vmaxu2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu));
            x = max(x & 0xffffu, x >> 16);
#pragma unroll
            for (int off = kLanes / 2; off > 0; off >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, off));
            if (lane % kLanes == 0) shared[2 * ((row & ~31) + i * kRows + lane / kLanes) + part] = x;
        }
        pair_sync(pair);
        auto largest_of = [&](int rr) {
            const uint2 x = reinterpret_cast<const uint2*>(shared)[rr];
            return max(x.x, x.y);
        };
        // a row's scale 2^-e: e = the exponent of its largest magnitude less 7
        auto exponent = [](uint32_t x) { return max((int)(x >> 7) - 127 - 7, -120); };
        auto power = [](int e) { return __uint_as_float((uint32_t)(127 + e) << 23); };
        const uint32_t mine = largest_of(row);
        factor = __fmul_rn(__fmul_rn(a.scale, kLog2e), power(exponent(mine)));
        if (mine >= 0x7f80u) factor = __uint_as_float(0x7fffffffu);  // a row that is not finite
        const int r = r0 + (row & 31);
        valid = r < rows;
        pos = valid ? c + of.token(row & 31) : -1;
        pos_first = r0 < rows ? c + of.token(0) : -1;
        pos_last = r0 + 31 < rows ? c + of.token(31) : -1;
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int rr = (row & ~31) + i * kRows + lane / kLanes;
            const float down = power(-exponent(largest_of(rr)));
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t x = j ? w[i].z : w[i].x, y = j ? w[i].w : w[i].y;
                const float f[4] = {bf16_lo(x) * down, bf16_hi(x) * down, bf16_lo(y) * down, bf16_hi(y) * down};
                hi[j] = e4m3_pair(f[0], f[1]) | (e4m3_pair(f[2], f[3]) << 16);
                const uint32_t h0 = e4m3x2_to_f16x2(hi[j]), h1 = e4m3x2_to_f16x2_hi(hi[j]);
                const float2 g0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
                const float2 g1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
                lo[j] = e4m3_pair(f[0] - g0.x, f[1] - g0.y) | (e4m3_pair(f[2] - g1.x, f[3] - g1.y) << 16);
            }
            const int at = part * kCols + lane % kLanes * 8;
            uint8_t* dst = q_tile + Tc<D>::place(rr, at >> 4) + (at & 8);
            *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(dst + Tc<D>::kPiece) = make_uint2(lo[0], lo[1]);
        }
    }

    // This part's sums at `o` (tensor memory) times `by`.
    __device__ __forceinline__ void rescale(uint32_t o, float by) {
#pragma unroll 1
        for (int c = 0; c < kCols; c += 16) {
            uint32_t r[16];
            tmem_ld_16(o + c, r);
            tc_wait_ld_16(r);
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * by);
            tc_st_16(o + c, r);
        }
        tmem_wait_st();
    }

    // The part's 32 keys of a half: scores at `s` become weights at `dst`.  k0: the first key; o:
    // this part's sums, which hold something where `some`, and everything handed over so far
    // once `summed` has run.  False: one of the row group's warps has failed.
    template <class Summed>
    __device__ __forceinline__ bool step(const KvAttendArgs& a, uint32_t s, uint32_t dst, uint32_t o,
                                         const float4* scales, int k0, bool some, bool failed, int row, int part,
                                         float* shared, int pair, Summed summed) {
        uint32_t r[32];
        tmem_ld_32(s, r);
        const float4 x0 = scales[0], x1 = scales[1];
        float2 sc[2] = {make_float2(x0.x * factor, x0.y), make_float2(x1.x * factor, x1.y)};
        const int window = a.sh.window;
        const bool border = pos_first < k0 + 31 || pos_last < 0 || (window > 0 && pos_last - window >= k0);
        tc_wait_ld_32(r);
        if (border) hide(r, sc[0], sc[1], window > 0 ? pos - window + 1 - k0 : 0, pos - k0);
        // scales are positive: the largest product is the largest score's
        const float top = fmaxf(fmaf(largest(r), sc[0].x, sc[0].y), fmaf(largest(r + 16), sc[1].x, sc[1].y));
        // The maximum follows when it is behind by more than 2^8, row by row: no row's bits depend on another's.
        const bool behind = top > m + kTcHeadroom;
        tc_fence_before();
        const bool renew = pair_any(pair, behind || failed);
        tc_fence_after();
        if (renew) {
            constexpr uint32_t kFailed = 0x7fc0dead;  // no score's bits
            shared[2 * row + part] = failed ? __uint_as_float(kFailed) : top;
            pair_sync(pair);
            const float2 both = reinterpret_cast<const float2*>(shared)[row];
            if (__float_as_uint(both.x) == kFailed || __float_as_uint(both.y) == kFailed) return false;
            const float most = fmaxf(both.x, both.y);
            const float now = most > m + kTcHeadroom ? most : m, down = now == m ? 1.f : ex2(m - now);
            m = now;
            l *= down;
            if (some) {
                summed();
                rescale(o, down);
            }
        }
        const float base = m == -INFINITY ? 0.f : m - kTcWeightBits;
        uint32_t w[16];
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
            const float f = sc[gg].x, shift = sc[gg].y - base;
            const f32x2 f2 = pack2(f, f), shift2 = pack2(shift, shift);
            f32x2 sum = 0ull;
#pragma unroll
            for (int k = 16 * gg; k < 16 * gg + 16; k += 2) {
                float p0, p1;
                unpack2(fma2_of(pack2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), f2, shift2), p0, p1);
                p0 = ex2(p0);
                p1 = ex2(p1);
                sum = add2(sum, pack2(p0, p1));
                w[k / 2] = f16_pair(p0, p1);
            }
            float s0, s1;
            unpack2(sum, s0, s1);
            s0 += s1;
            if (s0 != 0.f) l = fmaf(s0, gg ? x1.z : x0.z, l);  // unseen keys leave a block's NaN scale alone
        }
        tc_st_16(dst, w);  // (scores there have been read: by the other part's warp, pair_any)
        tmem_wait_st();
        return true;
    }

    // Largest of 16 scores.
    __device__ static __forceinline__ float largest(const uint32_t* x) {
        float t = max3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
        float u = max3(__uint_as_float(x[3]), __uint_as_float(x[4]), __uint_as_float(x[5]));
#pragma unroll
        for (int i = 6; i < 14; i += 4) {
            t = max3(t, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            u = max3(u, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
        }
        t = max3(t, __uint_as_float(x[14]), __uint_as_float(x[15]));
        return fmaxf(t, u);
    }

    // 32 scores of which [lo, hi] are seen: the others to -inf.  s0, s1: the groups' factors and
    // addends, made such that -inf stays so whatever the scales are.  A group with a factor
    // that is not a number passes that on to the scores that are seen.
    __device__ static __forceinline__ void hide(uint32_t (&r)[32], float2& s0, float2& s1, int lo, int hi) {
        lo = max(lo, 0);
        hi = min(hi, 31);
        const uint32_t seen = hi < lo ? 0u : (0xffffffffu << lo) & (0xffffffffu >> (31 - hi));
        const uint32_t none = __float_as_uint(-INFINITY);
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
            float2& sc = gg ? s1 : s0;
            const bool bad = !(sc.x == sc.x) || !(sc.y == sc.y);
            sc = bad ? make_float2(1.f, 0.f) : make_float2(fmaxf(sc.x, 0x1p-126f), sc.y);
#pragma unroll
            for (int i = 16 * gg; i < 16 * gg + 16; ++i) {
                if (bad) r[i] = 0x7fffffffu;
                r[i] = seen & (1u << i) ? r[i] : none;
            }
        }
    }

    // This part's sums (tensor memory `o`) to the output row, or to the CTA's part of it, 64
    // bytes a row at a time through shared memory (`stage`, 2 KB a warp), so that an instruction
    // writes 8 rows' pieces and not 16 bytes of 32.
    __device__ __forceinline__ void finish(const KvAttendArgs& a, const KvWork& work, const TcWalk& walk, int t, int row,
                                           int part, uint32_t o, float* shared, int pair, uint8_t* stage) {
        const int lane = threadIdx.x & 31;
        shared[2 * row + part] = l;
        pair_sync(pair);
        const float2 both = reinterpret_cast<const float2*>(shared)[row];
        const KvPlace& p = walk.at;
        const bool whole = walk.whole();
        KvParts parts{0, 1, true};
        if (!whole) parts = kv_parts(work, p, walk.first);
        const int group = a.sh.group, rows = p.s.n * group, in_tile = t * kTcTile + row;
        const TcRows of(a, p, p.rt * a.sh.rows + in_tile - lane);  // the warp's rows
        const int r0 = of.r0;
        const float down = 0x1p-6f, sum = (both.x + both.y) * down;
        const float by = !whole ? down : sum == 0.f ? 0.f : __fdiv_rn(down, sum);
        const int cols = whole ? 32 : 16;  // channels of 64 bytes
#pragma unroll 1
        for (int c = 0; c < kCols; c += cols) {
            uint32_t v[16];
            if (whole) {
                uint32_t x[32];
                tmem_ld_32(o + c, x);
                tc_wait_ld_32(x);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[i] = bf16_pair(__uint_as_float(x[2 * i]) * by, __uint_as_float(x[2 * i + 1]) * by);
            } else {
                tmem_ld_16(o + c, v);
                tc_wait_ld_16(v);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * by);
            }
            auto place = [&](int r, int q) { return reinterpret_cast<uint4*>(stage + r * 64 + ((q ^ (r >> 1 & 3)) << 4)); };
            __syncwarp();  // the previous piece has been read
#pragma unroll
            for (int q = 0; q < 4; ++q) *place(lane, q) = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rr = i * 8 + (lane >> 2), q = lane & 3, col = part * kCols + c;
                if (r0 + rr >= rows) continue;
                uint8_t* dst = whole ? reinterpret_cast<uint8_t*>(a.out + of.out_row(rr) * D + col)
                                     : reinterpret_cast<uint8_t*>(
                                           a.part_o + ((size_t)parts.slot * a.sh.rows + in_tile - lane + rr) * D + col);
                reinterpret_cast<uint4*>(dst)[q] = *place(rr, q);
            }
        }
        if (!valid || part != 0) return;
        const int64_t at = of.out_row(lane);
        if (!whole)
            a.part_ml[(size_t)parts.slot * a.sh.rows + in_tile] = make_float2(m, sum);
        else if (a.lse != nullptr)
            a.lse[at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
        if (parts.leader) a.info[at] = make_int2(parts.slot, parts.parts * 256 + in_tile);
    }
};

template <int D>
__device__ __forceinline__ void tc_softmax(const KvAttendArgs& a, const KvWork& work, uint8_t* smem, const TcBars& bar,
                                           uint32_t tmem, const WaitCtl& ctl) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = warp >> 3, part = warp >> 2 & 1, row = (warp & 3) * 32 + lane, pair = 1 + t * 4 + (warp & 3);
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s = lanes + t * kTcTile, o = lanes + 2 * kTcTile + t * kTcTile + part * (D / 2);
    uint8_t* q_tile = smem + t * 2 * Tc<D>::kPiece;
    uint8_t* stage = smem + Tc<D>::kOffStage + warp * 2048;
    float* shared = reinterpret_cast<float*>(smem + Tc<D>::kOffShared) + t * 2 * kTcTile;  // [row][part]
    constexpr int kUse = 4 * kTcTile;  // each of its three uses has a place of its own
    TcRing v;
    uint32_t s_phase = 0;  // steps
    bool failed = false;   // a wait gave up
    bool passed = false;   // over a row tile without rows of this tile
    TcRow<D> mine;
    TcWalk walk(work);
    auto start = [&](TcRow<D>& r, const TcWalk& w) {
        if (!w.more() || t >= w.tiles(a)) return;
        r.start(a, w.at, t, row, part, q_tile, reinterpret_cast<uint32_t*>(shared + kUse), pair);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.q_full[t]);
    };
    start(mine, walk);
    while (walk.more()) {
        TcWalk next = walk;
        if (t >= walk.tiles(a)) {
            for (int j = 0; j < walk.n; ++j) v.step(kTcVS);
            passed = true;
            next.next(a);
            start(mine, next);
            walk = next;
            continue;
        }
        // Steps passed over have not been waited for here, but by the scores' issuer: with the first
        // scores it is known that the stage's fill before this one is done, whose end has the parity
        // that the wait below would take for this one's.  (v_full always waited for behind the
        // step's scores: the prompt 2 % slower.)
        if (passed) failed = !tc_wait(&bar.s_full[2 * t], s_phase, ctl) || failed;
        passed = false;
        for (int j = 0; j < walk.n; ++j) {
            failed = !tc_wait(&bar.v_full[v.stage], v.phase, ctl) || failed;  // its scales
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                failed = !tc_wait(&bar.s_full[2 * t + h], s_phase, ctl) || failed;
                tc_fence_after();
                const float4* scales =
                    reinterpret_cast<const float4*>(smem + Tc<D>::kOffScales) + 8 * v.stage + 4 * h + 2 * part;
                const bool ok = mine.step(
                    a, s + h * kTcHalf + 32 * part, s + h * kTcHalf + 16 * part, o, scales,
                    (walk.at.unit + j) * kTcTile + h * kTcHalf + 32 * part, j + h > 0, failed, row, part, shared, pair,
                    [&] {  // the half before, and with it all others
                        failed = !tc_wait(&bar.pv_done[2 * t + (h ^ 1)], h ? s_phase : s_phase ^ 1u, ctl) || failed;
                        tc_fence_after();
                    });
                if (!ok) return;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[2 * t + h]);
            }
            v.step(kTcVS);
            s_phase ^= 1u;
        }
        // the last scores are there, so the queries have been read: the next row tile's
        // take their place while the last product runs
        TcRow<D> after = mine;
        next.next(a);
        start(after, next);
        failed = !tc_wait(&bar.pv_done[2 * t + 1], s_phase ^ 1u, ctl) || failed;
        tc_fence_after();
        mine.finish(a, work, walk, t, row, part, o, shared + 2 * kUse, pair, stage);
        tc_fence_before();
        mine = after;
        walk = next;
    }
}

// ------------------------------------------------------------------ values
// WINDOW: the call has a window; values before it become 0, as those behind the sequence (a weight
// of 0 does not undo a NaN).  A kernel of its own, as the bound costs the others 4 to 7 % of a
// prompt (registers).
template <int D, bool WINDOW>
__device__ __forceinline__ void tc_values(const KvAttendArgs& a, const KvWork& work, uint8_t* smem, const TcBars& bar,
                                          const WaitCtl& ctl) {
    constexpr int kPerRow = D / 16, kRows = 128 / kPerRow, kPasses = kTcTile / kRows;  // rows of a pass
    const int tid = threadIdx.x - 32 * kTcValues0, lane = tid & 31;
    // A lane's 16 channels and key of a pass: 8 lanes that store together have two keys
    // and pieces 0, 2, 4, 6 of 128 bytes, which the swizzle puts into all banks.
    const int c = D == 128 ? (lane & 3) | (lane >> 1 & 4) : lane & 3;
    const int row = (tid >> 5) * (kRows / 4) + (D == 128 ? (lane >> 2 & 1) | (lane >> 3 & 2) : lane >> 2);
    uint4 w[kPasses];
    float ks = 0.f, vs = 0.f;
    TcWalk walk(work);
    int j = 0;  // the step whose codes are loaded next
    bool more = walk.more();
    // the pages of that step, 16 keys a lane of the first eight
    int ids = more ? tc_page(a, walk.at, walk.at.unit * kTcTile, lane & 7) : -1;
    auto load = [&] {
        const KvPlace& p = walk.at;
        const int k0 = (p.unit + j) * kTcTile, keys = p.s.len - k0;  // keys of the step that are there
        const int id = ids;
        const int from = WINDOW ? kv_first_key(p.s, a.sh, p.rt) - k0 : 0;
        const bool there = (unsigned)id < (unsigned)a.c.n_pages && (!WINDOW || 16 * (lane & 7) + 16 > from);
        // where this lane's group begins (a page that is not there: nothing)
        const int in_page = (16 * (lane & 7)) & (a.c.page - 1);
        const uint8_t* group = a.c.v + (there ? id * a.c.page_stride + ((p.head << a.c.page_bits) + in_page) * D : 0);
        const uint32_t lo = (uint32_t)reinterpret_cast<uintptr_t>(group),
                       hi = (uint32_t)(reinterpret_cast<uintptr_t>(group) >> 32);
        const uint32_t ok = __ballot_sync(0xffffffffu, there);
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int key = i * kRows + row, g = D == 128 ? i : key >> 4;
            const uint64_t at = (uint64_t)__shfl_sync(0xffffffffu, hi, g) << 32 | __shfl_sync(0xffffffffu, lo, g);
            w[i] = make_uint4(0, 0, 0, 0);
            if ((ok >> g & 1) && key < keys && (!WINDOW || key >= from))
                w[i] = __ldcg(reinterpret_cast<const uint4*>(at + ((key & 15) * D + c * 16)));
        }
        ks = 1.f;
        vs = 0.f;
        if (there && lane < 8) {
            ks = a.c.k_scale[id * a.c.scale_stride + p.head];
            vs = a.c.v_scale[id * a.c.scale_stride + p.head];
        }
        if (++j == walk.n) {
            walk.next(a);
            j = 0;
        }
        more = walk.more();
        if (more) ids = tc_page(a, walk.at, (walk.at.unit + j) * kTcTile, lane & 7);
    };
    if (!more) return;
    load();
    TcRing v;
    for (bool last = false; !last;) {
        last = !more;
        if (!tc_wait(&bar.v_empty[v.stage], v.phase ^ 1u, ctl)) return;
        uint8_t* dst = smem + Tc<D>::kOffV + v.stage * Tc<D>::kValues;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int key = i * kRows + row;
            const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h[2 * k] = e4m3x2_to_f16x2(x[k]);
                h[2 * k + 1] = e4m3x2_to_f16x2_hi(x[k]);
            }
            *reinterpret_cast<uint4*>(dst + Tc<D>::place_value(key, 2 * c)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(dst + Tc<D>::place_value(key, 2 * c + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        if (tid < 8) {
            float lg, inv;
            value_scale(vs, lg, inv);
            reinterpret_cast<float4*>(smem + Tc<D>::kOffScales)[8 * v.stage + tid] =
                make_float4(finite_scale(ks), lg, inv, 0.f);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.v_full[v.stage]);
        v.step(kTcVS);
        if (more) load();
    }
}

// ------------------------------------------------------------------ keys
template <int D>
__device__ __forceinline__ void tc_keys(const KvAttendArgs& a, const KvWork& work, uint8_t* smem, const TcBars& bar,
                                        const CUtensorMap* map, int no_page, const WaitCtl& ctl) {
    const int lane = threadIdx.x & 31, boxes = kTcTile / a.c.page, groups = a.c.page / 16;
    int ok = 1;
    if (lane == 0) ok = !a.stall || mbar_wait(bar.stall, 0, ctl);  // the test hook's wait runs out
    ok = __shfl_sync(0xffffffffu, ok, 0);
    TcRing k;
    uint32_t it = 0;
    TcWalk walk(work);
    int id = walk.more() && lane < boxes ? tc_page(a, walk.at, walk.at.unit * kTcTile, lane * groups) : -1;
    for (; ok && walk.more(); walk.next(a)) {
        for (int j = 0; j < walk.n; ++j, ++it) {
            if (j == 0 && it != 0 && lane < boxes) id = tc_page(a, walk.at, walk.at.unit * kTcTile, lane * groups);
            // a page that is not there is read as one behind the last: zeros
            // (bad pages are reported here, the values' warps having no register for it: 7 % of a prompt's time)
            const bool there = (unsigned)id < (unsigned)a.c.n_pages;
            const int page = there ? id : no_page, from = (walk.at.unit + j) * kTcTile + lane * a.c.page;
            if (!there && lane < boxes && from < walk.at.s.len &&
                from + a.c.page > kv_first_key(walk.at.s, a.sh, walk.at.rt))
                atomicOr(a.error, kErrDevice);
            if (lane < boxes && j + 1 < walk.n) id = tc_page(a, walk.at, (walk.at.unit + j + 1) * kTcTile, lane * groups);
            if (lane == 0) {
                ok = mbar_wait(&bar.k_empty[k.stage], k.phase ^ 1u, ctl);
                if (ok) mbar_arrive_expect_tx(&bar.k_full[k.stage], Tc<D>::kPiece);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (lane < boxes)
                tma_load_3d(smem + Tc<D>::kOffK + k.stage * Tc<D>::kPiece + lane * a.c.page * D, map,
                            &bar.k_full[k.stage], 0, walk.at.head * a.c.page, page);
            k.step(kTcKS);
        }
        if (!ok) break;
    }
    // drain: every copy issued must land before the CTA may exit
    if (lane == 0)
        for (uint32_t st = 0; st < (uint32_t)kTcKS && st < it; ++st) {
            const uint32_t last = it - 1 - ((it - 1 - st) % kTcKS);
            mbar_wait_drain(&bar.k_full[st], (last / kTcKS) & 1u);
        }
}

// ------------------------------------------------------------------ products
// The MMAs' operands are constants but for the low words of the descriptors, and one lane
// of the whole warp issues under a predicate, without a branch: what an MMA takes stays in
// uniform registers.  (64-bit descriptors in a branch of lane 0 cost 100 clocks an MMA,
// which itself is 64.)  The tensor memory's address is 0: the CTA has all of it.
#define TC_SCORE_MMA(A, B, ACC)                                                              \
    "add.u32 x, %1, " #A ";\n\tmov.b64 a, {x, %4};\n\tadd.u32 x, %2, " #B                    \
    ";\n\tmov.b64 b, {x, %4};\n\t@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, " #ACC ";\n\t"
// S = Q1 K^T + Q2 K^T of 64 keys at column `d`: 32 bytes of channels an MMA; q, k: low words
// of the descriptors; the second part is a tile's bytes on.
template <int D>
__device__ __forceinline__ void tc_mma_scores(uint32_t d, uint32_t q, uint32_t k, uint32_t hi) {
    if constexpr (D == 128)
        asm volatile(
            "{\n\t.reg .pred e, n, t;\n\t.reg .b64 a, b;\n\t.reg .b32 x;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 n, %3, %3;\n\tsetp.eq.b32 t, %3, %3;\n\t"
            TC_SCORE_MMA(0, 0, n) TC_SCORE_MMA(2, 2, t) TC_SCORE_MMA(4, 4, t) TC_SCORE_MMA(6, 6, t)
            TC_SCORE_MMA(1024, 0, t) TC_SCORE_MMA(1026, 2, t) TC_SCORE_MMA(1028, 4, t) TC_SCORE_MMA(1030, 6, t)
            "}" ::"r"(d), "r"(q), "r"(k), "r"(idesc_e4m3(kTcTile, kTcHalf)), "r"(hi) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred e, n, t;\n\t.reg .b64 a, b;\n\t.reg .b32 x;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 n, %3, %3;\n\tsetp.eq.b32 t, %3, %3;\n\t"
            TC_SCORE_MMA(0, 0, n) TC_SCORE_MMA(2, 2, t) TC_SCORE_MMA(512, 0, t) TC_SCORE_MMA(514, 2, t)
            "}" ::"r"(d), "r"(q), "r"(k), "r"(idesc_e4m3(kTcTile, kTcHalf)), "r"(hi) : "memory");
}
static_assert(kTcTile * 128 / 16 == 1024 && kTcTile * 64 / 16 == 512, "a tile's bytes in the descriptors' units");

#define TC_VALUE_MMA(A, B, ACC)                                                                  \
    "add.u32 x, %2, " #B ";\n\tmov.b64 b, {x, %4};\n\tadd.u32 y, %1, " #A                        \
    ";\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [y], b, %3, " #ACC ";\n\t"
// O (+)= P V of 64 keys at column `d`: 16 keys an MMA, 8 columns of weights and 2 KB of values.
template <int D>
__device__ __forceinline__ void tc_mma_values(uint32_t d, uint32_t p, uint32_t v, uint32_t hi, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, n, t;\n\t.reg .b64 b;\n\t.reg .b32 x, y;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 n, %5, 0;\n\tsetp.eq.b32 t, %3, %3;\n\t"
        TC_VALUE_MMA(0, 0, n) TC_VALUE_MMA(8, 128, t) TC_VALUE_MMA(16, 256, t) TC_VALUE_MMA(24, 384, t)
        "}" ::"r"(d), "r"(p), "r"(v), "r"(idesc_f16_f32(kTcTile, D) | (1u << 16)),  // values: channels contiguous
        "r"(hi), "r"(accumulate) : "memory");
}
// Arrives on `bar` when the MMAs issued so far are done.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// A warp a tile.  A step is two halves of 64 keys, each with a buffer of its own for its
// scores, whose place the weights take: the scores of a half are asked for before the
// weights of the half before are there, so that the softmax finds them done.  (With one
// buffer a step of 128 keys was a chain of scores, softmax and weighted values, 4800
// clocks; one warp for both tiles was no different.)
// The ring of values needs no wait of its own: the softmax has waited for the stage before
// it hands over the weights.
template <int D>
__device__ __forceinline__ void tc_products(const KvAttendArgs& a, const KvWork& work, uint8_t* smem,
                                            const TcBars& bar, int t, const WaitCtl& ctl) {
    const uint64_t q_desc = Tc<D>::desc(smem_u32(smem)), v_desc = Tc<D>::desc_values(smem_u32(smem) + Tc<D>::kOffV);
    const uint32_t q0 = (uint32_t)q_desc + t * 2 * (Tc<D>::kPiece >> 4), k0 = (uint32_t)q_desc + (Tc<D>::kOffK >> 4);
    const uint32_t v0 = (uint32_t)v_desc;
    const int lane = threadIdx.x & 31;
    TcRing k, v;
    uint32_t q_phase = 0, p_phase = 0;  // row tiles; steps
    uint32_t done[2] = {0, 0};          // weighted halves issued
    auto scores = [&](int half) {
        tc_fence_after();
        tc_mma_scores<D>(t * kTcTile + half * kTcHalf, q0,
                         k0 + k.stage * (Tc<D>::kPiece >> 4) + half * (Tc<D>::kPiece >> 5), (uint32_t)(q_desc >> 32));
        tc_commit(&bar.s_full[2 * t + half]);
        if (half == 1) {
            tc_commit(&bar.k_empty[k.stage]);
            k.step(kTcKS);
        }
    };
    auto weighted = [&](int half, bool some) {
        if (!tc_wait(&bar.p_full[2 * t + half], p_phase, ctl)) return false;
        tc_fence_after();
        tc_mma_values<D>(2 * kTcTile + t * kTcTile, t * kTcTile + half * kTcHalf,
                         v0 + v.stage * (Tc<D>::kValues >> 4) + half * (kTcHalf * 128 >> 4), (uint32_t)(v_desc >> 32),
                         some ? 1u : 0u);
        tc_commit(&bar.pv_done[2 * t + half]);
        ++done[half];
        if (half == 1) {
            tc_commit(&bar.v_empty[v.stage]);
            v.step(kTcVS);
            p_phase ^= 1u;
        }
        return true;
    };
    // the weights in a half's buffer have been read.  (A barrier a half: with one for both, the
    // wait for the second could take the end of the one before the first for it.)
    auto free_buffer = [&](int half) {
        return done[half] == 0 || tc_wait(&bar.pv_done[2 * t + half], (done[half] - 1) & 1u, ctl);
    };
    bool ok = true;
    for (TcWalk walk(work); ok && walk.more(); walk.next(a)) {
        if (t >= walk.tiles(a)) {  // no rows: the other tile's stages are free as far as this one goes
            for (int j = 0; ok && j < walk.n; ++j) {
                ok = tc_wait(&bar.k_full[k.stage], k.phase, ctl) && tc_wait(&bar.v_full[v.stage], v.phase, ctl);
                if (ok && lane == 0) {
                    mbar_arrive(&bar.k_empty[k.stage]);
                    mbar_arrive(&bar.v_empty[v.stage]);
                }
                k.step(kTcKS);
                v.step(kTcVS);
            }
            continue;
        }
        ok = tc_wait(&bar.q_full[t], q_phase, ctl) && tc_wait(&bar.k_full[k.stage], k.phase, ctl) &&
             free_buffer(0) && free_buffer(1);
        q_phase ^= 1u;
        if (!ok) break;
        scores(0);
        scores(1);
        ok = weighted(0, false);
        for (int j = 1; ok && j < walk.n; ++j) {
            ok = tc_wait(&bar.k_full[k.stage], k.phase, ctl) && free_buffer(0);
            if (!ok) break;
            scores(0);
            ok = weighted(1, true) && free_buffer(1);
            if (!ok) break;
            scores(1);
            ok = weighted(0, true);
        }
        ok = ok && weighted(1, true);
    }
    tc_commit(&bar.teardown[t]);
    if (lane == 0) mbar_wait_drain(&bar.teardown[t], 0);
}

template <int D, bool WINDOW>
__global__ void __launch_bounds__(kTcThreads, 1)
    kv_attend_kernel(const __grid_constant__ CUtensorMap keys, const KvAttendArgs a, int no_page) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((smem_u32(smem) & 1023u) != 0u) {
        if (threadIdx.x == 0) atomicOr(a.error, kErrDevice);
        return;
    }
    const TcBars bar(smem + Tc<D>::kOffBars);
    KvWork* work = reinterpret_cast<KvWork*>(smem + Tc<D>::kOffWork);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Tc<D>::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Tc<D>::kOffMisc + 8);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bar.q_full[t], 8);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&bar.s_full[2 * t + h], 1);
                mbar_init(&bar.p_full[2 * t + h], 8);
                mbar_init(&bar.pv_done[2 * t + h], 1);
            }
            mbar_init(&bar.teardown[t], 1);
        }
        for (int i = 0; i < kTcKS; ++i) {
            mbar_init(&bar.k_full[i], 1);
            mbar_init(&bar.k_empty[i], 2);
        }
        for (int i = 0; i < kTcVS; ++i) {
            mbar_init(&bar.v_full[i], 4);
            mbar_init(&bar.v_empty[i], 2);
        }
        mbar_init(bar.stall, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&keys);
    }
    if (warp == kTcProducts0) {
        tmem_alloc(tmem_slot, kTcCols);
        tmem_relinquish();
    }
    pdl_wait();
    if (warp == kTcProducts0) pdl_trigger();  // not before the tensor memory is this CTA's
    kv_find_work<kTcThreads>(a, gridDim.x, 1, work, reinterpret_cast<int64_t*>(smem + Tc<D>::kOffMisc + 64));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl ctl{abort_flag, a.error, a.timeout_ns, 0u};
    if (tmem != 0u && threadIdx.x == 0) atomicOr(a.error, kErrDevice);  // all columns begin at 0
    if (work->u1 > work->u0 && tmem == 0u) {
        if (warp < kTcValues0)
            tc_softmax<D>(a, *work, smem, bar, tmem, ctl);
        else if (warp < kTcKeys0)
            tc_values<D, WINDOW>(a, *work, smem, bar, ctl);
        else if (warp == kTcKeys0)
            tc_keys<D>(a, *work, smem, bar, &keys, no_page, ctl);
        else if (warp < kTcProducts0 + 2)
            tc_products<D>(a, *work, smem, bar, warp - kTcProducts0, ctl);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kTcProducts0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTcCols);
    }
}

template <int D, bool WINDOW>
cudaError_t launch_tc(const KvAttendArgs& a, cudaStream_t st, bool pdl) {
    auto kern = kv_attend_kernel<D, WINDOW>;
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [&] {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D>::kSmem);
    });
    if (err != cudaSuccess) return err;
    CUtensorMap keys;
    const int pages = a.c.n_pages > 0 ? a.c.n_pages : 1;
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.c.heads * a.c.page, (uint64_t)pages};
    const uint64_t strides[2] = {(uint64_t)D, (uint64_t)a.c.page_stride};
    const uint32_t box[3] = {(uint32_t)D, (uint32_t)a.c.page, 1};
    if (!make_tensor_map_3d(&keys, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.c.k, dims, strides, box,
                            D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    return launch_kernel(kern, dim3(kv_tc_ctas()), dim3(kTcThreads), Tc<D>::kSmem, st, pdl, keys, a, pages);
}

}  // namespace

int kv_tc_ctas() { return num_sms(); }

cudaError_t launch_kv_attend(KvAttendArgs a, cudaStream_t st, bool pdl) {
    a.sh.rows = kKvRows;
    a.sh.tokens = kTcTile;
    a.sh.extra = kTcExtra;
    a.slots = 2 * kv_tc_ctas();
    const bool d64 = a.c.dim == 64;
    const cudaError_t e = a.sh.window > 0 ? (d64 ? launch_tc<64, true>(a, st, pdl) : launch_tc<128, true>(a, st, pdl))
                                          : (d64 ? launch_tc<64, false>(a, st, pdl) : launch_tc<128, false>(a, st, pdl));
    return e != cudaSuccess ? e : launch_kv_join(a, st, pdl);
}

}  // namespace moe
