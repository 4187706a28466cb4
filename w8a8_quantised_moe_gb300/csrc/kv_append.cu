// kv_append.cu -- new tokens' keys and values into the pages of the cache, keys and
// queries turned by their positions on the way:
//
//   half-split pairs (i, i + R/2), neighbours (2 i, 2 i + 1):
//     a' = a cos - b sin,  b' = b cos + a sin     (R rotated channels, then the rest)
//   block (page, head): s = 2^E, E the least integer >= -64 with max |value| <= 448 2^E
//     code = E4M3 nearest to value / s, ties to the even mantissa
//   a page that holds tokens already: s' = max(s, the new tokens' s); where s' > s its
//     codes are rounded again, E4M3(code s / s')
//   a token at a position behind its sequence's pages, or the table of angles: left out, reported
//
// A power of two costs nothing: E4M3 keeps the same relative precision at any scale,
// quotients by it are exact, and rounding codes again is exact but for subnormals, so
// that tokens that come one at a time and a whole prompt lead to nearly the same cache.
// The turned keys keep what lies below their binary32 value in its last bit (rounding
// to odd), so that the codes are those of the exact products with the table's values:
// about 1 in 10^6 would differ by a step otherwise.
//
// Bound by HBM for a prompt (16-bit rows in, 8-bit pages and turned queries out), by
// the latency of the lengths, the rows and the page's scale for single tokens.  A task is
// one page run (the new tokens of one page), head and K or V: W warps hold its values, two
// units of 16 a thread, so that they are read and turned once.  (64 registers, for four blocks
// an SM: the compiler spills 160 to 240 bytes a thread.)  8192 tokens, 32 query and 8 key heads
// of 128 channels (189 MB): 48 us, 0.58 of the copy's rate: each block has a chain of
// dependent loads (lengths, rows, page), which four blocks an SM do not cover.  Measured on
// the way: eight warps a task and its page looked up first 83; queries two units in flight,
// three blocks an SM 64; four blocks 58; the page not waited for before the rows 55; the
// runs' sequences from a sum over the batch in each block 51.  Pages of 16 tokens: 99 with
// eight warps a task, 57 with two.  64 single tokens: 4.7 us (5.0 with that sum).
#include "block_dev.cuh"
#include "kv_dev.cuh"

namespace moe {
namespace {

constexpr int kApThreads = 256;

// v rounded to odd: v is binary32, rest what lies between it and the exact value.
__device__ __forceinline__ float to_odd(float v, float rest) {
    const float hi = __fadd_rn(v, rest), lo = __fsub_rn(rest, __fsub_rn(hi, v));
    uint32_t bits = __float_as_uint(hi);
    if (lo != 0.f && !(bits & 1u)) bits += (lo > 0.f) == (hi > 0.f) ? 1u : ~0u;
    return __uint_as_float(bits);
}
// a c + b s: exact products, their sum and what it leaves, rounded to odd.
__device__ __forceinline__ float turn_odd(float a, float c, float b, float s) {
    const float p = __fmul_rn(a, c), pe = fmaf(a, c, -p), w = __fmul_rn(b, s), we = fmaf(b, s, -w);
    const float sum = __fadd_rn(p, w), bb = __fsub_rn(sum, p);
    const float t = __fadd_rn(__fsub_rn(p, __fsub_rn(sum, bb)), __fsub_rn(w, bb));
    return to_odd(sum, __fadd_rn(t, __fadd_rn(pe, we)));
}
__device__ __forceinline__ float turn_rn(float a, float c, float b, float s) { return fmaf(a, c, __fmul_rn(b, s)); }

// 16 channels of a row that are turned together (or not at all): the two runs of 8.
struct Unit {
    int c0, c1, angle;  // first channels of the runs; first angle, or -1
    bool pairs;
    __device__ __forceinline__ Unit(int u, int rope_dim, int interleaved) {
        const int turned = rope_dim / 16;
        pairs = interleaved != 0;
        angle = u < turned ? 8 * u : -1;
        if (u < turned && !pairs) {
            c0 = 8 * u;
            c1 = rope_dim / 2 + 8 * u;
        } else {
            c0 = 16 * u;
            c1 = c0 + 8;
        }
    }
};

template <bool ODD>
__device__ __forceinline__ void turn_unit(float (&f)[16], const Unit& u, const float* row, int half) {
    const float4* pc = reinterpret_cast<const float4*>(row + u.angle);
    const float4* ps = reinterpret_cast<const float4*>(row + half + u.angle);
    const float4 c0 = pc[0], c1 = pc[1], s0 = ps[0], s1 = ps[1];
    const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    auto turn = [&](float& a, float& b, int i) {
        const float x = ODD ? turn_odd(a, c[i], -b, s[i]) : turn_rn(a, c[i], -b, s[i]);
        const float y = ODD ? turn_odd(b, c[i], a, s[i]) : turn_rn(b, c[i], a, s[i]);
        a = x;
        b = y;
    };
    if (u.pairs) {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn(f[2 * i], f[2 * i + 1], i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn(f[i], f[8 + i], i);
    }
}

__device__ __forceinline__ void load16(const uint16_t* row, const Unit& u, float (&f)[16]) {
    float lo[8], hi[8];
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(row + u.c0), lo);
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(row + u.c1), hi);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[i] = lo[i];
        f[8 + i] = hi[i];
    }
}

// The scale of a block whose largest magnitude is amax; NaN where that is not finite.
__device__ __forceinline__ float pow2_scale(float amax) {
    const uint32_t b = __float_as_uint(amax);
    if (b >= 0x7f800000u) return __uint_as_float(0x7fffffffu);
    int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
    if (e < -64) e = -64;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Codes of 4 values over the scale 1 / inv; inv 0 (a scale that is not finite): codes 0.
__device__ __forceinline__ uint32_t codes4(const float* f, float inv) {
    if (inv == 0.f) return 0u;
    return e4m3_pair(f[0] * inv, f[1] * inv) | (e4m3_pair(f[2] * inv, f[3] * inv) << 16);
}

// One E4M3 code times `ratio`, rounded to E4M3.
__device__ __forceinline__ uint32_t requant4(uint32_t w, float ratio) {
    const uint32_t lo = e4m3x2_to_f16x2(w), hi = e4m3x2_to_f16x2_hi(w);
    float f[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2 h = *reinterpret_cast<const __half2*>(i == 0 ? &lo : &hi);
        f[2 * i] = __low2float(h) * ratio;
        f[2 * i + 1] = __high2float(h) * ratio;
    }
    return e4m3_pair(f[0], f[1]) | (e4m3_pair(f[2], f[3]) << 16);
}

// Queries: the block's tokens [t0, t1), every head; two units of a thread in flight (four: 2 us
// more for a prompt of 8192 tokens).
constexpr int kApTokens = 16;  // of such a block, at most
__device__ __forceinline__ void turn_queries(const KvAppendArgs& a, int t0, int t1, int* pos) {
    // the tokens' positions; -1: none to turn
    if ((int)threadIdx.x < t1 - t0) {
        const int t = t0 + threadIdx.x;
        int lo = 0, hi = a.bt.B;  // the entries of q_start[1..B] that are not above t
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (a.bt.q_start[mid + 1] <= t) lo = mid + 1;
            else hi = mid;
        }
        int p = -1;
        if (lo < a.bt.B) {  // else a row behind the last sequence
            int over;
            const KvSeq s = kv_seq_stored(a.bt, lo, a.c.page, over);
            if (t >= s.q0 && t < s.q0 + s.n) p = s.len - s.n + t - s.q0;
        }
        if (a.rope_dim > 0 && p >= a.rope_rows) {
            atomicOr(a.error, kErrDevice);
            p = -1;
        }
        pos[threadIdx.x] = p;
    }
    __syncthreads();
    const int D = a.c.dim, upr = D / 16, bits = D == 128 ? 3 : 2, units = a.q_heads * upr, all = (t1 - t0) * units;
    constexpr int kFlight = 2;
    for (int i0 = threadIdx.x; i0 < all; i0 += kFlight * kApThreads) {
        uint4 w[kFlight][2];
        int p[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            const int i = i0 + k * kApThreads, tok = i / units;
            p[k] = i < all ? pos[tok] : -1;
            const uint16_t* row = a.q + (t0 + tok) * a.q_stride + ((i - tok * units) >> bits) * D;
            const Unit u(i & (upr - 1), a.rope_dim, a.interleaved);
            if (p[k] >= 0) {
                w[k][0] = *reinterpret_cast<const uint4*>(row + u.c0);
                w[k][1] = *reinterpret_cast<const uint4*>(row + u.c1);
            }
        }
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            if (p[k] < 0) continue;
            const int i = i0 + k * kApThreads, tok = i / units;
            const Unit u(i & (upr - 1), a.rope_dim, a.interleaved);
            float lo[8], hi[8], x[16];
            bf16x8_to_f32(w[k][0], lo);
            bf16x8_to_f32(w[k][1], hi);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = lo[j];
                x[8 + j] = hi[j];
            }
            if (u.angle >= 0) turn_unit<false>(x, u, a.rope + (size_t)p[k] * a.rope_dim, a.rope_dim / 2);
            uint16_t* out = a.q_out + (size_t)(t0 + tok) * a.q_heads * D + ((i - tok * units) >> bits) * D;
            *reinterpret_cast<uint4*>(out + u.c0) =
                make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
            *reinterpret_cast<uint4*>(out + u.c1) = make_uint4(
                bf16_pair(x[8], x[9]), bf16_pair(x[10], x[11]), bf16_pair(x[12], x[13]), bf16_pair(x[14], x[15]));
        }
    }
}

// W: warps of a task (1, 2, 4 or 8; 8 / W tasks of a run a block).  NU: units that a thread
// holds in registers; the others (a page with many new tokens where few were expected, the
// second half of one of 128 tokens) are read twice.
template <int W, int NU>
__global__ void __launch_bounds__(kApThreads, 4) kv_append_kernel(const KvAppendArgs a) {
    __shared__ int pos[kApTokens];
    __shared__ float amax_s[kApThreads / 32];
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x >= a.store_blocks) {
        const int t0 = ((int)blockIdx.x - a.store_blocks) * a.q_tokens;
        turn_queries(a, t0, kv_min(t0 + a.q_tokens, a.bt.T), pos);
        return;
    }
    const int slot = blockIdx.x / a.task_blocks, P = a.c.page, D = a.c.dim;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the slot's sequence, found by each warp for itself, 32 candidates at once
    int seq = 0;
    for (int span = a.bt.B; span > 1;) {
        const int step = (span + 31) / 32, i = lane * step;
        const bool begun = i < span && kv_first_slot(a.bt, seq + i, P, a.by_token) <= slot;
        const uint32_t all = __ballot_sync(0xffffffffu, begun);
        const int last = all == 0 ? 0 : 31 - __clz(all);
        seq += last * step;
        span = kv_min(step, span - last * step);
    }
    int over;
    const KvSeq s = kv_seq_stored(a.bt, seq, P, over);
    const int run = slot - kv_first_slot(a.bt, seq, P, a.by_token);
    if (over > 0 && run == 0 && threadIdx.x == 0) atomicOr(a.error, kErrDevice);  // no pages for them
    const int page = kv_slot_page(s, run, P, a.by_token);
    if (page < 0) return;
    // positions [lo, hi) of the page are new; those before lo are held already
    int lo = kv_max(page * P, kv_max(s.len - s.n, 0)), hi = kv_min(page * P + P, s.len);
    const int held = lo - page * P;
    if (a.rope_dim > 0 && hi > a.rope_rows) {
        if (threadIdx.x == 0) atomicOr(a.error, kErrDevice);
        hi = a.rope_rows;
    }
    const int id = a.bt.page_table[seq * a.bt.table_stride + page];  // not waited for before the rows are there
    const int task = (blockIdx.x % a.task_blocks) * (8 / W) + warp / W;
    // the warps of a task end as one, so that they meet at their barriers
    if (task >= 2 * a.c.heads || hi <= lo) return;
    const bool keys = task < a.c.heads;
    const int head = keys ? task : task - a.c.heads;
    const int upr = D / 16, bits = D == 128 ? 3 : 2, units = (hi - lo) * upr;
    const int tid = (int)threadIdx.x & (32 * W - 1);
    const int64_t stride = keys ? a.k_stride : a.v_stride;
    const int rope_dim = keys ? a.rope_dim : 0;
    const uint16_t* in = (keys ? a.k : a.v) + (int64_t)(s.q0 + lo - (s.len - s.n)) * stride + head * D;

    auto load = [&](int i, float(&f)[16]) {
        const int r = i >> bits;
        const Unit u(i & (upr - 1), rope_dim, a.interleaved);
        load16(in + r * stride, u, f);
        if (u.angle >= 0) turn_unit<true>(f, u, a.rope + (size_t)(lo + r) * a.rope_dim, a.rope_dim / 2);
    };
    float held_f[NU][16];
    float amax = 0.f;
    auto largest = [&](const float(&f)[16]) {
#pragma unroll
        for (int j = 0; j < 16; ++j) amax = amax_nan(amax, f[j]);
    };
#pragma unroll
    for (int k = 0; k < NU; ++k) {
        const int i = tid + k * 32 * W;
        if (i < units) {
            load(i, held_f[k]);
            largest(held_f[k]);
        }
    }
    for (int i = tid + NU * 32 * W; i < units; i += 32 * W) {
        float f[16];
        load(i, f);
        largest(f);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = amax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    auto task_sync = [&] {
        if (W == 1)
            __syncwarp();
        else
            asm volatile("barrier.sync %0, %1;" ::"r"(1 + warp / W), "n"(32 * W) : "memory");
    };
    if (W > 1) {
        if (lane == 0) amax_s[warp] = amax;
        task_sync();
#pragma unroll
        for (int w = 0; w < W; ++w) amax = amax_nan(amax, amax_s[warp / W * W + w]);
    }
    if ((unsigned)id >= (unsigned)a.c.n_pages) {
        if (tid == 0) atomicOr(a.error, kErrDevice);
        return;
    }
    uint8_t* block = (keys ? a.c.k : a.c.v) + id * a.c.page_stride + (size_t)head * P * D;
    float* scale = (keys ? a.c.k_scale : a.c.v_scale) + id * a.c.scale_stride + head;
    const float before_s = held > 0 ? *scale : 0.f;
    auto store = [&](int i, const float(&f)[16], float inv) {
        const Unit u(i & (upr - 1), rope_dim, a.interleaved);
        uint8_t* row = block + (size_t)(held + (i >> bits)) * D;
        *reinterpret_cast<uint2*>(row + u.c0) = make_uint2(codes4(f, inv), codes4(f + 4, inv));
        *reinterpret_cast<uint2*>(row + u.c1) = make_uint2(codes4(f + 8, inv), codes4(f + 12, inv));
    };
    float now = pow2_scale(amax);
    if (held > 0) now = now != now || before_s != before_s ? __uint_as_float(0x7fffffffu) : fmaxf(now, before_s);
    const float inv = now == now ? __frcp_rn(now) : 0.f;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
        const int i = tid + k * 32 * W;
        if (i < units) store(i, held_f[k], inv);
    }
    for (int i = tid + NU * 32 * W; i < units; i += 32 * W) {
        float f[16];
        load(i, f);
        store(i, f, inv);
    }
    if (held > 0 && now > before_s) {
        const float ratio = __fdiv_rn(before_s, now);
        uint4* codes = reinterpret_cast<uint4*>(block);
        for (int i = tid; i < held * D / 16; i += 32 * W) {
            const uint4 w = codes[i];
            codes[i] = make_uint4(requant4(w.x, ratio), requant4(w.y, ratio), requant4(w.z, ratio), requant4(w.w, ratio));
        }
    }
    if (held > 0) task_sync();  // every thread has read the scale
    if (tid == 0) *scale = now;
}

}  // namespace

cudaError_t launch_kv_append(KvAppendArgs a, cudaStream_t st, bool pdl) {
    a.by_token = kv_slot_by_token(a.bt.B, a.bt.T, a.c.page);
    // A warp a task where a sequence brings a few tokens; else as many as hold a page of
    // new tokens, two units a thread.
    const int page_units = a.c.page * a.c.dim / 16;
    const int W = (int64_t)a.bt.T <= 4 * (int64_t)a.bt.B ? 1 : page_units <= 64 ? 1 : page_units <= 128 ? 2 : page_units <= 256 ? 4 : 8;
    a.task_blocks = (2 * a.c.heads * W + 7) / 8;
    const int64_t store = kv_slots(a.bt.B, a.bt.T, a.c.page) * a.task_blocks;
    a.q_tokens = 1;
    while (a.q_tokens < kApTokens && (int64_t)a.bt.T / (2 * a.q_tokens) >= 8 * num_sms()) a.q_tokens *= 2;
    const int64_t q_blocks = a.q != nullptr ? (a.bt.T + a.q_tokens - 1) / a.q_tokens : 0;
    if (store + q_blocks > INT32_MAX) return cudaErrorInvalidValue;
    a.store_blocks = (int)store;
    const dim3 grid((unsigned)(store + q_blocks)), block(kApThreads);
    switch (W) {
        case 1: return launch_kernel(kv_append_kernel<1, 2>, grid, block, 0, st, pdl, a);
        case 2: return launch_kernel(kv_append_kernel<2, 2>, grid, block, 0, st, pdl, a);
        case 4: return launch_kernel(kv_append_kernel<4, 2>, grid, block, 0, st, pdl, a);
        default: return launch_kernel(kv_append_kernel<8, 2>, grid, block, 0, st, pdl, a);
    }
}

}  // namespace moe
