// gemm_block.cu -- the grouped block-scaled FP8 product on the tcgen05 tensor
// cores, for groups of many rows:
//
//   D[r][n] = sum_b sx[r][b] * sw[n / 128][b] * (sum_{k in block b} a[r][k] * w[n][k])
//
// with E4M3 a and w (their products are exact in binary32).  The tensor cores
// accumulate one 128-channel block at a time in tensor memory; the scales
// differ from block to block, so the block's partial sums go to registers,
// where they are multiplied by the block's scale and added to binary32 sums.
//
// Tile: 128 activation rows (the MMA's M, one TMEM lane each) x 256 weight rows
// (N) in two halves of 128.  With rows on the lanes a thread's scale is one value
// per half and block: sx of its row times sw of the half.  GateUp's halves are 64
// gate rows and the 64 up rows of the same channels, so the tile holds whole
// scale blocks of h: each thread applies silu(gate) * up to its 64 + 64 columns
// and h leaves the kernel as E4M3 codes with their scale, never as binary32.  (The
// second expert product's rows are binary32: fp16 rows with a scale per 128 columns
// saved 33 us of 546 at 8192 tokens, and rounded y twice.)
//   warp 0      TMA producer (ring of kBgNS stages: activation rows and four
//               quarters of the weight rows, 128 bytes of K each)
//   warp 1      MMA issuer (and TMEM allocator): four K = 32 MMAs a block into one
//               of two 256-column buffers
//   warps 4-11  scale and sum the blocks, then the epilogue: four warps a half
// Persistent grid, tiles dealt round-robin.  Every wait is bounded (ptx.cuh).
//
// What bounds it: a block of a tile takes about 845 clocks (4864 x 4864, K 4096 to
// 12288, 2070 MHz), of which the MMAs are 512.  Two chains of about that length
// meet there.  Shared memory: the MMAs read 48 KB and the copies write 48 KB, 750
// clocks at 128 B.  Tensor memory, full with two buffers: given back, a buffer is
// summed again after a wait, 512 clocks of MMAs and another wait, while the
// other's 128 columns a warp take four loads and their multiply-adds; without the
// sums a block still took 795 to 836.  What counts on both sides are a lone warp's
// instructions: 65 more per block and scheduler cost 115 clocks, 115 more (scalar
// multiply-adds) 180.  At 8192^3 (440 us beside its quantiser) the card's power
// limit sets the clock besides: 1370 W, about 1.75 GHz.
//
// Measured on the way, the layer of the quantiser and this kernel at 8192^3, us:
// issued by one thread whose addresses did not stay uniform, with an issuer a half
// (the activation rows read twice), 16 columns a load: 490; the issuer as below
// 484; one 256-column MMA for both halves and 32 columns a load 469.  One barrier
// for both halves' sums instead of one each 474.  Tried and slower before that:
// two issuers on alternate blocks, sixteen epilogue warps (624), scalar
// multiply-adds (540), tests of the next block's barriers ahead of time (504), row
// scales read four blocks at a time (520) or stored block by block (617).  CTA
// pairs (cta_group::2, 32 KB a CTA and block) came to 447 here, by drawing less
// power, and to the same time at 4096^3; 16 experts of 2048 rows took 992 against 837,
// which an idle CTA in each group's odd tile (one in 17 at most) does not explain: the
// cause was not found.  Weights multicast to two CTAs: 483 against 490.
#include <mutex>

#include "block.h"
#include "block_tiles.cuh"

namespace moe {
namespace {

constexpr int kBgRows = 128;     // activation rows of a CTA
constexpr int kBgCols = 256;     // weight rows of a tile
constexpr int kBgThreads = 384;  // producer, MMA issuer, tile table, idle and 8 epilogue warps
constexpr int kBgEpi0 = 4;       // first epilogue warp
constexpr int kBgEpiWarps = 8;
constexpr int kBgHalf = kBlk * kBlk;         // bytes of 128 rows x 128 channels
// per epilogue warp: 32 rows x 64 codes, or x 128 bytes of columns
__host__ __device__ constexpr int bg_staging(int epi) { return epi == (int)BlockEpi::GateUp ? 32 * 64 : 32 * 128; }
constexpr int kBgXch = 2 * 2 * kBgRows * 4;  // GateUp: row maxima [2 tiles][2 warps][rows]

// The launch gives every thread 168 registers; the epilogue warps hold 128 sums
// and their next columns each, so the first four warps pass them theirs: 128 x
// 40 + 256 x 232 = 384 x 168.
__device__ __forceinline__ void bg_regs_few() { asm volatile("setmaxnreg.dec.sync.aligned.u32 40;"); }
__device__ __forceinline__ void bg_regs_many() { asm volatile("setmaxnreg.inc.sync.aligned.u32 232;"); }

template <int N>
struct Int {
    static constexpr int value = N;
};

// This lane's 32 columns from OFF on, of the tensor memory at `a`.
template <int OFF>
__device__ __forceinline__ void bg_ld_32(uint32_t a, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32 + %33];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
          "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(a), "n"(OFF));
}

// Waits for this warp's tensor-memory loads; the registers pass through, so
// that no use of them moves above the wait.
__device__ __forceinline__ void bg_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])::"memory");
}

// An epilogue warp: 32 lanes' rows x the 128 columns of half w2.
struct BgWarp {
    int q, w2, row, lane;  // lane quarter, half of the columns, row of the CTA's 128
    __device__ __forceinline__ BgWarp(int warp, int ln) : q(warp & 3), w2((warp - kBgEpi0) >> 2), lane(ln) {
        row = q * 32 + lane;
    }
    // its columns of a 256-column buffer at `tmem`
    __device__ __forceinline__ uint32_t addr(uint32_t tmem) const {
        return tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(w2 * kBlk);
    }
};

// Adds the block's sums at `a` (this warp's 128 columns), times the scales of the
// first and last 64, to acc[part][column pair].  `release` runs once every column
// is in registers.  (Offsets within the instruction and 32 columns a load: each
// instruction less an epilogue warp spends on a block counted, see above.)
template <class Release>
__device__ __forceinline__ void bg_add_block(f32x2 (&acc)[2][32], uint32_t a, float s0, float s1, Release release) {
    const f32x2 sc[2] = {pack2(s0, s0), pack2(s1, s1)};
    auto step = [&](auto part) {
        constexpr int c = decltype(part)::value;
        uint32_t v[32];
        bg_ld_32<c * 32>(a, v);
        bg_wait_ld(v);
        if constexpr (c == 3) release();
#pragma unroll
        for (int j = 0; j < 16; ++j)
            fma2(acc[c >> 1][(c & 1) * 16 + j],
                 pack2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), sc[c >> 1]);
    };
    step(Int<0>{});
    step(Int<1>{});
    step(Int<2>{});
    step(Int<3>{});
}

// The scales that an epilogue thread applies, read one block ahead: its row's
// (blocks of a row are next to each other: seven of eight reads hit L1) and the
// weights' two, one where both halves' parts share it.  Measured at 8192^3 on the
// first forms of this kernel, us: this 522; the rows' scales stored block by block,
// one line a warp and block, 617; staged in shared memory by a fourth warp or by
// the producer's copies, behind barriers of their own, 608 and 728.
struct BgScales {
    const float *sx, *sw0, *sw1;
    float x, w0, w1;
    template <int EPI>
    __device__ __forceinline__ void start(const BlockGemmArgs& a, int g, int cb, int w2, int r, int nkb) {
        const int nb = blocks_of(a.w_rows);
        const int b0 = EPI == (int)BlockEpi::GateUp ? cb : min(2 * cb + w2, nb - 1);
        const int b1 = EPI == (int)BlockEpi::GateUp ? cb + a.up_offset / kBlk : b0;
        sx = a.act_scale + (size_t)r * nkb;
        sw0 = a.w_scale + ((size_t)g * nb + b0) * nkb;
        sw1 = a.w_scale + ((size_t)g * nb + b1) * nkb;
        x = __ldg(sx);
        w0 = __ldg(sw0);
        w1 = EPI == (int)BlockEpi::GateUp ? __ldg(sw1) : w0;
    }
    template <int EPI>
    __device__ __forceinline__ void next(int kb, int nkb, float& s0, float& s1) {
        s0 = __fmul_rn(x, w0);
        s1 = EPI == (int)BlockEpi::GateUp ? __fmul_rn(x, w1) : s0;
        if (kb + 1 < nkb) {
            x = __ldg(sx + kb + 1);
            w0 = __ldg(sw0 + kb + 1);
            if (EPI == (int)BlockEpi::GateUp) w1 = __ldg(sw1 + kb + 1);
        }
    }
};

// The warp's 32 rows x 16 N bytes (v: this lane's row; N 4 or 8) to memory through
// shared memory, so that an instruction writes whole pieces of 32 / N rows
// instead of 16 bytes of 32.  dst: row 0's piece; rows from `rows` on are not written.
template <int N>
__device__ __forceinline__ void bg_store_rows(uint8_t* staging, const uint4 (&v)[N], int lane, uint8_t* dst,
                                              size_t stride, int rows) {
    auto place = [&](int r, int c) {
        return reinterpret_cast<uint4*>(staging + r * 16 * N + ((c ^ (N == 8 ? r & 7 : r >> 1 & 3)) << 4));
    };
    __syncwarp();  // the previous piece has been read
#pragma unroll
    for (int c = 0; c < N; ++c) *place(lane, c) = v[c];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int r = i * (32 / N) + lane / N, c = lane % N;
        if (r < rows) *reinterpret_cast<uint4*>(dst + (size_t)r * stride + c * 16) = *place(r, c);
    }
}

// What a tile's sums become.  row0: the CTA's first row; nvalid: its rows; cb:
// channel block (GateUp) or 256-column block.  Returns false when a wait gave up.
template <int EPI>
__device__ __forceinline__ bool bg_output(const BlockGemmArgs& args, f32x2 (&acc)[2][32], const BgWarp& w, int row0,
                                          int nvalid, int cb, float* xch, uint64_t* pair_bar, uint32_t tl,
                                          uint8_t* staging, const WaitCtl& ctl) {
    const int rows = min(32, nvalid - w.q * 32);  // of this warp; may be negative
    const size_t r0 = (size_t)row0 + w.q * 32;
    if constexpr (EPI == (int)BlockEpi::GateUp) {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            float g0, g1, u0, u1;
            unpack2(acc[0][j], g0, g1);
            unpack2(acc[1][j], u0, u1);
            g0 = silu_mul(g0, u0);
            g1 = silu_mul(g1, u1);
            amax = amax_nan(amax_nan(amax, g0), g1);
            acc[0][j] = pack2(g0, g1);
        }
        // the row's other 64 columns are the partner warp's
        float* mine = xch + (tl & 1u) * 2 * kBgRows;
        mine[w.w2 * kBgRows + w.row] = amax;
        __syncwarp();
        if (w.lane == 0) mbar_arrive(&pair_bar[w.q]);
        if (!warp_wait(&pair_bar[w.q], tl & 1u, ctl)) return false;
        amax = amax_nan(amax, mine[(w.w2 ^ 1) * kBgRows + w.row]);
        const float s = block_scale(amax);
        const BlockQuot quot(s);
        const int n_ch = args.up_offset;
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float h[16];
            uint32_t c4[4];
#pragma unroll
            for (int j = 0; j < 8; ++j) unpack2(acc[0][i * 8 + j], h[2 * j], h[2 * j + 1]);
            quot.codes(h, c4);
            v[i] = make_uint4(c4[0], c4[1], c4[2], c4[3]);
        }
        bg_store_rows(staging, v, w.lane, args.q_out + r0 * n_ch + cb * kBlk + w.w2 * 64, n_ch, rows);
        if (w.w2 == 0 && w.lane < rows) args.s_out[(r0 + w.lane) * (n_ch / kBlk) + cb] = s;
    } else {
        const int col0 = cb * kBgCols + w.w2 * kBlk;  // this warp's 128 columns
        constexpr int kElem = EPI == (int)BlockEpi::F32 ? 4 : 2, kCols = 128 / kElem;  // columns of a piece
#pragma unroll
        for (int piece = 0; piece < kBlk / kCols; ++piece) {
            const int col = col0 + piece * kCols;
            if (col >= args.w_rows) continue;
            uint4 v[8];  // this lane's 128 bytes
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t c4[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int p = piece * kCols / 2 + (i * 4 + j) * kCols / 64;  // column pair
                    float a, b;
                    unpack2(acc[p >> 5][p & 31], a, b);
                    c4[j] = EPI != (int)BlockEpi::F32 ? bf16_pair(a, b) : __float_as_uint(j & 1 ? b : a);
                }
                v[i] = make_uint4(c4[0], c4[1], c4[2], c4[3]);
            }
            uint8_t* dst = static_cast<uint8_t*>(args.out) + (r0 * args.w_rows + col) * kElem;
            if (EPI == (int)BlockEpi::F32 || col + kCols <= args.w_rows) {  // F32: w_rows is a multiple of 128
                bg_store_rows(staging, v, w.lane, dst, (size_t)args.w_rows * kElem, rows);
            } else if (w.lane < rows) {  // the last 16 to 48 columns of a matrix
#pragma unroll
                for (int i = 0; i < 6; ++i)
                    if (col + i * 8 < args.w_rows)
                        reinterpret_cast<uint4*>(dst + (size_t)w.lane * args.w_rows * 2)[i] = v[i];
            }
        }
    }
    return true;
}

template <int EPI>
__host__ __device__ inline int bg_col_blocks(const BlockGemmArgs& a) {
    return EPI == (int)BlockEpi::GateUp ? a.up_offset / kBlk : (a.w_rows + kBgCols - 1) / kBgCols;
}

// First weight row of a tile's quarters of 64: GateUp's halves are 64 gate rows,
// then the same channels' up rows.
template <int EPI>
__device__ __forceinline__ int bg_weight_row(const BlockGemmArgs& a, int g, int cb, int i) {
    return EPI == (int)BlockEpi::GateUp ? g * a.w_rows + (i & 1) * a.up_offset + cb * kBlk + (i >> 1) * 64
                                        : g * a.w_rows + cb * kBgCols + i * 64;
}

constexpr int kBgNS = 4;  // stages
constexpr int kBgStage = 3 * kBgHalf;
constexpr int kBgOffBars = kBgNS * kBgStage;
constexpr int kBgNumBars = 2 * kBgNS + 8 + 2 + 4;  // full, empty, acc_full/empty[4], teardown, stall, pair[4]
constexpr int kBgOffTiles = kBgOffBars + kBgNumBars * 8;
constexpr int kBgOffMisc = (kBgOffTiles + (kMaxExperts + 1) * 4 * 2 + 15) / 16 * 16;
constexpr int kBgOffStaging = kBgOffMisc + 64;  // then GateUp's row maxima
__host__ __device__ constexpr int bg_off_xch(int epi) { return kBgOffStaging + kBgEpiWarps * bg_staging(epi); }
__host__ __device__ constexpr int bg_smem(int epi) {
    return bg_off_xch(epi) + (epi == (int)BlockEpi::GateUp ? kBgXch : 0);
}
static_assert(kBgOffTiles % 8 == 0 && kBgOffStaging % 16 == 0, "alignment");
static_assert(bg_smem(0) <= 232448 && bg_smem(1) <= 232448, "shared memory budget");

// Box heights of the activation maps: the smallest that covers a tile's rows.
__host__ __device__ constexpr int bg_box_rows(int i) { return i == 0 ? 32 : i == 1 ? 64 : kBgRows; }
__device__ __forceinline__ int bg_box_index(int nvalid) { return nvalid <= 32 ? 0 : nvalid <= 64 ? 1 : 2; }

template <int EPI>
__global__ void __launch_bounds__(kBgThreads, 1)
    block_gemm_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_a0,
                      const __grid_constant__ CUtensorMap tmap_a1, const __grid_constant__ CUtensorMap tmap_a2,
                      const BlockGemmArgs args) {
    // The budget leaves no room to round the base up to the swizzle's 1024 bytes;
    // dynamic shared memory starts there.
    extern __shared__ __align__(1024) uint8_t smem[];
    if ((smem_u32(smem) & 1023u) != 0u) {
        if (threadIdx.x == 0) atomicOr(args.error, kErrDevice);
        return;
    }
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBgOffBars);
    uint64_t* full = bars;              // [NS] the stage landed
    uint64_t* empty = full + kBgNS;     // [NS] the MMAs of the stage completed
    uint64_t* acc_full = empty + kBgNS; // [2 buffers][2 halves] a block's partial sums are in tensor memory
    uint64_t* acc_empty = acc_full + 4; // [2][2] the half's epilogue warps have read them
    uint64_t* teardown = acc_empty + 4;
    uint64_t* stall_bar = teardown + 1; // test hook: nothing arrives on it
    uint64_t* pair_bar = stall_bar + 1; // [4] the two warps of a lane quarter
    int* tile_start = reinterpret_cast<int*>(smem + kBgOffTiles);
    int* row_start = tile_start + (kMaxExperts + 1);
    float* xch = reinterpret_cast<float*>(smem + bg_off_xch(EPI));
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kBgOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kBgOffMisc + 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nkb = blocks_of(args.K);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kBgNS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int d = 0; d < 4; ++d) {
            mbar_init(&acc_full[d], 1);
            mbar_init(&acc_empty[d], kBgEpiWarps / 2);
        }
        mbar_init(teardown, 1);
        mbar_init(stall_bar, 1);
        for (int i = 0; i < 4; ++i) mbar_init(&pair_bar[i], 2);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmap_w);
        tma_prefetch_desc(&tmap_a2);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    pdl_wait();  // the previous kernel's outputs (offsets, codes, scales) are visible from here
    if (warp == 1) pdl_trigger();  // not before the tensor memory is this CTA's
    if (warp == 2) block_tile_table(args, kBgRows, bg_col_blocks<EPI>(args), tile_start, row_start, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total_tiles = tile_start[args.n_groups];
    const Tiles tiles{tile_start, row_start, args.n_groups};
    const WaitCtl ctl{abort_flag, args.error, args.timeout_ns, 0u};
    // halves of a tile that hold weight rows (GateUp: always both)
    auto halves_of = [&](int cb) {
        return EPI == (int)BlockEpi::GateUp || args.w_rows - cb * kBgCols > kBlk ? 2 : 1;
    };

    if (warp < kBgEpi0) {
        bg_regs_few();
        if (warp == 0) {
            // ---------------------------------------------------------- producer
            // lanes 0-4 issue one box each (64 weight rows each, the activation
            // rows) in the same warp instruction; lane 0 owns the waits
            if (lane < 5) {
                uint32_t it = 0;
                int ok = 1;
                if (lane == 0) ok = !args.stall || mbar_wait(stall_bar, 0, ctl);  // the test hook's wait runs out
                ok = __shfl_sync(0x1fu, ok, 0);
                for (int tile = blockIdx.x; ok && tile < total_tiles; tile += gridDim.x) {
                    int g, cb, row0, nvalid;
                    block_decode_tile(tiles, tile, kBgRows, g, cb, row0, nvalid);
                    const int halves = halves_of(cb);
                    const int bi = bg_box_index(nvalid);
                    const CUtensorMap* ma = bi == 0 ? &tmap_a0 : bi == 1 ? &tmap_a1 : &tmap_a2;
                    const uint32_t bytes = (uint32_t)((bg_box_rows(bi) + halves * kBlk) * kBlk);
                    const CUtensorMap* map = lane == 4 ? ma : &tmap_w;
                    const int row = lane == 4 ? row0 : bg_weight_row<EPI>(args, g, cb, lane);
                    const int off = lane == 4 ? 0 : kBgHalf + lane * (kBgHalf / 2);
                    for (int kb = 0; kb < nkb; ++kb, ++it) {
                        const uint32_t s = it % kBgNS, ph = (it / kBgNS) & 1u;
                        if (lane == 0) {
                            ok = mbar_wait(&empty[s], ph ^ 1u, ctl);
                            if (ok) mbar_arrive_expect_tx(&full[s], bytes);
                        }
                        ok = __shfl_sync(0x1fu, ok, 0);
                        if (!ok) break;
                        if (lane < 2 * halves || lane == 4)
                            tma_load_2d(smem + s * kBgStage + off, map, &full[s], kb * kBlk, row);
                    }
                }
                // drain: every fill issued must land before the CTA may exit
                if (lane == 0)
                    for (uint32_t s = 0; s < (uint32_t)kBgNS && s < it; ++s) {
                        const uint32_t last = it - 1 - ((it - 1 - s) % kBgNS);
                        mbar_wait_drain(&full[s], (last / kBgNS) & 1u);
                    }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------ MMA issuer
            // The whole warp runs the loop, so that what the MMAs take stays uniform, and
            // asks every barrier before it uses an answer; lane 0 issues.
            constexpr uint32_t idesc = idesc_e4m3(kBgRows, kBgCols);
            const uint64_t a0 = smem_desc_sw128(smem_u32(smem)), b0 = smem_desc_sw128(smem_u32(smem) + kBgHalf);
            const int cta = blockIdx.x, ctas = gridDim.x;
            const int my_tiles = cta < total_tiles ? (total_tiles - 1 - cta) / ctas + 1 : 0;
            uint32_t s = 0, ph = 0, d = 0, dph = 1;  // stage, its phase, buffer, its phase
            for (int n = my_tiles * nkb; n > 0; --n) {
                const bool free0 = mbar_try_wait(&acc_empty[d * 2], dph),
                           free1 = mbar_try_wait(&acc_empty[d * 2 + 1], dph),
                           landed = mbar_try_wait(&full[s], ph);
                if (!__all_sync(0xffffffffu, free0 && free1 && landed) &&
                    (!warp_wait(&acc_empty[d * 2], dph, ctl) || !warp_wait(&acc_empty[d * 2 + 1], dph, ctl) ||
                     !warp_wait(&full[s], ph, ctl)))
                    break;
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t a = a0 + (uint64_t)(s * (kBgStage >> 4)), b = b0 + (uint64_t)(s * (kBgStage >> 4));
#pragma unroll
                    for (int ks = 0; ks < kBlk / 32; ++ks)  // 32 bytes of K per MMA
                        mma_e4m3(tmem + d * kBgCols, a + (uint64_t)(ks * 2), b + (uint64_t)(ks * 2), idesc,
                                 ks != 0 ? 1u : 0u);
                    mma_commit(&acc_full[d * 2]);
                    mma_commit(&acc_full[d * 2 + 1]);
                    mma_commit(&empty[s]);
                }
                __syncwarp();
                if (++s == kBgNS) {
                    s = 0;
                    ph ^= 1u;
                }
                d ^= 1u;
                dph ^= d ^ 1u;
            }
            if (lane == 0) {
                mma_commit(teardown);
                mbar_wait_drain(teardown, 0);
            }
        }
    } else {
        bg_regs_many();
        // ------------------------------------- block sums and the epilogue
        const BgWarp w(warp, lane);
        uint8_t* staging = smem + kBgOffStaging + (warp - kBgEpi0) * bg_staging(EPI);
        uint32_t d = 0, ph = 0, tl = 0;  // buffer, its phase, tiles
        bool ok = true;
        for (int tile = blockIdx.x; ok && tile < total_tiles; tile += gridDim.x, ++tl) {
            int g, cb, row0, nvalid;
            block_decode_tile(tiles, tile, kBgRows, g, cb, row0, nvalid);
            f32x2 acc[2][32];  // [64 columns][column pair]
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[0][j] = acc[1][j] = 0ull;
            BgScales sc;
            sc.start<EPI>(args, g, cb, w.w2, row0 + min(w.row, nvalid - 1), nkb);
            for (int kb = 0; kb < nkb; ++kb) {
                float s0, s1;
                sc.next<EPI>(kb, nkb, s0, s1);
                if (!warp_wait(&acc_full[d * 2 + w.w2], ph, ctl)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                auto release = [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_empty[d * 2 + w.w2]);
                };
                if (EPI == (int)BlockEpi::BF16 || nvalid > w.q * 32)  // else none of this warp's rows
                    bg_add_block(acc, w.addr(tmem + d * kBgCols), s0, s1, release);
                else
                    release();
                d ^= 1u;
                ph ^= d ^ 1u;
            }
            ok = ok && bg_output<EPI>(args, acc, w, row0, nvalid, cb, xch, pair_bar, tl, staging, ctl);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int EPI>
cudaError_t launch_block_impl(const BlockGemmArgs& args, cudaStream_t st, bool pdl) {
    auto kern = block_gemm_kernel<EPI>;
    static std::once_flag once;
    static cudaError_t attr_err = cudaSuccess;
    std::call_once(once, [&] {
        attr_err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bg_smem(EPI));
    });
    if (attr_err != cudaSuccess) return attr_err;
    CUtensorMap tw, ta[3];
    if (!make_tensor_map_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, args.w, args.K,
                            (uint64_t)args.n_groups * args.w_rows, kBlk, 64, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    for (int i = 0; i < 3; ++i)
        if (!make_tensor_map_2d(&ta[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, args.act, args.K, (uint64_t)args.total_rows,
                                kBlk, bg_box_rows(i), CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    const long max_tiles =
        ((long)(args.total_rows + kBgRows - 1) / kBgRows + args.n_groups - 1) * bg_col_blocks<EPI>(args);
    long grid = num_sms();
    if (max_tiles < grid) grid = max_tiles;
    if (grid < 1) grid = 1;
    return launch_kernel(kern, dim3((unsigned)grid), dim3(kBgThreads), bg_smem(EPI), st, pdl, tw, ta[0], ta[1], ta[2],
                         args);
}

}  // namespace

cudaError_t launch_block_gemm(BlockEpi epi, const BlockGemmArgs& args, cudaStream_t st, bool pdl) {
    if (args.total_rows == 0) return cudaSuccess;
    switch (epi) {
        case BlockEpi::GateUp: return launch_block_impl<0>(args, st, pdl);
        case BlockEpi::F32: return launch_block_impl<1>(args, st, pdl);
        case BlockEpi::BF16: return launch_block_impl<2>(args, st, pdl);
    }
    return cudaErrorInvalidValue;
}

}  // namespace moe
