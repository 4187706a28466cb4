// gemm_block_few.cu -- the grouped block-scaled FP8 products for groups of a few
// rows (the layer for a few tokens): the streaming of the experts' weights.
//
// A weight byte is read once and meets a handful of rows, so HBM bounds the
// product and a tile is shaped for the copies: 256 weight rows x 128 channels
// (two 16 KB boxes) and NTOK activation rows a stage, five stages in flight.  The
// weights are the MMA's A (two M = 128 tiles), the activation rows its N = NTOK,
// so a block's sums are 2 NTOK columns of tensor memory: scaling and adding them
// costs the epilogue warps next to nothing (cf. gemm_block.cu, whose tile pays
// for 128 rows however few there are).  A thread holds one weight row's sums for
// every activation row; a column's scale is sx of the row (staged in shared
// memory a tile ahead) times sw of the half.
//
// At the tile's end the sums go through shared memory and a warp takes an
// activation row: GateUp forms h of 128 channels, a whole scale block, and writes
// its codes and scale; F32 writes 256 columns.
//
// SPLIT: where the tiles leave SMs without one (one token through two experts: 24
// tiles) a cluster of CTAs splits each tile's K, one tile a cluster, as long as
// all the clusters run at once, and adds up through distributed shared memory in
// the order of K.  (One token, the whole layer, cold: 52 us unsplit, 42, 40, 39
// with 2, 3, 4 CTAs, 52 with 6, of which 23 clusters fit.)
//   warp 0     TMA producer      warp 1  TMEM allocator, MMA issuer
//   warps 2-9  sums and output (warp w: weight rows 32 (w % 4).., half (w - 2) / 4)
// Every wait is bounded; the cluster barriers are reached on every path.
#include "block_tiles.cuh"

namespace moe {
namespace {

// Rows a group on average up to which this kernel is taken.  Measured, the whole layer,
// weights cold, this kernel / gemm_block.cu, us (E experts, top-k, H, I):
//   rows  E 64, 2, 4096, 1536    E 128, 4, 2048, 768    E 256, 8, 7168, 2048
//   1     156 / 156              94 / 108
//   2     194 / 207              113 / 133              1458 / 1516
//   4     214 / 219              125 / 140              1659 / 1688
//   16    261 / 252              157 / 163              2203 / 1786
// and with a Zipf(1.2) choice of experts, whose largest groups take many tiles of 16 rows:
//   2     86 / 91                58 / 63                450 / 386
//   4     127 / 97               75 / 71                700 / 483
// Even loads gain 3 to 12 % at 4 rows, uneven ones lose up to 45 %; at 2 they gain 4 to 15 %
// and lose at one shape.
constexpr long kFewRowsMax = 2;
// Activation rows of a tile then.  (32 of them leave room for a stage less: 64
// tokens 206, 256 tokens 249.)
constexpr int kFewTile = 16;

constexpr int kGfThreads = 320;
constexpr int kGfEpi0 = 2;
constexpr int kGfEpiWarps = 8;
constexpr int kGfBuf = 4;                     // tensor-memory buffers
constexpr int kGfStageA = 2 * kBlk * kBlk;    // both halves' weight rows
constexpr int kGfMaxSmem = 232448;

// Shared memory: ring of ns stages, partial sums [2][NTOK][128], scales of two
// tiles [2][nkb][NTOK], barriers, tables.
struct GfLayout {
    int ns, part, scales, bars, tiles, total;
};
__host__ __device__ inline GfLayout gf_layout(int ntok, int nkb) {
    GfLayout L{};
    const int stage = kGfStageA + ntok * kBlk;
    const int rest = 2 * ntok * kBlk * 4 + 2 * nkb * ntok * 4 + 512 + (kMaxExperts + 1) * 8 + 1024;
    L.ns = (kGfMaxSmem - rest) / stage;
    if (L.ns > 5) L.ns = 5;
    L.part = L.ns * stage;
    L.scales = L.part + 2 * ntok * kBlk * 4;
    L.bars = L.scales + 2 * nkb * ntok * 4;
    L.tiles = L.bars + 512;
    L.total = L.tiles + (kMaxExperts + 1) * 8 + 1024;  // + alignment slack
    return L;
}

__device__ __forceinline__ float4 gf_add(const float4& a, const float4& b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

template <int EPI>
__host__ __device__ inline int few_col_blocks(const BlockGemmArgs& a) {
    return EPI == (int)BlockEpi::GateUp ? a.up_offset / kBlk : (a.w_rows + 2 * kBlk - 1) / (2 * kBlk);
}

// First weight row of a tile's halves, and the row of the weights' scales.
template <int EPI>
__device__ __forceinline__ int few_weight_row(const BlockGemmArgs& a, int g, int cb, int half) {
    return EPI == (int)BlockEpi::GateUp ? g * a.w_rows + half * a.up_offset + cb * kBlk
                                        : g * a.w_rows + (2 * cb + half) * kBlk;
}
template <int EPI>
__device__ __forceinline__ int few_scale_block(const BlockGemmArgs& a, int cb, int half, int nb) {
    return EPI == (int)BlockEpi::GateUp ? cb + half * (a.up_offset / kBlk) : min(2 * cb + half, nb - 1);
}

template <int C>
__device__ __forceinline__ void few_wait_ld(uint32_t (&r)[C]);
template <>
__device__ __forceinline__ void few_wait_ld<16>(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])::"memory");
}
template <>
__device__ __forceinline__ void few_wait_ld<32>(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ void cp_async4(float* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// One activation row of a tile, a warp: a and b are this lane's four columns of
// the first and second half.
template <int EPI>
__device__ __forceinline__ void few_output(const BlockGemmArgs& args, int r, int cb, int lane, const float4& a,
                                           const float4& b) {
    if constexpr (EPI == (int)BlockEpi::GateUp) {
        const float h[4] = {silu_mul(a.x, b.x), silu_mul(a.y, b.y), silu_mul(a.z, b.z), silu_mul(a.w, b.w)};
        float amax = amax_nan(amax_nan(amax_nan(amax_nan(0.f, h[0]), h[1]), h[2]), h[3]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) amax = amax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        const float s = block_scale(amax);
        const size_t n_ch = (size_t)args.up_offset;
        *reinterpret_cast<uint32_t*>(args.q_out + (size_t)r * n_ch + cb * kBlk + lane * 4) =
            e4m3_quot4(h[0], h[1], h[2], h[3], s);
        if (lane == 0) args.s_out[(size_t)r * (n_ch / kBlk) + cb] = s;
    } else {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float4& f = half ? b : a;
            const int col = (2 * cb + half) * kBlk + lane * 4;
            if (col >= args.w_rows) continue;  // the same for the whole warp: w_rows is a multiple of 128
            *reinterpret_cast<float4*>(static_cast<float*>(args.out) + (size_t)r * args.w_rows + col) = f;
        }
    }
}

// TOK: the experts' ids to out[0 .. T k), the distinct ones among them, in the
// order of their first slots, from out[kFewSlots], their number to out[2 kFewSlots].
__device__ __forceinline__ void few_distinct(const BlockGemmArgs& args, int* out, int lane) {
    const int n = args.T * args.k;  // <= kFewSlots = 32
    int id = lane < n ? __ldcg(args.ids + lane) : -1;
    if (lane < n && !in_range(id, 0, args.n_groups, args.error)) id = 0;  // checked build
    const unsigned same = __match_any_sync(0xffffffffu, id);
    const bool first = lane < n && (same & ((1u << lane) - 1u)) == 0u;
    const unsigned firsts = __ballot_sync(0xffffffffu, first);
    out[lane] = id;
    if (first) out[kFewSlots + __popc(firsts & ((1u << lane) - 1u))] = id;
    if (lane == 0) out[2 * kFewSlots] = __popc(firsts);
}

// Whether this was the last of n experts to write its rows' columns of block cb.
// The rows were written before a barrier that the calling thread has passed.
__device__ __forceinline__ int few_last(const BlockGemmArgs& args, int cb, int n) {
    __threadfence();
    const bool last = atomicAdd(args.done + cb, 1u) == (unsigned)n - 1u;
    __threadfence();
    return last;
}

// y of every token over the 256 columns of block cb, in top-k order, by n threads.
__device__ __forceinline__ void few_combine(const BlockGemmArgs& args, int cb, int i0, int n) {
    const int H = args.w_rows, per = min(2 * kBlk, H - cb * 2 * kBlk) / 8;  // 8 columns a thread
    for (int i = i0; i < args.T * per; i += n) {
        const int t = i / per, col = cb * 2 * kBlk + (i - t * per) * 8;
        float a[8] = {};
        for (int j = 0; j < args.k; ++j) {
            const size_t slot = (size_t)t * args.k + j;
            const float4* o = reinterpret_cast<const float4*>(static_cast<const float*>(args.out) + slot * H + col);
            const float4 lo = __ldcg(o), hi = __ldcg(o + 1);
            const float w = __ldg(args.topk_w + slot), v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int c = 0; c < 8; ++c) a[c] = __fadd_rn(a[c], __fmul_rn(w, v[c]));
        }
        *reinterpret_cast<uint4*>(args.y + (size_t)t * H + col) =
            make_uint4(bf16_pair(a[0], a[1]), bf16_pair(a[2], a[3]), bf16_pair(a[4], a[5]), bf16_pair(a[6], a[7]));
    }
}

template <int EPI, int NTOK, bool SPLIT, bool TOK>
__global__ void __launch_bounds__(kGfThreads, 1)
    block_few_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_a,
                     const BlockGemmArgs args, int cs) {
    constexpr int kStage = kGfStageA + NTOK * kBlk;
    constexpr int kTmem = 2 * NTOK * kGfBuf;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int nkb = blocks_of(args.K);
    const GfLayout L = gf_layout(NTOK, nkb);
    const int NS = L.ns;
    float* part = reinterpret_cast<float*>(smem + L.part);
    float* scales = reinterpret_cast<float*>(smem + L.scales);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars);
    uint64_t* full = bars;                  // [NS] the stage landed
    uint64_t* empty = full + 8;             // [NS] its MMAs completed
    uint64_t* acc_full = empty + 8;         // [kGfBuf] a block's sums are in tensor memory
    uint64_t* acc_empty = acc_full + kGfBuf;  // [kGfBuf] the epilogue warps have read them
    uint64_t* teardown = acc_empty + kGfBuf;
    uint64_t* stall_bar = teardown + 1;     // test hook: nothing arrives on it
    uint64_t* epi_bar = stall_bar + 1;      // the epilogue warps
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(epi_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* last_flag = abort_flag + 1;  // TOK, F32: this tile was its columns' last
    int* tile_start = reinterpret_cast<int*>(smem + L.tiles);
    int* row_start = tile_start + (kMaxExperts + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = SPLIT ? (int)cluster_ctarank() : 0;
    const int kb0 = SPLIT ? nkb * rank / cs : 0, kb1 = SPLIT ? nkb * (rank + 1) / cs : nkb;
    int* ids_s = tile_start;  // TOK, instead of the tables: [T k] experts, then the distinct ones
    const int tile0 = SPLIT ? (int)blockIdx.x / cs : (int)blockIdx.x;
    const int tile_step = SPLIT ? 1 << 30 : (int)gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < kGfBuf; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], kGfEpiWarps);
        }
        mbar_init(teardown, 1);
        mbar_init(stall_bar, 1);
        mbar_init(epi_bar, kGfEpiWarps);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmap_w);
        tma_prefetch_desc(&tmap_a);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmem);
        tmem_relinquish();
    }
    // The expert offsets were complete before the kernel before this one passed
    // its own wait, and no kernel of the layer writes weights: the table and the
    // first stages' weights need not wait for it.
    // (TOK: the first product follows the router itself and waits; to the second
    // the same holds for the experts' ids.)
    if (TOK && EPI == (int)BlockEpi::GateUp) pdl_wait();
    if (warp == 2) {
        if (TOK) few_distinct(args, ids_s, lane);
        else block_tile_table(args, NTOK, few_col_blocks<EPI>(args), tile_start, row_start, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int n_cb = few_col_blocks<EPI>(args);
    const int total_tiles = TOK ? ids_s[2 * kFewSlots] * n_cb : tile_start[args.n_groups];
    const Tiles tiles{tile_start, row_start, args.n_groups};
    auto decode = [&](int tile, int& g, int& cb, int& row0, int& nvalid) {
        if (TOK) {
            g = ids_s[kFewSlots + tile / n_cb];
            cb = tile % n_cb;
            row0 = 0;
            nvalid = args.total_rows;
        } else {
            block_decode_tile(tiles, tile, NTOK, g, cb, row0, nvalid);
        }
    };
    // TOK: the slot that column m of expert g's tile is written to, or -1
    auto slot_of = [&](int g, int m) {
        if (EPI != (int)BlockEpi::GateUp) return ids_s[m] == g ? m : -1;
        int slot = -1;
        for (int j = 0; j < args.k; ++j)
            if (ids_s[m * args.k + j] == g) slot = m * args.k + j;
        return slot;
    };
    const WaitCtl ctl{abort_flag, args.error, args.timeout_ns, 0u};

    if (warp == 0) {
        // ---------------------------------------------------------- producer
        // lanes 0-2 issue one box each (the halves' weight rows, activation
        // rows); lane 0 owns the waits.  The first stages' activation rows follow
        // behind the wait for the kernel before.
        if (lane < 3) {
            int it = 0, ok = 1;
            bool early = true;
            if (lane == 0) ok = !args.stall || mbar_wait(stall_bar, 0, ctl);  // the test hook's wait runs out
            ok = __shfl_sync(0x7u, ok, 0);
            for (int tile = tile0; ok && tile < total_tiles; tile += tile_step) {
                int g, cb, row0, nvalid;
                decode(tile, g, cb, row0, nvalid);
                const bool two = EPI == (int)BlockEpi::GateUp || args.w_rows - cb * 2 * kBlk > kBlk;
                const uint32_t bytes = (uint32_t)(((two ? 2 : 1) * kBlk + NTOK) * kBlk);
                const int row = lane == 2 ? row0 : few_weight_row<EPI>(args, g, cb, lane);
                const int off = lane == 2 ? kGfStageA : lane * kBlk * kBlk;
                int first = 0;  // stages whose activation rows are still to come
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % NS;
                    if (early && it == NS) {
                        pdl_wait();
                        early = false;
                        if (lane == 2)
                            for (int i = 0; i < NS; ++i)
                                tma_load_2d(smem + i * kStage + off, &tmap_a, &full[i], (kb0 + i) * kBlk, row);
                    }
                    if (lane == 0) {
                        ok = mbar_wait(&empty[s], ((uint32_t)(it / NS) & 1u) ^ 1u, ctl);
                        if (ok) mbar_arrive_expect_tx(&full[s], bytes);
                    }
                    ok = __shfl_sync(0x7u, ok, 0);
                    if (!ok) break;
                    if (lane == 0 || (lane == 1 && two))
                        tma_load_2d(smem + s * kStage + off, &tmap_w, &full[s], kb * kBlk, row);
                    if (lane == 2 && !early) tma_load_2d(smem + s * kStage + off, &tmap_a, &full[s], kb * kBlk, row);
                    first = it + 1;
                }
                if (early) {  // a tile of at most NS stages
                    pdl_wait();
                    early = false;
                    if (lane == 2)
                        for (int i = 0; i < first; ++i)
                            tma_load_2d(smem + i * kStage + off, &tmap_a, &full[i], (kb0 + i) * kBlk, row);
                }
            }
            // drain: every fill issued must land before the CTA may exit
            if (lane == 0)
                for (int s = 0; s < NS && s < it; ++s) mbar_wait_drain(&full[s], (uint32_t)((it - 1 - s) / NS) & 1u);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3(kBlk, NTOK);
            int it = 0;
            bool ok = true;
            for (int tile = tile0; ok && tile < total_tiles; tile += tile_step)
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % NS, b = it % kGfBuf;
                    if (!mbar_wait(&acc_empty[b], ((uint32_t)(it / kGfBuf) & 1u) ^ 1u, ctl) ||
                        !mbar_wait(&full[s], (uint32_t)(it / NS) & 1u, ctl)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t base = smem_u32(smem + s * kStage);
                    const uint64_t bd = smem_desc_sw128(base + kGfStageA);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint64_t ad = smem_desc_sw128(base + h * kBlk * kBlk);
#pragma unroll
                        for (int ks = 0; ks < kBlk / 32; ++ks)
                            mma_e4m3(tmem + (b * 2 + h) * NTOK, ad + (uint64_t)(ks * 2), bd + (uint64_t)(ks * 2),
                                     idesc, ks != 0 ? 1u : 0u);
                    }
                    mma_commit(&empty[s]);
                    mma_commit(&acc_full[b]);
                }
            mma_commit(teardown);
            mbar_wait_drain(teardown, 0);
        }
    } else {
        // --------------------------------------------- block sums and output
        const int h = (warp - kGfEpi0) >> 2, row = (warp & 3) * 32 + lane;  // half, weight row in it
        const int et = threadIdx.x - kGfEpi0 * 32;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(h * NTOK);
        pdl_wait();  // the rows' codes and scales are visible from here
        pdl_trigger();
        // a tile's scales, [kb][NTOK], into buffer tl & 1; rows past the tile's
        // repeat its last
        auto stage_scales = [&](int tile, uint32_t tl) {
            if (tile < total_tiles) {
                int g, cb, row0, nvalid;
                decode(tile, g, cb, row0, nvalid);
                float* d = scales + (tl & 1u) * nkb * NTOK;
                for (int i = kb0 * NTOK + et; i < kb1 * NTOK; i += kGfEpiWarps * 32)
                    cp_async4(d + i, args.act_scale + (size_t)(row0 + min(i % NTOK, nvalid - 1)) * nkb + i / NTOK);
            }
            cp_async_commit();
        };
        stage_scales(tile0, 0);
        uint32_t tl = 0, sync = 0;
        int it = 0;
        bool ok = true;
        for (int tile = tile0; ok && tile < total_tiles; tile += tile_step, ++tl) {
            int g, cb, row0, nvalid;
            decode(tile, g, cb, row0, nvalid);
            const int nb = blocks_of(args.w_rows);
            const float* sw = args.w_scale + ((size_t)g * nb + few_scale_block<EPI>(args, cb, h, nb)) * nkb;
            float sw_next = __ldg(sw + kb0);
            cp_async_wait<0>();
            if (!(ok = epi_sync(epi_bar, sync, ctl))) break;  // this tile's scales; part is free
            if (!SPLIT) stage_scales(tile + tile_step, tl + 1);
            const float* sx = scales + (tl & 1u) * nkb * NTOK;
            float acc[NTOK];
#pragma unroll
            for (int j = 0; j < NTOK; ++j) acc[j] = 0.f;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int b = it % kGfBuf;
                const float w = sw_next;
                if (kb + 1 < kb1) sw_next = __ldg(sw + kb + 1);
                if (!warp_wait(&acc_full[b], (uint32_t)(it / kGfBuf) & 1u, ctl)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t v[NTOK];
#pragma unroll
                for (int c = 0; c < NTOK; c += 16)
                    tmem_ld_16(lanes + b * 2 * NTOK + c, *reinterpret_cast<uint32_t(*)[16]>(v + c));
                few_wait_ld(v);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[b]);
#pragma unroll
                for (int j = 0; j < NTOK; j += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(sx + kb * NTOK + j);
                    acc[j] = __fmaf_rn(__uint_as_float(v[j]), __fmul_rn(f.x, w), acc[j]);
                    acc[j + 1] = __fmaf_rn(__uint_as_float(v[j + 1]), __fmul_rn(f.y, w), acc[j + 1]);
                    acc[j + 2] = __fmaf_rn(__uint_as_float(v[j + 2]), __fmul_rn(f.z, w), acc[j + 2]);
                    acc[j + 3] = __fmaf_rn(__uint_as_float(v[j + 3]), __fmul_rn(f.w, w), acc[j + 3]);
                }
            }
            if (!ok) break;
#pragma unroll
            for (int j = 0; j < NTOK; ++j) part[(h * NTOK + j) * kBlk + row] = acc[j];
            if (SPLIT) break;  // the cluster adds up below
            if (!(ok = epi_sync(epi_bar, sync, ctl))) break;
            for (int m = warp - kGfEpi0; m < nvalid; m += kGfEpiWarps) {
                const int r = TOK ? slot_of(g, m) : row0 + m;
                if (r < 0) continue;
                const float4 a = *reinterpret_cast<const float4*>(part + m * kBlk + lane * 4);
                const float4 b = *reinterpret_cast<const float4*>(part + (NTOK + m) * kBlk + lane * 4);
                few_output<EPI>(args, r, cb, lane, a, b);
            }
            if (TOK && EPI == (int)BlockEpi::F32) {  // this expert's rows are written: the combine of the last
                if (!(ok = epi_sync(epi_bar, sync, ctl))) break;
                if (et == 0) *last_flag = few_last(args, cb, ids_s[2 * kFewSlots]);
                if (!(ok = epi_sync(epi_bar, sync, ctl))) break;
                if (*last_flag) few_combine(args, cb, et, kGfEpiWarps * 32);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (SPLIT) {
        cluster_sync_all();
        if (tile0 < total_tiles) {
            int g, cb, row0, nvalid;
            decode(tile0, g, cb, row0, nvalid);
            for (int m = rank + cs * warp; m < nvalid; m += cs * (kGfThreads / 32)) {  // a warp per row
                const int r_out = TOK ? slot_of(g, m) : row0 + m;
                if (r_out < 0) continue;
                float4 a[8], b[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < cs) {
                        a[r] = ld_dsmem(cluster_addr(part + m * kBlk + lane * 4, (uint32_t)r));
                        b[r] = ld_dsmem(cluster_addr(part + (NTOK + m) * kBlk + lane * 4, (uint32_t)r));
                    }
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    if (r < cs) {
                        a[0] = gf_add(a[0], a[r]);
                        b[0] = gf_add(b[0], b[r]);
                    }
                few_output<EPI>(args, r_out, cb, lane, a[0], b[0]);
            }
        }
        cluster_sync_all();  // no CTA leaves while another reads its part
        if (TOK && EPI == (int)BlockEpi::F32 && rank == 0 && tile0 < total_tiles) {
            // this expert's rows are written (by the cluster): the combine of the last
            const int cb = tile0 % n_cb;
            if (threadIdx.x == 0) *last_flag = few_last(args, cb, ids_s[2 * kFewSlots]);
            __syncthreads();
            if (*last_flag) few_combine(args, cb, threadIdx.x, kGfThreads);
        }
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

template <int EPI, int NTOK, bool SPLIT, bool TOK>
cudaError_t few_smem_limit() {
    static const cudaError_t e = cudaFuncSetAttribute(block_few_kernel<EPI, NTOK, SPLIT, TOK>,
                                                      cudaFuncAttributeMaxDynamicSharedMemorySize, kGfMaxSmem);
    return e;
}

// CTAs of a cluster that splits one of `tiles` tiles: 1 where they do not all run at once.
template <int EPI, int NTOK, bool TOK>
int few_cluster(long tiles, int nkb) {
    if (few_smem_limit<EPI, NTOK, true, TOK>() != cudaSuccess) return 1;
    static const ClusterCounts counts(reinterpret_cast<const void*>(block_few_kernel<EPI, NTOK, true, TOK>), kGfThreads,
                                      kGfMaxSmem);
    return counts.largest(tiles, nkb);
}

template <int EPI, int NTOK, bool SPLIT, bool TOK>
cudaError_t launch_few_impl(const BlockGemmArgs& args, long tiles, int cs, cudaStream_t st, bool pdl) {
    auto kern = block_few_kernel<EPI, NTOK, SPLIT, TOK>;
    const cudaError_t attr_err = few_smem_limit<EPI, NTOK, SPLIT, TOK>();
    if (attr_err != cudaSuccess) return attr_err;
    CUtensorMap tw, ta;
    if (!make_tensor_map_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, args.w, args.K,
                            (uint64_t)args.n_groups * args.w_rows, kBlk, kBlk, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, args.act, args.K, (uint64_t)args.total_rows, kBlk,
                            NTOK, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    long grid = SPLIT ? tiles * cs : tiles < num_sms() ? tiles : num_sms();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kGfThreads);
    cfg.dynamicSmemBytes = (size_t)gf_layout(NTOK, blocks_of(args.K)).total;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (SPLIT) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cs;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    if (injected(kInjectLaunchFail)) return cudaErrorLaunchFailure;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tw, ta, args, cs);
    if (e == cudaSuccess) count_launch();
    return e;
}

template <int EPI, int NTOK, bool TOK>
cudaError_t launch_few_ntok(const BlockGemmArgs& args, long tiles, cudaStream_t st, bool pdl) {
    const int cs = few_cluster<EPI, NTOK, TOK>(tiles, blocks_of(args.K));
    return cs > 1 ? launch_few_impl<EPI, NTOK, true, TOK>(args, tiles, cs, st, pdl)
                  : launch_few_impl<EPI, NTOK, false, TOK>(args, tiles, 1, st, pdl);
}

template <int EPI>
cudaError_t launch_few(const BlockGemmArgs& args, cudaStream_t st, bool pdl) {
    const long rows = args.total_rows;
    if (args.ids != nullptr) {
        const long slots = (long)args.T * args.k;
        const long tiles = (slots < args.n_groups ? slots : args.n_groups) * few_col_blocks<EPI>(args);
        return rows <= 16 ? launch_few_ntok<EPI, 16, true>(args, tiles, st, pdl)
                          : launch_few_ntok<EPI, 32, true>(args, tiles, st, pdl);
    }
    // at most this many groups have rows, and so many more tiles than whole ones
    const long groups = rows < args.n_groups ? rows : args.n_groups;
    const long tiles = (rows <= kFewTile ? groups : rows / kFewTile + groups) * few_col_blocks<EPI>(args);
    return launch_few_ntok<EPI, kFewTile, false>(args, tiles, st, pdl);
}

}  // namespace

bool block_gemm_few_wanted(const BlockGemmArgs& args) {
    return args.total_rows <= kFewRowsMax * (long)args.n_groups;
}

cudaError_t launch_block_gemm_few(BlockEpi epi, const BlockGemmArgs& args, cudaStream_t st, bool pdl) {
    if (args.total_rows == 0) return cudaSuccess;
    switch (epi) {
        case BlockEpi::GateUp: return launch_few<0>(args, st, pdl);
        case BlockEpi::F32: return launch_few<1>(args, st, pdl);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace moe
