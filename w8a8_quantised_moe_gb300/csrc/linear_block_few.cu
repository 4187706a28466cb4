// linear_block_few.cu -- the block-scaled FP8 linear layer for few rows (M <=
// 128).
//
// Few rows read all the weights for little work, so the layer should take as
// long as N K bytes take from HBM (2.5 us for 4096 x 4096); what stands in the
// way is latency.  The whole GPU therefore takes one step together: a tile is
// 128 weight rows, and a cluster of CTAs splits its K, so that about every SM
// has one or two CTAs and a CTA has its first four blocks of weights in flight
// from the start.
//
//   A  128 weight rows (the MMA's M) x 128 channels, by TMA
//   B  NTOK >= M quantised rows of x (N) x 128 channels: up to kLfFusedRows rows are
//      quantised here while the weights fly (FUSED: each CTA its part of K, written
//      in the 128-byte swizzle); more come by TMA from the quantiser's launch
//      before, which the weights' loads overlap.
//   D  one 128-channel block's sums, NTOK columns of tensor memory, four buffers
//
// The epilogue warps scale each block's sums by sx * sw (a column's scale, from
// shared memory) into binary32 registers; the cluster's CTAs then add up their
// parts of K through distributed shared memory, in the order of K, each CTA for
// its share of the rows of x.
//   warps 0-7  codes or scales of x, then scale and sum (warp w: lanes
//              32 (w % 4).., half w / 4 of the columns), the cluster sum, y
//   warp 8     TMEM allocator, MMA issuer
//   warp 9     TMA producer
// Every wait is bounded; the cluster barriers are reached on every path.
#include "block_tiles.cuh"

namespace moe {
namespace {

constexpr int kLfThreads = 320;
constexpr int kLfNS = 4;                  // weight stages, and tensor-memory buffers
constexpr int kLfStageA = kBlk * kBlk;    // 128 weight rows x 128 channels
// Up to this many rows are quantised here.  Measured at N = K = 4096, quantised here /
// by a launch before, us, from a graph: 1 row 7.6 / 8.0, 4 rows 8.3 / 8.2, 8 rows 9.1 /
// 8.7, 12 rows 10.7 / 8.7, 16 rows 11.5 / 8.9 (13.0 / 9.0 at 16 x 2048 x 7168); called one
// after the other from Python, where the second launch costs host time, 1 to 16 rows:
// 11.3 to 13.6 / 14.0 to 14.7.  Beyond 8 rows each cluster's repeat of all of x costs a
// graph more than the launch costs the host.
constexpr int kLfFusedRows = 8;
constexpr int kLfMaxSmem = 232448;

struct LinFewArgs {
    const uint16_t* x;     // bf16 [M][K] (FUSED)
    const float* x_scale;  // [M][blocks_of(K)] (else)
    const float* w_scale;  // [blocks_of(N)][blocks_of(K)]
    uint16_t* y;           // bf16 [M][N]
    int M, N, K;
    int cs;                // CTAs of a cluster: parts of K
    int* error;
    uint64_t timeout_ns;
    int stall;
};

// Shared memory: ring of stages (later the partial sums), codes (FUSED), scales,
// barriers.
struct LfLayout {
    int codes, scales, bars, total;
};
__host__ __device__ constexpr int lf_stage(int ntok, bool fused) { return kLfStageA + (fused ? 0 : ntok * kBlk); }
__host__ __device__ inline LfLayout lf_layout(int ntok, bool fused, int len_max) {
    LfLayout L{};
    const int ring = kLfNS * lf_stage(ntok, fused), part = ntok * kBlk * 4;
    L.codes = ring > part ? ring : part;
    L.scales = L.codes + (fused ? len_max * ntok * kBlk : 0);
    L.bars = L.scales + len_max * ntok * 4;
    L.total = L.bars + 160 + 1024;  // + alignment slack
    // A CTA that holds all of the tensor memory takes the SM for itself: no CTA of
    // another launch is to wait there for columns while its cluster holds other SMs.
    if (ntok * kLfNS == 512 && L.total < kLfMaxSmem) L.total = kLfMaxSmem;
    return L;
}

template <int CW>
struct LfCols;  // this warp's CW columns of a buffer
template <>
struct LfCols<8> {
    static __device__ __forceinline__ void load(uint32_t a, uint32_t (&r)[8]) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(a));
    }
};
template <>
struct LfCols<16> {
    static __device__ __forceinline__ void load(uint32_t a, uint32_t (&r)[16]) { tmem_ld_16(a, r); }
};

// Waits for this warp's tensor-memory loads; the registers pass through, so
// that no use of them moves above the wait.
template <int C>
__device__ __forceinline__ void lf_wait_ld(uint32_t (&r)[C]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < C; ++i) asm volatile("" : "+r"(r[i]));
}

template <int NTOK, bool FUSED>
__global__ void __launch_bounds__(kLfThreads, NTOK <= 64 ? 2 : 1)
    block_linear_few_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                            const LinFewArgs a) {
    constexpr int CW = NTOK / 2;              // columns of a warp
    constexpr int CL = CW < 16 ? CW : 16;     // columns of one tensor-memory load
    constexpr int kTmem = NTOK * kLfNS < 32 ? 32 : NTOK * kLfNS;
    constexpr int kStage = lf_stage(NTOK, FUSED);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int nkb = blocks_of(a.K);
    const int rank = (int)cluster_ctarank(), tile = (int)blockIdx.x / a.cs;
    const int kb0 = nkb * rank / a.cs, len = nkb * (rank + 1) / a.cs - kb0;
    const LfLayout L = lf_layout(NTOK, FUSED, (nkb + a.cs - 1) / a.cs);
    uint8_t* codes = smem + L.codes;                              // FUSED: [len][NTOK rows x 128] swizzled
    float* scales = reinterpret_cast<float*>(smem + L.scales);    // [len][NTOK]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars);
    uint64_t* full = bars;               // [NS] the stage landed
    uint64_t* done = full + kLfNS;       // [NS] the block's MMAs completed: sums readable, stage free
    uint64_t* drained = done + kLfNS;    // [NS] the 8 warps have read the sums
    uint64_t* teardown = drained + kLfNS;
    uint64_t* stall_bar = teardown + 1;  // test hook: nothing arrives on it
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(stall_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCtl ctl{abort_flag, a.error, a.timeout_ns, 0u};

    int fills = 0;  // producer: stages filled
    auto load_w = [&](int kb) {
        uint64_t* bar = &full[kb % kLfNS];
        mbar_arrive_expect_tx(bar, (uint32_t)kStage);
        tma_load_2d(smem + kb % kLfNS * kStage, &tmap_w, bar, (kb0 + kb) * kBlk, tile * kBlk);
    };
    auto load_x = [&](int kb) {
        if (!FUSED)
            tma_load_2d(smem + kb % kLfNS * kStage + kLfStageA, &tmap_x, &full[kb % kLfNS], (kb0 + kb) * kBlk, 0);
    };
    if (threadIdx.x == 9 * 32) {
        for (int s = 0; s < kLfNS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&done[s], 1);
            mbar_init(&drained[s], 8);
        }
        mbar_init(teardown, 1);
        mbar_init(stall_bar, 1);
        *abort_flag = 0;
        fence_barrier_init();
        // The first stages need no wait on the ring.  With a quantiser before
        // this kernel nothing else still runs (it began by waiting for what was
        // before it), and it does not write weights: their loads start now.
        if (FUSED) pdl_wait();
        if (!a.stall) {
            for (; fills < kLfNS && fills < len; ++fills) load_w(fills);
            if (!FUSED) {
                pdl_wait();
                for (int kb = 0; kb < fills; ++kb) load_x(kb);
            }
        }
    }
    if (warp == 8) {
        tmem_alloc(tmem_slot, kTmem);
        tmem_relinquish();
    }
    __syncwarp();
    pdl_wait();  // x, and its codes and scales, are visible from here; y is free
    if (warp == 8) pdl_trigger();  // not before the tensor memory is this CTA's
    const float* sw = a.w_scale + (size_t)tile * nkb + kb0;
    if (warp < 8 && !FUSED) {  // scales of x times the weights'; columns from M on are not stored
        for (int i = threadIdx.x; i < a.M * len; i += 256) {
            const int m = i / len, kb = i - m * len;
            scales[kb * NTOK + m] = __fmul_rn(a.x_scale[(size_t)m * nkb + kb0 + kb], __ldg(sw + kb));
        }
    } else if (warp < 8) {
        // this part of x to codes, 16 lanes a block, 8 channels a lane.  Rows
        // from M on hold whatever is there: they reach their own columns of D only.
        constexpr int kBatch = 4;  // loads in flight per lane
        const int l16 = threadIdx.x & 15, items = a.M * len;
        for (int i0 = threadIdx.x >> 4; i0 - (int)(threadIdx.x >> 4 & 1) < items; i0 += 16 * kBatch) {
            uint4 v[kBatch];
            float ws[kBatch];
            int m[kBatch], kb[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int i = i0 + 16 * b;
                m[b] = i / len;
                kb[b] = i - m[b] * len;
                const int col = (kb0 + kb[b]) * kBlk + l16 * 8;
                v[b] = make_uint4(0u, 0u, 0u, 0u);
                ws[b] = 0.f;
                if (i < items) {
                    if (col < a.K) v[b] = *reinterpret_cast<const uint4*>(a.x + (size_t)m[b] * a.K + col);
                    ws[b] = __ldg(sw + kb[b]);
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                float f[8], s;
                bf16x8_to_f32(v[b], f);
                const uint2 c = quant8(f, s);
                if (i0 + 16 * b < items) {
                    uint8_t* row = codes + (kb[b] * NTOK + m[b]) * kBlk;
                    *reinterpret_cast<uint2*>(row + (((l16 >> 1) ^ (m[b] & 7)) << 4) + (l16 & 1) * 8) = c;
                    if (l16 == 0) scales[kb[b] * NTOK + m[b]] = __fmul_rn(s, ws[b]);
                }
            }
        }
        fence_proxy_async_smem();  // the codes are the tensor cores' operand
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    float acc[CW];
    if (warp == 9) {
        if (lane == 0) {
            bool ok = !a.stall || mbar_wait(stall_bar, 0, ctl);  // the test hook's wait runs out
            for (; ok && fills < len; ++fills) {
                const int s = fills % kLfNS;
                ok = fills < kLfNS || mbar_wait(&done[s], (uint32_t)(fills / kLfNS + 1) & 1u, ctl);
                if (!ok) break;
                load_w(fills);
                load_x(fills);
            }
            for (int s = 0; s < kLfNS && s < fills; ++s)  // every fill lands before the CTA may exit
                mbar_wait_drain(&full[s], (uint32_t)((fills - 1 - s) / kLfNS) & 1u);
        }
    } else if (warp == 8) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3(128, NTOK);
            for (int kb = 0; kb < len; ++kb) {
                const int s = kb % kLfNS;
                const uint32_t ph = (uint32_t)(kb / kLfNS) & 1u;
                if (!mbar_wait(&full[s], ph, ctl) || !mbar_wait(&drained[s], ph ^ 1u, ctl)) break;
                tc_fence_after();
                const uint64_t ad = smem_desc_sw128(smem_u32(smem + s * kStage));
                const uint64_t bd =
                    smem_desc_sw128(smem_u32(FUSED ? codes + kb * NTOK * kBlk : smem + s * kStage + kLfStageA));
#pragma unroll
                for (int ks = 0; ks < kBlk / 32; ++ks)
                    mma_e4m3(tmem + s * NTOK, ad + (uint64_t)(ks * 2), bd + (uint64_t)(ks * 2), idesc, ks != 0 ? 1u : 0u);
                mma_commit(&done[s]);
            }
            mma_commit(teardown);
            mbar_wait_drain(teardown, 0);
        }
    } else {
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)((warp >> 2) * CW);
#pragma unroll
        for (int j = 0; j < CW; ++j) acc[j] = 0.f;
        for (int kb = 0; kb < len; ++kb) {
            const int s = kb % kLfNS;
            if (!warp_wait(&done[s], (uint32_t)(kb / kLfNS) & 1u, ctl)) break;
            tc_fence_after();
            const float* sc = scales + kb * NTOK + (warp >> 2) * CW;
#pragma unroll
            for (int c = 0; c < CW / CL; ++c) {
                uint32_t r[CL];
                LfCols<CL>::load(lanes + s * NTOK + c * CL, r);
                lf_wait_ld(r);
#pragma unroll
                for (int j = 0; j < CL; j += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(sc + c * CL + j);
                    float* d = acc + c * CL + j;
                    d[0] = __fmaf_rn(__uint_as_float(r[j]), f.x, d[0]);
                    d[1] = __fmaf_rn(__uint_as_float(r[j + 1]), f.y, d[1]);
                    d[2] = __fmaf_rn(__uint_as_float(r[j + 2]), f.z, d[2]);
                    d[3] = __fmaf_rn(__uint_as_float(r[j + 3]), f.w, d[3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&drained[s]);
        }
    }
    // the ring is free (every MMA has completed): it takes the partial sums [NTOK][128]
    __syncthreads();
    float* part = reinterpret_cast<float*>(smem);
    if (warp < 8) {
        const int row = (warp & 3) * 32 + lane, c0 = (warp >> 2) * CW;
#pragma unroll
        for (int j = 0; j < CW; ++j) part[(c0 + j) * kBlk + row] = acc[j];
    }
    cluster_sync_all();
    for (int m = rank + a.cs * warp; m < a.M; m += a.cs * (kLfThreads / 32)) {  // a warp per row of x
        float4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < a.cs) v[r] = ld_dsmem(cluster_addr(part + m * kBlk + lane * 4, (uint32_t)r));
        float4 s = v[0];
#pragma unroll
        for (int r = 1; r < 8; ++r)
            if (r < a.cs) s = make_float4(s.x + v[r].x, s.y + v[r].y, s.z + v[r].z, s.w + v[r].w);
        const int col = tile * kBlk + lane * 4;
        if (col < a.N)
            *reinterpret_cast<uint2*>(a.y + (size_t)m * a.N + col) = make_uint2(bf16_pair(s.x, s.y), bf16_pair(s.z, s.w));
    }
    tc_fence_before();
    cluster_sync_all();  // no CTA leaves while another reads its part
    if (warp == 8) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

int lf_ntok(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

template <int NTOK, bool FUSED>
cudaError_t lf_smem_limit() {
    static const cudaError_t e = cudaFuncSetAttribute(block_linear_few_kernel<NTOK, FUSED>,
                                                      cudaFuncAttributeMaxDynamicSharedMemorySize, kLfMaxSmem);
    return e;
}

// CTAs of a cluster: as many parts of K as still run at once, two CTAs an SM where
// their shared memory allows; 0 where no split fits (FUSED keeps all its part's
// codes).
template <int NTOK, bool FUSED>
int lf_cluster(int N, int nkb) {
    if (lf_smem_limit<NTOK, FUSED>() != cudaSuccess) return 0;
    const void* kern = reinterpret_cast<const void*>(block_linear_few_kernel<NTOK, FUSED>);
    static const ClusterCounts two(kern, kLfThreads, kLfMaxSmem / 2 - 1024), one(kern, kLfThreads, kLfMaxSmem);
    const int tiles = blocks_of(N), most = nkb < 8 ? nkb : 8;
    int best = 0;
    for (int cs = 1; cs <= most; ++cs) {
        const int smem = lf_layout(NTOK, FUSED, (nkb + cs - 1) / cs).total;
        if (smem > kLfMaxSmem) continue;
        const int at_once = (smem <= kLfMaxSmem / 2 - 1024 ? two : one).of[cs];
        if (best == 0 || tiles <= at_once) best = cs;
    }
    return best;
}
int lf_cluster(int ntok, bool fused, int N, int nkb) {
    if (fused) return lf_cluster<16, true>(N, nkb);
    return ntok == 16   ? lf_cluster<16, false>(N, nkb)
           : ntok == 32 ? lf_cluster<32, false>(N, nkb)
           : ntok == 64 ? lf_cluster<64, false>(N, nkb)
                        : lf_cluster<128, false>(N, nkb);
}

template <int NTOK, bool FUSED>
cudaError_t launch_lf(const CUtensorMap& tw, const CUtensorMap& tx, const LinFewArgs& a, cudaStream_t st, bool pdl) {
    auto kern = block_linear_few_kernel<NTOK, FUSED>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks_of(a.N) * a.cs));
    cfg.blockDim = dim3(kLfThreads);
    cfg.dynamicSmemBytes = (size_t)lf_layout(NTOK, FUSED, (blocks_of(a.K) + a.cs - 1) / a.cs).total;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    if (injected(kInjectLaunchFail)) return cudaErrorLaunchFailure;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tw, tx, a);
    if (e == cudaSuccess) count_launch();
    return e;
}

}  // namespace

bool block_linear_few_fused(int M) { return M <= kLfFusedRows; }

// 128 rows are what four buffers of tensor memory hold.  This kernel / gemm_block.cu at
// that limit, us, from a graph, weights cold: 128 x 4096 x 4096 12.7 / 18.6, 128 x 2048 x
// 7168 13.6 / 27.8, 128 x 7168 x 2048 11.7 / 12.6, 128 x 8192 x 8192 26.2 / 32.4, 128 x
// 7168 x 16384 44 / 59; a wide N alone goes the other way: 16384 x 4096 with 17 rows 18.9 /
// 20.6, 64 rows 24.6 / 21.0, 128 rows 26.7 / 21.5.  (129 x 4096 x 4096: 18.5 there.)
bool block_linear_few_supported(int M, int N, int K) {
    return M <= 128 && lf_cluster(lf_ntok(M), block_linear_few_fused(M), N, blocks_of(K)) > 0;
}

cudaError_t launch_block_linear_few(const BlockGemmArgs& g, const uint16_t* x, cudaStream_t st, bool pdl) {
    const int M = g.total_rows, N = g.w_rows, ntok = lf_ntok(M);
    const bool fused = block_linear_few_fused(M);
    const LinFewArgs a{x, g.act_scale, g.w_scale, static_cast<uint16_t*>(g.out), M, N, g.K,
                       lf_cluster(ntok, fused, N, blocks_of(g.K)), g.error, g.timeout_ns, g.stall};
    CUtensorMap tw, tx;
    if (a.cs == 0 || !make_tensor_map_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.w, (uint64_t)g.K, (uint64_t)N, kBlk,
                                         kBlk, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    if (fused) return launch_lf<16, true>(tw, tw, a, st, pdl);
    if (!make_tensor_map_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.act, (uint64_t)g.K, (uint64_t)M, kBlk,
                            (uint32_t)ntok, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    switch (ntok) {
        case 16: return launch_lf<16, false>(tw, tx, a, st, pdl);
        case 32: return launch_lf<32, false>(tw, tx, a, st, pdl);
        case 64: return launch_lf<64, false>(tw, tx, a, st, pdl);
        default: return launch_lf<128, false>(tw, tx, a, st, pdl);
    }
}

}  // namespace moe
