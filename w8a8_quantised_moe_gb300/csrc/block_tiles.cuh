// block_tiles.cuh -- tile tables of the grouped block-scaled products, and the
// cluster helpers that they and the linear layer share.
#pragma once

#include "block.h"
#include "block_dev.cuh"
#include "gemm_common.cuh"

namespace moe {
namespace {

// Tile table of a launch, by one warp: group g has ceil(rows_g / rows_tile) *
// n_cb tiles.
__device__ __forceinline__ void block_tile_table(const BlockGemmArgs& args, int rows_tile, int n_cb, int* tile_start,
                                                 int* row_start, int lane) {
    const int n = args.n_groups;
    int carry = 0;
    bool bad = false;  // checked build: an offset out of order or range
    for (int base = 0; base < n; base += 32) {
        const int g = base + lane;
        int r0 = 0, r1 = 0;
        if (g < n) {
            r0 = args.offsets ? args.offsets[g] : 0;
            r1 = args.offsets ? args.offsets[g + 1] : args.total_rows;
            if (!group_rows_ok(r0, r1, args.total_rows, args.error)) {
                bad = true;
                r0 = r1 = 0;
            }
            row_start[g] = r0;
            if (g == n - 1) row_start[n] = r1;
        }
        const int v = (g < n) ? ((r1 - r0 + rows_tile - 1) / rows_tile) * n_cb : 0;
        int incl = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        if (g < n) tile_start[g] = carry + incl - v;
        carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) tile_start[n] = carry;
    if (kChecked && __any_sync(0xffffffffu, bad)) {  // an empty, consistent table: no tile runs
        for (int g = lane; g <= n; g += 32) {
            row_start[g] = 0;
            tile_start[g] = 0;
        }
    }
}

// Tile -> group, column block, first row, valid rows (row blocks fastest, so
// that a group's row blocks run together and share weight tiles in L2).
__device__ __forceinline__ void block_decode_tile(const Tiles& t, int tile, int rows_tile, int& g, int& cb,
                                                  int& row0, int& nvalid) {
    g = last_le(t.tile_start, t.n_groups, tile);
    const int local = tile - t.tile_start[g];
    const int rows = t.row_start[g + 1] - t.row_start[g];
    const int ntb = (rows + rows_tile - 1) / rows_tile;
    cb = local / ntb;
    row0 = t.row_start[g] + (local - cb * ntb) * rows_tile;
    nvalid = min(rows_tile, t.row_start[g + 1] - row0);
}

// Four values from the shared memory of another CTA of the cluster (cluster_addr).
__device__ __forceinline__ float4 ld_dsmem(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Clusters of n CTAs that run at once, for n = 1..8: an SM's place within its GPC
// leaves fewer than the SMs by themselves would (152 SMs, one CTA each: 36
// clusters of 4, 23 of 6, 15 of 8).  Asked once for a kernel and CTA size; smem:
// shared memory of a CTA.
struct ClusterCounts {
    int of[9];
    ClusterCounts(const void* kern, int threads, int smem) {
        for (int n = 1; n <= 8; ++n) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = (unsigned)n;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3((unsigned)(8 * num_sms() / n * n));
            cfg.blockDim = dim3((unsigned)threads);
            cfg.dynamicSmemBytes = (size_t)smem;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&of[n], kern, &cfg) != cudaSuccess) {
                cudaGetLastError();
                of[n] = n == 1 ? num_sms() : 0;
            }
        }
    }
    // The largest n <= most, with `wanted` clusters at once; 1 if none.
    int largest(long wanted, int most) const {
        int n = most < 8 ? most : 8;
        while (n > 1 && of[n] < wanted) --n;
        return n;
    }
};

}  // namespace
}  // namespace moe
