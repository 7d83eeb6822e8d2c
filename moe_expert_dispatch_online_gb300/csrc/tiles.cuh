// What the grouped products of quantised rows share: a device work list of row tiles, the walk of a
// pair of CTAs over its units, the epilogue's barriers and byte tensor maps.
#pragma once

#include <cudaTypedefs.h>

#include "ptx.cuh"

namespace bep {
namespace {

// Work of a pair of CTAs: rows of one segment by a pair of 128-output tiles.
struct Unit {
    int row0, rows, expert, mp;
};

// A cluster's units lie `ncl` apart in (tile, pair of output tiles) order, the pair fastest: a walk
// over them without a division, since a unit may last only a few stages.
struct UnitWalk {
    int unit, tile, mp;        // the next unit
    int dtile, dmp, MP, ncl;   // its successor
    __device__ __forceinline__ UnitWalk(int first, int ncl_, int MP_)
        : unit(first), tile(first / MP_), mp(first % MP_), dtile(ncl_ / MP_), dmp(ncl_ % MP_), MP(MP_), ncl(ncl_) {}
    // The unit's tile and expert; expert < 0 for a slot whose expert is unknown (reported, skipped)
    // and past the last unit.
    template <typename P>   // P: tiles, slot_expert, E
    __device__ __forceinline__ Unit take(const P& p, int total) {
        if (unit >= total) return Unit{0, 0, -1, 0};
        const MTile t = p.tiles[tile];
        Unit u;
        u.row0 = t.row0;
        u.rows = t.rows;
        u.mp = mp;
        u.expert = t.wsel >= 0 ? t.wsel : p.slot_expert[-1 - t.wsel];
        if (u.expert >= p.E) u.expert = -1;
        unit += ncl;
        tile += dtile;
        mp += dmp;
        if (mp >= MP) {
            mp -= MP;
            ++tile;
        }
        return u;
    }
};

__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint64_t* bar, void* dst, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(const CUtensorMap* map, uint32_t bar_cl, void* dst, int c0,
                                                 int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cl), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Named barriers of four epilogue warps.
__device__ __forceinline__ void quad_sync(int id) {
    __syncwarp();
    asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool quad_all(int id, bool v) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %2, 0;\n\t"
        "bar.red.and.pred p, %1, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(id), "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

// Rows of a unit's MMA: N in steps of 32, half of it in each CTA.
__device__ __forceinline__ int mma_rows(int rows) { return (rows + 31) & ~31; }

// The work list: tiles of at most kRows rows of one segment, in (rank, row) order. One CTA; a thread holds four segments at a time, all loaded at once (8 ranks x 433 segments: 3 us; a
// thread with four consecutive segments loaded twice took 7). A table with any inconsistent
// segment is refused as a whole.
template <int kRows>
__global__ void __launch_bounds__(1024) row_tiles_kernel(const int32_t* cu, Dims d, FastDiv nrow, Workspace ws) {
    constexpr int kS = 4, kChunk = kS * 1024;
    __shared__ int s_sum[kS * 32];
    grid_launch_dependents();   // the product may set itself up
    // cu may still be being written up to here: no load of it may come earlier, nor take the
    // non-coherent path, which the compiler may move and which wants memory constant from the start
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x < kRgTickets) ws.tickets[threadIdx.x] = 0;   // for the products that count parts
    const int items = d.R * d.NROW;
    int a[kS], len[kS];
    auto segments = [&](int base) {
        int bad = 0;
#pragma unroll
        for (int r = 0; r < kS; ++r) {
            const int i = base + r * 1024 + threadIdx.x;
            a[r] = len[r] = 0;
            if (i < items) {
                const int u = (int)fast_div((uint32_t)i, nrow);
                a[r] = cu[i + u];   // rank u's table has one more entry than segments
                len[r] = cu[i + u + 1];
            }
        }
#pragma unroll
        for (int r = 0; r < kS; ++r) {
            bad |= a[r] < 0 || len[r] < a[r] || (int64_t)len[r] > d.C;
            len[r] -= a[r];
        }
        return bad;
    };
    int bad = 0;
    for (int base = 0; base < items; base += kChunk) bad |= segments(base);
    const bool ok = !__syncthreads_or(bad);
    int total = 0;
    for (int base = 0; base < items && ok; base += kChunk) {
        if (items > kChunk) segments(base);
        int before[kS];   // tiles of this warp's run of 32 segments before this lane's
#pragma unroll
        for (int r = 0; r < kS; ++r) {
            const int n = (len[r] + kRows - 1) / kRows;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            before[r] = incl - n;
            if (lane == 31) s_sum[r * 32 + warp] = incl;
        }
        __syncthreads();
        // every warp: exclusive prefix of the 128 runs; lane l of round r holds run (r, l)
        int run_base[kS], sum = total;
#pragma unroll
        for (int r = 0; r < kS; ++r) {
            const int n = s_sum[r * 32 + lane];
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            run_base[r] = sum + __shfl_sync(0xffffffffu, incl - n, warp);
            sum += __shfl_sync(0xffffffffu, incl, 31);
        }
        total = sum;
#pragma unroll
        for (int r = 0; r < kS; ++r) {
            if (len[r] <= 0) continue;
            const int i = base + r * 1024 + threadIdx.x;
            const int u = (int)fast_div((uint32_t)i, nrow), rho = i - u * d.NROW;
            MTile t;
            t.wsel = rho < d.E ? rho : -(1 + u * d.B + (rho - d.E));
            t.pad = 0;
            MTile* out = ws.tiles + run_base[r] + before[r];
            for (int m = 0; m < len[r]; m += kRows) {
                t.row0 = (int32_t)(u * d.C + a[r] + m);
                t.rows = min(kRows, len[r] - m);
                *out++ = t;
            }
        }
        __syncthreads();   // s_sum is written again by the next chunk
    }
    if (threadIdx.x == 0) {
        if (!ok) set_status(ws.status, BEP_DERR_BOUNDS);
        *ws.ntiles = ok ? total : 0;
    }
}

// Queues the work list. It may be launched early, and so may the product after it.
template <int kRows>
cudaError_t launch_row_tiles(const Dims& d, const Workspace& ws, const int32_t* cu, cudaStream_t st) {
    cudaLaunchConfig_t tc = {};
    cudaLaunchAttribute early;
    tc.gridDim = dim3(1, 1, 1);
    tc.blockDim = dim3(1024, 1, 1);
    tc.stream = st;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    tc.attrs = &early;
    tc.numAttrs = 1;
    return cudaLaunchKernelEx(&tc, row_tiles_kernel<kRows>, cu, d, make_fast_div((uint32_t)d.NROW), ws);
}

// u8 tensor of `dims` (innermost first, dense), 128-byte boxes of
// `box_rows` rows, 128-byte swizzle.
bool encode_u8(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, uint32_t box_rows) {
    void* fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t d[3], strides[2];
    cuuint32_t box[3] = {128, box_rows, 1}, estr[3] = {1, 1, 1};
    for (int i = 0; i < rank; ++i) d[i] = dims[i];
    strides[0] = d[0];
    if (rank == 3) strides[1] = d[0] * d[1];
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
               m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), d, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace bep
