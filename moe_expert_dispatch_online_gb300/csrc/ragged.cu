// Grouped products of any width (sm_103a, tcgen05): rows grouped by expert, each group by its expert's own
// matrix, and the matrices' gradients. Widths are multiples of 8 and need not be multiples of a tile, rows may
// lie apart, and the products of replicas and of overflow rows go to the expert itself:
//   y[row, :]  = alpha * x[row, :] W(e) + add[row, :]        W(e) = w[e] [K, N], or w[e]^T with w[e] [N, K]
//   g[e]      (+)= alpha * sum over the rows of e: x[row]^T dy[row]                              (fp32)
// e = rho for a segment rho < E and slot_expert[u][rho - E] for a prefetch slot.
//
// Both kernels are persistent, one CTA an SM:
//   warp 0      TMA (128-byte swizzle) into a ring of stages of 64 reduction steps
//   warp 1      tcgen05.mma.kind::f16, M = 128 (64 where experts have few rows, 256 on a pair of CTAs), N <= 256, into
//               one of two accumulators
//   the rest    epilogue (8 or 16 warps): TMEM, summed over chains of steps, turned in shared memory, to whole pieces of rows
// What lies outside a matrix arrives as zeros (the tensor maps end at the widths). Where there are fewer units
// than SMs, the reduction is cut into parts; each part leaves its fp32 tile in the context's workspace and the CTA that
// comes last adds them in the order of the parts, so that the result does not depend on who that was.
//
// Narrow products are bound by HBM: 131,072 rows of 7168 into 16: 307 us (6.4 TB/s), back from 16: 376 us (5.2 TB/s, all
// of it writes), their gradient 327 us (6.4 TB/s; 347 us added to what was there); 64 onto 2048 with another output to add
// to: 212 us (5.6 TB/s; 316 us with the epilogue loading that itself). Wide ones by the operands' way into shared memory:
// 65,536 rows by 1088 x 1600 201 us (1.13 PFLOP/s), back 180 us, by 1096 x 1544, whose rows start inside 128-byte lines and
// take two requests a piece, 236 us, back 215 us.

#include <cudaTypedefs.h>

#include "tiles.cuh"

namespace bep {
namespace {

constexpr int kRgThreads = 32 * 10;      // 8 epilogue warps
constexpr int kRgSumThreads = 32 * 18;   // 16, where the sums of more than 128 columns are held in registers
constexpr int kRgA = 128 * 128;          // bytes: 128 rows (columns) x 64 reduction steps
constexpr int kRgChunk = 64 * 128;       // bytes: 64 x 64 elements
constexpr int kRgBox = 32 * 128;         // bytes: an epilogue warp's box of 32 rows of 128 bytes
constexpr int kRgDwBox = 16 * 128;       // bytes: the same of 16 rows of 32 fp32, written by TMA
constexpr int kRgTmem = 512;
constexpr int kRgMaxStages = 12;
constexpr int kRgMaxAdds = 4;
constexpr int kRgMaxParts = 16;
constexpr int kRgLocal = 256;            // row tiles of a small call, whose list each CTA makes itself
// Shared memory: up to 1 KB lost to alignment, 1 KB of barriers, then the ring and what the epilogue turns its boxes in.
constexpr size_t kRgSmem = 227 * 1024;
constexpr int kRgBytes = 225 * 1024;
// The tensor core cuts its fp32 sum off at each step of 16, always towards zero (7.7e-5 of a sum of 16,384 positive
// products in one chain of steps); a chain is therefore ended after this many blocks of 64 and added, rounded to nearest,
// to a sum in registers. Outputs of 16 bits have longer chains than gradients of 32 (65,536 rows by 1088 x 1600: 201 us
// with 8 blocks, 208 us with 4).
constexpr int kRgChain = 4;
constexpr int kRgRowChain = 8;

struct RgParams {
    const MTile* tiles;
    const int32_t* ntiles;
    const int32_t* cu;        // the table itself, where the CTAs make the list
    const int32_t* slot_expert;
    uint16_t* y;
    const uint16_t* add;
    int64_t ldy, ldadd;
    float alpha;
    int E, N, kbn;            // output columns, reduction blocks of 64
    int BN, NT;               // columns of a tile, tiles
    FastDiv by_nt, by_nrow;
    int tile_rows, local;
    int R, B, NROW;
    int64_t C;
    int steps;                // of 16 in a block: 4, or fewer where the reduction is shorter than a block
    int stages, a_bytes, b_bytes, chunk, adds, add_bytes;
    int32_t* tickets;
    float* partial;
    int32_t* status;
};

struct RgDwParams {
    const MTile* blocks;      // up to 64 rows of one segment, by expert
    const int32_t* first;     // [E + 1]
    int m_inner;              // the M side lies along g's rows, else the N side
    float alpha;
    int E, Md, Nd;            // widths of the sides
    int BN, MT, NT, parts;    // columns of a tile, units along M and N
    FastDiv by_parts, by_unit, by_nt;
    int stages, b_bytes;
    int accumulate;
    int32_t* tickets;
    float* partial;
    int32_t* status;
};

// A box of g written, or added (one fp32 rounding an element).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void tma_reduce_add_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
// Operand descriptors reach the instruction as a low word (address in 16-byte units, leading offset) beside a constant
// high word: 8-row groups 1024 bytes apart, version 1, 128-byte swizzle. The issuing thread's time bounds reductions
// of narrow tiles, so a stage costs it one addition an operand and the 16-step pieces constant ones.
//   K-major: rows of 64 elements (128 bytes), a piece 32 bytes along them;
//   MN-major: chunks of 64 columns x 64 reduction steps (or fewer: `chunk` bytes), a piece 16 of their rows.
#define BEP_RG_OPERAND_HI "0x40004040"
template <bool kMN>
__device__ __forceinline__ uint32_t operand_lo(uint32_t saddr, uint32_t chunk = kRgChunk) {
    return ((saddr >> 4) & 0x3FFFu) | ((kMN ? chunk >> 4 : 1u) << 16);
}
template <bool kMN>
__host__ __device__ constexpr uint32_t piece_step() { return kMN ? 128 : 2; }

// Instruction descriptor, kind::f16: fp32 accumulator, bf16 A and B, major bits 15/16 (1: MN), M = 256 (a pair), 128 or 64.
__device__ __forceinline__ uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, " BEP_RG_OPERAND_HI "};\n\t"
        "mov.b64 db, {%2, " BEP_RG_OPERAND_HI "};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(idesc), "r"(add)
        : "memory");
}

// The same on a pair of SMs: M = 256, of which each CTA holds 128 rows of A and of D, and half of B's columns.
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, " BEP_RG_OPERAND_HI "};\n\t"
        "mov.b64 db, {%2, " BEP_RG_OPERAND_HI "};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(idesc), "r"(add)
        : "memory");
}

// All epilogue warps of a kernel.
template <int kWarps>
__device__ __forceinline__ void epi_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
}
template <int kWarps>
__device__ __forceinline__ bool epi_all(bool v) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, 1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "n"(32 * kWarps)
        : "memory");
    return r != 0;
}

// What both kernels set up and take down alike.
struct Frame {
    uint8_t* ring;
    uint64_t *full, *empty, *ready, *tfull, *tempty, *afull, *aempty, *drain;
    uint32_t* s_tmem;
    volatile int* s_abort;
    int* s_last;
    int* s_rows;   // valid rows of each stage
    uint32_t tmem;
};
// kPair: MMAs are a pair's (cta_group::2).
template <bool kPair = false>
__device__ __forceinline__ Frame open_frame(uint8_t* smem_raw, int stages, int epi_warps) {
    Frame f;
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* base = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    f.ring = base + 1024;
    f.full = reinterpret_cast<uint64_t*>(base);
    f.empty = f.full + kRgMaxStages;
    f.ready = f.empty + kRgMaxStages;
    f.tfull = f.ready + kRgMaxStages;
    f.tempty = f.tfull + 2;
    f.afull = f.tempty + 2;
    f.aempty = f.afull + kRgMaxAdds;
    f.drain = f.aempty + kRgMaxAdds;
    f.s_tmem = reinterpret_cast<uint32_t*>(f.drain + 1);
    f.s_abort = reinterpret_cast<volatile int*>(f.s_tmem + 1);
    f.s_last = reinterpret_cast<int*>(f.s_tmem + 2);
    f.s_rows = f.s_last + 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&f.full[s], 1);
            mbar_init(&f.empty[s], 1);
            mbar_init(&f.ready[s], 2);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&f.tfull[a], 1);
            mbar_init(&f.tempty[a], (kPair ? 2 : 1) * epi_warps);
        }
        for (int a = 0; a < kRgMaxAdds; ++a) {
            mbar_init(&f.afull[a], 1);
            mbar_init(&f.aempty[a], epi_warps);
        }
        mbar_init(f.drain, 1);
        *f.s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x < 32) {
        __syncwarp();
        if (kPair) {   // a warp of each CTA together
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(f.s_tmem)),
                         "r"(kRgTmem)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(f.s_tmem)),
                         "r"(kRgTmem)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    f.tmem = *f.s_tmem;
    return f;
}
// What the producer started: its place in a ring and how often it armed a barrier there.
struct Started {
    uint32_t at = 0, phase = 0, armed = 0;
    __device__ __forceinline__ void step(uint32_t n) {
        ++armed;
        if (++at == n) {
            at = 0;
            phase ^= 1u;
        }
    }
    __device__ __forceinline__ void drain(uint64_t* bars, uint32_t n) {
        for (uint32_t i = 0; i < armed && i < n; ++i) {
            if (at == 0) {
                at = n;
                phase ^= 1u;
            }
            --at;
            mbar_drain(&bars[at], phase);
        }
    }
};
template <bool kPair = false>
__device__ __forceinline__ void close_frame(const Frame& f, int stages, int adds, Started ring, Started add) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (*f.s_abort) {
        // A wait gave up: what was started lands before shared memory and TMEM are released, each wait bounded.
        if (warp == 0 && lane == 0) {
            ring.drain(f.full, stages);
            if (adds) add.drain(f.afull, adds);
        } else if (warp == 1 && lane == 0 && !(kPair && cluster_rank() != 0)) {
            if (kPair) mma_commit_pair_lead(f.drain);
            else mma_commit(f.drain);
            mbar_drain(f.drain, 0);
        }
        if (kPair && threadIdx.x == 0)   // what it started for the other CTA
            for (int i = 0; i < 20; ++i) __nanosleep(10000);
        __syncthreads();
    }
    if (kPair) cluster_sync();   // neither CTA leaves while the other may still write to it or signal it
    if (warp == 0) {
        tc_fence_after();
        __syncwarp();
        if (kPair)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(f.tmem), "r"(kRgTmem) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(f.tmem), "r"(kRgTmem) : "memory");
    }
}

// A part's tile in the workspace: [column][128 rows], so that a warp's rows lie together.
constexpr int kPartRows = 128;
__device__ __forceinline__ float* part_tile(float* base, int slot) {
    return base + (int64_t)slot * (kPartRows * kRgPartCols);
}
// This thread's row, 32 columns: to a part's tile, and the sum of a unit's parts in their order.
__device__ __forceinline__ void put_part(float* tile, int c0, int row, const float* v) {
#pragma unroll
    for (int j = 0; j < 32; ++j) __stcg(tile + (c0 + j) * kPartRows + row, v[j]);
}
// 32 columns of this warp's 32 rows of an accumulator.
__device__ __forceinline__ void read_tmem(uint32_t taddr, float* v) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(taddr, r);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}
__device__ __forceinline__ void sum_parts(float* base, int slot0, int parts, int c0, int row, float* v) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __ldcg(part_tile(base, slot0) + (c0 + j) * kPartRows + row);
    for (int z = 1; z < parts; ++z) {
        const float* t = part_tile(base, slot0 + z);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += __ldcg(t + (c0 + j) * kPartRows + row);
    }
}
// True in the CTA that brings a unit's last part (all epilogue warps call it, their parts written).
template <int kWarps>
__device__ __forceinline__ bool last_part(int32_t* ticket, int parts, int* s_last) {
    __threadfence();
    epi_sync<kWarps>();
    if (threadIdx.x == 64) {
        const int n = atomicAdd(ticket, 1);
        __threadfence();
        *s_last = n == parts - 1;
        if (n == parts - 1) *ticket = 0;   // for the next call
    }
    epi_sync<kWarps>();
    const bool last = *s_last != 0;
    epi_sync<kWarps>();   // read before the next unit writes it
    return last;
}

// ------------------------------------------------------------------------ rows
// The list of row_tiles_kernel for a table of few row tiles, made in shared memory by every CTA for itself, which
// saves a launch: up to kRgLocal tiles in (rank, row) order; returns their number (0 for a bad table).
template <int kThreads>
__device__ __forceinline__ int local_tiles(const RgParams& p, int* table, MTile* out, int* s_warp) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int items = p.R * p.NROW, per = (items + kThreads - 1) / kThreads;
#pragma unroll 8
    for (int i = t; i < items + p.R; i += kThreads) table[i] = p.cu[i];
    __syncthreads();
    const int lo = min(items, t * per), hi = min(items, lo + per);
    int n = 0, bad = 0;
    auto segment = [&](int i, int* u, int* rho, int* a, int* b) {
        *u = (int)fast_div(i, p.by_nrow);
        *rho = i - *u * p.NROW;
        *a = table[i + *u];   // rank u's table has one more entry than segments
        *b = table[i + *u + 1];
    };
    for (int i = lo; i < hi; ++i) {
        int u, rho, a, b;
        segment(i, &u, &rho, &a, &b);
        bad |= a < 0 || b < a || (int64_t)b > p.C;
        n += (b - a + p.tile_rows - 1) / p.tile_rows;
    }
    __syncwarp();   // lanes leave the loops of this list at different times
    bad = __syncthreads_or(bad);
    if (bad) {
        if (blockIdx.x == 0 && t == 0) set_status(p.status, BEP_DERR_BOUNDS);
        return 0;
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int at = incl - n, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) at += s_warp[w];
        total += s_warp[w];
    }
    if (n)
        for (int i = lo; i < hi; ++i) {
            int u, rho, a, b;
            segment(i, &u, &rho, &a, &b);
            for (; a < b; a += p.tile_rows, ++at)
                if (at < kRgLocal)
                    out[at] = MTile{(int32_t)(u * p.C + a), min(p.tile_rows, b - a),
                                    rho < p.E ? rho : -(1 + u * p.B + (rho - p.E)), 0};
        }
    __syncwarp();
    // the table's place is the ring's: what was read and written here comes before the copies that land there
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    return min(total, kRgLocal);
}

// One map for each height of a box of rows.
struct RowMaps {
    CUtensorMap m16, m32, m64, m128;
};
__device__ __forceinline__ const CUtensorMap* map_for(const RowMaps& m, int rows) {
    return rows <= 16 ? &m.m16 : rows <= 32 ? &m.m32 : rows <= 64 ? &m.m64 : &m.m128;
}
__device__ __forceinline__ int box_for(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

// A unit: up to 128 rows of a segment x BN columns, or up to 64 where experts have few rows. A small tile leaves the
// accumulator's other rows to whatever the stage holds behind its own; they are not stored.
// kAdd: what the product is added to arrives by TMA, up to four units ahead, in boxes of 64 columns that the epilogue
// then turns its outputs in.
// kSum: a reduction of more than kRgRowChain blocks, whose chains take the two accumulators in turn and are summed in
// registers by so many epilogue warps, 64 columns each (0: one chain, read out of the accumulator by 8).
// kPair: up to 256 rows x BN on two CTAs of a cluster (cta_group::2): CTA r holds rows 128 r.. of A and of the output and
// half of W's columns, 32 KB a stage for 256 columns where a CTA alone loads 48 for the same rows. CTA 0's producer arms a
// stage for both and its warp 1 issues the MMAs of both.
//   barrier    owner   arrivals
//   full[s]    CTA 0   its producer's expect_tx + the TMA bytes of both
//   empty[s]   each    the MMA thread's multicast commit
//   tfull[a]   each    the MMA thread's multicast commit at the end of a chain
//   tempty[a]  CTA 0   the 16 epilogue warps of each CTA
template <bool kTrans, bool kAdd, int kSum, bool kPair>
__global__ void __launch_bounds__(kSum == 16 ? kRgSumThreads : kRgThreads, 1)
    ragged_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ RowMaps tmX,
                  const __grid_constant__ RowMaps tmAdd, const RgParams p) {
    static_assert(!kPair || (kSum && !kAdd), "a pair's reduction is long, and it adds nothing");
    constexpr bool kChain = kSum != 0;
    constexpr int kThreads = kSum == 16 ? kRgSumThreads : kRgThreads, kEpi = kThreads / 32 - 2;
    extern __shared__ uint8_t smem_raw[];
    grid_launch_dependents();
    const int nbox = (p.BN + 63) / 64;   // boxes of 64 columns
    Frame f = open_frame<kPair>(smem_raw, p.stages, kChain ? 4 * nbox : kEpi);
    if (kPair) cluster_sync();   // both CTAs' barriers exist
    const int rank = kPair ? (int)cluster_rank() : 0;
    const int first = kPair ? (int)cluster_id() : (int)blockIdx.x, stride = kPair ? (int)cluster_count() : (int)gridDim.x;
    uint8_t* smA = f.ring;
    uint8_t* smB = smA + p.stages * p.a_bytes;
    uint8_t* smT = smB + p.stages * p.b_bytes;   // kAdd: the units' boxes, else a box of each epilogue warp with columns
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Started pr, ad;
    grid_wait();   // launched early: the work list and the rows are complete from here on

    const MTile* tiles = p.tiles;
    int ntiles;
    if (p.local) {
        MTile* list = reinterpret_cast<MTile*>(f.ring + kRgBytes - kRgLocal * sizeof(MTile));
        ntiles = local_tiles<kThreads>(p, reinterpret_cast<int*>(f.ring), list, f.s_rows);   // (the ring is not in use yet)
        tiles = list;
    } else {
        ntiles = *p.ntiles;
    }
    const int units = ntiles * p.NT;
    int parts = 1;
    if (p.partial && units > 0) parts = max(1, min(min((int)gridDim.x / units, p.kbn / 4), kRgMaxParts));
    const int total = units * parts;
    struct Item {
        int row0, rows, expert, n0, unit, kb0, kb1;
    };
    // A CTA's next tile is read a unit ahead: a unit may last no longer than the load.
    auto unit_of = [&](int i) { return parts == 1 ? i : i / parts; };
    auto tile_at = [&](int i) { return i < total ? tiles[fast_div(unit_of(i), p.by_nt)] : MTile{0, 0, 0, 0}; };
    auto item_of = [&](int i, const MTile& t) {
        Item it;
        it.unit = unit_of(i);
        it.row0 = t.row0;
        it.rows = t.rows;
        it.expert = t.wsel >= 0 ? t.wsel : p.slot_expert[-1 - t.wsel];
        if (it.expert >= p.E) it.expert = -1;
        it.n0 = (it.unit - (int)fast_div(it.unit, p.by_nt) * p.NT) * p.BN;
        it.kb0 = 0;
        it.kb1 = p.kbn;
        if (parts > 1) {
            const int part = i - it.unit * parts;
            it.kb0 = part * p.kbn / parts;
            it.kb1 = (part + 1) * p.kbn / parts;
        }
        return it;
    };
    MTile next = tile_at(first);

    if (warp == 0) {
        if (lane == 0) {
            bool live = true;
            uint32_t bar0 = kPair ? cluster_addr(f.full, 0) : 0;
            for (int i = first; i < total && live; i += stride) {
                const Item u = item_of(i, next);
                next = tile_at(i + stride);
                if (u.expert < 0) {
                    if (rank == 0) set_status(p.status, BEP_DERR_BOUNDS);
                    continue;
                }
                // rows of the unit's first 128 and of the others; this CTA's
                const int rows0 = kPair ? min(u.rows, 128) : u.rows, rows1 = u.rows - rows0;
                const int box0 = box_for(rows0), box1 = rows1 > 0 ? box_for(rows1) : 0;
                const int box = rank ? box1 : box0, row0 = u.row0 + 128 * rank;
                const CUtensorMap* mx = map_for(tmX, rank ? rows1 : rows0);
                const int bytes = kPair ? (box0 + box1) * 128 + 2 * p.b_bytes : box * 128 + p.b_bytes;
                const int n0 = kPair ? u.n0 + rank * (p.BN / 2) : u.n0;
                for (int kb = u.kb0; kb < u.kb1; ++kb) {
                    if (!mbar_wait_held(&f.empty[pr.at], pr.phase ^ 1u, f.s_abort, p.status)) {
                        live = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&f.full[pr.at], bytes);
                    uint8_t* a = smA + pr.at * p.a_bytes;
                    uint8_t* b = smB + pr.at * p.b_bytes;
                    if (kPair) {
                        const uint32_t bar = bar0 + pr.at * 8;
                        if (box) tma_load_2d_pair(mx, bar, a, kb * 64, row0);
                        if (kTrans)
                            tma_load_3d_pair(&tmW, bar, b, kb * 64, n0, u.expert);
                        else
                            for (int c = 0; c * p.chunk < p.b_bytes; ++c)
                                tma_load_3d_pair(&tmW, bar, b + c * p.chunk, n0 + c * 64, kb * 64, u.expert);
                    } else {
                        tma_load_2d(mx, &f.full[pr.at], a, kb * 64, row0);
                        if (kTrans)
                            tma_load_3d(&tmW, &f.full[pr.at], b, kb * 64, n0, u.expert);
                        else
                            for (int c = 0; c * p.chunk < p.b_bytes; ++c)
                                tma_load_3d(&tmW, &f.full[pr.at], b + c * p.chunk, n0 + c * 64, kb * 64, u.expert);
                    }
                    pr.step(p.stages);
                }
                if (kAdd && parts == 1 && live) {
                    if (!mbar_wait_held(&f.aempty[ad.at], ad.phase ^ 1u, f.s_abort, p.status)) break;
                    const CUtensorMap* ma = map_for(tmAdd, u.rows);
                    mbar_arrive_expect_tx(&f.afull[ad.at], p.add_bytes / 128 * box);
                    for (int c = 0; c * kRgA < p.add_bytes; ++c)
                        tma_load_2d(ma, &f.afull[ad.at], smT + ad.at * p.add_bytes + c * kRgA, u.n0 + c * 64, u.row0);
                    ad.step(p.adds);
                }
            }
            if (kPair && live) {   // CTA 0's commits have arrived
                Started e = pr;
                e.drain(f.empty, p.stages);
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            const uint32_t idesc = idesc_bf16(kPair ? 256 : p.tile_rows, p.BN, false, !kTrans);
            const uint32_t a0 = operand_lo<false>(smem_u32(smA)), b0 = operand_lo<!kTrans>(smem_u32(smB), p.chunk);
            const uint32_t a_step = p.a_bytes >> 4, b_step = p.b_bytes >> 4;
            constexpr uint32_t sa = piece_step<false>(), sb = piece_step<!kTrans>();
            auto mma = [&](uint32_t dt, uint32_t aa, uint32_t bb, uint32_t add) {
                if (kPair) mma_bf16_pair(dt, aa, bb, idesc, add);
                else mma_bf16(dt, aa, bb, idesc, add);
            };
            auto commit = [&](uint64_t* bar) {
                if (kPair) mma_commit_pair(bar);
                else mma_commit(bar);
            };
            uint32_t s = 0, ph = 0, a = a0, b = b0;
            int it = 0;
            bool live = true;
            for (int i = first; i < total && live; i += stride) {
                const Item u = item_of(i, next);
                next = tile_at(i + stride);
                if (u.expert < 0) continue;
                int left = u.kb1 - u.kb0;   // blocks
                // chains of about the same length: each hides the way of the one before into registers
                for (int nc = kChain ? (left + kRgRowChain - 1) / kRgRowChain : 1; nc > 0 && live; --nc, ++it) {
                    const int acc = it & 1, len = kChain ? (left + nc - 1) / nc : left;
                    left -= len;
                    if (!mbar_wait_held<kPair>(&f.tempty[acc], ((it >> 1) & 1) ^ 1u, f.s_abort, p.status)) {
                        live = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t dt = f.tmem + acc * 256;
                    for (int k = 0; k < len; ++k) {
                        if (!mbar_wait_held(&f.full[s], ph, f.s_abort, p.status)) {
                            live = false;
                            break;
                        }
                        tc_fence_after();
                        mma(dt, a, b, k != 0);
                        if (kChain || p.steps == 4) {
                            mma(dt, a + sa, b + sb, 1);
                            mma(dt, a + 2 * sa, b + 2 * sb, 1);
                            mma(dt, a + 3 * sa, b + 3 * sb, 1);
                        } else {
                            for (int kk = 1; kk < p.steps; ++kk) mma(dt, a + kk * sa, b + kk * sb, 1);
                        }
                        commit(&f.empty[s]);
                        a += a_step;
                        b += b_step;
                        if (++s == (uint32_t)p.stages) {
                            s = 0;
                            ph ^= 1u;
                            a = a0;
                            b = b0;
                        }
                    }
                    if (live) commit(&f.tfull[acc]);
                }
            }
        }
    } else {
        // The warps of each quarter of the accumulator's rows share its boxes of 64 columns. A box is turned in shared
        // memory, so that 8 lanes write 128 bytes of a row of y.
        // (a tile of 64 rows has 16 of them in each quarter's first lanes)
        const int q = warp & 3, group = (warp - 2) >> 2, span = kPair ? 32 : p.tile_rows / 4;
        const int sub = lane >> 3, piece = lane & 7;
        const int mine = kChain ? 1 : (nbox + 1) / 2;
        const int box0 = group * mine, box1 = min(nbox, box0 + mine);
        const bool idle = kChain && box0 >= box1;   // such warps only meet the others at barriers
        constexpr int kBoxes = kChain ? 1 : 2;       // a warp's at most
        constexpr bool kHalf = kChain && !kAdd;      // turned 16 rows at a time, which leaves room for more stages
        int it = 0;
        uint32_t as = 0, aph = 0;
        for (int i = first; i < total; i += stride) {
            const Item u = item_of(i, next);
            next = tile_at(i + stride);
            if (u.expert < 0) continue;
            const int rows = min(u.rows - 128 * rank - span * q, span);   // this warp's
            const int64_t row0 = (int64_t)u.row0 + 128 * rank + span * q;
            float sum[kChain ? 2 : 1][32];   // this thread's row of the warp's box, else of 32 columns at a time
            bool done = true, held = true;
            auto release = [&](int acc) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair) mbar_arrive_rank_relaxed(&f.tempty[acc], 0);
                    else mbar_arrive(&f.tempty[acc]);
                }
                held = false;
            };
            if (kChain) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[kChain ? h : 0][j] = 0.0f;
                for (int c0 = u.kb0; c0 < u.kb1 && !idle; c0 += kRgRowChain) {
                    const int acc = it & 1;
                    done = __all_sync(0xffffffffu, mbar_wait_held(&f.tfull[acc], (it >> 1) & 1, f.s_abort, p.status));
                    if (!done) break;
                    ++it;
                    tc_fence_after();
                    const uint32_t tacc = f.tmem + ((uint32_t)(q * 32) << 16) + acc * 256 + 64 * box0;
                    if (rows > 0)
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            if (64 * box0 + 16 * h >= p.BN) break;
                            uint32_t r[16];
                            tmem_ld_32x32b_x16(tacc + 16 * h, r);
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum[kChain ? h >> 1 : 0][16 * (h & 1) + j] += __uint_as_float(r[j]);
                        }
                    release(acc);
                }
            } else {
                done = __all_sync(0xffffffffu, mbar_wait_held(&f.tfull[it & 1], (it >> 1) & 1, f.s_abort, p.status));
            }
            if (kAdd && parts == 1 && !idle)
                done = done && __all_sync(0xffffffffu, mbar_wait_held(&f.afull[as], aph, f.s_abort, p.status));
            // (warps that meet at barriers give up together)
            if (parts > 1 ? !epi_all<kEpi>(done) : !done) break;
            const int acc = it & 1;   // (!kChain)
            const uint32_t tacc = f.tmem + ((uint32_t)(q * 32) << 16) + acc * 256;
            if (!kChain) {
                ++it;
                tc_fence_after();
            }
            const int slot0 = u.unit * parts;
            bool mine_to_store = true;
            if (parts > 1) {
                if (kChain) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (!idle && 64 * box0 + 32 * h < p.BN)
                            put_part(part_tile(p.partial, i), 64 * box0 + 32 * h, 32 * q + lane, sum[kChain ? h : 0]);
                } else {
                    for (int c0 = 64 * box0; c0 < min(64 * box1, p.BN); c0 += 32) {
                        float r[32];
                        read_tmem(tacc + c0, r);
                        put_part(part_tile(p.partial, i), c0, 32 * q + lane, r);
                    }
                    release(acc);
                }
                mine_to_store = last_part<kEpi>(p.tickets + u.unit, parts, f.s_last);
            }
#pragma unroll
            for (int b = 0; b < kBoxes; ++b) {
                const int bx = box0 + b;
                if (bx >= box1 || !mine_to_store || (kChain && rows <= 0)) break;
                uint8_t* stg = kAdd ? smT + as * p.add_bytes + bx * kRgA + q * span * 128
                                    : smT + (warp - 2) * (kHalf ? kRgBox / 2 : kRgBox);
                uint4* line = reinterpret_cast<uint4*>(stg + lane * 128);   // this lane's row of the box
                const int c = 64 * bx + 8 * piece;
                const bool in = c < p.BN && u.n0 + c < p.N;
                __syncwarp();   // the box before has been read
                if (kAdd && parts > 1) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (in && 4 * j + sub < rows)
                            *reinterpret_cast<uint4*>(stg + (4 * j + sub) * 128 + ((piece ^ ((4 * j + sub) & 7)) << 4)) =
                                *reinterpret_cast<const uint4*>(p.add + (row0 + 4 * j + sub) * p.ldadd + u.n0 + c);
                    __syncwarp();
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c0 = 64 * bx + 32 * h;
                    if (c0 >= p.BN) break;
                    float* r = sum[kChain ? h : 0];
                    if (parts > 1) sum_parts(p.partial, slot0, parts, c0, 32 * q + lane, r);
                    else if (!kChain) read_tmem(tacc + c0, r);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint4& at = line[(4 * h + j) ^ (lane & 7)];
                        uint32_t w[4];
                        if (kAdd) {
                            const uint4 t = lane < span ? at : make_uint4(0, 0, 0, 0);
                            w[0] = t.x;
                            w[1] = t.y;
                            w[2] = t.z;
                            w[3] = t.w;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float lo = r[8 * j + 2 * e], hi = r[8 * j + 2 * e + 1];
                            if (kAdd) {
                                lo = fmaf(p.alpha, lo, __uint_as_float(w[e] << 16));
                                hi = fmaf(p.alpha, hi, __uint_as_float(w[e] & 0xffff0000u));
                            } else {
                                lo *= p.alpha;
                                hi *= p.alpha;
                            }
                            w[e] = pack_bf16x2(lo, hi);
                        }
                        if (kHalf) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) r[4 * j + e] = __uint_as_float(w[e]);
                        } else if (lane < span) {   // (the others' place is another warp's)
                            at = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                if (!kChain && held && bx + 1 == box1) release(acc);   // this warp has read all its columns
                uint16_t* out = p.y + (row0 + sub) * p.ldy + u.n0 + c;
#pragma unroll
                for (int half = 0; half < (kHalf ? 2 : 1); ++half) {
                    if (kHalf) {
                        if (half) __syncwarp();   // the first 16 rows have been read
                        if ((lane >> 4) == half)
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                reinterpret_cast<float4*>(stg + (lane & 15) * 128)[j ^ (lane & 7)] = make_float4(
                                    sum[kChain ? j >> 2 : 0][4 * (j & 3)], sum[kChain ? j >> 2 : 0][4 * (j & 3) + 1],
                                    sum[kChain ? j >> 2 : 0][4 * (j & 3) + 2], sum[kChain ? j >> 2 : 0][4 * (j & 3) + 3]);
                    }
                    __syncwarp();
                    if (in) {
#pragma unroll
                        for (int j = 0; j < (kHalf ? 4 : 8); ++j) {
                            const int row = 4 * j + sub, at = 16 * half + 4 * j;   // in the box, and of the warp's rows
                            if (at + sub < rows)
                                *reinterpret_cast<uint4*>(out + (int64_t)at * p.ldy) =
                                    *reinterpret_cast<const uint4*>(stg + row * 128 + ((piece ^ (row & 7)) << 4));
                        }
                    }
                }
            }
            if (!kChain && held) release(acc);   // a warp without columns
            if (kAdd && parts == 1 && !idle) {
                // the boxes were read and written here; the next unit's come by TMA
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&f.aempty[as]);
                if (++as == (uint32_t)p.adds) {
                    as = 0;
                    aph ^= 1u;
                }
            }
        }
    }
    // (what CTA 1 loads counts on CTA 0's barriers)
    close_frame<kPair>(f, p.stages, kAdd ? p.adds : 0, rank ? Started() : pr, ad);
}

// ------------------------------------------------------------------------ matrices
// Blocks of up to 64 rows of each expert's segments: first its home rows', then its slots', each in (rank, row) order, at
// tiles[first[e] .. first[e + 1]). One CTA. A slot whose expert is unknown is reported and left out; a table with any
// inconsistent segment is refused as a whole.
__global__ void __launch_bounds__(1024) ragged_blocks_kernel(const int32_t* cu, const int32_t* slot_expert, Dims d,
                                                             Workspace ws) {
    static_assert(kMaxE == 2048, "two experts, and two slots, a thread");   // there are at most as many slots as experts
    __shared__ int s_home[kMaxE], s_pos[kMaxE];     // blocks of the expert's home rows; of all, then where they begin
    __shared__ int2 s_slot[kMaxE];                  // expert and blocks of each slot
    __shared__ int s_sum[32];
    grid_launch_dependents();
    grid_wait();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int nslots = d.R * d.B, pitch = d.NROW + 1;
    if (t < kRgTickets) ws.tickets[t] = 0;
    auto blocks = [](int a, int b) { return (b - a + 63) / 64; };
    int bad = 0, unknown = 0;
    constexpr int kU = 8;   // ranks whose entries are read at once
    for (int e = t; e < kMaxE; e += 1024) {
        int n = 0;
        if (e < d.E)
            for (int u0 = 0; u0 < d.R; u0 += kU) {
                int a[kU], b[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    a[u] = b[u] = 0;
                    if (u0 + u < d.R) {
                        a[u] = cu[(u0 + u) * pitch + e];
                        b[u] = cu[(u0 + u) * pitch + e + 1];
                    }
                }
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    bad |= a[u] < 0 || b[u] < a[u] || (int64_t)b[u] > d.C;
                    n += blocks(a[u], b[u]);
                }
            }
        s_home[e] = s_pos[e] = n;
    }
    __syncthreads();
    int sa[2] = {0, 0}, sb[2] = {0, 0}, se[2] = {-1, -1};   // this thread's slots
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = t + 1024 * k;
        if (i >= nslots) continue;
        const int u = i / d.B, j = i - u * d.B;
        sa[k] = cu[u * pitch + d.E + j];
        sb[k] = cu[u * pitch + d.E + j + 1];
        const int e = slot_expert[i];
        bad |= sa[k] < 0 || sb[k] < sa[k] || (int64_t)sb[k] > d.C;
        if (sb[k] > sa[k]) {
            if (e >= 0 && e < d.E) se[k] = e;
            else unknown = 1;
        }
        const int n = blocks(sa[k], sb[k]);
        s_slot[i] = make_int2(se[k], n);
        if (se[k] >= 0) atomicAdd(&s_pos[se[k]], n);
    }
    bad = __syncthreads_or(bad);
    unknown = __syncthreads_or(unknown);
    if ((bad || unknown) && t == 0) set_status(ws.status, BEP_DERR_BOUNDS);
    // exclusive scan of the blocks
    const int n0 = s_pos[2 * t], n1 = s_pos[2 * t + 1];
    int incl = n0 + n1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += s_sum[w];
    const int at = before + incl - n0 - n1;
    s_pos[2 * t] = at;
    s_pos[2 * t + 1] = at + n0;
    if (2 * t <= d.E) ws.blk_first[2 * t] = bad ? -1 : at;
    if (2 * t + 1 <= d.E) ws.blk_first[2 * t + 1] = bad ? -1 : at + n0;
    if (t == 1023 && d.E == kMaxE) ws.blk_first[kMaxE] = bad ? -1 : at + n0 + n1;
    __syncthreads();
    if (bad) return;
    // A warp's lanes hold a segment each; long ones are written by the warp together.
    auto put = [&](int at, int u, int a, int b) {
        const int n = blocks(a, b);
        const bool many = n > 8;
        if (!many)
            for (int k = 0; k < n; ++k)
                ws.tiles[at + k] = MTile{(int32_t)(u * d.C + a + 64 * k), min(64, b - a - 64 * k), 0, 0};
        for (unsigned todo = __ballot_sync(0xffffffffu, many); todo; todo &= todo - 1) {
            const int src = __ffs(todo) - 1;
            const int at1 = __shfl_sync(0xffffffffu, at, src), a1 = __shfl_sync(0xffffffffu, a, src);
            const int b1 = __shfl_sync(0xffffffffu, b, src), u1 = __shfl_sync(0xffffffffu, u, src), n1 = blocks(a1, b1);
            for (int k = lane; k < n1; k += 32)
                ws.tiles[at1 + k] = MTile{(int32_t)(u1 * d.C + a1 + 64 * k), min(64, b1 - a1 - 64 * k), 0, 0};
        }
    };
    for (int e = t; e < kMaxE; e += 1024) {
        int at = s_pos[e];
        for (int u = 0; u < d.R; ++u) {
            const int a = e < d.E ? cu[u * pitch + e] : 0, b = e < d.E ? cu[u * pitch + e + 1] : 0;
            put(at, u, a, b);
            at += blocks(a, b);
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {   // a slot lies behind the expert's earlier slots: several may hold one expert
        const int i = t + 1024 * k;
        int at = 0;
        if (se[k] >= 0) {
            at = s_pos[se[k]] + s_home[se[k]];
            for (int j = 0; j < i; ++j)
                if (s_slot[j].x == se[k]) at += s_slot[j].y;
        }
        put(at, i < nslots ? i / d.B : 0, se[k] >= 0 ? sa[k] : 0, se[k] >= 0 ? sb[k] : 0);
    }
}

// Zeroes the rows [tail, 16 * ceil(tail / 16)) of a stage's `chunks` chunks of 64 x 64 (whole 128-byte rows, so the
// swizzle does not matter) and makes that visible to the tensor core. Warp-wide.
__device__ __forceinline__ void zero_rows(uint8_t* chunk, int chunks, int tail, int lane) {
    const int rows = 16 - (tail & 15);
    for (int i = lane; i < rows * 8 * chunks; i += 32) {
        const int c = i / (rows * 8), rest = i - c * rows * 8;
        *reinterpret_cast<uint4*>(chunk + c * kRgChunk + (tail + (rest >> 3)) * 128 + (rest & 7) * 16) =
            make_uint4(0, 0, 0, 0);
    }
}

// A unit: MI x 128 x BN of an expert's gradient, MI = 2 where BN leaves both room in an accumulator. Both
// operands lie along the rows (MN-major).
// kPair: 256 x BN on two CTAs of a cluster (cta_group::2): CTA r holds 128 of the M side's columns and half of the N
// side's, 32 KB a stage where a CTA alone loads 48 for half of the tile (65,536 rows by 1096 x 1544: 325 us on CTAs of
// their own, 302 us where each loaded half of the N side for both, 272 us with MMAs of the pair). In each CTA one more
// warp waits for the stage, clears the rows behind the segment's last and tells CTA 0, whose warp 1 issues the MMAs of
// both. (That signal releases shared memory alone: one that waits for all of the thread's stores took 2,000 cycles a
// stage, twice the time.)
//   barrier    owner   arrivals
//   full[s]    each    the producer's expect_tx + TMA bytes
//   ready[s]   CTA 0   the clearing warp of each CTA
//   empty[s]   each    the MMA thread's multicast commit
//   tfull[a]   each    the MMA thread's multicast commit at the end of a chain
//   tempty[a]  CTA 0   the 16 epilogue warps of each CTA
template <int MI, bool kPair>
__global__ void __launch_bounds__(kRgSumThreads + (kPair ? 32 : 0), 1) ragged_dw_kernel(const __grid_constant__ CUtensorMap tmM,
                                                                  const __grid_constant__ CUtensorMap tmN,
                                                                  const __grid_constant__ CUtensorMap tmG,
                                                                  const RgDwParams p) {
    extern __shared__ uint8_t smem_raw[];
    grid_launch_dependents();
    Frame f = open_frame<kPair>(smem_raw, p.stages, 16);
    if (kPair) cluster_sync();   // both CTAs' barriers exist
    const int rank = kPair ? (int)cluster_rank() : 0;
    const int first = kPair ? (int)cluster_id() : (int)blockIdx.x, stride = kPair ? (int)cluster_count() : (int)gridDim.x;
    constexpr int a_bytes = MI * kRgA;
    const int stage = a_bytes + p.b_bytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Started pr;
    grid_wait();   // launched early: the segments and the rows are complete from here on

    const int parts = p.parts;
    const int total = p.first[0] < 0 ? 0 : p.E * p.MT * p.NT * parts;
    struct Item {
        int unit, expert, m0, n0, b0, b1;
    };
    auto expert_at = [&](int i) { return fast_div(fast_div(i, p.by_parts), p.by_unit); };
    // An expert's range of blocks is read a unit ahead.
    auto range_at = [&](int i) {
        const uint32_t e = i < total ? expert_at(i) : 0;
        return make_int2(p.first[e], p.first[e + 1]);
    };
    auto item_of = [&](int i, const int2& range) {
        Item it;
        it.unit = fast_div(i, p.by_parts);
        const int part = i - it.unit * parts;
        it.expert = fast_div(it.unit, p.by_unit);
        const int rest = it.unit - it.expert * p.MT * p.NT, m = fast_div(rest, p.by_nt);
        it.m0 = (kPair ? 2 * m + rank : m) * MI * 128;
        it.n0 = (rest - m * p.NT) * p.BN;
        const int64_t nb = range.y - range.x;
        it.b0 = parts == 1 ? range.x : range.x + (int)(part * nb / parts);
        it.b1 = parts == 1 ? range.y : range.x + (int)((part + 1) * nb / parts);
        return it;
    };
    int2 next = range_at(first);

    if (warp == 0) {
        // 32 blocks at a time, a lane each; a unit's first 32 are read while the unit before runs
        auto blocks_at = [&](int b, int end) { return b + lane < end ? p.blocks[b + lane] : MTile{0, 0, 0, 0}; };
        auto first_of = [&](int i) {
            if (i >= total) return MTile{0, 0, 0, 0};
            const Item u = item_of(i, next);
            return blocks_at(u.b0, u.b1);
        };
        bool live = true;
        MTile run = first_of(first);
        for (int i = first; i < total && live; i += stride) {
            const Item u = item_of(i, next);
            next = range_at(i + stride);
            MTile cur = run;
            run = first_of(i + stride);
            for (int b = u.b0; b < u.b1; ++b) {
                const int k = (b - u.b0) & 31;
                if (k == 0 && b != u.b0) cur = blocks_at(b, u.b1);
                const int row0 = __shfl_sync(0xffffffffu, cur.row0, k), rows = __shfl_sync(0xffffffffu, cur.rows, k);
                if (!__all_sync(0xffffffffu, mbar_wait_held(&f.empty[pr.at], pr.phase ^ 1u, f.s_abort, p.status))) {
                    live = false;
                    break;
                }
                if (elect_one()) {
                    f.s_rows[pr.at] = rows;   // for the warp that waits on `full`
                    mbar_arrive_expect_tx(&f.full[pr.at], stage);
                    uint8_t* at = f.ring + pr.at * stage;
                    for (int c = 0; c < 2 * MI; ++c)
                        tma_load_2d(&tmM, &f.full[pr.at], at + c * kRgChunk, u.m0 + 64 * c, row0);
                    const int n0 = u.n0 + rank * (p.BN / 2);
                    for (int c = 0; c * kRgChunk < p.b_bytes; ++c)
                        tma_load_2d(&tmN, &f.full[pr.at], at + a_bytes + c * kRgChunk, n0 + 64 * c, row0);
                }
                __syncwarp();
                pr.step(p.stages);
            }
        }
        if (kPair && live && lane == 0) {   // CTA 0's commits have arrived
            Started e = pr;
            e.drain(f.empty, p.stages);
        }
    } else if (warp == 1) {
        const uint32_t idesc = idesc_bf16(kPair ? 256 : 128, p.BN, true, true);
        uint32_t s = 0, ph = 0;
        int it = 0;
        bool live = !kPair || rank == 0;
        for (int i = first; i < total && live; i += stride) {
            const Item u = item_of(i, next);
            next = range_at(i + stride);
            for (int b = u.b0; b < u.b1 && live; ++b) {
                const int k = (b - u.b0) % kRgChain;
                const int acc = it & 1;
                const uint32_t dt = f.tmem + acc * 256;
                bool ok = k != 0 || mbar_wait_held<kPair>(&f.tempty[acc], ((it >> 1) & 1) ^ 1u, f.s_abort, p.status);
                ok = ok && mbar_wait_held<kPair>(kPair ? &f.ready[s] : &f.full[s], ph, f.s_abort, p.status);
                if (!__all_sync(0xffffffffu, ok)) {
                    live = false;
                    break;
                }
                const int rows = f.s_rows[s];
                uint8_t* at = f.ring + s * stage;
                if (!kPair && (rows & 15)) {   // the rows behind a segment's last are another's, or nobody's
                    zero_rows(at, stage / kRgChunk, rows, lane);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                if (elect_one()) {
                    tc_fence_after();
                    const uint32_t a = operand_lo<true>(smem_u32(at)), bb = a + (a_bytes >> 4);
                    constexpr uint32_t st = piece_step<true>();
#pragma unroll
                    for (int m = 0; m < MI; ++m)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            if (16 * kk < rows) {
                                if (kPair) mma_bf16_pair(dt, a + kk * st, bb + kk * st, idesc, k || kk);
                                else mma_bf16(dt + m * 128, a + m * (kRgA >> 4) + kk * st, bb + kk * st, idesc, k || kk);
                            }
                    const bool end = k == kRgChain - 1 || b == u.b1 - 1;
                    if (kPair) {
                        mma_commit_pair(&f.empty[s]);
                        if (end) mma_commit_pair(&f.tfull[acc]);
                    } else {
                        mma_commit(&f.empty[s]);
                        if (end) mma_commit(&f.tfull[acc]);
                    }
                }
                __syncwarp();
                if (k == kRgChain - 1 || b == u.b1 - 1) ++it;
                if (++s == (uint32_t)p.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
    } else if (kPair && warp == kRgSumThreads / 32) {
        uint32_t s = 0, ph = 0;
        bool live = true;
        for (int i = first; i < total && live; i += stride) {
            const Item u = item_of(i, next);
            next = range_at(i + stride);
            for (int b = u.b0; b < u.b1; ++b) {
                if (!__all_sync(0xffffffffu, mbar_wait_held(&f.full[s], ph, f.s_abort, p.status))) {
                    live = false;
                    break;
                }
                const int rows = f.s_rows[s];
                if (rows & 15) {
                    zero_rows(f.ring + s * stage, stage / kRgChunk, rows, lane);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_rank_shared(&f.ready[s], 0);
                if (++s == (uint32_t)p.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
    } else {
        const int q = warp & 3, group = (warp - 2) >> 2;   // four groups of four warps, one a quarter of the rows
        uint8_t* stg = f.ring + p.stages * stage + (warp - 2) * kRgDwBox;
        // A warp's two boxes of 32 columns: every fourth one of the tile, or every second one of one of two tiles.
        constexpr int step = MI == 2 ? 64 : 128;
        const int start = MI == 2 ? 32 * (group & 1) : 32 * group, tile = MI == 2 ? group >> 1 : 0;
        int it = 0;
        bool live = true;
        for (int i = first; i < total && live; i += stride) {
            const Item u = item_of(i, next);
            next = range_at(i + stride);
            if (u.b0 == u.b1 && parts == 1 && p.accumulate) continue;
            float sum[2][32];   // this thread's row
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[b][j] = 0.0f;
            for (int b0 = u.b0; b0 < u.b1; b0 += kRgChain) {
                const int acc = it & 1;
                if (!__all_sync(0xffffffffu, mbar_wait_held(&f.tfull[acc], (it >> 1) & 1, f.s_abort, p.status))) {
                    live = false;
                    break;
                }
                ++it;
                tc_fence_after();
                const uint32_t tacc = f.tmem + ((uint32_t)(q * 32) << 16) + acc * 256 + tile * 128;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int c0 = start + b * step;
                    if (c0 >= p.BN) break;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t r[16];
                        tmem_ld_32x32b_x16(tacc + c0 + 16 * h, r);
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[b][16 * h + j] += __uint_as_float(r[j]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (kPair) mbar_arrive_rank_relaxed(&f.tempty[acc], 0);
                    else mbar_arrive(&f.tempty[acc]);
                }
            }
            if (parts > 1) {
                // (warps that meet at barriers give up together)
                if (!epi_all<16>(live)) break;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (start + b * step >= p.BN) break;
                    put_part(part_tile(p.partial, i), start + b * step, 32 * q + lane, sum[b]);
                }
                if (!last_part<16>(p.tickets + u.unit, parts, f.s_last)) continue;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (start + b * step >= p.BN) break;
                    sum_parts(p.partial, u.unit * parts, parts, start + b * step, 32 * q + lane, sum[b]);
                }
            }
            if (!live) break;
            // Boxes of 16 rows of g, 32 values of each, leave by TMA, which ends them at g's edges: the M side's 32 of
            // 16 columns, or 16 of the M side by 32 columns. (128-byte swizzle: 16-byte pieces, turned by the row.)
            const int m0 = u.m0 + tile * 128 + 32 * q;   // this warp's 32 along M
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int c0 = start + b * step, n0 = u.n0 + c0;
                if (c0 >= p.BN || n0 >= p.Nd || m0 >= p.Md) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int m = p.m_inner ? m0 : m0 + 16 * h, n = p.m_inner ? n0 + 16 * h : n0;
                    if (m >= p.Md || n >= p.Nd || (p.m_inner && c0 + 16 * h >= p.BN)) break;
                    if (lane == 0) bulk_wait_read_all();   // the box before has been read
                    __syncwarp();
                    if (p.m_inner) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            *reinterpret_cast<float*>(stg + j * 128 + (((lane >> 2) ^ (j & 7)) << 4) + (lane & 3) * 4) =
                                p.alpha * sum[b][16 * h + j];
                    } else if ((lane >> 4) == h) {
                        uint8_t* line = stg + (lane & 15) * 128;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<float4*>(line + ((j ^ (lane & 7)) << 4)) =
                                make_float4(p.alpha * sum[b][4 * j], p.alpha * sum[b][4 * j + 1],
                                            p.alpha * sum[b][4 * j + 2], p.alpha * sum[b][4 * j + 3]);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        const int x = p.m_inner ? m : n, y = p.m_inner ? n : m;
                        if (p.accumulate) tma_reduce_add_3d(&tmG, stg, x, y, u.expert);
                        else tma_store_3d(&tmG, stg, x, y, u.expert);
                        bulk_commit();
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();
    }
    close_frame<kPair>(f, p.stages, 0, pr, Started());
}

// bf16 tensor of `dims` (innermost first) with row strides in elements, boxes of 64 x box_rows, 128-byte swizzle.
bool encode_rows(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* ld, uint32_t box_rows) {
    void* fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t d[3], strides[2];
    cuuint32_t box[3] = {64, box_rows, 1}, estr[3] = {1, 1, 1};
    for (int i = 0; i < rank; ++i) d[i] = dims[i];
    for (int i = 0; i + 1 < rank; ++i) strides[i] = ld[i] * 2;
    // L2 fetches lines in pairs where no row starts inside a pair: 262,144 rows of 600 and 1000, whose rows do, take 319 us
    // instead of 334 (product) and 353 instead of 412 (gradient) with single lines, 131,072 of 7168, which do not, 332 instead of 326.
    bool whole = reinterpret_cast<uintptr_t>(base) % 256 == 0;
    for (int i = 0; i + 1 < rank; ++i) whole = whole && strides[i] % 256 == 0;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
               m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               whole ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// g fp32 [E, K, N], boxes of 16 rows of 32, 128-byte swizzle.
bool encode_g(CUtensorMap* m, float* g, int E, int K, int N) {
    void* fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)N, (cuuint64_t)K, (cuuint64_t)E};
    const cuuint64_t strides[2] = {(cuuint64_t)N * 4, (cuuint64_t)N * K * 4};
    const cuuint32_t box[3] = {32, 16, 1}, estr[3] = {1, 1, 1};
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
               m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, g, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

cudaLaunchConfig_t rg_config(int grid, int threads, cudaStream_t st, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = kRgSmem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Pairs of CTAs.
cudaLaunchConfig_t rg_pair_config(int pairs, int threads, cudaStream_t st, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = rg_config(2 * pairs, threads, st, attr);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cfg;
}

using RowKernel = void (*)(CUtensorMap, RowMaps, RowMaps, RgParams);
template <int kSum, bool kPair>
RowKernel row_kernel(bool trans, bool add) {
    if (kPair || !add) return trans ? ragged_kernel<true, false, kSum, kPair> : ragged_kernel<false, false, kSum, kPair>;
    return trans ? ragged_kernel<true, !kPair, kSum, kPair> : ragged_kernel<false, !kPair, kSum, kPair>;
}

// `width` in tiles of at most `most` columns, all of one size (a multiple of 16, or of `unit` where there are several).
void cut(int width, int most, int* tile, int* tiles, int unit = 16) {
    *tiles = (width + most - 1) / most;
    if (*tiles == 1) unit = 16;
    *tile = ((width + *tiles - 1) / *tiles + unit - 1) / unit * unit;
}

}  // namespace

cudaError_t ragged_setup(int num_sms, int* pairs) {
    const void* kernels[] = {
        (const void*)ragged_kernel<false, false, 0, false>, (const void*)ragged_kernel<true, false, 0, false>,
        (const void*)ragged_kernel<false, true, 0, false>, (const void*)ragged_kernel<true, true, 0, false>,
        (const void*)ragged_kernel<false, false, 8, false>, (const void*)ragged_kernel<true, false, 8, false>,
        (const void*)ragged_kernel<false, true, 8, false>, (const void*)ragged_kernel<true, true, 8, false>,
        (const void*)ragged_kernel<false, false, 16, false>, (const void*)ragged_kernel<true, false, 16, false>,
        (const void*)ragged_kernel<false, true, 16, false>, (const void*)ragged_kernel<true, true, 16, false>,
        (const void*)ragged_kernel<false, false, 16, true>, (const void*)ragged_kernel<true, false, 16, true>,
        (const void*)ragged_dw_kernel<1, false>, (const void*)ragged_dw_kernel<2, false>,
        (const void*)ragged_dw_kernel<1, true>};
    for (const void* k : kernels) {
        const cudaError_t err = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRgSmem);
        if (err != cudaSuccess) return err;
    }
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = rg_pair_config(num_sms / 2, kRgSumThreads + 32, nullptr, attr);   // (an SM holds one CTA of either kernel)
    return cudaOccupancyMaxActiveClusters(pairs, ragged_dw_kernel<1, true>, &cfg);
}

cudaError_t launch_ragged(const Dims& d, const Workspace& ws, const int32_t* cu, const int32_t* slot_expert,
                          const uint16_t* x, int64_t ldx, int K, const uint16_t* w, int N, int trans, float alpha,
                          const uint16_t* add, int64_t ldadd, uint16_t* y, int64_t ldy, int num_sms, int pairs,
                          cudaStream_t st) {
    const int64_t rows = (int64_t)d.R * d.C;
    RgParams p = {};
    p.tiles = ws.tiles;
    p.ntiles = ws.ntiles;
    p.cu = cu;
    p.slot_expert = slot_expert;
    p.y = y;
    p.add = add;
    p.ldy = ldy;
    p.ldadd = ldadd;
    p.alpha = alpha;
    p.E = d.E;
    p.R = d.R;
    p.B = d.B;
    p.NROW = d.NROW;
    p.C = d.C;
    p.N = N;
    p.kbn = (K + 63) / 64;
    p.status = ws.status;
    p.tickets = ws.tickets;
    // Few rows an expert: half the stage bytes for rows, more stages. (384 experts, 16 onto 2048: 40 rows an expert 54 us,
    // 68 with tiles of 128 rows; 48 60 and 69; 56 67 and 69. 7168 into 16: 73.8 and 74.0, 73.7 and 75.3, 94.9 and 77.4.)
    const bool few = rows / d.E <= 48;
    p.tile_rows = few ? 64 : 128;
    p.a_bytes = few ? kRgA / 2 : kRgA;
    const int64_t segs = (int64_t)d.R * d.NROW < rows ? (int64_t)d.R * d.NROW : rows;
    const int64_t most = rows / p.tile_rows + segs;   // row tiles at most
    p.local = most <= kRgLocal && (int64_t)d.R * d.NROW <= 32 * kRgThreads;
    // Tiles of 64 columns, whose reduction may be cut into parts, where even as many row tiles as there can be do not
    // make a unit for every SM with wider ones. With a short reduction and something to add, a unit is mostly what
    // it adds and writes: smaller tiles, more of them under way.
    const bool thin = add && p.kbn < 16 && !few;
    const int wide = thin ? 128 : 256;
    cut(N, most * ((N + wide - 1) / wide) < num_sms ? 64 : wide, &p.BN, &p.NT);
    // Tiles of 256 rows on pairs of SMs where experts have several and the reduction is in chains anyway: one SM's MMAs do
    // not hide the way of their operands into shared memory. (64 experts to 1024 columns. Rows of 1024: 320 an expert 63 us
    // on pairs and 64 without, 448 67 and 70, 1024 120 and 133, 2048 205 and 237; 512 rows of 640 55 and 59, of 512 50 and 44.)
    const bool pair = !add && !p.local && p.BN > 128 && p.kbn > kRgRowChain && rows / d.E >= 384 && pairs > 0;
    const int sum = p.kbn <= kRgRowChain ? 0 : p.BN <= 128 ? 8 : 16;
    if (pair) {
        p.tile_rows = 256;
        p.BN = (p.BN + 31) / 32 * 32;   // halves of 16
    }
    p.by_nt = make_fast_div((uint32_t)p.NT);
    p.by_nrow = make_fast_div((uint32_t)d.NROW);
    if (p.BN <= kRgPartCols) p.partial = ws.partial;
    p.steps = K >= 64 ? 4 : (K + 15) / 16;
    p.chunk = p.steps * 16 * 128;   // W [K, N]: boxes of 64 columns no taller than the reduction
    const int bn = pair ? p.BN / 2 : p.BN;   // W's columns in a CTA
    p.b_bytes = trans ? bn * 128 : (bn + 63) / 64 * p.chunk;
    p.adds = add ? (thin ? kRgMaxAdds : few || p.BN <= 64 ? 2 : 1) : 0;
    p.add_bytes = (p.BN + 63) / 64 * kRgA;
    const int rest = kRgBytes - (p.local ? kRgLocal * (int)sizeof(MTile) : 0) - (add ? p.adds * p.add_bytes : sum ? 2 * ((p.BN + 63) / 64) * kRgBox : 8 * kRgBox);
    const int fit = rest / (p.a_bytes + p.b_bytes);
    p.stages = fit < kRgMaxStages ? fit : kRgMaxStages;

    CUtensorMap tmW;
    RowMaps tmX, tmAdd = {};
    const uint64_t xd[2] = {(uint64_t)K, (uint64_t)rows}, xs[1] = {(uint64_t)ldx};
    const uint64_t ad[2] = {(uint64_t)N, (uint64_t)rows}, as[1] = {(uint64_t)ldadd};
    CUtensorMap* mx[4] = {&tmX.m16, &tmX.m32, &tmX.m64, &tmX.m128};
    CUtensorMap* ma[4] = {&tmAdd.m16, &tmAdd.m32, &tmAdd.m64, &tmAdd.m128};
    for (int i = 0; i < 4; ++i) {
        if (!encode_rows(mx[i], x, 2, xd, xs, 16u << i)) return cudaErrorInvalidValue;
        if (add && !encode_rows(ma[i], add, 2, ad, as, 16u << i)) return cudaErrorInvalidValue;
    }
    const uint64_t wd[3] = {(uint64_t)(trans ? K : N), (uint64_t)(trans ? N : K), (uint64_t)d.E};
    const uint64_t wl[2] = {wd[0], wd[0] * wd[1]};
    if (!encode_rows(&tmW, w, 3, wd, wl, trans ? (uint32_t)bn : (uint32_t)p.steps * 16)) return cudaErrorInvalidValue;
    if (!p.local) {
        const cudaError_t err = pair  ? launch_row_tiles<256>(d, ws, cu, st)
                                : few ? launch_row_tiles<64>(d, ws, cu, st)
                                      : launch_row_tiles<128>(d, ws, cu, st);
        if (err != cudaSuccess) return err;
    }
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg =
        pair ? rg_pair_config(pairs, kRgSumThreads, st, attr) : rg_config(num_sms, sum == 16 ? kRgSumThreads : kRgThreads, st, attr);
    auto* kernel = pair        ? row_kernel<16, true>(trans, false)
                   : sum == 16 ? row_kernel<16, false>(trans, add)
                   : sum == 8  ? row_kernel<8, false>(trans, add)
                               : row_kernel<0, false>(trans, add);
    return cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, tmAdd, p);
}

cudaError_t launch_ragged_dw(const Dims& d, const Workspace& ws, const int32_t* cu, const int32_t* slot_expert,
                             const uint16_t* x, int64_t ldx, int K, const uint16_t* dy, int64_t lddy, int N, float alpha,
                             int accumulate, float* g, int num_sms, int pairs, cudaStream_t st) {
    const int64_t rows = (int64_t)d.R * d.C;
    RgDwParams p = {};
    p.blocks = ws.tiles;
    p.first = ws.blk_first;
    p.alpha = alpha;
    p.E = d.E;
    // The M side is padded to 128 and the other to 16, so it is the wider one; x where that costs little, since then
    // a row of g leaves in 16-byte pieces.
    const int64_t pad_x = (int64_t)((K + 127) / 128 * 128) * ((N + 15) / 16 * 16);
    const int64_t pad_y = (int64_t)((N + 127) / 128 * 128) * ((K + 15) / 16 * 16);
    const bool x_wide = pad_x <= pad_y + pad_y / 4;
    p.Md = x_wide ? K : N;
    p.Nd = x_wide ? N : K;
    p.m_inner = !x_wide;
    p.accumulate = accumulate;
    p.tickets = ws.tickets;
    p.partial = ws.partial;
    p.status = ws.status;
    // two tiles along M a unit (half the units, each block of the narrow side read half as often) where they fill the SMs
    const int MI = p.Nd <= 128 && (int64_t)d.E * ((p.Md + 255) / 256) >= 2 * num_sms ? 2 : 1;
    p.MT = (p.Md + 128 * MI - 1) / (128 * MI);
    const int64_t units = (int64_t)d.E * p.MT * ((p.Nd + 255) / 256);
    cut(p.Nd, units < num_sms ? 64 : 256, &p.BN, &p.NT, 32);   // (a box of 32 columns is one tile's)
    p.parts = 1;
    const int64_t n = (int64_t)d.E * p.MT * p.NT;
    if (p.BN <= kRgPartCols && n < num_sms) {
        // a block takes a third of the time that adding a part does: for an expert of mean length, parts^2 <= blocks / 2
        const int64_t fit = num_sms / n, len = rows / 64 / d.E / 2;
        while (p.parts < kRgMaxParts && p.parts < fit && (int64_t)(p.parts + 1) * (p.parts + 1) <= len) ++p.parts;
    }
    // Tiles of 256 along M on pairs of CTAs, where there are enough of them for two rounds; an odd tile's partner only
    // brings its half of the N side. (262,144 rows of 64 experts by 1024 x 1024: 535 -> 425 us, by 600 x 1000, five tiles,
    // 450 -> 366 us (353 with single L2 lines), by 360 x 1000, three, 307 -> 264 us; 8,192 rows by 1096 x 1544: 114 -> 97 us, by 360 x 1000 the same.)
    const bool pair = MI == 1 && p.BN > 128 && p.MT > 1 && pairs > 0 &&
                      (int64_t)d.E * ((p.MT + 1) / 2) * p.NT >= 2 * pairs;
    if (pair) {
        p.MT = (p.MT + 1) / 2;
        p.BN = (p.BN + 31) / 32 * 32;   // halves of 16
    }
    p.by_parts = make_fast_div((uint32_t)p.parts);
    p.by_unit = make_fast_div((uint32_t)(p.MT * p.NT));
    p.by_nt = make_fast_div((uint32_t)p.NT);
    p.b_bytes = ((pair ? p.BN / 2 : p.BN) + 63) / 64 * kRgChunk;
    const int fit = (kRgBytes - 16 * kRgDwBox) / (MI * kRgA + p.b_bytes);
    p.stages = fit < kRgMaxStages ? fit : kRgMaxStages;

    CUtensorMap tx, ty, tg;
    if (!encode_g(&tg, g, d.E, K, N)) return cudaErrorInvalidValue;
    const uint64_t xd[2] = {(uint64_t)K, (uint64_t)rows}, xs[1] = {(uint64_t)ldx};
    const uint64_t yd[2] = {(uint64_t)N, (uint64_t)rows}, ys[1] = {(uint64_t)lddy};
    if (!encode_rows(&tx, x, 2, xd, xs, 64) || !encode_rows(&ty, dy, 2, yd, ys, 64)) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = rg_config(1, 1024, st, attr);
    cfg.dynamicSmemBytes = 0;
    cudaError_t err = cudaLaunchKernelEx(&cfg, ragged_blocks_kernel, cu, slot_expert, d, ws);
    if (err != cudaSuccess) return err;
    if (pair) {
        cfg = rg_pair_config(pairs, kRgSumThreads + 32, st, attr);
        return cudaLaunchKernelEx(&cfg, ragged_dw_kernel<1, true>, x_wide ? tx : ty, x_wide ? ty : tx, tg, p);
    }
    cfg = rg_config(num_sms, kRgSumThreads, st, attr);
    return cudaLaunchKernelEx(&cfg, MI == 2 ? ragged_dw_kernel<2, false> : ragged_dw_kernel<1, false>, x_wide ? tx : ty, x_wide ? ty : tx,
                              tg, p);
}

}  // namespace bep
