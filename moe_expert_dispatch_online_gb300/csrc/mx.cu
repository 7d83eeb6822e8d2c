// Experts with 4-bit weights (sm_103a): quantisation to microscaled e2m1 (mxfmt.cuh) and the
// grouped product of quantised rows with quantised weights on the block-scaled tensor cores.
//
//   y[row, n] = sum_h x4[row, h] * w4[expert(row), h, n],  fp32 accumulation, bf16 out
//
// Layouts. Two codes a byte, the even element in the low 4 bits; both operands lie along the
// reduction, so the weights are transposed when they are quantised:
//   row codes     [rows, H/2]            row scales     [rows, 16 * ceil(H/512)] bytes
//   weight codes  [E, H', H/2]           weight scales  [E, ceil(H'/128), ceil(H/128), 512]
// A 512-byte weight-scale block is the order in which the tensor core takes the scales of 128
// rows x 4 blocks of 32: row r, block k at byte (r % 32) * 16 + (r / 32) * 4 + k.

#include <cudaTypedefs.h>

#include "mxfmt.cuh"
#include "ptx.cuh"

namespace bep {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void block_to_f32(const uint4* v, float* f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) bf16x8_to_f32(v[j], f + 8 * j);
}

// ------------------------------------------------------------------------ weights
// One CTA: 64 columns n x 256 rows h of one expert. Each warp quantises a block of 32 rows h
// for all 64 columns (lane l: columns 2l and 2l + 1, so that a load covers 128 bytes); the
// codes meet in shared memory and leave as 128-byte runs along h.
__global__ void __launch_bounds__(kThreads) mx_weight_kernel(const uint32_t* __restrict__ w,
                                                             uint4* __restrict__ codes,
                                                             uint8_t* __restrict__ scales, int H,
                                                             int Hp) {
    __shared__ uint4 s_codes[64][9];   // 8 blocks of 16 bytes a column, one more against conflicts
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nt = Hp / 64;
    const int e = blockIdx.y, n0 = (blockIdx.x % nt) * 64, hb0 = (blockIdx.x / nt) * 8;
    const int nblk = H / kMxBlock, hb = hb0 + warp;
    const int MT = (Hp + 127) / 128, KB = (H + 127) / 128;
    if (hb < nblk) {
        const uint32_t* src = w + (((int64_t)e * H + (int64_t)hb * kMxBlock) * Hp + n0) / 2 + lane;
        float f0[kMxBlock], f1[kMxBlock];
#pragma unroll
        for (int i = 0; i < kMxBlock; ++i) {
            const uint32_t v = __ldcs(src + (int64_t)i * (Hp / 2));
            f0[i] = __uint_as_float(v << 16);
            f1[i] = __uint_as_float(v & 0xffff0000u);
        }
        const uint32_t b0 = mx4_block(f0, &s_codes[2 * lane][warp]);
        const uint32_t b1 = mx4_block(f1, &s_codes[2 * lane + 1][warp]);
        const int n = n0 + 2 * lane;
        uint8_t* sc = scales + (((int64_t)e * MT + n / 128) * KB + hb / 4) * 512 + (hb & 3);
        const int r = n & 127;
        sc[(r & 31) * 16 + (r >> 5) * 4] = (uint8_t)b0;
        sc[((r & 31) + 1) * 16 + (r >> 5) * 4] = (uint8_t)b1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * 8; i += kThreads) {
        const int n = i >> 3, b = i & 7;
        if (hb0 + b < nblk)
            codes[((int64_t)e * Hp + n0 + n) * nblk + hb0 + b] = s_codes[n][b];
    }
}

// ------------------------------------------------------------------------ dispatch
// codes[dest[tok, k]], scales[dest[tok, k]] = mx4(x[tok]). One warp per (token, run of 32
// blocks): a lane quantises one block once and stores its 16 bytes of codes and its scale
// byte to the K destination rows.
__global__ void __launch_bounds__(kThreads) dispatch_mx_kernel(const uint4* __restrict__ x,
                                                               const int32_t* __restrict__ dest,
                                                               uint4* __restrict__ codes,
                                                               uint8_t* __restrict__ scales,
                                                               int64_t ntok, int K, int nblk,
                                                               int runs, int pitch, int64_t nrows,
                                                               int32_t* status) {
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    const int64_t nitem = ntok * runs;
    for (int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; item < nitem;
         item += nwarps) {
        const int64_t tok = runs == 1 ? item : item / runs;
        const int b = (int)(item - tok * runs) * 32 + lane;
        int dl = 0;
        bool ok = true;
        if (lane < K) {
            dl = dest[tok * K + lane];
            ok = dl >= 0 && (int64_t)dl < nrows;
        }
        uint4 q = make_uint4(0, 0, 0, 0);
        uint32_t byte = 0;
        if (b < nblk) {
            uint4 v[4];
            const uint4* src = x + (tok * nblk + b) * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __ldg(src + j);
            float f[kMxBlock];
            block_to_f32(v, f);
            byte = mx4_block(f, &q);
        }
        const unsigned m = __ballot_sync(0xffffffffu, ok);
        if (m != 0xffffffffu && lane == 0) set_status(status, BEP_DERR_BOUNDS);
        for (int k = 0; k < K; ++k) {
            const int64_t row = __shfl_sync(0xffffffffu, dl, k);
            if (!((m >> k) & 1u) || b >= nblk) continue;
            codes[row * nblk + b] = q;
            scales[row * pitch + b] = (uint8_t)byte;
        }
    }
}

// ------------------------------------------------------------------------ activation
// codes, scales = mx4(g * sigmoid(g) * u) for h = [g | u]: one block of 32 a thread. The
// activation stays in fp32 until its one rounding to e2m1.
__global__ void __launch_bounds__(kThreads) swiglu_mx_kernel(const uint4* __restrict__ h,
                                                             uint4* __restrict__ codes,
                                                             uint8_t* __restrict__ scales,
                                                             int64_t nblocks, int nblk, int pitch) {
    grid_launch_dependents();
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < nblocks; i += step) {
        const int64_t row = i / nblk;
        const int b = (int)(i - row * nblk);
        const uint4* src = h + (row * 2 * nblk + b) * 4;
        float a[kMxBlock];
        uint4 v[4], t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = __ldg(src + j);
            t[j] = __ldg(src + (int64_t)nblk * 4 + j);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float g[8], u[8];
            bf16x8_to_f32(v[j], g);
            bf16x8_to_f32(t[j], u);
            gated8(g, u, a + 8 * j);
        }
        uint4 q;
        const uint32_t byte = mx4_block(a, &q);
        codes[i] = q;
        scales[row * pitch + b] = (uint8_t)byte;
    }
}

// ------------------------------------------------------------------------ product
// The weights are the M operand and the rows of one segment the N operand (32..224), so that a
// segment of a few rows costs a narrow MMA and not a 128-row one. A cluster of two CTAs shares a
// tile of 256 outputs x N rows (cta_group::2): CTA r holds outputs 128 r.. and half of the rows,
// so that a stage brings 33 KB to each SM for what takes one CTA 47 KB. Few rows: the weights'
// HBM stream bounds it (96 rows by 384 experts' 1024 x 7168, 1.30 GB: 195 us, 99% of the copy rate).
// Many rows: a stage of 224 rows takes the tensor pipe 390 cycles for its MMAs and about 120 for the
// six scale copies, which share the pipe, and the stage's bytes about as long to arrive in shared
// memory that the MMAs are reading; the two overlap to about 600 cycles. 524,288 rows by 7168 x 2048:
// 4.97 ms with one CTA and N <= 128, 2.92 with pairs and N <= 192, 2.67 with N <= 224, 2.46-2.6 now
// (5.9-6.3 PFLOP/s; the ordered hand-over of the row scales, below, is 3% of it).
//   warp 0     TMA: codes of 128 outputs and of N/2 rows; 256 reduction steps a stage
//   warp 1     (CTA 0) copies each stage's scales to both TMEMs, issues tcgen05.mma.kind::mxf4
//   warps 2, 3 put all N rows' scales (any row offset, so no TMA) in tensor-core order, make them
//              visible to the async proxy and arrive on CTA 0's barrier behind a release of shared memory
//              alone (a release of everything at cluster scope takes about 1,800 cycles a stage: 7.1 ms
//              at 524,288 rows by 7168 x 2048)
//   warps 4-11 epilogue: TMEM to bf16 y, while the next unit runs in the other accumulator
// Launches overlap: the kernel that writes the rows lets the work list's kernel be launched at once, and
// that one lets this kernel set up its barriers and TMEM. Both wait for the end of what precedes them
// before they read anything: the kernel before them need not be one of this library, and whatever it is
// may be what writes cu_seqlens.
// A polling warp takes issue slots from the warps that issue MMAs and scales, so every role but the
// scale warps is held in its waits by the hardware, and one of four epilogue warps waits for all four
// (96 rows by 384 experts' 1024 x 7168: 195 us, 220 us with every warp polling).
//   barrier    owner   arrivals
//   full[s]    CTA 0   CTA 0's producer (expect_tx), a scale warp of each CTA + both CTAs' TMA bytes
//   empty[s]   both    the MMA thread's multicast commit
//   tfull[a]   both    the MMA thread's multicast commit at the end of a unit
//   tempty[a]  CTA 0   the 8 epilogue warps of each CTA
constexpr int kMxRows = 224;                   // rows of a tile at most
constexpr int kMxEpiWarps = 8;                 // two for each quarter of TMEM's lanes
constexpr int kMxThreads = 32 * (4 + kMxEpiWarps);   // producer, MMA, two scale warps, epilogue
// Stages, compared before the row scales' hand-over cost its 3%: five 2.42 ms at 524,288 rows by 7168 x 2048 and
// 76.5 us at 64, six 2.54 ms and 75.1 us, four 2.64 ms and 81 us.
constexpr int kMxStages = 5;
constexpr int kMxK = 256;                      // reduction elements a stage: 128 bytes of codes
constexpr int kMxA = 128 * 128;                // bytes: 128 outputs x 128 bytes
constexpr int kMxB = kMxRows / 2 * 128;        // bytes: half of the rows
constexpr int kMxSfa = 1024;                   // bytes: 2 blocks of 512
constexpr int kMxSfb = 2048;                   // bytes: (2 reduction blocks) x (rows 0..127, 128..255)
constexpr int kMxOut = 32 * 256;               // bytes: four epilogue warps' 32 rows x 128 outputs
constexpr int kMxStageBytes = kMxA + kMxB + kMxSfa + kMxSfb;
constexpr int kMxTmemCols = 512;
constexpr int kMxSfBase = 2 * kMxRows;         // two accumulators lie before
constexpr int kMxSfCols = 24;                  // TMEM columns of a stage's scales: A 2 x 4, B 2 x 8
constexpr int kMxSlots = (kMxTmemCols - kMxSfBase) / kMxSfCols;   // 2
static_assert(kMxSlots >= 2 && kMxSlots <= kMxStages, "a slot is free once its stage is");
// A parity wait tells two neighbouring phases apart, no more. A scale warp fills two stages of every
// 2 kMxScaleWarps, and to fill them it had to see the ring's previous round; with at most a ring
// between its turns, the phase it waits for next is at most one ahead of the barrier's.
constexpr int kMxScaleWarps = 2;
static_assert(2 * kMxScaleWarps <= kMxStages, "a scale warp's turns lie at most one ring apart");

struct MxParams {
    const MTile* tiles;
    const int32_t* ntiles;
    const int32_t* slot_expert;
    const uint8_t* row_scales;
    uint16_t* y;
    int64_t nrows;
    int E, H, Hp, MT, KB, pitch;
    int32_t* status;
};

struct MxUnit {
    int row0, rows, expert, mp;
};

// A cluster's units lie `ncl` apart in (tile, pair of output tiles) order, the pair fastest: a walk
// over them without a division, since a unit may last only a few stages.
struct MxWalk {
    int unit, tile, mp;        // the next unit
    int dtile, dmp, MP, ncl;   // its successor
    __device__ __forceinline__ MxWalk(int first, int ncl_, int MP_)
        : unit(first), tile(first / MP_), mp(first % MP_), dtile(ncl_ / MP_), dmp(ncl_ % MP_), MP(MP_), ncl(ncl_) {}
    // The unit's tile and expert; expert < 0 for a slot whose expert is unknown (reported, skipped)
    // and past the last unit.
    __device__ __forceinline__ MxUnit take(const MxParams& p, int total) {
        if (unit >= total) return MxUnit{0, 0, -1, 0};
        const MTile t = p.tiles[tile];
        MxUnit u;
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

__device__ __forceinline__ void tma_load_3d_pair(const CUtensorMap* map, uint32_t bar_cl, void* dst, int c0,
                                                 int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cl), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Descriptors reach the instructions as a low word (address in 16-byte units; operands: leading
// offset 1) beside a constant high word. Operands: 8-row groups 1024 bytes apart, version 1, 128-byte
// swizzle. Scales: 32 rows of 16 bytes, groups of 8 rows 128 bytes apart, version 1, no swizzle.
#define BEP_MX_OPERAND_HI "0x40004040"
#define BEP_MX_SCALES_HI "0x00004008"
__device__ __forceinline__ uint32_t operand_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | (1u << 16); }
__device__ __forceinline__ uint32_t scales_lo(uint32_t saddr) { return (saddr >> 4) & 0x3FFFu; }

// In each CTA of the pair: 32 rows x 16 bytes of scales from its shared memory to 4 columns of
// its TMEM, in each of the four 32-lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t lo) {
    asm volatile(
        "{\n\t.reg .b64 d;\n\t"
        "mov.b64 d, {%1, " BEP_MX_SCALES_HI "};\n\t"
        "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr),
        "r"(lo)
        : "memory");
}

// Instruction descriptor, kind::mxf4, M = 256: e2m1 operands (1 at bits 7 and 10), N >> 3 at bit
// 17, e8m0 scales (bit 23), M >> 7 at bit 27; the first of the K step's two scale bytes (0 or 2
// of the TMEM word's four) at bits 4 (B) and 29 (A).
__device__ __forceinline__ uint32_t idesc_mxf4(int N, uint32_t sf) {
    return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | (2u << 27) |
           (sf << 29);
}

// kAdd: adds to the accumulator; otherwise when `add` is not 0.
template <bool kAdd>
__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t add = 1) {
    if (kAdd)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
            "mov.b64 da, {%1, " BEP_MX_OPERAND_HI "};\n\t"
            "mov.b64 db, {%2, " BEP_MX_OPERAND_HI "};\n\t"
            "setp.eq.u32 p, 0, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %3, [%4], [%5], p;\n\t}" ::
                "r"(d_tmem),
            "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
            "mov.b64 da, {%1, " BEP_MX_OPERAND_HI "};\n\t"
            "mov.b64 db, {%2, " BEP_MX_OPERAND_HI "};\n\t"
            "setp.ne.u32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %3, [%4], [%5], p;\n\t}" ::
                "r"(d_tmem),
            "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(add)
            : "memory");
}

// Named barriers of four epilogue warps.
__device__ __forceinline__ void quad_sync(int id) {
    asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool quad_all(int id, bool v) {
    uint32_t r;
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

// The work list: tiles of at most kMxRows rows of one segment, in (rank, row) order. One CTA; a
// thread holds four segments at a time, all loaded at once (8 ranks x 433 segments: 3 us; a
// thread with four consecutive segments loaded twice took 7). A table with any inconsistent
// segment is refused as a whole.
__global__ void __launch_bounds__(1024) mx_tiles_kernel(const int32_t* cu, Dims d, FastDiv nrow, Workspace ws) {
    constexpr int kS = 4, kChunk = kS * 1024;
    __shared__ int s_sum[kS * 32];
    grid_launch_dependents();   // the product may set itself up
    // cu may still be being written up to here: no load of it may come earlier, nor take the
    // non-coherent path, which the compiler may move and which wants memory constant from the start
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
            const int n = (len[r] + kMxRows - 1) / kMxRows;
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
            for (int m = 0; m < len[r]; m += kMxRows) {
                t.row0 = (int32_t)(u * d.C + a[r] + m);
                t.rows = min(kMxRows, len[r] - m);
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

__global__ void __launch_bounds__(kMxThreads, 1) grouped_gemm_mx_kernel(
    const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmS,
    const __grid_constant__ CUtensorMap tmX16, const __grid_constant__ CUtensorMap tmX32,
    const __grid_constant__ CUtensorMap tmX64, const __grid_constant__ CUtensorMap tmXtop,
    const MxParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t* smA = smem;
    uint8_t* smB = smA + kMxStages * kMxA;
    uint8_t* smSA = smB + kMxStages * kMxB;
    uint8_t* smSB = smSA + kMxStages * kMxSfa;
    uint8_t* smO = smSB + kMxStages * kMxSfb;
    uint64_t* full = reinterpret_cast<uint64_t*>(smO + kMxEpiWarps / 4 * kMxOut);
    uint64_t* empty = full + kMxStages;
    uint64_t* tfull = empty + kMxStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    int32_t* status = p.status;
    const uint32_t rank = cluster_rank();
    const bool lead = rank == 0;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 32) {
        const CUtensorMap* maps[] = {&tmW, &tmS, &tmX16, &tmX32, &tmX64, &tmXtop};
        for (const CUtensorMap* m : maps)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMxStages; ++s) {
            mbar_init(&full[s], 3);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 2 * kMxEpiWarps);
        }
        mbar_init(drain, 1);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        // one warp of each CTA performs the pair's allocation together (all of both TMEMs)
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(s_tmem)),
                     "r"(kMxTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers exist before any remote arrive or multicast commit
    tc_fence_after();
    const uint32_t tmem_base = *s_tmem;
    grid_wait();      // launched early: the work list and the rows are complete from here on

    const int MP = (p.MT + 1) / 2;             // pairs of 128-output tiles
    const int total = *p.ntiles * MP;
    const int nst = (p.H + kMxK - 1) / kMxK;   // stages a unit
    const int cl0 = (int)cluster_id(), ncl = (int)cluster_count();
    uint32_t pr_s = 0, pr_ph = 0, pr_armed = 0;

    if (warp == 0) {
        if (lane == 0) {
            bool live = true;
            MxWalk walk(cl0, ncl, MP);
            MxUnit next = walk.take(p, total);   // read a unit ahead
            for (int unit = cl0; unit < total && live; unit += ncl) {
                const MxUnit u = next;
                next = walk.take(p, total);
                if (u.expert < 0) {
                    if (lead) set_status(status, BEP_DERR_BOUNDS);
                    continue;
                }
                const int half = mma_rows(u.rows) / 2;
                const CUtensorMap* tmX = half <= 16 ? &tmX16 : half <= 32 ? &tmX32 : half <= 64 ? &tmX64 : &tmXtop;
                const int box = half <= 16 ? 16 : half <= 32 ? 32 : half <= 64 ? 64 : kMxRows / 2;
                const int mt = 2 * u.mp + (int)rank;   // past H' for the last odd tile: zeros
                const int srow = (u.expert * p.MT + mt) * p.KB;
                for (int k = 0; k < nst; ++k) {
                    if (!mbar_wait_held(&empty[pr_s], pr_ph ^ 1u, s_abort, status)) {
                        live = false;
                        break;
                    }
                    if (lead) mbar_arrive_expect_tx(&full[pr_s], 2 * (kMxA + kMxSfa + box * 128));
                    ++pr_armed;
                    const uint32_t bar = cluster_addr(&full[pr_s], 0);
                    tma_load_3d_pair(&tmW, bar, smA + pr_s * kMxA, k * 128, mt * 128, u.expert);
                    tma_load_2d_pair(tmX, bar, smB + pr_s * kMxB, k * 128, u.row0 + (int)rank * half);
                    tma_load_2d_pair(&tmS, bar, smSA + pr_s * kMxSfa, 0, srow + 2 * k);
                    if (++pr_s == kMxStages) {
                        pr_s = 0;
                        pr_ph ^= 1u;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lead && elect_one()) {
            // one thread, known to the compiler as one (524,288 rows by 7168 x 2048: 2.50 ms; with the
            // whole warp in the waits and one lane at the instructions 2.56-2.68 ms)
            const uint32_t da = operand_lo(smem_u32(smA)), db = operand_lo(smem_u32(smB));
            const uint32_t dsa = scales_lo(smem_u32(smSA)), dsb = scales_lo(smem_u32(smSB));
            uint32_t s = 0, ph = 0;                    // ring stage
            uint32_t slot = 0;                         // TMEM scale columns
            uint32_t old = 0, old_ph = 0, done = 0;    // the stage that used the slot before
            int it = 0;
            bool live = true;
            MxWalk walk(cl0, ncl, MP);
            MxUnit next = walk.take(p, total);   // read a unit ahead
            for (int unit = cl0; unit < total && live; unit += ncl) {
                const MxUnit u = next;
                next = walk.take(p, total);
                if (u.expert < 0) continue;
                const int N = mma_rows(u.rows);
                const int acc = it & 1;
                if (!mbar_wait_held<true>(&tempty[acc], ((it >> 1) & 1) ^ 1u, s_abort, status)) break;
                ++it;
                const uint32_t dt = tmem_base + acc * kMxRows;
                const uint32_t id0 = idesc_mxf4(N, 0), id2 = idesc_mxf4(N, 2);
                for (int k = 0; k < nst; ++k) {
                    // a slot's scales are overwritten once the MMAs that read them have completed
                    if (done >= (uint32_t)kMxSlots) {
                        if (!mbar_wait_held(&empty[old], old_ph, s_abort, status)) {
                            live = false;
                            break;
                        }
                        if (++old == kMxStages) {
                            old = 0;
                            old_ph ^= 1u;
                        }
                    } else {
                        ++done;
                    }
                    if (!mbar_wait_held<true>(&full[s], ph, s_abort, status)) {
                        live = false;
                        break;
                    }
                    tc_fence_after();
                    // descriptors count 16-byte units: a K step is 2 of them, a scale block 32
                    const uint32_t a = da + s * (kMxA / 16), b = db + s * (kMxB / 16);
                    const uint32_t sa = dsa + s * (kMxSfa / 16), sb = dsb + s * (kMxSfb / 16);
                    const uint32_t ta = tmem_base + kMxSfBase + slot * kMxSfCols, tb = ta + 8;
                    const int steps = min(4, (p.H - k * kMxK) / 64);
                    copy_scales(ta, sa);
                    copy_scales(tb, sb);
                    if (N > 128) copy_scales(tb + 4, sb + 32);
                    mma_mxf4<false>(dt, a, b, id0, ta, tb, k != 0);
                    if (steps > 1) mma_mxf4<true>(dt, a + 2, b + 2, id2, ta, tb);
                    if (steps > 2) {
                        copy_scales(ta + 4, sa + 32);
                        copy_scales(tb + 8, sb + 64);
                        if (N > 128) copy_scales(tb + 12, sb + 96);
                        mma_mxf4<true>(dt, a + 4, b + 4, id0, ta + 4, tb + 8);
                        if (steps > 3) mma_mxf4<true>(dt, a + 6, b + 6, id2, ta + 4, tb + 8);
                    }
                    mma_commit_pair(&empty[s]);
                    if (k == nst - 1) mma_commit_pair(&tfull[acc]);
                    if (++s == kMxStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                    if (++slot == kMxSlots) slot = 0;
                }
            }
        }
    } else if (warp < 2 + kMxScaleWarps) {
        // A 16-byte piece of a row's scales serves two stages; the two warps take the pieces in turn,
        // across units. Loads run two of a warp's own pieces ahead of the stores, across units, so that
        // their latency is hidden at four stages a unit as well.
        constexpr int kC = kMxRows / 32;
        static_assert(kC == 7, "four words of the first 128 rows and three of the rest");
        const int mine = warp - 2;
        const int pieces = (nst + 1) / 2;
        const uint4* src[kC] = {};
        MxWalk l_walk(cl0, ncl, MP);   // the load cursor: unit, piece and rows
        int l_piece = pieces + mine, l_rows = 0;
        auto load = [&](uint4* v) {
            while (l_piece >= pieces) {   // the next unit that has a piece for this warp
                if (l_walk.unit >= total) return;
                const MxUnit u = l_walk.take(p, total);
                if (u.expert < 0) continue;
                l_piece -= pieces;
                if (l_piece >= pieces) continue;   // all of this unit's are the other warp's
                l_rows = mma_rows(u.rows);
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    const int64_t row = min((int64_t)u.row0 + 32 * c + lane, p.nrows - 1);
                    src[c] = reinterpret_cast<const uint4*>(p.row_scales + row * p.pitch);
                }
            }
#pragma unroll
            for (int c = 0; c < kC; ++c)
                if (32 * c < l_rows) v[c] = src[c][l_piece];   // written while this kernel was starting: no __ldg
            l_piece += kMxScaleWarps;
        };
        uint4 v0[kC] = {}, v1[kC] = {};
        load(v0);
        load(v1);
        uint32_t s = 0, ph = 0;
        bool live = true;
        int own = mine;   // this warp's next piece of the unit
        MxWalk walk(cl0, ncl, MP);
        MxUnit u = walk.take(p, total);
        for (int unit = cl0; unit < total && live; unit += ncl) {
            const MxUnit cur = u;
            u = walk.take(p, total);
            if (cur.expert < 0) continue;
            const int N = mma_rows(cur.rows);
            for (int g = 0; g < pieces && live; ++g) {
                const int here = min(2, nst - 2 * g);   // stages of this piece
                if (g != own) {
                    s += here;
                    if (s >= kMxStages) {
                        s -= kMxStages;
                        ph ^= 1u;
                    }
                    continue;
                }
                own += kMxScaleWarps;
                uint4 v[kC];
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    v[c] = v0[c];
                    v0[c] = v1[c];
                }
                load(v1);
                for (int half = 0; half < here; ++half) {
                    if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1u, s_abort, status))) {
                        live = false;
                        break;
                    }
                    // row 32 c + lane of an atom's 128: word c of the lane's 16 bytes
                    uint4* d = reinterpret_cast<uint4*>(smSB + s * kMxSfb) + lane;
                    d[0] = half ? make_uint4(v[0].z, v[1].z, v[2].z, v[3].z) : make_uint4(v[0].x, v[1].x, v[2].x, v[3].x);
                    d[64] = half ? make_uint4(v[0].w, v[1].w, v[2].w, v[3].w) : make_uint4(v[0].y, v[1].y, v[2].y, v[3].y);
                    if (N > 128) {
                        d[32] = half ? make_uint4(v[4].z, v[5].z, v[6].z, 0) : make_uint4(v[4].x, v[5].x, v[6].x, 0);
                        d[96] = half ? make_uint4(v[4].w, v[5].w, v[6].w, 0) : make_uint4(v[4].y, v[5].y, v[6].y, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive_rank_shared(&full[s], 0);
                    if (++s == kMxStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            own -= pieces;
        }
    } else {
        // Four warps, one for each quarter of TMEM's lanes, own every second run of 32 rows. A lane
        // holds one output of 32 rows, and a row's outputs lie together in y, so the run is turned in
        // shared memory (2-byte stores with fixed offsets, conflict-free) and leaves as whole rows of
        // 256 bytes, 16 a lane. One warp a scheduler issues slowly and 64-byte pieces of rows write
        // slowly: 131,000 rows of 256 by 5760 took 991 us with 4 warps that traded outputs by shuffles
        // and stored 4 bytes a lane, 415 us with 8 that each turned and stored their own 64 bytes.
        const int quarter = warp & 3, second = (warp - 4) >> 2;
        uint8_t* stg = smO + second * kMxOut;
        int it = 0;
        MxWalk walk(cl0, ncl, MP);
        MxUnit next = walk.take(p, total);
        for (int unit = cl0; unit < total; unit += ncl) {
            const MxUnit u = next;
            next = walk.take(p, total);
            if (u.expert < 0) continue;
            const int acc = it & 1;
            // one warp waits for the accumulator and the others for it at their barrier, which costs the
            // busy warps no issue slots; the four give up together, so that none waits for another there
            const bool ready = quarter != 0 || mbar_wait_held(&tfull[acc], (it >> 1) & 1, s_abort, status);
            if (!quad_all(1 + second, ready)) break;
            ++it;
            tc_fence_after();
            // lane l of quarter q holds output n = 128 mt + 32 q + l, its columns the rows
            const int n0 = (2 * u.mp + (int)rank) * 128;
            const uint32_t tacc = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * kMxRows;
            bool held = true;
            for (int c0 = 32 * second; c0 < u.rows; c0 += 64) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(tacc + c0, r);
                if (c0 + 64 >= u.rows) {   // this warp has read all its runs: free them before the stores
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_rank_relaxed(&tempty[acc], 0);
                    held = false;
                }
                quad_sync(1 + second);   // the run before has been read (two buffers measured 3% slower)
                uint16_t* col = reinterpret_cast<uint16_t*>(stg) + quarter * 32 + lane;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint32_t two = pack_bf16x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                    col[(2 * j) * 128] = (uint16_t)two;
                    col[(2 * j + 1) * 128] = (uint16_t)(two >> 16);
                }
                quad_sync(1 + second);   // the run is staged
                const int row = quarter * 8 + (lane >> 4), n = n0 + (lane & 15) * 8;
                const uint4* piece = reinterpret_cast<const uint4*>(stg) + quarter * 128 + lane;
                uint16_t* out = p.y + ((int64_t)u.row0 + c0 + row) * p.Hp + n;
                const int left = n < p.Hp ? u.rows - c0 - row : 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (2 * j < left) *reinterpret_cast<uint4*>(out + (int64_t)(2 * j) * p.Hp) = piece[32 * j];
            }
            if (held) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_rank_relaxed(&tempty[acc], 0);
            }
        }
    }

    __syncthreads();
    if (*s_abort) {
        // A wait gave up: what was started lands before shared memory and TMEM are released, each
        // wait bounded. CTA 0's full phases count CTA 1's bytes too; CTA 1's loads of a stage that
        // CTA 0 never armed cannot be observed, and the short sleep bounds those.
        if (warp == 0 && lane == 0 && lead) {
            for (uint32_t i = 0; i < pr_armed && i < (uint32_t)kMxStages; ++i) {
                if (pr_s == 0) {
                    pr_s = kMxStages;
                    pr_ph ^= 1u;
                }
                --pr_s;
                mbar_drain(&full[pr_s], pr_ph);
            }
        } else if (warp == 1 && lane == 0 && lead) {
            mma_commit_pair_lead(drain);
            mbar_drain(drain, 0);
        }
        if (threadIdx.x == 0)
            for (int i = 0; i < 20; ++i) __nanosleep(10000);
        __syncthreads();
    }
    cluster_sync();   // neither CTA leaves while the other may still signal it or read its tiles
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(kMxTmemCols)
                     : "memory");
    }
}

constexpr size_t kMxSmem =
    1024 + (size_t)kMxStages * kMxStageBytes + kMxEpiWarps / 4 * kMxOut + (2 * kMxStages + 5) * 8 + 16;

// Scale blocks as rows of 128 words, 2 rows a box.
bool encode_scales(CUtensorMap* m, const void* base, uint64_t blocks) {
    void* fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t d[2] = {128, blocks}, strides[1] = {512};
    const cuuint32_t box[2] = {128, 2}, estr[2] = {1, 1};
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
               m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), d, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

cudaLaunchConfig_t mx_config(int clusters, cudaStream_t st, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * clusters, 1, 1);
    cfg.blockDim = dim3(kMxThreads, 1, 1);
    cfg.dynamicSmemBytes = kMxSmem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

// CTAs for `warps` items: all of them at once, in memory order (524,288 rows of 7168: 425 us, 490
// with 8 CTAs an SM that stride over the items), or, under an SM budget, 8 an SM of that many.
int grid_for(int64_t warps, int sms, int num_sms) {
    const int64_t g = (warps + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t cap = sms < num_sms ? (int64_t)sms * 8 : (int64_t)INT32_MAX;
    return (int)(g < cap ? (g > 0 ? g : 1) : cap);
}

}  // namespace

// *clusters: clusters of two that can be resident at once: the grid, so that the units are spread evenly over
// CTAs that run from the start.
cudaError_t mx_setup(int device, int* clusters) {
    cudaError_t err = cudaFuncSetAttribute(grouped_gemm_mx_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)kMxSmem);
    if (err != cudaSuccess) return err;
    int nsm = 0;
    err = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, device);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = mx_config(nsm / 2, nullptr, attr);
    return cudaOccupancyMaxActiveClusters(clusters, grouped_gemm_mx_kernel, &cfg);
}

cudaError_t launch_mx_weight(const Dims& d, const uint16_t* w, uint8_t* codes, uint8_t* scales,
                             cudaStream_t st) {
    const dim3 grid((unsigned)(d.Hp / 64) * ((d.H + 255) / 256), (unsigned)d.E);
    mx_weight_kernel<<<grid, kThreads, 0, st>>>(reinterpret_cast<const uint32_t*>(w),
                                                reinterpret_cast<uint4*>(codes), scales, d.H, d.Hp);
    return cudaGetLastError();
}

cudaError_t launch_dispatch_mx(const Dims& d, const Workspace& ws, const uint16_t* x,
                               const int32_t* dest, uint8_t* codes, uint8_t* scales, int sms, int num_sms,
                               cudaStream_t st) {
    const int64_t ntok = (int64_t)d.R * d.S;
    const int nblk = d.H / kMxBlock, runs = (nblk + 31) / 32;
    dispatch_mx_kernel<<<grid_for(ntok * runs, sms, num_sms), kThreads, 0, st>>>(
        reinterpret_cast<const uint4*>(x), dest, reinterpret_cast<uint4*>(codes), scales, ntok, d.K,
        nblk, runs, mx_scale_pitch(d.H), (int64_t)d.R * d.C, ws.status);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_mx(int64_t rows, int F, const uint16_t* h, uint8_t* codes,
                             uint8_t* scales, cudaStream_t st) {
    const int nblk = F / kMxBlock;
    swiglu_mx_kernel<<<grid_for((rows * nblk + 31) / 32, 1, 1), kThreads, 0, st>>>(
        reinterpret_cast<const uint4*>(h), reinterpret_cast<uint4*>(codes), scales, rows * nblk, nblk,
        mx_scale_pitch(F));
    return cudaGetLastError();
}

cudaError_t launch_grouped_gemm_mx(const Dims& d, const Workspace& ws, const int32_t* cu,
                                   const int32_t* slot_expert, const uint8_t* codes,
                                   const uint8_t* scales, const uint8_t* w_codes,
                                   const uint8_t* w_scales, uint16_t* y, int clusters,
                                   cudaStream_t st) {
    const uint64_t wd[3] = {(uint64_t)d.H / 2, (uint64_t)d.Hp, (uint64_t)d.E};
    const uint64_t xd[2] = {(uint64_t)d.H / 2, (uint64_t)d.R * d.C};
    const uint32_t boxes[4] = {16, 32, 64, kMxRows / 2};
    MxParams p;
    p.tiles = ws.tiles;
    p.ntiles = ws.ntiles;
    p.slot_expert = slot_expert;
    p.row_scales = scales;
    p.y = y;
    p.nrows = (int64_t)d.R * d.C;
    p.E = d.E;
    p.H = d.H;
    p.Hp = d.Hp;
    p.MT = (d.Hp + 127) / 128;
    p.KB = (d.H + 127) / 128;
    p.pitch = mx_scale_pitch(d.H);
    p.status = ws.status;
    CUtensorMap tmW, tmS, tmX[4];
    if (!encode_u8(&tmW, w_codes, 3, wd, 128)) return cudaErrorInvalidValue;
    if (!encode_scales(&tmS, w_scales, (uint64_t)d.E * p.MT * p.KB)) return cudaErrorInvalidValue;
    for (int i = 0; i < 4; ++i)
        if (!encode_u8(&tmX[i], codes, 2, xd, boxes[i])) return cudaErrorInvalidValue;
    cudaLaunchConfig_t tc = {};
    cudaLaunchAttribute early;
    tc.gridDim = dim3(1, 1, 1);
    tc.blockDim = dim3(1024, 1, 1);
    tc.stream = st;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    tc.attrs = &early;
    tc.numAttrs = 1;
    const cudaError_t err =
        cudaLaunchKernelEx(&tc, mx_tiles_kernel, cu, d, make_fast_div((uint32_t)d.NROW), ws);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = mx_config(clusters, st, attr);
    return cudaLaunchKernelEx(&cfg, grouped_gemm_mx_kernel, tmW, tmS, tmX[0], tmX[1], tmX[2], tmX[3], p);
}

}  // namespace bep
