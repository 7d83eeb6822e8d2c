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
    for (int j = 0; j < 4; ++j) {
        const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[8 * j + 2 * i] = __uint_as_float(w[i] << 16);
            f[8 * j + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
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
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < nblocks; i += step) {
        const int64_t row = i / nblk;
        const int b = (int)(i - row * nblk);
        const uint4* src = h + (row * 2 * nblk + b) * 4;
        float g[kMxBlock], u[kMxBlock];
        uint4 v[4], t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = __ldg(src + j);
            t[j] = __ldg(src + (int64_t)nblk * 4 + j);
        }
        block_to_f32(v, g);
        block_to_f32(t, u);
#pragma unroll
        for (int j = 0; j < kMxBlock; ++j) g[j] = g[j] * fast_sigmoid(g[j]) * u[j];
        uint4 q;
        const uint32_t byte = mx4_block(g, &q);
        codes[i] = q;
        scales[row * pitch + b] = (uint8_t)byte;
    }
}

// ------------------------------------------------------------------------ product
// The weights are the M operand (128 outputs n a tile) and the rows the N operand (16..128 of
// one segment), so that a segment of a few rows costs a narrow MMA and not a 128-row one.
//   warp 0  TMA: weight codes, weight scales and row codes of 256 reduction steps a stage
//   warp 1  copies the stage's scales to TMEM and issues tcgen05.mma.kind::mxf4 (K = 64)
//   warps 2, 3  put the rows' scales (any row offset, so no TMA) in tensor-core order
//   warps 4-7  epilogue: TMEM to bf16 y, while the next unit runs in the other accumulator
constexpr int kMxStages = 6;
constexpr int kMxK = 256;                 // reduction elements a stage: 128 bytes of codes
constexpr int kMxTile = 128 * 128;        // bytes: 128 rows x 128 bytes
constexpr int kMxSf = 1024;               // bytes: scales of 128 rows x 8 blocks
constexpr int kMxStageBytes = 2 * kMxTile + 2 * kMxSf;
constexpr int kMxTmemCols = 512;
constexpr int kMxSfCols = 16;             // TMEM columns of one stage's scales (A 8, B 8)
constexpr int kMxSfBase = 256;            // two accumulators of 128 columns lie before

struct MxParams {
    const MTile* tiles;
    const int32_t* ntiles;
    const int32_t* slot_expert;
    const uint8_t* row_scales;
    const uint8_t* w_scales;
    uint16_t* y;
    int64_t nrows;
    int E, H, Hp, MT, KB, pitch;
    int32_t* status;
};

struct MxUnit {
    int row0, rows, expert, mt;
};

// The unit's tile and expert; expert < 0 for a slot whose expert is unknown (reported, skipped).
__device__ __forceinline__ MxUnit mx_unit(const MxParams& p, int unit) {
    const int t = unit / p.MT;
    const MTile tile = p.tiles[t];
    MxUnit u;
    u.row0 = tile.row0;
    u.rows = tile.rows;
    u.mt = unit - t * p.MT;
    u.expert = tile.wsel >= 0 ? tile.wsel : p.slot_expert[-1 - tile.wsel];
    if (u.expert >= p.E) u.expert = -1;
    return u;
}

__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint64_t* bar, void* dst,
                                            int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// Shared-memory descriptor of a 512-byte scale block: 32 rows of 16 bytes, no swizzle, groups
// of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
// 32 rows x 16 bytes of scales to 4 TMEM columns, in each of the four 32-lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t sdesc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc)
                 : "memory");
}

// Instruction descriptor, kind::mxf4: e2m1 operands (1 at bits 7 and 10), N >> 3 at bit 17,
// e8m0 scales (bit 23), M >> 7 at bit 27; the first of the K step's two scale bytes (0 or 2 of
// the TMEM word's four) at bits 4 (B) and 29 (A).
__device__ __forceinline__ uint32_t idesc_mxf4(int N, uint32_t sf) {
    return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | (1u << 27) |
           (sf << 29);
}

__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
            "r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ int round16(int v) { return (v + 15) & ~15; }

__global__ void __launch_bounds__(kThreads, 1) grouped_gemm_mx_kernel(
    const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX16,
    const __grid_constant__ CUtensorMap tmX32, const __grid_constant__ CUtensorMap tmX64,
    const __grid_constant__ CUtensorMap tmX128, const MxParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t* smA = smem;
    uint8_t* smB = smA + kMxStages * kMxTile;
    uint8_t* smSA = smB + kMxStages * kMxTile;
    uint8_t* smSB = smSA + kMxStages * kMxSf;
    uint64_t* full = reinterpret_cast<uint64_t*>(smSB + kMxStages * kMxSf);
    uint64_t* empty = full + kMxStages;
    uint64_t* tfull = empty + kMxStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    int32_t* status = p.status;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMxStages; ++s) {
            mbar_init(&full[s], 2);   // the TMA thread (with its bytes) and the scale warp
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 4);
        }
        mbar_init(drain, 1);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(s_tmem)),
                     "r"(kMxTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *s_tmem;

    const int total = *p.ntiles * p.MT;
    const int nst = (p.H + kMxK - 1) / kMxK;   // stages a unit
    uint32_t pr_s = 0, pr_ph = 0, pr_armed = 0;

    if (warp == 0) {
        if (lane == 0) {
            bool live = true;
            for (int unit = blockIdx.x; unit < total && live; unit += gridDim.x) {
                const MxUnit u = mx_unit(p, unit);
                if (u.expert < 0) {
                    set_status(status, BEP_DERR_BOUNDS);
                    continue;
                }
                const CUtensorMap* tmX = u.rows <= 16   ? &tmX16
                                         : u.rows <= 32 ? &tmX32
                                         : u.rows <= 64 ? &tmX64
                                                        : &tmX128;
                const int box = u.rows <= 16 ? 16 : u.rows <= 32 ? 32 : u.rows <= 64 ? 64 : 128;
                const uint8_t* sf = p.w_scales + ((int64_t)u.expert * p.MT + u.mt) * p.KB * 512;
                for (int k = 0; k < nst; ++k) {
                    if (!mbar_wait(&empty[pr_s], pr_ph ^ 1u, s_abort, status)) {
                        live = false;
                        break;
                    }
                    const uint32_t sf_bytes = 2 * k + 1 < p.KB ? 1024 : 512;
                    mbar_arrive_expect_tx(&full[pr_s], kMxTile + box * 128 + sf_bytes);
                    ++pr_armed;
                    tma_load_3d(&tmW, &full[pr_s], smA + pr_s * kMxTile, k * 128, u.mt * 128, u.expert);
                    tma_load_2d(tmX, &full[pr_s], smB + pr_s * kMxTile, k * 128, u.row0);
                    bulk_load(smSA + pr_s * kMxSf, sf + (int64_t)k * 1024, sf_bytes, &full[pr_s]);
                    if (++pr_s == kMxStages) {
                        pr_s = 0;
                        pr_ph ^= 1u;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint64_t da = sdesc_sw128(smem_u32(smA), 16, 1024), db = sdesc_sw128(smem_u32(smB), 16, 1024);
            const uint64_t dsa = sdesc_scales(smem_u32(smSA)), dsb = sdesc_scales(smem_u32(smSB));
            uint32_t s = 0, ph = 0;
            int it = 0;
            bool live = true;
            for (int unit = blockIdx.x; unit < total && live; unit += gridDim.x) {
                const MxUnit u = mx_unit(p, unit);
                if (u.expert < 0) continue;
                const int N = round16(u.rows);
                const int acc = it & 1;
                if (!mbar_wait(&tempty[acc], ((it >> 1) & 1) ^ 1u, s_abort, status)) break;
                ++it;
                const uint32_t dt = tmem_base + acc * 128;
                const uint32_t id0 = idesc_mxf4(N, 0), id2 = idesc_mxf4(N, 2);
                for (int k = 0; k < nst; ++k) {
                    if (!mbar_wait(&full[s], ph, s_abort, status)) {
                        live = false;
                        break;
                    }
                    tc_fence_after();
                    // descriptors count 16-byte units: a tile is 1024 of them, a K step 2, a scale block 32
                    const uint64_t a = da + s * (kMxTile / 16), b = db + s * (kMxTile / 16);
                    const uint64_t sa = dsa + s * (kMxSf / 16), sb = dsb + s * (kMxSf / 16);
                    // the scales' TMEM columns belong to the ring stage: they are overwritten only
                    // after the stage's last use has been committed
                    const uint32_t ta = tmem_base + kMxSfBase + s * kMxSfCols, tb = ta + 8;
                    const int steps = min(4, (p.H - k * kMxK) / 64);
                    copy_scales(ta, sa);
                    copy_scales(tb, sb);
                    mma_mxf4(dt, a, b, id0, ta, tb, k != 0);
                    if (steps > 1) mma_mxf4(dt, a + 2, b + 2, id2, ta, tb, 1);
                    if (steps > 2) {
                        copy_scales(ta + 4, sa + 32);
                        copy_scales(tb + 4, sb + 32);
                        mma_mxf4(dt, a + 4, b + 4, id0, ta + 4, tb + 4, 1);
                        if (steps > 3) mma_mxf4(dt, a + 6, b + 6, id2, ta + 4, tb + 4, 1);
                    }
                    mma_commit(&empty[s]);
                    if (++s == kMxStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (live) mma_commit(&tfull[acc]);
            }
        }
    } else if (warp < 4) {
        // A 16-byte piece of a row's scales serves two stages; the two warps take the pieces in
        // turn and hold two of their own in flight, so a load has four pieces (eight stages) to
        // arrive: with one warp one piece ahead these loads, not the operands', set the pace
        // (decode of 64 rows by 384 experts' 7168 x 2048: 120 us instead of 95).
        const int mine = warp - 2;
        uint32_t s = 0, ph = 0;
        bool live = true;
        const int pieces = (nst + 1) / 2;
        for (int unit = blockIdx.x; unit < total && live; unit += gridDim.x) {
            const MxUnit u = mx_unit(p, unit);
            if (u.expert < 0) continue;
            const int N = round16(u.rows);
            const uint4* src[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int64_t row = min((int64_t)u.row0 + 32 * c + lane, p.nrows - 1);
                src[c] = reinterpret_cast<const uint4*>(p.row_scales + row * p.pitch);
            }
            uint4 v0[4] = {}, v1[4] = {};
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (32 * c < N) {
                    if (mine < pieces) v0[c] = __ldg(src[c] + mine);
                    if (mine + 2 < pieces) v1[c] = __ldg(src[c] + mine + 2);
                }
            for (int g = 0; g < pieces && live; ++g) {
                const int here = min(2, nst - 2 * g);   // stages of this piece
                if ((g & 1) != mine) {
                    s += here;
                    if (s >= kMxStages) {
                        s -= kMxStages;
                        ph ^= 1u;
                    }
                    continue;
                }
                uint4 v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    v[c] = v0[c];
                    v0[c] = v1[c];
                    if (32 * c < N && g + 4 < pieces) v1[c] = __ldg(src[c] + g + 4);
                }
                for (int half = 0; half < here; ++half) {
                    if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1u, s_abort, status))) {
                        live = false;
                        break;
                    }
                    uint32_t* d = reinterpret_cast<uint32_t*>(smSB + s * kMxSf) + lane * 4;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (32 * c < N) {
                            d[c] = half ? v[c].z : v[c].x;
                            d[128 + c] = half ? v[c].w : v[c].y;
                        }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[s]);
                    if (++s == kMxStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
        }
    } else if (warp >= 4) {
        const int quarter = warp - 4;
        int it = 0;
        for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
            const MxUnit u = mx_unit(p, unit);
            if (u.expert < 0) continue;
            const int acc = it & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], (it >> 1) & 1, s_abort, status))) break;
            ++it;
            tc_fence_after();
            // lane l of quarter q holds output n = 128 mt + 32 q + l, its columns the rows
            const int n0 = u.mt * 128 + quarter * 32;
            const bool odd = lane & 1;
            for (int c0 = 0; c0 < u.rows; c0 += 32) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * 128 + c0, r);
                // lanes 2i and 2i + 1 trade a row each, so that a lane stores two outputs of one row
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float keep = __uint_as_float(odd ? r[2 * j + 1] : r[2 * j]);
                    const float give = __uint_as_float(odd ? r[2 * j] : r[2 * j + 1]);
                    const float got = __shfl_xor_sync(0xffffffffu, give, 1);
                    const int c = c0 + 2 * j + (odd ? 1 : 0);
                    if (c < u.rows && n0 < p.Hp)
                        *reinterpret_cast<uint32_t*>(p.y + ((int64_t)u.row0 + c) * p.Hp + n0 + (lane & ~1)) =
                            odd ? pack_bf16x2(got, keep) : pack_bf16x2(keep, got);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[acc]);
        }
    }

    __syncthreads();
    if (*s_abort) {
        // A wait gave up: what was started lands before shared memory and TMEM are released.
        if (warp == 0 && lane == 0) {
            for (uint32_t i = 0; i < pr_armed && i < (uint32_t)kMxStages; ++i) {
                if (pr_s == 0) {
                    pr_s = kMxStages;
                    pr_ph ^= 1u;
                }
                --pr_s;
                mbar_drain(&full[pr_s], pr_ph);
            }
        } else if (warp == 1 && lane == 0) {
            mma_commit(drain);
            mbar_drain(drain, 0);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                     "r"(kMxTmemCols)
                     : "memory");
    }
}

constexpr size_t kMxSmem = 1024 + (size_t)kMxStages * kMxStageBytes + (2 * kMxStages + 5) * 8 + 16;

// u8 tensor of `dims` (innermost first, dense but for `pitch` bytes a row), 128-byte boxes of
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

int grid_for(int64_t warps, int num_sms) {
    const int64_t g = (warps + kThreads / 32 - 1) / (kThreads / 32), cap = (int64_t)num_sms * 8;
    return (int)(g < cap ? (g > 0 ? g : 1) : cap);
}

}  // namespace

cudaError_t mx_setup() {
    return cudaFuncSetAttribute(grouped_gemm_mx_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)kMxSmem);
}

cudaError_t launch_mx_weight(const Dims& d, const uint16_t* w, uint8_t* codes, uint8_t* scales,
                             cudaStream_t st) {
    const dim3 grid((unsigned)(d.Hp / 64) * ((d.H + 255) / 256), (unsigned)d.E);
    mx_weight_kernel<<<grid, kThreads, 0, st>>>(reinterpret_cast<const uint32_t*>(w),
                                                reinterpret_cast<uint4*>(codes), scales, d.H, d.Hp);
    return cudaGetLastError();
}

cudaError_t launch_dispatch_mx(const Dims& d, const Workspace& ws, const uint16_t* x,
                               const int32_t* dest, uint8_t* codes, uint8_t* scales, int num_sms,
                               cudaStream_t st) {
    const int64_t ntok = (int64_t)d.R * d.S;
    const int nblk = d.H / kMxBlock, runs = (nblk + 31) / 32;
    dispatch_mx_kernel<<<grid_for(ntok * runs, num_sms), kThreads, 0, st>>>(
        reinterpret_cast<const uint4*>(x), dest, reinterpret_cast<uint4*>(codes), scales, ntok, d.K,
        nblk, runs, mx_scale_pitch(d.H), (int64_t)d.R * d.C, ws.status);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_mx(int64_t rows, int F, const uint16_t* h, uint8_t* codes,
                             uint8_t* scales, int num_sms, cudaStream_t st) {
    const int nblk = F / kMxBlock;
    swiglu_mx_kernel<<<grid_for((rows * nblk + 31) / 32, num_sms), kThreads, 0, st>>>(
        reinterpret_cast<const uint4*>(h), reinterpret_cast<uint4*>(codes), scales, rows * nblk, nblk,
        mx_scale_pitch(F));
    return cudaGetLastError();
}

cudaError_t launch_grouped_gemm_mx(const Dims& d, const Workspace& ws, const int32_t* cu,
                                   const int32_t* slot_expert, const uint8_t* codes,
                                   const uint8_t* scales, const uint8_t* w_codes,
                                   const uint8_t* w_scales, uint16_t* y, int num_sms,
                                   cudaStream_t st) {
    const uint64_t wd[3] = {(uint64_t)d.H / 2, (uint64_t)d.Hp, (uint64_t)d.E};
    const uint64_t xd[2] = {(uint64_t)d.H / 2, (uint64_t)d.R * d.C};
    CUtensorMap tmW, tmX[4];
    if (!encode_u8(&tmW, w_codes, 3, wd, 128)) return cudaErrorInvalidValue;
    for (int i = 0; i < 4; ++i)
        if (!encode_u8(&tmX[i], codes, 2, xd, 16u << i)) return cudaErrorInvalidValue;
    MxParams p;
    p.tiles = ws.tiles;
    p.ntiles = ws.ntiles;
    p.slot_expert = slot_expert;
    p.row_scales = scales;
    p.w_scales = w_scales;
    p.y = y;
    p.nrows = (int64_t)d.R * d.C;
    p.E = d.E;
    p.H = d.H;
    p.Hp = d.Hp;
    p.MT = (d.Hp + 127) / 128;
    p.KB = (d.H + 127) / 128;
    p.pitch = mx_scale_pitch(d.H);
    p.status = ws.status;
    const cudaError_t err = launch_gemm_tiles(d, ws, cu, st);
    if (err != cudaSuccess) return err;
    grouped_gemm_mx_kernel<<<num_sms, kThreads, kMxSmem, st>>>(tmW, tmX[0], tmX[1], tmX[2], tmX[3], p);
    return cudaGetLastError();
}

}  // namespace bep
