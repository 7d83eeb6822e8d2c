// Grouped products of any width (sm_103a, tcgen05): rows grouped by expert, each group by its expert's own
// matrix, and the matrices' gradients. Widths are multiples of 8 and need not be multiples of a tile, rows may
// lie apart, and the products of replicas and of overflow rows go to the expert itself:
//   y[row, :]  = alpha * x[row, :] W(e) + add[row, :]        W(e) = w[e] [K, N], or w[e]^T with w[e] [N, K]
//   g[e]      (+)= alpha * sum over the rows of e: x[row]^T dy[row]                              (fp32)
// e = rho for a segment rho < E and slot_expert[u][rho - E] for a prefetch slot.
//
// Both kernels are persistent, one CTA an SM:
//   warp 0      TMA (128-byte swizzle) into a ring of stages of 64 reduction steps
//   warp 1      tcgen05.mma.kind::f16, M = 128, N <= 256, into one of two accumulators
//   warps 2-9   epilogue: TMEM, turned in shared memory, to whole pieces of rows
// What lies outside a matrix arrives as zeros (the tensor maps end at the widths). Where there are fewer units
// than SMs, the reduction is cut into parts; each part leaves its fp32 tile in the context's workspace and the CTA that
// comes last adds them in the order of the parts, so that the result does not depend on who that was.

#include <cudaTypedefs.h>

#include "tiles.cuh"

namespace bep {
namespace {

constexpr int kRgThreads = 32 * 10;
constexpr int kRgA = 128 * 128;          // bytes: 128 rows (columns) x 64 reduction steps
constexpr int kRgChunk = 64 * 128;       // bytes: 64 x 64 elements
constexpr int kRgBox = 32 * 128;         // bytes: an epilogue warp's 32 x 32 fp32
constexpr int kRgTmem = 512;
constexpr int kRgMaxStages = 12;
constexpr int kRgBars = 2 * kRgMaxStages + 5;
constexpr int kRgRing = 227 * 1024 - 1024 - 8 * kRgBox - kRgBars * 8 - 32;   // bytes of stages
constexpr int kRgMaxParts = 16;

struct RgParams {
    const MTile* tiles;
    const int32_t* ntiles;
    const int32_t* slot_expert;
    uint16_t* y;
    const uint16_t* add;      // or null
    int64_t ldy, ldadd;
    float alpha;
    int E, N, kbn;            // output columns, reduction blocks of 64
    int BN, NT;               // columns of a tile, tiles
    int stages, a_bytes, b_bytes;
    int32_t* tickets;
    float* partial;
    int32_t* status;
};

struct RgDwParams {
    const MTile* segs;        // segments by expert, in (rank, row) order
    const int32_t* first;     // [E + 1]
    const int32_t* blocks;    // [E], blocks of 64 rows
    float* g;
    int64_t g_expert;         // elements of an expert's gradient
    int64_t ldm, ldn;         // strides of g along the M side and the N side: one of them is 1
    float alpha;
    int E, Md, Nd;            // widths of the sides
    int BN, MT, NT, parts;
    int stages, b_bytes;
    int accumulate;
    int32_t* tickets;
    float* partial;
    int32_t* status;
};

__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint64_t* bar, void* dst, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Operand descriptor of 16 reduction steps of a stage: K-major rows of 64 elements (128 bytes), or MN-major
// chunks of 64 columns x 64 reduction steps, 8 KB each.
template <bool kMN>
__device__ __forceinline__ uint64_t operand(uint32_t base, int kk) {
    return kMN ? sdesc_sw128(base + kk * 2048, kRgChunk, 1024) : sdesc_sw128(base + kk * 32, 16, 1024);
}

// Instruction descriptor, kind::f16: fp32 accumulator, bf16 A and B, major bits 15/16 (1: MN), M = 128.
__device__ __forceinline__ uint32_t idesc_bf16(int N, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

// The 8 epilogue warps.
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool epi_all(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, 1, 256, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

// What both kernels set up and take down alike.
struct Frame {
    uint8_t* ring;
    uint8_t* boxes;
    uint64_t *full, *empty, *tfull, *tempty, *drain;
    uint32_t* s_tmem;
    volatile int* s_abort;
    int* s_last;
    uint32_t tmem;
};
__device__ __forceinline__ Frame open_frame(uint8_t* smem_raw, int stages) {
    Frame f;
    const uint32_t raw = smem_u32(smem_raw);
    f.ring = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    f.boxes = f.ring + kRgRing / 1024 * 1024;
    f.full = reinterpret_cast<uint64_t*>(f.boxes + 8 * kRgBox);
    f.empty = f.full + kRgMaxStages;
    f.tfull = f.empty + kRgMaxStages;
    f.tempty = f.tfull + 2;
    f.drain = f.tempty + 2;
    f.s_tmem = reinterpret_cast<uint32_t*>(f.drain + 1);
    f.s_abort = reinterpret_cast<volatile int*>(f.s_tmem + 1);
    f.s_last = reinterpret_cast<int*>(f.s_tmem + 2);
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&f.full[s], 1);
            mbar_init(&f.empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&f.tfull[a], 1);
            mbar_init(&f.tempty[a], 8);
        }
        mbar_init(f.drain, 1);
        *f.s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x < 32) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(f.s_tmem)),
                     "r"(kRgTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    f.tmem = *f.s_tmem;
    return f;
}
// pr_s, pr_ph, pr_armed: the producer's ring position and the stages that it armed.
__device__ __forceinline__ void close_frame(const Frame& f, int stages, uint32_t pr_s, uint32_t pr_ph, uint32_t pr_armed) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (*f.s_abort) {
        // A wait gave up: what was started lands before shared memory and TMEM are released, each wait bounded.
        if (warp == 0 && lane == 0) {
            for (uint32_t i = 0; i < pr_armed && i < (uint32_t)stages; ++i) {
                if (pr_s == 0) {
                    pr_s = stages;
                    pr_ph ^= 1u;
                }
                --pr_s;
                mbar_drain(&f.full[pr_s], pr_ph);
            }
        } else if (warp == 1 && lane == 0) {
            mma_commit(f.drain);
            mbar_drain(f.drain, 0);
        }
        __syncthreads();
    }
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(f.tmem), "r"(kRgTmem) : "memory");
    }
}

// A part's tile in the workspace: [column][128 rows], so that a warp's rows lie together.
constexpr int kPartRows = 128;
__device__ __forceinline__ float* part_tile(float* base, int slot) {
    return base + (int64_t)slot * (kPartRows * kRgPartCols);
}
// This thread's row, 32 columns: to a part's tile, and the sum of a unit's parts in their order.
__device__ __forceinline__ void put_part(float* tile, int c0, int row, const uint32_t* r) {
#pragma unroll
    for (int j = 0; j < 32; ++j) __stcg(tile + (c0 + j) * kPartRows + row, __uint_as_float(r[j]));
}
__device__ __forceinline__ void sum_parts(float* base, int slot0, int parts, int c0, int row, uint32_t* r) {
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __ldcg(part_tile(base, slot0) + (c0 + j) * kPartRows + row);
    for (int z = 1; z < parts; ++z) {
        const float* t = part_tile(base, slot0 + z);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] += __ldcg(t + (c0 + j) * kPartRows + row);
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(v[j]);
}
// True in the CTA that brings a unit's last part (all 8 epilogue warps call it, their parts written).
__device__ __forceinline__ bool last_part(int32_t* ticket, int parts, int* s_last) {
    __threadfence();
    epi_sync();
    if (threadIdx.x == 64) {
        const int n = atomicAdd(ticket, 1);
        __threadfence();
        *s_last = n == parts - 1;
    }
    epi_sync();
    const bool last = *s_last != 0;
    epi_sync();   // read before the next unit writes it
    return last;
}

// ------------------------------------------------------------------------ rows
// A unit: up to 128 rows of a segment x BN columns. A small tile leaves the accumulator's other rows to whatever the
// stage holds behind its own; they are not stored.
template <bool kTrans>
__global__ void __launch_bounds__(kRgThreads, 1) ragged_kernel(
    const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX16,
    const __grid_constant__ CUtensorMap tmX32, const __grid_constant__ CUtensorMap tmX64,
    const __grid_constant__ CUtensorMap tmX128, const RgParams p) {
    extern __shared__ uint8_t smem_raw[];
    Frame f = open_frame(smem_raw, p.stages);
    uint8_t* smA = f.ring;
    uint8_t* smB = smA + p.stages * p.a_bytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t pr_s = 0, pr_ph = 0, pr_armed = 0;
    grid_wait();   // launched early: the work list and the rows are complete from here on

    const int units = *p.ntiles * p.NT;
    int parts = 1;
    if (p.partial && units > 0) parts = max(1, min(min((int)gridDim.x / units, p.kbn / 4), kRgMaxParts));
    const int total = units * parts;
    struct Item {
        int row0, rows, expert, n0, unit, kb0, kb1;
    };
    auto item_at = [&](int i) {
        Item it;
        it.unit = i / parts;
        const int part = i - it.unit * parts, tile = it.unit / p.NT;
        const MTile t = p.tiles[tile];
        it.row0 = t.row0;
        it.rows = t.rows;
        it.expert = t.wsel >= 0 ? t.wsel : p.slot_expert[-1 - t.wsel];
        if (it.expert >= p.E) it.expert = -1;
        it.n0 = (it.unit - tile * p.NT) * p.BN;
        it.kb0 = part * p.kbn / parts;
        it.kb1 = (part + 1) * p.kbn / parts;
        return it;
    };

    if (warp == 0) {
        if (lane == 0) {
            bool live = true;
            for (int i = blockIdx.x; i < total && live; i += gridDim.x) {
                const Item u = item_at(i);
                if (u.expert < 0) {
                    set_status(p.status, BEP_DERR_BOUNDS);
                    continue;
                }
                const CUtensorMap* tmX = u.rows <= 16 ? &tmX16 : u.rows <= 32 ? &tmX32 : u.rows <= 64 ? &tmX64 : &tmX128;
                const int box = u.rows <= 16 ? 16 : u.rows <= 32 ? 32 : u.rows <= 64 ? 64 : 128;
                for (int kb = u.kb0; kb < u.kb1; ++kb) {
                    if (!mbar_wait_held(&f.empty[pr_s], pr_ph ^ 1u, f.s_abort, p.status)) {
                        live = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&f.full[pr_s], box * 128 + p.b_bytes);
                    ++pr_armed;
                    tma_load_2d(tmX, &f.full[pr_s], smA + pr_s * p.a_bytes, kb * 64, u.row0);
                    uint8_t* b = smB + pr_s * p.b_bytes;
                    if (kTrans)
                        tma_load_3d(&tmW, &f.full[pr_s], b, kb * 64, u.n0, u.expert);
                    else
                        for (int c = 0; c * kRgChunk < p.b_bytes; ++c)
                            tma_load_3d(&tmW, &f.full[pr_s], b + c * kRgChunk, u.n0 + c * 64, kb * 64, u.expert);
                    if (++pr_s == (uint32_t)p.stages) {
                        pr_s = 0;
                        pr_ph ^= 1u;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t idesc = idesc_bf16(p.BN, false, !kTrans);
            uint32_t s = 0, ph = 0;
            int it = 0;
            bool live = true;
            for (int i = blockIdx.x; i < total && live; i += gridDim.x) {
                const Item u = item_at(i);
                if (u.expert < 0) continue;
                const int acc = it & 1;
                if (!mbar_wait_held(&f.tempty[acc], ((it >> 1) & 1) ^ 1u, f.s_abort, p.status)) break;
                ++it;
                tc_fence_after();
                const uint32_t dt = f.tmem + acc * 256;
                for (int kb = u.kb0; kb < u.kb1; ++kb) {
                    if (!mbar_wait_held(&f.full[s], ph, f.s_abort, p.status)) {
                        live = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = smem_u32(smA + s * p.a_bytes), b = smem_u32(smB + s * p.b_bytes);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_bf16(dt, operand<false>(a, kk), operand<!kTrans>(b, kk), idesc, (kb != u.kb0) || kk);
                    mma_commit(&f.empty[s]);
                    if (++s == (uint32_t)p.stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (live) mma_commit(&f.tfull[acc]);
            }
        }
    } else {
        const int q = warp & 3, second = (warp - 2) >> 2;
        uint8_t* stg = f.boxes + (warp - 2) * kRgBox;
        const int sub = lane >> 2, piece = lane & 3;   // on the way out: 4 lanes take 32 columns of a row
        int it = 0;
        for (int i = blockIdx.x; i < total; i += gridDim.x) {
            const Item u = item_at(i);
            if (u.expert < 0) continue;
            const int acc = it & 1;
            const int rows = u.rows - 32 * q;          // of this warp's 32
            const int64_t row0 = (int64_t)u.row0 + 32 * q;
            // what the product is added to is on its way while the product is computed
            uint4 pre[4][4];
            if (p.add && parts == 1) {
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int c = 32 * (2 * b + second) + 8 * piece;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (c < p.BN && u.n0 + c < p.N && 8 * j + sub < rows)
                            pre[b][j] = *reinterpret_cast<const uint4*>(p.add + (row0 + 8 * j + sub) * p.ldadd + u.n0 + c);
                }
            }
            const bool done = __all_sync(0xffffffffu, mbar_wait_held(&f.tfull[acc], (it >> 1) & 1, f.s_abort, p.status));
            // (warps that meet at barriers give up together)
            if (parts > 1 ? !epi_all(done) : !done) break;
            ++it;
            tc_fence_after();
            const uint32_t tacc = f.tmem + ((uint32_t)(q * 32) << 16) + acc * 256;
            bool held = true;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&f.tempty[acc]);
                held = false;
            };
            const int slot0 = u.unit * parts;
            if (parts > 1) {
                for (int c0 = 32 * second; c0 < p.BN; c0 += 64) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tacc + c0, r);
                    put_part(part_tile(p.partial, i), c0, 32 * q + lane, r);
                }
                release();
                if (!last_part(p.tickets + u.unit, parts, f.s_last)) continue;
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int c0 = 32 * (2 * b + second);
                if (c0 >= p.BN) break;
                uint32_t r[32];
                if (parts > 1) sum_parts(p.partial, slot0, parts, c0, 32 * q + lane, r);
                else tmem_ld_32x32b_x32(tacc + c0, r);
                if (held && c0 + 64 >= p.BN) release();
                uint4* line = reinterpret_cast<uint4*>(stg + lane * 128);
                __syncwarp();   // the box before has been read
#pragma unroll
                for (int j = 0; j < 8; ++j) line[j ^ (lane & 7)] = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                __syncwarp();
                const int c = c0 + 8 * piece;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int rr = 8 * j + sub;
                    const float4 lo = *reinterpret_cast<const float4*>(stg + rr * 128 + (((2 * piece) ^ (rr & 7)) << 4));
                    const float4 hi = *reinterpret_cast<const float4*>(stg + rr * 128 + (((2 * piece + 1) ^ (rr & 7)) << 4));
                    if (c >= p.BN || u.n0 + c >= p.N || rr >= rows) continue;
                    float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    if (p.add) {
                        const uint4 t = parts == 1 ? pre[b][j]
                                                   : *reinterpret_cast<const uint4*>(p.add + (row0 + rr) * p.ldadd + u.n0 + c);
                        const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            v[2 * e] = fmaf(p.alpha, v[2 * e], __uint_as_float(w[e] << 16));
                            v[2 * e + 1] = fmaf(p.alpha, v[2 * e + 1], __uint_as_float(w[e] & 0xffff0000u));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] *= p.alpha;
                    }
                    *reinterpret_cast<uint4*>(p.y + (row0 + rr) * p.ldy + u.n0 + c) =
                        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                   pack_bf16x2(v[6], v[7]));
                }
            }
            if (held) release();   // a warp without columns
        }
    }
    close_frame(f, p.stages, pr_s, pr_ph, pr_armed);
}

// ------------------------------------------------------------------------ matrices
// The segments of each expert, in (rank, row) order: segs[first[e] .. first[e + 1]). One CTA. A slot whose expert is
// unknown is reported and left out; a table with any inconsistent segment is refused as a whole.
__global__ void __launch_bounds__(1024) ragged_segments_kernel(const int32_t* cu, const int32_t* slot_expert, Dims d,
                                                               Workspace ws) {
    __shared__ int s_pos[kMaxE], s_blk[kMaxE];
    __shared__ int s_sum[32];
    grid_launch_dependents();
    grid_wait();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    for (int e = t; e < kMaxE; e += 1024) s_pos[e] = s_blk[e] = 0;
    if (t < kRgTickets) ws.tickets[t] = 0;
    __syncthreads();
    auto expert_of = [&](int u, int rho) {
        const int e = rho < d.E ? rho : slot_expert[u * d.B + rho - d.E];
        return e >= 0 && e < d.E ? e : -1;
    };
    int bad = 0, unknown = 0;
    for (int u = 0; u < d.R; ++u)
        for (int rho = t; rho < d.NROW; rho += 1024) {
            const int a = cu[u * (d.NROW + 1) + rho], b = cu[u * (d.NROW + 1) + rho + 1];
            bad |= a < 0 || b < a || (int64_t)b > d.C;
            if (b <= a) continue;
            const int e = expert_of(u, rho);
            if (e < 0) {
                unknown = 1;
            } else {
                atomicAdd(&s_pos[e], 1);
                atomicAdd(&s_blk[e], (b - a + 63) / 64);
            }
        }
    bad = __syncthreads_or(bad);
    if (__syncthreads_or(unknown) && t == 0) set_status(ws.status, BEP_DERR_BOUNDS);
    if (bad && t == 0) set_status(ws.status, BEP_DERR_BOUNDS);
    for (int e = t; e < d.E; e += 1024) ws.seg_blocks[e] = s_blk[e];
    // exclusive scan of the counts: two experts a thread
    static_assert(kMaxE == 2048, "two experts a thread");
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
    const int at = bad ? -1 : before + incl - n0 - n1;
    s_pos[2 * t] = at;
    s_pos[2 * t + 1] = at + n0;
    if (2 * t <= d.E) ws.seg_first[2 * t] = bad ? -1 : at;
    if (2 * t + 1 <= d.E) ws.seg_first[2 * t + 1] = bad ? -1 : at + n0;
    if (t == 1023 && d.E == kMaxE) ws.seg_first[kMaxE] = bad ? -1 : at + n0 + n1;
    __syncthreads();
    if (bad) return;
    for (int u = 0; u < d.R; ++u) {
        const int32_t* row = cu + u * (d.NROW + 1);
        // home rows: every one its own expert
        for (int e = t; e < d.E; e += 1024) {
            const int a = row[e], b = row[e + 1];
            if (b > a) ws.tiles[s_pos[e]++] = MTile{(int32_t)(u * d.C + a), b - a, e, 0};
        }
        __syncthreads();
        // slots: several of a rank may hold one expert, so a slot counts those before it
        for (int j0 = 0; j0 < d.B; j0 += 1024) {
            const int j = j0 + t;
            int e = -1, a = 0, b = 0, ahead = 0;
            if (j < d.B) {
                a = row[d.E + j];
                b = row[d.E + j + 1];
                if (b > a) e = expert_of(u, d.E + j);
            }
            if (e >= 0)
                for (int i = j0; i < j; ++i)
                    ahead += slot_expert[u * d.B + i] == e && row[d.E + i + 1] > row[d.E + i];
            if (e >= 0) ws.tiles[s_pos[e] + ahead] = MTile{(int32_t)(u * d.C + a), b - a, e, 0};
            __syncthreads();
            if (e >= 0) atomicAdd(&s_pos[e], 1);
            __syncthreads();
        }
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

// Calls op(row, rows of the block) for the blocks [b0, b1) until it returns false.
template <typename F>
__device__ __forceinline__ bool each_block(const RgDwParams& p, int e, int b0, int b1, F&& op) {
    int b = 0;
    for (int s = p.first[e]; s < p.first[e + 1] && b < b1; ++s) {
        const MTile t = p.segs[s];
        const int n = (t.rows + 63) / 64;
        for (int k = max(0, b0 - b); k < n && b + k < b1; ++k)
            if (!op(t.row0 + 64 * k, min(64, t.rows - 64 * k))) return false;
        b += n;
    }
    return true;
}

// A unit: 128 x BN of an expert's gradient. The wider side is the M operand; both lie along the rows (MN-major).
__global__ void __launch_bounds__(kRgThreads, 1) ragged_dw_kernel(const __grid_constant__ CUtensorMap tmM,
                                                                  const __grid_constant__ CUtensorMap tmN,
                                                                  const RgDwParams p) {
    extern __shared__ uint8_t smem_raw[];
    Frame f = open_frame(smem_raw, p.stages);
    const int stage = kRgA + p.b_bytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t pr_s = 0, pr_ph = 0, pr_armed = 0;
    grid_wait();   // launched early: the segments and the rows are complete from here on

    const int parts = p.parts;
    const int total = p.first[0] < 0 ? 0 : p.E * p.MT * p.NT * parts;
    struct Item {
        int unit, expert, m0, n0, b0, b1;
    };
    auto item_at = [&](int i) {
        Item it;
        it.unit = i / parts;
        const int part = i - it.unit * parts, per = p.MT * p.NT;
        it.expert = it.unit / per;
        const int rest = it.unit - it.expert * per;
        it.m0 = rest / p.NT * 128;
        it.n0 = rest % p.NT * p.BN;
        const int64_t nb = p.blocks[it.expert];
        it.b0 = (int)(part * nb / parts);
        it.b1 = (int)((part + 1) * nb / parts);
        return it;
    };

    if (warp == 0) {
        if (lane == 0) {
            bool live = true;
            for (int i = blockIdx.x; i < total && live; i += gridDim.x) {
                const Item u = item_at(i);
                live = each_block(p, u.expert, u.b0, u.b1, [&](int row, int) {
                    if (!mbar_wait_held(&f.empty[pr_s], pr_ph ^ 1u, f.s_abort, p.status)) return false;
                    mbar_arrive_expect_tx(&f.full[pr_s], stage);
                    ++pr_armed;
                    uint8_t* a = f.ring + pr_s * stage;
                    for (int c = 0; c < 2; ++c) tma_load_2d(&tmM, &f.full[pr_s], a + c * kRgChunk, u.m0 + 64 * c, row);
                    for (int c = 0; c * kRgChunk < p.b_bytes; ++c)
                        tma_load_2d(&tmN, &f.full[pr_s], a + kRgA + c * kRgChunk, u.n0 + 64 * c, row);
                    if (++pr_s == (uint32_t)p.stages) {
                        pr_s = 0;
                        pr_ph ^= 1u;
                    }
                    return true;
                });
            }
        }
    } else if (warp == 1) {
        const uint32_t idesc = idesc_bf16(p.BN, true, true);
        uint32_t s = 0, ph = 0;
        int it = 0;
        for (int i = blockIdx.x; i < total; i += gridDim.x) {
            const Item u = item_at(i);
            if (u.b0 == u.b1) continue;
            const int acc = it & 1;
            if (!__all_sync(0xffffffffu, mbar_wait_held(&f.tempty[acc], ((it >> 1) & 1) ^ 1u, f.s_abort, p.status))) break;
            ++it;
            tc_fence_after();
            const uint32_t dt = f.tmem + acc * 256;
            uint32_t add = 0;
            const bool live = each_block(p, u.expert, u.b0, u.b1, [&](int, int rows) {
                if (!__all_sync(0xffffffffu, mbar_wait_held(&f.full[s], ph, f.s_abort, p.status))) return false;
                uint8_t* at = f.ring + s * stage;
                if (rows & 15) {   // the rows behind a segment's last are another's, or nobody's
                    zero_rows(at, stage / kRgChunk, rows, lane);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                if (lane == 0) {
                    tc_fence_after();
                    const uint32_t a = smem_u32(at), b = a + kRgA;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (16 * kk < rows) {
                            mma_bf16(dt, operand<true>(a, kk), operand<true>(b, kk), idesc, add);
                            add = 1;
                        }
                    mma_commit(&f.empty[s]);
                }
                __syncwarp();
                if (++s == (uint32_t)p.stages) {
                    s = 0;
                    ph ^= 1u;
                }
                return true;
            });
            if (!live) break;
            if (lane == 0) mma_commit(&f.tfull[acc]);
            __syncwarp();
        }
    } else {
        const int q = warp & 3, second = (warp - 2) >> 2;
        uint8_t* stg = f.boxes + (warp - 2) * kRgBox;
        const int sub = lane >> 3, piece = lane & 7;   // on the way out: 8 lanes take 32 columns of a row
        int it = 0;
        for (int i = blockIdx.x; i < total; i += gridDim.x) {
            const Item u = item_at(i);
            const bool none = u.b0 == u.b1;
            const int acc = it & 1;
            if (!none) {
                const bool done = __all_sync(0xffffffffu, mbar_wait_held(&f.tfull[acc], (it >> 1) & 1, f.s_abort, p.status));
                if (parts > 1 ? !epi_all(done) : !done) break;
                ++it;
                tc_fence_after();
            }
            bool held = !none;
            const uint32_t tacc = f.tmem + ((uint32_t)(q * 32) << 16) + acc * 256;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&f.tempty[acc]);
                held = false;
            };
            auto read = [&](int c0, uint32_t* r) {
                if (none) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = 0u;
                } else {
                    tmem_ld_32x32b_x32(tacc + c0, r);
                }
            };
            if (parts > 1) {
                for (int c0 = 32 * second; c0 < p.BN; c0 += 64) {
                    uint32_t r[32];
                    read(c0, r);
                    put_part(part_tile(p.partial, i), c0, 32 * q + lane, r);
                }
                if (held) release();
                if (!last_part(p.tickets + u.unit, parts, f.s_last)) continue;
            } else if (none && p.accumulate) {
                continue;
            }
            const int m0 = u.m0 + 32 * q;   // this warp's 32 along M
            float* g = p.g + (int64_t)u.expert * p.g_expert;
            for (int c0 = 32 * second; c0 < p.BN; c0 += 64) {
                uint32_t r[32];
                if (parts > 1) sum_parts(p.partial, u.unit * parts, parts, c0, 32 * q + lane, r);
                else read(c0, r);
                if (held && c0 + 64 >= p.BN) release();
                const int n0 = u.n0 + c0;
                if (p.ldm == 1) {   // the lanes' 32 lie together
                    if (m0 + lane < p.Md) {
                        float* out = g + (int64_t)n0 * p.ldn + m0 + lane;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (c0 + j < p.BN && n0 + j < p.Nd) {
                                float v = p.alpha * __uint_as_float(r[j]);
                                if (p.accumulate) v += out[(int64_t)j * p.ldn];
                                out[(int64_t)j * p.ldn] = v;
                            }
                    }
                } else {
                    uint4* line = reinterpret_cast<uint4*>(stg + lane * 128);
                    __syncwarp();   // the box before has been read
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        line[j ^ (lane & 7)] = make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                    __syncwarp();
                    const int c = c0 + 4 * piece;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int rr = 4 * j + sub;
                        float4 v = *reinterpret_cast<const float4*>(stg + rr * 128 + ((piece ^ (rr & 7)) << 4));
                        if (c >= p.BN || u.n0 + c >= p.Nd || m0 + rr >= p.Md) continue;
                        float4* out = reinterpret_cast<float4*>(g + (int64_t)(m0 + rr) * p.ldm + u.n0 + c);
                        v.x *= p.alpha;
                        v.y *= p.alpha;
                        v.z *= p.alpha;
                        v.w *= p.alpha;
                        if (p.accumulate) {
                            const float4 o = *out;
                            v.x += o.x;
                            v.y += o.y;
                            v.z += o.z;
                            v.w += o.w;
                        }
                        *out = v;
                    }
                }
            }
            if (held) release();   // a warp without columns
        }
    }
    close_frame(f, p.stages, pr_s, pr_ph, pr_armed);
}

constexpr size_t kRgSmem = 227 * 1024;

// bf16 tensor of `dims` (innermost first) with row strides in elements, boxes of 64 x box_rows, 128-byte swizzle.
bool encode_rows(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* ld, uint32_t box_rows) {
    void* fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t d[3], strides[2];
    cuuint32_t box[3] = {64, box_rows, 1}, estr[3] = {1, 1, 1};
    for (int i = 0; i < rank; ++i) d[i] = dims[i];
    for (int i = 0; i + 1 < rank; ++i) strides[i] = ld[i] * 2;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
               m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaLaunchConfig_t rg_config(int grid, cudaStream_t st, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kRgThreads, 1, 1);
    cfg.dynamicSmemBytes = kRgSmem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// `width` in tiles of at most `most` columns, all of one size (a multiple of 16).
void cut(int width, int most, int* tile, int* tiles) {
    *tiles = (width + most - 1) / most;
    *tile = ((width + *tiles - 1) / *tiles + 15) / 16 * 16;
}

}  // namespace

cudaError_t ragged_setup() {
    cudaError_t err =
        cudaFuncSetAttribute(ragged_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRgSmem);
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(ragged_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRgSmem);
    if (err == cudaSuccess)
        err = cudaFuncSetAttribute(ragged_dw_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRgSmem);
    return err;
}

cudaError_t launch_ragged(const Dims& d, const Workspace& ws, const int32_t* cu, const int32_t* slot_expert,
                          const uint16_t* x, int64_t ldx, int K, const uint16_t* w, int N, int trans, float alpha,
                          const uint16_t* add, int64_t ldadd, uint16_t* y, int64_t ldy, int num_sms, cudaStream_t st) {
    const int64_t rows = (int64_t)d.R * d.C;
    RgParams p = {};
    p.tiles = ws.tiles;
    p.ntiles = ws.ntiles;
    p.slot_expert = slot_expert;
    p.y = y;
    p.add = add;
    p.ldy = ldy;
    p.ldadd = ldadd;
    p.alpha = alpha;
    p.E = d.E;
    p.N = N;
    p.kbn = (K + 63) / 64;
    p.status = ws.status;
    p.tickets = ws.tickets;
    // Tiles of 64 columns, whose reduction may be cut into parts, where even as many row tiles as there can be do not
    // make a unit for every SM with wider ones.
    const int64_t segs = (int64_t)d.R * d.NROW < rows ? (int64_t)d.R * d.NROW : rows;
    const int64_t most = rows / 128 + segs;
    cut(N, most * ((N + 255) / 256) < num_sms ? 64 : 256, &p.BN, &p.NT);
    if (p.BN <= kRgPartCols) p.partial = ws.partial;
    // few rows an expert: half the stage bytes for rows, more stages
    const bool few = rows / d.E <= 48;
    p.a_bytes = few ? kRgA / 2 : kRgA;
    p.b_bytes = trans ? p.BN * 128 : (p.BN + 63) / 64 * kRgChunk;
    // (the last stage of small row tiles is read as 128 rows: up to kRgA / 2 behind the rows' stages, inside the ring)
    const int fit = kRgRing / 1024 * 1024 / (p.a_bytes + p.b_bytes);
    p.stages = fit < kRgMaxStages ? fit : kRgMaxStages;

    CUtensorMap tmW, tmX[4];
    const uint64_t xd[2] = {(uint64_t)K, (uint64_t)rows}, xs[1] = {(uint64_t)ldx};
    const uint32_t boxes[4] = {16, 32, 64, 128};
    for (int i = 0; i < 4; ++i)
        if (!encode_rows(&tmX[i], x, 2, xd, xs, boxes[i])) return cudaErrorInvalidValue;
    const uint64_t wd[3] = {(uint64_t)(trans ? K : N), (uint64_t)(trans ? N : K), (uint64_t)d.E};
    const uint64_t wl[2] = {wd[0], wd[0] * wd[1]};
    if (!encode_rows(&tmW, w, 3, wd, wl, trans ? (uint32_t)p.BN : 64)) return cudaErrorInvalidValue;
    const cudaError_t err = few ? launch_row_tiles<64>(d, ws, cu, st) : launch_row_tiles<128>(d, ws, cu, st);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = rg_config(num_sms, st, attr);
    return cudaLaunchKernelEx(&cfg, trans ? ragged_kernel<true> : ragged_kernel<false>, tmW, tmX[0], tmX[1], tmX[2],
                              tmX[3], p);
}

cudaError_t launch_ragged_dw(const Dims& d, const Workspace& ws, const int32_t* cu, const int32_t* slot_expert,
                             const uint16_t* x, int64_t ldx, int K, const uint16_t* dy, int64_t lddy, int N, float alpha,
                             int accumulate, float* g, int num_sms, cudaStream_t st) {
    const int64_t rows = (int64_t)d.R * d.C;
    RgDwParams p = {};
    p.segs = ws.tiles;
    p.first = ws.seg_first;
    p.blocks = ws.seg_blocks;
    p.g = g;
    p.g_expert = (int64_t)K * N;
    p.alpha = alpha;
    p.E = d.E;
    const bool x_wide = K >= N;
    p.Md = x_wide ? K : N;
    p.Nd = x_wide ? N : K;
    p.ldm = x_wide ? N : 1;
    p.ldn = x_wide ? 1 : N;
    p.accumulate = accumulate;
    p.tickets = ws.tickets;
    p.partial = ws.partial;
    p.status = ws.status;
    p.MT = (p.Md + 127) / 128;
    const int64_t units = (int64_t)d.E * p.MT * ((p.Nd + 255) / 256);
    cut(p.Nd, units < num_sms ? 64 : 256, &p.BN, &p.NT);
    p.parts = 1;
    const int64_t n = (int64_t)d.E * p.MT * p.NT;
    if (p.BN <= kRgPartCols && n < num_sms) {
        // parts of at least 4 blocks of an expert of mean length
        const int64_t fit = num_sms / n, len = rows / 64 / d.E / 4;
        int64_t z = fit < len ? fit : len;
        z = z < kRgMaxParts ? z : kRgMaxParts;
        p.parts = z > 1 ? (int)z : 1;
    }
    p.b_bytes = (p.BN + 63) / 64 * kRgChunk;
    const int fit = kRgRing / 1024 * 1024 / (kRgA + p.b_bytes);
    p.stages = fit < kRgMaxStages ? fit : kRgMaxStages;

    CUtensorMap tx, ty;
    const uint64_t xd[2] = {(uint64_t)K, (uint64_t)rows}, xs[1] = {(uint64_t)ldx};
    const uint64_t yd[2] = {(uint64_t)N, (uint64_t)rows}, ys[1] = {(uint64_t)lddy};
    if (!encode_rows(&tx, x, 2, xd, xs, 64) || !encode_rows(&ty, dy, 2, yd, ys, 64)) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = rg_config(1, st, attr);
    cfg.blockDim = dim3(1024, 1, 1);
    cfg.dynamicSmemBytes = 0;
    cudaError_t err = cudaLaunchKernelEx(&cfg, ragged_segments_kernel, cu, slot_expert, d, ws);
    if (err != cudaSuccess) return err;
    cfg = rg_config(num_sms, st, attr);
    return cudaLaunchKernelEx(&cfg, ragged_dw_kernel, x_wide ? tx : ty, x_wide ? ty : tx, p);
}

}  // namespace bep
