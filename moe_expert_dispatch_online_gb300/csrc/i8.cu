// Experts in 8-bit integers (sm_103a): quantisation of weights, tokens and activations with one
// scale a row (channel), and the grouped product of the integers.
//
//   v = [v_h]: m = max |v|, q_h = round-half-even(127 v_h / m), s = m / 127
//   y[row, n] = (sum_h q[row, h] qw[expert(row), n, h]) * sw[expert, n] * s[row]      (bf16 out)
//
// Layouts. Both operands lie along the reduction, so the weights are transposed when they are
// quantised: row codes [rows, H], row scales [rows] fp32, weight codes [E, H', H], scales [E, H'].

#include <cuda_fp16.h>

#include "mxfmt.cuh"
#include "tiles.cuh"

namespace bep {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------------ format
// A row's grid: values are multiplied by the power of two `up`, which brings the largest to [1, 4) (and far
// smaller ones to 0, which their integer is anyway), then by c = 127 / m: the product is within 2^-22 of 127 v / m.
// Of two bf16 numbers that quotient is a tie k + 1/2 or at least 2^-17 of itself away from one, so its mantissa is
// rounded to 19 bits before it becomes an integer: what was a tie is one again, and nothing else becomes one. (16,384
// tokens of 7168 to 8 rows each: 180 us, 6.5 TB/s; 377 us with IEEE divisions.)
struct Grid {
    float up, c, scale;
};
__device__ __forceinline__ Grid grid_of(uint32_t amax_bits) {
    Grid g;
    if (amax_bits >= 0x7f800000u) {   // an infinity or a NaN: every value of the row is NaN
        g.up = g.c = 0.0f;
        g.scale = __uint_as_float(0x7fc00000u);
        return g;
    }
    const float m = __uint_as_float(amax_bits);
    g.up = __uint_as_float((uint32_t)max(254 - (int)(amax_bits >> 23), 1) << 23);
    g.c = amax_bits ? __fdiv_rn(127.0f, m * g.up) : 0.0f;
    g.scale = __fdiv_rn(m, 127.0f);
    return g;
}
// The integer is in the low byte: adding 1.5 * 2^23 rounds to the nearest one, ties to even. (A row whose values
// are NaN is cleared by its writer.)
__device__ __forceinline__ uint32_t code_of(float v, const Grid& g) {
    const uint32_t q = (__float_as_uint(v * g.up * g.c) + 8u) & 0xfffffff0u;
    return __float_as_uint(__uint_as_float(q) + 12582912.0f);
}
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
__device__ __forceinline__ uint2 codes8(const float* f, const Grid& g) {
    const uint2 r = make_uint2(pack4(code_of(f[0], g), code_of(f[1], g), code_of(f[2], g), code_of(f[3], g)),
                               pack4(code_of(f[4], g), code_of(f[5], g), code_of(f[6], g), code_of(f[7], g)));
    return g.up == 0.0f ? make_uint2(0, 0) : r;
}
// The same of eight fp32 values, whose quotients may lie arbitrarily close to a tie without being one: the fused product
// is within 127 * 2^-23 < kNear of 127 v / m. `off` is the largest distance of a product from its integer so far; from
// 1/2 - kNear on, the writer calls codes8_near_tie instead.
constexpr float kNear = 0x1p-15f, kMagic = 12582912.0f;   // 1.5 * 2^23
__device__ __forceinline__ float off_code(float v, const Grid& g, uint32_t* q) {
    const float s = v * g.up, r = fmaf(s, g.c, kMagic);
    *q = __float_as_uint(r);
    return fmaf(s, g.c, kMagic - r);
}
__device__ __forceinline__ uint2 codes8_f32(const float* f, const Grid& g, float* off) {
    uint32_t q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) *off = fmaxf(*off, fabsf(off_code(f[k], g, &q[k])));
    const uint2 r = make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
    return g.up == 0.0f ? make_uint2(0, 0) : r;
}
// Between j and j + 1, by 254 v against (2 j + 1) m, both exact in fp64 (m: the row's largest magnitude).
__device__ __noinline__ uint2 codes8_near_tie(float4 lo, float4 hi, Grid g, float m) {
    const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float d = off_code(f[k], g, &q[k]);
        if (fabsf(d) > 0.5f - kNear) {
            const int j = (int)(__uint_as_float(q[k]) - kMagic) - (d > 0.0f ? 0 : 1);
            const double x = 254.0 * (double)f[k], t = (double)(2 * j + 1) * (double)m;
            q[k] = (uint32_t)(x > t || (x == t && (j & 1)) ? j + 1 : j);
        }
    }
    return make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
}
// Largest magnitude of eight bf16, as two bf16 bit patterns in a word (NaN above infinity above all).
__device__ __forceinline__ uint32_t top2(const uint4& v) {
    const uint32_t m = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
}
__device__ __forceinline__ uint32_t top_f32(uint32_t two) { return max(two & 0xffffu, two >> 16) << 16; }

// ------------------------------------------------------------------------ weights
// One CTA: 32 columns n of one expert over the whole reduction, twice: the columns' largest magnitudes, then
// their integers, which meet in shared memory, 256 rows h at a time, and leave as runs along h. The CTAs under way hold more
// than L2 where the reduction is long, so w comes from HBM twice: 384 experts of 7168 x 2048, 11.3 GB, 4.18 ms (6.7 TB/s
// with both reads), of 1024 x 7168 1.59 ms.
constexpr int kWCols = 32, kWRows = 256;
__global__ void __launch_bounds__(kThreads) i8_weight_kernel(const uint4* __restrict__ w, int8_t* __restrict__ codes,
                                                             float* __restrict__ scales, int H, int Hp) {
    __shared__ uint32_t s_top[kThreads / 4][kWCols];
    __shared__ Grid s_grid[kWCols];
    __shared__ uint32_t s_codes[kWCols][kWRows / 4 + 1];   // a word more a column: stores of a warp conflict-free
    const int e = blockIdx.y, n0 = blockIdx.x * kWCols;
    const int v = threadIdx.x & 3, r = threadIdx.x >> 2;
    const int pitch = Hp / 8;
    const uint4* src = w + (int64_t)e * H * pitch + n0 / 8 + v;
    uint32_t t[4] = {0, 0, 0, 0};
#pragma unroll 4
    for (int h = r; h < H; h += kThreads / 4) {
        const uint4 x = __ldg(src + (int64_t)h * pitch);
        t[0] = __vmaxu2(t[0], x.x & 0x7fff7fffu);
        t[1] = __vmaxu2(t[1], x.y & 0x7fff7fffu);
        t[2] = __vmaxu2(t[2], x.z & 0x7fff7fffu);
        t[3] = __vmaxu2(t[3], x.w & 0x7fff7fffu);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        s_top[r][8 * v + 2 * j] = t[j] << 16;
        s_top[r][8 * v + 2 * j + 1] = t[j] & 0xffff0000u;
    }
    __syncthreads();
    if (threadIdx.x < kWCols) {
        uint32_t top = 0;
        for (int i = 0; i < kThreads / 4; ++i) top = max(top, s_top[i][threadIdx.x]);
        const Grid g = grid_of(top);
        s_grid[threadIdx.x] = g;
        scales[(int64_t)e * Hp + n0 + threadIdx.x] = g.scale;
    }
    __syncthreads();
    for (int h0 = 0; h0 < H; h0 += kWRows) {
        const int h = h0 + 4 * r;
        if (h < H) {
            float f[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) bf16x8_to_f32(__ldg(src + (int64_t)(h + i) * pitch), f[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const Grid g = s_grid[8 * v + j];
                const uint32_t q = pack4(code_of(f[0][j], g), code_of(f[1][j], g), code_of(f[2][j], g), code_of(f[3][j], g));
                s_codes[8 * v + j][r] = g.up == 0.0f ? 0 : q;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = threadIdx.x; i < kWCols * kWRows / 16; i += kThreads) {
            const int n = i / (kWRows / 16), p = i % (kWRows / 16);
            if (h0 + 16 * p < H) {
                const uint32_t* c = &s_codes[n][4 * p];
                *reinterpret_cast<uint4*>(codes + ((int64_t)e * Hp + n0 + n) * H + h0 + 16 * p) =
                    make_uint4(c[0], c[1], c[2], c[3]);
            }
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------ dispatch
// Largest of a value over the CTA (every thread calls it).
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* s_warp) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (blockDim.x == 32) return v;
    __syncthreads();   // the last row's maxima have been read
    if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31, n = blockDim.x >> 5;
    return __reduce_max_sync(0xffffffffu, lane < n ? s_warp[lane] : 0u);
}

// codes[dest[tok, k]], scales[dest[tok, k]] = i8(x[tok]). A CTA per token: a thread holds kHold pieces of 16
// elements between the two passes over them, and what lies beyond (rows of more than 8192 * kHold) it reads again.
// Bound by HBM: 65,536 tokens of 7168 to 8 rows each, 4.7 GB, 703 us (6.7 TB/s).
constexpr int kDispatchThreads = 512, kHold = 2;   // (1 and 4 measured the same)
__global__ void __launch_bounds__(kDispatchThreads) dispatch_i8_kernel(const uint4* __restrict__ x,
                                                                       const int32_t* __restrict__ dest,
                                                                       uint4* __restrict__ codes,
                                                                       float* __restrict__ scales, int64_t ntok, int K,
                                                                       int pieces, int64_t nrows, int32_t* status) {
    __shared__ uint32_t s_warp[kDispatchThreads / 32];
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    for (int64_t tok = blockIdx.x; tok < ntok; tok += gridDim.x) {
        int dl = 0;
        bool ok = true;
        if (lane < K) {
            dl = dest[tok * K + lane];
            ok = dl >= 0 && (int64_t)dl < nrows;
        }
        const uint4* src = x + tok * pieces * 2;
        uint4 a[kHold], b[kHold];
#pragma unroll
        for (int j = 0; j < kHold; ++j) {
            const int p = threadIdx.x + j * blockDim.x;
            a[j] = b[j] = make_uint4(0, 0, 0, 0);
            if (p < pieces) {
                a[j] = __ldcs(src + 2 * p);
                b[j] = __ldcs(src + 2 * p + 1);
            }
        }
        const unsigned m = __ballot_sync(0xffffffffu, ok);
        if (m != 0xffffffffu && threadIdx.x == 0) set_status(status, BEP_DERR_BOUNDS);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < kHold; ++j) top = __vmaxu2(top, __vmaxu2(top2(a[j]), top2(b[j])));
        for (int p = threadIdx.x + kHold * blockDim.x; p < pieces; p += blockDim.x)
            top = __vmaxu2(top, __vmaxu2(top2(__ldg(src + 2 * p)), top2(__ldg(src + 2 * p + 1))));
        const Grid g = grid_of(block_max(top_f32(top), s_warp));
        if (threadIdx.x < K && ok) scales[dl] = g.scale;
        auto codes16 = [&](const uint4& lo, const uint4& hi) {
            float f[16];
            bf16x8_to_f32(lo, f);
            bf16x8_to_f32(hi, f + 8);
            const uint2 c0 = codes8(f, g), c1 = codes8(f + 8, g);
            return make_uint4(c0.x, c0.y, c1.x, c1.y);
        };
#pragma unroll
        for (int j = 0; j < kHold; ++j) a[j] = codes16(a[j], b[j]);
        for (int k = 0; k < K; ++k) {
            const int64_t row = __shfl_sync(0xffffffffu, dl, k);
            if (!((m >> k) & 1u)) continue;
            uint4* out = codes + row * pieces;
#pragma unroll
            for (int j = 0; j < kHold; ++j) {
                const int p = threadIdx.x + j * blockDim.x;
                if (p < pieces) out[p] = a[j];
            }
        }
        for (int p = threadIdx.x + kHold * blockDim.x; p < pieces; p += blockDim.x) {
            const uint4 c = codes16(__ldg(src + 2 * p), __ldg(src + 2 * p + 1));
            for (int k = 0; k < K; ++k)
                if ((m >> k) & 1u) codes[(int64_t)dest[tok * K + k] * pieces + p] = c;
        }
    }
}

// ------------------------------------------------------------------------ activation
// codes, scales = i8(g * sigmoid(g) * u) for h = [g | u]: kWarps warps a row. The activation stays in fp32
// until its integers; a thread holds 8 * kActHold of its values between the two passes and makes the others
// (rows longer than 8192) again. 524,288 rows of 1024 + 1024, 2.7 GB: 453 us (5.9 TB/s; 497 us with three CTAs an SM
// instead of four), the rest of the copy rate goes to the row's maximum between its loads and its stores.
constexpr int kActHold = 4;
template <int kWarps>
__global__ void __launch_bounds__(kThreads, 4) swiglu_i8_kernel(const uint4* __restrict__ h, uint2* __restrict__ codes,
                                                             float* __restrict__ scales, int64_t rows, int F8) {
    __shared__ uint32_t s_warp[kThreads / 32];
    constexpr int kRowThreads = 32 * kWarps, kRows = kThreads / kRowThreads;
    grid_launch_dependents();
    const int sub = threadIdx.x / kRowThreads, t = threadIdx.x % kRowThreads;
    const int64_t row = (int64_t)blockIdx.x * kRows + sub;
    const bool in = row < rows;
    const uint4* src = h + (in ? row : 0) * 2 * F8;
    const int n = in ? F8 : 0;
    auto act = [&](const uint4& vg, const uint4& vu, float* a) {
        float g[8], u[8];
        bf16x8_to_f32(vg, g);
        bf16x8_to_f32(vu, u);
        gated8(g, u, a);
    };
    uint4 vg[kActHold], vu[kActHold];
#pragma unroll
    for (int j = 0; j < kActHold; ++j) {
        const int c = t + j * kRowThreads;
        vg[j] = vu[j] = make_uint4(0, 0, 0, 0);
        if (c < n) {
            vg[j] = __ldcs(src + c);
            vu[j] = __ldcs(src + F8 + c);
        }
    }
    float a[kActHold][8];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kActHold; ++j) {
        act(vg[j], vu[j], a[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(a[j][i]) & 0x7fffffffu);
    }
    for (int c = t + kActHold * kRowThreads; c < n; c += kRowThreads) {
        float b[8];
        act(__ldg(src + c), __ldg(src + F8 + c), b);
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(b[i]) & 0x7fffffffu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (kWarps > 1) {
        if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top = max(top, s_warp[sub * kWarps + i]);
    }
    const Grid g = grid_of(top);
    if (in && t == 0) scales[row] = g.scale;
    uint2* out = codes + row * F8;
    float off = 0.0f;
    auto exact = [&](const float* v) {
        return codes8_near_tie(make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7]), g, __uint_as_float(top));
    };
#pragma unroll
    for (int j = 0; j < kActHold; ++j) {
        const int c = t + j * kRowThreads;
        if (c < n) out[c] = codes8_f32(a[j], g, &off);
    }
    if (off > 0.5f - kNear)   // one thread in 500
#pragma unroll
        for (int j = 0; j < kActHold; ++j) {
            const int c = t + j * kRowThreads;
            if (c < n) out[c] = exact(a[j]);
        }
    for (int c = t + kActHold * kRowThreads; c < n; c += kRowThreads) {
        float b[8];
        act(__ldg(src + c), __ldg(src + F8 + c), b);
        off = 0.0f;
        out[c] = codes8_f32(b, g, &off);
        if (off > 0.5f - kNear) out[c] = exact(b);
    }
}

// ------------------------------------------------------------------------ product
// This GPU's tensor cores multiply integers at a small fraction of their bf16 rate, so the integers become
// fp16 on the way, which holds them exactly: 1 byte an element in HBM and L2, kind::f16 in the tensor core. Their
// products and the sums below 2^24 are exact in the fp32 accumulator (any sum of 1,040 products; of rows
// as they occur, all of them), larger sums are truncated to fp32 at each step of 16.
// The weights are the M operand, written to TMEM by the warps that convert them, so that shared memory carries
// them once (1 byte) and not three times; the rows of one segment are the N operand (32..256), in shared memory.
// A cluster of two CTAs shares a tile of 256 outputs x N rows (cta_group::2): CTA r holds outputs 128 r.. and
// converts half of the rows.
//   warp 0        TMA: codes of 128 outputs and of half of the rows, 128 reduction steps a stage
//   warp 1        (CTA 0) tcgen05.mma, A from TMEM
//   warps 2-9     weights: two groups of four take the stages in turn; a thread turns one output's 128 codes
//   warps 10-17   rows: two groups of four in turn; a thread turns up to 128 codes
//   warps 18-25   epilogue: TMEM, scaled, to bf16 y
// The kinds of warps only meet at barriers whose signals take about 500 cycles between the CTAs, so the operand
// stages (kSlots) have to cover filling, signalling, multiplying and freeing one.
//   barrier    owner   arrivals
//   wfull[i]   each    the producer's expect_tx + TMA bytes
//   wempty[i]  each    a weight group's and a row group's four warps
//   ready[s]   CTA 0   the same of both CTAs
//   free[s]    both    the MMA thread's multicast commit
//   tfull[a]   both    the MMA thread's multicast commit at the end of a unit
//   tempty[a]  CTA 0   the 8 epilogue warps of each CTA
// Few rows: the weights' stream bounds it (64 rows by 384 experts of 7168 x 2048: 158 us, 5.5 TB/s with its start and
// end). Many: the tensor pipe (80% active), the hand-over of three stages and, in a long run, power (524,288 rows by 7168 x
// 2048: 9.2-9.6 ms, 1.6-1.7 PFLOP/s, of 1.68 that a plain product sustains; 22 ms with two groups of warps that turned weights and rows both, 12 ms with the rows' codes loaded by
// the warps themselves a turn ahead). The conversion (five instructions for four codes) keeps the integer pipe at
// half of its rate; it and the narrow MMAs are what a short reduction with few rows feels (768 rows by 384 experts of
// 1024 x 7168: 439 us, 5.6 TB/s; 402 us without either).
constexpr int kI8K = 128;                       // reduction elements a stage
constexpr int kI8W = 128 * kI8K;                // bytes: 128 outputs' codes
constexpr int kI8EpiWarps = 8;
constexpr int kI8Threads = 32 * (2 + 8 + 8 + kI8EpiWarps);
constexpr int kI8Out = 32 * 256;                // bytes: four epilogue warps' 32 rows x 128 outputs
constexpr int kI8Tmem = 512;
constexpr int kI8Parts = 8;                     // of a unit's reduction at most, each of at least 7 stages

// kRows: rows of a tile at most. Fewer rows leave room for more stages under way.
template <int kRows>
struct I8Cfg {
    static constexpr int kAcc = kRows < 128 ? kRows : 128;     // TMEM columns of an accumulator, of which there are two
    static constexpr int kSlots = kRows <= 64 ? 6 : kRows <= 128 ? 4 : 3;   // stages of fp16 operands
    static constexpr int kRing = kRows <= 64 ? 8 : kRows <= 128 ? 6 : 3;    // stages of codes under way
    static constexpr int kStage = kI8W + kRows / 2 * kI8K;     // bytes: outputs' codes, half of the rows' codes
    static constexpr int kB = kRows / 2 * kI8K * 2;            // bytes: half of the rows in fp16
    static constexpr int kSub = kB / 2;                        // 64 reduction steps of them
    static constexpr int kABase = 2 * kAcc, kACols = kI8K / 2;
    static constexpr size_t kSmem = 1024 + (size_t)kRing * kStage + (size_t)kSlots * kB + kI8EpiWarps / 4 * kI8Out + kRows * 4 +
                                    (2 * kRing + 2 * kSlots + 5) * 8 + 16;
    static_assert(kABase + kSlots * kACols <= kI8Tmem, "TMEM");
    static_assert(kSlots >= 2 && kRing >= 2, "two groups of warps take turns: neither may step past the end");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct I8Params {
    const MTile* tiles;
    const int32_t* ntiles;
    const int32_t* slot_expert;
    const float* scales;
    const float* w_scales;
    uint16_t* y;
    int64_t nrows;
    int E, H, Hp, MT;
    int32_t* tickets;
    float* partial;
    int32_t* status;
};

// Work of a pair of CTAs: whole units, or, in the form for so few units that most pairs would have none, a unit's part
// z of the reduction's stages. A part leaves its fp32 sums in the workspace, and the CTA of each rank that comes last
// adds them in order (one token through two experts of 7168 x 512, four units: 26.8 us whole, 13.3 us in eight parts).
struct I8Geo {
    int items, z, nst;
};
struct I8Item : Unit {
    int unit, part, k0, k1;   // (parts only) stages of the reduction
};
template <bool kSplit>
struct I8Walk {
    UnitWalk w;
    int item;
    __device__ __forceinline__ I8Walk(int first, int ncl, int MP) : w(first, ncl, MP), item(first) {}
    __device__ __forceinline__ I8Item take(const I8Params& p, const I8Geo& g) {
        I8Item u;
        u.k0 = 0;
        u.k1 = g.nst;
        if (!kSplit) {
            static_cast<Unit&>(u) = w.take(p, g.items);
        } else {
            u.unit = item / g.z;
            u.part = item - u.unit * g.z;
            UnitWalk one(u.unit, w.ncl, w.MP);
            static_cast<Unit&>(u) = one.take(p, g.items / g.z);
            u.k0 = u.part * g.nst / g.z;
            u.k1 = (u.part + 1) * g.nst / g.z;
            item += w.ncl;
        }
        return u;
    }
};

// 32 columns of this warp's 32 TMEM lanes, and the wait for them, where a vote has brought the warp together and nothing
// since has branched. (A __syncwarp in front of each: 32,768 rows, 384 experts of 1024 x 7168 661 us instead of 636, of
// 7168 x 2048 1090 instead of 1061.)
__device__ __forceinline__ void tmem_wait_st_converged() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_32x32b_x32_converged(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// Instruction descriptor, kind::f16: fp32 accumulator, fp16 A and B (0), both K-major, M = 256.
__device__ __forceinline__ uint32_t idesc_f16(int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | (16u << 24);
}

// D (+)= A B^T over 16 reduction steps: A in TMEM (each CTA its own 128 outputs), B in shared memory (each CTA
// half of the rows).
__device__ __forceinline__ void mma_f16_pair_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(add)
        : "memory");
}

// All eight epilogue warps.
__device__ __forceinline__ bool octet_all(bool v) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, 3, 256, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

// Four int8 to four fp16, as weight-only quantisation is known to do it: the byte with its sign bit turned, behind 0x64, is
// 1024 + 128 + q in fp16.
__device__ __forceinline__ void i8x4_to_f16(uint32_t w, uint32_t* out) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half((unsigned short)0x6480));   // 1152
    const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), off);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), off);
    out[0] = *reinterpret_cast<const uint32_t*>(&a);
    out[1] = *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void i8x16_to_f16(const uint4& v, uint32_t* out) {
    i8x4_to_f16(v.x, out);
    i8x4_to_f16(v.y, out + 2);
    i8x4_to_f16(v.z, out + 4);
    i8x4_to_f16(v.w, out + 6);
}

template <int kRows, bool kSplit>
__global__ void __launch_bounds__(kI8Threads, 1) grouped_gemm_i8_kernel(
    const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX16,
    const __grid_constant__ CUtensorMap tmX32, const __grid_constant__ CUtensorMap tmX64,
    const __grid_constant__ CUtensorMap tmX128, const I8Params p) {
    using C = I8Cfg<kRows>;
    constexpr int kRing = C::kRing, kSlots = C::kSlots;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t* smW = smem;
    uint8_t* smB = smW + kRing * C::kStage;
    uint8_t* smO = smB + kSlots * C::kB;
    float* smC = reinterpret_cast<float*>(smO + kI8EpiWarps / 4 * kI8Out);   // rows' scales of a unit
    uint64_t* wfull = reinterpret_cast<uint64_t*>(smC + kRows);
    uint64_t* wempty = wfull + kRing;
    uint64_t* ready = wempty + kRing;
    uint64_t* free_ = ready + kSlots;
    uint64_t* tfull = free_ + kSlots;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    int* s_last = reinterpret_cast<int*>(s_tmem + 2);
    int32_t* status = p.status;
    const uint32_t rank = cluster_rank();
    const bool lead = rank == 0;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 32) {
        const CUtensorMap* maps[] = {&tmW, &tmX16, &tmX32, &tmX64, &tmX128};
        for (const CUtensorMap* m : maps)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&wfull[i], 1);
            mbar_init(&wempty[i], 8);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&ready[s], 16);
            mbar_init(&free_[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 2 * kI8EpiWarps);
        }
        mbar_init(drain, 1);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                     "r"(kI8Tmem)
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
    const int cl0 = (int)cluster_id(), ncl = (int)cluster_count();
    I8Geo geo{*p.ntiles * MP, 1, (p.H + kI8K - 1) / kI8K};
    if (kSplit && geo.items > 0) {
        static_assert(!kSplit || kRows <= kRgPartCols, "a part's tile");
        geo.z = max(1, min(min(ncl / geo.items, geo.nst / 7), kI8Parts));
        geo.items *= geo.z;
    }
    const int total = geo.items;
    uint32_t pr_i = 0, pr_ph = 0, pr_armed = 0;

    if (warp == 0) {
        if (lane == 0) {
            bool live = true;
            I8Walk<kSplit> walk(cl0, ncl, MP);
            I8Item next = walk.take(p, geo);   // read a unit ahead
            for (int unit = cl0; unit < total && live; unit += ncl) {
                const I8Item u = next;
                next = walk.take(p, geo);
                if (u.expert < 0) {
                    if (lead) set_status(status, BEP_DERR_BOUNDS);
                    continue;
                }
                const int mt = 2 * u.mp + (int)rank;   // past H' for the last odd tile: zeros
                const int half = mma_rows(u.rows) / 2, row = u.row0 + (int)rank * half;
                const CUtensorMap* tmX = half <= 16 ? &tmX16 : half <= 32 ? &tmX32 : half <= 64 ? &tmX64 : &tmX128;
                const int bytes = kI8W + (half <= 16 ? 16 : half <= 32 ? 32 : half <= 64 ? 64 : 128) * kI8K;
                for (int k = u.k0; k < u.k1; ++k) {
                    if (!mbar_wait_held(&wempty[pr_i], pr_ph ^ 1u, s_abort, status)) {
                        live = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&wfull[pr_i], bytes);
                    ++pr_armed;
                    uint8_t* stage = smW + pr_i * C::kStage;
                    tma_load_3d(&tmW, &wfull[pr_i], stage, k * kI8K, mt * 128, u.expert);
                    tma_load_2d(tmX, &wfull[pr_i], stage + kI8W, k * kI8K, row);
                    if (++pr_i == kRing) {
                        pr_i = 0;
                        pr_ph ^= 1u;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lead && elect_one()) {
            uint32_t s = 0, ph = 0;   // operand slot
            uint32_t half = 0;        // accumulator of the next unit of up to 128 rows
            uint32_t aph[2] = {1, 1};   // the phases that free the accumulators
            bool live = true;
            I8Walk<kSplit> walk(cl0, ncl, MP);
            I8Item next = walk.take(p, geo);
            for (int unit = cl0; unit < total && live; unit += ncl) {
                const I8Item u = next;
                next = walk.take(p, geo);
                if (u.expert < 0) continue;
                const int N = mma_rows(u.rows);
                const bool big = N > C::kAcc;
                if (big) half = 0;
                if (!mbar_wait_held<true>(&tempty[half], aph[half], s_abort, status)) break;
                if (big && !mbar_wait_held<true>(&tempty[1], aph[1], s_abort, status)) break;
                aph[half] ^= 1u;
                if (big) aph[1] ^= 1u;
                const uint32_t dt = tmem_base + half * C::kAcc;
                const uint32_t idesc = idesc_f16(N);
                for (int k = u.k0; k < u.k1; ++k) {
                    if (!mbar_wait_held<true>(&ready[s], ph, s_abort, status)) {
                        live = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = tmem_base + C::kABase + s * C::kACols;
                    const uint32_t b = smem_u32(smB + s * C::kB);
                    const int steps = min(kI8K, p.H - k * kI8K) / 16;   // 4 or 8
#pragma unroll
                    for (int kk = 0; kk < kI8K / 16; ++kk)
                        if (kk < steps)
                            mma_f16_pair_ts(dt, a + kk * 8, sdesc_sw128(b + (kk >> 2) * C::kSub + (kk & 3) * 32, 16, 1024),
                                            idesc, k != u.k0 || kk != 0);
                    mma_commit_pair(&free_[s]);
                    if (k == u.k1 - 1) {
                        mma_commit_pair(&tfull[half]);
                        if (big) mma_commit_pair(&tfull[1]);
                    }
                    if (++s == kSlots) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!big) half ^= 1u;
            }
        }
    } else if (warp < 10) {
        const int group = (warp - 2) >> 2, quarter = warp & 3;   // four consecutive warps: each quarter of TMEM's lanes once
        const int n = quarter * 32 + lane;                       // output of this thread, lane of TMEM
        uint32_t i = group, iph = 0, s = group, sph = 0;         // ring stage and operand slot of this turn
        int turn = 0;
        bool live = true;
        I8Walk<kSplit> walk(cl0, ncl, MP);
        for (int unit = cl0; unit < total && live; unit += ncl) {
            const I8Item u = walk.take(p, geo);
            if (u.expert < 0) continue;
            for (int k = u.k0; k < u.k1; ++k, turn ^= 1) {
                if (turn != group) continue;
                if (!__all_sync(0xffffffffu, mbar_wait_held(&free_[s], sph ^ 1u, s_abort, status)) ||
                    !__all_sync(0xffffffffu, mbar_wait_held(&wfull[i], iph, s_abort, status))) {
                    live = false;
                    break;
                }
                const uint8_t* wrow = smW + i * C::kStage + n * 128;
                const uint32_t ta = tmem_base + ((uint32_t)(quarter * 32) << 16) + C::kABase + s * C::kACols;
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t f[32];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        i8x16_to_f16(*reinterpret_cast<const uint4*>(wrow + (((4 * q + j) ^ (n & 7)) << 4)), f + 8 * j);
                    tmem_st_32x32b_x32_converged(ta + 32 * q, f);
                }
                tmem_wait_st_converged();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&wempty[i]);
                    mbar_arrive_rank_shared(&ready[s], 0);
                }
                i += 2;
                if (i >= kRing) {
                    i -= kRing;
                    iph ^= 1u;
                }
                s += 2;
                if (s >= kSlots) {
                    s -= kSlots;
                    sph ^= 1u;
                }
            }
        }
    } else if (warp < 18) {
        const int group = (warp - 10) >> 2;
        // 4 lanes take 64 bytes of a row, a warp 8 rows and the group 32 at a time. Eight lanes in a run take rows r and
        // r ^ 5, whose swizzled pieces of 16 bytes lie in different banks in the codes and in the fp16 both.
        const int run = lane >> 2, piece = lane & 3;
        const int r = ((warp - 10) & 3) * 8 + ((run >> 1) ^ ((run & 1) * 5)), x = r & 7;
        const int from = kI8W + r * 128, to = r * 128;
        const int f0 = (piece ^ x) << 4, f1 = f0 ^ 64;                                // pieces of 16 codes
        const int t0 = ((2 * piece) ^ x) << 4, t1 = t0 ^ 16;                          // pieces of 8 fp16
        uint32_t i = group, iph = 0, s = group, sph = 0;   // ring stage and operand slot of this turn
        int turn = 0;
        bool live = true;
        I8Walk<kSplit> walk(cl0, ncl, MP);
        for (int unit = cl0; unit < total && live; unit += ncl) {
            const I8Item u = walk.take(p, geo);
            if (u.expert < 0) continue;
            const int half = mma_rows(u.rows) / 2;
            for (int k = u.k0; k < u.k1; ++k, turn ^= 1) {
                if (turn != group) continue;
                if (!__all_sync(0xffffffffu, mbar_wait_held(&free_[s], sph ^ 1u, s_abort, status)) ||
                    !__all_sync(0xffffffffu, mbar_wait_held(&wfull[i], iph, s_abort, status))) {
                    live = false;
                    break;
                }
                // 16 codes become two 16-byte pieces of a row of 64 fp16 (128-byte swizzle)
                const uint8_t* codes = smW + i * C::kStage + from;
                uint8_t* slot = smB + s * C::kB + to;
#pragma unroll
                for (int j = 0; j < (kRows / 2 + 31) / 32; ++j)
                    if (32 * j + r < half) {
                        const uint4 c0 = *reinterpret_cast<const uint4*>(codes + j * 4096 + f0);
                        const uint4 c1 = *reinterpret_cast<const uint4*>(codes + j * 4096 + f1);
                        uint32_t f[8];
                        i8x16_to_f16(c0, f);
                        *reinterpret_cast<uint4*>(slot + j * 4096 + t0) = make_uint4(f[0], f[1], f[2], f[3]);
                        *reinterpret_cast<uint4*>(slot + j * 4096 + t1) = make_uint4(f[4], f[5], f[6], f[7]);
                        i8x16_to_f16(c1, f);
                        *reinterpret_cast<uint4*>(slot + C::kSub + j * 4096 + t0) = make_uint4(f[0], f[1], f[2], f[3]);
                        *reinterpret_cast<uint4*>(slot + C::kSub + j * 4096 + t1) = make_uint4(f[4], f[5], f[6], f[7]);
                    }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&wempty[i]);
                    mbar_arrive_rank_shared(&ready[s], 0);
                }
                i += 2;
                if (i >= kRing) {
                    i -= kRing;
                    iph ^= 1u;
                }
                s += 2;
                if (s >= kSlots) {
                    s -= kSlots;
                    sph ^= 1u;
                }
            }
        }
    } else {
        // Four warps, one for each quarter of TMEM's lanes, own every second run of 32 rows. A lane holds one output
        // of 32 rows, and a row's outputs lie together in y, so the run is turned in shared memory, as words of two
        // rows, and leaves as whole rows of 256 bytes, 16 a lane. The rows' scales come from shared memory, four
        // to a load: the loads and stores of the warps that convert are what the epilogue competes with.
        const int quarter = warp & 3, second = (warp - 18) >> 2;
        uint8_t* stg = smO + second * kI8Out;
        float* sc = smC + second * (kRows / 2);
        uint32_t half = 0, tph[2] = {0, 0};
        I8Walk<kSplit> walk(cl0, ncl, MP);
        I8Item next = walk.take(p, geo);
        for (int unit = cl0; unit < total; unit += ncl) {
            const I8Item u = next;
            next = walk.take(p, geo);
            if (u.expert < 0) continue;
            const bool big = mma_rows(u.rows) > C::kAcc;
            if (big) half = 0;
            const int n0 = (2 * u.mp + (int)rank) * 128;
            const int n = n0 + quarter * 32 + lane;
            const float ws = n < p.Hp ? p.w_scales[(int64_t)u.expert * p.Hp + n] : 0.0f;
            // run `quarter` of this half's: the four warps have read the last unit's (a row behind the segment's
            // last is never stored)
            const int64_t srow = (int64_t)u.row0 + 32 * second + 64 * quarter + lane;
            if (64 * quarter < kRows) sc[32 * quarter + lane] = p.scales[i64min(srow, p.nrows - 1)];
            // one warp waits and the others for it at their barrier; the four give up together
            bool done = quarter != 0 || mbar_wait_held(&tfull[half], tph[half], s_abort, status);
            if (big && quarter == 0 && done) done = mbar_wait_held(&tfull[1], tph[1], s_abort, status);
            // (all eight warps together where they will meet)
            if (kSplit ? !octet_all(done) : !quad_all(1 + second, done)) break;
            tph[half] ^= 1u;
            if (big) tph[1] ^= 1u;
            tc_fence_after();
            const uint32_t tacc = tmem_base + ((uint32_t)(quarter * 32) << 16) + half * C::kAcc;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_rank_relaxed(&tempty[half], 0);
                    if (big) mbar_arrive_rank_relaxed(&tempty[1], 0);
                }
            };
            bool held = true, last = true;
            const int lane0 = quarter * 32 + lane;   // output of the tile
            if (kSplit && geo.z > 1) {
                float* out = p.partial + (int64_t)(2 * unit + (int)rank) * (kRgPartCols * 128) + lane0;
                for (int c0 = 32 * second; c0 < u.rows; c0 += 64) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tacc + c0, r);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c0 + j < u.rows) __stcg(out + (c0 + j) * 128, __uint_as_float(r[j]));
                }
                release();
                held = false;
                __threadfence();
                octet_all(true);
                if (quarter == 0 && second == 0 && lane == 0) {
                    int32_t* ticket = p.tickets + 2 * u.unit + (int)rank;
                    const int n = atomicAdd(ticket, 1);
                    __threadfence();
                    *s_last = n == geo.z - 1;
                    if (n == geo.z - 1) *ticket = 0;   // for the next call
                }
                octet_all(true);
                last = *s_last != 0;   // (no pair has two parts: written once a launch)
            }
            for (int c0 = 32 * second; last && c0 < u.rows; c0 += 64) {
                uint32_t r[32];
                if (kSplit && geo.z > 1) {
                    const float* in = p.partial + (int64_t)(2 * u.unit * geo.z + (int)rank) * (kRgPartCols * 128) + lane0;
                    // four rows of all parts at a time
#pragma unroll
                    for (int j0 = 0; j0 < 32; j0 += 4) {
                        float v[4][kI8Parts];
                        if (c0 + j0 >= u.rows) break;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int z = 0; z < kI8Parts; ++z)
                                v[j][z] = z < geo.z && c0 + j0 + j < u.rows
                                              ? __ldcg(in + (int64_t)2 * z * (kRgPartCols * 128) + (c0 + j0 + j) * 128)
                                              : 0.0f;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float sum = v[j][0];
#pragma unroll
                            for (int z = 1; z < kI8Parts; ++z) sum += v[j][z];
                            r[j0 + j] = __float_as_uint(sum);
                        }
                    }
                } else {
                    tmem_ld_32x32b_x32(tacc + c0, r);
                }
                if (held && c0 + 64 >= u.rows) {   // this warp has read all its runs: free them before the stores
                    release();
                    held = false;
                }
                const float4* s4 = reinterpret_cast<const float4*>(sc + (c0 >> 6) * 32);
                uint32_t two[16];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 f = s4[j];
                    two[2 * j] = pack_bf16x2(__uint_as_float(r[4 * j]) * ws * f.x, __uint_as_float(r[4 * j + 1]) * ws * f.y);
                    two[2 * j + 1] =
                        pack_bf16x2(__uint_as_float(r[4 * j + 2]) * ws * f.z, __uint_as_float(r[4 * j + 3]) * ws * f.w);
                }
                quad_sync(1 + second);   // the run before has been read, and this one's scales
                uint32_t* col = reinterpret_cast<uint32_t*>(stg) + quarter * 32 + lane;
#pragma unroll
                for (int j = 0; j < 16; ++j) col[j * 128] = two[j];
                quad_sync(1 + second);   // the run is staged
                // rows 2 j and 2 j + 1, j = 4 quarter + 2 i + (lane / 16): eight outputs a lane
                const int j0 = quarter * 4 + (lane >> 4), no = n0 + (lane & 15) * 8;
                const uint4* pc = reinterpret_cast<const uint4*>(stg) + j0 * 32 + (lane & 15) * 2;
                uint16_t* out = p.y + ((int64_t)u.row0 + c0 + 2 * j0) * p.Hp + no;
                const int rest = no < p.Hp ? u.rows - c0 - 2 * j0 : 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 a = pc[64 * i], b = pc[64 * i + 1];
                    if (4 * i < rest)
                        *reinterpret_cast<uint4*>(out + (int64_t)(4 * i) * p.Hp) =
                            make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                                       __byte_perm(b.x, b.y, 0x5410), __byte_perm(b.z, b.w, 0x5410));
                    if (4 * i + 1 < rest)
                        *reinterpret_cast<uint4*>(out + (int64_t)(4 * i + 1) * p.Hp) =
                            make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                                       __byte_perm(b.x, b.y, 0x7632), __byte_perm(b.z, b.w, 0x7632));
                }
            }
            if (held) release();
            if (!big) half ^= 1u;
        }
    }

    __syncthreads();
    if (*s_abort) {
        // A wait gave up: what was started lands before shared memory and TMEM are released, each wait bounded.
        if (warp == 0 && lane == 0) {
            for (uint32_t i = 0; i < pr_armed && i < (uint32_t)kRing; ++i) {
                if (pr_i == 0) {
                    pr_i = kRing;
                    pr_ph ^= 1u;
                }
                --pr_i;
                mbar_drain(&wfull[pr_i], pr_ph);
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
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kI8Tmem)
                     : "memory");
    }
}

template <int kRows>
cudaLaunchConfig_t i8_config(int clusters, cudaStream_t st, cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * clusters, 1, 1);
    cfg.blockDim = dim3(kI8Threads, 1, 1);
    cfg.dynamicSmemBytes = I8Cfg<kRows>::kSmem;
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

template <int kRows, bool kSplit>
cudaError_t i8_attributes() {
    return cudaFuncSetAttribute(grouped_gemm_i8_kernel<kRows, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)I8Cfg<kRows>::kSmem);
}

template <int kRows, bool kSplit = false>
cudaError_t run_gemm_i8(const Dims& d, const Workspace& ws, const int32_t* cu, const CUtensorMap& tmW, const CUtensorMap* tmX,
                        const I8Params& p,
                        int clusters, cudaStream_t st) {
    const cudaError_t err = launch_row_tiles<kRows>(d, ws, cu, st);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = i8_config<kRows>(clusters, st, attr);
    return cudaLaunchKernelEx(&cfg, grouped_gemm_i8_kernel<kRows, kSplit>, tmW, tmX[0], tmX[1], tmX[2], tmX[3], p);
}

template <int kWarps>
void run_swiglu_i8(int64_t rows, int F8, const uint4* h, uint2* codes, float* scales, cudaStream_t st) {
    constexpr int kRows = 8 / kWarps;
    swiglu_i8_kernel<kWarps><<<(unsigned)((rows + kRows - 1) / kRows), kThreads, 0, st>>>(h, codes, scales, rows, F8);
}

}  // namespace

// *clusters: pairs of CTAs that can be resident at once (an SM holds one CTA of any kind): the grid of the product.
cudaError_t i8_setup(int device, int* clusters) {
    cudaError_t err = i8_attributes<64, true>();
    if (err == cudaSuccess) err = i8_attributes<64, false>();
    if (err == cudaSuccess) err = i8_attributes<128, false>();
    if (err == cudaSuccess) err = i8_attributes<256, false>();
    if (err != cudaSuccess) return err;
    int nsm = 0;
    err = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, device);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = i8_config<256>(nsm / 2, nullptr, attr);
    return cudaOccupancyMaxActiveClusters(clusters, grouped_gemm_i8_kernel<256, false>, &cfg);
}

cudaError_t launch_i8_weight(const Dims& d, const uint16_t* w, int8_t* codes, float* scales, cudaStream_t st) {
    const dim3 grid((unsigned)(d.Hp / kWCols), (unsigned)d.E);
    i8_weight_kernel<<<grid, kThreads, 0, st>>>(reinterpret_cast<const uint4*>(w), codes, scales, d.H, d.Hp);
    return cudaGetLastError();
}

cudaError_t launch_dispatch_i8(const Dims& d, const Workspace& ws, const uint16_t* x, const int32_t* dest,
                               int8_t* codes, float* scales, int sms, int num_sms, cudaStream_t st) {
    const int64_t ntok = (int64_t)d.R * d.S;
    const int pieces = d.H / 16;
    const int want = (pieces + kHold - 1) / kHold;
    const int threads = want < kDispatchThreads ? (want + 31) / 32 * 32 : kDispatchThreads;
    // every token its own CTA, or, under an SM budget, what that many SMs hold
    const int64_t cap = sms < num_sms ? (int64_t)sms * (2048 / threads < 32 ? 2048 / threads : 32) : (int64_t)INT32_MAX;
    dispatch_i8_kernel<<<(unsigned)(ntok < cap ? ntok : cap), threads, 0, st>>>(
        reinterpret_cast<const uint4*>(x), dest, reinterpret_cast<uint4*>(codes), scales, ntok, d.K, pieces,
        (int64_t)d.R * d.C, ws.status);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_i8(int64_t rows, int F, const uint16_t* h, int8_t* codes, float* scales, int num_sms,
                             cudaStream_t st) {
    const int F8 = F / 8;
    const uint4* hp = reinterpret_cast<const uint4*>(h);
    uint2* cp = reinterpret_cast<uint2*>(codes);
    // as few warps a row as hold it (kActHold * 256 elements each), so that small rows share a CTA; more where
    // the rows alone would leave SMs idle
    int warps = 1;
    while (warps < 8 && (F8 > warps * 32 * kActHold || (rows * warps < num_sms * 16 && F8 > warps * 32))) warps *= 2;
    switch (warps) {
        case 1: run_swiglu_i8<1>(rows, F8, hp, cp, scales, st); break;
        case 2: run_swiglu_i8<2>(rows, F8, hp, cp, scales, st); break;
        case 4: run_swiglu_i8<4>(rows, F8, hp, cp, scales, st); break;
        default: run_swiglu_i8<8>(rows, F8, hp, cp, scales, st); break;
    }
    return cudaGetLastError();
}

cudaError_t launch_grouped_gemm_i8(const Dims& d, const Workspace& ws, const int32_t* cu, const int32_t* slot_expert,
                                   const int8_t* codes, const float* scales, const int8_t* w_codes,
                                   const float* w_scales, uint16_t* y, int clusters, cudaStream_t st) {
    I8Params p;
    p.tiles = ws.tiles;
    p.ntiles = ws.ntiles;
    p.slot_expert = slot_expert;
    p.scales = scales;
    p.w_scales = w_scales;
    p.y = y;
    p.nrows = (int64_t)d.R * d.C;
    p.E = d.E;
    p.H = d.H;
    p.Hp = d.Hp;
    p.MT = (d.Hp + 127) / 128;
    p.tickets = ws.tickets;
    p.partial = ws.partial;
    p.status = ws.status;
    const uint64_t wd[3] = {(uint64_t)d.H, (uint64_t)d.Hp, (uint64_t)d.E};
    const uint64_t xd[2] = {(uint64_t)d.H, (uint64_t)d.R * d.C};
    const uint32_t boxes[4] = {16, 32, 64, 128};
    CUtensorMap tmW, tmX[4];
    if (!encode_u8(&tmW, w_codes, 3, wd, 128)) return cudaErrorInvalidValue;
    for (int i = 0; i < 4; ++i)
        if (!encode_u8(&tmX[i], codes, 2, xd, boxes[i])) return cudaErrorInvalidValue;
    // Rows a tile by the mean segment: a tile of fewer rows leaves room for more weight codes under way, but a second tile of
    // a segment reads the weights again. (96 experts of 7168 x 2048, segments of half to one and a half of the mean: 40 rows
    // 254 us with tiles of 64, 256 with 128; 48 279 and 260; 96 298 with 128, 330 with 256; 112 345 and 323.)
    const int64_t mean = p.nrows / d.E;
    // Every row a tile of its own, at most: units for less than half of the pairs. (Below 14 stages there is one part, and
    // the form without parts is 1.4 us quicker.)
    if (p.nrows <= 64 && p.nrows * ((p.MT + 1) / 2) * 2 <= clusters && d.H >= 14 * kI8K)
        return run_gemm_i8<64, true>(d, ws, cu, tmW, tmX, p, clusters, st);
    if (mean <= 40) return run_gemm_i8<64>(d, ws, cu, tmW, tmX, p, clusters, st);
    if (mean <= 96) return run_gemm_i8<128>(d, ws, cu, tmW, tmX, p, clusters, st);
    return run_gemm_i8<256>(d, ws, cu, tmW, tmX, p, clusters, st);
}

}  // namespace bep
