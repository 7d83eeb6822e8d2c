// Gated activation between an expert's two projections (sm_103a), and its backward from an
// 8-bit checkpoint.
//
//   h = [g | u], bf16 [rows, 2F];  a = g * sigmoid(g) * u                    (bf16 out)
//   checkpoint: h in int8 with a power-of-two scale per 32 elements (mxfmt.cuh)
//   backward, with g^, u^ the checkpoint's values and s = sigmoid(g^):
//     dg = da * u^ * s * (1 + g^ (1 - s)),  du = da * g^ * s,  a^ = g^ * s * u^
// All arithmetic is fp32 with one rounding at the end of each output.
//
// Element-wise over rows, so bound by HBM: forward 4F + 2F + 2F (1 + 1/32) bytes a row,
// backward 2F (1 + 1/32) + 2F + 4F + 2F. A thread owns 8 columns of both halves (16-byte
// loads and stores of bf16, 8-byte of int8); the 4 threads of a block of 32 find its largest
// magnitude with two shuffles.

#include "mxfmt.cuh"

namespace bep {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack8(const float* f) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// Quantises this thread's 8 of a block's 32 values; the scale byte is the block's.
__device__ __forceinline__ uint2 quantise8(const float* f, uint32_t* byte) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(f[i]) & 0x7fffffffu);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    *byte = mx8_scale_byte(amax);
    if (*byte == kMxNan) return make_uint2(0, 0);
    const float inv = mx_inverse(*byte);
    return make_uint2(pack_int8x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                      pack_int8x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

// One pass, no loop: a CTA takes kU runs of 256 consecutive vectors, all of whose loads are in
// flight at once, and the CTAs follow one another through memory. A grid that strides over the
// rows instead reaches 87-93% of the copy rate; this reaches 101-104%.
// 524,288 rows of 1024 + 1024 (4.33 GB, 5.40 GB): forward 625 us, 746 with the striding grid; backward 803 us.
// n: vectors of 8 columns in all rows (rows * F / 8, a multiple of 4, below 2^31).
template <bool kSave, int kU>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const uint4* __restrict__ h,
                                                          uint4* __restrict__ a,
                                                          uint2* __restrict__ codes,
                                                          uint8_t* __restrict__ scales, uint32_t n,
                                                          FastDiv cols) {
    const uint32_t i0 = blockIdx.x * (kThreads * kU) + threadIdx.x;
    uint4 vg[kU], vu[kU];
    uint64_t at[kU];   // gate vector; the up vector is cols.d on
    uint32_t c[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
        const uint32_t i = i0 + j * kThreads;
        vg[j] = vu[j] = make_uint4(0, 0, 0, 0);   // past the end: whole warps stay for the shuffles
        const uint32_t row = fast_div(i < n ? i : 0, cols);
        c[j] = i - row * cols.d;
        at[j] = (uint64_t)row * (2 * cols.d) + c[j];
        if (i < n) {
            vg[j] = __ldcs(h + at[j]);
            vu[j] = __ldcs(h + at[j] + cols.d);
        }
    }
#pragma unroll
    for (int j = 0; j < kU; ++j) {
        const uint32_t i = i0 + j * kThreads;
        const bool in = i < n;
        float g[8], u[8];
        bf16x8_to_f32(vg[j], g);
        bf16x8_to_f32(vu[j], u);
        if (kSave) {
            uint32_t bg, bu;
            const uint2 qg = quantise8(g, &bg), qu = quantise8(u, &bu);
            if (in) {
                __stcs(codes + at[j], qg);
                __stcs(codes + at[j] + cols.d, qu);
                if ((c[j] & 3u) == 0) {
                    scales[at[j] >> 2] = (uint8_t)bg;
                    scales[(at[j] + cols.d) >> 2] = (uint8_t)bu;
                }
            }
        }
        float o[8];
        gated8(g, u, o);
        if (in) __stcs(a + i, pack8(o));
    }
}

// One vector a thread: two or more in flight measured no faster here.
__global__ void __launch_bounds__(kThreads) swiglu_bwd_kernel(const uint4* __restrict__ da,
                                                              const uint2* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales,
                                                              uint4* __restrict__ dh,
                                                              uint4* __restrict__ a, uint32_t n,
                                                              FastDiv cols) {
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const uint32_t row = fast_div(i, cols);
    const uint64_t at = (uint64_t)row * (2 * cols.d) + (i - row * cols.d);
    const uint2 qg = __ldcs(codes + at), qu = __ldcs(codes + at + cols.d);
    const float sg = mx_scale(scales[at >> 2]), su = mx_scale(scales[(at + cols.d) >> 2]);
    float d[8], og[8], ou[8], oa[8];
    bf16x8_to_f32(__ldcs(da + i), d);
    asm volatile("" ::"r"(qg.x), "r"(qu.x), "f"(d[0]));   // all loads before the branch
    // Codes are 127 at most: with a scale of 1/2 or less no gate of the block lies beyond 63.5. A tiny one is
    // left to a loop that reads its elements again, so that the rare case costs the other one no registers
    // (524,288 rows of 1024 + 1024, side by side: 807 us; both forms unrolled 836 us; the common one alone 798 us).
    if (sg > 0.5f) {
        float low = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) low = fminf(low, int8_at(k < 4 ? qg.x : qg.y, k & 3));
        if (low * sg < kTinyGate) {
            const int8_t* g8 = reinterpret_cast<const int8_t*>(codes + at);
            const int8_t* u8 = reinterpret_cast<const int8_t*>(codes + at + cols.d);
            const __nv_bfloat16* d16 = reinterpret_cast<const __nv_bfloat16*>(da + i);
            __nv_bfloat16* og16 = reinterpret_cast<__nv_bfloat16*>(dh + at);
            __nv_bfloat16* ou16 = reinterpret_cast<__nv_bfloat16*>(dh + at + cols.d);
            __nv_bfloat16* oa16 = reinterpret_cast<__nv_bfloat16*>(a + i);
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
                const float g = (float)g8[k] * sg, u = (float)u8[k] * su, dk = __bfloat162float(d16[k]);
                const Gate s = gate_of(g);
                const float rest = g < 0.0f ? s.r : s.e * s.r;   // 1 - sigmoid(g)
                og16[k] = __float2bfloat16_rn(dk * u * s.m * s.m * (s.r * fmaf(g, rest, 1.0f)));
                ou16[k] = __float2bfloat16_rn(gated(g, s, dk));
                if (a) oa16[k] = __float2bfloat16_rn(gated(g, s, u));
            }
            return;
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float g = int8_at(k < 4 ? qg.x : qg.y, k & 3) * sg;
        const float u = int8_at(k < 4 ? qu.x : qu.y, k & 3) * su;
        const float s = hw_sigmoid(g);
        const float gs = g * s;
        og[k] = d[k] * u * (s + gs * (1.0f - s));
        ou[k] = d[k] * gs;
        oa[k] = gs * u;
    }
    __stcs(dh + at, pack8(og));
    __stcs(dh + at + cols.d, pack8(ou));
    if (a) __stcs(a + i, pack8(oa));
}

// Rows are taken in slabs of fewer than 2^31 vectors, so that positions fit 32 bits.
template <typename F>
cudaError_t by_slabs(int64_t rows, int F8, F&& launch) {
    const int64_t most = ((int64_t)1 << 30) / F8 > 0 ? ((int64_t)1 << 30) / F8 : 1;
    for (int64_t r0 = 0; r0 < rows; r0 += most) {
        const int64_t nr = rows - r0 < most ? rows - r0 : most;
        const cudaError_t err = launch(r0, (uint32_t)(nr * F8));
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

// Three vectors a thread from 2^22 of them on (67 million: 691 -> 622 us); below, one, which spreads
// a small call over more CTAs (2,048 vectors: 1.9 us, 2.4 us with three; 670,000: the same either way).
constexpr uint32_t kManyVectors = 1u << 22;

template <bool kSave, int kU>
void run_swiglu(const uint4* h, uint4* a, uint2* codes, uint8_t* scales, uint32_t n, FastDiv cols,
                cudaStream_t st) {
    swiglu_kernel<kSave, kU><<<(n + kThreads * kU - 1) / (kThreads * kU), kThreads, 0, st>>>(
        h, a, codes, scales, n, cols);
}

}  // namespace

cudaError_t launch_swiglu(int64_t rows, int F, const uint16_t* h, uint16_t* a, int8_t* codes,
                          uint8_t* scales, cudaStream_t st) {
    const int F8 = F / 8;
    const FastDiv cols = make_fast_div((uint32_t)F8);
    return by_slabs(rows, F8, [&](int64_t r0, uint32_t n) {
        const uint4* hp = reinterpret_cast<const uint4*>(h) + r0 * 2 * F8;
        uint4* ap = reinterpret_cast<uint4*>(a) + r0 * F8;
        if (codes) {
            uint2* cp = reinterpret_cast<uint2*>(codes) + r0 * 2 * F8;
            uint8_t* sp = scales + r0 * (F8 / 2);
            n >= kManyVectors ? run_swiglu<true, 3>(hp, ap, cp, sp, n, cols, st)
                              : run_swiglu<true, 1>(hp, ap, cp, sp, n, cols, st);
        } else {
            n >= kManyVectors ? run_swiglu<false, 3>(hp, ap, nullptr, nullptr, n, cols, st)
                              : run_swiglu<false, 1>(hp, ap, nullptr, nullptr, n, cols, st);
        }
        return cudaGetLastError();
    });
}

cudaError_t launch_swiglu_bwd(int64_t rows, int F, const uint16_t* da, const int8_t* codes,
                              const uint8_t* scales, uint16_t* dh, uint16_t* a, cudaStream_t st) {
    const int F8 = F / 8;
    const FastDiv cols = make_fast_div((uint32_t)F8);
    return by_slabs(rows, F8, [&](int64_t r0, uint32_t n) {
        swiglu_bwd_kernel<<<(n + kThreads - 1) / kThreads, kThreads, 0, st>>>(
            reinterpret_cast<const uint4*>(da) + r0 * F8,
            reinterpret_cast<const uint2*>(codes) + r0 * 2 * F8, scales + r0 * (F8 / 2),
            reinterpret_cast<uint4*>(dh) + r0 * 2 * F8,
            a ? reinterpret_cast<uint4*>(a) + r0 * F8 : nullptr, n, cols);
        return cudaGetLastError();
    });
}

}  // namespace bep
