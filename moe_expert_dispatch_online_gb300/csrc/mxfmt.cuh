// Microscaled number formats: blocks of 32 elements share a power of two, held as the byte
// e + 127 (e8m0; 0xFF stands for NaN). e is the smallest exponent >= -127 with
// amax <= top * 2^e, where top is the element type's largest magnitude (6 for e2m1, 127 for
// int8), so no element saturates. The scaling is exact (a power of two), so the only rounding
// is the element's own: to nearest, ties to even. A block that holds an infinity or a NaN
// gets the byte 0xFF and zero elements: all its 32 values are NaN.
#pragma once

#include <cuda_bf16.h>

#include "bep_internal.cuh"

namespace bep {
namespace {

constexpr int kMxBlock = 32;
constexpr uint32_t kMxNan = 0xFFu;

// e8m0 byte for a block's largest magnitude (its fp32 bits, sign cleared). kLead: floor(log2(top));
// kLimit: fraction bits of top / 2^kLead (6 = 1.5 * 2^2, 127 = 1.984375 * 2^6).
template <int kLead, uint32_t kLimit>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return kMxNan;
    const int e = (int)(amax_bits >> 23) - kLead + ((amax_bits & 0x7fffffu) > kLimit ? 1 : 0);
    return (uint32_t)max(e, 0);   // biased exponent, e >= -127
}
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) {
    return mx_scale_byte<2, 0x400000u>(amax_bits);
}
__device__ __forceinline__ uint32_t mx8_scale_byte(uint32_t amax_bits) {
    return mx_scale_byte<6, 0x7e0000u>(amax_bits);
}
// 2^-e and 2^e of a scale byte: e in [-127, 126] (a NaN byte gives 0 and NaN)
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
    return byte == kMxNan ? 0.0f : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float mx_scale(uint32_t byte) {
    if (byte == kMxNan) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(byte ? byte << 23 : 0x400000u);
}

// Eight floats (already scaled) to eight e2m1 codes, the first in the lowest 4 bits.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float* f) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return r;
}

// The block's 32 values (fp32) to 16 bytes of e2m1 codes; returns the scale byte.
__device__ __forceinline__ uint32_t mx4_block(const float* f, uint4* codes) {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < kMxBlock; ++i) amax = max(amax, __float_as_uint(f[i]) & 0x7fffffffu);
    const uint32_t byte = mx4_scale_byte(amax);
    if (byte == kMxNan) {
        *codes = make_uint4(0, 0, 0, 0);
        return byte;
    }
    const float inv = mx_inverse(byte);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = f[8 * j + i] * inv;
        w[j] = pack_e2m1x8(s);
    }
    *codes = make_uint4(w[0], w[1], w[2], w[3]);
    return byte;
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Four floats (already scaled, magnitudes <= 127) to four int8. Adding 1.5 * 2^23 rounds to the
// nearest integer, ties to even, and leaves it in the low byte in two's complement.
__device__ __forceinline__ uint32_t pack_int8x4(float a, float b, float c, float d) {
    const float k = 12582912.0f;
    const uint32_t lo = __byte_perm(__float_as_uint(a + k), __float_as_uint(b + k), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(c + k), __float_as_uint(d + k), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}
// int8 element `i` of a packed word as fp32
__device__ __forceinline__ float int8_at(uint32_t w, int i) {
    return (float)(int8_t)(w >> (8 * i));
}

// sigmoid(x) by the hardware's exponential and reciprocal, 2 units in the last place of fp32 or fewer each, and
// the rounding of the exponential's argument, 2^-24 |x|: what it enters is rounded to 8 bits or fewer
// afterwards. 0 from x = -87.3 down, where the divisor passes 2^126.
__device__ __forceinline__ float hw_sigmoid(float x) {
    return __fdividef(1.0f, 1.0f + __expf(-x));
}

// The same for any gate, as r m^2 with r = 1 / (1 + e^-|g|) and m = 1, or e^(g/2) for g < 0. The two factors m
// meet the other factors one at a time, so that a tiny sigmoid beside a large up value does not vanish on
// the way: m is 0 only from g = -174 down. Twice the instructions, so a thread takes it only if one of its
// gates is below kTinyGate (524,288 rows of 1024 + 1024, forward and backward: 1522 us with it throughout,
// 1413 us without).
constexpr float kTinyGate = -80.0f;
struct Gate {
    float r, m, e;   // e = e^-|g|
};
__device__ __forceinline__ Gate gate_of(float g) {
    Gate s;
    const float t = __expf(-0.5f * fabsf(g));
    s.e = t * t;
    s.r = __fdividef(1.0f, 1.0f + s.e);
    s.m = g < 0.0f ? t : 1.0f;
    return s;
}
// g * sigmoid(g) * u
__device__ __forceinline__ float gated(float g, const Gate& s, float u) { return (g * s.r * s.m) * (s.m * u); }
// The same of 8 gates and up values.
__device__ __forceinline__ void gated8(const float* g, const float* u, float* a) {
    float low = g[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) low = fminf(low, g[k]);
    if (low >= kTinyGate) {
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = g[k] * hw_sigmoid(g[k]) * u[k];
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = gated(g[k], gate_of(g[k]), u[k]);
    }
}

}  // namespace
}  // namespace bep
