// Routing of tokens to experts (sm_103a): scores, groups, top-K, gates, loads, and the
// gradient of the logits.
//
//   s_e  = sigmoid(l_e), or softmax(l)_e over the token's E logits        (fp32)
//   key  = s_e + bias_e; the K largest keys are chosen, ties to the lowest index,
//          from the top_groups groups whose group_top largest keys sum highest
//   g_k  = scale * s_k / sum_j s_j (renorm; 0 where every chosen expert is masked), or scale * s_k
// Backward, with dv_k = dL/ds_k:
//   dv_k = scale * dg_k, or with renorm scale * (dg_k - sum_j dg_j w_j) / Z, w = s / Z
//   sigmoid: dl_k = dv_k s_k (1 - s_k), other experts 0
//   softmax: dl_e = s_e (dv_e - sum_k dv_k s_k). With renorm that sum is 0 and
//            dl_k = scale * w_k (dg_k - sum_j dg_j w_j), other experts 0, where w is the
//            softmax of the K chosen logits alone: no other logit is read.
//
// One warp owns one token; lane l holds experts l, l + 32, ... in registers, so each load
// instruction covers 32 consecutive logits whatever E and its alignment are.

#include <cuda_bf16.h>
#include <float.h>

#include "bep_internal.cuh"

namespace bep {
namespace {

// Threads of a CTA: large CTAs, since each adds its loads to memory once; half as many where a
// lane's experts need more than 128 registers.
constexpr int threads_for(int V) { return V > 16 ? 256 : 512; }
constexpr unsigned kAll = 0xffffffffu;

// Ranks below every key of an expert that can be chosen.
constexpr uint32_t kGone = 0u;     // chosen already, outside the kept groups, or no expert
constexpr uint32_t kMasked = 1u;   // logit at the type's lowest value or below

template <typename T>
__device__ __forceinline__ float load_logit(const T* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) {
    return __ldg(p);
}
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const uint16_t* p) {
    return __uint_as_float((uint32_t)__ldg(p) << 16);
}
// lowest finite value of the logits' type: at or below it an expert is masked
template <typename T>
__device__ __forceinline__ float lowest() {
    return sizeof(T) == 4 ? -FLT_MAX : __uint_as_float(0xff7f0000u);
}
template <typename T>
__device__ __forceinline__ void store_grad(T* p, float v);
template <>
__device__ __forceinline__ void store_grad<float>(float* p, float v) {
    *p = v;
}
template <>
__device__ __forceinline__ void store_grad<uint16_t>(uint16_t* p, float v) {
    *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Unsigned order of the result = order of the floats; -0 counts as +0. Results are >= 0x7fffff.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t b = __float_as_uint(f + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

__device__ __forceinline__ float warp_max(float v) {
    return unordered(__reduce_max_sync(kAll, ordered(v)));
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// down to the smallest subnormal (x = -103), where 1 / (1 + e^-x) would be 0 from -89 on
__device__ __forceinline__ float sigmoid(float x) {
    const float e = expf(-fabsf(x));
    return (x < 0.0f ? e : 1.0f) / (1.0f + e);
}

// The scores of all E experts of an ordinary row (keys, and the softmax's sum) use the hardware's 2^x and
// reciprocal, 2 units in the last place of fp32 each beside the rounding of x log2(e), in 2 and 4
// instructions; the K gates, and the keys of other rows, use expf and a rounded division. Results below
// 2^-126 are 0, which an ordinary row's never are.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float fast_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float fast_sigmoid(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + fast_exp2(x * -kLog2e)));
    return r;
}
// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A token's logits, lane l's at l + 32 i (the last expert again past E).
template <int V, bool kFull, typename T>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int E, int lane, float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = load_logit(row + (kFull ? lane + 32 * i : min(lane + 32 * i, E - 1)));
}
// An ordinary row's magnitudes are all kOrdinary at most: nothing is masked in it, and no score or
// exponential underflows. Other rows are looked at element by element: masked logits become -inf and
// *bad is set for a NaN or +inf among them. *top: the softmax's reference, the row's largest logit (0 if
// there is none, and for sigmoids). Without a reference the argument's rounding would grow with the
// logits and not with their distance from the largest: 8 logits near 36 then have scores 2.4e-6 off, and
// 2.6e-7 with it. Past E: -inf in either case.
constexpr float kOrdinary = 40.0f;
template <int V, bool kFull, typename T>
__device__ __forceinline__ bool look_over(int E, int lane, bool softmax, float (&x)[V], float* top, int* bad) {
    float hi = -INFINITY, far = 0.0f;
    if (softmax) {
        float lo = INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            hi = max_nan(hi, x[i]);
            lo = fminf(lo, x[i]);
        }
        far = max_nan(hi, -lo);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) far = max_nan(far, fabsf(x[i]));
    }
    const bool ordinary = __all_sync(kAll, far <= kOrdinary);
    *top = 0.0f;
    if (ordinary) {
        if (softmax) *top = warp_max(hi);
    } else {
        hi = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (!(x[i] <= FLT_MAX)) {
                *bad = 1;
                x[i] = -INFINITY;
            }
            if (x[i] <= lowest<T>()) x[i] = -INFINITY;
            hi = fmaxf(hi, x[i]);
        }
        hi = warp_max(hi);
        if (softmax && hi > -INFINITY) *top = hi;   // else nothing to choose from: all scores 0
    }
    if (!kFull) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i >= E) x[i] = -INFINITY;
    }
    return ordinary;
}

// e^(x - top); the difference first, so that a large top costs no precision
__device__ __forceinline__ float exp_of(float x, float top) { return fast_exp2((x - top) * kLog2e); }

struct RouteParams {
    int64_t ntok;
    int E, K;
    int groups, top_groups, group_top, group_size;
    int softmax, renorm;
    float scale;
};

// Larger two of (a1 >= a2) and (b1 >= b2).
__device__ __forceinline__ void merge2(uint32_t& a1, uint32_t& a2, uint32_t b1, uint32_t b2) {
    const uint32_t lo = min(a1, b1);
    a1 = max(a1, b1);
    a2 = max(lo, max(a2, b2));
}

// ------------------------------------------------------------------------------ forward
// Selection. A key's leading bits and the expert's index (complemented) make one 32-bit word,
// so that a round is one warp-wide maximum that names the winner and breaks ties. Each lane keeps
// its three largest words. Where that does not decide -- a lane's three have all won (about 5
// tokens in 100 at 8 of 384), or two of the K + 1 leading words agree in all their key bits (as
// many) -- the choice is made again on whole keys, with a second reduction for the index.
// 65,536 tokens, 8 of 384 by softmax and bias: 130 us with whole keys in every round and
// element-by-element checks, 86 us with two words a lane, rescanned when both have won, 42 us
// now; bound by the integer pipe and the chain of reductions (490 instructions a token).
template <int V>
struct Packed {
    static constexpr int kBits = V <= 1 ? 6 : V <= 3 ? 7 : V <= 7 ? 8 : V <= 15 ? 9 : V <= 16 ? 10 : V <= 32 ? 11 : 12;
    static_assert(32 * V < (1 << kBits), "an index and its complement differ from 0");
    static constexpr uint32_t kIndex = (1u << kBits) - 1;
};

// The K experts of the largest keys, lane k for the k-th. kAny: every key is an expert's.
// exact: the words hold whole keys. raw: the keys are the floats' own bits, in order only from +0
// on, which is decided as long as K + 1 keys are not negative (two integer instructions an expert
// fewer than keys in order throughout).
template <int V, bool kAny>
__device__ __forceinline__ int choose_packed(const uint32_t (&key)[V], int K, int lane, bool exact, bool raw,
                                             bool* decided) {
    constexpr uint32_t kIndex = Packed<V>::kIndex;
    const uint32_t c = (kIndex - lane) + (raw ? 0x80000000u : 0u);
    uint32_t t1 = 0, t2 = 0, t3 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        uint32_t w = (key[i] & ~kIndex) ^ (c - 32 * i);
        if (!kAny && key[i] == kGone) w = 0;
        if (V > 2) t3 = max(t3, min(t2, w));
        t2 = max(t2, min(t1, w));
        t1 = max(t1, w);
    }
    const bool any = t1 != 0;
    uint32_t mine = 0;
    for (int k = 0; k < K; ++k) {
        const uint32_t m = __reduce_max_sync(kAll, t1);
        if (lane == k) mine = m;
        if (t1 == m) {
            t1 = t2;
            t2 = t3;
            t3 = 0;
        }
    }
    const bool spent = V > 3 && any && t1 == 0;   // this lane may have had a fourth
    const uint32_t next = __reduce_max_sync(kAll, t1);   // the first that is not chosen
    uint32_t after = __shfl_down_sync(kAll, mine, 1);   // every lane takes part
    if (lane == K - 1) after = next;
    const bool near = !exact && lane < K && (mine ^ after) <= kIndex;
    *decided = !__any_sync(kAll, spent || near) && (!raw || next >= 0x80000000u);
    return (int)(kIndex - (mine & kIndex));
}

// The same on whole keys: the warp's largest key, then the lowest expert that has it.
template <int V>
__device__ __forceinline__ int choose_whole(uint32_t (&key)[V], int K, int lane) {
    int mine = 0;
    for (int k = 0; k < K; ++k) {
        uint32_t best = kGone;
        int at = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > best) {
                best = key[i];
                at = lane + 32 * i;
            }
        const uint32_t m = __reduce_max_sync(kAll, best);
        const int e = (int)__reduce_min_sync(kAll, best == m ? (unsigned)at : 0x7fffffffu);
        if (lane == k) mine = e;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 32 * i == e) key[i] = kGone;
    }
    return mine;
}

// V: experts a lane holds (E <= 32 V). Scores of all E experts are needed only where keys
// are more than the logits' order (a bias, sums of two keys) or where the softmax is not
// renormalised over the chosen ones.
// kFull: E = 32 V. kGroups: some groups are cut.
template <int V, typename T, bool kFull, bool kGroups>
__global__ void __launch_bounds__(threads_for(V)) route_kernel(const T* __restrict__ logits,
                                                         const float* __restrict__ bias,
                                                         int32_t* __restrict__ topk,
                                                         float* __restrict__ gates,
                                                         int32_t* __restrict__ load,
                                                         const RouteParams p, int32_t* status) {
    constexpr int kThreads = threads_for(V), kWarps = kThreads / 32;
    extern __shared__ uint32_t smem[];   // loads [E], the bias [E], then each warp's keys [E]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int* s_load = reinterpret_cast<int*>(smem);
    float* s_bias = reinterpret_cast<float*>(smem + p.E);
    uint32_t* s_key = smem + (2 + warp) * p.E;
    int bias_nan = 0;
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
        s_load[e] = 0;
        const float b = bias ? __ldg(bias + e) : 0.0f;
        s_bias[e] = b;
        bias_nan |= b != b;
    }
    bias_nan = __syncthreads_or(bias_nan);
    const float low = lowest<T>();
    const bool by_score = bias != nullptr || (kGroups && p.group_top > 1);
    const bool row_sum = p.softmax && (by_score || !p.renorm);
    int per = 32;   // lanes that scan a group
    while (kGroups && per * p.groups > 32) per >>= 1;
    const int g = lane / per, part = lane & (per - 1);
    int bad = 0;
    const int64_t step = (int64_t)gridDim.x * kWarps;
    float x[V];
    int64_t tok = (int64_t)blockIdx.x * kWarps + warp;
    if (tok < p.ntok) load_row<V, kFull>(logits + tok * p.E, p.E, lane, x);
    for (; tok < p.ntok; tok += step) {
        const T* row = logits + tok * p.E;
        float top;
        const bool ordinary = look_over<V, kFull, T>(p.E, lane, row_sum, x, &top, &bad) && !bias_nan;
        float inv = 0.0f;   // 1 / sum of exp(l - top)
        uint32_t key[V];
        if (row_sum) {
            float ex[V], sum = 0.0f;
            if (ordinary) {
#pragma unroll
                for (int i = 0; i < V; ++i) ex[i] = exp_of(x[i], top);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) ex[i] = expf(x[i] - top);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) sum += ex[i];
            sum = warp_sum(sum);
            inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                key[i] = by_score ? __float_as_uint(fmaf(ex[i], inv, s_bias[kFull ? lane + 32 * i : min(lane + 32 * i, p.E - 1)]))
                                  : __float_as_uint(x[i]);
        } else if (by_score) {
            float sg[V];
            if (ordinary) {
#pragma unroll
                for (int i = 0; i < V; ++i) sg[i] = fast_sigmoid(x[i]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) sg[i] = sigmoid(x[i]);
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                key[i] = __float_as_uint(
                    __fadd_rn(sg[i], s_bias[kFull ? lane + 32 * i : min(lane + 32 * i, p.E - 1)]));
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = __float_as_uint(x[i]);
        }
        const bool raw = kFull && !kGroups && by_score && ordinary;   // a score with a bias: never -0
        if (!raw) {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = ordered(__uint_as_float(key[i]));
        }
        if (!ordinary) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 32 * i;
                if (by_score && e < p.E && s_bias[e] != s_bias[e]) {
                    bad = 1;
                    key[i] = kMasked;
                }
                if (x[i] == -INFINITY) key[i] = kMasked;
            }
        }
        if (!kFull) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane + 32 * i >= p.E) key[i] = kGone;
        }
        if (kGroups) {
            // `per` lanes (a power of two) scan each group's keys for its two largest
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (kFull || lane + 32 * i < p.E) s_key[lane + 32 * i] = key[i];
            __syncwarp();
            uint32_t k1 = kGone, k2 = kGone;
            if (g < p.groups)
                for (int j = part; j < p.group_size; j += per) {
                    const uint32_t k = s_key[g * p.group_size + j];
                    k2 = max(k2, min(k1, k));
                    k1 = max(k1, k);
                }
            for (int o = 1; o < per; o <<= 1) {
                const uint32_t b1 = __shfl_xor_sync(kAll, k1, o), b2 = __shfl_xor_sync(kAll, k2, o);
                merge2(k1, k2, b1, b2);
            }
            // the group's score: its leading keys that are numbers; a group without any is last
            uint32_t score = kGone;
            if (g < p.groups) {
                if (k1 <= kMasked) score = kMasked;
                else if (p.group_top == 1 || k2 <= kMasked) score = k1;
                else score = ordered(unordered(k1) + unordered(k2));
            }
            int rank = 0;
            for (int o = 0; o < p.groups; ++o) {
                const uint32_t other = __shfl_sync(kAll, score, o * per);
                rank += other > score || (other == score && o < g);
            }
            if (g < p.groups && rank >= p.top_groups)
                for (int j = part; j < p.group_size; j += per) s_key[g * p.group_size + j] = kGone;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (kFull || lane + 32 * i < p.E) key[i] = s_key[lane + 32 * i];
            if (by_score && !bias) {
                // scores were for the groups' sums: without a bias their order is the logits', which
                // for bf16 logits, often equal, the words below hold whole
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (key[i] > kMasked) key[i] = ordered(x[i]);
            }
        }
        // the keys hold all the choice needs: the next token's logits arrive while it is made
        if (tok + step < p.ntok) load_row<V, kFull>(row + step * p.E, p.E, lane, x);
        bool decided;
        int mine = choose_packed<V, kFull && !kGroups>(key, p.K, lane, sizeof(T) == 2 && !bias, raw, &decided);
        if (!decided) {
            if (raw) {
#pragma unroll
                for (int i = 0; i < V; ++i) key[i] = ordered(__uint_as_float(key[i]));
            }
            mine = choose_whole(key, p.K, lane);
        }
        // gates of the chosen experts, lane k for the k-th
        float xs = -INFINITY;
        if (lane < p.K) {
            xs = load_logit(row + mine);
            if (!(xs <= FLT_MAX) || xs <= low) xs = -INFINITY;
        }
        // renormalised, the row's sum cancels: the largest chosen logit is the reference, as in the
        // backward, so that experts far below the row's largest (kept from it by a bias) keep their ratios
        const float ref = p.renorm ? warp_max(xs) : top;
        float sc = 0.0f;
        if (xs != -INFINITY) {
            if (p.softmax) sc = expf(xs - ref) * (p.renorm ? 1.0f : inv);
            else sc = p.renorm && ref < -kOrdinary ? expf(xs - ref) : sigmoid(xs);   // e^x itself there
        }
        if (p.renorm) {
            const float z = warp_sum(sc);
            sc = z > 0.0f ? sc / z : 0.0f;
        }
        if (lane < p.K) {
            topk[tok * p.K + lane] = mine;
            gates[tok * p.K + lane] = p.scale * sc;
            if (load) atomicAdd(&s_load[mine], 1);
        }
    }
    if (__any_sync(kAll, bad) && lane == 0) set_status(status, BEP_DERR_NONFINITE);
    if (load) {
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += kThreads)
            if (s_load[e]) atomicAdd(&load[e], s_load[e]);
    }
}

// ------------------------------------------------------------------------------ backward
// kDense: softmax without renorm, every logit has a gradient. Otherwise only the K chosen
// logits are read: the row is written as zeros and the K values over it. kFull: E = 32 V.
template <int V, typename T, bool kDense, bool kFull>
__global__ void __launch_bounds__(threads_for(V)) route_bwd_kernel(const T* __restrict__ logits,
                                                             const int32_t* __restrict__ topk,
                                                             const float* __restrict__ dgates,
                                                             T* __restrict__ dlogits,
                                                             const RouteParams p, int32_t* status) {
    constexpr int kWarps = threads_for(V) / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float low = lowest<T>();
    int bad = 0;
    const int64_t step = (int64_t)gridDim.x * kWarps;
    float next[V];
    int64_t tok = (int64_t)blockIdx.x * kWarps + warp;
    if (kDense && tok < p.ntok) load_row<V, kFull>(logits + tok * p.E, p.E, lane, next);
    for (; tok < p.ntok; tok += step) {
        const T* row = logits + tok * p.E;
        T* out = dlogits + tok * p.E;
        float x[V];
        if (kDense) {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = next[i];
            if (tok + step < p.ntok) load_row<V, kFull>(row + step * p.E, p.E, lane, next);
        }
        int e = -1;
        float dg = 0.0f, xs = -INFINITY;
        if (lane < p.K) {
            e = topk[tok * p.K + lane];
            dg = dgates[tok * p.K + lane];
            if (e < 0 || e >= p.E) {
                bad |= BEP_DERR_EXPERT_ID;
                e = -1;
                dg = 0.0f;
            }
        }
        auto chosen_logit = [&]() {
            if (e < 0) return -INFINITY;
            const float v = load_logit(row + e);
            return !(v <= FLT_MAX) || v <= low ? -INFINITY : v;
        };
        float v;   // dL/dl of this lane's chosen expert
        if (kDense) {
            float top, sum = 0.0f;
            int masked = 0;   // reported by the forward
            look_over<V, kFull, T>(p.E, lane, true, x, &top, &masked);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[i] = exp_of(x[i], top);
                sum += x[i];
            }
            sum = warp_sum(sum);
            const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
            xs = chosen_logit();
            const float s = xs == -INFINITY ? 0.0f : expf(xs - top) * inv;
            const float dot = warp_sum(s * dg);
            v = p.scale * s * (dg - dot);
            const float c = -p.scale * dot * inv;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (kFull || lane + 32 * i < p.E) store_grad(out + lane + 32 * i, c * x[i]);
        } else {
            float s, w = 0.0f, z = 0.0f;
            xs = chosen_logit();
            const float top = warp_max(xs);
            if (p.softmax || (p.renorm && top < -kOrdinary)) {
                s = xs == -INFINITY ? 0.0f : expf(xs - top);
            } else {
                s = xs == -INFINITY ? 0.0f : sigmoid(xs);
            }
            float d = dg;
            if (p.renorm) {
                z = warp_sum(s);
                w = z > 0.0f ? s / z : 0.0f;
                d = dg - warp_sum(dg * w);
            }
            if (p.softmax) v = p.scale * w * d;                                       // renorm
            else v = p.scale * (p.renorm ? w : s) * d * (xs == -INFINITY ? 0.0f : sigmoid(-xs));
            const uint32_t bytes = (uint32_t)p.E * sizeof(T);
            if (((reinterpret_cast<uintptr_t>(out) | bytes) & 15) == 0) {
                for (uint32_t j = lane; j < bytes / 16; j += 32)
                    reinterpret_cast<uint4*>(out)[j] = make_uint4(0, 0, 0, 0);
            } else {
                for (int j = lane; j < p.E; j += 32) store_grad(out + j, 0.0f);
            }
        }
        __syncwarp();   // the row's fill is ordered before the chosen experts' values
        if (e >= 0) store_grad(out + e, v);
    }
    const unsigned any = __reduce_or_sync(kAll, (unsigned)bad);
    if (any && lane == 0) set_status(status, (int)any);
}

RouteParams params_of(const Dims& d, const bep_route_config& rc) {
    RouteParams p;
    p.ntok = (int64_t)d.R * d.S;
    p.E = d.E;
    p.K = d.K;
    p.groups = rc.groups;
    p.top_groups = rc.top_groups;
    p.group_top = rc.group_top;
    p.group_size = d.E / rc.groups;
    p.softmax = rc.score == BEP_SCORE_SOFTMAX;
    p.renorm = rc.renorm != 0;
    p.scale = rc.scale;
    return p;
}

// Two CTAs an SM at most: what the registers let in.
int grid_for(int64_t ntok, int num_sms, int threads) {
    const int warps = threads / 32;
    const int64_t g = (ntok + warps - 1) / warps, cap = (int64_t)num_sms * 2;
    return (int)(g < cap ? g : cap);
}

// Calls fn with the smallest per-lane count that holds E experts.
template <typename F>
cudaError_t with_width(int E, F&& fn) {
    if (E <= 32) return fn(std::integral_constant<int, 1>());
    if (E <= 64) return fn(std::integral_constant<int, 2>());
    if (E <= 96) return fn(std::integral_constant<int, 3>());
    if (E <= 128) return fn(std::integral_constant<int, 4>());
    if (E <= 160) return fn(std::integral_constant<int, 5>());
    if (E <= 192) return fn(std::integral_constant<int, 6>());
    if (E <= 256) return fn(std::integral_constant<int, 8>());
    if (E <= 384) return fn(std::integral_constant<int, 12>());
    if (E <= 512) return fn(std::integral_constant<int, 16>());
    if (E <= 1024) return fn(std::integral_constant<int, 32>());
    return fn(std::integral_constant<int, 64>());
}

template <typename T>
cudaError_t route_typed(const Dims& d, const Workspace& ws, const RouteParams& p, const T* logits,
                        const float* bias, int32_t* topk, float* gates, int32_t* load, int num_sms,
                        cudaStream_t st) {
    const bool cut = p.top_groups < p.groups;
    return with_width(d.E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        // shared memory: the loads and the bias, and the keys of each warp where groups are cut
        const size_t smem = (2 * (size_t)d.E + (cut ? (size_t)(threads_for(V) / 32) * d.E : 0)) * 4;
        const bool all = d.E == 32 * V;
        const auto kernel = all ? (cut ? route_kernel<V, T, true, true> : route_kernel<V, T, true, false>)
                                : (cut ? route_kernel<V, T, false, true> : route_kernel<V, T, false, false>);
        if (smem > 48 * 1024) {
            const cudaError_t err =
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (err != cudaSuccess) return err;
        }
        kernel<<<grid_for(p.ntok, num_sms, threads_for(V)), threads_for(V), smem, st>>>(logits, bias, topk, gates, load, p,
                                                                     ws.status);
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t route_bwd_typed(const Dims& d, const Workspace& ws, const RouteParams& p,
                            const T* logits, const int32_t* topk, const float* dgates, T* dlogits,
                            int num_sms, cudaStream_t st) {
    if (!p.softmax || p.renorm) {
        route_bwd_kernel<1, T, false, false>
            <<<grid_for(p.ntok, num_sms, threads_for(1)), threads_for(1), 0, st>>>(logits, topk, dgates,
                                                                                dlogits, p, ws.status);
        return cudaGetLastError();
    }
    return with_width(d.E, [&](auto v) {
        constexpr int V = decltype(v)::value;
        const auto kernel = d.E == 32 * V ? route_bwd_kernel<V, T, true, true> : route_bwd_kernel<V, T, true, false>;
        kernel<<<grid_for(p.ntok, num_sms, threads_for(V)), threads_for(V), 0, st>>>(
            logits, topk, dgates, dlogits, p, ws.status);
        return cudaGetLastError();
    });
}

}  // namespace

cudaError_t launch_route(const Dims& d, const Workspace& ws, const bep_route_config& rc,
                         const void* logits, int logits_type, const float* bias, int32_t* topk,
                         float* gates, int32_t* load, int num_sms, cudaStream_t st) {
    const RouteParams p = params_of(d, rc);
    if (p.ntok == 0) return cudaSuccess;
    if (logits_type == BEP_F32)
        return route_typed(d, ws, p, static_cast<const float*>(logits), bias, topk, gates, load,
                           num_sms, st);
    return route_typed(d, ws, p, static_cast<const uint16_t*>(logits), bias, topk, gates, load,
                       num_sms, st);
}

cudaError_t launch_route_bwd(const Dims& d, const Workspace& ws, const bep_route_config& rc,
                             const void* logits, int logits_type, const int32_t* topk,
                             const float* dgates, void* dlogits, int num_sms, cudaStream_t st) {
    const RouteParams p = params_of(d, rc);
    if (p.ntok == 0) return cudaSuccess;
    if (logits_type == BEP_F32)
        return route_bwd_typed(d, ws, p, static_cast<const float*>(logits), topk, dgates,
                               static_cast<float*>(dlogits), num_sms, st);
    return route_bwd_typed(d, ws, p, static_cast<const uint16_t*>(logits), topk, dgates,
                           static_cast<uint16_t*>(dlogits), num_sms, st);
}

}  // namespace bep
