// Weights of logits as whole numbers, and an order of (logit, index): what the kernels that
// choose tokens (ce_sample, ce_beam) share.
#pragma once

#include "vce_internal.cuh"

namespace vce {
namespace {

constexpr int kSteps = 64;            // values of n per octave
constexpr int kFracBits = 36;         // of s
constexpr int kIndexBits = 20;      // vocabulary of at most 2^20

__device__ const uint64_t kExp2Table[kSteps] = {
#include "exp2_table.inc"
};

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN stays
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ uint32_t order_bits(float z) {  // monotone in z
    const uint32_t b = __float_as_uint(z);
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order_bits(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// (logit, index) as one number: larger comes first.  -0 counts as 0.
__device__ __forceinline__ uint64_t key_of(float z, int i) {
    return uint64_t(order_bits(z + 0.f)) << kIndexBits | uint32_t((1 << kIndexBits) - 1 - i);
}
__device__ __forceinline__ float key_logit(uint64_t k) { return from_order_bits(uint32_t(k >> kIndexBits)); }
__device__ __forceinline__ int key_index(uint64_t k) { return (1 << kIndexBits) - 1 - int(k & ((1 << kIndexBits) - 1)); }

// A row's scale: m its largest logit, ch + cl = log2(e) / T as an unevaluated sum.
struct Scale {
    float m, ch, cl;
};

__device__ __forceinline__ Scale make_scale(float m, float t) {
    const float lh = 1.44269502162933349609375f, ll = 1.92596299e-8f;  // log2(e) = lh + ll
    t = fminf(fmaxf(t, 1e-30f), 1e30f);
    const float ch = lh / t;
    const float r = fmaf(-ch, t, lh) + ll;  // the division's remainder, exact
    return {m, ch, r / t};
}

// The leading term of (z - m) c, monotone in z.
__device__ __forceinline__ float log2_weight(const Scale& s, float z) { return __fmul_rn(z - s.m, s.ch); }

// The element's n (as the bin -n) and s of a log2_weight above least_log2.
//   (z - m) and its product with c are carried as sums of two floats (TwoSum, FMA), about
//   2^-47 relative.  The exponent is n / 64 + f with |f| <= 2^-7; 2^f - 1 from its series
//   to the fifth power, its linear term split into a multiple of 2^-29 and a rest.
//   round(64 p) is taken by adding 1.5 x 2^23.
__device__ __forceinline__ int bin_of(float p) { return 0x4b400000 - __float_as_int(fmaf(p, float(kSteps), 12582912.f)); }

struct Step {
    int bin;
    int g;  // s - 2^kFracBits
};
__device__ __forceinline__ Step step_of(const Scale& s, float z) {
    const float d = z - s.m;
    const float b = d - z;
    const float dl = (z - (d - b)) - (s.m + b);
    const float p = __fmul_rn(d, s.ch);
    float e = fmaf(d, s.ch, -p);
    e = fmaf(d, s.cl, e);
    e = fmaf(dl, s.ch, e);
    const float t = fmaf(p, float(kSteps), 12582912.f);
    const float f = fmaf(t - 12582912.f, -1.f / kSteps, p);
    const float lh = 0.693147182464599609375f, ll = -1.904654323148236e-9f;  // ln 2 = lh + ll
    const float a = f * lh;
    float r = fmaf(f, lh, -a);
    r = fmaf(f, ll, r);
    r = fmaf(e, lh, r);
    // ln2^k / k! for k = 2 .. 5
    const float c2 = 0.24022650695910072f, c3 = 0.05550410866482158f, c4 = 0.009618129107628477f,
                c5 = 0.0013333558146428443f;
    const float fe = f + e;
    r = fmaf(fe * fe, fmaf(fmaf(fmaf(c5, f, c4), f, c3), f, c2), r);
    const float big = 1.5f * 0x1p-6f;  // |a| < 2^-7: the sum stays in big's binade, whose last bit is 2^-29
    const float u = a + big;
    const int hi = __float_as_int(u) - __float_as_int(big);
    r += a - (u - big);
    const int lo = __float_as_int(fmaf(r, 0x1p36f, 12582912.f)) - 0x4b400000;
    return {0x4b400000 - __float_as_int(t), hi * 128 + lo};
}

// round(2^Q 2^(-bin / 64) sum / 2^36) for a sum of s below 2^57
__device__ __forceinline__ uint64_t scale_up(uint64_t sum, int bin, const uint64_t* table, int q_bits) {
    const int n = -bin;
    const uint64_t t = table[n & (kSteps - 1)];                       // 63 fractional bits
    const int shift = 63 + kFracBits - q_bits - (n >> 6);             // 55 .. 102
    const uint64_t hi = __umul64hi(sum, t), lo = sum * t;
    uint64_t q, rest;  // the value rounded down (2^63 for a row of full weights), and the bits below it from the top down
    if (shift < 64) {
        q = hi << (64 - shift) | lo >> shift;
        rest = lo << (64 - shift);
    } else {
        q = hi >> (shift - 64);
        rest = shift == 64 ? lo : hi << (128 - shift);
    }
    return q + (rest >> 63);
}

__device__ __forceinline__ uint64_t weight_of(const Scale& s, float z, const uint64_t* table, int q_bits) {
    const Step st = step_of(s, z);
    return scale_up((uint64_t(1) << kFracBits) + int64_t(st.g), st.bin, table, q_bits);
}

template <typename T>
__device__ __forceinline__ float element(uint4 v, int e);
template <>
__device__ __forceinline__ float element<float>(uint4 v, int e) {
    return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
}
template <>
__device__ __forceinline__ float element<__nv_bfloat16>(uint4 v, int e) {
    const uint32_t w = (e >> 1) == 0 ? v.x : (e >> 1) == 1 ? v.y : (e >> 1) == 2 ? v.z : v.w;
    return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
}
__device__ __forceinline__ float one(const float* p) { return *p; }
__device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }

}  // namespace
}  // namespace vce
