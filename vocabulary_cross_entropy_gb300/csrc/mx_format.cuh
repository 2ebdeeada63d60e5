// Microscaled formats: one E8M0 scale (a power of two) per 32 consecutive columns.
//
// Scale of a block with largest magnitude amax: the least e with
// amax <= M 2^e, M the format's largest value (448 for E4M3, 6 for E2M1), so no
// value of a block saturates and at most one binade of the format is unused.
// From the bits of amax = 1.f x 2^a (a subnormal one is below 2^-126): both maxima
// are 1.m x 2^E (1.75 x 2^8 and 1.5 x 2^2), hence e = a - E + (1.f > 1.m), an
// exponent subtraction and one comparison of mantissa bits.
//
// Codes are stored in rows padded with zeros to a multiple of 128 columns.
// Scales are stored in tiles of 128 rows x 4 blocks (512 bytes), the shape in which
// tcgen05.cp takes them into tensor memory: inside a tile, the scale of row r,
// block b is byte (r % 32) * 16 + (r / 32) * 4 + b.  Tiles of a row range are
// consecutive along the columns.
#pragma once

#include "vce_internal.cuh"

namespace vce {
namespace mx {

constexpr int kBlock = 32;      // columns per scale
constexpr int kRowTile = 128;   // rows per scale tile
constexpr int kColTile = 128;   // columns per scale tile (4 blocks); codes are padded to it
constexpr int kTileBytes = 512;
constexpr uint32_t kNanScale = 255;

inline __host__ __device__ int64_t padded(int64_t x) { return (x + 127) / 128 * 128; }

// Byte offset of the scale of (row, block); ``col_tiles`` = padded columns / 128.
__device__ __forceinline__ int64_t scale_offset(int64_t row, int64_t block, int64_t col_tiles) {
    const int r = int(row & 127);
    return ((row >> 7) * col_tiles + (block >> 2)) * kTileBytes + (r & 31) * 16 + (r >> 5) * 4 + int(block & 3);
}

// Scale byte from the bits of a block's largest magnitude (sign cleared).  A block
// that holds an infinity or a NaN has no scale: it gets the NaN code and zero codes.
template <int kFmt>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return kNanScale;
    constexpr int emax = kFmt == VCE_MX_E4M3 ? 8 : 2;
    constexpr uint32_t mant = kFmt == VCE_MX_E4M3 ? 0x600000u : 0x400000u;  // 1.75, 1.5
    const int biased = int(amax_bits >> 23) - emax + ((amax_bits & 0x7fffffu) > mant ? 1 : 0);
    return uint32_t(biased < 0 ? 0 : biased);  // at most 254 - emax + 1
}

// The factor 2^-(byte - 127), exact in FP32: the exponents 127 .. -126 are all normal.
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// The scale itself; 2^-127 is subnormal, byte 255 a NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
    if (byte == kNanScale) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

// Two values as codes, the first in the low bits: round to nearest even, saturating.
// (The conversion instructions by name: the toolkit's wrappers cost several times as many
// instructions, which at eight columns per thread was what bound the quantisation.)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    return c;
}
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t c;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
        : "=r"(c)
        : "f"(hi), "f"(lo));
    return c;
}

// max(m, |x|) that keeps a NaN
__device__ __forceinline__ float max_abs(float m, float x) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(x)));
    return r;
}

// Two codes (bits 0-3 and 4-7, or 0-7 and 8-15 of ``c``) as FP32 values.
//   E4M3 by the conversion instruction: every value is one of FP16, and its NaN (which
// mx_quantize never writes but other sources may) stays one.
//   E2M1 by bits: a code's exponent and mantissa put at the same places of a BF16 are the
// value times 2^-126 (exponent bias 1), the subnormal among them; the product is exact.
template <int kFmt>
__device__ __forceinline__ float2 decode_pair(uint32_t c) {
    if (kFmt == VCE_MX_E2M1) {
        const uint32_t t = (c & 0xfu) | (c & 0xf0u) << 12;
        const uint32_t pair = (t & 0x00070007u) << 6 | (t & 0x00080008u) << 12;
        return make_float2(__uint_as_float(pair << 16) * 0x1p126f, __uint_as_float(pair & 0xffff0000u) * 0x1p126f);
    }
    float2 v;
    asm("{\n\t.reg .b32 h;\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.f16x2.e4m3x2 h, %2;\n\tmov.b32 {lo, hi}, h;\n\t"
        "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(v.x), "=f"(v.y)
        : "h"(uint16_t(c)));
    return v;
}

}  // namespace mx
}  // namespace vce
