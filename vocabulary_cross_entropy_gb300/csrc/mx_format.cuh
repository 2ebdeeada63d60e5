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

#include <cuda_fp4.h>
#include <cuda_fp8.h>

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

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    return uint32_t(__nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest));
}

}  // namespace mx
}  // namespace vce
