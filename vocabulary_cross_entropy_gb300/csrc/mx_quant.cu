// Quantisation of a BF16 or FP32 matrix to microscaled E2M1 or E4M3, and back
// (mx_format.cuh has the formats).  Both are copies in what they cost: one thread
// takes eight consecutive columns, four neighbouring lanes share a block of 32 and
// find its largest magnitude with two shuffles.

#include "vce_internal.cuh"
#include "mx_format.cuh"

namespace vce {
namespace {

constexpr int kThreads = 256;

struct QuantArgs {
    const void* x;
    int64_t rows, cols, stride, padded, rows_padded;
    uint8_t *codes, *scales;
    int vector_ok;  // rows start 16-byte aligned and cols is a multiple of 8
    int tpr;        // threads per row: a power of two, 16 .. kThreads
    int* dev_status;
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// One thread per eight columns and step; ``tpr`` threads walk one row.  The grid covers the
// scale rows that fill the last tile too.
template <typename T, int kFmt>
__global__ void __launch_bounds__(kThreads) mx_quantize_kernel(const QuantArgs a) {
    const int units = int(a.padded / 8);  // per row, a multiple of 16: half warps share a scale tile
    const int64_t row = int64_t(blockIdx.x) * (kThreads / a.tpr) + threadIdx.x / a.tpr;
    if (row >= a.rows_padded) return;
    const bool live = row < a.rows;
    const T* x = static_cast<const T*>(a.x) + row * a.stride;
    const int64_t tile_row = mx::scale_offset(row, 0, a.padded / mx::kColTile);
#pragma unroll 2
    for (int u = threadIdx.x % a.tpr; u < units; u += a.tpr) {  // whole half warps
        const int col = u * 8;
        float v[8];
        if (live && a.vector_ok && col < a.cols) {
            load8<T>(x + col, v);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = live && col + k < a.cols ? load1(x + col + k) : 0.f;
        }
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
        const unsigned lanes = 0xffffu << (threadIdx.x & 16);
        m = max(m, __shfl_xor_sync(lanes, m, 1));
        m = max(m, __shfl_xor_sync(lanes, m, 2));
        const uint32_t sb = mx::scale_byte<kFmt>(m);
        const bool bad = sb == mx::kNanScale;
        const float inv = bad ? 0.f : mx::inverse_scale(sb);
        // the four scales of a tile's row as one word
        uint32_t word = sb | __shfl_down_sync(lanes, sb, 4, 16) << 8;
        word |= __shfl_down_sync(lanes, word, 8, 16) << 16;
        if ((threadIdx.x & 15) == 0 && VCE_BOUNDS(col % mx::kColTile == 0 && col < a.padded, a.dev_status))
            *reinterpret_cast<uint32_t*>(a.scales + tile_row + int64_t(col / mx::kColTile) * mx::kTileBytes) = word;
        if (!live || !VCE_BOUNDS(row >= 0 && col + 8 <= a.padded, a.dev_status)) continue;
        if (kFmt == VCE_MX_E4M3) {
            uint32_t c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = bad ? 0u : mx::e4m3x2(v[2 * k] * inv, v[2 * k + 1] * inv);
            *reinterpret_cast<uint2*>(a.codes + row * a.padded + col) =
                make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
        } else {
            uint32_t c = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) c |= (bad ? 0u : mx::e2m1x2(v[2 * k] * inv, v[2 * k + 1] * inv)) << (8 * k);
            *reinterpret_cast<uint32_t*>(a.codes + (row * a.padded + col) / 2) = c;
        }
    }
}

struct DequantArgs {
    const uint8_t *codes, *scales;
    int64_t rows, cols, stride, padded;
    void* out;
    int vector_ok;
    int tpr;
    int* dev_status;
};

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<uint32_t*>(&b);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(u[0], u[1], u[2], u[3]));
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// A value of either format fits 4 significant bits, so its product with the scale is
// exact in FP32, and in BF16 unless it is subnormal there.
template <typename T, int kFmt>
__global__ void __launch_bounds__(kThreads) mx_dequantize_kernel(const DequantArgs a) {
    const int units = int((a.cols + 7) / 8);
    const int64_t row = int64_t(blockIdx.x) * (kThreads / a.tpr) + threadIdx.x / a.tpr;
    if (row >= a.rows) return;
    const uint8_t* scales = a.scales + mx::scale_offset(row, 0, a.padded / mx::kColTile);
    T* out = static_cast<T*>(a.out) + row * a.stride;
#pragma unroll 2
    for (int u = threadIdx.x % a.tpr; u < units; u += a.tpr) {
        const int col = u * 8;
        if (!VCE_BOUNDS(row >= 0 && col + 8 <= a.padded, a.dev_status)) continue;
        const float s = mx::scale_value(scales[(col / mx::kColTile) * mx::kTileBytes + (col / mx::kBlock & 3)]);
        float v[8];
        if (kFmt == VCE_MX_E4M3) {
            const uint2 c = __ldcs(reinterpret_cast<const uint2*>(a.codes + row * a.padded + col));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t w = (k < 2 ? c.x : c.y) >> (16 * (k & 1));
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w & 0xffff), __NV_E4M3);
                const float2 f = __half22float2(__half2(h));
                v[2 * k] = f.x * s, v[2 * k + 1] = f.y * s;
            }
        } else {
            const uint32_t c = __ldcs(reinterpret_cast<const uint32_t*>(a.codes + (row * a.padded + col) / 2));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __half2_raw h =
                    __nv_cvt_fp4x2_to_halfraw2(__nv_fp4x2_storage_t(c >> (8 * k) & 0xff), __NV_E2M1);
                const float2 f = __half22float2(__half2(h));
                v[2 * k] = f.x * s, v[2 * k + 1] = f.y * s;
            }
        }
        if (a.vector_ok) {
            store8(out + col, v);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (col + k < a.cols) store1(out + col + k, v[k]);
        }
    }
}

// Threads per row: the least power of two that covers its units of eight columns, at
// most a block.
int threads_per_row(int64_t units) {
    int t = 16;
    while (t < kThreads && t < units) t *= 2;
    return t;
}

bool vectors_fit(const void* p, int64_t cols, int64_t stride, size_t es) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && cols % 8 == 0 && (stride * int64_t(es)) % 16 == 0;
}

}  // namespace

vce_status launch_mx_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t stride, int fmt,
                              uint8_t* codes, uint8_t* scales, int* dev_status, cudaStream_t s) {
    if (rows == 0) return VCE_OK;
    QuantArgs a{x, rows, cols, stride, mx::padded(cols), mx::padded(rows), codes, scales, 0, 0, dev_status};
    a.vector_ok = vectors_fit(x, cols, stride, dtype == VCE_BF16 ? 2 : 4);
    a.tpr = threads_per_row(a.padded / 8);
    const int per = kThreads / a.tpr;
    const unsigned g = unsigned((a.rows_padded + per - 1) / per);
    count_launch();
    if (dtype == VCE_BF16) {
        if (fmt == VCE_MX_E4M3) mx_quantize_kernel<__nv_bfloat16, VCE_MX_E4M3><<<g, kThreads, 0, s>>>(a);
        else mx_quantize_kernel<__nv_bfloat16, VCE_MX_E2M1><<<g, kThreads, 0, s>>>(a);
    } else {
        if (fmt == VCE_MX_E4M3) mx_quantize_kernel<float, VCE_MX_E4M3><<<g, kThreads, 0, s>>>(a);
        else mx_quantize_kernel<float, VCE_MX_E2M1><<<g, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

vce_status launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int fmt, int64_t rows, int64_t cols,
                                void* out, int dtype, int64_t stride, int* dev_status, cudaStream_t s) {
    if (rows == 0) return VCE_OK;
    DequantArgs a{codes, scales, rows, cols, stride, mx::padded(cols), out, 0, 0, dev_status};
    a.vector_ok = vectors_fit(out, cols, stride, dtype == VCE_BF16 ? 2 : 4);
    a.tpr = threads_per_row((cols + 7) / 8);
    const int per = kThreads / a.tpr;
    const unsigned g = unsigned((rows + per - 1) / per);
    count_launch();
    if (dtype == VCE_BF16) {
        if (fmt == VCE_MX_E4M3) mx_dequantize_kernel<__nv_bfloat16, VCE_MX_E4M3><<<g, kThreads, 0, s>>>(a);
        else mx_dequantize_kernel<__nv_bfloat16, VCE_MX_E2M1><<<g, kThreads, 0, s>>>(a);
    } else {
        if (fmt == VCE_MX_E4M3) mx_dequantize_kernel<float, VCE_MX_E4M3><<<g, kThreads, 0, s>>>(a);
        else mx_dequantize_kernel<float, VCE_MX_E2M1><<<g, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

}  // namespace vce
