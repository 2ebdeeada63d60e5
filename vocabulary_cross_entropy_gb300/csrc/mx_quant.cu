// Quantisation of a BF16 or FP32 matrix to microscaled E2M1 or E4M3, and back
// (mx_format.cuh has the formats).  Both are copies in what they cost: one thread
// takes eight consecutive columns, four neighbouring lanes share a block of 32 and
// find its largest magnitude with two shuffles.  65536 x 4096 BF16 to E2M1 125 us, back
// 109 us (680 MB each, 0.81 and 0.93 of the copy rate); instructions are the rest.

#include "head_internal.cuh"
#include "mx_format.cuh"

namespace vce {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

struct QuantArgs {
    const void* x;
    int64_t rows, cols, stride, padded, rows_padded;
    uint8_t *codes, *scales;
    int tpr;        // threads per row: a power of two, 16 .. kThreads
    int* dev_status;
};

// Eight columns as loaded.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void load_some(const float* p, int n) {  // the first n, then zeros
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < n ? p[k] : 0.f;
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
};
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int n) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = (2 * k < n ? uint32_t(q[2 * k]) : 0u) | (2 * k + 1 < n ? uint32_t(q[2 * k + 1]) : 0u) << 16;
        a = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
};

// One thread per eight columns and step, kUnroll steps loaded ahead; ``tpr`` threads walk
// one row.  The grid covers the scale rows that fill the last tile too.
template <typename T, int kFmt, bool kVector>
__global__ void __launch_bounds__(kThreads) mx_quantize_kernel(const QuantArgs a) {
    const int units = int(a.padded / 8);  // per row, a multiple of 16: half warps share a scale tile
    const int64_t row = int64_t(blockIdx.x) * (kThreads / a.tpr) + threadIdx.x / a.tpr;
    if (row >= a.rows_padded) return;
    const int cols = row < a.rows ? int(a.cols) : 0;
    const T* x = static_cast<const T*>(a.x) + (cols ? row : 0) * a.stride;
    uint8_t* codes = a.codes + row * (kFmt == VCE_MX_E4M3 ? a.padded : a.padded / 2);
    uint8_t* scales = a.scales + mx::scale_offset(row, 0, a.padded / mx::kColTile);
    const unsigned lanes = 0xffffu << (threadIdx.x & 16);
    for (int u0 = threadIdx.x % a.tpr; u0 < units; u0 += kUnroll * a.tpr) {  // whole half warps
        Raw8<T> raw[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int col = (u0 + k * a.tpr) * 8;
            if (kVector && col < cols) raw[k].load(x + col);
            else raw[k].load_some(x + col, kVector ? 0 : cols - col);
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int u = u0 + k * a.tpr, col = u * 8;
            if (u >= units) break;
            float v[8];
            raw[k].get(v);
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = mx::max_abs(top, v[i]);
            uint32_t m = __float_as_uint(top);  // bits order magnitudes, a NaN above all
            m = max(m, __shfl_xor_sync(lanes, m, 1));
            m = max(m, __shfl_xor_sync(lanes, m, 2));
            const uint32_t sb = mx::scale_byte<kFmt>(m);
            const bool bad = sb == mx::kNanScale;
            const float inv = mx::inverse_scale(bad ? 0u : sb);
            // the four scales of a tile's row as one word
            uint32_t word = sb | __shfl_down_sync(lanes, sb, 4, 16) << 8;
            word |= __shfl_down_sync(lanes, word, 8, 16) << 16;
            if ((threadIdx.x & 15) == 0 && VCE_BOUNDS(col % mx::kColTile == 0 && col < a.padded, a.dev_status))
                *reinterpret_cast<uint32_t*>(scales + (col / mx::kColTile) * mx::kTileBytes) = word;
            if (row >= a.rows || !VCE_BOUNDS(row >= 0 && col + 8 <= a.padded, a.dev_status)) continue;
            if (kFmt == VCE_MX_E4M3) {
                uint32_t c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) c[i] = mx::e4m3x2(v[2 * i] * inv, v[2 * i + 1] * inv);
                const uint2 w = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
                *reinterpret_cast<uint2*>(codes + col) = bad ? make_uint2(0, 0) : w;
            } else {
                uint32_t c = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) c |= mx::e2m1x2(v[2 * i] * inv, v[2 * i + 1] * inv) << (8 * i);
                *reinterpret_cast<uint32_t*>(codes + col / 2) = bad ? 0u : c;
            }
        }
    }
}

struct DequantArgs {
    const uint8_t *codes, *scales;
    int64_t rows, cols, stride, padded;
    void* out;
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
    const int cols = int(a.cols), units = (cols + 7) / 8;
    const int64_t row = int64_t(blockIdx.x) * (kThreads / a.tpr) + threadIdx.x / a.tpr;
    if (row >= a.rows) return;
    const uint8_t* codes = a.codes + row * (kFmt == VCE_MX_E4M3 ? a.padded : a.padded / 2);
    const uint8_t* scales = a.scales + mx::scale_offset(row, 0, a.padded / mx::kColTile);
    T* out = static_cast<T*>(a.out) + row * a.stride;
    for (int u0 = threadIdx.x % a.tpr; u0 < units; u0 += kUnroll * a.tpr) {
        uint2 c[kUnroll];
        uint32_t sb[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int u = u0 + k * a.tpr, col = u * 8;
            if (u >= units || !VCE_BOUNDS(row >= 0 && col + 8 <= a.padded, a.dev_status)) break;
            if (kFmt == VCE_MX_E4M3) c[k] = __ldcs(reinterpret_cast<const uint2*>(codes + col));
            else c[k].x = __ldcs(reinterpret_cast<const uint32_t*>(codes + col / 2));
            sb[k] = scales[(col / mx::kColTile) * mx::kTileBytes + (col / mx::kBlock & 3)];
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int u = u0 + k * a.tpr, col = u * 8;
            if (u >= units || !VCE_BOUNDS(row >= 0 && col + 8 <= a.padded, a.dev_status)) break;
            const float s = mx::scale_value(sb[k]);
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 q =
                    kFmt == VCE_MX_E4M3 ? mx::decode_pair<kFmt>((i < 2 ? c[k].x : c[k].y) >> (16 * (i & 1)) & 0xffffu)
                                        : mx::decode_pair<kFmt>(c[k].x >> (8 * i) & 0xffu);
                v[2 * i] = q.x * s;  // exact but for results below 2^-126
                v[2 * i + 1] = q.y * s;
            }
            store8(out + col, v);
        }
    }
}

// Rows that do not allow 16-byte stores: one column per lane, a warp to a block of 32, so
// that stores stay neighbours (16000 x 4097 BF16: 176 us with eight columns per thread,
// 91 this way; the loads of the quantisation do better with eight, 68 against 113 us).
template <typename T, int kFmt>
__global__ void __launch_bounds__(kThreads) mx_dequantize_odd_kernel(const DequantArgs a) {
    const int lane = threadIdx.x & 31, warps = a.tpr / 32;
    const int cols = int(a.cols), blocks = (cols + mx::kBlock - 1) / mx::kBlock;
    const int64_t row = int64_t(blockIdx.x) * (kThreads / a.tpr) + threadIdx.x / a.tpr;
    if (row >= a.rows) return;
    const uint8_t* codes = a.codes + row * (kFmt == VCE_MX_E4M3 ? a.padded : a.padded / 2);
    const uint8_t* scales = a.scales + mx::scale_offset(row, 0, a.padded / mx::kColTile);
    T* out = static_cast<T*>(a.out) + row * a.stride;
    for (int b0 = (threadIdx.x % a.tpr) / 32 * 4; b0 < blocks; b0 += warps * 4) {
        uint32_t c[4];
        const uint32_t word = *reinterpret_cast<const uint32_t*>(scales + (b0 >> 2) * mx::kTileBytes);
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // (codes are padded to whole scale tiles)
            const int col = (b0 + k) * mx::kBlock + lane;
            if (!VCE_BOUNDS(col < a.padded, a.dev_status)) continue;
            c[k] = kFmt == VCE_MX_E4M3 ? codes[col] : (codes[col / 2] >> (4 * (lane & 1))) & 0xfu;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int col = (b0 + k) * mx::kBlock + lane;
            if (col < cols) store1(out + col, mx::decode_pair<kFmt>(c[k]).x * mx::scale_value(word >> (8 * k) & 0xffu));
        }
    }
}

// Threads per row: few enough that a thread has several units of eight columns over
// which its set-up is spread (two units per thread took 1.6 times as long as eight at
// 4096 columns: the kernels were bound by instructions), at least the half warp that
// shares a scale tile.
int threads_per_row(int64_t units, int least = 16) {
    int t = least;
    while (t < kThreads && t * 8 < units) t *= 2;
    return t;
}

bool vectors_fit(const void* p, int64_t cols, int64_t stride, size_t es) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && cols % 8 == 0 && (stride * int64_t(es)) % 16 == 0;
}

template <typename T, int kFmt>
void quantize(const QuantArgs& a, bool vector, unsigned grid, cudaStream_t s) {
    if (vector) mx_quantize_kernel<T, kFmt, true><<<grid, kThreads, 0, s>>>(a);
    else mx_quantize_kernel<T, kFmt, false><<<grid, kThreads, 0, s>>>(a);
}

template <typename T, int kFmt>
void dequantize(const DequantArgs& a, bool vector, unsigned grid, cudaStream_t s) {
    if (vector) mx_dequantize_kernel<T, kFmt><<<grid, kThreads, 0, s>>>(a);
    else mx_dequantize_odd_kernel<T, kFmt><<<grid, kThreads, 0, s>>>(a);
}

}  // namespace

vce_status launch_mx_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t stride, int fmt,
                              uint8_t* codes, uint8_t* scales, int* dev_status, cudaStream_t s) {
    if (rows == 0) return VCE_OK;
    const int64_t padded = mx::padded(cols);
    const bool vec = vectors_fit(x, cols, stride, dtype == VCE_BF16 ? 2 : 4);
    const QuantArgs a{x, rows, cols, stride, padded, mx::padded(rows), codes, scales, threads_per_row(padded / 8),
                      dev_status};
    const int per = kThreads / a.tpr;
    const unsigned g = unsigned((a.rows_padded + per - 1) / per);
    count_launch();
    if (dtype == VCE_BF16) {
        if (fmt == VCE_MX_E4M3) quantize<__nv_bfloat16, VCE_MX_E4M3>(a, vec, g, s);
        else quantize<__nv_bfloat16, VCE_MX_E2M1>(a, vec, g, s);
    } else {
        if (fmt == VCE_MX_E4M3) quantize<float, VCE_MX_E4M3>(a, vec, g, s);
        else quantize<float, VCE_MX_E2M1>(a, vec, g, s);
    }
    return cudaGetLastError() == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

vce_status launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int fmt, int64_t rows, int64_t cols,
                                void* out, int dtype, int64_t stride, int* dev_status, cudaStream_t s) {
    if (rows == 0) return VCE_OK;
    const bool vec = vectors_fit(out, cols, stride, dtype == VCE_BF16 ? 2 : 4);
    const DequantArgs a{codes, scales, rows, cols, stride, mx::padded(cols), out, threads_per_row((cols + 7) / 8, vec ? 16 : 32),
                        dev_status};
    const int per = kThreads / a.tpr;
    const unsigned g = unsigned((rows + per - 1) / per);
    count_launch();
    if (dtype == VCE_BF16) {
        if (fmt == VCE_MX_E4M3) dequantize<__nv_bfloat16, VCE_MX_E4M3>(a, vec, g, s);
        else dequantize<__nv_bfloat16, VCE_MX_E2M1>(a, vec, g, s);
    } else {
        if (fmt == VCE_MX_E4M3) dequantize<float, VCE_MX_E4M3>(a, vec, g, s);
        else dequantize<float, VCE_MX_E2M1>(a, vec, g, s);
    }
    return cudaGetLastError() == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

}  // namespace vce
