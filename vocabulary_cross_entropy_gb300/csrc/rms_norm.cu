// Root-mean-square norm of hidden states with the residual's addition, its 8-bit
// microscaled form, and its backward pass.
//
//   h = round(x + residual)      (h = x without a residual)
//   r = 1 / sqrt(mean_i h_i^2 + eps)
//   y_i = h_i r w_i
//
//   g_i = w_i dy_i,  c = r^2 mean_i (g_i h_i)
//   dx_i = r (g_i - h_i c) + dh_i  (the gradient of x and of the residual)
//   dw_i = sum over rows of dy_i h_i r
//
// The norm is taken of the rounded sum, the value the caller keeps as the residual
// stream, so that the backward pass differentiates the very numbers the forward
// pass used.  All arithmetic and every sum is FP32; the one rounding to fewer bits
// besides h is the store of y (dx, dw).
//
// All three are bound by memory: a row is read once into registers, reduced over
// its threads and written from registers.  16384 x 4096 BF16 with a residual (537 MB, 80 us
// at the copy rate): forward 82 us, backward 99 us.  The 8-bit form is bound by
// instructions (54 us without a residual, 202 MB).

#include "head_internal.cuh"
#include "mx_format.cuh"

#include <math.h>
#include <algorithm>
#include <initializer_list>
#include <mutex>
#include <utility>

namespace vce {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kRingThreads = 1024;  // (64 registers)

template <typename T, int VE>
struct alignas(sizeof(T) * VE) Vec {
    T e[VE];
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// A vector's values as FP32, and back (BF16: two values per conversion instruction).
template <int VE>
__device__ __forceinline__ void unpack(const Vec<float, VE>& v, float (&f)[VE]) {
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = v.e[i];
}
template <int VE>
__device__ __forceinline__ void unpack(const Vec<__nv_bfloat16, VE>& v, float (&f)[VE]) {
    if constexpr (VE == 1) {
        f[0] = to_f(v.e[0]);
    } else {
        const uint32_t* u = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
}
template <int VE>
__device__ __forceinline__ void pack(const float (&f)[VE], Vec<float, VE>& v) {
#pragma unroll
    for (int i = 0; i < VE; ++i) v.e[i] = f[i];
}
template <int VE>
__device__ __forceinline__ void pack(const float (&f)[VE], Vec<__nv_bfloat16, VE>& v) {
    if constexpr (VE == 1) {
        v.e[0] = __float2bfloat16_rn(f[0]);
    } else {
        uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
    }
}

template <int VE>
__device__ __forceinline__ void load_weight(const void* w, int w_f32, int64_t at, float (&out)[VE]) {
    if (w_f32) {
        if constexpr (VE == 8) {  // two 16-byte loads
            const Vec<float, 4> a = *reinterpret_cast<const Vec<float, 4>*>(static_cast<const float*>(w) + at);
            const Vec<float, 4> b = *reinterpret_cast<const Vec<float, 4>*>(static_cast<const float*>(w) + at + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i] = a.e[i], out[i + 4] = b.e[i];
        } else {
            const Vec<float, VE> a = *reinterpret_cast<const Vec<float, VE>*>(static_cast<const float*>(w) + at);
#pragma unroll
            for (int i = 0; i < VE; ++i) out[i] = a.e[i];
        }
    } else {
        const Vec<__nv_bfloat16, VE> a =
            *reinterpret_cast<const Vec<__nv_bfloat16, VE>*>(static_cast<const __nv_bfloat16*>(w) + at);
        unpack<VE>(a, out);
    }
}

// Sum over the ``tpr`` threads of a row (a warp, or the whole block); every thread
// gets it.  ``slot`` holds one float per warp and is not reused before the next barrier.
__device__ __forceinline__ float row_sum(float v, int tpr, float* slot) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr == 32) return v;
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
    __syncthreads();
    const int warps = tpr >> 5;
    v = (threadIdx.x & 31) < warps ? slot[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct NormArgs {
    const void *x, *residual, *weight;
    int w_f32;
    int64_t n, hidden, x_stride, r_stride, h_stride, y_stride;
    float eps;
    void *h, *y;
    float* rstd;
    uint8_t *codes, *scales;  // 8-bit form: [n, padded], scale tiles
    int64_t padded, rows_padded;
    int tpr;  // threads per row: 32, or the block
    int* dev_status;
};

// The 8-bit form's stores of VE consecutive values at column ``col`` (a multiple of
// VE) of the row whose codes and scales start at ``codes`` and ``scales``.  The 32 / VE
// lanes that hold one block find its largest magnitude together; every lane of the
// warp calls.
template <int VE>
__device__ __forceinline__ void store_mx(const NormArgs& a, uint8_t* codes, uint8_t* scales, int col,
                                         const float (&y)[VE]) {
    constexpr int kLanes = mx::kBlock / VE;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < VE; ++i) top = mx::max_abs(top, y[i]);
    uint32_t m = __float_as_uint(top);
    if constexpr (kLanes == 32) {
        m = __reduce_max_sync(0xffffffffu, m);
    } else {
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    const uint32_t sb = mx::scale_byte<VCE_MX_E4M3>(m);
    const bool bad = sb == mx::kNanScale;
    const float inv = mx::inverse_scale(bad ? 0u : sb);
    uint32_t word = sb;
    if constexpr (VE >= 4) {  // a warp holds whole scale tiles: four scales to a word
        word |= __shfl_down_sync(0xffffffffu, word, kLanes) << 8;
        word |= __shfl_down_sync(0xffffffffu, word, 2 * kLanes) << 16;
    }
    if (col >= a.padded || !VCE_BOUNDS(col >= 0 && col + VE <= a.padded, a.dev_status)) return;
    uint8_t* dst = codes + col;
    if constexpr (VE == 1) {
        *dst = bad ? 0 : uint8_t(mx::e4m3x2(y[0] * inv, 0.f) & 0xff);
    } else {
        uint32_t c[VE / 2];
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) c[i] = bad ? 0 : mx::e4m3x2(y[2 * i] * inv, y[2 * i + 1] * inv);
        if constexpr (VE == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
        else if constexpr (VE == 4) *reinterpret_cast<uint32_t*>(dst) = c[0] | c[1] << 16;
        else *reinterpret_cast<uint16_t*>(dst) = uint16_t(c[0]);
    }
    uint8_t* at = scales + (col / mx::kColTile) * mx::kTileBytes;
    if (VE >= 4) {
        if (col % mx::kColTile == 0) *reinterpret_cast<uint32_t*>(at) = word;
    } else if (col % mx::kBlock == 0) {
        at[col / mx::kBlock & 3] = uint8_t(sb);
    }
}

// Scales of the rows past the last one in the last tile.
__device__ __forceinline__ void zero_scale_row(const NormArgs& a, int64_t row, int t, int tpr) {
    for (int64_t b = t; b < a.padded / mx::kBlock; b += tpr)
        a.scales[mx::scale_offset(row, b, a.padded / mx::kColTile)] = 0;
}

// One row per ``tpr`` threads, NV vectors of VE elements per thread in registers.
template <typename T, int VE, int NV, bool kMx>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_rows(const NormArgs a) {
    uint8_t *codes = nullptr, *scales = nullptr;
    __shared__ float slot[32];
    const int tpr = a.tpr;
    const int t = threadIdx.x % tpr;
    const int64_t row = int64_t(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
    if (kMx && row >= a.n) {  // (whole warps: a row's threads are whole warps)
        if (row < a.rows_padded) zero_scale_row(a, row, t, tpr);
        return;
    }
    if (row >= a.n) return;
    if (kMx) {
        codes = a.codes + row * a.padded;
        scales = a.scales + mx::scale_offset(row, 0, a.padded / mx::kColTile);
    }
    using V = Vec<T, VE>;
    const int hidden = int(a.hidden);
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.r_stride : nullptr;
    T* h = a.residual ? static_cast<T*>(a.h) + row * a.h_stride : nullptr;
    V v[NV], u[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (j * tpr + t) * VE;
        if (col < hidden) v[j] = *reinterpret_cast<const V*>(x + col);
    }
    if (res) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * tpr + t) * VE;
            if (col < hidden) u[j] = *reinterpret_cast<const V*>(res + col);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (j * tpr + t) * VE;
        if (col < hidden) {
            float f[VE];
            unpack<VE>(v[j], f);
            if (res) {
                float g[VE];
                unpack<VE>(u[j], g);
#pragma unroll
                for (int i = 0; i < VE; ++i) f[i] += g[i];
                pack<VE>(f, v[j]);
                unpack<VE>(v[j], f);
                if (VCE_BOUNDS(col >= 0 && col + VE <= a.hidden && row < a.n, a.dev_status))
                    *reinterpret_cast<V*>(h + col) = v[j];
            }
#pragma unroll
            for (int i = 0; i < VE; ++i) ss = fmaf(f[i], f[i], ss);
        }
    }
    ss = row_sum(ss, tpr, slot);
    const float r = __frsqrt_rn(ss / float(a.hidden) + a.eps);
    if (t == 0 && a.rstd) a.rstd[row] = r;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (j * tpr + t) * VE;
        float y[VE];
        if (col < hidden) {
            float f[VE];
            load_weight<VE>(a.weight, a.w_f32, col, y);
            unpack<VE>(v[j], f);
#pragma unroll
            for (int i = 0; i < VE; ++i) y[i] = f[i] * r * y[i];
            if (!kMx) {
                V o;
                pack<VE>(y, o);
                if (VCE_BOUNDS(col >= 0 && col + VE <= a.hidden && row < a.n, a.dev_status))
                    *reinterpret_cast<V*>(static_cast<T*>(a.y) + row * a.y_stride + col) = o;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i) y[i] = 0.f;
        }
        if constexpr (kMx) store_mx<VE>(a, codes, scales, col, y);
    }
}

// Rows that start off 16-byte boundaries, at the same offset in all operands: the block's rows
// are a multiple of VE rows apart, so that they share the offset ``off`` and the weight can be
// laid out by it in shared memory; vector v holds columns v VE - off ....  The first and the
// last one hold elements of the neighbouring rows too, which are masked (the tensor's own
// first and last bytes are loaded one by one).
template <typename T, int NV>
__global__ void __launch_bounds__(kMaxThreads, 2) rms_norm_rows_shift(const NormArgs a) {
    constexpr int VE = 16 / sizeof(T);
    using V = Vec<T, VE>;
    extern __shared__ __align__(16) float shift_smem[];
    float* slots = shift_smem;    // [2][32]
    float* sw = shift_smem + 64;  // [vectors][VE]
    const int t = threadIdx.x, tpr = blockDim.x, hidden = int(a.hidden);
    const int off = int(reinterpret_cast<uintptr_t>(static_cast<const T*>(a.x) + blockIdx.x * a.x_stride) / sizeof(T) % VE);
    for (int i = t; i < (hidden + off + VE - 1) / VE * VE; i += tpr) {
        float w[1] = {0.f};
        if (i >= off && i - off < hidden) load_weight<1>(a.weight, a.w_f32, i - off, w);
        sw[i] = w[0];
    }
    __syncthreads();
    auto load = [&](const T* src, int64_t row, int col) {
        V v;
        if ((row == 0 && col < 0) || (row == a.n - 1 && col + VE > hidden)) {
#pragma unroll
            for (int i = 0; i < VE; ++i) v.e[i] = from_f<T>(0.f);
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (uint32_t(col + i) < uint32_t(hidden)) v.e[i] = src[col + i];
        } else if (VCE_BOUNDS(aligned16(src + col), a.dev_status)) {
            v = *reinterpret_cast<const V*>(src + col);
        }
        return v;
    };
    auto store = [&](T* dst, int64_t row, int col, const V& v) {
        if (col >= 0 && col + VE <= hidden) {
            if (VCE_BOUNDS(aligned16(dst + col) && row < a.n, a.dev_status)) *reinterpret_cast<V*>(dst + col) = v;
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (uint32_t(col + i) < uint32_t(hidden)) dst[col + i] = v.e[i];
        }
    };
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
        const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.r_stride : nullptr;
        T* h = a.residual ? static_cast<T*>(a.h) + row * a.h_stride : nullptr;
        V v[NV], u[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * tpr + t) * VE - off;
            if (col < hidden) v[j] = load(x, row, col);
        }
        if (res) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int col = (j * tpr + t) * VE - off;
                if (col < hidden) u[j] = load(res, row, col);
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * tpr + t) * VE - off;
            if (col < hidden) {
                float f[VE];
                unpack<VE>(v[j], f);
                if (res) {
                    float g[VE];
                    unpack<VE>(u[j], g);
#pragma unroll
                    for (int i = 0; i < VE; ++i) f[i] += g[i];
                    pack<VE>(f, v[j]);
                    unpack<VE>(v[j], f);
                    store(h, row, col, v[j]);
                }
                if (col < 0 || col + VE > hidden) {
#pragma unroll
                    for (int i = 0; i < VE; ++i)
                        if (uint32_t(col + i) >= uint32_t(hidden)) f[i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < VE; ++i) ss = fmaf(f[i], f[i], ss);
            }
        }
        ss = row_sum(ss, tpr, slots + parity * 32);
        parity ^= 1;
        const float r = __frsqrt_rn(ss / float(a.hidden) + a.eps);
        if (t == 0 && a.rstd) a.rstd[row] = r;
        T* y = static_cast<T*>(a.y) + row * a.y_stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int vec = j * tpr + t, col = vec * VE - off;
            if (col < hidden) {
                float f[VE];
                unpack<VE>(v[j], f);
#pragma unroll
                for (int i = 0; i < VE; ++i) f[i] = f[i] * r * sw[vec * VE + i];
                V o;
                pack<VE>(f, o);
                store(y, row, col, o);
            }
        }
    }
}

// Rows longer than the registers hold: two passes over the row, one block per row,
// one element per thread and step.  Each thread reads back only what it wrote.
template <typename T, bool kMx>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_long(const NormArgs a) {
    __shared__ float slot[32];
    const int64_t row = blockIdx.x;
    if (row >= a.n) {
        if (kMx && row < a.rows_padded) zero_scale_row(a, row, threadIdx.x, blockDim.x);
        return;
    }
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.r_stride : nullptr;
    T* h = a.residual ? static_cast<T*>(a.h) + row * a.h_stride : nullptr;
    float ss = 0.f, comp = 0.f;  // compensated: one thread adds many terms
    for (int64_t col = threadIdx.x; col < a.hidden; col += blockDim.x) {
        T v = x[col];
        if (res) {
            v = from_f<T>(to_f(v) + to_f(res[col]));
            h[col] = v;
        }
        const float q = fmaf(to_f(v), to_f(v), -comp);
        const float s = ss + q;
        comp = (s - ss) - q;
        ss = s;
    }
    ss = row_sum(ss, blockDim.x, slot);
    const float r = __frsqrt_rn(ss / float(a.hidden) + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[row] = r;
    const T* src = res ? h : x;
    const int64_t end = kMx ? a.padded : a.hidden;  // both passes give a thread the same columns
    uint8_t* codes = a.codes + row * a.padded;
    uint8_t* scales = a.scales + mx::scale_offset(row, 0, a.padded / mx::kColTile);
    for (int64_t c0 = 0; c0 < end; c0 += blockDim.x) {
        const int64_t col = c0 + threadIdx.x;
        float y[1] = {0.f}, w[1];
        if (col < a.hidden) {
            load_weight<1>(a.weight, a.w_f32, col, w);
            y[0] = to_f(src[col]) * r * w[0];
            if (!kMx) static_cast<T*>(a.y)[row * a.y_stride + col] = from_f<T>(y[0]);
        }
        if constexpr (kMx) store_mx<1>(a, codes, scales, int(col), y);
    }
}

struct NormBwdArgs {
    const void *dy, *h, *weight, *dh;
    const float* rstd;
    int w_f32;
    int64_t n, hidden, dy_stride, h_stride, dh_stride, dx_stride;
    void* dx;
    float* part;  // [parts][hidden] partial sums of dw
    int parts;
    int tpr;
    int* dev_status;
};

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...: a thread keeps the same columns for
// all of them and sums their dw in registers; the block writes one partial row.
template <typename T, int VE, int NV>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_backward_rows(const NormBwdArgs a) {
    extern __shared__ float smem[];  // [2][32] reduction slots, then [hidden] (several rows per block)
    using V = Vec<T, VE>;
    const int tpr = a.tpr, groups = blockDim.x / tpr;
    const int t = threadIdx.x % tpr, g = threadIdx.x / tpr;
    float acc[NV][VE];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VE; ++i) acc[j][i] = 0.f;
    int parity = 0;
    const float inv_h = 1.f / float(a.hidden);
    for (int64_t row = int64_t(blockIdx.x) * groups + g; row < a.n; row += int64_t(gridDim.x) * groups) {
        const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
        const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
        const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.dh_stride : nullptr;
        T* dx = static_cast<T*>(a.dx) + row * a.dx_stride;
        V vg[NV], vh[NV], ve[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * tpr + t) * VE;
            if (col < a.hidden) {
                vg[j] = *reinterpret_cast<const V*>(dy + col);
                vh[j] = *reinterpret_cast<const V*>(h + col);
                if (dh) ve[j] = *reinterpret_cast<const V*>(dh + col);
            }
        }
        const float r = a.rstd[row];
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * tpr + t) * VE;
            if (col < a.hidden) {
                float w[VE], d[VE], f[VE];
                load_weight<VE>(a.weight, a.w_f32, col, w);
                unpack<VE>(vg[j], d);
                unpack<VE>(vh[j], f);
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const float hat = f[i] * r;
                    acc[j][i] = fmaf(d[i], hat, acc[j][i]);
                    s = fmaf(d[i] * w[i], hat, s);
                }
            }
        }
        s = row_sum(s, tpr, smem + parity * 32) * inv_h;
        parity ^= 1;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * tpr + t) * VE;
            if (col < a.hidden) {
                float w[VE], d[VE], f[VE];
                load_weight<VE>(a.weight, a.w_f32, col, w);
                unpack<VE>(vg[j], d);
                unpack<VE>(vh[j], f);
#pragma unroll
                for (int i = 0; i < VE; ++i) d[i] = r * (d[i] * w[i] - f[i] * r * s);
                if (dh) {
                    unpack<VE>(ve[j], f);
#pragma unroll
                    for (int i = 0; i < VE; ++i) d[i] += f[i];
                }
                V o;
                pack<VE>(d, o);
                if (VCE_BOUNDS(col >= 0 && col + VE <= a.hidden && row < a.n, a.dev_status))
                    *reinterpret_cast<V*>(dx + col) = o;
            }
        }
    }
    float* out = a.part + int64_t(blockIdx.x) * a.hidden;
    if (groups == 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * tpr + t) * VE;
            if (col < a.hidden && VCE_BOUNDS(int(blockIdx.x) < a.parts, a.dev_status))
#pragma unroll
                for (int i = 0; i < VE; ++i) out[col + i] = acc[j][i];
        }
        return;
    }
    float* sum = smem + 64;  // the block's row groups add theirs in turn: a fixed order
    for (int k = 0; k < groups; ++k) {
        if (g == k) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int col = (j * tpr + t) * VE;
                if (col < a.hidden)
#pragma unroll
                    for (int i = 0; i < VE; ++i) sum[col + i] = (k == 0 ? 0.f : sum[col + i]) + acc[j][i];
            }
        }
        __syncthreads();
    }
    for (int64_t c = threadIdx.x; c < a.hidden; c += blockDim.x)
        if (VCE_BOUNDS(int(blockIdx.x) < a.parts, a.dev_status)) out[c] = sum[c];
}

__device__ __forceinline__ void copy16_async(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}

// The same with rows of one block each read by 16 bytes, the loads of the next kStages - 1
// rows in flight: a thread copies its own vectors to its own slots of shared memory and
// reads them back itself, so the ring needs no barrier.
//   kShift: rows that start anywhere, at the same offset from a 16-byte boundary in all
// operands.  A block's rows are a multiple of VE rows apart, so that they share one offset
// ``off`` and a thread keeps its columns; vector v holds columns v VE - off ....  The first and
// the last vector of a row hold elements of its neighbours too, which are masked; where there
// is no neighbour (the tensor's own first and last bytes) the elements are loaded one by one.
// The weight is laid out by the same offset in shared memory.
template <typename T, int NV, int kStages, bool kShift>
__global__ void __launch_bounds__(kRingThreads) rms_norm_backward_ring(const NormBwdArgs a) {
    constexpr int VE = 16 / sizeof(T);
    using V = Vec<T, VE>;
    extern __shared__ __align__(16) uint8_t ring_raw[];
    float* slots = reinterpret_cast<float*>(ring_raw);  // [2][32]
    float* sw = slots + 64;                             // kShift: [vectors][VE]
    const int t = threadIdx.x, tpr = blockDim.x, streams = a.dh ? 3 : 2, hidden = int(a.hidden);
    const int off = kShift ? int(reinterpret_cast<uintptr_t>(static_cast<const T*>(a.dy) + blockIdx.x * a.dy_stride) /
                                 sizeof(T) % VE)
                           : 0;
    V* ring = reinterpret_cast<V*>(kShift ? sw + (hidden + 2 * VE - 1) / VE * VE : sw);  // [kStages][streams][NV][threads]
    const int stage_vecs = streams * NV * tpr;
    if constexpr (kShift) {
        for (int i = t; i < (hidden + off + VE - 1) / VE * VE; i += tpr) {
            float w[1] = {0.f};
            if (i >= off && i - off < hidden) load_weight<1>(a.weight, a.w_f32, i - off, w);
            sw[i] = w[0];
        }
        __syncthreads();
    }
    float acc[NV][VE];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VE; ++i) acc[j][i] = 0.f;
    auto whole = [&](int col) { return !kShift || (col >= 0 && col + VE <= hidden); };
    // one vector of an operand to its slot
    auto copy = [&](V* dst, const void* base, int64_t stride, int64_t row, int col) {
        const T* src = static_cast<const T*>(base) + row * stride + col;
        if (kShift && ((row == 0 && col < 0) || (row == a.n - 1 && col + VE > hidden))) {
            V v;
#pragma unroll
            for (int i = 0; i < VE; ++i) v.e[i] = from_f<T>(0.f);
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (uint32_t(col + i) < uint32_t(hidden)) v.e[i] = src[i];
            *dst = v;
        } else if (VCE_BOUNDS(aligned16(src), a.dev_status)) {
            copy16_async(dst, src);
        }
    };
    auto prefetch = [&](int64_t row, int stage) {
        if (row < a.n) {
            V* dst = ring + stage * stage_vecs + t;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int col = (j * tpr + t) * VE - off;
                if (col < hidden) {
                    copy(dst + j * tpr, a.dy, a.dy_stride, row, col);
                    copy(dst + (NV + j) * tpr, a.h, a.h_stride, row, col);
                    if (streams == 3) copy(dst + (2 * NV + j) * tpr, a.dh, a.dh_stride, row, col);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");  // one group per row, empty past the end
    };
    // a vector's dy, h and weight, zeros outside the row
    auto load = [&](const V* src, int j, int col, float (&d)[VE], float (&f)[VE], float (&w)[VE]) {
        if constexpr (kShift) {
#pragma unroll
            for (int i = 0; i < VE; ++i) w[i] = sw[(j * tpr + t) * VE + i];
        } else {
            load_weight<VE>(a.weight, a.w_f32, col, w);
        }
        unpack<VE>(src[j * tpr], d);
        unpack<VE>(src[(NV + j) * tpr], f);
        if (!whole(col)) {
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (uint32_t(col + i) >= uint32_t(hidden)) d[i] = f[i] = 0.f;
        }
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) prefetch(int64_t(blockIdx.x) + int64_t(s) * gridDim.x, s);
    const float inv_h = 1.f / float(a.hidden);
    int stage = 0, parity = 0;
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        // the slots of the row before this one have been read (by this thread)
        prefetch(row + int64_t(kStages - 1) * gridDim.x, stage == 0 ? kStages - 1 : stage - 1);
        const float r = a.rstd[row];
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        const V* src = ring + stage * stage_vecs + t;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * tpr + t) * VE - off;
            if (col < hidden) {
                float w[VE], d[VE], f[VE];
                load(src, j, col, d, f, w);
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const float hat = f[i] * r;
                    acc[j][i] = fmaf(d[i], hat, acc[j][i]);
                    s = fmaf(d[i] * w[i], hat, s);
                }
            }
        }
        s = row_sum(s, tpr, slots + parity * 32) * inv_h;
        parity ^= 1;
        T* dx = static_cast<T*>(a.dx) + row * a.dx_stride;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (j * tpr + t) * VE - off;
            if (col < hidden) {
                float w[VE], d[VE], f[VE];
                load(src, j, col, d, f, w);
#pragma unroll
                for (int i = 0; i < VE; ++i) d[i] = r * (d[i] * w[i] - f[i] * r * s);
                if (streams == 3) {
                    const V ve = src[(2 * NV + j) * tpr];
                    unpack<VE>(ve, f);
#pragma unroll
                    for (int i = 0; i < VE; ++i) d[i] += f[i];
                }
                V o;
                pack<VE>(d, o);
                if (whole(col)) {
                    if (VCE_BOUNDS(col >= 0 && col + VE <= hidden && row < a.n && aligned16(dx + col), a.dev_status))
                        *reinterpret_cast<V*>(dx + col) = o;
                } else {
#pragma unroll
                    for (int i = 0; i < VE; ++i)
                        if (uint32_t(col + i) < uint32_t(hidden)) dx[col + i] = o.e[i];
                }
            }
        }
        if (++stage == kStages) stage = 0;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    float* out = a.part + int64_t(blockIdx.x) * a.hidden;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (j * tpr + t) * VE - off;
        if (col < hidden && VCE_BOUNDS(int(blockIdx.x) < a.parts, a.dev_status))
#pragma unroll
            for (int i = 0; i < VE; ++i)
                if (!kShift || uint32_t(col + i) < uint32_t(hidden)) out[col + i] = acc[j][i];
    }
}

// Rows longer than the registers hold: dx by one block per row (after dw: dx may
// be written over dy) ...
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_backward_long(const NormBwdArgs a) {
    __shared__ float slot[32];
    const int64_t row = blockIdx.x;
    const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
    const T* h = static_cast<const T*>(a.h) + row * a.h_stride;
    const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.dh_stride : nullptr;
    const float r = a.rstd[row];
    float s = 0.f, comp = 0.f, w[1];
    for (int64_t col = threadIdx.x; col < a.hidden; col += blockDim.x) {
        load_weight<1>(a.weight, a.w_f32, col, w);
        const float q = fmaf(to_f(dy[col]) * w[0], to_f(h[col]) * r, -comp);
        const float n = s + q;
        comp = (n - s) - q;
        s = n;
    }
    s = row_sum(s, blockDim.x, slot) / float(a.hidden);
    for (int64_t col = threadIdx.x; col < a.hidden; col += blockDim.x) {
        load_weight<1>(a.weight, a.w_f32, col, w);
        float d = r * (to_f(dy[col]) * w[0] - to_f(h[col]) * r * s);
        if (dh) d += to_f(dh[col]);
        static_cast<T*>(a.dx)[row * a.dx_stride + col] = from_f<T>(d);
    }
}

// ... and dw by columns: block (x, y) sums rows y, y + parts, ... of 256 columns.
template <typename T>
__global__ void __launch_bounds__(256) rms_norm_dweight_long(const NormBwdArgs a) {
    const int64_t col = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (col >= a.hidden) return;
    float s = 0.f;
    for (int64_t row = blockIdx.y; row < a.n; row += a.parts)
        s = fmaf(to_f(static_cast<const T*>(a.dy)[row * a.dy_stride + col]),
                 to_f(static_cast<const T*>(a.h)[row * a.h_stride + col]) * a.rstd[row], s);
    a.part[int64_t(blockIdx.y) * a.hidden + col] = s;
}

// dw = the sum of the partial rows, in a fixed order: 32 columns per block, VE per thread,
// the partial rows dealt out to the threads that share columns, whose loads are then all on
// their way at once.  Launched so that it overlaps the end of the kernel before (16384 x 4096
// BF16 101 -> 99 us; started earlier than that kernel's last blocks, 2880 FP32 columns lost 6%).
template <int VE>
__global__ void __launch_bounds__(1024) rms_norm_dweight_sum(const float* __restrict__ part, int parts, int64_t hidden,
                                                             void* dw, int w_f32) {
    constexpr int kLanes = 32 / VE, kSplit = 1024 / kLanes;
    __shared__ float sm[kSplit][33];
    const int lc = threadIdx.x % kLanes, sp = threadIdx.x / kLanes;
    const int64_t col0 = int64_t(blockIdx.x) * 32, col = col0 + lc * VE;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for the partial rows
    float s[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) s[i] = 0.f;
    if (col < hidden) {
#pragma unroll 8
        for (int p = sp; p < parts; p += kSplit) {
            const Vec<float, VE> v = *reinterpret_cast<const Vec<float, VE>*>(part + int64_t(p) * hidden + col);
#pragma unroll
            for (int i = 0; i < VE; ++i) s[i] += v.e[i];
        }
    }
#pragma unroll
    for (int i = 0; i < VE; ++i) sm[sp][lc * VE + i] = s[i];
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;  // a warp per column
    float t = 0.f;
#pragma unroll
    for (int k = lane; k < kSplit; k += 32) t += sm[k][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane != 0 || col0 + warp >= hidden) return;
    if (w_f32) static_cast<float*>(dw)[col0 + warp] = t;
    else static_cast<__nv_bfloat16*>(dw)[col0 + warp] = __float2bfloat16_rn(t);
}

// Elements per access: the widest of the kernel's choices that divides the row length and
// every stride and to which every pointer is aligned.
int pick_ve(int full, int64_t hidden, size_t es, std::initializer_list<const void*> ptrs,
            std::initializer_list<int64_t> strides, const void* weight, int w_f32) {
    for (int ve : {full, 2}) {
        bool ok = hidden % ve == 0;
        for (const void* p : ptrs) ok = ok && reinterpret_cast<uintptr_t>(p) % (ve * es) == 0;
        for (int64_t s : strides) ok = ok && s % ve == 0;
        const size_t wa = w_f32 ? (ve * 4 > 16 ? 16 : ve * 4) : ve * 2;
        ok = ok && reinterpret_cast<uintptr_t>(weight) % wa == 0;
        if (ok) return ve;
    }
    return 1;
}

// Whether every row starts at the same offset from a 16-byte boundary as that of ``p``.
bool same_offset(size_t es, const void* p, int64_t stride,
                 std::initializer_list<std::pair<const void*, int64_t>> others) {
    bool same = true;
    for (const auto& o : others)
        same = same && (reinterpret_cast<uintptr_t>(o.first) ^ reinterpret_cast<uintptr_t>(p)) % 16 == 0 &&
               (o.second - stride) * int64_t(es) % 16 == 0;
    return same;
}

// threads in whole warps
int warps_for(int64_t x) { return x <= 32 ? 32 : int((x + 31) / 32 * 32); }

template <typename T, bool kMx>
vce_status norm_forward(NormArgs a, int ve, bool same_offset, cudaStream_t s, const DeviceInfo& dev) {
    constexpr int kFull = 16 / sizeof(T);
    // Rows off 16-byte boundaries by vectors all the same, with narrow accesses / this way, BF16:
    // 16000 x 4097 215 / 82 us, with a residual 249 / 138, 3035 x 2317 21 / 12.  Where accesses of
    // two elements are possible only long rows without a residual gain: 16000 x 4098 98 / 82, with
    // a residual 119 / 137, 16000 x 300 10.5 / 12.3.
    const bool gains = ve == 1 || (!a.residual && a.hidden >= 2048);
    if (!kMx && ve != kFull && same_offset && gains) {
        const int64_t wide = (a.hidden + 2 * kFull - 2) / kFull;  // vectors of a row, at most
        const int threads = warps_for((wide + 3) / 4);
        const size_t smem = (64 + size_t((a.hidden + 2 * kFull - 1) / kFull * kFull)) * sizeof(float);
        if (wide > 32 && threads <= kMaxThreads && smem <= 48 << 10) {
            // as many blocks as run at once (64 registers for each of 1024 threads)
            int64_t grid = dev.num_sms * std::min(int64_t((228 << 10) / (smem + 1024)), int64_t(1024 / threads));
            if (grid >= a.n) grid = a.n;
            else grid -= grid % kFull;  // a block's rows share their offset
            count_launch();
            rms_norm_rows_shift<T, 4><<<unsigned(grid), threads, smem, s>>>(a);
            return cudaGetLastError() == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
        }
    }
    const int64_t cols = kMx ? a.padded : a.hidden;
    const int64_t nvec = (cols + ve - 1) / ve;
    const int64_t rows = kMx ? a.rows_padded : a.n;
    count_launch();
    // Four vectors per thread keep enough loads in flight from few threads; with fewer
    // rows than fill the SMs, one vector per thread finishes a row sooner.
    int nv = a.n < 2 * dev.num_sms ? 1 : 4;
    if (ve != kFull) nv = 8;
    while (nv < 8 && nvec > int64_t(kMaxThreads) * nv) nv *= 2;
    if (nvec > int64_t(kMaxThreads) * nv) {
        rms_norm_long<T, kMx><<<unsigned(rows), kMaxThreads, 0, s>>>(a);
        return cudaGetLastError() == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
    }
    a.tpr = warps_for((nvec + nv - 1) / nv);
    const int block = a.tpr == 32 ? 128 : a.tpr;  // four rows of one warp each, or one row
    const unsigned grid = unsigned((rows + block / a.tpr - 1) / (block / a.tpr));
    if (ve == kFull) {
        if (nv == 1) rms_norm_rows<T, kFull, 1, kMx><<<grid, block, 0, s>>>(a);
        else if (nv == 2) rms_norm_rows<T, kFull, 2, kMx><<<grid, block, 0, s>>>(a);
        else if (nv == 4) rms_norm_rows<T, kFull, 4, kMx><<<grid, block, 0, s>>>(a);
        else rms_norm_rows<T, kFull, 8, kMx><<<grid, block, 0, s>>>(a);
    } else if (ve == 2) {
        rms_norm_rows<T, 2, 8, kMx><<<grid, block, 0, s>>>(a);
    } else {
        rms_norm_rows<T, 1, 8, kMx><<<grid, block, 0, s>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

constexpr int kRingStages = 2;
constexpr int kRingVecs = 2;                // vectors per thread
constexpr size_t kRingMost = 148 << 10;  // of shared memory per block

template <typename T, int NV, bool kShift>
vce_status launch_ring(const NormBwdArgs& a, int threads, size_t smem, cudaStream_t s, int device) {
    static std::mutex mu;
    static bool ready[64];
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!ready[device]) {
            if (cudaFuncSetAttribute(rms_norm_backward_ring<T, NV, kRingStages, kShift>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, int(kRingMost)) != cudaSuccess)
                return VCE_ERR_CUDA;
            ready[device] = true;
        }
    }
    count_launch();
    rms_norm_backward_ring<T, NV, kRingStages, kShift><<<a.parts, threads, smem, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

template <typename T>
vce_status norm_backward(NormBwdArgs a, int ve, bool same_offset, int& parts, cudaStream_t s, const DeviceInfo& dev) {
    constexpr int kFull = 16 / sizeof(T);
    constexpr int kNv = 32 / kFull;  // 32 sums of dw per thread
    const int64_t nvec = (a.hidden + ve - 1) / ve;
    int nv = ve == kFull ? kNv : 8;
    a.parts = parts;
    // The ring where a row is longer than 128 vectors and its stages fit: as many blocks as an
    // SM holds (and the workspace has partial rows for), so that all run at once.  Rows that
    // start off 16-byte boundaries, with narrow accesses / in the ring: 16000 x 4097 BF16 285 /
    // 121 us, 3035 x 2317 44 / 26, 16000 x 300 31 / 27.  Two stages: more blocks per SM beat
    // more stages (16384 x 4096 BF16, with the sum of partials: 104 us with two stages, 112 with
    // three, 127 with four).
    const bool shift = ve != kFull && same_offset;
    const int64_t wide = shift ? (a.hidden + 2 * kFull - 2) / kFull : nvec;  // vectors of a row, at most
    const int threads = warps_for((wide + kRingVecs - 1) / kRingVecs);
    const size_t ring = 64 * sizeof(float) + (shift ? size_t((a.hidden + 2 * kFull - 1) / kFull * kFull) * sizeof(float) : 0) +
                        size_t(kRingStages) * (a.dh ? 3 : 2) * kRingVecs * threads * 16;
    if (a.n > 0 && (ve == kFull || shift) && wide > (shift ? 32 : 128) && threads <= kRingThreads && ring <= kRingMost) {
        // resident at once: by shared memory, and by registers (64 for each of 1024 threads)
        const int64_t fit = int64_t(dev.num_sms) *
                            std::min(int64_t((228 << 10) / (ring + 1024)), int64_t(kRingThreads / threads));
        if (parts > fit) parts = int(fit);
        if (shift && parts < a.n) parts -= parts % kFull;  // a block's rows share their offset
        a.parts = parts;
        return shift ? launch_ring<T, kRingVecs, true>(a, threads, ring, s, dev.ordinal)
                     : launch_ring<T, kRingVecs, false>(a, threads, ring, s, dev.ordinal);
    }
    if (a.n > 0 && nvec > int64_t(kMaxThreads) * nv) {
        count_launch();  // dw first: dx may be written over dy
        rms_norm_dweight_long<T><<<dim3(unsigned((a.hidden + 255) / 256), unsigned(parts)), 256, 0, s>>>(a);
        count_launch();
        rms_norm_backward_long<T><<<unsigned(a.n), kMaxThreads, 0, s>>>(a);
    } else if (a.n > 0) {
        while (nv > 1 && nvec <= 32 * (nv / 2) && ve == kFull) nv /= 2;
        a.tpr = warps_for((nvec + nv - 1) / nv);
        const int block = a.tpr == 32 ? 128 : a.tpr;
        const size_t smem = 64 * sizeof(float) + (block == a.tpr ? 0 : size_t(a.hidden) * sizeof(float));
        count_launch();
        if (ve == kFull) {
            if (nv == kNv) rms_norm_backward_rows<T, kFull, kNv><<<parts, block, smem, s>>>(a);
            else if (nv == kNv / 2) rms_norm_backward_rows<T, kFull, kNv / 2><<<parts, block, smem, s>>>(a);
            else rms_norm_backward_rows<T, kFull, kNv / 4><<<parts, block, smem, s>>>(a);
        } else if (ve == 2) {
            rms_norm_backward_rows<T, 2, 8><<<parts, block, smem, s>>>(a);
        } else {
            rms_norm_backward_rows<T, 1, 8><<<parts, block, smem, s>>>(a);
        }
    }
    return cudaGetLastError() == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

}  // namespace

// Partial rows of dw, one per block: four blocks per SM, up to sixteen where rows are
// short and blocks small (four of 64 threads left most of an SM idle), but at most one
// per row.
int rms_norm_parts(int64_t n, int64_t hidden, int num_sms) {
    const int64_t most = int64_t(num_sms) * (hidden <= 1024 ? 16 : hidden <= 2048 ? 8 : 4);
    return int(n < most ? n : most);
}

vce_status launch_rms_norm(const void* x, const void* residual, const void* weight, int dtype, int w_dtype,
                           int64_t n, int64_t hidden, int64_t x_stride, int64_t r_stride, int64_t h_stride,
                           int64_t y_stride, float eps, void* h, void* y, float* rstd, uint8_t* codes,
                           uint8_t* scales, int* dev_status, cudaStream_t s, const DeviceInfo& dev) {
    if (n == 0) return VCE_OK;
    NormArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.w_f32 = w_dtype == VCE_F32;
    a.n = n; a.hidden = hidden; a.x_stride = x_stride; a.r_stride = r_stride; a.h_stride = h_stride;
    a.y_stride = y_stride; a.eps = eps; a.h = h; a.y = y; a.rstd = rstd; a.codes = codes; a.scales = scales;
    a.padded = mx::padded(hidden); a.rows_padded = mx::padded(n); a.dev_status = dev_status;
    const size_t es = dtype == VCE_BF16 ? 2 : 4;
    const void* any = x;  // absent operands do not limit the access width
    const bool same = same_offset(es, x, x_stride,
                                  {{residual ? residual : any, residual ? r_stride : x_stride},
                                   {residual ? h : any, residual ? h_stride : x_stride},
                                   {codes ? any : y, codes ? x_stride : y_stride}});
    const int ve = pick_ve(int(16 / es), hidden, es,
                           {x, residual ? residual : any, residual ? h : any, codes ? any : y},
                           {x_stride, residual ? r_stride : 0, residual ? h_stride : 0, codes ? 0 : y_stride},
                           weight, a.w_f32);
    if (dtype == VCE_BF16)
        return codes ? norm_forward<__nv_bfloat16, true>(a, ve, same, s, dev)
                     : norm_forward<__nv_bfloat16, false>(a, ve, same, s, dev);
    return codes ? norm_forward<float, true>(a, ve, same, s, dev) : norm_forward<float, false>(a, ve, same, s, dev);
}

vce_status launch_rms_norm_backward(const void* dy, const void* h, const void* weight, const float* rstd,
                                    const void* dh, int dtype, int w_dtype, int64_t n, int64_t hidden,
                                    int64_t dy_stride, int64_t h_stride, int64_t dh_stride, int64_t dx_stride,
                                    void* dx, void* dweight, void* ws, int* dev_status, cudaStream_t s,
                                    const DeviceInfo& dev) {
    NormBwdArgs a{};
    a.dy = dy; a.h = h; a.weight = weight; a.dh = dh; a.rstd = rstd; a.w_f32 = w_dtype == VCE_F32;
    a.n = n; a.hidden = hidden; a.dy_stride = dy_stride; a.h_stride = h_stride; a.dh_stride = dh_stride;
    a.dx_stride = dx_stride; a.dx = dx; a.part = static_cast<float*>(ws); a.dev_status = dev_status;
    const size_t es = dtype == VCE_BF16 ? 2 : 4;
    int parts = rms_norm_parts(n, hidden, dev.num_sms);
    const int ve = n == 0 ? 1
                          : pick_ve(int(16 / es), hidden, es, {dy, h, dh ? dh : h, dx},
                                    {dy_stride, h_stride, dh ? dh_stride : 0, dx_stride}, weight, a.w_f32);
    const bool same = same_offset(es, dy, dy_stride, {{h, h_stride}, {dh ? dh : dy, dh ? dh_stride : dy_stride},
                                                      {dx, dx_stride}});
    vce_status st = dtype == VCE_BF16 ? norm_backward<__nv_bfloat16>(a, ve, same, parts, s, dev)
                                      : norm_backward<float>(a, ve, same, parts, s, dev);
    if (st) return st;
    count_launch();
    cudaLaunchConfig_t cfg{};  // its launch overlaps the end of the kernel before, for which it waits
    cfg.gridDim = dim3(unsigned((hidden + 31) / 32));
    cfg.blockDim = dim3(1024);
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const float* part = a.part;
    const auto sum = hidden % 4 == 0 ? rms_norm_dweight_sum<4> : rms_norm_dweight_sum<1>;
    return cudaLaunchKernelEx(&cfg, sum, part, parts, hidden, dweight, a.w_f32) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

}  // namespace vce
