// The C ABI of libvce.so: argument validation, workspace carving and dispatch.
// Every host-detectable error returns before any launch; nothing here
// allocates, frees or synchronises.

#include "head_internal.cuh"
#include "mx_format.cuh"

#include <atomic>
#include <mutex>

namespace vce {

namespace {
std::atomic<unsigned long long> g_launches{0};
}

void count_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

vce_status current_device(DeviceInfo& info) {
    static std::mutex mu;
    static DeviceInfo cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return VCE_ERR_CUDA;
    if (dev < 0 || dev >= 64) return VCE_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (cache[dev].ordinal != dev) {
            DeviceInfo d;
            d.ordinal = dev;
            int v = 0, l2 = 0;
            if (cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&v, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&l2, cudaDevAttrL2CacheSize, dev) != cudaSuccess)
                return VCE_ERR_CUDA;
            d.max_smem_optin = size_t(v);
            d.l2_bytes = size_t(l2);
            cache[dev] = d;
        }
        info = cache[dev];
    }
    if (info.cc_major != 10 || info.cc_minor != 3) return VCE_ERR_ARCH;
    return VCE_OK;
}

}  // namespace vce

using namespace vce;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool eps_ok(float eps) { return eps >= 0.f && eps <= 1.f; }  // false for NaN too

bool reduce_ok(int r) { return r == VCE_REDUCE_NONE || r == VCE_REDUCE_MEAN || r == VCE_REDUCE_SUM; }

size_t elem_size(int dtype) { return dtype == VCE_BF16 ? 2 : 4; }

bool dtype_ok(int dtype) { return dtype == VCE_BF16 || dtype == VCE_F32; }

bool mx_ok(int fmt) { return fmt == VCE_MX_E4M3 || fmt == VCE_MX_E2M1; }

// Row counts and lengths the row kernels index with: a grid dimension of rows (and of
// the rows that fill a scale tile), 32-bit columns inside a row.
constexpr int64_t kMaxRows = 0x7fffff00;
constexpr int64_t kMaxCols = int64_t(1) << 28;
constexpr int64_t kMaxTokens = int64_t(1) << 27;  // of adapter_linear, whose grid has eight blocks for each
constexpr int64_t kMaxReorder = int64_t(1) << 23;  // requests of beam_reorder: a grid dimension of groups of 256

vce_status check_norm(int dtype, int64_t n, int64_t hidden, const void* x, int64_t x_stride, const void* residual,
                      int64_t residual_stride, const void* weight, int weight_dtype, float eps, const void* h,
                      int64_t h_stride, const float* rstd) {
    if (!dtype_ok(dtype) || !dtype_ok(weight_dtype)) return VCE_ERR_DTYPE;
    if (n < 0 || n > kMaxRows || hidden < 1 || hidden > kMaxCols || x_stride < hidden || !(eps >= 0.f))
        return VCE_ERR_INVALID_ARG;
    if (n > 0 && (!x || !weight)) return VCE_ERR_INVALID_ARG;
    if (n > 0 && residual && (!h || residual_stride < hidden || h_stride < hidden)) return VCE_ERR_INVALID_ARG;
    const size_t es = elem_size(dtype);
    if (!aligned(x, es) || !aligned(residual, es) || !aligned(h, es) || !aligned(weight, elem_size(weight_dtype)) ||
        !aligned(rstd, 4))
        return VCE_ERR_ALIGN;
    return VCE_OK;
}

}  // namespace

extern "C" {

const char* vce_status_string(int status) {
    switch (status) {
        case VCE_OK: return "VCE_OK";
        case VCE_ERR_INVALID_ARG: return "VCE_ERR_INVALID_ARG";
        case VCE_ERR_DTYPE: return "VCE_ERR_DTYPE";
        case VCE_ERR_ALIGN: return "VCE_ERR_ALIGN";
        case VCE_ERR_WORKSPACE: return "VCE_ERR_WORKSPACE";
        case VCE_ERR_ARCH: return "VCE_ERR_ARCH";
        case VCE_ERR_CUDA: return "VCE_ERR_CUDA";
        default: return "VCE_UNKNOWN_STATUS";
    }
}

int vce_version(void) { return 100; }

unsigned long long vce_kernel_launches(void) { return g_launches.load(std::memory_order_relaxed); }

int vce_bounds_check_build(void) {
#ifdef VCE_BOUNDS_CHECK
    return 1;
#else
    return 0;
#endif
}

size_t ce_workspace_size(int64_t n_rows, int64_t vocab, int reduce_loss) {
    (void)vocab;
    if (!reduce_loss || n_rows <= 0) return 0;
    return align256(size_t(n_rows) * sizeof(float));
}

vce_status ce_forward(const void* logits, int dtype, int64_t n_rows, int64_t vocab,
                      int64_t row_stride, const int64_t* target, float label_smoothing,
                      int reduce_loss, int64_t ignore_idx, float* loss, float* stats,
                      int64_t* n_valid, void* ws, size_t ws_bytes, int* dev_status,
                      void* stream) {
    if (dtype != VCE_BF16 && dtype != VCE_F32) return VCE_ERR_DTYPE;
    if (n_rows < 0 || vocab < 1 || row_stride < vocab || !eps_ok(label_smoothing) || !reduce_ok(reduce_loss))
        return VCE_ERR_INVALID_ARG;
    if (!loss || (n_rows > 0 && (!logits || !target || !stats))) return VCE_ERR_INVALID_ARG;
    if (reduce_loss == VCE_REDUCE_MEAN && !n_valid) return VCE_ERR_INVALID_ARG;
    if (!aligned(logits, elem_size(dtype)) || !aligned(stats, 8)) return VCE_ERR_ALIGN;
    const size_t need = ce_workspace_size(n_rows, vocab, reduce_loss);
    if (need > 0 && (!ws || ws_bytes < need)) return VCE_ERR_WORKSPACE;
    if (ws && !aligned(ws, 256)) return VCE_ERR_ALIGN;
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_ce_forward(logits, dtype, n_rows, vocab, row_stride, target, label_smoothing,
                             reduce_loss, ignore_idx, loss, stats, n_valid, ws, dev_status,
                             static_cast<cudaStream_t>(stream), dev);
}

vce_status ce_backward(const void* logits, int dtype, int64_t n_rows, int64_t vocab,
                       int64_t row_stride, const int64_t* target, const float* stats,
                       const int64_t* n_valid, const float* grad_output,
                       float label_smoothing, int reduce_loss, int64_t ignore_idx,
                       void* dlogits, int* dev_status, void* stream) {
    if (dtype != VCE_BF16 && dtype != VCE_F32) return VCE_ERR_DTYPE;
    if (n_rows < 0 || vocab < 1 || row_stride < vocab || !eps_ok(label_smoothing) || !reduce_ok(reduce_loss))
        return VCE_ERR_INVALID_ARG;
    if (n_rows > 0 && (!logits || !target || !stats || !grad_output || !dlogits))
        return VCE_ERR_INVALID_ARG;
    if (n_rows > 0 && reduce_loss == VCE_REDUCE_MEAN && !n_valid) return VCE_ERR_INVALID_ARG;
    const size_t es = elem_size(dtype);
    if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(stats, 8)) return VCE_ERR_ALIGN;
    // logits and dlogits rows must share their offset within 16 bytes (vector path)
    if (((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(dlogits)) & 15) != 0)
        return VCE_ERR_ALIGN;
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_ce_backward(logits, dtype, n_rows, vocab, row_stride, target, stats, n_valid,
                              grad_output, label_smoothing, reduce_loss, ignore_idx, dlogits,
                              dev_status, static_cast<cudaStream_t>(stream), dev);
}

vce_status ce_forward_backward(const void* logits, int dtype, int64_t n_rows, int64_t vocab,
                               int64_t row_stride, const int64_t* target, float label_smoothing,
                               int reduce_loss, int64_t ignore_idx, const float* grad_output,
                               float* loss, float* stats, int64_t* n_valid, void* dlogits, void* ws,
                               size_t ws_bytes, int* dev_status, void* stream) {
    if (dtype != VCE_BF16 && dtype != VCE_F32) return VCE_ERR_DTYPE;
    if (n_rows < 0 || vocab < 1 || row_stride < vocab || !eps_ok(label_smoothing) || !reduce_ok(reduce_loss))
        return VCE_ERR_INVALID_ARG;
    if (!loss || (n_rows > 0 && (!logits || !target || !stats || !grad_output || !dlogits)))
        return VCE_ERR_INVALID_ARG;
    if (reduce_loss == VCE_REDUCE_MEAN && !n_valid) return VCE_ERR_INVALID_ARG;
    const size_t es = elem_size(dtype);
    if (!aligned(logits, es) || !aligned(dlogits, es) || !aligned(stats, 8)) return VCE_ERR_ALIGN;
    if (((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(dlogits)) & 15) != 0)
        return VCE_ERR_ALIGN;
    const size_t need = ce_workspace_size(n_rows, vocab, reduce_loss);
    if (need > 0 && (!ws || ws_bytes < need)) return VCE_ERR_WORKSPACE;
    if (ws && !aligned(ws, 256)) return VCE_ERR_ALIGN;
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_ce_forward_backward(logits, dtype, n_rows, vocab, row_stride, target, label_smoothing,
                                      reduce_loss, ignore_idx, grad_output, loss, stats, n_valid, dlogits, ws,
                                      dev_status, static_cast<cudaStream_t>(stream), dev);
}

vce_status shift_targets(const int64_t* target, int64_t n, int64_t seq_len, int64_t ignore_idx,
                         int64_t* shifted, void* stream) {
    if (n < 0 || seq_len < 1 || (n > 0 && (!target || !shifted))) return VCE_ERR_INVALID_ARG;
    if (n > 0 && target == shifted) return VCE_ERR_INVALID_ARG;  // the kernel reads target[i + 1]
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_shift_targets(target, n, seq_len, ignore_idx, shifted, static_cast<cudaStream_t>(stream));
}

size_t lce_workspace_size(int64_t n, int64_t h, int64_t v, int reduce_loss,
                          size_t max_slab_bytes) {
    if (n <= 0 || h <= 0 || v <= 0) return 0;
    const size_t fwd = lce_forward_ws_bytes(n, v, reduce_loss);
    if (max_slab_bytes == 0) max_slab_bytes = VCE_DEFAULT_SLAB_BYTES;
    const int64_t cap = int64_t(max_slab_bytes / (size_t(n) * 2)) / 256 * 256;  // at most 2^63 - 1
    const int64_t slab = cap < 256 ? 256 : (cap < v ? cap : v);
    const size_t bwd = lce_backward_ws_bytes(n, h, v, slab);
    return fwd > bwd ? fwd : bwd;
}

vce_status lce_forward(const void* X, const void* W, int64_t n, int64_t h, int64_t v,
                       const int64_t* target, float label_smoothing, int reduce_loss,
                       int64_t ignore_idx, float* loss, float* lse, float* entropy,
                       int64_t* n_valid, void* ws, size_t ws_bytes, int* dev_status,
                       void* stream) {
    if (n < 0 || h < 1 || v < 1 || !eps_ok(label_smoothing) || !reduce_ok(reduce_loss)) return VCE_ERR_INVALID_ARG;
    if (!loss || (n > 0 && (!X || !W || !target || !lse))) return VCE_ERR_INVALID_ARG;
    if (reduce_loss == VCE_REDUCE_MEAN && !n_valid) return VCE_ERR_INVALID_ARG;
    if (h % 8 != 0 || !aligned(X, 16) || !aligned(W, 16)) return VCE_ERR_ALIGN;
    if (n > 0) {
        const size_t need = lce_forward_ws_bytes(n, v, reduce_loss);
        if (!ws || ws_bytes < need) return VCE_ERR_WORKSPACE;
        if (!aligned(ws, 256)) return VCE_ERR_ALIGN;
    }
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_lce_forward(X, W, n, h, v, target, label_smoothing, reduce_loss, ignore_idx,
                              loss, lse, entropy, n_valid, ws, dev_status,
                              static_cast<cudaStream_t>(stream), dev);
}

vce_status lce_backward(const void* X, const void* W, int64_t n, int64_t h, int64_t v,
                        const int64_t* target, const float* lse, const int64_t* n_valid,
                        const float* grad_output, float label_smoothing, int reduce_loss,
                        int64_t ignore_idx, void* dX, void* dW, void* ws, size_t ws_bytes,
                        int* dev_status, void* stream) {
    if (n < 0 || h < 1 || v < 1 || !eps_ok(label_smoothing) || !reduce_ok(reduce_loss)) return VCE_ERR_INVALID_ARG;
    if (!dW || (n > 0 && (!X || !W || !target || !lse || !grad_output || !dX)))
        return VCE_ERR_INVALID_ARG;
    if (n > 0 && reduce_loss == VCE_REDUCE_MEAN && !n_valid) return VCE_ERR_INVALID_ARG;
    if (h % 8 != 0 || !aligned(X, 16) || !aligned(W, 16) || !aligned(dX, 16) || !aligned(dW, 16))
        return VCE_ERR_ALIGN;
    int64_t slab = 0;
    if (n > 0) {
        slab = lce_slab_for_ws(n, h, v, ws ? ws_bytes : 0);
        if (slab <= 0) return VCE_ERR_WORKSPACE;
        if (!aligned(ws, 256)) return VCE_ERR_ALIGN;
    }
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_lce_backward(X, W, n, h, v, target, lse, n_valid, grad_output, label_smoothing,
                               reduce_loss, ignore_idx, dX, dW, ws, slab, dev_status,
                               static_cast<cudaStream_t>(stream), dev);
}

vce_status rms_norm_forward(const void* x, int dtype, int64_t n, int64_t hidden, int64_t x_stride,
                            const void* residual, int64_t residual_stride, const void* weight,
                            int weight_dtype, float eps, void* h, int64_t h_stride, void* y,
                            int64_t y_stride, float* rstd, int* dev_status, void* stream) {
    if (vce_status st = check_norm(dtype, n, hidden, x, x_stride, residual, residual_stride, weight, weight_dtype,
                                   eps, h, h_stride, rstd))
        return st;
    if (n > 0 && (!y || y_stride < hidden)) return VCE_ERR_INVALID_ARG;
    if (!aligned(y, elem_size(dtype))) return VCE_ERR_ALIGN;
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_rms_norm(x, residual, weight, dtype, weight_dtype, n, hidden, x_stride, residual_stride, h_stride,
                           y_stride, eps, h, y, rstd, nullptr, nullptr, dev_status,
                           static_cast<cudaStream_t>(stream), dev);
}

vce_status rms_norm_mx(const void* x, int dtype, int64_t n, int64_t hidden, int64_t x_stride,
                       const void* residual, int64_t residual_stride, const void* weight,
                       int weight_dtype, float eps, void* h, int64_t h_stride, void* codes,
                       void* scales, float* rstd, int* dev_status, void* stream) {
    if (vce_status st = check_norm(dtype, n, hidden, x, x_stride, residual, residual_stride, weight, weight_dtype,
                                   eps, h, h_stride, rstd))
        return st;
    if (n > 0 && (!codes || !scales)) return VCE_ERR_INVALID_ARG;
    if (!aligned(codes, 16) || !aligned(scales, 16)) return VCE_ERR_ALIGN;
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_rms_norm(x, residual, weight, dtype, weight_dtype, n, hidden, x_stride, residual_stride, h_stride,
                           0, eps, h, nullptr, rstd, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                           dev_status, static_cast<cudaStream_t>(stream), dev);
}

size_t rms_norm_workspace_size(int64_t n, int64_t hidden) {
    DeviceInfo dev;
    if (n <= 0 || hidden <= 0 || current_device(dev) != VCE_OK) return 0;
    return align256(size_t(rms_norm_parts(n, hidden, dev.num_sms)) * size_t(hidden) * sizeof(float));
}

vce_status rms_norm_backward(const void* dy, int dtype, int64_t n, int64_t hidden, int64_t dy_stride,
                             const void* h, int64_t h_stride, const void* weight, int weight_dtype,
                             const float* rstd, const void* dh, int64_t dh_stride, void* dx,
                             int64_t dx_stride, void* dweight, void* ws, size_t ws_bytes,
                             int* dev_status, void* stream) {
    if (!dtype_ok(dtype) || !dtype_ok(weight_dtype)) return VCE_ERR_DTYPE;
    if (n < 0 || n > kMaxRows || hidden < 1 || hidden > kMaxCols || !dweight) return VCE_ERR_INVALID_ARG;
    if (n > 0 && (!dy || !h || !weight || !rstd || !dx || dy_stride < hidden || h_stride < hidden ||
                  dx_stride < hidden || (dh && dh_stride < hidden) || dx == h))
        return VCE_ERR_INVALID_ARG;
    const size_t es = elem_size(dtype), ews = elem_size(weight_dtype);
    if (!aligned(dy, es) || !aligned(h, es) || !aligned(dh, es) || !aligned(dx, es) || !aligned(weight, ews) ||
        !aligned(dweight, ews) || !aligned(rstd, 4))
        return VCE_ERR_ALIGN;
    DeviceInfo dev;
    if (n > 0 && !ws) return VCE_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return VCE_ERR_ALIGN;
    if (vce_status st = current_device(dev)) return st;
    if (n > 0 && ws_bytes < rms_norm_workspace_size(n, hidden)) return VCE_ERR_WORKSPACE;
    return launch_rms_norm_backward(dy, h, weight, rstd, dh, dtype, weight_dtype, n, hidden, dy_stride, h_stride,
                                    dh_stride, dx_stride, dx, dweight, ws, dev_status,
                                    static_cast<cudaStream_t>(stream), dev);
}

size_t mx_codes_size(int64_t rows, int64_t cols, int fmt) {
    if (rows <= 0 || cols <= 0 || !mx_ok(fmt)) return 0;
    return size_t(rows) * size_t(mx::padded(cols)) / (fmt == VCE_MX_E2M1 ? 2 : 1);
}

size_t mx_scales_size(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0) return 0;
    return size_t(mx::padded(rows)) * size_t(mx::padded(cols)) / mx::kBlock;
}

vce_status mx_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t row_stride, int fmt,
                       void* codes, void* scales, int* dev_status, void* stream) {
    if (!dtype_ok(dtype) || !mx_ok(fmt)) return VCE_ERR_DTYPE;
    if (rows < 0 || rows > kMaxRows || cols < 1 || cols > kMaxCols || row_stride < cols) return VCE_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !codes || !scales)) return VCE_ERR_INVALID_ARG;
    if (!aligned(x, elem_size(dtype)) || !aligned(codes, 16) || !aligned(scales, 16)) return VCE_ERR_ALIGN;
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_mx_quantize(x, dtype, rows, cols, row_stride, fmt, static_cast<uint8_t*>(codes),
                              static_cast<uint8_t*>(scales), dev_status, static_cast<cudaStream_t>(stream));
}

vce_status mx_dequantize(const void* codes, const void* scales, int fmt, int64_t rows, int64_t cols,
                         void* out, int dtype, int64_t row_stride, int* dev_status, void* stream) {
    if (!dtype_ok(dtype) || !mx_ok(fmt)) return VCE_ERR_DTYPE;
    if (rows < 0 || rows > kMaxRows || cols < 1 || cols > kMaxCols || row_stride < cols) return VCE_ERR_INVALID_ARG;
    if (rows > 0 && (!out || !codes || !scales)) return VCE_ERR_INVALID_ARG;
    if (!aligned(out, elem_size(dtype)) || !aligned(codes, 16) || !aligned(scales, 16)) return VCE_ERR_ALIGN;
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_mx_dequantize(static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), fmt, rows,
                                cols, out, dtype, row_stride, dev_status, static_cast<cudaStream_t>(stream));
}

vce_status mx_linear(const void* x_codes, const void* x_scales, const void* w_codes, const void* w_scales,
                     int64_t n, int64_t h, int64_t v, void* out, int out_dtype, int64_t out_stride,
                     int* dev_status, void* stream) {
    if (!dtype_ok(out_dtype)) return VCE_ERR_DTYPE;
    if (n < 0 || n > kMaxRows || v < 1 || v > kMaxRows || h < 1 || h > kMaxCols || out_stride < v)
        return VCE_ERR_INVALID_ARG;
    if (n > 0 && (!x_codes || !x_scales || !w_codes || !w_scales || !out)) return VCE_ERR_INVALID_ARG;
    if (!aligned(x_codes, 16) || !aligned(x_scales, 16) || !aligned(w_codes, 32) || !aligned(w_scales, 16) ||
        !aligned(out, elem_size(out_dtype)))
        return VCE_ERR_ALIGN;
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_mx_linear(x_codes, x_scales, w_codes, w_scales, n, v, h, out, out_dtype, out_stride, dev_status,
                            static_cast<cudaStream_t>(stream), dev);
}

vce_status ce_sample(const void* logits, int dtype, int64_t n_rows, int64_t vocab, int64_t row_stride,
                     const float* uniform, const float* temperature, const int32_t* top_k,
                     const float* top_p, const float* min_p, int64_t* token, float* logprob,
                     int* dev_status, void* stream) {
    if (!dtype_ok(dtype)) return VCE_ERR_DTYPE;
    if (n_rows < 0 || n_rows > kMaxRows || vocab < 1 || vocab > VCE_SAMPLE_MAX_VOCAB || row_stride < vocab)
        return VCE_ERR_INVALID_ARG;
    if (n_rows > 0 && (!logits || !uniform || !token)) return VCE_ERR_INVALID_ARG;
    if (!aligned(logits, elem_size(dtype)) || !aligned(uniform, 4) || !aligned(temperature, 4) ||
        !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(token, 8) || !aligned(logprob, 4))
        return VCE_ERR_ALIGN;
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_ce_sample(logits, dtype, n_rows, vocab, row_stride, uniform, temperature, top_k, top_p, min_p,
                            token, logprob, dev_status, static_cast<cudaStream_t>(stream), dev);
}

size_t ce_beam_workspace_size(int64_t batch, int beams, int count) {
    if (batch <= 0 || batch > kMaxRows || beams < 1 || beams > VCE_BEAM_MAX_BEAMS || count < 1 ||
        count > VCE_BEAM_MAX_COUNT)
        return 0;
    return ce_beam_ws_bytes(batch * beams, count);
}

vce_status ce_beam(const void* logits, int dtype, int64_t batch, int beams, int64_t vocab, int64_t row_stride,
                   const float* score, const uint8_t* ended, const int32_t* length, int64_t end,
                   double length_penalty, int count, int keep_places, int64_t* token, int64_t* parent,
                   float* out_score, uint8_t* out_ended, int32_t* out_length, void* ws, size_t ws_bytes,
                   int* dev_status, void* stream) {
    if (!dtype_ok(dtype)) return VCE_ERR_DTYPE;
    if (batch < 0 || batch > kMaxRows || beams < 1 || beams > VCE_BEAM_MAX_BEAMS || batch * beams > kMaxRows ||
        vocab < 1 || vocab > VCE_SAMPLE_MAX_VOCAB || row_stride < vocab || count < 1 || count > VCE_BEAM_MAX_COUNT ||
        (keep_places && count != beams) || end < -1 || end >= vocab || (ended && end < 0) ||
        !(length_penalty >= -16.0 && length_penalty <= 16.0) || (length_penalty != 0.0 && !length))
        return VCE_ERR_INVALID_ARG;
    if (batch > 0 && (!logits || !score || !token || !parent || !out_score || ((ended || end >= 0) && !out_ended) ||
                      (length && !out_length)))
        return VCE_ERR_INVALID_ARG;
    if (!length && out_length) return VCE_ERR_INVALID_ARG;
    // a request's results over another one's state
    if (batch > 0 && count != beams && (out_score == score || (ended && out_ended == ended) || (length && out_length == length)))
        return VCE_ERR_INVALID_ARG;
    if (!aligned(logits, elem_size(dtype)) || !aligned(score, 4) || !aligned(length, 4) || !aligned(token, 8) ||
        !aligned(parent, 8) || !aligned(out_score, 4) || !aligned(out_length, 4) || !aligned(ws, 256))
        return VCE_ERR_ALIGN;
    if (batch > 0 && (!ws || ws_bytes < ce_beam_workspace_size(batch, beams, count))) return VCE_ERR_WORKSPACE;
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_ce_beam(logits, dtype, batch, beams, vocab, row_stride, score, ended, length, end, length_penalty,
                          count, keep_places != 0, token, parent, out_score, out_ended, out_length, ws, dev_status,
                          static_cast<cudaStream_t>(stream), dev);
}

vce_status beam_reorder(const vce_state* states, int count, const int64_t* parent, int64_t batch, int beams,
                        const int32_t* lengths, int* dev_status, void* stream) {
    constexpr int64_t kMost = int64_t(1) << 46;  // bytes of a row, and of a stride
    if (count < 0 || (count > 0 && !states) || batch < 0 || batch > kMaxRows || beams < 1 ||
        beams > VCE_BEAM_MAX_BEAMS || batch * beams > kMaxRows || batch > kMaxReorder)
        return VCE_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        const vce_state& s = states[i];
        if (s.parts < 0 || s.positions < 0 || s.position_bytes < 0 || s.parts > kMost || s.positions > kMost ||
            s.position_bytes > kMost)
            return VCE_ERR_INVALID_ARG;
        if (s.parts == 0 || s.positions == 0 || s.position_bytes == 0) continue;
        if (s.positions > kMost / s.position_bytes || s.positions * s.position_bytes > kMost / s.parts)
            return VCE_ERR_INVALID_ARG;
        if (batch > 0 && (!s.src || !s.dst)) return VCE_ERR_INVALID_ARG;
        for (int64_t stride : {s.src_row_stride, s.dst_row_stride, s.src_part_stride, s.dst_part_stride})
            if (stride < 0 || stride > kMost) return VCE_ERR_INVALID_ARG;
        if (s.src == s.dst && (s.src_row_stride != s.dst_row_stride || s.src_part_stride != s.dst_part_stride))
            return VCE_ERR_INVALID_ARG;
    }
    if (batch > 0 && count > 0 && !parent) return VCE_ERR_INVALID_ARG;
    if (!aligned(parent, 8) || !aligned(lengths, 4)) return VCE_ERR_ALIGN;
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_beam_reorder(states, count, parent, batch, beams, lengths, dev_status,
                               static_cast<cudaStream_t>(stream), dev);
}

size_t adapter_workspace_size(int64_t n, int64_t adapters, int rank) {
    if (n <= 0 || n > kMaxRows || adapters < 1 || adapters > VCE_MAX_ADAPTERS || rank < 1 || rank > VCE_MAX_ADAPTER_RANK)
        return 0;
    return adapter_ws_bytes(n, adapters, rank);
}

vce_status adapter_linear(const void* y, int y_dtype, int64_t n, int64_t vocab, int64_t y_stride, const void* x,
                          int x_dtype, int64_t hidden, int64_t x_stride, const void* A, const void* B,
                          int64_t adapters, int rank, const int32_t* index, const float* scale, void* out,
                          int64_t out_stride, void* ws, size_t ws_bytes, int* dev_status, void* stream) {
    if (!dtype_ok(y_dtype) || !dtype_ok(x_dtype)) return VCE_ERR_DTYPE;
    if (n < 0 || n > kMaxTokens || vocab < 1 || vocab > kMaxCols || y_stride < vocab || out_stride < vocab ||
        hidden < 1 || hidden > kMaxCols || x_stride < hidden || adapters < 1 || adapters > VCE_MAX_ADAPTERS ||
        rank < 1 || rank > VCE_MAX_ADAPTER_RANK || rank % 8)
        return VCE_ERR_INVALID_ARG;
    if (n > 0 && (!y || !x || !A || !B || !index || !out)) return VCE_ERR_INVALID_ARG;
    if (out == y && out_stride != y_stride) return VCE_ERR_INVALID_ARG;
    const int64_t es = int64_t(elem_size(x_dtype));
    if (!aligned(y, elem_size(y_dtype)) || !aligned(out, elem_size(y_dtype)) || !aligned(x, 16) || !aligned(A, 16) ||
        !aligned(B, 16) || !aligned(index, 4) || !aligned(scale, 4) || !aligned(ws, 256) || hidden % 8 ||
        (n > 1 && x_stride * es % 16))
        return VCE_ERR_ALIGN;
    if (n > 0 && (!ws || ws_bytes < adapter_workspace_size(n, adapters, rank))) return VCE_ERR_WORKSPACE;
    DeviceInfo dev;
    if (vce_status st = current_device(dev)) return st;
    return launch_adapter_linear(y, y_dtype, n, vocab, y_stride, x, x_dtype, hidden, x_stride, A, B, adapters, rank, index,
                                 scale, out, out_stride, ws, dev_status, static_cast<cudaStream_t>(stream), dev);
}

}  // extern "C"
