// Launchers of the output head's operators.
#pragma once

#include "vce_internal.cuh"

namespace vce {

// ---- sampling (ce_sample.cu) ----
vce_status launch_ce_sample(const void* logits, int dtype, int64_t n, int64_t vocab, int64_t stride,
                            const float* uniform, const float* temperature, const int* top_k, const float* top_p,
                            const float* min_p, int64_t* token, float* logprob, int* dev_status, cudaStream_t s,
                            const DeviceInfo& dev);

// ---- the norm before the classifier (rms_norm.cu) ----
int rms_norm_parts(int64_t n, int64_t hidden, int num_sms);
vce_status launch_rms_norm(const void* x, const void* residual, const void* weight, int dtype, int w_dtype,
                           int64_t n, int64_t hidden, int64_t x_stride, int64_t r_stride, int64_t h_stride,
                           int64_t y_stride, float eps, void* h, void* y, float* rstd, uint8_t* codes,
                           uint8_t* scales, int* dev_status, cudaStream_t s, const DeviceInfo& dev);
vce_status launch_rms_norm_backward(const void* dy, const void* h, const void* weight, const float* rstd,
                                    const void* dh, int dtype, int w_dtype, int64_t n, int64_t hidden,
                                    int64_t dy_stride, int64_t h_stride, int64_t dh_stride, int64_t dx_stride,
                                    void* dx, void* dweight, void* ws, int* dev_status, cudaStream_t s,
                                    const DeviceInfo& dev);

// ---- microscaled tensors (mx_quant.cu) ----
vce_status launch_mx_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t stride, int fmt,
                              uint8_t* codes, uint8_t* scales, int* dev_status, cudaStream_t s);
vce_status launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int fmt, int64_t rows, int64_t cols,
                                void* out, int dtype, int64_t stride, int* dev_status, cudaStream_t s);

// ---- product of microscaled matrices (mx_linear.cu) ----
vce_status launch_mx_linear(const void* x_codes, const void* x_scales, const void* w_codes, const void* w_scales,
                            int64_t n, int64_t v, int64_t h, void* out, int out_dtype, int64_t out_stride,
                            int* dev_status, cudaStream_t s, const DeviceInfo& dev);

}  // namespace vce
