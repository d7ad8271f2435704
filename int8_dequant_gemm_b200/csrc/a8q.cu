// Launchers of the 8-bit row operators: the element type picks the unit that
// holds its kernels (a8q.cuh).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "a8q.cuh"

namespace rtq {

extern template cudaError_t row_operator<float>(int, int, const RowArgs &, cudaStream_t);
extern template cudaError_t row_operator<__half>(int, int, const RowArgs &, cudaStream_t);
extern template cudaError_t row_operator<__nv_bfloat16>(int, int, const RowArgs &, cudaStream_t);
extern template cudaError_t row_values<float>(int, const uint8_t *, const float *, void *, int, int,
                                              cudaStream_t);
extern template cudaError_t row_values<__half>(int, const uint8_t *, const float *, void *, int, int,
                                               cudaStream_t);
extern template cudaError_t row_values<__nv_bfloat16>(int, const uint8_t *, const float *, void *,
                                                      int, int, cudaStream_t);

namespace {

cudaError_t rows(int mode, int fmt, int dtype, const RowArgs &a, cudaStream_t s) {
    if (dtype == RT_DTYPE_F32) return row_operator<float>(mode, fmt, a, s);
    if (dtype == RT_DTYPE_F16) return row_operator<__half>(mode, fmt, a, s);
    return row_operator<__nv_bfloat16>(mode, fmt, a, s);
}

}  // namespace

cudaError_t launch_quantize_a8(int fmt, int dtype, const void *X, uint8_t *codes, float *scales,
                               int M, int K, DevCtl *ctl, cudaStream_t s) {
    return rows(kModeQuant, fmt, dtype,
                {X, nullptr, nullptr, 0.f, 0.f, nullptr, codes, scales, M, K, ctl}, s);
}

cudaError_t launch_addnorm_a8(int fmt, int dtype, const void *X, const void *R, const float *gain,
                              float eps, void *H, uint8_t *codes, float *scales, int M, int K,
                              DevCtl *ctl, cudaStream_t s) {
    return rows(kModeNorm, fmt, dtype,
                {X, R, gain, eps, 1.f / static_cast<float>(K), H, codes, scales, M, K, ctl}, s);
}

cudaError_t launch_gate_a8(int fmt, int dtype, const void *U, uint8_t *codes, float *scales, int M,
                           int F, DevCtl *ctl, cudaStream_t s) {
    return rows(kModeGate, fmt, dtype,
                {U, nullptr, nullptr, 0.f, 0.f, nullptr, codes, scales, M, F, ctl}, s);
}

cudaError_t launch_dequant_a8(int fmt, int dtype, const uint8_t *codes, const float *scales,
                              void *out, int M, int K, cudaStream_t s) {
    if (dtype == RT_DTYPE_F32) return row_values<float>(fmt, codes, scales, out, M, K, s);
    if (dtype == RT_DTYPE_F16) return row_values<__half>(fmt, codes, scales, out, M, K, s);
    return row_values<__nv_bfloat16>(fmt, codes, scales, out, M, K, s);
}

}  // namespace rtq
