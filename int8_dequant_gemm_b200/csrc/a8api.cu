// C ABI of the 8-bit activation operators (declared in include/rtq.h):
// argument checks, then one launch each.  None of them needs a workspace.
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "../../include/rtq.h"
#include "kernels.cuh"

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1024;   // tile ends stay in 32 bits
constexpr int64_t kMaxSumK = 131056;   // 128 * 128 * K < 2^31: the int32 sum cannot overflow

struct Span {
    const void *p;
    int64_t bytes;
};

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + static_cast<uintptr_t>(b.bytes) && b0 < a0 + static_cast<uintptr_t>(a.bytes);
}

int type_bytes(int dtype) { return dtype == RT_DTYPE_F32 ? 4 : 2; }
bool dtype_valid(int d) { return d == RT_DTYPE_F32 || d == RT_DTYPE_F16 || d == RT_DTYPE_BF16; }
bool fmt8_valid(int f) { return f == RT_FMT_Q8 || f == RT_FMT_E4M3; }

// Sizes and formats of the row operators, before any pointer is looked at.
rt_status check_rows(int fmt, int dtype, int64_t M, int64_t K, int64_t max_k) {
    if (!fmt8_valid(fmt) || !dtype_valid(dtype) || M < 0 || M > kMaxRows || K < 1)
        return RT_ERR_INVALID_ARG;
    if (K % 16 != 0 || K > max_k) return RT_ERR_UNSUPPORTED_SHAPE;
    return RT_OK;
}

// Codes and scales of an [M, K] result against the n inputs they are made of.
rt_status check_result(const void *codes, const void *scales, int64_t M, int64_t K, const Span *in,
                       int n) {
    if (!codes || !scales) return RT_ERR_INVALID_ARG;
    if (!aligned(codes, 16) || !aligned(scales, 4)) return RT_ERR_ALIGNMENT;
    const Span c = {codes, M * K}, s = {scales, M * 4};
    if (overlap(c, s)) return RT_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (overlap(c, in[i]) || overlap(s, in[i])) return RT_ERR_INVALID_ARG;
    return RT_OK;
}

rt_status from_cuda(cudaError_t e) { return e == cudaSuccess ? RT_OK : RT_ERR_CUDA; }

}  // namespace

extern "C" {

rt_status rt_quantize_a8(int fmt, int dtype, const void *X, void *codes, float *scales, int64_t M,
                         int64_t K, void *stream) {
    rt_status st = check_rows(fmt, dtype, M, K, rtq::kMaxRowK);
    if (st != RT_OK || M == 0) return st;
    if (!X) return RT_ERR_INVALID_ARG;
    if (!aligned(X, 16)) return RT_ERR_ALIGNMENT;
    const Span in[] = {{X, M * K * type_bytes(dtype)}};
    if ((st = check_result(codes, scales, M, K, in, 1)) != RT_OK) return st;
    rtq::DevCtl *ctl = nullptr;
    if ((st = rtq::device_ctl(&ctl)) != RT_OK) return st;
    return from_cuda(rtq::launch_quantize_a8(fmt, dtype, X, static_cast<uint8_t *>(codes), scales,
                                             static_cast<int>(M), static_cast<int>(K), ctl,
                                             static_cast<cudaStream_t>(stream)));
}

rt_status rt_addnorm_a8(int fmt, int dtype, const void *X, const void *R, const float *gain,
                        float eps, void *H, void *codes, float *scales, int64_t M, int64_t K,
                        void *stream) {
    rt_status st = check_rows(fmt, dtype, M, K, rtq::kMaxRowK);
    if (st != RT_OK) return st;
    if (!(eps >= FLT_MIN && eps <= FLT_MAX)) return RT_ERR_INVALID_ARG;
    if (M == 0) return RT_OK;
    if (!X) return RT_ERR_INVALID_ARG;
    if (!aligned(X, 16) || (R && !aligned(R, 16)) || (H && !aligned(H, 16)) ||
        (gain && !aligned(gain, 16)))
        return RT_ERR_ALIGNMENT;
    const int64_t bytes = M * K * type_bytes(dtype);
    const Span in[] = {{X, bytes}, {R, R ? bytes : 0}, {gain, gain ? K * 4 : 0}, {H, H ? bytes : 0}};
    if ((st = check_result(codes, scales, M, K, in, 4)) != RT_OK) return st;
    // H may be X or R itself, but not a part of one shifted against it
    if (H && ((H != X && overlap(in[3], in[0])) || (H != R && overlap(in[3], in[1])) ||
              overlap(in[3], in[2])))
        return RT_ERR_INVALID_ARG;
    rtq::DevCtl *ctl = nullptr;
    if ((st = rtq::device_ctl(&ctl)) != RT_OK) return st;
    return from_cuda(rtq::launch_addnorm_a8(fmt, dtype, X, R, gain, eps, H,
                                            static_cast<uint8_t *>(codes), scales,
                                            static_cast<int>(M), static_cast<int>(K), ctl,
                                            static_cast<cudaStream_t>(stream)));
}

rt_status rt_gate_a8(int fmt, int dtype, const void *U, void *codes, float *scales, int64_t M,
                     int64_t F, void *stream) {
    rt_status st = check_rows(fmt, dtype, M, F, rtq::kMaxRowK);
    if (st != RT_OK || M == 0) return st;
    if (!U) return RT_ERR_INVALID_ARG;
    if (!aligned(U, 16)) return RT_ERR_ALIGNMENT;
    const Span in[] = {{U, 2 * M * F * type_bytes(dtype)}};
    if ((st = check_result(codes, scales, M, F, in, 1)) != RT_OK) return st;
    rtq::DevCtl *ctl = nullptr;
    if ((st = rtq::device_ctl(&ctl)) != RT_OK) return st;
    return from_cuda(rtq::launch_gate_a8(fmt, dtype, U, static_cast<uint8_t *>(codes), scales,
                                         static_cast<int>(M), static_cast<int>(F), ctl,
                                         static_cast<cudaStream_t>(stream)));
}

rt_status rt_dequant_a8(int fmt, int dtype, const void *codes, const float *scales, void *out,
                        int64_t M, int64_t K, void *stream) {
    rt_status st = check_rows(fmt, dtype, M, K, kMaxSumK);
    if (st != RT_OK || M == 0) return st;
    if (!codes || !scales || !out) return RT_ERR_INVALID_ARG;
    if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(out, 16)) return RT_ERR_ALIGNMENT;
    const Span o = {out, M * K * type_bytes(dtype)};
    if (overlap(o, {codes, M * K}) || overlap(o, {scales, M * 4})) return RT_ERR_INVALID_ARG;
    return from_cuda(rtq::launch_dequant_a8(fmt, dtype, static_cast<const uint8_t *>(codes), scales,
                                            out, static_cast<int>(M), static_cast<int>(K),
                                            static_cast<cudaStream_t>(stream)));
}

rt_status rt_qgemm_a8(int fmt, int dtype, const void *Xq, const float *x_scales, const void *Wq,
                      const float *w_scales, const float *bias, void *Y, int64_t M, int64_t N,
                      int64_t K, void *stream) {
    if (!fmt8_valid(fmt) || !dtype_valid(dtype) || M < 0 || N < 1 || K < 1 || M > kMaxRows ||
        N > kMaxRows)
        return RT_ERR_INVALID_ARG;
    if (K % 16 != 0 || K > kMaxSumK) return RT_ERR_UNSUPPORTED_SHAPE;
    // a q8 weight always has row scales; e4m3 weights may have none
    if (!Wq || (fmt == RT_FMT_Q8 && !w_scales)) return RT_ERR_INVALID_ARG;
    if (M == 0) return RT_OK;
    if (!Xq || !x_scales || !Y) return RT_ERR_INVALID_ARG;
    const int es = type_bytes(dtype);
    if (!aligned(Xq, 16) || !aligned(Wq, 16) || !aligned(Y, 16) || !aligned(x_scales, 4) ||
        (w_scales && !aligned(w_scales, 4)) || (bias && !aligned(bias, 4)))
        return RT_ERR_ALIGNMENT;
    const Span y = {Y, M * N * es};
    if (overlap(y, {Xq, M * K}) || overlap(y, {x_scales, M * 4}) || overlap(y, {Wq, N * K}) ||
        overlap(y, {w_scales, N * 4}) || overlap(y, {bias, N * 4}))
        return RT_ERR_INVALID_ARG;
    rtq::DevCtl *ctl = nullptr;
    rt_status st = rtq::device_ctl(&ctl);
    if (st != RT_OK) return st;
    const int m = static_cast<int>(M), n = static_cast<int>(N), k = static_cast<int>(K);
    return from_cuda(rtq::launch_qgemm_a8(rtq::plan_a8(fmt, m, n, k, rtq::sm_count()), fmt, dtype, Xq,
                                          x_scales, Wq, w_scales, bias, Y, m, n, k, ctl,
                                          static_cast<cudaStream_t>(stream)));
}

int rt_qgemm_a8_plan(int fmt, int64_t M, int64_t N, int64_t K, int *tile_rows, int *split) {
    if (!fmt8_valid(fmt) || M < 0 || N < 1 || K < 1 || M > kMaxRows || N > kMaxRows || K % 16 != 0 || K > kMaxSumK)
        return -1;
    const rtq::A8Plan p = rtq::plan_a8(fmt, static_cast<int>(M), static_cast<int>(N),
                                       static_cast<int>(K), rtq::sm_count());
    if (tile_rows) *tile_rows = p.bn;
    if (split) *split = p.split;
    return p.few ? 4 : p.pair | (p.small << 1);
}

}  // extern "C"
