// Product of a few 8-bit activation rows with 8-bit weights on the CUDA cores: at
// these sizes the call is set-up and latency, and a warp that reads its operands
// straight into registers has neither the tensor path's set-up nor its trip
// through shared memory and TMEM.
//
// A warp takes RW weight rows and MT activation rows and walks K in 512-byte
// steps, 16 bytes of every row a lane; the activation rows come from L1.  int8:
// four-way integer dot products, exact in int32.  e4m3: exact products, fp32 sums.  The RW * MT sums
// are added over the lanes by halving (each step trades half of the values for
// the other half), so a value ends in 32 / (RW MT) lanes of its own; the order of
// the additions is fixed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kernels.cuh"
#include "ptx.cuh"

namespace rtq {
namespace {

constexpr int kWarps = 4;                    // a block

__device__ __forceinline__ float to_type(float v, const float *) { return v; }
__device__ __forceinline__ __half to_type(float v, const __half *) { return __float2half_rn(v); }
__device__ __forceinline__ __nv_bfloat16 to_type(float v, const __nv_bfloat16 *) {
    return __float2bfloat16_rn(v);
}

// Two e4m3 codes (low 16 bits) as fp32, exact.
__device__ __forceinline__ float2 e4m3x2(uint32_t w) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ void codes16(const uint4 &u, float2 (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = e4m3x2(w[i]);
        f[2 * i + 1] = e4m3x2(w[i] >> 16);
    }
}

template <int FMT, typename YT, int MT, int RW>
__global__ void __launch_bounds__(kWarps * 32)
    a8_few_kernel(const uint8_t *__restrict__ Xq, const float *__restrict__ xs,
                  const uint8_t *__restrict__ Wq, const float *__restrict__ ws,
                  const float *__restrict__ bias, YT *__restrict__ Y, int M, int N, int K,
                  DevCtl *ctl) {
    using Acc = std::conditional_t<FMT == kFmtQ8, int, float>;
    constexpr int kVals = RW * MT;
    static_assert(kVals <= 32, "a value a lane");
    // every operand may be the previous kernel's output
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t o0 = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * RW;
    if (o0 >= N) return;
    const int m0 = static_cast<int>(blockIdx.y) * MT;
    const uint8_t *w[RW], *x[MT];
#pragma unroll
    for (int r = 0; r < RW; ++r) w[r] = Wq + min(o0 + r, static_cast<int64_t>(N) - 1) * K;
#pragma unroll
    for (int m = 0; m < MT; ++m) x[m] = Xq + static_cast<int64_t>(min(m0 + m, M - 1)) * K;
    Acc acc[kVals] = {};
    constexpr int kSteps = RW > 2 ? 2 : 4;   // 512-byte steps with loads in flight at once
    for (int k0 = lane * 16; k0 < K; k0 += kSteps * 512) {
        uint4 wv[kSteps][RW];
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int r = 0; r < RW; ++r)
                wv[s][r] = k0 + 512 * s < K ? ldg_nc_v4(w[r] + k0 + 512 * s) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            if (s > 0 && k0 + 512 * s >= K) break;
            if constexpr (FMT == kFmtQ8) {
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint4 xv = ldg_v4(x[m] + k0 + 512 * s);
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        int a = acc[m * RW + r];
                        a = __dp4a(static_cast<int>(wv[s][r].x), static_cast<int>(xv.x), a);
                        a = __dp4a(static_cast<int>(wv[s][r].y), static_cast<int>(xv.y), a);
                        a = __dp4a(static_cast<int>(wv[s][r].z), static_cast<int>(xv.z), a);
                        acc[m * RW + r] = __dp4a(static_cast<int>(wv[s][r].w),
                                                 static_cast<int>(xv.w), a);
                    }
                }
            } else {
                float2 xf[MT][8];
#pragma unroll
                for (int m = 0; m < MT; ++m) codes16(ldg_v4(x[m] + k0 + 512 * s), xf[m]);
#pragma unroll
                for (int r = 0; r < RW; ++r) {
                    float2 wf[8];
                    codes16(wv[s][r], wf);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            acc[m * RW + r] = fmaf(wf[i].x, xf[m][i].x, acc[m * RW + r]);
                            acc[m * RW + r] = fmaf(wf[i].y, xf[m][i].y, acc[m * RW + r]);
                        }
                }
            }
        }
    }
    int d = 16;
#pragma unroll
    for (int half = kVals / 2; half >= 1; half /= 2, d /= 2) {
        const bool hi = (lane & d) != 0;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const Acc send = hi ? acc[i] : acc[i + half], keep = hi ? acc[i + half] : acc[i];
            acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, d);
        }
    }
#pragma unroll
    for (int e = 32 / kVals / 2; e >= 1; e /= 2) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], e);
    // lane group lane / (32 / kVals) holds value m * RW + r
    const int v = lane / (32 / kVals), m = m0 + v / RW;
    const int64_t o = o0 + v % RW;
    float out = 0.f;
    if (lane % (32 / kVals) == 0 && m < M && o < N) {
        const float s = static_cast<float>(acc[0]);
        const YT y = to_type(fmaf(s * (ws ? __ldg(ws + o) : 1.f), __ldg(xs + m),
                                  bias ? __ldg(bias + o) : 0.f), Y);
        Y[static_cast<int64_t>(m) * N + o] = y;
        out = static_cast<float>(y);
    }
    if (__any_sync(0xffffffffu, !(fabsf(out) <= 3.4028234663852886e38f)) && lane == 0)
        atomicOr(&ctl->status, 1u << kStatusRange);
}

template <int FMT, typename YT, int MT, int RW>
cudaError_t launch_few(const void *Xq, const float *xs, const void *Wq, const float *wsc,
                       const float *bias, void *Y, int M, int N, int K, DevCtl *ctl,
                       cudaStream_t st) {
    const uint8_t *x = static_cast<const uint8_t *>(Xq), *w = static_cast<const uint8_t *>(Wq);
    YT *y = static_cast<YT *>(Y);
    void *args[] = {&x, &xs, &w, &wsc, &bias, &y, &M, &N, &K, &ctl};
    cudaLaunchConfig_t cfg = {};
    const int64_t rows = static_cast<int64_t>(RW) * kWarps;
    cfg.gridDim = dim3(static_cast<unsigned>((N + rows - 1) / rows),
                       static_cast<unsigned>((M + MT - 1) / MT), 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(
        &cfg, reinterpret_cast<const void *>(a8_few_kernel<FMT, YT, MT, RW>), args);
}

template <int FMT, typename YT>
cudaError_t launch_few_m(int rw, const void *Xq, const float *xs, const void *Wq, const float *wsc,
                         const float *bias, void *Y, int M, int N, int K, DevCtl *ctl,
                         cudaStream_t s) {
#define RTQ_FEW(mt)                                                                            \
    return rw == 1 ? launch_few<FMT, YT, mt, 1>(Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s)     \
                   : launch_few<FMT, YT, mt, 4>(Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s)
    if (M == 1) RTQ_FEW(1);
    if (M == 2) RTQ_FEW(2);
    if (M <= 4) RTQ_FEW(4);
    RTQ_FEW(8);
#undef RTQ_FEW
}

template <int FMT>
cudaError_t launch_few_y(int rw, int dtype, const void *Xq, const float *xs, const void *Wq,
                         const float *wsc, const float *bias, void *Y, int M, int N, int K,
                         DevCtl *ctl, cudaStream_t s) {
    if (dtype == RT_DTYPE_F32)
        return launch_few_m<FMT, float>(rw, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
    if (dtype == RT_DTYPE_F16)
        return launch_few_m<FMT, __half>(rw, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
    return launch_few_m<FMT, __nv_bfloat16>(rw, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
}

}  // namespace

cudaError_t launch_qgemm_a8_few(int rw, int fmt, int dtype, const void *Xq, const float *xs,
                                const void *Wq, const float *wsc, const float *bias, void *Y, int M,
                                int N, int K, DevCtl *ctl, cudaStream_t s) {
    return fmt == kFmtQ8
               ? launch_few_y<kFmtQ8>(rw, dtype, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s)
               : launch_few_y<kFmtE4M3>(rw, dtype, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
}

}  // namespace rtq
