// Activations into 8 bits, one scale a row: plain quantization, residual
// addition + root-mean-square norm, and the gated SiLU, each followed in the
// same kernel by
//
//   s0 = max_k |v_k| / Q,   code_k = v_k / s0 rounded to nearest even
//
// (Q = 127 onto int8, the rule of rt_quantize_q8_row, s0 rounded to fp32; Q = 448
// onto FP8 E4M3, s0 unrounded in the codes).
//
// Norm: y = h * rstd * g with rstd = 1 / sqrt(mean(h^2) + eps) > 0, so
// y_k / max|y| = (h g)_k / max|h g|: the codes need only v = h * g, and rstd
// enters the scale alone, scale = s0 * rstd.  Sum of squares and maximum
// therefore come from one pass over the row and one reduction, and no value
// waits for rstd.
//
// A row stays with a group of TPR threads (NV vectors of 16 bytes a thread and
// input), so each input is read once and nothing is written but the sum h, the
// codes and the scale.  It stays in registers up to K = 16384 (fp32 norm and gate: 8192);
// longer rows need more than the 64 that each of 1024 threads has, and the rest
// is spilled (K = 32768: 2.4 to 5.7 TB/s).  Sums, maxima and values are fp32.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>

#include "kernels.cuh"
#include "ptx.cuh"

namespace rtq {

constexpr int kModeQuant = 0, kModeNorm = 1, kModeGate = 2;

struct RowArgs {
    const void *X, *R;
    const float *gain;
    float eps, inv_k;
    void *H;
    uint8_t *codes;
    float *scales;
    int M, K;
    DevCtl *ctl;
};

// The row operators of one element type; each type is a compilation unit
// (a8q_f32.cu, a8q_f16.cu, a8q_bf16.cu).
template <typename T>
cudaError_t row_operator(int mode, int fmt, const RowArgs &a, cudaStream_t s);
template <typename T>
cudaError_t row_values(int fmt, const uint8_t *codes, const float *scales, void *out, int M, int K,
                       cudaStream_t s);

namespace {

template <typename T>
struct Vec {
    static constexpr int n = 16 / static_cast<int>(sizeof(T));
};

__device__ __forceinline__ void unpack(const uint4 &u, float (&f)[4], const float *) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
}

__device__ __forceinline__ void unpack(const uint4 &u, float (&f)[8], const __nv_bfloat16 *) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void unpack(const uint4 &u, float (&f)[8], const __half *) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

__device__ __forceinline__ uint4 pack(const float (&f)[4], const float *) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
}

__device__ __forceinline__ uint4 pack(const float (&f)[8], const __nv_bfloat16 *) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 pack(const float (&f)[8], const __half *) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// |v| as bits: an order on magnitudes in which infinity is above every finite
// value and NaN above infinity, so that one unsigned maximum finds both.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;
constexpr uint32_t kTinyBits = 0x0D800000u;   // 2^-100: from here on 1 / (max / Q) is finite

// max(mx, abs_bits(v)) in one instruction (any NaN becomes the NaN of all ones).
__device__ __forceinline__ uint32_t max_bits(uint32_t mx, float v) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(__uint_as_float(mx)), "f"(fabsf(v)));
    return __float_as_uint(m);
}

// Unsigned maximum and (SUM) sum over the TPR threads of a row's group; every
// thread gets both.  TPR > 32: through shared memory, `part` = one slot per
// warp of the block, two buffers used in turn so that one barrier a call is
// enough.  A group of whole warps smaller than the block syncs the block: all
// of a block's groups run the same number of calls.
template <int TPR, bool SUM>
__device__ __forceinline__ void row_reduce(float &sum, uint32_t &mx, float2 *part, int &turn) {
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (SUM) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    }
    if (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        float2 *buf = part + turn * 32;
        turn ^= 1;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) buf[warp] = make_float2(sum, __uint_as_float(mx));
        __syncthreads();
        const float2 p = buf[warp / kWarps * kWarps + (lane % kWarps)];
        mx = __reduce_max_sync(0xffffffffu, __float_as_uint(p.y));
        if (SUM) {
            sum = p.x;
#pragma unroll
            for (int d = kWarps / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        }
    }
}

// a / Q correctly rounded, a = 0 or at least 2^-100: the quotient from the
// rounded reciprocal, corrected by its exact remainder (Markstein's division).
template <int FMT>
__device__ __forceinline__ float over_top(float a) {
    constexpr float kTop = FMT == kFmtQ8 ? 127.f : 448.f;
    constexpr float kInv = 1.f / kTop;
    const float q = a * kInv;
    return fmaf(fmaf(-q, kTop, a), kInv, q);
}

// 1.5 * 2^23 + n for an integer |n| <= 128: n in the low mantissa bits.
constexpr float kMagic = 12582912.f;

// The integer nearest v / s0 (ties to even), in kMagic form, from m = kMagic +
// the integer nearest an approximation of the quotient that is within 3e-5.
// The residual r = v - n s0 of one fused multiply-add is exact where it is near
// s0 / 2 in magnitude; n moves toward its sign if |r| > s0 / 2, or if |r| = s0 / 2
// and n is odd (magnitudes compare as their bits do).
__device__ __forceinline__ float nearest_code(float v, float s0, float m) {
    const float r = fmaf(kMagic - m, s0, v);
    const uint32_t b = __float_as_uint(m);
    const bool move = abs_bits(r) + (b & 1u) > __float_as_uint(0.5f * s0);
    return __uint_as_float(move ? b + (r < 0.f ? 0xFFFFFFFFu : 1u) : b);
}

// The same for s0 below 2^-100, down to subnormals and 0, where twice the residual
// against s0 is still a multiple of the smallest subnormal.  A subnormal s0
// is so coarse that quotients can pass 127: they are held there.
__device__ __noinline__ float tiny_code(float v, float s0) {
    if (s0 == 0.f) return kMagic;
    const float n = rintf(fminf(200.f, fmaxf(-200.f, __fdiv_rn(v, s0))));
    const float r = fmaf(-2.f * n, s0, 2.f * v);
    const bool move = abs_bits(r) + (static_cast<int>(n) & 1) > __float_as_uint(s0);
    return kMagic + fminf(127.f, fmaxf(-127.f, move ? (r < 0.f ? n - 1.f : n + 1.f) : n));
}

// Codes of one 16-byte input vector's values.  int8: v * inv is within 3e-5 of
// v / s0 at |code| <= 127 (inv is within 2^-23 of 1 / s0), and one fused
// multiply-add onto 1.5 * 2^23 rounds it to an integer in the low mantissa bits.
// Only a product that close to a rounding border can round to another integer
// than the quotient; those are decided exactly, and the codes are the host
// quantizer's.  e4m3: v * (inv + inv_lo), inv + inv_lo = Q / max|v| to about
// 2^-45, so that the quotient is rounded once before it is rounded to 8 bits.
// `slow`: s0 is too small for 1 / s0.
template <int FMT, int N>
__device__ __forceinline__ void encode(const float (&v)[N], float s0, float inv, float inv_lo,
                                       bool slow, uint32_t (&w)[N / 4]) {
    if (FMT == kFmtQ8) {
        float m[N], edge = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            m[i] = fmaf(v[i], inv, kMagic);
            edge = fmaxf(edge, fabsf(fmaf(v[i], inv, kMagic - m[i])));
        }
        if (edge > 0.49996f) {
#pragma unroll
            for (int i = 0; i < N; ++i) m[i] = nearest_code(v[i], s0, m[i]);
        }
        if (slow) {
#pragma unroll
            for (int i = 0; i < N; ++i) m[i] = tiny_code(v[i], s0);
        }
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            uint32_t b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(m[4 * i + j]);
            w[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040),
                               0x5410);
        }
    } else {
        float t[N];
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = fmaf(v[i], inv, v[i] * inv_lo);
        if (slow) {
#pragma unroll
            for (int i = 0; i < N; ++i) t[i] = s0 > 0.f ? __fdiv_rn(v[i], s0) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(t[4 * i], t[4 * i + 1]),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(t[4 * i + 2], t[4 * i + 3]),
                                                         __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        }
    }
}

// a * sigmoid(a) * b = a b / (1 + e^-a) of two values.  With s = a log2 e,
// rounded, 2^-s is e^-a but for what s lost, up to 2^-24 |a|: the factor
// e^-(a - s ln 2), to first order.  Off by at most 5 units of 2^-24 from a = -20 on and 7
// from -80 on, where a / (1 + expf(-a)) is by 4.2 and 2^-s alone by 18 and 64
// (65536 x 2048 bf16: 114 us; 185 and 111).  Below a = -87.3 the reciprocal is 0:
// sigmoid(a) < 2^-126 counts as 0.
__device__ __forceinline__ float2 silu_mul(float2 a, float2 b) {
    const float2 x = make_float2(fminf(a.x, 128.f), fminf(a.y, 128.f));     // e^-128 adds nothing to 1
    const float2 s = __fmul2_rn(x, make_float2(1.4426950408889634f, 1.4426950408889634f));
    const float2 m = __ffma2_rn(s, make_float2(-0.69314718055994531f, -0.69314718055994531f), x);
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(-s.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(-s.y));
    const float2 one = make_float2(1.f, 1.f);
    const float2 den = __ffma2_rn(e, __ffma2_rn(m, make_float2(-1.f, -1.f), one), one);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(den.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(den.y));
    return __fmul2_rn(__fmul2_rn(a, r), b);
}

// Rows of [M, K] by groups of TPR threads, blockDim.x / TPR rows a block at a
// time; the blocks stay and walk the rows, and each thread loads its part of
// the next row before it works on this one, so a row's arithmetic, reduction
// and stores run under the next row's loads (65536 x 2048 bf16 gate: 110 us,
// with one row a block 140).  Inputs: X [M, K] (gate: [M, 2K],
// the halves a | b), R [M, K] or NULL, gain [K] or NULL; H [M, K] or NULL
// receives x + r.  H may be X or R: a row is written after it was read, by the
// threads that read it.
template <typename T, int MODE, int FMT, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
    a8_rows_kernel(const T *X, const T *R, const float *__restrict__ gain, float eps, float inv_k,
                   T *H, uint8_t *__restrict__ codes, float *__restrict__ scales, int M, int K,
                   DevCtl *ctl) {
    constexpr int V = Vec<T>::n;
    __shared__ float2 part[64];
    int turn = 0;
    // X may be the previous kernel's output, and the outputs its input.  The
    // codes may be the next product's weights: whatever reads weights before
    // its own wait is launched by a pre-pass that has waited for this grid.
    pdl_wait_prior_grid();
    const int per_block = blockDim.x / TPR;
    const int t = threadIdx.x % TPR;
    const int64_t step = static_cast<int64_t>(gridDim.x) * per_block;
    int64_t row = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / TPR;

    uint4 in0[NV], in1[NV];               // x, or a; the residual, or b
    const auto load = [&](int64_t at) {
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = (i * TPR + t) * V;
            const bool have = at < M && k < K;
            const T *p = X + (MODE == kModeGate ? at * 2 * K : at * K) + k;
            in0[i] = have ? *reinterpret_cast<const uint4 *>(p) : zero;
            if (MODE == kModeGate) in1[i] = have ? *reinterpret_cast<const uint4 *>(p + K) : zero;
            if (MODE == kModeNorm && R)
                in1[i] = have ? *reinterpret_cast<const uint4 *>(R + at * K + k) : zero;
        }
    };
    load(row);
    // the block's groups make the same number of turns: they share barriers
    for (int64_t lead = row - threadIdx.x / TPR; lead < M; lead += step, row += step) {
        const bool live = row < M;
        float v[NV][V];
        float ss = 0.f;
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack(in0[i], v[i], X);
            if (MODE == kModeGate || (MODE == kModeNorm && R)) {
                float b[V];
                unpack(in1[i], b, X);
                if (MODE == kModeGate) {
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        const float2 y = silu_mul(make_float2(v[i][j], v[i][j + 1]),
                                                  make_float2(b[j], b[j + 1]));
                        v[i][j] = y.x;
                        v[i][j + 1] = y.y;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) v[i][j] += b[j];
                }
            }
        }
        load(row + step);
        if (MODE == kModeNorm && H) {
            // rounded once to the stream's type; the norm below is of the fp32 sum
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int k = (i * TPR + t) * V;
                if (live && k < K) *reinterpret_cast<uint4 *>(H + row * K + k) = pack(v[i], X);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = (i * TPR + t) * V;
            if (MODE == kModeNorm) {
#pragma unroll
                for (int j = 0; j < V; ++j) ss = fmaf(v[i][j], v[i][j], ss);
                if (gain && k < K) {
#pragma unroll
                    for (int j = 0; j < V; j += 4) {
                        const float4 g = __ldg(reinterpret_cast<const float4 *>(gain + k + j));
                        const float gg[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            mx = max(mx, abs_bits(v[i][j + q] * gg[q]));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) mx = max(mx, abs_bits(v[i][j]));
                }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    mx = MODE == kModeGate ? max_bits(mx, v[i][j]) : max(mx, abs_bits(v[i][j]));
            }
        }
        row_reduce<TPR, MODE == kModeNorm>(ss, mx, part, turn);
        float mul = 1.f;                  // scale = s0 * mul
        if (MODE == kModeNorm) {
            mul = rsqrtf(fmaf(ss, inv_k, eps));
            // The squares or h * gain have left fp32's range, or the products
            // are so small that their quotients would lose digits: the row once
            // more as y itself, from h * 2^-80 where the squares overflowed.  A
            // group agrees on this; groups that share barriers take the block's
            // vote.
            const bool redo = live && (!(ss <= FLT_MAX) || mx >= kInfBits || mx < kTinyBits);
            const bool any = (TPR == 32 || TPR >= 256) ? redo : __syncthreads_or(redo) != 0;
            if (any) {
                const float f = ss <= FLT_MAX ? 1.f : 0x1p-80f;
                float s2 = 0.f, none = 0.f;
                uint32_t m2 = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) s2 = fmaf(v[i][j] * f, v[i][j] * f, s2);
                row_reduce<TPR, true>(s2, m2, part, turn);
                const float r2 = rsqrtf(fmaf(s2, inv_k, eps * f * f));
                m2 = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int k = (i * TPR + t) * V;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        if (redo) v[i][j] = v[i][j] * f * r2;
                        m2 = max(m2,
                                 abs_bits(v[i][j] * (gain && k < K ? __ldg(gain + k + j) : 1.f)));
                    }
                }
                row_reduce<TPR, false>(none, m2, part, turn);
                if (redo) {
                    mx = m2;
                    mul = 1.f;
                }
            }
        }
        if (!live) continue;
        // A value that is not finite: the row has no scale; its codes are 0 and
        // the product gives NaN for it, and for it alone.
        const bool bad = mx >= kInfBits;
        const float amax = __uint_as_float(mx);
        const bool slow = mx < kTinyBits;
        const float s0 = slow ? __fdiv_rn(amax, FMT == kFmtQ8 ? 127.f : 448.f) : over_top<FMT>(amax);
        float inv = slow ? 0.f : __fdividef(1.f, s0), inv_lo = 0.f;
        if (FMT == kFmtE4M3 && !slow) {
            // the rest of Q / amax beyond inv, from its exact remainder
            inv = fmaf(fmaf(-inv, s0, 1.f), inv, inv);
            inv_lo = fmaf(-inv, amax, 448.f) * (inv * (1.f / 448.f));
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int k = (i * TPR + t) * V;
            if (k >= K) continue;
            if (MODE == kModeNorm) {
#pragma unroll
                for (int j = 0; j < V && gain; j += 4) {
                    const float4 g = __ldg(reinterpret_cast<const float4 *>(gain + k + j));
                    v[i][j] *= g.x;
                    v[i][j + 1] *= g.y;
                    v[i][j + 2] *= g.z;
                    v[i][j + 3] *= g.w;
                }
            }
            uint32_t w[V / 4];
            encode<FMT, V>(v[i], s0, inv, inv_lo, slow, w);
            if (bad) w[0] = w[V / 4 - 1] = 0u;
            if (V == 4)
                *reinterpret_cast<uint32_t *>(codes + row * K + k) = w[0];
            else
                *reinterpret_cast<uint2 *>(codes + row * K + k) = make_uint2(w[0], w[V / 4 - 1]);
        }
        if (t == 0) {
            scales[row] = bad ? __uint_as_float(0x7FC00000u) : s0 * mul;
            if (bad) atomicOr(&ctl->status, 1u << kStatusRange);
        }
    }
}

// Values of 8-bit rows: code * scale in fp32, rounded once to the type.  A warp
// takes kSpan vectors of one row at a time, all of its loads in flight at once.
constexpr int kSpan = 4 * 32;

template <typename T, int FMT>
__global__ void __launch_bounds__(256)
    a8_values_kernel(const uint8_t *__restrict__ codes, const float *__restrict__ scales,
                     T *__restrict__ out, int M, int vecs) {
    constexpr int V = Vec<T>::n;
    pdl_wait_prior_grid();
    const int lane = threadIdx.x & 31;
    const int spans = (vecs + kSpan - 1) / kSpan;
    const int64_t total = static_cast<int64_t>(M) * spans;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
         u < total; u += step) {
        const int64_t row = total <= INT32_MAX ? static_cast<int>(u) / spans : u / spans;
        const int first = static_cast<int>(u - row * spans) * kSpan + lane;
        const float s = __ldg(scales + row);
        uint2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = first + 32 * i;
            w[i] = make_uint2(0u, 0u);
            if (k < vecs) {
                const int64_t at = row * vecs + k;
                if (V == 4) w[i].x = __ldg(reinterpret_cast<const uint32_t *>(codes) + at);
                else w[i] = __ldg(reinterpret_cast<const uint2 *>(codes) + at);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = first + 32 * i;
            if (k >= vecs) break;
            float f[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint32_t b = ((j < 4 ? w[i].x : w[i].y) >> (8 * (j & 3))) & 0xFFu;
                if (FMT == kFmtQ8) {
                    f[j] = static_cast<float>(static_cast<int8_t>(b)) * s;
                } else {
                    const __half_raw h = __nv_cvt_fp8_to_halfraw(
                        static_cast<__nv_fp8_storage_t>(b), __NV_E4M3);
                    f[j] = __half2float(__half(h)) * s;
                }
            }
            reinterpret_cast<uint4 *>(out)[row * vecs + k] = pack(f, out);
        }
    }
}

cudaError_t launch_pdl(const void *fn, unsigned grid, unsigned block, void **args,
                       cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// Blocks of `kernel` that the current device holds at once (cached).
template <typename Kernel>
int resident_blocks(Kernel kernel, int threads, std::atomic<int> (&cache)[kMaxDevices]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
    int n = cache[dev].load(std::memory_order_acquire);
    if (n > 0) return n;
    int per = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, 0) != cudaSuccess ||
        per < 1) {
        cudaGetLastError();
        per = 1;
    }
    n = per * sm_count();
    cache[dev].store(n, std::memory_order_release);
    return n;
}

template <typename T, int MODE, int FMT, int TPR, int NV>
cudaError_t launch_rows(RowArgs a, cudaStream_t s) {
    constexpr int kBlock = TPR < 256 ? 256 : TPR;
    constexpr int kRows = kBlock / TPR;
    const T *X = static_cast<const T *>(a.X), *R = static_cast<const T *>(a.R);
    T *H = static_cast<T *>(a.H);
    void *args[] = {&X, &R, &a.gain, &a.eps, &a.inv_k, &H, &a.codes, &a.scales, &a.M, &a.K, &a.ctl};
    const auto kernel = a8_rows_kernel<T, MODE, FMT, TPR, NV>;
    static std::atomic<int> resident[kMaxDevices];
    const int64_t want = (static_cast<int64_t>(a.M) + kRows - 1) / kRows;
    const int64_t most = resident_blocks(kernel, kBlock, resident);
    unsigned grid = static_cast<unsigned>(want < most ? want : most), block = kBlock;
    if (kRows > 1 && want < 2 * sm_count()) {      // few rows: blocks of fewer rows, on more SMs
        const int rows = static_cast<int>((a.M + 2 * sm_count() - 1) / (2 * sm_count()));
        block = static_cast<unsigned>(rows * TPR);
        grid = static_cast<unsigned>((a.M + rows - 1) / rows);
    }
    return launch_pdl(reinterpret_cast<const void *>(kernel), grid, block, args, s);
}

// A group of `tpr` threads (32 to 1024), NV vectors a thread.
template <typename T, int MODE, int FMT, int NV>
cudaError_t launch_rows_nv(const RowArgs &a, int tpr, cudaStream_t s) {
    if (tpr <= 32) return launch_rows<T, MODE, FMT, 32, NV>(a, s);
    if (tpr == 64) return launch_rows<T, MODE, FMT, 64, NV>(a, s);
    if (tpr == 128) return launch_rows<T, MODE, FMT, 128, NV>(a, s);
    if (tpr == 256) return launch_rows<T, MODE, FMT, 256, NV>(a, s);
    if (tpr == 512) return launch_rows<T, MODE, FMT, 512, NV>(a, s);
    return launch_rows<T, MODE, FMT, 1024, NV>(a, s);
}

// Threads a row and vectors a thread.  Few rows, up to half of the threads that the
// device holds: 1 vector, for the shortest chain (80 x 512 bf16 norm: 1.7 us, with 2
// 2.4; 1001 x 512: 2.2 and 2.5; beyond, 1180 x 1024 fp32: 3.4 and 3.1).  Many rows: 3 where that
// leaves fewer threads idle than a power of two, else what keeps most bytes in
// flight for the registers it takes.  16-bit types 2: 65536 x 2048 bf16 gate 107
// us (1: 119, 4: 107), norm 144 (1: 152, 4: 159).  fp32 quantization 4: 65536 x 512
// 26 us (2: 28, 1: 37); gate 2: 4096 x 2048 12.8 us (4: 13.7); norm 1 up to 128
// vectors, then 2: 65536 x 512 68 us (2: 71, 4: 73), 65536 x 2048 267 us (1: 280).
// The longest rows take what 1024 threads need.
template <typename T, int MODE, int FMT>
cudaError_t launch_rows_k(const RowArgs &a, cudaStream_t s) {
    constexpr bool kWide = Vec<T>::n == 4;            // fp32
    constexpr int kMany = kWide && MODE == kModeQuant ? 4 : 2;
    const int vecs = a.K / Vec<T>::n;
    int room = 32;                                    // a power of two that holds the row
    while (room < vecs) room *= 2;
    if (room <= 512 && static_cast<int64_t>(a.M) * room <= 1024 * sm_count())
        return launch_rows_nv<T, MODE, FMT, 1>(a, room, s);
    if (room >= 128 && room <= 4096 && 4 * vecs <= 3 * room)
        return launch_rows_nv<T, MODE, FMT, 3>(a, room / 4, s);
    if (room == 32 || (kWide && MODE == kModeNorm && room <= 128))
        return launch_rows_nv<T, MODE, FMT, 1>(a, room, s);
    if (room == 64) return launch_rows<T, MODE, FMT, 32, 2>(a, s);
    if (room <= 1024 * kMany) return launch_rows_nv<T, MODE, FMT, kMany>(a, room / kMany, s);
    if (kMany < 4 && room <= 4096) return launch_rows<T, MODE, FMT, 1024, 4>(a, s);
    return launch_rows<T, MODE, FMT, 1024, kWide ? 8 : 4>(a, s);     // up to kMaxRowK
}

template <typename T, int MODE>
cudaError_t launch_rows_f(int fmt, const RowArgs &a, cudaStream_t s) {
    return fmt == kFmtQ8 ? launch_rows_k<T, MODE, kFmtQ8>(a, s)
                         : launch_rows_k<T, MODE, kFmtE4M3>(a, s);
}

template <typename T>
cudaError_t launch_values(int fmt, const uint8_t *codes, const float *scales, T *out, int M, int K,
                          cudaStream_t s) {
    int vecs = K / Vec<T>::n;
    void *args[] = {&codes, &scales, &out, &M, &vecs};
    const int64_t warps = static_cast<int64_t>(M) * ((vecs + kSpan - 1) / kSpan);
    const int64_t want = (warps + 7) / 8, most = 16 * static_cast<int64_t>(sm_count());
    const unsigned grid = static_cast<unsigned>(want < most ? want : most);
    const void *fn = fmt == kFmtQ8 ? reinterpret_cast<const void *>(a8_values_kernel<T, kFmtQ8>)
                                   : reinterpret_cast<const void *>(a8_values_kernel<T, kFmtE4M3>);
    return launch_pdl(fn, grid, 256, args, s);
}

}  // namespace

template <typename T>
cudaError_t row_operator(int mode, int fmt, const RowArgs &a, cudaStream_t s) {
    if (mode == kModeQuant) return launch_rows_f<T, kModeQuant>(fmt, a, s);
    if (mode == kModeNorm) return launch_rows_f<T, kModeNorm>(fmt, a, s);
    return launch_rows_f<T, kModeGate>(fmt, a, s);
}

template <typename T>
cudaError_t row_values(int fmt, const uint8_t *codes, const float *scales, void *out, int M, int K,
                       cudaStream_t s) {
    return launch_values(fmt, codes, scales, static_cast<T *>(out), M, K, s);
}

}  // namespace rtq
