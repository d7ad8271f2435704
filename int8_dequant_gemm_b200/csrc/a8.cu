// Product of 8-bit activations and 8-bit weights on the tensor cores' 8-bit
// instructions:
//
//   Y[m, o] = (sum_k Xc[m, k] * Wc[o, k]) * ws[o] * xs[m] + bias[o]
//
// with int8 codes (tcgen05.mma kind::i8, the sum exact in int32) or FP8 E4M3
// codes (kind::f8f6f4, fp32 sum).  The scales leave the sum because each is
// constant along k, so nothing is dequantized and both operands go from HBM to
// the tensor core as they are stored: TMA boxes of 128 bytes of K in the
// 128-byte-swizzled operand layout.
//
// Orientation as in the other tensor-core kernels: weight rows are the MMA's M
// (TMEM lanes), activation rows its N (TMEM columns).  A warp of the epilogue
// then holds 32 neighbouring outputs of one Y row, so plain stores are whole
// 128-byte segments of Y for every N, and few activation rows cost few columns.
// Measured and not kept: activation rows in lanes with 32-byte stores (a quarter
// of the store instructions; 276 against 204 us for 65536 x 4096 x 512 into
// fp32, 181 against 175 into bf16, then), and tiles of Y staged in shared memory
// and stored by TMA (19.8 against 17.5 us for 4096 x 4096 x 512).
// What bounds large products: 8192^3 the tensor cores (94 % of their cycles at 4096 x
// 8192 x 8192; 365 us); fp32 results of short K the bytes between L2 and the SMs,
// operands and Y together 10 TB/s, L1 82 % busy (65536 x 4096 x 512 205 us).  16-bit results
// move a third fewer with activations that stay (143 us, 7 TB/s): no unit is above 57 %
// (issue slots, L1; tensor cores 44), so it is the latency of the epilogue's steps; the
// same for ragged ones (20001 x 2003 x 1040 50 to 53 us, 7 TB/s, L1 64 %, issue slots 35 %,
// with two stores for one).
//
// Roles (20 warps): warp 0 TMA, warp 1 MMA issue, warps 4-19 epilogue (four per
// TMEM lane quadrant); warps 2-3 idle.
//
// Three shapes of the same code:
//   - persistent tiles of 128 weight rows x bn activation rows, one CTA each,
//     two accumulators so that a tile's epilogue runs under the next one's MMAs;
//   - the same on CTA pairs (PAIR): one cta_group::2 MMA over 256 weight rows,
//     each CTA staging its own 128 weight rows and half of the activation rows,
//     which stay for all weight tiles where K is short (RES);
//   - few tiles: K split over a cluster of `split` CTAs (SPLIT), one tile a cluster,
//     partial sums sent through distributed shared memory and added in rank order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kernels.cuh"
#include "tmapipe.cuh"

namespace rtq {
namespace {

constexpr int kKBytes = 128;                       // K of an atom: one swizzled row
constexpr int kABytes = kTileRows * kKBytes;       // 16 KB of weights an atom
// Atoms a stage: issuing a stage costs about 330 cycles beside its MMAs' 25 each,
// which one atom of a pair's 256-wide MMAs (128 cycles each) covers; narrower
// tiles take two at a time (80 x 512 x 2048 e4m3 5.0 -> 4.6 us, 512 x 4096 x 4096
// 12.3 -> 10.4; 8192^3 on pairs 369 -> 381).
constexpr int stage_atoms(int pair) { return pair ? 1 : 2; }
// Epilogue groups G of four warps, one per TMEM lane quadrant: 4 for persistent
// tiles, 1 where a CTA has one narrow tile: 192 threads, at most half an SM's
// registers and, up to 80 rows (32 with a split), half its shared memory, so that the next
// kernel's CTA starts beside it.  Wider tiles need more for their two stages and the
// split's partial sums, 119 to 199 KB.
constexpr int epi_warp0(int G) { return G == 1 ? 2 : 4; }
constexpr int cta_threads(int G) { return (epi_warp0(G) + 4 * G) * 32; }
constexpr int kMaxStages = 8;
constexpr int kResAtoms = 9;                       // K atoms of activations that stay (RES)
constexpr int kBand = 8;                           // activation tiles walked together
constexpr uint16_t kBoth = 3;                      // multicast mask: both CTAs of a pair
constexpr int kSmemMax = 200 * 1024;               // ring of stages (RES: and the activations)
constexpr int kSmemSmall = 100 * 1024;             // ring and partial sums for G = 1
constexpr int kChunk = 16;                         // activation rows an epilogue warp takes at once

struct A8Args {
    const float *xs, *ws, *bias;
    void *Y;
    int M, N, K, bn, stages, split;
    int n_o, n_m;            // weight tiles, activation tiles
    int acc_cols;
    int alt;                 // two epilogue sets take turns
    int res_off;             // after the ring, RES: the activations' atoms
    int red_off;             // after the ring, split: partial sums of this rank's columns,
                             // [rank][column][128]
    int tail_off;            // after these: each epilogue warp's activation
                             // scales [4 G][2][kWarpWords], barriers and words
};

__host__ __device__ constexpr int atom_bytes(int bn, int pair) {
    return kABytes + (pair ? bn / 2 : bn) * kKBytes;
}
__host__ __device__ constexpr int stage_bytes(int bn, int pair) {
    return stage_atoms(pair) * atom_bytes(bn, pair);
}

// RES: the K atoms of a CTA's activation rows.
__host__ inline int res_bytes(int bn, int nkb) { return nkb * (bn / 2) * kKBytes; }
constexpr int kWarpRows = 128;                     // activation rows of a tile an epilogue warp takes
constexpr int kWarpWords = kWarpRows + 64;         // their scales, then each lane's ws and bias
constexpr int scale_bytes(int G) { return 4 * G * 2 * kWarpWords * 4; }
constexpr int tail_bytes(int G) { return scale_bytes(G) + (2 * kMaxStages + 2 * kResAtoms + 5) * 8 + 16; }

// Instruction descriptors (A and B K-major): accumulator s32 (2) or f32 (1),
// operand type 1 = s8 of kind::i8, 0 = e4m3 of kind::f8f6f4.
__host__ __device__ constexpr uint32_t idesc_8bit(int fmt, int M, int N) {
    return ((fmt == kFmtQ8 ? 2u : 1u) << 4) | ((fmt == kFmtQ8 ? 1u : 0u) << 7) |
           ((fmt == kFmtQ8 ? 1u : 0u) << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

template <int FMT, bool PAIR>
__device__ __forceinline__ void mma_8bit(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
#define RTQ_MMA8(group, kind)                                                   \
    asm volatile(                                                               \
        "{\n\t.reg .pred p;\n\t"                                                \
        "setp.ne.b32 p, %4, 0;\n\t"                                             \
        "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, p;\n\t}" \
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)                   \
        : "memory")
    if (FMT == kFmtQ8) {
        if (PAIR) RTQ_MMA8("2", "i8");
        else RTQ_MMA8("1", "i8");
    } else {
        if (PAIR) RTQ_MMA8("2", "f8f6f4");
        else RTQ_MMA8("1", "f8f6f4");
    }
#undef RTQ_MMA8
}

// TMA load of a CTA of a pair: into this CTA's shared memory, its bytes
// counted on the mbarrier at `cbar` (a shared::cluster address in either CTA).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y,
                                                 uint32_t cbar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(cbar)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

template <int FMT>
__device__ __forceinline__ float acc_f32(uint32_t v) {
    return FMT == kFmtQ8 ? __int2float_rn(static_cast<int>(v)) : __uint_as_float(v);
}

__device__ __forceinline__ float to_type(float v, const float *) { return v; }
__device__ __forceinline__ __half to_type(float v, const __half *) { return __float2half_rn(v); }
__device__ __forceinline__ __nv_bfloat16 to_type(float v, const __nv_bfloat16 *) {
    return __float2bfloat16_rn(v);
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Two results of one output column (rows i, i + 1) as one register of the type.
__device__ __forceinline__ uint32_t pair_bits(float a, float b, const __half *) {
    const __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t pair_bits(float a, float b, const __nv_bfloat16 *) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// Turns NaN in either half once a result is not finite in its type.
__device__ __forceinline__ void watch(uint32_t &nf, uint32_t w, const __half *) {
    asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(nf) : "r"(w), "r"(0u));
}
__device__ __forceinline__ void watch(uint32_t &nf, uint32_t w, const __nv_bfloat16 *) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(nf) : "r"(w), "r"(0u));
}
__device__ __forceinline__ void watch(uint32_t &nf, float v) {
    nf = __float_as_uint(fmaf(v, 0.f, __uint_as_float(nf)));
}

// A chunk of 16 activation rows of one weight row: y = acc * ws * xs + bias in
// fp32 (fp32 results), or rounded and packed, rows 2i and 2i + 1 in word i
// (16-bit results).  `xs`: the rows' scales in shared memory.  `nf` turns NaN once
// one of the chunk's results, beyond the tensor's edge or not, is not finite.
template <int FMT, typename YT>
__device__ __forceinline__ void finish_chunk(uint32_t (&v)[kChunk], uint32_t xs, float ws, float bo,
                                             uint32_t &nf, const YT *type) {
    const float2 ws2 = make_float2(ws, ws), bo2 = make_float2(bo, bo);
#pragma unroll
    for (int i = 0; i < kChunk; i += 4) {
        const uint4 f = lds_v4(xs + 4 * i);
        const float2 x0 = make_float2(__uint_as_float(f.x), __uint_as_float(f.y));
        const float2 x1 = make_float2(__uint_as_float(f.z), __uint_as_float(f.w));
        const float2 a0 = make_float2(acc_f32<FMT>(v[i]), acc_f32<FMT>(v[i + 1]));
        const float2 a1 = make_float2(acc_f32<FMT>(v[i + 2]), acc_f32<FMT>(v[i + 3]));
        const float2 y0 = __ffma2_rn(__fmul2_rn(a0, ws2), x0, bo2);
        const float2 y1 = __ffma2_rn(__fmul2_rn(a1, ws2), x1, bo2);
        if constexpr (sizeof(YT) == 2) {
            v[i / 2] = pair_bits(y0.x, y0.y, type);
            v[i / 2 + 1] = pair_bits(y1.x, y1.y, type);
            watch(nf, v[i / 2], type);
            watch(nf, v[i / 2 + 1], type);
        } else {
            watch(nf, y0.x);
            watch(nf, y0.y);
            watch(nf, y1.x);
            watch(nf, y1.y);
            v[i] = __float_as_uint(y0.x);
            v[i + 1] = __float_as_uint(y0.y);
            v[i + 2] = __float_as_uint(y1.x);
            v[i + 3] = __float_as_uint(y1.y);
        }
    }
}

// A finished chunk of 32 weight rows: y = lane 0's output of its first row, the same in
// all lanes, so that rows step in uniform registers (65536 x 4096 x 512 bf16 157 us;
// with 64-bit addresses a lane, 58 % of all issue slots taken, 174).
// `whole`: every lane of the warp has an output.  16-bit results of an even N
// go out as pairs: lanes 2i and 2i + 1 trade one value of two rows, and each
// stores two neighbours of one row.  `seen`: finish_chunk's nf of this chunk; of a
// chunk at the edge only the results that exist count toward nf.
template <typename YT>
__device__ __forceinline__ void store_chunk(const uint32_t (&v)[kChunk], YT *y, int N, int rows,
                                            bool live, bool whole, uint32_t seen, uint32_t &nf) {
    const size_t ld = static_cast<size_t>(N) * sizeof(YT);
    const uint32_t lane = threadIdx.x & 31;
    char *yr = reinterpret_cast<char *>(y);
    if (whole && rows >= kChunk) {
        nf |= seen;
        if constexpr (sizeof(YT) == 2) {
            if ((N & 1) == 0 && N < (1 << 30)) {       // a row fits a 32-bit offset
                const uint32_t odd = lane & 1;
                const uint32_t sel = odd ? 0x3276u : 0x5410u;
                const uint32_t at = (lane - odd) * 2 + (odd ? static_cast<uint32_t>(ld) : 0u);
#pragma unroll
                for (int i = 0; i < kChunk / 2; ++i, yr += 2 * ld) {
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, v[i], 1);
                    *reinterpret_cast<uint32_t *>(yr + at) = __byte_perm(v[i], got, sel);
                }
                return;
            }
#pragma unroll
            for (int i = 0; i < kChunk; ++i, yr += ld)
                *reinterpret_cast<uint16_t *>(yr + lane * 2) =
                    static_cast<uint16_t>(v[i / 2] >> (16 * (i & 1)));
        } else {
#pragma unroll
            for (int i = 0; i < kChunk; ++i, yr += ld)
                *reinterpret_cast<uint32_t *>(yr + lane * 4) = v[i];
        }
        return;
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < kChunk; ++i, yr += ld)
        if (i < rows) {
            if constexpr (sizeof(YT) == 2) {
                const uint32_t one = (v[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
                watch(nf, one, y);
                *reinterpret_cast<uint16_t *>(yr + lane * 2) = static_cast<uint16_t>(one);
            } else {
                watch(nf, __uint_as_float(v[i]));
                *reinterpret_cast<uint32_t *>(yr + lane * 4) = v[i];
            }
        }
}

// Tile t of the walk: bands of kBand activation tiles, all weight tiles of a
// band, activation tile fastest.  The tiles that run at once then share few
// operand rows, which stay in L2.  `res`: all weight tiles of one activation tile
// after another, each group of CTAs a contiguous share.
struct TileAt {
    int m, o;
    __device__ TileAt(int t, int n_m, int n_o, bool res) {
        if (res) {
            m = t / n_o;
            o = t - m * n_o;
            return;
        }
        const int band = t / (kBand * n_o);
        const int m0 = band * kBand, mb = min(kBand, n_m - m0);
        const int r = t - band * kBand * n_o;
        m = m0 + r % mb;
        o = r / mb;
    }
};

__host__ __device__ inline int share_of(int n, int i, int parts) {
    return static_cast<int>(static_cast<int64_t>(n) * i / parts);
}

template <int FMT, typename YT, bool PAIR, int G, bool SPLIT, bool RES>
__global__ void __launch_bounds__(cta_threads(G), G == 1 ? 2 : 1)
    a8_qgemm_kernel(const __grid_constant__ CUtensorMap w_map,
                    const __grid_constant__ CUtensorMap x_map, const A8Args a, DevCtl *ctl) {
    constexpr int kEpiWarp0 = epi_warp0(G), kEpiWarps = 4 * G, kAtoms = stage_atoms(PAIR);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t base = smem_addr(smem);
    uint8_t *tail = smem + a.tail_off;
    float *xs_s = reinterpret_cast<float *>(tail);
    uint64_t *full = reinterpret_cast<uint64_t *>(tail + scale_bytes(G));
    uint64_t *empty = full + kMaxStages;
    uint64_t *acc_full = empty + kMaxStages, *acc_empty = acc_full + 2, *drain = acc_empty + 2;
    uint64_t *x_full = drain + 1, *x_empty = x_full + kResAtoms;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(x_empty + kResAtoms);
    volatile uint32_t *failed = tmem_slot + 1;     // split: a rank has no sum

    // (warp: by a shuffle, so that the compiler knows it to be the same in all lanes)
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = static_cast<int>(threadIdx.x & 31);
    const int split = SPLIT ? a.split : 1;
    const int csize = PAIR ? 2 : split;
    const int rank = csize > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const bool leader = !PAIR || rank == 0;
    const int nkb = (a.K + kKBytes - 1) / kKBytes;
    const int kb0 = SPLIT ? nkb * rank / split : 0, kb1 = SPLIT ? nkb * (rank + 1) / split : nkb;
    const int n_tiles = a.n_o * a.n_m;
    // tiles first, first + step, ... below end
    const int group = static_cast<int>(blockIdx.x) / csize;
    const int groups_n = static_cast<int>(gridDim.x) / csize;
    const int first = RES ? share_of(n_tiles, group, groups_n) : group;
    const int end = RES ? share_of(n_tiles, group + 1, groups_n) : n_tiles;
    const int step = RES ? 1 : groups_n;
    const int abytes = RES ? kABytes : atom_bytes(a.bn, PAIR), sbytes = kAtoms * abytes;
    const int xbytes = atom_bytes(a.bn, PAIR) - kABytes;
    const unsigned long long *lim = &ctl->wait_ns;
    const bool inject = leader && ctl->inject;     // read before the wait below

    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], (PAIR ? 2 : 1) * (a.alt ? kEpiWarps / 2 : kEpiWarps));
        }
        if (RES)
            for (int i = 0; i < nkb; ++i) {
                mbar_init(&x_full[i], 1);
                mbar_init(&x_empty[i], 1);
            }
        mbar_init(drain, 1);
        *failed = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 64) {
        prefetch_map(&w_map);
        prefetch_map(&x_map);
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(tmem_slot, static_cast<uint32_t>(a.acc_cols));
            tmem_relinquish_pair();
        } else {
            tmem_alloc(tmem_slot, static_cast<uint32_t>(a.acc_cols));
            tmem_relinquish();
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (PAIR) cluster_sync();      // the peer's barriers are initialised
    else if (SPLIT) cluster_arrive();      // this rank takes its peers' sums
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // Every operand, the weights and scales too, may be the previous kernel's
    // output.
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    bool ok = true;
    float wsc[4] = {1.f, 1.f, 1.f, 1.f}, bo[4] = {};       // of the split-K sum's weight rows
    if (SPLIT && warp >= kEpiWarp0) {
        const TileAt at(first, a.n_m, a.n_o, RES);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = at.o * kTileRows + 4 * lane + i;
            if (n < a.N && a.ws) wsc[i] = __ldg(a.ws + n);
            if (n < a.N && a.bias) bo[i] = __ldg(a.bias + n);
        }
    }

    // The TMA and MMA warps run their loops whole and in uniform control flow -- a
    // wait that gives up clears `good`, which skips later waits and issues but
    // no loop -- so that counters and descriptors stay in uniform registers.  With
    // loops left early, or run by one lane, a stage took 300 ns to issue.
    if (warp == 0) {
        // ============================================================ TMA
        // (Test hook: with `inject` the first weight box is never requested.)
        bool good = true;
        int s = 0, j = 0, x_loads = 0;
        uint32_t par = 1;
        for (int t = first; t < end; t += step) {
            const TileAt at(t, a.n_m, a.n_o, RES);
            const int oy = (PAIR ? 2 * at.o + rank : at.o) * kTileRows;
            const int my = at.m * a.bn + (PAIR ? rank * (a.bn / 2) : 0);
            const bool x_new = RES && (t == first || at.o == 0);
            if (x_new) ++x_loads;
            for (int kb = kb0; kb < kb1; kb += kAtoms, ++j) {
                if (x_new) {
                    // this atom of the last activation tile has been multiplied
                    if (good && x_loads > 1)
                        good = mbar_wait(&x_empty[kb], static_cast<uint32_t>(x_loads) & 1u, lim);
                    if (elect_one() && good) {
                        const uint32_t cbar = cluster_map(smem_addr(&x_full[kb]), 0);
                        if (leader) mbar_expect_tx(&x_full[kb], static_cast<uint32_t>(2 * xbytes));
                        tma_load_2d_pair(base + static_cast<uint32_t>(a.res_off + kb * xbytes), &x_map,
                                         kb * kKBytes, my, cbar);
                    }
                }
                if (good && j >= a.stages) good = mbar_wait(&empty[s], par, lim);
                const int atoms = min(kAtoms, kb1 - kb);
                const uint32_t bytes = static_cast<uint32_t>((PAIR ? 2 : 1) * atoms * abytes);
                if (elect_one() && good) {
                    const uint32_t cbar = PAIR ? cluster_map(smem_addr(&full[s]), 0) : 0;
                    if (leader) mbar_expect_tx(&full[s], bytes);
#pragma unroll
                    for (int u = 0; u < kAtoms; ++u) {
                        if (u == atoms) break;
                        const uint32_t dst = base + static_cast<uint32_t>(s * sbytes + u * abytes);
                        const int x = (kb + u) * kKBytes;
                        const bool skip = inject && j == 0 && u == 0;
                        if (PAIR) {
                            if (!skip) tma_load_2d_pair(dst, &w_map, x, oy, cbar);
                            if (!RES) tma_load_2d_pair(dst + kABytes, &x_map, x, my, cbar);
                        } else {
                            if (!skip) tma_load_2d(dst, &w_map, x, oy, &full[s]);
                            tma_load_2d(dst + kABytes, &x_map, x, my, &full[s]);
                        }
                    }
                }
                if (++s == a.stages) {
                    s = 0;
                    par ^= 1;
                }
            }
        }
        // Before the CTA may exit, every box it requested has landed (immediate
        // unless a consumer gave up; a pair's boxes are counted by its even CTA,
        // which the odd one meets before it exits).  A box that was not
        // requested after a failure makes its wait run out.
        if (leader) {
            for (int i = 0; i < a.stages && i < j; ++i) {
                const int last_j = i + ((j - 1 - i) / a.stages) * a.stages;
                if (good && !(last_j == 0 && inject))
                    mbar_wait(&full[i], static_cast<uint32_t>(last_j / a.stages) & 1u, lim);
            }
            if (RES)
                for (int kb = 0; kb < nkb && x_loads > 0 && good; ++kb)
                    mbar_wait(&x_full[kb], static_cast<uint32_t>(x_loads - 1) & 1u, lim);
        }
        ok = __all_sync(0xffffffffu, good);
    } else if (warp == 1) {
        // ============================================================ MMA issue
        if (leader) {
            const uint32_t idesc = idesc_8bit(FMT, (PAIR ? 2 : 1) * kTileRows, a.bn);
            bool good = true;
            int s = 0, n_local = 0, x_loads = 0;
            uint32_t par = 0;
            for (int t = first; t < end; t += step, ++n_local) {
                const int o_at = RES ? t % a.n_o : 0;
                const bool x_new = RES && (t == first || o_at == 0);
                const bool x_last = RES && (t + 1 == end || o_at == a.n_o - 1);
                if (x_new) ++x_loads;
                const int b = n_local & 1;
                if (good && n_local >= 2)
                    good = mbar_wait(&acc_empty[b], static_cast<uint32_t>((n_local / 2) - 1) & 1u,
                                     lim);
                const uint32_t d = tmem + static_cast<uint32_t>(b * a.bn);
                for (int kb = kb0; kb < kb1; kb += kAtoms) {
                    if (x_new && good)
                        good = mbar_wait(&x_full[kb], static_cast<uint32_t>(x_loads - 1) & 1u, lim);
                    if (good) good = mbar_wait(&full[s], par, lim);
                    tc_fence_after_sync();
                    const uint32_t st = base + static_cast<uint32_t>(s * sbytes);
                    const uint64_t ad = sw128_kmajor_desc(st);
                    const uint64_t bd = sw128_kmajor_desc(
                        RES ? base + static_cast<uint32_t>(a.res_off + kb * xbytes) : st + kABytes);
                    const uint64_t next = static_cast<uint64_t>(abytes >> 4);
                    // K left in this CTA's slice; the rest of the last atom is zero fill
                    const int left = min(a.K, kb1 * kKBytes) - kb * kKBytes;
                    if (elect_one() && good) {
#pragma unroll
                        for (int kk = 0; kk < 4 * kAtoms; ++kk)        // 32 K each
                            if (kk * 32 < left)
                                mma_8bit<FMT, PAIR>(d, ad + (kk >> 2) * next + 2 * (kk & 3),
                                                    bd + (kk >> 2) * next + 2 * (kk & 3), idesc,
                                                    (kb > kb0 || kk > 0) ? 1u : 0u);
                        if (PAIR) tc_commit_pair_mc(&empty[s], kBoth);
                        else tc_commit(&empty[s]);
                        if (x_last) tc_commit_pair_mc(&x_empty[kb], kBoth);
                    }
                    if (++s == a.stages) {
                        s = 0;
                        par ^= 1;
                    }
                }
                if (elect_one() && good) {
                    if (PAIR) tc_commit_pair_mc(&acc_full[b], kBoth);
                    else tc_commit(&acc_full[b]);
                }
            }
            ok = __all_sync(0xffffffffu, good);
            if (!ok) {                       // issued MMAs end before the CTA does
                if (elect_one()) {
                    if (PAIR) tc_commit_pair_mc(drain, 1);
                    else tc_commit(drain);
                    mbar_wait(drain, 0, lim);
                }
                __syncwarp();
            }
        }
    } else if (warp >= kEpiWarp0) {
        // ============================================================ epilogue
        // Several tiles a CTA (alt): two sets of eight warps take turns, so that
        // one set's loads and arithmetic run under the other's stores and each
        // has two tiles' time for its latencies.  One tile: all warps share it.
        const int q = warp & 3;
        const int ew = warp - kEpiWarp0;
        const int set = a.alt ? ew >> 3 : 0, groups = a.alt ? G / 2 : G;
        const int h = a.alt ? (ew >> 2) & 1 : ew >> 2;
        const int turn = a.alt ? 2 : 1, chunk_step = 2 * kChunk * groups;
        const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
        YT *const Y = static_cast<YT *>(a.Y);
        uint32_t nf = 0;                     // NaN once an output is not finite
        // The next tile's scales and bias are copied while this one is stored, past
        // the registers, of which the arithmetic needs all.  Each warp keeps the scales
        // of its own activation rows: the warps share no barrier, which a warp whose
        // wait gave up would not come to.
        uint32_t xs_w = smem_addr(xs_s) + ew * (2 * kWarpWords * 4), flip = 0;
        auto fetch = [&](int t, uint32_t to) {
            if (SPLIT || t >= end) return;
            const TileAt at(t, a.n_m, a.n_o, RES);
#pragma unroll
            for (int i = 0; i < kWarpRows / 32; ++i) {
                const int c = 32 * h + chunk_step * i + lane, m = at.m * a.bn + c;
                const bool there = c < a.bn && m < a.M;
                cp_async_word(to + 4 * (32 * i + lane), a.xs + (there ? m : 0), there);
            }
            const int o = (PAIR ? 2 * at.o + rank : at.o) * kTileRows + q * 32 + lane;
            const bool there = o < a.N;
            const uint32_t own = to + 4 * (kWarpRows + lane);
            if (a.ws) cp_async_word(own, a.ws + (there ? o : 0), there);
            else sts_u32(own, __float_as_uint(1.f));
            if (a.bias) cp_async_word(own + 128, a.bias + (there ? o : 0), there);
            else sts_u32(own + 128, 0);
        };
        fetch(first + set * step, xs_w);
        if (SPLIT) cluster_wait();      // the peers have started
        int n_local = set;
        for (int t = first + set * step; t < end && ok; t += turn * step, n_local += turn) {
            const TileAt at(t, a.n_m, a.n_o, RES);
            const int b = n_local & 1;
            const int m0 = at.m * a.bn;
            const int mlim = min(a.bn, a.M - m0);
            if (SPLIT) {
                // each rank's columns of this partial sum into its shared memory
                ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[0], 0, lim));
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t own = static_cast<uint32_t>(a.bn / split);
                const uint32_t to = base + static_cast<uint32_t>(a.red_off) +
                                    (rank * own * kTileRows + q * 32 + lane) * 4;
                uint32_t peer = 0, at_p = 0;
                for (int c = 0; c < a.bn; c += kChunk) {
                    uint32_t v[kChunk];
                    tmem_ld_x16(tq + static_cast<uint32_t>(c), v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < kChunk; ++i) {
                        st_cluster_u32(cluster_map(to + at_p * kTileRows * 4, peer), v[i]);
                        if (++at_p == own) {
                            at_p = 0;
                            ++peer;
                        }
                    }
                }
                break;
            }
            const uint32_t mine = xs_w + flip;
            flip ^= kWarpWords * 4;
            cp_async_wait_all();
            __syncwarp();                    // and the tile before's have been read
            const float ws = __uint_as_float(lds_u32(mine + 4 * (kWarpRows + lane)));
            const float bo = __uint_as_float(lds_u32(mine + 4 * (kWarpRows + 32 + lane)));
            const int o = (PAIR ? 2 * at.o + rank : at.o) * kTileRows + q * 32 + lane;
            const bool live = o < a.N;
            fetch(t + turn * step, xs_w + flip);
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&acc_full[b], static_cast<uint32_t>(n_local / 2) & 1u, lim));
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t tb = tq + static_cast<uint32_t>(b * a.bn);
            YT *yo = Y + static_cast<size_t>(m0) * a.N + (o - lane);
            const bool whole = __all_sync(0xffffffffu, live);
            const auto put = [&](uint32_t (&v)[kChunk], int c, uint32_t xs) {
                uint32_t seen = 0;
                finish_chunk<FMT>(v, xs, ws, bo, seen, Y);
                store_chunk(v, yo + static_cast<size_t>(c) * a.N, a.N, mlim - c, live, whole, seen,
                            nf);
            };
            int c = 2 * kChunk * h;
            uint32_t xs = mine;
            do {
                uint32_t v0[kChunk], v1[kChunk];
                if (c < a.bn) tmem_ld_x16(tb + static_cast<uint32_t>(c), v0);
                if (c + kChunk < a.bn) tmem_ld_x16(tb + static_cast<uint32_t>(c + kChunk), v1);
                tmem_ld_wait();
                if (c + chunk_step >= a.bn) {    // the accumulator has been read
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR) mbar_arrive_remote(cluster_map(smem_addr(&acc_empty[b]), 0));
                        else mbar_arrive(&acc_empty[b]);
                    }
                }
                if (c < a.bn) put(v0, c, xs);
                if (c + kChunk < a.bn) put(v1, c + kChunk, xs + 4 * kChunk);
                c += chunk_step;
                xs += 4 * 32;
            } while (c < a.bn);
        }
        cp_async_wait_all();                 // after a wait that gave up
        if (__any_sync(0xffffffffu, (nf & 0x7FFF7FFFu) != 0) && lane == 0)
            atomicOr(&ctl->status, 1u << kStatusRange);
    }
    if (SPLIT && warp < kEpiWarp0) cluster_wait();
    if (!ok) {
        atomicOr(&ctl->status, 1u << kStatusTimeout);
        if (SPLIT)
            for (int r = 0; r < split; ++r)
                st_cluster_u32(cluster_map(smem_addr(const_cast<uint32_t *>(failed)),
                                           static_cast<uint32_t>(r)), 1);
    }
    tc_fence_before_sync();
    if (PAIR || SPLIT) cluster_sync();
    else __syncthreads();
    if (SPLIT && warp >= kEpiWarp0 && *failed == 0) {
        // ============================================================ split-K sum
        // Each rank has sent its peers their columns, a store a column and warp, and
        // one cluster barrier orders them (80 x 512 x 2048 e4m3: 3.7 us; with the sums
        // read from the peers, between two barriers, 4.6).  Rank r of the cluster adds
        // and stores columns [bn r / split, bn (r + 1) / split): all ranks' partial sums
        // of them, in rank order.
        const TileAt at(first, a.n_m, a.n_o, RES);
        YT *const Y = static_cast<YT *>(a.Y);
        float nf = 0.f;
        const int own = a.bn / split, m0 = at.m * a.bn + rank * own;
        const int c1 = min(own, a.M - m0);
        const int o = at.o * kTileRows + 4 * lane;
        for (int c = warp - kEpiWarp0; c < c1; c += kEpiWarps) {
            const float xv = __ldg(a.xs + m0 + c);
            const float *part =
                reinterpret_cast<const float *>(smem + a.red_off) + c * kTileRows + 4 * lane;
            float sf[4] = {0.f, 0.f, 0.f, 0.f};
            int si[4] = {0, 0, 0, 0};
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < split) {
                    const float4 p = *reinterpret_cast<const float4 *>(part + r * own * kTileRows);
                    const float e[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (FMT == kFmtQ8) si[i] += __float_as_int(e[i]);
                        else sf[i] += e[i];
                    }
                }
            YT *yo = Y + static_cast<size_t>(m0 + c) * a.N + o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (o + i < a.N) {
                    const float s = FMT == kFmtQ8 ? __int2float_rn(si[i]) : sf[i];
                    const YT y = to_type(fmaf(s * wsc[i], xv, bo[i]), Y);
                    nf = fmaf(to_f32(y), 0.f, nf);
                    yo[i] = y;
                }
            }
        }
        if (__any_sync(0xffffffffu, nf != 0.f) && lane == 0)
            atomicOr(&ctl->status, 1u << kStatusRange);
    }
    if (warp == 1) {
        tc_fence_after_sync();
        if (PAIR) tmem_dealloc_pair(tmem, static_cast<uint32_t>(a.acc_cols));
        else tmem_dealloc(tmem, static_cast<uint32_t>(a.acc_cols));
    }
}

template <int FMT, typename YT, bool PAIR, int G, bool SPLIT, bool RES>
cudaError_t launch_a8(const A8Plan &plan, const void *Xq, const float *xs, const void *Wq,
                      const float *wsc, const float *bias, void *Y, int M, int N, int K,
                      DevCtl *ctl, cudaStream_t st) {
    static std::atomic<bool> attr_done[kMaxDevices];
    static std::atomic<int> pairs_cache[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const auto kernel = a8_qgemm_kernel<FMT, YT, PAIR, G, SPLIT, RES>;
    if ((e = smem_attr_once(kernel, 227 * 1024, dev, attr_done)) != cudaSuccess) return e;
    A8Args a = {};
    a.xs = xs;
    a.ws = wsc;
    a.bias = bias;
    a.Y = Y;
    a.M = M;
    a.N = N;
    a.K = K;
    a.bn = plan.bn;
    a.split = SPLIT ? plan.split : 1;
    const int nkb = (K + kKBytes - 1) / kKBytes;
    const int ot = PAIR ? 2 * kTileRows : kTileRows;
    a.n_o = static_cast<int>((static_cast<int64_t>(N) + ot - 1) / ot);
    a.n_m = static_cast<int>((static_cast<int64_t>(M) + a.bn - 1) / a.bn);
    const int csize = PAIR ? 2 : a.split;
    const int64_t tiles = static_cast<int64_t>(a.n_o) * a.n_m;
    if (tiles > (int64_t(1) << 30)) return cudaErrorInvalidValue;

    CUtensorMap x_map, w_map;
    if (!encode_tma_2d(&x_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, Xq, K, M, kKBytes,
                       CU_TENSOR_MAP_SWIZZLE_128B, PAIR ? a.bn / 2 : a.bn) ||
        !encode_tma_2d(&w_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, Wq, K, N, kKBytes,
                       CU_TENSOR_MAP_SWIZZLE_128B, kTileRows))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(cta_threads(G), 1, 1);
    cfg.stream = st;
    int64_t grid = tiles * a.split;          // G = 1: one tile a CTA or cluster
    if (PAIR) {
        // the clusters' shared memory barely depends on the plan: one count serves all
        cudaLaunchConfig_t most = cfg;
        most.dynamicSmemBytes = kSmemMax + tail_bytes(G) + 1024;
        grid = 2 * std::min<int64_t>(tiles, resident_pairs(kernel, most, dev, pairs_cache));
    } else if (G > 1 && a.split == 1) {
        grid = std::min<int64_t>(tiles, sm_count());
    }
    const int64_t share = (tiles * csize + grid - 1) / grid;   // tiles a CTA or cluster
    a.alt = share > 1;
    // Clusters wait for their peers, so none of their CTAs may wait in tcgen05.alloc
    // for another cluster's: pairs leave no registers beside them on an SM, and a CTA
    // of a split takes a larger part of the shared memory than of the 512 columns
    // (128, 64, 32 columns: at least 98, 75, 52 KB of 227).
    a.acc_cols = 32;
    while (a.acc_cols < (a.alt ? 2 : 1) * a.bn) a.acc_cols *= 2;
    const int sbytes = RES ? kABytes : stage_bytes(a.bn, PAIR);
    const int res = RES ? res_bytes(a.bn, nkb) : 0, red = a.split > 1 ? a.bn * kTileRows * 4 : 0;
    const int fit = std::max(2, ((G == 1 ? kSmemSmall : kSmemMax) - red - res) / sbytes);
    a.stages = static_cast<int>(std::min<int64_t>(
        std::min(kMaxStages, fit),
        share * ((((nkb + a.split - 1) / a.split) + stage_atoms(PAIR) - 1) / stage_atoms(PAIR))));
    a.res_off = a.stages * sbytes;
    a.red_off = a.res_off + res;
    a.tail_off = a.red_off + red;
    cfg.dynamicSmemBytes = a.tail_off + tail_bytes(G) + 1024;
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cudaLaunchAttribute attr[2];
    int n = 0;
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
    if (csize > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = csize;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, w_map, x_map, a, ctl);
}

// Pairs: an activation tile stays in shared memory for all weight tiles (RES), which
// takes half of the operand bytes off the way from L2, where the other operand's ring
// keeps enough stages, the weights stay in L2 and there is more than one weight
// tile.  It gains most where rows of K lie across L2 lines, a piece over two; it
// loses where rows of Y begin inside a 32-byte sector and Y is larger than L2, unless
// K is long: its walk leaves the sectors at its tiles' edges half written for
// longer.  Time kept over time streamed, means of 2200 timings (M 12000 to 65536, N
// 300 to 8192):
//   K not a multiple of 64, by pieces of 128   2     3     4     5     7     8
//     Y of 128 MB and more, whole rows, bf16  0.95  0.91  0.85  0.82  0.80  0.80
//     the same, fp32                          1.04  0.99  0.94  0.90  0.87  0.89
//     ragged rows, bf16                       1.26  1.21  1.10  0.99  0.86  0.82
//     ragged rows, fp32                       1.07  1.16  1.21  1.13  0.98  0.88
//     Y below 128 MB, the worst of the four   1.12  1.07  1.00  0.98  0.97  0.97
//     and the best                            0.95  0.88  0.88  0.88  0.88  0.85
//   K an odd multiple of 64, 6 and 8 pieces: bf16 0.94 to 1.07, fp32 0.90 to 1.03 (ragged
//     and large 1.22 and 1.05); 3 pieces 1.0 to 1.3, 9 0.9 to 1.1
//   K a multiple of 128: 1.0 to 1.3, but for whole rows of N >= 4096, bf16 up to 6
//     pieces 0.93 to 1.01, fp32 6 pieces 0.90 to 0.96
// One weight tile: 0.99 to 1.06 bf16, 0.90 to 1.03 fp32.
bool activations_stay(int M, int N, int K, size_t y_bytes) {
    const int nkb = (K + kKBytes - 1) / kKBytes;
    if (nkb > kResAtoms || static_cast<int64_t>(N) * K > (int64_t(32) << 20) || N <= 2 * kTileRows)
        return false;
    const bool half = y_bytes == 2, whole = N * y_bytes % 32 == 0;
    const bool large = M * (N * y_bytes) >= (size_t(128) << 20);
    if (K % 128 == 0) return whole && N >= 4096 && nkb <= 6 && (half || nkb == 6);
    if (K % 64 == 0) return nkb >= 6 && nkb <= 8 && (whole || half || !large);
    if (large && whole && half) return nkb >= 2;
    return nkb >= (large && !whole ? (half ? 5 : 8) : 4);
}

template <int FMT, typename YT>
cudaError_t launch_a8_p(const A8Plan &p, const void *Xq, const float *xs, const void *Wq,
                        const float *wsc, const float *bias, void *Y, int M, int N, int K,
                        DevCtl *ctl, cudaStream_t s) {
    if (p.pair && activations_stay(M, N, K, sizeof(YT)))
        return launch_a8<FMT, YT, true, 4, false, true>(p, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
    if (p.pair)
        return launch_a8<FMT, YT, true, 4, false, false>(p, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
    if (p.split > 1)
        return launch_a8<FMT, YT, false, 1, true, false>(p, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
    if (p.small)
        return launch_a8<FMT, YT, false, 1, false, false>(p, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
    return launch_a8<FMT, YT, false, 4, false, false>(p, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
}

template <int FMT>
cudaError_t launch_a8_y(const A8Plan &p, int dtype, const void *Xq, const float *xs, const void *Wq,
                        const float *wsc, const float *bias, void *Y, int M, int N, int K,
                        DevCtl *ctl, cudaStream_t s) {
    if (dtype == RT_DTYPE_F32)
        return launch_a8_p<FMT, float>(p, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
    if (dtype == RT_DTYPE_F16)
        return launch_a8_p<FMT, __half>(p, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
    return launch_a8_p<FMT, __nv_bfloat16>(p, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
}

}  // namespace

int sm_count() {
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return n;
    }
    const int known = cache[dev].load(std::memory_order_acquire);
    if (known > 0) return known;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    cache[dev].store(n, std::memory_order_release);
    return n;
}

// The plan of least estimated time.  The estimate (in us, beyond the 1.76 that a launch
// takes): an SM takes in 128-byte rows of operands at one per 0.98 to 1.16 ns (the
// smaller ring of G = 1 less well), which is slower than the MMAs they feed; a tile's
// epilogue takes 0.04 + 0.0094 bn; a split adds its cluster and the exchange of partial
// sums, a pair its handshakes; in a walk of tiles load and epilogue hide little of each
// other, since both are bytes between the SM and L2.  Rows whose length is no
// multiple of 128 bytes lie across two L2 lines a piece and count 1.5 times (20001 x
// 2048 x 1040 bf16 47 us, K = 1024 36).  Weights of more than 60 MB come from HBM,
// faster the more CTAs ask for them (16 x 8192 x 8192 on 64, 128 and 256 CTAs: 22, 16
// and 14.7 us).  The constants are a fit to timings of every plan at M = 1 to
// 4096 and twelve weight shapes from 512 x 64 to 8192 x 8192, on the kernels of then; the
// plan taken was on average 1 % slower than the best of a shape, at most 20 %.
A8Plan plan_a8(int fmt, int M, int N, int K, int sms) {
    const int nkb = (K + kKBytes - 1) / kKBytes;
    const int n_o = static_cast<int>((static_cast<int64_t>(N) + kTileRows - 1) / kTileRows);
    const int n_op = (n_o + 1) / 2;
    const auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const float lines = K % kKBytes ? 1.5f : 1.f;
    const auto rows_us = [=](float us, int rows, int kb) {
        return lines * us * static_cast<float>(rows) * static_cast<float>(kb);
    };
    const auto epi_us = [](int bn) { return 0.04f + 0.0094f * static_cast<float>(bn); };
    const float mbytes = 1e-6f * static_cast<float>(N) * static_cast<float>(K);
    const auto hbm_us = [&](float tbps) { return mbytes > 60.f ? mbytes / tbps : 0.f; };
    A8Plan best = {16, 1, 0, 1, 0};
    float least = 1e30f;
    const auto offer = [&](const A8Plan &p, float us) {
        if (us < least) {
            least = us;
            best = p;
        }
    };
    // one narrow tile a CTA, or shared by a cluster along K
    const int64_t widest = std::max<int64_t>(16, up(M, 16) * 16);
    for (int bn = 16; bn <= 128 && bn <= widest; bn += 16) {
        const int64_t tiles = n_o * up(std::max(M, 1), bn);
        for (int log = 0; log < 4; ++log) {
            const int split = 1 << log;
            constexpr float kCluster[4] = {0.f, 0.59f, 0.58f, 0.75f};
            if (split > nkb || tiles * split > 6 * sms) break;
            const float per = static_cast<float>(up(tiles * split, sms));
            const float load = per * rows_us(0.00116f, kTileRows + bn, (nkb + split - 1) / split);
            const float hbm = hbm_us(n_o * split * 2 >= 3 * sms   ? 5.9f
                                     : n_o * split * 4 >= 3 * sms ? 5.1f
                                                                  : 3.4f);
            offer({bn, split, 0, 1, 0},
                  std::max(load, hbm) + 0.84f * (per - 1.f) + epi_us(bn) +
                      (split > 1 ? 0.025f * static_cast<float>(bn) : 0.f) + kCluster[log]);
        }
    }
    // persistent tiles, on single CTAs and on pairs
    for (int pair = 0; pair < 2; ++pair)
        for (int bn = 64; bn <= 256 && bn <= std::max<int64_t>(64, up(M, 32) * 32); bn += 32) {
            const int64_t tiles = (pair ? n_op : n_o) * up(std::max(M, 1), bn);
            const float per = static_cast<float>(up(tiles, pair ? sms / 2 : sms));
            const float load = pair ? rows_us(0.00116f, kTileRows + bn / 2, nkb)
                                    : rows_us(0.00098f, kTileRows + bn, nkb);
            const float epi = epi_us(bn);
            const float walk =
                load + (per - 1.f) * (std::max(load, epi) + 0.95f * std::min(load, epi));
            offer({bn, 1, pair, 0, 0},
                  std::max(walk, hbm_us(4.8f)) + epi + 0.2f + (pair ? 0.98f : 0.f));
        }
    // A few rows on the CUDA cores, 1 or 4 weight rows a warp (us beyond 1.76): a
    // 512-byte step of K costs a load's latency, a byte of weights its load or its
    // arithmetic, in whole steps.  Up to four activation rows: one weight row a warp, whose
    // loads of K all run at once, but four where K is short (below 1024) and there are enough
    // weight rows (above 2048) to fill the SMs with a quarter of the warps.  One over
    // four, int8, M = 1: 2048 x 512 0.94, 4096 x 512 1.29, 32768 x 512 1.62, 4096 x 1024
    // 0.72, 4096 x 2048 0.68; M = 4: 1.00, 1.12, 1.74, 0.91, 0.67; e4m3, M = 1: 0.91,
    // 1.29, 1.60, 1.00, 0.80.  (From N = 32768 on four are faster at K = 1024 too, 1.24, and
    // one at 2048, 0.88.)  More activation rows: one where four would leave SMs without
    // warps.  Measured, us, CUDA cores and tensor
    // cores: M = 1, int8, 512 x 512: 1.5 and 2.6, 512 x 2048 (K): 1.9 and 3.3, 8192 x
    // 8192: 12.2 and 14.0; M = 8, 4096 x 4096: 6.7 and 4.6; M = 80, 512 x 512: 2.4 and
    // 2.7, 2048 x 512: 5.5 and 2.8; e4m3, M = 1, 8192 x 8192: 17.1 and 14.1; M = 80,
    // 512 x 512: 3.6 and 2.9; one and four weight rows, M = 8, int8: 512 x 2048 2.7
    // and 3.1, 4096 x 512 2.9 and 2.4.
    if (M >= 1 && M <= 128) {
        const int64_t steps = up(K, 512), groups = up(M, 8);
        const float step_us = static_cast<float>(steps - 1);
        const float mb = 1e-6f * static_cast<float>(N) * static_cast<float>(512 * steps);
        const bool q8 = fmt == kFmtQ8;
        if (M <= 4 && !(K < 1024 && N > 2048)) {
            const float byte_us = q8 ? 0.08f + 0.031f * M : 0.14f + 0.089f * M;
            offer({8, 1, 0, 0, 1},
                  -0.48f + 0.08f * step_us + std::max(byte_us * mb, hbm_us(5.9f)));
        } else {
            const float work = lines * mb * static_cast<float>(M <= 4 ? M : 8 * groups);
            offer({8, 1, 0, 0, M > 4 && N * groups <= 1024 ? 1 : 4},
                  q8 ? -0.41f + 0.3f * step_us + (K <= 512 ? 0.045f : 0.03f) * work
                     : -0.16f + 0.7f * step_us * (M <= 4 ? 0.125f * M : 1.f) + 0.085f * work);
        }
    }
    return best;
}

cudaError_t launch_qgemm_a8(const A8Plan &plan, int fmt, int dtype, const void *Xq, const float *xs,
                            const void *Wq, const float *wsc, const float *bias, void *Y, int M,
                            int N, int K, DevCtl *ctl, cudaStream_t s) {
    if (plan.few)
        return launch_qgemm_a8_few(plan.few, fmt, dtype, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
    return fmt == kFmtQ8
               ? launch_a8_y<kFmtQ8>(plan, dtype, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s)
               : launch_a8_y<kFmtE4M3>(plan, dtype, Xq, xs, Wq, wsc, bias, Y, M, N, K, ctl, s);
}

}  // namespace rtq
