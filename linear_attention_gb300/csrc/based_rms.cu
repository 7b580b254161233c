// based_rms.cu: the root-mean-square norm of a residual stream (declared in include/based_ops.h).
//
//     s = x + residual (rounded to the stream's type),   y = s r w,   r = 1 / sqrt(mean(s^2) + eps)
//     ds = r (d - s r mean(d s r)) + dsum with d = dy w,   dw = sum over rows of dy s r
//
// A row lies in the registers of THREADS threads, up to four packs of eight channels each, so one reading of it serves the
// sum of squares, the largest magnitude of an 8-bit output and the result. Bound by memory. Rows of up to 64 packs take a part of
// a warp or a warp; longer ones two to sixteen warps, which meet once (8 bits: twice) in shared memory. CTAs walk over the rows with the weights in
// registers; backward the weights' gradients add up there too, in an order that the sizes and the rows' alignment fix.
#include <type_traits>

#include "ops_common.cuh"

namespace based {
namespace {

constexpr int kPack = 8, kMostPacks = 4, kMostThreads = 512;
constexpr int kRmsMaxC = kPack * kMostPacks * kMostThreads;
constexpr int kRmsCtas = 304;  // partial sums of the weights' gradient: two CTAs on each of 152 SMs

struct RmsParams {
    const void *x, *residual, *weight, *dy, *dsum;
    int64_t x_sr, res_sr, dy_sr, dsum_sr;
    int64_t R;
    int C, p_dtype, ctas;
    float eps;
    void *sum, *y, *ds, *dx, *dweight;
    float *scales, *partial;
};

// Channel e of pack j of a thread. Packs that are words lie side by side; single channels are dealt out one to a thread, so that either way
// neighbouring threads read neighbouring addresses.
template <bool WORDS>
__device__ __forceinline__ int channel(int t, int threads, int j, int e) {
    return WORDS ? (t + threads * j) * kPack + e : t + threads * (j * kPack + e);
}
// A pack as it lies in memory: the loads of several packs go out together, the conversion comes after
template <bool WORDS, typename T>
struct Raw {
    Pack<T, kPack> p;
    __device__ __forceinline__ void load(const T *from, int t, int threads, int j, int C) {
        if constexpr (WORDS) {
            const int c = channel<true>(t, threads, j, 0);
            uint4 *const w = reinterpret_cast<uint4 *>(&p);
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(p)) / 16; ++i) {
                w[i] = make_uint4(0, 0, 0, 0);
                if (c < C) w[i] = __ldcs(reinterpret_cast<const uint4 *>(from + c) + i);
            }
        } else {
#pragma unroll
            for (int e = 0; e < kPack; ++e) {
                const int c = channel<false>(t, threads, j, e);
                p.v[e] = from_f32<T>(0.0f);
                if (c < C) p.v[e] = from[c];
            }
        }
    }
    __device__ __forceinline__ float operator[](int e) const { return to_f32(p.v[e]); }
};
template <bool WORDS, typename T>
__device__ __forceinline__ void store_pack(T *p, const float (&x)[kPack], int t, int threads, int j, int C) {
    if constexpr (WORDS) {
        const int c = channel<true>(t, threads, j, 0);
        if (c < C) {
            Pack<T, kPack> w;
#pragma unroll
            for (int e = 0; e < kPack; ++e) w.v[e] = from_f32<T>(x[e]);
            *reinterpret_cast<Pack<T, kPack> *>(p + c) = w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kPack; ++e) {
            const int c = channel<false>(t, threads, j, e);
            if (c < C) p[c] = from_f32<T>(x[e]);
        }
    }
}
// Two elements in e4m3, to nearest even; beyond 448 they become 448
__device__ __forceinline__ uint32_t e4m3_pair(float x, float y) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
    return r;
}
template <bool WORDS>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&x)[kPack], int t, int threads, int j, int C) {
    if constexpr (WORDS) {
        const int c = channel<true>(t, threads, j, 0);
        if (c < C)
            *reinterpret_cast<uint2 *>(p + c) = make_uint2(e4m3_pair(x[0], x[1]) | e4m3_pair(x[2], x[3]) << 16,
                                                           e4m3_pair(x[4], x[5]) | e4m3_pair(x[6], x[7]) << 16);
    } else {
#pragma unroll
        for (int e = 0; e < kPack; ++e) {
            const int c = channel<false>(t, threads, j, e);
            if (c < C) p[c] = static_cast<uint8_t>(e4m3_pair(x[e], 0.0f));
        }
    }
}
template <typename T, bool WORDS>
__device__ __forceinline__ void load_weight(float (&w)[kPack], const RmsParams &p, int t, int threads, int j) {
    Raw<WORDS, T> a;
    Raw<WORDS, float> b;
    if (p.weight && p.p_dtype == BASED_F32)
        b.load(static_cast<const float *>(p.weight), t, threads, j, p.C);
    else if (p.weight)
        a.load(static_cast<const T *>(p.weight), t, threads, j, p.C);
#pragma unroll
    for (int e = 0; e < kPack; ++e) w[e] = !p.weight ? 1.0f : p.p_dtype == BASED_F32 ? b[e] : a[e];
}

__host__ __device__ constexpr int cta_of(int threads) { return threads < 256 ? 256 : threads; }

// The threads of a row meet; the CTA's other rows go on.
template <int THREADS>
__device__ __forceinline__ void meet_row() {
    if constexpr (THREADS < cta_of(THREADS))
        named_bar_sync(1 + threadIdx.x / THREADS, THREADS);
    else
        __syncthreads();
}
// The sum or the largest of v over the THREADS threads of a row; red: 32 floats of the CTA, two rows of them used in turn
template <int THREADS, bool MOST>
__device__ __forceinline__ float over_row(float v, float *red, int &turn) {
    constexpr int kLanes = THREADS < 32 ? THREADS : 32, kWarps = THREADS / 32;
#pragma unroll
    for (int d = 1; d < kLanes; d *= 2) {
        const float o = __shfl_xor_sync(0xffffffffu, v, d);
        v = MOST ? fmaxf(v, o) : v + o;
    }
    if constexpr (kWarps > 1) {
        float *const at = red + turn * 32 + threadIdx.x / THREADS * kWarps;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) at[threadIdx.x % THREADS / 32] = v;
        meet_row<THREADS>();
        v = at[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) v = MOST ? fmaxf(v, at[i]) : v + at[i];
    }
    return v;
}

// Two sums at once
template <int THREADS>
__device__ __forceinline__ void over_row2(float &a, float &b, float *red, int &turn) {
    constexpr int kLanes = THREADS < 32 ? THREADS : 32, kWarps = THREADS / 32;
#pragma unroll
    for (int d = 1; d < kLanes; d *= 2) a += __shfl_xor_sync(0xffffffffu, a, d), b += __shfl_xor_sync(0xffffffffu, b, d);
    if constexpr (kWarps > 1) {
        float2 *const at = reinterpret_cast<float2 *>(red) + turn * 16 + threadIdx.x / THREADS * kWarps;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) at[threadIdx.x % THREADS / 32] = make_float2(a, b);
        meet_row<THREADS>();
        float2 v = at[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) v.x += at[i].x, v.y += at[i].y;
        a = v.x, b = v.y;
    }
}

template <typename T, typename S, int THREADS, int PACKS, bool WORDS>
__global__ void __launch_bounds__(cta_of(THREADS)) based_rms_fwd_kernel(RmsParams p) {
    constexpr int kRows = cta_of(THREADS) / THREADS;
    __shared__ __align__(8) float red[64];
    int turn = 0;
    const int t = threadIdx.x % THREADS, slot = threadIdx.x / THREADS;
    griddep_wait();
    float w[PACKS][kPack];
#pragma unroll
    for (int j = 0; j < PACKS; ++j) load_weight<T, WORDS>(w[j], p, t, THREADS, j);
    const float mean = 1.0f / p.C;
    // The next row's loads go out in front of a row's sums where registers hold both
    constexpr bool kAhead = WORDS && PACKS * (sizeof(T) + sizeof(S)) <= 12;
    Raw<WORDS, T> x[PACKS];
    Raw<WORDS, S> r[PACKS];
    const auto load = [&](int64_t row) {
        const int C = row < p.R ? p.C : 0;
#pragma unroll
        for (int j = 0; j < PACKS; ++j) x[j].load(static_cast<const T *>(p.x) + row * p.x_sr, t, THREADS, j, C);
        if (p.residual) {
#pragma unroll
            for (int j = 0; j < PACKS; ++j) r[j].load(static_cast<const S *>(p.residual) + row * p.res_sr, t, THREADS, j, C);
        }
    };
    if (kAhead) load(static_cast<int64_t>(blockIdx.x) * kRows + slot);
    // all threads of the CTA go round equally often: rows behind the last are computed as zeros and not stored
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRows; first < p.R; first += static_cast<int64_t>(gridDim.x) * kRows) {
        const int64_t row = first + slot;
        const bool there = row < p.R;
        const int C = there ? p.C : 0;
        float s[PACKS][kPack], sq = 0.0f;
        if (!kAhead) load(row);
        if (p.residual) {
#pragma unroll
            for (int j = 0; j < PACKS; ++j)
#pragma unroll
                for (int e = 0; e < kPack; ++e) s[j][e] = to_f32(from_f32<S>(x[j][e] + r[j][e]));  // what is written is what is normed
        } else {
#pragma unroll
            for (int j = 0; j < PACKS; ++j)
#pragma unroll
                for (int e = 0; e < kPack; ++e) s[j][e] = x[j][e];
        }
        if (kAhead) load(row + static_cast<int64_t>(gridDim.x) * kRows);
        if (p.residual) {
#pragma unroll
            for (int j = 0; j < PACKS; ++j) store_pack<WORDS>(static_cast<S *>(p.sum) + row * p.C, s[j], t, THREADS, j, C);
        }
#pragma unroll
        for (int j = 0; j < PACKS; ++j)
#pragma unroll
            for (int e = 0; e < kPack; ++e) sq = fmaf(s[j][e], s[j][e], sq);
        const float norm = rsqrtf(over_row<THREADS, false>(sq, red, turn) * mean + p.eps);
        float most = 0.0f;
#pragma unroll
        for (int j = 0; j < PACKS; ++j)
#pragma unroll
            for (int e = 0; e < kPack; ++e) {
                s[j][e] = s[j][e] * norm * w[j][e];
                asm("max.NaN.f32 %0, %1, %2;" : "=f"(most) : "f"(most), "f"(fabsf(s[j][e])));
            }
        if (p.scales) {
            most = over_row<THREADS, true>(most, red, turn);
            const float scale = most > 0.0f ? fmaxf(most / 448.0f, 1.17549435e-38f) : 1.0f, inverse = 1.0f / scale;
#pragma unroll
            for (int j = 0; j < PACKS; ++j) {
#pragma unroll
                for (int e = 0; e < kPack; ++e) s[j][e] *= inverse;
                store_e4m3<WORDS>(static_cast<uint8_t *>(p.y) + row * p.C, s[j], t, THREADS, j, C);
            }
            if (t == 0 && there) p.scales[row] = scale;
        } else {
#pragma unroll
            for (int j = 0; j < PACKS; ++j) store_pack<WORDS>(static_cast<T *>(p.y) + row * p.C, s[j], t, THREADS, j, C);
        }
    }
}

template <typename T, typename S, int THREADS, int PACKS, bool WORDS>
__global__ void __launch_bounds__(cta_of(THREADS), cta_of(THREADS) == 256 ? 2 : 1) based_rms_bwd_kernel(RmsParams p) {
    constexpr int kCta = cta_of(THREADS), kRows = kCta / THREADS;
    __shared__ __align__(8) float red[64];
    extern __shared__ float sums[];  // rows' threads' sums of the weights' gradient, where a CTA takes several rows
    int turn = 0;
    const int t = threadIdx.x % THREADS, slot = threadIdx.x / THREADS;
    griddep_wait();
    float w[PACKS][kPack], dw[PACKS][kPack] = {};
#pragma unroll
    for (int j = 0; j < PACKS; ++j) load_weight<T, WORDS>(w[j], p, t, THREADS, j);
    const float mean = 1.0f / p.C;
    constexpr bool kAhead = WORDS && PACKS * (sizeof(T) + 2 * sizeof(S)) <= 12;  // as forward
    Raw<WORDS, S> ns[PACKS], ng[PACKS];
    Raw<WORDS, T> nd[PACKS];
    const auto load = [&](int64_t row) {
        const int C = row < p.R ? p.C : 0;
#pragma unroll
        for (int j = 0; j < PACKS; ++j) {
            ns[j].load(static_cast<const S *>(p.x) + row * p.x_sr, t, THREADS, j, C);
            nd[j].load(static_cast<const T *>(p.dy) + row * p.dy_sr, t, THREADS, j, C);
        }
#pragma unroll
        for (int j = 0; j < PACKS; ++j) ng[j].load(static_cast<const S *>(p.dsum) + row * p.dsum_sr, t, THREADS, j, p.dsum ? C : 0);
    };
    if (kAhead) load(static_cast<int64_t>(blockIdx.x) * kRows + slot);
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRows; first < p.R; first += static_cast<int64_t>(gridDim.x) * kRows) {
        const int64_t row = first + slot;
        const int C = row < p.R ? p.C : 0;
        Raw<WORDS, S> s[PACKS], g[PACKS];
        Raw<WORDS, T> d[PACKS];
        float sq = 0.0f, ds = 0.0f;
        if (!kAhead) load(row);
#pragma unroll
        for (int j = 0; j < PACKS; ++j) s[j] = ns[j], g[j] = ng[j], d[j] = nd[j];
        if (kAhead) load(row + static_cast<int64_t>(gridDim.x) * kRows);
#pragma unroll
        for (int j = 0; j < PACKS; ++j)
#pragma unroll
            for (int e = 0; e < kPack; ++e) sq = fmaf(s[j][e], s[j][e], sq), ds = fmaf(d[j][e] * w[j][e], s[j][e], ds);
        over_row2<THREADS>(sq, ds, red, turn);
        // (rows behind the last add nothing to the weights' gradient, whatever eps is)
        const float r = row < p.R ? rsqrtf(sq * mean + p.eps) : 0.0f, back = ds * mean * r * r;  // mean(d s) r^2
#pragma unroll
        for (int j = 0; j < PACKS; ++j) {
            float x[kPack];
#pragma unroll
            for (int e = 0; e < kPack; ++e) {
                dw[j][e] = fmaf(d[j][e], s[j][e] * r, dw[j][e]);
                x[e] = fmaf(r, d[j][e] * w[j][e] - s[j][e] * back, g[j][e]);
            }
            store_pack<WORDS>(static_cast<S *>(p.ds) + row * p.C, x, t, THREADS, j, C);
            if constexpr (!std::is_same<T, S>::value) store_pack<WORDS>(static_cast<T *>(p.dx) + row * p.C, x, t, THREADS, j, C);
        }
    }
    if (!p.dweight) return;
    float *const out = p.partial + static_cast<int64_t>(blockIdx.x) * p.C;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int j = 0; j < PACKS; ++j) store_pack<WORDS>(out, dw[j], t, THREADS, j, p.C);
    } else {
#pragma unroll
        for (int j = 0; j < PACKS; ++j)
#pragma unroll
            for (int e = 0; e < kPack; ++e) {
                const int c = channel<WORDS>(t, THREADS, j, e);
                if (c < p.C) sums[slot * p.C + c] = dw[j][e];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < p.C; c += kCta) {
            float v = sums[c];
            for (int i = 1; i < kRows; ++i) v += sums[i * p.C + c];
            out[c] = v;
        }
    }
}

// dweight from the CTAs' sums: 32 channels a CTA, its 32 warps take every 32nd sum
template <typename P>
__global__ void __launch_bounds__(1024) based_rms_sum_kernel(RmsParams p) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    griddep_wait();
    float v = 0.0f;
    if (c < p.C) {
#pragma unroll 10
        for (int i = warp; i < p.ctas; i += 32) v += p.partial[static_cast<int64_t>(i) * p.C + c];
    }
    part[warp][lane] = v;
    __syncthreads();
    v = part[lane][warp];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
    const int to = blockIdx.x * 32 + warp;
    if (lane == 0 && to < p.C) static_cast<P *>(p.dweight)[to] = from_f32<P>(v);
}

// ------------------------------------------------------------------------------------------------
// Host
// ------------------------------------------------------------------------------------------------
template <typename T, typename S, int THREADS, int PACKS, bool WORDS>
int launch_fwd(RmsParams &p, int sms, cudaStream_t st) {
    constexpr int kCta = cta_of(THREADS), kRows = kCta / THREADS;
    const int64_t groups = (p.R + kRows - 1) / kRows;
    void (*const fwd)(RmsParams) = based_rms_fwd_kernel<T, S, THREADS, PACKS, WORDS>;
    int resident = 0;
    if (const int rc = resident_clusters(reinterpret_cast<const void *>(fwd), kCta, 0, 1, &resident)) return rc;
    const int64_t most = resident > 0 ? resident : sms;
    OPS_CUDA(launch_op(fwd, static_cast<unsigned>(groups < most ? groups : most), kCta, 0, st, p));
    return BASED_OK;
}
template <typename T, typename S, int THREADS, int PACKS, bool WORDS>
int launch_bwd(RmsParams &p, cudaStream_t st) {
    constexpr int kCta = cta_of(THREADS), kRows = kCta / THREADS;
    const int64_t groups = (p.R + kRows - 1) / kRows;
    p.ctas = static_cast<int>(groups < kRmsCtas ? groups : kRmsCtas);
    const size_t smem = kRows > 1 ? static_cast<size_t>(kRows) * p.C * 4 : 0;
    OPS_CUDA(launch_op(based_rms_bwd_kernel<T, S, THREADS, PACKS, WORDS>, p.ctas, kCta, smem, st, p));
    if (p.dweight) {
        void (*const sum)(RmsParams) = p.p_dtype == BASED_F32 ? based_rms_sum_kernel<float> : based_rms_sum_kernel<T>;
        OPS_CUDA(launch_op(sum, (p.C + 31) / 32, 1024, 0, st, p));
    }
    return BASED_OK;
}
// Threads for a row: as few as hold it in two packs each, which leaves registers for the next row's loads (three where that fits better and both
// streams have 16 bits), so that a warp or a part of one serves short rows and sums stay in it. bf16, with the next row ahead and without: 29296 x 2048 75 us (four packs
// 84), 7324 x 8192 81 (109), a float32 stream of 20000 x 3000 114 (134). 16-bit inputs beside a float32 stream of more than 3584 channels do better in four packs
// without it: of 60 million elements 4096 channels take 115 us (e4m3 out: 111) instead of 126 (117), 3840 115 (112) instead of 126 (113), 3584 117 (115) and 124 (111),
// 3200 124 (119) and 120 (111); float32 throughout 3200 to 4096 channels take 179 to 193 us in four packs and 158 to 169 in two.
// Backward 24000 x 1536 51 us, without 64, with four packs 79. Single channels, not words, go by four or two packs.
template <typename T, typename S>
int launch_rms(RmsParams &p, bool words, bool bwd, int sms, cudaStream_t st) {
    const int packs = (p.C + kPack - 1) / kPack;
    if (bwd) {
        if (!words) {
            if (packs <= 64) return launch_bwd<T, S, 32, 2, false>(p, st);
            if (packs <= 512) return launch_bwd<T, S, 256, 2, false>(p, st);
            return launch_bwd<T, S, 512, 4, false>(p, st);
        }
        if (packs <= 8) return launch_bwd<T, S, 8, 1, true>(p, st);
        if (packs <= 32) return launch_bwd<T, S, 16, 2, true>(p, st);
        if (packs <= 64) return launch_bwd<T, S, 32, 2, true>(p, st);
        if (packs <= 128) return launch_bwd<T, S, 64, 2, true>(p, st);
        if (packs <= 256) return launch_bwd<T, S, 128, 2, true>(p, st);
        if (packs <= 512) return launch_bwd<T, S, 256, 2, true>(p, st);
        if (packs <= 1024) return launch_bwd<T, S, 512, 2, true>(p, st);
        return launch_bwd<T, S, 512, 4, true>(p, st);
    }
    if (!words) {
        if (packs <= 128) return launch_fwd<T, S, 32, 4, false>(p, sms, st);
        if (packs <= 512) return launch_fwd<T, S, 128, 4, false>(p, sms, st);
        return launch_fwd<T, S, 512, 4, false>(p, sms, st);
    }
    if (packs <= 8) return launch_fwd<T, S, 8, 1, true>(p, sms, st);
    if (packs <= 32) return launch_fwd<T, S, 16, 2, true>(p, sms, st);
    if (packs <= 64) return launch_fwd<T, S, 32, 2, true>(p, sms, st);
    if (packs <= 128) return launch_fwd<T, S, 64, 2, true>(p, sms, st);
    if constexpr (sizeof(S) == 2)
        if (packs <= 192) return launch_fwd<T, S, 64, 3, true>(p, sms, st);
    if (packs <= 256) return launch_fwd<T, S, 128, 2, true>(p, sms, st);
    if constexpr (sizeof(S) == 2)
        if (packs <= 384) return launch_fwd<T, S, 128, 3, true>(p, sms, st);
    if constexpr (sizeof(T) == 2 && sizeof(S) == 4)
        if (packs > 448 && packs <= 512) return launch_fwd<T, S, 128, 4, true>(p, sms, st);
    if (packs <= 512) return launch_fwd<T, S, 256, 2, true>(p, sms, st);
    if (packs <= 1024) return launch_fwd<T, S, 512, 2, true>(p, sms, st);
    return launch_fwd<T, S, 512, 4, true>(p, sms, st);
}

int run_rms(RmsParams &p, int dtype, int s_dtype, bool bwd, void *workspace, size_t ws_bytes, based_stream_t stream) {
    if (!type_ok(dtype) || !type_ok(s_dtype) || (s_dtype != dtype && s_dtype != BASED_F32)) return BASED_ERR_UNSUPPORTED_TYPE;
    if (p.weight && p.p_dtype != dtype && p.p_dtype != BASED_F32) return BASED_ERR_UNSUPPORTED_TYPE;
    if (!(p.eps >= 0.0f)) return BASED_ERR_BAD_ARGUMENT;
    if (p.R < 1 || p.C < 1 || p.C > kRmsMaxC || p.R > (static_cast<int64_t>(1) << 46) / p.C) return BASED_ERR_BAD_SIZE;
    if (p.x_sr < 0 || p.res_sr < 0 || p.dy_sr < 0 || p.dsum_sr < 0) return BASED_ERR_BAD_STRIDE;
    const int64_t R = p.R, C = p.C;
    const size_t es = elem_size(dtype), ss = elem_size(s_dtype), ps = elem_size(p.p_dtype), xs = bwd ? ss : es;
    if (!aligned(p.x, xs) || !aligned(p.residual, ss) || !aligned(p.weight, ps) || !aligned(p.dy, es) || !aligned(p.dsum, ss) ||
        !aligned(p.sum, ss) || (!p.scales && !aligned(p.y, es)) || !aligned(p.scales, 4) || !aligned(p.ds, ss) || !aligned(p.dx, es) ||
        !aligned(p.dweight, ps))
        return BASED_ERR_MISALIGNED;
    const Span x = span(p.x, (R - 1) * p.x_sr + C - 1, xs), res = span(p.residual, (R - 1) * p.res_sr + C - 1, ss),
               w = span(p.weight, C - 1, ps), dy = span(p.dy, (R - 1) * p.dy_sr + C - 1, es), dsum = span(p.dsum, (R - 1) * p.dsum_sr + C - 1, ss);
    size_t need = 0;
    if (bwd && p.dweight) {
        need = static_cast<size_t>(R < kRmsCtas ? R : kRmsCtas) * C * 4;
        if (!workspace || ws_bytes < need || !aligned(workspace, 16)) return BASED_ERR_WORKSPACE;
        p.partial = static_cast<float *>(workspace);
    }
    const Span in[] = {x, res, w, dy, dsum};
    const Span out[] = {span(p.sum, R * C - 1, ss), span(p.y, R * C - 1, p.scales ? 1 : es), span(p.scales, R - 1, 4), span(p.ds, R * C - 1, ss),
                        span(p.dx, R * C - 1, es), span(p.dweight, C - 1, ps), span(p.partial, static_cast<int64_t>(need / 4) - 1, 4)};
    for (int i = 0; i < 7; ++i) {
        for (int j = 0; j < 5; ++j) {
            // the sum may replace the residual, and the gradient of the sum the one that is added to it
            const bool place = (i == 0 && j == 1 && p.sum == p.residual && p.res_sr == C) || (i == 3 && j == 4 && p.ds == p.dsum && p.dsum_sr == C);
            if (!place && overlap(out[i], in[j])) return BASED_ERR_ALIASING;
        }
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return BASED_ERR_ALIASING;
    }
    int sms;
    if (const int rc = host_device(&sms)) return rc;
    const auto words = [&](const void *q, int64_t stride, size_t size) {
        return !q || (aligned(q, size * kPack < 16 ? size * kPack : 16) && (stride * static_cast<int64_t>(size)) % 16 == 0);
    };
    const bool wide = C % kPack == 0 && words(p.x, p.x_sr, xs) && words(p.residual, p.res_sr, ss) && words(p.weight, 0, ps) &&
                      words(p.dy, p.dy_sr, es) && words(p.dsum, p.dsum_sr, ss) && words(p.sum, 0, ss) && words(p.y, 0, p.scales ? 1 : es) &&
                      words(p.ds, 0, ss) && words(p.dx, 0, es);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == BASED_F32) return launch_rms<float, float>(p, wide, bwd, sms, st);
    if (dtype == BASED_BF16)
        return s_dtype == BASED_F32 ? launch_rms<__nv_bfloat16, float>(p, wide, bwd, sms, st)
                                    : launch_rms<__nv_bfloat16, __nv_bfloat16>(p, wide, bwd, sms, st);
    return s_dtype == BASED_F32 ? launch_rms<__half, float>(p, wide, bwd, sms, st) : launch_rms<__half, __half>(p, wide, bwd, sms, st);
}

}  // namespace
}  // namespace based

extern "C" {

int based_rms_fwd(const void *x, int64_t x_sr, const void *residual, int64_t res_sr, int s_dtype, const void *weight, int p_dtype, int64_t R,
                  int C, float eps, void *sum, void *y, int dtype, float *scales, based_stream_t stream) {
    if (!x || !y || !residual != !sum) return BASED_ERR_NULL_POINTER;
    based::RmsParams p = {};
    p.x = x, p.x_sr = x_sr, p.residual = residual, p.res_sr = res_sr, p.weight = weight, p.p_dtype = weight ? p_dtype : dtype;
    p.R = R, p.C = C, p.eps = eps, p.sum = sum, p.y = y, p.scales = scales;
    return based::run_rms(p, dtype, residual ? s_dtype : dtype, false, nullptr, 0, stream);
}

int based_rms_bwd(const void *dy, int64_t dy_sr, const void *s, int64_t s_sr, int s_dtype, const void *weight, int p_dtype, const void *dsum,
                  int64_t dsum_sr, int64_t R, int C, float eps, void *ds, void *dx, void *dweight, int dtype, void *workspace, size_t ws_bytes,
                  based_stream_t stream) {
    if (!dy || !s || !ds || (s_dtype == dtype) != !dx || (dweight && !weight)) return BASED_ERR_NULL_POINTER;
    based::RmsParams p = {};
    p.dy = dy, p.dy_sr = dy_sr, p.x = s, p.x_sr = s_sr, p.weight = weight, p.p_dtype = weight ? p_dtype : dtype, p.dsum = dsum, p.dsum_sr = dsum_sr;
    p.R = R, p.C = C, p.eps = eps, p.ds = ds, p.dx = dx, p.dweight = dweight;
    return based::run_rms(p, dtype, s_dtype, true, workspace, ws_bytes, stream);
}

size_t based_rms_bwd_workspace_size(int64_t R, int C) {
    if (R < 1 || C < 1 || C > based::kRmsMaxC || R > (static_cast<int64_t>(1) << 46) / C) return 0;
    return static_cast<size_t>(R < based::kRmsCtas ? R : based::kRmsCtas) * C * 4;
}

}  // extern "C"
