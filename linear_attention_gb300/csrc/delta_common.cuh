// delta_common.cuh: what the kernels of the gated delta rule share: parameters, the layout of a chunk's records,
// float16 pairs and the matrix instructions on them.
//
// The kernels multiply on tensor cores and keep float32's accuracy. A float32 operand x goes in as two
// float16 terms, hi = x s and lo = x s - hi with a power of two s that brings the largest |x| of what shares it
// to 2^14: together 22 bits, off by 2^-23 of that largest where bfloat16 pairs would be off by 2^-17. A product
// of two pairs is three matrix products (lo lo, 2^-22 of the result, is left out); 16-bit inputs are one term.
// Sums are float32. Per multiprocessor and cycle mma.sync makes 1019 float16 products (measured), a quarter of what
// tcgen05.mma does, but its accumulators are registers: a chunk's chain of products runs
// in one warp, which hands its results to itself without a barrier or a trip through memory.
#pragma once
#include <cstring>

#include "ops_common.cuh"

namespace based {

constexpr int kChunk = 64;         // rows of a chunk
constexpr int kMaxKeys = 128;      // channels of a key
constexpr int kDeltaMaxV = 1 << 16;

struct DeltaParams {
    const void *q, *k, *v, *beta, *gate, *dout;
    int64_t q_sb, q_st, q_sh, k_sb, k_st, k_sh, v_sb, v_st, v_sh, do_sb, do_st, do_sh, beta_sb, beta_st, gate_sb, gate_st;
    int B, T, H, HK, K, V, chunks;
    int qk_vec, v_vec, do_vec, o_vec;  // rows can be read (written) as 16-byte words
    float scale;
    const int32_t *lengths;
    const float *state;       // forward: the first state; backward: dfinal
    float *final_state;       // forward: the last state; backward: dstate
    uint8_t *saved;           // forward's records of the slices (SliceRec), or NULL
    void *out;                // forward: o; backward: dv
    void *dq, *dk, *dbeta, *dgate;
    uint8_t *qk_rec, *g_rec;  // the records of the chunks
    uint8_t *slice_rec;       // backward's records of the slices
};

// The terms of an operand. Inputs of 16 bits are one float16 term (bfloat16 fits one after its scaling: 8 bits). Results that are
// rounded to bfloat16 (half a step is 2^-8) take one term, 2^-11, of what is computed; other outputs, and all that goes into a state, two. With two
// 8 x 4096 rows of 16 heads of 128 x 128 took 3091 us in training where one took 2327, 1 x 16384 forward 638 and 579; off the 64-bit results are
// 0.166 % with two (the rounding alone) and 0.168 % with one.
template <typename T>
struct Terms {
    static constexpr int in = 1, out = 2;
};
template <>
struct Terms<__nv_bfloat16> {
    static constexpr int in = 1, out = 1;
};
template <>
struct Terms<float> {
    static constexpr int in = 2, out = 2;
};

// A chunk's records in the workspace: images of shared memory, copied as they are.
//   of a key head: the scaled keys and queries, TERMS x 64 x KP float16 each
//   of a value head: the inverse below its diagonal of ones (two terms; forward: its rows times their steps, its columns over theirs), the
//   masked scores (forward: Terms::out, times beta of their columns over their steps; backward: two), 64 x 64 float16 each, and float32
//   numbers: per row grow = exp(b), rest = exp(b_last - b) (forward: grow times the row's step), beta (forward: the step), b in two parts (b: the sum
//   of log decays up to the row), beta grow (forward: beta rest over the step), then the scales' inverses, and of each 16 rows the
//   largest |beta grow| (forward: the largest |beta rest| over the step) and the largest grow.
constexpr int kSquare = kChunk * kChunk * 2;  // bytes
enum { F_GROW = 0, F_REST = 64, F_BETA = 128, F_BHI = 192, F_BLO = 256, F_BF = 320, F_INV = 384, F_P, F_WHOLE, F_K, F_Q, F_BFMOST = 392, F_GROWMOST = 396, F_COUNT = 400 };
enum { F_GROWSTEP = F_REST, F_STEP = F_BETA };  // forward
template <typename T, int KP>
struct Rec {
    static constexpr int term = kChunk * KP * 2, img = Terms<T>::in * term, qk = 2 * img;
    __host__ __device__ static constexpr int scores(bool bwd) { return bwd ? 2 : Terms<T>::out; }
    __host__ __device__ static constexpr int g(bool bwd) { return (2 + scores(bwd)) * kSquare + F_COUNT * 4; }
};

// What the passes through the chunks leave for the gradients, per chunk, value head and slice of 16 channels of the values: float16 terms
// in the order of left operands, 16 x 16 blocks of four 8 x 8 blocks (rows 0-7 and 8-15 of columns 0-7, the same of columns 8-15) of 128
// bytes, rows the slice's channels; behind them the scales' inverses, one for the state, and one for each 16 of the chunk's rows of E (whose rows are times
// their steps), dR and dO.
constexpr int kSlice = 16;
constexpr int kRowsTerm = kSlice * kChunk * 2;
template <typename T, int KP>
struct SliceRec {
    static constexpr int in = Terms<T>::in, out = Terms<T>::out;
    static constexpr int state_term = kSlice * KP * 2, states = out * state_term;
    // forward: the state in front of the chunk, E
    static constexpr int e = states, fwd_scales = e + out * kRowsTerm, fwd = fwd_scales + 32;
    // backward: the gradient of the state behind the chunk, dR, dO
    static constexpr int dr = states, dout = dr + out * kRowsTerm, bwd_scales = dout + in * kRowsTerm, bwd = bwd_scales + 48;
};

// ------------------------------------------------------------------------------------------------
// Images: rows of COLS float16, their 16-byte words exchanged by the row so that eight rows of one column of
// words lie in different banks
// ------------------------------------------------------------------------------------------------
template <int COLS>
__device__ __forceinline__ uint32_t word_at(int row, int word) {
    return row * (COLS * 2) + ((word ^ (row & 7)) << 4);
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
// Operands of a 16 x 8 x 16 product from an image X. The second operand's register pairs {r0, r1} and {r2, r3} are two blocks of
// eight columns n:
//   left:    A[m][k] = X[row + m][col + k]
//   left_t:  A[m][k] = X[row + k][col + m]
//   right:   B[k][n] = X[row + n][col + k]     (16 n)
//   right_t: B[k][n] = X[row + k][col + n]     (16 n)
// row and col are multiples of 16.
template <int COLS>
__device__ __forceinline__ void left(uint32_t (&r)[4], uint32_t img, int row, int col, int lane) {
    ldsm(r, img + word_at<COLS>(row + (lane & 15), (col >> 3) + (lane >> 4)));
}
template <int COLS>
__device__ __forceinline__ void left_t(uint32_t (&r)[4], uint32_t img, int row, int col, int lane) {
    ldsm_t(r, img + word_at<COLS>(row + (lane & 7) + ((lane >> 4) << 3), (col >> 3) + ((lane >> 3) & 1)));
}
template <int COLS>
__device__ __forceinline__ void right(uint32_t (&r)[4], uint32_t img, int row, int col, int lane) {
    ldsm(r, img + word_at<COLS>(row + (lane & 7) + ((lane >> 4) << 3), (col >> 3) + ((lane >> 3) & 1)));
}
template <int COLS>
__device__ __forceinline__ void right_t(uint32_t (&r)[4], uint32_t img, int row, int col, int lane) {
    ldsm_t(r, img + word_at<COLS>(row + (lane & 15), (col >> 3) + (lane >> 4)));
}

using Acc = float[4];  // a 16 x 8 block: rows lane / 4 and + 8, columns 2 (lane % 4) and + 1

__device__ __forceinline__ void mma(Acc &d, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int N>
__device__ __forceinline__ void clear(Acc (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.0f;
}
// Two 16 x 8 blocks += the left operand's LT terms times the RT terms of a right operand. The tensor cores cut a sum's last bits off at every
// step; for float32 results (T) the step's sum is taken from zero, small terms first, and added in float32: a backward pass's errors
// are 0.4e-6 instead of 1.1e-6 (2 x 777 rows, 3 heads of 40 x 75), where float32 products give 0.3e-6.
template <typename T, int LT, int RT>
__device__ __forceinline__ void products(Acc &x, Acc &y, const uint32_t (&a)[LT][4], const uint32_t (&b)[RT][4]) {
    if constexpr (Terms<T>::in == 2) {
        Acc s[2];
        clear(s);
#pragma unroll
        for (int j = RT - 1; j >= 0; --j)
#pragma unroll
            for (int i = LT - 1; i >= 0; --i)
                if (i + j < 2) {
                    mma(s[0], a[i], b[j][0], b[j][1]);
                    mma(s[1], a[i], b[j][2], b[j][3]);
                }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += s[0][e], y[e] += s[1][e];
    } else {
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
            for (int i = 0; i < LT; ++i)
                if (i + j < 2) {
                    mma(x, a[i], b[j][0], b[j][1]);
                    mma(y, a[i], b[j][2], b[j][3]);
                }
    }
}

// Pairs of a block's columns times y; x += t c
__device__ __forceinline__ void by_pairs(Acc &x, const Vec<2> &y) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        const Vec<2> r = vmul(Vec<2>{{x[e], x[e + 1]}}, y);
        x[e] = r.v[0], x[e + 1] = r.v[1];
    }
}
__device__ __forceinline__ void add_times(Acc &x, const Acc &t, float c) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        const Vec<2> r = vfma(Vec<2>{{t[e], t[e + 1]}}, splat<2>(c), Vec<2>{{x[e], x[e + 1]}});
        x[e] = r.v[0], x[e + 1] = r.v[1];
    }
}
// ... times c: of several products whose left operands differ in their scales each is a sum of its own
template <int LT, int RT>
__device__ __forceinline__ void products_by(Acc &x, Acc &y, const uint32_t (&a)[LT][4], const uint32_t (&b)[RT][4], float c) {
    Acc s[2];
    clear(s);
#pragma unroll
    for (int j = RT - 1; j >= 0; --j)
#pragma unroll
        for (int i = LT - 1; i >= 0; --i)
            if (i + j < 2) {
                mma(s[0], a[i], b[j][0], b[j][1]);
                mma(s[1], a[i], b[j][2], b[j][3]);
            }
    add_times(x, s[0], c), add_times(y, s[1], c);
}

// ------------------------------------------------------------------------------------------------
// float16 pairs
// ------------------------------------------------------------------------------------------------
// The power of two that brings `most` (finite, >= 0) to [2^14, 2^15): between 2^-100 and 2^60, so that a
// product of two inverses is a float32 number unless the product of the values is none.
__device__ __forceinline__ float scale_for(float most) {
    int e = 268 - static_cast<int>(__float_as_uint(most) >> 23);
    e = e < 27 ? 27 : e > 187 ? 187 : e;
    return __uint_as_float(static_cast<uint32_t>(e) << 23);
}
constexpr float kTop = 32768.0f;  // what scaled magnitudes stay below: |x| < kTop * inverse
__device__ __forceinline__ float inverse_of(float pow2) { return __uint_as_float((254u << 23) - __float_as_uint(pow2)); }

// A row's step: the power of two at or below |beta|, from 2^-12 to 1. What a row holds before it is times beta is an operand times its step,
// and the other operand is over it: a row that hardly writes (beta 0: a masked token) takes no bits from the 16 that it is scaled with, whatever
// its values are, and beta's own gradient still has them.
__device__ __forceinline__ float step_of(float beta) {
    return fminf(fmaxf(__uint_as_float(__float_as_uint(beta) & 0x7f800000u), 2.44140625e-4f), 1.0f);
}

__device__ __forceinline__ uint32_t half2_of(float x, float y) { return pack<__half>(Vec<2>{{x, y}}); }
// hi and lo terms of two elements
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = half2_of(x, y);
    const Vec<2> h = unpack<__half>(hi);
    lo = half2_of(x - h.v[0], y - h.v[1]);
}
template <int TERMS>
__device__ __forceinline__ void terms(float x, float y, uint32_t (&w)[TERMS]) {
    if constexpr (TERMS == 2)
        split(x, y, w[0], w[1]);
    else
        w[0] = half2_of(x, y);
}
// The left operand made of two neighbouring accumulator blocks
template <int TERMS>
__device__ __forceinline__ void left_of(uint32_t (&a)[TERMS][4], const Acc &x, const Acc &y, float s) {
    uint32_t w[TERMS];
    terms<TERMS>(x[0] * s, x[1] * s, w);
#pragma unroll
    for (int i = 0; i < TERMS; ++i) a[i][0] = w[i];
    terms<TERMS>(x[2] * s, x[3] * s, w);
#pragma unroll
    for (int i = 0; i < TERMS; ++i) a[i][1] = w[i];
    terms<TERMS>(y[0] * s, y[1] * s, w);
#pragma unroll
    for (int i = 0; i < TERMS; ++i) a[i][2] = w[i];
    terms<TERMS>(y[2] * s, y[3] * s, w);
#pragma unroll
    for (int i = 0; i < TERMS; ++i) a[i][3] = w[i];
}
// The scale of the warp's N blocks
template <int N>
__device__ __forceinline__ float warp_scale(const Acc (&x)[N]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(fmaxf(m, fmaxf(fabsf(x[i][0]), fabsf(x[i][1]))), fmaxf(fabsf(x[i][2]), fabsf(x[i][3])));
    return scale_for(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))));
}

// ------------------------------------------------------------------------------------------------
// Copies
// ------------------------------------------------------------------------------------------------
// 16 bytes, of which the first `bytes` are read and the others become zero
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes = 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 4 bytes
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// bytes (a multiple of 16, as both addresses are), counted on a barrier
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
                 "r"(bar)
                 : "memory");
}

// Eight elements at p as they lie there, of which the first n exist; the others are zero. words: p is on 16 bytes and n is at least 8, or 0 or less (in
// float32 also 4). The loads of several calls go out together; the conversion comes after.
template <typename T>
struct Raw {
    uint32_t w[2 * sizeof(T)];
    __device__ __forceinline__ void load(const T *p, int n, bool words) {
        constexpr int kEl = 16 / sizeof(T);
        if (words) {
#pragma unroll
            for (int i = 0; i < 8 / kEl; ++i) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (i * kEl < n) x = reinterpret_cast<const uint4 *>(p)[i];
                w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
            }
        } else {
            T x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = from_f32<T>(0.0f);
                if (i < n) x[i] = p[i];
            }
            memcpy(w, x, sizeof(w));
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        constexpr int kEach = 4 / sizeof(T);
#pragma unroll
        for (int i = 0; i < 8 / kEach; ++i) {
            const Vec<kEach> f = unpack<T>(w[i]);
#pragma unroll
            for (int e = 0; e < kEach; ++e) x[i * kEach + e] = f.v[e];
        }
    }
};
// The terms of eight scaled elements as a word of each term's image
template <int TERMS>
__device__ __forceinline__ void words_of(uint4 (&w)[TERMS], const float (&x)[8], float s) {
    uint32_t t[4][TERMS];
#pragma unroll
    for (int i = 0; i < 4; ++i) terms<TERMS>(x[2 * i] * s, x[2 * i + 1] * s, t[i]);
#pragma unroll
    for (int j = 0; j < TERMS; ++j) w[j] = make_uint4(t[0][j], t[1][j], t[2][j], t[3][j]);
}
__device__ __forceinline__ float most8(float m, const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    return m;
}
// The largest of the CTA's m >= 0; at: WARPS places that nothing else uses between the barriers in front and behind
template <int WARPS>
__device__ __forceinline__ float cta_most(float m, float *at) {
    const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
    if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = __uint_as_float(w);
    __syncthreads();
    float r = at[0];
#pragma unroll
    for (int i = 1; i < WARPS; ++i) r = fmaxf(r, at[i]);
    __syncthreads();
    return r;
}

// The rows of batch entry b that exist.
__device__ __forceinline__ int live_rows(const DeltaParams &p, int b) {
    if (!p.lengths) return p.T;
    const int n = p.lengths[b];
    return n < 0 ? 0 : n > p.T ? p.T : n;
}

}  // namespace based
