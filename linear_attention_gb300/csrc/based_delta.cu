// based_delta.cu: the gated delta rule (declared in include/based_ops.h).
//
//     S_t = a_t S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - a_t S_{t-1}^T k_t),   o_t = scale S_t^T q_t
//
// A chunk of 64 rows takes a few matrix products instead of 64 steps. With b_i the sum of log decays up to row i of
// the chunk, D_ij = exp(b_i - b_j) for j <= i, S0 the state in front, grow_i = exp(b_i) and rest_i = exp(b_last - b_i):
//     X = V - grow K S0,   E = (1 + L)^-1 X with L_ij = D_ij (k_i k_j) beta_j below the diagonal,   U = beta E,
//     O = scale grow Q S0 + P U with P_ij = scale D_ij (q_i k_j),   S = grow_last S0 + (rest K)^T U.
// delta_prep_kernel has all that does not depend on the state (the inverse and P), for all chunks at once;
// delta_fwd_kernel runs through the chunks. Backward, with G the gradient of the state behind the chunk and A_ij = beta_i D_ij (k_i k_j):
//     dU = P^T dO + rest K G,   dR = (1 + A)^-T dU,   dV = beta dR,
//     G' = grow_last G + scale (grow Q)^T dO - (beta grow K)^T dR
// runs through the chunks from the last (delta_bwd_kernel), and what is left is again for all chunks at once
// (delta_grad_kernel, where its formulas are).
#include "delta_common.cuh"

namespace based {
namespace {

// ------------------------------------------------------------------------------------------------
// What does not depend on the state
// ------------------------------------------------------------------------------------------------
constexpr int kPrepWarps = 4;
constexpr int kLd = 68;  // floats in a row of the square matrices in shared memory

template <typename T, int KP>
struct PrepSmem {
    static constexpr int squares = kChunk * kLd * 4;
    static constexpr int images = Rec<T, KP>::qk, work = 2 * squares + 32 * 36 * 4;
    static constexpr int shared = images > work ? images : work;  // the images, then the inverse's work in their place
    static constexpr int bytes = shared + 2 * squares + (3 * kChunk + 16) * 4;
};

// Rows of q or k into their images, in shared memory and in the record; returns the scale's inverse.
template <typename T, int KP>
__device__ __forceinline__ float make_image(const T *src, int64_t stride, int rows, int K, bool vec, uint8_t *img, uint8_t *rec, float *red) {
    constexpr int kWords = KP / 8, kEach = kChunk * kWords / (32 * kPrepWarps), kStep = 32 * kPrepWarps / kWords;
    const int word = threadIdx.x % kWords, row0 = threadIdx.x / kWords;
    float x[kEach][8], most = 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int row = row0 + i * kStep;
        load8(x[i], src + row * stride + word * 8, row < rows ? K - word * 8 : 0, vec);
        most = most8(most, x[i]);
    }
    const float s = scale_for(cta_most<kPrepWarps>(most, red));
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        uint4 w[Terms<T>::in];
        words_of<Terms<T>::in>(w, x[i], s);
        const uint32_t at = word_at<KP>(row0 + i * kStep, word);
#pragma unroll
        for (int j = 0; j < Terms<T>::in; ++j) {
            *reinterpret_cast<uint4 *>(img + j * Rec<T, KP>::term + at) = w[j];
            *reinterpret_cast<uint4 *>(rec + j * Rec<T, KP>::term + at) = w[j];
        }
    }
    return inverse_of(s);
}

// The terms of a 64 x 64 matrix, held in x as rows (threadIdx.x / 8) + 16 r and words threadIdx.x % 8, into the record
template <int TERMS>
__device__ __forceinline__ float put_square(const float (&x)[4][8], uint8_t *rec, float *red) {
    float most = 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) most = most8(most, x[r]);
    const float s = scale_for(cta_most<kPrepWarps>(most, red));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        uint4 w[TERMS];
        words_of<TERMS>(w, x[r], s);
        const uint32_t at = word_at<kChunk>(threadIdx.x / 8 + 16 * r, threadIdx.x % 8);
#pragma unroll
        for (int j = 0; j < TERMS; ++j) *reinterpret_cast<uint4 *>(rec + j * kSquare + at) = w[j];
    }
    return inverse_of(s);
}

// C = sign A B for N x N blocks in shared memory, by `count` threads of which this is number i
template <int N>
__device__ __forceinline__ void small_product(float *c, int ldc, const float *a, int lda, const float *b, int ldb, float sign, int i, int count) {
    for (int e = i * 4; e < N * N; e += count * 4) {
        const int row = e / N, col = e % N;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int m = 0; m < N; ++m) {
            const float x = a[row * lda + m];
            const float4 y = *reinterpret_cast<const float4 *>(b + m * ldb + col);
            s.x = fmaf(x, y.x, s.x), s.y = fmaf(x, y.y, s.y), s.z = fmaf(x, y.z, s.z), s.w = fmaf(x, y.w, s.w);
        }
        *reinterpret_cast<float4 *>(c + row * ldc + col) = make_float4(sign * s.x, sign * s.y, sign * s.z, sign * s.w);
    }
}

// h = (1 + m)^-1 for m strictly lower triangular, by blocks: the inverses of the 16 x 16 blocks on the diagonal by substitution,
// then twice [A 0; C B]^-1 = [A^-1 0; -B^-1 C A^-1 B^-1]. float32 throughout: the inverse's rounding is that of plain substitution.
__device__ __forceinline__ void invert(float *h, const float *m, float *w) {
    const int tid = threadIdx.x;
    if (tid < kChunk) {
        const int block = tid & ~15, j = tid & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = 0.0f;
#pragma unroll
            for (int l = 0; l < i; ++l) s = fmaf(m[(block + i) * kLd + block + l], x[l], s);
            x[i] = i == j ? 1.0f : i < j ? 0.0f : -s;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) h[(block + i) * kLd + tid] = x[i];
    }
    __syncthreads();
    {
        const int pair = tid / 64, a = 32 * pair, b = a + 16;
        float *const t = w + pair * 16 * 36;
        small_product<16>(t, 36, m + b * kLd + a, kLd, h + a * kLd + a, kLd, 1.0f, tid % 64, 64);
        __syncthreads();
        small_product<16>(h + b * kLd + a, kLd, h + b * kLd + b, kLd, t, 36, -1.0f, tid % 64, 64);
    }
    __syncthreads();
    small_product<32>(w, 36, m + 32 * kLd, kLd, h, kLd, 1.0f, tid, 32 * kPrepWarps);
    __syncthreads();
    small_product<32>(h + 32 * kLd, kLd, h + 32 * kLd + 32, kLd, w, 36, -1.0f, tid, 32 * kPrepWarps);
    __syncthreads();
}

// One chunk of one key head, and all value heads that share it.
template <typename T, int KP, bool BWD>
__global__ void __launch_bounds__(32 * kPrepWarps) based_delta_prep_kernel(DeltaParams p) {
    using R = Rec<T, KP>;
    using Sm = PrepSmem<T, KP>;
    extern __shared__ __align__(128) uint8_t smem[];
    float *const gk = reinterpret_cast<float *>(smem + Sm::shared), *const gq = gk + kChunk * kLd;
    float *const m = reinterpret_cast<float *>(smem), *const h = m + kChunk * kLd, *const w = h + kChunk * kLd;
    float *const bhi = gq + kChunk * kLd, *const blo = bhi + kChunk, *const beta = blo + kChunk, *const red = beta + kChunk;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = blockIdx.x, hk = blockIdx.y, group = p.H / p.HK;
    griddep_wait();
    for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
        const int rows = min(kChunk, live_rows(p, b) - n * kChunk);
        if (rows <= 0) continue;  // the same for all threads
        const int64_t t0 = static_cast<int64_t>(n) * kChunk;
        uint8_t *const rec = p.qk_rec + ((static_cast<int64_t>(b) * p.HK + hk) * p.chunks + n) * R::qk;
        const T *const ks = static_cast<const T *>(p.k) + b * p.k_sb + t0 * p.k_st + hk * p.k_sh;
        const T *const qs = static_cast<const T *>(p.q) + b * p.q_sb + t0 * p.q_st + hk * p.q_sh;
        __syncthreads();  // the batch entry before
        const float ik = make_image<T, KP>(ks, p.k_st, rows, p.K, p.qk_vec, smem, rec, red);
        const float iq = make_image<T, KP>(qs, p.q_st, rows, p.K, p.qk_vec, smem + R::img, rec + R::img, red);
        __syncthreads();
        {  // the products of keys with keys and queries: rows 16 warp .. + 15, columns up to the diagonal
            Acc sk[8] = {}, sq[8] = {};
            const uint32_t kimg = smem_u32(smem), qimg = kimg + R::img;
            constexpr int NT = Terms<T>::in;
#pragma unroll
            for (int kk = 0; kk < KP / 16; ++kk) {
                uint32_t a[NT][4], c[NT][4];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    left<KP>(a[j], kimg + j * R::term, 16 * warp, 16 * kk, lane);
                    left<KP>(c[j], qimg + j * R::term, 16 * warp, 16 * kk, lane);
                }
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    if (np > warp) continue;
                    uint32_t x[NT][4];
#pragma unroll
                    for (int j = 0; j < NT; ++j) right<KP>(x[j], kimg + j * R::term, 16 * np, 16 * kk, lane);
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i + j < NT; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                mma(sk[2 * np + e], a[i], x[j][2 * e], x[j][2 * e + 1]);
                                mma(sq[2 * np + e], c[i], x[j][2 * e], x[j][2 * e + 1]);
                            }
                }
            }
            const float fk = ik * ik, fq = iq * ik * p.scale;
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const int at = (16 * warp + lane / 4) * kLd + 8 * nt + 2 * (lane % 4);
                *reinterpret_cast<float2 *>(gk + at) = make_float2(sk[nt][0] * fk, sk[nt][1] * fk);
                *reinterpret_cast<float2 *>(gk + at + 8 * kLd) = make_float2(sk[nt][2] * fk, sk[nt][3] * fk);
                *reinterpret_cast<float2 *>(gq + at) = make_float2(sq[nt][0] * fq, sq[nt][1] * fq);
                *reinterpret_cast<float2 *>(gq + at + 8 * kLd) = make_float2(sq[nt][2] * fq, sq[nt][3] * fq);
            }
        }
        for (int hh = 0; hh < group; ++hh) {
            const int head = hk * group + hh;
            uint8_t *const g = p.g_rec + ((static_cast<int64_t>(b) * p.H + head) * p.chunks + n) * R::g(BWD);
            float *const f = reinterpret_cast<float *>(g + (2 + R::scores(BWD)) * kSquare);
            if (warp == 0) {
                // Sums of log decays in 64 bits, kept as two floats: differences of neighbours then have float32's relative
                // accuracy however much has decayed before. -1e5 stands for anything below it, -inf among it: its decay is 0.
                double x[2], be[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 2 * lane + e;
                    float v = 0.0f, y = 0.0f;
                    if (i < rows) {
                        if (p.gate) v = to_f32(static_cast<const T *>(p.gate)[b * p.gate_sb + (t0 + i) * p.gate_st + head]);
                        y = to_f32(static_cast<const T *>(p.beta)[b * p.beta_sb + (t0 + i) * p.beta_st + head]);
                    }
                    x[e] = v < -1e5f ? -1e5 : static_cast<double>(v), be[e] = y;
                }
                x[1] += x[0];
                double sum = x[1];
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const double o = __shfl_up_sync(0xffffffffu, sum, d);
                    if (lane >= d) sum += o;
                }
                const double before = sum - x[1];
                const double last = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 2 * lane + e;
                    const double v = before + x[e];
                    bhi[i] = static_cast<float>(v), blo[i] = static_cast<float>(v - bhi[i]), beta[i] = static_cast<float>(be[e]);
                    f[F_GROW + i] = expf(static_cast<float>(v)), f[F_REST + i] = expf(static_cast<float>(last - v));
                    f[F_BETA + i] = beta[i], f[F_BHI + i] = bhi[i], f[F_BLO + i] = blo[i];
                }
                if (lane == 0) f[F_WHOLE] = expf(static_cast<float>(last)), f[F_K] = ik, f[F_Q] = iq;
            }
            __syncthreads();  // the sums, and the images are done with
            float x[4][8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = tid / 8 + 16 * r, j0 = tid % 8 * 8;
                float k8[8], q8[8], y[8];
                load8(k8, gk + i * kLd + j0, 8, true), load8(q8, gq + i * kLd + j0, 8, true);
                const float hi = bhi[i], lo = blo[i], bi = beta[i];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = j0 + e;
                    const float d = j <= i ? expf((hi - bhi[j]) + (lo - blo[j])) : 0.0f;
                    x[r][e] = j <= i ? d * q8[e] : 0.0f;
                    y[e] = j < i ? d * k8[e] * (BWD ? bi : beta[j]) : 0.0f;
                }
                float4 *const to = reinterpret_cast<float4 *>(m + i * kLd + j0), *const zero = reinterpret_cast<float4 *>(h + i * kLd + j0);
                to[0] = make_float4(y[0], y[1], y[2], y[3]), to[1] = make_float4(y[4], y[5], y[6], y[7]);
                zero[0] = zero[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            const float ip = put_square<R::scores(BWD)>(x, g + 2 * kSquare, red);  // with a barrier
            invert(h, m, w);
#pragma unroll
            for (int r = 0; r < 4; ++r) load8(x[r], h + (tid / 8 + 16 * r) * kLd + tid % 8 * 8, 8, true);
            const float ih = put_square<2>(x, g, red);
            if (tid == 0) f[F_INV] = ih, f[F_P] = ip;
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Through the chunks. A warp owns 16 channels of the values: the state's transpose, 16 x KP, lies in its accumulators, so every
// product's left operand comes from the warp's own registers, and the records in shared memory serve all warps of the CTA.
// ------------------------------------------------------------------------------------------------
constexpr int kSlice = 16;
constexpr int kMostWarps = 8;

template <typename T, int KP>
struct SeqSmem {
    static constexpr int row = sizeof(T) == 2 ? 32 : 80;  // bytes of a row of 16 values: 32-bit ones lie apart so that four rows' banks differ
    static constexpr int tile = kChunk * row;
    // of float32 with 128 channels of keys, two chunks' records leave room for the tiles of two warps
    static constexpr int warps = sizeof(T) == 4 && KP == 128 ? 2 : kMostWarps;
    __host__ __device__ static constexpr int stage(bool bwd) { return Rec<T, KP>::qk + Rec<T, KP>::g(bwd); }
    static constexpr int bytes(bool bwd, int warps) { return 2 * stage(bwd) + 2 * warps * tile; }
};

// A warp's 64 x 16 tile of v, dout or an output: where its words lie
template <typename T>
__device__ __forceinline__ uint32_t tile_word(int row, int word) {
    if constexpr (sizeof(T) == 2) return row * 32 + ((word ^ (row >> 2 & 1)) << 4);
    return row * 80 + (word << 4);
}
// Rows [0, rows) of the channels [0, cols) at src; zeros elsewhere. By one warp.
template <typename T>
__device__ __forceinline__ void load_tile(uint8_t *tile, const T *src, int64_t stride, int rows, int cols, bool vec, int lane) {
    constexpr int kWords = sizeof(T), kEl = 16 / sizeof(T);  // two words of eight, or four of four elements a row
    if (vec) {
#pragma unroll
        for (int i = 0; i < 2 * kWords; ++i) {
            const int row = (lane + 32 * i) / kWords, word = (lane + 32 * i) % kWords;
            const bool there = row < rows && word * kEl < cols;
            copy16(smem_u32(tile) + tile_word<T>(row, word), there ? src + row * stride + word * kEl : src, there ? 16 : 0);
        }
    } else {
#pragma unroll 4
        for (int i = lane; i < kChunk * kSlice; i += 32) {
            const int row = i / kSlice, c = i % kSlice;
            T v = from_f32<T>(0.0f);
            if (row < rows && c < cols) v = src[row * stride + c];
            *reinterpret_cast<T *>(tile + tile_word<T>(row, c / kEl) + c % kEl * sizeof(T)) = v;
        }
    }
}
// The tile's transpose as accumulator blocks: rows are channels, columns the chunk's rows
template <typename T>
__device__ __forceinline__ void read_tile(Acc (&x)[8], const uint8_t *tile, int lane) {
#pragma unroll
    for (int np = 0; np < 4; ++np) {
        if constexpr (sizeof(T) == 2) {
            uint32_t r[4];
            ldsm_t(r, smem_u32(tile) + tile_word<T>(16 * np + (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Vec<2> f = unpack<T>(r[i]);
                x[2 * np + i / 2][2 * (i % 2)] = f.v[0], x[2 * np + i / 2][2 * (i % 2) + 1] = f.v[1];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = 16 * np + 8 * (e / 4) + 2 * (lane & 3) + e % 2, c = (lane >> 2) + 8 * (e / 2 % 2);
                x[2 * np + e / 4][e % 4] = *reinterpret_cast<const float *>(tile + row * 80 + c * 4);
            }
        }
    }
}
template <typename T>
__device__ __forceinline__ void write_tile(uint8_t *tile, const Acc (&x)[8], int lane) {
#pragma unroll
    for (int np = 0; np < 4; ++np) {
        if constexpr (sizeof(T) == 2) {
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = pack<T>(Vec<2>{{x[2 * np + i / 2][2 * (i % 2)], x[2 * np + i / 2][2 * (i % 2) + 1]}});
            stsm_t(smem_u32(tile) + tile_word<T>(16 * np + (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1), r[0], r[1], r[2], r[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = 16 * np + 8 * (e / 4) + 2 * (lane & 3) + e % 2, c = (lane >> 2) + 8 * (e / 2 % 2);
                *reinterpret_cast<float *>(tile + row * 80 + c * 4) = x[2 * np + e / 4][e % 4];
            }
        }
    }
}
// Rows [0, rows) of the tile, and zeros up to row `all`, to dst
template <typename T>
__device__ __forceinline__ void store_tile(T *dst, int64_t stride, const uint8_t *tile, int rows, int all, int cols, bool vec, int lane) {
    constexpr int kWords = sizeof(T), kEl = 16 / sizeof(T);
    if (vec) {
#pragma unroll
        for (int i = 0; i < 2 * kWords; ++i) {
            const int row = (lane + 32 * i) / kWords, word = (lane + 32 * i) % kWords;
            if (row < all && word * kEl < cols)
                *reinterpret_cast<uint4 *>(dst + row * stride + word * kEl) =
                    row < rows ? *reinterpret_cast<const uint4 *>(tile + tile_word<T>(row, word)) : make_uint4(0, 0, 0, 0);
        }
    } else {
#pragma unroll 4
        for (int i = lane; i < kChunk * kSlice; i += 32) {
            const int row = i / kSlice, c = i % kSlice;
            if (row < all && c < cols)
                dst[row * stride + c] =
                    row < rows ? *reinterpret_cast<const T *>(tile + tile_word<T>(row, c / kEl) + c % kEl * sizeof(T)) : from_f32<T>(0.0f);
        }
    }
}
// A state (K,V) at p, or its transpose in the accumulators
template <int KP>
__device__ __forceinline__ void read_state(Acc (&s)[KP / 8], const float *p, int K, int V, int v0, int lane) {
#pragma unroll
    for (int j = 0; j < KP / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = 8 * j + 2 * (lane & 3) + e % 2, v = v0 + (lane >> 2) + 8 * (e / 2);
            s[j][e] = p && k < K && v < V ? p[static_cast<int64_t>(k) * V + v] : 0.0f;
        }
}
template <int KP>
__device__ __forceinline__ void write_state(float *p, const Acc (&s)[KP / 8], int K, int V, int v0, int lane) {
#pragma unroll
    for (int j = 0; j < KP / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = 8 * j + 2 * (lane & 3) + e % 2, v = v0 + (lane >> 2) + 8 * (e / 2);
            if (k < K && v < V) p[static_cast<int64_t>(k) * V + v] = s[j][e];
        }
}
// The transpose of rows of 32-bit values, (rows) x (V), as they lie in the accumulators
__device__ __forceinline__ void write_rows(float *p, int64_t stride, const Acc (&x)[8], int rows, int V, int v0, int lane) {
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = 8 * nt + 2 * (lane & 3) + e % 2, v = v0 + (lane >> 2) + 8 * (e / 2);
            if (row < rows && v < V) p[row * stride + v] = x[nt][e];
        }
}
// Elements of columns of x times f[column] and by rows times c0 or c1
__device__ __forceinline__ void by_columns(Acc (&x)[8], const float *f, float c0, float c1, int lane) {
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
        const float2 y = *reinterpret_cast<const float2 *>(f + 8 * nt + 2 * (lane & 3));
        x[nt][0] *= y.x * c0, x[nt][1] *= y.y * c0, x[nt][2] *= y.x * c1, x[nt][3] *= y.y * c1;
    }
}
__device__ __forceinline__ void by_rows(Acc (&x)[8], float c0, float c1) {
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) x[nt][0] *= c0, x[nt][1] *= c0, x[nt][2] *= c1, x[nt][3] *= c1;
}
template <int N>
__device__ __forceinline__ void clear(Acc (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.0f;
}
// Two 16 x 8 blocks += the left operand's LT terms times the RT terms of a right operand
template <int LT, int RT>
__device__ __forceinline__ void products(Acc &x, Acc &y, const uint32_t (&a)[LT][4], const uint32_t (&b)[RT][4]) {
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int i = 0; i < LT; ++i)
            if (i + j < 2) {
                mma(x, a[i], b[j][0], b[j][1]);
                mma(y, a[i], b[j][2], b[j][3]);
            }
}

// x = M^T or M of the record (a lower triangular 64 x 64 image of RT terms) applied to y along its columns:
// TURN false: x[.][i] = sum over j <= i of y[.][j] M[i][j]; true: x[.][j] = sum over i >= j of y[.][i] M[i][j]
template <bool TURN, int LT, int RT>
__device__ __forceinline__ void triangle(Acc (&x)[8], const Acc (&y)[8], float s0, float s1, uint32_t img, int lane) {
    clear(x);
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
        uint32_t a[LT][4];
        left_of<LT>(a, y[2 * kb], y[2 * kb + 1], s0, s1);
#pragma unroll
        for (int np = TURN ? 0 : kb; np < (TURN ? kb + 1 : 4); ++np) {
            uint32_t b[RT][4];
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                if (TURN)
                    right_t<kChunk>(b[j], img + j * kSquare, 16 * kb, 16 * np, lane);
                else
                    right<kChunk>(b[j], img + j * kSquare, 16 * np, 16 * kb, lane);
            }
            products<LT, RT>(x[2 * np], x[2 * np + 1], a, b);
        }
    }
}

// The records of a chunk, by all threads of the CTA
__device__ __forceinline__ void copy_records(uint8_t *to, const uint8_t *qk, int qk_bytes, const uint8_t *g, int g_bytes) {
    const uint32_t at = smem_u32(to);
    for (int i = threadIdx.x * 16; i < qk_bytes; i += blockDim.x * 16) copy16(at + i, qk + i);
    for (int i = threadIdx.x * 16; i < g_bytes; i += blockDim.x * 16) copy16(at + qk_bytes + i, g + i);
}

template <typename T, int KP>
__global__ void __launch_bounds__(32 * kMostWarps, 1) based_delta_fwd_kernel(DeltaParams p) {
    using R = Rec<T, KP>;
    using Sm = SeqSmem<T, KP>;
    constexpr int NI = Terms<T>::in, NO = Terms<T>::out, kStage = Sm::stage(false);
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int head = blockIdx.y, hk = head / (p.H / p.HK), v0 = (blockIdx.x * warps + warp) * kSlice;
    uint8_t *const tiles = smem + 2 * kStage + 2 * warp * Sm::tile;
    const int cols = p.V - v0;  // of this warp; may be none
    griddep_wait();
    for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
        const int live = live_rows(p, b), count = (live + kChunk - 1) / kChunk;
        const int64_t st = static_cast<int64_t>(b) * p.H + head, first = static_cast<int64_t>(b) * p.T;
        const uint8_t *const qk = p.qk_rec + (static_cast<int64_t>(b) * p.HK + hk) * p.chunks * R::qk;
        const uint8_t *const g = p.g_rec + st * p.chunks * R::g(false);
        const T *const v = static_cast<const T *>(p.v) + b * p.v_sb + head * p.v_sh + v0;
        T *const o = static_cast<T *>(p.out) + (first * p.H + head) * p.V + v0;
        const int64_t row_o = static_cast<int64_t>(p.H) * p.V;
        const auto fetch = [&](int n) {
            copy_records(smem + (n & 1) * kStage, qk + static_cast<int64_t>(n) * R::qk, R::qk, g + static_cast<int64_t>(n) * R::g(false), R::g(false));
            if (cols > 0)
                load_tile(tiles + (n & 1) * Sm::tile, v + static_cast<int64_t>(n) * kChunk * p.v_st, p.v_st, live - n * kChunk, cols, p.v_vec, lane);
            copies_commit();
        };
        Acc s[KP / 8];
        read_state<KP>(s, p.state ? p.state + st * p.K * p.V : nullptr, p.K, p.V, v0, lane);
        __syncthreads();  // the batch entry before
        if (count > 0) fetch(0);
        for (int n = 0; n < count; ++n) {
            copies_wait();
            __syncthreads();  // chunk n is there, and chunk n - 1 done with
            if (n + 1 < count) fetch(n + 1);
            if (cols <= 0) continue;
            const int rows = live - n * kChunk < kChunk ? live - n * kChunk : kChunk;
            const int64_t t0 = static_cast<int64_t>(n) * kChunk;
            uint8_t *const tile = tiles + (n & 1) * Sm::tile;
            const uint32_t kimg = smem_u32(smem) + (n & 1) * kStage, qimg = kimg + R::img, inv = kimg + R::qk;
            const float *const f = reinterpret_cast<const float *>(smem + (n & 1) * kStage + R::qk + (2 + NO) * kSquare);
            if (p.states) write_state<KP>(p.states + ((static_cast<int64_t>(b) * p.chunks + n) * p.H + head) * p.K * p.V, s, p.K, p.V, v0, lane);
            float s0, s1;
            row_scales(s, s0, s1);
            Acc x[8], y[8], z[8];
            clear(x), clear(z);
#pragma unroll
            for (int kk = 0; kk < KP / 16; ++kk) {  // x = S0^T K^T, z = S0^T Q^T
                uint32_t a[2][4];
                left_of<2>(a, s[2 * kk], s[2 * kk + 1], s0, s1);
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    uint32_t r[NI][4];
#pragma unroll
                    for (int j = 0; j < NI; ++j) right<KP>(r[j], kimg + j * R::term, 16 * np, 16 * kk, lane);
                    products<2, NI>(x[2 * np], x[2 * np + 1], a, r);
#pragma unroll
                    for (int j = 0; j < NI; ++j) right<KP>(r[j], qimg + j * R::term, 16 * np, 16 * kk, lane);
                    products<NO, NI>(z[2 * np], z[2 * np + 1], reinterpret_cast<const uint32_t(&)[NO][4]>(a), r);
                }
            }
            s0 = inverse_of(s0), s1 = inverse_of(s1);
            by_columns(x, f + F_GROW, s0 * f[F_K], s1 * f[F_K], lane);
            by_columns(z, f + F_GROW, s0 * f[F_Q] * p.scale, s1 * f[F_Q] * p.scale, lane);
            read_tile<T>(y, tile, lane);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[nt][e] = y[nt][e] - x[nt][e];
            row_scales(x, s0, s1);
            triangle<false, 2, 2>(y, x, s0, s1, inv, lane);
            by_rows(y, inverse_of(s0) * f[F_INV], inverse_of(s1) * f[F_INV]);  // E
            if (p.errors) write_rows(p.errors + ((first + t0) * p.H + head) * p.V, row_o, y, rows, p.V, v0, lane);
            by_columns(y, f + F_BETA, 1.0f, 1.0f, lane);  // U
            row_scales(y, s0, s1);
            triangle<false, NO, NO>(x, y, s0, s1, inv + 2 * kSquare, lane);
            by_rows(x, inverse_of(s0) * f[F_P], inverse_of(s1) * f[F_P]);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[nt][e] += x[nt][e];
            __syncwarp();  // the tile is read
            write_tile<T>(tile, z, lane);
            __syncwarp();
            store_tile<T>(o + t0 * row_o, row_o, tile, rows, static_cast<int>(p.T - t0 < kChunk ? p.T - t0 : kChunk), cols, p.o_vec, lane);
            by_columns(y, f + F_REST, 1.0f, 1.0f, lane);
            row_scales(y, s0, s1);
            uint32_t a[4][2][4];
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) left_of<2>(a[kb], y[2 * kb], y[2 * kb + 1], s0, s1);
            s0 = inverse_of(s0) * f[F_K], s1 = inverse_of(s1) * f[F_K];
            const float whole = f[F_WHOLE];
#pragma unroll
            for (int jp = 0; jp < KP / 32; ++jp) {  // S = whole S0 + K^T U, 32 keys' channels at a time
                Acc t[4];
                clear(t);
#pragma unroll
                for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t r[NI][4];
#pragma unroll
                        for (int j = 0; j < NI; ++j) right_t<KP>(r[j], kimg + j * R::term, 16 * kb, 32 * jp + 16 * e, lane);
                        products<2, NI>(t[2 * e], t[2 * e + 1], a[kb], r);
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    Acc &w = s[4 * jp + i];
                    w[0] = fmaf(t[i][0], s0, w[0] * whole), w[1] = fmaf(t[i][1], s0, w[1] * whole);
                    w[2] = fmaf(t[i][2], s1, w[2] * whole), w[3] = fmaf(t[i][3], s1, w[3] * whole);
                }
            }
        }
        if (cols > 0) {
            for (int n = count; n < p.chunks; ++n) {
                const int64_t t0 = static_cast<int64_t>(n) * kChunk;
                store_tile<T>(o + t0 * row_o, row_o, tiles, 0, static_cast<int>(p.T - t0 < kChunk ? p.T - t0 : kChunk), cols, p.o_vec, lane);
            }
            if (p.final_state) write_state<KP>(p.final_state + st * p.K * p.V, s, p.K, p.V, v0, lane);
        }
    }
}

template <typename T, int KP>
__global__ void __launch_bounds__(32 * kMostWarps, 1) based_delta_bwd_kernel(DeltaParams p) {
    using R = Rec<T, KP>;
    using Sm = SeqSmem<T, KP>;
    constexpr int NI = Terms<T>::in, kStage = Sm::stage(true);
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int head = blockIdx.y, hk = head / (p.H / p.HK), v0 = (blockIdx.x * warps + warp) * kSlice;
    uint8_t *const tiles = smem + 2 * kStage + 2 * warp * Sm::tile;
    const int cols = p.V - v0;
    griddep_wait();
    for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
        const int live = live_rows(p, b), count = (live + kChunk - 1) / kChunk;
        const int64_t st = static_cast<int64_t>(b) * p.H + head, first = static_cast<int64_t>(b) * p.T;
        const uint8_t *const qk = p.qk_rec + (static_cast<int64_t>(b) * p.HK + hk) * p.chunks * R::qk;
        const uint8_t *const grec = p.g_rec + st * p.chunks * R::g(true);
        const T *const dout = static_cast<const T *>(p.dout) + b * p.do_sb + head * p.do_sh + v0;
        T *const dv = static_cast<T *>(p.out) + (first * p.H + head) * p.V + v0;
        const int64_t row_o = static_cast<int64_t>(p.H) * p.V;
        const auto fetch = [&](int n) {
            copy_records(smem + (n & 1) * kStage, qk + static_cast<int64_t>(n) * R::qk, R::qk, grec + static_cast<int64_t>(n) * R::g(true), R::g(true));
            if (cols > 0)
                load_tile(tiles + (n & 1) * Sm::tile, dout + static_cast<int64_t>(n) * kChunk * p.do_st, p.do_st, live - n * kChunk, cols, p.do_vec, lane);
            copies_commit();
        };
        Acc g[KP / 8];
        read_state<KP>(g, p.state ? p.state + st * p.K * p.V : nullptr, p.K, p.V, v0, lane);
        __syncthreads();
        if (count > 0) fetch(count - 1);
        for (int n = count - 1; n >= 0; --n) {
            copies_wait();
            __syncthreads();
            if (n > 0) fetch(n - 1);
            if (cols <= 0) continue;
            const int rows = live - n * kChunk < kChunk ? live - n * kChunk : kChunk;
            const int64_t t0 = static_cast<int64_t>(n) * kChunk;
            uint8_t *const tile = tiles + (n & 1) * Sm::tile;
            const uint32_t kimg = smem_u32(smem) + (n & 1) * kStage, qimg = kimg + R::img, inv = kimg + R::qk;
            const float *const f = reinterpret_cast<const float *>(smem + (n & 1) * kStage + R::qk + 4 * kSquare);
            write_state<KP>(p.dstates + ((static_cast<int64_t>(b) * p.chunks + n) * p.H + head) * p.K * p.V, g, p.K, p.V, v0, lane);
            float s0, s1;
            row_scales(g, s0, s1);
            Acc x[8], y[8], z[8];
            clear(x);
#pragma unroll
            for (int kk = 0; kk < KP / 16; ++kk) {  // x = G^T K^T
                uint32_t a[2][4];
                left_of<2>(a, g[2 * kk], g[2 * kk + 1], s0, s1);
#pragma unroll
                for (int np = 0; np < 4; ++np) {
                    uint32_t r[NI][4];
#pragma unroll
                    for (int j = 0; j < NI; ++j) right<KP>(r[j], kimg + j * R::term, 16 * np, 16 * kk, lane);
                    products<2, NI>(x[2 * np], x[2 * np + 1], a, r);
                }
            }
            by_columns(x, f + F_REST, inverse_of(s0) * f[F_K], inverse_of(s1) * f[F_K], lane);
            read_tile<T>(z, tile, lane);  // dO
            row_scales(z, s0, s1);
            triangle<true, NI, 2>(y, z, s0, s1, inv + 2 * kSquare, lane);
            s0 = inverse_of(s0) * f[F_P], s1 = inverse_of(s1) * f[F_P];
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[nt][e] = fmaf(y[nt][e], e < 2 ? s0 : s1, x[nt][e]);  // dU
            row_scales(x, s0, s1);
            triangle<true, 2, 2>(y, x, s0, s1, inv, lane);
            by_rows(y, inverse_of(s0) * f[F_INV], inverse_of(s1) * f[F_INV]);  // dR
            write_rows(p.dr + ((first + t0) * p.H + head) * p.V, row_o, y, rows, p.V, v0, lane);
            by_columns(y, f + F_BETA, 1.0f, 1.0f, lane);  // dV
            __syncwarp();
            write_tile<T>(tile, y, lane);
            __syncwarp();
            store_tile<T>(dv + t0 * row_o, row_o, tile, rows, static_cast<int>(p.T - t0 < kChunk ? p.T - t0 : kChunk), cols, p.o_vec, lane);
            by_columns(y, f + F_GROW, -1.0f, -1.0f, lane);
            by_columns(z, f + F_GROW, p.scale, p.scale, lane);
            uint32_t a[4][2][4], c[4][2][4];
            float u0, u1;
            row_scales(y, s0, s1), row_scales(z, u0, u1);
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {
                left_of<2>(a[kb], y[2 * kb], y[2 * kb + 1], s0, s1);
                left_of<2>(c[kb], z[2 * kb], z[2 * kb + 1], u0, u1);
            }
            s0 = inverse_of(s0) * f[F_K], s1 = inverse_of(s1) * f[F_K];
            u0 = inverse_of(u0) * f[F_Q], u1 = inverse_of(u1) * f[F_Q];
            const float whole = f[F_WHOLE];
#pragma unroll
            for (int jp = 0; jp < KP / 16; ++jp) {
                Acc t[2], w[2];
                clear(t), clear(w);
#pragma unroll
                for (int kb = 0; kb < 4; ++kb) {
                    uint32_t r[NI][4];
#pragma unroll
                    for (int j = 0; j < NI; ++j) right_t<KP>(r[j], kimg + j * R::term, 16 * kb, 16 * jp, lane);
                    products<2, NI>(t[0], t[1], a[kb], r);
#pragma unroll
                    for (int j = 0; j < NI; ++j) right_t<KP>(r[j], qimg + j * R::term, 16 * kb, 16 * jp, lane);
                    products<2, NI>(w[0], w[1], c[kb], r);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    Acc &d = g[2 * jp + i];
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[e] = fmaf(t[i][e], e < 2 ? s0 : s1, fmaf(w[i][e], e < 2 ? u0 : u1, d[e] * whole));
                }
            }
        }
        if (cols > 0) {
            for (int n = count; n < p.chunks; ++n) {
                const int64_t t0 = static_cast<int64_t>(n) * kChunk;
                store_tile<T>(dv + t0 * row_o, row_o, tiles, 0, static_cast<int>(p.T - t0 < kChunk ? p.T - t0 : kChunk), cols, p.o_vec, lane);
            }
            if (p.final_state) write_state<KP>(p.final_state + st * p.K * p.V, g, p.K, p.V, v0, lane);
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Gradients that need no order. With dP = dO U^T and dA = -dR U^T (below the diagonal),
//     dQ = scale grow dO S0^T + (scale D dP) K,
//     dK = rest U G^T - beta grow dR S0^T + (scale D dP)^T Q + (beta D dA) K + (beta D dA)^T K,
//     dbeta = rows of dR E,
// and the gradient of b_i, the sum of log decays up to row i, is what row i reads minus what it has written:
//     db_i = q_i (scale grow dO S0^T)_i - k_i (beta grow dR S0^T + rest U G^T)_i + sum_j (N_ij - N_ji),  N = dP P + dA A,
// with grow_last <S0, G> + sum_i k_i (rest U G^T)_i more at the last row; dgate_i is the sum of db from i on.
// A CTA takes one chunk of one key head and adds up the value heads that share it, so that nothing is added by atomics.
// ------------------------------------------------------------------------------------------------
constexpr int kGradWarps = 8;
constexpr int kTileV = 64;

template <typename T, int KP>
struct GradSmem {
    static constexpr int NO = Terms<T>::out;
    static constexpr int f = Rec<T, KP>::qk, dout = f + F_COUNT * 4, u = dout + NO * kSquare, dr = u + NO * kSquare, s = dr + NO * kSquare,
                         g = s + NO * KP * kTileV * 2, inv = g + NO * KP * kTileV * 2;  // the images' rows' inverse scales
    static constexpr int part = inv + (3 * kChunk + 2 * KP) * 4;                        // sums: rows 2 x 64, next 2 x 64, columns 4 x 64, dbeta 64
    static constexpr int red = part + 9 * kChunk * 4, bytes = red + 64;
};

// Rows of eight words into an image of 64 columns, each row with its own scale. x: the word that this thread holds
template <int NO>
__device__ __forceinline__ void put_row(uint8_t *img, int term, float *inv, int row, int word, const float (&x)[8]) {
    float m = most8(0.0f, x);
#pragma unroll
    for (int d = 1; d < 8; d *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float s = scale_for(m);
    uint4 w[NO];
    words_of<NO>(w, x, s);
#pragma unroll
    for (int j = 0; j < NO; ++j) *reinterpret_cast<uint4 *>(img + j * term + word_at<kTileV>(row, word)) = w[j];
    if (word == 0) inv[row] = inverse_of(s);
}
// Two neighbouring elements of an image of key or query rows
template <typename T, int KP>
__device__ __forceinline__ float2 image_pair(const uint8_t *img, int row, int col, float inv) {
    const uint8_t *const at = img + word_at<KP>(row, col >> 3) + (col & 7) * 2;
    const Vec<2> h = unpack<__half>(*reinterpret_cast<const uint32_t *>(at));
    float2 r = make_float2(h.v[0], h.v[1]);
    if constexpr (Terms<T>::in == 2) {
        const Vec<2> l = unpack<__half>(*reinterpret_cast<const uint32_t *>(at + Rec<T, KP>::term));
        r.x += l.v[0], r.y += l.v[1];
    }
    return make_float2(r.x * inv, r.y * inv);
}
// Two elements of a row of dq or dk
template <typename T>
__device__ __forceinline__ void store_pair(T *p, int col, int K, bool pair, float x, float y) {
    if (pair && col + 1 < K) {
        *reinterpret_cast<Pack<T, 2> *>(p + col) = {{from_f32<T>(x), from_f32<T>(y)}};
    } else {
        if (col < K) p[col] = from_f32<T>(x);
        if (col + 1 < K) p[col + 1] = from_f32<T>(y);
    }
}

template <typename T, int KP>
__global__ void __launch_bounds__(32 * kGradWarps) based_delta_grad_kernel(DeltaParams p) {
    using R = Rec<T, KP>;
    using Sm = GradSmem<T, KP>;
    constexpr int NI = Terms<T>::in, NO = Terms<T>::out, NB = KP / 16;  // a warp's blocks of keys' channels
    constexpr int kStateTerm = KP * kTileV * 2;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wm = warp & 3, wn = warp >> 2;
    const int n = blockIdx.x, hk = blockIdx.y, group = p.H / p.HK;
    const int r0 = 16 * wm + (lane >> 2), r1 = r0 + 8, col0 = wn * (KP / 2) + 2 * (lane & 3);  // this thread's accumulators
    float *const f = reinterpret_cast<float *>(smem + Sm::f);
    float *const inv_do = reinterpret_cast<float *>(smem + Sm::inv), *const inv_u = inv_do + kChunk, *const inv_dr = inv_u + kChunk,
                *const inv_s = inv_dr + kChunk, *const inv_g = inv_s + KP;
    float *const part_row = reinterpret_cast<float *>(smem + Sm::part), *const part_next = part_row + 2 * kChunk,
                *const part_col = part_next + 2 * kChunk, *const part_beta = part_col + 4 * kChunk, *const red = reinterpret_cast<float *>(smem + Sm::red);
    const uint32_t base = smem_u32(smem), kimg = base, qimg = base + R::img, i_do = base + Sm::dout, i_u = base + Sm::u, i_dr = base + Sm::dr,
                   i_s = base + Sm::s, i_g = base + Sm::g;
    const bool vec32 = p.V % 4 == 0, pair = p.K % 2 == 0;
    griddep_wait();
    for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
        const int64_t t0 = static_cast<int64_t>(n) * kChunk, first = static_cast<int64_t>(b) * p.T + t0;
        const int rows = min(kChunk, live_rows(p, b) - n * kChunk), all = static_cast<int>(p.T - t0 < kChunk ? p.T - t0 : kChunk);
        T *const dq = static_cast<T *>(p.dq) + (first * p.HK + hk) * p.K, *const dk = static_cast<T *>(p.dk) + (first * p.HK + hk) * p.K;
        const int64_t row_k = static_cast<int64_t>(p.HK) * p.K;
        // padding
        for (int i = tid; i < (all - (rows < 0 ? 0 : rows)) * p.K; i += 32 * kGradWarps) {
            const int row = (rows < 0 ? 0 : rows) + i / p.K, c = i % p.K;
            dq[row * row_k + c] = dk[row * row_k + c] = from_f32<T>(0.0f);
        }
        for (int i = tid; i < (all - (rows < 0 ? 0 : rows)) * group; i += 32 * kGradWarps) {
            const int64_t at = (first + (rows < 0 ? 0 : rows) + i / group) * p.H + hk * group + i % group;
            static_cast<T *>(p.dbeta)[at] = from_f32<T>(0.0f);
            if (p.dgate) static_cast<T *>(p.dgate)[at] = from_f32<T>(0.0f);
        }
        if (rows <= 0) continue;
        __syncthreads();  // the batch entry before
        copy_records(smem, p.qk_rec + ((static_cast<int64_t>(b) * p.HK + hk) * p.chunks + n) * R::qk, R::qk, nullptr, 0);
        copies_commit();
        Acc aq[NB], ak[NB];
        clear(aq), clear(ak);
        for (int hh = 0; hh < group; ++hh) {
            const int head = hk * group + hh;
            const uint8_t *const rec = p.g_rec + ((static_cast<int64_t>(b) * p.H + head) * p.chunks + n) * R::g(true) + 4 * kSquare;
            __syncthreads();  // the head before
            for (int i = tid; i < F_COUNT; i += 32 * kGradWarps) f[i] = reinterpret_cast<const float *>(rec)[i];
            if (tid < kChunk) part_beta[tid] = 0.0f;
            copies_wait();
            __syncthreads();
            const float ik = f[F_K], iq = f[F_Q];
            float row0 = 0.0f, row1 = 0.0f, next0 = 0.0f, next1 = 0.0f, dot = 0.0f;
            Acc dp[4], da[4];
            clear(dp), clear(da);
            const T *const dout = static_cast<const T *>(p.dout) + b * p.do_sb + t0 * p.do_st + head * p.do_sh;
            const int64_t val = (first * p.H + head) * p.V, row_v = static_cast<int64_t>(p.H) * p.V;
            const int64_t st = ((static_cast<int64_t>(b) * p.chunks + n) * p.H + head) * p.K * p.V;
            for (int v0 = 0; v0 < p.V; v0 += kTileV) {
                const int word = tid & 7, c = v0 + 8 * word;
                if (v0) __syncthreads();  // the tiles before
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = (tid >> 3) + 32 * i, there = row < rows ? p.V - c : 0;
                    float x[8], e[8];
                    load8(x, dout + row * p.do_st + c, there, p.do_vec);
                    put_row<NO>(smem + Sm::dout, kSquare, inv_do, row, word, x);
                    load8(e, p.errors + val + row * row_v + c, there, vec32);
                    load8(x, p.dr + val + row * row_v + c, there, vec32);
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum = fmaf(x[j], e[j], sum), e[j] *= f[F_BETA + row];
                    put_row<NO>(smem + Sm::u, kSquare, inv_u, row, word, e);
                    put_row<NO>(smem + Sm::dr, kSquare, inv_dr, row, word, x);
#pragma unroll
                    for (int d = 1; d < 8; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                    if (word == 0) part_beta[row] += sum;
                }
#pragma unroll
                for (int i = 0; i < KP / 32; ++i) {
                    const int row = (tid >> 3) + 32 * i, there = row < p.K ? p.V - c : 0;
                    float x[8], y[8];
                    load8(x, p.states + st + static_cast<int64_t>(row) * p.V + c, there, vec32);
                    load8(y, p.dstates + st + static_cast<int64_t>(row) * p.V + c, there, vec32);
#pragma unroll
                    for (int j = 0; j < 8; ++j) dot = fmaf(x[j], y[j], dot);
                    put_row<NO>(smem + Sm::s, kStateTerm, inv_s, row, word, x);
                    put_row<NO>(smem + Sm::g, kStateTerm, inv_g, row, word, y);
                }
                __syncthreads();
                // the left operand's rows 16 wm .. + 15 by the rows of a state's image
                const auto by_state = [&](Acc(&t)[NB], uint32_t l, uint32_t r) {
                    clear(t);
#pragma unroll
                    for (int kk = 0; kk < kTileV / 16; ++kk) {
                        uint32_t a[NO][4];
#pragma unroll
                        for (int j = 0; j < NO; ++j) left<kTileV>(a[j], l + j * kSquare, 16 * wm, 16 * kk, lane);
#pragma unroll
                        for (int jp = 0; jp < NB / 2; ++jp) {
                            uint32_t x[NO][4];
#pragma unroll
                            for (int j = 0; j < NO; ++j) right<kTileV>(x[j], r + j * kStateTerm, wn * (KP / 2) + 16 * jp, 16 * kk, lane);
                            products<NO, NO>(t[2 * jp], t[2 * jp + 1], a, x);
                        }
                    }
                };
                // to += t by rows' and columns' factors; returns its rows' products with the image's
                const auto add = [&](Acc(&to)[NB], const Acc(&t)[NB], float c0, float c1, const float *cols, const uint8_t *img, float inv, float &d0, float &d1) {
                    d0 = d1 = 0.0f;
#pragma unroll
                    for (int nt = 0; nt < NB; ++nt) {
                        const int col = col0 + 8 * nt;
                        const float2 y = *reinterpret_cast<const float2 *>(cols + col);
                        const float2 x0 = image_pair<T, KP>(img, r0, col, inv), x1 = image_pair<T, KP>(img, r1, col, inv);
                        const float z[4] = {t[nt][0] * (c0 * y.x), t[nt][1] * (c0 * y.y), t[nt][2] * (c1 * y.x), t[nt][3] * (c1 * y.y)};
                        d0 = fmaf(z[0], x0.x, fmaf(z[1], x0.y, d0)), d1 = fmaf(z[2], x1.x, fmaf(z[3], x1.y, d1));
#pragma unroll
                        for (int e = 0; e < 4; ++e) to[nt][e] += z[e];
                    }
                };
                {
                    Acc t[NB];
                    float d0, d1;
                    by_state(t, i_do, i_s);
                    add(aq, t, p.scale * f[F_GROW + r0] * inv_do[r0], p.scale * f[F_GROW + r1] * inv_do[r1], inv_s, smem + R::img, iq, d0, d1);
                    row0 += d0, row1 += d1;
                    by_state(t, i_dr, i_s);
                    add(ak, t, -f[F_BETA + r0] * f[F_GROW + r0] * inv_dr[r0], -f[F_BETA + r1] * f[F_GROW + r1] * inv_dr[r1], inv_s, smem, ik, d0, d1);
                    row0 += d0, row1 += d1;
                    by_state(t, i_u, i_g);
                    add(ak, t, f[F_REST + r0] * inv_u[r0], f[F_REST + r1] * inv_u[r1], inv_g, smem, ik, d0, d1);
                    next0 += d0, next1 += d1;
                }
                // dP and -dA: 32 columns of this warp
                Acc tp[4], ta[4];
                clear(tp), clear(ta);
#pragma unroll
                for (int kk = 0; kk < kTileV / 16; ++kk) {
                    uint32_t a[NO][4], c4[NO][4];
#pragma unroll
                    for (int j = 0; j < NO; ++j) {
                        left<kTileV>(a[j], i_do + j * kSquare, 16 * wm, 16 * kk, lane);
                        left<kTileV>(c4[j], i_dr + j * kSquare, 16 * wm, 16 * kk, lane);
                    }
#pragma unroll
                    for (int jp = 0; jp < 2; ++jp) {
                        if (2 * wn + jp > wm) continue;
                        uint32_t x[NO][4];
#pragma unroll
                        for (int j = 0; j < NO; ++j) right<kTileV>(x[j], i_u + j * kSquare, 32 * wn + 16 * jp, 16 * kk, lane);
                        products<NO, NO>(tp[2 * jp], tp[2 * jp + 1], a, x);
                        products<NO, NO>(ta[2 * jp], ta[2 * jp + 1], c4, x);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const float2 y = *reinterpret_cast<const float2 *>(inv_u + 32 * wn + 8 * nt + 2 * (lane & 3));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float w = e % 2 ? y.y : y.x;
                        dp[nt][e] = fmaf(tp[nt][e], w * inv_do[e < 2 ? r0 : r1], dp[nt][e]);
                        da[nt][e] = fmaf(ta[nt][e], -w * inv_dr[e < 2 ? r0 : r1], da[nt][e]);
                    }
                }
            }
            // the products of queries and keys with keys, and with them the pairs' sums and the factors of dQ and dK
            float pair0 = 0.0f, pair1 = 0.0f;
            {
                Acc sq[4], sk[4];
                clear(sq), clear(sk);
#pragma unroll
                for (int kk = 0; kk < KP / 16; ++kk) {
                    uint32_t a[NI][4], c4[NI][4];
#pragma unroll
                    for (int j = 0; j < NI; ++j) {
                        left<KP>(a[j], qimg + j * R::term, 16 * wm, 16 * kk, lane);
                        left<KP>(c4[j], kimg + j * R::term, 16 * wm, 16 * kk, lane);
                    }
#pragma unroll
                    for (int jp = 0; jp < 2; ++jp) {
                        if (2 * wn + jp > wm) continue;
                        uint32_t x[NI][4];
#pragma unroll
                        for (int j = 0; j < NI; ++j) right<KP>(x[j], kimg + j * R::term, 32 * wn + 16 * jp, 16 * kk, lane);
                        products<NI, NI>(sq[2 * jp], sq[2 * jp + 1], a, x);
                        products<NI, NI>(sk[2 * jp], sk[2 * jp + 1], c4, x);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    float col[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = e < 2 ? r0 : r1, j = 32 * wn + 8 * nt + 2 * (lane & 3) + e % 2;
                        const float d = j <= i ? expf((f[F_BHI + i] - f[F_BHI + j]) + (f[F_BLO + i] - f[F_BLO + j])) : 0.0f;
                        const float dq_ = j <= i ? d * p.scale : 0.0f, dk_ = j < i ? d * f[F_BETA + i] : 0.0f;
                        dp[nt][e] = j <= i ? dp[nt][e] * dq_ : 0.0f, da[nt][e] = j < i ? da[nt][e] * dk_ : 0.0f;
                        const float sum = j <= i ? dp[nt][e] * sq[nt][e] * (iq * ik) + da[nt][e] * sk[nt][e] * (ik * ik) : 0.0f;
                        (e < 2 ? pair0 : pair1) += sum;
                        col[e % 2] += sum;
                    }
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) col[0] += __shfl_xor_sync(0xffffffffu, col[0], d), col[1] += __shfl_xor_sync(0xffffffffu, col[1], d);
                    if (lane < 4) part_col[wm * kChunk + 32 * wn + 8 * nt + 2 * lane] = col[0], part_col[wm * kChunk + 32 * wn + 8 * nt + 2 * lane + 1] = col[1];
                }
            }
            row0 += pair0 - next0, row1 += pair1 - next1;
#pragma unroll
            for (int d = 1; d < 4; d *= 2) {
                row0 += __shfl_xor_sync(0xffffffffu, row0, d), row1 += __shfl_xor_sync(0xffffffffu, row1, d);
                next0 += __shfl_xor_sync(0xffffffffu, next0, d), next1 += __shfl_xor_sync(0xffffffffu, next1, d);
            }
            if ((lane & 3) == 0) {
                part_row[wn * kChunk + r0] = row0, part_row[wn * kChunk + r1] = row1;
                part_next[wn * kChunk + r0] = next0, part_next[wn * kChunk + r1] = next1;
            }
#pragma unroll
            for (int d = 1; d < 32; d *= 2) dot += __shfl_xor_sync(0xffffffffu, dot, d);
            float mp = 0.0f, ma = 0.0f;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) mp = fmaxf(mp, fabsf(dp[nt][e])), ma = fmaxf(ma, fabsf(da[nt][e]));
            mp = scale_for(cta_most<kGradWarps>(mp, red)), ma = scale_for(cta_most<kGradWarps>(ma, red));  // with barriers: the tiles are done with
            if (lane == 0) red[warp] = dot;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t at = word_at<kChunk>(e ? r1 : r0, 4 * wn + nt) + 4 * (lane & 3);
                    uint32_t w[NO];
                    terms<NO>(dp[nt][2 * e] * mp, dp[nt][2 * e + 1] * mp, w);
#pragma unroll
                    for (int j = 0; j < NO; ++j) *reinterpret_cast<uint32_t *>(smem + Sm::dout + j * kSquare + at) = w[j];
                    terms<NO>(da[nt][2 * e] * ma, da[nt][2 * e + 1] * ma, w);
#pragma unroll
                    for (int j = 0; j < NO; ++j) *reinterpret_cast<uint32_t *>(smem + Sm::dr + j * kSquare + at) = w[j];
                }
            __syncthreads();
            if (warp == 0) {
                float dots = 0.0f;
#pragma unroll
                for (int i = 0; i < kGradWarps; ++i) dots += red[i];
                float x[2], nx[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 2 * lane + e;
                    float c = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) c += part_col[j * kChunk + i];
                    x[e] = part_row[i] + part_row[kChunk + i] - c, nx[e] = part_next[i] + part_next[kChunk + i];
                }
                float end = nx[0] + nx[1];
#pragma unroll
                for (int d = 1; d < 32; d *= 2) end += __shfl_xor_sync(0xffffffffu, end, d);
                end = fmaf(f[F_WHOLE], dots, end);
                float sum = x[0] + x[1];  // from this lane's rows on
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const float o = __shfl_down_sync(0xffffffffu, sum, d);
                    if (lane + d < 32) sum += o;
                }
                const float behind = sum - (x[0] + x[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 2 * lane + e;
                    const float from = e ? behind + x[1] : behind + x[1] + x[0];
                    if (i < rows) {
                        const int64_t at = (first + i) * p.H + head;
                        static_cast<T *>(p.dbeta)[at] = from_f32<T>(part_beta[i]);
                        if (p.dgate) static_cast<T *>(p.dgate)[at] = from_f32<T>(from + end);
                    }
                }
            }
            {
                const auto rank = [&](Acc(&to)[NB], uint32_t l, uint32_t r, float c) {  // to += c times the lower triangle (TURN: its transpose) of l by the rows of r
                    Acc t[NB];
                    clear(t);
#pragma unroll
                    for (int kb = 0; kb < 4; ++kb) {
                        if (kb > wm) continue;
                        uint32_t a[NO][4];
#pragma unroll
                        for (int j = 0; j < NO; ++j) left<kChunk>(a[j], l + j * kSquare, 16 * wm, 16 * kb, lane);
#pragma unroll
                        for (int jp = 0; jp < NB / 2; ++jp) {
                            uint32_t x[NI][4];
#pragma unroll
                            for (int j = 0; j < NI; ++j) right_t<KP>(x[j], r + j * R::term, 16 * kb, wn * (KP / 2) + 16 * jp, lane);
                            products<NO, NI>(t[2 * jp], t[2 * jp + 1], a, x);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NB; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) to[nt][e] = fmaf(t[nt][e], c, to[nt][e]);
                };
                const auto rank_t = [&](Acc(&to)[NB], uint32_t l, uint32_t r, float c) {
                    Acc t[NB];
                    clear(t);
#pragma unroll
                    for (int kb = 0; kb < 4; ++kb) {
                        if (kb < wm) continue;
                        uint32_t a[NO][4];
#pragma unroll
                        for (int j = 0; j < NO; ++j) left_t<kChunk>(a[j], l + j * kSquare, 16 * kb, 16 * wm, lane);
#pragma unroll
                        for (int jp = 0; jp < NB / 2; ++jp) {
                            uint32_t x[NI][4];
#pragma unroll
                            for (int j = 0; j < NI; ++j) right_t<KP>(x[j], r + j * R::term, 16 * kb, wn * (KP / 2) + 16 * jp, lane);
                            products<NO, NI>(t[2 * jp], t[2 * jp + 1], a, x);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NB; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) to[nt][e] = fmaf(t[nt][e], c, to[nt][e]);
                };
                mp = inverse_of(mp), ma = inverse_of(ma) * ik;
                rank(aq, i_do, kimg, mp * ik);
                rank_t(ak, i_do, qimg, mp * iq);
                rank(ak, i_dr, kimg, ma);
                rank_t(ak, i_dr, kimg, ma);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NB; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = e ? r1 : r0, col = col0 + 8 * nt;
                if (row >= rows) continue;
                store_pair(dq + row * row_k, col, p.K, pair, aq[nt][2 * e], aq[nt][2 * e + 1]);
                store_pair(dk + row * row_k, col, p.K, pair, ak[nt][2 * e], ak[nt][2 * e + 1]);
            }
    }
}

// ------------------------------------------------------------------------------------------------
// One row of each of N sequences whose states lie in a pool. A CTA takes 32 channels of the values of one state, all of it in registers:
// S^T k and S^T q come from one reading of it, with o = scale (a S^T q + (k q) u), so the state is read once and written once. Bound by memory.
// ------------------------------------------------------------------------------------------------
constexpr int kStepWarps = 8;
struct DeltaStepParams {
    const void *q, *k, *v, *beta, *gate;
    int64_t q_sn, q_sh, k_sn, k_sh, v_sn, v_sh, beta_sn, gate_sn;
    int N, H, HK, K, V, S;
    float scale;
    float *pool;
    const int32_t *slots;
    void *o;
};
template <typename T, int VEC>
__global__ void __launch_bounds__(32 * kStepWarps) based_delta_step_kernel(DeltaStepParams p) {
    constexpr int kLanes = 32 / VEC, kRows = 32 / kLanes * kStepWarps, kEach = kMaxKeys / kRows;  // a row's lanes, rows of a pass, passes
    __shared__ float sk[kMaxKeys], sq[kMaxKeys], red[3][kStepWarps][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, head = blockIdx.y, hk = head / (p.H / p.HK);
    const int c = blockIdx.x * 32 + lane % kLanes * VEC, row0 = warp * (32 / kLanes) + lane / kLanes;
    griddep_wait();
    for (int n = blockIdx.z; n < p.N; n += gridDim.z) {
        const int slot = p.slots ? p.slots[n] : n;
        T *const o = static_cast<T *>(p.o) + (static_cast<int64_t>(n) * p.H + head) * p.V + c;
        if (slot < 0 || slot >= p.S) {  // an idle sequence
            if (row0 == 0 && c < p.V)
                for (int j = 0; j < VEC && c + j < p.V; ++j) o[j] = from_f32<T>(0.0f);
            continue;
        }
        float *const state = p.pool + (static_cast<int64_t>(slot) * p.H + head) * p.K * p.V + c;
        Pack<float, VEC> s[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row0 + i * kRows;
            if (row < p.K && c < p.V) s[i] = *reinterpret_cast<const Pack<float, VEC> *>(state + static_cast<int64_t>(row) * p.V);
        }
        __syncthreads();  // the sequence before
        if (tid < p.K) {
            sk[tid] = to_f32(static_cast<const T *>(p.k)[n * p.k_sn + hk * p.k_sh + tid]);
            sq[tid] = to_f32(static_cast<const T *>(p.q)[n * p.q_sn + hk * p.q_sh + tid]);
        }
        const float a = p.gate ? expf(to_f32(static_cast<const T *>(p.gate)[n * p.gate_sn + head])) : 1.0f;
        const float beta = to_f32(static_cast<const T *>(p.beta)[n * p.beta_sn + head]);
        __syncthreads();
        float x[VEC] = {}, y[VEC] = {}, kq = 0.0f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row0 + i * kRows;
            if (row < p.K && c < p.V) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    s[i].v[j] *= a;
                    x[j] = fmaf(s[i].v[j], sk[row], x[j]), y[j] = fmaf(s[i].v[j], sq[row], y[j]);
                }
            }
        }
        for (int i = lane; i < p.K; i += 32) kq = fmaf(sk[i], sq[i], kq);
#pragma unroll
        for (int d = 1; d < 32; d *= 2) kq += __shfl_xor_sync(0xffffffffu, kq, d);
#pragma unroll
        for (int d = kLanes; d < 32; d *= 2)
#pragma unroll
            for (int j = 0; j < VEC; ++j) x[j] += __shfl_xor_sync(0xffffffffu, x[j], d), y[j] += __shfl_xor_sync(0xffffffffu, y[j], d);
        if (lane < kLanes) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) red[0][warp][lane * VEC + j] = x[j], red[1][warp][lane * VEC + j] = y[j];
        }
        __syncthreads();
        if (tid < 32) {
            float sx = 0.0f, sy = 0.0f, u = 0.0f;
#pragma unroll
            for (int w = 0; w < kStepWarps; ++w) sx += red[0][w][tid], sy += red[1][w][tid];
            const int col = blockIdx.x * 32 + tid;
            if (col < p.V) {
                u = beta * (to_f32(static_cast<const T *>(p.v)[n * p.v_sn + head * p.v_sh + col]) - sx);
                static_cast<T *>(p.o)[(static_cast<int64_t>(n) * p.H + head) * p.V + col] = from_f32<T>(p.scale * fmaf(kq, u, sy));
            }
            red[2][0][tid] = u;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = red[2][0][lane % kLanes * VEC + j];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row0 + i * kRows;
            if (row < p.K && c < p.V) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) s[i].v[j] = fmaf(sk[row], x[j], s[i].v[j]);
                *reinterpret_cast<Pack<float, VEC> *>(state + static_cast<int64_t>(row) * p.V) = s[i];
            }
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Host
// ------------------------------------------------------------------------------------------------
constexpr int kMostGrid = 65535;

// The parts of a workspace, each on 256 bytes
struct DeltaSpace {
    size_t qk, g, dr, dstates, total;
};
inline int padded_keys(int K) { return K <= 64 ? 64 : 128; }
template <typename T, int KP>
DeltaSpace delta_space(int B, int T_, int H, int HK, int K, int V, bool bwd) {
    const size_t chunks = (static_cast<size_t>(T_) + kChunk - 1) / kChunk, up = 255;
    DeltaSpace s;
    s.qk = 0;
    s.g = (s.qk + chunks * B * HK * Rec<T, KP>::qk + up) & ~up;
    s.dr = (s.g + chunks * B * H * Rec<T, KP>::g(bwd) + up) & ~up;
    s.dstates = bwd ? (s.dr + static_cast<size_t>(B) * T_ * H * V * 4 + up) & ~up : s.dr;
    s.total = bwd ? (s.dstates + chunks * B * H * K * V * 4 + up) & ~up : s.dr;
    return s;
}
DeltaSpace delta_space(int B, int T, int H, int HK, int K, int V, int dtype, bool bwd) {
    const bool wide = padded_keys(K) == 128;
    // (the records of bfloat16 and float16 differ in the terms of the scores)
    if (dtype == BASED_F32) return wide ? delta_space<float, 128>(B, T, H, HK, K, V, bwd) : delta_space<float, 64>(B, T, H, HK, K, V, bwd);
    if (dtype == BASED_BF16)
        return wide ? delta_space<__nv_bfloat16, 128>(B, T, H, HK, K, V, bwd) : delta_space<__nv_bfloat16, 64>(B, T, H, HK, K, V, bwd);
    return wide ? delta_space<__half, 128>(B, T, H, HK, K, V, bwd) : delta_space<__half, 64>(B, T, H, HK, K, V, bwd);
}

int check_delta_sizes(int64_t B, int64_t T, int H, int HK, int K, int V) {
    if (B < 1 || T < 1 || H < 1 || HK < 1 || K < 1 || V < 1 || H % HK != 0 || K > kMaxKeys || V > kDeltaMaxV || H > kMostGrid || T > (1 << 30) ||
        B > (1 << 30) / T || B * T > (static_cast<int64_t>(1) << 40) / (static_cast<int64_t>(H) * (K > V ? K : V)))
        return BASED_ERR_BAD_SIZE;
    return BASED_OK;
}

template <typename T, int KP>
int launch_delta(DeltaParams &p, bool bwd, int sms, cudaStream_t st) {
    using Sm = SeqSmem<T, KP>;
    const int slices = (p.V + kSlice - 1) / kSlice;
    const unsigned z = p.B < kMostGrid ? p.B : kMostGrid;
    void (*const prep)(DeltaParams) = bwd ? based_delta_prep_kernel<T, KP, true> : based_delta_prep_kernel<T, KP, false>;
    OPS_CUDA(allow(prep, PrepSmem<T, KP>::bytes));
    OPS_CUDA(launch_op(prep, dim3(p.chunks, p.HK, z), 32 * kPrepWarps, PrepSmem<T, KP>::bytes, st, p));
    // As many warps to a CTA (they share its records) as leave a CTA for every SM
    static_assert(Sm::bytes(true, Sm::warps) <= 227 * 1024 && GradSmem<T, KP>::bytes <= 227 * 1024, "shared memory of a CTA");
    int warps = Sm::warps;
    while (warps > 1 && (warps / 2 >= slices || static_cast<int64_t>(p.B) * p.H * ((slices + warps - 1) / warps) < sms)) warps /= 2;
    void (*const seq)(DeltaParams) = bwd ? based_delta_bwd_kernel<T, KP> : based_delta_fwd_kernel<T, KP>;
    OPS_CUDA(allow(seq, Sm::bytes(bwd, Sm::warps)));
    OPS_CUDA(launch_op(seq, dim3((slices + warps - 1) / warps, p.H, z), 32 * warps, Sm::bytes(bwd, warps), st, p));
    if (bwd) {
        void (*const grad)(DeltaParams) = based_delta_grad_kernel<T, KP>;
        OPS_CUDA(allow(grad, GradSmem<T, KP>::bytes));
        OPS_CUDA(launch_op(grad, dim3(p.chunks, p.HK, z), 32 * kGradWarps, GradSmem<T, KP>::bytes, st, p));
    }
    return BASED_OK;
}
template <typename T>
int launch_delta(DeltaParams &p, bool bwd, int sms, cudaStream_t st) {
    return padded_keys(p.K) == 64 ? launch_delta<T, 64>(p, bwd, sms, st) : launch_delta<T, 128>(p, bwd, sms, st);
}

struct Region {
    Span s;
    bool out;
};
// Whether an output overlaps anything else
template <int N>
bool clash(const Region (&r)[N]) {
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < i; ++j)
            if ((r[i].out || r[j].out) && overlap(r[i].s, r[j].s)) return true;
    return false;
}

int run_delta(DeltaParams &p, int dtype, bool bwd, void *workspace, size_t ws_bytes, based_stream_t stream) {
    if (!p.q || !p.k || !p.v || !p.beta || !p.out) return BASED_ERR_NULL_POINTER;
    if (bwd && (!p.dout || !p.states || !p.errors || !p.dq || !p.dk || !p.dbeta || !p.gate != !p.dgate)) return BASED_ERR_NULL_POINTER;
    if (!bwd && !p.states != !p.errors) return BASED_ERR_NULL_POINTER;
    if (!type_ok(dtype)) return BASED_ERR_UNSUPPORTED_TYPE;
    if (!(p.scale == p.scale)) return BASED_ERR_BAD_ARGUMENT;
    const int B = p.B, T = p.T, H = p.H, HK = p.HK, K = p.K, V = p.V;
    if (const int rc = check_delta_sizes(B, T, H, HK, K, V)) return rc;
    p.chunks = (T + kChunk - 1) / kChunk;
    const int64_t strides[] = {p.q_sb, p.q_st, p.q_sh, p.k_sb, p.k_st, p.k_sh, p.v_sb, p.v_st, p.v_sh, p.do_sb, p.do_st, p.do_sh,
                               p.beta_sb, p.beta_st, p.gate_sb, p.gate_st};
    int64_t bits = 0;
    for (const int64_t s : strides) {
        if (s < 0) return BASED_ERR_BAD_STRIDE;
        bits |= s;
    }
    const size_t es = elem_size(dtype);
    const void *const typed[] = {p.q, p.k, p.v, p.beta, p.gate, p.dout, p.out, p.dq, p.dk, p.dbeta, p.dgate};
    for (const void *t : typed)
        if (!aligned(t, es)) return BASED_ERR_MISALIGNED;
    if (!aligned(p.lengths, 4) || !aligned(p.state, 4) || !aligned(p.final_state, 4) || !aligned(p.states, 16) || !aligned(p.errors, 16) ||
        !aligned(p.dq, 2 * es) || !aligned(p.dk, 2 * es))
        return BASED_ERR_MISALIGNED;
    const DeltaSpace space = delta_space(B, T, H, HK, K, V, dtype, bwd);
    if (!workspace || ws_bytes < space.total || !aligned(workspace, 16)) return BASED_ERR_WORKSPACE;
    const auto three = [&](const void *t, int64_t sb, int64_t s1, int64_t sh, int h, int c) {
        return span(t, (B - 1) * sb + (T - 1) * s1 + (h - 1) * sh + c - 1, es);
    };
    const int64_t bth = static_cast<int64_t>(B) * T * H, states = static_cast<int64_t>(B) * H * K * V;
    const Region regions[] = {
        {three(p.q, p.q_sb, p.q_st, p.q_sh, HK, K), false}, {three(p.k, p.k_sb, p.k_st, p.k_sh, HK, K), false},
        {three(p.v, p.v_sb, p.v_st, p.v_sh, H, V), false}, {three(p.dout, p.do_sb, p.do_st, p.do_sh, H, V), false},
        {three(p.beta, p.beta_sb, p.beta_st, 1, H, 1), false}, {three(p.gate, p.gate_sb, p.gate_st, 1, H, 1), false},
        {span(p.lengths, B - 1, 4), false},
        {p.state == p.final_state ? Span{0, 0} : span(p.state, states - 1, 4), false},  // may be replaced in place
        {span(p.states, states * p.chunks - 1, 4), !bwd}, {span(p.errors, bth * V - 1, 4), !bwd},
        {span(p.out, bth * V - 1, es), true}, {span(p.final_state, states - 1, 4), true},
        {span(p.dq, static_cast<int64_t>(B) * T * HK * K - 1, es), true}, {span(p.dk, static_cast<int64_t>(B) * T * HK * K - 1, es), true},
        {span(p.dbeta, bth - 1, es), true}, {span(p.dgate, bth - 1, es), true}, {span(workspace, static_cast<int64_t>(space.total) - 1, 1), true}};
    if (clash(regions)) return BASED_ERR_ALIASING;
    int sms;
    if (const int rc = host_device(&sms)) return rc;
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    p.qk_rec = ws + space.qk, p.g_rec = ws + space.g;
    if (bwd) p.dr = reinterpret_cast<float *>(ws + space.dr), p.dstates = reinterpret_cast<float *>(ws + space.dstates);
    const int64_t e = static_cast<int64_t>(es);
    const auto words = [&](const void *t, int64_t sb, int64_t s1, int64_t sh, int c) {
        return (sb | s1 | sh | c) * e % 16 == 0 && aligned(t, 16);
    };
    p.qk_vec = words(p.q, p.q_sb, p.q_st, p.q_sh, K) && words(p.k, p.k_sb, p.k_st, p.k_sh, K);
    p.v_vec = words(p.v, p.v_sb, p.v_st, p.v_sh, V), p.o_vec = words(p.out, 0, 0, 0, V);
    p.do_vec = p.dout && words(p.dout, p.do_sb, p.do_st, p.do_sh, V);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == BASED_F32) return launch_delta<float>(p, bwd, sms, st);
    if (dtype == BASED_BF16) return launch_delta<__nv_bfloat16>(p, bwd, sms, st);
    return launch_delta<__half>(p, bwd, sms, st);
}

// The default scale is K^-1/2.
inline float delta_scale(float scale, int K) { return scale > 0.0f || K < 1 ? scale : 1.0f / sqrtf(static_cast<float>(K)); }

template <typename T>
int launch_delta_step(const DeltaStepParams &p, cudaStream_t st) {
    const bool quad = p.V % 4 == 0 && aligned(p.pool, 16);
    const dim3 grid((p.V + 31) / 32, p.H, p.N < kMostGrid ? p.N : kMostGrid);
    OPS_CUDA(launch_op(quad ? based_delta_step_kernel<T, 4> : based_delta_step_kernel<T, 1>, grid, 32 * kStepWarps, 0, st, p));
    return BASED_OK;
}

}  // namespace
}  // namespace based

extern "C" {

int based_delta_fwd(const void *q, int64_t q_sb, int64_t q_st, int64_t q_sh, const void *k, int64_t k_sb, int64_t k_st, int64_t k_sh, const void *v,
                    int64_t v_sb, int64_t v_st, int64_t v_sh, const void *beta, int64_t beta_sb, int64_t beta_st, const void *gate,
                    int64_t gate_sb, int64_t gate_st, int B, int T, int H, int HK, int K, int V, int dtype, float scale, const float *state,
                    const int32_t *lengths, void *o, float *final_state, float *states, float *errors, void *workspace, size_t ws_bytes,
                    based_stream_t stream) {
    based::DeltaParams p = {};
    p.q = q, p.q_sb = q_sb, p.q_st = q_st, p.q_sh = q_sh, p.k = k, p.k_sb = k_sb, p.k_st = k_st, p.k_sh = k_sh;
    p.v = v, p.v_sb = v_sb, p.v_st = v_st, p.v_sh = v_sh, p.beta = beta, p.beta_sb = beta_sb, p.beta_st = beta_st;
    p.gate = gate, p.gate_sb = gate_sb, p.gate_st = gate_st;
    p.B = B, p.T = T, p.H = H, p.HK = HK, p.K = K, p.V = V, p.scale = based::delta_scale(scale, K);
    p.state = state, p.lengths = lengths, p.out = o, p.final_state = final_state, p.states = states, p.errors = errors;
    return based::run_delta(p, dtype, false, workspace, ws_bytes, stream);
}

int based_delta_bwd(const void *q, int64_t q_sb, int64_t q_st, int64_t q_sh, const void *k, int64_t k_sb, int64_t k_st, int64_t k_sh, const void *v,
                    int64_t v_sb, int64_t v_st, int64_t v_sh, const void *beta, int64_t beta_sb, int64_t beta_st, const void *gate,
                    int64_t gate_sb, int64_t gate_st, const void *dout, int64_t do_sb, int64_t do_st, int64_t do_sh, const float *states,
                    const float *errors, int B, int T, int H, int HK, int K, int V, int dtype, float scale, const float *dfinal,
                    const int32_t *lengths, void *dq, void *dk, void *dv, void *dbeta, void *dgate, float *dstate, void *workspace,
                    size_t ws_bytes, based_stream_t stream) {
    based::DeltaParams p = {};
    p.q = q, p.q_sb = q_sb, p.q_st = q_st, p.q_sh = q_sh, p.k = k, p.k_sb = k_sb, p.k_st = k_st, p.k_sh = k_sh;
    p.v = v, p.v_sb = v_sb, p.v_st = v_st, p.v_sh = v_sh, p.beta = beta, p.beta_sb = beta_sb, p.beta_st = beta_st;
    p.gate = gate, p.gate_sb = gate_sb, p.gate_st = gate_st, p.dout = dout, p.do_sb = do_sb, p.do_st = do_st, p.do_sh = do_sh;
    p.B = B, p.T = T, p.H = H, p.HK = HK, p.K = K, p.V = V, p.scale = based::delta_scale(scale, K);
    p.state = dfinal, p.lengths = lengths, p.out = dv, p.dq = dq, p.dk = dk, p.dbeta = dbeta, p.dgate = dgate, p.final_state = dstate;
    p.states = const_cast<float *>(states), p.errors = const_cast<float *>(errors);
    return based::run_delta(p, dtype, true, workspace, ws_bytes, stream);
}

size_t based_delta_workspace_size(int B, int T, int H, int HK, int K, int V, int dtype, int backward) {
    if (based::check_delta_sizes(B, T, H, HK, K, V) != BASED_OK || !based::type_ok(dtype)) return 0;
    return based::delta_space(B, T, H, HK, K, V, dtype, backward != 0).total;
}

int based_delta_step(const void *q, int64_t q_sn, int64_t q_sh, const void *k, int64_t k_sn, int64_t k_sh, const void *v, int64_t v_sn, int64_t v_sh,
                     const void *beta, int64_t beta_sn, const void *gate, int64_t gate_sn, int N, int H, int HK, int K, int V, int S, int dtype,
                     float scale, float *pool, const int32_t *slots, void *o, based_stream_t stream) {
    using namespace based;
    if (!q || !k || !v || !beta || !pool || !o) return BASED_ERR_NULL_POINTER;
    if (!type_ok(dtype)) return BASED_ERR_UNSUPPORTED_TYPE;
    if (!(scale == scale)) return BASED_ERR_BAD_ARGUMENT;
    if (check_delta_sizes(N, 1, H, HK, K, V) != BASED_OK || S < 1 || (!slots && S < N)) return BASED_ERR_BAD_SIZE;
    if (q_sn < 0 || q_sh < 0 || k_sn < 0 || k_sh < 0 || v_sn < 0 || v_sh < 0 || beta_sn < 0 || gate_sn < 0) return BASED_ERR_BAD_STRIDE;
    const size_t es = elem_size(dtype);
    const void *const typed[] = {q, k, v, beta, gate, o};
    for (const void *t : typed)
        if (!aligned(t, es)) return BASED_ERR_MISALIGNED;
    if (!aligned(pool, 4) || !aligned(slots, 4)) return BASED_ERR_MISALIGNED;
    const Region regions[] = {{span(q, (N - 1) * q_sn + (HK - 1) * q_sh + K - 1, es), false},
                              {span(k, (N - 1) * k_sn + (HK - 1) * k_sh + K - 1, es), false},
                              {span(v, (N - 1) * v_sn + (H - 1) * v_sh + V - 1, es), false},
                              {span(beta, (N - 1) * beta_sn + H - 1, es), false}, {span(gate, (N - 1) * gate_sn + H - 1, es), false},
                              {span(slots, N - 1, 4), false}, {span(pool, static_cast<int64_t>(S) * H * K * V - 1, 4), true},
                              {span(o, static_cast<int64_t>(N) * H * V - 1, es), true}};
    if (clash(regions)) return BASED_ERR_ALIASING;
    int sms;
    if (const int rc = host_device(&sms)) return rc;
    const DeltaStepParams p = {q, k, v, beta, gate, q_sn, q_sh, k_sn, k_sh, v_sn, v_sh, beta_sn, gate_sn, N, H, HK, K, V, S,
                               delta_scale(scale, K), pool, slots, o};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == BASED_F32) return launch_delta_step<float>(p, st);
    if (dtype == BASED_BF16) return launch_delta_step<__nv_bfloat16>(p, st);
    return launch_delta_step<__half>(p, st);
}

}  // extern "C"
