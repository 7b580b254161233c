// based_delta.cu: the gated delta rule (declared in include/based_ops.h).
//
//     S_t = a_t S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - a_t S_{t-1}^T k_t),   o_t = scale S_t^T q_t
//
// A chunk of 64 rows takes a few matrix products instead of 64 steps. With b_i the sum of log decays up to row i of
// the chunk, D_ij = exp(b_i - b_j) for j <= i, S0 the state in front, grow_i = exp(b_i) and rest_i = exp(b_last - b_i):
//     X = V - grow K S0,   E = (1 + L)^-1 X with L_ij = D_ij (k_i k_j) beta_j below the diagonal,   U = beta E,
//     O = scale grow Q S0 + P U with P_ij = scale D_ij (q_i k_j),   S = grow_last S0 + (rest K)^T U.
// The inverse's diagonal of ones is left to the float32 registers that X lies in: its product is only what other rows add.
// based_delta_prep_kernel has all that does not depend on the state (the inverse and P), for all chunks at once;
// based_delta_fwd_kernel runs through the chunks. Backward, with G the gradient of the state behind the chunk and
// A_ij = beta_i D_ij (k_i k_j) below the diagonal:
//     dU = P^T dO + rest K G,   dR = (1 + A)^-T dU,   dV = beta dR,
//     G' = grow_last G + scale (grow Q)^T dO - (beta grow K)^T dR
// runs through the chunks from the last (based_delta_bwd_kernel), and what is left is again for all chunks at once
// (based_delta_grad_kernel, where its formulas are).
#include <cmath>

#include "delta_common.cuh"

namespace based {
namespace {

// ------------------------------------------------------------------------------------------------
// What does not depend on the state
// ------------------------------------------------------------------------------------------------
constexpr int kPrepWarps = 8;
constexpr int kLd = 68;  // floats in a row of the square matrices in shared memory

template <typename T, int KP>
struct PrepSmem {
    static constexpr int images = Rec<T, KP>::qk, work = (2 * kChunk * kLd + 32 * 36) * 4;
    static constexpr int shared = images > work ? images : work;  // the images, then the inverse's work in their place
    static constexpr int bytes = shared + (9 * kChunk + 16) * 4;
};

// Rows of q or k into their images, in shared memory and in the record; returns the scale's inverse.
__host__ __device__ constexpr int prep_words(int KP) { return kChunk * KP / 8 / (32 * kPrepWarps); }  // of a thread
template <typename T, int KP>
__device__ __forceinline__ void read_rows(Raw<T> (&raw)[prep_words(KP)], const T *src, int64_t stride, int rows, int K, bool words) {
    constexpr int kWords = KP / 8, kStep = 32 * kPrepWarps / kWords;
    const int word = threadIdx.x % kWords, row0 = threadIdx.x / kWords;
#pragma unroll
    for (int i = 0; i < prep_words(KP); ++i) {
        const int row = row0 + i * kStep;
        raw[i].load(src + row * stride + word * 8, row < rows ? K - word * 8 : 0, words);
    }
}
template <typename T, int KP>
__device__ __forceinline__ float make_image(const Raw<T> (&raw)[prep_words(KP)], uint8_t *img, uint8_t *rec, float *red) {
    constexpr int kWords = KP / 8, kStep = 32 * kPrepWarps / kWords;
    const int word = threadIdx.x % kWords, row0 = threadIdx.x / kWords;
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < prep_words(KP); ++i) {
        float x[8];
        raw[i].get(x);
        most = most8(most, x);
    }
    const float s = scale_for(cta_most<kPrepWarps>(most, red));
#pragma unroll
    for (int i = 0; i < prep_words(KP); ++i) {
        float x[8];
        raw[i].get(x);
        uint4 w[Terms<T>::in];
        words_of<Terms<T>::in>(w, x, s);
        const uint32_t at = word_at<KP>(row0 + i * kStep, word);
#pragma unroll
        for (int j = 0; j < Terms<T>::in; ++j) {
            *reinterpret_cast<uint4 *>(img + j * Rec<T, KP>::term + at) = w[j];
            *reinterpret_cast<uint4 *>(rec + j * Rec<T, KP>::term + at) = w[j];
        }
    }
    return inverse_of(s);
}

// C = sign A B for N x N blocks in shared memory, by `count` threads of which this is number i. A thread holds a column of B and takes rows of A that
// its neighbours take too: a word of A serves a warp at once, where four results to a thread took five times the wavefronts.
template <int N>
__device__ __forceinline__ void small_product(float *c, int ldc, const float *a, int lda, const float *b, int ldb, float sign, int i, int count) {
    const int col = i % N;
    float x[N];
#pragma unroll
    for (int m = 0; m < N; ++m) x[m] = b[m * ldb + col];
    for (int row = i / N; row < N; row += count / N) {
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int m = 0; m < N; m += 4) {
            const float4 y = *reinterpret_cast<const float4 *>(a + row * lda + m);
            s[0] = fmaf(y.x, x[m], s[0]), s[1] = fmaf(y.y, x[m + 1], s[1]), s[0] = fmaf(y.z, x[m + 2], s[0]), s[1] = fmaf(y.w, x[m + 3], s[1]);
        }
        c[row * ldc + col] = sign * (s[0] + s[1]);
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
            for (int l = 0; l < i; l += 4) {
                const float4 y = *reinterpret_cast<const float4 *>(m + (block + i) * kLd + block + l);
                s = fmaf(y.x, x[l], s);
                if (l + 1 < i) s = fmaf(y.y, x[l + 1], s);
                if (l + 2 < i) s = fmaf(y.z, x[l + 2], s);
                if (l + 3 < i) s = fmaf(y.w, x[l + 3], s);
            }
            x[i] = i == j ? 1.0f : i < j ? 0.0f : -s;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) h[(block + i) * kLd + tid] = x[i];
    }
    __syncthreads();
    {
        const int pair = tid / 128, a = 32 * pair, b = a + 16;
        float *const t = w + pair * 16 * 36;
        small_product<16>(t, 36, m + b * kLd + a, kLd, h + a * kLd + a, kLd, 1.0f, tid % 128, 128);
        __syncthreads();
        small_product<16>(h + b * kLd + a, kLd, h + b * kLd + b, kLd, t, 36, -1.0f, tid % 128, 128);
    }
    __syncthreads();
    small_product<32>(w, 36, m + 32 * kLd, kLd, h, kLd, 1.0f, tid, 32 * kPrepWarps);
    __syncthreads();
    small_product<32>(h + 32 * kLd, kLd, h + 32 * kLd + 32, kLd, w, 36, -1.0f, tid, 32 * kPrepWarps);
    __syncthreads();
}

// A number as a float and what it is off by
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two plus(const Two &a, const Two &b) {
    const float s = a.hi + b.hi, v = s - a.hi, e = (a.hi - (s - v)) + (b.hi - v) + (a.lo + b.lo), h = s + e;
    return {h, e - (h - s)};
}

// One chunk of one key head, and all value heads that share it.
template <typename T, int KP, bool BWD>
__global__ void __launch_bounds__(32 * kPrepWarps, sizeof(T) == 2 ? 4 : 2) based_delta_prep_kernel(DeltaParams p) {
    using R = Rec<T, KP>;
    using Sm = PrepSmem<T, KP>;
    constexpr int NI = Terms<T>::in, NP = R::scores(BWD);
    extern __shared__ __align__(128) uint8_t smem[];
    float *const m = reinterpret_cast<float *>(smem), *const h = m + kChunk * kLd, *const w = h + kChunk * kLd;
    float *const bhi = reinterpret_cast<float *>(smem + Sm::shared), *const blo = bhi + kChunk, *const beta = blo + kChunk, *const till = beta + kChunk,
                *const over = till + kChunk, *const since = over + kChunk, *const red = since + 4 * kChunk;
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
        const auto record = [&](int head) { return p.g_rec + ((static_cast<int64_t>(b) * p.H + head) * p.chunks + n) * R::g(BWD); };
        const auto scan = [&](int head) {
            if (warp != 0) return;
            float *const f = reinterpret_cast<float *>(record(head) + (2 + NP) * kSquare);
            // Sums of log decays as two floats each (64-bit floats are slow here): differences of neighbours then have float32's relative
            // accuracy however much has decayed before. -1e5 stands for anything below it, -inf among it: its decay is 0.
            Two x[2];
            float be[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                float v = 0.0f;
                be[e] = 0.0f;
                if (i < rows) {
                    if (p.gate) v = to_f32(static_cast<const T *>(p.gate)[b * p.gate_sb + (t0 + i) * p.gate_st + head]);
                    be[e] = to_f32(static_cast<const T *>(p.beta)[b * p.beta_sb + (t0 + i) * p.beta_st + head]);
                }
                x[e] = {v < -1e5f ? -1e5f : v, 0.0f};
            }
            x[1] = plus(x[0], x[1]);
            Two sum = x[1];
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const Two o = {__shfl_up_sync(0xffffffffu, sum.hi, d), __shfl_up_sync(0xffffffffu, sum.lo, d)};
                if (lane >= d) sum = plus(o, sum);
            }
            Two before = {__shfl_up_sync(0xffffffffu, sum.hi, 1), __shfl_up_sync(0xffffffffu, sum.lo, 1)};
            if (lane == 0) before = {0.0f, 0.0f};
            const Two last = {__shfl_sync(0xffffffffu, sum.hi, 31), __shfl_sync(0xffffffffu, sum.lo, 31)};
            // the sum up to the last of each 16 rows
            const Two end = {__shfl_sync(0xffffffffu, sum.hi, lane | 7), __shfl_sync(0xffffffffu, sum.lo, lane | 7)};
            float most = 0.0f, grow_most = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                const Two v = plus(before, x[e]);
                const float grow = expf(v.hi + v.lo), rest = expf((last.hi - v.hi) + (last.lo - v.lo)), y = be[e];
                const float step = BWD ? 1.0f : step_of(y), bf = BWD ? y * grow : y * inverse_of(step) * rest;
                bhi[i] = v.hi, blo[i] = v.lo, beta[i] = y, over[i] = inverse_of(step), till[i] = expf((end.hi - v.hi) + (end.lo - v.lo));
                f[F_GROW + i] = grow, f[F_REST + i] = BWD ? rest : grow * step, f[F_BETA + i] = BWD ? y : step;
                f[F_BHI + i] = v.hi, f[F_BLO + i] = v.lo, f[F_BF + i] = bf;
                most = fmaxf(most, fabsf(bf)), grow_most = fmaxf(grow_most, grow);
            }
#pragma unroll
            for (int d = 1; d < 8; d *= 2)
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d)), grow_most = fmaxf(grow_most, __shfl_xor_sync(0xffffffffu, grow_most, d));
            if (lane % 8 == 0) f[F_BFMOST + lane / 8] = most, f[F_GROWMOST + lane / 8] = grow_most;
            if (lane == 0) f[F_WHOLE] = expf(last.hi + last.lo);
        };
        __syncthreads();  // the batch entry before
        float ik, iq;
        if constexpr (sizeof(T) == 2) {  // (registers for both only in 16 bits)
            Raw<T> rk[prep_words(KP)], rq[prep_words(KP)];
            read_rows<T, KP>(rk, ks, p.k_st, rows, p.K, p.qk_vec);
            read_rows<T, KP>(rq, qs, p.q_st, rows, p.K, p.qk_vec);
            scan(hk * group);  // while the rows are on their way
            ik = make_image<T, KP>(rk, smem, rec, red);
            iq = make_image<T, KP>(rq, smem + R::img, rec + R::img, red);
        } else {
            Raw<T> raw[prep_words(KP)];
            read_rows<T, KP>(raw, ks, p.k_st, rows, p.K, p.qk_vec);
            scan(hk * group);
            ik = make_image<T, KP>(raw, smem, rec, red);
            read_rows<T, KP>(raw, qs, p.q_st, rows, p.K, p.qk_vec);
            iq = make_image<T, KP>(raw, smem + R::img, rec + R::img, red);
        }
        __syncthreads();
        // the products of keys with keys and queries: a warp has 16 rows and 32 columns, up to the diagonal
        const int wm = warp & 3, wn = warp >> 2;
        Acc sk[4], sq[4];
        clear(sk), clear(sq);
        {
            const uint32_t kimg = smem_u32(smem), qimg = kimg + R::img;
#pragma unroll
            for (int kk = 0; kk < KP / 16; ++kk) {
                if (2 * wn > wm) continue;
                uint32_t a[NI][4], c[NI][4];
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    left<KP>(a[j], kimg + j * R::term, 16 * wm, 16 * kk, lane);
                    left<KP>(c[j], qimg + j * R::term, 16 * wm, 16 * kk, lane);
                }
#pragma unroll
                for (int np = 0; np < 2; ++np) {
                    if (2 * wn + np > wm) continue;
                    uint32_t x[NI][4];
#pragma unroll
                    for (int j = 0; j < NI; ++j) right<KP>(x[j], kimg + j * R::term, 32 * wn + 16 * np, 16 * kk, lane);
                    products<T, NI, NI>(sk[2 * np], sk[2 * np + 1], a, x);
                    products<T, NI, NI>(sq[2 * np], sq[2 * np + 1], c, x);
                }
            }
        }
        const float fk = ik * ik, fq = iq * ik * p.scale;
        for (int hh = 0; hh < group; ++hh) {
            const int head = hk * group + hh;
            uint8_t *const g = record(head);
            float *const f = reinterpret_cast<float *>(g + (2 + NP) * kSquare);
            if (hh) scan(head);
            for (int i = tid; i < kChunk * kLd / 4; i += 32 * kPrepWarps)
                if (hh) reinterpret_cast<float4 *>(h)[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            __syncthreads();  // the sums, and the images are done with
            if (!hh)
                for (int i = tid; i < kChunk * kLd / 4; i += 32 * kPrepWarps) reinterpret_cast<float4 *>(h)[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            {  // decays since the last of each 16 rows
                const int i = tid & 63, end = 16 * (tid >> 6) + 15;
                since[tid] = expf((bhi[i] - bhi[end]) + (blo[i] - blo[end]));
            }
            __syncthreads();
            Acc pv[4];
            float most = 0.0f;
            {
                const int r0 = 16 * wm + (lane >> 2), c0 = 32 * wn + 2 * (lane & 3);
                const float hi[2] = {bhi[r0], bhi[r0 + 8]}, lo[2] = {blo[r0], blo[r0 + 8]}, bi[2] = {beta[r0], beta[r0 + 8]};
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const int block = 2 * wn + nt / 2, c = c0 + 8 * nt;
                    if (block > wm) {  // above the diagonal
#pragma unroll
                        for (int e = 0; e < 4; ++e) pv[nt][e] = 0.0f;
                        continue;
                    }
                    const float2 jb = *reinterpret_cast<const float2 *>(beta + c), jo = *reinterpret_cast<const float2 *>(over + c);
                    float d[4];
                    if (block < wm) {  // D_ij by the last row of j's 16: two factors
                        const float2 t = *reinterpret_cast<const float2 *>(till + c);
                        const float s0 = since[64 * block + r0], s1 = since[64 * block + r0 + 8];
                        d[0] = s0 * t.x, d[1] = s0 * t.y, d[2] = s1 * t.x, d[3] = s1 * t.y;
                    } else {
                        const float2 jh = *reinterpret_cast<const float2 *>(bhi + c), jl = *reinterpret_cast<const float2 *>(blo + c);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = (hi[e / 2] - (e % 2 ? jh.y : jh.x)) + (lo[e / 2] - (e % 2 ? jl.y : jl.x));
                            d[e] = c + e % 2 <= r0 + 8 * (e / 2) ? expf(x) : 0.0f;
                        }
                    }
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = r0 + 8 * (e / 2), j = c + e % 2;
                        const float bj = e % 2 ? jb.y : jb.x;
                        pv[nt][e] = j <= i ? d[e] * (sq[nt][e] * fq) * (BWD ? 1.0f : bj * (e % 2 ? jo.y : jo.x)) : 0.0f;
                        y[e] = j < i ? d[e] * (sk[nt][e] * fk) * (BWD ? bi[e / 2] : bj) : 0.0f;
                        most = fmaxf(most, fabsf(pv[nt][e]));
                    }
                    float *const to = m + r0 * kLd + c;
                    *reinterpret_cast<float2 *>(to) = make_float2(y[0], y[1]);
                    *reinterpret_cast<float2 *>(to + 8 * kLd) = make_float2(y[2], y[3]);
                }
            }
            const float sp = scale_for(cta_most<kPrepWarps>(most, red));  // with a barrier
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t x[NP];
                    terms<NP>(pv[nt][2 * e] * sp, pv[nt][2 * e + 1] * sp, x);
                    const uint32_t at = word_at<kChunk>(16 * wm + (lane >> 2) + 8 * e, 4 * wn + nt) + 4 * (lane & 3);
#pragma unroll
                    for (int j = 0; j < NP; ++j) *reinterpret_cast<uint32_t *>(g + (2 + j) * kSquare + at) = x[j];
                }
            invert(h, m, w);
            float x[2][8];
            most = 0.0f;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float4 *const from = reinterpret_cast<const float4 *>(h + (tid / 8 + 32 * r) * kLd + tid % 8 * 8);
                const float4 u = from[0], v = from[1];
                x[r][0] = u.x, x[r][1] = u.y, x[r][2] = u.z, x[r][3] = u.w, x[r][4] = v.x, x[r][5] = v.y, x[r][6] = v.z, x[r][7] = v.w;
                const float step = inverse_of(over[tid / 8 + 32 * r]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = tid % 8 * 8 + e;
                    x[r][e] = j < tid / 8 + 32 * r ? x[r][e] * (BWD ? 1.0f : over[j] * step) : 0.0f;
                }
                most = most8(most, x[r]);
            }
            const float sh = scale_for(cta_most<kPrepWarps>(most, red));
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                uint4 z[2];
                words_of<2>(z, x[r], sh);
                const uint32_t at = word_at<kChunk>(tid / 8 + 32 * r, tid % 8);
                *reinterpret_cast<uint4 *>(g + at) = z[0], *reinterpret_cast<uint4 *>(g + kSquare + at) = z[1];
            }
            if (tid == 0) f[F_INV] = inverse_of(sh), f[F_P] = inverse_of(sp), f[F_K] = ik, f[F_Q] = iq;
        }
    }
}

// ------------------------------------------------------------------------------------------------
// Through the chunks. Four warps own 16 channels of the values, a slice. The state's transpose lies in their accumulators, a quarter of the keys'
// channels each, so what a state's product needs of the state is never stored in float32 and read back; a chunk's rows are shared out too, 16 to each
// warp. Three times a chunk the warps hand one another left operands: the state's, X's and E's (backward: the gradient's, dU's and dR's).
// A chunk's records in shared memory serve all slices of a CTA.
// ------------------------------------------------------------------------------------------------
constexpr int kQuad = 128;  // threads of a slice

template <typename T, int KP>
struct SeqSmem {
    static constexpr int row = sizeof(T) == 2 ? 32 : 80;  // bytes of a row of 16 values: 32-bit ones lie apart so that four rows' banks differ
    static constexpr int tile = 16 * row;                 // of a warp: its rows of the values
    __host__ __device__ static constexpr int stage(bool bwd) { return Rec<T, KP>::qk + Rec<T, KP>::g(bwd); }
    // left operands, 512 bytes a term of a 16 x 16 block: the state's; E's or dO's; what is added to the state (backward: two); X's or dU's
    // (backward in the place of the state's, which all warps are done with by then)
    static constexpr int state = 0, e = state + KP / 16 * 1024, e_block = (Terms<T>::in > Terms<T>::out ? Terms<T>::in : Terms<T>::out) * 512, u = e + 4 * e_block,
                         w = u + 4096;
    __host__ __device__ static constexpr int x(bool bwd) { return bwd ? state : w; }
    static constexpr int scales = w + 4096, slice = scales + 128 + 8 * tile;
    static constexpr int bytes(bool bwd, int slices) { return 2 * stage(bwd) + slices * slice + 32; }
    // Slices of a CTA, at most: 512 threads, and what shared memory holds
    static constexpr int most(bool bwd) { return bytes(bwd, 4) <= 227 * 1024 ? 4 : bytes(bwd, 3) <= 227 * 1024 ? 3 : bytes(bwd, 2) <= 227 * 1024 ? 2 : 1; }
};

// A warp's 16 rows by 16 channels of v, dout or an output: where its words lie
template <typename T>
__device__ __forceinline__ uint32_t tile_word(int row, int word) {
    if constexpr (sizeof(T) == 2) return row * 32 + ((word ^ (row >> 2 & 1)) << 4);
    return row * 80 + (word << 4);
}
// Rows [0, rows) of the channels [0, cols) at src; zeros elsewhere
template <typename T>
__device__ __forceinline__ void load_tile(uint8_t *tile, const T *src, int64_t stride, int rows, int cols, bool words, int lane) {
    constexpr int kWords = sizeof(T), kEl = 16 / sizeof(T);  // two words of eight, or four of four elements a row
    if (words) {
#pragma unroll
        for (int i = 0; i < kWords / 2; ++i) {
            const int row = (lane + 32 * i) / kWords, word = (lane + 32 * i) % kWords;
            const bool there = row < rows && word * kEl < cols;
            copy16(smem_u32(tile) + tile_word<T>(row, word), there ? src + row * stride + word * kEl : src, there ? 16 : 0);
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = (lane >> 4) + 2 * i, c = lane & 15;
            const bool there = row < rows && c < cols;
            copy4(smem_u32(tile) + row * 80 + c * 4, there ? src + row * stride + c : src, there ? 4 : 0);
        }
    } else {
        T x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = (lane >> 4) + 2 * i, c = lane & 15;
            x[i] = from_f32<T>(0.0f);
            if (row < rows && c < cols) x[i] = src[row * stride + c];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = (lane >> 4) + 2 * i, c = lane & 15;
            *reinterpret_cast<T *>(tile + tile_word<T>(row, c / kEl) + c % kEl * sizeof(T)) = x[i];
        }
    }
}
// The tile's transpose as two accumulator blocks: rows are channels, columns the warp's 16 rows
template <typename T>
__device__ __forceinline__ void read_tile(Acc (&x)[2], const uint8_t *tile, int lane) {
    if constexpr (sizeof(T) == 2) {
        uint32_t r[4];
        ldsm_t(r, smem_u32(tile) + tile_word<T>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Vec<2> f = unpack<T>(r[i]);
            x[i / 2][2 * (i % 2)] = f.v[0], x[i / 2][2 * (i % 2) + 1] = f.v[1];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e / 4][e % 4] = *reinterpret_cast<const float *>(tile + (8 * (e / 4) + 2 * (lane & 3) + e % 2) * 80 + ((lane >> 2) + 8 * (e / 2 % 2)) * 4);
    }
}
template <typename T>
__device__ __forceinline__ void write_tile(uint8_t *tile, const Acc (&x)[2], int lane) {
    if constexpr (sizeof(T) == 2) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = pack<T>(Vec<2>{{x[i / 2][2 * (i % 2)], x[i / 2][2 * (i % 2) + 1]}});
        stsm_t(smem_u32(tile) + tile_word<T>((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1), r[0], r[1], r[2], r[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float *>(tile + (8 * (e / 4) + 2 * (lane & 3) + e % 2) * 80 + ((lane >> 2) + 8 * (e / 2 % 2)) * 4) = x[e / 4][e % 4];
    }
}
// Rows [0, rows) of the tile, and zeros up to row `all`, to dst
template <typename T>
__device__ __forceinline__ void store_tile(T *dst, int64_t stride, const uint8_t *tile, int rows, int all, int cols, bool words, int lane) {
    constexpr int kWords = sizeof(T), kEl = 16 / sizeof(T);
    if (words) {
#pragma unroll
        for (int i = 0; i < kWords / 2; ++i) {
            const int row = (lane + 32 * i) / kWords, word = (lane + 32 * i) % kWords;
            if (row < all && word * kEl < cols)
                *reinterpret_cast<uint4 *>(dst + row * stride + word * kEl) =
                    row < rows ? *reinterpret_cast<const uint4 *>(tile + tile_word<T>(row, word)) : make_uint4(0, 0, 0, 0);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = (lane >> 4) + 2 * i, c = lane & 15;
            if (row < all && c < cols)
                dst[row * stride + c] =
                    row < rows ? *reinterpret_cast<const T *>(tile + tile_word<T>(row, c / kEl) + c % kEl * sizeof(T)) : from_f32<T>(0.0f);
        }
    }
}
// A quarter (N blocks) of a state (K,V)'s transpose
template <int N>
__device__ __forceinline__ void read_state(Acc (&s)[N], const float *p, int k0, int K, int V, int v0, int lane) {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = k0 + 8 * j + 2 * (lane & 3) + e % 2, v = v0 + (lane >> 2) + 8 * (e / 2);
            s[j][e] = 0.0f;
            if (p && k < K && v < V) s[j][e] = p[static_cast<int64_t>(k) * V + v];
        }
}
template <int N>
__device__ __forceinline__ void write_state(float *p, const Acc (&s)[N], int k0, int K, int V, int v0, int lane) {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = k0 + 8 * j + 2 * (lane & 3) + e % 2, v = v0 + (lane >> 2) + 8 * (e / 2);
            if (k < K && v < V) p[static_cast<int64_t>(k) * V + v] = s[j][e];
        }
}
// Columns of two blocks times f[column] (and c)
__device__ __forceinline__ void by_columns(Acc (&x)[2], const float *f, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) by_pairs(x[i], *reinterpret_cast<const Vec<2> *>(f + 8 * i + 2 * (lane & 3)));
}
__device__ __forceinline__ void by_columns(Acc (&x)[2], const float *f, float c, int lane) {
#pragma unroll
    for (int i = 0; i < 2; ++i) by_pairs(x[i], vmul(*reinterpret_cast<const Vec<2> *>(f + 8 * i + 2 * (lane & 3)), splat<2>(c)));
}
template <int N>
__device__ __forceinline__ void scale_all(Acc (&x)[N], float c) {
#pragma unroll
    for (int i = 0; i < N; ++i) by_pairs(x[i], splat<2>(c));
}
template <int N>
__device__ __forceinline__ void add(Acc (&x)[N], const Acc (&t)[N], float c) {
#pragma unroll
    for (int i = 0; i < N; ++i) add_times(x[i], t[i], c);
}
// Left operands, handed over through shared memory or left in a record
template <int TERMS>
__device__ __forceinline__ void give(uint8_t *to, const uint32_t (&a)[TERMS][4], int lane) {
#pragma unroll
    for (int j = 0; j < TERMS; ++j) *reinterpret_cast<uint4 *>(to + j * 512 + lane * 16) = make_uint4(a[j][0], a[j][1], a[j][2], a[j][3]);
}
template <int TERMS>
__device__ __forceinline__ void take(uint32_t (&a)[TERMS][4], const uint8_t *from, int lane) {
#pragma unroll
    for (int j = 0; j < TERMS; ++j) {
        const uint4 x = *reinterpret_cast<const uint4 *>(from + j * 512 + lane * 16);
        a[j][0] = x.x, a[j][1] = x.y, a[j][2] = x.z, a[j][3] = x.w;
    }
}
template <int TERMS, int N>
__device__ __forceinline__ void leave(uint8_t *to, int term, const uint32_t (&a)[N][4], int lane) {
#pragma unroll
    for (int j = 0; j < TERMS; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) *reinterpret_cast<uint32_t *>(to + j * term + r * 128 + lane * 4) = a[j][r];
}

// Records come by bulk copies that one thread issues (as 16-byte copies of all threads they took 1250 of a chunk's 4200 cycles where one slice
// has an SM to itself: 1 x 16384, 16 heads of 128 x 128). A barrier counts a stage's bytes, and all threads wait for it; another counts the warps
// that are done with the stage, and only the thread that fills it again waits for that: slices that share records need not keep step (8 x 4096
// rows, 16 heads of 128 x 128: forward 572 to 511 us, backward 666 to 607).
__device__ unsigned int g_delta_status;  // bit 0: a wait for records gave up
constexpr uint64_t kDeltaWaitNs = 1000000000ull;

struct Stages {
    uint32_t bars, done;  // a barrier of eight bytes for each stage
    uint32_t late = 0, parities = 0;  // stages whose copies were given up, and the phases they belong to

    static constexpr int bytes(int count) { return 16 * count; }
    __device__ __forceinline__ void begin(uint8_t *at, int count) {
        bars = smem_u32(at), done = bars + 8 * count;
        if (threadIdx.x == 0) {
            for (int i = 0; i < count; ++i) mbar_init(bars + 8 * i, 1), mbar_init(done + 8 * i, blockDim.x / 32);
            fence_mbar_init();
        }
        __syncthreads();
    }
    // Two records, one behind the other, by thread 0, once all warps are done with what the stage held. use: how often it was filled before (0 where a barrier
    // of the CTA has said so).
    __device__ __forceinline__ void copy(int stage, int use, uint8_t *to, const uint8_t *a, int a_bytes, const uint8_t *b, int b_bytes) {
        if (threadIdx.x != 0) return;
        const uint32_t bar = bars + 8 * stage, at = smem_u32(to);
        if (use > 0 && !mbar_try_wait(done + 8 * stage, use - 1 & 1) && (late || !come(done + 8 * stage, use - 1 & 1))) late |= 1u << 31;
        mbar_arrive_expect_tx(bar, a_bytes + b_bytes);
        bulk_copy(at, a, a_bytes, bar);
        if (b_bytes) bulk_copy(at + a_bytes, b, b_bytes, bar);
    }
    // A wait that gives up (a second: the copy has not come) sets the status word; later ones look only once, so that the kernel ends.
    __device__ __forceinline__ void wait(int stage, int parity) {
        if (mbar_try_wait(bars + 8 * stage, parity)) return;
        if (late || !come(bars + 8 * stage, parity)) late |= 1u << stage, parities = (parities & ~(1u << stage)) | static_cast<uint32_t>(parity) << stage;
    }
    // The warp is done with the stage.
    __device__ __forceinline__ void leave(int stage) const {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(done + 8 * stage);
    }
    // Before the CTA ends: what was given up may still be on its way into its shared memory
    __device__ __forceinline__ void end() const {
        if (late)
            for (int i = 0; i < 8; ++i)
                if (late >> i & 1) come(bars + 8 * i, parities >> i & 1);
    }
    __device__ static __noinline__ bool come(uint32_t bar, int parity) {
        const uint64_t began = global_timer_ns();
        while (!mbar_try_wait(bar, parity)) {
            if (global_timer_ns() - began > kDeltaWaitNs) {
                atomicOr(&g_delta_status, 1u);
                return false;
            }
        }
        return true;
    }
};

// Operands of another scale than what they are added up with come to the largest's by a power of two: what that takes from their last bits
// is below the sum's. The exponent of a power of two, and 2^e for e <= 0 as two halves
__device__ __forceinline__ int exponent(float pow2) { return static_cast<int>(__float_as_uint(pow2) >> 23) - 127; }
__device__ __forceinline__ uint32_t halves(int e) {
    const uint32_t h = e >= -14 ? static_cast<uint32_t>(15 + e) << 10 : e >= -24 ? 1u << (24 + e) : 0u;
    return h | h << 16;
}
template <int TERMS>
__device__ __forceinline__ void times(uint32_t (&to)[TERMS][4], const uint32_t (&a)[TERMS][4], uint32_t f) {
#pragma unroll
    for (int j = 0; j < TERMS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(to[j][i]) : "r"(a[j][i]), "r"(f));
}

// What both directions have in common: this warp's place, and the parts of shared memory
template <typename T, int KP, bool BWD>
struct Seq {
    using R = Rec<T, KP>;
    using Sm = SeqSmem<T, KP>;
    static constexpr int NI = Terms<T>::in, NO = Terms<T>::out, kSteps = KP / 64, kStage = Sm::stage(BWD);  // steps: of 16 of the keys' channels
    const DeltaParams &p;
    uint8_t *smem, *mine;  // the records; the slice's
    int lane, w, slice, head, hk, v0, cols;
    float *sc;  // inverse scales of operands
    enum { SC_QUARTER = 0, SC_X = 4, SC_E = 8, SC_U = 12, SC_W = 16, SC_STATE = 20 };  // of each quarter, of 16 rows of x, e, u and w each, of the state
    uint8_t *tiles;

    __device__ __forceinline__ Seq(const DeltaParams &p_, uint8_t *smem_) : p(p_), smem(smem_) {
        const int quad = threadIdx.x / kQuad, quads = blockDim.x / kQuad;
        lane = threadIdx.x & 31, w = threadIdx.x >> 5 & 3;
        head = blockIdx.y, hk = head / (p.H / p.HK);
        slice = blockIdx.x * quads + quad, v0 = slice * kSlice, cols = p.V - v0;
        mine = smem + 2 * kStage + quad * Sm::slice;
        sc = reinterpret_cast<float *>(mine + Sm::scales);
        tiles = mine + Sm::scales + 128 + 2 * w * Sm::tile;
    }
    __device__ __forceinline__ void meet() const { named_bar_sync(1 + threadIdx.x / kQuad, kQuad); }
    // The largest of this warp's quarter of the state, as an inverse scale; and, once all four are known, the quarter's left operands for the others and
    // for the record. Operands are scaled by what they hold, not by bounds from what they are made of: the largest factors may belong to different rows
    // (a token masked by beta 0, values in front of a cleared state). By such bounds 1 x 16384 rows of 16 heads of 128 x 128 took 581 us where this takes 627, and
    // 8 x 4096 rows in training 2336 where this takes 2385, but a masked row 10^4 times the others cost the results behind it all but 11 bits.
    __device__ __forceinline__ void measure(const Acc (&s)[2 * kSteps]) const {
        const float own = inverse_of(warp_scale(s));
        if (lane == 0) sc[SC_QUARTER + w] = own;
    }
    __device__ __forceinline__ void hand_over(const Acc (&s)[2 * kSteps], uint8_t *rec, float *rec_scale) const {
        const float4 of = *reinterpret_cast<const float4 *>(sc + SC_QUARTER);
        const float inverse = fmaxf(fmaxf(of.x, of.y), fmaxf(of.z, of.w)), f = inverse_of(inverse);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            uint32_t a[2][4];
            left_of<2>(a, s[2 * i], s[2 * i + 1], f);
            give<2>(mine + Sm::state + (w * kSteps + i) * 1024, a, lane);
            if (rec) leave<NO>(rec + (w * kSteps + i) * 512, SliceRec<T, KP>::state_term, a, lane);
        }
        if (lane == 0 && w == 0) {
            sc[SC_STATE] = inverse;
            if (rec) *rec_scale = inverse;
        }
    }
    // Rows' left operand, scaled by its own largest, for the others: at number `place` of sc, and of a record
    template <int TERMS>
    __device__ __forceinline__ void hand_rows(const Acc (&x)[2], float f, uint8_t *to, int place, uint8_t *rec = nullptr, float *rec_scale = nullptr) const {
        uint32_t a[TERMS][4];
        left_of<TERMS>(a, x[0], x[1], f);
        if (to) give<TERMS>(to, a, lane);
        if (rec) leave<TERMS>(rec, kRowsTerm, a, lane);
        if (lane == 0) {
            if (to) sc[place + w] = inverse_of(f);
            if (rec) *rec_scale = inverse_of(f);
        }
    }
};

template <typename T, int KP>
__global__ void __launch_bounds__(512, 1) based_delta_fwd_kernel(DeltaParams p) {
    using R = Rec<T, KP>;
    using Sm = SeqSmem<T, KP>;
    using SR = SliceRec<T, KP>;
    using Q = Seq<T, KP, false>;
    constexpr int NI = Q::NI, NO = Q::NO, kSteps = Q::kSteps, kStage = Q::kStage;
    extern __shared__ __align__(128) uint8_t smem[];
    const Q q(p, smem);
    const int lane = q.lane, w = q.w, head = q.head, v0 = q.v0, cols = q.cols, slices = (p.V + kSlice - 1) / kSlice;
    // The next chunk's records are asked for at once where a slice has the CTA to itself, else after a chunk's first products: other
    // slices may still be in the chunk before.
    const bool alone = blockDim.x == kQuad;
    Stages stages;
    stages.begin(smem + 2 * kStage + blockDim.x / kQuad * Sm::slice, 2);
    int turn = 0;  // chunks up to this batch entry
    griddep_wait();
    for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
        const int live = live_rows(p, b), count = (live + kChunk - 1) / kChunk;
        const int64_t st = static_cast<int64_t>(b) * p.H + head, first = static_cast<int64_t>(b) * p.T, row_o = static_cast<int64_t>(p.H) * p.V;
        const uint8_t *const qk = p.qk_rec + (static_cast<int64_t>(b) * p.HK + q.hk) * p.chunks * R::qk, *const g = p.g_rec + st * p.chunks * R::g(false);
        const T *const v = static_cast<const T *>(p.v) + b * p.v_sb + head * p.v_sh + v0;
        T *const o = static_cast<T *>(p.out) + (first * p.H + head) * p.V + v0;
        const auto record = [&](int n) { return p.saved ? p.saved + (((static_cast<int64_t>(b) * p.chunks + n) * p.H + head) * slices + q.slice) * SR::fwd : nullptr; };
        const auto fetch = [&](int n) {
            const int at = turn + n & 1;
            stages.copy(at, turn + n >> 1, smem + at * kStage, qk + static_cast<int64_t>(n) * R::qk, R::qk, g + static_cast<int64_t>(n) * R::g(false), R::g(false));
        };
        const auto values = [&](int n) {
            const int at = turn + n & 1;
            const int64_t t = static_cast<int64_t>(n) * kChunk + 16 * w;
            if (cols > 0) load_tile(q.tiles + at * Sm::tile, t < live ? v + t * p.v_st : v, p.v_st, static_cast<int>(live - t), cols, p.v_vec, lane);
            copies_commit();
        };
        Acc s[2 * kSteps];
        read_state(s, p.state ? p.state + st * p.K * p.V : nullptr, w * (KP / 4), p.K, p.V, v0, lane);
        __syncthreads();  // the batch entry before
        if (count > 0) {
            fetch(0), values(0);
            uint8_t *const rec = cols > 0 ? record(0) : nullptr;
            q.measure(s);
            q.meet();
            q.hand_over(s, rec, reinterpret_cast<float *>(rec + SR::fwd_scales));
        }
        for (int n = 0; n < count; ++n) {
            const int stage = turn + n & 1;
            stages.wait(stage, turn + n >> 1 & 1);
            if (cols <= 0) {  // the same for the slice's warps (the CTA's first slice has channels)
                stages.leave(stage);
                continue;
            }
            copies_wait<0>();
            q.meet();  // chunk n's values and the state's operands are there
            if (n + 1 < count) values(n + 1);
            if (n + 1 < count && alone) fetch(n + 1);
            const int64_t t0 = static_cast<int64_t>(n) * kChunk + 16 * w;  // this warp's first row
            uint8_t *const tile = q.tiles + stage * Sm::tile;
            const uint32_t kimg = smem_u32(smem) + stage * kStage, qimg = kimg + R::img, inv = kimg + R::qk, pimg = inv + 2 * kSquare;
            const float *const f = reinterpret_cast<const float *>(smem + stage * kStage + R::qk + (2 + NO) * kSquare);
            uint8_t *const rec = record(n);
            float *const rec_scales = reinterpret_cast<float *>(rec + SR::fwd_scales);
            Acc x[2], z[2], y[2];  // S0^T K^T, S0^T Q^T
            clear(x), clear(z);
            const float is = q.sc[Q::SC_STATE];
            {
                uint32_t a[2][2][4], r[2][NI][4], c[2][NI][4];
                const auto load = [&](int kk) {
                    take<2>(a[kk & 1], q.mine + Sm::state + kk * 1024, lane);
#pragma unroll
                    for (int j = 0; j < NI; ++j)
                        right<KP>(r[kk & 1][j], kimg + j * R::term, 16 * w, 16 * kk, lane), right<KP>(c[kk & 1][j], qimg + j * R::term, 16 * w, 16 * kk, lane);
                };
                load(0);
#pragma unroll
                for (int kk = 0; kk < KP / 16; ++kk) {
                    if (kk + 1 < KP / 16) load(kk + 1);  // a step ahead: often a warp has its scheduler to itself
                    products<T, 2, NI>(x[0], x[1], a[kk & 1], r[kk & 1]);
                    products<T, NO, NI>(z[0], z[1], reinterpret_cast<const uint32_t(&)[NO][4]>(a[kk & 1]), c[kk & 1]);
                }
            }
            by_columns(x, f + F_GROWSTEP + 16 * w, f[F_K] * is, lane);
            by_columns(z, f + F_GROW + 16 * w, f[F_Q] * p.scale * is, lane);
            read_tile<T>(y, tile, lane);
            by_columns(y, f + F_STEP + 16 * w, lane);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][e] = y[i][e] - x[i][e];
            q.template hand_rows<2>(x, warp_scale(x), q.mine + Sm::x(false) + w * 1024, Q::SC_X);
            if (n + 1 < count && !alone) fetch(n + 1);
            q.meet();
            {  // E: X and what the rows in front have written. X and E are times their rows' steps from here on
                uint32_t a[2][2][4], r[2][2][4];
                const auto load = [&](int kb) {
                    take<2>(a[kb & 1], q.mine + Sm::x(false) + kb * 1024, lane);
                    right<kChunk>(r[kb & 1][0], inv, 16 * w, 16 * kb, lane), right<kChunk>(r[kb & 1][1], inv + kSquare, 16 * w, 16 * kb, lane);
                };
                load(0);
#pragma unroll
                for (int kb = 0; kb < 4; ++kb) {
                    if (kb > w) break;
                    if (kb < 3) load(kb + 1);  // (of the last one nothing comes)
                    products_by<2, 2>(x[0], x[1], a[kb & 1], r[kb & 1], q.sc[Q::SC_X + kb] * f[F_INV]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[i][e] = x[i][e];
            by_columns(y, f + F_BF + 16 * w, lane);
            {
                // (U is E times factors of up to F_BFMOST in these rows)
                const float se = warp_scale(x), su = scale_for(kTop * inverse_of(se) * f[F_BFMOST + w]);
                q.template hand_rows<2>(y, su, q.mine + Sm::u + w * 1024, Q::SC_U);
                q.template hand_rows<NO>(x, se, q.mine + Sm::e + w * Sm::e_block, Q::SC_E, rec ? rec + SR::e + w * 512 : nullptr, rec_scales + 1 + w);
            }
            q.meet();
            {
                uint32_t a[2][NO][4], r[2][NO][4];
                const auto load = [&](int kb) {
                    take<NO>(a[kb & 1], q.mine + Sm::e + kb * Sm::e_block, lane);
#pragma unroll
                    for (int j = 0; j < NO; ++j) right<kChunk>(r[kb & 1][j], pimg + j * kSquare, 16 * w, 16 * kb, lane);
                };
                load(0);
#pragma unroll
                for (int kb = 0; kb < 4; ++kb) {
                    if (kb > w) break;
                    if (kb < 3) load(kb + 1);
                    products_by<NO, NO>(z[0], z[1], a[kb & 1], r[kb & 1], q.sc[Q::SC_E + kb] * f[F_P]);
                }
            }
            // S = whole S0 + K^T U, this warp's quarter
            const float ik = f[F_K];
            scale_all(s, f[F_WHOLE]);
            {
                uint32_t a[2][2][4], r[2][kSteps][NI][4];
                const auto load = [&](int kb) {
                    take<2>(a[kb & 1], q.mine + Sm::u + kb * 1024, lane);
#pragma unroll
                    for (int i = 0; i < kSteps; ++i)
#pragma unroll
                        for (int j = 0; j < NI; ++j) right_t<KP>(r[kb & 1][i][j], kimg + j * R::term, 16 * kb, w * (KP / 4) + 16 * i, lane);
                };
                load(0);
#pragma unroll
                for (int kb = 0; kb < 4; ++kb) {
                    if (kb < 3) load(kb + 1);
                    const float iu = q.sc[Q::SC_U + kb] * ik;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) products_by<2, NI>(s[2 * i], s[2 * i + 1], a[kb & 1], r[kb & 1][i], iu);
                }
            }
            stages.leave(stage);
            q.measure(s);
            if (t0 < p.T) {
                write_tile<T>(tile, z, lane);
                __syncwarp();
                store_tile<T>(o + t0 * row_o, row_o, tile, static_cast<int>(live - t0), static_cast<int>(p.T - t0), cols, p.o_vec, lane);
            }
            if (n + 1 < count) {
                uint8_t *const next = record(n + 1);
                q.meet();
                q.hand_over(s, next, reinterpret_cast<float *>(next + SR::fwd_scales));
            }
        }
        turn += count;
        if (cols > 0) {
            for (int64_t t = static_cast<int64_t>(count) * kChunk + 16 * w; t < p.T; t += kChunk)
                store_tile<T>(o + t * row_o, row_o, q.tiles, 0, static_cast<int>(p.T - t), cols, p.o_vec, lane);
            if (p.final_state) write_state(p.final_state + st * p.K * p.V, s, w * (KP / 4), p.K, p.V, v0, lane);
        }
    }
    stages.end();
}

template <typename T, int KP>
__global__ void __launch_bounds__(512, 1) based_delta_bwd_kernel(DeltaParams p) {
    using R = Rec<T, KP>;
    using Sm = SeqSmem<T, KP>;
    using SR = SliceRec<T, KP>;
    using Q = Seq<T, KP, true>;
    constexpr int NI = Q::NI, NO = Q::NO, kSteps = Q::kSteps, kStage = Q::kStage;
    extern __shared__ __align__(128) uint8_t smem[];
    const Q q(p, smem);
    const int lane = q.lane, w = q.w, head = q.head, v0 = q.v0, cols = q.cols, slices = (p.V + kSlice - 1) / kSlice;
    // The next chunk's records are asked for at once where a slice has the CTA to itself, else after a chunk's first products: other
    // slices may still be in the chunk before.
    const bool alone = blockDim.x == kQuad;
    Stages stages;
    stages.begin(smem + 2 * kStage + blockDim.x / kQuad * Sm::slice, 2);
    int turn = 0;  // chunks up to this batch entry
    griddep_wait();
    for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
        const int live = live_rows(p, b), count = (live + kChunk - 1) / kChunk;
        const int64_t st = static_cast<int64_t>(b) * p.H + head, first = static_cast<int64_t>(b) * p.T, row_o = static_cast<int64_t>(p.H) * p.V;
        const uint8_t *const qk = p.qk_rec + (static_cast<int64_t>(b) * p.HK + q.hk) * p.chunks * R::qk, *const grec = p.g_rec + st * p.chunks * R::g(true);
        const T *const dout = static_cast<const T *>(p.dout) + b * p.do_sb + head * p.do_sh + v0;
        T *const dv = static_cast<T *>(p.out) + (first * p.H + head) * p.V + v0;
        const auto record = [&](int n) { return p.slice_rec + (((static_cast<int64_t>(b) * p.chunks + n) * p.H + head) * slices + q.slice) * SR::bwd; };
        const auto fetch = [&](int n) {
            const int at = turn + count - 1 - n & 1;
            stages.copy(at, turn + count - 1 - n >> 1, smem + at * kStage, qk + static_cast<int64_t>(n) * R::qk, R::qk,
                        grec + static_cast<int64_t>(n) * R::g(true), R::g(true));
        };
        const auto values = [&](int n) {
            const int at = turn + count - 1 - n & 1;
            const int64_t t = static_cast<int64_t>(n) * kChunk + 16 * w;
            if (cols > 0) load_tile(q.tiles + at * Sm::tile, t < live ? dout + t * p.do_st : dout, p.do_st, static_cast<int>(live - t), cols, p.do_vec, lane);
            copies_commit();
        };
        Acc g[2 * kSteps];
        read_state(g, p.state ? p.state + st * p.K * p.V : nullptr, w * (KP / 4), p.K, p.V, v0, lane);
        __syncthreads();
        if (count > 0) {
            fetch(count - 1), values(count - 1);
            if (cols > 0) {
                q.measure(g);
                q.meet();
                q.hand_over(g, record(count - 1), reinterpret_cast<float *>(record(count - 1) + SR::bwd_scales));
            }
        }
        for (int n = count - 1; n >= 0; --n) {
            const int stage = turn + count - 1 - n & 1;
            stages.wait(stage, turn + count - 1 - n >> 1 & 1);
            if (cols <= 0) {
                stages.leave(stage);
                continue;
            }
            copies_wait<0>();
            q.meet();
            if (n > 0) values(n - 1);
            if (n > 0 && alone) fetch(n - 1);
            const int64_t t0 = static_cast<int64_t>(n) * kChunk + 16 * w;
            uint8_t *const tile = q.tiles + stage * Sm::tile;
            const uint32_t kimg = smem_u32(smem) + stage * kStage, qimg = kimg + R::img, inv = kimg + R::qk, pimg = inv + 2 * kSquare;
            const float *const f = reinterpret_cast<const float *>(smem + stage * kStage + R::qk + 4 * kSquare);
            uint8_t *const rec = record(n);
            float *const rec_scales = reinterpret_cast<float *>(rec + SR::bwd_scales);
            Acc x[2], y[2];
            read_tile<T>(y, tile, lane);  // dO
            const float so = warp_scale(y);
            q.template hand_rows<NI>(y, so, q.mine + Sm::e + w * Sm::e_block, Q::SC_E, rec + SR::dout + w * 512, rec_scales + 5 + w);
            clear(x);  // dU
            const float is = q.sc[Q::SC_STATE];
            {
                uint32_t a[2][2][4], r[2][NI][4];
                const auto load = [&](int kk) {
                    take<2>(a[kk & 1], q.mine + Sm::state + kk * 1024, lane);
#pragma unroll
                    for (int j = 0; j < NI; ++j) right<KP>(r[kk & 1][j], kimg + j * R::term, 16 * w, 16 * kk, lane);
                };
                load(0);
#pragma unroll
                for (int kk = 0; kk < KP / 16; ++kk) {
                    if (kk + 1 < KP / 16) load(kk + 1);
                    products<T, 2, NI>(x[0], x[1], a[kk & 1], r[kk & 1]);
                }
            }
            by_columns(x, f + F_REST + 16 * w, f[F_K] * is, lane);
            if (n > 0 && !alone) fetch(n - 1);
            q.meet();
            {  // (from the last rows up: all warps have those)
                uint32_t a[2][NI][4], r[2][2][4];
                const auto load = [&](int kb) {
                    take<NI>(a[kb & 1], q.mine + Sm::e + kb * Sm::e_block, lane);
                    right_t<kChunk>(r[kb & 1][0], pimg, 16 * kb, 16 * w, lane), right_t<kChunk>(r[kb & 1][1], pimg + kSquare, 16 * kb, 16 * w, lane);
                };
                load(3);
#pragma unroll
                for (int kb = 3; kb >= 0; --kb) {
                    if (kb < w) break;
                    if (kb > 0) load(kb - 1);
                    products_by<NI, 2>(x[0], x[1], a[kb & 1], r[kb & 1], q.sc[Q::SC_E + kb] * f[F_P]);
                }
            }
            by_columns(y, f + F_GROW + 16 * w, p.scale, lane);
            {
                const float sx = warp_scale(x), su = scale_for(kTop * inverse_of(so) * f[F_GROWMOST + w] * fabsf(p.scale));
                q.template hand_rows<2>(x, sx, q.mine + Sm::x(true) + w * 1024, Q::SC_X);
                q.template hand_rows<2>(y, su, q.mine + Sm::u + w * 1024, Q::SC_U);
            }
            q.meet();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[i][e] = x[i][e];
            {  // dR: dU and what the rows behind take back
                uint32_t a[2][2][4], r[2][2][4];
                const auto load = [&](int kb) {
                    take<2>(a[kb & 1], q.mine + Sm::x(true) + kb * 1024, lane);
                    right_t<kChunk>(r[kb & 1][0], inv, 16 * kb, 16 * w, lane), right_t<kChunk>(r[kb & 1][1], inv + kSquare, 16 * kb, 16 * w, lane);
                };
                load(3);
#pragma unroll
                for (int kb = 3; kb >= 0; --kb) {
                    if (kb < w) break;
                    if (kb > 0) load(kb - 1);
                    products_by<2, 2>(y[0], y[1], a[kb & 1], r[kb & 1], q.sc[Q::SC_X + kb] * f[F_INV]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][e] = y[i][e];
            by_columns(y, f + F_BF + 16 * w, -1.0f, lane);
            {
                const float sr = warp_scale(x), sw = scale_for(kTop * inverse_of(sr) * f[F_BFMOST + w]);
                q.template hand_rows<2>(y, sw, q.mine + Sm::w + w * 1024, Q::SC_W);
                q.template hand_rows<NO>(x, sr, nullptr, 0, rec + SR::dr + w * 512, rec_scales + 1 + w);
            }
            by_columns(x, f + F_BETA + 16 * w, lane);  // dV
            q.meet();
            const float ik = f[F_K], iq = f[F_Q];
            scale_all(g, f[F_WHOLE]);
#pragma unroll
            for (int kb = 0; kb < 4; ++kb) {  // (a step ahead there would be registers for neither)
                uint32_t a[2][4], c[2][4];
                take<2>(a, q.mine + Sm::u + kb * 1024, lane), take<2>(c, q.mine + Sm::w + kb * 1024, lane);
                const float iu = q.sc[Q::SC_U + kb] * iq, iw = q.sc[Q::SC_W + kb] * ik;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    uint32_t r[NI][4];
#pragma unroll
                    for (int j = 0; j < NI; ++j) right_t<KP>(r[j], qimg + j * R::term, 16 * kb, w * (KP / 4) + 16 * i, lane);
                    products_by<2, NI>(g[2 * i], g[2 * i + 1], a, r, iu);
#pragma unroll
                    for (int j = 0; j < NI; ++j) right_t<KP>(r[j], kimg + j * R::term, 16 * kb, w * (KP / 4) + 16 * i, lane);
                    products_by<2, NI>(g[2 * i], g[2 * i + 1], c, r, iw);
                }
            }
            stages.leave(stage);
            q.measure(g);
            if (t0 < p.T) {
                write_tile<T>(tile, x, lane);
                __syncwarp();
                store_tile<T>(dv + t0 * row_o, row_o, tile, static_cast<int>(live - t0), static_cast<int>(p.T - t0), cols, p.o_vec, lane);
            }
            if (n > 0) {
                q.meet();
                q.hand_over(g, record(n - 1), reinterpret_cast<float *>(record(n - 1) + SR::bwd_scales));
            }
        }
        turn += count;
        if (cols > 0) {
            for (int64_t t = static_cast<int64_t>(count) * kChunk + 16 * w; t < p.T; t += kChunk)
                store_tile<T>(dv + t * row_o, row_o, q.tiles, 0, static_cast<int>(p.T - t), cols, p.o_vec, lane);
            if (p.final_state) write_state(p.final_state + st * p.K * p.V, g, w * (KP / 4), p.K, p.V, v0, lane);
        }
    }
    stages.end();
}

// ------------------------------------------------------------------------------------------------
// Gradients that need no order. With dP = dO U^T and dA = -dR U^T (below the diagonal),
//     dQ = scale grow dO S0^T + (scale D dP) K,
//     dK = rest U G^T - beta grow dR S0^T + (scale D dP)^T Q + (beta D dA) K + (beta D dA)^T K,
//     dbeta = the diagonal of dR E^T,
// and the gradient of b_i, the sum of log decays up to row i, is what row i reads minus what it has written:
//     db_i = q_i (scale grow dO S0^T)_i - k_i (beta grow dR S0^T + rest U G^T)_i + sum_j (N_ij - N_ji),  N = dP P + dA A,
// with grow_last <S0, G> + sum_i k_i (rest U G^T)_i more at the last row; dgate_i is the sum of db from i on.
// A CTA takes one chunk of one key head and adds up the value heads that share it, so that nothing is added by atomics. Its eight warps share out
// the products' results, 16 rows and half of the columns each; the slices' records come in by a ring of stages and are used as they lie. With
// 16 warps of a quarter of the columns left operands were read twice as often (8 x 4096 rows, 16 heads of 128 x 128: 782 us, now 756; without the
// barrier of each slice 797). The pairs' sums N come from the products of queries and keys again, 16 % of a CTA's time: taken from q dq - k dk
// they would be differences of rounded sums, and where decays are steep dgate would be what that rounding leaves.
// ------------------------------------------------------------------------------------------------
constexpr int kGradWarps = 8;

template <typename T, int KP>
struct GradSmem {
    using SR = SliceRec<T, KP>;
    static constexpr int stages = Terms<T>::out == 1 ? 4 : 3, stage = SR::fwd + SR::bwd;
    static constexpr int f = Rec<T, KP>::qk, ring = f + F_COUNT * 4, dp = ring + stages * stage, da = dp + Terms<T>::out * kSquare,
                         part = da + Terms<T>::out * kSquare;  // sums: rows 2 x 64, next 2 x 64, columns 4 x 64, dbeta 64
    static constexpr int red = part + 9 * kChunk * 4, bars = red + 2 * kGradWarps * 4, bytes = bars + Stages::bytes(stages + 1);
};

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
// A left operand's transpose, 16 of the chunk's rows by a slice's channels, and a right operand, a slice's channels by 16 columns, from the
// blocks of a record
__device__ __forceinline__ void left_blocks(uint32_t (&r)[4], uint32_t at, int lane) {
    ldsm_t(r, at + ((lane >> 4) + 2 * (lane >> 3 & 1)) * 128 + (lane & 7) * 16);
}
__device__ __forceinline__ void right_blocks(uint32_t (&r)[4], uint32_t at, int lane) { ldsm_t(r, at + lane * 16); }

// Slices differ in their scales: their products are brought to the largest's on one operand.
template <typename T, int KP>
__global__ void __launch_bounds__(32 * kGradWarps, 1) based_delta_grad_kernel(DeltaParams p) {
    using R = Rec<T, KP>;
    using SR = SliceRec<T, KP>;
    using Sm = GradSmem<T, KP>;
    constexpr int NI = Terms<T>::in, NO = Terms<T>::out, NQ = KP / 32, kThreads = 32 * kGradWarps;  // NQ: 16 columns of a warp's half
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wm = warp & 3, wn = warp >> 2;
    const int n = blockIdx.x, hk = blockIdx.y, group = p.H / p.HK, slices = (p.V + kSlice - 1) / kSlice;
    const int r0 = 16 * wm + (lane >> 2), r1 = r0 + 8, col0 = wn * (KP / 2) + 2 * (lane & 3);  // this thread's accumulators
    const bool traces = warp < KP / 16;
    float *const f = reinterpret_cast<float *>(smem + Sm::f);
    float *const part_row = reinterpret_cast<float *>(smem + Sm::part), *const part_next = part_row + 2 * kChunk,
                *const part_col = part_next + 2 * kChunk, *const part_beta = part_col + 4 * kChunk, *const red = reinterpret_cast<float *>(smem + Sm::red);
    const uint32_t base = smem_u32(smem), kimg = base, qimg = base + R::img;
    constexpr int kKeysStage = Sm::stages;  // the stage of the queries' and keys' images
    Stages stages;
    stages.begin(smem + Sm::bars, Sm::stages + 1);
    int turn = 0, entry = 0;  // slices and batch entries up to this one
    griddep_wait();
    for (int b = blockIdx.z; b < p.B; b += gridDim.z) {
        const int64_t t0 = static_cast<int64_t>(n) * kChunk, first = static_cast<int64_t>(b) * p.T + t0;
        const int rows = min(kChunk, live_rows(p, b) - n * kChunk), all = static_cast<int>(p.T - t0 < kChunk ? p.T - t0 : kChunk);
        T *const dq = static_cast<T *>(p.dq) + (first * p.HK + hk) * p.K, *const dk = static_cast<T *>(p.dk) + (first * p.HK + hk) * p.K;
        const int64_t row_k = static_cast<int64_t>(p.HK) * p.K;
        if (rows > 0) {
            __syncthreads();  // the batch entry before
            stages.copy(kKeysStage, 0, smem, p.qk_rec + ((static_cast<int64_t>(b) * p.HK + hk) * p.chunks + n) * R::qk, R::qk, nullptr, 0);
        }
        const int from = rows < 0 ? 0 : rows;  // padding
        for (int i = tid; i < (all - from) * p.K; i += kThreads) {
            const int64_t at = (from + i / p.K) * row_k + i % p.K;
            dq[at] = dk[at] = from_f32<T>(0.0f);
        }
        for (int i = tid; i < (all - from) * group; i += kThreads) {
            const int64_t at = (first + from + i / group) * p.H + hk * group + i % group;
            static_cast<T *>(p.dbeta)[at] = from_f32<T>(0.0f);
            if (p.dgate) static_cast<T *>(p.dgate)[at] = from_f32<T>(0.0f);
        }
        if (rows <= 0) continue;
        Acc aq[2 * NQ], ak[2 * NQ];
        clear(aq), clear(ak);
        for (int hh = 0; hh < group; ++hh) {
            const int head = hk * group + hh;
            const uint8_t *const rec = p.g_rec + ((static_cast<int64_t>(b) * p.H + head) * p.chunks + n) * R::g(true) + 4 * kSquare;
            const int64_t at0 = ((static_cast<int64_t>(b) * p.chunks + n) * p.H + head) * slices;
            const uint8_t *const fwd = p.saved + at0 * SR::fwd, *const bwd = p.slice_rec + at0 * SR::bwd;
            const auto fetch = [&](int sl) {
                const int at = (turn + sl) % Sm::stages;
                if (sl < slices)
                    stages.copy(at, 0, smem + Sm::ring + at * Sm::stage, fwd + static_cast<int64_t>(sl) * SR::fwd, SR::fwd,
                                bwd + static_cast<int64_t>(sl) * SR::bwd, SR::bwd);
            };
            __syncthreads();  // the head before
#pragma unroll
            for (int i = 0; i < Sm::stages - 1; ++i) fetch(i);
            for (int i = tid; i < F_COUNT; i += kThreads) f[i] = reinterpret_cast<const float *>(rec)[i];
            // The largest exponents of the slices' products for this warp: dO S0, dR S0, E G, S0 G, and by 16 columns dO E, dR E
            enum { OS, RS, EG, SG, OE, RE = OE + 2, kProducts = RE + 2 };
            int top[kProducts];
#pragma unroll
            for (int i = 0; i < kProducts; ++i) top[i] = -1000;
            const auto exponents = [&](int (&x)[kProducts], int sl) {
                const float *const a = reinterpret_cast<const float *>(fwd + static_cast<int64_t>(sl) * SR::fwd + SR::fwd_scales),
                                   *const c = reinterpret_cast<const float *>(bwd + static_cast<int64_t>(sl) * SR::bwd + SR::bwd_scales);
                const int s = exponent(a[0]), g = exponent(c[0]), r = exponent(c[1 + wm]), o = exponent(c[5 + wm]);
                x[OS] = o + s, x[RS] = r + s, x[EG] = exponent(a[1 + wm]) + g, x[SG] = s + g;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int e = exponent(a[1 + 2 * wn + i]);
                    x[OE + i] = o + e, x[RE + i] = r + e;
                }
            };
            uint32_t by[kProducts];  // lane i: the factors of slice i (of 32)
            for (int sl = lane; sl < slices; sl += 32) {
                int x[kProducts];
                exponents(x, sl);
#pragma unroll
                for (int i = 0; i < kProducts; ++i) top[i] = max(top[i], x[i]);
            }
#pragma unroll
            for (int i = 0; i < kProducts; ++i) top[i] = __reduce_max_sync(0xffffffffu, top[i]);
            Acc aos[2 * NQ], ars[2 * NQ], aeg[2 * NQ], dp[4], da[4];
            Acc diagonal[2];
            clear(aos), clear(ars), clear(aeg), clear(dp), clear(da), clear(diagonal);
            for (int sl = 0; sl < slices; ++sl) {
                const int at = (turn + sl) % Sm::stages;
                stages.wait(at, (turn + sl) / Sm::stages & 1);
                __syncthreads();  // the slice is there, and the one whose place comes next is done with
                fetch(sl + Sm::stages - 1);
                const uint8_t *const x = smem + Sm::ring + at * Sm::stage, *const y = x + SR::fwd;
                if (sl % 32 == 0) {
                    int e[kProducts] = {};
                    if (sl + lane < slices) exponents(e, sl + lane);
#pragma unroll
                    for (int i = 0; i < kProducts; ++i) by[i] = halves(e[i] - top[i]);
                }
                uint32_t factor[kProducts];
#pragma unroll
                for (int i = 0; i < kProducts; ++i) factor[i] = __shfl_sync(0xffffffffu, by[i], sl % 32);
                const uint32_t xa = smem_u32(x), ya = smem_u32(y);
                uint32_t lo[NI][4], lr[NO][4], le[NO][4], c[NO][4], d[NI][4], v[NO][4];
#pragma unroll
                for (int j = 0; j < NI; ++j) left_blocks(lo[j], ya + SR::dout + j * kRowsTerm + wm * 512, lane);
#pragma unroll
                for (int j = 0; j < NO; ++j) left_blocks(lr[j], ya + SR::dr + j * kRowsTerm + wm * 512, lane), left_blocks(le[j], xa + SR::e + j * kRowsTerm + wm * 512, lane);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (2 * wn + i > wm) break;
                    times<NI>(d, lo, factor[OE + i]), times<NO>(c, lr, factor[RE + i]);
#pragma unroll
                    for (int j = 0; j < NO; ++j) right_blocks(v[j], xa + SR::e + j * kRowsTerm + (2 * wn + i) * 512, lane);
                    products<T, NI, NO>(dp[2 * i], dp[2 * i + 1], d, v);
                    products<T, NO, NO>(da[2 * i], da[2 * i + 1], c, v);
                }
                times<NI>(d, lo, factor[OS]), times<NO>(c, lr, factor[RS]), times<NO>(le, le, factor[EG]);
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
#pragma unroll
                    for (int j = 0; j < NO; ++j) right_blocks(v[j], xa + j * SR::state_term + (wn * NQ + i) * 512, lane);
                    products<T, NI, NO>(aos[2 * i], aos[2 * i + 1], d, v);
                    products<T, NO, NO>(ars[2 * i], ars[2 * i + 1], c, v);
#pragma unroll
                    for (int j = 0; j < NO; ++j) right_blocks(v[j], ya + j * SR::state_term + (wn * NQ + i) * 512, lane);
                    products<T, NO, NO>(aeg[2 * i], aeg[2 * i + 1], le, v);
                }
                // <S0, G>: the diagonal of S0^T G, 16 channels to a warp
                if (traces) {
#pragma unroll
                    for (int j = 0; j < NO; ++j) left_blocks(c[j], xa + j * SR::state_term + warp * 512, lane), right_blocks(v[j], ya + j * SR::state_term + warp * 512, lane);
                    times<NO>(c, c, factor[SG]);
                    products<T, NO, NO>(diagonal[0], diagonal[1], c, v);
                }
            }
            turn += slices;
            if (hh == 0) stages.wait(kKeysStage, entry & 1);
            float dot = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (traces && 2 * (lane & 3) + e == lane >> 2) dot += diagonal[0][e] + diagonal[1][2 + e];
            dot = ldexpf(dot, top[SG]);
            // rows' and columns' factors, and the rows' products with queries and keys
            const float ik = f[F_K], iq = f[F_Q], c0 = f[F_GROW + r0], c1 = f[F_GROW + r1], b0 = f[F_BETA + r0], b1 = f[F_BETA + r1];
            float row0 = 0.0f, row1 = 0.0f, next0 = 0.0f, next1 = 0.0f;
            {
                const float so = ldexpf(p.scale, top[OS]), sr = ldexpf(-1.0f, top[RS]), se = ldexpf(1.0f, top[EG]);
                const float n0 = b0 * inverse_of(step_of(b0)), n1 = b1 * inverse_of(step_of(b1));  // (E's rows are times their steps)
#pragma unroll
                for (int i = 0; i < 2 * NQ; ++i) {
                    const int col = col0 + 8 * i;
                    const float2 q0 = image_pair<T, KP>(smem + R::img, r0, col, iq), q1 = image_pair<T, KP>(smem + R::img, r1, col, iq);
                    const float2 k0 = image_pair<T, KP>(smem, r0, col, ik), k1 = image_pair<T, KP>(smem, r1, col, ik);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float c = e < 2 ? c0 : c1, be = e < 2 ? b0 : b1, re = f[F_REST + (e < 2 ? r0 : r1)];
                        const float x = aos[i][e] * so * c, y = ars[i][e] * sr * (be * c), z = aeg[i][e] * se * (re * (e < 2 ? n0 : n1));
                        const float qv = e == 0 ? q0.x : e == 1 ? q0.y : e == 2 ? q1.x : q1.y, kv = e == 0 ? k0.x : e == 1 ? k0.y : e == 2 ? k1.x : k1.y;
                        (e < 2 ? row0 : row1) += x * qv + y * kv;
                        (e < 2 ? next0 : next1) += z * kv;
                        aq[i][e] += x, ak[i][e] += y + z;
                    }
                }
            }
            // the products of queries and keys with keys, and with them the pairs' sums and the factors of dQ and dK
            row0 -= next0, row1 -= next1;
            float col[4][2] = {}, mp = 0.0f, ma = 0.0f;
            if (2 * wn <= wm) {
                Acc sq[4], sk[4];
                clear(sq), clear(sk);
#pragma unroll
                for (int kk = 0; kk < KP / 16; ++kk) {
                    if (!p.dgate) break;  // nobody asks for the pairs' sums
                    uint32_t a[NI][4], c4[NI][4], x[NI][4];
#pragma unroll
                    for (int j = 0; j < NI; ++j) {
                        left<KP>(a[j], qimg + j * R::term, 16 * wm, 16 * kk, lane);
                        left<KP>(c4[j], kimg + j * R::term, 16 * wm, 16 * kk, lane);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (2 * wn + i > wm) break;
#pragma unroll
                        for (int j = 0; j < NI; ++j) right<KP>(x[j], kimg + j * R::term, 32 * wn + 16 * i, 16 * kk, lane);
                        products<T, NI, NI>(sq[2 * i], sq[2 * i + 1], a, x);
                        products<T, NI, NI>(sk[2 * i], sk[2 * i + 1], c4, x);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const float sp = ldexpf(1.0f, top[OE + nt / 2]), sa = ldexpf(-1.0f, top[RE + nt / 2]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = e < 2 ? r0 : r1, j = 32 * wn + 8 * nt + 2 * (lane & 3) + e % 2;
                        const float over = inverse_of(step_of(f[F_BETA + j])), bj = f[F_BETA + j] * over;
                        if (i == j) part_beta[i] = -da[nt][e] * sa * over;
                        const float d = j <= i ? expf((f[F_BHI + i] - f[F_BHI + j]) + (f[F_BLO + i] - f[F_BLO + j])) : 0.0f;
                        dp[nt][e] = j <= i ? dp[nt][e] * sp * bj * (d * p.scale) : 0.0f;
                        da[nt][e] = j < i ? da[nt][e] * sa * bj * (d * f[F_BETA + i]) : 0.0f;
                        const float sum = j <= i ? dp[nt][e] * (sq[nt][e] * (iq * ik)) + da[nt][e] * (sk[nt][e] * (ik * ik)) : 0.0f;
                        (e < 2 ? row0 : row1) += sum;
                        col[nt][e % 2] += sum;
                        mp = fmaxf(mp, fabsf(dp[nt][e])), ma = fmaxf(ma, fabsf(da[nt][e]));
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
                for (int d = 4; d < 32; d *= 2) col[nt][0] += __shfl_xor_sync(0xffffffffu, col[nt][0], d), col[nt][1] += __shfl_xor_sync(0xffffffffu, col[nt][1], d);
                if (lane < 4) *reinterpret_cast<float2 *>(part_col + wm * kChunk + 32 * wn + 8 * nt + 2 * lane) = make_float2(col[nt][0], col[nt][1]);
            }
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
            if (lane == 0) red[kGradWarps + warp] = dot;
            mp = scale_for(cta_most<kGradWarps>(mp, red)), ma = scale_for(cta_most<kGradWarps>(ma, red));
            if (2 * wn <= wm) {
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t at = word_at<kChunk>(e ? r1 : r0, 4 * wn + nt) + 4 * (lane & 3);
                        uint32_t w[NO];
                        terms<NO>(dp[nt][2 * e] * mp, dp[nt][2 * e + 1] * mp, w);
#pragma unroll
                        for (int j = 0; j < NO; ++j) *reinterpret_cast<uint32_t *>(smem + Sm::dp + j * kSquare + at) = w[j];
                        terms<NO>(da[nt][2 * e] * ma, da[nt][2 * e + 1] * ma, w);
#pragma unroll
                        for (int j = 0; j < NO; ++j) *reinterpret_cast<uint32_t *>(smem + Sm::da + j * kSquare + at) = w[j];
                    }
            }
            __syncthreads();
            if (warp == 0) {
                float dots = 0.0f;
#pragma unroll
                for (int i = 0; i < kGradWarps; ++i) dots += red[kGradWarps + i];
                float x[2], nx[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 2 * lane + e;
                    x[e] = nx[e] = 0.0f;
#pragma unroll
                    for (int j = 0; j < 2; ++j) x[e] += part_row[j * kChunk + i], nx[e] += part_next[j * kChunk + i];
                    float c = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) c += part_col[j * kChunk + i];
                    x[e] -= c;
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
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 2 * lane + e;
                    if (i < rows) {
                        const int64_t at = (first + i) * p.H + head;
                        static_cast<T *>(p.dbeta)[at] = from_f32<T>(part_beta[i]);
                        if (p.dgate) {  // (a decay of 0 has no gradient, whatever the sums' rounding leaves)
                            const float log = i ? (f[F_BHI + i] - f[F_BHI + i - 1]) + (f[F_BLO + i] - f[F_BLO + i - 1]) : f[F_BHI];
                            static_cast<T *>(p.dgate)[at] = from_f32<T>(expf(log) == 0.0f ? 0.0f : sum - (e ? x[0] : 0.0f) + end);
                        }
                    }
                }
            }
            {
                const uint32_t i_dp = base + Sm::dp, i_da = base + Sm::da;
                mp = inverse_of(mp), ma = inverse_of(ma) * ik;
                Acc tq[2 * NQ], tk[2 * NQ], ta[2 * NQ];
                clear(tq), clear(tk), clear(ta);
#pragma unroll
                for (int kb = 0; kb < 4; ++kb) {
                    uint32_t a[NO][4], c[NO][4], e[NO][4];
                    if (kb <= wm) {  // the triangles' rows
#pragma unroll
                        for (int j = 0; j < NO; ++j)
                            left<kChunk>(a[j], i_dp + j * kSquare, 16 * wm, 16 * kb, lane), left<kChunk>(c[j], i_da + j * kSquare, 16 * wm, 16 * kb, lane);
                    }
#pragma unroll
                    for (int i = 0; i < NQ; ++i) {
                        uint32_t x[NI][4];
#pragma unroll
                        for (int j = 0; j < NI; ++j) right_t<KP>(x[j], kimg + j * R::term, 16 * kb, wn * (KP / 2) + 16 * i, lane);
                        if (kb <= wm) {
                            products<T, NO, NI>(tq[2 * i], tq[2 * i + 1], a, x);
                            products<T, NO, NI>(ta[2 * i], ta[2 * i + 1], c, x);
                        }
                        if (kb >= wm) {  // their columns
#pragma unroll
                            for (int j = 0; j < NO; ++j) left_t<kChunk>(e[j], i_da + j * kSquare, 16 * kb, 16 * wm, lane);
                            products<T, NO, NI>(ta[2 * i], ta[2 * i + 1], e, x);
#pragma unroll
                            for (int j = 0; j < NO; ++j) left_t<kChunk>(e[j], i_dp + j * kSquare, 16 * kb, 16 * wm, lane);
#pragma unroll
                            for (int j = 0; j < NI; ++j) right_t<KP>(x[j], qimg + j * R::term, 16 * kb, wn * (KP / 2) + 16 * i, lane);
                            products<T, NO, NI>(tk[2 * i], tk[2 * i + 1], e, x);
                        }
                    }
                }
                add(aq, tq, mp * ik), add(ak, tk, mp * iq), add(ak, ta, ma);
            }
        }
        ++entry;
#pragma unroll
        for (int i = 0; i < 2 * NQ; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = e ? r1 : r0, c = col0 + 8 * i;
                if (row >= rows) continue;
                store_pair(dq + row * row_k, c, p.K, p.K % 2 == 0, aq[i][2 * e], aq[i][2 * e + 1]);
                store_pair(dk + row * row_k, c, p.K, p.K % 2 == 0, ak[i][2 * e], ak[i][2 * e + 1]);
            }
    }
    stages.end();
}

// ------------------------------------------------------------------------------------------------
// One row of each of N sequences whose states lie in a pool. A CTA takes 32 channels of the values of one state (with keys of up to 64 or 32 channels,
// 64 or 128 of them, that it has enough to load: 75 sequences of 24 heads of 32 x 224 23 us instead of 47), all of it in registers: S^T k and S^T q come from one reading of it, with o = scale (a S^T q + (k q) u), so the state is read once and written once. Bound by memory.
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
template <typename T, int VEC, int GROUPS>
__global__ void __launch_bounds__(32 * kStepWarps, 5) based_delta_step_kernel(DeltaStepParams p) {
    // warps of 32 channels, a row's lanes, rows of a pass, passes
    constexpr int kWarps = kStepWarps / GROUPS, kLanes = 32 / VEC, kRows = 32 / kLanes * kWarps, kEach = kMaxKeys / GROUPS / kRows;
    __shared__ float sk[kMaxKeys], sq[kMaxKeys], red[3][kStepWarps][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, head = blockIdx.y, hk = head / (p.H / p.HK);
    const int group = warp / kWarps, c = (blockIdx.x * GROUPS + group) * 32 + lane % kLanes * VEC, row0 = warp % kWarps * (32 / kLanes) + lane / kLanes;
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
        if (warp < GROUPS) {
            float sx = 0.0f, sy = 0.0f, u = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sx += red[0][warp * kWarps + w][lane], sy += red[1][warp * kWarps + w][lane];
            const int col = blockIdx.x * GROUPS * 32 + tid;
            if (col < p.V) {
                u = beta * (to_f32(static_cast<const T *>(p.v)[n * p.v_sn + head * p.v_sh + col]) - sx);
                static_cast<T *>(p.o)[(static_cast<int64_t>(n) * p.H + head) * p.V + col] = from_f32<T>(p.scale * fmaf(kq, u, sy));
            }
            red[2][warp][lane] = u;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = red[2][group][lane % kLanes * VEC + j];
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

// The parts of a workspace, each on 256 bytes, and the bytes that the forward pass saves
struct DeltaSpace {
    size_t qk, g, slices, total, saved;
};
inline int padded_keys(int K) { return K <= 64 ? 64 : 128; }
template <typename T, int KP>
DeltaSpace delta_space(int B, int T_, int H, int HK, int V, bool bwd) {
    const size_t chunks = (static_cast<size_t>(T_) + kChunk - 1) / kChunk, up = 255, slices = chunks * B * H * ((V + kSlice - 1) / kSlice);
    DeltaSpace s;
    s.qk = 0;
    s.g = (s.qk + chunks * B * HK * Rec<T, KP>::qk + up) & ~up;
    s.slices = (s.g + chunks * B * H * Rec<T, KP>::g(bwd) + up) & ~up;
    s.total = bwd ? (s.slices + slices * SliceRec<T, KP>::bwd + up) & ~up : s.slices;
    s.saved = slices * SliceRec<T, KP>::fwd;
    return s;
}
DeltaSpace delta_space(int B, int T, int H, int HK, int K, int V, int dtype, bool bwd) {
    const bool wide = padded_keys(K) == 128;
    if (dtype == BASED_F32) return wide ? delta_space<float, 128>(B, T, H, HK, V, bwd) : delta_space<float, 64>(B, T, H, HK, V, bwd);
    if (dtype == BASED_BF16)
        return wide ? delta_space<__nv_bfloat16, 128>(B, T, H, HK, V, bwd) : delta_space<__nv_bfloat16, 64>(B, T, H, HK, V, bwd);
    return wide ? delta_space<__half, 128>(B, T, H, HK, V, bwd) : delta_space<__half, 64>(B, T, H, HK, V, bwd);
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
    static_assert(Sm::bytes(true, Sm::most(true)) <= 227 * 1024 && Sm::bytes(false, Sm::most(false)) <= 227 * 1024 && GradSmem<T, KP>::bytes <= 227 * 1024,
                  "shared memory of a CTA");
    const int slices = (p.V + kSlice - 1) / kSlice;
    const unsigned z = p.B < kMostGrid ? p.B : kMostGrid;
    void (*const prep)(DeltaParams) = bwd ? based_delta_prep_kernel<T, KP, true> : based_delta_prep_kernel<T, KP, false>;
    OPS_CUDA(allow(prep, PrepSmem<T, KP>::bytes));
    OPS_CUDA(launch_op(prep, dim3(p.chunks, p.HK, z), 32 * kPrepWarps, PrepSmem<T, KP>::bytes, st, p));
    // A CTA's slices share its records but also its SM: as many as take the least time, which is the rounds of CTAs (those of equal lengths end together)
    // by what a round takes: 1, 1.29, 1.57 and 2.09 with one to four slices. 8 x 4096 rows, 16 heads, with one, two, three and four: 128 x 128 bf16 forward 935, 674, 602
    // and 527 us, backward 1132, 816, 723 and 636; f16 1035, 750 and 682 (three fit), 1155, 837 and 746; 64 x 64 bf16 288, 281, 344 and 208, 546, 338, 421 and 253;
    // 4 x 4096 float32 of 64 x 64 286, 184 and 232, 311, 202 and 258. It takes the fastest of each.
    constexpr double kRound[5] = {0.0, 1.0, 1.29, 1.57, 2.09};
    int per = 1;
    const auto cost = [&](int n) {
        const double rounds = static_cast<double>(p.B) * p.H * ((slices + n - 1) / n) / sms;
        return (p.lengths && rounds > 1.0 ? rounds : ceil(rounds)) * kRound[n];
    };
    for (int n = 2; n <= Sm::most(bwd) && n <= slices; ++n)
        if (cost(n) <= cost(per)) per = n;
    void (*const seq)(DeltaParams) = bwd ? based_delta_bwd_kernel<T, KP> : based_delta_fwd_kernel<T, KP>;
    OPS_CUDA(allow(seq, Sm::bytes(bwd, Sm::most(bwd))));
    OPS_CUDA(launch_op(seq, dim3((slices + per - 1) / per, p.H, z), kQuad * per, Sm::bytes(bwd, per), st, p));
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
    if (bwd && (!p.dout || !p.saved || !p.dq || !p.dk || !p.dbeta || !p.gate != !p.dgate)) return BASED_ERR_NULL_POINTER;
    if (!type_ok(dtype)) return BASED_ERR_UNSUPPORTED_TYPE;
    if (!(p.scale == p.scale)) return BASED_ERR_BAD_ARGUMENT;
    const int B = p.B, T = p.T, H = p.H, HK = p.HK, K = p.K, V = p.V;
    if (const int rc = check_delta_sizes(B, T, H, HK, K, V)) return rc;
    p.chunks = (T + kChunk - 1) / kChunk;
    const int64_t strides[] = {p.q_sb, p.q_st, p.q_sh, p.k_sb, p.k_st, p.k_sh, p.v_sb, p.v_st, p.v_sh, p.do_sb, p.do_st, p.do_sh,
                               p.beta_sb, p.beta_st, p.gate_sb, p.gate_st};
    for (const int64_t s : strides)
        if (s < 0) return BASED_ERR_BAD_STRIDE;
    const size_t es = elem_size(dtype);
    const void *const typed[] = {p.q, p.k, p.v, p.beta, p.gate, p.dout, p.out, p.dq, p.dk, p.dbeta, p.dgate};
    for (const void *t : typed)
        if (!aligned(t, es)) return BASED_ERR_MISALIGNED;
    if (!aligned(p.lengths, 4) || !aligned(p.state, 4) || !aligned(p.final_state, 4) || !aligned(p.saved, 16) ||
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
        {span(p.saved, static_cast<int64_t>(space.saved) - 1, 1), !bwd},
        {span(p.out, bth * V - 1, es), true}, {span(p.final_state, states - 1, 4), true},
        {span(p.dq, static_cast<int64_t>(B) * T * HK * K - 1, es), true}, {span(p.dk, static_cast<int64_t>(B) * T * HK * K - 1, es), true},
        {span(p.dbeta, bth - 1, es), true}, {span(p.dgate, bth - 1, es), true}, {span(workspace, static_cast<int64_t>(space.total) - 1, 1), true}};
    if (clash(regions)) return BASED_ERR_ALIASING;
    int sms;
    if (const int rc = host_device(&sms)) return rc;
    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    p.qk_rec = ws + space.qk, p.g_rec = ws + space.g, p.slice_rec = ws + space.slices;
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
inline float delta_scale(float scale, int K) { return !(scale <= 0.0f) || K < 1 ? scale : 1.0f / sqrtf(static_cast<float>(K)); }

template <typename T, int VEC>
int launch_delta_step(const DeltaStepParams &p, cudaStream_t st) {
    const int groups = p.K <= 32 && p.V > 64 ? 4 : p.K <= 64 && p.V > 32 ? 2 : 1;
    void (*const step)(DeltaStepParams) = groups == 4 ? based_delta_step_kernel<T, VEC, 4> : groups == 2 ? based_delta_step_kernel<T, VEC, 2> : based_delta_step_kernel<T, VEC, 1>;
    const dim3 grid((p.V + 32 * groups - 1) / (32 * groups), p.H, p.N < kMostGrid ? p.N : kMostGrid);
    OPS_CUDA(launch_op(step, grid, 32 * kStepWarps, 0, st, p));
    return BASED_OK;
}
template <typename T>
int launch_delta_step(const DeltaStepParams &p, cudaStream_t st) {
    if (p.V % 4 == 0 && aligned(p.pool, 16)) return launch_delta_step<T, 4>(p, st);
    if (p.V % 2 == 0 && aligned(p.pool, 8)) return launch_delta_step<T, 2>(p, st);
    return launch_delta_step<T, 1>(p, st);
}

}  // namespace

cudaError_t delta_status(unsigned int *status, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(status, g_delta_status, sizeof(unsigned int));
    if (e == cudaSuccess && clear && *status) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_delta_status, &zero, sizeof(unsigned int));
    }
    return e;
}
}  // namespace based

extern "C" {

int based_delta_fwd(const void *q, int64_t q_sb, int64_t q_st, int64_t q_sh, const void *k, int64_t k_sb, int64_t k_st, int64_t k_sh, const void *v,
                    int64_t v_sb, int64_t v_st, int64_t v_sh, const void *beta, int64_t beta_sb, int64_t beta_st, const void *gate,
                    int64_t gate_sb, int64_t gate_st, int B, int T, int H, int HK, int K, int V, int dtype, float scale, const float *state,
                    const int32_t *lengths, void *o, float *final_state, void *saved, void *workspace, size_t ws_bytes,
                    based_stream_t stream) {
    based::DeltaParams p = {};
    p.q = q, p.q_sb = q_sb, p.q_st = q_st, p.q_sh = q_sh, p.k = k, p.k_sb = k_sb, p.k_st = k_st, p.k_sh = k_sh;
    p.v = v, p.v_sb = v_sb, p.v_st = v_st, p.v_sh = v_sh, p.beta = beta, p.beta_sb = beta_sb, p.beta_st = beta_st;
    p.gate = gate, p.gate_sb = gate_sb, p.gate_st = gate_st;
    p.B = B, p.T = T, p.H = H, p.HK = HK, p.K = K, p.V = V, p.scale = based::delta_scale(scale, K);
    p.state = state, p.lengths = lengths, p.out = o, p.final_state = final_state, p.saved = static_cast<uint8_t *>(saved);
    return based::run_delta(p, dtype, false, workspace, ws_bytes, stream);
}

int based_delta_bwd(const void *q, int64_t q_sb, int64_t q_st, int64_t q_sh, const void *k, int64_t k_sb, int64_t k_st, int64_t k_sh, const void *v,
                    int64_t v_sb, int64_t v_st, int64_t v_sh, const void *beta, int64_t beta_sb, int64_t beta_st, const void *gate,
                    int64_t gate_sb, int64_t gate_st, const void *dout, int64_t do_sb, int64_t do_st, int64_t do_sh, const void *saved, int B, int T, int H, int HK, int K, int V, int dtype, float scale, const float *dfinal,
                    const int32_t *lengths, void *dq, void *dk, void *dv, void *dbeta, void *dgate, float *dstate, void *workspace,
                    size_t ws_bytes, based_stream_t stream) {
    based::DeltaParams p = {};
    p.q = q, p.q_sb = q_sb, p.q_st = q_st, p.q_sh = q_sh, p.k = k, p.k_sb = k_sb, p.k_st = k_st, p.k_sh = k_sh;
    p.v = v, p.v_sb = v_sb, p.v_st = v_st, p.v_sh = v_sh, p.beta = beta, p.beta_sb = beta_sb, p.beta_st = beta_st;
    p.gate = gate, p.gate_sb = gate_sb, p.gate_st = gate_st, p.dout = dout, p.do_sb = do_sb, p.do_st = do_st, p.do_sh = do_sh;
    p.B = B, p.T = T, p.H = H, p.HK = HK, p.K = K, p.V = V, p.scale = based::delta_scale(scale, K);
    p.state = dfinal, p.lengths = lengths, p.out = dv, p.dq = dq, p.dk = dk, p.dbeta = dbeta, p.dgate = dgate, p.final_state = dstate;
    p.saved = static_cast<uint8_t *>(const_cast<void *>(saved));
    return based::run_delta(p, dtype, true, workspace, ws_bytes, stream);
}

size_t based_delta_workspace_size(int B, int T, int H, int HK, int K, int V, int dtype, int backward) {
    if (based::check_delta_sizes(B, T, H, HK, K, V) != BASED_OK || !based::type_ok(dtype)) return 0;
    return based::delta_space(B, T, H, HK, K, V, dtype, backward != 0).total;
}

size_t based_delta_saved_size(int B, int T, int H, int K, int V, int dtype) {
    if (based::check_delta_sizes(B, T, H, 1, K, V) != BASED_OK || !based::type_ok(dtype)) return 0;
    return based::delta_space(B, T, H, 1, K, V, dtype, false).saved;
}

int based_delta_step(const void *q, int64_t q_sn, int64_t q_sh, const void *k, int64_t k_sn, int64_t k_sh, const void *v, int64_t v_sn, int64_t v_sh,
                     const void *beta, int64_t beta_sn, const void *gate, int64_t gate_sn, int N, int H, int HK, int K, int V, int S, int dtype,
                     float scale, float *pool, const int32_t *slots, void *o, based_stream_t stream) {
    using namespace based;
    if (!q || !k || !v || !beta || !pool || !o) return BASED_ERR_NULL_POINTER;
    if (!type_ok(dtype)) return BASED_ERR_UNSUPPORTED_TYPE;
    if (!(scale == scale)) return BASED_ERR_BAD_ARGUMENT;
    if (check_delta_sizes(N, 1, H, HK, K, V) != BASED_OK || S < 1 || (!slots && S < N) ||
        S > (static_cast<int64_t>(1) << 56) / (static_cast<int64_t>(H) * K * V))
        return BASED_ERR_BAD_SIZE;
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
