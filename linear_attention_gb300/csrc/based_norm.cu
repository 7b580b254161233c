// based_norm.cu: per-token group norm with an activation (declared in include/based_ops.h).
//
//     v = hat w + b,  hat = (x - mean) rstd;    y = v act(z) with a gate z, act(v) without
// backward, with dv = dy act(z) (or dy act'(v)) and q = dv w:
//     dx = rstd (q - mean(q) - hat mean(q hat)),  dz = dy v act'(z),  dw = sum dv hat,  db = sum dv
//
// A group is held by `tpg` neighbouring threads (a power of two), eight channels each, in
// registers: one read of x serves the mean, the squared deviations and the result. Up to 32
// threads reduce by shuffles; larger groups take a whole CTA. A CTA keeps its channels and walks
// over rows, so that weights are loaded once and their gradients add up in registers. At 24000 x 1536 in 12
// groups (bf16, gated) the forward pass takes 40 us, 83 % of the floor of its reads and writes, bound by
// the latency of the loads (one row ahead, 30 warps an SM); the backward pass 67 us, 82 %, with the issue slots
// 60 % busy and 6 us for the column sums.
#include <type_traits>

#include "ops_common.cuh"

namespace based {
namespace {

constexpr int kMaxGroup = 4096;  // channels of a group: 512 threads x 8
constexpr int kElems = 8;        // channels of a thread

struct NormParams {
    const void *x, *gate, *dy, *weight, *bias;
    int64_t x_sr, gate_sr, dy_sr, R;
    int C, G, Cg;
    int tpg, gpb, rp;  // threads of a group; groups and rows side by side in a CTA
    int p_dtype, act;
    float eps;
    void *y, *dx, *dgate;
    float *partial;  // (gridDim.x, 2, C): the CTAs' sums for dweight and dbias
};

__device__ __forceinline__ float load_param(const void *p, int dtype, int i, float none) {
    if (!p) return none;
    if (dtype == BASED_F32) return static_cast<const float *>(p)[i];
    if (dtype == BASED_BF16) return to_f32(static_cast<const __nv_bfloat16 *>(p)[i]);
    return to_f32(static_cast<const __half *>(p)[i]);
}

// Eight channels of a row, by what lies in a word. kOctets: consecutive ones, loaded as 16-byte words. kPairs:
// pairs of neighbours, tpg pairs apart. kSingles: channels l, l + tpg, ... of the group.
// `held`: a bit for each that the thread holds. A load leaves what the thread does not hold as it
// is (zero from clear()).
enum Words { kSingles, kPairs, kOctets };
template <typename T, Words W>
struct Row;
template <typename T>
struct Row<T, kOctets> {
    static constexpr int kQuads = sizeof(T) * kElems / 16;
    uint32_t w[kQuads * 4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < 4 * kQuads; ++k) w[k] = 0;
    }
    // ONCE: the data is not kept in L2 over what others read again
    template <bool ONCE>
    __device__ __forceinline__ void load(const T *p, unsigned held, int) {
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
            if (!held) continue;
            const uint4 *at = reinterpret_cast<const uint4 *>(p) + k, q = ONCE ? __ldcs(at) : *at;
            w[4 * k] = q.x, w[4 * k + 1] = q.y, w[4 * k + 2] = q.z, w[4 * k + 3] = q.w;
        }
    }
    __device__ __forceinline__ void store(T *p, unsigned held, int) const {
#pragma unroll
        for (int k = 0; k < kQuads; ++k)
            if (held) reinterpret_cast<uint4 *>(p)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
    __device__ __forceinline__ void keep(unsigned) {}
    __device__ __forceinline__ Vec<2> get(int k) const {
        if constexpr (sizeof(T) == 4)
            return {{__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1])}};
        else
            return unpack<T>(w[k]);
    }
    __device__ __forceinline__ void set(int k, const Vec<2> &v) {
        if constexpr (sizeof(T) == 4)
            w[2 * k] = __float_as_uint(v.v[0]), w[2 * k + 1] = __float_as_uint(v.v[1]);
        else
            w[k] = pack<T>(v);
    }
};
// A pair at the start or the end of a group may have one half in the next group. It is loaded whole, as the row goes
// on there, and keep() clears the half; a store leaves it alone.
template <typename T>
struct Row<T, kPairs> {
    static constexpr int kPairWords = sizeof(T) / 2;
    uint32_t w[kElems / 2 * kPairWords];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < kElems / 2 * kPairWords; ++k) w[k] = 0;
    }
    template <bool ONCE>
    __device__ __forceinline__ void load(const T *p, unsigned held, int tpg) {
#pragma unroll
        for (int k = 0; k < kElems / 2; ++k) {
            if (!(held >> (2 * k) & 3)) continue;
            const T *from = p + k * 2 * tpg;
            if constexpr (sizeof(T) == 4) {
                const uint2 q = *reinterpret_cast<const uint2 *>(from);
                w[2 * k] = q.x, w[2 * k + 1] = q.y;
            } else {
                w[k] = *reinterpret_cast<const uint32_t *>(from);
            }
        }
    }
    __device__ __forceinline__ void keep(unsigned held) {
#pragma unroll
        for (int k = 0; k < kElems / 2; ++k) {
            if constexpr (sizeof(T) == 4) {
                if (!(held >> (2 * k) & 1)) w[2 * k] = 0;
                if (!(held >> (2 * k) & 2)) w[2 * k + 1] = 0;
            } else {
                if (!(held >> (2 * k) & 1)) w[k] &= 0xffff0000u;
                if (!(held >> (2 * k) & 2)) w[k] &= 0xffffu;
            }
        }
    }
    __device__ __forceinline__ void store(T *p, unsigned held, int tpg) const {
#pragma unroll
        for (int k = 0; k < kElems / 2; ++k) {
            const unsigned both = held >> (2 * k) & 3;
            T *to = p + k * 2 * tpg;
            if constexpr (sizeof(T) == 4) {
                if (both == 3)
                    *reinterpret_cast<uint2 *>(to) = make_uint2(w[2 * k], w[2 * k + 1]);
                else if (both)
                    *reinterpret_cast<uint32_t *>(to + (both >> 1)) = both & 1 ? w[2 * k] : w[2 * k + 1];
            } else {
                if (both == 3)
                    *reinterpret_cast<uint32_t *>(to) = w[k];
                else if (both)
                    *reinterpret_cast<uint16_t *>(to + (both >> 1)) = static_cast<uint16_t>(both & 1 ? w[k] : w[k] >> 16);
            }
        }
    }
    __device__ __forceinline__ Vec<2> get(int k) const {
        if constexpr (sizeof(T) == 4)
            return {{__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1])}};
        else
            return unpack<T>(w[k]);
    }
    __device__ __forceinline__ void set(int k, const Vec<2> &v) {
        if constexpr (sizeof(T) == 4)
            w[2 * k] = __float_as_uint(v.v[0]), w[2 * k + 1] = __float_as_uint(v.v[1]);
        else
            w[k] = pack<T>(v);
    }
};
template <typename T>
struct Row<T, kSingles> {
    T w[kElems];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < kElems; ++k) w[k] = from_f32<T>(0.0f);
    }
    template <bool ONCE>
    __device__ __forceinline__ void load(const T *p, unsigned held, int tpg) {
#pragma unroll
        for (int k = 0; k < kElems; ++k)
            if (held >> k & 1) w[k] = p[k * tpg];
    }
    __device__ __forceinline__ void keep(unsigned) {}
    __device__ __forceinline__ void store(T *p, unsigned held, int tpg) const {
#pragma unroll
        for (int k = 0; k < kElems; ++k)
            if (held >> k & 1) p[k * tpg] = w[k];
    }
    __device__ __forceinline__ Vec<2> get(int k) const { return {{to_f32(w[2 * k]), to_f32(w[2 * k + 1])}}; }
    __device__ __forceinline__ void set(int k, const Vec<2> &v) {
        w[2 * k] = from_f32<T>(v.v[0]);
        w[2 * k + 1] = from_f32<T>(v.v[1]);
    }
};

// Sums of K values over the threads of a group. BIG: groups may span warps (then they are the whole
// CTA); `red` holds 16 K floats, and calls in a row use different ones.
template <int K, bool BIG>
__device__ __forceinline__ void group_sum(float (&v)[K], int tpg, float *red) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        if (tpg <= d) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(~0u, v[k], d);
    }
    if (!BIG || tpg <= 32) return;
    const int warps = tpg >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) red[k * 16 + (threadIdx.x >> 5)] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        v[k] = 0.0f;
        for (int w = 0; w < warps; ++w) v[k] += red[k * 16 + w];
    }
}
__device__ __forceinline__ float total(const Vec<2> (&v)[kElems / 2]) {
    const Vec<2> s = vadd(vadd(v[0], v[1]), vadd(v[2], v[3]));
    return s.v[0] + s.v[1];
}

// act(v) and act'(v)
template <int ACT>
__device__ __forceinline__ void activate(Vec<2> v, Vec<2> &f, Vec<2> &df) {
    if (ACT == BASED_ACT_NONE) {
        f = v, df = splat<2>(1.0f);
        return;
    }
    Vec<2> s, t;
    vsigmoid(v, s, t);  // v is -87 at least: a type's lowest value times the smallest sigma is far from 0
    if (ACT == BASED_ACT_SIGMOID)
        f = s, df = vmul(s, t);
    else
        f = vmul(v, s), df = vfma(f, t, s);
}

// f with the activation as a compile-time constant
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
    if (act == BASED_ACT_SILU)
        f(std::integral_constant<int, BASED_ACT_SILU>());
    else if (act == BASED_ACT_SIGMOID)
        f(std::integral_constant<int, BASED_ACT_SIGMOID>());
    else
        f(std::integral_constant<int, BASED_ACT_NONE>());
}

// Registers: the forward kernel fits 64, the backward kernel, which also holds the sums for dweight
// and dbias, 80 (100 where x is float32): weight and bias wait in shared memory, four 16-byte reads a
// row. By pairs and singles they take up to 85 and 128. BIG ones may have 512 threads.
constexpr int norm_threads(Words w, bool bwd, bool big) { return big ? 512 : w == kOctets && bwd ? 128 : 256; }
constexpr int norm_ctas(Words w, bool bwd, bool big, bool x32) {
    return big ? 1 : w == kOctets ? (bwd ? (x32 ? 5 : 6) : 4) : (bwd ? 2 : 3);
}
template <typename TX, typename TY, Words W, bool GATED, bool BWD, bool BIG>
__global__ void __launch_bounds__(norm_threads(W, BWD, BIG), norm_ctas(W, BWD, BIG, sizeof(TX) == 4))
    based_norm_kernel(const NormParams p) {
    constexpr int P = kElems / 2;
    constexpr bool VEC = W == kOctets;
    extern __shared__ __align__(16) float smem[];
    const int slot = threadIdx.x / p.tpg, l = threadIdx.x % p.tpg;
    const int r = slot / p.gpb, g = blockIdx.y * p.gpb + slot % p.gpb;
    const int per = p.gpb * p.tpg;
    const bool on = r < p.rp && g < p.G;
    // pairs start on even channels: in a group that starts on an odd one with the channel before it
    const int first = W == kOctets ? l * kElems : W == kPairs ? 2 * l - (g * p.Cg & 1) : l;
    auto place = [&](int i) { return W == kOctets ? i : W == kPairs ? i / 2 * 2 * p.tpg + i % 2 : i * p.tpg; };
    unsigned held = 0;
#pragma unroll
    for (int i = 0; i < kElems; ++i)
        if (on && first + place(i) >= 0 && first + place(i) < p.Cg) held |= 1u << i;
    const int64_t c = static_cast<int64_t>(g) * p.Cg + first;
    const float inv = 1.0f / p.Cg;
    griddep_wait();
    griddep_launch_dependents();
    // (4, per) quads: elements 0-3 and 4-7 of the weights, then of the biases, of a row's threads
    float4 *params = reinterpret_cast<float4 *>(smem + 64);
    const float4 *mine = params + threadIdx.x % per;
    if (r == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = (q & 1) * 4 + j, o = static_cast<int>(c) + place(i);
                v[j] = held >> i & 1 ? load_param(q < 2 ? p.weight : p.bias, p.p_dtype, o, q < 2 ? 1.0f : 0.0f) : 0.0f;
            }
            params[q * per + threadIdx.x] = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
    Vec<2> dw[P], db[P];
#pragma unroll
    for (int k = 0; k < P; ++k) dw[k] = db[k] = splat<2>(0.0f);
    // the next row is loaded while a row is worked on
    Row<TX, W> nx;
    Row<TY, W> nz, nd;
    nx.clear(), nz.clear(), nd.clear();
    const int64_t turn = static_cast<int64_t>(gridDim.x) * p.rp;
    int64_t row = static_cast<int64_t>(blockIdx.x) * p.rp + r;
    const TX *px = static_cast<const TX *>(p.x) + row * p.x_sr + c;
    const TY *pz = static_cast<const TY *>(p.gate) + row * p.gate_sr + c;
    const TY *pd = static_cast<const TY *>(p.dy) + row * p.dy_sr + c;
    int64_t out = row * p.C + c;
    // past the last row the registers keep an earlier one
    auto fetch = [&] {
        const unsigned m = row < p.R ? held : 0;
        // streaming loads forward (16384 x 1024, float32 in: 23.3 to 18.7 us), ordinary ones backward (they
        // take 67 us there, streaming ones 69)
        nx.template load<!BWD>(px, m, p.tpg);
        if (GATED) nz.template load<!BWD>(pz, m, p.tpg);
        if (BWD) nd.template load<!BWD>(pd, m, p.tpg);
    };
    fetch();
    __syncthreads();
    // every thread takes part in the sums of every turn: the bound is the CTA's first row
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * p.rp; base < p.R; base += turn) {
        Row<TX, W> rx = nx;
        Row<TY, W> rz, rd;
        if (GATED) rz = nz;
        if (BWD) rd = nd;
        const unsigned mh = row < p.R ? held : 0;
        rx.keep(held);
        if (GATED) rz.keep(held);
        if (BWD) rd.keep(held);
        row += turn;
        px += turn * p.x_sr, pz += turn * p.gate_sr, pd += turn * p.dy_sr;
        fetch();
        if (BWD && !mh) {  // adds nothing to dweight and dbias, whatever the earlier row's gate was
            rd.clear();
            if (GATED) rz.clear();
        }
        Vec<2> h[P], sq[P];
#pragma unroll
        for (int k = 0; k < P; ++k) h[k] = rx.get(k);
        float s1[1] = {total(h)};
        group_sum<1, BIG>(s1, p.tpg, smem);
        const Vec<2> mean = splat<2>(-s1[0] * inv);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            h[k] = vadd(h[k], mean);
            if (!VEC) {
                if (!(mh >> (2 * k) & 1)) h[k].v[0] = 0.0f;
                if (!(mh >> (2 * k) & 2)) h[k].v[1] = 0.0f;
            }
            sq[k] = vmul(h[k], h[k]);
        }
        float s2[1] = {total(sq)};
        if (VEC && !mh) s2[0] = 0.0f;
        group_sum<1, BIG>(s2, p.tpg, smem + 16);
        // a thread without channels scales by 0, so that nothing it adds to a sum is NaN where eps is 0
        const float rstd = mh ? rsqrtf(fmaf(s2[0], inv, p.eps)) : 0.0f;
        auto param = [&](int k, int which) {  // pair k of the weights (0) or biases (1)
            const float4 q = mine[(2 * which + k / 2) * per];
            return k % 2 ? Vec<2>{{q.z, q.w}} : Vec<2>{{q.x, q.y}};
        };
        if (!BWD) {
            Row<TY, W> ry;
            with_act(p.act, [&](auto act) {
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const Vec<2> v = vfma(vmul(h[k], splat<2>(rstd)), param(k, 0), param(k, 1));
                    Vec<2> f, df;
                    activate<decltype(act)::value>(GATED ? rz.get(k) : v, f, df);
                    ry.set(k, GATED ? vmul(v, f) : f);
                }
            });
            ry.store(static_cast<TY *>(p.y) + out, mh, p.tpg);
        } else {
            Row<TY, W> oz;
            Row<TX, W> ox;
            Vec<2> q[P], s0 = splat<2>(0.0f), sh = splat<2>(0.0f);
            with_act(p.act, [&](auto act) {
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    h[k] = vmul(h[k], splat<2>(rstd));
                    const Vec<2> w = param(k, 0), v = vfma(h[k], w, param(k, 1)), d = rd.get(k);
                    Vec<2> f, df;
                    activate<decltype(act)::value>(GATED ? rz.get(k) : v, f, df);
                    const Vec<2> dv = vmul(d, GATED ? f : df);
                    if (GATED) oz.set(k, vmul(vmul(d, v), df));
                    dw[k] = vfma(dv, h[k], dw[k]);
                    db[k] = vadd(db[k], dv);
                    q[k] = vmul(dv, w);
                    s0 = vadd(s0, q[k]);
                    sh = vfma(q[k], h[k], sh);
                }
            });
            if (GATED) oz.store(static_cast<TY *>(p.dgate) + out, mh, p.tpg);
            float s[2] = {s0.v[0] + s0.v[1], sh.v[0] + sh.v[1]};
            group_sum<2, BIG>(s, p.tpg, smem + 32);
            const Vec<2> m0 = splat<2>(-s[0] * inv), m1 = splat<2>(-s[1] * inv), scale = splat<2>(rstd);
#pragma unroll
            for (int k = 0; k < P; ++k) ox.set(k, vmul(scale, vfma(h[k], m1, vadd(q[k], m0))));
            ox.store(static_cast<TX *>(p.dx) + out, mh, p.tpg);
        }
        out += turn * p.C;
    }
    if (BWD && p.partial) {
        // the CTA's rows side by side are added in shared memory, in order
        float *part = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.C;
        Vec<2> *sum = reinterpret_cast<Vec<2> *>(params + 4 * per);
        for (int k = 1; k < p.rp; ++k) {
            __syncthreads();
            if (r == k && on) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    sum[(i * 2) * per + threadIdx.x % per] = dw[i];
                    sum[(i * 2 + 1) * per + threadIdx.x % per] = db[i];
                }
            }
            __syncthreads();
            if (r == 0 && on) {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    dw[i] = vadd(dw[i], sum[(i * 2) * per + threadIdx.x]);
                    db[i] = vadd(db[i], sum[(i * 2 + 1) * per + threadIdx.x]);
                }
            }
        }
        if (r == 0) {
#pragma unroll
            for (int i = 0; i < kElems; ++i) {
                const int o = place(i);
                if (held >> i & 1) {
                    part[c + o] = dw[i / 2].v[i % 2];
                    part[p.C + c + o] = db[i / 2].v[i % 2];
                }
            }
        }
    }
}

struct NormSumParams {
    const float *partial;
    int parts, C, p_dtype;
    void *dweight, *dbias;
};

// dweight and dbias from the CTAs' sums: 32 columns a CTA, one row of partial sums a warp.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) based_norm_sum_kernel(const NormSumParams p) {
    __shared__ float red[kSumWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;  // 0 .. 2 C - 1: dweight, then dbias
    griddep_wait();
    griddep_launch_dependents();
    float s = 0.0f;
    // loads under way at once: the sums of 640 CTAs in one go (608 at 24000 x 1536); others, up to eight CTAs an SM of
    // 96 threads, take two
    constexpr int kAhead = 20;
    for (int k0 = warp; k0 < p.parts && c < 2 * p.C; k0 += kAhead * kSumWarps) {
        float v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int k = k0 + i * kSumWarps;
            v[i] = k < p.parts ? p.partial[static_cast<int64_t>(k) * 2 * p.C + c] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) s += v[i];
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= 2 * p.C) return;
    for (int w = 1; w < kSumWarps; ++w) s += red[w][lane];
    void *out = c < p.C ? p.dweight : p.dbias;
    const int o = c < p.C ? c : c - p.C;
    if (!out) return;
    if (p.p_dtype == BASED_F32)
        static_cast<float *>(out)[o] = s;
    else if (p.p_dtype == BASED_BF16)
        static_cast<__nv_bfloat16 *>(out)[o] = from_f32<__nv_bfloat16>(s);
    else
        static_cast<__half *>(out)[o] = from_f32<__half>(s);
}

// How a launch lays groups on threads and rows on CTAs.
struct NormShape {
    int tpg, gpb, rp, threads, grid_x, grid_y;
};
NormShape norm_shape(int64_t R, int C, int G, int sms, bool bwd, bool vec, bool x32) {
    NormShape s;
    const int per = (C / G + kElems - 1) / kElems;
    for (s.tpg = 1; s.tpg < per;) s.tpg *= 2;
    if (s.tpg > 32) {
        s.gpb = s.rp = 1;
        s.threads = s.tpg;
    } else {
        // columns in blocks of about equal width, rows side by side where one block is narrow
        const int limit = bwd && vec ? 128 : 256, blocks = (G * s.tpg + limit - 1) / limit;
        s.gpb = (G + blocks - 1) / blocks;
        s.rp = limit / (s.gpb * s.tpg);
        s.threads = (s.gpb * s.rp * s.tpg + 31) / 32 * 32;
    }
    s.grid_y = (G + s.gpb - 1) / s.gpb;
    // as many CTAs as are resident at once, in whole turns over the column blocks, by what groups of up to 256
    // channels hold. Larger groups' kernels take up to 128 registers, and a half-empty last wave (16384 x 2048 in one
    // group: 32 us forward and 86 us backward, of 20 and 30 at the memory's rate).
    const int held = vec ? (bwd ? (x32 ? 640 : 768) : 1024) : (bwd ? 512 : 768);
    const int resident = sms * (held / s.threads > 1 ? held / s.threads : 1);
    const int64_t turns = (R + s.rp - 1) / s.rp, most = resident / s.grid_y > 1 ? resident / s.grid_y : 1;
    s.grid_x = static_cast<int>(turns < most ? turns : most);
    return s;
}

bool norm_sizes_ok(int64_t R, int C, int G) {
    return R >= 1 && R < (1ll << 40) && C >= 1 && C <= (1 << 20) && G >= 1 && C % G == 0 && C / G <= kMaxGroup;
}

int check_norm(const NormParams &p, int x_dtype, int dtype, bool bwd, const void *dweight, const void *dbias) {
    if (!p.x || (bwd ? (!p.dy || !p.dx || !p.dgate != !p.gate) : !p.y)) return BASED_ERR_NULL_POINTER;
    if (!type_ok(x_dtype) || !type_ok(dtype) || !type_ok(p.p_dtype) || (x_dtype != BASED_F32 && x_dtype != dtype))
        return BASED_ERR_UNSUPPORTED_TYPE;
    if (p.act != BASED_ACT_NONE && p.act != BASED_ACT_SILU && p.act != BASED_ACT_SIGMOID) return BASED_ERR_BAD_ARGUMENT;
    if (!(p.eps >= 0.0f)) return BASED_ERR_BAD_ARGUMENT;
    if (!norm_sizes_ok(p.R, p.C, p.G)) return BASED_ERR_BAD_SIZE;
    if (p.x_sr < 0 || p.gate_sr < 0 || p.dy_sr < 0) return BASED_ERR_BAD_STRIDE;
    const size_t xs = elem_size(x_dtype), es = elem_size(dtype), ps = elem_size(p.p_dtype);
    if (!aligned(p.x, xs) || !aligned(p.dx, xs) || !aligned(p.gate, es) || !aligned(p.dy, es) || !aligned(p.y, es) ||
        !aligned(p.dgate, es) || !aligned(p.weight, ps) || !aligned(p.bias, ps) || !aligned(dweight, ps) ||
        !aligned(dbias, ps))
        return BASED_ERR_MISALIGNED;
    auto rows = [&](const void *q, int64_t sr, size_t e) { return span(q, (p.R - 1) * sr + p.C - 1, e); };
    const Span in[] = {rows(p.x, p.x_sr, xs), rows(p.gate, p.gate_sr, es), rows(p.dy, p.dy_sr, es),
                       span(p.weight, p.C - 1, ps), span(p.bias, p.C - 1, ps)};
    const Span out[] = {rows(p.y, p.C, es), rows(p.dx, p.C, xs), rows(p.dgate, p.C, es), span(dweight, p.C - 1, ps),
                        span(dbias, p.C - 1, ps)};
    for (int i = 0; i < 5; ++i) {
        for (int k = 0; k < 5; ++k) {
            // y over the whole of x or of the gate: a thread reads its channels of a row before it writes them
            if (i == 0 && ((k == 0 && p.y == p.x && xs == es && p.x_sr == p.C) ||
                           (k == 1 && p.y == p.gate && p.gate_sr == p.C)))
                continue;
            if (overlap(out[i], in[k])) return BASED_ERR_ALIASING;
        }
        for (int k = 0; k < i; ++k)
            if (overlap(out[i], out[k])) return BASED_ERR_ALIASING;
    }
    return BASED_OK;
}

template <typename TX, typename TY, bool BWD, Words W>
int launch_norm(const NormParams &p, const NormShape &s, cudaStream_t st) {
    const dim3 grid(s.grid_x, s.grid_y);
    // the sums' 64 floats, weight and bias, and where rows lie side by side their dweight and dbias
    const size_t smem = (64 + (BWD && s.rp > 1 ? 4 : 2) * kElems * s.gpb * s.tpg) * sizeof(float);
    void (*kernel)(NormParams);
    if (s.tpg > 32)
        kernel = p.gate ? based_norm_kernel<TX, TY, W, true, BWD, true> : based_norm_kernel<TX, TY, W, false, BWD, true>;
    else
        kernel = p.gate ? based_norm_kernel<TX, TY, W, true, BWD, false> : based_norm_kernel<TX, TY, W, false, BWD, false>;
    OPS_CUDA(launch_op(kernel, grid, s.threads, smem, st, p));
    return BASED_OK;
}
template <typename TX, typename TY, bool BWD>
int launch_norm(const NormParams &p, const NormShape &s, Words w, cudaStream_t st) {
    if (w == kOctets) return launch_norm<TX, TY, BWD, kOctets>(p, s, st);
    if (w == kPairs) return launch_norm<TX, TY, BWD, kPairs>(p, s, st);
    return launch_norm<TX, TY, BWD, kSingles>(p, s, st);
}

template <bool BWD>
int dispatch_norm(const NormParams &p, const NormShape &s, Words w, int x_dtype, int dtype, cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (x_dtype == BASED_F32) {
        if (dtype == BASED_F32) return launch_norm<float, float, BWD>(p, s, w, st);
        if (dtype == BASED_BF16) return launch_norm<float, bf, BWD>(p, s, w, st);
        return launch_norm<float, __half, BWD>(p, s, w, st);
    }
    if (dtype == BASED_BF16) return launch_norm<bf, bf, BWD>(p, s, w, st);
    return launch_norm<__half, __half, BWD>(p, s, w, st);
}

NormParams norm_params(const void *x, int64_t x_sr, const void *gate, int64_t gate_sr, const void *weight,
                       const void *bias, int p_dtype, int64_t R, int C, int G, float eps, int act) {
    NormParams p = {};
    p.x = x, p.x_sr = x_sr, p.gate = gate, p.gate_sr = gate ? gate_sr : 0;
    p.weight = weight, p.bias = bias, p.p_dtype = p_dtype;
    p.R = R, p.C = C, p.G = G, p.eps = eps, p.act = act;
    return p;
}

// The widest words on which every group of every row starts (pairs: on, or on the second half of one).
// 24000 x 1536 in 12 groups takes 40 us forward and 66 us backward by octets, 63 and 117 by singles; 24000 x 1500,
// whose groups of 125 start on even and odd channels, 57 and 105 by pairs, 65 and 119 by singles.
Words row_words(const NormParams &p, int x_dtype, int dtype) {
    const size_t xs = elem_size(x_dtype), es = elem_size(dtype);
    auto on = [&](size_t x_bytes, size_t bytes) {
        auto row = [](const void *q, int64_t sr, size_t e, size_t b) { return !q || (aligned(q, b) && sr * e % b == 0); };
        return row(p.x, p.x_sr, xs, x_bytes) && row(p.gate, p.gate_sr, es, bytes) && row(p.dy, p.dy_sr, es, bytes) &&
               row(p.y, p.C, es, bytes) && row(p.dx, p.C, xs, x_bytes) && row(p.dgate, p.C, es, bytes);
    };
    return p.C / p.G % kElems == 0 && on(16, 16) ? kOctets : on(2 * xs, 2 * es) ? kPairs : kSingles;
}

void place(NormParams &p, const NormShape &s) {
    p.Cg = p.C / p.G;
    p.tpg = s.tpg, p.gpb = s.gpb, p.rp = s.rp;
}

}  // namespace
}  // namespace based

extern "C" {

int based_norm_fwd(const void *x, int64_t x_sr, int x_dtype, const void *gate, int64_t gate_sr, const void *weight,
                   const void *bias, int p_dtype, int64_t R, int C, int G, float eps, int act, void *y, int dtype,
                   based_stream_t stream) {
    using namespace based;
    NormParams p = norm_params(x, x_sr, gate, gate_sr, weight, bias, p_dtype, R, C, G, eps, act);
    p.y = y;
    int sms, rc = check_norm(p, x_dtype, dtype, false, nullptr, nullptr);
    if (rc != BASED_OK || (rc = host_device(&sms)) != BASED_OK) return rc;
    const Words w = row_words(p, x_dtype, dtype);
    const NormShape s = norm_shape(R, C, G, sms, false, w == kOctets, x_dtype == BASED_F32);
    place(p, s);
    return dispatch_norm<false>(p, s, w, x_dtype, dtype, reinterpret_cast<cudaStream_t>(stream));
}

size_t based_norm_bwd_workspace_size(int64_t R, int C, int G) {
    int sms;
    if (!based::norm_sizes_ok(R, C, G) || based::host_device(&sms) != BASED_OK) return 0;
    // the most that any alignment and type takes
    int parts = 0;
    for (int k = 0; k < 4; ++k) {
        const int n = based::norm_shape(R, C, G, sms, true, k & 1, k & 2).grid_x;
        parts = n > parts ? n : parts;
    }
    return static_cast<size_t>(parts) * 2 * C * sizeof(float);
}

int based_norm_bwd(const void *dy, int64_t dy_sr, const void *x, int64_t x_sr, int x_dtype, const void *gate,
                   int64_t gate_sr, const void *weight, const void *bias, int p_dtype, int64_t R, int C, int G,
                   float eps, int act, void *dx, void *dgate, void *dweight, void *dbias, int dtype, void *workspace,
                   size_t ws_bytes, based_stream_t stream) {
    using namespace based;
    NormParams p = norm_params(x, x_sr, gate, gate_sr, weight, bias, p_dtype, R, C, G, eps, act);
    p.dy = dy, p.dy_sr = dy_sr, p.dx = dx, p.dgate = dgate;
    int sms, rc = check_norm(p, x_dtype, dtype, true, dweight, dbias);
    if (rc != BASED_OK || (rc = host_device(&sms)) != BASED_OK) return rc;
    const Words w = row_words(p, x_dtype, dtype);
    const NormShape s = norm_shape(R, C, G, sms, true, w == kOctets, x_dtype == BASED_F32);
    place(p, s);
    const bool sums = dweight || dbias;
    if (sums) {
        if (!workspace || !aligned(workspace, 16) || ws_bytes < static_cast<size_t>(s.grid_x) * 2 * C * sizeof(float))
            return BASED_ERR_WORKSPACE;
        const size_t xs = elem_size(x_dtype), es = elem_size(dtype), ps = elem_size(p_dtype);
        const Span sw = span(workspace, static_cast<int64_t>(s.grid_x) * 2 * C - 1, sizeof(float));
        const Span all[] = {span(x, (R - 1) * x_sr + C - 1, xs),   span(gate, (R - 1) * p.gate_sr + C - 1, es),
                            span(dy, (R - 1) * dy_sr + C - 1, es), span(dx, R * C - 1, xs),
                            span(dgate, R * C - 1, es),            span(weight, C - 1, ps),
                            span(bias, C - 1, ps),                 span(dweight, C - 1, ps),
                            span(dbias, C - 1, ps)};
        for (const Span &t : all)
            if (overlap(sw, t)) return BASED_ERR_ALIASING;
        p.partial = static_cast<float *>(workspace);
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((rc = dispatch_norm<true>(p, s, w, x_dtype, dtype, st)) != BASED_OK || !sums) return rc;
    const NormSumParams q = {p.partial, s.grid_x, C, p_dtype, dweight, dbias};
    OPS_CUDA(launch_op(based_norm_sum_kernel, dim3((2 * C + 31) / 32), 32 * kSumWarps, 0, st, q));
    return BASED_OK;
}

}  // extern "C"
