// based_norm.cu: per-token group norm with an activation (declared in include/based_ops.h).
//
//     v = hat w + b,  hat = (x - mean) rstd;    y = v act(z) with a gate z, act(v) without
// backward, with dv = dy act(z) (or dy act'(v)) and q = dv w:
//     dx = rstd (q - mean(q) - hat mean(q hat)),  dz = dy v act'(z),  dw = sum dv hat,  db = sum dv
//
// A group is held by `tpg` neighbouring threads (a power of two), eight channels each, in
// registers: one read of x serves the mean, the squared deviations and the result. Up to 32
// threads reduce by shuffles; larger groups take a whole CTA. A CTA keeps its channels and walks
// over rows, so that weights are loaded once and their gradients add up in registers.
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

// Eight channels of a row. VEC: consecutive ones, loaded as 16-byte words; otherwise channels
// l, l + tpg, ... of the group. n: the channels of the group from this thread's first on.
template <typename T, bool VEC>
struct Row {
    static constexpr int kPer = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;  // channels of a word
    using Word = Pack<T, kPer>;
    Word w[kElems / kPer];
    __device__ __forceinline__ void load(const T *p, int n, int step) {
#pragma unroll
        for (int k = 0; k < kElems / kPer; ++k)
            if (VEC ? n > 0 : k * step < n) w[k] = *reinterpret_cast<const Word *>(p + k * (VEC ? kPer : step));
    }
    __device__ __forceinline__ void store(T *p, int n, int step) const {
#pragma unroll
        for (int k = 0; k < kElems / kPer; ++k)
            if (VEC ? n > 0 : k * step < n) *reinterpret_cast<Word *>(p + k * (VEC ? kPer : step)) = w[k];
    }
    __device__ __forceinline__ T &at(int i) { return w[i / kPer].v[i % kPer]; }
};

// Sums of K values over the threads of a group. For groups of more than a warp, `red` holds
// 16 K floats, and calls in a row use different ones.
template <int K>
__device__ __forceinline__ void group_sum(float (&v)[K], int tpg, float *red) {
    for (int d = min(tpg, 32) >> 1; d > 0; d >>= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(~0u, v[k], d);
    }
    if (tpg <= 32) return;
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

// act(v) and act'(v)
__device__ __forceinline__ void activate(int act, float v, float &f, float &df) {
    if (act == BASED_ACT_NONE) {
        f = v, df = 1.0f;
        return;
    }
    float s, t;
    sigmoid_pair(v, s, t);
    if (act == BASED_ACT_SIGMOID)
        f = s, df = s * t;
    else
        f = v * s, df = fmaf(f, t, s);
}

template <typename TX, typename TY, bool VEC, bool GATED, bool BWD>
__global__ void __launch_bounds__(512) based_norm_kernel(const NormParams p) {
    extern __shared__ float smem[];
    const int slot = threadIdx.x / p.tpg, l = threadIdx.x % p.tpg;
    const int r = slot / p.gpb, g = blockIdx.y * p.gpb + slot % p.gpb;
    const int first = VEC ? l * kElems : l, step = p.tpg;
    const bool on = r < p.rp && g < p.G;
    const int n = on ? p.Cg - first : 0;  // > 0: this thread holds channels
    const int64_t c = static_cast<int64_t>(g) * p.Cg + first;
    const float inv = 1.0f / p.Cg;
    griddep_wait();
    griddep_launch_dependents();
    float w[kElems], b[kElems], dw[kElems], db[kElems];
    bool in[kElems];
#pragma unroll
    for (int i = 0; i < kElems; ++i) {
        const int o = VEC ? i : i * step;
        in[i] = VEC ? n > 0 : o < n;
        w[i] = in[i] ? load_param(p.weight, p.p_dtype, static_cast<int>(c) + o, 1.0f) : 0.0f;
        b[i] = in[i] ? load_param(p.bias, p.p_dtype, static_cast<int>(c) + o, 0.0f) : 0.0f;
        dw[i] = db[i] = 0.0f;
    }
    // every thread takes part in the sums of every turn: the bound is the CTA's first row
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * p.rp; base < p.R; base += static_cast<int64_t>(gridDim.x) * p.rp) {
        const int64_t row = base + r;
        const int m = row < p.R ? n : 0;
        Row<TX, VEC> rx;
        Row<TY, VEC> rz, rd;
        rx.load(static_cast<const TX *>(p.x) + row * p.x_sr + c, m, step);
        if (GATED) rz.load(static_cast<const TY *>(p.gate) + row * p.gate_sr + c, m, step);
        if (BWD) rd.load(static_cast<const TY *>(p.dy) + row * p.dy_sr + c, m, step);
        float h[kElems];
        float s1[1] = {0.0f}, s2[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < kElems; ++i) {
            in[i] = VEC ? m > 0 : i * step < m;
            h[i] = in[i] ? to_f32(rx.at(i)) : 0.0f;
            s1[0] += h[i];
        }
        group_sum(s1, p.tpg, smem);
        const float mean = s1[0] * inv;
#pragma unroll
        for (int i = 0; i < kElems; ++i) {
            h[i] = in[i] ? h[i] - mean : 0.0f;
            s2[0] = fmaf(h[i], h[i], s2[0]);
        }
        group_sum(s2, p.tpg, smem + 16);
        const float rstd = rsqrtf(fmaf(s2[0], inv, p.eps));
        if (!BWD) {
            Row<TY, VEC> ry;
#pragma unroll
            for (int i = 0; i < kElems; ++i) {
                const float v = fmaf(h[i] * rstd, w[i], b[i]);
                float f, df;
                activate(p.act, GATED ? to_f32(rz.at(i)) : v, f, df);
                ry.at(i) = from_f32<TY>(GATED ? v * f : f);
            }
            ry.store(static_cast<TY *>(p.y) + row * p.C + c, m, step);
        } else {
            Row<TY, VEC> oz;
            Row<TX, VEC> ox;
            float q[kElems], s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < kElems; ++i) {
                h[i] *= rstd;
                const float v = fmaf(h[i], w[i], b[i]);
                const float d = in[i] ? to_f32(rd.at(i)) : 0.0f;
                float f, df;
                activate(p.act, GATED ? (in[i] ? to_f32(rz.at(i)) : 0.0f) : v, f, df);
                const float dv = d * (GATED ? f : df);
                if (GATED) oz.at(i) = from_f32<TY>(d * v * df);
                dw[i] = fmaf(dv, h[i], dw[i]);
                db[i] += dv;
                q[i] = dv * w[i];
                s[0] += q[i];
                s[1] = fmaf(q[i], h[i], s[1]);
            }
            group_sum(s, p.tpg, smem + 32);
#pragma unroll
            for (int i = 0; i < kElems; ++i)
                ox.at(i) = from_f32<TX>(rstd * (q[i] - s[0] * inv - h[i] * (s[1] * inv)));
            ox.store(static_cast<TX *>(p.dx) + row * p.C + c, m, step);
            if (GATED) oz.store(static_cast<TY *>(p.dgate) + row * p.C + c, m, step);
        }
    }
    if (BWD && p.partial) {
        // the CTA's rows side by side are added in shared memory, in order
        float *part = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.C;
        const int per = p.gpb * p.tpg;  // threads of a row
        float *sum = smem + 64;
        for (int k = 1; k < p.rp; ++k) {
            __syncthreads();
            if (r == k && on) {
#pragma unroll
                for (int i = 0; i < kElems; ++i) {
                    sum[(i * 2) * per + threadIdx.x % per] = dw[i];
                    sum[(i * 2 + 1) * per + threadIdx.x % per] = db[i];
                }
            }
            __syncthreads();
            if (r == 0 && on) {
#pragma unroll
                for (int i = 0; i < kElems; ++i) {
                    dw[i] += sum[(i * 2) * per + threadIdx.x];
                    db[i] += sum[(i * 2 + 1) * per + threadIdx.x];
                }
            }
        }
        if (r == 0) {
#pragma unroll
            for (int i = 0; i < kElems; ++i) {
                const int o = VEC ? i : i * step;
                if (VEC ? n > 0 : o < n) {
                    part[c + o] = dw[i];
                    part[p.C + c + o] = db[i];
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

// dweight and dbias from the CTAs' sums: 32 columns a CTA, eight rows of partials at a time.
__global__ void __launch_bounds__(256) based_norm_sum_kernel(const NormSumParams p) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;  // 0 .. 2 C - 1: dweight, then dbias
    griddep_wait();
    griddep_launch_dependents();
    float s = 0.0f;
    if (c < 2 * p.C)
        for (int k = warp; k < p.parts; k += 8) s += p.partial[static_cast<int64_t>(k) * 2 * p.C + c];
    red[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= 2 * p.C) return;
    for (int w = 1; w < 8; ++w) s += red[w][lane];
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
NormShape norm_shape(int64_t R, int C, int G, int sms, bool bwd) {
    NormShape s;
    const int per = (C / G + kElems - 1) / kElems;
    for (s.tpg = 1; s.tpg < per;) s.tpg *= 2;
    if (s.tpg > 32) {
        s.gpb = s.rp = 1;
        s.threads = s.tpg;
    } else {
        s.gpb = 256 / s.tpg < G ? 256 / s.tpg : G;
        s.rp = 256 / (s.gpb * s.tpg);
        s.threads = (s.gpb * s.rp * s.tpg + 31) / 32 * 32;
    }
    s.grid_y = (G + s.gpb - 1) / s.gpb;
    // as many CTAs as are resident at once, in whole turns over the column blocks
    const int resident = sms * ((bwd ? 1024 : 2048) / (s.threads > 256 ? 512 : 256));
    const int64_t turns = (R + s.rp - 1) / s.rp, most = resident / s.grid_y > 1 ? resident / s.grid_y : 1;
    s.grid_x = static_cast<int>(turns < most ? turns : most);
    return s;
}

int check_norm(const NormParams &p, int x_dtype, int dtype, bool bwd, const void *dweight, const void *dbias) {
    if (!p.x || (bwd ? (!p.dy || !p.dx || !p.dgate != !p.gate) : !p.y)) return BASED_ERR_NULL_POINTER;
    if (!type_ok(x_dtype) || !type_ok(dtype) || !type_ok(p.p_dtype) || (x_dtype != BASED_F32 && x_dtype != dtype))
        return BASED_ERR_UNSUPPORTED_TYPE;
    if (p.act != BASED_ACT_NONE && p.act != BASED_ACT_SILU && p.act != BASED_ACT_SIGMOID) return BASED_ERR_BAD_ARGUMENT;
    if (!(p.eps >= 0.0f)) return BASED_ERR_BAD_ARGUMENT;
    if (p.R < 1 || p.C < 1 || p.G < 1 || p.C % p.G != 0 || p.C / p.G > kMaxGroup || p.C > (1 << 20) ||
        p.R >= (1ll << 40))
        return BASED_ERR_BAD_SIZE;
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

template <typename TX, typename TY, bool BWD>
int launch_norm(const NormParams &p, const NormShape &s, cudaStream_t st) {
    const size_t xs = sizeof(TX), es = sizeof(TY);
    auto wide = [](const void *q, int64_t sr, size_t e) { return aligned(q, 16) && sr * e % 16 == 0; };
    // 16-byte words where every group of every row starts on one
    const bool vec = p.Cg % kElems == 0 && wide(p.x, p.x_sr, xs) && wide(p.gate, p.gate_sr, es) &&
                     wide(p.dy, p.dy_sr, es) && aligned(p.y, 16) && aligned(p.dx, 16) && aligned(p.dgate, 16);
    const dim3 grid(s.grid_x, s.grid_y);
    const size_t smem = (64 + (BWD && s.rp > 1 ? 2 * kElems * s.gpb * s.tpg : 0)) * sizeof(float);
    void (*kernel)(NormParams);
    if (p.gate)
        kernel = vec ? based_norm_kernel<TX, TY, true, true, BWD> : based_norm_kernel<TX, TY, false, true, BWD>;
    else
        kernel = vec ? based_norm_kernel<TX, TY, true, false, BWD> : based_norm_kernel<TX, TY, false, false, BWD>;
    OPS_CUDA(launch_op(kernel, grid, s.threads, smem, st, p));
    return BASED_OK;
}

template <bool BWD>
int dispatch_norm(const NormParams &p, const NormShape &s, int x_dtype, int dtype, cudaStream_t st) {
    using bf = __nv_bfloat16;
    if (x_dtype == BASED_F32) {
        if (dtype == BASED_F32) return launch_norm<float, float, BWD>(p, s, st);
        if (dtype == BASED_BF16) return launch_norm<float, bf, BWD>(p, s, st);
        return launch_norm<float, __half, BWD>(p, s, st);
    }
    if (dtype == BASED_BF16) return launch_norm<bf, bf, BWD>(p, s, st);
    return launch_norm<__half, __half, BWD>(p, s, st);
}

NormParams norm_params(const void *x, int64_t x_sr, const void *gate, int64_t gate_sr, const void *weight,
                       const void *bias, int p_dtype, int64_t R, int C, int G, float eps, int act) {
    NormParams p = {};
    p.x = x, p.x_sr = x_sr, p.gate = gate, p.gate_sr = gate ? gate_sr : 0;
    p.weight = weight, p.bias = bias, p.p_dtype = p_dtype;
    p.R = R, p.C = C, p.G = G, p.eps = eps, p.act = act;
    return p;
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
    const NormShape s = norm_shape(R, C, G, sms, false);
    place(p, s);
    return dispatch_norm<false>(p, s, x_dtype, dtype, reinterpret_cast<cudaStream_t>(stream));
}

size_t based_norm_bwd_workspace_size(int64_t R, int C, int G) {
    int sms;
    if (R < 1 || C < 1 || G < 1 || C % G != 0 || C / G > based::kMaxGroup || based::host_device(&sms) != BASED_OK)
        return 0;
    return static_cast<size_t>(based::norm_shape(R, C, G, sms, true).grid_x) * 2 * C * sizeof(float);
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
    const NormShape s = norm_shape(R, C, G, sms, true);
    place(p, s);
    const bool sums = dweight || dbias;
    if (sums) {
        if (!workspace || !aligned(workspace, 16) || ws_bytes < static_cast<size_t>(s.grid_x) * 2 * C * sizeof(float))
            return BASED_ERR_WORKSPACE;
        p.partial = static_cast<float *>(workspace);
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((rc = dispatch_norm<true>(p, s, x_dtype, dtype, st)) != BASED_OK || !sums) return rc;
    const NormSumParams q = {p.partial, s.grid_x, C, p_dtype, dweight, dbias};
    OPS_CUDA(launch_op(based_norm_sum_kernel, dim3((2 * C + 31) / 32), 256, 0, st, q));
    return BASED_OK;
}

}  // extern "C"
