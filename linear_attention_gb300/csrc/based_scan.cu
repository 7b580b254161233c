// based_scan.cu: the gated linear recurrence (declared in include/based_ops.h).
//
//     h_t = a_t h_{t-1} + u_t    per batch entry and channel
//
// A stretch of rows acts on the state as the affine map h -> A h + H with A the product of its
// decays and H the state it ends in from zero; two stretches compose as (A2 A1, A2 H1 + H2). The
// kernels cut time into tiles, a tile's rows among the warps of a CTA, take each warp's map in one
// pass over registers, compose the maps in front of each warp, and then run the rows from the
// right state. Nothing but the inputs is read and nothing but the outputs is written.
#include "ops_common.cuh"

namespace based {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kSave = BASED_SCAN_SAVE_ROWS;

struct ScanParams {
    const void *gate, *x, *dy;
    int64_t gate_sb, gate_st, x_sb, x_st, dy_sb, dy_st;
    int B, T, D, slabs;
    const float *state;   // forward: h_{-1}; backward: dfinal
    const int32_t *lengths;
    void *y;              // forward: h; backward: dgate
    void *dx;
    float *final_state;   // forward: the last state; backward: dstate
    float *saved;         // forward: written; backward: read
};

template <int MODE>
__device__ __forceinline__ void decay(float g, float x, float &a, float &u) {
    if (MODE == BASED_GATE_LOG) {
        a = expf(g);
        u = x;
    } else {
        float rest;
        sigmoid_pair(g, a, rest);
        u = rest * x;
    }
}

// One CTA: 32 N channels of one batch entry, tiles of kWarps * R rows in turn. Lane: N channels;
// warp w: rows [w R, w R + R) of a tile.
template <typename T, int N, int MODE>
__global__ void __launch_bounds__(kThreads, 2) based_scan_fwd_kernel(const ScanParams p) {
    constexpr int R = 16;
    constexpr int kTile = R * kWarps;
    using W = Pack<T, N>;
    __shared__ float agg[2][kWarps][2 * N][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / p.slabs, c = (blockIdx.x % p.slabs) * 32 * N + lane * N;
    const bool on = c < p.D;
    griddep_wait();
    griddep_launch_dependents();
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    const int64_t plane = static_cast<int64_t>(b) * p.D + c;
    const T *gate = static_cast<const T *>(p.gate) + b * p.gate_sb + c;
    const T *x = static_cast<const T *>(p.x) + b * p.x_sb + c;
    T *y = static_cast<T *>(p.y) + static_cast<int64_t>(b) * p.T * p.D + c;
    const int n_saved = (p.T + kSave - 1) / kSave;
    float carry[N];
#pragma unroll
    for (int j = 0; j < N; ++j) carry[j] = on && p.state ? p.state[plane + j] : 0.0f;
    const int tiles = (p.T + kTile - 1) / kTile;
    for (int tile = 0; tile < tiles; ++tile) {
        const int row0 = tile * kTile + warp * R;
        float a[R][N], u[R][N], A[N], H[N];
#pragma unroll
        for (int j = 0; j < N; ++j) A[j] = 1.0f, H[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (on && row0 + i < len) {
                const W g = *reinterpret_cast<const W *>(gate + (row0 + i) * p.gate_st);
                const W v = *reinterpret_cast<const W *>(x + (row0 + i) * p.x_st);
#pragma unroll
                for (int j = 0; j < N; ++j) decay<MODE>(to_f32(g.v[j]), to_f32(v.v[j]), a[i][j], u[i][j]);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) a[i][j] = 1.0f, u[i][j] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                H[j] = fmaf(a[i][j], H[j], u[i][j]);
                A[j] *= a[i][j];
            }
        float(&slot)[kWarps][2 * N][32] = agg[tile & 1];
#pragma unroll
        for (int j = 0; j < N; ++j) slot[warp][j][lane] = A[j], slot[warp][N + j][lane] = H[j];
        __syncthreads();  // the two buffers alternate: one barrier a tile is enough
        float h[N];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (w == warp) h[j] = carry[j];
                carry[j] = fmaf(slot[w][j][lane], carry[j], slot[w][N + j][lane]);
            }
        }
        if (!on) continue;
        if (p.saved && row0 % kSave == 0 && row0 < p.T) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                p.saved[(static_cast<int64_t>(b) * n_saved + row0 / kSave) * p.D + c + j] = h[j];
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (row0 + i < p.T) {
                W o;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    h[j] = fmaf(a[i][j], h[j], u[i][j]);
                    o.v[j] = from_f32<T>(row0 + i < len ? h[j] : 0.0f);
                }
                *reinterpret_cast<W *>(y + static_cast<int64_t>(row0 + i) * p.D) = o;
            }
        }
    }
    if (on && warp == 0 && p.final_state) {
#pragma unroll
        for (int j = 0; j < N; ++j) p.final_state[plane + j] = carry[j];
    }
}

// Backward: the tiles from the last to the first. With mu = what the rows after a row pass back to
// it, lam_t = dy_t + mu and mu <- a_t lam_t: the map of a stretch in reversed time is mu -> A mu + M
// with the same A. h inside a tile is rebuilt from the state saved before it.
template <typename T, int N, int MODE>
__global__ void __launch_bounds__(kThreads, 2) based_scan_bwd_kernel(const ScanParams p) {
    constexpr int R = kSave / kWarps;
    using W = Pack<T, N>;
    __shared__ float agg[2][kWarps][3 * N][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / p.slabs, c = (blockIdx.x % p.slabs) * 32 * N + lane * N;
    const bool on = c < p.D;
    griddep_wait();
    griddep_launch_dependents();
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    const int64_t plane = static_cast<int64_t>(b) * p.D + c;
    const T *gate = static_cast<const T *>(p.gate) + b * p.gate_sb + c;
    const T *x = static_cast<const T *>(p.x) + b * p.x_sb + c;
    const T *dy = static_cast<const T *>(p.dy) + b * p.dy_sb + c;
    T *dgate = static_cast<T *>(p.y) + static_cast<int64_t>(b) * p.T * p.D + c;
    T *dx = static_cast<T *>(p.dx) + static_cast<int64_t>(b) * p.T * p.D + c;
    const int tiles = (p.T + kSave - 1) / kSave;
    float carry[N];
#pragma unroll
    for (int j = 0; j < N; ++j) carry[j] = on && p.state ? p.state[plane + j] : 0.0f;
    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int row0 = tile * kSave + warp * R;
        float a[R][N], rest[R][N], v[R][N], d[R][N], before[R][N], h[N], A[N], H[N], M[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            A[j] = 1.0f, H[j] = 0.0f, M[j] = 0.0f;
            h[j] = on ? p.saved[(static_cast<int64_t>(b) * tiles + tile) * p.D + c + j] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (on && row0 + i < len) {
                const W wg = *reinterpret_cast<const W *>(gate + (row0 + i) * p.gate_st);
                const W wx = *reinterpret_cast<const W *>(x + (row0 + i) * p.x_st);
                const W wd = *reinterpret_cast<const W *>(dy + (row0 + i) * p.dy_st);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    if (MODE == BASED_GATE_LOG)
                        a[i][j] = expf(to_f32(wg.v[j])), rest[i][j] = 1.0f;
                    else
                        sigmoid_pair(to_f32(wg.v[j]), a[i][j], rest[i][j]);
                    v[i][j] = to_f32(wx.v[j]);
                    d[i][j] = to_f32(wd.v[j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) a[i][j] = 1.0f, rest[i][j] = 0.0f, v[i][j] = 0.0f, d[i][j] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                H[j] = fmaf(a[i][j], H[j], rest[i][j] * v[i][j]);
                A[j] *= a[i][j];
                const int k = R - 1 - i;
                M[j] = a[k][j] * (d[k][j] + M[j]);
            }
        float(&slot)[kWarps][3 * N][32] = agg[tile & 1];
#pragma unroll
        for (int j = 0; j < N; ++j)
            slot[warp][j][lane] = A[j], slot[warp][N + j][lane] = H[j], slot[warp][2 * N + j][lane] = M[j];
        __syncthreads();
        float mu[N];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int k = kWarps - 1 - w;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (w < warp) h[j] = fmaf(slot[w][j][lane], h[j], slot[w][N + j][lane]);
                if (k == warp) mu[j] = carry[j];
                carry[j] = fmaf(slot[k][j][lane], carry[j], slot[k][2 * N + j][lane]);
            }
        }
        if (!on) continue;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                before[i][j] = h[j];
                h[j] = fmaf(a[i][j], h[j], rest[i][j] * v[i][j]);
            }
#pragma unroll
        for (int i = R - 1; i >= 0; --i) {
            if (row0 + i < p.T) {
                W og, ox;
                const bool live = row0 + i < len;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float lam = d[i][j] + mu[j];
                    mu[j] = a[i][j] * lam;
                    float dg, dv;
                    if (MODE == BASED_GATE_LOG)
                        dg = mu[j] * before[i][j], dv = lam;
                    else
                        dg = mu[j] * rest[i][j] * (before[i][j] - v[i][j]), dv = rest[i][j] * lam;
                    og.v[j] = from_f32<T>(live ? dg : 0.0f);
                    ox.v[j] = from_f32<T>(live ? dv : 0.0f);
                }
                *reinterpret_cast<W *>(dgate + static_cast<int64_t>(row0 + i) * p.D) = og;
                *reinterpret_cast<W *>(dx + static_cast<int64_t>(row0 + i) * p.D) = ox;
            }
        }
    }
    if (on && warp == 0 && p.final_state) {
#pragma unroll
        for (int j = 0; j < N; ++j) p.final_state[plane + j] = carry[j];
    }
}

struct StepParams {
    const void *gate, *x;
    int64_t gate_sn, x_sn;
    int N, D, S;
    float *pool;
    const int32_t *slots;
    void *y;
};

// One row for N sequences: grid (channel blocks, sequences), N_ consecutive channels a thread.
template <typename T, int N, int MODE>
__global__ void __launch_bounds__(128) based_scan_step_kernel(const StepParams p) {
    using W = Pack<T, N>;
    const int c = (blockIdx.x * 128 + threadIdx.x) * N;
    griddep_wait();
    griddep_launch_dependents();
    if (c >= p.D) return;
    for (int64_t n = blockIdx.y; n < p.N; n += gridDim.y) {
        const int64_t s = p.slots ? p.slots[n] : n;
        W o;
        if (s >= 0 && s < p.S) {
            const W g = *reinterpret_cast<const W *>(static_cast<const T *>(p.gate) + n * p.gate_sn + c);
            const W v = *reinterpret_cast<const W *>(static_cast<const T *>(p.x) + n * p.x_sn + c);
            Pack<float, N> h = *reinterpret_cast<const Pack<float, N> *>(p.pool + s * p.D + c);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float a, u;
                decay<MODE>(to_f32(g.v[j]), to_f32(v.v[j]), a, u);
                h.v[j] = fmaf(a, h.v[j], u);
                o.v[j] = from_f32<T>(h.v[j]);
            }
            *reinterpret_cast<Pack<float, N> *>(p.pool + s * p.D + c) = h;
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) o.v[j] = from_f32<T>(0.0f);
        }
        *reinterpret_cast<W *>(static_cast<T *>(p.y) + n * p.D + c) = o;
    }
}

int check_scan(const ScanParams &p, int dtype, int mode, bool bwd) {
    if (!p.gate || !p.x || !p.y || (bwd && (!p.dy || !p.dx || !p.saved))) return BASED_ERR_NULL_POINTER;
    if (!type_ok(dtype)) return BASED_ERR_UNSUPPORTED_TYPE;
    if (mode != BASED_GATE_LOG && mode != BASED_GATE_SIGMOID) return BASED_ERR_BAD_ARGUMENT;
    if (p.B < 1 || p.T < 1 || p.D < 1) return BASED_ERR_BAD_SIZE;
    if (static_cast<int64_t>(p.B) * p.D >= (1ll << 31) || p.T > (1 << 30)) return BASED_ERR_BAD_SIZE;
    if (p.gate_sb < 0 || p.gate_st < 0 || p.x_sb < 0 || p.x_st < 0 || p.dy_sb < 0 || p.dy_st < 0)
        return BASED_ERR_BAD_STRIDE;
    const size_t es = elem_size(dtype);
    if (!aligned(p.gate, es) || !aligned(p.x, es) || !aligned(p.y, es) || !aligned(p.dy, es) || !aligned(p.dx, es) ||
        !aligned(p.state, 4) || !aligned(p.lengths, 4) || !aligned(p.final_state, 4) || !aligned(p.saved, 4))
        return BASED_ERR_MISALIGNED;
    auto last = [&](int64_t sb, int64_t st) { return (p.B - 1) * sb + (p.T - 1) * st + p.D - 1; };
    const int64_t all = static_cast<int64_t>(p.B) * p.T * p.D - 1, plane = static_cast<int64_t>(p.B) * p.D - 1;
    const int64_t saved = static_cast<int64_t>(p.B) * ((p.T + kSave - 1) / kSave) * p.D - 1;
    const Span in[] = {span(p.gate, last(p.gate_sb, p.gate_st), es), span(p.x, last(p.x_sb, p.x_st), es),
                       span(p.dy, last(p.dy_sb, p.dy_st), es), span(p.lengths, p.B - 1, 4),
                       span(p.state, plane, 4), bwd ? span(p.saved, saved, 4) : Span{0, 0}};
    const Span out[] = {span(p.y, all, es), span(p.dx, all, es), span(p.final_state, plane, 4),
                        bwd ? Span{0, 0} : span(p.saved, saved, 4)};
    for (int i = 0; i < 4; ++i) {
        for (const Span &s : in)
            if (overlap(out[i], s) && !(p.state && p.final_state == p.state && i == 2 && s.a == in[4].a && s.b == in[4].b))
                return BASED_ERR_ALIASING;
        for (int k = 0; k < i; ++k)
            if (overlap(out[i], out[k])) return BASED_ERR_ALIASING;
    }
    return BASED_OK;
}

template <typename T, int N>
int launch_scan(ScanParams &p, int mode, bool bwd, cudaStream_t st) {
    p.slabs = (p.D + 32 * N - 1) / (32 * N);
    const dim3 grid(static_cast<unsigned>(p.slabs) * p.B);
    if (bwd)
        OPS_CUDA(launch_op(mode == BASED_GATE_LOG ? based_scan_bwd_kernel<T, N, BASED_GATE_LOG>
                                                  : based_scan_bwd_kernel<T, N, BASED_GATE_SIGMOID>,
                           grid, kThreads, 0, st, p));
    else
        OPS_CUDA(launch_op(mode == BASED_GATE_LOG ? based_scan_fwd_kernel<T, N, BASED_GATE_LOG>
                                                  : based_scan_fwd_kernel<T, N, BASED_GATE_SIGMOID>,
                           grid, kThreads, 0, st, p));
    return BASED_OK;
}

int run_scan(ScanParams &p, int dtype, int mode, bool bwd, based_stream_t stream) {
    int rc = check_scan(p, dtype, mode, bwd), sms;
    if (rc != BASED_OK || (rc = host_device(&sms)) != BASED_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == BASED_F32) return launch_scan<float, 1>(p, mode, bwd, st);
    // two 16-bit channels a lane where every row starts on a 4-byte boundary
    const bool pair = ((p.D | p.gate_sb | p.gate_st | p.x_sb | p.x_st | p.dy_sb | p.dy_st) & 1) == 0 &&
                      aligned(p.gate, 4) && aligned(p.x, 4) && aligned(p.dy, 4) && aligned(p.y, 4) && aligned(p.dx, 4);
    if (dtype == BASED_BF16)
        return pair ? launch_scan<__nv_bfloat16, 2>(p, mode, bwd, st) : launch_scan<__nv_bfloat16, 1>(p, mode, bwd, st);
    return pair ? launch_scan<__half, 2>(p, mode, bwd, st) : launch_scan<__half, 1>(p, mode, bwd, st);
}

template <typename T, int N>
int launch_step(const StepParams &p, int mode, cudaStream_t st) {
    const int64_t blocks = (p.D + 128ll * N - 1) / (128 * N);
    const dim3 grid(static_cast<unsigned>(blocks), p.N < 65535 ? p.N : 65535);
    OPS_CUDA(launch_op(mode == BASED_GATE_LOG ? based_scan_step_kernel<T, N, BASED_GATE_LOG>
                                              : based_scan_step_kernel<T, N, BASED_GATE_SIGMOID>,
                       grid, 128, 0, st, p));
    return BASED_OK;
}

}  // namespace
}  // namespace based

extern "C" {

int based_scan_fwd(const void *gate, int64_t gate_sb, int64_t gate_st, const void *x, int64_t x_sb, int64_t x_st,
                   int B, int T, int D, int dtype, int mode, const float *state, const int32_t *lengths, void *y,
                   float *final_state, float *saved, based_stream_t stream) {
    based::ScanParams p = {};
    p.gate = gate, p.gate_sb = gate_sb, p.gate_st = gate_st;
    p.x = x, p.x_sb = x_sb, p.x_st = x_st;
    p.B = B, p.T = T, p.D = D;
    p.state = state, p.lengths = lengths, p.y = y, p.final_state = final_state, p.saved = saved;
    return based::run_scan(p, dtype, mode, false, stream);
}

int based_scan_bwd(const void *gate, int64_t gate_sb, int64_t gate_st, const void *x, int64_t x_sb, int64_t x_st,
                   const void *dy, int64_t dy_sb, int64_t dy_st, const float *saved, int B, int T, int D, int dtype,
                   int mode, const float *dfinal, const int32_t *lengths, void *dgate, void *dx, float *dstate,
                   based_stream_t stream) {
    based::ScanParams p = {};
    p.gate = gate, p.gate_sb = gate_sb, p.gate_st = gate_st;
    p.x = x, p.x_sb = x_sb, p.x_st = x_st;
    p.dy = dy, p.dy_sb = dy_sb, p.dy_st = dy_st;
    p.B = B, p.T = T, p.D = D;
    p.state = dfinal, p.lengths = lengths, p.y = dgate, p.dx = dx, p.final_state = dstate;
    p.saved = const_cast<float *>(saved);
    return based::run_scan(p, dtype, mode, true, stream);
}

int based_scan_step(const void *gate, int64_t gate_sn, const void *x, int64_t x_sn, int N, int D, int S, int dtype,
                    int mode, float *pool, const int32_t *slots, void *y, based_stream_t stream) {
    using namespace based;
    if (!gate || !x || !pool || !y) return BASED_ERR_NULL_POINTER;
    if (!type_ok(dtype)) return BASED_ERR_UNSUPPORTED_TYPE;
    if (mode != BASED_GATE_LOG && mode != BASED_GATE_SIGMOID) return BASED_ERR_BAD_ARGUMENT;
    if (N < 1 || D < 1 || S < 1 || D > (1 << 30) || (!slots && S < N)) return BASED_ERR_BAD_SIZE;
    if (gate_sn < 0 || x_sn < 0) return BASED_ERR_BAD_STRIDE;
    const size_t es = elem_size(dtype);
    if (!aligned(gate, es) || !aligned(x, es) || !aligned(y, es) || !aligned(pool, 4) || !aligned(slots, 4))
        return BASED_ERR_MISALIGNED;
    const Span in[] = {span(gate, (N - 1) * gate_sn + D - 1, es), span(x, (N - 1) * x_sn + D - 1, es),
                       span(slots, N - 1, 4)};
    const Span sy = span(y, static_cast<int64_t>(N) * D - 1, es), sp = span(pool, static_cast<int64_t>(S) * D - 1, 4);
    for (const Span &s : in)
        if (overlap(s, sy) || overlap(s, sp)) return BASED_ERR_ALIASING;
    if (overlap(sy, sp)) return BASED_ERR_ALIASING;
    int sms;
    const int rc = host_device(&sms);
    if (rc != BASED_OK) return rc;
    const StepParams p = {gate, x, gate_sn, x_sn, N, D, S, pool, slots, y};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // four channels a thread where the rows of every tensor allow their loads
    const bool quad = ((D | gate_sn | x_sn) & 3) == 0 && aligned(gate, 4 * es) && aligned(x, 4 * es) &&
                      aligned(y, 4 * es) && aligned(pool, 16);
    if (dtype == BASED_F32) return quad ? launch_step<float, 4>(p, mode, st) : launch_step<float, 1>(p, mode, st);
    if (dtype == BASED_BF16)
        return quad ? launch_step<__nv_bfloat16, 4>(p, mode, st) : launch_step<__nv_bfloat16, 1>(p, mode, st);
    return quad ? launch_step<__half, 4>(p, mode, st) : launch_step<__half, 1>(p, mode, st);
}

}  // extern "C"
