// based_scan.cu: the gated linear recurrence (declared in include/based_ops.h).
//
//     h_t = a_t h_{t-1} + u_t    per batch entry and channel
//
// A stretch of rows acts on the state as the affine map h -> A h + H with A the product of its
// decays and H the state it ends in from zero; two stretches compose as (A2 A1, A2 H1 + H2). Time
// is cut into tiles of 64 rows. The CTAs of a cluster take the tiles in turn; each warp of a CTA
// takes its rows' map in one pass over registers, the maps of a CTA's warps and of the cluster's
// CTAs are exchanged through (distributed) shared memory, and every warp then runs its rows from
// the state in front of them. So each input is read once and each output written once, however
// few channels there are, and no CTA waits for one that may not be resident.
#include <mutex>

#include "ops_common.cuh"

namespace based {
namespace {

constexpr int kSave = BASED_SCAN_SAVE_ROWS;
constexpr int kTile = kSave;       // rows of a tile: one saved state each
constexpr int kRowBytes = 128;     // a tile's row: 64 channels of 16 bits or 32 of 32
constexpr int kMaxCluster = 16;

struct ScanParams {
    const void *gate, *x, *dy;
    int64_t gate_sb, gate_st, x_sb, x_st, dy_sb, dy_st;
    int B, T, D, slabs;
    int cluster;          // CTAs of a cluster
    int word;             // bytes of a copy to shared memory that every row's start allows: 16, 4 or 2
    int pair;             // two 16-bit outputs can be stored as one word
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

// ------------------------------------------------------------------------------------------------
// Copies of a tile's rows into shared memory
// ------------------------------------------------------------------------------------------------
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src) {
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows [0, rows) of channels [0, cols) of a tensor at src into the tile at dst, by all THREADS
// threads of the CTA. The other places keep what they held; nothing that is stored depends on it.
template <typename T, int THREADS, int BYTES>
__device__ __forceinline__ void copy_words(uint8_t *dst, const T *src, int64_t stride, int rows, int cols) {
    constexpr int kPer = BYTES / static_cast<int>(sizeof(T)), kWords = kRowBytes / BYTES, kStep = THREADS / kWords;
    const int col = static_cast<int>(threadIdx.x) % kWords, row0 = static_cast<int>(threadIdx.x) / kWords;
    if (col * kPer >= cols) return;
    const T *from = src + row0 * stride + col * kPer;
    const uint32_t to = smem_u32(dst) + row0 * kRowBytes + col * BYTES;
#pragma unroll
    for (int k = 0; k < kTile / kStep; ++k) {
        if (row0 + k * kStep < rows) cp_async<BYTES>(to + k * kStep * kRowBytes, from);
        from += kStep * stride;
    }
}
template <typename T, int THREADS>
__device__ __forceinline__ void copy_tile(uint8_t *dst, const T *src, int64_t stride, int rows, int cols, int word) {
    if (word == 16) {
        copy_words<T, THREADS, 16>(dst, src, stride, rows, cols);
    } else if (word == 4) {
        copy_words<T, THREADS, 4>(dst, src, stride, rows, cols);
    } else {
        // rows that start on an odd 16-bit element: no asynchronous copy is that narrow
        constexpr int kCols = kRowBytes / sizeof(T);
        for (int i = threadIdx.x; i < rows * kCols; i += THREADS)
            if (i % kCols < cols) reinterpret_cast<T *>(dst)[i] = src[(i / kCols) * stride + i % kCols];
    }
}

// ------------------------------------------------------------------------------------------------
// Clusters
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The map h -> a h + b of N channels.
template <int N>
struct alignas(8 * N) Map {
    float a[N], b[N];
};
template <int N>
__device__ __forceinline__ void send(Map<N> *slot, uint32_t rank, const Map<N> &m) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(slot)), "r"(rank));
    if (N == 2)
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(m.a[0]), "f"(m.a[N - 1]),
                     "f"(m.b[0]), "f"(m.b[N - 1])
                     : "memory");
    else
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(m.a[0]), "f"(m.b[0]) : "memory");
}
// The maps of the cluster's CTAs, in the order of their tiles: `at` becomes the value in front of
// tile `rank`, `carry` the one behind the last.
template <int N>
__device__ __forceinline__ void fold(const Map<N> (*maps)[32], int cluster, int rank, int lane, float (&at)[N], float (&carry)[N]) {
    for (int r = 0; r < cluster; ++r) {
        const Map<N> m = maps[r][lane];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            at[j] = r == rank ? carry[j] : at[j];
            carry[j] = fmaf(m.a[j], carry[j], m.b[j]);
        }
    }
}

template <typename T, int N>
__device__ __forceinline__ void store_channels(T *dst, const float (&v)[N], int n, int pair) {
    if (N == 2 && pair) {
        Pack<T, N> w;
#pragma unroll
        for (int j = 0; j < N; ++j) w.v[j] = from_f32<T>(v[j]);
        *reinterpret_cast<Pack<T, N> *>(dst) = w;
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < n) dst[j] = from_f32<T>(v[j]);
    }
}

// Shared memory: the stages of the copies, the warps' maps, the cluster's maps (two of each, used in
// turn, so that one barrier a tile orders their reuse).
template <int N, int WARPS, int TENSORS, int STAGES>
struct ScanSmem {
    uint8_t tile[STAGES][TENSORS][kTile * kRowBytes];
    Map<N> warp[2][WARPS][32];
    float rev[2][WARPS][N][32];  // backward: the reversed map's increment
    static constexpr size_t bytes(int cluster) { return sizeof(ScanSmem) + (cluster > 1 ? 2 * cluster * 32 * sizeof(Map<N>) : 0); }
};

// ------------------------------------------------------------------------------------------------
// Forward
// ------------------------------------------------------------------------------------------------
constexpr int kFwdWarps = 4, kFwdStages = 2;
template <typename T>
struct ScanCfg {
    static constexpr int N = 4 / sizeof(T);  // channels of a lane: one 32-bit word
    using Fwd = ScanSmem<N, kFwdWarps, 2, kFwdStages>;
};

// A cluster: 32 N channels of one batch entry. Lane: N channels; warp w of the CTA: rows
// [16 w, 16 w + 16) of its tile.
template <typename T, int MODE>
__global__ void __launch_bounds__(32 * kFwdWarps, 4) based_scan_fwd_kernel(const ScanParams p) {
    constexpr int N = ScanCfg<T>::N, R = kTile / kFwdWarps, kThreads = 32 * kFwdWarps;
    using Smem = typename ScanCfg<T>::Fwd;
    using W = Pack<T, N>;
    extern __shared__ __align__(128) uint8_t raw[];
    Smem &sm = *reinterpret_cast<Smem *>(raw);
    Map<N>(*maps)[32] = reinterpret_cast<Map<N>(*)[32]>(raw + sizeof(Smem));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cs = p.cluster, rank = cs > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int slab = static_cast<int>(blockIdx.x / cs), b = slab / p.slabs, c0 = (slab % p.slabs) * 32 * N, c = c0 + lane * N;
    const int n = min(max(p.D - c, 0), N), cols = min(p.D - c0, 32 * N);
    griddep_wait();
    griddep_launch_dependents();
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    const int64_t plane = static_cast<int64_t>(b) * p.D + c;
    const T *gate = static_cast<const T *>(p.gate) + b * p.gate_sb + c0;
    const T *x = static_cast<const T *>(p.x) + b * p.x_sb + c0;
    T *y = static_cast<T *>(p.y) + static_cast<int64_t>(b) * p.T * p.D + c;
    const int tiles = (p.T + kTile - 1) / kTile, steps = (tiles + cs - 1) / cs;
    float carry[N];
#pragma unroll
    for (int j = 0; j < N; ++j) carry[j] = j < n && p.state ? p.state[plane + j] : 0.0f;
    auto fetch = [&](int step) {
        const int row = (step * cs + rank) * kTile, rows = min(len - row, kTile);
        if (rows > 0) {
            copy_tile<T, kThreads>(sm.tile[step % kFwdStages][0], gate + row * p.gate_st, p.gate_st, rows, cols, p.word);
            copy_tile<T, kThreads>(sm.tile[step % kFwdStages][1], x + row * p.x_st, p.x_st, rows, cols, p.word);
        }
    };
#pragma unroll
    for (int k = 0; k < kFwdStages - 1; ++k) {
        if (k < steps) fetch(k);
        cp_async_commit();
    }
    if (cs > 1) {  // every CTA of the cluster runs before another one writes to its shared memory
        cluster_arrive();
        cluster_wait();
    }
    for (int step = 0; step < steps; ++step) {
        const int tile = step * cs + rank, row0 = tile * kTile + warp * R;
        cp_async_wait<kFwdStages - 2>();
        __syncthreads();  // the tile has landed, and the stage before it is free
        if (step + kFwdStages - 1 < steps) fetch(step + kFwdStages - 1);
        cp_async_commit();
        const uint8_t *sg = sm.tile[step % kFwdStages][0] + warp * R * kRowBytes + lane * 4;
        const uint8_t *sx = sm.tile[step % kFwdStages][1] + warp * R * kRowBytes + lane * 4;
        float a[R][N], u[R][N];
        Map<N> m;
#pragma unroll
        for (int j = 0; j < N; ++j) m.a[j] = 1.0f, m.b[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const W g = *reinterpret_cast<const W *>(sg + i * kRowBytes);
            const W v = *reinterpret_cast<const W *>(sx + i * kRowBytes);
            const bool live = row0 + i < len;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                decay<MODE>(to_f32(g.v[j]), to_f32(v.v[j]), a[i][j], u[i][j]);
                a[i][j] = live ? a[i][j] : 1.0f;
                u[i][j] = live ? u[i][j] : 0.0f;
                m.b[j] = fmaf(a[i][j], m.b[j], u[i][j]);
                m.a[j] *= a[i][j];
            }
        }
        sm.warp[step & 1][warp][lane] = m;
        __syncthreads();
        // this warp's start as a map of the tile's start, then the tile's start itself
        Map<N> pre, all;
#pragma unroll
        for (int j = 0; j < N; ++j) all.a[j] = 1.0f, all.b[j] = 0.0f;
#pragma unroll
        for (int w = 0; w < kFwdWarps; ++w) {
            const Map<N> o = sm.warp[step & 1][w][lane];
            if (w == warp) pre = all;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                all.b[j] = fmaf(o.a[j], all.b[j], o.b[j]);
                all.a[j] *= o.a[j];
            }
        }
        float h[N];
        if (cs > 1) {
            Map<N>(*mine)[32] = maps + (step & 1) * cs;
            for (int r = warp; r < cs; r += kFwdWarps) send(&mine[rank][lane], r, all);
            cluster_arrive();
            cluster_wait();
            fold<N>(mine, cs, rank, lane, h, carry);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                h[j] = carry[j];
                carry[j] = fmaf(all.a[j], carry[j], all.b[j]);
            }
        }
        if (warp == 0 && p.saved && row0 < p.T) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j < n) p.saved[(static_cast<int64_t>(b) * tiles + tile) * p.D + c + j] = h[j];
        }
#pragma unroll
        for (int j = 0; j < N; ++j) h[j] = fmaf(pre.a[j], h[j], pre.b[j]);
        if (n > 0) {
            T *to = y + static_cast<int64_t>(row0) * p.D;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float o[N];
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    h[j] = fmaf(a[i][j], h[j], u[i][j]);
                    o[j] = row0 + i < len ? h[j] : 0.0f;
                }
                if (row0 + i < p.T) store_channels<T, N>(to, o, n, p.pair);
                to += p.D;
            }
        }
    }
    if (warp == 0 && rank == 0 && p.final_state) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < n) p.final_state[plane + j] = carry[j];
    }
}

// ------------------------------------------------------------------------------------------------
// Backward
// ------------------------------------------------------------------------------------------------
// The tiles from the last to the first. With mu = what the rows after a row pass back to it,
// lam_t = dy_t + mu and mu <- a_t lam_t: the map of a stretch in reversed time is mu -> A mu + M
// with the same A. h inside a tile is rebuilt from the state saved before it.
constexpr int kBwdWarps = 8, kBwdStages = 3;
template <typename T, int MODE>
__global__ void __launch_bounds__(32 * kBwdWarps, 2) based_scan_bwd_kernel(const ScanParams p) {
    constexpr int N = ScanCfg<T>::N, R = kTile / kBwdWarps, kThreads = 32 * kBwdWarps;
    using Smem = ScanSmem<N, kBwdWarps, 3, kBwdStages>;
    using W = Pack<T, N>;
    extern __shared__ __align__(128) uint8_t raw[];
    Smem &sm = *reinterpret_cast<Smem *>(raw);
    Map<N>(*maps)[32] = reinterpret_cast<Map<N>(*)[32]>(raw + sizeof(Smem));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cs = p.cluster, rank = cs > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int slab = static_cast<int>(blockIdx.x / cs), b = slab / p.slabs, c0 = (slab % p.slabs) * 32 * N, c = c0 + lane * N;
    const int n = min(max(p.D - c, 0), N), cols = min(p.D - c0, 32 * N);
    griddep_wait();
    griddep_launch_dependents();
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    const int64_t plane = static_cast<int64_t>(b) * p.D + c;
    const T *gate = static_cast<const T *>(p.gate) + b * p.gate_sb + c0;
    const T *x = static_cast<const T *>(p.x) + b * p.x_sb + c0;
    const T *dy = static_cast<const T *>(p.dy) + b * p.dy_sb + c0;
    T *dgate = static_cast<T *>(p.y) + static_cast<int64_t>(b) * p.T * p.D + c;
    T *dx = static_cast<T *>(p.dx) + static_cast<int64_t>(b) * p.T * p.D + c;
    const int tiles = (p.T + kTile - 1) / kTile, steps = (tiles + cs - 1) / cs;
    float carry[N];
#pragma unroll
    for (int j = 0; j < N; ++j) carry[j] = j < n && p.state ? p.state[plane + j] : 0.0f;
    auto fetch = [&](int step) {
        const int row = (tiles - 1 - (step * cs + rank)) * kTile, rows = min(len - row, kTile);
        if (row >= 0 && rows > 0) {
            uint8_t(*to)[kTile * kRowBytes] = sm.tile[step % kBwdStages];
            copy_tile<T, kThreads>(to[0], gate + row * p.gate_st, p.gate_st, rows, cols, p.word);
            copy_tile<T, kThreads>(to[1], x + row * p.x_st, p.x_st, rows, cols, p.word);
            copy_tile<T, kThreads>(to[2], dy + row * p.dy_st, p.dy_st, rows, cols, p.word);
        }
    };
    float next[N];  // the state in front of the next tile
    auto fetch_state = [&](int step) {
        const int tile = tiles - 1 - (step * cs + rank);
#pragma unroll
        for (int j = 0; j < N; ++j)
            next[j] = tile >= 0 && j < n ? p.saved[(static_cast<int64_t>(b) * tiles + tile) * p.D + c + j] : 0.0f;
    };
    fetch_state(0);
#pragma unroll
    for (int k = 0; k < kBwdStages - 1; ++k) {
        if (k < steps) fetch(k);
        cp_async_commit();
    }
    if (cs > 1) {  // every CTA of the cluster runs before another one writes to its shared memory
        cluster_arrive();
        cluster_wait();
    }
    for (int step = 0; step < steps; ++step) {
        const int tile = tiles - 1 - (step * cs + rank), row0 = tile * kTile + warp * R;
        float h[N];
#pragma unroll
        for (int j = 0; j < N; ++j) h[j] = next[j];
        cp_async_wait<kBwdStages - 2>();
        __syncthreads();
        if (step + kBwdStages - 1 < steps) fetch(step + kBwdStages - 1);
        cp_async_commit();
        fetch_state(step + 1);
        const uint8_t(*st)[kTile * kRowBytes] = sm.tile[step % kBwdStages];
        const int off = warp * R * kRowBytes + lane * 4;
        float a[R][N], rest[R][N], rev[N];
        W v[R], d[R];
        Map<N> m;
#pragma unroll
        for (int j = 0; j < N; ++j) m.a[j] = 1.0f, m.b[j] = 0.0f, rev[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const W g = *reinterpret_cast<const W *>(st[0] + off + i * kRowBytes);
            v[i] = *reinterpret_cast<const W *>(st[1] + off + i * kRowBytes);
            d[i] = *reinterpret_cast<const W *>(st[2] + off + i * kRowBytes);
            const bool live = tile >= 0 && row0 + i < len;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (MODE == BASED_GATE_LOG)
                    a[i][j] = expf(to_f32(g.v[j])), rest[i][j] = 1.0f;
                else
                    sigmoid_pair(to_f32(g.v[j]), a[i][j], rest[i][j]);
                if (!live) {
                    a[i][j] = 1.0f, rest[i][j] = 0.0f;
                    v[i].v[j] = from_f32<T>(0.0f);
                    d[i].v[j] = from_f32<T>(0.0f);
                }
                m.b[j] = fmaf(a[i][j], m.b[j], rest[i][j] * to_f32(v[i].v[j]));
                m.a[j] *= a[i][j];
            }
        }
#pragma unroll
        for (int i = R - 1; i >= 0; --i)
#pragma unroll
            for (int j = 0; j < N; ++j) rev[j] = a[i][j] * (to_f32(d[i].v[j]) + rev[j]);
        sm.warp[step & 1][warp][lane] = m;
#pragma unroll
        for (int j = 0; j < N; ++j) sm.rev[step & 1][warp][j][lane] = rev[j];
        __syncthreads();
        // the rows behind this warp's as a map, and the tile's map
        Map<N> pre, all;
#pragma unroll
        for (int j = 0; j < N; ++j) all.a[j] = 1.0f, all.b[j] = 0.0f;
#pragma unroll
        for (int k = 0; k < kBwdWarps; ++k) {
            const int w = kBwdWarps - 1 - k;
            const Map<N> o = sm.warp[step & 1][w][lane], f = sm.warp[step & 1][k][lane];
            if (w == warp) pre = all;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                all.b[j] = fmaf(o.a[j], all.b[j], sm.rev[step & 1][w][j][lane]);
                all.a[j] *= o.a[j];
                h[j] = k < warp ? fmaf(f.a[j], h[j], f.b[j]) : h[j];
            }
        }
        float mu[N];
        if (cs > 1) {
            Map<N>(*mine)[32] = maps + (step & 1) * cs;
            for (int r = warp; r < cs; r += kBwdWarps) send(&mine[rank][lane], r, all);
            cluster_arrive();
            cluster_wait();
            fold<N>(mine, cs, rank, lane, mu, carry);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                mu[j] = carry[j];
                carry[j] = fmaf(all.a[j], carry[j], all.b[j]);
            }
        }
        float before[R][N];
#pragma unroll
        for (int j = 0; j < N; ++j) mu[j] = fmaf(pre.a[j], mu[j], pre.b[j]);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                before[i][j] = h[j];
                h[j] = fmaf(a[i][j], h[j], rest[i][j] * to_f32(v[i].v[j]));
            }
        if (n > 0 && tile >= 0) {
            const int64_t at = static_cast<int64_t>(row0) * p.D;
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                float og[N], ox[N];
                const bool live = row0 + i < len;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float lam = to_f32(d[i].v[j]) + mu[j];
                    mu[j] = a[i][j] * lam;
                    if (MODE == BASED_GATE_LOG)
                        og[j] = mu[j] * before[i][j], ox[j] = lam;
                    else
                        og[j] = mu[j] * rest[i][j] * (before[i][j] - to_f32(v[i].v[j])), ox[j] = rest[i][j] * lam;
                    og[j] = live ? og[j] : 0.0f;
                    ox[j] = live ? ox[j] : 0.0f;
                }
                if (row0 + i < p.T) {
                    store_channels<T, N>(dgate + at + static_cast<int64_t>(i) * p.D, og, n, p.pair);
                    store_channels<T, N>(dx + at + static_cast<int64_t>(i) * p.D, ox, n, p.pair);
                }
            }
        }
    }
    if (warp == 0 && rank == 0 && p.final_state) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < n) p.final_state[plane + j] = carry[j];
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
    if (static_cast<int64_t>(p.B) * p.D >= (1ll << 30) || p.T > (1 << 30)) return BASED_ERR_BAD_SIZE;
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

// Once per kernel and process: its shared memory above 48 KB and clusters of 16.
template <typename K>
cudaError_t allow(K *kernel, size_t smem) {
    static std::mutex m;
    static K *done[32];
    std::lock_guard<std::mutex> lk(m);
    int i = 0;
    for (; i < 32 && done[i]; ++i)
        if (done[i] == kernel) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && i < 32) done[i] = kernel;
    return e;
}

// per_sm: CTAs that an SM holds. Time is shared out among as many CTAs as there are slots and
// tiles for, so that few channels fill the GPU too.
template <typename T, typename Smem>
int launch_scan(ScanParams &p, void (*kernel)(ScanParams), int threads, int per_sm, int sms, cudaStream_t st) {
    p.slabs = (p.D + 32 * ScanCfg<T>::N - 1) / (32 * ScanCfg<T>::N);
    const int64_t blocks = static_cast<int64_t>(p.slabs) * p.B, tiles = (p.T + kTile - 1) / kTile;
    p.cluster = 1;
    while (p.cluster < kMaxCluster && p.cluster < tiles && blocks * p.cluster * 2 <= static_cast<int64_t>(sms) * per_sm)
        p.cluster *= 2;
    OPS_CUDA(allow(kernel, Smem::bytes(kMaxCluster)));
    OPS_CUDA(launch_op(kernel, dim3(static_cast<unsigned>(blocks * p.cluster)), threads, Smem::bytes(p.cluster), st, p, p.cluster));
    return BASED_OK;
}
template <typename T>
int launch_scan(ScanParams &p, int mode, bool bwd, int sms, cudaStream_t st) {
    const bool log = mode == BASED_GATE_LOG;
    if (bwd)
        return launch_scan<T, ScanSmem<ScanCfg<T>::N, kBwdWarps, 3, kBwdStages>>(
            p, log ? based_scan_bwd_kernel<T, BASED_GATE_LOG> : based_scan_bwd_kernel<T, BASED_GATE_SIGMOID>,
            32 * kBwdWarps, 2, sms, st);
    return launch_scan<T, typename ScanCfg<T>::Fwd>(
        p, log ? based_scan_fwd_kernel<T, BASED_GATE_LOG> : based_scan_fwd_kernel<T, BASED_GATE_SIGMOID>,
        32 * kFwdWarps, 4, sms, st);
}

int run_scan(ScanParams &p, int dtype, int mode, bool bwd, based_stream_t stream) {
    int rc = check_scan(p, dtype, mode, bwd), sms;
    if (rc != BASED_OK || (rc = host_device(&sms)) != BASED_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // the widest word that every row of every input starts on, and ends on
    const int64_t es = static_cast<int64_t>(elem_size(dtype));
    const int64_t bits = (p.D | p.gate_sb | p.gate_st | p.x_sb | p.x_st | p.dy_sb | p.dy_st) * es |
                         static_cast<int64_t>(reinterpret_cast<uintptr_t>(p.gate) | reinterpret_cast<uintptr_t>(p.x) |
                                              reinterpret_cast<uintptr_t>(p.dy));
    p.word = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
    p.pair = p.D % 2 == 0 && aligned(p.y, 4) && aligned(p.dx, 4);
    if (dtype == BASED_F32) return launch_scan<float>(p, mode, bwd, sms, st);
    if (dtype == BASED_BF16) return launch_scan<__nv_bfloat16>(p, mode, bwd, sms, st);
    return launch_scan<__half>(p, mode, bwd, sms, st);
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
