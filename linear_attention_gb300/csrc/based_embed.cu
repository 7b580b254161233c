// based_embed.cu: scaled embedding lookup and its gradient (declared in include/based_ops.h).
//
//     y_i = s E[id_i],    dE_v = s sum over i with id_i = v of dy_i
//
// The gradient is summed by sorted tokens. The (id, position) pairs are sorted by id with a stable
// counting sort, digit by digit; the sorted order is cut into tiles, a CTA sums the runs of equal
// ids in its tile, and runs that cross tiles are joined from float32 partial sums. The order of
// every sum follows from the ids alone, so that results repeat bit for bit, and a token that
// occurs thousands of times is spread over many CTAs.
#include "ops_common.cuh"

namespace based {
namespace {

constexpr int kSortThreads = 256;
constexpr int kSortChunk = 1024;    // keys a CTA ranks at a time, 128 a warp
constexpr int kMaxSortBlocks = 128;
constexpr int kMaxDigits = 1024;
constexpr int kTileRows = 32;       // sorted positions of a tile

struct EmbedParams {
    const void *ids, *table;
    int64_t table_sr, N;
    int ids64, V, D;
    float scale;
    void *y;
};

__device__ __forceinline__ int load_id(const void *ids, int ids64, int64_t i, int V) {
    const int64_t id = ids64 ? static_cast<const int64_t *>(ids)[i] : static_cast<const int32_t *>(ids)[i];
    return id >= 0 && id < V ? static_cast<int>(id) : V;  // V: padding
}

// blockDim.x threads along a row, N channels each; blockDim.y rows at a time.
template <typename T, int N>
__global__ void __launch_bounds__(256) based_embed_fwd_kernel(const EmbedParams p) {
    using W = Pack<T, N>;
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; i < p.N;
         i += static_cast<int64_t>(gridDim.x) * blockDim.y) {
        const int id = load_id(p.ids, p.ids64, i, p.V);
        const T *src = static_cast<const T *>(p.table) + id * p.table_sr;
        T *dst = static_cast<T *>(p.y) + i * p.D;
        for (int c = threadIdx.x * N; c < p.D; c += blockDim.x * N) {
            W w;
            if (id < p.V) w = *reinterpret_cast<const W *>(src + c);
#pragma unroll
            for (int j = 0; j < N; ++j) w.v[j] = from_f32<T>(id < p.V ? to_f32(w.v[j]) * p.scale : 0.0f);
            *reinterpret_cast<W *>(dst + c) = w;
        }
    }
}

struct SortParams {
    const void *ids;       // the first pass reads ids, the others key_in and pos_in
    const int32_t *key_in, *pos_in;
    int32_t *key_out, *pos_out, *hist;  // hist: (blocks, digits)
    int N, V, ids64, per;  // per: keys of a CTA, a multiple of kSortChunk
    int shift, digits;
};

__device__ __forceinline__ int sort_key(const SortParams &p, int i) {
    return p.ids ? load_id(p.ids, p.ids64, i, p.V) : p.key_in[i];
}

// How often each digit occurs among a CTA's keys.
__global__ void __launch_bounds__(kSortThreads) based_embed_count_kernel(const SortParams p) {
    __shared__ int cnt[kMaxDigits];
    griddep_wait();
    griddep_launch_dependents();
    for (int d = threadIdx.x; d < p.digits; d += kSortThreads) cnt[d] = 0;
    __syncthreads();
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * p.per, end = min(begin + p.per, static_cast<int64_t>(p.N));
    for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads)
        atomicAdd(&cnt[(sort_key(p, static_cast<int>(i)) >> p.shift) & (p.digits - 1)], 1);
    __syncthreads();
    for (int d = threadIdx.x; d < p.digits; d += kSortThreads)
        p.hist[static_cast<int64_t>(blockIdx.x) * p.digits + d] = cnt[d];
}

// Moves a CTA's keys to their places: those of smaller digits, then those of the same digit in
// earlier CTAs, earlier warps, earlier rounds and lower lanes come first.
__global__ void __launch_bounds__(kSortThreads) based_embed_place_kernel(const SortParams p) {
    __shared__ int base[kMaxDigits];
    __shared__ int cnt[kSortThreads / 32][kMaxDigits];
    __shared__ int warp_sum[kSortThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_wait();
    griddep_launch_dependents();
    const int blocks = gridDim.x, me = blockIdx.x;
    for (int d = threadIdx.x; d < kMaxDigits; d += kSortThreads) {
        int total = 0, before = 0;
        if (d < p.digits) {
#pragma unroll 8
            for (int k = 0; k < blocks; ++k) {
                const int v = p.hist[static_cast<int64_t>(k) * p.digits + d];
                total += v;
                before += k < me ? v : 0;
            }
        }
        base[d] = before;
        cnt[0][d] = total;
    }
    __syncthreads();
    {
        // exclusive sum of the digits' totals, four digits a thread
        int v[4], s = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = cnt[0][threadIdx.x * 4 + j], s += v[j];
        int incl = s;
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(~0u, incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int off = incl - s;
        for (int w = 0; w < warp; ++w) off += warp_sum[w];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            base[threadIdx.x * 4 + j] += off;
            off += v[j];
        }
    }
    const int64_t begin = static_cast<int64_t>(me) * p.per, end = min(begin + p.per, static_cast<int64_t>(p.N));
    for (int64_t chunk = begin; chunk < end; chunk += kSortChunk) {
        __syncthreads();
        for (int d = threadIdx.x; d < p.digits; d += kSortThreads) {
#pragma unroll
            for (int w = 0; w < kSortThreads / 32; ++w) cnt[w][d] = 0;
        }
        __syncthreads();
        constexpr int kRounds = kSortChunk / kSortThreads;
        int key[kRounds], rank[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int64_t i = chunk + warp * (32 * kRounds) + r * 32 + lane;
            key[r] = i < end ? sort_key(p, static_cast<int>(i)) : -1;
            const int d = key[r] < 0 ? -1 : (key[r] >> p.shift) & (p.digits - 1);
            const unsigned same = __match_any_sync(~0u, d);
            const int leader = __ffs(same) - 1;
            int old = 0;
            if (lane == leader && d >= 0) {
                old = cnt[warp][d];
                cnt[warp][d] = old + __popc(same);
            }
            rank[r] = __shfl_sync(~0u, old, leader) + __popc(same & ((1u << lane) - 1));
            __syncwarp();
        }
        __syncthreads();
        for (int d = threadIdx.x; d < p.digits; d += kSortThreads) {
            int off = base[d];
#pragma unroll
            for (int w = 0; w < kSortThreads / 32; ++w) {
                const int t = cnt[w][d];
                cnt[w][d] = off;
                off += t;
            }
            base[d] = off;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            if (key[r] < 0) continue;
            const int i = static_cast<int>(chunk) + warp * (32 * kRounds) + r * 32 + lane;
            const int at = cnt[warp][(key[r] >> p.shift) & (p.digits - 1)] + rank[r];
            p.key_out[at] = key[r];
            p.pos_out[at] = p.ids ? i : p.pos_in[i];
        }
    }
}

struct FillParams {
    void *out;
    int64_t words;  // 16-byte words
    int64_t bytes;
};

__global__ void __launch_bounds__(256) based_embed_zero_kernel(const FillParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t step = static_cast<int64_t>(gridDim.x) * 256, at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    for (int64_t i = at; i < p.words; i += step) static_cast<uint4 *>(p.out)[i] = make_uint4(0, 0, 0, 0);
    // the rest, or all of a table that starts off a 16-byte boundary, in the 2 bytes of the smallest type
    for (int64_t i = p.words * 8 + at; i < p.bytes / 2; i += step) static_cast<uint16_t *>(p.out)[i] = 0;
}

struct SumParams {
    const int32_t *key, *pos;
    const void *dy;
    int64_t dy_sr;
    int N, V, D;
    float scale;
    float *partial;  // (tiles, 2, D): of the run that began before a tile, and of one that goes on after it
    void *out;
};

template <typename G, int N>
__device__ __forceinline__ void store_row(const SumParams &p, int row, int c, const float (&acc)[N]) {
    G *out = static_cast<G *>(p.out) + static_cast<int64_t>(row) * p.D + c;
    constexpr int kPer = sizeof(G) * N > 16 ? 16 / sizeof(G) : N;
#pragma unroll
    for (int k = 0; k < N / kPer; ++k) {
        Pack<G, kPer> w;
#pragma unroll
        for (int j = 0; j < kPer; ++j) w.v[j] = from_f32<G>(acc[k * kPer + j] * p.scale);
        *reinterpret_cast<Pack<G, kPer> *>(out + k * kPer) = w;
    }
}

// A CTA sums the runs of one tile of the sorted order, N channels a thread.
template <typename T, typename G, int N>
__global__ void __launch_bounds__(256) based_embed_sum_kernel(const SumParams p) {
    constexpr int kPer = sizeof(T) * N > 16 ? 16 / sizeof(T) : N, kWords = N / kPer, kAhead = 8;
    using W = Pack<T, kPer>;
    __shared__ int key[kTileRows + 2], pos[kTileRows];
    griddep_wait();
    griddep_launch_dependents();
    const int tile = blockIdx.x, c = (blockIdx.y * blockDim.x + threadIdx.x) * N;
    const int64_t begin = static_cast<int64_t>(tile) * kTileRows;
    const int n = static_cast<int>(min(static_cast<int64_t>(kTileRows), p.N - begin));
    for (int i = threadIdx.x; i < kTileRows + 2; i += blockDim.x) {
        const int64_t at = begin + i - 1;
        key[i] = at >= 0 && at < p.N ? p.key[at] : -1;
        if (i < n) pos[i] = p.pos[begin + i];
    }
    __syncthreads();
    if (c >= p.D) return;
    const T *dy = static_cast<const T *>(p.dy) + c;
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    bool before = key[0] == key[1];  // the run began in an earlier tile
    float *partial = p.partial + (static_cast<int64_t>(tile) * 2) * p.D + c;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        W w[kAhead][kWords];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i0 + k < n && key[i0 + k + 1] < p.V) {
                const T *row = dy + pos[i0 + k] * p.dy_sr;
#pragma unroll
                for (int q = 0; q < kWords; ++q) w[k][q] = *reinterpret_cast<const W *>(row + q * kPer);
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k;
            if (i >= n || key[i + 1] >= p.V) break;  // padding sorts last
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += to_f32(w[k][j / kPer].v[j % kPer]);
            const bool last = i == n - 1;
            if (!last && key[i + 2] == key[i + 1]) continue;
            const bool after = last && key[i + 2] == key[i + 1];
            if (!before && !after) {
                store_row<G, N>(p, key[i + 1], c, acc);
            } else {
                float *to = partial + (before ? 0 : p.D);
#pragma unroll
                for (int j = 0; j < N; ++j) to[j] = acc[j];
            }
            before = false;
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = 0.0f;
        }
    }
}

// Joins each run that crosses tiles, in the CTA of the tile it begins in.
template <typename G, int N>
__global__ void __launch_bounds__(256) based_embed_join_kernel(const SumParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int tile = blockIdx.x, c = (blockIdx.y * blockDim.x + threadIdx.x) * N;
    const int64_t begin = static_cast<int64_t>(tile) * kTileRows, end = begin + kTileRows;
    if (end >= p.N || c >= p.D) return;  // nothing goes on after the last tile
    const int k = p.key[end - 1];
    if (k >= p.V || p.key[end] != k) return;
    if (begin > 0 && p.key[begin] == k && p.key[begin - 1] == k) return;  // it began earlier
    float acc[N];
    const float *from = p.partial + (static_cast<int64_t>(tile) * 2 + 1) * p.D + c;
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = from[j];
    for (int64_t t = tile + 1; t * kTileRows < p.N && p.key[t * kTileRows] == k; ++t) {
        from = p.partial + t * 2 * p.D + c;
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += from[j];
    }
    store_row<G, N>(p, k, c, acc);
}

// Where the parts of based_embed_bwd's workspace lie.
struct EmbedPlan {
    int passes, bits, blocks, per, tiles;
    size_t key, pos, hist, partial, bytes;  // key and pos: two buffers each
};
bool embed_plan(int64_t N, int V, int D, EmbedPlan &e) {
    if (N < 1 || V < 1 || D < 1 || N >= (1ll << 30)) return false;
    int bits = 1;
    while ((static_cast<int64_t>(V) >> bits) != 0) ++bits;  // V itself is the key of padding
    e.passes = (bits + 9) / 10;                              // at most kMaxDigits digits a pass
    e.bits = (bits + e.passes - 1) / e.passes;
    int64_t per = (N + kMaxSortBlocks - 1) / kMaxSortBlocks;
    per = (per + kSortChunk - 1) / kSortChunk * kSortChunk;
    e.per = static_cast<int>(per);
    e.blocks = static_cast<int>((N + per - 1) / per);
    e.tiles = static_cast<int>((N + kTileRows - 1) / kTileRows);
    auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
    const size_t list = up(static_cast<size_t>(N) * 4);
    e.key = 0;
    e.pos = 2 * list;
    e.hist = 4 * list;
    e.partial = e.hist + up(static_cast<size_t>(e.blocks) * (1 << e.bits) * 4);
    e.bytes = e.partial + static_cast<size_t>(e.tiles) * 2 * D * 4;
    return true;
}

template <typename T, typename G, int N>
int launch_sums(const SumParams &p, int tiles, cudaStream_t st) {
    const int need = (p.D + N - 1) / N, threads = need >= 256 ? 256 : (need + 31) / 32 * 32;
    const dim3 grid(tiles, (need + threads - 1) / threads);
    OPS_CUDA(launch_op(based_embed_sum_kernel<T, G, N>, grid, threads, 0, st, p));
    OPS_CUDA(launch_op(based_embed_join_kernel<G, N>, grid, threads, 0, st, p));
    return BASED_OK;
}
template <typename T>
int launch_sums(const SumParams &p, int g_dtype, bool wide, int tiles, cudaStream_t st) {
    if (g_dtype == BASED_F32) return wide ? launch_sums<T, float, 8>(p, tiles, st) : launch_sums<T, float, 1>(p, tiles, st);
    return wide ? launch_sums<T, T, 8>(p, tiles, st) : launch_sums<T, T, 1>(p, tiles, st);
}

template <typename T, int N>
int launch_embed(const EmbedParams &p, int sms, cudaStream_t st) {
    int tx = 32;
    while (tx < 256 && tx * N < p.D) tx *= 2;
    const int ty = 256 / tx;
    const int64_t need = (p.N + ty - 1) / ty, most = sms * 8ll;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(need < most ? need : most));
    cfg.blockDim = dim3(tx, ty);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    OPS_CUDA(cudaLaunchKernelEx(&cfg, based_embed_fwd_kernel<T, N>, p));
    return BASED_OK;
}

}  // namespace
}  // namespace based

extern "C" {

int based_embed_fwd(const void *ids, int ids64, const void *table, int64_t table_sr, int64_t N, int V, int D,
                    int dtype, float scale, void *y, based_stream_t stream) {
    using namespace based;
    if (!ids || !table || !y) return BASED_ERR_NULL_POINTER;
    if (!type_ok(dtype)) return BASED_ERR_UNSUPPORTED_TYPE;
    if (N < 1 || V < 1 || D < 1 || D > (1 << 30) || N >= (1ll << 40)) return BASED_ERR_BAD_SIZE;
    if (table_sr < 0) return BASED_ERR_BAD_STRIDE;
    const size_t es = elem_size(dtype), is = ids64 ? 8 : 4;
    if (!aligned(ids, is) || !aligned(table, es) || !aligned(y, es)) return BASED_ERR_MISALIGNED;
    const Span sy = span(y, N * D - 1, es);
    if (overlap(sy, span(ids, N - 1, is)) || overlap(sy, span(table, (V - 1) * table_sr + D - 1, es)))
        return BASED_ERR_ALIASING;
    int sms;
    const int rc = host_device(&sms);
    if (rc != BASED_OK) return rc;
    const EmbedParams p = {ids, table, table_sr, N, ids64 ? 1 : 0, V, D, scale, y};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool wide = aligned(table, 16) && aligned(y, 16) && table_sr * es % 16 == 0 && D * es % 16 == 0;
    if (dtype == BASED_F32) return wide ? launch_embed<float, 4>(p, sms, st) : launch_embed<float, 1>(p, sms, st);
    if (dtype == BASED_BF16)
        return wide ? launch_embed<__nv_bfloat16, 8>(p, sms, st) : launch_embed<__nv_bfloat16, 1>(p, sms, st);
    return wide ? launch_embed<__half, 8>(p, sms, st) : launch_embed<__half, 1>(p, sms, st);
}

size_t based_embed_bwd_workspace_size(int64_t N, int V, int D) {
    based::EmbedPlan e;
    return based::embed_plan(N, V, D, e) ? e.bytes : 0;
}

int based_embed_bwd(const void *ids, int ids64, const void *dy, int64_t dy_sr, int64_t N, int V, int D, int dtype,
                    float scale, void *dtable, int g_dtype, void *workspace, size_t ws_bytes, based_stream_t stream) {
    using namespace based;
    if (!ids || !dy || !dtable) return BASED_ERR_NULL_POINTER;
    if (!type_ok(dtype) || !type_ok(g_dtype) || (g_dtype != BASED_F32 && g_dtype != dtype))
        return BASED_ERR_UNSUPPORTED_TYPE;
    EmbedPlan e;
    if (!embed_plan(N, V, D, e) || D > (1 << 20)) return BASED_ERR_BAD_SIZE;
    if (dy_sr < 0) return BASED_ERR_BAD_STRIDE;
    const size_t es = elem_size(dtype), gs = elem_size(g_dtype), is = ids64 ? 8 : 4;
    if (!aligned(ids, is) || !aligned(dy, es) || !aligned(dtable, gs)) return BASED_ERR_MISALIGNED;
    const Span so = span(dtable, static_cast<int64_t>(V) * D - 1, gs);
    if (overlap(so, span(ids, N - 1, is)) || overlap(so, span(dy, (N - 1) * dy_sr + D - 1, es)))
        return BASED_ERR_ALIASING;
    if (!workspace || !aligned(workspace, 16) || ws_bytes < e.bytes) return BASED_ERR_WORKSPACE;
    int sms;
    const int rc = host_device(&sms);
    if (rc != BASED_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    int32_t *key[2], *pos[2];
    for (int i = 0; i < 2; ++i) {
        key[i] = reinterpret_cast<int32_t *>(ws + e.key + i * (e.pos / 2));
        pos[i] = reinterpret_cast<int32_t *>(ws + e.pos + i * (e.pos / 2));
    }
    const int64_t out_bytes = static_cast<int64_t>(V) * D * gs;
    const FillParams f = {dtable, aligned(dtable, 16) ? out_bytes / 16 : 0, out_bytes};
    OPS_CUDA(launch_op(based_embed_zero_kernel, dim3(sms * 8), 256, 0, st, f));
    for (int i = 0; i < e.passes; ++i) {
        const SortParams s = {i == 0 ? ids : nullptr,
                              key[(i + 1) & 1],
                              pos[(i + 1) & 1],
                              key[i & 1],
                              pos[i & 1],
                              reinterpret_cast<int32_t *>(ws + e.hist),
                              static_cast<int>(N),
                              V,
                              ids64 ? 1 : 0,
                              e.per,
                              i * e.bits,
                              1 << e.bits};
        OPS_CUDA(launch_op(based_embed_count_kernel, dim3(e.blocks), kSortThreads, 0, st, s));
        OPS_CUDA(launch_op(based_embed_place_kernel, dim3(e.blocks), kSortThreads, 0, st, s));
    }
    const int done = (e.passes - 1) & 1;
    const SumParams p = {key[done], pos[done], dy, dy_sr, static_cast<int>(N), V, D, scale,
                         reinterpret_cast<float *>(ws + e.partial), dtable};
    const bool wide = D % 8 == 0 && aligned(dy, 16) && dy_sr * es % 16 == 0 && aligned(dtable, 16);
    if (dtype == BASED_F32) return launch_sums<float>(p, g_dtype, wide, e.tiles, st);
    if (dtype == BASED_BF16) return launch_sums<__nv_bfloat16>(p, g_dtype, wide, e.tiles, st);
    return launch_sums<__half>(p, g_dtype, wide, e.tiles, st);
}

}  // extern "C"
