// based_embed.cu: scaled embedding lookup and its gradient (declared in include/based_ops.h).
//
//     y_i = s E[id_i],    dE_v = s sum over i with id_i = v of dy_i
//
// The gradient is summed by sorted tokens, in three launches. One cluster sorts the (id, position)
// pairs by id with a stable counting sort, digit by digit, while the other clusters of the same
// launch write the zeros of the gradient. The sorted order is cut into tiles, a CTA sums the runs of
// equal ids in its tile, and runs that cross tiles are joined from float32 partial sums. The order
// of every sum follows from the ids alone, so that results repeat bit for bit, and a token that
// occurs thousands of times is spread over many CTAs. A few tokens (up to 1024) take two launches:
// each finds its place by counting the smaller ones, and a CTA sums a whole run.
#include "ops_common.cuh"

namespace based {
namespace {

constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;  // two CTAs an SM
constexpr int kSortCluster = 8, kWideCluster = 16;         // CTAs that sort
constexpr int kSortRounds = 8;                             // keys that a thread holds, at most
constexpr int kSortChunk = kSortThreads * kSortRounds;
constexpr int kMaxBits = 9;                                // of a digit
constexpr int kFewTokens = 1024, kFewVocab = 1 << 22;      // tokens that are ranked directly (ids of 22 bits)
constexpr int kTileRows = 32;                              // sorted positions of a tile, at most

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
    const void *ids;
    int32_t *key0, *key1, *pos0, *pos1;  // pass i writes lists i & 1; the first reads ids
    int N, V, ids64, few, passes, bits;
    void *out;                 // the gradient: `words` 16-byte words, then bytes up to `bytes`
    int64_t words, bytes;
};

__device__ __forceinline__ int load_remote(const int *p, int rank) {
    uint32_t at;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

struct SortSmem {
    int hist[1 << kMaxBits];   // digits of this CTA's keys
    int base[1 << kMaxBits];   // where the next key of each digit goes
    int warp_sum[kSortWarps];
    int cnt[kSortWarps][1 << kMaxBits];
};

constexpr int kFillBytes = 16384;  // zeros that one copy writes
static_assert(sizeof(SortSmem) >= kFillBytes, "the zeros lie in the sort's shared memory");
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, int bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

// A chunk of a CTA's keys in registers: `rounds` keys a thread, a warp's keys consecutive.
struct SortChunk {
    int key[kSortRounds], pos[kSortRounds], rank[kSortRounds];
    int rounds;
    int64_t first;

    __device__ __forceinline__ void load(const SortParams &p, int pass, int64_t begin, int64_t end) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int64_t n = min(end - begin, static_cast<int64_t>(kSortChunk)), last = begin + n;
        rounds = static_cast<int>((n + kSortThreads - 1) / kSortThreads);
        first = begin + warp * 32 * rounds + lane;
        if (n <= 0) return;
        // loads that depend on nothing (past the end the last key again), so that all are under way at once
        int64_t at[kSortRounds];
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) at[r] = min(first + r * 32, last - 1);
        if (pass > 0) {
            const int32_t *key_in = pass & 1 ? p.key0 : p.key1, *pos_in = pass & 1 ? p.pos0 : p.pos1;
#pragma unroll
            for (int r = 0; r < kSortRounds; ++r) key[r] = __ldcg(key_in + at[r]);
#pragma unroll
            for (int r = 0; r < kSortRounds; ++r) pos[r] = __ldcg(pos_in + at[r]);
        } else {
            int64_t id[kSortRounds];
            if (p.ids64) {
#pragma unroll
                for (int r = 0; r < kSortRounds; ++r) id[r] = static_cast<const int64_t *>(p.ids)[at[r]];
            } else {
#pragma unroll
                for (int r = 0; r < kSortRounds; ++r) id[r] = static_cast<const int32_t *>(p.ids)[at[r]];
            }
#pragma unroll
            for (int r = 0; r < kSortRounds; ++r) {
                key[r] = id[r] >= 0 && id[r] < p.V ? static_cast<int>(id[r]) : p.V;
                pos[r] = static_cast<int>(at[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r)
            if (r >= rounds || first + r * 32 >= last) key[r] = -1;
    }
    // rank: how many earlier keys of the warp have the key's digit; cnt[warp]: the warp's digits
    __device__ __forceinline__ void count(SortSmem &sm, int shift, int digits) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        for (int d = lane; d < digits; d += 32) sm.cnt[warp][d] = 0;
        __syncwarp();
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) {
            if (r >= rounds) break;
            // lanes with the same digit, bit by bit: nine votes are faster than matching whole
            // digits (25 instead of 27 us for the sort of 32768 tokens)
            const int d = (key[r] >> shift) & (digits - 1);
            unsigned same = __ballot_sync(~0u, key[r] >= 0);
#pragma unroll
            for (int b = 0; b < kMaxBits; ++b) {
                const unsigned set = __ballot_sync(~0u, d >> b & 1);
                same &= d >> b & 1 ? set : ~set;
            }
            const int leader = same ? __ffs(same) - 1 : 0;
            int old = 0;
            if (lane == leader && key[r] >= 0) {
                old = sm.cnt[warp][d];
                sm.cnt[warp][d] = old + __popc(same);
            }
            rank[r] = __shfl_sync(~0u, old, leader) + __popc(same & ((1u << lane) - 1));
            __syncwarp();
        }
    }
    // cnt[warp][d] becomes the count in earlier warps, counted from `start`; returns the end
    __device__ __forceinline__ static int scan_warps(SortSmem &sm, int d, int start) {
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int t = sm.cnt[w][d];
            sm.cnt[w][d] = start;
            start += t;
        }
        return start;
    }
    // base: added to the counts (where a chunk is a CTA's only one), or NULL
    __device__ __forceinline__ void place(const SortParams &p, const SortSmem &sm, int pass, int shift, int digits, const int *base) {
        int32_t *key_out = pass & 1 ? p.key1 : p.key0, *pos_out = pass & 1 ? p.pos1 : p.pos0;
        const int warp = threadIdx.x >> 5;
#pragma unroll
        for (int r = 0; r < kSortRounds; ++r) {
            if (r >= rounds || key[r] < 0) continue;
            const int d = (key[r] >> shift) & (digits - 1), at = sm.cnt[warp][d] + rank[r] + (base ? base[d] : 0);
            key_out[at] = key[r];
            pos_out[at] = pos[r];
        }
    }
};

// Few tokens: a token's place is the number of smaller (id, position) pairs, and every pair fits one
// word. Each CTA of the first cluster places an eighth of the tokens, 512 / (N / 8) threads a token.
// With the kernel that sums whole runs, the gradient of 512 tokens (8192 x 512) takes 8.4 us, where the
// counting sort, tiles and joins take 11.3; of 1024 tokens 10.3, where they take 13.0.
__device__ __forceinline__ void rank_few(const SortParams &p, uint32_t *all) {
    const int tid = threadIdx.x, n4 = (p.N + 3) / 4;
    for (int i = tid; i < n4 * 4; i += kSortThreads)
        all[i] = i < p.N ? static_cast<uint32_t>(load_id(p.ids, p.ids64, i, p.V)) << 10 | i : ~0u;
    __syncthreads();
    const int per = (p.N + kSortCluster - 1) / kSortCluster;  // tokens of a CTA: at most 128
    const int split = per <= 16 ? 32 : per <= 32 ? 16 : per <= 64 ? 8 : 4, part = tid % split, mine = tid / split;
    const int i = static_cast<int>(blockIdx.x) * per + mine;
    const bool on = mine < per && i < p.N;
    const uint32_t me = on ? all[i] : 0;
    int rank = 0;
    for (int j = part; j < n4; j += split) {
        const uint4 q = reinterpret_cast<const uint4 *>(all)[j];
        rank += (q.x < me) + (q.y < me) + (q.z < me) + (q.w < me);
    }
    for (int d = split >> 1; d > 0; d >>= 1) rank += __shfl_xor_sync(~0u, rank, d);
    if (on && part == 0) {
        p.key0[rank] = static_cast<int>(me >> 10);
        p.pos0[rank] = i;
    }
}

// The first cluster sorts: each of its CTAs takes an equal part of the keys. Per pass and CTA: count the
// digits; read the other CTAs' counts through distributed shared memory; move each key behind those
// of smaller digits, then those of the same digit in earlier CTAs, warps, rounds and lanes. On one
// cluster a pass costs barriers of a few hundred nanoseconds where launches of their own cost
// microseconds. Up to 4096 tokens a CTA every key is loaded once a pass; more go through twice, in chunks.
template <int CLUSTER>
__global__ void __launch_bounds__(kSortThreads, 2) based_embed_sort_kernel(const SortParams p) {
    extern __shared__ __align__(128) int raw[];
    SortSmem &sm = *reinterpret_cast<SortSmem *>(raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x >= CLUSTER) {
        const int64_t step = static_cast<int64_t>(gridDim.x - CLUSTER) * kSortThreads;
        const int64_t at = static_cast<int64_t>(blockIdx.x - CLUSTER) * kSortThreads + tid;
        // bulk copies of zeros from shared memory, by one thread
        for (int i = tid; i < kFillBytes / 16; i += kSortThreads) reinterpret_cast<uint4 *>(raw)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            const int64_t n = p.words * 16;
            for (int64_t i = static_cast<int64_t>(blockIdx.x - CLUSTER) * kFillBytes; i < n;
                 i += static_cast<int64_t>(gridDim.x - CLUSTER) * kFillBytes)
                bulk_store(static_cast<uint8_t *>(p.out) + i, smem_u32(raw), static_cast<int>(min(n - i, static_cast<int64_t>(kFillBytes))));
            bulk_commit_group();
            bulk_wait_group_all();
        }
        // the rest, or all of a table that starts off a 16-byte boundary, in the 2 bytes of the smallest type
        for (int64_t i = p.words * 8 + at; i < p.bytes / 2; i += step) static_cast<uint16_t *>(p.out)[i] = 0;
        return;
    }
    if (p.few) {
        rank_few(p, reinterpret_cast<uint32_t *>(raw));
        return;
    }
    const int rank = static_cast<int>(cluster_rank()), digits = 1 << p.bits;
    const int64_t begin = static_cast<int64_t>(p.N) * rank / CLUSTER;
    const int64_t end = static_cast<int64_t>(p.N) * (rank + 1) / CLUSTER;
    const bool once = end - begin <= kSortChunk;
    SortChunk ch;
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * p.bits;
        if (once) {
            ch.load(p, pass, begin, end);
            ch.count(sm, shift, digits);
            __syncthreads();
            if (tid < digits) sm.hist[tid] = SortChunk::scan_warps(sm, tid, 0);
        } else {
            int mine = 0;
            for (int64_t chunk = begin; chunk < end; chunk += kSortChunk) {
                ch.load(p, pass, chunk, end);
                ch.count(sm, shift, digits);
                __syncthreads();
                if (tid < digits) {
#pragma unroll
                    for (int w = 0; w < kSortWarps; ++w) mine += sm.cnt[w][tid];
                }
                __syncthreads();
            }
            if (tid < digits) sm.hist[tid] = mine;
        }
        cluster_sync();
        int total = 0, before = 0;
        if (tid < digits) {
            int v[CLUSTER];
#pragma unroll
            for (int r = 0; r < CLUSTER; ++r) v[r] = load_remote(&sm.hist[tid], r);
#pragma unroll
            for (int r = 0; r < CLUSTER; ++r) {
                total += v[r];
                before += r < rank ? v[r] : 0;
            }
        }
        // exclusive sum of the totals over the digits
        int incl = total;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(~0u, incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 31) sm.warp_sum[warp] = incl;
        __syncthreads();
        if (tid < digits) {
            int off = incl - total + before;
            for (int w = 0; w < warp; ++w) off += sm.warp_sum[w];
            sm.base[tid] = off;
        }
        __syncthreads();
        if (once) {
            ch.place(p, sm, pass, shift, digits, sm.base);
        } else {
            for (int64_t chunk = begin; chunk < end; chunk += kSortChunk) {
                ch.load(p, pass, chunk, end);
                ch.count(sm, shift, digits);
                __syncthreads();
                if (tid < digits) sm.base[tid] = SortChunk::scan_warps(sm, tid, sm.base[tid]);
                __syncthreads();
                ch.place(p, sm, pass, shift, digits, nullptr);
                __syncthreads();
            }
        }
        // the counts were read and the keys are in place everywhere before the next pass
        cluster_sync();
    }
}

struct SumParams {
    const int32_t *key, *pos;
    const void *dy;
    int64_t dy_sr;
    int N, V, D;
    int rows;        // sorted positions of a tile
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

// A CTA sums the runs of one tile of the sorted order, N channels a thread. Bound by the latency of the rows it
// gathers, eight under way a thread: 19 us for 32768 rows of 1024, 60 MB read and 40 MB written (15 us at
// the memory's rate).
template <typename T, typename G, int N>
__global__ void __launch_bounds__(256) based_embed_sum_kernel(const SumParams p) {
    constexpr int kPer = sizeof(T) * N > 16 ? 16 / sizeof(T) : N, kWords = N / kPer, kAhead = 8;
    using W = Pack<T, kPer>;
    __shared__ int key[kTileRows + 2], pos[kTileRows];
    griddep_wait();
    griddep_launch_dependents();
    const int tile = blockIdx.x, c = (blockIdx.y * blockDim.x + threadIdx.x) * N;
    const int64_t begin = static_cast<int64_t>(tile) * p.rows;
    const int n = static_cast<int>(min(static_cast<int64_t>(p.rows), p.N - begin));
    for (int i = threadIdx.x; i < p.rows + 2; i += blockDim.x) {
        const int64_t at = begin + i - 1;
        key[i] = at >= 0 && at < p.N ? p.key[at] : -1;
        if (i < n) pos[i] = p.pos[begin + i];
    }
    // padding sorts last: the rows in front of it
    const int live = __syncthreads_count(static_cast<int>(threadIdx.x) < n && p.key[begin + threadIdx.x] < p.V);
    if (c >= p.D) return;
    const T *dy = static_cast<const T *>(p.dy) + c;
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    bool before = key[0] == key[1];  // the run began in an earlier tile
    float *partial = p.partial + (static_cast<int64_t>(tile) * 2) * p.D + c;
    for (int i0 = 0; i0 < live; i0 += kAhead) {
        // loads that depend on no condition (past the end the last row again), so that all are under way at once
        W w[kAhead][kWords];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const T *row = dy + pos[min(i0 + k, live - 1)] * p.dy_sr;
#pragma unroll
            for (int q = 0; q < kWords; ++q) w[k][q] = *reinterpret_cast<const W *>(row + q * kPer);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k;
            if (i < live) {
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] += to_f32(w[k][j / kPer].v[j % kPer]);
                const bool same = key[i + 2] == key[i + 1];
                if (!same || i == n - 1) {
                    if (!before && !same) {
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
    }
}

// Few tokens: the CTA of the sorted position where a run begins sums all of it. blockDim.x threads
// along the columns, N channels each; blockDim.y share the rows.
constexpr int kRunLanes = 8;
template <typename T, typename G, int N>
__global__ void __launch_bounds__(32 * kRunLanes) based_embed_run_kernel(const SumParams p) {
    constexpr int kPer = sizeof(T) * N > 16 ? 16 / sizeof(T) : N, kWords = N / kPer, kAhead = 4;
    using W = Pack<T, kPer>;
    __shared__ float red[kRunLanes][N][32];
    griddep_wait();
    griddep_launch_dependents();
    const int first = blockIdx.x, lane = threadIdx.x, row = threadIdx.y, c = (blockIdx.y * 32 + lane) * N;
    const int k = p.key[first];
    if (k >= p.V || (first > 0 && p.key[first - 1] == k)) return;
    int last = first;  // 32 positions at a time
    for (unsigned same = ~0u; same == ~0u;) {
        const int at = last + 1 + lane;
        same = __ballot_sync(~0u, at < p.N && p.key[at < p.N ? at : 0] == k);
        last += same == ~0u ? 32 : __ffs(~same) - 1;
    }
    float acc[N];
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
    const T *dy = static_cast<const T *>(p.dy) + (c < p.D ? c : 0);
    for (int i0 = first + row; i0 <= last; i0 += kAhead * kRunLanes) {
        W w[kAhead][kWords];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const T *src = dy + p.pos[min(i0 + a * kRunLanes, last)] * p.dy_sr;
#pragma unroll
            for (int q = 0; q < kWords; ++q) w[a][q] = *reinterpret_cast<const W *>(src + q * kPer);
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += i0 + a * kRunLanes <= last ? to_f32(w[a][j / kPer].v[j % kPer]) : 0.0f;
        }
    }
    if (last > first) {
#pragma unroll
        for (int j = 0; j < N; ++j) red[row][j][lane] = acc[j];
        __syncthreads();
        if (row == 0) {
#pragma unroll
            for (int r = 1; r < kRunLanes; ++r) {
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] += red[r][j][lane];
            }
        }
    }
    if (row == 0 && c < p.D) store_row<G, N>(p, k, c, acc);
}

// Joins each run that crosses tiles: a warp looks at one tile and 32 N columns, and sums the run that begins
// there and goes on after it; the CTA's warps share a run of more than kJoinAlone tiles.
constexpr int kJoinWarps = 8, kJoinAlone = 8;
template <typename G, int N>
__global__ void __launch_bounds__(32 * kJoinWarps) based_embed_join_kernel(const SumParams p) {
    __shared__ float red[kJoinWarps][N][32];
    __shared__ int64_t last_of[kJoinWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (blockIdx.y * 32 + lane) * N;
    // lane i: the partial sums of tiles first + i, first + i + step, ... up to last
    auto add = [&](float (&acc)[N], int64_t tile, int64_t first, int64_t last, int step) {
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = 0.0f;
        if (c >= p.D) return;
#pragma unroll 4
        for (int64_t t = first; t <= last; t += step) {
            const float *from = p.partial + (t * 2 + (t == tile ? 1 : 0)) * p.D + c;
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += from[j];
        }
    };
    const int64_t tile0 = static_cast<int64_t>(blockIdx.x) * kJoinWarps, tile = tile0 + warp;
    const int64_t begin = tile * p.rows, end = begin + p.rows;
    int64_t last = -1;  // the last tile of the run that begins in this one and goes on; -1: none does
    if (end < p.N) {
        // the tile's last key, the next one, its first and the one before; then the first keys of the tiles after the next
        const int k = p.key[end], in = p.key[end - 1], first = p.key[begin], earlier = begin > 0 ? p.key[begin - 1] : -1;
        if (k < p.V && in == k && !(first == k && earlier == k)) {
            last = tile;
            for (unsigned same = ~0u; same == ~0u;) {  // 32 tiles at a time
                const int64_t at = (last + 1 + lane) * p.rows;
                same = __ballot_sync(~0u, at < p.N && p.key[at < p.N ? at : 0] == k);
                last += same == ~0u ? 32 : __ffs(~same) - 1;
            }
            if (last - tile < kJoinAlone) {
                float acc[N];
                add(acc, tile, tile, last, 1);
                if (c < p.D) store_row<G, N>(p, k, c, acc);
                last = -1;
            }
        }
    }
    if (lane == 0) last_of[warp] = last;
    __syncthreads();
    for (int w = 0; w < kJoinWarps; ++w) {
        if (last_of[w] < 0) continue;
        float acc[N];
        add(acc, tile0 + w, tile0 + w + warp, last_of[w], kJoinWarps);
#pragma unroll
        for (int j = 0; j < N; ++j) red[warp][j][lane] = acc[j];
        __syncthreads();
        if (warp == 0 && c < p.D) {
#pragma unroll
            for (int i = 1; i < kJoinWarps; ++i) {
#pragma unroll
                for (int j = 0; j < N; ++j) acc[j] += red[i][j][lane];
            }
            store_row<G, N>(p, p.key[(tile0 + w + 1) * p.rows], c, acc);
        }
        __syncthreads();
    }
}

// Where the parts of based_embed_bwd's workspace lie.
struct EmbedPlan {
    int few, passes, bits, rows, tiles;
    size_t list, partial, bytes;  // two lists of keys, two of positions, the partial sums
};
bool embed_plan(int64_t N, int V, int D, EmbedPlan &e) {
    if (N < 1 || V < 1 || D < 1 || N >= (1ll << 30) || D > (1 << 20)) return false;
    int bits = 1;
    while ((static_cast<int64_t>(V) >> bits) != 0) ++bits;  // V itself is the key of padding
    e.few = N <= kFewTokens && V < kFewVocab;
    e.passes = e.few ? 1 : (bits + kMaxBits - 1) / kMaxBits;
    e.bits = (bits + e.passes - 1) / e.passes;
    // Fewer tokens: shorter tiles, so that more CTAs share them. Tiles of 8 and of 32 take 16.0 and 18.3 us
    // for 2048 tokens, 17.9 and 18.9 for 6000, 80 and 63 for 32768 (with their partial sums' traffic).
    e.rows = N >= 8192 ? kTileRows : 8;
    e.tiles = static_cast<int>((N + e.rows - 1) / e.rows);
    e.list = (static_cast<size_t>(N) * 4 + 255) & ~static_cast<size_t>(255);
    e.partial = 4 * e.list;
    e.bytes = e.partial + (e.few ? 0 : static_cast<size_t>(e.tiles) * 2 * D * 4);
    return true;
}

template <typename T, typename G, int N>
int launch_sums(const SumParams &p, const EmbedPlan &e, cudaStream_t st) {
    const int need = (p.D + N - 1) / N, threads = need >= 256 ? 256 : (need + 31) / 32 * 32;
    const unsigned tiles = static_cast<unsigned>(e.tiles);
    if (e.few) {
        OPS_CUDA(launch_op(based_embed_run_kernel<T, G, N>, dim3(p.N, (need + 31) / 32), dim3(32, kRunLanes), 0, st, p));
        return BASED_OK;
    }
    OPS_CUDA(launch_op(based_embed_sum_kernel<T, G, N>, dim3(tiles, (need + threads - 1) / threads), threads, 0, st, p));
    OPS_CUDA(launch_op(based_embed_join_kernel<G, N>, dim3((tiles + kJoinWarps - 1) / kJoinWarps, (need + 31) / 32),
                       32 * kJoinWarps, 0, st, p));
    return BASED_OK;
}
template <typename T>
int launch_sums(const SumParams &p, int g_dtype, bool wide, const EmbedPlan &e, cudaStream_t st) {
    if (g_dtype == BASED_F32) return wide ? launch_sums<T, float, 8>(p, e, st) : launch_sums<T, float, 1>(p, e, st);
    return wide ? launch_sums<T, T, 8>(p, e, st) : launch_sums<T, T, 1>(p, e, st);
}

template <typename T, int N>
int launch_embed(const EmbedParams &p, int sms, cudaStream_t st) {
    int tx = 32;
    while (tx < 256 && tx * N < p.D) tx *= 2;
    const int ty = 256 / tx;
    const int64_t need = (p.N + ty - 1) / ty, most = sms * 8ll;
    OPS_CUDA(launch_op(based_embed_fwd_kernel<T, N>, dim3(static_cast<unsigned>(need < most ? need : most)), dim3(tx, ty), 0, st, p));
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
    // 16-byte words where every row starts on one (32768 rows of 1024: 17 us, 46 by single elements)
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
    if (!embed_plan(N, V, D, e)) return BASED_ERR_BAD_SIZE;
    if (dy_sr < 0) return BASED_ERR_BAD_STRIDE;
    const size_t es = elem_size(dtype), gs = elem_size(g_dtype), is = ids64 ? 8 : 4;
    if (!aligned(ids, is) || !aligned(dy, es) || !aligned(dtable, gs)) return BASED_ERR_MISALIGNED;
    const Span so = span(dtable, static_cast<int64_t>(V) * D - 1, gs);
    if (overlap(so, span(ids, N - 1, is)) || overlap(so, span(dy, (N - 1) * dy_sr + D - 1, es)))
        return BASED_ERR_ALIASING;
    if (!workspace || !aligned(workspace, 16) || ws_bytes < e.bytes) return BASED_ERR_WORKSPACE;
    const Span sw = span(workspace, static_cast<int64_t>(e.bytes) - 1, 1);
    if (overlap(sw, so) || overlap(sw, span(ids, N - 1, is)) || overlap(sw, span(dy, (N - 1) * dy_sr + D - 1, es)))
        return BASED_ERR_ALIASING;
    int sms;
    int rc = host_device(&sms);
    if (rc != BASED_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    int32_t *lists[4];
    for (int i = 0; i < 4; ++i) lists[i] = reinterpret_cast<int32_t *>(ws + i * e.list);
    const int64_t out_bytes = static_cast<int64_t>(V) * D * gs;
    const SortParams s = {ids, lists[0], lists[1], lists[2], lists[3], static_cast<int>(N), V, ids64 ? 1 : 0, e.few,
                          e.passes, e.bits, dtable, aligned(dtable, 16) ? out_bytes / 16 : 0, out_bytes};
    // one cluster sorts; enough others write the zeros: the rest of what is resident at once, or 16 words a thread
    // Sixteen CTAs sort where the sort would take longer than the zeros (some 0.7 ns a token with eight CTAs), or where
    // eight cannot hold the tokens: 32768 tokens, 50000 x 64: 26 us, 31 with eight; 65536 tokens, 50000 x 1024: 83 and
    // 105. Their clusters leave more of the GPU unused for the zeros (32768 tokens, 50000 x 1024: 66 us, 61 with eight).
    const bool wider = N > kSortCluster * kSortChunk || (N > 8192 && out_bytes < 4480 * N);
    const int cluster = wider ? kWideCluster : kSortCluster;
    void (*const sort)(SortParams) =
        cluster == kWideCluster ? based_embed_sort_kernel<kWideCluster> : based_embed_sort_kernel<kSortCluster>;
    OPS_CUDA(allow(sort, sizeof(SortSmem)));
    int resident;
    if ((rc = resident_clusters(reinterpret_cast<const void *>(sort), kSortThreads, sizeof(SortSmem), cluster, &resident)) != BASED_OK)
        return rc;
    int64_t fill = (out_bytes / 16 + cluster * kSortThreads * 16 - 1) / (cluster * kSortThreads * 16);
    // (of the eight-CTA clusters four fifths: 32768 tokens, 50000 x 1024 take 79 us forward and backward with 30 of
    // them, 80 with 32, 84 with 34, 87 with all, 82 with 26; from 2048 x 50000 x 1024 to 8192 x 128000 x 2048 and
    // 4096 x 32000 x 4096 all of them take 9 to 22 % longer; of the sixteen-CTA ones all but the sorting one)
    const int64_t some = wider ? resident - 1 : 2 * sms / cluster * 4 / 5, most = some > 1 ? some : 1;
    fill = fill < 1 ? 1 : fill < most ? fill : most;
    OPS_CUDA(launch_op(sort, dim3(static_cast<unsigned>((fill + 1) * cluster)), kSortThreads, sizeof(SortSmem), st, s, cluster));
    const int done = (e.passes - 1) & 1;
    const SumParams p = {lists[done], lists[2 + done], dy, dy_sr, static_cast<int>(N), V, D, e.rows, scale,
                         reinterpret_cast<float *>(ws + e.partial), dtable};
    // eight columns a thread where rows start on 16 bytes, one otherwise (63 and 78 us for 32768 tokens of 1024)
    const bool wide = D % 8 == 0 && aligned(dy, 16) && dy_sr * es % 16 == 0 && aligned(dtable, 16);
    if (dtype == BASED_F32) return launch_sums<float>(p, g_dtype, wide, e, st);
    if (dtype == BASED_BF16) return launch_sums<__nv_bfloat16>(p, g_dtype, wide, e, st);
    return launch_sums<__half>(p, g_dtype, wide, e, st);
}

}  // extern "C"
