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
#include <cstddef>
#include <type_traits>

#include "ops_common.cuh"

namespace based {
namespace {

constexpr int kSave = BASED_SCAN_SAVE_ROWS;
constexpr int kTile = kSave;       // rows of a tile: one saved state each
constexpr int kRowBytes = 128;     // a tile's row: 64 channels of 16 bits or 32 of 32
constexpr int kMaxCluster = 16;
constexpr int kMaxGrid = 65535;    // blocks along y and z
constexpr int kMaxD = 1 << 20;     // channels: blocks of them along y; a tile of an output spans less than 2^32 bytes

struct ScanParams {
    const void *gate, *x, *dy;
    int64_t gate_sb, gate_st, x_sb, x_st, dy_sb, dy_st;
    int B, T, D, b0;      // b0: the launch's first batch entry
    int cluster, steps;   // CTAs of a cluster; tiles that each of them takes, at most
    int fast;             // every row of every input starts on 16 bytes, a tile's rows within 2^32 bytes
    int pair;             // two 16-bit outputs can be stored as one word
    const float *state;   // forward: h_{-1}; backward: dfinal
    const int32_t *lengths;
    void *y;              // forward: h; backward: dgate
    void *dx;
    float *final_state;   // forward: the last state; backward: dstate
    float *saved;         // forward: written; backward: read
};

// The decay a and its complement 1 - a (unused for log decays), and the increment u.
template <int MODE, int N>
__device__ __forceinline__ void decay(Vec<N> g, Vec<N> &a, Vec<N> &rest) {
    if (MODE == BASED_GATE_LOG) {
        a = vexp(g);
        rest = splat<N>(1.0f);
    } else {
        vsigmoid(g, a, rest);
    }
}
template <int MODE, int N>
__device__ __forceinline__ Vec<N> increment(const Vec<N> &rest, const Vec<N> &x) {
    return MODE == BASED_GATE_LOG ? x : vmul(rest, x);
}

// ------------------------------------------------------------------------------------------------
// Copies of a tile's rows into shared memory
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows [0, rows) of the first `cols` bytes of rows at src, `stride` bytes apart, into the tile at dst, by
// all THREADS threads of the CTA. The other places keep what they held; nothing that is stored depends
// on it. src is the same for all threads and their offsets from it fit 32 bits: one addition a copy.
template <int THREADS>
__device__ __forceinline__ void copy_aligned(uint8_t *dst, const uint8_t *src, uint32_t stride, int rows, int cols) {
    constexpr int kWords = kRowBytes / 16, kStep = THREADS / kWords;
    const int col = static_cast<int>(threadIdx.x) % kWords, row0 = static_cast<int>(threadIdx.x) / kWords;
    if (col * 16 >= cols) return;
    uint32_t off = row0 * stride + col * 16;
    const uint32_t to = smem_u32(dst) + row0 * kRowBytes + col * 16;
    if (rows == kTile) {
#pragma unroll
        for (int k = 0; k < kTile / kStep; ++k) {
            cp_async_16(to + k * kStep * kRowBytes, src + off);
            off += kStep * stride;
        }
    } else {
        for (int k = 0; k < kTile / kStep && row0 + k * kStep < rows; ++k) {
            cp_async_16(to + k * kStep * kRowBytes, src + off);
            off += kStep * stride;
        }
    }
}

// Rows that start anywhere: a row's 16-byte words from the one its first element lies in, nine at most, at the
// row's place in a tile with room for them. Words that reach past the tensor [first, end) are
// copied element by element: nothing outside it is read.
constexpr int kWideRow = kRowBytes + 16;
template <typename T, int THREADS>
__device__ __forceinline__ void copy_anywhere(uint8_t *dst, const T *src, int64_t stride, int rows, int cols,
                                              const T *first, const T *end) {
    constexpr int kWords = kRowBytes / 16, kStep = THREADS / kWords;
    static_assert(THREADS >= kTile && kTile % kStep == 0, "a thread for each row's ninth word");
    static_assert(kStep * sizeof(T) % 16 == 0, "a thread's rows start alike");
    const uintptr_t at = reinterpret_cast<uintptr_t>(src);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(first), hi = reinterpret_cast<uintptr_t>(end);
    const uint32_t bytes = cols * static_cast<uint32_t>(sizeof(T)), low = static_cast<uint32_t>(at);
    const uintptr_t begin = at & ~static_cast<uintptr_t>(15), stop = at + (rows - 1) * stride * sizeof(T) + bytes + 15;
    const int word = static_cast<int>(threadIdx.x) % kWords, row0 = static_cast<int>(threadIdx.x) / kWords;
    if (stride < (1 << 24) && begin >= lo && (stop & ~static_cast<uintptr_t>(15)) <= hi) {
        const uint32_t pitch = static_cast<uint32_t>(stride) * sizeof(T);
        const uint8_t *const from = reinterpret_cast<const uint8_t *>(begin);
        uint32_t off = (low & 15) + row0 * pitch, to = smem_u32(dst) + row0 * kWideRow + word * 16;
        if (word * 16 < (off & 15) + bytes) {
            off = (off & ~15u) + word * 16;
            if (rows == kTile) {
#pragma unroll
                for (int k = 0; k < kTile / kStep; ++k) {
                    cp_async_16(to + k * kStep * kWideRow, from + off);
                    off += kStep * pitch;
                }
            } else {
                for (int row = row0; row < rows; row += kStep) {
                    cp_async_16(to, from + off);
                    to += kStep * kWideRow, off += kStep * pitch;
                }
            }
        }
        const uint32_t ninth = threadIdx.x, last = (low & 15) + ninth * pitch;
        if (ninth < static_cast<uint32_t>(rows) && kRowBytes < (last & 15) + bytes)
            cp_async_16(smem_u32(dst) + ninth * kWideRow + kRowBytes, from + ((last & ~15u) + kRowBytes));
    } else {
#pragma unroll 1
        for (int i = threadIdx.x; i < rows * (kWords + 1); i += THREADS) {
            const int row = i % rows, k = i / rows;
            const uintptr_t start = at + row * stride * sizeof(T), part = (start & ~static_cast<uintptr_t>(15)) + k * 16;
            uint8_t *to = dst + row * kWideRow + k * 16;
            if (part >= lo && part + 16 <= hi && part < start + bytes)
                cp_async_16(smem_u32(to), reinterpret_cast<const void *>(part));
            else
                for (uintptr_t e = k ? part : start; e < part + 16 && e < start + bytes; e += sizeof(T))
                    *reinterpret_cast<T *>(to + (e - part)) = *reinterpret_cast<const T *>(e);
        }
    }
}

// One of the kernels' inputs: what a CTA needs to copy its tiles and to read them. FAST: the rows start on 16 bytes.
template <typename T, int THREADS, bool FAST>
struct Input {
    const T *at;      // row 0, first channel of the CTA
    int64_t stride;
    const T *first, *end;  // the tensor
    __device__ __forceinline__ Input(const void *p, int64_t sb, int64_t st, int b, int c0, const ScanParams &s)
        : at(static_cast<const T *>(p) + b * sb + c0), stride(st), first(static_cast<const T *>(p)),
          end(first + (s.B - 1) * sb + (s.T - 1) * st + s.D) {}
    __device__ __forceinline__ void copy(uint8_t *dst, int row, int rows, int cols) const {
        if (FAST)
            copy_aligned<THREADS>(dst, reinterpret_cast<const uint8_t *>(at + row * stride),
                                  static_cast<uint32_t>(stride) * sizeof(T), rows, cols * static_cast<int>(sizeof(T)));
        else
            copy_anywhere<T, THREADS>(dst, at + row * stride, stride, rows, cols, first, end);
    }
    // A lane's word of the i-th of a warp's rows, which are at `rows`. How far from a word of 16 bytes a row starts
    // is the same for every warp and tile, as those begin sixteen rows apart: uniform registers hold it.
    __device__ __forceinline__ uint32_t word(const uint8_t *rows, int i, int lane) const {
        if (FAST) return reinterpret_cast<const uint32_t *>(rows + i * kRowBytes)[lane];
        const uint32_t begin = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at)) +
                               i * static_cast<uint32_t>(stride) * static_cast<uint32_t>(sizeof(T));
        const uint32_t *from = reinterpret_cast<const uint32_t *>(rows + i * kWideRow + (begin & 12)) + lane;
        return sizeof(T) == 4 ? from[0] : __funnelshift_r(from[0], from[1], (begin & 2) * 8);
    }
    // A warp's R rows moved to where aligned rows have them.
    template <int R>
    __device__ __forceinline__ void realign(uint8_t *rows, int lane) const {
        static_assert(R * sizeof(T) % 16 == 0, "rows of other warps and tiles start alike");
        if constexpr (!FAST) {
            uint32_t w[R];
#pragma unroll
            for (int i = 0; i < R; ++i) w[i] = word(rows, i, lane);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < R; ++i) reinterpret_cast<uint32_t *>(rows + i * kWideRow)[lane] = w[i];
        }
    }
};

// ------------------------------------------------------------------------------------------------
// Maps h -> a h + b of N channels, and their exchange in a cluster
// ------------------------------------------------------------------------------------------------
template <int N>
struct alignas(8 * N) Map {
    Vec<N> a, b;
};
template <int N>
__device__ __forceinline__ Vec<N> apply(const Map<N> &m, const Vec<N> &h) {
    return vfma(m.a, h, m.b);
}
template <int N>  // first `in`, then `m`
__device__ __forceinline__ Map<N> compose(const Map<N> &m, const Map<N> &in) {
    return {vmul(m.a, in.a), vfma(m.a, in.b, m.b)};
}

// Where decays grow (positive log gates), the product over a tile can pass float32 although every row of the recurrence
// is finite: the state in front of it may be 0, or small. Such a map holds the negative cube root of its product
// (past 2^300 any state but 0 overflows: the root stays at 2^100). Sixteen rows alone are one product in float32:
// where that is infinite, a state of 0 stays 0 and any other becomes infinite. And where a product underflows, an
// infinite state in front of it stays infinite, as it does row by row. The functions named far do that. They are
// for tiles in which a warp's map is not plain(), which a barrier's vote tells, and for steps through the cluster's maps
// that meet such a map or an infinite state. There they are made of selections: with branches on which the lanes of a
// warp differ the loops over the tiles take longer (8 x 4096 x 2047 bf16, log decays, forward: 139 us, 129 here, 124
// without any of this; 1 x 16384 x 2048 40.9 and 39.9 us).
template <int N>
__device__ __forceinline__ bool finite(const Vec<N> &v) {
    return fabsf(v.v[0]) + (N == 2 ? fabsf(v.v[N - 1]) : 0.0f) < INFINITY;
}
// Whether this map and three more of its kind compose in float32.
template <int N>
__device__ __forceinline__ bool plain(const Vec<N> &a, const Vec<N> &b) {
    return a.v[0] < 0x1p31f && a.v[N - 1] < 0x1p31f && finite(b);
}
// a h + b of one channel, as fmaf() has it for maps of the common kind
__device__ __forceinline__ float far_apply(float a, float b, float h) {
    const bool root = a < 0.0f, stays = (a == 0.0f && isinf(h)) || (a == INFINITY && h == 0.0f);
    return fmaf(stays ? 1.0f : fabsf(a), root ? a * (a * h) : h, b);
}
__device__ __forceinline__ float far_product(float a, float b) {
    if (a == 0.0f || b == 0.0f) return 0.0f;
    if (a > 0.0f && b > 0.0f && a * b < INFINITY) return a * b;
    const float root = (a < 0.0f ? -a : cbrtf(a)) * (b < 0.0f ? -b : cbrtf(b));
    return root > 0x1p100f ? -0x1p100f : -root;  // NaN stays NaN
}
template <int N>
__device__ __forceinline__ Vec<N> far_apply(const Map<N> &m, const Vec<N> &h) {
    Vec<N> r;
#pragma unroll
    for (int j = 0; j < N; ++j) r.v[j] = far_apply(m.a.v[j], m.b.v[j], h.v[j]);
    return r;
}
// A product that overflowed before a decay of 0 is NaN; its increment is not, as it is where a gate was.
template <int N>
__device__ __forceinline__ Map<N> far_clear(Map<N> m) {
#pragma unroll
    for (int j = 0; j < N; ++j) m.a.v[j] = isnan(m.a.v[j]) && !isnan(m.b.v[j]) ? 0.0f : m.a.v[j];
    return m;
}

// The warps' maps composed, the first first: to[i] is the map of the first i + 1. far: some lane's map is not plain().
template <int COUNT, int N, typename F>
__device__ __forceinline__ void in_order(F map, Map<N> (&to)[COUNT], bool far) {
    to[0] = map(0);
#pragma unroll
    for (int i = 1; i < COUNT; ++i) to[i] = compose(map(i), to[i - 1]);
    if (far) {
        to[0] = far_clear(to[0]);
#pragma unroll
        for (int i = 1; i < COUNT; ++i) {
            const Map<N> m = far_clear(map(i));
#pragma unroll
            for (int j = 0; j < N; ++j) to[i].a.v[j] = far_product(m.a.v[j], to[i - 1].a.v[j]);
            to[i].b = far_apply(m, to[i - 1].b);
        }
    }
}
// What a kernel looks at in its steps through the cluster's maps: nothing; results; results and the maps' signs.
enum Far { kNever, kInfinite, kGrowing };

__device__ unsigned int g_scan_status;  // bit 0: a wait on the cluster's maps gave up
constexpr uint64_t kScanWaitNs = 1000000000ull;

// The maps of a cluster's tiles, two sets in turn. A CTA's warp sends its tile's map into every CTA
// of the cluster with stores that count their bytes on that CTA's mbarrier: nothing else has to be
// ordered or flushed, as a barrier of the whole cluster would.
template <int N>
struct Exchange {
    uint64_t full[2];
    Map<N> maps[1][32];  // (2, cluster, 32)

    static constexpr size_t bytes(int cluster) { return 16 + 2 * cluster * 32 * sizeof(Map<N>); }

    __device__ __forceinline__ void init() {
        mbar_init(smem_u32(&full[0]), 1);
        mbar_init(smem_u32(&full[1]), 1);
        fence_mbar_init();
    }
    // one warp: sends `m`, waits for the set of this step; returns false where the wait gave up
    __device__ __forceinline__ bool swap(int step, int cluster, int rank, int lane, const Map<N> &m) {
        const uint32_t bar = smem_u32(&full[step & 1]), slot = smem_u32(&maps[(step & 1) * cluster + rank][lane]);
        if (lane == 0) mbar_arrive_expect_tx(bar, cluster * 32 * sizeof(Map<N>));
        for (int r = 0; r < cluster; ++r) {
            uint32_t to, to_bar;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(slot), "r"(r));
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to_bar) : "r"(bar), "r"(r));
            if (N == 2)
                asm volatile(
                    "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                    "f"(m.a.v[0]), "f"(m.a.v[N - 1]), "f"(m.b.v[0]), "f"(m.b.v[N - 1]), "r"(to_bar)
                    : "memory");
            else
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to),
                             "f"(m.a.v[0]), "f"(m.b.v[0]), "r"(to_bar)
                             : "memory");
        }
        const uint32_t parity = (step >> 1) & 1;
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t began = global_timer_ns();
        while (!mbar_try_wait(bar, parity))
            if (global_timer_ns() - began > kScanWaitNs) {
                atomicOr(&g_scan_status, 1u);
                return false;
            }
        return true;
    }
    // `at`: the value in front of tile `rank`; `carry` becomes the one behind the last tile. signs: of the maps' products
    __device__ __forceinline__ void fold(int step, int cluster, int rank, int lane, Vec<N> &at, Vec<N> &carry, uint32_t &signs) {
        const Map<N>(*set)[32] = maps + (step & 1) * cluster;
        at = carry;
#pragma unroll 4
        for (int r = 0; r < cluster; ++r) {
            const Map<N> m = set[r][lane];
#pragma unroll
            for (int j = 0; j < N; ++j) signs |= __float_as_uint(m.a.v[j]);
            carry = apply(m, carry);
            if (r + 1 == rank) at = carry;
        }
    }
    __device__ __forceinline__ void far_fold(int step, int cluster, int rank, int lane, Vec<N> &at, Vec<N> &carry) {
        const Map<N>(*set)[32] = maps + (step & 1) * cluster;
        at = carry;
#pragma unroll 1
        for (int r = 0; r < cluster; ++r) {
            carry = far_apply(set[r][lane], carry);
            if (r + 1 == rank) at = carry;
        }
    }
    // From the maps of a CTA's COUNT stretches, composed, what is in front of each of them, through the exchange where
    // there are several CTAs (waiting: no wait has given up); `carry` moves on.
    template <Far FAR, int COUNT>
    __device__ __forceinline__ void advance(const Map<N> (&to)[COUNT], int step, int cluster, int rank, int lane, bool &waiting,
                                            Vec<N> &carry, Vec<N> (&front)[COUNT]) {
        const Vec<N> before = carry;
        uint32_t signs = 0;
        front[0] = carry;
        if (cluster > 1) {
            if (waiting) waiting = swap(step, cluster, rank, lane, to[COUNT - 1]);
            fold(step, cluster, rank, lane, front[0], carry, signs);
        } else {
            carry = apply(to[COUNT - 1], carry);
#pragma unroll
            for (int j = 0; j < N; ++j) signs |= __float_as_uint(to[COUNT - 1].a.v[j]);
        }
#pragma unroll
        for (int i = 1; i < COUNT; ++i) {
            front[i] = apply(to[i - 1], front[0]);
#pragma unroll
            for (int j = 0; j < N; ++j) signs |= __float_as_uint(to[i - 1].a.v[j]);
        }
        if (FAR == kNever) return;
        if (__any_sync(~0u, (FAR == kGrowing && static_cast<int32_t>(signs) < 0) || !finite(carry))) {
            carry = front[0] = before;
            if (cluster > 1)
                far_fold(step, cluster, rank, lane, front[0], carry);
            else
                carry = far_apply(to[COUNT - 1], carry);
#pragma unroll
            for (int i = 1; i < COUNT; ++i) front[i] = far_apply(to[i - 1], front[0]);
        }
    }
};

template <typename T, int N>
__device__ __forceinline__ void store_some(T *dst, const Vec<N> &v, int n) {
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < n) dst[j] = from_f32<T>(v.v[j]);
}
// A row's values, one lane's at `to` each, the whole warp together. FAST: whole words on their places, and no
// lane without its own. Otherwise 16-bit rows that start between two words are stored one element further
// on, each lane's first with the last of the lane before it (8 x 4096 x 2047: 128 us forward and 263 backward
// with these stores and copy_anywhere(), 199 and 341 element by element).
template <typename T, bool FAST, int N>
__device__ __forceinline__ void store_row(uint8_t *to, const Vec<N> &v, int lane, int n, int cols) {
    const uint32_t w = pack<T>(v);
    if (FAST || N == 1) {
        if (FAST || n) *reinterpret_cast<uint32_t *>(to) = w;
    } else if ((reinterpret_cast<uintptr_t>(to) & 2) == 0) {
        if (n == 2)
            *reinterpret_cast<uint32_t *>(to) = w;
        else if (n)
            *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(w);
    } else {
        const uint32_t before = __shfl_up_sync(~0u, w, 1);
        if (n && lane)
            *reinterpret_cast<uint32_t *>(to - 2) = __funnelshift_l(before, w, 16);
        else if (n)
            *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(w);
        if (n == 2 && 2 * lane + 2 >= cols) *reinterpret_cast<uint16_t *>(to + 2) = static_cast<uint16_t>(w >> 16);
    }
}
template <int N>
__device__ __forceinline__ void load_state(const float *src, int n, Vec<N> &v) {
#pragma unroll
    for (int j = 0; j < N; ++j) v.v[j] = src && j < n ? src[j] : 0.0f;
}

// The rows of sequence b before its padding. The loops over the tiles run to T all the same, and steps in
// the padding skip their work between the barriers: a bound that comes from memory makes the loop one
// of threads that might diverge, which costs a third more time. Kernels without lengths (RAGGED
// false) and those whose rows start anywhere (FAST false, which take lengths or none) are instances
// of their own, as both cost the others registers.
template <bool RAGGED>
__device__ __forceinline__ int sequence_length(const ScanParams &p, int b) {
    return RAGGED && p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
}

// Zeros in an output's rows [row0, row0 + R).
template <int R, typename T>
__device__ __forceinline__ void zero_rows(T *to, const ScanParams &p, int row0, int n) {
    constexpr int N = 4 / sizeof(T);
    for (int i = 0; i < R && row0 + i < p.T; ++i) {
        if (p.pair && n == N)
            *reinterpret_cast<uint32_t *>(to) = 0;
        else
            store_some(to, splat<N>(0.0f), n);
        to += p.D;
    }
}

// What both kernels know about their place: 32 N channels of one batch entry for a cluster, N
// channels for a lane; the cluster's CTAs take the tiles in turn.
template <typename T>
struct Place {
    static constexpr int N = 4 / sizeof(T);  // channels of a lane: one 32-bit word
    int lane, warp, rank, b, c0, c, n, cols, tiles;
    __device__ __forceinline__ explicit Place(const ScanParams &p) {
        lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        // the grid: the CTAs of a cluster, the channel blocks, the batch entries
        rank = static_cast<int>(blockIdx.x), b = p.b0 + static_cast<int>(blockIdx.z);
        c0 = static_cast<int>(blockIdx.y) * 32 * N, c = c0 + lane * N;
        n = min(max(p.D - c, 0), N), cols = min(p.D - c0, 32 * N);
        tiles = (p.T + kTile - 1) / kTile;
    }
};

// ------------------------------------------------------------------------------------------------
// Forward
// ------------------------------------------------------------------------------------------------
// Warp w of a CTA: rows [16 w, 16 w + 16) of its tile. Sixteen rows a thread keep the maps' share of the work small
// (eight rows and twice the warps: 494 us where this takes 270, 8 x 16384 x 2048). Four CTAs an SM, by registers
// and shared memory, with two tiles ahead each keep the memory busy: 6.0 TB/s and 90 % of the floor at that
// size. Where few channels leave each CTA many steps, a step's own latencies bound it, 1.6 us: the pass over the rows,
// the exchange and the second pass, one after the other.
constexpr int kFwdWarps = 4, kFwdStages = 2;
template <int N, int PITCH>  // PITCH: bytes of a tile's row
struct FwdSmem {
    uint8_t tile[kFwdStages][2][kTile * PITCH];
    Map<N> warp[kFwdWarps][32];  // each warp's rows; then in b the state in front of them
    Exchange<N> ex;
    static constexpr size_t bytes(int cluster) { return offsetof(FwdSmem, ex) + (cluster > 1 ? Exchange<N>::bytes(cluster) : 0); }
};

template <typename T, int MODE, bool RAGGED, bool FAST>
__global__ void __launch_bounds__(32 * kFwdWarps, 4) based_scan_fwd_kernel(const ScanParams p) {
    constexpr int N = Place<T>::N, R = kTile / kFwdWarps, kThreads = 32 * kFwdWarps, P = FAST ? kRowBytes : kWideRow;
    constexpr Far kFar = MODE == BASED_GATE_LOG ? kGrowing : kInfinite;
    extern __shared__ __align__(128) uint8_t raw[];
    FwdSmem<N, P> &sm = *reinterpret_cast<FwdSmem<N, P> *>(raw);
    const Place<T> at(p);
    const int lane = at.lane, warp = at.warp, cs = p.cluster;
    if (cs > 1) {
        if (threadIdx.x == 0) sm.ex.init();
        cluster_sync();  // every CTA's mbarriers are there before another CTA counts on them
    }
    griddep_wait();
    griddep_launch_dependents();
    const int len = sequence_length<RAGGED>(p, at.b);
    const int64_t plane = static_cast<int64_t>(at.b) * p.D + at.c;
    const Input<T, kThreads, FAST> gate(p.gate, p.gate_sb, p.gate_st, at.b, at.c0, p);
    const Input<T, kThreads, FAST> x(p.x, p.x_sb, p.x_st, at.b, at.c0, p);
    T *y = static_cast<T *>(p.y) + static_cast<int64_t>(at.b) * p.T * p.D;
    const uint32_t off0 = (warp * R * p.D + at.c) * static_cast<uint32_t>(sizeof(T));
    const uint32_t off_row = p.D * static_cast<uint32_t>(sizeof(T));
    const bool wide = !FAST || (p.pair && at.n == N);  // store_row() takes rows that are whole in time
    Vec<N> carry = splat<N>(0.0f);  // warp 0's: the state in front of the cluster's tiles
    if (warp == 0) {
        load_state(p.state ? p.state + plane : nullptr, at.n, carry);
        // The store needs the loaded value: this CTA has read the state before it sends its first map, and so before
        // any CTA of the cluster can have the last state, which may be written to the same place.
        sm.warp[0][lane].b = carry;
    }
    bool waiting = true;
    auto fetch = [&](int step) {
        const int row = (step * cs + at.rank) * kTile, rows = min(len - row, kTile);
        if (rows > 0) {
            gate.copy(sm.tile[step % kFwdStages][0], row, rows, at.cols);
            x.copy(sm.tile[step % kFwdStages][1], row, rows, at.cols);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kFwdStages; ++k) fetch(k);
    cp_async_wait<kFwdStages - 1>();
    __syncthreads();
    for (int step = 0; step < p.steps; ++step) {
        const int tile = step * cs + at.rank, row0 = tile * kTile + warp * R;
        const bool live = !RAGGED || step * cs * kTile < len;  // some row of the cluster's tiles is no padding
        const uint8_t *sg = sm.tile[step % kFwdStages][0] + warp * R * P;
        const uint8_t *sx = sm.tile[step % kFwdStages][1] + warp * R * P;
        Vec<N> a[R], u[R];
        const bool full = row0 + R <= len;
        Map<N> m = {splat<N>(1.0f), splat<N>(0.0f)};
        auto rows = [&](auto all_live) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                Vec<N> rest;
                decay<MODE>(unpack<T>(gate.word(sg, i, lane)), a[i], rest);
                u[i] = increment<MODE>(rest, unpack<T>(x.word(sx, i, lane)));
                if (!decltype(all_live)::value && row0 + i >= len) a[i] = splat<N>(1.0f), u[i] = splat<N>(0.0f);
                m = compose(Map<N>{a[i], u[i]}, m);
            }
        };
        if (full)
            rows(std::true_type());
        else if (row0 < len)
            rows(std::false_type());
        sm.warp[warp][lane] = m;
        const bool far = __syncthreads_or(!plain(m.a, m.b));  // the maps are there, and this step's stage is free
        fetch(step + kFwdStages);
        if (warp == 0) {
            Vec<N> h = carry;
            if (live) {
                Map<N> to[kFwdWarps];
                Vec<N> front[kFwdWarps];
                in_order<kFwdWarps, N>([&](int w) { return sm.warp[w][lane]; }, to, far);
                sm.ex.template advance<kFar>(to, step, cs, at.rank, lane, waiting, carry, front);
#pragma unroll
                for (int w = 0; w < kFwdWarps; ++w) sm.warp[w][lane].b = front[w];
                h = front[0];
            }
            if (p.saved && tile < at.tiles)
                store_some(p.saved + (static_cast<int64_t>(at.b) * at.tiles + tile) * p.D + at.c, h, at.n);
        }
        cp_async_wait<kFwdStages - 1>();
        __syncthreads();  // the starts are there, and the next step's tile
        uint8_t *to = reinterpret_cast<uint8_t *>(y + static_cast<int64_t>(tile) * kTile * p.D);
        uint32_t off = off0;
        if (full && wide) {
            Vec<N> h = sm.warp[warp][lane].b;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                h = vfma(a[i], h, u[i]);
                store_row<T, FAST>(to + off, h, lane, at.n, at.cols);
                off += off_row;
            }
        } else if (row0 < len) {
            Vec<N> h = sm.warp[warp][lane].b;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                h = vfma(a[i], h, u[i]);
                if (row0 + i < p.T) store_some(reinterpret_cast<T *>(to + off), row0 + i < len ? h : splat<N>(0.0f), at.n);
                off += off_row;
            }
        } else if (RAGGED) {
            zero_rows<R>(reinterpret_cast<T *>(to + off0), p, row0, at.n);
        }
    }
    if (warp == 0 && at.rank == 0 && p.final_state) store_some(p.final_state + plane, carry, at.n);
    if (cs > 1) cluster_sync();  // no CTA leaves while another one may still write to it
}

// ------------------------------------------------------------------------------------------------
// Backward
// ------------------------------------------------------------------------------------------------
// The tiles from the last to the first. With mu = what the rows after a row pass back to it,
// lam_t = dy_t + mu and mu <- a_t lam_t: the map of a stretch in reversed time is mu -> A mu + M
// with the same A. h inside a tile is rebuilt from the state saved before it.
// Warp w of a CTA: rows [16 w, 16 w + 16) of its tile. A thread keeps its rows' decays and what the mode
// needs besides: 1 - a for logistic gates, the states in front of the rows for log decays. The rest stays in
// shared memory, where the differences h_{t-1} - x_t of logistic gates take the places of the gate and x (each thread
// reads and writes its own words alone). Eight rows a thread and twice the warps took 489 us where this takes
// 437 (8 x 16384 x 2048, log decays, 92 % of the floor).
constexpr int kBwdWarps = 4, kBwdStages = 2;
template <int N, int PITCH>
struct BwdSmem {
    uint8_t tile[kBwdStages][3][kTile * PITCH];
    Map<N> warp[kBwdWarps][32];  // each warp's rows; then in b the state in front of them
    Vec<N> rev[kBwdWarps][32];   // the reversed map's increment; then mu behind the warp's rows
    Exchange<N> ex;
    static constexpr size_t bytes(int cluster) { return offsetof(BwdSmem, ex) + (cluster > 1 ? Exchange<N>::bytes(cluster) : 0); }
};

template <typename T, int MODE, bool RAGGED, bool FAST>
__global__ void __launch_bounds__(32 * kBwdWarps, FAST ? 4 : 3) based_scan_bwd_kernel(const ScanParams p) {
    constexpr int N = Place<T>::N, R = kTile / kBwdWarps, kThreads = 32 * kBwdWarps, P = FAST ? kRowBytes : kWideRow;
    constexpr Far kFar = MODE == BASED_GATE_LOG ? kGrowing : kNever;
    extern __shared__ __align__(128) uint8_t raw[];
    BwdSmem<N, P> &sm = *reinterpret_cast<BwdSmem<N, P> *>(raw);
    const Place<T> at(p);
    const int lane = at.lane, warp = at.warp, cs = p.cluster;
    if (cs > 1) {
        if (threadIdx.x == 0) sm.ex.init();
        cluster_sync();
    }
    griddep_wait();
    griddep_launch_dependents();
    const int len = sequence_length<RAGGED>(p, at.b);
    const int64_t plane = static_cast<int64_t>(at.b) * p.D + at.c;
    const Input<T, kThreads, FAST> gate(p.gate, p.gate_sb, p.gate_st, at.b, at.c0, p);
    const Input<T, kThreads, FAST> x(p.x, p.x_sb, p.x_st, at.b, at.c0, p);
    const Input<T, kThreads, FAST> dy(p.dy, p.dy_sb, p.dy_st, at.b, at.c0, p);
    T *dgate = static_cast<T *>(p.y) + static_cast<int64_t>(at.b) * p.T * p.D;
    T *dx = static_cast<T *>(p.dx) + static_cast<int64_t>(at.b) * p.T * p.D;
    const uint32_t off0 = (warp * R * p.D + at.c) * static_cast<uint32_t>(sizeof(T));
    const uint32_t off_row = p.D * static_cast<uint32_t>(sizeof(T));
    const bool wide = !FAST || (p.pair && at.n == N);  // store_row() takes rows that are whole in time
    Vec<N> carry = splat<N>(0.0f);  // warp 1's: mu behind the cluster's tiles
    if (warp == 1) load_state(p.state ? p.state + plane : nullptr, at.n, carry);
    bool waiting = true;
    int exchanges = 0;
    auto tile_of = [&](int step) { return at.tiles - 1 - (step * cs + at.rank); };
    auto fetch = [&](int step) {
        const int row = tile_of(step) * kTile, rows = min(len - row, kTile);
        if (row >= 0 && rows > 0) {
            uint8_t(*to)[kTile * P] = sm.tile[step % kBwdStages];
            gate.copy(to[0], row, rows, at.cols);
            x.copy(to[1], row, rows, at.cols);
            dy.copy(to[2], row, rows, at.cols);
        }
        cp_async_commit();
    };
    Vec<N> saved;  // warp 0's: the state in front of the next tile
    auto fetch_state = [&](int step) {
        const int tile = tile_of(step);
        load_state(tile >= 0 ? p.saved + (static_cast<int64_t>(at.b) * at.tiles + tile) * p.D + at.c : nullptr, at.n, saved);
    };
    if (warp == 0) fetch_state(0);
    fetch(0);
    for (int step = 0; step < p.steps; ++step) {
        const int tile = tile_of(step), row0 = tile * kTile + warp * R;
        const bool live = !RAGGED || (at.tiles - (step + 1) * cs) * kTile < len;  // some row of the cluster's tiles is no padding
        cp_async_wait<0>();
        __syncthreads();  // the tile has landed, and the other stage is free
        fetch(step + 1);
        x.template realign<R>(sm.tile[step % kBwdStages][1] + warp * R * P, lane);
        dy.template realign<R>(sm.tile[step % kBwdStages][2] + warp * R * P, lane);
        uint8_t *sg = sm.tile[step % kBwdStages][0] + warp * R * P + lane * 4;
        uint8_t *sx = sg + kTile * P, *sd = sx + kTile * P;
        auto word = [&](uint8_t *s, int i) -> uint32_t & { return *reinterpret_cast<uint32_t *>(s + i * P); };
        const bool full = tile >= 0 && row0 + R <= len, some = tile >= 0 && row0 < len;
        Vec<N> a[R], other[R], rev = splat<N>(0.0f);  // other: 1 - a, or the states in front of the rows
        Map<N> m = {splat<N>(1.0f), splat<N>(0.0f)};
        auto rows = [&](auto all_live) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                Vec<N> rest;
                decay<MODE>(unpack<T>(gate.word(sg - lane * 4, i, lane)), a[i], rest);
                if (!decltype(all_live)::value && row0 + i >= len) {
                    a[i] = splat<N>(1.0f), rest = splat<N>(0.0f);
                    word(sx, i) = word(sd, i) = 0;
                }
                if (MODE == BASED_GATE_SIGMOID) other[i] = rest;
                m = compose(Map<N>{a[i], increment<MODE>(rest, unpack<T>(word(sx, i)))}, m);
            }
#pragma unroll
            for (int i = R - 1; i >= 0; --i) rev = vmul(a[i], vadd(unpack<T>(word(sd, i)), rev));
        };
        if (full)
            rows(std::true_type());
        else if (some)
            rows(std::false_type());
        sm.warp[warp][lane] = m;
        sm.rev[warp][lane] = rev;
        bool far = false;
        if (kFar != kNever)
            far = __syncthreads_or(!plain(m.a, m.b) || !finite(rev));  // the maps are there
        else
            __syncthreads();
        if (warp == 0) {
            Map<N> m[kBwdWarps];
            Vec<N> h[kBwdWarps];
            h[0] = saved;
#pragma unroll
            for (int w = 1; w < kBwdWarps; ++w) m[w] = sm.warp[w - 1][lane], h[w] = apply(m[w], h[w - 1]);
            if (far) {
#pragma unroll
                for (int w = 1; w < kBwdWarps; ++w) h[w] = far_apply(far_clear(m[w]), h[w - 1]);
            }
#pragma unroll
            for (int w = 0; w < kBwdWarps; ++w) sm.warp[w][lane].b = h[w];
            fetch_state(step + 1);
        } else if (warp == 1 && live) {
            // the tile's map in reversed time, composed for one CTA as for several: no bit depends on their number
            Map<N> to[kBwdWarps];
            Vec<N> front[kBwdWarps];
            in_order<kBwdWarps, N>([&](int i) { return Map<N>{sm.warp[kBwdWarps - 1 - i][lane].a, sm.rev[kBwdWarps - 1 - i][lane]}; }, to, far);
            sm.ex.template advance<kFar>(to, exchanges++, cs, at.rank, lane, waiting, carry, front);
#pragma unroll
            for (int w = 0; w < kBwdWarps; ++w) sm.rev[kBwdWarps - 1 - w][lane] = front[w];
        }
        __syncthreads();  // the starts are there
        uint8_t *const to_g = reinterpret_cast<uint8_t *>(dgate + static_cast<int64_t>(tile) * kTile * p.D);
        uint8_t *const to_x = reinterpret_cast<uint8_t *>(dx + static_cast<int64_t>(tile) * kTile * p.D);
        if (some) {
            Vec<N> h = sm.warp[warp][lane].b, mu = sm.rev[warp][lane];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const Vec<N> v = unpack<T>(word(sx, i));
                if constexpr (MODE == BASED_GATE_LOG) {
                    other[i] = h;
                    h = vfma(a[i], h, v);
                } else {
                    const Vec<N> diff = vfma(v, splat<N>(-1.0f), h);
                    h = vfma(a[i], h, vmul(other[i], v));
                    word(sg, i) = __float_as_uint(diff.v[0]);
                    if (N == 2) word(sx, i) = __float_as_uint(diff.v[N - 1]);
                }
            }
            uint32_t off = off0 + (R - 1) * off_row;
            auto back = [&](auto all_live) {
#pragma unroll
                for (int i = R - 1; i >= 0; --i) {
                    // shared memory is read four rows ahead at most: all 16 at once spill registers, which
                    // costs a third of the time
                    if (i % 4 == 3) asm volatile("" ::: "memory");
                    const Vec<N> lam = vadd(unpack<T>(word(sd, i)), mu);
                    mu = vmul(a[i], lam);
                    Vec<N> og, ox;
                    if constexpr (MODE == BASED_GATE_LOG) {
                        og = vmul(mu, other[i]), ox = lam;
                    } else {
                        Vec<N> diff;
                        diff.v[0] = __uint_as_float(word(sg, i));
                        if (N == 2) diff.v[N - 1] = __uint_as_float(word(sx, i));
                        og = vmul(vmul(mu, other[i]), diff);
                        ox = vmul(other[i], lam);
                    }
                    if (decltype(all_live)::value) {
                        store_row<T, FAST>(to_g + off, og, lane, at.n, at.cols);
                        store_row<T, FAST>(to_x + off, ox, lane, at.n, at.cols);
                    } else if (row0 + i < p.T) {
                        store_some(reinterpret_cast<T *>(to_g + off), row0 + i < len ? og : splat<N>(0.0f), at.n);
                        store_some(reinterpret_cast<T *>(to_x + off), row0 + i < len ? ox : splat<N>(0.0f), at.n);
                    }
                    off -= off_row;
                }
            };
            if (full && wide)
                back(std::true_type());
            else
                back(std::false_type());
        } else if (RAGGED && tile >= 0) {
            zero_rows<R>(reinterpret_cast<T *>(to_g + off0), p, row0, at.n);
            zero_rows<R>(reinterpret_cast<T *>(to_x + off0), p, row0, at.n);
        }
    }
    if (warp == 1 && at.rank == 0 && p.final_state) store_some(p.final_state + plane, carry, at.n);
    if (cs > 1) cluster_sync();
}

struct StepParams {
    const void *gate, *x;
    int64_t gate_sn, x_sn;
    int N, D, S;
    float *pool;
    const int32_t *slots;
    void *y;
};

// One row for N sequences: bound by launch and latency (1.4 us for one sequence of 1024 channels in a graph, 2.8 us for
// 256 of 4096, where the memory's rate gives 2.2). Grid (channel blocks, sequences), N consecutive channels
// a thread.
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
                Vec<1> a, rest;
                decay<MODE>(Vec<1>{{to_f32(g.v[j])}}, a, rest);
                h.v[j] = fmaf(a.v[0], h.v[j], increment<MODE>(rest, Vec<1>{{to_f32(v.v[j])}}).v[0]);
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
    if (static_cast<int64_t>(p.B) * p.D >= (1ll << 30) || p.T > (1 << 30) || p.D > kMaxD) return BASED_ERR_BAD_SIZE;
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
            // the last state may take the place of the first
            if (overlap(out[i], s) && !(!bwd && p.state && p.final_state == p.state && i == 2 && s.a == in[4].a && s.b == in[4].b))
                return BASED_ERR_ALIASING;
        for (int k = 0; k < i; ++k)
            if (overlap(out[i], out[k])) return BASED_ERR_ALIASING;
    }
    return BASED_OK;
}

// What a kernel's steps take, measured: `us` by a CTA's own latencies where the GPU is not full, `bytes` of copies
// and stores at `rate` bytes per us where it is, and `us_rank` more for each CTA of a cluster.
struct StepCost {
    double us, bytes, rate, us_rank;
};

// CTAs of a cluster: those whose estimated time is least, a CTA having two steps' worth of start and end besides
// its share of the tiles. Of sequences with padding a little more than half is taken to be alive (5 x 2112 x 1024 bf16
// forward, lengths from a quarter to all of the rows 14.2 us, all full 14.8, one full and four an eighth 12.0; with all
// taken to be alive 15.0, 15.8, 14.0; nine other shapes the same within 1 %). Against the best
// of all sizes on eleven shapes the choice costs up to 6 % (8 x 3000 x 1536: 1, 2, 3, 4 CTAs take
// 54, 42, 38, 49 us, and 3 are chosen).
// slots[cs]: clusters of cs CTAs that the device holds at once.
int choose_cluster(int64_t blocks, int64_t tiles, const int (&slots)[kMaxCluster + 1], const StepCost &c, bool ragged) {
    int best = 1;
    double least = 0.0;
    for (int cs = 1; cs <= kMaxCluster && (cs == 1 || cs / 2 < tiles); ++cs) {
        if (slots[cs] < 1) continue;
        auto step = [&](int64_t resident) {
            const double us = resident * cs * c.bytes * (ragged ? 0.6 : 1.0) / c.rate;
            return (us > c.us ? us : c.us) + c.us_rank * cs;
        };
        const int64_t waves = blocks / slots[cs], rest = blocks % slots[cs];
        const double us = ((tiles + cs - 1) / cs + 2) * (waves * step(slots[cs]) + (rest ? step(rest) : 0.0));
        if (cs == 1 || us < 0.98 * least) best = cs, least = us;
    }
    return best;
}

// The cluster size of a call, from a per-thread cache of the last few shapes: a call repeats the
// shapes of the calls before it far more often than not. All that `choose` looks at is in the key.
template <typename F>
int recent_cluster(ScanParams &p, void (*kernel)(ScanParams), F choose) {
    struct Entry {
        void (*kernel)(ScanParams);
        int dev, B, T, D, ragged, cluster;
    };
    constexpr int kEntries = 8;
    static thread_local Entry recent[kEntries];
    static thread_local int next = 0;
    int dev;
    OPS_CUDA(cudaGetDevice(&dev));
    const int ragged = p.lengths != nullptr;
    for (const Entry &e : recent) {
        if (e.kernel == kernel && e.dev == dev && e.B == p.B && e.T == p.T && e.D == p.D && e.ragged == ragged) {
            p.cluster = e.cluster;
            return BASED_OK;
        }
    }
    const int rc = choose(&p.cluster);
    if (rc != BASED_OK) return rc;
    recent[next] = {kernel, dev, p.B, p.T, p.D, ragged, p.cluster};
    next = (next + 1) % kEntries;
    return BASED_OK;
}

template <typename T, typename Smem>
int launch_scan(ScanParams &p, void (*kernel)(ScanParams), int threads, int sms, const StepCost &cost, cudaStream_t st) {
    const int slabs = (p.D + 32 * Place<T>::N - 1) / (32 * Place<T>::N);
    const int64_t blocks = static_cast<int64_t>(slabs) * p.B, tiles = (p.T + kTile - 1) / kTile;
    constexpr int64_t kMost = 227 * 1024;
    const int rc = recent_cluster(p, kernel, [&](int *cluster) -> int {
        OPS_CUDA(allow(kernel, kMost));
        int slots[kMaxCluster + 1];
        for (int cs = 1; cs <= kMaxCluster; ++cs) {
            const int rc = resident_clusters(reinterpret_cast<const void *>(kernel), threads, Smem::bytes(cs), cs, &slots[cs]);
            if (rc != BASED_OK) return rc;
        }
        *cluster = choose_cluster(blocks, tiles, slots, cost, p.lengths != nullptr);
        return BASED_OK;
    });
    if (rc != BASED_OK) return rc;
    p.steps = static_cast<int>((tiles + p.cluster - 1) / p.cluster);
    // CTAs that are all resident at once spread evenly where no SM can take more than its share: each asks for
    // that share of the shared memory (8 x 3000 x 1536 backward: 84 us with up to four on an SM, 69 us with three).
    // One more with large clusters, which have to find their SMs within a part of the GPU.
    const int64_t per_sm = (blocks * p.cluster + sms - 1) / sms + (p.cluster > 8 ? 1 : 0);
    const int64_t share = per_sm < 4 ? 228 * 1024 / per_sm - 1024 : 0;
    size_t smem = Smem::bytes(p.cluster);
    if (share > static_cast<int64_t>(smem)) smem = static_cast<size_t>(share < kMost ? share : kMost);
    for (p.b0 = 0; p.b0 < p.B; p.b0 += kMaxGrid) {
        const dim3 grid(p.cluster, slabs, p.B - p.b0 < kMaxGrid ? p.B - p.b0 : kMaxGrid);
        OPS_CUDA(launch_op(kernel, grid, threads, smem, st, p, p.cluster));
    }
    return BASED_OK;
}
template <typename T>
int launch_scan(ScanParams &p, int mode, bool bwd, int sms, cudaStream_t st) {
    constexpr int kLog = BASED_GATE_LOG, kSig = BASED_GATE_SIGMOID;
    const bool log = mode == BASED_GATE_LOG, fast = p.fast != 0, ragged = p.lengths;
    const StepCost fwd_cost = {1.6, 3.0 * kTile * kRowBytes, 6.7e6, 0.02};
    const StepCost bwd_cost = {2.6, 5.0 * kTile * kRowBytes, 6.6e6, 0.03};
    constexpr int N = Place<T>::N;
    if (bwd) {
        if (!fast)
            return launch_scan<T, BwdSmem<N, kWideRow>>(
                p, log ? based_scan_bwd_kernel<T, kLog, true, false> : based_scan_bwd_kernel<T, kSig, true, false>,
                32 * kBwdWarps, sms, bwd_cost, st);
        void (*const k)(ScanParams) =
            ragged ? (log ? based_scan_bwd_kernel<T, kLog, true, true> : based_scan_bwd_kernel<T, kSig, true, true>)
                   : (log ? based_scan_bwd_kernel<T, kLog, false, true> : based_scan_bwd_kernel<T, kSig, false, true>);
        return launch_scan<T, BwdSmem<N, kRowBytes>>(p, k, 32 * kBwdWarps, sms, bwd_cost, st);
    }
    if (!fast)
        return launch_scan<T, FwdSmem<N, kWideRow>>(
            p, log ? based_scan_fwd_kernel<T, kLog, true, false> : based_scan_fwd_kernel<T, kSig, true, false>,
            32 * kFwdWarps, sms, fwd_cost, st);
    void (*const k)(ScanParams) =
        ragged ? (log ? based_scan_fwd_kernel<T, kLog, true, true> : based_scan_fwd_kernel<T, kSig, true, true>)
               : (log ? based_scan_fwd_kernel<T, kLog, false, true> : based_scan_fwd_kernel<T, kSig, false, true>);
    return launch_scan<T, FwdSmem<N, kRowBytes>>(p, k, 32 * kFwdWarps, sms, fwd_cost, st);
}

int run_scan(ScanParams &p, int dtype, int mode, bool bwd, based_stream_t stream) {
    int rc = check_scan(p, dtype, mode, bwd), sms;
    if (rc != BASED_OK || (rc = host_device(&sms)) != BASED_OK) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int64_t es = static_cast<int64_t>(elem_size(dtype));
    const int64_t bits = (p.D | p.gate_sb | p.gate_st | p.x_sb | p.x_st | p.dy_sb | p.dy_st) * es |
                         static_cast<int64_t>(reinterpret_cast<uintptr_t>(p.gate) | reinterpret_cast<uintptr_t>(p.x) |
                                              reinterpret_cast<uintptr_t>(p.dy));
    const bool near = (p.gate_st | p.x_st | p.dy_st) < (1 << 24);  // a tile's rows within 2^32 bytes
    // (8 x 4096 x 2048 and 2047 bfloat16: 67 + 117 us forward and backward by aligned words, 128 + 263 by shifted ones, 199
    // + 341 element by element. Rows of 4-byte words are copied as rows that start anywhere, too: by such words
    // 2 x 2047 x 777 float32 took 14.2 + 21.6 us where this took 11.5 + 18.2, and 8 x 4096 x 1023 95 + 230, this 85 + 145,
    // both before float32 decays took expf(), 0.6 us of 12; 2 x 4096 x 1022 bfloat16 alone would be faster, 19.4 + 35.6
    // where this takes 21.3 + 38.1.)
    p.fast = bits % 16 == 0 && near;
    p.pair = es == 4 || (p.D % 2 == 0 && aligned(p.y, 4) && aligned(p.dx, 4));
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

cudaError_t scan_status(unsigned int *status, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(status, g_scan_status, sizeof(unsigned int));
    if (e == cudaSuccess && clear && *status) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_scan_status, &zero, sizeof(unsigned int));
    }
    return e;
}
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
    // four channels a thread where the rows of every tensor allow their loads, one otherwise (256 rows of
    // 4096: 2.8 and 8.9 us)
    const bool quad = ((D | gate_sn | x_sn) & 3) == 0 && aligned(gate, 4 * es) && aligned(x, 4 * es) &&
                      aligned(y, 4 * es) && aligned(pool, 16);
    if (dtype == BASED_F32) return quad ? launch_step<float, 4>(p, mode, st) : launch_step<float, 1>(p, mode, st);
    if (dtype == BASED_BF16)
        return quad ? launch_step<__nv_bfloat16, 4>(p, mode, st) : launch_step<__nv_bfloat16, 1>(p, mode, st);
    return quad ? launch_step<__half, 4>(p, mode, st) : launch_step<__half, 1>(p, mode, st);
}

}  // extern "C"
