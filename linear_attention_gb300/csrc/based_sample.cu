// based_sample.cu: the choice of a next token (declared in include/based_ops.h).
//
// With w_i = exp((x_i - max) / temperature), each of top-k, top-p and min-p keeps a prefix of the tokens in the order of falling
// logits (equal ones by rising index), so what is kept is one comparison with a cut: the whole order is never needed. A row lies in the
// shared memory of a cluster. A small top-k is cut among the tokens above a bound that the threads' largest ones give, and what it keeps is
// sorted and summed by one CTA. Else one pass over the row counts tokens (or sums masses) in 2048 bins of x's distance from the largest; the bin of the cut follows
// from the bins' sums, and the cut from the tokens of that bin, or of all bins up to it, which one CTA sorts. A last pass sums the kept masses by
// warps, and the warp in which the random number falls finds the token. Masses are whole numbers, w 2^40 in 64 bits: their sums
// do not depend on an order, so the same call gives the same token. Bound by the passes' instructions where there are many rows, by the
// barriers between them where there are few.
#include "ops_common.cuh"

namespace based {
namespace {

constexpr int kSampleThreads = 512, kSampleWarps = kSampleThreads / 32;
constexpr int kBins = 2048, kFew = 2048;  // bins; tokens that one CTA sorts
constexpr uint32_t kListed = 256;
constexpr float kReach = 46.0f;           // the last bin begins at w = 2^-46
constexpr float kMass = 1099511627776.0f; // 2^40
constexpr int kSampleCluster = 16;
constexpr int kSampleMostV = 1 << 22;     // whose masses' sum is below 2^63

struct SampleParams {
    const void *logits;
    int64_t stride;
    int V, slice, cluster, resident;  // tokens of a CTA, a multiple of eight; whether they lie in shared memory
    int words;                        // rows can be read as 16-byte words
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    float temperature_all, top_p_all, min_p_all;
    int top_k_all;
    int32_t *tokens;
    float *probs;
};

using u64 = unsigned long long;

struct SampleShared {
    union {
        uint32_t bins[3][kBins];  // counts; or masses, 14 bits of them in each (64-bit atomics on shared memory are loops)
        struct {
            u64 place[kFew], mass[kFew];
        } few;  // the tokens to sort: in the first CTA, once all have read its bins
    };
    u64 slots[2][4];  // what this CTA hands to the others, two sets in turn
    u64 warp[4][kSampleWarps];
    u64 found[4];
    uint32_t count, pad[3];
};
static_assert(sizeof(SampleShared) % 16 == 0, "the tokens lie behind it");

__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);  // -0 and 0 are equal
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
// Where the kept tokens end in the order: the last one. (Of none -inf is kept.)
struct Cut {
    float x = -INFINITY;
    int index = -1;
    __device__ __forceinline__ bool keeps(float v, int i) const { return v > x || (v == x && i <= index); }
};
// A token's place in the order: larger is earlier
__device__ __forceinline__ u64 place_of(float x, int index) { return static_cast<u64>(ordered(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(index)); }

// Moves the cut up to a place
__device__ __forceinline__ void raise(Cut &cut, u64 place) {
    const float x = unordered(static_cast<uint32_t>(place >> 32));
    const int i = static_cast<int>(0xffffffffu - static_cast<uint32_t>(place));
    if (place && (x > cut.x || (x == cut.x && i < cut.index))) cut.x = x, cut.index = i;
}
// The same variable in the shared memory of another CTA of the cluster
template <typename P>
__device__ __forceinline__ uint32_t peer(P *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ u64 peer_load(uint32_t at) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t peer_load32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void peer_store(uint32_t at, u64 v) { asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory"); }
__device__ __forceinline__ uint32_t peer_add(uint32_t at, uint32_t v) {
    uint32_t r;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(at), "r"(v) : "memory");
    return r;
}

template <bool MOST>
__device__ __forceinline__ u64 over_warp(u64 v) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const u64 o = __shfl_xor_sync(0xffffffffu, v, d);
        v = MOST ? (o > v ? o : v) : v + o;
    }
    return v;
}

template <typename T>
struct Sampler {
    const SampleParams &p;
    SampleShared &sh;
    const T *row;    // this CTA's tokens, in shared memory or the row itself
    int first, len;  // their indices
    uint32_t rank;
    int turn = 0;
    int tid = threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    __device__ __forceinline__ void meet() {
        if (p.cluster > 1)
            cluster_sync();
        else
            __syncthreads();
    }
    // Sums (or largest) over all threads of the cluster of up to three numbers, and the sums of the CTAs in front of this one. All
    // threads get them.
    template <int N, bool MOST = false>
    __device__ __forceinline__ void total(u64 (&v)[N], u64 (&before)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = over_warp<MOST>(v[i]);
            if (lane == 0) sh.warp[i][warp] = v[i];
        }
        __syncthreads();
        if (tid < N) {
            u64 s = 0;
            for (int w = 0; w < kSampleWarps; ++w) s = MOST ? (sh.warp[tid][w] > s ? sh.warp[tid][w] : s) : s + sh.warp[tid][w];
            sh.slots[turn][tid] = s;
        }
        meet();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            u64 o = 0;  // lane r: what CTA r handed over
            if (lane < p.cluster) o = p.cluster > 1 ? peer_load(peer(&sh.slots[turn][i], lane)) : sh.slots[turn][i];
            v[i] = over_warp<MOST>(o);
            before[i] = over_warp<false>(lane < static_cast<int>(rank) ? o : 0);
        }
        turn ^= 1;
        // (the next call writes the other set; sh.warp is read before meet())
    }
    template <int N, bool MOST = false>
    __device__ __forceinline__ void total(u64 (&v)[N]) {
        u64 before[N];
        total<N, MOST>(v, before);
    }

    // f(x, index in the slice) for this thread's tokens, in the order of their indices within a warp's rounds
    template <typename F>
    __device__ __forceinline__ void each(F f) {
        each(f, [](int) {});
    }
    // ... and g(index of the first) after every eight
    template <typename F, typename G>
    __device__ __forceinline__ void each(F f, G g) {
        const int per = (len + kSampleWarps * 8 - 1) / (kSampleWarps * 8) * 8, from = warp * per, to = min(len, from + per);
        for (int i = from + 8 * lane; i < to; i += 256) {
            eight(i, to, f);
            g(i);
        }
    }
    template <typename F>
    __device__ __forceinline__ void eight(int i, int to, F f) {
        if (i + 8 <= to && p.resident) {
            const Pack<T, 8> w = *reinterpret_cast<const Pack<T, 8> *>(row + i);
#pragma unroll
            for (int e = 0; e < 8; ++e) f(to_f32(w.v[e]), i + e);
        } else {
#pragma unroll 1
            for (int e = 0; e < 8 && i + e < to; ++e) {
                const float x = to_f32(row[i + e]);
                f(x == x ? x : -INFINITY, i + e);
            }
        }
    }
};

// w = 2^-t, t = (most - x) log2(e) / temperature, with the product's rounding made good
struct Weigh {
    float most, hi, lo;
    // The bin, as a number whose whole part it is. The last one takes all that is far below the largest, also where the product is beyond
    // float32 (a type's lowest value as a mask, a small temperature) or no number (a difference beyond it, an infinite temperature).
    __device__ __forceinline__ float place(float x) const { return fminf((most - x) * hi * (kBins / kReach), kBins - 1.0f); }
    __device__ __forceinline__ float weight(float x) const {
        const float d = most - x, t = d * hi, r = fmaf(d, lo, fmaf(d, hi, -t));
        const float w = ex2(-t);
        return t < 120.0f ? fmaf(w, -0.6931471806f * r, w) : 0.0f;
    }
    __device__ __forceinline__ u64 mass(float x) const { return static_cast<u64>(__float2ull_rn(weight(x) * kMass)); }
    __device__ __forceinline__ int bin(float x) const { return static_cast<int>(place(x)); }
};

// Prefix sums over the CTA, in the order of threads; all: the sum
__device__ __forceinline__ u64 cta_prefix(u64 v, u64 *by_warp, u64 &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 up = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const u64 o = __shfl_up_sync(0xffffffffu, up, d);
        if (lane >= d) up += o;
    }
    if (lane == 31) by_warp[warp] = up;
    __syncthreads();
    u64 before = up - v;
    all = 0;
    for (int w = 0; w < kSampleWarps; ++w) {
        const u64 o = by_warp[w];
        if (w < warp) before += o;
        all += o;
    }
    __syncthreads();
    return before;
}
// The tokens to sort, into falling places
__device__ __forceinline__ void sort_few(SampleShared &sh, int n) {
    int size = 2;
    while (size < n) size *= 2;
    for (int i = n + threadIdx.x; i < size; i += kSampleThreads) sh.few.place[i] = sh.few.mass[i] = 0;
    for (int k = 2; k <= size; k *= 2)
        for (int d = k / 2; d > 0; d /= 2) {
            __syncthreads();
            for (int i = threadIdx.x; i < size / 2; i += kSampleThreads) {
                const int a = 2 * i - (i & (d - 1)), b = a + d;
                const u64 x = sh.few.place[a], y = sh.few.place[b];
                if (((a & k) == 0) == (x < y)) {
                    const u64 m = sh.few.mass[a];
                    sh.few.place[a] = y, sh.few.place[b] = x, sh.few.mass[a] = sh.few.mass[b], sh.few.mass[b] = m;
                }
            }
        }
    __syncthreads();
}

// (up to 2^18 of at most 2^40, or their sums: the highest part takes what is above)
__device__ __forceinline__ void add_mass(SampleShared &sh, int bin, u64 v) {
    atomicAdd(&sh.bins[0][bin], static_cast<uint32_t>(v) & 0x3fffu);
    atomicAdd(&sh.bins[1][bin], static_cast<uint32_t>(v >> 14) & 0x3fffu);
    atomicAdd(&sh.bins[2][bin], static_cast<uint32_t>(v >> 28));
}

// share * total, rounded up (UP) or down to a whole number; share in (0, 1)
template <bool UP>
__device__ __forceinline__ u64 share_of(float share, u64 total) {
    const uint32_t b = __float_as_uint(share), e = b >> 23, m = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
    const uint32_t shift = 150 - (e ? e : 1);  // share = m 2^-shift, shift from 24 on
    const u64 low = total * m, high = __umul64hi(total, m);
    if (shift >= 128) return UP && (low | high) ? 1 : 0;
    if (shift >= 64) return (shift == 64 ? high : high >> (shift - 64)) + (UP && (low | (shift == 64 ? 0 : high << (128 - shift))) ? 1 : 0);
    return (high << (64 - shift) | low >> shift) + (UP && low << (64 - shift) ? 1 : 0);
}

// The mass in front of the token that a random number takes
__device__ __forceinline__ u64 target_of(float u, u64 all) {
    const u64 target = u > 0.0f ? u < 1.0f ? share_of<false>(u, all) : all : 0;
    return target >= all ? all - 1 : target;
}

// Moves the cut up: by count to the k'th token of those at or above it and, where all of those could be sorted, on to the first at which the masses
// reach `share` of theirs (DONE; LISTED: the first CTA has them in `few`, found[2] of them, at most kListed); by mass (k is 0) to the latter.
// quick: only each thread's largest, `top`, is counted. The k'th of those bounds the k'th of all, and in a row of any order but few tokens lie above
// it. Where they do not fit (MANY) nothing is moved.
enum Moved { CUT, DONE, LISTED, MANY };
template <typename T>
__device__ Moved move_cut(Sampler<T> &s, const Weigh &w, int k, float share, Cut &cut, bool quick, float top) {
    SampleShared &sh = s.sh;
    const SampleParams &p = s.p;
    const bool by_mass = k == 0;
    u64 last = 0;  // the last bin's tokens, which may be most, without atomics
    const auto count = [&](float x, int i) {
        if (!cut.keeps(x, s.first + i)) return;
        const int bin = w.bin(x);
        if (by_mass) {
            const u64 v = w.mass(x);
            if (bin == kBins - 1)
                last += v;
            else
                add_mass(sh, bin, v);
        } else if (bin == kBins - 1) {
            ++last;
        } else {
            atomicAdd(&sh.bins[0][bin], 1u);
        }
    };
    if (quick)
        count(top, 0);
    else
        s.each(count);
    last = over_warp<false>(last);
    if (s.lane == 0 && last) by_mass ? add_mass(sh, kBins - 1, last) : static_cast<void>(atomicAdd(&sh.bins[0][kBins - 1], static_cast<uint32_t>(last)));
    s.meet();
    // this CTA's part of the bins over all CTAs: up to four neighbouring bins a thread
    constexpr int kMost = kBins / kSampleThreads;
    const int part = kBins / p.cluster, per = part < kSampleThreads ? 1 : part / kSampleThreads, mine = threadIdx.x * per;
    u64 v[kMost], sum = 0;
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
        v[j] = 0;
        if (j < per && mine + j < part) {
            const int at = s.rank * part + mine + j;
#pragma unroll
            for (int c = 0; c < 3; ++c) {
                if (c && !by_mass) continue;
                u64 all_of = 0;
                if (p.cluster > 1) {
#pragma unroll
                    for (int r = 0; r < kSampleCluster; ++r)
                        if (r < p.cluster) all_of += peer_load32(peer(&sh.bins[c][at], r));
                } else {
                    all_of = sh.bins[c][at];
                }
                v[j] += all_of << (14 * c);
            }
        }
        sum += v[j];
    }
    u64 all[1], others[1], in_cta;
    u64 before = cta_prefix(sum, sh.warp[3], in_cta);
    all[0] = threadIdx.x == 0 ? in_cta : 0;
    if (threadIdx.x == 0) sh.found[0] = sh.found[1] = sh.found[2] = 0;
    s.template total<1>(all, others);
    before += others[0];
    const u64 target = by_mass ? share_of<true>(share, all[0]) : static_cast<u64>(k);  // (whole numbers: 64-bit floats are slow here)
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
        if (before < target && before + v[j] >= target)
            sh.found[0] = s.rank * part + mine + j + 1, sh.found[1] = before, sh.found[2] = before + v[j];
        before += v[j];
    }
    __syncthreads();
    u64 at[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) at[i] = s.tid == 0 ? sh.found[i] : 0;
    s.template total<3>(at);
    // fewer tokens than k: all are kept, and sorted where they are few
    const bool enough = at[0] != 0, whole = !by_mass && (quick || (enough ? at[2] : all[0]) <= kFew);
    if (quick ? at[0] == 0 || at[0] == kBins : !enough && !whole) return quick ? MANY : CUT;
    const int bin = enough ? static_cast<int>(at[0]) - 1 : kBins - 1, low = whole ? 0 : bin;
    const float from = static_cast<float>(low), to = static_cast<float>(bin + 1);
    uint32_t hits = 0;  // of eight tokens: what follows is needed for few, so it is there once
    s.each([&](float x, int i) {
        const float b = w.place(x);
        if (b < to && b >= from && cut.keeps(x, s.first + i)) hits |= 1u << (i & 7);
    }, [&](int i0) {
        while (hits) {
            const int i = i0 + __ffs(hits) - 1;
            hits &= hits - 1;
            const float x = to_f32(s.row[i]);
            const uint32_t n = p.cluster > 1 ? peer_add(peer(&sh.count, 0), 1) : atomicAdd(&sh.count, 1u);
            if (n >= kFew) continue;
            const u64 pl = place_of(x, s.first + i), m = w.mass(x);
            if (p.cluster > 1)
                peer_store(peer(&sh.few.place[n], 0), pl), peer_store(peer(&sh.few.mass[n], 0), m);
            else
                sh.few.place[n] = pl, sh.few.mass[n] = m;
        }
    });
    s.meet();
    if (s.tid == 0) sh.found[0] = sh.found[1] = sh.found[2] = 0;
    const uint32_t few = s.rank == 0 ? sh.count : 0;
    __syncthreads();
    if (s.rank == 0) {
        if (s.tid == 0) sh.count = 0, sh.found[1] = few > kFew, sh.found[2] = few;
        const int n = static_cast<int>(few);
        if (n > 0 && n <= kFew) {
            sort_few(sh, n);
            // the k'th of all, or what is behind the bins in front: no more than are listed
            const u64 base = whole ? 0 : at[1];
            const int nth = by_mass || !enough ? n : min(n, static_cast<int>(static_cast<u64>(k) - base));
            if (share < 1.0f && (by_mass || whole)) {
                u64 m[kFew / kSampleThreads], sums = 0, up_to;
#pragma unroll
                for (int j = 0; j < kFew / kSampleThreads; ++j) {
                    const int i = threadIdx.x * (kFew / kSampleThreads) + j;
                    m[j] = i < nth ? sh.few.mass[i] : 0;
                    sums += m[j];
                }
                u64 now = (by_mass ? base : 0) + cta_prefix(sums, sh.warp[3], up_to);
                const u64 reach = by_mass ? target : share_of<true>(share, up_to);
#pragma unroll
                for (int j = 0; j < kFew / kSampleThreads; ++j) {
                    if (now < reach && now + m[j] >= reach)
                        sh.found[0] = sh.few.place[threadIdx.x * (kFew / kSampleThreads) + j];
                    now += m[j];
                }
            } else if (s.tid == 0) {
                sh.found[0] = sh.few.place[nth - 1];
            }
        }
    }
    __syncthreads();
    u64 result[3] = {s.tid == 0 ? sh.found[0] : 0, s.tid == 0 ? sh.found[1] : 0, s.tid == 0 ? sh.found[2] : 0};
    s.template total<3>(result);
    if (!result[1]) {
        raise(cut, result[0]);
        return !whole ? CUT : result[2] <= kListed ? LISTED : DONE;
    }
    if (quick) return MANY;
    // Many tokens lie close together (equal logits, a high temperature): the cut bit by bit, the largest place with enough at or above it
    u64 found = 0;
    for (int bit = 63; bit >= 0; --bit) {
        const u64 trial = found | 1ull << bit;
        u64 c[1] = {0};
        s.each([&](float x, int i) {
            if (cut.keeps(x, s.first + i) && place_of(x, s.first + i) >= trial) c[0] += by_mass ? w.mass(x) : 1;
        });
        s.template total<1>(c);
        if (c[0] >= target) found = trial;
    }
    raise(cut, found);
    return CUT;
}

// The token, by the first CTA alone, where move_cut has left it all that are kept. It sorts them again, by indices; above kListed that takes as long
// as the passes over the row which it saves. Masses are rounded by eight neighbouring tokens, as in those passes: which way a call goes depends on its
// number of rows and on alignment, and its tokens do not.
template <typename T>
__device__ void take_listed(const Sampler<T> &s, const Weigh &w, const Cut &cut, float min_p, int64_t n) {
    SampleShared &sh = s.sh;
    constexpr int kEach = kFew / kSampleThreads;
    const int count = static_cast<int>(sh.found[2]), mine = s.tid * kEach;
    u64 v[kEach], m[kEach], kept = 0, all;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        v[j] = m[j] = 0;
        if (mine + j < count) {
            const u64 place = sh.few.place[mine + j];
            const float x = unordered(static_cast<uint32_t>(place >> 32)), weight = w.weight(x);
            m[j] = __float_as_uint(weight);
            if (cut.keeps(x, static_cast<int>(0xffffffffu - static_cast<uint32_t>(place))) && weight >= min_p) v[j] = place & 0xffffffffu, ++kept;
        }
    }
    u64 at = cta_prefix(kept, sh.warp[0], all);  // (with barriers)
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (v[j]) sh.few.place[at] = v[j], sh.few.mass[at++] = m[j];
    const int keep = static_cast<int>(all);
    __syncthreads();
    sort_few(sh, keep);  // by rising indices
    const auto token = [&](int i) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(sh.few.place[i])); };
    const auto weight = [&](int i) { return __uint_as_float(static_cast<uint32_t>(sh.few.mass[i])); };
    u64 sum = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {  // the first of its eight has their mass
        const int i = mine + j;
        v[j] = 0;
        if (i < keep && (i == 0 || token(i - 1) >> 3 != token(i) >> 3)) {
            float eight = 0.0f;
            for (int l = i; l < keep && token(l) >> 3 == token(i) >> 3; ++l) eight += weight(l);
            v[j] = static_cast<u64>(__float2ull_rn(eight * kMass));
        }
        sum += v[j];
    }
    u64 now = cta_prefix(sum, sh.warp[0], all);
    const u64 target = target_of(s.p.u[n], all);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        if (now <= target && now + v[j] > target) {  // as in the passes
            const int i = mine + j;
            const float left = static_cast<float>(target - now) / kMass;
            float up_to = 0.0f, taken = 0.0f;
            int to = -1;
            bool passed = false;
            for (int l = i; l < keep && token(l) >> 3 == token(i) >> 3; ++l) {
                up_to += weight(l);
                if (weight(l) > 0.0f && !passed) to = token(l), taken = weight(l), passed = up_to > left;
            }
            s.p.tokens[n] = to;
            if (s.p.probs) s.p.probs[n] = static_cast<float>(static_cast<double>(taken) * kMass / static_cast<double>(all));
        }
        now += v[j];
    }
}

template <typename T>
__global__ void __launch_bounds__(kSampleThreads) based_sample_kernel(SampleParams p) {
    extern __shared__ __align__(16) uint8_t memory[];
    SampleShared &sh = *reinterpret_cast<SampleShared *>(memory);
    T *const tokens = reinterpret_cast<T *>(memory + sizeof(SampleShared));
    const int64_t n = blockIdx.x / p.cluster;
    const uint32_t rank = p.cluster > 1 ? cluster_rank() : 0;
    const int first = static_cast<int>(rank) * p.slice, len = max(0, min(p.slice, p.V - first));
    griddep_wait();
    const T *const src = static_cast<const T *>(p.logits) + n * p.stride + first;
    Sampler<T> s = {p, sh, p.resident ? tokens : src, first, len, rank};
    for (int i = threadIdx.x; i < 3 * kBins; i += kSampleThreads) sh.bins[0][i] = 0;
    if (threadIdx.x == 0) sh.count = 0;
    float top = -INFINITY;
    int top_at = 0;
    const auto look = [&](float x, int i) {
        if (x > top) top = x, top_at = i;  // indices rise: the first of equals
    };
    if (p.resident && p.words) {
        constexpr int kEl = 16 / sizeof(T);
        const int words = (len + kEl - 1) / kEl;  // the row's last word is whole: p.words has V a multiple of it
#pragma unroll 4
        for (int i = threadIdx.x; i < words; i += kSampleThreads) {
            Pack<T, kEl> w = *reinterpret_cast<const Pack<T, kEl> *>(src + i * kEl);
#pragma unroll
            for (int e = 0; e < kEl; ++e) {
                float x = to_f32(w.v[e]);
                if (!(x == x)) x = -INFINITY, w.v[e] = from_f32<T>(x);
                look(x, i * kEl + e);
            }
            *reinterpret_cast<Pack<T, kEl> *>(tokens + i * kEl) = w;
        }
        __syncthreads();
    } else if (p.resident) {
#pragma unroll 8
        for (int i = threadIdx.x; i < len; i += kSampleThreads) {
            float x = to_f32(src[i]);
            if (!(x == x)) x = -INFINITY;
            tokens[i] = from_f32<T>(x);
            look(x, i);
        }
        __syncthreads();
    } else {
        s.each(look);
    }
    u64 best[1] = {place_of(top, first + top_at)};
    s.template total<1, true>(best);
    const float most = unordered(static_cast<uint32_t>(best[0] >> 32));
    const float temperature = p.temperature ? p.temperature[n] : p.temperature_all;
    const bool none = !(most > -INFINITY);
    if (none || !(temperature > 0.0f) || most == INFINITY) {
        if (rank == 0 && threadIdx.x == 0) {
            p.tokens[n] = none ? -1 : static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(best[0]));
            if (p.probs) p.probs[n] = none ? 0.0f : 1.0f;
        }
        s.meet();  // shared memory stays until the others have read it
        return;
    }
    Weigh w;
    w.most = most, w.hi = 1.44269502f / temperature, w.lo = (fmaf(-w.hi, temperature, 1.44269502f) + 1.92596303e-8f) / temperature;
    if (!(w.hi < 3e38f)) w.hi = 3e38f, w.lo = 0.0f;
    if (temperature == INFINITY) w.lo = 0.0f;  // (hi is 0: all alike)
    int k = p.top_k ? p.top_k[n] : p.top_k_all;
    float top_p = p.top_p ? p.top_p[n] : p.top_p_all;
    float min_p = p.min_p ? p.min_p[n] : p.min_p_all;
    min_p = min_p > 0.0f ? fminf(min_p, 1.0f) : 0.0f;
    if (k <= 0 || k > p.V) k = p.V;
    if (!(top_p < 1.0f)) top_p = 1.0f;
    if (top_p <= 0.0f) k = 1, top_p = 1.0f;
    Cut cut;
    const auto clear = [&] {
        for (int i = threadIdx.x; i < 3 * kBins; i += kSampleThreads) sh.bins[0][i] = 0;
        __syncthreads();
    };
    // (256 x 50000 bf16: top-k 50 by the threads' largest 54 us, by all tokens 73; 61 x 130000 float32: 46 and 60, but top-k 1000, where more lies above
    // their bound and is sorted, 118 and 93)
    Moved moved = MANY;
    if (k < p.V) {
        if (k <= static_cast<int>(kListed) && 2 * k <= p.cluster * kSampleThreads) moved = move_cut(s, w, k, top_p, cut, true, top);
        if (moved == MANY) {
            clear();
            moved = move_cut(s, w, k, top_p, cut, false, top);
        }
        if (moved == LISTED) {
            s.meet();
            if (rank == 0) take_listed(s, w, cut, min_p, n);
            return;
        }
        if (moved == CUT && top_p < 1.0f) clear();
    }
    if (moved != DONE && top_p < 1.0f) move_cut(s, w, 0, top_p, cut, false, top);
    const auto kept = [&](float x, int i) -> float {
        if (!cut.keeps(x, first + i)) return 0.0f;
        const float v = w.weight(x);
        return v >= min_p ? v : 0.0f;
    };
    // the mass of eight tokens: the same in both passes
    const auto mass_of = [&](int i, int to) -> u64 {
        float sum = 0.0f;
        s.eight(i, to, [&](float x, int e) { sum += kept(x, e); });
        return static_cast<u64>(__float2ull_rn(sum * kMass));
    };
    const int per = (len + kSampleWarps * 8 - 1) / (kSampleWarps * 8) * 8, begin = s.warp * per, to = min(len, begin + per);
    u64 sum[1] = {0}, before[1];
    for (int i = begin + 8 * s.lane; i < to; i += 256) sum[0] += mass_of(i, to);
    s.template total<1>(sum, before);  // leaves the warps' sums in sh.warp
    const float u = p.u[n];
    const u64 target = target_of(u, sum[0]);
    // the warp at which the sum passes the target, then its round, lane and token
    u64 at = before[0];
    for (int i = 0; i < s.warp; ++i) at += sh.warp[0][i];
    if (at <= target && at + sh.warp[0][s.warp] > target) {
        for (int i0 = begin; i0 < to; i0 += 256) {
            const int i = i0 + 8 * s.lane;
            const u64 m = i < to ? mass_of(i, to) : 0;
            u64 up = m;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const u64 o = __shfl_up_sync(0xffffffffu, up, d);
                if (s.lane >= d) up += o;
            }
            const u64 mine = at + up - m;
            if (m && mine <= target && mine + m > target) {
                // the token in the eight: the first at which their sum passes what is left, or the last that is kept
                const float left = static_cast<float>(target - mine) / kMass;
                float now = 0.0f, weight = 0.0f;
                int token = -1;
                bool passed = false;
                s.eight(i, to, [&](float x, int e) {
                    const float v = kept(x, e);
                    now += v;
                    if (v > 0.0f && !passed) token = first + e, weight = v, passed = now > left;
                });
                p.tokens[n] = token;
                if (p.probs) p.probs[n] = static_cast<float>(static_cast<double>(weight) * kMass / static_cast<double>(sum[0]));
            }
            at += __shfl_sync(0xffffffffu, up, 31);
            if (at > target) break;
        }
    }
    s.meet();
}

// ------------------------------------------------------------------------------------------------
// Host
// ------------------------------------------------------------------------------------------------
template <typename T>
int launch_sample(SampleParams &p, int N, int sms, cudaStream_t st) {
    constexpr int64_t kRoom = 226 * 1024 - static_cast<int64_t>(sizeof(SampleShared));
    constexpr int64_t kShare = 113 * 1024 - static_cast<int64_t>(sizeof(SampleShared));  // two CTAs on an SM
    const auto bytes = [&](int cluster) {
        return ((static_cast<int64_t>(p.V) + cluster - 1) / cluster + 7) / 8 * 8 * static_cast<int64_t>(sizeof(T));
    };
    // As many CTAs to a row as leave no more than the SMs', and as its tokens need to lie in shared memory
    int cluster = 1;
    while (cluster < kSampleCluster && (bytes(cluster) > kShare || static_cast<int64_t>(N) * cluster * 2 <= sms) && p.V / (2 * cluster) >= 1024) cluster *= 2;
    p.cluster = cluster, p.slice = static_cast<int>(bytes(cluster) / sizeof(T)), p.resident = bytes(cluster) <= kRoom;
    const size_t smem = sizeof(SampleShared) + (p.resident ? bytes(cluster) : 0);
    OPS_CUDA(allow(based_sample_kernel<T>, 227 * 1024));
    OPS_CUDA(launch_op(based_sample_kernel<T>, dim3(static_cast<unsigned>(N) * cluster), kSampleThreads, smem, st, p, cluster));
    return BASED_OK;
}

}  // namespace
}  // namespace based

extern "C" int based_sample(const void *logits, int64_t stride, int dtype, int N, int V, const float *u, const float *temperature,
                            float temperature_all, const int32_t *top_k, int top_k_all, const float *top_p, float top_p_all, const float *min_p,
                            float min_p_all, int32_t *tokens, float *probs, based_stream_t stream) {
    using namespace based;
    if (!logits || !u || !tokens) return BASED_ERR_NULL_POINTER;
    if (!type_ok(dtype)) return BASED_ERR_UNSUPPORTED_TYPE;
    if (N < 1 || V < 1 || N > (1 << 26) || V > kSampleMostV) return BASED_ERR_BAD_SIZE;
    if (stride < 0) return BASED_ERR_BAD_STRIDE;
    const size_t es = elem_size(dtype);
    if (!aligned(logits, es) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) ||
        !aligned(tokens, 4) || !aligned(probs, 4))
        return BASED_ERR_MISALIGNED;
    const Span in[] = {span(logits, (N - 1) * stride + V - 1, es), span(u, N - 1, 4), span(temperature, N - 1, 4), span(top_k, N - 1, 4),
                       span(top_p, N - 1, 4), span(min_p, N - 1, 4)};
    const Span st = span(tokens, N - 1, 4), sp = span(probs, N - 1, 4);
    for (const Span &s : in)
        if (overlap(s, st) || overlap(s, sp)) return BASED_ERR_ALIASING;
    if (overlap(st, sp)) return BASED_ERR_ALIASING;
    int sms;
    if (const int rc = host_device(&sms)) return rc;
    SampleParams p = {};
    p.logits = logits, p.stride = stride, p.V = V, p.u = u;
    p.temperature = temperature, p.temperature_all = temperature_all, p.top_k = top_k, p.top_k_all = top_k_all;
    p.top_p = top_p, p.top_p_all = top_p_all, p.min_p = min_p, p.min_p_all = min_p_all, p.tokens = tokens, p.probs = probs;
    p.words = aligned(logits, 16) && stride * static_cast<int64_t>(es) % 16 == 0 && V * es % 16 == 0;
    cudaStream_t stm = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == BASED_F32) return launch_sample<float>(p, N, sms, stm);
    if (dtype == BASED_BF16) return launch_sample<__nv_bfloat16>(p, N, sms, stm);
    return launch_sample<__half>(p, N, sms, stm);
}
