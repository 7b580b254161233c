// ops_common.cuh: what the kernels and host code of the operators in include/based_ops.h share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/based_ops.h"
#include "sm103_ptx.cuh"

namespace based {

// defined in based_fwd.cu
int host_cuda_fail(cudaError_t e, const char *what);
int host_device(int *sms);  // checks that the current device is an sm_103 GPU
// defined in based_scan.cu: the current device's status word of the scan kernels
cudaError_t scan_status(unsigned int *status, bool clear);
// defined in based_delta.cu: that of the delta rule's kernels
cudaError_t delta_status(unsigned int *status, bool clear);

#define OPS_CUDA(call)                                            \
    do {                                                          \
        cudaError_t e_ = (call);                                  \
        if (e_ != cudaSuccess) return host_cuda_fail(e_, #call);  \
    } while (0)

// ------------------------------------------------------------------------------------------------
// Host: argument checks
// ------------------------------------------------------------------------------------------------
inline size_t elem_size(int dtype) { return dtype == BASED_F32 ? 4 : 2; }
inline bool type_ok(int dtype) { return dtype == BASED_F32 || dtype == BASED_BF16 || dtype == BASED_F16; }
inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The bytes an argument spans: from its first element to one past its last. Empty where it is NULL.
struct Span {
    uintptr_t a, b;
};
inline Span span(const void *p, int64_t last_elem, size_t es) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return p ? Span{a, a + (static_cast<uintptr_t>(last_elem) + 1) * es} : Span{0, 0};
}
inline bool overlap(const Span &x, const Span &y) { return x.a < y.b && y.a < x.b; }

// Launches kernel<<<grid, block, smem, st>>>(arg) as a programmatic dependent of the kernel before
// it in the stream: its CTAs may start while that kernel finishes, and every thread that touches
// memory first waits for it (griddep_wait). cluster: CTAs per cluster along x.
template <typename P>
cudaError_t launch_op(void (*kernel)(P), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const P &arg,
                      int cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, arg);
}

// Lets a kernel have `smem` bytes of dynamic shared memory and clusters of 16; once per kernel and
// device. K: a kernel's function type.
template <typename K>
cudaError_t allow(K *kernel, size_t smem) {
    struct Done {
        K *kernel;
        uint64_t devices;
    };
    static std::mutex m;
    static Done done[64];
    int dev, i = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(m);
    while (i < 63 && done[i].kernel && done[i].kernel != kernel) ++i;
    if (done[i].kernel == kernel && (done[i].devices >> (dev & 63) & 1)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done[i] = {kernel, (done[i].kernel == kernel ? done[i].devices : 0) | 1ull << (dev & 63)};
    return e;
}

// How many clusters of `cluster` CTAs of a kernel the current device holds at once: a cluster lies within
// one of the parts that the SMs form, and those are not all equal. Asked once per kernel, device and size.
inline int resident_clusters(const void *kernel, int threads, size_t smem, int cluster, int *out) {
    struct Entry {
        const void *kernel;
        int dev, cluster, n;
    };
    static std::mutex m;
    static Entry table[1024];
    static int used = 0;
    int dev;
    OPS_CUDA(cudaGetDevice(&dev));
    std::lock_guard<std::mutex> lk(m);
    for (int i = 0; i < used; ++i) {
        const Entry &e = table[i];
        if (e.kernel == kernel && e.dev == dev && e.cluster == cluster) {
            *out = e.n;
            return BASED_OK;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    OPS_CUDA(cudaOccupancyMaxActiveClusters(&n, kernel, &cfg));
    if (used < 1024) table[used++] = {kernel, dev, cluster, n};
    *out = n;
    return BASED_OK;
}

// ------------------------------------------------------------------------------------------------
// Device: clusters
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ------------------------------------------------------------------------------------------------
// Device: element types
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
    return __float2half_rn(v);
}

// N consecutive elements that are loaded and stored as one word (4 to 32 bytes; 32 as two of 16)
template <typename T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Pack {
    T v[N];
};

// ------------------------------------------------------------------------------------------------
// Device: float32 vectors of one or two elements. Two go through the packed instructions, which
// take one issue slot for both.
// ------------------------------------------------------------------------------------------------
template <int N>
struct Vec;
template <>
struct Vec<1> {
    float v[1];
};
template <>
struct alignas(8) Vec<2> {
    float v[2];
};
template <int N>
__device__ __forceinline__ Vec<N> splat(float s) {
    Vec<N> r;
#pragma unroll
    for (int j = 0; j < N; ++j) r.v[j] = s;
    return r;
}
__device__ __forceinline__ uint64_t bits2(const Vec<2> &a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.v[0]), "f"(a.v[1]));
    return r;
}
__device__ __forceinline__ Vec<2> from_bits2(uint64_t b) {
    Vec<2> r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.v[0]), "=f"(r.v[1]) : "l"(b));
    return r;
}
__device__ __forceinline__ Vec<1> vfma(const Vec<1> &a, const Vec<1> &b, const Vec<1> &c) { return {fmaf(a.v[0], b.v[0], c.v[0])}; }
__device__ __forceinline__ Vec<1> vmul(const Vec<1> &a, const Vec<1> &b) { return {a.v[0] * b.v[0]}; }
__device__ __forceinline__ Vec<1> vadd(const Vec<1> &a, const Vec<1> &b) { return {a.v[0] + b.v[0]}; }
__device__ __forceinline__ Vec<2> vfma(const Vec<2> &a, const Vec<2> &b, const Vec<2> &c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return from_bits2(r);
}
__device__ __forceinline__ Vec<2> vmul(const Vec<2> &a, const Vec<2> &b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return from_bits2(r);
}
__device__ __forceinline__ Vec<2> vadd(const Vec<2> &a, const Vec<2> &b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return from_bits2(r);
}
// A 32-bit word as one float32 or two 16-bit elements, the first in the low half.
template <typename T>
__device__ __forceinline__ Vec<4 / sizeof(T)> unpack(uint32_t w);
template <>
__device__ __forceinline__ Vec<1> unpack<float>(uint32_t w) {
    return {{__uint_as_float(w)}};
}
template <>
__device__ __forceinline__ Vec<2> unpack<__nv_bfloat16>(uint32_t w) {
    return {{__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)}};
}
template <>
__device__ __forceinline__ Vec<2> unpack<__half>(uint32_t w) {
    Vec<2> r;
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}"
        : "=f"(r.v[0]), "=f"(r.v[1])
        : "r"(w));
    return r;
}
template <typename T>
__device__ __forceinline__ uint32_t pack(const Vec<4 / sizeof(T)> &a);
template <>
__device__ __forceinline__ uint32_t pack<float>(const Vec<1> &a) {
    return __float_as_uint(a.v[0]);
}
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(const Vec<2> &a) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(a.v[1]), "f"(a.v[0]));
    return w;
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(const Vec<2> &a) {
    uint32_t w;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(a.v[1]), "f"(a.v[0]));
    return w;
}

// ------------------------------------------------------------------------------------------------
// Device: exp and the logistic function
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ float ex2(float t) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
    return r;
}
__device__ __forceinline__ float rcp(float d) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    return r;
}
// e^x. A single element, as float32 recurrences have it, takes expf(). Of two at once (16-bit elements, and the norm's
// activations) it is 2^t with t = x log2(e) rounded once, off by 2^-22 (the approximation of 2^t) and |x| 2^-24: where a
// decay e^x is near 1 and errors add up over many rows, |x| is small, and an output of 16 bits shows neither.
// (2 x 2047 x 777 float32 by expf: 11.7 + 18.1 us forward and backward, 11.3 + 17.4 by 2^t, and 7.7e-7 off the 64-bit
// result where 2^t was 1.3e-6 off, with log decays of some 400 rows.)
template <int N>
__device__ __forceinline__ Vec<N> vexp(const Vec<N> &x) {
    if (N == 1) return splat<N>(expf(x.v[0]));
    Vec<N> t = vmul(x, splat<N>(1.4426950408889634f));
#pragma unroll
    for (int j = 0; j < N; ++j) t.v[j] = ex2(t.v[j]);
    return t;
}
// p = sigma(g), q = sigma(-g) = 1 - p, each with its own relative accuracy (q = e^-g p, not 1 - p). Below
// g = -87, where p is under 2e-38, g becomes -87, so that e^-g stays finite and g p near 0; NaN stays NaN. A single element's p
// above 1/2 is 1 - q, as close to 1 as float32 has it: the reciprocal's error would add up over a recurrence's rows.
template <int N>
__device__ __forceinline__ void vsigmoid(Vec<N> &g, Vec<N> &p, Vec<N> &q) {
#pragma unroll
    for (int j = 0; j < N; ++j) asm("max.NaN.f32 %0, %1, %2;" : "=f"(g.v[j]) : "f"(g.v[j]), "f"(-87.0f));
    Vec<N> e;
    if (N == 1) {
        e = splat<N>(expf(-g.v[0]));
    } else {
        e = vmul(g, splat<N>(-1.4426950408889634f));
#pragma unroll
        for (int j = 0; j < N; ++j) e.v[j] = ex2(e.v[j]);
    }
    const Vec<N> d = vadd(e, splat<N>(1.0f));
#pragma unroll
    for (int j = 0; j < N; ++j) p.v[j] = rcp(d.v[j]);
    q = vmul(e, p);
    if (N == 1 && e.v[0] < 1.0f) p.v[0] = 1.0f - q.v[0];
}

}  // namespace based
