// ops_common.cuh: what the kernels and host code of the operators in include/based_ops.h share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/based_ops.h"
#include "sm103_ptx.cuh"

namespace based {

// defined in based_fwd.cu
int host_cuda_fail(cudaError_t e, const char *what);
int host_device(int *sms);  // checks that the current device is an sm_103 GPU

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
cudaError_t launch_op(void (*kernel)(P), dim3 grid, int block, size_t smem, cudaStream_t st, const P &arg,
                      int cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
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

// exp and the logistic function to about one unit of float32's last place: the recurrence
// multiplies thousands of decays, so that the error of a faster approximation would add up.
// 1 / d by the hardware's approximation and one step of Newton's method.
__device__ __forceinline__ float recip(float d) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    return fmaf(r, fmaf(-d, r, 1.0f), r);
}
// p = sigma(g), q = sigma(-g) = 1 - p, each with its own relative accuracy. Below g = -87, where p
// is under 2e-38, g counts as -87, so that exp(-g) and its reciprocal stay in range; NaN stays NaN.
__device__ __forceinline__ void sigmoid_pair(float g, float &p, float &q) {
    float c;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(g), "f"(-87.0f));
    const float e = expf(-c);
    p = recip(1.0f + e);
    q = e * p;
}

}  // namespace based
