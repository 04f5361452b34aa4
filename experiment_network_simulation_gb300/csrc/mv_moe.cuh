// Shared by the routed-expert operators (mv_route.cu, mv_exchange.cu,
// mv_experts.cu): element types, warp reductions, launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/mv.h"

namespace mvmoe {

using u32 = uint32_t;
using u64 = uint64_t;

constexpr u32 kFull = 0xFFFFFFFFu;
constexpr u32 kMaxTopk = MV_MOE_MAX_TOPK;
constexpr u32 kMaxExperts = MV_MOE_MAX_EXPERTS;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}

// Reductions over aligned groups of W lanes, in a fixed order (the same
// result on every run, in every lane).
template <int W> __device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int d = W / 2; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}
template <int W> __device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int d = W / 2; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
    return v;
}

// 2^v and 1 / v to 2^-22 of their values or so.
__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float reciprocal_fast(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

inline bool aligned(const void *p, u64 bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline u64 dtype_size(u32 dtype) { return dtype == MV_F32 ? 4 : 2; }

// One launch; its own status, whatever an earlier call left behind.  With
// `early` the kernel may start before the stream's previous one has ended: it
// waits for that one itself (griddepcontrol.wait).
template <class... P, class... A>
int launch_as(bool early, void (*kernel)(P...), dim3 grid, u32 threads, u32 smem, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess ? MV_OK : MV_ECUDA;
}
template <class... P, class... A>
int launch(void (*kernel)(P...), dim3 grid, u32 threads, u32 smem, cudaStream_t stream, A... args)
{
    return launch_as(false, kernel, grid, threads, smem, stream, args...);
}
template <class... P, class... A>
int launch_after(void (*kernel)(P...), dim3 grid, u32 threads, u32 smem, cudaStream_t stream, A... args)
{
    return launch_as(true, kernel, grid, threads, smem, stream, args...);
}

// SMs of the current device (0 if there is none).
inline u32 sm_count()
{
    static int cached[64] = {};
    int dev = -1, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
    if (dev < 64 && cached[dev]) return (u32)cached[dev];
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) cached[dev] = n;
    return (u32)n;
}

}  // namespace mvmoe
