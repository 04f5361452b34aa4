// Shared by the block operators (mv_linear.cu, mv_activation.cu, mv_norm.cu).
#pragma once

#include <cstring>
#include <type_traits>

#include "mv_moe.cuh"

namespace mvblock {

using namespace mvmoe;

// 1 / (1 + exp(-v)) to some units of 2^-22 of its value, and |v| 2^-23 more where v is negative (the
// exponent's rounding); 0 under -88, where the exponential is infinite.
__device__ __forceinline__ float logistic(float v) { return reciprocal_fast(1.0f + exp2_fast(-kLog2e * v)); }

constexpr float kRootHalf = 0.70710678118654752f;
constexpr float kTanhOuter = 1.5957691216057308f;       // 2 sqrt(2 / pi)
constexpr float kTanhInner = 0.044715f;

// Tanh's form of gelu is z logistic(2 v), v = sqrt(2 / pi) (z + 0.044715 z^3),
// since (1 + tanh v) / 2 is the logistic function of 2 v: small values keep
// their relative precision, which 1 + tanh v would lose.  erfc does the same
// for gelu itself.  An infinite z counts as its limit.
__device__ __forceinline__ float activation(u32 act, float z)
{
    switch (act) {
    case MV_ACT_RELU: return z < 0.0f ? 0.0f : z;                      // a NaN stays one
    case MV_ACT_GELU: return z == -INFINITY ? 0.0f : 0.5f * z * erfcf(-kRootHalf * z);
    case MV_ACT_GELU_TANH: return z == -INFINITY ? 0.0f : z * logistic(kTanhOuter * fmaf(kTanhInner * z * z, z, z));
    case MV_ACT_SILU: return z == -INFINITY ? 0.0f : z * logistic(z);
    default: return z;
    }
}

__device__ __forceinline__ float activation_slope(u32 act, float z)
{
    switch (act) {
    case MV_ACT_RELU: return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
    case MV_ACT_GELU: {
        const float bell = 0.39894228040143268f * exp2_fast(-0.5f * kLog2e * z * z);
        return 0.5f * erfcf(-kRootHalf * z) + (bell > 0.0f ? z * bell : 0.0f);
    }
    case MV_ACT_GELU_TANH: {
        // q + z q (1 - q) dv/dz; q (1 - q) from |v|, where both factors are precise
        const float zz = z * z, v = kTanhOuter * fmaf(kTanhInner * zz, z, z);
        const float e = exp2_fast(-kLog2e * fabsf(v)), p = reciprocal_fast(1.0f + e);
        const float both = e * p * p, dv = kTanhOuter * fmaf(3.0f * kTanhInner, zz, 1.0f);
        return (v < 0.0f ? e * p : p) + (both > 0.0f ? z * both * dv : 0.0f);
    }
    case MV_ACT_SILU: {
        const float e = exp2_fast(-kLog2e * fabsf(z)), p = reciprocal_fast(1.0f + e), both = e * p * p;
        return (z < 0.0f ? e * p : p) + (both > 0.0f ? z * both : 0.0f);
    }
    default: return 1.0f;
    }
}

// The normal distribution Phi(z) and its density, two values an instruction where
// there is one, for 16-bit results: to 2e-7 of 1, less than a hundredth of their
// rounding, and with a fraction of erfc's instructions.  With a = |z| and
// t = 1 / (1 + 0.4 a) the tail is t 2^(p(t) - a^2 log2(e) / 2); p is a Chebyshev fit
// (degree 8, to 1.3e-7) of what that leaves of its logarithm.
__device__ __forceinline__ float2 normal2(float2 z, float2 &density)
{
    constexpr float kTail[9] = {0.275790244f, -1.41183841f, 2.81971717f, -2.53615332f, 0.788428247f, -0.264325142f, 0.537471354f, 1.43842268f, -2.64751267f};
    auto all = [](float v) { return make_float2(v, v); };
    const float2 a = make_float2(fabsf(z.x), fabsf(z.y)), below = __ffma2_rn(a, all(0.4f), all(1.0f));
    const float2 t = make_float2(reciprocal_fast(below.x), reciprocal_fast(below.y));
    float2 p = all(kTail[0]);
#pragma unroll
    for (int i = 1; i < 9; i++) p = __ffma2_rn(p, t, all(kTail[i]));
    const float2 square = __fmul2_rn(__fmul2_rn(a, a), all(-0.5f * kLog2e));
    p = __fadd2_rn(p, square);
    const float2 tail = __fmul2_rn(t, make_float2(exp2_fast(p.x), exp2_fast(p.y)));
    density = __fmul2_rn(make_float2(exp2_fast(square.x), exp2_fast(square.y)), all(0.39894228040143268f));
    return make_float2(z.x > 0.0f ? 1.0f - tail.x : tail.x, z.y > 0.0f ? 1.0f - tail.y : tail.y);
}

// logistic() of two values, at the same price an instruction where there is one.
__device__ __forceinline__ float2 logistic2(float2 v)
{
    const float2 w = __fmul2_rn(v, make_float2(-kLog2e, -kLog2e));
    const float2 below = __fadd2_rn(make_float2(exp2_fast(w.x), exp2_fast(w.y)), make_float2(1.0f, 1.0f));
    return make_float2(reciprocal_fast(below.x), reciprocal_fast(below.y));
}
// activation() of N values, by pairs.  SHORT: for 16-bit results.
template <u32 ACT, int N, bool SHORT> __device__ __forceinline__ void activate(float *v)
{
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 z = make_float2(v[i], v[i + 1]);
        if constexpr (ACT == MV_ACT_GELU_TANH || ACT == MV_ACT_SILU || (ACT == MV_ACT_GELU && SHORT)) {
            float2 q, rest;
            if constexpr (ACT == MV_ACT_GELU) {
                q = normal2(z, rest);
            } else if constexpr (ACT == MV_ACT_SILU) {
                q = logistic2(z);
            } else {
                const float2 zz = __fmul2_rn(__fmul2_rn(z, z), make_float2(kTanhInner * kTanhOuter, kTanhInner * kTanhOuter));
                q = logistic2(__fmul2_rn(__fadd2_rn(zz, make_float2(kTanhOuter, kTanhOuter)), z));
            }
            const float2 y = __fmul2_rn(z, q);
            v[i] = z.x == -INFINITY ? 0.0f : y.x;
            v[i + 1] = z.y == -INFINITY ? 0.0f : y.y;
        } else {
            v[i] = activation(ACT, z.x);
            v[i + 1] = activation(ACT, z.y);
        }
    }
}
template <int N, bool SHORT> __device__ __forceinline__ void activate(u32 act, float *v)
{
    if (act == MV_ACT_RELU) activate<MV_ACT_RELU, N, SHORT>(v);
    else if (act == MV_ACT_GELU) activate<MV_ACT_GELU, N, SHORT>(v);
    else if (act == MV_ACT_GELU_TANH) activate<MV_ACT_GELU_TANH, N, SHORT>(v);
    else if (act == MV_ACT_SILU) activate<MV_ACT_SILU, N, SHORT>(v);
}

// 16 bytes of a row as 32-bit values; N neighbours (16 bytes or more, or one) from and to memory.
template <class T, int N> __device__ __forceinline__ void widen_piece(const uint4 &w, float *v)
{
    const u32 words[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = __uint_as_float(words[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                v[2 * i] = __uint_as_float(words[i] << 16);
                v[2 * i + 1] = __uint_as_float(words[i] & 0xFFFF0000u);
            } else {
                __half2 h;
                memcpy(&h, &words[i], 4);
                const float2 f = __half22float2(h);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}
template <class T, int N> __device__ __forceinline__ void get(const T *p, float *v)
{
    if constexpr (N == 1) {
        v[0] = to_float(*p);
    } else {
        constexpr int kEach = 16 / sizeof(T);       // of a 16-byte word
#pragma unroll
        for (int i = 0; i < N; i += kEach) widen_piece<T, kEach>(*reinterpret_cast<const uint4 *>(p + i), v + i);
    }
}
template <class T, int N> __device__ __forceinline__ void put(T *p, const float *v)
{
    if constexpr (N == 1) {
        *p = from_float<T>(v[0]);
    } else {
        constexpr int kEach = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < N; i += kEach) {
            uint4 w;
            if constexpr (sizeof(T) == 4) {
                w = make_uint4(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3]));
            } else {
                u32 words[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(v[i + 2 * j], v[i + 2 * j + 1]);
                        memcpy(&words[j], &h, 4);
                    } else {
                        const __half2 h = __floats2half2_rn(v[i + 2 * j], v[i + 2 * j + 1]);
                        memcpy(&words[j], &h, 4);
                    }
                }
                w = make_uint4(words[0], words[1], words[2], words[3]);
            }
            *reinterpret_cast<uint4 *>(p + i) = w;
        }
    }
}
}  // namespace mvblock
