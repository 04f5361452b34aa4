// dz = scale * dy * act'(z) (mv_activation_backward in include/mv.h): two
// arrays read and one written, so memory bounds it: 8192 x 20480 bfloat16 (1.0 GB)
// gelu_tanh 163 us, 6.2 TB/s; silu 154; gelu 171, where instructions come near.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "mv_block.cuh"

namespace mvblock {

struct SlopeArgs {
    const void *dy, *z;
    void *dz;
    u64 tokens, cols, dy_stride, z_stride;
    float scale;
};

constexpr u32 kSlopeThreads = 256;

// scale * dy * act'(z) of two neighbours: the formulas of activation_slope(),
// two values an instruction where there is one, as one value at a time it is
// instructions, not memory, that bound 16-bit arrays (8192 x 20480: gelu_tanh 172 us,
// so 163; gelu 316, so 171).
// SHORT: for a 16-bit result.
template <u32 ACT, bool SHORT> __device__ __forceinline__ float2 slope2(float2 z, float2 dy, float scale)
{
    const float2 s = make_float2(scale, scale);
    if constexpr (ACT == MV_ACT_GELU_TANH || ACT == MV_ACT_SILU) {
        auto all = [](float v) { return make_float2(v, v); };
        float2 v = z, dv = all(1.0f);
        if constexpr (ACT == MV_ACT_GELU_TANH) {
            const float2 zz = __fmul2_rn(z, z);
            v = __fmul2_rn(__ffma2_rn(__fmul2_rn(zz, all(kTanhInner)), z, z), all(kTanhOuter));
            dv = __ffma2_rn(zz, all(3.0f * kTanhInner * kTanhOuter), all(kTanhOuter));
        }
        const float2 e = make_float2(exp2_fast(-kLog2e * fabsf(v.x)), exp2_fast(-kLog2e * fabsf(v.y)));
        const float2 below = __fadd2_rn(e, all(1.0f)), p = make_float2(reciprocal_fast(below.x), reciprocal_fast(below.y));
        const float2 ep = __fmul2_rn(e, p), both = __fmul2_rn(ep, p);
        const float2 q = make_float2(v.x < 0.0f ? ep.x : p.x, v.y < 0.0f ? ep.y : p.y);
        float2 more = __fmul2_rn(z, both);
        if constexpr (ACT == MV_ACT_GELU_TANH) more = __fmul2_rn(more, dv);
        // far out `both` is 0, and what it is multiplied by may be infinite
        more = make_float2(both.x > 0.0f ? more.x : 0.0f, both.y > 0.0f ? more.y : 0.0f);
        return __fmul2_rn(__fmul2_rn(dy, __fadd2_rn(q, more)), s);
    } else if constexpr (ACT == MV_ACT_GELU && SHORT) {
        // Phi(z) + z phi(z)
        float2 bell;
        const float2 q = normal2(z, bell);
        float2 more = __fmul2_rn(z, bell);
        more = make_float2(bell.x > 0.0f ? more.x : 0.0f, bell.y > 0.0f ? more.y : 0.0f);
        return __fmul2_rn(__fmul2_rn(dy, __fadd2_rn(q, more)), s);
    } else {
        return __fmul2_rn(__fmul2_rn(dy, make_float2(activation_slope(ACT, z.x), activation_slope(ACT, z.y))), s);
    }
}

// Dense arrays are one long row; 16 bytes of each array a step, four steps of a thread under way.
template <class T, u32 ACT> __global__ void __launch_bounds__(kSlopeThreads) k_slope(const SlopeArgs a)
{
    constexpr u32 N = 16 / sizeof(T), kAhead = 4;
    const u64 pieces = a.cols / N, n = a.tokens * pieces, step = (u64)kSlopeThreads;
    const T *dy = static_cast<const T *>(a.dy), *z = static_cast<const T *>(a.z);
    T *dz = static_cast<T *>(a.dz);
    for (u64 i0 = (u64)blockIdx.x * (kSlopeThreads * kAhead) + threadIdx.x; i0 < n; i0 += (u64)gridDim.x * (kSlopeThreads * kAhead)) {
        uint4 g[kAhead], v[kAhead];
        u64 to[kAhead];
#pragma unroll
        for (u32 j = 0; j < kAhead; j++) {
            const u64 i = i0 + j * step;
            if (i >= n) break;
            const u64 r = a.tokens == 1 ? 0 : i / pieces, c = (i - r * pieces) * N;
            g[j] = __ldcs(reinterpret_cast<const uint4 *>(dy + r * a.dy_stride + c));
            v[j] = __ldcs(reinterpret_cast<const uint4 *>(z + r * a.z_stride + c));
            to[j] = r * a.cols + c;
        }
#pragma unroll
        for (u32 j = 0; j < kAhead; j++) {
            if (i0 + j * step >= n) break;
            float gt[N], vt[N];
            widen_piece<T, N>(g[j], gt);
            widen_piece<T, N>(v[j], vt);
#pragma unroll
            for (u32 e = 0; e < N; e += 2) {
                const float2 d = slope2<ACT, sizeof(T) == 2>(make_float2(vt[e], vt[e + 1]), make_float2(gt[e], gt[e + 1]), a.scale);
                gt[e] = d.x;
                gt[e + 1] = d.y;
            }
            put<T, N>(dz + to[j], gt);
        }
    }
}

// Rows that no 16-byte access fits.
template <class T, u32 ACT> __global__ void __launch_bounds__(kSlopeThreads) k_slope_each(const SlopeArgs a)
{
    const T *dy = static_cast<const T *>(a.dy), *z = static_cast<const T *>(a.z);
    const u64 n = a.tokens * a.cols;
    for (u64 i = (u64)blockIdx.x * kSlopeThreads + threadIdx.x; i < n; i += (u64)gridDim.x * kSlopeThreads) {
        const u64 r = a.tokens == 1 ? 0 : i / a.cols, c = i - r * a.cols;
        static_cast<T *>(a.dz)[i] =
            from_float<T>(a.scale * (to_float(dy[r * a.dy_stride + c]) * activation_slope(ACT, to_float(z[r * a.z_stride + c]))));
    }
}

template <class T, u32 ACT> int run_slope(SlopeArgs a, cudaStream_t stream)
{
    if (a.dy_stride == a.cols && a.z_stride == a.cols) { a.cols *= a.tokens; a.tokens = 1; a.dy_stride = a.z_stride = a.cols; }
    constexpr u32 N = 16 / sizeof(T);
    const bool wide = a.cols % N == 0 && (a.tokens == 1 || (a.dy_stride % N == 0 && a.z_stride % N == 0)) && aligned(a.dy, 16) &&
                      aligned(a.z, 16) && aligned(a.dz, 16);
    const u64 each = wide ? (u64)kSlopeThreads * 4 * N : kSlopeThreads * 4;
    const u32 blocks = (u32)std::min<u64>((a.tokens * a.cols + each - 1) / each, 1u << 20);
    return wide ? launch(k_slope<T, ACT>, dim3(blocks), kSlopeThreads, 0, stream, a)
                : launch(k_slope_each<T, ACT>, dim3(blocks), kSlopeThreads, 0, stream, a);
}

template <class T> int run_slope(const SlopeArgs &a, u32 act, cudaStream_t stream)
{
    switch (act) {
    case MV_ACT_RELU: return run_slope<T, MV_ACT_RELU>(a, stream);
    case MV_ACT_GELU: return run_slope<T, MV_ACT_GELU>(a, stream);
    case MV_ACT_GELU_TANH: return run_slope<T, MV_ACT_GELU_TANH>(a, stream);
    case MV_ACT_SILU: return run_slope<T, MV_ACT_SILU>(a, stream);
    default: return run_slope<T, MV_ACT_NONE>(a, stream);
    }
}

}  // namespace mvblock

using namespace mvblock;

extern "C" int mv_activation_backward(const mv_act_grad_desc *d, void *stream)
{
    if (!d || d->dtype > MV_BF16 || d->act > MV_ACT_SILU || !std::isfinite(d->scale)) return MV_EINVAL;
    if (d->tokens == 0 || d->cols == 0) return MV_OK;
    if (d->dy_stride < d->cols || d->z_stride < d->cols || !d->dy || !d->z || !d->dz || !aligned(d->dy, dtype_size(d->dtype)) ||
        !aligned(d->z, dtype_size(d->dtype)) || !aligned(d->dz, dtype_size(d->dtype)))
        return MV_EINVAL;
    if (d->tokens > 1ull << 31 || d->cols > 1ull << 31 || d->dy_stride > 1ull << 36 || d->z_stride > 1ull << 36) return MV_EOVERFLOW;
    const SlopeArgs a = {d->dy, d->z, d->dz, d->tokens, d->cols, d->dy_stride, d->z_stride, d->scale};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (d->dtype == MV_F32) return run_slope<float>(a, d->act, s);
    return d->dtype == MV_F16 ? run_slope<__half>(a, d->act, s) : run_slope<__nv_bfloat16>(a, d->act, s);
}
