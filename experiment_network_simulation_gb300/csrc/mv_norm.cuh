// Shared by mv_norm.cu and mv_norm_grad.cu: rows held by blocks.
#pragma once

#include "mv_block.cuh"

namespace mvblock {

struct NormArgs {
    const void *y, *residual, *dn, *dr;
    const void *weight, *bias, *post, *post_bias, *gate;
    void *n, *r, *dy, *dresidual, *dgate;
    u64 tokens, y_stride, residual_stride, dn_stride, dr_stride;
    u64 run, rows;                                  // tokens that share a gate; rows a block (backward)
    u32 hidden, layer, params_f32;
    float alpha, eps, inv_hidden;
    u64 pitch;                                      // hidden, up to whole fours
    float *sums;                                    // a block's sums for weight, bias, post, post_bias  [blocks, 4, pitch]
    float *gate_sums;                               // and for its first and last gates                  [blocks, 2, pitch]
};

struct NormShape {
    u32 n, pieces, threads;
    bool whole;                                     // the threads' pieces are the row, and no more
    u32 at_once;                                    // rows that go together (backward)
};
template <class T> int run_norm_grad(const NormArgs &a, const NormShape &s, u64 blocks, u32 smem, bool post, bool bias, cudaStream_t stream);

// A thread's E elements of a row (or of a parameter): pieces of N neighbours (16
// bytes, or one where rows lie on no 16-byte boundary), threads next to each
// other.  WHOLE: the threads' pieces are the row, and nothing lies beyond.  Else a
// piece beyond it is its first one over again, read without a branch, and is
// hidden where it would count.  Arithmetic goes by pairs, two values an instruction.
template <int N> __device__ __forceinline__ u32 column_of(u32 i, u32 hidden, u32 threads)
{
    const u32 c = (i * threads + threadIdx.x) * N;
    return c < hidden ? c : 0;
}
template <class T, int N, bool WHOLE, int E> __device__ __forceinline__ void get_row(const T *row, u32 hidden, u32 threads, float (&v)[E])
{
#pragma unroll
    for (int i = 0; i < E / N; i++) get<T, N>(row + (WHOLE ? (i * threads + threadIdx.x) * N : column_of<N>(i, hidden, threads)), &v[i * N]);
}
template <int N, bool WHOLE, int E> __device__ __forceinline__ void hide(u32 hidden, u32 threads, float (&v)[E])
{
    if constexpr (!WHOLE)
#pragma unroll
        for (int i = 0; i < E / N; i++)
            if ((i * threads + threadIdx.x) * N >= hidden)
#pragma unroll
                for (int j = 0; j < N; j++) v[i * N + j] = 0.0f;
}
template <class T, int N, bool WHOLE, int E> __device__ __forceinline__ void put_row(T *row, u32 hidden, u32 threads, const float (&v)[E])
{
    row += threadIdx.x * N;
#pragma unroll
    for (int i = 0; i < E / N; i++)
        if (WHOLE || (i * threads + threadIdx.x) * N < hidden) put<T, N>(row + i * threads * N, &v[i * N]);
}

__device__ __forceinline__ float2 two(const float *v) { return make_float2(v[0], v[1]); }
__device__ __forceinline__ void set(float *v, float2 w) { v[0] = w.x; v[1] = w.y; }
// d = a b + c; d = a b; d = a + b, of E elements; one operand may be a number.
template <int E> __device__ __forceinline__ void fma_row(float (&d)[E], const float (&a)[E], const float (&b)[E], const float (&c)[E])
{
#pragma unroll
    for (int i = 0; i < E; i += 2) set(&d[i], __ffma2_rn(two(&a[i]), two(&b[i]), two(&c[i])));
}
template <int E> __device__ __forceinline__ void fma_row(float (&d)[E], const float (&a)[E], float b, const float (&c)[E])
{
#pragma unroll
    for (int i = 0; i < E; i += 2) set(&d[i], __ffma2_rn(two(&a[i]), make_float2(b, b), two(&c[i])));
}
template <int E> __device__ __forceinline__ void mul_row(float (&d)[E], const float (&a)[E], const float (&b)[E])
{
#pragma unroll
    for (int i = 0; i < E; i += 2) set(&d[i], __fmul2_rn(two(&a[i]), two(&b[i])));
}
template <int E> __device__ __forceinline__ void mul_row(float (&d)[E], const float (&a)[E], float b)
{
#pragma unroll
    for (int i = 0; i < E; i += 2) set(&d[i], __fmul2_rn(two(&a[i]), make_float2(b, b)));
}
template <int E> __device__ __forceinline__ void add_row(float (&d)[E], const float (&a)[E], const float (&b)[E])
{
#pragma unroll
    for (int i = 0; i < E; i += 2) set(&d[i], __fadd2_rn(two(&a[i]), two(&b[i])));
}
template <int E> __device__ __forceinline__ void add_row(float (&d)[E], const float (&a)[E], float b)
{
#pragma unroll
    for (int i = 0; i < E; i += 2) set(&d[i], __fadd2_rn(two(&a[i]), make_float2(b, b)));
}
template <int E> __device__ __forceinline__ float sum_row(const float (&a)[E])
{
    float2 s = two(&a[0]);
#pragma unroll
    for (int i = 2; i < E; i += 2) s = __fadd2_rn(s, two(&a[i]));
    return s.x + s.y;
}
template <int E> __device__ __forceinline__ float dot_row(const float (&a)[E], const float (&b)[E])
{
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < E; i += 2) s = __ffma2_rn(two(&a[i]), two(&b[i]), s);
    return s.x + s.y;
}

// Sums over the block of a value a thread, in a fixed order; the two halves of
// `part` are used in turn, so that one barrier is enough.  After it
// every thread adds the warps' sums itself: a second round of shuffles would
// take twice as long.
struct Reducer {
    float (*part)[32];
    u32 turn, warps;
    __device__ __forceinline__ static float warps_sum(const float *p, u32 warps)
    {
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (u32 i = 0; i < 32; i += 4) {
            if (i >= warps) break;
            const float4 w = *reinterpret_cast<const float4 *>(p + i);
            s = __fadd2_rn(s, __fadd2_rn(make_float2(w.x, w.y), make_float2(w.z, w.w)));
        }
        return s.x + s.y;
    }
    __device__ __forceinline__ void start()         // warps that are not there add nothing
    {
        if (threadIdx.x < 32)
            for (u32 i = threadIdx.x; i < 64; i += 32) part[0][i] = 0.0f;
        __syncthreads();
    }
    __device__ __forceinline__ float operator()(float a)
    {
        a = group_sum<32>(a);
        if (warps == 1) return a;
        if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = a;
        __syncthreads();
        const float s = warps_sum(part[turn], warps);
        turn ^= 1;
        return s;
    }
};

// v becomes N(v) without its parameters.  The deviation is taken from the differences to the mean, so a mean
// far from 0 costs it nothing.
template <int N, bool WHOLE, int E> __device__ __forceinline__ void normalise(const NormArgs &a, bool layer, Reducer &sum, float (&v)[E], u32 threads)
{
    hide<N, WHOLE>(a.hidden, threads, v);
    if (layer) {
        add_row(v, v, -(sum(sum_row(v)) * a.inv_hidden));
        hide<N, WHOLE>(a.hidden, threads, v);
    }
    // divided before they are added up: the sum of a long row's squares may be beyond 32 bits where their mean is not
    const float inverse = rsqrtf(sum(dot_row(v, v) * a.inv_hidden) + a.eps);
    mul_row(v, v, inverse);
}

constexpr u32 kMostThreads = MV_NORM_MAX_HIDDEN / 32;   // a block: 32 elements a thread where rows are longest

// The backward pass: threads a block where each has 96 registers, and where it has 72 (beyond: 64).
template <bool FEW> constexpr int kGradThreads = FEW ? 640 : 896;

}  // namespace mvblock
