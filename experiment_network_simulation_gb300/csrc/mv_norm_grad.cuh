// Gradients of the norms around a residual (mv_norm_backward in include/mv.h);
// a translation unit a type, as each takes a while to compile.
//
// With G = dr + the gradient through N(r), whose g = dn weight:
//   N'(x): (g - mean(g x^) x^ - [layer] mean(g)) / deviation, x^ = N(x)
//   dresidual = alpha G, dgate = sum G u, du = gate G, dpost = sum du y^,
//   dpost_bias = sum du, dy = N'(y) of du post, dweight = sum dn r^, dbias = sum dn.
// A block takes a run of rows and adds up its columns' sums in registers.  The
// statistics are computed again from y and the residual, which costs no bytes.
// The next row is copied to shared memory while this one is worked on, every
// thread its own pieces, so that nothing waits for another's.
#pragma once

#include "mv_norm.cuh"

namespace mvblock {

template <class T, class P, int N, int E, bool POST, bool BIAS>
__global__ void __launch_bounds__(kMostThreads) k_norm_grad(const NormArgs a)
{
    constexpr bool kCanStage = N * sizeof(T) >= 4;
    constexpr u32 kBytes = N * sizeof(T), kPieces = E / N;
    extern __shared__ __align__(16) unsigned char stage[];
    __shared__ float2 part[2][32];
    const u32 threads = blockDim.x, tid = threadIdx.x, hidden = a.hidden;
    const bool layer = BIAS && a.layer, post = POST && a.post, gated = POST && a.gate, staged = kCanStage && a.staged;
    Reducer sum = {part, 0, threads / 32};
    const u64 first = blockIdx.x * a.rows, last = min(first + a.rows, a.tokens);
    const T *const from[4] = {static_cast<const T *>(a.y), static_cast<const T *>(a.residual), static_cast<const T *>(a.dn),
                              static_cast<const T *>(a.dr)};
    const u64 strides[4] = {a.y_stride, a.residual_stride, a.dn_stride, a.dr_stride};
    const u32 stage_at = (u32)__cvta_generic_to_shared(stage) + tid * kBytes, piece_bytes = threads * kBytes;
    auto fetch = [&](u64 t, u32 buffer) {
        if constexpr (kCanStage) {
            if (t < last) {
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    if (!from[k]) continue;
                    const T *row = from[k] + t * strides[k];
#pragma unroll
                    for (u32 i = 0; i < kPieces; i++) {
                        const u32 c = (i * threads + tid) * N;
                        const u32 to = stage_at + ((buffer * 4 + k) * kPieces + i) * piece_bytes;
                        if (c < hidden) {
                            if constexpr (kBytes == 16)
                                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(row + c) : "memory");
                            else
                                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(row + c) : "memory");
                        }
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    u64 t = first;
    u32 buffer = 0;
    auto load = [&](int k, float (&v)[E]) {
        if (staged) {
#pragma unroll
            for (u32 i = 0; i < kPieces; i++) {
                const u32 at = stage_at + ((buffer * 4 + k) * kPieces + i) * piece_bytes;
                if constexpr (kBytes == 16) {
                    uint4 w;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at));
                    widen_piece<T, N>(w, &v[i * N]);
                } else {
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[i]) : "r"(at));
                }
            }
        } else {
            get_row<T, N>(from[k] + t * strides[k], hidden, threads, v);
        }
    };
    auto param = [&](const void *p, float (&v)[E]) { get_row<P, N>(static_cast<const P *>(p), hidden, threads, v); };
    if (staged)                             // beyond the row nothing is ever copied
        for (u32 i = 0; i < 8 * kPieces; i++) {
            if constexpr (kBytes == 16) asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(stage_at + i * piece_bytes), "r"(0u) : "memory");
            else asm volatile("st.shared.b32 [%0], %1;" ::"r"(stage_at + i * piece_bytes), "r"(0u) : "memory");
        }
    // the sums: of weight, bias, post, post_bias, gate
    float dw[E] = {}, db[BIAS ? E : 2] = {}, dp[POST ? E : 2] = {}, dpb[POST && BIAS ? E : 2] = {}, dg[POST ? E : 2] = {};
    u64 gate = gated ? first / a.run : 0, gate_end = gated ? (gate + 1) * a.run : ~0ull;
    if (staged) fetch(first, 0);
    for (; t < last; t++, buffer ^= 1) {
        if (staged) {
            fetch(t + 1, buffer ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        }
        if constexpr (POST) {
            if (t == gate_end) {
                if (!a.dgate) put_row<float, N>(a.gate_sums + (blockIdx.x + gate) * a.pitch, hidden, threads, dg);
                gate++;
                gate_end += a.run;
#pragma unroll
                for (int i = 0; i < E; i++) dg[i] = 0.0f;
            }
        }
        const P *gates = static_cast<const P *>(a.gate) + gate * hidden;
        float v[E], w[E], g[E];
        load(0, v);
        // as in the forward pass; y's norm is gone back to by its mean and deviation
        float2 my = make_float2(0.0f, 1.0f);
        if (post) {
            my = normalise<N>(a, layer, sum, v, threads);
            param(a.post, w);
            mul_row(v, v, w);
            if constexpr (BIAS) {
                if (a.post_bias) {
                    param(a.post_bias, w);
                    add_row(v, v, w);
                }
            }
        }
        if (gated) {
            param(gates, w);
            mul_row(v, v, w);
        }
        if (from[1]) {
            load(1, w);
            fma_row(v, w, a.alpha, v);
        }
        const float inverse = normalise<N>(a, layer, sum, v, threads).y;
        load(2, g);
        fma_row(dw, g, v, dw);
        if constexpr (BIAS) add_row(db, g, db);
        param(a.weight, w);
        mul_row(g, g, w);
        float mean = 0.0f, slope;
        if (layer) {
            const float2 m = sum(sum_row(g), dot_row(g, v));
            mean = m.x * a.inv_hidden;
            slope = m.y * a.inv_hidden;
        } else {
            slope = sum(dot_row(g, v)) * a.inv_hidden;
        }
        fma_row(v, v, -slope, g);
        if (layer) add_row(v, v, -mean);
        if (from[3]) {
            load(3, w);
            fma_row(v, v, inverse, w);
        } else {
            mul_row(v, v, inverse);
        }
        if (a.dresidual) {
            mul_row(w, v, a.alpha);
            put_row<T, N>(static_cast<T *>(a.dresidual) + t * hidden, hidden, threads, w);
        }
        if constexpr (POST) {
            load(0, g);
            if (post) {
                if (layer) add_row(g, g, -my.x);
                mul_row(g, g, my.y);               // y^
                param(a.post, w);
            }
            if (gated) {
                float u[E];
                if (post) {
                    mul_row(u, g, w);
                    if constexpr (BIAS) {
                        if (a.post_bias) {
                            float b[E];
                            param(a.post_bias, b);
                            add_row(u, u, b);
                        }
                    }
                    if (a.dgate) mul_row(u, u, v);
                    else fma_row(dg, u, v, dg);
                } else {
                    if (a.dgate) mul_row(u, g, v);
                    else fma_row(dg, g, v, dg);
                }
                if (a.dgate) put_row<P, N>(static_cast<P *>(a.dgate) + gate * hidden, hidden, threads, u);
                param(gates, u);
                mul_row(v, v, u);
            }
            if (post) {
                fma_row(dp, v, g, dp);
                if constexpr (BIAS) add_row(dpb, dpb, v);
                mul_row(v, v, w);
                if (layer) {
                    const float2 m = sum(sum_row(v), dot_row(v, g));
                    mean = m.x * a.inv_hidden;
                    slope = m.y * a.inv_hidden;
                } else {
                    slope = sum(dot_row(v, g)) * a.inv_hidden;
                }
                fma_row(v, g, -slope, v);
                if (layer) add_row(v, v, -mean);
                mul_row(v, v, my.y);
            }
        }
        put_row<T, N>(static_cast<T *>(a.dy) + t * hidden, hidden, threads, v);
    }
    if (staged) asm volatile("cp.async.wait_group 0;" ::: "memory");
    float *to = a.sums + (u64)blockIdx.x * 4 * a.pitch;
    put_row<float, N>(to, hidden, threads, dw);
    if constexpr (BIAS) put_row<float, N>(to + a.pitch, hidden, threads, db);
    if constexpr (POST) {
        put_row<float, N>(to + 2 * a.pitch, hidden, threads, dp);
        if (gated && !a.dgate) put_row<float, N>(a.gate_sums + (blockIdx.x + gate) * a.pitch, hidden, threads, dg);
    }
    if constexpr (POST && BIAS) put_row<float, N>(to + 3 * a.pitch, hidden, threads, dpb);
}

template <class T, class P, int N, int E, bool POST, bool BIAS>
int run_grad(const NormArgs &a, const NormShape &s, u64 blocks, u32 smem, cudaStream_t stream)
{
    const auto kernel = k_norm_grad<T, P, N, E, POST, BIAS>;
    if (smem > 32 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return MV_ECUDA;
    return launch(kernel, dim3((u32)blocks), s.threads, smem, stream, a);
}
// Rows that are rare (longest, or on no 16-byte boundary) have the kernel with
// all the sums, as it is without work that is not there.
template <class T, class P, int N, int E>
int run_grad(const NormArgs &a, const NormShape &s, u64 blocks, u32 smem, bool post, bool bias, cudaStream_t stream)
{
    if constexpr (E == 32) {
        return run_grad<T, P, N, E, true, true>(a, s, blocks, smem, stream);
    } else {
        if constexpr (N > 1)
            if (!bias) return post ? run_grad<T, P, N, E, true, false>(a, s, blocks, smem, stream) : run_grad<T, P, N, E, false, false>(a, s, blocks, smem, stream);
        return post ? run_grad<T, P, N, E, true, true>(a, s, blocks, smem, stream) : run_grad<T, P, N, E, false, true>(a, s, blocks, smem, stream);
    }
}
template <class T, class P> int run_grad(const NormArgs &a, const NormShape &s, u64 blocks, u32 smem, bool post, bool bias, cudaStream_t stream)
{
    constexpr int N = 16 / sizeof(T);
    const u32 e = s.n * s.pieces;
    if (s.n > 1) {
        if (e == N) return run_grad<T, P, N, N>(a, s, blocks, smem, post, bias, stream);
        if (e == 16) return run_grad<T, P, N, 16>(a, s, blocks, smem, post, bias, stream);
        return run_grad<T, P, N, 32>(a, s, blocks, smem, post, bias, stream);
    }
    if (e == 4) return run_grad<T, P, 1, 4>(a, s, blocks, smem, post, bias, stream);
    if (e == 16) return run_grad<T, P, 1, 16>(a, s, blocks, smem, post, bias, stream);
    return run_grad<T, P, 1, 32>(a, s, blocks, smem, post, bias, stream);
}

template <class T> int run_norm_grad(const NormArgs &a, const NormShape &s, u64 blocks, u32 smem, bool post, bool bias, cudaStream_t stream)
{
    return a.params_f32 ? run_grad<T, float>(a, s, blocks, smem, post, bias, stream) : run_grad<T, T>(a, s, blocks, smem, post, bias, stream);
}

}  // namespace mvblock
