// Gradients of the norms around a residual (mv_norm_backward in include/mv.h);
// a translation unit a type, as each takes a while to compile.
//
// With G = dr + the gradient through N(r), whose g = dn weight:
//   N'(x): (g - mean(g x^) x^ - [layer] mean(g)) / deviation, x^ = N(x)
//   dresidual = alpha G, dgate = sum G u, du = gate G, dpost = sum du y^,
//   dpost_bias = sum du, dy = N'(y) of du post, dweight = sum dn r^, dbias = sum dn.
// A block takes a run of rows and adds up its columns' sums in registers.  The
// statistics are computed again from y and the residual, which costs no bytes.
// A row is a chain of four sums over the block, so two rows go through it
// together: half the barriers, and parameters are read once for both.  The next
// rows are copied to shared memory meanwhile, every thread its own pieces, so
// that nothing waits for another's: each array as soon as its last use is over,
// y, which is used to the end, in two buffers.
//
// 16384 x 7168 bfloat16 with both norms, residual and gate (1.41 GB): 373 us, 3.8
// TB/s, and 16384 x 7168 with one norm 226 us, 6.2 TB/s.  What bounds the first is
// instructions (57 an element) that issue at half rate, 28 warps an SM being what
// 72 registers leave, with 100 bytes of a thread's spilled (300 with biases); barriers are not it (a chain of two sums a row instead of
// four took 557 us: more is computed).  Steps on the way: 689 us; arithmetic by
// pairs, sixteen elements a thread 434; two rows at a time, 32-bit row numbers 378.
// 16384 x 5120 with biases and gates (layer): 451 us, so 218.  4099 x 1437 in 32 bits,
// rows on no 16-byte boundary: 80 us, so 51; element by element, and its blocks' sums
// (6.7 MB) added by a second kernel.
#pragma once

#include "mv_norm.cuh"

namespace mvblock {

// R rows at a time; E elements a thread; MOST threads a block.
template <class T, class P, int N, int E, int R, bool POST, bool BIAS, int MOST>
__global__ void __launch_bounds__(MOST, 1) k_norm_grad(const NormArgs a)
{
    // pieces of 2 bytes cannot be copied, and the longest rows do not fit: they are read where they are used
    constexpr bool staged = N * sizeof(T) >= 4 && E == 8;
    constexpr u32 kBytes = N * sizeof(T), kPieces = E / N;        // in five places: y twice, residual, dn, dr
    extern __shared__ __align__(16) unsigned char stage[];
    __shared__ float2 part[2][R][32];
    const u32 threads = blockDim.x, tid = threadIdx.x, hidden = a.hidden;
    const bool layer = BIAS && a.layer, post = POST && a.post, gated = POST && a.gate;
    // pieces of this thread; a piece beyond the row is taken from its start, and counts for nothing
    const bool ragged = threads * E != hidden;
    bool within[kPieces];
    u32 column[kPieces];
#pragma unroll
    for (u32 i = 0; i < kPieces; i++) {
        column[i] = (i * threads + tid) * N;
        within[i] = column[i] < hidden;
        if (!within[i]) column[i] = 0;
    }
    const u32 first = blockIdx.x * (u32)a.rows, last = (u32)min((u64)first + a.rows, a.tokens), run = (u32)a.run;
    // Rows that go together share their gate; a second one that is not there is the first again, and counts for nothing.
    u32 gate = gated ? first / run : 0;
    u64 gate_end = gated ? (u64)(gate + 1) * run : ~0ull;
    auto end_of = [&](u32 t) {
        u32 end = min(t + R, last);
        if (gated) end = (u32)min((u64)end, t < gate_end ? gate_end : gate_end + run);
        return end;
    };
    const void *const from[4] = {a.y, a.residual, a.dn, a.dr};
    auto row_of = [&](int k, u32 row) {
        const u64 stride = k == 0 ? a.y_stride : k == 1 ? a.residual_stride : k == 2 ? a.dn_stride : a.dr_stride;
        return static_cast<const T *>(from[k]) + row * stride;
    };
    const u32 stage_at = (u32)__cvta_generic_to_shared(stage) + tid * kBytes, piece_bytes = threads * kBytes;
    auto fetch = [&](int k, u32 t, u32 end, u32 slot) {
        if constexpr (staged) {
            if (from[k] && t < last) {
#pragma unroll
                for (int r = 0; r < R; r++) {
                    const T *row = row_of(k, r ? end - 1 : t);
#pragma unroll
                    for (u32 i = 0; i < kPieces; i++) {
                        const u32 to = stage_at + ((slot * R + r) * kPieces + i) * piece_bytes;
                        if constexpr (kBytes == 16)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(row + column[i]) : "memory");
                        else
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(row + column[i]) : "memory");
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    auto load = [&](int k, u32 t, u32 end, int r, u32 slot, float (&v)[E]) {
        if constexpr (staged) {
#pragma unroll
            for (u32 i = 0; i < kPieces; i++) {
                const u32 at = stage_at + ((slot * R + r) * kPieces + i) * piece_bytes;
                if constexpr (kBytes == 16) {
                    uint4 w;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at));
                    widen_piece<T, N>(w, &v[i * N]);
                } else {
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[i]) : "r"(at));
                }
            }
        } else {
            const T *row = row_of(k, r ? end - 1 : t);
#pragma unroll
            for (u32 i = 0; i < kPieces; i++) get<T, N>(row + column[i], &v[i * N]);
        }
    };
    auto param = [&](const void *p, float (&v)[E]) {
#pragma unroll
        for (u32 i = 0; i < kPieces; i++) get<P, N>(static_cast<const P *>(p) + column[i], &v[i * N]);
    };
    auto store = [&](void *p, u32 t, const float (&v)[E]) {
        T *row = static_cast<T *>(p) + (u64)t * hidden;
#pragma unroll
        for (u32 i = 0; i < kPieces; i++)
            if (within[i]) put<T, N>(row + column[i], &v[i * N]);
    };
    auto store_sums = [&](float *p, const float (&v)[E]) {
#pragma unroll
        for (u32 i = 0; i < kPieces; i++)
            if (within[i]) put<float, N>(p + column[i], &v[i * N]);
    };
    auto hide = [&](float (&v)[E]) {                          // what lies beyond the row
        if (!ragged) return;
#pragma unroll
        for (u32 i = 0; i < kPieces; i++)
            if (!within[i])
#pragma unroll
                for (int j = 0; j < N; j++) v[i * N + j] = 0.0f;
    };
    // Sums over the block of a value of each of R rows; or of two.
    const u32 warps = threads / 32, lane = tid & 31;
    u32 turn = 0;
    auto sums2 = [&](float2 (&s)[R]) {
        float mine[R];
        const bool upper = lane & 16;
#pragma unroll
        for (int r = 0; r < R; r++) {                         // the first exchange leaves x to the lower half-warp, y to the upper
            mine[r] = (upper ? s[r].y : s[r].x) + __shfl_xor_sync(kFull, upper ? s[r].x : s[r].y, 16);
            mine[r] = group_sum<16>(mine[r]);
        }
        if (warps > 1) {
            if ((lane & 15) == 0)
#pragma unroll
                for (int r = 0; r < R; r++) (upper ? part[turn][r][tid >> 5].y : part[turn][r][tid >> 5].x) = mine[r];
            __syncthreads();
#pragma unroll
            for (int r = 0; r < R; r++) {
                const float2 w = lane < warps ? part[turn][r][lane] : make_float2(0.0f, 0.0f);
                mine[r] = (upper ? w.y : w.x) + __shfl_xor_sync(kFull, upper ? w.x : w.y, 16);
                mine[r] = group_sum<16>(mine[r]);
            }
            turn ^= 1;
        }
#pragma unroll
        for (int r = 0; r < R; r++) s[r] = make_float2(__shfl_sync(kFull, mine[r], 0), __shfl_sync(kFull, mine[r], 16));
    };
    auto sums = [&](float (&s)[R]) {
        if constexpr (R == 2) {                               // two rows' values as one row's two
            const bool upper = lane & 16;
            float mine = (upper ? s[1] : s[0]) + __shfl_xor_sync(kFull, upper ? s[0] : s[1], 16);
            mine = group_sum<16>(mine);
            if (warps > 1) {
                if ((lane & 15) == 0) (upper ? part[turn][0][tid >> 5].y : part[turn][0][tid >> 5].x) = mine;
                __syncthreads();
                const float2 w = lane < warps ? part[turn][0][lane] : make_float2(0.0f, 0.0f);
                mine = (upper ? w.y : w.x) + __shfl_xor_sync(kFull, upper ? w.x : w.y, 16);
                mine = group_sum<16>(mine);
                turn ^= 1;
            }
            s[0] = __shfl_sync(kFull, mine, 0);
            s[1] = __shfl_sync(kFull, mine, 16);
        } else {
            float mine = group_sum<32>(s[0]);
            if (warps > 1) {
                if (lane == 0) part[turn][0][tid >> 5].x = mine;
                __syncthreads();
                mine = group_sum<32>(lane < warps ? part[turn][0][lane].x : 0.0f);
                turn ^= 1;
            }
            s[0] = mine;
        }
    };
    // v becomes N(v) of every row; means and what they were divided by, inverted
    auto normalise = [&](float (&v)[R][E], float (&mean)[R], float (&inverse)[R]) {
        float s[R];
#pragma unroll
        for (int r = 0; r < R; r++) mean[r] = 0.0f;
        if (layer) {
#pragma unroll
            for (int r = 0; r < R; r++) { hide(v[r]); s[r] = sum_row(v[r]); }
            sums(s);
#pragma unroll
            for (int r = 0; r < R; r++) { mean[r] = s[r] * a.inv_hidden; add_row(v[r], v[r], -mean[r]); }
        }
#pragma unroll
        for (int r = 0; r < R; r++) { hide(v[r]); s[r] = dot_row(v[r], v[r]) * a.inv_hidden; }
        sums(s);
#pragma unroll
        for (int r = 0; r < R; r++) { inverse[r] = rsqrtf(s[r] + a.eps); mul_row(v[r], v[r], inverse[r]); }
    };
    // means of g and of g x^, of every row
    auto slopes = [&](const float (&g)[R][E], const float (&x)[R][E], float (&mean)[R], float (&slope)[R]) {
        if (layer) {
            float2 s[R];
#pragma unroll
            for (int r = 0; r < R; r++) s[r] = make_float2(sum_row(g[r]), dot_row(g[r], x[r]));
            sums2(s);
#pragma unroll
            for (int r = 0; r < R; r++) { mean[r] = s[r].x * a.inv_hidden; slope[r] = s[r].y * a.inv_hidden; }
        } else {
#pragma unroll
            for (int r = 0; r < R; r++) slope[r] = dot_row(g[r], x[r]);
            sums(slope);
#pragma unroll
            for (int r = 0; r < R; r++) { mean[r] = 0.0f; slope[r] *= a.inv_hidden; }
        }
    };

    // the sums: of weight, bias, post, post_bias, gate
    float dw[E] = {}, db[BIAS ? E : 2] = {}, dp[POST ? E : 2] = {}, dpb[POST && BIAS ? E : 2] = {}, dg[POST ? E : 2] = {};
    // A gate whose rows are all this block's is done with them; of another the block has a
    // part, in one of two places: its first gate's, or another's, which goes on after it.
    auto store_gate = [&] {
        if constexpr (POST) {
            if ((u64)gate * run >= first && gate_end <= last) {
                P *to = static_cast<P *>(a.dgate) + (u64)gate * hidden;
#pragma unroll
                for (u32 i = 0; i < kPieces; i++)
                    if (within[i]) put<P, N>(to + column[i], &dg[i * N]);
            } else {
                store_sums(a.gate_sums + (blockIdx.x * 2ull + (gate != first / run)) * a.pitch, dg);
            }
        }
    };
    u32 buffer = 0;
    u32 end = end_of(first);
    fetch(0, first, end, 0);
    fetch(1, first, end, 2);
    fetch(2, first, end, 3);
    fetch(3, first, end, 4);
    for (u32 t = first; t < last; buffer ^= 1) {
        if constexpr (POST) {
            if (t == gate_end) {
                store_gate();
                gate++;
                gate_end += run;
#pragma unroll
                for (int i = 0; i < E; i++) dg[i] = 0.0f;
            }
        }
        const u32 next = end, next_end = end_of(next);
        const bool lone = R == 2 && end - t < 2;              // only the first of two rows counts
        const P *const gate_row = POST ? static_cast<const P *>(a.gate) + (u64)gate * hidden : nullptr;
        fetch(0, next, next_end, buffer ^ 1);
        float v[R][E], w[E], mean[R], inverse[R], my[R], iy[R], slope[R];
        if constexpr (staged) asm volatile("cp.async.wait_group 4;" ::: "memory");
#pragma unroll
        for (int r = 0; r < R; r++) load(0, t, end, r, buffer, v[r]);
        // as in the forward pass
        if (post) {
            normalise(v, my, iy);
            param(a.post, w);
#pragma unroll
            for (int r = 0; r < R; r++) mul_row(v[r], v[r], w);
            if constexpr (BIAS) {
                if (a.post_bias) {
                    param(a.post_bias, w);
#pragma unroll
                    for (int r = 0; r < R; r++) add_row(v[r], v[r], w);
                }
            }
        }
        if (gated) {
            param(gate_row, w);
#pragma unroll
            for (int r = 0; r < R; r++) mul_row(v[r], v[r], w);
        }
        if constexpr (staged) asm volatile("cp.async.wait_group 3;" ::: "memory");
        if (from[1])
#pragma unroll
            for (int r = 0; r < R; r++) {
                load(1, t, end, r, 2, w);
                fma_row(v[r], w, a.alpha, v[r]);
            }
        fetch(1, next, next_end, 2);
        normalise(v, mean, inverse);
        if constexpr (staged) asm volatile("cp.async.wait_group 3;" ::: "memory");
        float g[R][E];
#pragma unroll
        for (int r = 0; r < R; r++) load(2, t, end, r, 3, g[r]);
        fetch(2, next, next_end, 3);
        if (R == 2 && lone)
#pragma unroll
            for (int i = 0; i < E; i++) g[R - 1][i] = 0.0f;
        param(a.weight, w);
#pragma unroll
        for (int r = 0; r < R; r++) {
            fma_row(dw, g[r], v[r], dw);
            if constexpr (BIAS) add_row(db, g[r], db);
            mul_row(g[r], g[r], w);
            hide(g[r]);
        }
        slopes(g, v, mean, slope);
        if constexpr (staged) asm volatile("cp.async.wait_group 3;" ::: "memory");
#pragma unroll
        for (int r = 0; r < R; r++) {
            fma_row(v[r], v[r], -slope[r], g[r]);
            if (layer) add_row(v[r], v[r], -mean[r]);
            if (from[3]) {
                load(3, t, end, r, 4, w);
                fma_row(v[r], v[r], inverse[r], w);
            } else {
                mul_row(v[r], v[r], inverse[r]);
            }
            if (R == 2 && r && lone)
#pragma unroll
                for (int i = 0; i < E; i++) v[r][i] = 0.0f;
            if (a.dresidual) {
                mul_row(w, v[r], a.alpha);
                if (!(R == 2 && r && lone)) store(a.dresidual, t + r, w);
            }
        }
        fetch(3, next, next_end, 4);
        if constexpr (POST) {
#pragma unroll
            for (int r = 0; r < R; r++) {
                load(0, t, end, r, buffer, g[r]);
                if (post) {
                    if (layer) add_row(g[r], g[r], -my[r]);
                    mul_row(g[r], g[r], iy[r]);               // y^
                }
            }
            if (gated) {
                float u[E];
                if (post) param(a.post, w);
#pragma unroll
                for (int r = 0; r < R; r++) {
                    if (post) {
                        mul_row(u, g[r], w);
                        if constexpr (BIAS) {
                            if (a.post_bias) {
                                float b[E];
                                param(a.post_bias, b);
                                add_row(u, u, b);
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < E; i++) u[i] = g[r][i];
                    }
                    fma_row(dg, u, v[r], dg);
                }
                param(gate_row, w);
#pragma unroll
                for (int r = 0; r < R; r++) mul_row(v[r], v[r], w);
            }
            if (post) {
                param(a.post, w);
#pragma unroll
                for (int r = 0; r < R; r++) {
                    fma_row(dp, v[r], g[r], dp);
                    if constexpr (BIAS) add_row(dpb, dpb, v[r]);
                    mul_row(v[r], v[r], w);
                    hide(v[r]);
                }
                slopes(v, g, mean, slope);
#pragma unroll
                for (int r = 0; r < R; r++) {
                    fma_row(v[r], g[r], -slope[r], v[r]);
                    if (layer) add_row(v[r], v[r], -mean[r]);
                    mul_row(v[r], v[r], iy[r]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; r++)
            if (!(R == 2 && r && lone)) store(a.dy, t + r, v[r]);
        t = next;
        end = next_end;
    }
    if constexpr (staged) asm volatile("cp.async.wait_group 0;" ::: "memory");
    float *to = a.sums + (u64)blockIdx.x * 4 * a.pitch;
    store_sums(to, dw);
    if constexpr (BIAS) store_sums(to + a.pitch, db);
    if constexpr (POST) {
        store_sums(to + 2 * a.pitch, dp);
        if (gated) store_gate();
    }
    if constexpr (POST && BIAS) store_sums(to + 3 * a.pitch, dpb);
}

template <class T, class P, int N, int E, int R, bool POST, bool BIAS, int MOST>
int run_grad(const NormArgs &a, const NormShape &s, u64 blocks, u32 smem, cudaStream_t stream)
{
    const auto kernel = k_norm_grad<T, P, N, E, R, POST, BIAS, MOST>;
    if (smem > 32 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return MV_ECUDA;
    return launch(kernel, dim3((u32)blocks), s.threads, smem, stream, a);
}
// Fewer threads leave more registers to each, which the kernels with the most
// sums need.  Rarer rows (longest, of 32 bits and long, or on no 16-byte boundary)
// have kernels with more sums than they may need.  Blocks of 1024 threads have 64 registers
// each: with post 400 to 500 bytes of a thread's are spilled, and 800 of rows beyond 8192.
// 4096 x 8192 bfloat16 with both norms (403 MB) 206 us, 2.0 TB/s; 4096 x 16384 562 us, 1.4 TB/s.
template <class T, class P, int N, int R, int MOST>
int run_grad(const NormArgs &a, const NormShape &s, u64 blocks, u32 smem, bool post, bool bias, cudaStream_t stream)
{
    constexpr int kMany = kGradThreads<false>, kPlain = N > 1 && MOST < kMany ? kMany : MOST;       // without post: as many threads as may be
    if constexpr (N > 1 && R == 2 && MOST <= kMany)
        if (!bias) return post ? run_grad<T, P, N, 8, R, true, false, MOST>(a, s, blocks, smem, stream)
                               : run_grad<T, P, N, 8, R, false, false, kPlain>(a, s, blocks, smem, stream);
    return post ? run_grad<T, P, N, 8, R, true, true, MOST>(a, s, blocks, smem, stream)
                : run_grad<T, P, N, 8, R, false, true, kPlain>(a, s, blocks, smem, stream);
}
template <class T, class P, int N> int run_grad(const NormArgs &a, const NormShape &s, u64 blocks, u32 smem, bool post, bool bias, cudaStream_t stream)
{
    constexpr int kFew = kGradThreads<true>, kMany = kGradThreads<false>;
    if (s.pieces * s.n == 16) return run_grad<T, P, N, 16, 1, true, true, 1024>(a, s, blocks, smem, stream);
    if constexpr (sizeof(T) == 4)           // two rows at a time do not fit where they are long
        if (s.at_once == 1)
            return s.threads <= kMany ? run_grad<T, P, N, 1, kMany>(a, s, blocks, smem, post, bias, stream)
                                      : run_grad<T, P, N, 1, 1024>(a, s, blocks, smem, post, bias, stream);
    if (s.threads <= kFew) return run_grad<T, P, N, 2, kFew>(a, s, blocks, smem, post, bias, stream);
    return s.threads <= kMany ? run_grad<T, P, N, 2, kMany>(a, s, blocks, smem, post, bias, stream)
                              : run_grad<T, P, N, 2, 1024>(a, s, blocks, smem, post, bias, stream);
}
template <class T, class P> int run_grad(const NormArgs &a, const NormShape &s, u64 blocks, u32 smem, bool post, bool bias, cudaStream_t stream)
{
    return s.n > 1 ? run_grad<T, P, 16 / (int)sizeof(T)>(a, s, blocks, smem, post, bias, stream) : run_grad<T, P, 1>(a, s, blocks, smem, post, bias, stream);
}

template <class T> int run_norm_grad(const NormArgs &a, const NormShape &s, u64 blocks, u32 smem, bool post, bool bias, cudaStream_t stream)
{
    return a.params_f32 ? run_grad<T, float>(a, s, blocks, smem, post, bias, stream) : run_grad<T, T>(a, s, blocks, smem, post, bias, stream);
}

}  // namespace mvblock
