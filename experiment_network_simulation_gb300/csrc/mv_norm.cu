// Norms after one branch and before the next, with the branch's gate and the
// residual between them (mv_norm, mv_norm_backward in include/mv.h):
//   u = N(y) post + post_bias,   r = alpha residual + gate u,   n = N(r) weight + bias
// A block holds a row: it is read once, and the stream between the two norms is
// normed from its 32-bit values.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "mv_block.cuh"

namespace mvblock {

struct NormArgs {
    const void *y, *residual, *dn, *dr;
    const void *weight, *bias, *post, *post_bias, *gate;
    void *n, *r, *dy, *dresidual, *dgate;           // dgate: where every token has a gate of its own
    u64 tokens, y_stride, residual_stride, dn_stride, dr_stride;
    u64 run, rows;                                  // tokens that share a gate; rows a block (backward)
    u32 hidden, layer, params_f32, staged;
    float alpha, eps, inv_hidden;
    float *sums;                                    // a block's sums for weight, bias, post, post_bias  [blocks, 4, hidden]
    float *gate_sums;                               // and for the gates of its rows                     [blocks + gates, hidden]
};

// ---- pieces of a row --------------------------------------------------------
// A thread's elements: PIECES pieces of N neighbours, threads next to each
// other; N = 1 where rows lie on no 16-byte boundary.
template <class T, int N> __device__ __forceinline__ void get(const T *p, float (&v)[N])
{
    if constexpr (N == 1) {
        v[0] = to_float(*p);
    } else {
        constexpr int kWords = N * sizeof(T) / 16;
        uint4 w[kWords];
        T t[N];
#pragma unroll
        for (int i = 0; i < kWords; i++) w[i] = reinterpret_cast<const uint4 *>(p)[i];
        memcpy(t, w, sizeof w);
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = to_float(t[i]);
    }
}
template <class T, int N> __device__ __forceinline__ void put(T *p, const float (&v)[N])
{
    if constexpr (N == 1) {
        *p = from_float<T>(v[0]);
    } else {
        constexpr int kWords = N * sizeof(T) / 16;
        uint4 w[kWords];
        T t[N];
#pragma unroll
        for (int i = 0; i < N; i++) t[i] = from_float<T>(v[i]);
        memcpy(w, t, sizeof w);
#pragma unroll
        for (int i = 0; i < kWords; i++) reinterpret_cast<uint4 *>(p)[i] = w[i];
    }
}
template <class T, int N> __device__ __forceinline__ void get_param(const NormArgs &a, const void *p, u64 at, float (&v)[N])
{
    if constexpr (sizeof(T) != 4)
        if (!a.params_f32) return get<T, N>(static_cast<const T *>(p) + at, v);
    get<float, N>(static_cast<const float *>(p) + at, v);
}

// Sums over the block of up to two values a thread, in a fixed order; the
// two halves of `part` are used in turn, so that one barrier is enough.
struct Reducer {
    float2 (*part)[32];
    u32 turn, warps;
    __device__ __forceinline__ float2 operator()(float a, float b)
    {
        a = group_sum<32>(a);
        b = group_sum<32>(b);
        if (warps == 1) return make_float2(a, b);
        if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const u32 lane = threadIdx.x & 31;
        float2 v = lane < warps ? part[turn][lane] : make_float2(0.0f, 0.0f);
        turn ^= 1;
        return make_float2(group_sum<32>(v.x), group_sum<32>(v.y));
    }
    __device__ __forceinline__ float operator()(float a)
    {
        a = group_sum<32>(a);
        if (warps == 1) return a;
        if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5].x = a;
        __syncthreads();
        const u32 lane = threadIdx.x & 31;
        const float v = lane < warps ? part[turn][lane].x : 0.0f;
        turn ^= 1;
        return group_sum<32>(v);
    }
};

// (mean, 1 / deviation) of a row; values beyond it are 0.  The deviation comes
// from the differences to the mean, so a mean far from 0 costs it nothing.
template <int N, int PIECES>
__device__ __forceinline__ float2 moments(const NormArgs &a, Reducer &sum, const float (&v)[PIECES][N], u32 threads)
{
    float mean = 0.0f, s = 0.0f;
    if (a.layer) {
#pragma unroll
        for (int i = 0; i < PIECES; i++)
#pragma unroll
            for (int j = 0; j < N; j++) s += v[i][j];
        mean = sum(s) * a.inv_hidden;
        s = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < PIECES; i++)
        if ((i * threads + threadIdx.x) * N < a.hidden)
#pragma unroll
            for (int j = 0; j < N; j++) s = fmaf(v[i][j] - mean, v[i][j] - mean, s);
    return make_float2(mean, 1.0f / sqrtf(fmaf(sum(s), a.inv_hidden, a.eps)));
}

// Threads a block at most, by shape_of().
template <class T, int N, int PIECES> constexpr u32 kMostThreads = PIECES < (N > 1 ? 4 : 16) ? 512 : MV_NORM_MAX_HIDDEN / (N * PIECES);

// ---- forward ----------------------------------------------------------------
template <class T, int N, int PIECES> __global__ void __launch_bounds__(kMostThreads<T, N, PIECES>) k_norm(const NormArgs a)
{
    __shared__ float2 part[2][32];
    const u32 threads = blockDim.x;
    Reducer sum = {part, 0, threads / 32};
    for (u64 t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        float v[PIECES][N], res[PIECES][N];
        const T *y = static_cast<const T *>(a.y) + t * a.y_stride, *residual = static_cast<const T *>(a.residual) + t * a.residual_stride;
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
            const u32 c = (i * threads + threadIdx.x) * N;
#pragma unroll
            for (int j = 0; j < N; j++) v[i][j] = res[i][j] = 0.0f;
            if (c < a.hidden) {
                get<T, N>(y + c, v[i]);
                if (a.residual) get<T, N>(residual + c, res[i]);
            }
        }
        if (a.post) {
            const float2 m = moments<N, PIECES>(a, sum, v, threads);
#pragma unroll
            for (int i = 0; i < PIECES; i++) {
                const u32 c = (i * threads + threadIdx.x) * N;
                if (c >= a.hidden) continue;
                float w[N], b[N];
#pragma unroll
                for (int j = 0; j < N; j++) b[j] = 0.0f;
                get_param<T, N>(a, a.post, c, w);
                if (a.post_bias) get_param<T, N>(a, a.post_bias, c, b);
#pragma unroll
                for (int j = 0; j < N; j++) v[i][j] = fmaf((v[i][j] - m.x) * m.y, w[j], b[j]);
            }
        }
        const u64 gate_row = a.gate ? t / a.run * a.hidden : 0;
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
            const u32 c = (i * threads + threadIdx.x) * N;
            if (c >= a.hidden) continue;
            if (a.gate) {
                float g[N];
                get_param<T, N>(a, a.gate, gate_row + c, g);
#pragma unroll
                for (int j = 0; j < N; j++) v[i][j] *= g[j];
            }
            if (a.residual)
#pragma unroll
                for (int j = 0; j < N; j++) v[i][j] = fmaf(a.alpha, res[i][j], v[i][j]);
            if (a.r) put<T, N>(static_cast<T *>(a.r) + t * a.hidden + c, v[i]);
        }
        const float2 m = moments<N, PIECES>(a, sum, v, threads);
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
            const u32 c = (i * threads + threadIdx.x) * N;
            if (c >= a.hidden) continue;
            float w[N], b[N];
#pragma unroll
            for (int j = 0; j < N; j++) b[j] = 0.0f;
            get_param<T, N>(a, a.weight, c, w);
            if (a.bias) get_param<T, N>(a, a.bias, c, b);
#pragma unroll
            for (int j = 0; j < N; j++) w[j] = fmaf((v[i][j] - m.x) * m.y, w[j], b[j]);
            put<T, N>(static_cast<T *>(a.n) + t * a.hidden + c, w);
        }
    }
}

// ---- backward ---------------------------------------------------------------
// With G = dr + the gradient through N(r), whose g = dn weight:
//   N'(x): (g - mean(g x^) x^ - [layer] mean(g)) / deviation, x^ = N(x)
//   dresidual = alpha G, dgate = sum G u, du = gate G, dpost = sum du y^,
//   dpost_bias = sum du, dy = N'(y) of du post, dweight = sum dn r^, dbias = sum dn.
// A block takes a run of rows and adds up its columns' sums in registers.  The
// statistics are computed again from y and the residual, which costs no bytes.
// The next row is copied to shared memory while this one is worked on, every
// thread its own pieces, so that nothing waits for another's.
template <class T, int N, int PIECES, bool POST, bool BIAS>
__global__ void __launch_bounds__(kMostThreads<T, N, PIECES>) k_norm_grad(const NormArgs a)
{
    constexpr bool kCanStage = N * sizeof(T) >= 4;
    constexpr u32 kBytes = N * sizeof(T);
    extern __shared__ __align__(16) unsigned char stage[];
    __shared__ float2 part[2][32];
    const u32 threads = blockDim.x, tid = threadIdx.x;
    Reducer sum = {part, 0, threads / 32};
    const u64 first = blockIdx.x * a.rows, last = min(first + a.rows, a.tokens);
    const void *const from[4] = {a.y, a.residual, a.dn, a.dr};
    const u64 strides[4] = {a.y_stride, a.residual_stride, a.dn_stride, a.dr_stride};
    const u32 stage_at = (u32)__cvta_generic_to_shared(stage);
    auto fetch = [&](u64 t, u32 buffer) {
        if constexpr (kCanStage) {
            if (t < last)
#pragma unroll
                for (int k = 0; k < 4; k++)
                    if (from[k])
#pragma unroll
                        for (int i = 0; i < PIECES; i++) {
                            const u32 c = (i * threads + tid) * N;
                            if (c >= a.hidden) continue;
                            const u32 to = stage_at + (((buffer * 4 + k) * PIECES + i) * threads + tid) * kBytes;
                            const T *p = static_cast<const T *>(from[k]) + t * strides[k] + c;
                            if constexpr (kBytes == 16)
                                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
                            else
                                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(p) : "memory");
                        }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
    auto piece = [&](u64 t, u32 buffer, int k, int i, float (&v)[N]) {
        const u32 c = (i * threads + tid) * N;
        if (kCanStage && a.staged)
            get<T, N>(reinterpret_cast<const T *>(stage + (((buffer * 4 + k) * PIECES + i) * threads + tid) * kBytes), v);
        else
            get<T, N>(static_cast<const T *>(from[k]) + t * strides[k] + c, v);
    };
    float dw[PIECES][N], db[BIAS ? PIECES : 1][N], dp[POST ? PIECES : 1][N], dpb[POST && BIAS ? PIECES : 1][N], dg[POST ? PIECES : 1][N];
#pragma unroll
    for (int i = 0; i < PIECES; i++)
#pragma unroll
        for (int j = 0; j < N; j++) {
            dw[i][j] = 0.0f;
            if constexpr (BIAS) db[i][j] = 0.0f;
            if constexpr (POST) dp[i][j] = dg[i][j] = 0.0f;
            if constexpr (POST && BIAS) dpb[i][j] = 0.0f;
        }
    auto store_gate = [&](u64 g) {
        if constexpr (POST) {
#pragma unroll
            for (int i = 0; i < PIECES; i++) {
                const u32 c = (i * threads + tid) * N;
                if (c >= a.hidden) continue;
                put<float, N>(a.gate_sums + (blockIdx.x + g) * a.hidden + c, dg[i]);
#pragma unroll
                for (int j = 0; j < N; j++) dg[i][j] = 0.0f;
            }
        }
    };
    if (a.staged) fetch(first, 0);
    u64 gate = POST && a.gate ? first / a.run : 0;
    u32 buffer = 0;
    for (u64 t = first; t < last; t++, buffer ^= 1) {
        if (a.staged) {
            fetch(t + 1, buffer ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        }
        if (POST && a.gate && !a.dgate && t / a.run != gate) {
            store_gate(gate);
            gate = t / a.run;
        }
        const u64 gate_row = POST && a.gate ? t / a.run * a.hidden : 0;
        float v[PIECES][N];
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
#pragma unroll
            for (int j = 0; j < N; j++) v[i][j] = 0.0f;
            if ((i * threads + tid) * N < a.hidden) piece(t, buffer, 0, i, v[i]);
        }
        float2 my = make_float2(0.0f, 1.0f);
        const bool post = POST && a.post;
        if (post) my = moments<N, PIECES>(a, sum, v, threads);
        // y of a piece, normed where it is, and the branch before its gate
        auto branch = [&](u32 c, float (&yn)[N], float (&u)[N]) {
#pragma unroll
            for (int j = 0; j < N; j++) u[j] = yn[j];
            if (post) {
                float w[N], b[N];
#pragma unroll
                for (int j = 0; j < N; j++) b[j] = 0.0f;
                get_param<T, N>(a, a.post, c, w);
                if (BIAS && a.post_bias) get_param<T, N>(a, a.post_bias, c, b);
#pragma unroll
                for (int j = 0; j < N; j++) {
                    yn[j] = (yn[j] - my.x) * my.y;
                    u[j] = fmaf(yn[j], w[j], b[j]);
                }
            }
        };
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
            const u32 c = (i * threads + tid) * N;
            if (c >= a.hidden) continue;
            float u[N];
            branch(c, v[i], u);
            if (POST && a.gate) {
                float g[N];
                get_param<T, N>(a, a.gate, gate_row + c, g);
#pragma unroll
                for (int j = 0; j < N; j++) u[j] *= g[j];
            }
            if (a.residual) {
                float s[N];
                piece(t, buffer, 1, i, s);
#pragma unroll
                for (int j = 0; j < N; j++) u[j] = fmaf(a.alpha, s[j], u[j]);
            }
#pragma unroll
            for (int j = 0; j < N; j++) v[i][j] = u[j];
        }
        const float2 mr = moments<N, PIECES>(a, sum, v, threads);
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
            const u32 c = (i * threads + tid) * N;
            if (c >= a.hidden) continue;
            float d[N], w[N];
            piece(t, buffer, 2, i, d);
            get_param<T, N>(a, a.weight, c, w);
#pragma unroll
            for (int j = 0; j < N; j++) {
                v[i][j] = (v[i][j] - mr.x) * mr.y;
                dw[i][j] = fmaf(d[j], v[i][j], dw[i][j]);
                if constexpr (BIAS) db[i][j] += d[j];
                const float g = d[j] * w[j];
                s0 += g;
                s1 = fmaf(g, v[i][j], s1);
            }
        }
        float2 m = sum(s0, s1);
        float mean = a.layer ? m.x * a.inv_hidden : 0.0f, slope = m.y * a.inv_hidden;
        s0 = s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
            const u32 c = (i * threads + tid) * N;
            if (c >= a.hidden) continue;
            float d[N], w[N], e[N];
            piece(t, buffer, 2, i, d);
            get_param<T, N>(a, a.weight, c, w);
#pragma unroll
            for (int j = 0; j < N; j++) e[j] = 0.0f;
            if (a.dr) piece(t, buffer, 3, i, e);
#pragma unroll
            for (int j = 0; j < N; j++) v[i][j] = fmaf(fmaf(-slope, v[i][j], fmaf(d[j], w[j], -mean)), mr.y, e[j]);
            if (a.dresidual) {
#pragma unroll
                for (int j = 0; j < N; j++) e[j] = a.alpha * v[i][j];
                put<T, N>(static_cast<T *>(a.dresidual) + t * a.hidden + c, e);
            }
            if constexpr (POST) {
                float yn[N], u[N];
                piece(t, buffer, 0, i, yn);
                branch(c, yn, u);
                if (a.gate) {
                    float g[N];
                    get_param<T, N>(a, a.gate, gate_row + c, g);
                    if (a.dgate) {
#pragma unroll
                        for (int j = 0; j < N; j++) u[j] *= v[i][j];
                        if (a.params_f32) put<float, N>(static_cast<float *>(a.dgate) + gate_row + c, u);
                        else put<T, N>(static_cast<T *>(a.dgate) + gate_row + c, u);
                    } else {
#pragma unroll
                        for (int j = 0; j < N; j++) dg[i][j] = fmaf(v[i][j], u[j], dg[i][j]);
                    }
#pragma unroll
                    for (int j = 0; j < N; j++) v[i][j] *= g[j];
                }
                if (post) {
                    get_param<T, N>(a, a.post, c, w);
#pragma unroll
                    for (int j = 0; j < N; j++) {
                        dp[i][j] = fmaf(v[i][j], yn[j], dp[i][j]);
                        if constexpr (BIAS) dpb[i][j] += v[i][j];
                        v[i][j] *= w[j];
                        s0 += v[i][j];
                        s1 = fmaf(v[i][j], yn[j], s1);
                    }
                }
            }
        }
        if (post) {
            m = sum(s0, s1);
            mean = a.layer ? m.x * a.inv_hidden : 0.0f;
            slope = m.y * a.inv_hidden;
        }
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
            const u32 c = (i * threads + tid) * N;
            if (c >= a.hidden) continue;
            if (post) {
                float yn[N];
                piece(t, buffer, 0, i, yn);
#pragma unroll
                for (int j = 0; j < N; j++) v[i][j] = (v[i][j] - mean - slope * ((yn[j] - my.x) * my.y)) * my.y;
            }
            put<T, N>(static_cast<T *>(a.dy) + t * a.hidden + c, v[i]);
        }
    }
    if (kCanStage && a.staged) asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (POST && a.gate && !a.dgate && first < last) store_gate(gate);
    float *to = a.sums + (u64)blockIdx.x * 4 * a.hidden;
#pragma unroll
    for (int i = 0; i < PIECES; i++) {
        const u32 c = (i * threads + tid) * N;
        if (c >= a.hidden) continue;
        put<float, N>(to + c, dw[i]);
        if constexpr (BIAS) put<float, N>(to + a.hidden + c, db[i]);
        if constexpr (POST) put<float, N>(to + 2 * a.hidden + c, dp[i]);
        if constexpr (POST && BIAS) put<float, N>(to + 3 * a.hidden + c, dpb[i]);
    }
}

// The blocks' sums, added in their order: 32 columns a block of threads, every
// warp the blocks w, w + 32, ..., then the warps'.
struct AddArgs {
    const float *sums, *gate_sums;
    void *to[4], *dgate;
    u64 hidden, blocks, run, rows, gates;
    u32 params_f32;
};
template <class T> __global__ void __launch_bounds__(1024) k_norm_add(const AddArgs a)
{
    __shared__ float part[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const u32 x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const u64 c = (u64)blockIdx.x * 32 + x;
    // what: four parameters, then the gates
    for (u64 what = blockIdx.y; what < 4 + a.gates; what += gridDim.y) {
        void *out = what < 4 ? a.to[what] : a.dgate;
        if (!out) continue;
        const float *from = a.sums + what * a.hidden;
        u64 pitch = 4 * a.hidden, first = 0, last = a.blocks, at = 0;
        if (what >= 4) {
            const u64 g = what - 4;
            first = g * a.run / a.rows;
            last = ((g + 1) * a.run - 1) / a.rows + 1;
            from = a.gate_sums + g * a.hidden;
            pitch = a.hidden;
            at = g * a.hidden;
        }
        float s = 0.0f;
        if (c < a.hidden)
#pragma unroll 4
            for (u64 b = first + y; b < last; b += 32) s += from[b * pitch + c];
        __syncthreads();
        part[y][x] = s;
        __syncthreads();
        s = group_sum<32>(part[x][y]);                       // column y of the block's 32
        const u64 mine = (u64)blockIdx.x * 32 + y;
        if (x == 0 && mine < a.hidden) {
            if (a.params_f32) static_cast<float *>(out)[at + mine] = s;
            else static_cast<T *>(out)[at + mine] = from_float<T>(s);
        }
    }
}

// ---- host ---------------------------------------------------------------
struct Shape {
    u32 n, pieces, threads;
};
// Few pieces a thread where the row is short, more where a block would pass 512 threads.
Shape shape_of(u32 hidden, u32 size, bool wide)
{
    const u32 n = wide ? 16 / size : 1;
    u32 pieces = wide ? 1 : 4;
    while (pieces < (wide ? 4u : 16u) && hidden > n * pieces * 512) pieces *= wide ? 2 : 4;
    const u32 threads = (hidden + n * pieces - 1) / (n * pieces);
    return {n, pieces, (threads + 31) / 32 * 32};
}

bool dense(const void *p, u64 stride, u32 n, u32 size) { return !p || (aligned(p, 16) && stride % n == 0 && (n * size == 16)); }

int check(const mv_norm_desc *d, bool grad)
{
    if (!d || !d->hidden || d->dtype > MV_BF16 || (d->param_dtype != d->dtype && d->param_dtype != MV_F32) ||
        d->kind > MV_NORM_LAYER || !std::isfinite(d->alpha) || !(d->eps >= 0.0f) || !std::isfinite(d->eps) ||
        (d->gate && (d->gates == 0 || d->tokens % d->gates)) || (d->post_bias && !d->post))
        return MV_EINVAL;
    if (d->hidden > MV_NORM_MAX_HIDDEN || d->tokens > 1ull << 31 || d->y_stride > 1ull << 31 || d->residual_stride > 1ull << 31)
        return MV_EOVERFLOW;
    const u64 size = dtype_size(d->dtype), param = dtype_size(d->param_dtype);
    if (d->y_stride < d->hidden || (d->residual && d->residual_stride < d->hidden) || !aligned(d->y, size) ||
        !aligned(d->residual, size) || !aligned(d->weight, param) || !aligned(d->bias, param) || !aligned(d->post, param) ||
        !aligned(d->post_bias, param) || !aligned(d->gate, param))
        return MV_EINVAL;
    if (d->tokens && (!d->y || !d->weight)) return MV_EINVAL;
    (void)grad;
    return MV_OK;
}

bool wide_row(const mv_norm_desc *d)
{
    const u32 size = (u32)dtype_size(d->dtype), n = 16 / size;
    return d->hidden % n == 0 && dense(d->y, d->y_stride, n, size) && dense(d->residual, d->residual_stride, n, size) &&
           aligned(d->weight, 16) && aligned(d->bias, 16) && aligned(d->post, 16) && aligned(d->post_bias, 16) && aligned(d->gate, 16);
}

NormArgs arguments(const mv_norm_desc *d)
{
    NormArgs a = {};
    a.y = d->y;
    a.residual = d->residual;
    a.weight = d->weight;
    a.bias = d->bias;
    a.post = d->post;
    a.post_bias = d->post_bias;
    a.gate = d->gate;
    a.tokens = d->tokens;
    a.y_stride = d->y_stride;
    a.residual_stride = d->residual_stride;
    a.run = d->gate ? d->tokens / d->gates : 1;
    a.hidden = (u32)d->hidden;
    a.layer = d->kind == MV_NORM_LAYER;
    a.params_f32 = d->param_dtype == MV_F32;
    a.alpha = d->alpha;
    a.eps = d->eps;
    a.inv_hidden = 1.0f / (float)d->hidden;
    return a;
}

template <class T> int run_norm(const NormArgs &a, const Shape &s, u32 sms, cudaStream_t stream)
{
    const u32 an_sm = std::max(1u, 1536 / s.threads);
    const dim3 grid((u32)std::min<u64>(a.tokens, (u64)sms * an_sm));
    constexpr int N = 16 / sizeof(T);
    if (s.n > 1) {
        if (s.pieces == 1) return launch(k_norm<T, N, 1>, grid, s.threads, 0, stream, a);
        if (s.pieces == 2) return launch(k_norm<T, N, 2>, grid, s.threads, 0, stream, a);
        return launch(k_norm<T, N, 4>, grid, s.threads, 0, stream, a);
    }
    if (s.pieces == 4) return launch(k_norm<T, 1, 4>, grid, s.threads, 0, stream, a);
    return launch(k_norm<T, 1, 16>, grid, s.threads, 0, stream, a);
}

struct GradPlan {
    Shape shape;
    bool staged, each;                  // each: every token has a gate of its own
    u32 smem;
    u64 blocks, rows, sums, gate_sums, total;
};
GradPlan grad_plan(const mv_norm_desc *d, bool wide)
{
    GradPlan p = {};
    const u32 size = (u32)dtype_size(d->dtype);
    p.shape = shape_of((u32)d->hidden, size, wide);
    const u32 smem = 2 * 4 * p.shape.pieces * p.shape.threads * p.shape.n * size;
    p.staged = p.shape.n * size >= 4 && smem <= 200 * 1024;
    p.smem = p.staged ? smem : 0;
    const u32 sms = std::max(1u, sm_count());
    const u32 an_sm = std::max(1u, std::min(512 / p.shape.threads, p.smem ? 220u * 1024 / (p.smem + 2048) : 16u));
    const u64 blocks = std::min<u64>((d->tokens + 3) / 4, (u64)sms * std::min(an_sm, 16u));
    p.rows = (d->tokens + blocks - 1) / blocks;
    p.blocks = (d->tokens + p.rows - 1) / p.rows;
    p.each = d->gate && d->gates == d->tokens;
    p.sums = 0;
    p.gate_sums = (p.blocks * 4 * d->hidden * 4 + 255) / 256 * 256;
    p.total = p.gate_sums + (d->gate && !p.each ? (p.blocks + d->gates) * d->hidden * 4 : 0);
    return p;
}

template <class T, int N, int PIECES, bool POST, bool BIAS> int run_grad(const NormArgs &a, const GradPlan &p, cudaStream_t stream)
{
    const auto kernel = k_norm_grad<T, N, PIECES, POST, BIAS>;
    if (p.smem > 32 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem) != cudaSuccess)
        return MV_ECUDA;
    return launch(kernel, dim3((u32)p.blocks), p.shape.threads, p.smem, stream, a);
}
template <class T, int N, int PIECES> int run_grad(const NormArgs &a, const GradPlan &p, bool post, bool bias, cudaStream_t stream)
{
    if (post) return bias ? run_grad<T, N, PIECES, true, true>(a, p, stream) : run_grad<T, N, PIECES, true, false>(a, p, stream);
    return bias ? run_grad<T, N, PIECES, false, true>(a, p, stream) : run_grad<T, N, PIECES, false, false>(a, p, stream);
}
template <class T> int run_grad(const NormArgs &a, const GradPlan &p, bool post, bool bias, const AddArgs &add, cudaStream_t stream)
{
    constexpr int N = 16 / sizeof(T);
    int rc;
    if (p.shape.n > 1) {
        rc = p.shape.pieces == 1 ? run_grad<T, N, 1>(a, p, post, bias, stream)
           : p.shape.pieces == 2 ? run_grad<T, N, 2>(a, p, post, bias, stream) : run_grad<T, N, 4>(a, p, post, bias, stream);
    } else {
        rc = p.shape.pieces == 4 ? run_grad<T, 1, 4>(a, p, post, bias, stream) : run_grad<T, 1, 16>(a, p, post, bias, stream);
    }
    if (rc != MV_OK) return rc;
    const dim3 grid((u32)((add.hidden + 31) / 32), (u32)std::min<u64>(4 + add.gates, 65535));
    return launch_after(k_norm_add<T>, grid, 1024, 0, stream, add);
}

}  // namespace mvblock

using namespace mvblock;

extern "C" int mv_norm(const mv_norm_desc *d, void *n, void *r, void *stream)
{
    const int rc = check(d, false);
    if (rc != MV_OK || d->tokens == 0) return rc;
    const u64 size = dtype_size(d->dtype);
    if (!n || !aligned(n, size) || !aligned(r, size)) return MV_EINVAL;
    const u32 sms = sm_count();
    if (!sms) return MV_ECUDA;
    NormArgs a = arguments(d);
    a.n = n;
    a.r = r;
    const Shape s = shape_of(a.hidden, (u32)size, wide_row(d) && aligned(n, 16) && aligned(r, 16));
    cudaStream_t on = static_cast<cudaStream_t>(stream);
    if (d->dtype == MV_F32) return run_norm<float>(a, s, sms, on);
    return d->dtype == MV_F16 ? run_norm<__half>(a, s, sms, on) : run_norm<__nv_bfloat16>(a, s, sms, on);
}

static int check_grad(const mv_norm_desc *d, const mv_norm_grads *g)
{
    const int rc = check(d, true);
    if (rc != MV_OK) return rc;
    if (!g) return MV_EINVAL;
    const u64 size = dtype_size(d->dtype), param = dtype_size(d->param_dtype);
    if ((d->tokens && (!g->dn || !g->dy || g->dn_stride < d->hidden || (g->dr && g->dr_stride < d->hidden))) || !g->dweight ||
        (d->bias != nullptr) != (g->dbias != nullptr) || (d->post != nullptr) != (g->dpost != nullptr) ||
        (d->post_bias != nullptr) != (g->dpost_bias != nullptr) || (d->gate != nullptr) != (g->dgate != nullptr) ||
        (d->tokens && (d->residual != nullptr) != (g->dresidual != nullptr)) || !aligned(g->dn, size) || !aligned(g->dr, size) ||
        !aligned(g->dy, size) || !aligned(g->dresidual, size) || !aligned(g->dweight, param) || !aligned(g->dbias, param) ||
        !aligned(g->dpost, param) || !aligned(g->dpost_bias, param) || !aligned(g->dgate, param))
        return MV_EINVAL;
    if (g->dn_stride > 1ull << 31 || g->dr_stride > 1ull << 31) return MV_EOVERFLOW;
    return MV_OK;
}
static bool wide_grad(const mv_norm_desc *d, const mv_norm_grads *g)
{
    const u32 size = (u32)dtype_size(d->dtype), n = 16 / size;
    return wide_row(d) && dense(g->dn, g->dn_stride, n, size) && dense(g->dr, g->dr_stride, n, size) && aligned(g->dy, 16) &&
           aligned(g->dresidual, 16) && aligned(g->dgate, 16);
}

extern "C" int mv_norm_backward_workspace_bytes(const mv_norm_desc *d, const mv_norm_grads *g, uint64_t *bytes)
{
    if (!bytes) return MV_EINVAL;
    *bytes = 0;
    const int rc = check_grad(d, g);
    if (rc != MV_OK || d->tokens == 0) return rc;
    *bytes = grad_plan(d, wide_grad(d, g)).total;
    return MV_OK;
}

extern "C" int mv_norm_backward(const mv_norm_desc *d, const mv_norm_grads *g, void *workspace, uint64_t ws_bytes, void *stream)
{
    const int rc = check_grad(d, g);
    if (rc != MV_OK) return rc;
    cudaStream_t on = static_cast<cudaStream_t>(stream);
    const u64 param = dtype_size(d->param_dtype);
    if (d->tokens == 0) {               // sums of nothing
        void *const to[5] = {g->dweight, g->dbias, g->dpost, g->dpost_bias, g->dgate};
        for (int i = 0; i < 5; i++)
            if (to[i] && cudaMemsetAsync(to[i], 0, param * d->hidden * (i == 4 ? d->gates : 1), on) != cudaSuccess) return MV_ECUDA;
        return MV_OK;
    }
    const GradPlan p = grad_plan(d, wide_grad(d, g));
    if (!workspace || !aligned(workspace, 256)) return MV_EINVAL;
    if (ws_bytes < p.total) return MV_ENOMEM;
    if (!sm_count()) return MV_ECUDA;
    char *ws = static_cast<char *>(workspace);
    NormArgs a = arguments(d);
    a.dn = g->dn;
    a.dr = g->dr;
    a.dn_stride = g->dn_stride;
    a.dr_stride = g->dr_stride;
    a.dy = g->dy;
    a.dresidual = g->dresidual;
    a.dgate = p.each ? g->dgate : nullptr;
    a.rows = p.rows;
    a.staged = p.staged;
    a.sums = reinterpret_cast<float *>(ws + p.sums);
    a.gate_sums = reinterpret_cast<float *>(ws + p.gate_sums);
    AddArgs add = {};
    add.sums = a.sums;
    add.gate_sums = a.gate_sums;
    add.to[0] = g->dweight;
    add.to[1] = g->dbias;
    add.to[2] = g->dpost;
    add.to[3] = g->dpost_bias;
    add.dgate = d->gate && !p.each ? g->dgate : nullptr;
    add.hidden = d->hidden;
    add.blocks = p.blocks;
    add.run = a.run;
    add.rows = p.rows;
    add.gates = add.dgate ? d->gates : 0;
    add.params_f32 = a.params_f32;
    const bool post = d->post || d->gate, bias = d->bias || d->post_bias;
    if (d->dtype == MV_F32) return run_grad<float>(a, p, post, bias, add, on);
    return d->dtype == MV_F16 ? run_grad<__half>(a, p, post, bias, add, on) : run_grad<__nv_bfloat16>(a, p, post, bias, add, on);
}
