// Norms after one branch and before the next, with the branch's gate and the
// residual between them (mv_norm, mv_norm_backward in include/mv.h):
//   u = N(y) post + post_bias,   r = alpha residual + gate u,   n = N(r) weight + bias
// A block holds a row: it is read once, the next one on its way, and the stream
// between the two norms is normed from its 32-bit values.
//
// Memory bounds it where a row is normed once: 16384 x 5120 bfloat16, layer, with
// residual and gates (671 MB) 111 us, 6.0 TB/s.  With both norms it is the row's
// chain of sums and the instructions between them: 16384 x 7168, 195 us, 4.8 TB/s.
// Steps on the way to the first figure: 191 us; the next row's loads ahead and
// arithmetic by pairs 111; registers by block size, for parameters of 32 bits and
// biases.  Rows on no 16-byte boundary go element by element: 16384 x 1437, 2.8 TB/s.
#include <algorithm>
#include <cmath>

#include "mv_norm.cuh"

namespace mvblock {

// Registers decide: blocks of at most 320 threads go two an SM with 96 registers a
// thread, larger ones alone.  16384 x 7168 with both norms took 214 us in two blocks of
// 64 registers, 195 in one; 16384 x 5120 with biases 152 us in one block, 115 in two;
// unaligned rows, 16384 x 1437 in 16 bits, 99 us with 64 registers, 66 with 96.
constexpr int kFewThreads = 320, kMoreThreads = 640;

// A row as it lies in memory, so that the next one costs few registers.
template <class T, int N, int E, bool WHOLE> struct RawRow {
    static constexpr int kPieces = E / N;
    std::conditional_t<N == 1, T, uint4> piece[kPieces];
    __device__ __forceinline__ void fetch(const T *row, u32 hidden, u32 threads)
    {
#pragma unroll
        for (int i = 0; i < kPieces; i++) {
            const u32 c = WHOLE ? (i * threads + threadIdx.x) * N : column_of<N>(i, hidden, threads);
            if constexpr (N == 1) piece[i] = row[c];
            else piece[i] = *reinterpret_cast<const uint4 *>(row + c);
        }
    }
    __device__ __forceinline__ void widen(float (&v)[E]) const
    {
#pragma unroll
        for (int i = 0; i < kPieces; i++) {
            if constexpr (N == 1) v[i] = to_float(piece[i]);
            else widen_piece<T, N>(piece[i], &v[i * N]);
        }
    }
};

template <class T, class P, int N, int E, bool WHOLE, int MOST> __global__ void __launch_bounds__(MOST, MOST == kFewThreads ? 2 : 1) k_norm(const NormArgs a)
{
    __shared__ __align__(16) float part[2][32];
    const u32 threads = blockDim.x, hidden = a.hidden;
    const bool layer = a.layer;
    Reducer sum = {part, 0, threads / 32};
    sum.start();
    const T *y = static_cast<const T *>(a.y), *residual = static_cast<const T *>(a.residual);
    RawRow<T, N, E, WHOLE> next_y, next_residual;
    auto fetch = [&](u64 t) {
        if (t >= a.tokens) return;
        next_y.fetch(y + t * a.y_stride, hidden, threads);
        if (residual) next_residual.fetch(residual + t * a.residual_stride, hidden, threads);
    };
    fetch(blockIdx.x);
    for (u64 t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        float v[E], w[E];
        next_y.widen(v);
        RawRow<T, N, E, WHOLE> res = next_residual;
        fetch(t + gridDim.x);
        if (a.post) {
            normalise<N, WHOLE>(a, layer, sum, v, threads);
            get_row<P, N, WHOLE>(static_cast<const P *>(a.post), hidden, threads, w);
            mul_row(v, v, w);
            if (a.post_bias) {
                get_row<P, N, WHOLE>(static_cast<const P *>(a.post_bias), hidden, threads, w);
                add_row(v, v, w);
            }
        }
        if (a.gate) {
            get_row<P, N, WHOLE>(static_cast<const P *>(a.gate) + (u64)((u32)t / (u32)a.run) * hidden, hidden, threads, w);
            mul_row(v, v, w);
        }
        if (residual) {
            res.widen(w);
            fma_row(v, w, a.alpha, v);
        }
        if (a.r) put_row<T, N, WHOLE>(static_cast<T *>(a.r) + t * hidden, hidden, threads, v);
        normalise<N, WHOLE>(a, layer, sum, v, threads);
        get_row<P, N, WHOLE>(static_cast<const P *>(a.weight), hidden, threads, w);
        mul_row(v, v, w);
        if (a.bias) {
            get_row<P, N, WHOLE>(static_cast<const P *>(a.bias), hidden, threads, w);
            add_row(v, v, w);
        }
        put_row<T, N, WHOLE>(static_cast<T *>(a.n) + t * hidden, hidden, threads, v);
    }
}

// The blocks' sums, added in their order: two columns a lane, every sixteenth
// block's a warp, then the warps'.
constexpr u32 kAddWarps = 16, kAddColumns = 64;
struct AddArgs {
    const float *sums, *gate_sums;
    void *to[4], *dgate;
    u64 tokens, hidden, pitch, blocks, run, rows;
    u32 shared, gates_first, params_f32;
};
template <class T> __global__ void __launch_bounds__(32 * kAddWarps) k_norm_add(const AddArgs a)
{
    __shared__ float2 part[kAddWarps][32];
    const u32 lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const u64 c = ((u64)blockIdx.x * 32 + lane) * 2;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // what: four parameters, then the gates that more than one block has a part of: one of every gate
    // or, where those are more, of every block, the gate that begins in it and goes on after it
    for (u32 what = blockIdx.y; what < 4 + a.shared; what += gridDim.y) {
        void *out = what < 4 ? a.to[what] : a.dgate;
        if (!out) continue;
        const float *from = a.sums + what * a.pitch;
        u64 step = 4 * a.pitch, first = 0, last = a.blocks, at = 0, own = 0;
        if (what >= 4) {
            const u32 i = what - 4, g = a.gates_first ? i : (u32)(min((i + 1) * a.rows, a.tokens) - 1) / (u32)a.run;
            const u32 b = a.gates_first ? (u32)(g * a.run) / (u32)a.rows : i;
            const u64 begin = b * a.rows, end = min(begin + a.rows, a.tokens);
            if (g * a.run < begin || (g + 1) * a.run <= end) continue;
            // this block's part, and as their first gates' those of the blocks up to its end
            first = b;
            last = ((g + 1) * a.run - 1) / a.rows + 1;
            from = a.gate_sums;
            step = 2 * a.pitch;
            at = g * a.hidden;
            own = g != (u32)begin / (u32)a.run ? a.pitch : 0;
        }
        float2 s = make_float2(0.0f, 0.0f);
        if (c < a.hidden) {
            const float *p = from + (first + warp) * step + c;
            u32 left = (u32)(last - first);
            left = left > warp ? (left - warp + kAddWarps - 1) / kAddWarps : 0;
            if (own && warp == 0) {
                s = *reinterpret_cast<const float2 *>(p + own);
                p += kAddWarps * step;
                left--;
            }
#pragma unroll 8
            for (; left; left--, p += kAddWarps * step) {
                const float2 w = *reinterpret_cast<const float2 *>(p);
                s.x += w.x; s.y += w.y;
            }
        }
        __syncthreads();
        part[warp][lane] = s;
        __syncthreads();
        if (threadIdx.x >= kAddColumns) continue;
        const u64 mine = (u64)blockIdx.x * kAddColumns + threadIdx.x;
        if (mine >= a.hidden) continue;
        float v = 0.0f;
#pragma unroll
        for (u32 i = 0; i < kAddWarps; i++) v += reinterpret_cast<const float *>(part[i])[threadIdx.x];
        if (a.params_f32) static_cast<float *>(out)[at + mine] = v;
        else static_cast<T *>(out)[at + mine] = from_float<T>(v);
    }
}

// ---- host ---------------------------------------------------------------
// Sixteen elements a thread: with eight the block's sums are a larger part of the
// work (16384 x 7168 with both norms 220 us instead of 214, 16384 x 5120 layer 160
// instead of 128, when they were measured), with 32, for rows that 512 threads would not hold
// otherwise, registers leave one block an SM.  Rows on no 16-byte boundary have eight, or
// sixteen where 1024 threads need them.  Short rows are one warp's.
NormShape shape_of(u32 hidden, u32 size, bool wide)
{
    const u32 n = wide ? 16 / size : 1, few = wide ? n : 4;
    const u32 e = hidden <= 32 * few ? few : !wide ? (hidden <= 8192 ? 8 : 16) : hidden <= 16 * kMostThreads ? 16 : 32;
    const u32 threads = (hidden + e - 1) / e;
    return {n, e / n, (threads + 31) / 32 * 32, hidden % (32 * e) == 0, 1};
}

// rows of pieces of n elements, 16 bytes
bool dense(const void *p, u64 stride, u32 n) { return !p || (aligned(p, 16) && stride % n == 0); }

int check(const mv_norm_desc *d)
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
    return MV_OK;
}

bool wide_row(const mv_norm_desc *d)
{
    const u32 n = 16 / (u32)dtype_size(d->dtype);
    return d->hidden % n == 0 && dense(d->y, d->y_stride, n) && dense(d->residual, d->residual_stride, n) &&
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

template <class T, class P> int run_norm(const NormArgs &a, const NormShape &s, u32 sms, cudaStream_t stream)
{
    const u32 e = s.n * s.pieces, few = e <= 16 && s.threads <= kFewThreads;
    const u32 an_sm = few ? std::min(16u, 2 * kFewThreads / s.threads) : 1;
    const dim3 grid((u32)std::min<u64>(a.tokens, (u64)sms * an_sm));
    constexpr int N = 16 / sizeof(T), kFew = kFewThreads, kMost = kMostThreads;
    auto run = [&](auto kernel) { return launch(kernel, grid, s.threads, 0, stream, a); };
    if (s.n > 1) {
        if (e == N) return run(k_norm<T, P, N, N, false, kFew>);
        if (e == 16 && s.whole) return few ? run(k_norm<T, P, N, 16, true, kFew>) : run(k_norm<T, P, N, 16, true, kMost>);
        if (e == 16) return few ? run(k_norm<T, P, N, 16, false, kFew>) : run(k_norm<T, P, N, 16, false, kMost>);
        return run(k_norm<T, P, N, 32, false, kMost>);
    }
    if (e == 4) return run(k_norm<T, P, 1, 4, false, kFew>);
    if (e == 8) return few ? run(k_norm<T, P, 1, 8, false, kFew>) : s.threads <= kMoreThreads ? run(k_norm<T, P, 1, 8, false, kMoreThreads>)
                                                                                              : run(k_norm<T, P, 1, 8, false, 1024>);
    return run(k_norm<T, P, 1, 16, false, 1024>);
}
template <class T> int run_norm(const NormArgs &a, const NormShape &s, u32 sms, cudaStream_t stream)
{
    return a.params_f32 ? run_norm<T, float>(a, s, sms, stream) : run_norm<T, T>(a, s, sms, stream);
}

struct GradPlan {
    NormShape shape;
    u32 smem;
    u64 blocks, rows, pitch, gate_sums, total;
};
GradPlan grad_plan(const mv_norm_desc *d, bool wide)
{
    GradPlan p = {};
    const u32 size = (u32)dtype_size(d->dtype);
    const u32 hidden = (u32)d->hidden, n = wide ? 16 / size : 1;
    // eight elements a thread and two rows at a time (or one, where two do not fit), copied ahead;
    // sixteen and one where a row is too long for that
    auto shape = [&](u32 e, u32 at_once) { return NormShape{n, e / n, ((hidden + e - 1) / e + 31) / 32 * 32, false, at_once}; };
    p.shape = shape(8, 2);
    if (p.shape.threads <= 1024) {
        p.smem = n * size >= 4 ? 5 * 2 * 8 * p.shape.threads * size : 0;
        if (p.smem > 216 * 1024) {
            p.shape.at_once = 1;
            p.smem /= 2;
        }
    } else {
        p.shape = shape(16, 1);
    }
    const u32 threads = p.shape.threads;
    const u32 sms = std::max(1u, sm_count());
    const u32 held = (threads <= (u32)kGradThreads<true> ? kGradThreads<true> : kGradThreads<false>) / threads;
    const u32 an_sm = std::max(1u, std::min(held, p.smem ? 224u * 1024 / (p.smem + 2048) : 16u));
    // at least four rows a block: its sums are written and read once for all of them
    const u64 blocks = std::min<u64>((d->tokens + 3) / 4, (u64)sms * std::min(an_sm, 16u));
    p.rows = (d->tokens + blocks - 1) / blocks;
    p.blocks = (d->tokens + p.rows - 1) / p.rows;
    p.pitch = (d->hidden + 3) / 4 * 4;
    p.gate_sums = (p.blocks * 4 * p.pitch * 4 + 255) / 256 * 256;
    p.total = p.gate_sums + (d->gate ? p.blocks * 2 * p.pitch * 4 : 0);
    return p;
}

}  // namespace mvblock

using namespace mvblock;

extern "C" int mv_norm(const mv_norm_desc *d, void *n, void *r, void *stream)
{
    const int rc = check(d);
    if (rc != MV_OK || d->tokens == 0) return rc;
    const u64 size = dtype_size(d->dtype);
    if (!n || !aligned(n, size) || !aligned(r, size)) return MV_EINVAL;
    const u32 sms = sm_count();
    if (!sms) return MV_ECUDA;
    NormArgs a = arguments(d);
    a.n = n;
    a.r = r;
    const NormShape s = shape_of(a.hidden, (u32)size, wide_row(d) && aligned(n, 16) && aligned(r, 16));
    cudaStream_t on = static_cast<cudaStream_t>(stream);
    if (d->dtype == MV_F32) return run_norm<float>(a, s, sms, on);
    return d->dtype == MV_F16 ? run_norm<__half>(a, s, sms, on) : run_norm<__nv_bfloat16>(a, s, sms, on);
}

static int check_grad(const mv_norm_desc *d, const mv_norm_grads *g)
{
    const int rc = check(d);
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
    const u32 n = 16 / (u32)dtype_size(d->dtype);
    return wide_row(d) && dense(g->dn, g->dn_stride, n) && dense(g->dr, g->dr_stride, n) && aligned(g->dy, 16) &&
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
    a.dgate = g->dgate;
    a.rows = p.rows;
    a.sums = reinterpret_cast<float *>(ws);
    a.gate_sums = reinterpret_cast<float *>(ws + p.gate_sums);
    AddArgs add = {};
    add.sums = a.sums;
    add.gate_sums = a.gate_sums;
    add.to[0] = g->dweight;
    add.to[1] = g->dbias;
    add.to[2] = g->dpost;
    add.to[3] = g->dpost_bias;
    add.dgate = g->dgate;
    add.tokens = d->tokens;
    add.gates_first = d->gates <= p.blocks;
    add.shared = add.dgate ? (u32)std::min<u64>(d->gates, p.blocks) : 0;
    add.hidden = d->hidden;
    add.pitch = a.pitch = p.pitch;
    add.blocks = p.blocks;
    add.run = a.run;
    add.rows = p.rows;
    add.params_f32 = a.params_f32;
    const bool post = d->post || d->gate, bias = a.layer || d->bias || d->post_bias;
    const int done = d->dtype == MV_F32 ? run_norm_grad<float>(a, p.shape, p.blocks, p.smem, post, bias, on)
                   : d->dtype == MV_F16 ? run_norm_grad<__half>(a, p.shape, p.blocks, p.smem, post, bias, on)
                                        : run_norm_grad<__nv_bfloat16>(a, p.shape, p.blocks, p.smem, post, bias, on);
    if (done != MV_OK) return done;
    const dim3 grid((u32)((d->hidden + kAddColumns - 1) / kAddColumns), 4 + std::min(add.shared, 16u));
    return d->dtype == MV_BF16 ? launch_after(k_norm_add<__nv_bfloat16>, grid, 32 * kAddWarps, 0, on, add)
                               : launch_after(k_norm_add<__half>, grid, 32 * kAddWarps, 0, on, add);
}
