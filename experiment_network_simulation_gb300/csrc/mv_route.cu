// Routing of tokens to experts, and its gradient (mv_route,
// mv_route_backward in include/mv.h, which states the formulas).
#include <cmath>

#include "mv_moe.cuh"

namespace mvmoe {

// What the experts of a row are ordered by.
enum Order { kByLogit = 0, kBySigmoid = 1, kBySoftmax = 2 };

struct RouteArgs {
    const void *logits;
    const float *bias;
    int32_t *ids;
    float *weights;
    u64 tokens, stride;
    u32 experts, topk, groups, top_groups;
    bool softmax, renorm, top_two;
    float scale;
};

// An unsigned integer that orders like the float: 0 is below every number,
// and stands for a closed expert.  Adding 0 makes -0 and 0 the same.
__device__ __forceinline__ u32 ordered(float v)
{
    const u32 u = __float_as_uint(v + 0.0f);
    return u ^ ((u32)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(u32 k)
{
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// Neither -inf nor NaN.
__device__ __forceinline__ bool open(float v) { return v > -INFINITY; }
// exp(v - m) for v <= m; 1 at the maximum, an infinite one included.
__device__ __forceinline__ float exp_below(float v, float m) { return v == m ? 1.0f : expf(v - m); }
__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// Weights of a row's choices.  Lane r of the W lanes holds slot r: its
// expert (or -1) and that expert's logit; m and sum are the row's softmax
// statistics where the weights need them.
template <int W>
__device__ __forceinline__ float slot_weight(const RouteArgs &a, int id, float x, float m, float sum)
{
    float w = 0.0f;
    if (a.softmax && a.renorm) {
        const float best = group_max<W>(id >= 0 ? x : -INFINITY);
        w = id >= 0 ? exp_below(x, best) : 0.0f;
    } else if (id >= 0) {
        w = a.softmax ? exp_below(x, m) / sum : sigmoid(x);
    }
    if (a.renorm) {
        const float total = group_sum<W>(w);
        w = total > 0.0f ? w / total : 0.0f;
    }
    return w * a.scale;
}

// One row by one warp, by comparing every expert's exact order value.
// key: the warp's own `experts` words of shared memory.
template <class T, int ORDER>
__device__ void route_row(const RouteArgs &a, u64 row, u32 *key)
{
    const u32 lane = threadIdx.x & 31, E = a.experts;
    const T *x = static_cast<const T *>(a.logits) + row * a.stride;
    float m = -INFINITY, sum = 0.0f;
    if (a.softmax && (ORDER == kBySoftmax || !a.renorm)) {
        for (u32 e = lane; e < E; e += 32) {
            const float v = to_float(x[e]);
            if (open(v)) m = fmaxf(m, v);
        }
        m = group_max<32>(m);
        for (u32 e = lane; e < E; e += 32) {
            const float v = to_float(x[e]);
            if (open(v)) sum += exp_below(v, m);
        }
        sum = group_sum<32>(sum);
    }
    for (u32 e = lane; e < E; e += 32) {
        const float v = to_float(x[e]), b = a.bias ? a.bias[e] : 0.0f;
        float by = v;
        if (ORDER == kBySigmoid) by = sigmoid(v) + b;
        if (ORDER == kBySoftmax) by = exp_below(v, m) / sum + b;
        key[e] = open(v) && open(b) ? ordered(by) : 0u;
    }
    __syncwarp();
    if (a.groups > 1) {
        const u32 size = E / a.groups;
        u32 mine = 0;
        if (lane < a.groups) {
            u32 first = 0, second = 0;
            for (u32 i = 0; i < size; i++) {
                const u32 k = key[lane * size + i];
                second = max(second, min(first, k));
                first = max(first, k);
            }
            mine = first;
            if (a.top_two && second) mine = ordered(unordered(first) + unordered(second));
        }
        u32 before = 0;
        for (u32 g = 0; g < a.groups; g++) {
            const u32 other = __shfl_sync(kFull, mine, g);
            before += other > mine || (other == mine && g < lane);
        }
        const u32 stays = __ballot_sync(kFull, lane < a.groups && before < a.top_groups);
        __syncwarp();
        for (u32 e = lane; e < E; e += 32)
            if (!((stays >> (e / size)) & 1)) key[e] = 0;
        __syncwarp();
    }
    int id = -1;
    for (u32 r = 0; r < a.topk; r++) {
        u32 best = 0, at = kFull;
        for (u32 e = lane; e < E; e += 32)
            if (key[e] > best) { best = key[e]; at = e; }
        const u32 top = __reduce_max_sync(kFull, best);
        if (!top) break;
        const u32 e = __reduce_min_sync(kFull, best == top ? at : kFull);
        if (lane == r) id = (int)e;
        if (lane == 0) key[e] = 0;
        __syncwarp();
    }
    const float v = id >= 0 ? to_float(x[id]) : 0.0f;
    const float w = slot_weight<32>(a, id, v, m, sum);
    if (lane < a.topk) {
        a.ids[row * a.topk + lane] = id;
        a.weights[row * a.topk + lane] = w;
    }
    __syncwarp();
}

constexpr u32 kRouteWarps = 8;

template <class T, int ORDER>
__global__ void __launch_bounds__(kRouteWarps * 32) k_route(const RouteArgs a)
{
    extern __shared__ u32 keys[];
    u32 *key = keys + (threadIdx.x >> 5) * a.experts;
    const u64 step = (u64)gridDim.x * kRouteWarps;
    for (u64 row = (u64)blockIdx.x * kRouteWarps + (threadIdx.x >> 5); row < a.tokens; row += step)
        route_row<T, ORDER>(a, row, key);
}

struct RouteGradArgs {
    const void *logits;
    const int32_t *ids;
    const float *dweights;
    void *dlogits;
    u64 tokens, stride;
    u32 experts, topk;
    bool softmax, renorm;
    float scale;
};

// The gradient of one row by one warp.  With G the slots' gradients laid out
// over the experts, and p the softmax: dx = scale p (G - sum G p), dense.
// In the other forms only the chosen experts' logits matter.
constexpr u32 kGradWarps = 8;

template <class T>
__global__ void __launch_bounds__(kGradWarps * 32) k_route_grad(const RouteGradArgs a)
{
    extern __shared__ float grads[];
    const u32 lane = threadIdx.x & 31, E = a.experts;
    float *G = grads + (threadIdx.x >> 5) * E;
    const u64 step = (u64)gridDim.x * kGradWarps;
    for (u64 row = (u64)blockIdx.x * kGradWarps + (threadIdx.x >> 5); row < a.tokens; row += step) {
        const T *x = static_cast<const T *>(a.logits) + row * a.stride;
        T *dx = static_cast<T *>(a.dlogits) + row * E;
        for (u32 e = lane; e < E; e += 32) G[e] = 0.0f;
        int id = lane < a.topk ? a.ids[row * a.topk + lane] : -1;
        if ((u32)id >= E) id = -1;
        const float g = id >= 0 ? a.dweights[row * a.topk + lane] : 0.0f;
        __syncwarp();
        if (a.softmax && !a.renorm) {
            if (id >= 0) G[id] = g;
            __syncwarp();
            float m = -INFINITY, sum = 0.0f, dot = 0.0f;
            for (u32 e = lane; e < E; e += 32) {
                const float v = to_float(x[e]);
                if (open(v)) m = fmaxf(m, v);
            }
            m = group_max<32>(m);
            for (u32 e = lane; e < E; e += 32) {
                const float v = to_float(x[e]), p = open(v) ? exp_below(v, m) : 0.0f;
                sum += p;
                dot += p * G[e];
            }
            sum = group_sum<32>(sum);
            dot = group_sum<32>(dot);
            const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
            dot *= inv;
            for (u32 e = lane; e < E; e += 32) {
                const float v = to_float(x[e]), p = open(v) ? exp_below(v, m) * inv : 0.0f;
                dx[e] = from_float<T>(p * (G[e] - dot) * a.scale);
            }
        } else {
            const float v = id >= 0 ? to_float(x[id]) : -INFINITY;
            float d;
            if (a.softmax) {
                const float best = group_max<32>(v);
                float w = id >= 0 ? exp_below(v, best) : 0.0f;
                const float sum = group_sum<32>(w);
                w = sum > 0.0f ? w / sum : 0.0f;
                d = w * (g - group_sum<32>(g * w));
            } else {
                const float s = id >= 0 ? sigmoid(v) : 0.0f;
                d = g;
                if (a.renorm) {
                    const float sum = group_sum<32>(s), dot = group_sum<32>(g * s);
                    d = sum > 0.0f ? (g - dot / sum) / sum : 0.0f;
                }
                d *= s * (1.0f - s);
            }
            if (id >= 0) G[id] = d * a.scale;
            __syncwarp();
            for (u32 e = lane; e < E; e += 32) dx[e] = from_float<T>(G[e]);
        }
        __syncwarp();
    }
}

template <class T> int run_route(const RouteArgs &a, Order order, cudaStream_t stream)
{
    const u32 blocks = (u32)std::fmin((double)((a.tokens + kRouteWarps - 1) / kRouteWarps),
                                      (double)sm_count() * 8);
    const u32 smem = kRouteWarps * a.experts * 4;
    if (!blocks) return MV_ECUDA;
    if (order == kByLogit) return launch(k_route<T, kByLogit>, blocks, kRouteWarps * 32, smem, stream, a);
    if (order == kBySigmoid)
        return launch(k_route<T, kBySigmoid>, blocks, kRouteWarps * 32, smem, stream, a);
    return launch(k_route<T, kBySoftmax>, blocks, kRouteWarps * 32, smem, stream, a);
}

template <class T> int run_route_grad(const RouteGradArgs &a, cudaStream_t stream)
{
    const u32 blocks = (u32)std::fmin((double)((a.tokens + kGradWarps - 1) / kGradWarps),
                                      (double)sm_count() * 8);
    if (!blocks) return MV_ECUDA;
    return launch(k_route_grad<T>, blocks, kGradWarps * 32, kGradWarps * a.experts * 4, stream, a);
}

}  // namespace mvmoe

using namespace mvmoe;

extern "C" int mv_route(const mv_route_desc *d, void *stream)
{
    if (!d || !d->experts || !d->topk || d->topk > d->experts || d->dtype > MV_BF16 ||
        d->scores > MV_SCORE_SIGMOID || d->group_rule > MV_GROUP_TOPTWO || !d->groups ||
        d->groups > 32 || d->experts % d->groups || !d->top_groups || d->top_groups > d->groups ||
        d->topk > d->top_groups * (d->experts / d->groups) || !std::isfinite(d->scale))
        return MV_EINVAL;
    if (d->experts > kMaxExperts || d->topk > kMaxTopk) return MV_EOVERFLOW;
    if (d->tokens == 0) return MV_OK;
    if (!d->logits || !d->ids || !d->weights || d->row_stride < d->experts ||
        !aligned(d->logits, dtype_size(d->dtype)) || !aligned(d->bias, 4) || !aligned(d->ids, 4) ||
        !aligned(d->weights, 4))
        return MV_EINVAL;
    if (d->tokens > (1ull << 40) || d->row_stride > (1ull << 31)) return MV_EOVERFLOW;
    RouteArgs a;
    a.logits = d->logits;
    a.bias = d->bias;
    a.ids = d->ids;
    a.weights = d->weights;
    a.tokens = d->tokens;
    a.stride = d->row_stride;
    a.experts = d->experts;
    a.topk = d->topk;
    a.groups = d->groups;
    a.top_groups = d->top_groups;
    a.softmax = d->scores == MV_SCORE_SOFTMAX;
    a.renorm = d->renorm != 0;
    a.top_two = d->groups > 1 && d->group_rule == MV_GROUP_TOPTWO;
    a.scale = d->scale;
    const Order order = !d->bias && !a.top_two ? kByLogit : a.softmax ? kBySoftmax : kBySigmoid;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (d->dtype == MV_F32) return run_route<float>(a, order, s);
    if (d->dtype == MV_F16) return run_route<__half>(a, order, s);
    return run_route<__nv_bfloat16>(a, order, s);
}

extern "C" int mv_route_backward(const mv_route_grad_desc *d, void *stream)
{
    if (!d || !d->experts || !d->topk || d->topk > d->experts || d->dtype > MV_BF16 ||
        d->scores > MV_SCORE_SIGMOID || !std::isfinite(d->scale))
        return MV_EINVAL;
    if (d->experts > kMaxExperts || d->topk > kMaxTopk) return MV_EOVERFLOW;
    if (d->tokens == 0) return MV_OK;
    const u64 size = dtype_size(d->dtype);
    if (!d->logits || !d->ids || !d->dweights || !d->dlogits || d->row_stride < d->experts ||
        !aligned(d->logits, size) || !aligned(d->ids, 4) || !aligned(d->dweights, 4) ||
        !aligned(d->dlogits, size))
        return MV_EINVAL;
    if (d->tokens > (1ull << 40) || d->row_stride > (1ull << 31)) return MV_EOVERFLOW;
    RouteGradArgs a;
    a.logits = d->logits;
    a.ids = d->ids;
    a.dweights = d->dweights;
    a.dlogits = d->dlogits;
    a.tokens = d->tokens;
    a.stride = d->row_stride;
    a.experts = d->experts;
    a.topk = d->topk;
    a.softmax = d->scores == MV_SCORE_SOFTMAX;
    a.renorm = d->renorm != 0;
    a.scale = d->scale;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (d->dtype == MV_F32) return run_route_grad<float>(a, s);
    if (d->dtype == MV_F16) return run_route_grad<__half>(a, s);
    return run_route_grad<__nv_bfloat16>(a, s);
}
