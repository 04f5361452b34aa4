// Routing of tokens to experts, and its gradient (mv_route,
// mv_route_backward in include/mv.h, which states the formulas).
#include <cmath>
#include <cstring>

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
__device__ __noinline__ void route_row(const RouteArgs &a, u64 row, u32 *key)
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

// ---- the fast way ---------------------------------------------------------
// L lanes share a row, V experts a lane.  Every expert becomes one unsigned
// key that orders like its value and ends in its place, so that keys differ
// and ties fall to the lowest index; a lane sorts its keys by a network of
// min and max, and the row's greatest head is taken topk times.  16-bit
// logits fit a key whole.  Longer values lose their last bits to the place
// (and scores come from the approximate exponential and reciprocal): where
// two neighbours in the order are closer than that, the row is done again by
// route_row, which compares exact values.
constexpr u32 kRouteWarps = 8;

// How the lanes of a row share the experts: a group of experts takes
// 1 << shift lanes, `per` experts each.
struct Shares {
    u32 shift, per, size;
    bool wide;                      // lanes load their experts by 16 bytes
};

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

template <int L> __device__ __forceinline__ u32 row_max(u32 v)
{
    if (L == 32) return __reduce_max_sync(kFull, v);
#pragma unroll
    for (int d = L / 2; d; d >>= 1) v = max(v, __shfl_xor_sync(kFull, v, d));
    return v;
}

__device__ __forceinline__ void order_two(u32 &a, u32 &b)
{
    const u32 hi = max(a, b), lo = min(a, b);
    a = hi;
    b = lo;
}
// Batcher's odd-even merge sort, greatest first.
template <int V> __device__ __forceinline__ void sort_keys(u32 (&k)[V])
{
#pragma unroll
    for (int p = 1; p < V; p <<= 1)
#pragma unroll
        for (int d = p; d > 0; d >>= 1)
#pragma unroll
            for (int j = d % p; j + d < V; j += 2 * d)
#pragma unroll
                for (int i = 0; i < d; i++)
                    if (i + j + d < V && (i + j) / (2 * p) == (i + j + d) / (2 * p)) order_two(k[i + j], k[i + j + d]);
}

template <class T, int V>
__device__ __forceinline__ void load_share(const T *x, u32 n, bool wide, float (&v)[V])
{
    constexpr int kPer = 16 / sizeof(T);
    if (wide && n == V) {
#pragma unroll
        for (int i = 0; i < V / kPer; i++) {
            const uint4 q = reinterpret_cast<const uint4 *>(x)[i];
            const u32 w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (sizeof(T) == 4) {
                    v[i * kPer + j] = __uint_as_float(w[j]);
                } else {
                    T pair[2];
                    memcpy(pair, &w[j], 4);
                    v[i * kPer + 2 * j] = to_float(pair[0]);
                    v[i * kPer + 2 * j + 1] = to_float(pair[1]);
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) v[i] = i < n ? to_float(x[i]) : -INFINITY;
    }
}

template <class T, int ORDER, int L, int V, bool FEW>
__global__ void __launch_bounds__(kRouteWarps * 32) k_route(const RouteArgs a, const Shares sh)
{
    extern __shared__ u32 keys[];
    constexpr bool EXACT = sizeof(T) == 2 && ORDER == kByLogit;
    constexpr u32 kPlace = EXACT ? L * V - 1 : V - 1;        // a key's bits for the place
    constexpr u32 kRows = 32 / L;
    const u32 lane = threadIdx.x & 31, sub = lane & (L - 1), warp = threadIdx.x >> 5;
    const u32 in_group = sub & ((1u << sh.shift) - 1), group = sub >> sh.shift;
    const u32 base = group * sh.size + in_group * sh.per;
    const u32 n = group < a.groups && in_group * sh.per < sh.size ? min(sh.per, sh.size - in_group * sh.per) : 0;
    const bool stats = a.softmax && (ORDER == kBySoftmax || !a.renorm);
    float bias[V];
    if (ORDER != kByLogit) {
#pragma unroll
        for (int i = 0; i < V; i++) bias[i] = i < n ? (a.bias ? a.bias[base + i] : 0.0f) : -INFINITY;
    }
    const u64 step = (u64)gridDim.x * kRouteWarps * kRows;
    for (u64 first = ((u64)blockIdx.x * kRouteWarps + warp) * kRows; first < a.tokens; first += step) {
        const u64 row = first + lane / L;
        const bool here = row < a.tokens;
        const T *x = static_cast<const T *>(a.logits) + (here ? row : first) * a.stride;
        float v[V];
        load_share<T, V>(x + base, n, sh.wide, v);
        float m = -INFINITY, sum = 0.0f;
        if (stats) {
#pragma unroll
            for (int i = 0; i < V; i++) m = fmaxf(m, v[i]);          // passes NaN by
            m = group_max<L>(m);
#pragma unroll
            for (int i = 0; i < V; i++)
                sum += open(v[i]) ? (v[i] == m ? 1.0f : exp2_fast((v[i] - m) * kLog2e)) : 0.0f;
            sum = group_sum<L>(sum);
        }
        u32 key[V];
        const float inv = ORDER == kBySoftmax ? reciprocal_fast(sum) : 0.0f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            float by = v[i];
            if (ORDER == kBySigmoid) by = reciprocal_fast(1.0f + exp2_fast(-v[i] * kLog2e)) + bias[i];
            if (ORDER == kBySoftmax) by = (v[i] == m ? 1.0f : exp2_fast((v[i] - m) * kLog2e)) * inv + bias[i];
            const bool is_open = open(v[i]) && (ORDER == kByLogit || open(bias[i]));
            key[i] = is_open ? (ordered(by) & ~kPlace) | (kPlace - (EXACT ? base + i : i)) : 0u;
        }
        sort_keys<V>(key);
        // a value's error: the bits that made room, and the approximations
        const float rel = EXACT || ORDER == kByLogit ? 0.0f : V * 0x1p-23f;
        const float eps = ORDER == kByLogit ? 0.0f : ORDER == kBySigmoid ? 1e-6f : 2e-6f;
        bool close = false;
        if (a.groups > 1) {
            u32 f = key[0], s = key[1];
            for (u32 d = 1; d < 1u << sh.shift; d <<= 1) {
                const u32 f2 = __shfl_xor_sync(kFull, f, d), s2 = __shfl_xor_sync(kFull, s, d);
                s = max(max(s, s2), min(f, f2));
                f = max(f, f2);
            }
            u32 mine = f;
            float value = 0.0f, size = 0.0f;
            if (!EXACT) {
                value = unordered(f & ~kPlace);
                size = fabsf(value);
                if (a.top_two && s) {
                    const float v2 = unordered(s & ~kPlace);
                    value += v2;
                    size += fabsf(v2);
                }
                mine = f ? ordered(value) : 0u;
            }
            u32 before = 0;
            for (u32 g = 0; g < a.groups; g++) {
                const u32 other = __shfl_sync(kFull, mine, g << sh.shift, L);
                before += other > mine || (other == mine && g < group);
            }
            const bool stays = group < a.groups && before < a.top_groups;
            if (!EXACT) {
                // the best that leaves against each that stays
                const u32 out = row_max<L>(stays || group >= a.groups ? 0u : mine);
                const float most = __uint_as_float(row_max<L>(f ? __float_as_uint(size) : 0u));
                const float tol = 4 * eps + 4 * rel * most;
                if (stays && mine && out)
                    close = ORDER == kByLogit ? (mine ^ out) <= kPlace : !(value - unordered(out) > tol);
            }
            if (!stays)
#pragma unroll
                for (int i = 0; i < V; i++) key[i] = 0;
        }
        // lane r of the row keeps slot r; one look further tells how sure the last is
        u32 got = 0, from = 0, after = 0;
        auto take = [&](u32 r, int depth) {
            const u32 top = row_max<L>(key[0]);
            bool won = key[0] == top;
            u32 who = 0;
            if (!EXACT) {
                u32 all = __ballot_sync(kFull, won);
                if (L < 32) all = (all >> (lane & ~(L - 1))) & ((1u << L) - 1);
                who = __ffs(all) - 1;
                won = sub == who;
            }
            if (sub == r) { got = top; from = who; }
            if (r == a.topk) after = top;
#pragma unroll
            for (int i = 0; i + 1 < V; i++)
                if (i < depth) key[i] = won ? key[i + 1] : key[i];
            if (depth >= V - 1) key[V - 1] = won ? 0u : key[V - 1];
        };
        const u32 looks = a.topk + (EXACT ? 0 : 1);
        if (FEW) {                                   // topk <= 8: only what can still be reached moves up
#pragma unroll
            for (int r = 0; r < 9; r++)
                if (r < looks) take(r, 8 - r);
        } else {
            for (u32 r = 0; r < looks; r++) take(r, V);
        }
        int id = -1;
        if (sub < a.topk && got) {
            const u32 place = kPlace - (got & kPlace);
            id = (int)(EXACT ? place
                             : (from >> sh.shift) * sh.size + (from & ((1u << sh.shift) - 1)) * sh.per + place);
        }
        if (!EXACT) {
            u32 next = __shfl_down_sync(kFull, got, 1, L);
            if (sub + 1 == a.topk) next = after;
            if (id >= 0 && next) {
                if (ORDER == kByLogit) {
                    close = close || (got ^ next) <= kPlace;
                } else {
                    const float p = unordered(got & ~kPlace), q = unordered(next & ~kPlace);
                    close = close || !(p - q > 2 * eps + 2 * rel * (fabsf(p) + fabsf(q)));
                }
            }
        }
        float logit = 0.0f;
        if (EXACT) {
            // a negative number's key is its complement: the place's bits were ones
            const u32 k = (got >> 31) ? got & ~kPlace : got | kPlace;
            if (id >= 0) logit = unordered(k);
        } else if (id >= 0) {
            logit = to_float(x[id]);
        }
        const float w = slot_weight<L>(a, id, logit, m, sum);
        u32 again = EXACT ? 0u : __ballot_sync(kFull, close && here);
        if (L < 32) again = (again >> (lane & ~(L - 1))) & ((1u << L) - 1);
        if (here && !again && sub < a.topk) {
            a.ids[row * a.topk + sub] = id;
            a.weights[row * a.topk + sub] = w;
        }
        if (!EXACT) {
            u32 rows = __ballot_sync(kFull, again != 0 && sub == 0);
            while (rows) {
                const u32 at = __ffs(rows) - 1;
                rows &= rows - 1;
                route_row<T, ORDER>(a, first + at / L, keys + warp * a.experts);
            }
        }
    }
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

template <class T, int ORDER, int L, int V, bool FEW>
int run_route(const RouteArgs &a, const Shares &sh, cudaStream_t stream)
{
    constexpr u32 kRowsABlock = kRouteWarps * (32 / L);
    const u32 blocks = (u32)std::fmin((double)((a.tokens + kRowsABlock - 1) / kRowsABlock), 8.0 * sm_count());
    if (!blocks) return MV_ECUDA;
    const bool exact = sizeof(T) == 2 && ORDER == kByLogit;
    return launch(k_route<T, ORDER, L, V, FEW>, blocks, kRouteWarps * 32,
                  exact ? 0 : kRouteWarps * a.experts * 4, stream, a, sh);
}

// The smallest of the shapes (lanes, experts a lane) that holds the experts,
// a lane to a slot and whole lanes to a group.
template <class T, int ORDER> int run_route(const RouteArgs &a, cudaStream_t stream)
{
    auto fits = [&](u32 L, u32 V, Shares &sh) {
        if (a.topk > L || a.groups > L) return false;
        sh.shift = 0;
        while (a.groups << (sh.shift + 1) <= L) sh.shift++;
        sh.size = a.experts / a.groups;
        sh.per = a.groups == 1 ? V : (sh.size + (1u << sh.shift) - 1) >> sh.shift;
        if (sh.per > V || sh.size > sh.per << sh.shift) return false;
        sh.wide = sh.per == V && aligned(a.logits, 16) && a.stride * sizeof(T) % 16 == 0 &&
                  (a.groups == 1 || sh.size * sizeof(T) % 16 == 0);
        return true;
    };
    Shares sh;
    const bool few = a.topk <= 8;
    if (few && fits(8, 8, sh)) return run_route<T, ORDER, 8, 8, true>(a, sh, stream);
    if (few && fits(16, 8, sh)) return run_route<T, ORDER, 16, 8, true>(a, sh, stream);
    if (fits(32, 8, sh))
        return few ? run_route<T, ORDER, 32, 8, true>(a, sh, stream) : run_route<T, ORDER, 32, 8, false>(a, sh, stream);
    if (fits(32, 16, sh)) return run_route<T, ORDER, 32, 16, false>(a, sh, stream);
    if (fits(32, 32, sh)) return run_route<T, ORDER, 32, 32, false>(a, sh, stream);
    return MV_EOVERFLOW;
}

template <class T> int run_route(const RouteArgs &a, Order order, cudaStream_t stream)
{
    if (order == kByLogit) return run_route<T, kByLogit>(a, stream);
    if (order == kBySigmoid) return run_route<T, kBySigmoid>(a, stream);
    return run_route<T, kBySoftmax>(a, stream);
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
