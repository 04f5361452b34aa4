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
// Renormalised sigmoids whose sum is below this lose bits, and all are 0 under
// logits of -88 or so.  There sigmoid(v) is exp(v) to 2^-26, and what is left of
// the ratio is a softmax of the chosen.  Under -700 (1e-304) a logit is taken for
// what it must be, a mask by the type's lowest value, whose score is 0.
constexpr float kTinySum = 0x1p-26f, kMasked = -700.0f;
__device__ __forceinline__ float tiny_score(float v, float best) { return best >= kMasked ? exp_below(v, best) : 0.0f; }

// Weights of a row's choices, of one row a warp (W is 32).  Lane r holds slot
// r: its expert (or -1) and that expert's logit; m and sum are the row's softmax
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
        float total = group_sum<W>(w);
        if (!a.softmax && total < kTinySum) {        // the same in all of the warp
            const float best = group_max<W>(id >= 0 ? x : -INFINITY);
            w = id >= 0 ? tiny_score(x, best) : 0.0f;
            total = group_sum<W>(w);
        }
        w = total > 0.0f ? w / total : 0.0f;
    }
    return w * a.scale;
}

// One row by one warp, by comparing every expert's exact order value: the
// definition that the faster kernels fall back on where two neighbours in the
// order are nearer than their shortened keys can tell.  How many rows those are
// is up to the data.  By the keys' resolution, 256 standard normal logits with a
// bias of 0.05: two to five in a thousand; 1024 experts by softmax, bias 3e-4: 6
// in a hundred; sigmoids of logits about -8, bias 1e-3: 17 in a hundred; rows of
// ties: all.  2^16 rows take 32 us, 254 (224 with a bias of 0.05), 53 and 111 so.
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

// ---- the fast ways --------------------------------------------------------
// Every expert becomes one unsigned key that orders like its value and ends
// in its place, so that keys differ and ties fall to the lowest index.  Keys
// are sorted by networks of min and max; the row's greatest is taken topk
// times.  16-bit logits fit a key whole.  Longer values lose their last bits
// to the place (and scores come from the approximate exponential and
// reciprocal): where two neighbours in the order are closer than that, the
// row is done again by route_row, which compares exact values.
constexpr u32 kRouteWarps = 8;

// How the lanes of a row share the experts: a group of experts takes
// 1 << shift lanes, `per` experts each.
struct Shares {
    u32 shift, per, size;
    bool wide;                      // lanes load their experts by 16 bytes
};

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

// More than eight slots, and short batches: a warp has a row, a lane V experts,
// all of them sorted.
template <class T, int ORDER, int V>
__global__ void __launch_bounds__(kRouteWarps * 32) k_route(const RouteArgs a, const Shares sh)
{
    extern __shared__ u32 keys[];
    constexpr bool EXACT = sizeof(T) == 2 && ORDER == kByLogit;
    constexpr u32 kPlace = EXACT ? 32 * V - 1 : V - 1;        // a key's bits for the place
    const u32 lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const u32 in_group = lane & ((1u << sh.shift) - 1), group = lane >> sh.shift;
    const u32 base = group * sh.size + in_group * sh.per;
    const u32 n = group < a.groups && in_group * sh.per < sh.size ? min(sh.per, sh.size - in_group * sh.per) : 0;
    const bool stats = a.softmax && (ORDER == kBySoftmax || !a.renorm);
    float bias[V];
    if (ORDER != kByLogit) {
#pragma unroll
        for (int i = 0; i < V; i++) bias[i] = i < n ? (a.bias ? a.bias[base + i] : 0.0f) : -INFINITY;
    }
    const u64 step = (u64)gridDim.x * kRouteWarps;
    for (u64 row = (u64)blockIdx.x * kRouteWarps + warp; row < a.tokens; row += step) {
        const T *x = static_cast<const T *>(a.logits) + row * a.stride;
        float v[V];
        load_share<T, V>(x + base, n, sh.wide, v);
        float m = -INFINITY, sum = 0.0f;
        if (stats) {
#pragma unroll
            for (int i = 0; i < V; i++) m = fmaxf(m, v[i]);          // passes NaN by
            m = group_max<32>(m);
#pragma unroll
            for (int i = 0; i < V; i++)
                sum += open(v[i]) ? (v[i] == m ? 1.0f : exp2_fast((v[i] - m) * kLog2e)) : 0.0f;
            sum = group_sum<32>(sum);
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
                const u32 other = __shfl_sync(kFull, mine, g << sh.shift);
                before += other > mine || (other == mine && g < group);
            }
            const bool stays = group < a.groups && before < a.top_groups;
            if (!EXACT) {
                // the best that leaves against each that stays
                const u32 out = __reduce_max_sync(kFull, stays || group >= a.groups ? 0u : mine);
                const float most = __uint_as_float(__reduce_max_sync(kFull, f ? __float_as_uint(size) : 0u));
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
        const u32 looks = a.topk + (EXACT ? 0 : 1);
        for (u32 r = 0; r < looks; r++) {
            const u32 top = __reduce_max_sync(kFull, key[0]);
            bool won = key[0] == top;
            u32 who = 0;
            if (!EXACT) {
                who = __ffs(__ballot_sync(kFull, won)) - 1;
                won = lane == who;
            }
            if (lane == r) { got = top; from = who; }
            if (r == a.topk) after = top;
#pragma unroll
            for (int i = 0; i + 1 < V; i++) key[i] = won ? key[i + 1] : key[i];
            key[V - 1] = won ? 0u : key[V - 1];
        }
        int id = -1;
        if (lane < a.topk && got) {
            const u32 place = kPlace - (got & kPlace);
            id = (int)(EXACT ? place
                             : (from >> sh.shift) * sh.size + (from & ((1u << sh.shift) - 1)) * sh.per + place);
        }
        if (!EXACT) {
            u32 next = __shfl_down_sync(kFull, got, 1);
            if (lane + 1 == a.topk) next = after;
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
        const float w = slot_weight<32>(a, id, logit, m, sum);
        if (!EXACT && __any_sync(kFull, close)) {
            route_row<T, ORDER>(a, row, keys + warp * a.experts);
        } else if (lane < a.topk) {
            a.ids[row * a.topk + lane] = id;
            a.weights[row * a.topk + lane] = w;
        }
    }
}

// Up to eight slots.  Four lanes share a row, so a warp has eight rows at a
// time: what a row costs in cross-lane steps is shared by eight.  A lane
// takes eight consecutive experts of every 32, sorts their keys and merges
// them into its best eight.  With groups a first pass finds the groups'
// values, and the second goes through those that stay; it computes their keys
// again, which costs less than the shared memory to keep them (2^16 rows of 256
// in eight groups: 42 us against 45).
//
// Bound by instructions, not by memory: 2^20 rows of 256 bfloat16 take 205 us
// (2.9 TB/s) with the half-rate min / max / logic pipe 83% busy, 160
// instructions a row; 2^16 rows of 256 float32, sigmoid, biased, in groups 38
// us (1.9 TB/s), some 380 instructions a row.  A warp a row with its keys in 32
// lanes took 466 and 65 us, comparing exact values alone 876 and 129 us.  Seven
// blocks an SM leave 72 registers a thread: eight (64) take 205 and 43 us, six
// 215 and 41.  The instances of float32 by logit and by softmax spill 8 to 136
// bytes at that (2^16 rows of 256 by logit: 30 us).
//
// Score keys are fixed point: score * f + bias' lies in (4, 6), where floats
// are 2^-21 apart, and their last 22 bits move to the top of the key; 4
// itself is closed.
constexpr u32 kFew = 8, kPiece = 8, kBatch = 32, kFewWarps = 4;

// f: power of two; bias' = bias * f + shift; close: units that may be an error.
struct Scale {
    float f, shift;
    u32 close;
    bool usable;                    // false: a bias range that no scale holds
};

template <class T> struct Bits16;   // ordered 16-bit patterns
template <> struct Bits16<__nv_bfloat16> {
    static constexpr u32 kLowest = 0xFF80FF80, kClosed = 0x007F, kInf = 0xFF80;
    static __device__ __forceinline__ u32 plus_zero(u32 w)
    {
        u32 d;
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(0u));
        return d;
    }
    static __device__ __forceinline__ float value(u32 bits) { return __uint_as_float(bits << 16); }
};
template <> struct Bits16<__half> {
    static constexpr u32 kLowest = 0xFC00FC00, kClosed = 0x03FF, kInf = 0xFC00;
    static __device__ __forceinline__ u32 plus_zero(u32 w)
    {
        u32 d;
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(0u));
        return d;
    }
    static __device__ __forceinline__ float value(u32 bits) { return __half2float(__ushort_as_half((unsigned short)bits)); }
};
template <> struct Bits16<float> {   // not used: keeps the other branch well formed
    static constexpr u32 kLowest = 0xFF800000, kClosed = 0, kInf = 0;
    static __device__ __forceinline__ u32 plus_zero(u32 w) { return w; }
    static __device__ __forceinline__ float value(u32) { return 0.0f; }
};

// Eight consecutive logits as they lie in memory (absent ones: -inf).
template <class T> struct Piece {
    static constexpr int kWords = kPiece * sizeof(T) / 4;
    u32 w[kWords];
    template <bool WHOLE> __device__ __forceinline__ void load(const T *x, u32 n, bool wide)
    {
        if (WHOLE || (wide && n == kPiece)) {
#pragma unroll
            for (int i = 0; i < kWords / 4; i++) {
                const uint4 q = reinterpret_cast<const uint4 *>(x)[i];
                w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
            }
            if (WHOLE) return;
        }
        if (wide && n == kPiece) return;
#pragma unroll
        for (int i = 0; i < kWords; i++) w[i] = Bits16<T>::kLowest;
#pragma unroll
        for (int i = 0; i < (int)kPiece; i++)
            if ((u32)i < n) {
                if constexpr (sizeof(T) == 4) {
                    w[i] = __float_as_uint(x[i]);
                } else {
                    unsigned short v;
                    memcpy(&v, x + i, 2);
                    w[i / 2] = i & 1 ? (w[i / 2] & 0xFFFFu) | (u32)v << 16 : (w[i / 2] & 0xFFFF0000u) | v;
                }
            }
    }
    __device__ __forceinline__ float value(int i) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return Bits16<T>::value(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu);
    }
};

__device__ __forceinline__ float quad_max(float v)
{
    v = fmaxf(v, __shfl_xor_sync(kFull, v, 2));
    return fmaxf(v, __shfl_xor_sync(kFull, v, 1));
}
__device__ __forceinline__ float quad_sum(float v)
{
    v += __shfl_xor_sync(kFull, v, 2);
    return v + __shfl_xor_sync(kFull, v, 1);
}

// A row's words for its groups: their values, and eight each to find them.
__host__ __device__ constexpr u32 few_value_words(u32 groups) { return (groups + 1) / 2 * 2 + 8 * groups; }

// WHOLE: groups are whole batches and loads are wide.
template <class T, int ORDER, bool WHOLE>
__global__ void __launch_bounds__(kFewWarps * 32, 7) k_route_few(const RouteArgs a, const bool wide)
{
    extern __shared__ float shared[];
    __shared__ float lowest[kFewWarps], highest[kFewWarps];
    constexpr bool EXACT = sizeof(T) == 2 && ORDER == kByLogit;
    const u32 E = a.experts, lane = threadIdx.x & 31, q = lane & 3, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const u32 size = E / a.groups, parts = (size + kBatch - 1) / kBatch;
    const bool grouped = a.groups > 1 && a.top_groups < a.groups;
    const u32 batches = parts * a.groups;
    // a warp's own words: route_row's keys or the groups' values
    const u32 value_words = few_value_words(a.groups);
    const u32 values = (max(E, grouped ? 8 * value_words : 0) + 3) & ~3u;
    float *bias = shared;
    u32 *mine = reinterpret_cast<u32 *>(shared + (ORDER == kByLogit ? 0 : (E + 3) & ~3u)) + warp * values;
    // bits of a key that hold the place
    const u32 place = EXACT ? 0xFFFFu : ORDER != kByLogit ? 1023u : (2u << (31 - __clz((E - 1) | 1))) - 1;

    Scale sc = {1.0f, 0.0f, 0, true};
    if (ORDER != kByLogit) {
        float lo = INFINITY, hi = -INFINITY;
        for (u32 e = threadIdx.x; e < E; e += blockDim.x) {
            const float b = a.bias ? a.bias[e] : 0.0f;
            if (open(b)) { lo = fminf(lo, b); hi = fmaxf(hi, b); }
        }
        lo = -group_max<32>(-lo);
        hi = group_max<32>(hi);
        if (lane == 0) { lowest[warp] = lo; highest[warp] = hi; }
        __syncthreads();
        for (u32 i = 0; i < warps; i++) { lo = fminf(lo, lowest[i]); hi = fmaxf(hi, highest[i]); }
        if (!(lo <= hi)) lo = hi = 0.0f;             // no expert is open
        const float range = hi - lo + 1.0f;
        while (range * sc.f > 1.875f && sc.f > 0x1p-20f) sc.f *= 0.5f;
        sc.usable = range * sc.f <= 1.875f && fmaxf(fabsf(lo), fabsf(hi)) * sc.f <= 64.0f;
        sc.shift = 4.0f + 0x1p-6f - lo * sc.f;
        // the approximations' 2e-6, three roundings here, two of the exact value
        sc.close = sc.usable ? 8 + (u32)(fmaxf(fabsf(lo), fabsf(hi)) * sc.f) : 0;
        for (u32 e = threadIdx.x; e < E; e += blockDim.x) {
            const float b = a.bias ? a.bias[e] : 0.0f;
            bias[e] = open(b) ? fmaf(b, sc.f, sc.shift) : __int_as_float(0x7FFFFFFF);
        }
        __syncthreads();
    }
    const int zero = sc.usable ? (int)((sc.shift - 4.0f) * 0x1p21f) : 0;       // a value of 0, in units

    const u64 step = (u64)gridDim.x * warps * 8;
    for (u64 first = ((u64)blockIdx.x * warps + warp) * 8; first < a.tokens; first += step) {
        const u64 row = first + (lane >> 2);
        const bool here = row < a.tokens;
        const T *x = static_cast<const T *>(a.logits) + (here ? row : first) * a.stride;
        float m = -INFINITY, sum = 0.0f, inv = 0.0f;
        // A batch is part p of group g (WHOLE: the groups' batches follow on
        // from one another), the last of a group in four equal shares; this
        // lane's piece starts at expert from().
        struct Batch {
            u32 b, g, p;
        };
        auto share = [&](const Batch &i) { return min(kPiece, (size - i.p * kBatch + 3) / 4); };
        auto from = [&](const Batch &i) {
            return WHOLE ? i.b * kBatch + q * kPiece : i.g * size + i.p * kBatch + q * share(i);
        };
        auto many = [&](const Batch &i) {
            const u32 at = WHOLE ? 0 : i.p * kBatch + q * share(i);
            return WHOLE ? kPiece : at < size ? min(share(i), size - at) : 0u;
        };
        auto after = [&](const Batch &i) {
            return i.p + 1 == parts ? Batch{i.b + 1, i.g + 1, 0} : Batch{i.b + 1, i.g, i.p + 1};
        };
        // calls f(batch, piece) for every batch, the next one's loads under way
        auto each = [&](auto f) {
            Piece<T> now, next;
            Batch i = {0, 0, 0};
            now.template load<WHOLE>(x + from(i), many(i), wide);
            while (i.b < batches) {
                const Batch then = after(i);
                if (then.b < batches) next.template load<WHOLE>(x + from(then), many(then), wide);
                f(i, now);
                now = next;
                i = then;
            }
        };
        auto statistics = [&](bool with_max) {
            if (with_max) {
                each([&](const Batch &, const Piece<T> &v) {
#pragma unroll
                    for (int i = 0; i < (int)kPiece; i++) m = fmaxf(m, v.value(i));           // passes NaN by
                });
                m = quad_max(m);
            }
            each([&](const Batch &, const Piece<T> &v) {
#pragma unroll
                for (int i = 0; i < (int)kPiece; i++) sum += exp2_fast((fmaxf(v.value(i), -INFINITY) - m) * kLog2e);
            });
            sum = quad_sum(sum);
        };
        auto keys_of = [&](const Piece<T> &v, const Batch &at, u32 (&key)[kPiece]) {
            const u32 e0 = from(at), n = many(at);
            if (EXACT) {
                u32 tag = (0xFFFEu - e0) << 16 | (0xFFFFu - e0);
#pragma unroll
                for (int i = 0; i < (int)kPiece / 2; i++) {
                    const u32 z = Bits16<T>::plus_zero(v.w[i % Piece<T>::kWords]);
                    u32 negative;                             // each half's sign in all of its bits
                    asm("prmt.b32 %0, %1, %1, 0xBB99;" : "=r"(negative) : "r"(z));
                    const u32 o = z ^ (negative | 0x80008000u);
                    key[2 * i] = __byte_perm(o, tag, 0x1054);
                    key[2 * i + 1] = __byte_perm(o, tag, 0x3276);
                    tag -= 0x00020002u;
                }
            } else if (ORDER == kByLogit) {
#pragma unroll
                for (int i = 0; i < (int)kPiece; i++)
                    key[i] = (ordered(v.value(i)) & ~place) | ((place - e0 - i) & place);
            } else {
                float add[kPiece];
                if (WHOLE) {
                    *reinterpret_cast<float4 *>(add) = *reinterpret_cast<const float4 *>(bias + e0);
                    *reinterpret_cast<float4 *>(add + 4) = *reinterpret_cast<const float4 *>(bias + e0 + 4);
                } else {
#pragma unroll
                    for (int i = 0; i < (int)kPiece; i++) add[i] = (u32)i < n ? bias[e0 + i] : 0.0f;
                }
                const u32 tag = 1023u - e0;
#pragma unroll
                for (int i = 0; i < (int)kPiece; i++) {
                    const float l = v.value(i);
                    float capped, s;
                    // NaN for -inf, NaN and closed biases; a logit of +inf is open
                    asm("min.NaN.f32 %0, %1, %2;" : "=f"(capped) : "f"(l), "f"(1e30f));
                    if (ORDER == kBySigmoid) s = reciprocal_fast(1.0f + exp2_fast(-l * kLog2e));
                    else s = exp2_fast((l - m) * kLog2e) * inv;
                    const float y = fmaxf(fmaf(s, sc.f, fmaf(capped, 0.0f, add[i])), 4.0f);
                    key[i] = __float_as_uint(y) * 1024u + (WHOLE ? tag - i : (tag - i) & 1023u);
                }
            }
        };
        auto is_open = [&](u32 k) {
            return EXACT ? (k >> 16) > Bits16<T>::kClosed : ORDER == kByLogit ? (k & ~place) > 0x007FFFFFu : k > 1023u;
        };
        // too near each other for these keys to tell
        auto near = [&](u32 greater, u32 less) {
            return !EXACT && (ORDER == kByLogit ? (greater ^ less) <= place : greater - less < (sc.close + 1) * 1024u);
        };
        bool close = ORDER != kByLogit && !sc.usable;
        if (ORDER == kBySoftmax) {
            statistics(true);
            inv = reciprocal_fast(sum);
            close = close || m == INFINITY;
        }

        u32 stays = kFull;
        if (grouped) {
            u32 *value = mine + (lane >> 2) * value_words;
            // a lane's two greatest of its pieces of a group, side by side with the other three's
            uint2 *two = reinterpret_cast<uint2 *>(value + (a.groups + 1) / 2 * 2);
            u32 f = 0, s = 0;
            each([&](const Batch &i, const Piece<T> &v) {
                u32 key[kPiece];
                keys_of(v, i, key);
#pragma unroll
                for (int j = 0; j < (int)kPiece; j++) {
                    if (ORDER != kByLogit) s = max(s, min(f, key[j]));
                    f = max(f, key[j]);
                }
                if (i.p + 1 < parts) return;                 // the group goes on
                two[i.g * 4 + q] = make_uint2(f, s);
                f = s = 0;
            });
            __syncwarp();
            for (u32 g = q; g < a.groups; g += 4) {
                u32 f = 0, s = 0;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const uint2 o = two[g * 4 + j];
                    if (ORDER != kByLogit) s = max(max(s, o.y), min(f, o.x));
                    f = max(f, o.x);
                }
                // scores: units, moved up so that 0 is below every open group
                if (ORDER != kByLogit)
                    f = !is_open(f) ? 0u
                                    : (u32)((int)(f >> 10) + (a.top_two ? is_open(s) ? (int)(s >> 10) : zero : 0)) + (1u << 30);
                value[g] = f;
            }
            __syncwarp();
            u32 mask = 0, in = kFull, out = 0;
            for (u32 g = q; g < a.groups; g += 4) {
                const u32 v = value[g];
                u32 before = 0;
                for (u32 o = 0; o < a.groups; o++) before += value[o] > v || (value[o] == v && o < g);
                if (before < a.top_groups) {
                    mask |= 1u << g;
                    in = min(in, v);
                } else {
                    out = max(out, v);
                }
            }
#pragma unroll
            for (int d = 1; d < 4; d <<= 1) {
                mask |= __shfl_xor_sync(kFull, mask, d);
                in = min(in, __shfl_xor_sync(kFull, in, d));
                out = max(out, __shfl_xor_sync(kFull, out, d));
            }
            stays = mask;
            // the worst that stays against the best that leaves
            if (ORDER == kByLogit) close = close || (!EXACT && is_open(out) && (in ^ out) <= place);
            else close = close || (out && in - out <= 2 * sc.close);
            __syncwarp();
        }

        u32 best[kFew];
#pragma unroll
        for (int i = 0; i < (int)kFew; i++) best[i] = 0;
        auto merge = [&](u32 (&key)[kPiece]) {
            sort_keys<kPiece>(key);
            // the eight greatest of two sorted eights, sorted again
#pragma unroll
            for (int i = 0; i < (int)kFew; i++) best[i] = max(best[i], key[kFew - 1 - i]);
#pragma unroll
            for (int d = 4; d; d >>= 1)
#pragma unroll
                for (int i = 0; i < (int)kFew; i++)
                    if (!(i & d)) order_two(best[i], best[i + d]);
        };
        if (grouped) {
            // each row goes through the groups that stay of its own
            u32 left = stays;
            auto lowest_of = [&](u32 set) { const u32 g = (u32)__ffs(set) - 1; return Batch{g * parts, g, 0}; };
            Batch i = lowest_of(left);
            Piece<T> now, next;
            now.template load<WHOLE>(x + from(i), many(i), wide);
            for (u32 n = a.top_groups * parts; n; n--) {
                Batch then = {i.b + 1, i.g, i.p + 1};
                if (then.p == parts) {
                    left &= left - 1;
                    then = lowest_of(left);
                }
                if (n > 1) next.template load<WHOLE>(x + from(then), many(then), wide);
                u32 key[kPiece];
                keys_of(now, i, key);
                merge(key);
                now = next;
                i = then;
            }
        } else {
            each([&](const Batch &i, const Piece<T> &v) {
                u32 key[kPiece];
                keys_of(v, i, key);
                merge(key);
            });
        }

        // Lane q of the four keeps slots q and q + 4.  One look further tells
        // how sure the last is, unless one lane has given all of its eight.
        u32 got[2] = {0, 0}, last = 0, given = 0;
#pragma unroll
        for (int r = 0; r <= (int)kFew; r++) {
            if ((u32)r >= a.topk + (EXACT ? 0 : 1)) break;
            u32 top = max(best[0], __shfl_xor_sync(kFull, best[0], 2));
            top = max(top, __shfl_xor_sync(kFull, top, 1));
            const bool won = best[0] == top;
            if (r < (int)kFew) given += won;
            else close = close || given == kFew;
#pragma unroll
            for (int i = 0; i + 1 < (int)kFew; i++)
                if (i < (int)kFew - r) best[i] = won ? best[i + 1] : best[i];
            if (r == 0) best[kFew - 1] = won ? 0u : best[kFew - 1];
            if (r == 0 && ORDER == kByLogit)                  // a NaN sorts above infinity
                close = EXACT ? (top >> 16) > Bits16<T>::kInf : close || (top & ~place) > 0xFF800000u;
            if (r > 0) close = close || (near(last, top) && is_open(top));
            last = top;
            if ((u32)r < a.topk && q == (r & 3)) got[(r >> 2) & 1] = top;
        }
        int id[2];
        float logit[2], w[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            id[i] = -1;
            logit[i] = 0.0f;
            if (!is_open(got[i])) continue;
            id[i] = (int)(place - (got[i] & place));
            if (EXACT) {
                const u32 o = got[i] >> 16;
                logit[i] = Bits16<T>::value(o ^ ((o & 0x8000u) ? 0x8000u : 0xFFFFu));
            } else {
                logit[i] = to_float(x[id[i]]);
            }
        }
        if (ORDER == kByLogit && a.softmax && !a.renorm) {
            m = __shfl_sync(kFull, id[0] >= 0 ? logit[0] : -INFINITY, 0, 4);     // slot 0 has the maximum
            close = close || m == INFINITY;
            statistics(false);
        }
        if (a.softmax && a.renorm) {
            const float top = quad_max(fmaxf(id[0] >= 0 ? logit[0] : -INFINITY, id[1] >= 0 ? logit[1] : -INFINITY));
#pragma unroll
            for (int i = 0; i < 2; i++) w[i] = id[i] >= 0 ? exp_below(logit[i], top) : 0.0f;
        } else {
#pragma unroll
            for (int i = 0; i < 2; i++)
                w[i] = id[i] < 0 ? 0.0f : a.softmax ? exp_below(logit[i], m) / sum : sigmoid(logit[i]);
        }
        if (a.renorm) {
            float total = quad_sum(w[0] + w[1]);
            const bool tiny = !a.softmax && total < kTinySum;
            if (__any_sync(kFull, tiny)) {
                const float top = quad_max(fmaxf(id[0] >= 0 ? logit[0] : -INFINITY, id[1] >= 0 ? logit[1] : -INFINITY));
#pragma unroll
                for (int i = 0; i < 2; i++)
                    if (tiny) w[i] = id[i] >= 0 ? tiny_score(logit[i], top) : 0.0f;
                total = quad_sum(w[0] + w[1]);
            }
#pragma unroll
            for (int i = 0; i < 2; i++) w[i] = total > 0.0f ? w[i] / total : 0.0f;
        }
        const u32 again = __ballot_sync(kFull, close && here);
        const bool redo = (again >> (lane & ~3u)) & 15;
#pragma unroll
        for (int i = 0; i < 2; i++)
            if (here && !redo && q + 4 * i < a.topk) {
                a.ids[row * a.topk + q + 4 * i] = id[i];
                a.weights[row * a.topk + q + 4 * i] = w[i] * a.scale;
            }
        for (u32 rows = __ballot_sync(kFull, redo && q == 0); rows; rows &= rows - 1)
            route_row<T, ORDER>(a, first + (__ffs(rows) - 1) / 4, mine);
        __syncwarp();
    }
}

// Sizes that no lane layout holds: every row by its exact values.  2^16 rows of
// 960 float32 logits in 12 groups, 9 slots: 354 us (in 8 groups k_route takes 373).
template <class T, int ORDER> __global__ void __launch_bounds__(kRouteWarps * 32) k_route_rows(const RouteArgs a)
{
    extern __shared__ u32 keys[];
    const u32 warp = threadIdx.x >> 5;
    const u64 step = (u64)gridDim.x * kRouteWarps;
    for (u64 row = (u64)blockIdx.x * kRouteWarps + warp; row < a.tokens; row += step)
        route_row<T, ORDER>(a, row, keys + warp * a.experts);
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

// The gradient of a row.  With G the slots' gradients laid out over the
// experts, and p the softmax: dx = scale p (G - sum G p), dense.  In the
// other forms only the chosen experts' logits matter and the rest is zeros.
// L lanes share a row, V experts a lane: eight neighbours of every 8 L, whose
// sums do not depend on how the row lies in memory.  G, or the slots' results,
// are scattered into the row's floats in shared memory; rows that 16-byte
// accesses do not fit (not WIDE) come and go through there too.  The row is
// read once and held in registers: 2^16 rows of 256 float32 take 30.6 us, 4.5
// TB/s (three passes over memory took 63).
constexpr u32 kGradWarps = 8;

template <class T, int L, int V, bool WIDE>
__global__ void __launch_bounds__(kGradWarps * 32) k_route_grad(const RouteGradArgs a)
{
    extern __shared__ float grads[];
    constexpr u32 kRows = 32 / L;
    const u32 E = a.experts, pitch = (E + 7) & ~7u, lane = threadIdx.x & 31, sub = lane & (L - 1);
    float *G = grads + (threadIdx.x / L) * pitch;
    const bool dense = a.softmax && !a.renorm;
    auto place = [&](int i) { return (i / 8) * (L * 8) + sub * 8 + i % 8; };
    // this lane's experts out of the row in shared memory, whose pitch is a whole number of eights
    auto gather = [&](float (&at)[V]) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4 *>(at + i) =
                (u32)place(i) < pitch ? *reinterpret_cast<const float4 *>(G + place(i)) : make_float4(0, 0, 0, 0);
    };
    const u64 step = (u64)gridDim.x * kGradWarps * kRows;
    for (u64 first = ((u64)blockIdx.x * kGradWarps + (threadIdx.x >> 5)) * kRows; first < a.tokens; first += step) {
        const u64 row = first + lane / L;
        const bool here = row < a.tokens;
        const T *x = static_cast<const T *>(a.logits) + (here ? row : first) * a.stride;
        alignas(16) float v[V];
        if (dense) {
            if (WIDE) {
#pragma unroll
                for (int i = 0; i < V; i += 8) {
                    Piece<T> piece;
                    piece.template load<false>(x + place(i), (u32)place(i) < E ? 8 : 0, true);
#pragma unroll
                    for (int j = 0; j < 8; j++) v[i + j] = piece.value(j);
                }
            } else {
                for (u32 e = sub; e < pitch; e += L) G[e] = e < E ? to_float(x[e]) : -INFINITY;
                __syncwarp();
                gather(v);
#pragma unroll
                for (int i = 0; i < V; i++)
                    if ((u32)place(i) >= E) v[i] = -INFINITY;
                __syncwarp();
            }
        }
        int id = here && sub < a.topk ? a.ids[row * a.topk + sub] : -1;
        if ((u32)id >= E) id = -1;
        const float g = id >= 0 ? a.dweights[row * a.topk + sub] : 0.0f;
        for (u32 e = sub * 4; e < pitch; e += L * 4) *reinterpret_cast<float4 *>(G + e) = make_float4(0, 0, 0, 0);
        __syncwarp();
        if (dense) {
            if (id >= 0) G[id] = g;
            float m = -INFINITY, sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < V; i++) m = fmaxf(m, v[i]);          // passes NaN by
            m = group_max<L>(m);
            __syncwarp();
            alignas(16) float at[V];
            gather(at);
#pragma unroll
            for (int i = 0; i < V; i++) {
                v[i] = !open(v[i]) ? 0.0f : v[i] == m ? 1.0f : exp2_fast((v[i] - m) * kLog2e);
                sum += v[i];
                dot += v[i] * at[i];
            }
            sum = group_sum<L>(sum);
            dot = group_sum<L>(dot);
            const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
            dot *= inv;
#pragma unroll
            for (int i = 0; i < V; i++) v[i] = v[i] * inv * (at[i] - dot) * a.scale;
        } else {
            const float l = id >= 0 ? to_float(x[id]) : -INFINITY;
            float d;
            if (a.softmax) {
                const float best = group_max<L>(l);
                float w = id >= 0 ? exp_below(l, best) : 0.0f;
                const float sum = group_sum<L>(w);
                w = sum > 0.0f ? w / sum : 0.0f;
                d = w * (g - group_sum<L>(g * w));
            } else {
                // the score s and its complement (1 - s would end at s's last bit) from one exponential
                const float e = expf(-fabsf(l)), n = 1.0f + e;
                float s = (l < 0.0f ? e : 1.0f) / n;
                d = g;
                if (a.renorm) {
                    float sum = group_sum<L>(s);
                    const bool tiny = sum < kTinySum;
                    if (__any_sync(kFull, tiny)) {
                        const float best = group_max<L>(l);
                        if (tiny) s = id >= 0 ? tiny_score(l, best) : 0.0f;
                        sum = group_sum<L>(s);
                    }
                    const float dot = group_sum<L>(g * s);
                    d = sum > 0.0f ? (g - dot / sum) / sum : 0.0f;
                }
                d *= s * ((l < 0.0f ? 1.0f : e) / n);
            }
            if (id >= 0) G[id] = d * a.scale;
            __syncwarp();
            gather(v);
        }
        __syncwarp();
        T *dx = static_cast<T *>(a.dlogits) + row * E;
        if (WIDE) {
#pragma unroll
            for (int i = 0; i < V; i += 8) {
                if ((u32)place(i) >= E || !here) continue;
                T out[8];
#pragma unroll
                for (int j = 0; j < 8; j++) out[j] = from_float<T>(v[i + j]);
#pragma unroll
                for (int j = 0; j < (int)sizeof(T) / 2; j++) {
                    uint4 q;
                    memcpy(&q, reinterpret_cast<const char *>(out) + 16 * j, 16);
                    reinterpret_cast<uint4 *>(dx + place(i))[j] = q;
                }
            }
        } else {
            if (dense)
#pragma unroll
                for (int i = 0; i < V; i += 4)
                    if ((u32)place(i) < pitch) *reinterpret_cast<float4 *>(G + place(i)) = *reinterpret_cast<float4 *>(v + i);
            __syncwarp();
            if (here)
                for (u32 e = sub; e < E; e += L) dx[e] = from_float<T>(G[e]);
            __syncwarp();
        }
    }
}

template <class T, int L, int V> int run_route_grad(const RouteGradArgs &a, cudaStream_t stream)
{
    constexpr u32 kRowsABlock = kGradWarps * 32 / L;
    const u32 sms = sm_count(), smem = kRowsABlock * ((a.experts + 7) & ~7u) * 4;
    if (!sms) return MV_ECUDA;
    const bool wide = a.experts % 8 == 0 && aligned(a.logits, 16) && a.stride * sizeof(T) % 16 == 0 && aligned(a.dlogits, 16);
    const u32 blocks = (u32)std::fmin((double)((a.tokens + kRowsABlock - 1) / kRowsABlock), 16.0 * sms);
    return launch(wide ? k_route_grad<T, L, V, true> : k_route_grad<T, L, V, false>, blocks, kGradWarps * 32, smem, stream, a);
}

// The smallest shape that holds the experts, and a lane to a slot.
template <class T> int run_route_grad(const RouteGradArgs &a, cudaStream_t stream)
{
    if (a.experts <= 64 && a.topk <= 8) return run_route_grad<T, 8, 8>(a, stream);
    if (a.experts <= 128 && a.topk <= 16) return run_route_grad<T, 16, 8>(a, stream);
    if (a.experts <= 256) return run_route_grad<T, 32, 8>(a, stream);
    if (a.experts <= 512) return run_route_grad<T, 32, 16>(a, stream);
    return run_route_grad<T, 32, 32>(a, stream);
}

template <class T, int ORDER> int run_route_few(const RouteArgs &a, cudaStream_t stream)
{
    const u32 sms = sm_count(), size = a.experts / a.groups;
    if (!sms) return MV_ECUDA;
    const bool grouped = a.groups > 1 && a.top_groups < a.groups;
    const bool wide = aligned(a.logits, 16) && a.stride * sizeof(T) % 16 == 0 && (a.groups == 1 || size % kPiece == 0);
    const u32 rows = grouped ? 8 * few_value_words(a.groups) : 0, values = ((rows > a.experts ? rows : a.experts) + 3) & ~3u;
    // Eight rows a warp: short batches spread over the SMs in small blocks.
    const u64 warps = (a.tokens + 7) / 8;
    const u32 a_block = warps < 16ull * sms ? 1 : kFewWarps;
    const u32 smem = 4 * ((ORDER == kByLogit ? 0 : (a.experts + 3) & ~3u) + a_block * values);
    const u32 blocks = (u32)std::fmin((double)((warps + a_block - 1) / a_block), 64.0 * sms);
    const auto kernel = size % kBatch == 0 && wide ? k_route_few<T, ORDER, true> : k_route_few<T, ORDER, false>;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return MV_ECUDA;
    return launch(kernel, blocks, a_block * 32, smem, stream, a, wide);
}

// Blocks of a warp a row (0: no device).
inline u32 route_blocks(const RouteArgs &a)
{
    return (u32)std::fmin((double)((a.tokens + kRouteWarps - 1) / kRouteWarps), 8.0 * sm_count());
}

template <class T, int ORDER, int V> int run_route(const RouteArgs &a, const Shares &sh, cudaStream_t stream)
{
    const u32 blocks = route_blocks(a);
    if (!blocks) return MV_ECUDA;
    const bool exact = sizeof(T) == 2 && ORDER == kByLogit;
    return launch(k_route<T, ORDER, V>, blocks, kRouteWarps * 32, exact ? 0 : kRouteWarps * a.experts * 4,
                  stream, a, sh);
}

// Up to eight slots by four lanes a row; more by a warp a row, in the
// smallest shape that gives every group whole lanes.  A batch of up to 16 rows
// an SM goes by a warp a row too, where what counts is one row's latency (256
// experts: one row with groups 3.2 us against 8.6, 2432 rows 8.6 against 13.8,
// 9728 rows 15.7 against 14.9; without groups 2.2 against 3.3, 2.9 against 3.8,
// 6.2 against 4.3) - unless the weights need a sum over the row, whose order
// is that of the lanes.
template <class T, int ORDER> int run_route(const RouteArgs &a, cudaStream_t stream)
{
    const bool sums = a.softmax && (ORDER == kBySoftmax || !a.renorm);
    if (a.topk <= kFew && (sums || a.tokens > 16ull * sm_count() || a.experts > 256)) return run_route_few<T, ORDER>(a, stream);
    auto fits = [&](u32 V, Shares &sh) {
        sh.shift = 0;
        while (a.groups << (sh.shift + 1) <= 32) sh.shift++;
        sh.size = a.experts / a.groups;
        sh.per = a.groups == 1 ? V : (sh.size + (1u << sh.shift) - 1) >> sh.shift;
        if (sh.per > V || sh.size > sh.per << sh.shift) return false;
        sh.wide = sh.per == V && aligned(a.logits, 16) && a.stride * sizeof(T) % 16 == 0 &&
                  (a.groups == 1 || sh.size * sizeof(T) % 16 == 0);
        return true;
    };
    Shares sh;
    if (fits(8, sh)) return run_route<T, ORDER, 8>(a, sh, stream);
    if (a.topk <= kFew) return run_route_few<T, ORDER>(a, stream);
    if (fits(16, sh)) return run_route<T, ORDER, 16>(a, sh, stream);
    if (fits(32, sh)) return run_route<T, ORDER, 32>(a, sh, stream);
    // More than eight slots of large groups, 3, 5 to 7, 9 to 15 or 17 to 31 of
    // them: some lanes would have none and the others more than 32 experts.
    if (a.top_groups == a.groups) {                  // groups decide nothing
        RouteArgs whole = a;
        whole.groups = whole.top_groups = 1;
        return run_route<T, ORDER>(whole, stream);
    }
    const u32 blocks = route_blocks(a);
    if (!blocks) return MV_ECUDA;
    return launch(k_route_rows<T, ORDER>, blocks, kRouteWarps * 32, kRouteWarps * a.experts * 4, stream, a);
}

template <class T> int run_route(const RouteArgs &a, Order order, cudaStream_t stream)
{
    if (order == kByLogit) return run_route<T, kByLogit>(a, stream);
    if (order == kBySigmoid) return run_route<T, kBySigmoid>(a, stream);
    return run_route<T, kBySoftmax>(a, stream);
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
