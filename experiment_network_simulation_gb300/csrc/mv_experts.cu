// The routed experts' SwiGLU products with 4-bit weights (mv_experts in
// include/mv.h).
#include <cmath>

#include "mv_moe.cuh"

namespace mvmoe {

struct ExpertArgs {
    const void *x;
    const int32_t *ids;
    const float *weights;
    const uint8_t *w13, *w2;
    const void *s13, *s2;
    void *y;
    float *h;                       // [pairs, inner]
    u64 tokens, stride;
    u32 topk, experts, hidden, inner, group;
};

constexpr u32 kExpertWarps = 8;

// Sum over a row of packed weights: (q - 8) x scale x value, by one warp.
template <class T, class X>
__device__ float dot_row(const uint8_t *q, const T *scale, const X *v, u32 n, u32 group)
{
    float sum = 0.0f;
    for (u32 k = (threadIdx.x & 31) * 2; k < n; k += 64) {
        const u32 b = q[k >> 1];
        const float s = to_float(scale[k / group]);
        sum += s * ((float)((int)(b & 15) - 8) * to_float(v[k]) +
                    (float)((int)(b >> 4) - 8) * to_float(v[k + 1]));
    }
    return group_sum<32>(sum);
}

// h = silu(W1 x) (W3 x) of one (token, slot) a grid row, one inner row a warp.
template <class T> __global__ void __launch_bounds__(kExpertWarps * 32) k_gate_up(const ExpertArgs a)
{
    for (u64 p = blockIdx.y; p < a.tokens * a.topk; p += gridDim.y) {
        const u32 e = (u32)a.ids[p];
        if (e >= a.experts) continue;
        const T *x = static_cast<const T *>(a.x) + p / a.topk * a.stride;
        for (u32 i = blockIdx.x * kExpertWarps + (threadIdx.x >> 5); i < a.inner;
             i += gridDim.x * kExpertWarps) {
            const u64 r1 = (u64)e * 2 * a.inner + i, r3 = r1 + a.inner;
            const T *s = static_cast<const T *>(a.s13);
            const u32 groups = a.hidden / a.group;
            const float g = dot_row(a.w13 + r1 * (a.hidden / 2), s + r1 * groups, x, a.hidden, a.group);
            const float u = dot_row(a.w13 + r3 * (a.hidden / 2), s + r3 * groups, x, a.hidden, a.group);
            if ((threadIdx.x & 31) == 0) a.h[p * a.inner + i] = g / (1.0f + expf(-g)) * u;
        }
    }
}

// y = sum over the slots, in their order, of weight x (W2 h).
template <class T> __global__ void __launch_bounds__(kExpertWarps * 32) k_down(const ExpertArgs a)
{
    for (u64 t = blockIdx.y; t < a.tokens; t += gridDim.y)
        for (u32 i = blockIdx.x * kExpertWarps + (threadIdx.x >> 5); i < a.hidden;
             i += gridDim.x * kExpertWarps) {
            float y = 0.0f;
            for (u64 p = t * a.topk; p < (t + 1) * a.topk; p++) {
                const u32 e = (u32)a.ids[p];
                if (e >= a.experts) continue;
                const u64 r = (u64)e * a.hidden + i;
                y += a.weights[p] * dot_row(a.w2 + r * (a.inner / 2),
                                            static_cast<const T *>(a.s2) + r * (a.inner / a.group),
                                            a.h + p * a.inner, a.inner, a.group);
            }
            if ((threadIdx.x & 31) == 0) static_cast<T *>(a.y)[t * a.hidden + i] = from_float<T>(y);
        }
}

int check(const mv_experts_desc *d)
{
    if (!d || !d->experts || !d->topk || (d->dtype != MV_F16 && d->dtype != MV_BF16) ||
        (d->group != 32 && d->group != 64 && d->group != 128) || !d->hidden || !d->inner ||
        d->hidden % d->group || d->inner % d->group)
        return MV_EINVAL;
    if (d->experts > kMaxExperts || d->topk > kMaxTopk || d->hidden > (1u << 20) ||
        d->inner > (1u << 20) || d->tokens > (1u << 24) || d->row_stride > (1ull << 31))
        return MV_EOVERFLOW;
    return MV_OK;
}

template <class T> int run_experts(const ExpertArgs &a, cudaStream_t stream)
{
    const u32 gi = (a.inner + kExpertWarps - 1) / kExpertWarps, gh = (a.hidden + kExpertWarps - 1) / kExpertWarps;
    const u32 gp = (u32)std::fmin((double)(a.tokens * a.topk), 65535.0), gt = (u32)std::fmin((double)a.tokens, 65535.0);
    int rc = launch(k_gate_up<T>, dim3(gi, gp), kExpertWarps * 32, 0, stream, a);
    if (rc == MV_OK) rc = launch(k_down<T>, dim3(gh, gt), kExpertWarps * 32, 0, stream, a);
    return rc;
}

}  // namespace mvmoe

using namespace mvmoe;

extern "C" int mv_experts_workspace_bytes(const mv_experts_desc *d, uint64_t *bytes)
{
    if (!bytes) return MV_EINVAL;
    *bytes = 0;
    const int rc = check(d);
    if (rc != MV_OK) return rc;
    *bytes = (4 * d->tokens * d->topk * d->inner + 255) / 256 * 256;
    return MV_OK;
}

extern "C" int mv_experts(const mv_experts_desc *d, void *workspace, uint64_t ws_bytes, void *stream)
{
    uint64_t need = 0;
    const int rc = mv_experts_workspace_bytes(d, &need);
    if (rc != MV_OK || d->tokens == 0) return rc;
    if (!d->x || !d->ids || !d->weights || !d->w13 || !d->s13 || !d->w2 || !d->s2 || !d->y ||
        !workspace || d->row_stride < d->hidden || d->row_stride % 8 || !aligned(d->x, 16) ||
        !aligned(d->ids, 4) || !aligned(d->weights, 4) || !aligned(d->w13, 16) ||
        !aligned(d->s13, 16) || !aligned(d->w2, 16) || !aligned(d->s2, 16) || !aligned(d->y, 16) ||
        !aligned(workspace, 256))
        return MV_EINVAL;
    if (ws_bytes < need) return MV_ENOMEM;
    ExpertArgs a;
    a.x = d->x;
    a.ids = d->ids;
    a.weights = d->weights;
    a.w13 = d->w13;
    a.s13 = d->s13;
    a.w2 = d->w2;
    a.s2 = d->s2;
    a.y = d->y;
    a.h = static_cast<float *>(workspace);
    a.tokens = d->tokens;
    a.stride = d->row_stride;
    a.topk = d->topk;
    a.experts = d->experts;
    a.hidden = d->hidden;
    a.inner = d->inner;
    a.group = d->group;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return d->dtype == MV_F16 ? run_experts<__half>(a, s) : run_experts<__nv_bfloat16>(a, s);
}
