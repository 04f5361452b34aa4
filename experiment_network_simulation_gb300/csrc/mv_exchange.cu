// Token counts of an expert-parallel exchange (mv_exchange in include/mv.h).
#include "mv_moe.cuh"

namespace mvmoe {

struct ExchangeArgs {
    const int32_t *ids, *place;
    const int64_t *starts;          // sources + 1 token offsets, or null: even shares
    int32_t *load, *sent;
    u64 batches, tokens;
    u32 topk, experts, sources, ranks;
    bool once;
};

constexpr u32 kExchangeThreads = 256;

// One block a (batch, source): counts in shared memory, one row written.
__global__ void __launch_bounds__(kExchangeThreads) k_exchange(const ExchangeArgs a)
{
    extern __shared__ int32_t counts[];
    int32_t *row = counts, *load = counts + a.ranks;
    const u64 item = blockIdx.x, b = item / a.sources, s = item % a.sources;
    for (u32 i = threadIdx.x; i < a.ranks + a.experts; i += kExchangeThreads) counts[i] = 0;
    __syncthreads();
    u64 t0 = s * (a.tokens / a.sources), t1 = t0 + a.tokens / a.sources;
    if (a.starts) {
        t0 = min((u64)max(a.starts[s], (int64_t)0), a.tokens);
        t1 = min((u64)max(a.starts[s + 1], (int64_t)0), a.tokens);
    }
    for (u64 t = t0 + threadIdx.x; t < t1; t += kExchangeThreads) {
        const int32_t *ids = a.ids + (b * a.tokens + t) * a.topk;
        int to[kMaxTopk];
        for (u32 j = 0; j < a.topk; j++) {
            const u32 e = (u32)ids[j];
            to[j] = -1;
            if (e >= a.experts) continue;
            atomicAdd(&load[e], 1);
            const u32 d = (u32)a.place[e];
            bool count = d < a.ranks;
            if (a.once)
                for (u32 i = 0; i < j; i++) count = count && to[i] != (int)d;
            to[j] = (int)d;
            if (count) atomicAdd(&row[d], 1);
        }
    }
    __syncthreads();
    for (u32 i = threadIdx.x; i < a.ranks; i += kExchangeThreads)
        a.sent[item * a.ranks + i] = row[i];
    for (u32 i = threadIdx.x; i < a.experts; i += kExchangeThreads)
        if (load[i]) atomicAdd(&a.load[b * a.experts + i], load[i]);
}

}  // namespace mvmoe

using namespace mvmoe;

extern "C" int mv_exchange(const mv_exchange_desc *d, void *stream)
{
    if (!d || !d->experts || !d->topk || !d->sources || !d->ranks) return MV_EINVAL;
    if (d->experts > kMaxExperts || d->topk > kMaxTopk || d->ranks > MV_MOE_MAX_RANKS ||
        d->sources > (1u << 24) || d->batches > (1u << 24) || d->tokens > (1ull << 31) - 1 ||
        d->batches * d->sources > (1ull << 31) - 1 ||
        d->tokens * d->topk > (1ull << 31) - 1)           // a count is a 32-bit number
        return MV_EOVERFLOW;
    if (!d->starts && d->tokens % d->sources) return MV_EINVAL;
    if (d->batches == 0) return MV_OK;
    if ((d->tokens && !d->ids) || !d->place || !d->load || !d->sent || !aligned(d->ids, 4) ||
        !aligned(d->place, 4) || !aligned(d->starts, 8) || !aligned(d->load, 4) || !aligned(d->sent, 4))
        return MV_EINVAL;
    ExchangeArgs a;
    a.ids = d->ids;
    a.place = d->place;
    a.starts = d->starts;
    a.load = d->load;
    a.sent = d->sent;
    a.batches = d->batches;
    a.tokens = d->tokens;
    a.topk = d->topk;
    a.experts = d->experts;
    a.sources = d->sources;
    a.ranks = d->ranks;
    a.once = d->once != 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(a.load, 0, 4 * d->batches * d->experts, s) != cudaSuccess) return MV_ECUDA;
    return launch(k_exchange, dim3((u32)(d->batches * d->sources)), kExchangeThreads,
                  4 * (a.ranks + a.experts), s, a);
}
