// Token counts of an expert-parallel exchange (mv_exchange in include/mv.h).
#include "mv_moe.cuh"

namespace mvmoe {

struct ExchangeArgs {
    const int32_t *ids, *place;
    const int64_t *starts;          // sources + 1 token offsets, or null: even shares
    int32_t *load, *sent;
    u64 tokens, items;              // items: batches * sources * splits
    u32 topk, experts, sources, ranks;
    u32 splits;                     // parts a source's tokens are cut into; their rows meet in `sent`
    u32 count_blocks;               // the first blocks count a batch's load each; 0: the items do
    u32 share;                      // items a warp
    u32 warps;                      // warps a block
};

// Token t0 .. t1 of an item: part `split` of a source's tokens.
__device__ __forceinline__ void item_tokens(const ExchangeArgs &a, u32 source, u32 split, u64 &t0, u64 &t1)
{
    t0 = source * (a.tokens / a.sources);
    t1 = t0 + a.tokens / a.sources;
    if (a.starts) {
        t0 = min((u64)max(a.starts[source], (int64_t)0), a.tokens);
        t1 = max(t0, min((u64)max(a.starts[source + 1], (int64_t)0), a.tokens));
    }
    const u64 n = t1 - t0;
    t1 = t0 + n * (split + 1) / a.splits;
    t0 += n * split / a.splits;
}

// A warp takes a run of items, one source's tokens (or a part of them) at a
// time, and counts in shared memory of its own: no block ever waits.  Lanes
// read neighbouring slots, so that a token's first choices, often the same
// popular expert, meet in few lanes of one counting step.
//
// Without ONCE an item's slots are counted by expert, one atomic a slot; the
// experts' counts then make the row of ranks and the load.  With ONCE a
// token's lanes look for equal ranks among themselves and the first counts.
constexpr u32 kExchangeWarps = 8;
constexpr int kAhead = 8;               // loads of ids under way a lane

template <bool ONCE> __global__ void __launch_bounds__(kExchangeWarps * 32) k_exchange(const ExchangeArgs a)
{
    extern __shared__ int32_t shared[];
    const u32 lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.experts;
    if (blockIdx.x < a.count_blocks) {                  // the load of one batch
        for (u32 e = threadIdx.x; e < E; e += blockDim.x) shared[e] = 0;
        __syncthreads();
        const int32_t *ids = a.ids + (u64)blockIdx.x * a.tokens * a.topk;
        for (u64 i = threadIdx.x; i < a.tokens * a.topk; i += blockDim.x) {
            const u32 e = (u32)ids[i];
            if (e < E) atomicAdd(&shared[e], 1);
        }
        __syncthreads();
        for (u32 e = threadIdx.x; e < E; e += blockDim.x) a.load[(u64)blockIdx.x * E + e] = shared[e];
        return;
    }
    const bool loads = a.count_blocks == 0;
    int32_t *place = shared, *row = shared + E + warp * (a.ranks + 2 * E);
    int32_t *hist = row + a.ranks, *sum = hist + E;      // an item's experts; the batch's so far
    for (u32 e = threadIdx.x; e < E; e += blockDim.x) place[e] = a.place[e];
    for (u32 e = lane; e < E; e += 32) hist[e] = sum[e] = 0;
    __syncthreads();

    const u64 first = ((u64)(blockIdx.x - a.count_blocks) * a.warps + warp) * a.share;
    const u64 last = min(first + a.share, a.items);
    u64 at_batch = ~0ull;
    auto flush = [&]() {
        if (!loads || at_batch == ~0ull) return;
        int32_t *counts = ONCE ? hist : sum;
        __syncwarp();
        for (u32 e = lane; e < E; e += 32) {
            if (counts[e]) atomicAdd(&a.load[at_batch * E + e], counts[e]);
            counts[e] = 0;
        }
        __syncwarp();
    };
    for (u64 item = first; item < last; item++) {
        const u64 pair = item / a.splits, b = pair / a.sources;
        if (b != at_batch) {
            flush();
            at_batch = b;
        }
        u64 t0, t1;
        item_tokens(a, (u32)(pair % a.sources), (u32)(item % a.splits), t0, t1);
        for (u32 d = lane; d < a.ranks; d += 32) row[d] = 0;
        __syncwarp();
        const int32_t *ids = a.ids + (b * a.tokens + t0) * a.topk;
        const u64 slots = (t1 - t0) * a.topk;
        if (ONCE) {
            const u32 used = 32 / a.topk * a.topk, token = lane / a.topk;
            for (u64 i = 0; i < slots; i += kAhead * used) {
                u32 id[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; j++) {
                    const u64 at = i + j * used + lane;
                    id[j] = lane < used && at < slots ? (u32)ids[at] : kFull;
                }
#pragma unroll
                for (int j = 0; j < kAhead; j++) {
                    if (i + j * used >= slots) break;
                    u32 d = kFull;
                    if (id[j] < E) {
                        if (loads) atomicAdd(&hist[id[j]], 1);
                        d = (u32)place[id[j]];
                    }
                    // ranks are below 2^13; what counts nowhere matches nothing
                    const u32 same = __match_any_sync(kFull, d < a.ranks ? token << 16 | d : 1u << 31 | lane);
                    if (d < a.ranks && lane + 1 == (u32)__ffs(same)) atomicAdd(&row[d], 1);
                }
            }
        } else {
            for (u64 i = lane; i < slots; i += kAhead * 32) {
                u32 id[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; j++) id[j] = i + j * 32 < slots ? (u32)ids[i + j * 32] : kFull;
#pragma unroll
                for (int j = 0; j < kAhead; j++)
                    if (id[j] < E) atomicAdd(&hist[id[j]], 1);
            }
            __syncwarp();
            for (u32 e = lane; e < E; e += 32) {
                const int32_t n = hist[e];
                const u32 d = (u32)place[e];
                hist[e] = 0;
                if (!n) continue;
                sum[e] += n;
                if (d < a.ranks) atomicAdd(&row[d], n);
            }
        }
        __syncwarp();
        int32_t *sent = a.sent + pair * a.ranks;
        for (u32 d = lane; d < a.ranks; d += 32) {
            if (a.splits == 1) sent[d] = row[d];
            else if (row[d]) atomicAdd(&sent[d], row[d]);
        }
        __syncwarp();
    }
    flush();
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
    a.tokens = d->tokens;
    a.topk = d->topk;
    a.experts = d->experts;
    a.sources = d->sources;
    a.ranks = d->ranks;
    const u32 sms = sm_count();
    if (!sms) return MV_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Few sources with many tokens are cut, down to 256 tokens a part: the
    // device has room for some 16 warps an SM.
    const u64 pairs = d->batches * d->sources, room = 16ull * sms, mean = d->tokens / d->sources;
    a.splits = 1;
    if (pairs < room && mean > 256) {
        const u64 want = (room + pairs - 1) / pairs, can = (mean + 255) / 256;
        a.splits = (u32)(want < can ? want : can);
    }
    a.items = pairs * a.splits;
    // A small batch's load is counted by a block of its own, which saves
    // clearing it; a large one's by the warps that have read the ids anyway.
    a.count_blocks = d->tokens * d->topk <= 32768 && d->batches <= 4 * sms ? (u32)d->batches : 0;
    const u32 a_warp = 4 * (a.ranks + 2 * a.experts);
    a.warps = kExchangeWarps;
    while (a.warps > 1 && 4 * a.experts + a.warps * a_warp > 72 * 1024) a.warps /= 2;
    const u32 smem = 4 * a.experts + a.warps * a_warp, held = 227 * 1024 / (smem + 1024);
    const u64 resident = (u64)sms * a.warps * (held < 64 / a.warps ? held : 64 / a.warps);
    a.share = (u32)((a.items + 2 * resident - 1) / (2 * resident));
    if (!a.count_blocks && cudaMemsetAsync(a.load, 0, 4 * d->batches * d->experts, s) != cudaSuccess) return MV_ECUDA;
    if (a.splits > 1 && cudaMemsetAsync(a.sent, 0, 4 * pairs * a.ranks, s) != cudaSuccess) return MV_ECUDA;
    const auto kernel = d->once ? k_exchange<true> : k_exchange<false>;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return MV_ECUDA;
    const u64 a_block = (u64)a.share * a.warps;
    return launch(kernel, dim3((u32)(a.count_blocks + (a.items + a_block - 1) / a_block)), a.warps * 32, smem, s, a);
}
