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

// Tokens t0 .. t1 of the sources first .. last.
__device__ __forceinline__ void source_tokens(const ExchangeArgs &a, u32 first, u32 last, u64 &t0, u64 &t1)
{
    t0 = first * (a.tokens / a.sources);
    t1 = (last + 1) * (a.tokens / a.sources);
    if (a.starts) {
        t0 = min((u64)max(a.starts[first], (int64_t)0), a.tokens);
        t1 = max(t0, min((u64)max(a.starts[last + 1], (int64_t)0), a.tokens));
    }
}

// Those of an item: part `split` of a source's tokens.
__device__ __forceinline__ void item_tokens(const ExchangeArgs &a, u32 source, u32 split, u64 &t0, u64 &t1)
{
    source_tokens(a, source, source, t0, t1);
    const u64 n = t1 - t0;
    t1 = t0 + n * (split + 1) / a.splits;
    t0 += n * split / a.splits;
}

// Counts slots first, first + step, ... (a warp's 32, or what whole tokens
// fill of them, a step) of a source's `slots`.  Lanes read neighbouring slots,
// so that a token's first choices, often the same popular expert, meet in few
// lanes of one counting step.
//
// Without ONCE slots are counted by expert, one atomic a slot; the experts'
// counts then make the row of ranks and the load.  With ONCE a token's lanes
// look for equal ranks among themselves and the first counts.
constexpr u32 kExchangeWarps = 8;
constexpr int kAhead = 8;               // loads of ids under way a lane

template <bool ONCE>
__device__ __forceinline__ void count_slots(const ExchangeArgs &a, const int32_t *ids, u64 slots, u64 first, u64 step,
                                            bool loads, const int32_t *place, int32_t *hist, int32_t *row)
{
    const u32 lane = threadIdx.x & 31, used = ONCE ? 32 / a.topk * a.topk : 32, token = lane / a.topk;
    for (u64 i = first; i < slots; i += kAhead * step) {
        u32 id[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            const u64 at = i + j * step + lane;
            id[j] = lane < used && at < slots ? (u32)ids[at] : kFull;
        }
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            if (i + j * step >= slots) break;
            if (id[j] < a.experts && (loads || !ONCE)) atomicAdd(&hist[id[j]], 1);
            if (!ONCE) continue;
            const u32 d = id[j] < a.experts ? (u32)place[id[j]] : kFull;
            // ranks are below 2^13; what counts nowhere matches nothing
            const u32 same = __match_any_sync(kFull, d < a.ranks ? token << 16 | d : 1u << 31 | lane);
            if (d < a.ranks && lane + 1 == (u32)__ffs(same)) atomicAdd(&row[d], 1);
        }
    }
}

// Many sources: a warp takes a run of items, one source's tokens at a time,
// and counts in shared memory of its own: no warp waits for another.  64
// batches of 512 sources x 128 tokens x 8 slots to 512 ranks: 52 us, 3.9 TB/s.
// A block a source with two shared-memory atomics a slot took 128 us, so they
// are held to be the bound; no counter shows it.  With ONCE, two atomics and a
// match a slot: 277 us.  A long source is one warp's, however many short ones
// there are.
template <bool ONCE> __global__ void __launch_bounds__(kExchangeWarps * 32) k_exchange(const ExchangeArgs a)
{
    extern __shared__ int32_t shared[];
    const u32 lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.experts;
    int32_t *place = shared, *row = shared + E + warp * (a.ranks + 2 * E);
    int32_t *hist = row + a.ranks, *sum = hist + E;      // an item's experts; the batch's so far
    for (u32 e = threadIdx.x; e < E; e += blockDim.x) place[e] = a.place[e];
    for (u32 e = lane; e < E; e += 32) hist[e] = sum[e] = 0;
    __syncthreads();

    const u64 first = ((u64)blockIdx.x * a.warps + warp) * a.share;
    const u64 last = min(first + a.share, a.items);
    u64 at_batch = ~0ull;
    auto flush = [&]() {
        if (at_batch == ~0ull) return;
        int32_t *counts = ONCE ? hist : sum;
        __syncwarp();
        for (u32 e = lane; e < E; e += 32) {
            if (counts[e]) atomicAdd(&a.load[at_batch * E + e], counts[e]);
            counts[e] = 0;
        }
        __syncwarp();
    };
    for (u64 item = first; item < last; item++) {
        const u64 b = item / a.sources;
        if (b != at_batch) {
            flush();
            at_batch = b;
        }
        u64 t0, t1;
        item_tokens(a, (u32)(item % a.sources), 0, t0, t1);
        for (u32 d = lane; d < a.ranks; d += 32) row[d] = 0;
        __syncwarp();
        count_slots<ONCE>(a, a.ids + (b * a.tokens + t0) * a.topk, (t1 - t0) * a.topk, 0,
                          ONCE ? 32 / a.topk * a.topk : 32, true, place, hist, row);
        __syncwarp();
        if (!ONCE) {
            for (u32 e = lane; e < E; e += 32) {
                const int32_t n = hist[e];
                const u32 d = (u32)place[e];
                hist[e] = 0;
                if (!n) continue;
                sum[e] += n;
                if (d < a.ranks) atomicAdd(&row[d], n);
            }
            __syncwarp();
        }
        for (u32 d = lane; d < a.ranks; d += 32) a.sent[item * a.ranks + d] = row[d];
        __syncwarp();
    }
    flush();
}

// Few sources: a block counts one item, a source's tokens or a part of them (64
// uneven sources of 37 tokens on average: 7 us on the device, a warp each took
// 25); parts' rows meet in `sent`.  The first blocks count a small batch's load,
// which saves clearing it beforehand.
constexpr u32 kTogether = 512;

template <bool ONCE> __global__ void __launch_bounds__(kTogether) k_exchange_together(const ExchangeArgs a)
{
    extern __shared__ int32_t shared[];
    const u32 E = a.experts, warp = threadIdx.x >> 5;
    int32_t *place = shared, *hist = place + E, *row = hist + E;
    const bool load_only = blockIdx.x < a.count_blocks, loads = load_only || a.count_blocks == 0;
    const u64 item = blockIdx.x - a.count_blocks, pair = item / a.splits, b = load_only ? blockIdx.x : pair / a.sources;
    u64 t0, t1;
    if (load_only) source_tokens(a, 0, a.sources - 1, t0, t1);      // tokens of no source count nowhere
    else item_tokens(a, (u32)(pair % a.sources), (u32)(item % a.splits), t0, t1);
    for (u32 e = threadIdx.x; e < E; e += kTogether) {
        place[e] = a.place[e];
        hist[e] = 0;
    }
    for (u32 d = threadIdx.x; d < a.ranks; d += kTogether) row[d] = 0;
    __syncthreads();
    const int32_t *ids = a.ids + (b * a.tokens + t0) * a.topk;
    const u64 slots = (t1 - t0) * a.topk;
    if (load_only) {
        count_slots<false>(a, ids, slots, warp * 32, kTogether, true, place, hist, row);
    } else {
        const u32 used = ONCE ? 32 / a.topk * a.topk : 32;
        count_slots<ONCE>(a, ids, slots, warp * used, used * (kTogether / 32), loads, place, hist, row);
    }
    __syncthreads();
    if (loads) {
        for (u32 e = threadIdx.x; e < E; e += kTogether) {
            if (load_only) a.load[b * E + e] = hist[e];
            else if (hist[e]) atomicAdd(&a.load[b * E + e], hist[e]);
        }
        if (load_only) return;
    }
    if (!ONCE) {
        for (u32 e = threadIdx.x; e < E; e += kTogether)
            if (hist[e] && (u32)place[e] < a.ranks) atomicAdd(&row[place[e]], hist[e]);
        __syncthreads();
    }
    int32_t *sent = a.sent + pair * a.ranks;
    for (u32 d = threadIdx.x; d < a.ranks; d += kTogether) {
        if (a.splits == 1) sent[d] = row[d];
        else if (row[d]) atomicAdd(&sent[d], row[d]);
    }
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
    const u64 pairs = d->batches * d->sources, mean = d->tokens / d->sources;
    a.splits = 1;
    a.count_blocks = 0;
    if (pairs < 8ull * sms) {
        // Sources of more than 2048 tokens are cut until every SM has two blocks:
        // 16 of 16384 tokens x 8 take 25 us on the device (whole: 138), of 4096 25 (40).
        // Those of 2048 stay whole, at 23 (parts of 512 tokens: 13).
        const u64 want = (2ull * sms + pairs - 1) / pairs, can = (mean + 2047) / 2048;
        if (can > 1 && want > 1) a.splits = (u32)(want < can ? want : can);
        // One set of 64 sources: up to 16384 slots 3 to 4 us by counting blocks (6.3
        // with the load cleared and added up by the items), 32768 6.2 (7.1), 65536 9.9 (8.4).
        if (d->tokens * d->topk <= 32768) a.count_blocks = (u32)d->batches;
    }
    a.items = pairs * a.splits;
    if (!a.count_blocks && cudaMemsetAsync(a.load, 0, 4 * d->batches * d->experts, s) != cudaSuccess) return MV_ECUDA;
    if (a.splits > 1 && cudaMemsetAsync(a.sent, 0, 4 * pairs * a.ranks, s) != cudaSuccess) return MV_ECUDA;
    if (pairs < 8ull * sms)
        return launch(d->once ? k_exchange_together<true> : k_exchange_together<false>,
                      dim3((u32)(a.count_blocks + a.items)), kTogether, 4 * (2 * a.experts + a.ranks), s, a);
    const u32 a_warp = 4 * (a.ranks + 2 * a.experts);
    a.warps = kExchangeWarps;
    while (a.warps > 1 && 4 * a.experts + a.warps * a_warp > 72 * 1024) a.warps /= 2;
    const u32 smem = 4 * a.experts + a.warps * a_warp, held = 227 * 1024 / (smem + 1024);
    const u64 resident = (u64)sms * a.warps * (held < 64 / a.warps ? held : 64 / a.warps);
    a.share = (u32)((a.items + 2 * resident - 1) / (2 * resident));
    const auto kernel = d->once ? k_exchange<true> : k_exchange<false>;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return MV_ECUDA;
    const u64 a_block = (u64)a.share * a.warps;
    return launch(kernel, dim3((u32)((a.items + a_block - 1) / a_block)), a.warps * 32, smem, s, a);
}
