// The routed experts' SwiGLU products with 4-bit weights (mv_experts in
// include/mv.h), for the few tokens of a decode step.
//
// Bytes decide: an expert of 7168 x 2048 is 22 MB of weights and 0.7 MB of
// scales, read for one token or for twenty.  So pairs of token and expert are
// grouped by expert, and each visited expert's weights are streamed once, in a
// chain of four kernels (group; W1 and W3 with silu; W2; combine), each
// starting as the one before it ends.  With at most 24 columns of activations
// the matrix instruction that takes its operands from registers fits: weights
// are widened in registers and never written back, and the tensor pipe is 17 to
// 46% busy.  Widening is most of the work: about 64 instructions for 32 x 32
// weights of W1/W3 (92 of W2, whose activations are in two parts), of the 89
// issue slots that memory speed would leave.  The issue slots are half used:
// what is left is latency at 16 warps an SM.
//
// 64 tokens on 32 of 256 such experts (633 MB): 150 us, 4.2 TB/s, W1/W3 at 5.0,
// W2 3.5; one token (182 MB): 54 us, of which W1/W3 30 (256 blocks for 152 SMs),
// W2 21, grouping and combining 7 (the kernels overlap); 7 tokens over 33 experts
// of 2880 x 1440 with scales every 32 columns: 59 us; 200 tokens over 60
// experts of 2048 x 1408 (277 MB, three tiles of activations): 156 us.  Steps on
// the way, us for 64, 1 and 200 tokens: a dot product a row and pair 1801, 280,
// 6486; matrix instructions 212, 99, 177; scales copied ahead of their use 198,
// 84, 162; activations as half and constants as arguments 166, 66, 182; kernels
// started early 153, 58, 154; steps without checks 136 to 143, 53, 139; inner
// activations in two parts, not rounded to the type, 150, 54, 156.
#include <cmath>
#include <cstring>
#include <type_traits>

#include "mv_moe.cuh"

namespace mvmoe {

// A token's slot is a pair; pairs are grouped by expert, and up to 8, 16 or 24
// of one expert's pairs make an item: what one pass over its weights serves.
u32 item_pairs(u64 tokens) { return tokens <= 8 ? 8 : tokens <= 16 ? 16 : 24; }

struct alignas(16) Item {
    u32 expert, first, count, none; // pairs[first .. first + count); a count of 0: none, nor any after it
};

// Bit patterns of a widening, as kernel arguments: an instruction holds one
// constant, and two that the compiler knew would cost it another one.
struct Patterns {
    u32 low, high;                  // nibbles 0 and 4, 1 and 5 of a word
    u32 power, offset;              // what they are masked into, and that plus 8
    u32 sixteenth, offset16;        // 1 / 16 and -(power / 16 + 8)
};

struct ExpertArgs {
    Patterns half, brain;           // for half, for bfloat16
    const void *x;
    const int32_t *ids;
    const float *weights;
    const uint8_t *w13, *w2;
    const void *s13, *s2;
    void *y;
    u64 tokens, stride;
    u32 topk, experts, hidden, inner, group, item_pairs;
    // workspace
    __half *xp;                     // x / x_unit, permuted      [tokens, hidden]
    float *x_unit;                  // powers of two             [tokens]
    __nv_bfloat16 *h;               // silu(W1 x) (W3 x) in two parts, permuted [pairs, 2, inner]
    float *o;                       // W2 h                      [pairs, hidden]
    uint2 *pairs;                   // pairs by expert, each with its token
    Item *items;
    u32 most_items;
};

// ---- packed weights against 16-bit activations ---------------------------
// Widening by mask and subtraction (Kim, Henry, Fahim and Hassan Awadalla, "Who
// Says Elephants Can't Run", 2022).
// A 32-bit word holds the 4-bit numbers of columns 0..7.  Masking nibbles i
// and i + 4 into the halves of a word that holds a power of two makes that
// power plus q in both halves, exactly; one subtraction leaves q - 8.  The
// columns then come as pairs (0,4) (1,5) (2,6) (3,7), so activations are kept
// with every eight columns in that order.
__device__ __forceinline__ u32 column_place(u32 c) { return (c & ~7u) | ((c & 3) << 1) | ((c >> 2) & 1); }

template <class T> struct Math;
template <> struct Math<__half> {
    static constexpr bool kOneShift = true;
    static constexpr Patterns kPatterns = {0x000F000F, 0x00F000F0, 0x64006400, 0x64086408, 0x2C002C00, 0xD480D480};   // 1024
    static __device__ __forceinline__ u32 sub(u32 a, u32 b)
    {
        u32 d;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ void mma(float (&c)[4], u32 a0, u32 a1, u32 a2, u32 a3, u32 b0, u32 b1)
    {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};
template <> struct Math<__nv_bfloat16> {
    static constexpr bool kOneShift = false;
    static constexpr Patterns kPatterns = {0x000F000F, 0, 0x43004300, 0x43084308, 0, 0};                             // 128
    static __device__ __forceinline__ u32 sub(u32 a, u32 b)
    {
        u32 d;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ void mma(float (&c)[4], u32 a0, u32 a1, u32 a2, u32 a3, u32 b0, u32 b1)
    {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};
// The first product of a sum starts it.
template <class T>
__device__ __forceinline__ void mma_from_zero(float (&c)[4], u32 a0, u32 a1, u32 a2, u32 a3, u32 b0, u32 b1)
{
    c[0] = c[1] = c[2] = c[3] = 0.0f;
    Math<T>::mma(c, a0, a1, a2, a3, b0, b1);
}
template <class T> __device__ __forceinline__ void widen(const Patterns &c, u32 word, u32 (&p)[4])
{
    if constexpr (Math<T>::kOneShift) {
        // half's ten bits hold a nibble in place: 1024 + 16 q, over 16, less 72
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const u32 w = word >> (4 * i);
            p[i] = Math<T>::sub((w & c.low) | c.power, c.offset);
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(p[i + 1]) : "r"((w & c.high) | c.power), "r"(c.sixteenth), "r"(c.offset16));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) p[i] = Math<T>::sub(((word >> (4 * i)) & c.low) | c.power, c.offset);
    }
}

__device__ __forceinline__ void copy16(u32 to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
template <int N> __device__ __forceinline__ void copies_left()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <class T> __device__ __forceinline__ float shared_value(u32 at)
{
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
    T t;
    memcpy(&t, &v, 2);
    return to_float(t);
}

// A kernel of the chain may start while the one before it ends, and waits
// here for what that one has written.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---- grouping ------------------------------------------------------------
constexpr u32 kPrepThreads = 512;

// Block 0 groups the pairs by expert (counts, their prefix sums, a cursor an
// expert); the other blocks write x in the products' column order.  The order
// of an expert's pairs may differ from run to run: a pair's result does not
// depend on its place.
//
// x is kept as half, whose products take fewer instructions to feed than
// bfloat16's.  A bfloat16 row is divided by a power of two first, so that its
// greatest magnitude lies in [2^14, 2^15): its eight bits fit half's eleven
// exactly down to 2^-28 of the greatest, and below that the error is under
// 2^-39 of it, less than the 32-bit sums' own.
template <class T> __global__ void __launch_bounds__(kPrepThreads) k_prepare(const ExpertArgs a)
{
    const u32 tid = threadIdx.x;
    let_next_start();
    if (blockIdx.x) {
        __shared__ float greatest[kPrepThreads / 32];
        const u32 eights = a.hidden / 8;
        for (u64 t = blockIdx.x - 1; t < a.tokens; t += gridDim.x - 1) {
            const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + t * a.stride);
            uint4 *to = reinterpret_cast<uint4 *>(a.xp + t * a.hidden);
            float unit = 1.0f, inverse = 1.0f;
            if constexpr (sizeof(T) == 2 && !Math<T>::kOneShift) {
                float m = 0.0f;
                for (u32 i = tid; i < eights; i += kPrepThreads) {
                    const uint4 v = x[i];
                    const u32 w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xFFFF0000u))));
                }
                m = group_max<32>(m);
                __syncthreads();                              // the last token's maxima are read
                if ((tid & 31) == 0) greatest[tid >> 5] = m;
                __syncthreads();
                for (u32 i = 0; i < kPrepThreads / 32; i++) m = fmaxf(m, greatest[i]);
                if (m > 0.0f && m < INFINITY) {
                    const int e = max((int)(__float_as_uint(m) >> 23) - 127, -100) - 14;
                    unit = __uint_as_float((u32)(e + 127) << 23);
                    inverse = __uint_as_float((u32)(127 - e) << 23);
                }
            }
            for (u32 i = tid; i < eights; i += kPrepThreads) {
                uint4 v = x[i];
                if constexpr (!Math<T>::kOneShift) {
                    u32 *w = reinterpret_cast<u32 *>(&v);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const __half2 h = __floats2half2_rn(__uint_as_float(w[j] << 16) * inverse,
                                                            __uint_as_float(w[j] & 0xFFFF0000u) * inverse);
                        memcpy(&w[j], &h, 4);
                    }
                }
                to[i] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                   __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
            }
            if (tid == 0) a.x_unit[t] = unit;
        }
        return;
    }
    __shared__ u32 count[kMaxExperts], first[kMaxExperts], item[kMaxExperts];
    const u32 n = (u32)(a.tokens * a.topk), most = a.item_pairs;
    for (u32 e = tid; e < a.experts; e += kPrepThreads) count[e] = 0;
    __syncthreads();
    for (u32 p = tid; p < n; p += kPrepThreads) {
        const u32 e = (u32)a.ids[p];
        if (e < a.experts) atomicAdd(&count[e], 1u);
    }
    __syncthreads();
    if (tid < 32) {                                     // prefix sums by one warp
        u32 pairs = 0, items = 0;
        for (u32 base = 0; base < a.experts; base += 32) {
            const u32 e = base + tid, c = e < a.experts ? count[e] : 0;
            const u32 k = (c + most - 1) / most;
            u32 sc = c, sk = k;
            for (u32 d = 1; d < 32; d <<= 1) {
                const u32 oc = __shfl_up_sync(kFull, sc, d), ok = __shfl_up_sync(kFull, sk, d);
                if (tid >= d) { sc += oc; sk += ok; }
            }
            if (e < a.experts) { first[e] = pairs + sc - c; item[e] = items + sk - k; }
            pairs += __shfl_sync(kFull, sc, 31);
            items += __shfl_sync(kFull, sk, 31);
        }
        for (u32 i = items + tid; i < a.most_items; i += 32) a.items[i] = {0, 0, 0, 0};
    }
    __syncthreads();
    for (u32 e = tid; e < a.experts; e += kPrepThreads)
        for (u32 i = 0; i * most < count[e]; i++)
            a.items[item[e] + i] = {e, first[e] + i * most, min(most, count[e] - i * most), 0};
    __syncthreads();
    for (u32 p = tid; p < n; p += kPrepThreads) {
        const u32 e = (u32)a.ids[p];
        if (e < a.experts) a.pairs[atomicAdd(&first[e], 1u)] = make_uint2(p, p / a.topk);
    }
}

// ---- products ------------------------------------------------------------
// The inner activations h = silu(W1 x) (W3 x) are the next product's operand:
// two bfloat16, the nearest to h and the nearest to what that leaves, together
// within 2^-18 of h at any magnitude that 32 bits hold (float16 would end at
// 65504).  Both parts meet the same widened weights and add to the same sums,
// so the second costs matrix instructions and shared-memory loads, not
// widening.  All sums are held in 32 bits, and only y is rounded to x's type.
constexpr u32 kWarps = 8, kThreads = kWarps * 32;
constexpr u32 kRows = kWarps / 2 * 32;          // weight rows a block: 32 to each of four pairs of warps
constexpr u32 kStep = 256;                      // columns a step: half of them to each warp of a pair
constexpr u32 kWPitch = kStep / 4;              // bytes of a row of a warp's weights; piece p of row r lies at
constexpr u32 kWarpStage = 32 * kWPitch;        // p ^ (r / 2 & 3), so that eight rows' pieces are eight bank groups

// Scales come by epochs of 16 groups, two in shared memory.  A row's scales
// start anywhere, so the aligned 16-byte pieces around them are copied: three
// hold 16 groups at any offset.
constexpr u32 kEpoch = 16;
constexpr u32 kSPitch = kEpoch * 2 + 16;
constexpr u32 kScaleBytes = 2 * kRows * kSPitch;

// Weights are copied by the warp that uses them, kStagesOf steps in flight or
// in use, and no other warp waits for them.  Activations are the block's, in
// chunks of kChunkOf steps, two in shared memory; the block's warps meet once
// a chunk.  Epochs begin with a chunk.  What is copied is there kStagesOf - 1
// steps later: a chunk or an epoch at most.  NB: tiles of activations, 8 rows each;
// many of them leave room for less ahead.
template <int NB, u32 PER> constexpr int kStagesOf = NB == 1 && PER > 1 ? 4 : NB <= 3 ? 3 : 2;
template <int NB, u32 PER> constexpr u32 kChunkOf = NB == 1 && PER > 1 ? 4 : NB <= 3 ? 2 : 1;
template <int NB, u32 PER> constexpr u32 kXPitch = kChunkOf<NB, PER> * kStep * 2;      // odd rows' 64-byte halves are swapped
template <int NB, u32 PER> constexpr u32 kRing = kStagesOf<NB, PER> * kWarps * kWarpStage;
constexpr u32 kTable = 3 * 8 * 8;               // an item's pairs: where they go, and what x was divided by
template <int NB, u32 PER> constexpr u32 kRoom = kTable + kScaleBytes + kRing<NB, PER> + 2 * NB * 8 * kXPitch<NB, PER>;
template <u32 A, u32 B> constexpr u32 kLarger = A > B ? A : B;
// Parts of the activations: x is one half, h two bfloat16.
template <bool GATE> constexpr int kParts = GATE ? 1 : 2;
// Shared memory of a block whose items hold up to 8 MOST pairs.
template <bool GATE, int MOST, u32 PER, int P = kParts<GATE>> constexpr u32 kSmem =
    MOST == 1 ? kRoom<P, PER> : kLarger<kRoom<P, PER>, MOST == 2 ? kRoom<2 * P, PER> : kLarger<kRoom<2 * P, PER>, kRoom<3 * P, PER>>>;
template <bool GATE> constexpr u32 kMostSmem = kLarger<kSmem<GATE, 3, 1>, kSmem<GATE, 3, 4>>;
static_assert(2 * (kLarger<kMostSmem<true>, kMostSmem<false>> + 1024) <= 227 * 1024, "two blocks an SM");

// One tile of weight rows against up to 8 NT pairs' activations.  A warp
// holds 32 rows as two matrix operands of 16; an operand of 16 x 16 weights
// meets 16 x 8 activations in one mma.  Sums of a group of columns start at
// zero and are then added, times the rows' scales, in 32 bits; a pair of
// warps adds its two sums at the end.  The order of additions depends on the
// sizes alone, never on the other tokens.
//
// T: the type of the scales and of the result; C: of the activations' parts;
// PER: blocks of 32 columns a group.
template <class T, class C, int NT, bool GATE, u32 PER>
__device__ __forceinline__ void product(const ExpertArgs &a, const Item it, u32 tile, unsigned char *smem)
{
    constexpr int kP = kParts<GATE>, kTiles = NT * kP, kStages = kStagesOf<kTiles, PER>;
    constexpr u32 kGroup = PER * 32, kEpochSteps = kEpoch * kGroup / kStep, kChunk = kChunkOf<kTiles, PER>, kPitch = kXPitch<kTiles, PER>;
    static_assert(kEpochSteps % kChunk == 0 && kStages - 1 <= (int)kChunk, "copies arrive in time");
    const u32 tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const u32 half = tid >> 7, warp = (tid >> 5) & 3;         // columns, rows
    const u32 K = GATE ? a.hidden : a.inner, groups = K / kGroup;
    const Patterns patterns = GATE ? a.half : a.brain;
    uint2 *table = reinterpret_cast<uint2 *>(smem);
    const u32 scales = (u32)__cvta_generic_to_shared(smem) + kTable, ring = scales + kScaleBytes, rows = ring + kRing<kTiles, PER>;
    // block row r: warp r / 32's operand (r / 16) & 1, row r & 15
    auto weight_row = [&](u32 r) -> int64_t {
        if (GATE) {
            const u32 i = tile * (kRows / 2) + (r >> 5) * 16 + (r & 15);
            return i < a.inner ? (int64_t)((r & 16) ? a.inner + i : i) : -1;
        }
        const u32 i = tile * kRows + r;
        return i < a.hidden ? (int64_t)i : -1;
    };
    const u64 base_row = (u64)it.expert * (GATE ? 2 * a.inner : a.hidden);
    // This thread's pieces of a step: weights, activations, scales.  Rows
    // beyond the matrix are copied from its first one and not used.
    const uint8_t *wp[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int64_t row = weight_row(warp * 32 + j * 8 + (lane >> 2));
        wp[j] = (GATE ? a.w13 : a.w2) + (base_row + (u64)(row < 0 ? 0 : row)) * (K / 2) + half * (kStep / 4) + (lane & 3) * 16;
    }
    const u32 my_ring = ring + (tid >> 5) * kWarpStage, w_to = my_ring + (lane >> 2) * kWPitch + ((lane & 3) ^ (lane >> 3)) * 16;
    auto fetch_weights = [&](u32 s, u32 slot, bool whole) {   // pointers advance: called for s = 0, 1, ...
        if (whole || s * kStep + half * (kStep / 2) + (lane & 3) * 32 < K)
#pragma unroll
            for (int j = 0; j < 4; j++) copy16(w_to + slot * (kWarps * kWarpStage) + j * 8 * kWPitch, wp[j]);
#pragma unroll
        for (int j = 0; j < 4; j++) wp[j] += kStep / 2;
    };
    const u32 steps = (K + kStep - 1) / kStep;
    // the weights' copies start before anything is known of the pairs
#pragma unroll
    for (int s = 0; s < kStages - 1; s++)
        if ((u32)s < steps) fetch_weights(s, s, false);

    const C *xp[NT];
#pragma unroll
    for (int j = 0; j < NT; j++) {                            // a warp copies whole rows
        const u32 r = (tid >> 5) + j * 8;
        xp[j] = nullptr;
        if (r >= it.count) continue;
        const uint2 p = a.pairs[it.first + r];
        xp[j] = (GATE ? reinterpret_cast<const C *>(a.xp) + (u64)p.y * K : reinterpret_cast<const C *>(a.h) + (u64)p.x * kP * K) + lane * 8;
        if (lane == 0) table[r] = make_uint2(p.x, GATE ? __float_as_uint(a.x_unit[p.y]) : 0u);
    }
    const u32 x_to = rows + (tid >> 5) * kPitch + ((lane * 16) ^ ((tid & 32) * 2));
    auto fetch_rows = [&](u32 chunk, bool whole) {
#pragma unroll
        for (u32 i = 0; i < kChunk; i++) {
            const u32 c = (chunk * kChunk + i) * kStep;
            if (!whole && c + lane * 8 >= K) break;
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int part = 0; part < kP; part++)
                    if (xp[j]) copy16(x_to + ((chunk & 1) * kTiles + part * NT + j) * 8 * kPitch + i * kStep * 2, xp[j] + part * K + c);
        }
    };
    const T *all = static_cast<const T *>(GATE ? a.s13 : a.s2);
    const char *s_end = reinterpret_cast<const char *>(all + (u64)a.experts * (GATE ? 2 * a.inner : a.hidden) * groups);
    const int64_t srow = tid < kRows ? weight_row(tid) : -1;
    const char *s_row = srow < 0 ? nullptr : reinterpret_cast<const char *>(all + (base_row + (u64)srow) * groups);
    auto fetch_scales = [&](u32 epoch) {
        if (!s_row || epoch * kEpoch >= groups) return;
        const char *from = s_row + epoch * kEpoch * 2, *to = s_row + min((epoch + 1) * kEpoch, groups) * 2;
        from -= reinterpret_cast<uintptr_t>(from) & 15;
        u32 at = scales + ((epoch & 1) * kRows + tid) * kSPitch;
        for (; from < to; from += 16, at += 16) {
            const u32 bytes = s_end - from < 16 ? (u32)(s_end - from) : 16u;     // the array's end
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
        }
    };
    // where this lane's four rows have theirs
    u32 s_at[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const u32 r = warp * 32 + g + 8 * i;
        const int64_t row = weight_row(r);
        s_at[i] = scales + r * kSPitch + (u32)(((base_row + (u64)(row < 0 ? 0 : row)) * groups * 2) & 15);
    }

    float total[2][NT][4], sum[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; m++)
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int i = 0; i < 4; i++) total[m][n][i] = 0.0f;

    fetch_scales(0);
#pragma unroll
    for (int s = 0; s < kStages - 1; s++) {
        if (s == 0) fetch_rows(0, false);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    const u32 a_row = my_ring + ((lane & 7) + ((lane >> 3) & 1) * 8 + (lane >> 4) * 16) * kWPitch, a_turn = (lane >> 1) & 3;
    const u32 x_row = rows + g * kPitch + half * kStep, x_turn = (t * 16) ^ ((g & 1) * 64);
    // this half's blocks of 32 columns of a step, those below `blocks`
    auto multiply = [&](u32 s, u32 off, u32 x_off, u32 blocks) {
        // one tile: every operand of the step is under way before the first is used
        u32 w[kStep / 64][4], x[kStep / 64][kP][4];
        auto load_weights = [&](u32 b) {
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[b][0]), "=r"(w[b][1]), "=r"(w[b][2]), "=r"(w[b][3]) : "r"(a_row + off + (b ^ a_turn) * 16));
        };
        auto load_rows = [&](int part, int n, u32 b, u32 (&y)[4]) {
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                         : "r"(x_row + x_off + (part * NT + n) * 8 * kPitch + ((b * 64) ^ x_turn)));
        };
#pragma unroll
        for (u32 b = 0; b < kStep / 64; b++) {
            if (NT > 1) break;
            load_weights(b);
#pragma unroll
            for (int part = 0; part < kP; part++) load_rows(part, 0, b, x[b][part]);
        }
#pragma unroll
        for (u32 b = 0; b < kStep / 64; b++) {
            if (b >= blocks) break;
            if (NT > 1) load_weights(b);
            u32 q[4][4];
#pragma unroll
            for (int i = 0; i < 4; i++) widen<C>(patterns, w[b][i], q[i]);
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int part = 0; part < kP; part++) {
                    u32 y[4];
                    if (NT == 1) {
#pragma unroll
                        for (int i = 0; i < 4; i++) y[i] = x[b][part][i];
                    } else {
                        load_rows(part, n, b, y);
                    }
#pragma unroll
                    for (int m = 0; m < 2; m++) {
                        if (b % PER == 0 && part == 0) mma_from_zero<C>(sum[m][n], q[2 * m][0], q[2 * m + 1][0], q[2 * m][1], q[2 * m + 1][1], y[0], y[1]);
                        else Math<C>::mma(sum[m][n], q[2 * m][0], q[2 * m + 1][0], q[2 * m][1], q[2 * m + 1][1], y[0], y[1]);
                        Math<C>::mma(sum[m][n], q[2 * m][2], q[2 * m + 1][2], q[2 * m][3], q[2 * m + 1][3], y[2], y[3]);
                    }
                }
            if (b % PER == PER - 1) {                         // the group's last columns
                const u32 group = s * (kStep / kGroup) + half * (kStep / 2 / kGroup) + b / PER;
                const u32 s_off = ((group / kEpoch) & 1) * kRows * kSPitch + (group % kEpoch) * 2;
#pragma unroll
                for (int m = 0; m < 2; m++) {
                    const float s0 = shared_value<T>(s_at[2 * m] + s_off), s1 = shared_value<T>(s_at[2 * m + 1] + s_off);
#pragma unroll
                    for (int n = 0; n < NT; n++) {
                        total[m][n][0] += s0 * sum[m][n][0];
                        total[m][n][1] += s0 * sum[m][n][1];
                        total[m][n][2] += s1 * sum[m][n][2];
                        total[m][n][3] += s1 * sum[m][n][3];
                    }
                }
            }
        }
    };
    u32 slot = 0, ahead = kStages - 1;
    // step s, number i of its chunk; whole: nothing that it multiplies or copies ends at K
    auto step = [&](u32 s, u32 i, bool whole) {
        copies_left<kStages - 2>();
        if (i == 0) __syncthreads();
        else __syncwarp();
        if (whole || s + kStages - 1 < steps) fetch_weights(s + kStages - 1, ahead, whole);
        if (i == 0) fetch_rows(s / kChunk + 1, whole);
        if (i == 0 && s % kEpochSteps == 0) fetch_scales(s / kEpochSteps + 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        const u32 off = slot * (kWarps * kWarpStage), x_off = (s / kChunk & 1) * kTiles * 8 * kPitch + i * kStep * 2;
        if (whole || (NT == 1 && (s + 1) * kStep <= K)) {
            multiply(s, off, x_off, kStep / 64);
        } else {
            const u32 left = (K - s * kStep) / 32, mine = half * (kStep / 64);
            multiply(s, off, x_off, left > mine ? left - mine : 0);
        }
        slot = slot + 1 == kStages ? 0 : slot + 1;
        ahead = ahead + 1 == kStages ? 0 : ahead + 1;
    };
    u32 s = 0;
    if (NT == 1) {                                            // more tiles leave no registers for a second copy
        for (const u32 whole = K / kStep; s + kLarger<2 * kChunk, kChunk + kStages - 1> <= whole; s += kChunk)
#pragma unroll
            for (u32 i = 0; i < kChunk; i++) step(s + i, i, true);
    }
    for (; s < steps; s++) step(s, s % kChunk, false);
    copies_left<0>();
    // The halves' sums meet through the ring: the first half finishes the
    // operands' rows 0 to 7, the second rows 8 to 15.
    __syncthreads();
    float2 *sums = reinterpret_cast<float2 *>(smem + kTable + kScaleBytes) + (warp * 32 + lane);
#pragma unroll
    for (int m = 0; m < 2; m++)
#pragma unroll
        for (int n = 0; n < NT; n++)
            sums[((m * NT + n) * 2 + half) * 128] =
                half ? make_float2(total[m][n][0], total[m][n][1]) : make_float2(total[m][n][2], total[m][n][3]);
    __syncthreads();
    // value j of operand m, tile n: row g of the half's eight, pair 8 n + 2 t + j
#pragma unroll
    for (int n = 0; n < NT; n++) {
        float v[2][2];
#pragma unroll
        for (int m = 0; m < 2; m++) {
            const float2 other = sums[((m * NT + n) * 2 + 1 - half) * 128];
            v[m][0] = (half ? total[m][n][2] : total[m][n][0]) + other.x;
            v[m][1] = (half ? total[m][n][3] : total[m][n][1]) + other.y;
        }
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const u32 c = n * 8 + 2 * t + j, r = g + half * 8;
            if (c >= it.count) continue;
            const uint2 to = table[c];
            if (GATE) {
                const u32 row = tile * (kRows / 2) + warp * 16 + r;
                const float unit = __uint_as_float(to.y), z = v[0][j] * unit, up = v[1][j] * unit;
                if (row < a.inner) {
                    const float h = z * reciprocal_fast(1.0f + exp2_fast(-z * kLog2e)) * up;
                    const __nv_bfloat16 most = __float2bfloat16_rn(h);
                    __nv_bfloat16 *at = a.h + (u64)to.x * 2 * a.inner + column_place(row);
                    at[0] = most;
                    const float rest = h - __bfloat162float(most);
                    at[a.inner] = __float2bfloat16_rn(fabsf(rest) < INFINITY ? rest : 0.0f);          // of infinities nothing is left
                }
            } else {
#pragma unroll
                for (int m = 0; m < 2; m++) {
                    const u32 row = tile * kRows + warp * 32 + m * 16 + r;
                    if (row < a.hidden) a.o[(u64)to.x * a.hidden + row] = v[m][j];
                }
            }
        }
    }
}

template <class T, bool GATE, int MOST, u32 PER> __global__ void __launch_bounds__(kThreads, 2) k_product(const ExpertArgs a)
{
    using C = std::conditional_t<GATE, __half, __nv_bfloat16>;
    extern __shared__ __align__(16) unsigned char smem[];
    after_previous();
    let_next_start();
    for (u32 i = blockIdx.y; i < a.most_items; i += gridDim.y) {
        const uint4 v = *reinterpret_cast<const uint4 *>(a.items + i);
        const Item it = {v.x, v.y, v.z, 0};
        if (!it.count) return;
        if (MOST == 1 || it.count <= 8) product<T, C, 1, GATE, PER>(a, it, blockIdx.x, smem);
        else if (MOST == 2 || it.count <= 16) product<T, C, 2, GATE, PER>(a, it, blockIdx.x, smem);
        else product<T, C, MOST < 3 ? 1 : 3, GATE, PER>(a, it, blockIdx.x, smem);
        __syncthreads();
    }
}

// y = sum over the slots, in their order, of weight x (W2 h).  Four columns a
// thread; a token's ids and weights are read once and its rows eight at a time.
constexpr u32 kCombineThreads = 128;

template <class T> __global__ void __launch_bounds__(kCombineThreads) k_combine(const ExpertArgs a)
{
    after_previous();
    const u64 quads = a.hidden / 4, n = a.tokens * quads;
    for (u64 i = (u64)blockIdx.x * kCombineThreads + threadIdx.x; i < n; i += (u64)gridDim.x * kCombineThreads) {
        const u64 t = i / quads, c = (i % quads) * 4;
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (u32 j0 = 0; j0 < a.topk; j0 += 8) {
            float4 o[8];
            float w[8];
#pragma unroll
            for (u32 j = 0; j < 8; j++) {
                const u64 p = t * a.topk + j0 + j;
                const bool here = j0 + j < a.topk && (u32)a.ids[p] < a.experts;
                w[j] = here ? a.weights[p] : 0.0f;
                o[j] = here ? *reinterpret_cast<const float4 *>(a.o + p * a.hidden + c) : make_float4(0, 0, 0, 0);
            }
#pragma unroll
            for (u32 j = 0; j < 8; j++) {
                y[0] += w[j] * o[j].x; y[1] += w[j] * o[j].y; y[2] += w[j] * o[j].z; y[3] += w[j] * o[j].w;
            }
        }
        T out[4];
#pragma unroll
        for (int j = 0; j < 4; j++) out[j] = from_float<T>(y[j]);
        uint2 v;
        memcpy(&v, out, 8);
        *reinterpret_cast<uint2 *>(static_cast<T *>(a.y) + t * a.hidden + c) = v;
    }
}

// Workspace: offsets of its parts, each on a 256-byte boundary.
struct Layout {
    u64 xp, x_unit, h, o, pairs, items, total;
};
u64 most_items(const mv_experts_desc *d)
{
    const u64 pairs = d->tokens * d->topk;
    return (pairs < d->experts ? pairs : d->experts) + pairs / item_pairs(d->tokens);
}
Layout layout(const mv_experts_desc *d)
{
    const u64 pairs = d->tokens * d->topk;
    Layout l;
    u64 at = 0;
    auto take = [&](u64 bytes) { const u64 here = at; at += (bytes + 255) / 256 * 256; return here; };
    l.xp = take(d->tokens * d->hidden * 2);
    l.x_unit = take(d->tokens * 4);
    l.h = take(pairs * d->inner * 4);
    l.o = take(pairs * d->hidden * 4);
    l.pairs = take(pairs * sizeof(uint2));
    l.items = take(most_items(d) * sizeof(Item));
    l.total = at;
    return l;
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

template <class T, bool GATE, int MOST, u32 PER> int run_product(const ExpertArgs &a, u64 items, cudaStream_t stream)
{
    constexpr u32 smem = kSmem<GATE, MOST, PER>;
    const u32 tiles = GATE ? (a.inner + kRows / 2 - 1) / (kRows / 2) : (a.hidden + kRows - 1) / kRows;
    const auto kernel = k_product<T, GATE, MOST, PER>;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return MV_ECUDA;
    return launch_after(kernel, dim3(tiles, (u32)std::fmin((double)items, 65535.0)), kThreads, smem, stream, a);
}

template <class T, bool GATE, int MOST> int run_product(const ExpertArgs &a, u64 items, cudaStream_t stream)
{
    if (a.group == 32) return run_product<T, GATE, MOST, 1>(a, items, stream);
    if (a.group == 64) return run_product<T, GATE, MOST, 2>(a, items, stream);
    return run_product<T, GATE, MOST, 4>(a, items, stream);
}

template <class T, int MOST> int run_experts(const ExpertArgs &a, u64 items, cudaStream_t stream)
{
    const u32 sms = sm_count();
    if (!sms) return MV_ECUDA;
    const u32 share = (u32)std::fmin((double)a.tokens, 2.0 * sms);
    int rc = launch(k_prepare<T>, dim3(1 + share), kPrepThreads, 0, stream, a);
    if (rc == MV_OK) rc = run_product<T, true, MOST>(a, items, stream);
    if (rc == MV_OK) rc = run_product<T, false, MOST>(a, items, stream);
    const u64 quads = a.tokens * (a.hidden / 4);
    const u32 blocks = (u32)std::fmin((double)((quads + kCombineThreads - 1) / kCombineThreads), 16.0 * sms);
    if (rc == MV_OK) rc = launch_after(k_combine<T>, dim3(blocks), kCombineThreads, 0, stream, a);
    return rc;
}

template <class T> int run_experts(const ExpertArgs &a, u64 items, cudaStream_t stream)
{
    if (a.item_pairs == 8) return run_experts<T, 1>(a, items, stream);
    if (a.item_pairs == 16) return run_experts<T, 2>(a, items, stream);
    return run_experts<T, 3>(a, items, stream);
}

}  // namespace mvmoe

using namespace mvmoe;

extern "C" int mv_experts_workspace_bytes(const mv_experts_desc *d, uint64_t *bytes)
{
    if (!bytes) return MV_EINVAL;
    *bytes = 0;
    const int rc = check(d);
    if (rc != MV_OK) return rc;
    *bytes = layout(d).total;
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
    a.half = Math<__half>::kPatterns;
    a.brain = Math<__nv_bfloat16>::kPatterns;
    a.x = d->x;
    a.ids = d->ids;
    a.weights = d->weights;
    a.w13 = d->w13;
    a.s13 = d->s13;
    a.w2 = d->w2;
    a.s2 = d->s2;
    a.y = d->y;
    const Layout l = layout(d);
    char *ws = static_cast<char *>(workspace);
    a.xp = reinterpret_cast<__half *>(ws + l.xp);
    a.x_unit = reinterpret_cast<float *>(ws + l.x_unit);
    a.h = reinterpret_cast<__nv_bfloat16 *>(ws + l.h);
    a.o = reinterpret_cast<float *>(ws + l.o);
    a.pairs = reinterpret_cast<uint2 *>(ws + l.pairs);
    a.items = reinterpret_cast<Item *>(ws + l.items);
    a.most_items = (u32)most_items(d);
    a.tokens = d->tokens;
    a.stride = d->row_stride;
    a.topk = d->topk;
    a.experts = d->experts;
    a.hidden = d->hidden;
    a.inner = d->inner;
    a.group = d->group;
    a.item_pairs = item_pairs(d->tokens);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return d->dtype == MV_F16 ? run_experts<__half>(a, most_items(d), s)
                              : run_experts<__nv_bfloat16>(a, most_items(d), s);
}
