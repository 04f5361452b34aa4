// Matrix products with bias, activation and residual (mv_linear in
// include/mv.h), and their gradients (mv_linear_backward).
//
// All of them are C[m, n] = sum over k of A[m, k] B[n, k]; only the side that
// lies contiguous in memory differs:
//   y  = x w^T     A = x,  B = w      both contiguous along k
//   dx = dz w      A = dz,            B = w transposed: contiguous along n
//   dw = dz^T x    A = dz transposed, B = x transposed: both along m or n
// The tensor core takes either order from shared memory, so nothing is
// transposed on the way.  Tiles of A and B come by TMA, the sums stay in TMEM
// in 32 bits; one warp copies, one multiplies and four or eight finish tiles, the
// next tile's products running while the last one is finished.
//
// Large products are bound by the tensor pipe (92% busy) and, over a second or so,
// by power: 8192 x 5120 to 20480, bfloat16, with bias and gelu and the
// pre-activations kept, 912 us once (1.88 PFLOP/s; the library's plain product 830)
// and 1055 among others.  Tiles are 256 x 256 by pairs of blocks then, and what is
// left over after whole rounds goes in pieces along k.  Few rows are bound by the
// weights' bytes: x and w change places, so that 128 weight rows meet 16 or 64 of x,
// and up to six or eight blocks share a tile's k and add up in their cluster's shared
// memory: 1 x 20480 to 5120 39.4 us, 5.3 TB/s.  Between the two a product is bound
// by its start and its last, unfilled round: 2048 x 5120 by 2560, dx 46 and dw 40 us,
// where the library takes 36 to 41.  Steps of the first figure: a row of a tile
// at a time 2216 us; eight at a time by eight warps 916; stored by TMA, TMEM handed
// back without waiting for the stores 904 (dx of 65536 x 256 by 256 x 7168: 2030,
// 373, 203).
#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "mv_block.cuh"

namespace mvblock {

// ---- what becomes of a sum -------------------------------------------------
struct Finish {
    const void *bias, *residual;
    void *y, *z;
    u64 m, n;                       // rows and columns of the result
    u64 y_stride, residual_stride;  // z is dense
    u32 dtype, out, bias_type;      // of z; of y and the residual
    u32 act, residual_wide, bias_wide, y_wide, z_wide;   // *_wide: four columns are one aligned access
    u32 by_tma;                     // y and z are stored by TMA, the residual comes by it: rows are 16-byte aligned
    float scale;
};

template <class T> __device__ __forceinline__ void load4(const void *p, u64 at, bool wide, u32 n, float (&v)[4])
{
    const T *from = static_cast<const T *>(p) + at;
    if (wide && n == 4) {
        T t[4];
        if constexpr (sizeof(T) == 4) {
            const uint4 w = *reinterpret_cast<const uint4 *>(from);
            memcpy(t, &w, 16);
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(from);
            memcpy(t, &w, 8);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = to_float(t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = i < (int)n ? to_float(from[i]) : 0.0f;
    }
}
template <class T> __device__ __forceinline__ void store4(void *p, u64 at, bool wide, u32 n, const float (&v)[4])
{
    T *to = static_cast<T *>(p) + at;
    T t[4];
#pragma unroll
    for (int i = 0; i < 4; i++) t[i] = from_float<T>(v[i]);
    if (wide && n == 4) {
        if constexpr (sizeof(T) == 4) {
            uint4 w;
            memcpy(&w, t, 16);
            *reinterpret_cast<uint4 *>(to) = w;
        } else {
            uint2 w;
            memcpy(&w, t, 8);
            *reinterpret_cast<uint2 *>(to) = w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (i < (int)n) to[i] = t[i];
    }
}
__device__ __forceinline__ void load4_as(u32 type, const void *p, u64 at, bool wide, u32 n, float (&v)[4])
{
    if (type == MV_BF16) load4<__nv_bfloat16>(p, at, wide, n, v);
    else if (type == MV_F16) load4<__half>(p, at, wide, n, v);
    else load4<float>(p, at, wide, n, v);
}
__device__ __forceinline__ void store4_as(u32 type, void *p, u64 at, bool wide, u32 n, const float (&v)[4])
{
    if (type == MV_BF16) store4<__nv_bfloat16>(p, at, wide, n, v);
    else if (type == MV_F16) store4<__half>(p, at, wide, n, v);
    else store4<float>(p, at, wide, n, v);
}

// Columns c .. c + 3 of row r (those inside the matrix), from their sums.
__device__ __forceinline__ void finish4(const Finish &f, u64 r, u64 c, float (&v)[4])
{
    if (r >= f.m || c >= f.n) return;
    const u32 n = f.n - c < 4 ? (u32)(f.n - c) : 4;
    if (f.bias) {
        float b[4];
        load4_as(f.bias_type, f.bias, c, f.bias_wide, n, b);
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] += b[i];
    }
    if (f.z) store4_as(f.dtype, f.z, r * f.n + c, f.z_wide, n, v);
    if (f.act != MV_ACT_NONE)
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = activation(f.act, v[i]);
    if (f.residual) {
        float b[4];
        load4_as(f.out, f.residual, r * f.residual_stride + c, f.residual_wide, n, b);
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = fmaf(f.scale, v[i], b[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] *= f.scale;
    }
    store4_as(f.out, f.y, r * f.y_stride + c, f.y_wide, n, v);
}

// One column, where a warp's lanes hold neighbours of a row.
__device__ __forceinline__ float value_as(u32 type, const void *p, u64 at)
{
    return type == MV_BF16 ? to_float(static_cast<const __nv_bfloat16 *>(p)[at])
         : type == MV_F16 ? to_float(static_cast<const __half *>(p)[at]) : static_cast<const float *>(p)[at];
}
// Column c of N rows from r on, a lane's of a warp whose lanes have neighbours, so
// that their accesses are whole; rows may lie anywhere.  ALL: of as many rows.
// Residuals are read first and all at once (each in its turn, 3604 x 80 to 2449 with
// gelu, residual and pre-activations took 97 us, so 53).
template <class OUT, int N> __device__ __forceinline__ void read_residual(const Finish &f, u64 r, u64 c, u32 rows, OUT (&residual)[N])
{
    const OUT *from = static_cast<const OUT *>(f.residual) + r * f.residual_stride + c;
#pragma unroll
    for (u32 j = 0; j < N; j++) residual[j] = j < rows ? from[j * f.residual_stride] : from_float<OUT>(0.0f);
}
template <class OUT, int N> __device__ __forceinline__ void finish_column(const Finish &f, u64 r, u64 c, u32 rows, float (&v)[N], const OUT (&residual)[N])
{
    if (f.bias) {
        const float b = value_as(f.bias_type, f.bias, c);
#pragma unroll
        for (u32 j = 0; j < N; j++) v[j] += b;
    }
    if (f.z) {
        unsigned short *z = static_cast<unsigned short *>(f.z) + r * f.n + c;
#pragma unroll
        for (u32 j = 0; j < N; j++) {
            unsigned short w;
            if (f.dtype == MV_BF16) {
                const __nv_bfloat16 t = from_float<__nv_bfloat16>(v[j]);
                memcpy(&w, &t, 2);
            } else {
                const __half t = from_float<__half>(v[j]);
                memcpy(&w, &t, 2);
            }
            if (j < rows) z[j * f.n] = w;
        }
    }
    activate<N, sizeof(OUT) == 2>(f.act, v);
    OUT *y = static_cast<OUT *>(f.y) + r * f.y_stride + c;
#pragma unroll
    for (u32 j = 0; j < N; j++) {
        const float t = f.residual ? fmaf(f.scale, v[j], to_float(residual[j])) : f.scale * v[j];
        if (j < rows) y[j * f.y_stride] = from_float<OUT>(t);
    }
}
// The same of a warp's 32 x 32 in shared memory.
template <class OUT, bool ALL> __device__ __forceinline__ void finish_column(const Finish &f, u32 mine, u32 lane, u64 r, u64 c, u32 some)
{
    const u32 rows = ALL ? 32 : some;
    OUT residual[32];
    if (f.residual) read_residual(f, r, c, rows, residual);
    float v[32];
#pragma unroll
    for (u32 j = 0; j < 32; j++)
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[j]) : "r"(mine + j * 128 + (((lane >> 2) ^ (j & 7)) * 16) + (lane & 3) * 4));
    finish_column(f, r, c, rows, v, residual);
}
template <class OUT> __device__ __noinline__ void finish_column(const Finish &from, u32 mine, u32 lane, u64 r, u64 c)
{
    const Finish f = from;              // in registers: through the reference each would be read again after every store
    if (c >= f.n || r >= f.m) return;
    if (f.m - r >= 32) finish_column<OUT, true>(f, mine, lane, r, c, 32);
    else finish_column<OUT, false>(f, mine, lane, r, c, (u32)(f.m - r));
}

// ---- PTX -------------------------------------------------------------------
__device__ unsigned g_gave_up;          // warps that ended a wait by its limit

__device__ __forceinline__ u32 shared_at(const void *p) { return (u32)__cvta_generic_to_shared(p); }
__device__ __forceinline__ u64 nanoseconds()
{
    u64 t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ bool barrier_passed(u32 bar, u32 parity)
{
    u32 ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok;
}
// Waits for a phase, two seconds at most.
__device__ __forceinline__ bool barrier_wait(u32 bar, u32 parity)
{
    if (barrier_passed(bar, parity)) return true;
    const u64 end = nanoseconds() + 2000000000ull;
    while (!barrier_passed(bar, parity))
        if (nanoseconds() > end) return false;
    return true;
}
__device__ __forceinline__ void barrier_init(u32 bar, u32 count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ u32 at_leader(u32 address)
{
    u32 there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(there) : "r"(address));
    return there;
}
__device__ __forceinline__ bool one_lane()
{
    u32 ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok;
}
template <int CTAS> __device__ __forceinline__ void copy_tile(u32 to, const CUtensorMap *map, int x, int y, u32 bar)
{
    if constexpr (CTAS == 2)
        asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%3, %4}], [%2];" ::"r"(to), "l"(map), "r"(bar), "r"(x), "r"(y) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%3, %4}], [%2];" ::"r"(to), "l"(map), "r"(bar), "r"(x), "r"(y) : "memory");
}
// A and B in shared memory, by descriptors; the sums in TMEM.
template <int CTAS> __device__ __forceinline__ void multiply(u32 sums, u64 a, u64 b, u32 what, u32 add)
{
    if constexpr (CTAS == 2)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     ::"r"(sums), "l"(a), "l"(b), "r"(what), "r"(add) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     ::"r"(sums), "l"(a), "l"(b), "r"(what), "r"(add) : "memory");
}
// Arrives at the barrier, in every block of the pair, once all products issued so far are done.
template <int CTAS> __device__ __forceinline__ void arrive_after_products(u32 bar)
{
    if constexpr (CTAS == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     ::"r"(bar), "h"((unsigned short)3) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void load_sums(u32 at, u32 (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_sums(u32 at, const u32 (&v)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
        ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
          "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
          "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
          "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(at)
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_sums(u32 at, const u32 (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
        ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
          "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(at)
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void load_sums(u32 at, u32 (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void meet()          // the cluster's threads
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A lane's row of a tile, 128 bytes of it at a time: to shared memory in the
// 128-byte swizzle, and from there to the result by TMA, which leaves out what
// lies beyond the matrix.  Fewer instructions than by a lane's own stores,
// which have to change places for whole sectors: dx of 65536 x 256 by 256 x 7168
// took 308 us that way, 203 so.
template <class T> __device__ __forceinline__ void send_tile(u32 mine, u32 lane, const CUtensorMap *map, int x, int y)
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map), "r"(mine), "r"(x), "r"(y) : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}
// RESIDUAL: v is added, times the scale, to what lies there.
template <class T, bool RESIDUAL>
__device__ __forceinline__ void store_tile(u32 mine, u32 lane, const CUtensorMap *map, int x, int y, const float *v, float scale)
{
    constexpr u32 kEach = 16 / sizeof(T);
    if constexpr (!RESIDUAL) {
        // the store before this one has read the buffer
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
    }
#pragma unroll
    for (u32 j = 0; j < 8; j++) {
        const u32 at = mine + lane * 128 + ((j ^ (lane & 7)) * 16);
        T t[kEach];
        uint4 w;
        if constexpr (RESIDUAL) {
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
            memcpy(t, &w, 16);
        }
#pragma unroll
        for (u32 i = 0; i < kEach; i++)
            t[i] = from_float<T>(RESIDUAL ? fmaf(scale, v[j * kEach + i], to_float(t[i])) : v[j * kEach + i]);
        memcpy(&w, t, 16);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
    }
    send_tile<T>(mine, lane, map, x, y);
}
template <class T, int N> __device__ __forceinline__ void add_bias(const Finish &f, u64 c, float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        if (c + i >= f.n) break;
        float b[4];
        load4<T>(f.bias, c + i, f.bias_wide, f.n - (c + i) < 4 ? (u32)(f.n - (c + i)) : 4, b);
#pragma unroll
        for (int j = 0; j < 4; j++) v[i + j] += b[j];
    }
}
// The residual of the same 128 bytes, on its way to the same place; its arrival is at the barrier.
__device__ __forceinline__ void fetch_residual(u32 mine, u32 lane, u32 bar, const CUtensorMap *map, int x, int y)
{
    if (lane == 0) {
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(32 * 128) : "memory");
        copy_tile<1>(mine, map, x, y, bar);
    }
}
// Columns c .. of the lane's row, 128 bytes of OUT; the residual's are in shared memory.
template <class OUT, int N>
__device__ __forceinline__ void finish_tile(const Finish &f, u32 mine, u32 lane, const CUtensorMap *y_map, const CUtensorMap *z_map,
                                            u64 row0, u64 c, float (&v)[N])
{
    if (f.bias) {
        if (f.bias_type == MV_F32) add_bias<float>(f, c, v);
        else if (f.bias_type == MV_BF16) add_bias<__nv_bfloat16>(f, c, v);
        else add_bias<__half>(f, c, v);
    }
    if (f.z && f.residual) {            // z needs the place that the residual is in
        constexpr int kEach = 16 / sizeof(OUT);
        uint4 residual[8];
#pragma unroll
        for (u32 j = 0; j < 8; j++)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(residual[j].x), "=r"(residual[j].y), "=r"(residual[j].z), "=r"(residual[j].w)
                         : "r"(mine + lane * 128 + ((j ^ (lane & 7)) * 16)) : "memory");
        store_tile<OUT, false>(mine, lane, z_map, (int)c, (int)row0, v, 1.0f);
        activate<N, sizeof(OUT) == 2>(f.act, v);
#pragma unroll
        for (u32 j = 0; j < 8; j++) {
            OUT t[kEach];
            memcpy(t, &residual[j], 16);
#pragma unroll
            for (u32 i = 0; i < kEach; i++) v[j * kEach + i] = fmaf(f.scale, v[j * kEach + i], to_float(t[i]));
        }
        store_tile<OUT, false>(mine, lane, y_map, (int)c, (int)row0, v, 1.0f);
        return;
    }
    if (f.z) store_tile<OUT, false>(mine, lane, z_map, (int)c, (int)row0, v, 1.0f);
    activate<N, sizeof(OUT) == 2>(f.act, v);
    if (f.residual) {
        store_tile<OUT, true>(mine, lane, y_map, (int)c, (int)row0, v, f.scale);
        return;
    }
    if (f.scale != 1.0f)
#pragma unroll
        for (int i = 0; i < N; i++) v[i] *= f.scale;
    store_tile<OUT, false>(mine, lane, y_map, (int)c, (int)row0, v, 1.0f);
}

// ---- tiles -----------------------------------------------------------------
// A block's share of a step of 64 columns of k: 128 rows of A and BN / CTAS
// rows of B, 128 bytes each, in the 128-byte swizzle.  An operand that is
// contiguous along k lies as rows of 64 k; one that is contiguous along its own
// rows lies as pieces of 64 rows x 64 k, each k 128 bytes.
constexpr u32 kStep = 64;

template <int CTAS, int BN> struct Tile {
    static constexpr u32 kRows = 128 * CTAS;
    // a warp copies, one multiplies, the others finish: two to each quarter of TMEM's lanes where tiles are large
    static constexpr u32 kWorkers = BN >= 128 ? 8 : 4, kThreads = 64 + kWorkers * 32, kStaging = kWorkers * 32 * 128;
    static constexpr u32 kA = 128 * 128, kBRows = BN / CTAS, kB = kBRows * 128, kStage = kA + kB;
    // copies under way: as many as one block an SM has room for, or, where tiles are small and
    // blocks many, half of them to each of two
    static constexpr u32 fit(u32 room) { return (room - 2048 - kStaging) / kStage < 8 ? (room - 2048 - kStaging) / kStage : 8; }
    static constexpr u32 kStages = fit(227 * 1024), kFewStages = BN >= 128 ? kStages : fit(113 * 1024);
    // columns of TMEM: of one of two tiles under way, and of those and the sums of a long tile's earlier runs
    static constexpr u32 kColumns = BN < 32 ? 32 : BN, kAllColumns = BN == 256 ? 512 : 4 * kColumns;
    static constexpr u32 smem(u32 stages) { return 1024 + stages * kStage + kStaging + 256; }
};

struct Units {                      // what the blocks (or pairs) do, in order
    u32 tiles_m, tiles_n;
    u32 columns;                    // columns of tiles that come first
    u32 whole;                      // tiles done in one piece; of each one after them
    u32 parts;                      // this many pieces along k
    u32 total;                      // units in all
    u32 steps;                      // steps of k of a tile
    u32 stages;                     // copies under way a block
    u32 chain;                      // steps that are summed in one go (below)
    u32 half_steps;                 // steps after which A's second part begins (0: none)
};

struct Args {
    Units u;
    Finish f;
    u32 what;                       // instruction descriptor
    float *partial;                 // sums of tiles in pieces
};

// Tiles go in columns of eight along m, so that those under way share both operands in L2:
// first those of the first u.columns columns, then the others.
__device__ __forceinline__ void tile_at(const Units &u, u32 i, u32 &m, u32 &n)
{
    u32 start = 0, across = u.columns;
    if (i >= across * u.tiles_m) {
        i -= across * u.tiles_m;
        start = across;
        across = u.tiles_n - across;
    }
    const u32 band = 8 * across, b = i / band, rows = min(8u, u.tiles_m - 8 * b), j = i - b * band;
    n = j / rows;
    m = 8 * b + j - n * rows;
    n += start;
}

template <bool MN> __device__ __forceinline__ u64 operand(u32 at)
{
    // address / 16; distance of pieces / 16 (64 rows each) where the rows are contiguous; of eight
    // lines / 16; version 1; 128-byte swizzle
    const u64 pieces = MN ? 8192 / 16 : 1;
    return (u64)(at >> 4 & 0x3FFF) | pieces << 16 | (u64)(1024 / 16) << 32 | 1ull << 46 | 2ull << 61;
}

// SWAP: A holds the result's columns and B its rows, for fewer rows than a tile of A has.
template <int CTAS, int BN, bool A_MN, bool B_MN, bool SWAP>
__global__ void __launch_bounds__(Tile<CTAS, BN>::kThreads, BN >= 128 ? 1 : 2)
k_product(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap a2_map,
          const __grid_constant__ CUtensorMap b_map, const __grid_constant__ CUtensorMap y_map,
          const __grid_constant__ CUtensorMap z_map, const __grid_constant__ CUtensorMap residual_map,
          const __grid_constant__ Args args)
{
    using S = Tile<CTAS, BN>;
    extern __shared__ unsigned char raw[];
    const u32 base = (shared_at(raw) + 1023) & ~1023u;
    const u32 stages = S::kStages == S::kFewStages ? S::kStages : args.u.stages;
    const u32 staging = base + stages * S::kStage, bars = staging + S::kStaging;
    const u32 full = bars, empty = full + 8 * stages, done = empty + 8 * stages, taken = done + 16,
              drained = taken + 16, slot = drained + 8, residuals = slot + 8;
    const u32 warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    u32 rank = 0;
    if constexpr (CTAS == 2 || SWAP) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const Units &u = args.u;
    const u32 cluster = SWAP ? u.parts : CTAS, worker = blockIdx.x / cluster, workers = gridDim.x / cluster;
    const u32 pair_rank = CTAS == 2 ? rank : 0;

    if (threadIdx.x == 0) {
        for (u32 i = 0; i < stages; i++) {
            barrier_init(full + 8 * i, 1);
            barrier_init(empty + 8 * i, 1);
        }
        for (u32 i = 0; i < 2; i++) {
            barrier_init(done + 8 * i, 1);
            barrier_init(taken + 8 * i, S::kWorkers * CTAS);
        }
        barrier_init(drained, 1);
        for (u32 i = 0; i < S::kWorkers; i++) barrier_init(residuals + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (CTAS == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(S::kAllColumns) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(S::kAllColumns) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (CTAS == 2) meet();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    u32 tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    auto unit = [&](u32 i, u32 &m, u32 &n, u32 &first, u32 &last) {
        u32 tile = i, part = 0, parts = 1;
        if (SWAP) {
            part = rank;
            parts = u.parts;
        } else if (i >= u.whole) {
            tile = u.whole + (i - u.whole) / u.parts;
            part = (i - u.whole) % u.parts;
            parts = u.parts;
        }
        tile_at(u, tile, m, n);
        first = (u32)((u64)u.steps * part / parts);
        last = (u32)((u64)u.steps * (part + 1) / parts);
    };

    bool ok = true;
    if (warp == 0) {
        if (one_lane()) {                                         // copies
            u32 s = 0, turn = 0;
            u64 issued = 0;
            for (u32 i = worker; i < u.total && ok; i += workers) {
                u32 m, n, first, last;
                unit(i, m, n, first, last);
                const int row_a = (int)(m * S::kRows + pair_rank * 128), row_b = (int)(n * BN + pair_rank * S::kBRows);
                for (u32 k = first; k < last; k++) {
                    if (!barrier_wait(empty + 8 * s, turn ^ 1)) { ok = false; break; }
                    const bool second = u.half_steps && k >= u.half_steps;
                    const CUtensorMap *a = second ? &a2_map : &a_map;
                    const int at = (int)((second ? k - u.half_steps : k) * kStep);
                    const u32 to = base + s * S::kStage;
                    u32 bar = full + 8 * s;
                    if (pair_rank == 0)
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(CTAS * S::kStage) : "memory");
                    if constexpr (CTAS == 2) bar = at_leader(bar);
                    if constexpr (A_MN) {
                        copy_tile<CTAS>(to, a, row_a, at, bar);
                        copy_tile<CTAS>(to + 8192, a, row_a + 64, at, bar);
                    } else {
                        copy_tile<CTAS>(to, a, at, row_a, bar);
                    }
                    if constexpr (B_MN) {
#pragma unroll
                        for (u32 j = 0; j < S::kBRows / 64; j++) copy_tile<CTAS>(to + S::kA + j * 8192, &b_map, row_b + 64 * j, at, bar);
                    } else {
                        copy_tile<CTAS>(to + S::kA, &b_map, at, row_b, bar);
                    }
                    issued++;
                    if (++s == stages) { s = 0; turn ^= 1; }
                }
            }
            // The copies under way end before the block does, and so do the arrivals that tell
            // that they were used.  After a wait that ran out the former are waited for, both
            // blocks' of a pair, which the leader's barriers count; else the latter.
            if (ok || pair_rank == 0)
                for (u32 j = 0; j < stages && j < issued; j++) {
                    s = s ? s - 1 : stages - 1;
                    if (s == stages - 1) turn ^= 1;
                    barrier_wait((ok ? empty : full) + 8 * s, turn);
                }
        }
    } else if (warp == 1) {
        if (pair_rank == 0 && one_lane()) {                       // multiplies
            u32 s = 0, turn = 0, buffer = 0, buffer_turn = 0;
            for (u32 i = worker; i < u.total && ok; i += workers) {
                u32 m, n, first, last;
                unit(i, m, n, first, last);
                for (u32 k = first; k < last && ok;) {
                    ok = barrier_wait(taken + 8 * buffer, buffer_turn ^ 1);
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const u32 sums = tmem + buffer * S::kColumns, start = k, end = min(last, k + u.chain);
                    for (; k < end && ok; k++) {
                        ok = barrier_wait(full + 8 * s, turn);
                        if (!ok) break;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const u64 a = operand<A_MN>(base + s * S::kStage), b = operand<B_MN>(base + s * S::kStage + S::kA);
#pragma unroll
                        for (u32 j = 0; j < kStep / 16; j++)  // 16 k: 32 bytes along a line, or 16 lines
                            multiply<CTAS>(sums, a + j * (A_MN ? 2048 / 16 : 32 / 16), b + j * (B_MN ? 2048 / 16 : 32 / 16),
                                           args.what, k > start || j);
                        arrive_after_products<CTAS>(empty + 8 * s);
                        if (++s == stages) { s = 0; turn ^= 1; }
                    }
                    if (ok) arrive_after_products<CTAS>(done + 8 * buffer);
                    buffer ^= 1;
                    if (buffer == 0) buffer_turn ^= 1;
                }
            }
            if (!ok) {
                arrive_after_products<CTAS>(drained);
                barrier_wait(drained, 0);
            }
        }
    } else {                                                      // finish
        const u32 w = warp & 3;                                   // a warp reads its quarter of TMEM's lanes
        const u32 mine = staging + (warp - 2) * 32 * 128, share = (warp - 2) / 4;
        constexpr u32 kShares = S::kWorkers / 4;
        const u32 residual_bar = residuals + (warp - 2) * 8;
        u32 buffer = 0, buffer_turn = 0, residual_turn = 0;
        for (u32 i = worker; i < u.total && ok; i += workers) {
            u32 m, n, first, last;
            unit(i, m, n, first, last);
            constexpr u32 kRun = BN < 32 ? 16 : 32, kShare = BN / kShares;
            const u64 row0 = (u64)m * S::kRows + pair_rank * 128 + w * 32, col0 = (u64)n * BN;
            float *part = SWAP || i < u.whole ? nullptr
                        : args.partial + (u64)(i - u.whole) * (S::kRows * BN) + pair_rank * 128 * BN;
            // the residual is on its way while the tile is summed
            const bool fetched = !SWAP && !part && args.f.by_tma && args.f.residual && row0 < args.f.m && col0 + share * kShare < args.f.n;
            if (fetched) fetch_residual(mine, lane, residual_bar, &residual_map, (int)(col0 + share * kShare), (int)row0);
            // The tensor core's additions cut what is beyond 32 bits off, so an error of a long
            // chain grows with its length (2.4e-6 of the norm after 2048 products): where the result has 32 bits
            // or the chain is very long, it is summed in runs of u.chain steps, and a run's sum is
            // added, rounded to nearest, to the sum of those before it (in TMEM too).
            const u32 earlier = tmem + 2 * S::kColumns + (w << 21);
            u32 k = first;
            const auto arrived = [&] {
                ok = barrier_wait(done + 8 * buffer, buffer_turn);
                ok = __all_sync(kFull, ok);
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                return ok;
            };
            const auto taken_over = [&] {
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                // What it tells is that TMEM has been read (the fence above): a release would
                // also wait for this tile's stores, which took as long as a short tile's products.
                if (lane == 0) {
                    if constexpr (CTAS == 2)
                        asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(at_leader(taken + 8 * buffer)) : "memory");
                    else
                        asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(taken + 8 * buffer) : "memory");
                }
                buffer ^= 1;
                if (buffer == 0) buffer_turn ^= 1;
            };
            if constexpr (BN < 256) {
                for (; last - k > u.chain; k += u.chain) {
                    if (!arrived()) break;
                    const u32 sums = tmem + buffer * S::kColumns + (w << 21);
                    for (u32 c = share * kShare; c < (share + 1) * kShare; c += kRun) {
                        u32 v[kRun], e[kRun];
                        load_sums(sums + c, v);
                        if (k > first) {
                            load_sums(earlier + c, e);
#pragma unroll
                            for (u32 j = 0; j < kRun; j++) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(e[j]));
                        }
                        store_sums(earlier + c, v);
                    }
                    taken_over();
                }
            }
            if (!ok || !arrived()) {
                if (fetched) barrier_wait(residual_bar, residual_turn);
                break;
            }
            const u32 sums = tmem + buffer * S::kColumns + (w << 21);
            const auto load_all = [&](u32 c, auto &v) {           // the sums of columns c ..
                load_sums(sums + c, v);
                if constexpr (BN < 256)
                    if (k > first) {
                        std::remove_reference_t<decltype(v)> e;
                        load_sums(earlier + c, e);
#pragma unroll
                        for (u32 j = 0; j < sizeof(v) / 4; j++) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(e[j]));
                    }
            };
            if constexpr (SWAP) {
                // lanes are columns of the result, TMEM's columns its rows
                const u64 column = row0 + lane;
                constexpr int kAtOnce = BN < 32 ? BN : 32;
                const auto all = [&](auto type) {
                    using OUT = decltype(type);
                    for (u32 c = 0; c < BN && col0 + c < args.f.m; c += kAtOnce) {
                        const u32 rows = (u32)min((u64)kAtOnce, args.f.m - (col0 + c));
                        const bool inside = column < args.f.n;
                        OUT residual[kAtOnce];
                        if (args.f.residual && inside) read_residual(args.f, col0 + c, column, rows, residual);
                        float v[kAtOnce];
                        load_all(c, *reinterpret_cast<u32(*)[kAtOnce]>(&v[0]));
                        if (inside) finish_column(args.f, col0 + c, column, rows, v, residual);
                    }
                };
                if (u.parts > 1) {                                // [rows][128 columns], in the copies' place
                    for (u32 c = 0; c < BN && col0 + c < args.f.m; c += kAtOnce) {
                        u32 v[kAtOnce];
                        load_all(c, v);
#pragma unroll
                        for (int j = 0; j < kAtOnce; j++)
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + ((c + j) * 128 + w * 32 + lane) * 4), "r"(v[j]) : "memory");
                    }
                } else if (args.f.out == MV_BF16) {
                    all(__nv_bfloat16());
                } else if (args.f.out == MV_F16) {
                    all(__half());
                } else {
                    all(0.0f);
                }
            } else if (args.f.by_tma && !part) {
                const auto all = [&](auto type) {
                    using OUT = decltype(type);
                    constexpr int N = 128 / sizeof(OUT);
                    for (u32 c = share * kShare; c < (share + 1) * kShare && col0 + c < args.f.n; c += N) {
                        float v[N];
#pragma unroll
                        for (int j = 0; j < N; j += 32) load_all(c + j, *reinterpret_cast<u32(*)[32]>(&v[j]));
                        if (fetched) {
                            if (c != share * kShare) fetch_residual(mine, lane, residual_bar, &residual_map, (int)(col0 + c), (int)row0);
                            ok = barrier_wait(residual_bar, residual_turn);
                            ok = __all_sync(kFull, ok);
                            if (!ok) return;
                            residual_turn ^= 1;
                        }
                        if (row0 < args.f.m) finish_tile<OUT>(args.f, mine, lane, &y_map, &z_map, row0, col0 + c, v);
                    }
                };
                if (args.f.out == MV_BF16) all(__nv_bfloat16());
                else if (args.f.out == MV_F16) all(__half());
                else all(0.0f);
            } else {
                for (u32 c = share * kShare; c < (share + 1) * kShare && col0 + c < args.f.n; c += 32) {
                    u32 v[32];
                    load_all(c, v);
                    if (part) {                                   // [columns / 4][rows][4]
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            *reinterpret_cast<uint4 *>(part + ((c / 4 + j) * 128 + w * 32 + lane) * 4) =
                                make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                        continue;
                    }
                    // A lane holds a row: through shared memory, so that eight lanes share
                    // one and its accesses are whole sectors.
                    __syncwarp();
#pragma unroll
                    for (u32 j = 0; j < 8; j++)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + lane * 128 + ((j ^ (lane & 7)) * 16)),
                                     "r"(v[4 * j]), "r"(v[4 * j + 1]), "r"(v[4 * j + 2]), "r"(v[4 * j + 3]) : "memory");
                    __syncwarp();
                    if (args.f.out == MV_BF16) finish_column<__nv_bfloat16>(args.f, mine, lane, row0, col0 + c + lane);
                    else if (args.f.out == MV_F16) finish_column<__half>(args.f, mine, lane, row0, col0 + c + lane);
                    else finish_column<float>(args.f, mine, lane, row0, col0 + c + lane);
                }
            }
            taken_over();
        }
    }
    if (warp > 1 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");      // the stores have ended
    if (!ok && (warp < 2 || lane == 0)) atomicAdd(&g_gave_up, 1u);
    __syncwarp();
    if (SWAP && u.parts > 1) {
        // The pieces' sums meet through the cluster's shared memory: each block finishes
        // some of the quads of columns, adding the pieces in their order.
        u32 m, n;
        tile_at(u, worker, m, n);
        const u64 row0 = (u64)n * BN, column0 = (u64)m * 128;
        const u32 quads = (u32)min((u64)BN, args.f.m - row0) * 32;
        meet();
        for (u32 q = rank * S::kThreads + threadIdx.x; q < quads; q += u.parts * S::kThreads) {
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (u32 p = 0; p < u.parts; p++) {
                float w[4];
                u32 there;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(base + q * 16), "r"(p));
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]) : "r"(there) : "memory");
#pragma unroll
                for (int i = 0; i < 4; i++) v[i] += w[i];
            }
            finish4(args.f, row0 + q / 32, column0 + q % 32 * 4, v);
        }
        meet();
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (CTAS == 2) meet();
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if constexpr (CTAS == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kAllColumns));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kAllColumns));
    }
}

// Tiles done in pieces along k: the pieces' sums are added in their order, or,
// where few tiles would leave most SMs without work, those of each of eight
// groups of threads and then the groups' (4 tiles of 19 pieces: 10.9 us so 9.4;
// 28 tiles of 8: 16.5 us, in groups 23.6).
template <int CTAS, int BN, u32 GROUPS> __global__ void __launch_bounds__(256) k_join(const __grid_constant__ Args args)
{
    using S = Tile<CTAS, BN>;
    constexpr u32 kEach = 256 / GROUPS;     // groups of so many threads
    __shared__ float4 sums[GROUPS > 1 ? GROUPS : 1][32];
    const Units &u = args.u;
    // kEach / 8 rows x 32 of a tile a block
    constexpr u32 kDown = S::kRows / (kEach / 8), kAcross = BN / 32;
    const u32 tile = blockIdx.x / (kDown * kAcross), here = blockIdx.x % (kDown * kAcross), t = threadIdx.x % kEach, group = threadIdx.x / kEach;
    u32 m, n;
    tile_at(u, u.whole + tile, m, n);
    const u32 r = (here / kAcross) * (kEach / 8) + (t >> 3), c = (here % kAcross) * 32 + (t & 7) * 4;
    const u64 row = (u64)m * S::kRows + r, column = (u64)n * BN + c, at = (r / 128) * (128 * BN) + ((c / 4) * 128 + (r & 127)) * 4;
    const bool mine = row < args.f.m && column < args.f.n;
    constexpr u32 kPiece = S::kRows * BN;
    const float *p = args.partial + (u64)tile * u.parts * kPiece + at;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (mine)
#pragma unroll 8
        for (u32 i = group; i < u.parts; i += GROUPS) {
            const float4 w = *reinterpret_cast<const float4 *>(p + (u64)i * kPiece);
            v[0] += w.x; v[1] += w.y; v[2] += w.z; v[3] += w.w;
        }
    if constexpr (GROUPS > 1) {
        sums[group][t] = make_float4(v[0], v[1], v[2], v[3]);
        __syncthreads();
        if (group) return;
#pragma unroll
        for (u32 i = 1; i < GROUPS; i++) {
            const float4 w = sums[i][t];
            v[0] += w.x; v[1] += w.y; v[2] += w.z; v[3] += w.w;
        }
    }
    if (mine) finish4(args.f, row, column, v);
}

// ---- operands as the copies want them ---------------------------------------
// Rows that lie on no 16-byte boundary are copied to where they do, and 32-bit
// values are split into two bfloat16, the nearest and the nearest to what that
// leaves: together within 2^-17 of the value or, under 2^-117, within half of
// bfloat16's smallest step, 2^-134.
struct PackArgs {
    const unsigned short *from[2];
    unsigned short *to[2];
    u64 stride[2], rows[2], cols[2];
};
// Two arrays at most (blockIdx.y), eight values a thread and four such under way.
// They are read by aligned words of two values, each of which holds one of the row at least.
constexpr u32 kPackThreads = 256, kPackAhead = 4;
__global__ void __launch_bounds__(kPackThreads) k_pack(const PackArgs a)
{
    const u32 which = blockIdx.y;
    const u64 cols = a.cols[which], stride = a.stride[which], pieces = (cols + 7) / 8, n = a.rows[which] * pieces;
    const unsigned short *all = a.from[which];
    uint4 *to = reinterpret_cast<uint4 *>(a.to[which]);
    for (u64 i0 = (u64)blockIdx.x * (kPackThreads * kPackAhead) + threadIdx.x; i0 < n; i0 += (u64)gridDim.x * (kPackThreads * kPackAhead)) {
        u32 w[kPackAhead][5], odd[kPackAhead];
        u64 c[kPackAhead];
#pragma unroll
        for (u32 j = 0; j < kPackAhead; j++) {
            const u64 i = i0 + j * kPackThreads;
            if (i >= n) break;
            const u64 r = n >> 32 ? i / pieces : (u32)i / (u32)pieces;
            c[j] = (i - r * pieces) * 8;
            const unsigned short *from = all + r * stride;
            odd[j] = (u32)(reinterpret_cast<uintptr_t>(from) >> 1 & 1);
            const u32 *words = reinterpret_cast<const u32 *>(from - odd[j]) + c[j] / 2;
            const u64 left = (cols + odd[j] + 1) / 2 - c[j] / 2;           // words of the row from here on
#pragma unroll
            for (u32 k = 0; k < 5; k++) w[j][k] = k < left ? words[k] : 0;
        }
#pragma unroll
        for (u32 j = 0; j < kPackAhead; j++) {
            const u64 i = i0 + j * kPackThreads;
            if (i >= n) break;
            u32 v[4];
#pragma unroll
            for (u32 k = 0; k < 4; k++) {
                v[k] = odd[j] ? __funnelshift_r(w[j][k], w[j][k + 1], 16) : w[j][k];
                if (c[j] + 2 * k + 1 >= cols) v[k] = c[j] + 2 * k < cols ? v[k] & 0xFFFFu : 0;
            }
            to[i] = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
}
__global__ void __launch_bounds__(256) k_split(const float *from, u64 stride, u64 rows, u64 cols, __nv_bfloat16 *to, u64 to_stride, u64 second)
{
    const u64 n = rows * to_stride / 4, step = (u64)gridDim.x * 256, quads = to_stride / 4;
    const bool wide = stride % 4 == 0 && (reinterpret_cast<uintptr_t>(from) & 15) == 0;
    for (u64 i = (u64)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
        const u64 r = i / quads, c = (i - r * quads) * 4;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, rest[4];
        __nv_bfloat16 most[4];
        if (c < cols) load4<float>(from, r * stride + c, wide, cols - c < 4 ? (u32)(cols - c) : 4, v);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            most[j] = fabsf(v[j]) > 3.3895e38f && fabsf(v[j]) < INFINITY ? __float2bfloat16_rz(v[j])      // would round to infinity
                                                                         : __float2bfloat16_rn(v[j]);
            rest[j] = v[j] - __bfloat162float(most[j]);
            if (!(fabsf(rest[j]) < INFINITY)) rest[j] = 0.0f;        // of infinities nothing is left
        }
        uint2 w;
        memcpy(&w, most, 8);
        *reinterpret_cast<uint2 *>(to + i * 4) = w;
        store4<__nv_bfloat16>(to + second, i * 4, true, 4, rest);
    }
}

// ---- columns' sums (dbias) --------------------------------------------------
// A warp adds up every eighth row of a run, eight columns a lane; the block's
// eight warps' sums are added, and the runs' by the second kernel, both in order.
constexpr u32 kSumLanes = 8, kSumColumns = 8 * 32;
template <class T> __global__ void __launch_bounds__(256)
k_column_sums(const T *from, u64 stride, u64 rows, u64 cols, u64 run, u32 wide, float *sums)
{
    __shared__ float part[kSumLanes][kSumColumns];
    const u32 lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const u64 c = (u64)blockIdx.x * kSumColumns + lane * 8, first = blockIdx.y * run, last = min(first + run, rows);
    float s[8] = {};
    if (c < cols)
#pragma unroll 4
        for (u64 r = first + warp; r < last; r += kSumLanes)
#pragma unroll
            for (u32 i = 0; i < 8; i += 4) {
                float v[4];
                load4<T>(from, r * stride + c + i, wide, c + i >= cols ? 0 : cols - (c + i) < 4 ? (u32)(cols - (c + i)) : 4, v);
#pragma unroll
                for (u32 j = 0; j < 4; j++) s[i + j] += v[j];
            }
#pragma unroll
    for (u32 i = 0; i < 8; i++) part[warp][i * 32 + lane] = s[i];
    // the kernel before this one may still run: what is written here is nobody's until it has ended
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    const u64 mine = (u64)blockIdx.x * kSumColumns + (threadIdx.x & 31) * 8 + (threadIdx.x >> 5);
    if (mine < cols) {
        float v = part[0][threadIdx.x];
        for (u32 i = 1; i < kSumLanes; i++) v += part[i][threadIdx.x];
        sums[blockIdx.y * cols + mine] = v;
    }
}
template <class T> __global__ void __launch_bounds__(128) k_add_runs(const float *sums, u64 runs, u64 cols, T *to)
{
    const u64 c = (u64)blockIdx.x * 128 + threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c >= cols) return;
    float s = 0.0f;
#pragma unroll 16
    for (u64 i = 0; i < runs; i++) s += sums[i * cols + c];
    to[c] = from_float<T>(s);
}

// ---- host ------------------------------------------------------------------
using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                            const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encoder()
{
    static Encode found = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess) p = nullptr;
        return reinterpret_cast<Encode>(p);
    }();
    return found;
}

// One side of a product: `rows` by `k`, contiguous along k, or (mn) k by `rows`, contiguous along the rows.
struct Side {
    const void *p;
    u64 rows, k, stride;
    bool mn;
};
bool map_side(CUtensorMap *map, const Side &s, u32 dtype, u32 box_rows)
{
    const Encode encode = encoder();
    if (!encode) return false;
    const cuuint64_t dims[2] = {s.mn ? s.rows : s.k, s.mn ? s.k : s.rows}, strides[1] = {s.stride * 2};
    const cuuint32_t box[2] = {kStep, s.mn ? kStep : box_rows}, each[2] = {1, 1};
    return encode(map, dtype == MV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                  const_cast<void *>(s.p), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A result or residual, 32 rows of 128 bytes at a time.
bool map_result(CUtensorMap *map, void *p, u64 rows, u64 cols, u64 stride, u32 type)
{
    const u32 size = (u32)dtype_size(type);
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {stride * size};
    const cuuint32_t box[2] = {128 / size, 32}, each[2] = {1, 1};
    return encoder()(map, type == MV_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                        : type == MV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, dims, strides, box, each,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The kinds of tile: A's rows and B's a tile, and whether two blocks share an SM where there are enough.
enum Kind { kPair256, kPair128, kOne128, kOne64, kSwap64, kSwap16, kKinds };
struct KindOf {
    u32 rows, cols;
    bool two, swap;
};
constexpr KindOf kKind[kKinds] = {{256, 256, false, false}, {256, 128, false, false}, {128, 128, false, false}, {128, 64, true, false},
                                  {128, 64, true, true}, {128, 16, true, true}};
constexpr u64 kCluster = 8;             // blocks that share a tile of the kinds that swap, at most

struct Plan {
    Kind kind;
    bool two;                           // two blocks an SM
    Units u;
    u64 blocks, partial;                // blocks; bytes of pieces' sums
};

// What a product would take with one kind of tile, in cycles, as measured on
// GB300: a step of 64 k takes a pair of blocks 530 cycles (the products
// themselves 512), a single one what its copies take, 64 bytes a cycle and SM,
// but no less than a copy's 2000 cycles over the copies under way; memory gives 3300 bytes a cycle.
// Checked by forcing each kind, us: 2048 x 5120 to 2560: 45.7 (pairs), 51.9
// (128 x 128), 70.3 (128 x 64); 1 x 20480 to 5120: 39 (swapped, 16), 42
// (swapped, 64), 50 (128 x 128), 64 (pairs); 64 x 5120 to 5120: 20 (swapped, 64),
// 25 (swapped, 16), 23 (128 x 128).
//
// alike: every row's sums are to be made of the same pieces, so that equal rows have
// equal results: tiles go in pieces by whole columns.  What that costs: by this estimate
// 0.2% on average over sizes spread over their logarithm, and more than 6% for one product in a
// hundred, where few columns have many tiles each (20000 x 7168 to 256 took 78 us, so 104;
// 3000 x 4096 to 4096 in 32 bits 131, so 134; 2048 x 5120 to 5120 78 either way).
Plan plan_kind(Kind kind, u64 m, u64 n, u64 steps, u32 chain, bool alike, u32 sms, double &best)
{
    const KindOf &k = kKind[kind];
    const bool pair = kind <= kPair128;
    const u64 a = k.swap ? n : m, b = k.swap ? m : n, tm = (a + k.rows - 1) / k.rows, tn = (b + k.cols - 1) / k.cols, tiles = tm * tn;
    const u64 each = pair ? 2 : 1;                                     // blocks a unit
    const double bytes = (k.rows + k.cols) * (pair ? 64 : 128);
    const double memory = (double)(m + n) * (double)steps * 128 / (sms * 21.7);
    Plan p = {};
    best = INFINITY;
    auto consider = [&](u64 whole, u64 left, u64 parts, u64 blocks, u64 slots, bool two, double join) {
        // TMEM has no room for earlier sums beside the largest tiles
        if (kind == kPair256 && (steps + (whole ? 1 : parts) - 1) / (whole ? 1 : parts) > chain) return;
        const double step = kind == kPair256 ? 530 : kind == kPair128 ? 400 : std::max(bytes / 64 * (two ? 2 : 1), two || kind == kOne128 ? 400.0 : 250.0);
        // rounds of whole tiles, the last of which pieces may fill up, and of pieces
        const u64 full = (whole + slots - 1) / slots, rounds = (whole + left * parts + slots - 1) / slots - full;
        const double work = (double)full * ((double)steps * step + 400) +
                            (double)rounds * ((double)((steps + parts - 1) / parts) * step + 2000);
        const double cost = std::max(work, memory) + 0.35 * std::min(work, memory) + join + 2000;
        if (cost >= best) return;
        best = cost;
        p.kind = kind;
        p.two = two;
        p.u = {(u32)tm, (u32)tn, (u32)(k.swap || parts == 1 || !alike ? tn : whole / tm), (u32)(k.swap || parts == 1 ? tiles : whole), (u32)parts,
               (u32)(k.swap || parts == 1 ? tiles : whole + left * parts), (u32)steps, 0, chain, 0};
        p.blocks = blocks;
        p.partial = k.swap || parts == 1 ? 0 : left * parts * (u64)k.rows * k.cols * 4;
    };
    if (k.swap) {                       // every tile in as many pieces, a block each, in one cluster
        for (u64 parts = 1; parts <= std::min(kCluster, steps); parts++) {
            const bool two = tiles * parts > sms;
            // clusters of seven and eight leave SMs out: 1 x 20480 to 5120 in 6 pieces 39.4 us, in 7 49.2
            const u64 slots = parts > 6 ? (u64)sms * (two ? 3 : 2) / (two ? 2 : 3) : (u64)sms * (two ? 2 : 1);
            // more than one round costs its blocks' starts: 1 x 5120 to 20480 in one piece 39.6 us, in three 45.4
            if (parts > 1 && tiles * parts > slots) continue;
            consider(0, tiles, parts, tiles * parts, std::max<u64>(1, slots), two, parts > 1 ? 1000 : 0);
        }
        return p;
    }
    // whole tiles in rounds of all slots, and what is left in pieces: as many as fill one to four more rounds, or fewer
    const bool two = k.two && tiles > sms;
    const u64 slots = std::max<u64>(1, (u64)sms * (two ? 2 : 1) / each), rest = tiles % slots;
    auto in_parts = [&](u64 left, u64 parts) {
        const u64 whole = tiles - left;
        const double join = parts > 1 ? 6000 + (double)(parts * left) * k.rows * k.cols * 4 / (sms * 24.0) : 0;
        consider(whole, left, parts, std::min<u64>(whole + left * parts, slots) * each, slots, two, join);
    };
    in_parts(rest, 1);
    if (!rest) return p;
    // what goes in pieces: the rest, or columns, as few as hold that many tiles or up to two more
    const u64 unit = alike ? tm : rest, fewest = (rest + unit - 1) / unit, most = alike ? std::min(tn, fewest + 2) : 1;
    for (u64 units = fewest; units <= most; units++) {
        const u64 left = units * unit, begun = (tiles - left) % slots;      // of a round, by whole tiles
        for (u64 round = 1; round <= 4; round++) {
            const u64 parts = std::min<u64>(steps, (round * slots - begun) / left);
            if (parts > 1) in_parts(left, parts);
        }
        for (u64 parts : {2, 4, 8, 12})
            if (parts < slots / left && parts <= steps) in_parts(left, parts);
    }
    return p;
}

// chain: the longest run of steps that may be summed in one go.
Plan plan(u64 m, u64 n, u64 steps, u32 chain, bool swaps, bool alike, u32 sms)
{
    Plan best = {};
    double least = INFINITY;
    for (int kind = 0; kind < kKinds; kind++) {
        if (kKind[kind].swap && !swaps) continue;
        double cost;
        const Plan p = plan_kind((Kind)kind, m, n, steps, chain, alike, sms, cost);
        if (cost < least) { least = cost; best = p; }
    }
    return best;
}

template <int CTAS, int BN, bool A_MN, bool B_MN, bool SWAP>
int run_kind(const Side &a, const void *a2, const Side &b, u32 dtype, const Plan &p, Args &args, bool early, cudaStream_t stream)
{
    using S = Tile<CTAS, BN>;
    const auto kernel = k_product<CTAS, BN, A_MN, B_MN, SWAP>;
    CUtensorMap maps[6];
    Side second = a;
    second.p = a2 ? a2 : a.p;
    if (!map_side(&maps[0], a, dtype, 128) || !map_side(&maps[1], second, dtype, 128) ||
        !map_side(&maps[2], b, dtype, S::kBRows))
        return MV_ECUDA;
    maps[3] = maps[4] = maps[5] = maps[0];
    Finish &f = args.f;
    const u64 size = dtype_size(f.out);
    f.by_tma = !SWAP && f.n * size % 16 == 0 && aligned(f.y, 16) && aligned(f.z, 16) && !(f.z && f.out == MV_F32) &&
               (!f.residual || (aligned(f.residual, 16) && f.residual_stride * size % 16 == 0));
    if (f.by_tma && (!map_result(&maps[3], f.y, f.m, f.n, f.n, f.out) || (f.z && !map_result(&maps[4], f.z, f.m, f.n, f.n, f.out)) ||
                     (f.residual && !map_result(&maps[5], const_cast<void *>(f.residual), f.m, f.n, f.residual_stride, f.out))))
        return MV_ECUDA;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::smem(S::kStages)) != cudaSuccess) return MV_ECUDA;
    // type of the sums: 32 bits; of both operands; which side is contiguous; the tile
    args.what = 1u << 4 | (dtype == MV_BF16 ? 1u << 7 | 1u << 10 : 0u) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u) |
                (u32)(BN >> 3) << 17 | (u32)(128 * CTAS >> 4) << 24;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((u32)p.blocks);
    cfg.blockDim = dim3(S::kThreads);
    args.u.stages = p.two ? S::kFewStages : S::kStages;
    cfg.dynamicSmemBytes = S::smem(args.u.stages);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    u32 attrs = 0;
    if (early) {
        attr[attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[attrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    const u32 cluster = SWAP ? p.u.parts : CTAS;
    if (cluster > 1) {
        attr[attrs].id = cudaLaunchAttributeClusterDimension;
        attr[attrs++].val.clusterDim = {cluster, 1, 1};
    }
    cfg.attrs = attr;
    cfg.numAttrs = attrs;
    if (cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], maps[3], maps[4], maps[5], args) != cudaSuccess) return MV_ECUDA;
    if (SWAP || p.u.parts == 1) return MV_OK;
    const u32 left = (p.u.total - p.u.whole) / p.u.parts;
    const u32 blocks = left * (S::kRows * BN / 1024);
    if (blocks >= 4 * sm_count()) return launch_after(k_join<CTAS, BN, 1>, dim3(blocks), 256, 0, stream, args);
    return launch_after(k_join<CTAS, BN, 8>, dim3(8 * blocks), 256, 0, stream, args);
}

// C = A B^T into args.f; with a2, A is the sum of two.  early: after a kernel of this call.
template <bool A_MN, bool B_MN>
int product(const Side &a, const void *a2, const Side &b, u32 dtype, Plan p, const Finish &f, float *partial, bool early, cudaStream_t stream)
{
    Args args = {};
    args.u = p.u;
    args.f = f;
    args.partial = partial;
    args.u.half_steps = a2 ? p.u.steps / 2 : 0;
    switch (p.kind) {
    case kPair256: return run_kind<2, 256, A_MN, B_MN, false>(a, a2, b, dtype, p, args, early, stream);
    case kPair128: return run_kind<2, 128, A_MN, B_MN, false>(a, a2, b, dtype, p, args, early, stream);
    case kOne128: return run_kind<1, 128, A_MN, B_MN, false>(a, a2, b, dtype, p, args, early, stream);
    case kOne64: return run_kind<1, 64, A_MN, B_MN, false>(a, a2, b, dtype, p, args, early, stream);
    default: break;
    }
    if constexpr (!A_MN && !B_MN) {     // the forward product alone: A and B change places
        if (p.kind == kSwap64) return run_kind<1, 64, false, false, true>(b, nullptr, a, dtype, p, args, early, stream);
        if (p.kind == kSwap16) return run_kind<1, 16, false, false, true>(b, nullptr, a, dtype, p, args, early, stream);
    }
    return MV_EINVAL;
}

u64 up(u64 v, u64 to) { return (v + to - 1) / to * to; }
u64 steps_of(u64 k) { return (k + kStep - 1) / kStep; }
bool copies(const void *p, u64 stride) { return aligned(p, 16) && stride % 8 == 0; }
bool wide(const void *p, u64 stride, u32 dtype) { return aligned(p, 4 * dtype_size(dtype)) && stride % 4 == 0; }
// Steps of 64 products summed in one go: 512 products (5e-7 of error) where the result has 32 bits, 32768
// (4e-5 of the result's norm, where the rounding to bfloat16 is 1.7e-3 and to float16 2.1e-4) where it has 16.
constexpr u32 kChain32 = 8, kChain16 = 512;
constexpr u64 kMostRows = 1ull << 30, kMostTiles = 1ull << 31;

// Arrays to be copied, and the launch that does it.
struct Packing {
    PackArgs a = {};
    u32 count = 0;
    u64 most = 0;
    const void *add(const void *from, u64 &stride, u64 rows, u64 cols, void *to)
    {
        a.from[count] = static_cast<const unsigned short *>(from);
        a.to[count] = static_cast<unsigned short *>(to);
        a.stride[count] = stride;
        a.rows[count] = rows;
        a.cols[count++] = cols;
        most = std::max(most, rows * ((cols + 7) / 8));
        stride = up(cols, 8);
        return to;
    }
    int run(cudaStream_t stream)
    {
        const u32 pairs = count;
        if (!pairs) return MV_OK;
        const dim3 grid((u32)std::min<u64>((most + kPackThreads * kPackAhead - 1) / (kPackThreads * kPackAhead), 1u << 16), pairs);
        count = 0;
        most = 0;
        return launch(k_pack, grid, kPackThreads, 0, stream, a);
    }
};

struct LinearLayout {
    u64 x, w, partial, total;
    Plan plan;
};
struct GradLayout {
    u64 x, w, dz, runs, partial, total;
    u64 run;                            // rows of dz a block of the columns' sums adds
    Plan dx, dw;
};

u32 planned_sms() { const u32 n = sm_count(); return n ? n : 152; }

int check(const mv_linear_desc *d)
{
    if (!d || !d->cols || !d->rows || (d->dtype != MV_F16 && d->dtype != MV_BF16) ||
        (d->out_dtype != d->dtype && d->out_dtype != MV_F32) || (d->bias_dtype != d->dtype && d->bias_dtype != MV_F32) ||
        d->act > MV_ACT_SILU || !std::isfinite(d->scale) || d->x_stride < d->cols || d->w_stride < d->cols ||
        (d->residual && d->residual_stride < d->rows))
        return MV_EINVAL;
    if (d->tokens > kMostRows || d->cols > kMostRows || d->rows > kMostRows || d->x_stride > 1ull << 36 ||
        d->w_stride > 1ull << 36 || d->residual_stride > 1ull << 36 || (d->tokens / 128 + 1) * (d->rows / 16 + 1) > kMostTiles)
        return MV_EOVERFLOW;
    return MV_OK;
}
LinearLayout layout(const mv_linear_desc *d)
{
    LinearLayout l = {};
    u64 at = 0;
    auto take = [&](u64 bytes) { const u64 here = at; at += up(bytes, 256); return here; };
    l.plan = plan(d->tokens, d->rows, steps_of(d->cols), d->out_dtype == MV_F32 ? kChain32 : kChain16, d->tokens <= 256, true, planned_sms());
    l.x = take(copies(d->x, d->x_stride) ? 0 : d->tokens * up(d->cols, 8) * 2);
    l.w = take(copies(d->w, d->w_stride) ? 0 : d->rows * up(d->cols, 8) * 2);
    l.partial = take(l.plan.partial);
    l.total = at;
    return l;
}

int check(const mv_linear_grad_desc *d)
{
    if (!d || !d->cols || !d->rows || (d->dtype != MV_F16 && d->dtype != MV_BF16) ||
        (d->dz_dtype != d->dtype && !(d->dz_dtype == MV_F32 && d->dtype == MV_BF16)) || d->x_stride < d->cols ||
        d->w_stride < d->cols || d->dz_stride < d->rows)
        return MV_EINVAL;
    if (d->tokens > kMostRows || d->cols > kMostRows || d->rows > kMostRows || d->x_stride > 1ull << 36 ||
        d->w_stride > 1ull << 36 || d->dz_stride > 1ull << 36 || (d->tokens / 128 + 1) * (d->cols / 64 + 1) > kMostTiles ||
        (d->rows / 128 + 1) * (d->cols / 64 + 1) > kMostTiles)
        return MV_EOVERFLOW;
    return MV_OK;
}
GradLayout layout(const mv_linear_grad_desc *d)
{
    GradLayout l = {};
    u64 at = 0;
    auto take = [&](u64 bytes) { const u64 here = at; at += up(bytes, 256); return here; };
    const u64 parts = d->dz_dtype == MV_F32 ? 2 : 1, sms = planned_sms();
    if (d->dx) l.dx = plan(d->tokens, d->cols, parts * steps_of(d->rows), kChain16, false, false, (u32)sms);
    if (d->dw) l.dw = plan(d->rows, d->cols, parts * steps_of(d->tokens), kChain16, false, false, (u32)sms);
    l.x = take(!d->dw || copies(d->x, d->x_stride) ? 0 : d->tokens * up(d->cols, 8) * 2);
    l.w = take(!d->dx || copies(d->w, d->w_stride) ? 0 : d->rows * up(d->cols, 8) * 2);
    l.dz = take(parts == 1 && copies(d->dz, d->dz_stride) ? 0 : parts * d->tokens * up(d->rows, 8) * 2);
    // runs long enough to be worth adding, enough of them for all SMs
    const u64 across = (d->rows + kSumColumns - 1) / kSumColumns;
    u64 runs = std::max<u64>(1, 4 * sms / across);
    l.run = std::max<u64>(64, up((d->tokens + runs - 1) / runs, kSumLanes));
    runs = (d->tokens + l.run - 1) / l.run;
    l.runs = take(d->dbias ? runs * d->rows * 4 : 0);
    l.partial = take(std::max(l.dx.partial, l.dw.partial));
    l.total = at;
    return l;
}

}  // namespace mvblock

using namespace mvblock;

extern "C" int mv_linear_workspace_bytes(const mv_linear_desc *d, uint64_t *bytes)
{
    if (!bytes) return MV_EINVAL;
    *bytes = 0;
    const int rc = check(d);
    if (rc != MV_OK || d->tokens == 0) return rc;
    *bytes = layout(d).total;
    return MV_OK;
}

extern "C" int mv_linear(const mv_linear_desc *d, void *workspace, uint64_t ws_bytes, void *stream)
{
    int rc = check(d);
    if (rc != MV_OK || d->tokens == 0) return rc;
    if (!d->x || !d->w || !d->y || !aligned(d->x, 2) || !aligned(d->w, 2) || !aligned(d->y, dtype_size(d->out_dtype)) ||
        !aligned(d->z, 2) || !aligned(d->bias, dtype_size(d->bias_dtype)) || !aligned(d->residual, dtype_size(d->out_dtype)) ||
        !aligned(workspace, 256))
        return MV_EINVAL;
    const LinearLayout l = layout(d);
    if (ws_bytes < l.total) return MV_ENOMEM;
    if (l.total && !workspace) return MV_EINVAL;
    if (!sm_count()) return MV_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    Side x = {d->x, d->tokens, d->cols, d->x_stride, false}, w = {d->w, d->rows, d->cols, d->w_stride, false};
    Packing packing;
    if (!copies(d->x, d->x_stride)) x.p = packing.add(d->x, x.stride, d->tokens, d->cols, ws + l.x);
    if (!copies(d->w, d->w_stride)) w.p = packing.add(d->w, w.stride, d->rows, d->cols, ws + l.w);
    const bool packed = packing.count != 0;
    rc = packing.run(s);
    if (rc != MV_OK) return rc;
    Finish f = {};
    f.bias = d->bias;
    f.residual = d->residual;
    f.y = d->y;
    f.z = d->z;
    f.m = d->tokens;
    f.n = d->rows;
    f.y_stride = d->rows;
    f.residual_stride = d->residual_stride;
    f.dtype = d->dtype;
    f.out = d->out_dtype;
    f.bias_type = d->bias_dtype;
    f.act = d->act;
    f.scale = d->scale;
    f.residual_wide = wide(d->residual, d->residual_stride, d->out_dtype);
    f.bias_wide = wide(d->bias, 0, d->bias_dtype);
    f.y_wide = wide(d->y, d->rows, d->out_dtype);
    f.z_wide = wide(d->z, d->rows, d->dtype);
    return product<false, false>(x, nullptr, w, d->dtype, l.plan, f, reinterpret_cast<float *>(ws + l.partial), packed, s);
}

extern "C" int mv_linear_backward_workspace_bytes(const mv_linear_grad_desc *d, uint64_t *bytes)
{
    if (!bytes) return MV_EINVAL;
    *bytes = 0;
    const int rc = check(d);
    if (rc != MV_OK || d->tokens == 0) return rc;
    *bytes = layout(d).total;
    return MV_OK;
}

extern "C" int mv_linear_backward(const mv_linear_grad_desc *d, void *workspace, uint64_t ws_bytes, void *stream)
{
    int rc = check(d);
    if (rc != MV_OK) return rc;
    if ((d->tokens && (!d->dz || (d->dw && !d->x) || (d->dx && !d->w))) || !aligned(d->dz, dtype_size(d->dz_dtype)) ||
        !aligned(d->x, 2) || !aligned(d->w, 2) || !aligned(d->dx, 2) || !aligned(d->dw, 2) || !aligned(d->dbias, 2) ||
        !aligned(workspace, 256))
        return MV_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (d->tokens == 0) {               // sums of nothing
        if (d->dw && cudaMemsetAsync(d->dw, 0, d->rows * d->cols * 2, s) != cudaSuccess) return MV_ECUDA;
        if (d->dbias && cudaMemsetAsync(d->dbias, 0, d->rows * 2, s) != cudaSuccess) return MV_ECUDA;
        return MV_OK;
    }
    const GradLayout l = layout(d);
    if (ws_bytes < l.total) return MV_ENOMEM;
    if (l.total && !workspace) return MV_EINVAL;
    if (!sm_count()) return MV_ECUDA;
    char *ws = static_cast<char *>(workspace);
    const void *dz = d->dz, *dz2 = nullptr, *x = d->x, *w = d->w;
    u64 dz_stride = d->dz_stride, x_stride = d->x_stride, w_stride = d->w_stride;
    const u64 padded = up(d->rows, 8);
    Packing packing;
    if ((d->dx || d->dw) && d->dz_dtype == MV_F32) {
        const u64 n = d->tokens * padded;
        const u32 blocks = (u32)std::min<u64>((n / 4 + 255) / 256, 1u << 16);
        rc = launch(k_split, dim3(blocks), 256, 0, s, static_cast<const float *>(d->dz), d->dz_stride, d->tokens, d->rows,
                    reinterpret_cast<__nv_bfloat16 *>(ws + l.dz), padded, n);
        dz = ws + l.dz;
        dz2 = ws + l.dz + n * 2;
        dz_stride = padded;
    } else if ((d->dx || d->dw) && !copies(d->dz, d->dz_stride)) {
        dz = packing.add(d->dz, dz_stride, d->tokens, d->rows, ws + l.dz);
    }
    if (d->dw && !copies(d->x, d->x_stride)) x = packing.add(d->x, x_stride, d->tokens, d->cols, ws + l.x);
    if (rc == MV_OK && packing.count == 2) rc = packing.run(s);
    if (d->dx && !copies(d->w, d->w_stride)) w = packing.add(d->w, w_stride, d->rows, d->cols, ws + l.w);
    bool early = dz != d->dz || x != d->x || packing.count;
    if (rc == MV_OK) rc = packing.run(s);
    Finish f = {};
    f.n = d->cols;
    f.y_stride = d->cols;
    f.dtype = f.out = f.bias_type = d->dtype;
    f.act = MV_ACT_NONE;
    f.scale = 1.0f;
    float *partial = reinterpret_cast<float *>(ws + l.partial);
    if (rc == MV_OK && d->dx) {
        f.m = d->tokens;
        f.y = d->dx;
        f.y_wide = wide(d->dx, d->cols, d->dtype);
        rc = product<false, true>({dz, d->tokens, d->rows, dz_stride, false}, dz2, {w, d->cols, d->rows, w_stride, true}, d->dtype,
                                  l.dx, f, partial, early, s);
        early = true;
    }
    if (rc == MV_OK && d->dw) {
        f.m = d->rows;
        f.y = d->dw;
        f.y_wide = wide(d->dw, d->cols, d->dtype);
        rc = product<true, true>({dz, d->rows, d->tokens, dz_stride, true}, dz2, {x, d->cols, d->tokens, x_stride, true}, d->dtype,
                                 l.dw, f, partial, early, s);
        early = true;
    }
    if (rc == MV_OK && d->dbias) {
        const u64 runs = (d->tokens + l.run - 1) / l.run;
        float *sums = reinterpret_cast<float *>(ws + l.runs);
        const dim3 grid((u32)((d->rows + kSumColumns - 1) / kSumColumns), (u32)runs);
        const u32 adders = (u32)((d->rows + 127) / 128), whole = wide(d->dz, d->dz_stride, d->dz_dtype);
        // after another kernel of this call they start while it ends: dz itself was there before that one
        if (d->dz_dtype == MV_F32)
            rc = launch_as(early, k_column_sums<float>, grid, 256, 0, s, static_cast<const float *>(d->dz), d->dz_stride, d->tokens, d->rows, l.run, whole, sums);
        else if (d->dz_dtype == MV_F16)
            rc = launch_as(early, k_column_sums<__half>, grid, 256, 0, s, static_cast<const __half *>(d->dz), d->dz_stride, d->tokens, d->rows, l.run, whole, sums);
        else
            rc = launch_as(early, k_column_sums<__nv_bfloat16>, grid, 256, 0, s, static_cast<const __nv_bfloat16 *>(d->dz), d->dz_stride, d->tokens, d->rows, l.run, whole, sums);
        if (rc == MV_OK)
            rc = d->dtype == MV_F16 ? launch_after(k_add_runs<__half>, dim3(adders), 128, 0, s, sums, runs, d->rows, static_cast<__half *>(d->dbias))
                                    : launch_after(k_add_runs<__nv_bfloat16>, dim3(adders), 128, 0, s, sums, runs, d->rows, static_cast<__nv_bfloat16 *>(d->dbias));
    }
    return rc;
}

extern "C" int mv_block_status(uint32_t *gave_up)
{
    if (!gave_up) return MV_EINVAL;
    // the copy alone waits for the default stream, and not for those that do not wait for it either
    if (cudaDeviceSynchronize() != cudaSuccess) return MV_ECUDA;
    return cudaMemcpyFromSymbol(gave_up, g_gave_up, sizeof *gave_up) == cudaSuccess ? MV_OK : MV_ECUDA;
}
