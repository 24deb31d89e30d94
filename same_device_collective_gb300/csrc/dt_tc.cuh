// Thin wrappers over the fifth-generation tensor core instructions (tcgen05),
// tensor memory and tiled TMA loads, and the descriptors they take.
//
// Operands are bf16 tiles in shared memory, cut into boxes of 64 columns and up
// to 128 rows: rows of 128 bytes, in the 128-byte swizzle that the TMA load
// applies (16-byte chunk c of row r lies at chunk c ^ (r mod 8)).  A box
// begins on a 1024-byte boundary.  An operand whose rows run along K ("K
// major") is boxes of 64 of K and all of its M or N; one whose rows run along
// M or N ("MN major") is boxes of 64 of M or N, each 128 deep in K.  Both are
// what a TMA load of a row-major matrix leaves, so no operand is ever
// transposed in memory.
#pragma once

#include <cuda.h>

#include <cstdint>

namespace dt {

constexpr uint32_t kBoxBytes = 128 * 128;   // a box of 128 rows; MN-major boxes lie this far apart

// Shared memory matrix descriptor: address, leading and stride byte offsets
// (in 16-byte units), the descriptor version of this architecture (bit 46)
// and the 128-byte swizzle (2 at bit 61).
//   K major: stride offset = 8 rows of 128 bytes; the leading offset is not used.
//   MN major: leading offset = from 64 columns to the next (kBoxBytes), stride
//   offset = 8 rows of K.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool mn_major)
{
    const uint64_t lead = mn_major ? kBoxBytes / 16 : 1, stride = 1024 / 16;
    return (uint64_t)((addr >> 4) & 0x3FFF) | lead << 16 | stride << 32 | 1ull << 46 | 2ull << 61;
}

// Instruction descriptor of kind::f16: fp32 accumulator, bf16 operands, the
// operands' major-ness, N / 8 and M / 16.
__host__ __device__ constexpr uint32_t mma_desc(uint32_t m, uint32_t n, bool a_mn_major, bool b_mn_major)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)a_mn_major << 15 | (uint32_t)b_mn_major << 16 | (n / 8) << 17 |
           (m / 16) << 24;
}

// The forms below take the number of CTAs that share a tile, CG: 1, or 2 for
// the two CTAs of a cluster.  As a pair each CTA holds its half of the rows of
// A and of the columns of B in its own shared memory, and its rows of the
// accumulator in its own tensor memory; the first one issues the products.

// One M x N x 16 product into tensor memory; `add` false overwrites.
template <int CG>
__device__ __forceinline__ void mma_bf16(uint32_t tmem, uint64_t a, uint64_t b, uint32_t desc, bool add)
{
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
            "l"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
            "l"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
            : "memory");
}

// The barrier (of a pair: the barrier at this place in both CTAs) gets one
// arrival once every MMA this thread issued has finished.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
}

// A whole warp (of a pair: one of each CTA) allocates and frees tensor memory
// columns; the address is written to shared memory.
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t smem_slot, uint32_t columns)
{
    if constexpr (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_slot), "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_slot), "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns)
{
    if constexpr (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
}

// Both CTAs of a pair; every thread of them calls it.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Arrival at the barrier at this place in the pair's first CTA, which says that
// tensor memory has been read and nothing else: the loads have completed
// (tcgen05.wait::ld, tc_fence_before), and relaxed as it is it orders neither
// reads nor writes of shared or global memory.  (A release at cluster scope
// would wait for all of the thread's stores first.)
__device__ __forceinline__ void mbar_arrive_first(uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of this warp's 32 lanes: thread t gets row t of them.  The values
// may be used after tmem_wait.
__device__ __forceinline__ void tmem_load32(uint32_t tmem, float (&v)[32])
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(tmem)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 8 columns.
__device__ __forceinline__ void tmem_load8(uint32_t tmem, float (&v)[8])
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(tmem)
                 : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// One box of a row-major matrix at (column, row) into this CTA's shared
// memory; what lies outside the matrix is filled with zeros and counts towards
// the barrier's bytes.  Of a pair, both CTAs' loads complete on the barrier
// at this place in the first CTA.  The column is a multiple of eight 16-bit
// elements, so the copy starts on a 16-byte boundary.
template <int CG>
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int32_t col, int32_t row, uint32_t bar)
{
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
            ::"r"(dst), "l"(map), "r"(col), "r"(row), "r"(bar)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, 0;\n\t"
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
            "[%0], [%1, {%2, %3}], [a];\n\t}"
            ::"r"(dst), "l"(map), "r"(col), "r"(row), "r"(bar)
            : "memory");
}

// True for one lane of a whole warp, the same one each time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The larger of three (a NaN among them does not count), and two sums or
// products at a time.
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    uint64_t x, y, z;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(x), "l"(y));
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(z));
    return f;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t x, y, w, z;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(w) : "f"(c.x), "f"(c.y));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(z) : "l"(x), "l"(y), "l"(w));
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(z));
    return f;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    uint64_t x, y, z;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(x), "l"(y));
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(z));
    return f;
}

// 2^x, at most 2 ulp off.
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / x, at most 1 ulp off.
__device__ __forceinline__ float rcp_fast(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace dt
