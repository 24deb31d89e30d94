// Parts of the kernels that work on rows whose columns stay with one thread each:
// a row's elements in registers, the threads that share a row, and their sums.
#pragma once

#include <cstdint>

#include "dt_internal.h"
#include "dt_math.cuh"

namespace dt {

constexpr int kNormThreads = 512;    // most threads of a block, and of a row

// Two fp32 values in a pair of registers, for the instructions that work on
// both at once: the kernels are nearly bound by issue, and these halve the
// arithmetic's share of it.  The same functions on one float serve rows that
// are read element by element.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 pair(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split(F2 x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ F2 add(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float both(F2 x)
{
    float a, b;
    split(x, a, b);
    return a + b;
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float both(float x) { return x; }
__device__ __forceinline__ float first_of(F2 x)
{
    float a, b;
    split(x, a, b);
    return a;
}
__device__ __forceinline__ float second_of(F2 x)
{
    float a, b;
    split(x, a, b);
    return b;
}
__device__ __forceinline__ float first_of(float x) { return x; }

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ void from_f32(float f, float *p) { *p = f; }
__device__ __forceinline__ void from_f32(float f, uint16_t *p) { *p = f32_to_bf16(f); }

// VEC elements as they lie in memory: one 16-byte vector, or one element; in
// registers K values of V, pairs of floats or one float.
template <typename T, int VEC>
struct Chunk {
    static_assert(VEC * sizeof(T) == 16, "a vector is 16 bytes");
    using V = F2;
    static constexpr int K = VEC / 2;
    uint4 v;
    __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(V (&f)[K]) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < K; ++i) {
            if constexpr (VEC == 8) f[i] = pair(bf16_lo(w[i]), bf16_hi(w[i]));
            else f[i] = pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        }
    }
    static __device__ __forceinline__ void store(T *p, const V (&f)[K])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            float a, b;
            split(f[i], a, b);
            if constexpr (VEC == 8) {
                w[i] = pack_bf16x2(a, b);
            } else {
                w[2 * i] = __float_as_uint(a);
                w[2 * i + 1] = __float_as_uint(b);
            }
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ V all(float x) { return pair(x, x); }
};

template <typename T>
struct Chunk<T, 1> {
    using V = float;
    static constexpr int K = 1;
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ void get(V (&f)[1]) const { f[0] = to_f32(v); }
    static __device__ __forceinline__ void store(T *p, const V (&f)[1]) { from_f32(f[0], p); }
    static __device__ __forceinline__ V all(float x) { return x; }
};

// The threads that share a ring: one warp or more of one row, or a warp of 32 / L
// teams of L lanes, which take the rows of a stage in turn.
template <int L>
struct Team {
    static constexpr uint32_t kTeams = 32 / L;
    uint32_t tpr, group, team, t;
    explicit __device__ __forceinline__ Team(uint32_t threads)
        : tpr(L < 32 ? L : threads), group(threadIdx.x / (tpr * kTeams)), team(threadIdx.x / tpr % kTeams),
          t(threadIdx.x % tpr)
    {
    }
    __device__ __forceinline__ uint32_t threads() const { return tpr * kTeams; }
    __device__ __forceinline__ bool first() const { return team == 0 && t == 0; }
    __device__ __forceinline__ bool first_warp() const { return L < 32 || t < 32; }
};

// The sum over L lanes.
template <int L>
__device__ __forceinline__ float lane_sum(float v)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sums of V values (2, 4 or 8) over the threads that share a row, L lanes or
// several warps; every thread gets the same sums, added in the same order.
// Within a warp each step halves the values a lane still carries as well as the
// lanes that share one: 9 shuffles for 8 values, where one value after the
// other takes 40.  `red` is double-buffered like exchange()'s.
template <int V, int L>
__device__ __forceinline__ void row_sum(float (&v)[V], float (*red)[V][kNormThreads / 32], uint32_t &phase,
                                        const Team<L> &m)
{
    static_assert(V <= L, "a value to a lane at least");
    constexpr uint32_t kLanes = L / V;   // lanes that hold the same value in the end
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll
    for (int have = V, o = L / 2; o > 0; o >>= 1) {
        if (have > 1) {
            have /= 2;
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < have; ++i) {
                const float send = up ? v[i] : v[i + have], keep = up ? v[i + have] : v[i];
                v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
            }
        } else {
            v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
        }
    }
    float sum = v[0];                     // of value lane % L / kLanes
    if (L == 32 && m.tpr > 32) {
        const uint32_t warps = m.tpr >> 5, j = lane % kLanes;
        if (j == 0) red[phase][lane / kLanes][threadIdx.x >> 5] = sum;
        asm volatile("bar.sync %0, %1;" ::"r"(m.group + 1), "r"(m.tpr) : "memory");
        const float *of = &red[phase][lane / kLanes][m.group * warps];
        sum = 0.0f;
#pragma unroll
        for (uint32_t k = 0; k < kNormThreads / 32; k += kLanes)
            if (k + j < warps) sum += of[k + j];
#pragma unroll
        for (uint32_t o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        phase ^= 1;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, sum, i * kLanes, L);
}

// Another lane's value.
__device__ __forceinline__ float from_lane(float x, uint32_t o) { return __shfl_xor_sync(0xFFFFFFFFu, x, o); }
__device__ __forceinline__ F2 from_lane(F2 x, uint32_t o)
{
    float a, b;
    split(x, a, b);
    return pair(from_lane(a, o), from_lane(b, o));
}

}  // namespace dt
