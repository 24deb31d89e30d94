// Layer norm over the rows of P ranks, forward and backward, and the
// reduction of the weight's and bias' gradients over every rank's rows.
//
//   mu = mean_j x_j      v = mean_j (x_j - mu)^2      r = 1 / sqrt(v + eps)
//   h_j = (x_j - mu) r   y_j = h_j w_j + b_j
//   q_j = dy_j w_j       dx_j = r (q_j - mean(q) - h_j mean(q h))
//   dw_j = sum_rows dy_j h_j      db_j = sum_rows dy_j
//
// A call is one launch (two for the backward pass) whatever the number of
// ranks.  HBM bounds both directions (about 4 and 5 flops per byte), and close
// behind it the instructions an SM can issue and the time that one row takes,
// so every row is read once and crosses few threads: sums cost shuffles and
// barriers per warp that shares a row, not per element.
//
// norm_rows_kernel  forward, rows of whole vectors: a row in the registers of
//                   4, 8 or 16 lanes or of whole warps, blocks handed out by
//                   the hardware (4 x 2048 rows of 4096 bf16: 27.8 us, 4.8
//                   TB/s; PyTorch's copy of the same bytes 23.2)
// norm_kernel       forward, rows at other offsets or too long for that, and
// norm_backward_kernel: resident blocks whose groups of threads each have a
//                   ring of shared memory stages that bulk copies fill, so that
//                   up to 160 KB an SM are always under way.  A stage is a few
//                   rows; rows of any alignment are copied with the 16-byte
//                   blocks that their ends lie in, and then read element by
//                   element (3 x 5000 rows of 1021 f32: 24.4 us, 5.0 TB/s; with
//                   loads to registers 36).  A thread keeps its columns, 8 to
//                   32 of them, over all of its rows, and with them their
//                   weights and, backward, their shares of dw and db; up to four
//                   rows are summed at a time, and the rows of a warp's teams of
//                   lanes where rows are short.  Backward 4 x 2048 x 4096 bf16
//                   43 us, 4.7 TB/s; 8 x 8192 x 4096 272 us, 5.9 TB/s: the
//                   smaller call's blocks spend 5 us on their way to the first
//                   row and 3 between the first SM's end and the last's.
// norm_join_kernel  adds the blocks' shares of dw and db in a fixed order, so
//                   that the result depends on the device and the shapes alone,
//                   not on timing.
//
// The variance is the mean of the squared distances from the mean, not
// E[x^2] - mu^2, which loses every digit where |mu| is large.  All sums are
// fp32, and results are rounded once, at the store.
#include <algorithm>
#include <type_traits>

#include "dt_ops.h"

#include "dt_bounds.cuh"
#include "dt_device.cuh"
#include "dt_math.cuh"
#include "dt_timeline.cuh"

namespace dt {
namespace {

constexpr int kNormThreads = 512;    // most threads of a block, and of a row
// Rings, of the SM's 227 KB.  With more on its way than keeps HBM busy, some
// SMs get a larger share of it than others and wait for those at the end
// (backward, 4 x 8192 rows of 2048 f32: 145 us with 208 KB, the SMs busy for
// 202000 to 246000 cycles; 133 with 160).
constexpr uint32_t kSmemBytes = 160 * 1024;
constexpr uint32_t kMaxStages = 8;
constexpr uint32_t kStageTarget = 4096;
constexpr uint32_t kMostColumns = kNormThreads * 32;   // of a row in registers
constexpr int kLongThreads = 512;    // rows too long for registers
constexpr int kLongSlices = 32;      // row slices of the column sums there
constexpr int kJoinCols = 32;        // columns and row slices of a block that adds the shares
constexpr int kJoinSlices = 16;

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

// Bounds-checked builds: [a, a + n) lies in buffer `kind` (x 0, dy 1, y or dx 2,
// mean 3, rstd 4) of rank r, in the weight or bias, or in one of the others.
#define NORM_OK(kind, r, a, n) DT_IN_EXTENT(p, kBoundsNorm, (kind) * DT_MAX_RANKS + (r), (a), (n))
#define NORM_PARAM_OK(bias, q, n) DT_IN_EXTENT(p, kBoundsNorm, (bias) ? kNormBias : kNormWeight, (q), (n) * sizeof *(q))
#define NORM_BUFFER_OK(buffer, a, n) DT_IN_EXTENT(p, kBoundsNorm, (buffer), (a), (n))

// Element j of the weight (bias 0) or the bias (1), or what they are where the
// caller has none: 1 and 0.
template <int BIAS>
__device__ __forceinline__ float param(const NormParams &p, uint32_t j)
{
    const void *base = BIAS ? p.bias : p.weight;
    const float none = BIAS ? 0.0f : 1.0f;
    if (!base) return none;
    if (p.weight_bf16) {
        const uint16_t *q = static_cast<const uint16_t *>(base) + j;
        return NORM_PARAM_OK(BIAS, q, 1) ? bf16_to_f32(*q) : none;
    }
    const float *q = static_cast<const float *>(base) + j;
    return NORM_PARAM_OK(BIAS, q, 1) ? *q : none;
}

// A thread's weights or biases from element e on: whole vectors where they lie
// on 16-byte boundaries.
template <typename C, int VEC, int BIAS>
__device__ __forceinline__ void params(const NormParams &p, uint32_t e, typename C::V (&f)[C::K])
{
    const void *base = BIAS ? p.bias : p.weight;
    float v[VEC];
    const bool vec = VEC > 1 && (reinterpret_cast<uint64_t>(base) & 15) == 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = BIAS ? 0.0f : 1.0f;
    if (base && p.weight_bf16) {
        const uint16_t *q = static_cast<const uint16_t *>(base) + e;
        if (NORM_PARAM_OK(BIAS, q, VEC)) {
            uint32_t u[VEC > 1 ? VEC / 2 : 1];
            if (VEC > 1 && vec) {
                if constexpr (VEC == 8) *reinterpret_cast<uint4 *>(u) = *reinterpret_cast<const uint4 *>(q);
                if constexpr (VEC == 4) *reinterpret_cast<uint2 *>(u) = *reinterpret_cast<const uint2 *>(q);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; i += 2) u[i / 2] = q[i] | (VEC > 1 ? (uint32_t)q[i + (VEC > 1)] << 16 : 0u);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = i & 1 ? bf16_hi(u[i / 2]) : bf16_lo(u[i / 2]);
        }
    } else if (base) {
        const float *q = static_cast<const float *>(base) + e;
        if (NORM_PARAM_OK(BIAS, q, VEC)) {
            if (VEC > 1 && vec) {
#pragma unroll
                for (int i = 0; i < VEC / 4; ++i)
                    *reinterpret_cast<float4 *>(v + 4 * i) = *reinterpret_cast<const float4 *>(q + 4 * i);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[i] = q[i];
            }
        }
    }
    if constexpr (VEC == 1) {
        f[0] = v[0];
    } else {
#pragma unroll
        for (int i = 0; i < C::K; ++i) f[i] = pair(v[2 * i], v[2 * i + 1]);
    }
}

// The rank that row belongs to, and the row's number there.
__device__ __forceinline__ int find_rank(const NormParams &p, uint64_t row, uint64_t &local)
{
    int r = 0;
    uint64_t begin = 0;
    while (r + 1 < p.P && row >= p.row_end[r]) begin = p.row_end[r++];
    local = row - begin;
    return r;
}

// Values of each warp of a row to all of its threads: `red` is
// double-buffered by the caller's `phase`, and a buffer is written again only
// after the barrier of the exchange in between, which every reader of it has
// passed.  The result is the row's first entry.
using Exchange = float4[2][kNormThreads / 32];
__device__ __forceinline__ const float4 *exchange(float4 v, Exchange &red, uint32_t &phase, uint32_t tpr, uint32_t group)
{
    if ((threadIdx.x & 31) == 0) red[phase][threadIdx.x >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
    const float4 *first = &red[phase][group * (tpr >> 5)];
    phase ^= 1;
    return first;
}

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

// A group's walk over the rows: chunk c of the call is up to p.chunk_rows rows
// of one rank; group number `part` has chunks part, part + parts, ...  Its
// first warp starts the copies; the rest is the same in all of its threads.
// Dynamic shared memory holds the groups' rings and their barriers.
template <typename T, bool BACK>
struct Ring {
    const NormParams &p;
    uint32_t base, bars;             // the group's stages and their barriers in shared memory
    unsigned char *mem;
    uint32_t s = 0, parity = 0;
    bool late = false;               // a wait ran out: wait no more, and keep to the barriers

    // The rows of chunk c: rank, first row there, how many.
    __device__ __forceinline__ void chunk(uint64_t c, int &r, uint64_t &row, uint32_t &n) const
    {
        uint64_t begin = 0, rows = 0;
        r = 0;
        while (r + 1 < p.P && c >= p.chunk_end[r]) begin = p.chunk_end[r++];
        row = (c - begin) * p.chunk_rows;
        rows = p.row_end[r] - (r ? p.row_end[r - 1] : 0);
        n = rows - row < p.chunk_rows ? (uint32_t)(rows - row) : p.chunk_rows;
    }
    // The copies of a chunk: x, and backward dy, mean, rstd.
    static constexpr uint32_t kCopies = BACK ? 4 : 1;
    // Copies the 16-byte blocks of one of its buffers that hold rows [row, row + n) of rank r; how many bytes.
    __device__ __forceinline__ uint32_t copy(uint32_t which, int r, uint64_t row, uint32_t n, uint32_t stage) const
    {
        uint32_t dst = base + stage * p.stage_bytes;
        uint64_t row_bytes = p.cols * sizeof(T);
        const void *const *bases = p.x;
        if (BACK && which != 0) {
            bases = which == 1 ? p.dy : reinterpret_cast<const void *const *>(which == 2 ? p.mean : p.rstd);
            dst += which == 1 ? p.array_bytes : 2 * p.array_bytes + (which - 2) * p.stat_bytes;
            if (which >= 2) row_bytes = 4;
        }
        const uint64_t lo = reinterpret_cast<uint64_t>(bases[r]) + row * row_bytes, hi = lo + n * row_bytes;
        const uint64_t from = lo & ~15ull, to = (hi + 15) & ~15ull;
        if (!NORM_OK(which < 2 ? which : which + 1, r, reinterpret_cast<const void *>(lo), hi - lo)) return 0;
        bulk_load(dst, reinterpret_cast<const void *>(from), (uint32_t)(to - from), bars + 8 * stage);
        return (uint32_t)(to - from);
    }
    // All of them by one thread.
    __device__ __forceinline__ void load(uint64_t c, uint32_t stage) const
    {
        int r;
        uint64_t row;
        uint32_t n, bytes = 0;
        chunk(c, r, row, n);
#pragma unroll
        for (uint32_t k = 0; k < kCopies; ++k) bytes += copy(k, r, row, n, stage);
        mbar_expect_tx(bars + 8 * stage, bytes);
    }
    // The ring's first ones, by a warp, a lane to a copy: one after the other they
    // take 0.6 us a stage.  They come after the weights' loads, which behind 25 MB
    // of rows would take 6 us.
    __device__ __forceinline__ void load_first(uint64_t part) const
    {
        static_assert(kCopies * kMaxStages <= 32, "a lane to a copy");
        const uint32_t lane = threadIdx.x & 31, stage = lane / kCopies, which = lane % kCopies;
        const uint64_t c = part + (uint64_t)stage * p.parts;
        const bool mine = stage < p.stages && c < p.chunks;
        uint32_t bytes = 0;
        if (mine) {
            int r;
            uint64_t row;
            uint32_t n;
            chunk(c, r, row, n);
            bytes = copy(which, r, row, n, stage);
        }
#pragma unroll
        for (uint32_t o = 1; o < kCopies; o *= 2) bytes += __shfl_xor_sync(0xFFFFFFFFu, bytes, o);
        if (mine && which == 0) mbar_expect_tx(bars + 8 * stage, bytes);
    }
    __device__ __forceinline__ void wait()
    {
        const uint32_t bar = bars + 8 * s;
        for (int k = 0; k < 64 && !late; ++k)
            if (mbar_try_wait(bar, parity)) return;
        if (late || mbar_wait_bounded(bar, parity, p.sink.timeout_ns)) return;
        late = true;
        record_error(p.sink, DT_ERR_TIMEOUT, -1, blockIdx.x, 0);
    }
    // What was copied to `offset` bytes into the present stage from `src` on.
    template <typename E>
    __device__ __forceinline__ const E *at(uint32_t offset, const E *src) const
    {
        return reinterpret_cast<const E *>(mem + s * p.stage_bytes + offset + (reinterpret_cast<uint64_t>(src) & 15));
    }
    __device__ __forceinline__ void next()
    {
        if (++s == p.stages) s = 0, parity ^= 1;
    }
    // Before the block goes on after a wait that ran out, a last, bounded wait
    // for what is still under way: each stage's last copy of group `part`.
    __device__ __forceinline__ void drain(bool first, uint64_t part) const
    {
        if (!late || !first) return;
        const uint64_t n = (p.chunks - part + p.parts - 1) / p.parts;
        for (uint32_t k = 0; k < p.stages && k < n; ++k)
            mbar_wait_bounded(bars + 8 * k, (uint32_t)((n - k + p.stages - 1) / p.stages - 1) & 1, p.sink.timeout_ns);
    }
};

// The group's ring; the waits for the kernel before and of the one after.
template <typename T, bool BACK, int L>
__device__ __forceinline__ Ring<T, BACK> make_ring(const NormParams &p, unsigned char *smem, const Team<L> &m)
{
    const uint32_t groups = blockDim.x / m.threads(), mine = p.stages * p.stage_bytes;
    const uint32_t bars = smem_addr(smem) + groups * mine;
    if (threadIdx.x == 0) {
        for (uint32_t k = 0; k < groups * p.stages; ++k) mbar_init(bars + 8 * k, 1);
        mbar_init_fence();
    }
    __syncthreads();
    unsigned char *mem = smem + (size_t)m.group * mine;
    pdl_begin();
    return Ring<T, BACK>{p, smem_addr(mem), bars + 8 * m.group * p.stages, mem};
}

// A row of a stage in registers: chunk c of thread t is elements [(c * tpr +
// t) * VEC, + VEC).
template <typename T, int VEC, int N>
__device__ __forceinline__ void read_row(Chunk<T, VEC> (&c)[N], const NormParams &p, const T *row, uint32_t tpr, uint32_t t,
                                         bool there)
{
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint32_t e = (n * tpr + t) * VEC;
        if (there && e < p.cols) c[n].load(row + e);
        else c[n].zero();
    }
}

// Rows that are summed at a time, so that a barrier serves several: up to four,
// as long as they take at most 32 registers of a thread.
template <typename T, int VEC, int N, bool BACK>
__host__ __device__ constexpr int rows_at_once()
{
    constexpr int regs = N * (VEC == 1 ? 1 : 4) * (BACK ? 2 : 1);
    return regs <= 8 ? 4 : regs <= 16 ? 2 : 1;
}

// sum + low is the sum of what was added, to about twice fp32's digits: `low`
// collects what each addition rounds off, as Knuth's two-sum gives it exactly
// (The Art of Computer Programming, volume 2, section 4.2.2).
template <typename V>
__device__ __forceinline__ void exact_add(V &sum, V &low, V x, V minus_one)
{
    const V t = add(sum, x), of_x = fma(sum, minus_one, t);
    low = add(low, add(fma(fma(of_x, minus_one, t), minus_one, sum), fma(of_x, minus_one, x)));
    sum = t;
}

// Without it where the sum is no number.
__device__ __forceinline__ float with_low(float sum, float low) { return sum - sum == 0.0f ? sum + low : sum; }

// The mean and the sum of squared distances from it, of all warps that share a
// row from each one's own: M2 = sum of M2_w + n_w (mean_w - mean)^2.
__device__ __forceinline__ void row_moments(float sum, float &mean, float &m2, uint32_t mine, float inv_cols,
                                            Exchange &red, uint32_t &phase, uint32_t tpr, uint32_t group,
                                            float *lows = nullptr, float low = 0.0f)
{
    if (tpr == 32) {
        if (lows) mean = with_low(sum, low) * inv_cols;
        return;
    }
    if (lows && (threadIdx.x & 31) == 0) lows[threadIdx.x >> 5] = low;
    const float4 *of = exchange(make_float4(sum, m2, mean, (float)mine), red, phase, tpr, group);
    float all = 0.0f, rest = 0.0f;
#pragma unroll 4
    for (uint32_t q = 0; q < tpr >> 5; ++q) {
        if (!lows) {
            all += of[q].x;
        } else {
            rest += lows[q];
            exact_add(all, rest, of[q].x, -1.0f);
        }
    }
    mean = (lows ? with_low(all, rest) : all) * inv_cols;
    m2 = 0.0f;
#pragma unroll 4
    for (uint32_t q = 0; q < tpr >> 5; ++q) {
        const float4 v = of[q];
        m2 += fmaf(v.w * (v.z - mean), v.z - mean, v.y);
    }
}

// 1 / sqrt(v + eps), at most 2 ulp off.
__device__ __forceinline__ float rstd_of(float m2, float inv_cols, float eps) { return rsqrtf(fmaf(m2, inv_cols, eps)); }

template <typename T, int VEC, int N, int L>
__global__ void __launch_bounds__(kNormThreads, 1) norm_kernel(const __grid_constant__ NormParams p)
{
    constexpr bool kHold = N * VEC <= 16;   // wider rows read their weights again from L1
    constexpr int B = rows_at_once<T, VEC, N, false>();
    using C = Chunk<T, VEC>;
    using V = typename C::V;
    constexpr int K = C::K;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float red[2][B][kNormThreads / 32];
    DT_TL_BEGIN();
    const Team<L> team(p.tpr);
    constexpr uint32_t S = Team<L>::kTeams;
    const uint32_t tpr = team.tpr, t = team.t, cols = p.cols;
    const uint64_t part = (uint64_t)team.group * gridDim.x + blockIdx.x;
    Ring<T, false> ring = make_ring<T, false>(p, smem, team);
    DT_TL_WAITED();
    const float inv = p.inv_cols;
    uint32_t phase = 0;
    // the weights' loads before the stages' copies (Ring::load_first)
    V w[N][K], b[N][K];
    auto weights = [&](int n) {
        const uint32_t e = (n * tpr + t) * VEC;
        if (e >= cols) return;
        params<C, VEC, 0>(p, e, w[n]);
        params<C, VEC, 1>(p, e, b[n]);
    };
    if constexpr (kHold)
#pragma unroll
        for (int n = 0; n < N; ++n) weights(n);
    if (team.first_warp()) ring.load_first(part);

    for (uint64_t c = part; c < p.chunks; c += p.parts) {
        int r;
        uint64_t row;
        uint32_t rows;
        ring.chunk(c, r, row, rows);
        const T *src = ring.at(0, static_cast<const T *>(p.x[r]) + row * cols) + team.team * cols;
        T *y = static_cast<T *>(p.out[r]) + (row + team.team) * cols;
        float *means = p.mean[r] ? p.mean[r] + row : nullptr, *rstds = p.rstd[r] ? p.rstd[r] + row : nullptr;
        ring.wait();
        // this team's rows are the stage's k, k + S, ...
        for (uint32_t k = team.team; k - team.team < rows; k += B * S, src += B * S * cols, y += (uint64_t)(B * S) * cols) {
            // B rows at a time; the last ones of a stage may stand beside rows of zeros
            C x[B][N];
            float s[B], m2[B];
#pragma unroll
            for (int j = 0; j < B; ++j) {
                read_row<T, VEC, N>(x[j], p, src + j * S * cols, tpr, t, k + j * S < rows);
                V sum = C::all(0.0f);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    V f[K];
                    x[j][n].get(f);
#pragma unroll
                    for (int i = 0; i < K; ++i) sum = add(sum, f[i]);
                }
                s[j] = both(sum);
            }
            row_sum<B>(s, red, phase, team);
            if (tpr <= 32) __syncwarp();
            // every thread has read its part of the stage's last rows
            if (k - team.team + B * S >= rows && team.first() && c + (uint64_t)p.stages * p.parts < p.chunks)
                ring.load(c + (uint64_t)p.stages * p.parts, ring.s);
#pragma unroll
            for (int j = 0; j < B; ++j) {
                s[j] *= inv;
                V sum = C::all(0.0f);
                const V minus = C::all(-s[j]);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint32_t e = (n * tpr + t) * VEC;
                    if (e >= cols) continue;
                    V f[K];
                    x[j][n].get(f);
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        f[i] = add(f[i], minus);
                        sum = fma(f[i], f[i], sum);
                    }
                }
                m2[j] = both(sum);
            }
            row_sum<B>(m2, red, phase, team);
#pragma unroll
            for (int j = 0; j < B; ++j) {
                if (k + j * S >= rows) continue;
                m2[j] = rstd_of(m2[j], inv, p.eps);
                const V minus = C::all(-s[j]), scale = C::all(m2[j]);
                T *to = y + j * S * (uint64_t)cols;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint32_t e = (n * tpr + t) * VEC;
                    if (e >= cols) continue;
                    if constexpr (!kHold) weights(n);
                    V f[K];
                    x[j][n].get(f);
#pragma unroll
                    for (int i = 0; i < K; ++i) f[i] = fma(mul(add(f[i], minus), scale), w[n][i], b[n][i]);
                    if (NORM_OK(2, r, to + e, VEC * sizeof(T))) C::store(to + e, f);
                }
            }
            // one lane to a row, of the team's last warp
            const uint32_t lane = t - (tpr - L), at = k + lane * S;
            if (lane < B && at < rows) {
                float mean = s[0], rstd = m2[0];
#pragma unroll
                for (int j = 1; j < B; ++j)
                    if (lane == j) mean = s[j], rstd = m2[j];
                if (means && NORM_OK(3, r, means + at, 4)) means[at] = mean;
                if (rstds && NORM_OK(4, r, rstds + at, 4)) rstds[at] = rstd;
            }
        }
        ring.next();
    }
    ring.drain(team.first(), part);
    DT_TL_END_BLOCK(DT_TL_NORM);
}

// How a call's weights and biases are read; the kernel takes it as a constant
// within its loops, so that loads are not kept apart by branches.
enum ParamKind { kParamBf16, kParamF32, kParamAny };   // whole vectors of either type, or whatever there is

template <typename C, int VEC, int KIND, int BIAS>
__device__ __forceinline__ void read_param(const NormParams &p, uint32_t e, typename C::V (&f)[C::K])
{
    if constexpr (KIND == kParamBf16 && VEC == 8) {
        const uint16_t *q = static_cast<const uint16_t *>(BIAS ? p.bias : p.weight) + e;
        const uint4 u = NORM_PARAM_OK(BIAS, q, VEC) ? __ldg(reinterpret_cast<const uint4 *>(q)) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = pair(bf16_lo(w[i]), bf16_hi(w[i]));
    } else if constexpr (KIND == kParamF32 && VEC > 1) {
#pragma unroll
        for (int i = 0; i < C::K; i += 2) {
            const float *q = static_cast<const float *>(BIAS ? p.bias : p.weight) + e + 2 * i;
            const float4 u = NORM_PARAM_OK(BIAS, q, 4) ? __ldg(reinterpret_cast<const float4 *>(q)) : make_float4(0, 0, 0, 0);
            f[i] = pair(u.x, u.y);
            f[i + 1] = pair(u.z, u.w);
        }
    } else {
        params<C, VEC, BIAS>(p, e, f);
    }
}

// A row in the registers of tpr threads, mostly 4 vectors each, and blocks of a
// few rows that the hardware hands to the SMs as they come free: resident
// blocks that share the rows out evenly took 37 us for 4 x 2048 rows of 4096
// bf16, this 27.7.  64 registers a thread leave room for eight rows an SM; a
// row takes 3 us, of which 1 is its loads'.  Tried: 1, 2, 8, 16 vectors a
// thread 66, 43, 35, 38 us (with 4: 34 at that stage); the rows' weights in
// shared memory 40, bound by reading them there.
// L: lanes of a warp that share a row.  Short rows share a warp, four vectors a
// lane: a warp to a row took 230, 118, 67, 48 us for 100 MB of rows of 64, 128,
// 256, 512 bf16, this 46, 38, 41, 41.
// EARLY: the weights are loaded along with the row, for calls of few rows,
// where only the time from the first load to the last store counts.
template <typename T, int VEC, int N, int L, bool EARLY>
__global__ void __launch_bounds__(EARLY || N < 4 ? kNormThreads : 256, EARLY || N < 4 ? 1 : 4)
norm_rows_kernel(const __grid_constant__ NormParams p)
{
    using C = Chunk<T, VEC>;
    using V = typename C::V;
    __shared__ Exchange red;
    __shared__ float lows[kNormThreads / 32];
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    const uint32_t tpr = p.tpr, group = threadIdx.x / tpr, t = threadIdx.x % tpr, cols = p.cols;
    // A row of blocks to a rank, as a search for the rank takes a tenth of a row's
    // instructions; but one row of blocks for all where many would find no rows.
    int r = blockIdx.y;
    uint32_t block = blockIdx.x;
    if (p.chunks) {
        for (int step = DT_MAX_RANKS / 2; step > 0; step /= 2)
            if (r + step < p.P && block >= p.chunk_end[r + step - 1]) r += step;
        if (r) block -= (uint32_t)p.chunk_end[r - 1];
    }
    const uint64_t row = (uint64_t)block * (blockDim.x / tpr) + group;
    const bool there = row < p.row_end[r] - (r ? p.row_end[r - 1] : 0);
    if (L < 32 || there) {   // all rows of a warp pass through its shuffles
        const T *src = static_cast<const T *>(p.x[r]) + row * cols;
        T *y = static_cast<T *>(p.out[r]) + row * cols;
        C x[N];
        V w[EARLY ? N : 1][C::K], b[EARLY ? N : 1][C::K];
        uint32_t mine = 0, phase = 0;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint32_t first = (n * tpr + t / L * L) * VEC, e = (n * tpr + t) * VEC;
            mine += first < cols ? min(cols - first, (uint32_t)(L * VEC)) : 0;
            if (e < cols && there && NORM_OK(0, r, src + e, VEC * sizeof(T))) x[n].load(src + e);
            else x[n].zero();
        }
        if constexpr (EARLY)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint32_t e = (n * tpr + t) * VEC;
                if (e >= cols) continue;
                params<C, VEC, 0>(p, e, w[n]);
                params<C, VEC, 1>(p, e, b[n]);
            }
        const float inv_mine = mine ? __frcp_rn((float)mine) : 0.0f;
        // four sums, so that an addition does not wait for the one before
        V s[4] = {C::all(0.0f), C::all(0.0f), C::all(0.0f), C::all(0.0f)}, m[4] = {s[0], s[0], s[0], s[0]};
#pragma unroll
        for (int n = 0; n < N; ++n) {
            V f[C::K];
            x[n].get(f);
#pragma unroll
            for (int i = 0; i < C::K; ++i) s[(n * C::K + i) & 3] = add(s[(n * C::K + i) & 3], f[i]);
        }
        float sum = both(add(add(s[0], s[1]), add(s[2], s[3]))), low = 0.0f;
        if constexpr (EARLY) {
            // A mean near zero keeps few of its sum's digits, and a sum of twice the
            // digits costs nothing here (4 x 1 x 4096 bf16: 4.0 us either way), while
            // kernels of many rows are nearly bound by issue.  So a row's statistics may
            // differ in their last bits between a call of few rows and one of many, as
            // they do by the threads that share the row.
            V hi = C::all(0.0f), lo = C::all(0.0f);
#pragma unroll
            for (int n = 0; n < N; ++n) {
                V f[C::K];
                x[n].get(f);
#pragma unroll
                for (int i = 0; i < C::K; ++i) exact_add(hi, lo, f[i], C::all(-1.0f));
            }
            sum = first_of(hi);
            low = both(lo);
            if constexpr (VEC > 1) exact_add(sum, low, second_of(hi), -1.0f);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                low += __shfl_xor_sync(0xFFFFFFFFu, low, o);
                exact_add(sum, low, __shfl_xor_sync(0xFFFFFFFFu, sum, o), -1.0f);
            }
        } else {
            sum = lane_sum<L>(sum);
        }
        float mean = sum * inv_mine;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if ((n * tpr + t) * VEC >= cols) continue;
            V f[C::K];
            x[n].get(f);
#pragma unroll
            for (int i = 0; i < C::K; ++i) {
                const V d = add(f[i], C::all(-mean));
                m[(n * C::K + i) & 3] = fma(d, d, m[(n * C::K + i) & 3]);
            }
        }
        float m2 = lane_sum<L>(both(add(add(m[0], m[1]), add(m[2], m[3]))));
        if constexpr (L == 32)
            row_moments(sum, mean, m2, mine, p.inv_cols, red, phase, tpr, group, EARLY ? lows : nullptr, low);
        const float rstd = rstd_of(m2, p.inv_cols, p.eps);
        const V minus = C::all(-mean), scale = C::all(rstd);
        auto finish = [&](auto kind) {
            constexpr int KIND = decltype(kind)::value;
            (void)KIND;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint32_t e = (n * tpr + t) * VEC;
                if (e >= cols || !there) continue;
                constexpr int k = EARLY ? 1 : 0;
                if constexpr (!EARLY) {
                    read_param<C, VEC, KIND, 0>(p, e, w[0]);
                    read_param<C, VEC, KIND, 1>(p, e, b[0]);
                }
                V f[C::K];
                x[n].get(f);
#pragma unroll
                for (int i = 0; i < C::K; ++i) f[i] = fma(mul(add(f[i], minus), scale), w[n * k][i], b[n * k][i]);
                if (NORM_OK(2, r, y + e, VEC * sizeof(T))) C::store(y + e, f);
            }
        };
        if (EARLY || p.param_kind == kParamAny) finish(std::integral_constant<int, kParamAny>());
        else if (p.param_kind == kParamBf16) finish(std::integral_constant<int, kParamBf16>());
        else finish(std::integral_constant<int, kParamF32>());
        if (t == 0 && there) {
            if (p.mean[r] && NORM_OK(3, r, p.mean[r] + row, 4)) p.mean[r][row] = mean;
            if (p.rstd[r] && NORM_OK(4, r, p.rstd[r] + row, 4)) p.rstd[r][row] = rstd;
        }
    }
    DT_TL_END_BLOCK(DT_TL_NORM);
}

__device__ __forceinline__ float from_lane(float x, uint32_t o) { return __shfl_xor_sync(0xFFFFFFFFu, x, o); }
__device__ __forceinline__ F2 from_lane(F2 x, uint32_t o)
{
    float a, b;
    split(x, a, b);
    return pair(from_lane(a, o), from_lane(b, o));
}

template <typename T, int VEC, int N, int L>
__global__ void __launch_bounds__(kNormThreads, 1) norm_backward_kernel(const __grid_constant__ NormParams p)
{
    constexpr bool kHold = N * VEC <= 16;   // wider rows read their weights again from L1
    constexpr int B = rows_at_once<T, VEC, N, true>();
    using C = Chunk<T, VEC>;
    using V = typename C::V;
    constexpr int K = C::K;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float red[2][2 * B][kNormThreads / 32];
    DT_TL_BEGIN();
    const Team<L> team(p.tpr);
    constexpr uint32_t S = Team<L>::kTeams;
    const uint32_t tpr = team.tpr, t = team.t, cols = p.cols;
    const uint64_t part = (uint64_t)team.group * gridDim.x + blockIdx.x;
    Ring<T, true> ring = make_ring<T, true>(p, smem, team);
    DT_TL_WAITED();
    const float inv = p.inv_cols;
    uint32_t phase = 0;
    // the weights' loads before the stages' copies (Ring::load_first)
    V dw[N][K], db[N][K], w[N][K];
    auto weights = [&](int n) {
        const uint32_t e = (n * tpr + t) * VEC;
        if (e < cols) params<C, VEC, 0>(p, e, w[n]);
    };
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int i = 0; i < K; ++i) dw[n][i] = db[n][i] = w[n][i] = C::all(0.0f);
        if constexpr (kHold) weights(n);
    }
    if (team.first_warp()) ring.load_first(part);

    for (uint64_t c = part; c < p.chunks; c += p.parts) {
        int r;
        uint64_t row;
        uint32_t rows;
        ring.chunk(c, r, row, rows);
        const T *xs = ring.at(0, static_cast<const T *>(p.x[r]) + row * cols) + team.team * cols;
        const T *gs = ring.at(p.array_bytes, static_cast<const T *>(p.dy[r]) + row * cols) + team.team * cols;
        const float *means = ring.at(2 * p.array_bytes, p.mean[r] + row);
        const float *rstds = ring.at(2 * p.array_bytes + p.stat_bytes, p.rstd[r] + row);
        T *dx = static_cast<T *>(p.out[r]) + (row + team.team) * cols;
        ring.wait();
        // this team's rows are the stage's k, k + S, ...
        for (uint32_t k = team.team; k - team.team < rows;
             k += B * S, xs += B * S * cols, gs += B * S * cols, dx += (uint64_t)(B * S) * cols) {
            // B rows at a time; the last ones of a stage may stand beside rows of zeros
            float mean[B], rstd[B];
#pragma unroll
            for (int j = 0; j < B; ++j) {
                mean[j] = k + j * S < rows ? means[k + j * S] : 0.0f;
                rstd[j] = k + j * S < rows ? rstds[k + j * S] : 0.0f;
            }
            C x[B][N], g[B][N];
            float s[2 * B];
#pragma unroll
            for (int j = 0; j < B; ++j) {
                read_row<T, VEC, N>(x[j], p, xs + j * S * cols, tpr, t, k + j * S < rows);
                read_row<T, VEC, N>(g[j], p, gs + j * S * cols, tpr, t, k + j * S < rows);
                V sq = C::all(0.0f), sh = C::all(0.0f);
                const V minus = C::all(-mean[j]), scale = C::all(rstd[j]);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    if ((n * tpr + t) * VEC >= cols) continue;
                    if constexpr (!kHold) weights(n);
                    V f[K], d[K];
                    x[j][n].get(f);
                    g[j][n].get(d);
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        const V a = add(f[i], minus), q = mul(d[i], w[n][i]);   // h = a * rstd
                        sq = add(sq, q);
                        sh = fma(q, a, sh);
                        dw[n][i] = fma(mul(d[i], scale), a, dw[n][i]);
                        db[n][i] = add(db[n][i], d[i]);
                    }
                }
                s[2 * j] = both(sq);
                s[2 * j + 1] = both(sh);
            }
            row_sum<2 * B>(s, red, phase, team);
            if (tpr <= 32) __syncwarp();
            // every thread has read its part of the stage's last rows
            if (k - team.team + B * S >= rows && team.first() && c + (uint64_t)p.stages * p.parts < p.chunks)
                ring.load(c + (uint64_t)p.stages * p.parts, ring.s);
#pragma unroll
            for (int j = 0; j < B; ++j) {
                if (k + j * S >= rows) continue;
                // dx = rstd (q - mean(q)) - a rstd^2 mean(q h), h = a rstd
                const V c0 = C::all(-s[2 * j] * inv * rstd[j]);
                const V c1 = C::all(-s[2 * j + 1] * inv * rstd[j] * rstd[j] * rstd[j]);
                const V minus = C::all(-mean[j]), scale = C::all(rstd[j]);
                T *to = dx + j * S * (uint64_t)cols;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint32_t e = (n * tpr + t) * VEC;
                    if (e >= cols) continue;
                    if constexpr (!kHold) weights(n);
                    V f[K], d[K];
                    x[j][n].get(f);
                    g[j][n].get(d);
#pragma unroll
                    for (int i = 0; i < K; ++i) f[i] = fma(add(f[i], minus), c1, fma(mul(d[i], w[n][i]), scale, c0));
                    if (NORM_OK(2, r, to + e, VEC * sizeof(T))) C::store(to + e, f);
                }
            }
        }
        ring.next();
    }
    ring.drain(team.first(), part);
    if (p.partial) {
        // the teams of a warp add theirs, then the block its groups', in ascending
        // order, in the rings' place (512 threads' columns take at most 128 KB)
#pragma unroll
        for (uint32_t o = 16; o >= (uint32_t)L; o >>= 1)
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < K; ++i) {
                    dw[n][i] = add(dw[n][i], from_lane(dw[n][i], o));
                    db[n][i] = add(db[n][i], from_lane(db[n][i], o));
                }
        const uint32_t groups = blockDim.x / team.threads();
        float *out = p.partial + (uint64_t)blockIdx.x * 2 * cols, *all = reinterpret_cast<float *>(smem);
        if (groups > 1) __syncthreads();
        float *mine = groups > 1 ? all + (size_t)team.group * 2 * cols : out;
        if (team.team == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint32_t e = (n * tpr + t) * VEC;
                if (e >= cols) continue;
#pragma unroll
                for (int i = 0; i < K; ++i) {   // cols is even where there are pairs
                    V *a = reinterpret_cast<V *>(mine + e) + i, *c = reinterpret_cast<V *>(mine + cols + e) + i;
                    if (groups > 1 || NORM_BUFFER_OK(kNormWorkspace, a, sizeof(V))) *a = dw[n][i];
                    if (groups > 1 || NORM_BUFFER_OK(kNormWorkspace, c, sizeof(V))) *c = db[n][i];
                }
            }
        if (groups > 1) {
            __syncthreads();
#pragma unroll 4
            for (uint32_t e = threadIdx.x; e < 2 * cols; e += blockDim.x) {
                float v = all[e];
#pragma unroll 4
                for (uint32_t k = 1; k < groups; ++k) v += all[(size_t)k * 2 * cols + e];
                if (NORM_BUFFER_OK(kNormWorkspace, out + e, 4)) out[e] = v;
            }
        }
    }
    DT_TL_END_BLOCK(DT_TL_NORM);
}

// Adds the shares of dw (blockIdx.y 0) and db (1): thread (c, s) adds shares
// s, s + 16, ... of its column, then the 16 sums are added in a tree.
__global__ void __launch_bounds__(kJoinCols *kJoinSlices) norm_join_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float sum[kJoinSlices][kJoinCols + 1];
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    const uint32_t c = threadIdx.x % kJoinCols, s = threadIdx.x / kJoinCols;
    const uint32_t first = blockIdx.x * kJoinCols;
    float v = 0.0f;
    if (first + c < p.cols) {
        const float *in = p.partial + blockIdx.y * (uint64_t)p.cols + first + c;
        for (uint32_t k = s; k < p.parts; k += kJoinSlices * 10) {
            float o[10];   // on their way at the same time: 152 shares are 10 of each slice
#pragma unroll
            for (uint32_t j = 0; j < 10; ++j) {
                const uint32_t at = k + j * kJoinSlices;
                const float *from = in + (uint64_t)at * 2 * p.cols;
                o[j] = at < p.parts && NORM_BUFFER_OK(kNormWorkspace, from, 4) ? *from : 0.0f;
            }
#pragma unroll
            for (uint32_t j = 0; j < 10; ++j) v += o[j];
        }
    }
    sum[s][c] = v;
    __syncthreads();
    // half a warp to a column, a lane to a slice
    const uint32_t mine = threadIdx.x / kJoinSlices, col = first + mine;
    v = sum[threadIdx.x % kJoinSlices][mine];
#pragma unroll
    for (int o = kJoinSlices / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (threadIdx.x % kJoinSlices == 0 && col < p.cols) {
        if (p.avg) v = avg_of(v, p.P, p.avg_scale, p.avg_pow2);
        void *out = blockIdx.y ? p.dbias : p.dweight;
        if (out && p.weight_bf16) {
            uint16_t *to = static_cast<uint16_t *>(out) + col;
            if (NORM_BUFFER_OK(blockIdx.y ? kNormDbias : kNormDweight, to, 2)) *to = f32_to_bf16(v);
        } else if (out) {
            float *to = static_cast<float *>(out) + col;
            if (NORM_BUFFER_OK(blockIdx.y ? kNormDbias : kNormDweight, to, 4)) *to = v;
        }
    }
    DT_TL_END_BLOCK(DT_TL_NORM);
}

// Rows too long for registers: a block to a row, which it reads from memory
// (L2, mostly) once for each sum and once for the result.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) norm_long_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float red[2][2][kNormThreads / 32];
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    uint32_t phase = 0;
    for (uint64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        uint64_t local;
        const int r = find_rank(p, row, local);
        const T *x = static_cast<const T *>(p.x[r]) + local * p.cols;
        T *y = static_cast<T *>(p.out[r]) + local * p.cols;
        auto at = [&](uint32_t e) {
            return NORM_OK(0, r, x + e, sizeof(T)) ? to_f32(x[e]) : 0.0f;
        };
        float s[2] = {0.0f, 0.0f}, m2[2] = {0.0f, 0.0f};
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) s[0] += at(e);
        row_sum<2>(s, red, phase, Team<32>(kLongThreads));
        const float mean = s[0] * p.inv_cols;
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            const float d = at(e) - mean;
            m2[0] = fmaf(d, d, m2[0]);
        }
        row_sum<2>(m2, red, phase, Team<32>(kLongThreads));
        const float rstd = rstd_of(m2[0], p.inv_cols, p.eps);
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            const float f = fmaf((at(e) - mean) * rstd, param<0>(p, e), param<1>(p, e));
            if (NORM_OK(2, r, y + e, sizeof(T))) from_f32(f, y + e);
        }
        if (threadIdx.x == 0) {
            if (p.mean[r] && NORM_OK(3, r, p.mean[r] + local, 4)) p.mean[r][local] = mean;
            if (p.rstd[r] && NORM_OK(4, r, p.rstd[r] + local, 4)) p.rstd[r][local] = rstd;
        }
    }
    DT_TL_END_BLOCK(DT_TL_NORM);
}

template <typename T>
__global__ void __launch_bounds__(kLongThreads) norm_backward_long_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float red[2][2][kNormThreads / 32];
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    uint32_t phase = 0;
    for (uint64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        uint64_t local;
        const int r = find_rank(p, row, local);
        const T *x = static_cast<const T *>(p.x[r]) + local * p.cols;
        const T *dy = static_cast<const T *>(p.dy[r]) + local * p.cols;
        T *dx = static_cast<T *>(p.out[r]) + local * p.cols;
        const float mean = NORM_OK(3, r, p.mean[r] + local, 4) ? p.mean[r][local] : 0.0f;
        const float rstd = NORM_OK(4, r, p.rstd[r] + local, 4) ? p.rstd[r][local] : 0.0f;
        auto h_at = [&](uint32_t e) {
            return NORM_OK(0, r, x + e, sizeof(T)) ? (to_f32(x[e]) - mean) * rstd : 0.0f;
        };
        auto q_at = [&](uint32_t e) {
            return NORM_OK(1, r, dy + e, sizeof(T)) ? to_f32(dy[e]) * param<0>(p, e) : 0.0f;
        };
        float s[2] = {0.0f, 0.0f};
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            const float q = q_at(e);
            s[0] += q;
            s[1] = fmaf(q, h_at(e), s[1]);
        }
        row_sum<2>(s, red, phase, Team<32>(kLongThreads));
        const float mq = s[0] * p.inv_cols, mqh = s[1] * p.inv_cols;
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            const float f = rstd * (q_at(e) - mq - h_at(e) * mqh);
            if (NORM_OK(2, r, dx + e, sizeof(T))) from_f32(f, dx + e);
        }
    }
    DT_TL_END_BLOCK(DT_TL_NORM);
}

// The column sums of such rows: thread per column, block (x, s) over every
// parts-th row from s on.  It runs before the kernel above, whose dx may be
// written over dy.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_columns_long_kernel(const __grid_constant__ NormParams p)
{
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    const uint32_t e = blockIdx.x * kThreads + threadIdx.x;
    if (e < p.cols) {
        float dw = 0.0f, db = 0.0f;
        for (uint64_t row = blockIdx.y; row < p.rows; row += p.parts) {
            uint64_t local;
            const int r = find_rank(p, row, local);
            const uint64_t at = local * p.cols + e;
            const T *x = static_cast<const T *>(p.x[r]) + at, *dy = static_cast<const T *>(p.dy[r]) + at;
            if (!NORM_OK(0, r, x, sizeof(T)) || !NORM_OK(1, r, dy, sizeof(T)) || !NORM_OK(3, r, p.mean[r] + local, 4) ||
                !NORM_OK(4, r, p.rstd[r] + local, 4))
                continue;
            const float d = to_f32(*dy);
            dw = fmaf(d, (to_f32(*x) - p.mean[r][local]) * p.rstd[r][local], dw);
            db += d;
        }
        float *out = p.partial + (uint64_t)blockIdx.y * 2 * p.cols + e;
        if (NORM_BUFFER_OK(kNormWorkspace, out, 4)) *out = dw;
        if (NORM_BUFFER_OK(kNormWorkspace, out + p.cols, 4)) out[p.cols] = db;
    }
    DT_TL_END_BLOCK(DT_TL_NORM);
}

using NormFn = void (*)(NormParams);

// The kernel for rows of `cols` elements, either way, and the threads that
// share a row: 16 columns of bf16 or 8 of f32 a thread (bf16 8 where that leaves
// fewer threads idle), in as few lanes of a warp as that takes; or 16 where
// that keeps the row within 256 threads, so that two groups or more share an
// SM and one computes while another waits at its barrier (4 x 2048 x 4096
// backward: over 512 threads 47.0 us, over 256 46.6).  Past 256 threads of 32
// columns a row may have 512; beyond that, a thread's sums for its columns
// would not fit in registers (32 columns of f32 spill 540 bytes as it is, of
// bf16 94).  100 MB of rows of 64, 128, 384 bf16 backward: 8
// columns and a warp to a row 161, 93, 100 us; this 61, 61, 75.
struct NormPick {
    NormFn fn = nullptr;
    uint32_t tpr = 0, threads = 0, rows = 0;   // of a row; of a group, and the rows that it sums at a time
};

template <typename T, int VEC, int N, int L, bool BACK>
void try_pick(NormPick &k, uint32_t chunks, uint32_t most)
{
    const uint32_t tpr = L < 32 ? L : ((chunks + N - 1) / N + 31) / 32 * 32;
    if (k.fn || tpr > most || chunks > tpr * N) return;
    if constexpr (BACK) k.fn = norm_backward_kernel<T, VEC, N, L>;
    else k.fn = norm_kernel<T, VEC, N, L>;
    k.tpr = tpr;
    k.threads = L < 32 ? 32 : tpr;
    k.rows = rows_at_once<T, VEC, N, BACK>() * (32 / L);
}

template <typename T, int VEC, bool BACK>
NormPick pick_norm(uint32_t cols)
{
    NormPick k;
    const uint32_t chunks = (cols + VEC - 1) / VEC;
    if constexpr (VEC == 1) {   // 65 f32, 100 MB: a warp to a row 87 us forward, 8 lanes' 8 columns 44
        try_pick<T, VEC, 8, 8, BACK>(k, chunks, 32);
        try_pick<T, VEC, 8, 16, BACK>(k, chunks, 32);
        try_pick<T, VEC, 8, 32, BACK>(k, chunks, 256);
        try_pick<T, VEC, 16, 32, BACK>(k, chunks, kNormThreads);
    } else if constexpr (!BACK) {   // what is left to this kernel is longer than 256 threads of 4 vectors
        try_pick<T, VEC, 32 / VEC, 32, BACK>(k, chunks, kNormThreads);
    } else {
        try_pick<T, VEC, 2, 4, BACK>(k, chunks, 32);
        try_pick<T, VEC, 2, 8, BACK>(k, chunks, 32);
        try_pick<T, VEC, 2, 16, BACK>(k, chunks, 32);
        if constexpr (VEC == 8)
            if ((chunks + 31) / 32 * 32 * 1.1 < (chunks + 63) / 64 * 64) try_pick<T, VEC, 1, 32, BACK>(k, chunks, 256);
        try_pick<T, VEC, 2, 32, BACK>(k, chunks, 256);
        if constexpr (VEC == 4) try_pick<T, VEC, 4, 32, BACK>(k, chunks, 256);
        try_pick<T, VEC, 16 / VEC, 32, BACK>(k, chunks, kNormThreads);
        try_pick<T, VEC, 32 / VEC, 32, BACK>(k, chunks, kNormThreads);
    }
    return k;
}

template <bool BACK>
NormPick pick_norm(int dtype, bool vec, uint32_t cols)
{
    if (dtype == DT_BF16) return vec ? pick_norm<uint16_t, 8, BACK>(cols) : pick_norm<uint16_t, 1, BACK>(cols);
    return vec ? pick_norm<float, 4, BACK>(cols) : pick_norm<float, 1, BACK>(cols);
}

// The kernel that has a row in registers, and the threads of a row.  Few rows:
// as many threads as a row has vectors.  Else, for rows of whole vectors, 4
// vectors a thread in as few lanes of a warp as that takes, or 4 to 6 vectors
// and whole warps, whichever leaves the fewest threads idle (100 MB of rows of
// 2056 bf16: 4 and 5 vectors 58, 49 us; of 640 f32 40, 32; 5 and 6 vectors of
// bf16 spill 28 and 56 bytes of their 64 registers and are faster all the same).
template <typename T, int VEC>
NormPick pick_rows(uint32_t cols, bool few)
{
    NormPick k;
    const uint32_t chunks = (cols + VEC - 1) / VEC;
    auto take = [&](NormFn fn, uint32_t tpr) {
        k.fn = fn;
        k.tpr = tpr;
    };
    auto warps = [&](uint32_t n) { return ((chunks + n - 1) / n + 31) / 32 * 32; };
    if (few) {
        if (warps(1) <= kNormThreads) take(norm_rows_kernel<T, VEC, 1, 32, true>, warps(1));
        else if (warps(2) <= kNormThreads) take(norm_rows_kernel<T, VEC, 2, 32, true>, warps(2));
        if (k.fn) return k;
    }
    if constexpr (VEC > 1) {
        // what a row costs: its threads' vectors, and more where a block has one of an odd number of warps
        auto cost = [&](uint32_t n, uint32_t most, double factor) {
            const uint32_t t = warps(n);
            return t > most ? 1e30 : n * t * factor * (t & (t - 1) ? 1.15 : 1.0);
        };
        const double c4 = cost(4, 256, 1.0), c5 = cost(5, 128, 1.08), c6 = cost(6, 128, 1.12);
        if (chunks <= 16) take(norm_rows_kernel<T, VEC, 4, 4, false>, 4);
        else if (chunks <= 32) take(norm_rows_kernel<T, VEC, 4, 8, false>, 8);
        else if (chunks <= 64) take(norm_rows_kernel<T, VEC, 4, 16, false>, 16);
        else if (c4 <= c5 && c4 <= c6 && c4 < 1e30) take(norm_rows_kernel<T, VEC, 4, 32, false>, warps(4));
        else if (c5 <= c6 && c5 < 1e30) take(norm_rows_kernel<T, VEC, 5, 32, false>, warps(5));
        else if (c6 < 1e30) take(norm_rows_kernel<T, VEC, 6, 32, false>, warps(6));
    }
    return k;
}

NormPick pick_rows(int dtype, bool vec, uint32_t cols, bool few)
{
    if (dtype == DT_BF16) return vec ? pick_rows<uint16_t, 8>(cols, few) : pick_rows<uint16_t, 1>(cols, few);
    return vec ? pick_rows<float, 4>(cols, few) : pick_rows<float, 1>(cols, few);
}

// The grid, the groups and the rings of a call.
struct NormShape {
    uint32_t grid, threads;
    size_t smem;
};

NormShape norm_shape(NormParams &p, const NormPick &k, int dtype, bool vec, bool back, int device)
{
    const uint64_t row_bytes = (uint64_t)p.cols * (dtype == DT_BF16 ? 2 : 4), sms = (uint64_t)sm_count(device);
    p.tpr = k.tpr;
    uint64_t groups = kNormThreads / k.threads;
    if (k.threads > 32) groups = std::min<uint64_t>(groups, 15);   // named barriers
    // rows of a stage: those summed at once, and more where they are short,
    // but not so many that groups go without
    // (at most 256 backward, whose means and reciprocals take 8 bytes a row: all
    // groups' stages fit kSmemBytes then, or pass it by the stages' rounding)
    uint64_t per = std::max<uint64_t>(kStageTarget / std::max<uint64_t>(row_bytes, back ? 16 : 1), k.rows);
    per = std::max<uint64_t>(1, std::min(per, p.rows / (groups * sms)));
    p.chunk_rows = (uint32_t)per;
    p.chunks = 0;
    for (int r = 0; r < p.P; ++r)
        p.chunk_end[r] = p.chunks += (p.row_end[r] - (r ? p.row_end[r - 1] : 0) + per - 1) / per;
    const uint64_t grid = std::min(sms, p.chunks);
    groups = std::min(groups, (p.chunks + grid - 1) / grid);
    p.parts = (uint32_t)(grid * groups);
    // rows at other offsets are copied with up to 15 bytes at either end
    p.array_bytes = (uint32_t)((per * row_bytes + (vec ? 0 : 32) + 127) / 128 * 128);
    p.stat_bytes = back ? (uint32_t)((per * 4 + 32 + 63) / 64 * 64) : 0;
    p.stage_bytes = back ? 2 * (p.array_bytes + p.stat_bytes) : p.array_bytes;
    const uint64_t depth = (p.chunks + p.parts - 1) / p.parts;
    p.stages = (uint32_t)std::max<uint64_t>(1, std::min({(uint64_t)kMaxStages, kSmemBytes / (groups * p.stage_bytes), depth}));
    const size_t rings = groups * p.stages * (p.stage_bytes + 8), sums = back ? groups * 2 * (size_t)p.cols * sizeof(float) : 0;
    return {(uint32_t)grid, (uint32_t)(groups * k.threads), std::max(rings, sums)};
}

cudaError_t launch_rows(NormFn fn, const NormShape &n, const NormParams &p, cudaStream_t s)
{
    // A kernel may have 48 KB without asking, its static part (up to 1 KB of these) included.
    if (n.smem > 46 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(fn, dim3(n.grid), dim3(n.threads), n.smem, s, false, p);
}

}  // namespace

DT_TL_BINDER(bind_timeline_norm)

size_t norm_workspace(uint32_t cols, int device)
{
    // a share to a block, or to a slice of the rows where a row is too long for
    // any block's registers (and may be for those of one that takes it element by element)
    const int blocks = cols > kMostColumns ? 0 : sm_count(device);
    return (size_t)std::max(blocks, kLongSlices) * 2 * cols * sizeof(float);
}

cudaError_t launch_norm(NormParams p, int dtype, bool vec, int device, cudaStream_t s)
{
    const bool few = p.rows <= 2 * (uint64_t)sm_count(device);
    const NormPick rows = pick_rows(dtype, vec, p.cols, few);
    if (rows.fn) {
        const uint32_t threads = few ? rows.tpr : std::max(rows.tpr, 256 / rows.tpr * rows.tpr), per = threads / rows.tpr;
        uint64_t most = 0, blocks = 0;   // blocks of the rank with the most rows, and of all
        for (int r = 0; r < p.P; ++r) {
            const uint64_t n = (p.row_end[r] - (r ? p.row_end[r - 1] : 0) + per - 1) / per;
            most = std::max(most, n);
            p.chunk_end[r] = blocks += n;
        }
        if (blocks <= 0x7FFFFFFF) {
            // With one rank of 16 holding all rows, 67 MB of rows of 64, 256, 4096 bf16 took 289,
            // 164, 90 us on a grid of 16 rows of blocks; this way 34, 29, 31 (a single rank: 33,
            // 29, 31).  Ranks of 1 : 3 : 5 : 7, 4 x 2048 rows of 4096: 29.0 and 29.6.
            const bool even = most * p.P <= blocks + blocks / 4;
            p.chunks = even ? 0 : blocks;
            p.tpr = rows.tpr;
            const bool whole = p.weight && p.bias && ((uintptr_t)p.weight & 15) == 0 && ((uintptr_t)p.bias & 15) == 0;
            p.param_kind = !vec || !whole ? kParamAny : !p.weight_bf16 ? kParamF32 : dtype == DT_BF16 ? kParamBf16 : kParamAny;
            const dim3 grid(even ? (unsigned)most : (unsigned)blocks, even ? (unsigned)p.P : 1u);
            return launch_kernel(rows.fn, grid, dim3(threads), 0, s, false, p);
        }
    }
    const NormPick k = pick_norm<false>(dtype, vec, p.cols);
    if (k.fn) return launch_rows(k.fn, norm_shape(p, k, dtype, vec, false, device), p, s);
    const NormFn fn = dtype == DT_BF16 ? norm_long_kernel<uint16_t> : norm_long_kernel<float>;
    int resident = 0;
    const cudaError_t e = resident_blocks(reinterpret_cast<const void *>(fn), kLongThreads, device, &resident);
    if (e != cudaSuccess) return e;
    const uint64_t grid = std::min(p.rows, (uint64_t)resident);
    return launch_kernel(fn, dim3((unsigned)grid), dim3(kLongThreads), 0, s, false, p);
}

cudaError_t launch_norm_backward(NormParams p, int dtype, bool vec, int device, cudaStream_t s)
{
    const NormPick k = pick_norm<true>(dtype, vec, p.cols);
    cudaError_t e = cudaSuccess;
    if (p.rows == 0) {
        p.parts = 0;
    } else if (k.fn) {
        const NormShape n = norm_shape(p, k, dtype, vec, true, device);
        e = launch_rows(k.fn, n, p, s);
        p.parts = n.grid;   // a share to a block
    } else {
        const bool bf16 = dtype == DT_BF16;
        if (p.partial) {
            p.parts = (uint32_t)std::min<uint64_t>(p.rows, kLongSlices);
            e = launch_kernel(bf16 ? norm_columns_long_kernel<uint16_t> : norm_columns_long_kernel<float>,
                              dim3((p.cols + kThreads - 1) / kThreads, p.parts), dim3(kThreads), 0, s, false, p);
            if (e != cudaSuccess) return e;
        }
        const NormFn fn = bf16 ? norm_backward_long_kernel<uint16_t> : norm_backward_long_kernel<float>;
        int resident = 0;
        e = resident_blocks(reinterpret_cast<const void *>(fn), kLongThreads, device, &resident);
        if (e != cudaSuccess) return e;
        const uint64_t grid = std::min(p.rows, (uint64_t)resident);
        e = launch_kernel(fn, dim3((unsigned)grid), dim3(kLongThreads), 0, s, false, p);
    }
    if (e != cudaSuccess || !p.partial) return e;
    return launch_kernel(norm_join_kernel, dim3((p.cols + kJoinCols - 1) / kJoinCols, 2),
                         dim3(kJoinCols * kJoinSlices), 0, s, false, p);
}

}  // namespace dt
