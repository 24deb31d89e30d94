// Layer norm over the rows of P ranks, forward and backward, and the
// reduction of the weight's and bias' gradients over every rank's rows.
//
//   mu = mean_j x_j      v = mean_j (x_j - mu)^2      r = 1 / sqrt(v + eps)
//   h_j = (x_j - mu) r   y_j = h_j w_j + b_j
//   q_j = dy_j w_j       dx_j = r (q_j - mean(q) - h_j mean(q h))
//   dw_j = sum_rows dy_j h_j      db_j = sum_rows dy_j
//
// The ranks' rows are one list, so that a call is one launch (two for the
// backward pass) whatever the number of ranks.  Both directions are bound by
// HBM: about 4 and 5 flops per byte.  A row is read once: its elements stay
// in the registers of the `tpr` threads that share it, the variance is the
// mean of the squared distances from the mean (a second pass over registers,
// not E[x^2] - mu^2, which loses every digit where |mu| is large), and all
// sums are fp32.  Results are rounded once, at the store.
//
// Blocks stay resident and walk over the rows; each loads its next row before
// it works on the present one, so that loads are always in flight.  The
// backward pass keeps its share of dw and db in registers over all of its
// rows and writes it once; a second kernel adds the shares in a fixed order,
// so the result depends on the device and the shapes alone, not on timing.
#include "dt_ops.h"

#include "dt_bounds.cuh"
#include "dt_device.cuh"
#include "dt_math.cuh"
#include "dt_timeline.cuh"

namespace dt {
namespace {

constexpr int kNormThreads = 512;    // most threads of a block, and of a row
constexpr int kLongThreads = 512;    // rows too long for registers
constexpr int kLongSlices = 32;      // row slices of the column sums there
constexpr int kJoinCols = 32;        // columns and row slices of a block that adds the shares
constexpr int kJoinSlices = 16;

// VEC elements as they lie in memory: one 16-byte vector, or one element.
template <typename T, int VEC>
struct Chunk {
    static_assert(VEC * sizeof(T) == 16, "a vector is 16 bytes");
    uint4 v;
    __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[VEC]) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (VEC == 8) {
                f[2 * i] = bf16_lo(w[i]);
                f[2 * i + 1] = bf16_hi(w[i]);
            } else {
                f[i] = __uint_as_float(w[i]);
            }
        }
    }
    static __device__ __forceinline__ void store(T *p, const float (&f)[VEC])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (VEC == 8) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
            else w[i] = __float_as_uint(f[i]);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ void from_f32(float f, float *p) { *p = f; }
__device__ __forceinline__ void from_f32(float f, uint16_t *p) { *p = f32_to_bf16(f); }

template <typename T>
struct Chunk<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void zero() { v = 0; }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f32(v); }
    static __device__ __forceinline__ void store(T *p, const float (&f)[1]) { from_f32(f[0], p); }
};

// Element j of the weight or bias, `none` where there is none.
__device__ __forceinline__ float param(const void *p, int bf16, uint32_t j, float none)
{
    if (!p) return none;
    return bf16 ? bf16_to_f32(static_cast<const uint16_t *>(p)[j]) : static_cast<const float *>(p)[j];
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

#ifdef DT_BOUNDS
// [a, a + n) lies in rank r's buffer of `elem` bytes for each of its rows'
// elements (mean and rstd: cols = 1).
__device__ __forceinline__ bool in_rank(const NormParams &p, const void *const *base, int kind, int r,
                                        const void *a, uint64_t n, uint64_t row_bytes)
{
    const uint64_t lo = reinterpret_cast<uint64_t>(base[r]);
    const uint64_t rows = p.row_end[r] - (r ? p.row_end[r - 1] : 0);
    return DT_IN_BOUNDS(span_in(a, n, lo, lo + rows * row_bytes), p.sink, DT_BOUNDS_NORM,
                        kind * DT_MAX_RANKS + r, a, lo);
}
#define NORM_OK(base, kind, r, a, n, row_bytes) \
    in_rank(p, reinterpret_cast<const void *const *>(base), (kind), (r), (a), (n), (row_bytes))
#else
#define NORM_OK(base, kind, r, a, n, row_bytes) true
#endif

// Sums of K values over the tpr threads of a row; every thread gets the same
// sums, in the same order of addition.  `red` is double-buffered by the
// caller's `phase`: a buffer is written again only after the barrier of the
// sum in between, which every reader of it has passed.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*red)[32][2], uint32_t &phase, uint32_t tpr,
                                        uint32_t group)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
    if (tpr == 32) return;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t first = group * (tpr >> 5), warps = tpr >> 5;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) red[phase][warp][k] = v[k];
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lane < warps ? red[phase][first + lane][k] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
    phase ^= 1;
}

// A row in registers: chunk c of thread t is elements [(c * tpr + t) * VEC,
// + VEC).
template <typename T, int VEC, int N>
__device__ __forceinline__ void load_row(Chunk<T, VEC> (&c)[N], const NormParams &p, const void *const *base,
                                         int kind, uint64_t row, uint32_t t)
{
    uint64_t local;
    const int r = find_rank(p, row, local);
    const T *src = static_cast<const T *>(base[r]) + local * p.cols;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint32_t e = (n * p.tpr + t) * VEC;
        if (e < p.cols && NORM_OK(base, kind, r, src + e, VEC * sizeof(T), p.cols * sizeof(T))) c[n].load(src + e);
        else c[n].zero();
    }
}

template <typename T, int VEC, int N>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const __grid_constant__ NormParams p)
{
    // weights of up to 16 elements a thread stay in registers over all rows;
    // wider rows read them again from L1
    constexpr bool kHold = N * VEC <= 16;
    __shared__ float red[2][32][2];
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    const uint32_t tpr = p.tpr, groups = blockDim.x / tpr, group = threadIdx.x / tpr, t = threadIdx.x % tpr;
    const uint64_t step = (uint64_t)gridDim.x * groups;
    uint64_t row = (uint64_t)blockIdx.x * groups + group;
    uint32_t phase = 0;
    Chunk<T, VEC> next[N];
    if (row < p.rows) load_row<T, VEC, N>(next, p, p.x, 0, row, t);

    float w[kHold ? N * VEC : 1], b[kHold ? N * VEC : 1];
    if constexpr (kHold)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const uint32_t e = (n * tpr + t) * VEC + i;
                w[n * VEC + i] = e < p.cols ? param(p.weight, p.weight_bf16, e, 1.0f) : 0.0f;
                b[n * VEC + i] = e < p.cols ? param(p.bias, p.weight_bf16, e, 0.0f) : 0.0f;
            }

    for (; row < p.rows; row += step) {
        Chunk<T, VEC> x[N];
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = next[n];
        if (row + step < p.rows) load_row<T, VEC, N>(next, p, p.x, 0, row + step, t);

        float s[1] = {0.0f};
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float f[VEC];
            x[n].get(f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] += f[i];
        }
        row_sum<1>(s, red, phase, tpr, group);
        const float mean = __fdiv_rn(s[0], (float)p.cols);
        float m2[1] = {0.0f};
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if ((n * tpr + t) * VEC >= p.cols) continue;
            float f[VEC];
            x[n].get(f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) m2[0] = fmaf(f[i] - mean, f[i] - mean, m2[0]);
        }
        row_sum<1>(m2, red, phase, tpr, group);
        const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(m2[0], (float)p.cols) + p.eps));

        uint64_t local;
        const int r = find_rank(p, row, local);
        T *y = static_cast<T *>(p.out[r]) + local * p.cols;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint32_t e = (n * tpr + t) * VEC;
            if (e >= p.cols) continue;
            float f[VEC];
            x[n].get(f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float wi = kHold ? w[kHold ? n * VEC + i : 0] : param(p.weight, p.weight_bf16, e + i, 1.0f);
                const float bi = kHold ? b[kHold ? n * VEC + i : 0] : param(p.bias, p.weight_bf16, e + i, 0.0f);
                f[i] = fmaf((f[i] - mean) * rstd, wi, bi);
            }
            if (NORM_OK(p.out, 2, r, y + e, VEC * sizeof(T), p.cols * sizeof(T))) Chunk<T, VEC>::store(y + e, f);
        }
        if (t == 0) {
            if (p.mean[r] && NORM_OK(p.mean, 3, r, p.mean[r] + local, 4, 4)) p.mean[r][local] = mean;
            if (p.rstd[r] && NORM_OK(p.rstd, 4, r, p.rstd[r] + local, 4, 4)) p.rstd[r][local] = rstd;
        }
    }
    DT_TL_END_BLOCK(DT_TL_NORM);
}

template <typename T, int VEC, int N>
__global__ void __launch_bounds__(kNormThreads) norm_backward_kernel(const __grid_constant__ NormParams p)
{
    constexpr bool kAhead = N * VEC * sizeof(T) <= 32;   // the next row's registers fit beside the sums
    constexpr bool kHold = N * VEC <= 16;
    __shared__ float red[2][32][2];
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    const uint32_t tpr = p.tpr, groups = blockDim.x / tpr, group = threadIdx.x / tpr, t = threadIdx.x % tpr;
    const uint64_t step = (uint64_t)gridDim.x * groups;
    const uint64_t part = (uint64_t)blockIdx.x * groups + group;
    uint64_t row = part;
    uint32_t phase = 0;
    Chunk<T, VEC> xn[N], gn[N];
    if (kAhead && row < p.rows) {
        load_row<T, VEC, N>(xn, p, p.x, 0, row, t);
        load_row<T, VEC, N>(gn, p, p.dy, 1, row, t);
    }
    float dw[N * VEC], db[N * VEC], w[kHold ? N * VEC : 1];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const uint32_t e = (n * tpr + t) * VEC + i;
            dw[n * VEC + i] = db[n * VEC + i] = 0.0f;
            if constexpr (kHold) w[n * VEC + i] = e < p.cols ? param(p.weight, p.weight_bf16, e, 1.0f) : 0.0f;
        }

    for (; row < p.rows; row += step) {
        Chunk<T, VEC> x[N], g[N];
        uint64_t local;
        const int r = find_rank(p, row, local);
        const float mean = NORM_OK(p.mean, 3, r, p.mean[r] + local, 4, 4) ? p.mean[r][local] : 0.0f;
        const float rstd = NORM_OK(p.rstd, 4, r, p.rstd[r] + local, 4, 4) ? p.rstd[r][local] : 0.0f;
        if constexpr (kAhead) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                x[n] = xn[n];
                g[n] = gn[n];
            }
            if (row + step < p.rows) {
                load_row<T, VEC, N>(xn, p, p.x, 0, row + step, t);
                load_row<T, VEC, N>(gn, p, p.dy, 1, row + step, t);
            }
        } else {
            load_row<T, VEC, N>(x, p, p.x, 0, row, t);
            load_row<T, VEC, N>(g, p, p.dy, 1, row, t);
        }
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint32_t e = (n * tpr + t) * VEC;
            if (e >= p.cols) continue;
            float f[VEC], d[VEC];
            x[n].get(f);
            g[n].get(d);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float h = (f[i] - mean) * rstd;
                const float q = d[i] * (kHold ? w[kHold ? n * VEC + i : 0] : param(p.weight, p.weight_bf16, e + i, 1.0f));
                s[0] += q;
                s[1] = fmaf(q, h, s[1]);
                dw[n * VEC + i] = fmaf(d[i], h, dw[n * VEC + i]);
                db[n * VEC + i] += d[i];
            }
        }
        row_sum<2>(s, red, phase, tpr, group);
        const float mq = __fdiv_rn(s[0], (float)p.cols), mqh = __fdiv_rn(s[1], (float)p.cols);
        T *dx = static_cast<T *>(p.out[r]) + local * p.cols;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint32_t e = (n * tpr + t) * VEC;
            if (e >= p.cols) continue;
            float f[VEC], d[VEC];
            x[n].get(f);
            g[n].get(d);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float h = (f[i] - mean) * rstd;
                const float q = d[i] * (kHold ? w[kHold ? n * VEC + i : 0] : param(p.weight, p.weight_bf16, e + i, 1.0f));
                f[i] = rstd * (q - mq - h * mqh);
            }
            if (NORM_OK(p.out, 2, r, dx + e, VEC * sizeof(T), p.cols * sizeof(T))) Chunk<T, VEC>::store(dx + e, f);
        }
    }
    if (p.partial && part < p.parts) {
        float *out = p.partial + part * 2 * p.cols;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const uint32_t e = (n * tpr + t) * VEC + i;
                if (e >= p.cols) continue;
                out[e] = dw[n * VEC + i];
                out[p.cols + e] = db[n * VEC + i];
            }
    }
    DT_TL_END_BLOCK(DT_TL_NORM);
}

// Adds the shares of dw (blockIdx.y 0) and db (1): thread (c, s) adds shares
// s, s + 16, ... of its column, then the 16 sums are added in ascending order.
__global__ void __launch_bounds__(kJoinCols *kJoinSlices) norm_join_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float sum[kJoinSlices][kJoinCols];
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    const uint32_t c = threadIdx.x % kJoinCols, s = threadIdx.x / kJoinCols;
    const uint32_t col = blockIdx.x * kJoinCols + c;
    float v = 0.0f;
    if (col < p.cols) {
        const float *in = p.partial + blockIdx.y * (uint64_t)p.cols + col;
#pragma unroll 4
        for (uint32_t k = s; k < p.parts; k += kJoinSlices) v += in[(uint64_t)k * 2 * p.cols];
    }
    sum[s][c] = v;
    __syncthreads();
    if (s == 0 && col < p.cols) {
        for (int k = 1; k < kJoinSlices; ++k) v += sum[k][c];
        if (p.avg) v = avg_of(v, p.P, p.avg_scale, p.avg_pow2);
        void *out = blockIdx.y ? p.dbias : p.dweight;
        if (out) {
            if (p.weight_bf16) static_cast<uint16_t *>(out)[col] = f32_to_bf16(v);
            else static_cast<float *>(out)[col] = v;
        }
    }
    DT_TL_END_BLOCK(DT_TL_NORM);
}

// Rows too long for registers: a block to a row, which it reads from memory
// (L2, mostly) once for each sum and once for the result.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) norm_long_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float red[2][32][2];
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
            return NORM_OK(p.x, 0, r, x + e, sizeof(T), p.cols * sizeof(T)) ? to_f32(x[e]) : 0.0f;
        };
        float s[1] = {0.0f}, m2[1] = {0.0f};
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) s[0] += at(e);
        row_sum<1>(s, red, phase, kLongThreads, 0);
        const float mean = __fdiv_rn(s[0], (float)p.cols);
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            const float d = at(e) - mean;
            m2[0] = fmaf(d, d, m2[0]);
        }
        row_sum<1>(m2, red, phase, kLongThreads, 0);
        const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(m2[0], (float)p.cols) + p.eps));
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            const float f = fmaf((at(e) - mean) * rstd, param(p.weight, p.weight_bf16, e, 1.0f),
                                 param(p.bias, p.weight_bf16, e, 0.0f));
            if (NORM_OK(p.out, 2, r, y + e, sizeof(T), p.cols * sizeof(T))) from_f32(f, y + e);
        }
        if (threadIdx.x == 0) {
            if (p.mean[r] && NORM_OK(p.mean, 3, r, p.mean[r] + local, 4, 4)) p.mean[r][local] = mean;
            if (p.rstd[r] && NORM_OK(p.rstd, 4, r, p.rstd[r] + local, 4, 4)) p.rstd[r][local] = rstd;
        }
    }
    DT_TL_END_BLOCK(DT_TL_NORM);
}

template <typename T>
__global__ void __launch_bounds__(kLongThreads) norm_backward_long_kernel(const __grid_constant__ NormParams p)
{
    __shared__ float red[2][32][2];
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
        const float mean = NORM_OK(p.mean, 3, r, p.mean[r] + local, 4, 4) ? p.mean[r][local] : 0.0f;
        const float rstd = NORM_OK(p.rstd, 4, r, p.rstd[r] + local, 4, 4) ? p.rstd[r][local] : 0.0f;
        auto h_at = [&](uint32_t e) {
            return NORM_OK(p.x, 0, r, x + e, sizeof(T), p.cols * sizeof(T)) ? (to_f32(x[e]) - mean) * rstd : 0.0f;
        };
        auto q_at = [&](uint32_t e) {
            return NORM_OK(p.dy, 1, r, dy + e, sizeof(T), p.cols * sizeof(T))
                       ? to_f32(dy[e]) * param(p.weight, p.weight_bf16, e, 1.0f) : 0.0f;
        };
        float s[2] = {0.0f, 0.0f};
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            const float q = q_at(e);
            s[0] += q;
            s[1] = fmaf(q, h_at(e), s[1]);
        }
        row_sum<2>(s, red, phase, kLongThreads, 0);
        const float mq = __fdiv_rn(s[0], (float)p.cols), mqh = __fdiv_rn(s[1], (float)p.cols);
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            const float f = rstd * (q_at(e) - mq - h_at(e) * mqh);
            if (NORM_OK(p.out, 2, r, dx + e, sizeof(T), p.cols * sizeof(T))) from_f32(f, dx + e);
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
            if (!NORM_OK(p.x, 0, r, x, sizeof(T), p.cols * sizeof(T)) ||
                !NORM_OK(p.dy, 1, r, dy, sizeof(T), p.cols * sizeof(T)))
                continue;
            const float d = to_f32(*dy);
            dw = fmaf(d, (to_f32(*x) - p.mean[r][local]) * p.rstd[r][local], dw);
            db += d;
        }
        p.partial[(uint64_t)blockIdx.y * 2 * p.cols + e] = dw;
        p.partial[(uint64_t)blockIdx.y * 2 * p.cols + p.cols + e] = db;
    }
    DT_TL_END_BLOCK(DT_TL_NORM);
}

using NormFn = void (*)(NormParams);

// The kernel for rows of `chunks` chunks, and the threads that share a row.
// The fewest chunks a thread that keep a row within 256 threads: 4096 bf16
// elements are 2 x 16 bytes of 256 threads.  Backward instances stop where
// two sums for each element no longer fit in registers.
struct NormPick {
    NormFn fn = nullptr;
    uint32_t tpr = 0;
};

template <typename T, int VEC, int N, bool BACK>
bool try_pick(NormPick &k, uint32_t chunks, uint32_t most)
{
    const uint32_t tpr = ((chunks + N - 1) / N + 31) / 32 * 32;
    if (tpr > most) return false;
    if constexpr (BACK) k.fn = norm_backward_kernel<T, VEC, N>;
    else k.fn = norm_kernel<T, VEC, N>;
    k.tpr = tpr;
    return true;
}

template <typename T, int VEC, bool BACK>
NormPick pick_norm(uint32_t cols)
{
    NormPick k;
    const uint32_t chunks = (cols + VEC - 1) / VEC;
    constexpr int kMost = VEC == 1 ? 16 : BACK ? 16 / VEC * 2 : 8;   // chunks a thread
    if (try_pick<T, VEC, 1, BACK>(k, chunks, 32) || try_pick<T, VEC, 2, BACK>(k, chunks, 256) ||
        try_pick<T, VEC, 4, BACK>(k, chunks, 256))
        return k;
    if constexpr (kMost >= 8)
        if (try_pick<T, VEC, 8, BACK>(k, chunks, 256)) return k;
    try_pick<T, VEC, kMost, BACK>(k, chunks, kNormThreads);
    return k;
}

template <bool BACK>
NormPick pick_norm(int dtype, bool vec, uint32_t cols)
{
    if (dtype == DT_BF16) return vec ? pick_norm<uint16_t, 8, BACK>(cols) : pick_norm<uint16_t, 1, BACK>(cols);
    return vec ? pick_norm<float, 4, BACK>(cols) : pick_norm<float, 1, BACK>(cols);
}

constexpr int kBackBlocks = 2;   // blocks per SM of the backward pass, at most: each writes a share of dw and db

uint32_t groups_of(uint32_t tpr, uint32_t threads) { return tpr >= threads ? 1 : threads / tpr; }

}  // namespace

DT_TL_BINDER(bind_timeline_norm)

size_t norm_workspace(uint32_t cols, int device)
{
    // at least 32 threads a row, and at most 32 elements a thread
    uint32_t tpr = (cols + 31) / 32;
    tpr = tpr < 32 ? 32 : (tpr + 31) / 32 * 32;
    const uint64_t parts = (uint64_t)sm_count(device) * kBackBlocks * groups_of(tpr, kNormThreads);
    return (size_t)((parts > kLongSlices ? parts : kLongSlices) * 2 * cols * sizeof(float));
}

cudaError_t launch_norm(const NormParams &p0, int dtype, bool vec, int device, cudaStream_t s)
{
    NormParams p = p0;
    const NormPick k = pick_norm<false>(dtype, vec, p.cols);
    uint32_t threads = kLongThreads, groups = 1;
    NormFn fn = k.fn;
    if (fn) {
        p.tpr = k.tpr;
        groups = groups_of(k.tpr, 256);
        threads = groups * k.tpr;
    } else {
        fn = dtype == DT_BF16 ? norm_long_kernel<uint16_t> : norm_long_kernel<float>;
    }
    int resident = 0;
    cudaError_t e = resident_blocks(reinterpret_cast<const void *>(fn), (int)threads, device, &resident);
    if (e != cudaSuccess) return e;
    const uint64_t want = (p.rows + groups - 1) / groups;
    const unsigned grid = (unsigned)(want < (uint64_t)resident ? want : (uint64_t)resident);
    return launch_kernel(fn, dim3(grid), dim3(threads), 0, s, false, p);
}

cudaError_t launch_norm_backward(NormParams p, int dtype, bool vec, int device, cudaStream_t s)
{
    const NormPick k = pick_norm<true>(dtype, vec, p.cols);
    cudaError_t e = cudaSuccess;
    if (p.rows == 0) {
        p.parts = 0;
    } else if (k.fn) {
        p.tpr = k.tpr;
        const uint32_t groups = groups_of(k.tpr, kNormThreads), threads = groups * k.tpr;
        int resident = 0;
        e = resident_blocks(reinterpret_cast<const void *>(k.fn), (int)threads, device, &resident);
        if (e != cudaSuccess) return e;
        const uint64_t want = (p.rows + groups - 1) / groups, cap = (uint64_t)sm_count(device) * kBackBlocks;
        uint64_t grid = want < (uint64_t)resident ? want : (uint64_t)resident;
        if (grid > cap) grid = cap;
        p.parts = (uint32_t)(grid * groups < p.rows ? grid * groups : p.rows);
        e = launch_kernel(k.fn, dim3((unsigned)grid), dim3(threads), 0, s, false, p);
    } else {
        const bool bf16 = dtype == DT_BF16;
        if (p.partial) {
            p.parts = p.rows < kLongSlices ? (uint32_t)p.rows : kLongSlices;
            e = launch_kernel(bf16 ? norm_columns_long_kernel<uint16_t> : norm_columns_long_kernel<float>,
                              dim3((p.cols + kThreads - 1) / kThreads, p.parts), dim3(kThreads), 0, s, false, p);
            if (e != cudaSuccess) return e;
        }
        const NormFn fn = bf16 ? norm_backward_long_kernel<uint16_t> : norm_backward_long_kernel<float>;
        int resident = 0;
        e = resident_blocks(reinterpret_cast<const void *>(fn), kLongThreads, device, &resident);
        if (e != cudaSuccess) return e;
        const uint64_t grid = p.rows < (uint64_t)resident ? p.rows : (uint64_t)resident;
        e = launch_kernel(fn, dim3((unsigned)grid), dim3(kLongThreads), 0, s, false, p);
    }
    if (e != cudaSuccess || !p.partial) return e;
    return launch_kernel(norm_join_kernel, dim3((p.cols + kJoinCols - 1) / kJoinCols, 2),
                         dim3(kJoinCols * kJoinSlices), 0, s, false, p);
}

}  // namespace dt
