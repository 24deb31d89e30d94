// What stands between two blocks of a model whose tokens are split over P ranks:
// the norm of the block's output, its gate, the residual sum, and the norm before the
// next block, forward and backward, with the weights' gradients reduced over every
// rank's rows.
//
//   r1 = 1 / sqrt(mean o^2 + eps)   h = o r1   y = scale x + gate post h
//   r2 = 1 / sqrt(mean y^2 + eps)   n = y r2   z = n pre
//   q = dz pre     d = dy + r2 (q - n mean(q n))     dx = scale d
//   c = d gate post                 do = r1 (c - h mean(c h))
//   G = sum_rows d h    dpost = G gate    dgate = G post    dpre = sum_rows dz n
//
// Two weights' gradients come from one column sum, and both of a row's means from
// one reduction: with g = gate post and e = dy + r2 q, sum(c h) = sum(g h e) - r2
// mean(q n) sum(g h n), so that the three sums of a row cross its threads together.
//
// HBM bounds both directions (4 and 6 passes over the rows at 2 to 4 flops a byte), so
// every row is read once.  Resident blocks, whose groups of threads each have a ring of
// shared memory stages that bulk copies fill, walk over the rows; rows of any alignment
// are copied with the 16-byte blocks that their ends lie in.  A thread keeps its columns
// over all of its rows, and with them their weights and, backward, its shares of the
// column sums, which a second kernel adds in a fixed order.
//
// All sums are fp32, y enters the second norm before it is rounded, and results are
// rounded once, at the store.
#include <algorithm>

#include "dt_residual.h"

#include "dt_bounds.cuh"
#include "dt_device.cuh"
#include "dt_math.cuh"
#include "dt_rows.cuh"
#include "dt_timeline.cuh"

namespace dt {
namespace {

constexpr uint32_t kSmemBytes = 160 * 1024;   // rings, of the SM's 227 KB
constexpr uint32_t kMaxStages = 4;
constexpr uint32_t kStageTarget = 4096;
constexpr int kLongThreads = 512;             // rows too long for registers
constexpr int kJoinCols = 32;                 // columns and row slices of a block that adds the shares
constexpr int kJoinSlices = 16;

#define RESIDUAL_OK(buffer, a, n) DT_IN_EXTENT(p, kBoundsResidual, (buffer), (a), (n))

// N weights from element e on, or ones.
template <int N>
__device__ __forceinline__ void load_weights(const ResidualParams &p, const void *base, int buffer, uint32_t e, float (&v)[N])
{
    (void)buffer;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 1.0f;
    if (!base) return;
    if (p.weight_bf16) {
        const uint16_t *q = static_cast<const uint16_t *>(base) + e;
        if (!RESIDUAL_OK(buffer, q, 2 * N)) return;
        if (N == 8 && (reinterpret_cast<uintptr_t>(base) & 15) == 0) {
            const uint4 u = *reinterpret_cast<const uint4 *>(q);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = i & 1 ? bf16_hi(w[i / 2 % 4]) : bf16_lo(w[i / 2 % 4]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = bf16_to_f32(q[i]);
        }
    } else {
        const float *q = static_cast<const float *>(base) + e;
        if (!RESIDUAL_OK(buffer, q, 4 * N)) return;
        if (N % 4 == 0 && (reinterpret_cast<uintptr_t>(base) & 15) == 0) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) *reinterpret_cast<float4 *>(v + 4 * i) = *reinterpret_cast<const float4 *>(q + 4 * i);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = q[i];
        }
    }
}

// gate * post, and pre, of a thread's columns from e on.
template <typename C, int VEC>
__device__ __forceinline__ void weights(const ResidualParams &p, uint32_t e, typename C::V (&gp)[C::K], typename C::V (&pre)[C::K])
{
    float a[VEC], b[VEC], c[VEC];
    load_weights<VEC>(p, p.post, kResidualPost, e, a);
    load_weights<VEC>(p, p.gate, kResidualGate, e, b);
    load_weights<VEC>(p, p.pre, kResidualPre, e, c);
    if constexpr (VEC == 1) {
        gp[0] = a[0] * b[0];
        pre[0] = c[0];
    } else {
#pragma unroll
        for (int i = 0; i < C::K; ++i) {
            gp[i] = pair(a[2 * i] * b[2 * i], a[2 * i + 1] * b[2 * i + 1]);
            pre[i] = pair(c[2 * i], c[2 * i + 1]);
        }
    }
}

// A group's walk over the rows: chunk c of the call is up to p.chunk_rows rows of one
// rank; group number `part` has chunks part, part + parts, ...  Its first warp starts
// the copies.  Dynamic shared memory holds the groups' rings and their barriers.
template <typename T, bool BACK>
struct Ring {
    const ResidualParams &p;
    uint32_t base, bars;             // the group's stages and their barriers in shared memory
    unsigned char *mem;
    uint32_t s = 0, parity = 0;
    bool late = false;               // a wait ran out: wait no more, and keep to the barriers

    static constexpr uint32_t kArrays = BACK ? 4 : 2, kCopies = BACK ? 8 : 2;   // and two of rstd
    // The rows of chunk c: rank, first row there, how many.
    __device__ __forceinline__ void chunk(uint64_t c, int &r, uint64_t &row, uint32_t &n) const
    {
        uint64_t begin = 0;
        r = 0;
        while (r + 1 < p.P && c >= p.chunk_end[r]) begin = p.chunk_end[r++];
        row = (c - begin) * p.chunk_rows;
        const uint64_t rows = p.row_end[r] - (r ? p.row_end[r - 1] : 0);
        n = rows - row < p.chunk_rows ? (uint32_t)(rows - row) : p.chunk_rows;
    }
    // Copies the 16-byte blocks of one of its buffers that hold rows [row, row + n) of rank r; how many bytes.
    __device__ __forceinline__ uint32_t copy(uint32_t which, int r, uint64_t row, uint32_t n, uint32_t stage) const
    {
        if (which >= kArrays + (BACK ? 2 : 0) || (BACK && which == kDy && !p.has_dy)) return 0;
        const bool stat = BACK && which >= kArrays;
        const uint64_t row_bytes = stat ? 4 : p.cols * sizeof(T);
        const uint32_t dst = base + stage * p.stage_bytes + min(which, kArrays) * p.array_bytes +
                             (which == kArrays + 1 ? p.stat_bytes : 0);
        const void *from_base = stat ? p.rstd[which - kArrays][r] : p.src[which % kResidualSources][r];
        const uint64_t lo = reinterpret_cast<uint64_t>(from_base) + row * row_bytes, hi = lo + n * row_bytes;
        const uint64_t from = lo & ~15ull, to = (hi + 15) & ~15ull;
        if (!RESIDUAL_OK((stat ? kResidualRstd + (which - kArrays) * DT_MAX_RANKS : which * DT_MAX_RANKS) + r,
                         reinterpret_cast<const void *>(lo), hi - lo))
            return 0;
        bulk_load(dst, reinterpret_cast<const void *>(from), (uint32_t)(to - from), bars + 8 * stage);
        return (uint32_t)(to - from);
    }
    // A chunk's copies by a warp, a lane to a copy, for stages [first, first + stages) at once.
    __device__ __forceinline__ void load(uint64_t c, uint32_t first, uint32_t stages) const
    {
        static_assert(kCopies * kMaxStages <= 32, "a lane to a copy");
        const uint32_t lane = threadIdx.x & 31, k = lane / kCopies, which = lane % kCopies;
        c += (uint64_t)k * p.parts;
        const bool mine = k < stages && c < p.chunks;
        uint32_t bytes = 0;
        if (mine) {
            int r;
            uint64_t row;
            uint32_t n;
            chunk(c, r, row, n);
            bytes = copy(which, r, row, n, first + k);
        }
#pragma unroll
        for (uint32_t o = 1; o < kCopies; o *= 2) bytes += __shfl_xor_sync(0xFFFFFFFFu, bytes, o);
        if (mine && which == 0) mbar_expect_tx(bars + 8 * (first + k), bytes);
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
    __device__ __forceinline__ const T *row(uint32_t which, int r, uint64_t first) const
    {
        return at(which * p.array_bytes, static_cast<const T *>(p.src[which][r]) + first * p.cols);
    }
    __device__ __forceinline__ void next()
    {
        if (++s == p.stages) s = 0, parity ^= 1;
    }
    // Before the block goes on after a wait that ran out, a last, bounded wait
    // for what is still under way: each stage's last copy of group `part`.
    __device__ __forceinline__ void drain(bool first, uint64_t part) const
    {
        if (!late || !first || part >= p.chunks) return;
        const uint64_t n = (p.chunks - part + p.parts - 1) / p.parts;
        for (uint32_t k = 0; k < p.stages && k < n; ++k)
            mbar_wait_bounded(bars + 8 * k, (uint32_t)((n - k + p.stages - 1) / p.stages - 1) & 1, p.sink.timeout_ns);
    }
};

// The group's ring; the waits for the kernel before and of the one after.
template <typename T, bool BACK, int L>
__device__ __forceinline__ Ring<T, BACK> make_ring(const ResidualParams &p, unsigned char *smem, const Team<L> &m)
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
__device__ __forceinline__ void read_row(Chunk<T, VEC> (&c)[N], uint32_t cols, const T *row, uint32_t tpr, uint32_t t, bool there)
{
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint32_t e = (n * tpr + t) * VEC;
        if (there && e < cols) c[n].load(row + e);
        else c[n].zero();
    }
}

// Rows that are summed at a time, so that a barrier serves several: as many as leave
// room for a thread's values, its columns' weights and its sums among 128 registers.
template <typename T, int VEC, int N, int L, bool BACK>
__host__ __device__ constexpr int rows_at_once()
{
    constexpr int raw = N * (VEC == 1 ? 1 : 4), cols = N * VEC;
    constexpr int held = (BACK ? 4 : 2) * cols, row = 2 * raw + cols;
    constexpr int most = BACK && L < 16 ? L / 4 : 4;   // row_sum: a value to a lane at least
    constexpr int room = BACK ? 72 : 96;
    return most >= 4 && held + 4 * row <= room ? 4 : most >= 2 && held + 2 * row <= room ? 2 : 1;
}

__device__ __forceinline__ float rstd_of(float sum, float inv_cols, float eps) { return rsqrtf(fmaf(sum, inv_cols, eps)); }

template <typename T, int VEC, int N, int L>
__global__ void __launch_bounds__(kNormThreads, 1) residual_kernel(const __grid_constant__ ResidualParams p)
{
    constexpr int B = rows_at_once<T, VEC, N, L, false>();
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
    const V scale = C::all(p.scale);
    uint32_t phase = 0;
    V gp[N][K], pre[N][K];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint32_t e = (n * tpr + t) * VEC;
#pragma unroll
        for (int i = 0; i < K; ++i) gp[n][i] = pre[n][i] = C::all(0.0f);
        if (e < cols) weights<C, VEC>(p, e, gp[n], pre[n]);
    }
    if (team.first_warp()) ring.load(part, 0, p.stages);

    for (uint64_t c = part; c < p.chunks; c += p.parts) {
        int r;
        uint64_t row;
        uint32_t rows;
        ring.chunk(c, r, row, rows);
        const T *os = ring.row(kBranch, r, row) + team.team * cols, *xs = ring.row(kX, r, row) + team.team * cols;
        ring.wait();
        // this team's rows are the stage's k, k + S, ...
        for (uint32_t k = team.team; k - team.team < rows; k += B * S, os += B * S * cols, xs += B * S * cols) {
            // B rows at a time; the last ones of a stage may stand beside rows of zeros
            C o[B][N], x[B][N];
            float s[B];
#pragma unroll
            for (int j = 0; j < B; ++j) {
                read_row<T, VEC, N>(o[j], cols, os + j * S * cols, tpr, t, k + j * S < rows);
                read_row<T, VEC, N>(x[j], cols, xs + j * S * cols, tpr, t, k + j * S < rows);
                V sum = C::all(0.0f);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    V f[K];
                    o[j][n].get(f);
#pragma unroll
                    for (int i = 0; i < K; ++i) sum = fma(f[i], f[i], sum);
                }
                s[j] = both(sum);
            }
            row_sum<B>(s, red, phase, team);
            if (tpr <= 32) __syncwarp();
            // every thread has read its part of the stage's last rows
            if (k - team.team + B * S >= rows && team.first_warp() && c + (uint64_t)p.stages * p.parts < p.chunks)
                ring.load(c + (uint64_t)p.stages * p.parts, ring.s, 1);
            V y[B][N][K];
            float r1[B], r2[B];
#pragma unroll
            for (int j = 0; j < B; ++j) {
                r1[j] = rstd_of(s[j], inv, p.eps);
                const V scale1 = C::all(r1[j]);
                V sum = C::all(0.0f);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    V f[K], a[K];
                    o[j][n].get(f);
                    x[j][n].get(a);
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        y[j][n][i] = fma(mul(f[i], scale1), gp[n][i], mul(a[i], scale));
                        sum = fma(y[j][n][i], y[j][n][i], sum);
                    }
                }
                s[j] = both(sum);
            }
            row_sum<B>(s, red, phase, team);
#pragma unroll
            for (int j = 0; j < B; ++j) {
                if (k + j * S >= rows) continue;
                r2[j] = rstd_of(s[j], inv, p.eps);
                const V scale2 = C::all(r2[j]);
                const uint64_t at = row + k + j * S;
                T *to_y = static_cast<T *>(p.out[0][r]) + at * cols, *to_z = static_cast<T *>(p.out[1][r]) + at * cols;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint32_t e = (n * tpr + t) * VEC;
                    if (e >= cols) continue;
                    V z[K];
#pragma unroll
                    for (int i = 0; i < K; ++i) z[i] = mul(mul(y[j][n][i], scale2), pre[n][i]);
                    if (RESIDUAL_OK(kResidualOut + r, to_y + e, VEC * sizeof(T))) C::store(to_y + e, y[j][n]);
                    if (RESIDUAL_OK(kResidualOut + DT_MAX_RANKS + r, to_z + e, VEC * sizeof(T))) C::store(to_z + e, z);
                }
                if (t == 0) {
                    if (p.rstd[0][r] && RESIDUAL_OK(kResidualRstd + r, p.rstd[0][r] + at, 4)) p.rstd[0][r][at] = r1[j];
                    if (p.rstd[1][r] && RESIDUAL_OK(kResidualRstd + DT_MAX_RANKS + r, p.rstd[1][r] + at, 4)) p.rstd[1][r][at] = r2[j];
                }
            }
        }
        ring.next();
    }
    ring.drain(team.first(), part);
    DT_TL_END_BLOCK(DT_TL_RESIDUAL);
}

template <typename T, int VEC, int N, int L>
__global__ void __launch_bounds__(kNormThreads, 1) residual_backward_kernel(const __grid_constant__ ResidualParams p)
{
    constexpr int B = rows_at_once<T, VEC, N, L, true>();
    using C = Chunk<T, VEC>;
    using V = typename C::V;
    constexpr int K = C::K;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float red[2][4 * B][kNormThreads / 32];
    DT_TL_BEGIN();
    const Team<L> team(p.tpr);
    constexpr uint32_t S = Team<L>::kTeams;
    const uint32_t tpr = team.tpr, t = team.t, cols = p.cols;
    const uint64_t part = (uint64_t)team.group * gridDim.x + blockIdx.x;
    Ring<T, true> ring = make_ring<T, true>(p, smem, team);
    DT_TL_WAITED();
    const float inv = p.inv_cols;
    uint32_t phase = 0;
    V gp[N][K], pre[N][K], dh[N][K], dn[N][K];   // and the column sums of d h and dz n
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint32_t e = (n * tpr + t) * VEC;
#pragma unroll
        for (int i = 0; i < K; ++i) gp[n][i] = pre[n][i] = dh[n][i] = dn[n][i] = C::all(0.0f);
        if (e < cols) weights<C, VEC>(p, e, gp[n], pre[n]);
    }
    if (team.first_warp()) ring.load(part, 0, p.stages);

    for (uint64_t c = part; c < p.chunks; c += p.parts) {
        int r;
        uint64_t row;
        uint32_t rows;
        ring.chunk(c, r, row, rows);
        const T *src[kResidualSources];
#pragma unroll
        for (int a = 0; a < kResidualSources; ++a) src[a] = ring.row(a, r, row) + team.team * cols;
        const float *r1s = ring.at(4 * p.array_bytes, p.rstd[0][r] + row);
        const float *r2s = ring.at(4 * p.array_bytes + p.stat_bytes, p.rstd[1][r] + row);
        ring.wait();
        // this team's rows are the stage's k, k + S, ...
        for (uint32_t k = team.team; k - team.team < rows; k += B * S) {
            // B rows at a time; the last ones of a stage may stand beside rows of zeros.  Of
            // dz and dy only e = dy + rstd_pre q is kept, in fp32.
            C o[B][N], y[B][N];
            V e[B][N][K];
            float s[4 * B], r1[B], r2[B];
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const bool there = k + j * S < rows;
                r1[j] = there ? r1s[k + j * S] : 0.0f;
                r2[j] = there ? r2s[k + j * S] : 0.0f;
                read_row<T, VEC, N>(o[j], cols, src[kBranch] + j * S * cols, tpr, t, there);
                read_row<T, VEC, N>(y[j], cols, src[kY] + j * S * cols, tpr, t, there);
                C z[N], d[N];
                read_row<T, VEC, N>(z, cols, src[kDz] + j * S * cols, tpr, t, there);
                read_row<T, VEC, N>(d, cols, src[kDy] + j * S * cols, tpr, t, there && p.has_dy);
                // sums of q y, g e and g y, with g = gate post o: the other rstd factors come afterwards
                V qn = C::all(0.0f), he = qn, hn = qn;
                const V scale2 = C::all(r2[j]);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    V of[K], yf[K], zf[K], df[K];
                    o[j][n].get(of);
                    y[j][n].get(yf);
                    z[n].get(zf);
                    d[n].get(df);
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        const V q = mul(zf[i], pre[n][i]), g = mul(of[i], gp[n][i]);
                        e[j][n][i] = fma(q, scale2, df[i]);
                        qn = fma(q, yf[i], qn);
                        he = fma(g, e[j][n][i], he);
                        hn = fma(g, yf[i], hn);
                        dn[n][i] = fma(zf[i], mul(yf[i], scale2), dn[n][i]);
                    }
                }
                s[4 * j] = both(qn);
                s[4 * j + 1] = both(he);
                s[4 * j + 2] = both(hn);
                s[4 * j + 3] = 0.0f;
            }
            row_sum<4 * B>(s, red, phase, team);
            if (tpr <= 32) __syncwarp();
            // every thread has read its part of the stage's last rows
            if (k - team.team + B * S >= rows && team.first_warp() && c + (uint64_t)p.stages * p.parts < p.chunks)
                ring.load(c + (uint64_t)p.stages * p.parts, ring.s, 1);
#pragma unroll
            for (int j = 0; j < B; ++j) {
                if (k + j * S >= rows) continue;
                // d = e - y r2^2 mean(q n);  do = r1 c - o r1^2 mean(c h)
                const float m2 = s[4 * j] * r2[j] * inv;
                const float ch = r1[j] * fmaf(-m2 * r2[j] * r2[j], s[4 * j + 2], s[4 * j + 1]);
                const V back2 = C::all(-r2[j] * r2[j] * m2);
                const V scale1 = C::all(r1[j]), back1 = C::all(-r1[j] * (ch * inv)), scale = C::all(p.scale);
                const uint64_t at = row + k + j * S;
                T *to_x = static_cast<T *>(p.out[0][r]) + at * cols, *to_o = static_cast<T *>(p.out[1][r]) + at * cols;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint32_t c = (n * tpr + t) * VEC;
                    if (c >= cols) continue;
                    V of[K], yf[K], dx[K];
                    o[j][n].get(of);
                    y[j][n].get(yf);
#pragma unroll
                    for (int i = 0; i < K; ++i) {
                        const V d = fma(yf[i], back2, e[j][n][i]), h = mul(of[i], scale1);
                        dx[i] = mul(d, scale);
                        dh[n][i] = fma(d, h, dh[n][i]);
                        of[i] = fma(mul(d, gp[n][i]), scale1, mul(h, back1));
                    }
                    if (RESIDUAL_OK(kResidualOut + r, to_x + c, VEC * sizeof(T))) C::store(to_x + c, dx);
                    if (RESIDUAL_OK(kResidualOut + DT_MAX_RANKS + r, to_o + c, VEC * sizeof(T))) C::store(to_o + c, of);
                }
            }
#pragma unroll
            for (int a = 0; a < kResidualSources; ++a) src[a] += B * S * cols;
        }
        ring.next();
    }
    ring.drain(team.first(), part);
    if (p.partial) {
        // the teams of a warp add theirs, then the block its groups', in ascending
        // order, in the rings' place
#pragma unroll
        for (uint32_t o = 16; o >= (uint32_t)L; o >>= 1)
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < K; ++i) {
                    dh[n][i] = add(dh[n][i], from_lane(dh[n][i], o));
                    dn[n][i] = add(dn[n][i], from_lane(dn[n][i], o));
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
                    V *a = reinterpret_cast<V *>(mine + e) + i, *b = reinterpret_cast<V *>(mine + cols + e) + i;
                    if (groups > 1 || RESIDUAL_OK(kResidualWorkspace, a, sizeof(V))) *a = dh[n][i];
                    if (groups > 1 || RESIDUAL_OK(kResidualWorkspace, b, sizeof(V))) *b = dn[n][i];
                }
            }
        if (groups > 1) {
            __syncthreads();
#pragma unroll 4
            for (uint32_t e = threadIdx.x; e < 2 * cols; e += blockDim.x) {
                float v = all[e];
#pragma unroll 4
                for (uint32_t k = 1; k < groups; ++k) v += all[(size_t)k * 2 * cols + e];
                if (RESIDUAL_OK(kResidualWorkspace, out + e, 4)) out[e] = v;
            }
        }
    }
    DT_TL_END_BLOCK(DT_TL_RESIDUAL);
}

// Forward, few rows of whole vectors: a block to a row, whose threads load their vectors of
// it and their weights straight from memory, all at once (a decoding step of 4 rows of 4096
// bf16: by way of a ring 5.0 us, this 4.7).
template <typename T, int VEC, int N>
__global__ void __launch_bounds__(kNormThreads) residual_few_kernel(const __grid_constant__ ResidualParams p)
{
    using C = Chunk<T, VEC>;
    using V = typename C::V;
    constexpr int K = C::K;
    __shared__ float red[2][1][kNormThreads / 32];
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    const Team<32> team(p.tpr);
    int r = 0;
    uint64_t begin = 0;
    while (r + 1 < p.P && blockIdx.x >= p.row_end[r]) begin = p.row_end[r++];
    const uint64_t row = blockIdx.x - begin, first = row * p.cols;
    const T *os = static_cast<const T *>(p.src[kBranch][r]) + first, *xs = static_cast<const T *>(p.src[kX][r]) + first;
    C o[N], x[N];
    V gp[N][K], pre[N][K];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint32_t e = (n * team.tpr + team.t) * VEC;
        o[n].zero();
        x[n].zero();
        if (e < p.cols && RESIDUAL_OK(kBranch * DT_MAX_RANKS + r, os + e, 16)) o[n].load(os + e);
        if (e < p.cols && RESIDUAL_OK(kX * DT_MAX_RANKS + r, xs + e, 16)) x[n].load(xs + e);
#pragma unroll
        for (int i = 0; i < K; ++i) gp[n][i] = pre[n][i] = C::all(0.0f);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint32_t e = (n * team.tpr + team.t) * VEC;
        if (e < p.cols) weights<C, VEC>(p, e, gp[n], pre[n]);
    }
    uint32_t phase = 0;
    V sum = C::all(0.0f), y[N][K];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        o[n].get(y[n]);
#pragma unroll
        for (int i = 0; i < K; ++i) sum = fma(y[n][i], y[n][i], sum);
    }
    float s[1] = {both(sum)};
    row_sum<1>(s, red, phase, team);
    const float r1 = rstd_of(s[0], p.inv_cols, p.eps);
    sum = C::all(0.0f);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        V a[K];
        x[n].get(a);
#pragma unroll
        for (int i = 0; i < K; ++i) {
            y[n][i] = fma(mul(y[n][i], C::all(r1)), gp[n][i], mul(a[i], C::all(p.scale)));
            sum = fma(y[n][i], y[n][i], sum);
        }
    }
    s[0] = both(sum);
    row_sum<1>(s, red, phase, team);
    const float r2 = rstd_of(s[0], p.inv_cols, p.eps);
    T *to_y = static_cast<T *>(p.out[0][r]) + first, *to_z = static_cast<T *>(p.out[1][r]) + first;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint32_t e = (n * team.tpr + team.t) * VEC;
        if (e >= p.cols) continue;
        V z[K];
#pragma unroll
        for (int i = 0; i < K; ++i) z[i] = mul(mul(y[n][i], C::all(r2)), pre[n][i]);
        if (RESIDUAL_OK(kResidualOut + r, to_y + e, 16)) C::store(to_y + e, y[n]);
        if (RESIDUAL_OK(kResidualOut + DT_MAX_RANKS + r, to_z + e, 16)) C::store(to_z + e, z);
    }
    if (threadIdx.x == 0) {
        if (p.rstd[0][r] && RESIDUAL_OK(kResidualRstd + r, p.rstd[0][r] + row, 4)) p.rstd[0][r][row] = r1;
        if (p.rstd[1][r] && RESIDUAL_OK(kResidualRstd + DT_MAX_RANKS + r, p.rstd[1][r] + row, 4)) p.rstd[1][r][row] = r2;
    }
    DT_TL_END_BLOCK(DT_TL_RESIDUAL);
}

// The weights' gradients from the blocks' shares: of dpost and dgate (blockIdx.y 0) or
// dpre (1).  Thread (c, s) adds shares s, s + 16, ... of its column, then the 16 sums
// are added in a tree.
__global__ void __launch_bounds__(kJoinCols *kJoinSlices) residual_join_kernel(const __grid_constant__ ResidualParams p)
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
                o[j] = at < p.parts && RESIDUAL_OK(kResidualWorkspace, from, 4) ? *from : 0.0f;
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
    auto store = [&](void *out, int buffer, float f) {
        (void)buffer;
        if (!out) return;
        if (p.avg) f = avg_of(f, p.P, p.avg_scale, p.avg_pow2);
        if (p.weight_bf16) {
            uint16_t *to = static_cast<uint16_t *>(out) + col;
            if (RESIDUAL_OK(buffer, to, 2)) *to = f32_to_bf16(f);
        } else {
            float *to = static_cast<float *>(out) + col;
            if (RESIDUAL_OK(buffer, to, 4)) *to = f;
        }
    };
    if (threadIdx.x % kJoinSlices == 0 && col < p.cols) {
        if (blockIdx.y) {
            store(p.dpre, kResidualDpre, v);
        } else {
            float gate[1], post[1];
            load_weights<1>(p, p.gate, kResidualGate, col, gate);
            load_weights<1>(p, p.post, kResidualPost, col, post);
            store(p.dpost, kResidualDpost, v * gate[0]);
            store(p.dgate, kResidualDgate, v * post[0]);
        }
    }
    DT_TL_END_BLOCK(DT_TL_RESIDUAL);
}

// ---- rows too long for registers ------------------------------------------------
// A block to a row, which it reads from memory (or L2) again for each of its steps.

// The block's sums of N values a thread; every thread gets them.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (&red)[kLongThreads / 32][N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
    __syncthreads();   // the last sums have been read
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[threadIdx.x >> 5][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = red[0][i];
        for (int w = 1; w < kLongThreads / 32; ++w) v[i] += red[w][i];
    }
}

__device__ __forceinline__ int find_rank(const ResidualParams &p, uint64_t row, uint64_t &local)
{
    int r = 0;
    uint64_t begin = 0;
    while (r + 1 < p.P && row >= p.row_end[r]) begin = p.row_end[r++];
    local = row - begin;
    return r;
}

__device__ __forceinline__ float weight(const ResidualParams &p, const void *base, int buffer, uint32_t e)
{
    float v[1];
    load_weights<1>(p, base, buffer, e, v);
    return v[0];
}

template <typename T>
__device__ __forceinline__ float element(const ResidualParams &p, int which, int r, uint64_t at)
{
    const T *from = static_cast<const T *>(p.src[which][r]) + at;
    return RESIDUAL_OK(which * DT_MAX_RANKS + r, from, sizeof(T)) ? to_f32(*from) : 0.0f;
}

template <typename T>
__device__ __forceinline__ void put(const ResidualParams &p, int which, int r, uint64_t at, float v)
{
    T *to = static_cast<T *>(p.out[which][r]) + at;
    if (RESIDUAL_OK(kResidualOut + which * DT_MAX_RANKS + r, to, sizeof(T))) from_f32(v, to);
}

template <typename T>
__global__ void __launch_bounds__(kLongThreads) residual_long_kernel(const __grid_constant__ ResidualParams p)
{
    __shared__ float red[kLongThreads / 32][1];
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    for (uint64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        uint64_t local;
        const int r = find_rank(p, row, local);
        const uint64_t first = local * p.cols;
        float s[1] = {0.0f};
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            const float o = element<T>(p, kBranch, r, first + e);
            s[0] = fmaf(o, o, s[0]);
        }
        block_sum(s, red);
        const float r1 = rstd_of(s[0], p.inv_cols, p.eps);
        auto sum_at = [&](uint32_t e) {
            const float g = weight(p, p.post, kResidualPost, e) * weight(p, p.gate, kResidualGate, e);
            return fmaf(element<T>(p, kBranch, r, first + e) * r1, g, element<T>(p, kX, r, first + e) * p.scale);
        };
        s[0] = 0.0f;
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            const float y = sum_at(e);
            s[0] = fmaf(y, y, s[0]);
        }
        block_sum(s, red);
        const float r2 = rstd_of(s[0], p.inv_cols, p.eps);
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            const float y = sum_at(e);
            put<T>(p, 0, r, first + e, y);
            put<T>(p, 1, r, first + e, y * r2 * weight(p, p.pre, kResidualPre, e));
        }
        if (threadIdx.x == 0) {
            if (p.rstd[0][r] && RESIDUAL_OK(kResidualRstd + r, p.rstd[0][r] + local, 4)) p.rstd[0][r][local] = r1;
            if (p.rstd[1][r] && RESIDUAL_OK(kResidualRstd + DT_MAX_RANKS + r, p.rstd[1][r] + local, 4)) p.rstd[1][r][local] = r2;
        }
    }
    DT_TL_END_BLOCK(DT_TL_RESIDUAL);
}

// The block's shares of the column sums stay in memory, where a thread adds to its
// own columns row after row.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) residual_backward_long_kernel(const __grid_constant__ ResidualParams p)
{
    __shared__ float red[kLongThreads / 32][3];
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    float *share = p.partial ? p.partial + (uint64_t)blockIdx.x * 2 * p.cols : nullptr;
    if (share)
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            if (RESIDUAL_OK(kResidualWorkspace, share + e, 4)) share[e] = 0.0f;
            if (RESIDUAL_OK(kResidualWorkspace, share + p.cols + e, 4)) share[p.cols + e] = 0.0f;
        }
    for (uint64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        uint64_t local;
        const int r = find_rank(p, row, local);
        const uint64_t first = local * p.cols;
        const float r1 = RESIDUAL_OK(kResidualRstd + r, p.rstd[0][r] + local, 4) ? p.rstd[0][r][local] : 0.0f;
        const float r2 = RESIDUAL_OK(kResidualRstd + DT_MAX_RANKS + r, p.rstd[1][r] + local, 4) ? p.rstd[1][r][local] : 0.0f;
        auto gp = [&](uint32_t e) { return weight(p, p.post, kResidualPost, e) * weight(p, p.gate, kResidualGate, e); };
        float s[3] = {0.0f, 0.0f, 0.0f};
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            const uint64_t at = first + e;
            const float q = element<T>(p, kDz, r, at) * weight(p, p.pre, kResidualPre, e), y = element<T>(p, kY, r, at);
            const float g = element<T>(p, kBranch, r, at) * gp(e), d = p.has_dy ? element<T>(p, kDy, r, at) : 0.0f;
            s[0] = fmaf(q, y, s[0]);
            s[1] = fmaf(g, fmaf(q, r2, d), s[1]);
            s[2] = fmaf(g, y, s[2]);
        }
        block_sum(s, red);
        const float m2 = s[0] * r2 * p.inv_cols;
        const float m1 = r1 * fmaf(-m2 * r2 * r2, s[2], s[1]) * p.inv_cols;
        for (uint32_t e = threadIdx.x; e < p.cols; e += kLongThreads) {
            const uint64_t at = first + e;
            const float z = element<T>(p, kDz, r, at), y = element<T>(p, kY, r, at), o = element<T>(p, kBranch, r, at);
            const float d = (p.has_dy ? element<T>(p, kDy, r, at) : 0.0f) +
                            fmaf(z * weight(p, p.pre, kResidualPre, e), r2, y * (-r2 * r2 * m2));
            put<T>(p, 0, r, at, d * p.scale);
            put<T>(p, 1, r, at, fmaf(d * gp(e), r1, o * (-r1 * r1 * m1)));
            if (share && RESIDUAL_OK(kResidualWorkspace, share + e, 4)) share[e] = fmaf(d, o * r1, share[e]);
            if (share && RESIDUAL_OK(kResidualWorkspace, share + p.cols + e, 4))
                share[p.cols + e] = fmaf(z, y * r2, share[p.cols + e]);
        }
    }
    DT_TL_END_BLOCK(DT_TL_RESIDUAL);
}

using ResidualFn = void (*)(ResidualParams);

// The kernel for rows of `cols` elements, the threads that share a row and the rows
// that a group sums at a time.
struct Pick {
    ResidualFn fn = nullptr;
    uint32_t tpr = 0, threads = 0, rows = 0;
};

template <typename T, int VEC, int N, int L, bool BACK>
void try_pick(Pick &k, uint32_t vecs, uint32_t most)
{
    const uint32_t tpr = L < 32 ? L : ((vecs + N - 1) / N + 31) / 32 * 32;
    if (k.fn || tpr > most || vecs > tpr * N) return;
    if constexpr (BACK) k.fn = residual_backward_kernel<T, VEC, N, L>;
    else k.fn = residual_kernel<T, VEC, N, L>;
    k.tpr = tpr;
    k.threads = L < 32 ? 32 : tpr;
    k.rows = rows_at_once<T, VEC, N, L, BACK>() * (32 / L);
}

template <typename T, int VEC, bool BACK>
Pick pick(uint32_t cols)
{
    Pick k;
    const uint32_t vecs = (cols + VEC - 1) / VEC;
    constexpr int N = 8 / VEC;   // eight columns a thread, 16 where they are not enough
    try_pick<T, VEC, N, 8, BACK>(k, vecs, 32);
    try_pick<T, VEC, N, 16, BACK>(k, vecs, 32);
    try_pick<T, VEC, N, 32, BACK>(k, vecs, kNormThreads);
    try_pick<T, VEC, 2 * N, 32, BACK>(k, vecs, kNormThreads);
    return k;
}

template <bool BACK>
Pick pick(int dtype, bool vec, uint32_t cols)
{
    if (dtype == DT_BF16) return vec ? pick<uint16_t, 8, BACK>(cols) : pick<uint16_t, 1, BACK>(cols);
    return vec ? pick<float, 4, BACK>(cols) : pick<float, 1, BACK>(cols);
}

// The kernel for few rows of whole vectors, and the threads of a row.
template <typename T, int VEC>
Pick pick_few(uint32_t cols)
{
    Pick k;
    const uint32_t vecs = (cols + VEC - 1) / VEC;
    if (vecs <= kNormThreads) {
        k.fn = residual_few_kernel<T, VEC, 1>;
        k.tpr = (vecs + 31) / 32 * 32;
    } else if (vecs <= 2 * kNormThreads) {
        k.fn = residual_few_kernel<T, VEC, 2>;
        k.tpr = ((vecs + 1) / 2 + 31) / 32 * 32;
    }
    return k;
}

// The grid, the groups and the rings of a call.
cudaError_t launch_rows(const Pick &k, ResidualParams &p, int dtype, bool vec, bool back, int device, cudaStream_t s)
{
    const uint64_t row_bytes = (uint64_t)p.cols * (dtype == DT_BF16 ? 2 : 4), sms = (uint64_t)sm_count(device);
    p.tpr = k.tpr;
    uint64_t groups = kNormThreads / k.threads;
    if (k.threads > 32) groups = std::min<uint64_t>(groups, 15);   // named barriers
    // rows of a stage: those summed at once, and more where they are short, but not so
    // many that groups go without
    uint64_t per = std::max<uint64_t>(kStageTarget / std::max<uint64_t>(row_bytes, 16), k.rows);
    per = std::max<uint64_t>(1, std::min(per, p.rows / (groups * sms)));
    const uint64_t arrays = back ? 4 : 2;
    auto stage = [&] {
        // rows at other offsets are copied with up to 15 bytes at either end
        p.array_bytes = (uint32_t)((per * row_bytes + (vec ? 0 : 32) + 127) / 128 * 128);
        p.stat_bytes = back ? (uint32_t)((per * 4 + 32 + 63) / 64 * 64) : 0;
        p.stage_bytes = (uint32_t)(arrays * p.array_bytes + 2 * p.stat_bytes);
    };
    stage();
    while (per > 1 && groups * p.stage_bytes * 2 > kSmemBytes) per = (per + 1) / 2, stage();   // two stages at least
    p.chunk_rows = (uint32_t)per;
    p.chunks = 0;
    for (int r = 0; r < p.P; ++r)
        p.chunk_end[r] = p.chunks += (p.row_end[r] - (r ? p.row_end[r - 1] : 0) + per - 1) / per;
    const uint64_t grid = std::max<uint64_t>(1, std::min(sms, p.chunks));
    groups = std::max<uint64_t>(1, std::min(groups, (p.chunks + grid - 1) / grid));
    while (groups > 1 && groups * p.stage_bytes > kSmemBytes) --groups;
    p.parts = (uint32_t)(grid * groups);
    const uint64_t depth = (p.chunks + p.parts - 1) / p.parts;
    p.stages = (uint32_t)std::max<uint64_t>(1, std::min({(uint64_t)kMaxStages, kSmemBytes / (groups * p.stage_bytes), depth}));
    const size_t smem = std::max<size_t>(groups * p.stages * (p.stage_bytes + 8), back ? groups * 2 * (size_t)p.cols * sizeof(float) : 0);
    // A kernel may have 48 KB without asking, its static part (up to 2 KB of these) included.
    if (smem > 45 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(k.fn),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
        if (e != cudaSuccess) return e;
    }
    const cudaError_t e = launch_kernel(k.fn, dim3((unsigned)grid), dim3((unsigned)(groups * k.threads)), smem, s, false, p);
    p.parts = (uint32_t)grid;   // shares, to the join
    return e;
}

// Blocks that share the column sums where rows are too long for registers: one an SM,
// as long as their shares take at most 64 MB.
uint64_t long_blocks(uint32_t cols, int device)
{
    return std::max<uint64_t>(8, std::min<uint64_t>((uint64_t)sm_count(device), ((uint64_t)64 << 20) / (8ull * cols)));
}

}  // namespace

DT_TL_BINDER(bind_timeline_residual)

size_t residual_workspace(uint32_t cols, int device)
{
    const uint64_t blocks = std::max<uint64_t>(cols <= 16 * kNormThreads ? (uint64_t)sm_count(device) : 0, long_blocks(cols, device));
    return (size_t)blocks * 2 * cols * sizeof(float);
}

cudaError_t launch_residual(ResidualParams p, int dtype, bool vec, int device, cudaStream_t s)
{
    if (vec && p.rows <= 2 * (uint64_t)sm_count(device)) {
        const Pick few = dtype == DT_BF16 ? pick_few<uint16_t, 8>(p.cols) : pick_few<float, 4>(p.cols);
        p.tpr = few.tpr;
        if (few.fn) return launch_kernel(few.fn, dim3((unsigned)p.rows), dim3(few.tpr), 0, s, false, p);
    }
    const Pick k = pick<false>(dtype, vec, p.cols);
    if (k.fn) return launch_rows(k, p, dtype, vec, false, device, s);
    const uint64_t grid = std::min<uint64_t>(p.rows, (uint64_t)sm_count(device) * 4);
    return launch_kernel(dtype == DT_BF16 ? residual_long_kernel<uint16_t> : residual_long_kernel<float>, dim3((unsigned)grid),
                         dim3(kLongThreads), 0, s, false, p);
}

cudaError_t launch_residual_backward(ResidualParams p, int dtype, bool vec, int device, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    const Pick k = pick<true>(dtype, vec, p.cols);
    if (p.rows == 0) {
        p.parts = 0;
    } else if (k.fn) {
        e = launch_rows(k, p, dtype, vec, true, device, s);
    } else {
        p.parts = (uint32_t)std::min<uint64_t>(p.rows, long_blocks(p.cols, device));
        e = launch_kernel(dtype == DT_BF16 ? residual_backward_long_kernel<uint16_t> : residual_backward_long_kernel<float>,
                          dim3(p.parts), dim3(kLongThreads), 0, s, false, p);
    }
    if (e != cudaSuccess || !p.partial) return e;
    return launch_kernel(residual_join_kernel, dim3((p.cols + kJoinCols - 1) / kJoinCols, 2), dim3(kJoinCols * kJoinSlices), 0,
                         s, false, p);
}

}  // namespace dt
