// The linear layers over the ranks where few outputs or few tokens leave a tcgen05 tile's
// way through shared and tensor memory longer than its products: products by mma.sync,
// with operands read in place at any alignment, in one launch.
//
// linear_few_kernel    forward, up to 16 tokens: the weights' way from memory bounds it
// linear_small_kernel  any product and its gradients while a call is bound by launches and
//                      round trips to memory: nothing is laid out again before, no sums are
//                      joined after, and the gradient before the activation and the bias'
//                      gradient are made on the way
#include <algorithm>

#include "dt_linear.cuh"

#include "dt_bounds.cuh"
#include "dt_device.cuh"
#include "dt_math.cuh"
#include "dt_tc.cuh"
#include "dt_timeline.cuh"

namespace dt {
namespace {

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A float of another CTA of the cluster's shared memory.
__device__ __forceinline__ float cluster_load(const float *here, uint32_t rank)
{
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(smem_addr(here)), "r"(rank)
                 : "memory");
    return v;
}

// ---- few tokens --------------------------------------------------------------

// Forward products of up to 16 tokens, which the weights' way from memory bounds: 16
// rows of W to a group of warps that split the inner axis, with the weights straight
// from memory into the registers of mma.sync.m16n8k16 as its A, the tokens as its eight
// or sixteen columns.  (A tile of tcgen05 would be 128 rows of tokens, nearly all
// empty, and its way through shared and tensor memory is longer than the whole of a
// small call.)  A lane takes eight consecutive elements of a row, in one load, as its
// elements of two products: which of the inner axis' elements stand together in a
// product is free as long as both operands agree.  The warps' sums are added in shared
// memory, then those of the C CTAs of a cluster, which split the inner axis where there
// are few rows, in a fixed order.
constexpr uint32_t kFewRows = 16, kFewWarps = kThreads / 32;
// Of the inner axis, to a step of a warp: what its loads in flight leave registers for.
__host__ __device__ constexpr uint32_t few_depth(bool vec) { return vec ? 128 : 64; }

// Elements [k, k + 8) of a row of `len`; NULL: zeros.
template <bool VEC>
__device__ __forceinline__ void few_load(const LinearFew &p, const uint16_t *row, uint32_t k, uint32_t len, int buffer,
                                         Eight<VEC> &v)
{
    (void)p, (void)buffer;
    const uint32_t n = row && k < len ? min(len - k, 8u) : 0;
    v.load(row + k, n && LINEAR_OK(buffer, row + k, 2 * n) ? n : 0);
}

template <int KIND, int NT, bool VEC, int C>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kThreads) linear_few_kernel(const __grid_constant__ LinearFew p)
{
    __shared__ float sums[kFewWarps][NT * 8][kFewRows + 1];
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint32_t groups = kFewWarps / p.k_warps, group = warp / p.k_warps;
    const uint32_t part = C > 1 ? cluster_rank() : 0, block = blockIdx.x / C;
    // the block's rows of W: of one rank's features, or of the columns of a token
    uint32_t r = 0, begin = 0;
    if (KIND == kGather)
        while ((int)r + 1 < p.P && block >= p.block_end[r]) begin = p.block_end[r++];
    const uint32_t first = (block - begin) * groups * kFewRows, rows = KIND == kGather ? p.f_len[r] : p.dim;
    const uint32_t row = first + group * kFewRows + g;   // this lane's rows: this and the eighth after it
    // the tokens that this lane loads, and their rank
    const uint16_t *token[NT];
    int of[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const uint32_t t = n * 8 + g;
        token[n] = nullptr;
        of[n] = 0;
        if (KIND == kGather && t < p.tokens) {
            uint32_t at = 0;
            while (of[n] + 1 < p.P && t >= p.row_end[of[n]]) at = p.row_end[of[n]++];
            token[n] = p.x[of[n]] + (uint64_t)(t - at) * p.dim;
        }
    }
    float c[NT][4] = {};
    const uint32_t step = p.k_warps * C, mine = part * p.k_warps + warp % p.k_warps;
    constexpr uint32_t kDepth = few_depth(VEC), kParts = kDepth / 32;
    // steps of the inner axis, numbered through the ranks' pieces where it is features
    uint32_t i = mine;
    for (uint32_t f = KIND == kGather ? r : 0; f < (KIND == kGather ? r + 1 : (uint32_t)p.P); ++f) {
        const uint32_t len = KIND == kGather ? p.dim : p.f_len[f], steps = (len + kDepth - 1) / kDepth;
        const uint16_t *w0 = row < rows ? p.w[f] + (uint64_t)row * len : nullptr;
        const uint16_t *w1 = row + 8 < rows ? p.w[f] + (uint64_t)(row + 8) * len : nullptr;
        if (KIND == kReduce) {
#pragma unroll
            for (int n = 0; n < NT; ++n) token[n] = n * 8 + g < p.tokens ? p.x[f] + (uint64_t)(n * 8 + g) * len : nullptr;
        }
        for (; i < steps; i += step) {
            // a step's loads all go out before its products
            Eight<VEC> v0[kParts], v1[kParts], vb[NT][kParts];
#pragma unroll
            for (uint32_t j = 0; j < kParts; ++j) {
                const uint32_t k = i * kDepth + j * 32 + q * 8;
                few_load<VEC>(p, w0, k, len, kLinearW + f, v0[j]);
                few_load<VEC>(p, w1, k, len, kLinearW + f, v1[j]);
            }
#pragma unroll
            for (uint32_t j = 0; j < kParts; ++j)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    few_load<VEC>(p, token[n], i * kDepth + j * 32 + q * 8, len, kLinearX + (KIND == kGather ? of[n] : (int)f),
                                  vb[n][j]);
#pragma unroll
            for (uint32_t j = 0; j < kParts; ++j) {
                uint32_t a0[4], a1[4], b[NT][4];
                v0[j].get(a0);
                v1[j].get(a1);
#pragma unroll
                for (int n = 0; n < NT; ++n) vb[n][j].get(b[n]);
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {
                    const uint32_t a[4] = {a0[2 * h], a1[2 * h], a0[2 * h + 1], a1[2 * h + 1]};
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_16x8x16(c[n], a, b[n][2 * h], b[n][2 * h + 1]);
                }
            }
        }
        i -= steps;
    }
    // a lane holds rows g and g + 8 of tokens 2 q and 2 q + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        sums[warp][n * 8 + 2 * q][g] = c[n][0];
        sums[warp][n * 8 + 2 * q + 1][g] = c[n][1];
        sums[warp][n * 8 + 2 * q][g + 8] = c[n][2];
        sums[warp][n * 8 + 2 * q + 1][g + 8] = c[n][3];
    }
    __syncthreads();
    if (C > 1 && p.k_warps > 1) {   // the warps' sums into the first of each group
        for (uint32_t o = threadIdx.x; o < groups * p.tokens * kFewRows; o += kThreads) {
            const uint32_t at = o % kFewRows, t = o / kFewRows % p.tokens, w = o / kFewRows / p.tokens * p.k_warps;
            float v = sums[w][t][at];
            for (uint32_t k = 1; k < p.k_warps; ++k) v += sums[w + k][t][at];
            sums[w][t][at] = v;
        }
    }
    __syncwarp();
    if (C > 1) cluster_sync();
    for (uint32_t o = part * kThreads + threadIdx.x; o < groups * p.tokens * kFewRows; o += kThreads * C) {
        const uint32_t at = o % kFewRows, t = o / kFewRows % p.tokens, w = o / kFewRows / p.tokens, f = first + w * kFewRows + at;
        if (f >= rows) continue;
        float v[2] = {0.0f, 0.0f};
        if (C > 1) {
            for (uint32_t k = 0; k < C; ++k) v[0] += cluster_load(&sums[w * p.k_warps][t][at], k);
        } else {
            for (uint32_t k = 0; k < p.k_warps; ++k) v[0] += sums[w * p.k_warps + k][t][at];
        }
        if (KIND == kGather) {
            const uint64_t to = (uint64_t)t * rows + f;
            if (p.biased && LINEAR_OK(kLinearBias + r, p.bias[r] + f, 2)) v[0] += bf16_to_f32(p.bias[r][f]);
            if (p.keep && LINEAR_OK(kLinearPre + r, p.pre[r] + to, 2)) p.pre[r][to] = f32_to_bf16(v[0]);
            activate(v, p.act);
            if (LINEAR_OK(kLinearY + r, p.out[r] + to, 2)) p.out[r][to] = f32_to_bf16(v[0]);
        } else {
            uint32_t rank = 0, begin_row = 0;
            while ((int)rank + 1 < p.P && t >= p.row_end[rank]) begin_row = p.row_end[rank++];
            const uint64_t to = (uint64_t)(t - begin_row) * p.dim + f;
            if (p.biased && LINEAR_OK(kLinearBias, p.bias[0] + f, 2)) v[0] += bf16_to_f32(p.bias[0][f]);
            if (p.residuals && LINEAR_OK(kLinearResidual + rank, p.residual[rank] + to, 2))
                v[0] += bf16_to_f32(p.residual[rank][to]);
            if (LINEAR_OK(kLinearY + rank, p.out[rank] + to, 2)) p.out[rank][to] = f32_to_bf16(v[0]);
        }
    }
    __syncwarp();
    if (C > 1) cluster_sync();   // no CTA leaves while another reads its sums
    DT_TL_END_BLOCK(DT_TL_LINEAR);
}

// ---- small products ------------------------------------------------------------

// A tile of 64 x 64 outputs to four warps of 32 x 32 each; of the inner axis 64 at a time,
// 16 KB of both operands from memory to registers, where rows at any element are put right
// and a gradient is taken before its activation, and from there to shared memory, while the
// 64 before are multiplied.  An operand lies there as it does in memory, so that one whose
// rows run along the inner axis is read with ldmatrix' transposition.  A step takes a round
// trip to memory: where there are few tiles the CTAs of a cluster share the inner axis, and
// add their sums from one another's shared memory in rank order.  Tokens are numbered
// through the ranks, and each row of their matrix is looked up.  The gradient before an
// activation is two bf16 operands, its rounding and what that left, so that results of few
// tokens, over which its rounding would not average out, are as near as their own rounding
// leaves them (1 token of 424 to 8 x 192, silu: 2.6e-3 off by root mean square, so 2.0e-3;
// 7.1 -> 8.7 us).
constexpr uint32_t kSmallThreads = 128;
constexpr uint32_t kSumPitch = kSmallTile + 4;     // of the sums, in floats
constexpr uint32_t kSmallVecs = kSmallTile * kSmallTile / 8 / kSmallThreads;
using SmallOperand = uint16_t[kSmallTile * kSmallTile];

template <int KIND>
union SmallSmem {
    SmallOperand operand[2][KIND == kGatherBack ? 3 : 2];   // [step][A, B, what A's rounding left]
    float sum[kSmallTile][kSumPitch];
};

// Eight elements of an operand's row, from column `col` on (a multiple of eight): written a
// row to eight threads and read eight rows at a time without bank conflicts.
template <class T>
__device__ __forceinline__ T *operand_at(T *operand, uint32_t row, uint32_t col)
{
    return operand + row * kSmallTile + ((col >> 3 ^ (row & 7)) << 3);
}

// Row `row` of a matrix (of the piece `piece`), NULL past its last; its width and buffer.
template <class R, int MATRIX>
__device__ __forceinline__ const uint16_t *matrix_row(const LinearSmall &p, uint32_t piece, uint32_t row, uint32_t &width,
                                                      int &buffer)
{
    if (MATRIX == kTok) {
        width = p.dim;
        if (row >= p.tokens) return nullptr;
        uint32_t r = 0, begin = 0;
        while ((int)r + 1 < p.P && row >= p.row_end[r]) begin = p.row_end[r++];
        buffer = (R::kind == kGather || R::kind == kGatherBack ? kLinearX : kLinearDy) + r;
        return p.tok[r] + (uint64_t)(row - begin) * p.dim;
    }
    if (MATRIX == kFeat) {
        width = p.f_len[piece];
        buffer = (R::kind == kGatherBack ? kLinearDy : kLinearX) + piece;
        return row < p.tokens ? p.feat[piece] + (uint64_t)row * width : nullptr;
    }
    width = R::w_by_feature ? p.dim : p.f_len[piece];
    buffer = kLinearW + piece;
    return row < (R::w_by_feature ? p.f_len[piece] : p.dim) ? p.weight[piece] + (uint64_t)row * width : nullptr;
}

// A thread's vectors of an operand's 64 x 64, step after step along the inner axis: four
// rows, eight elements of each.  Rows are looked up where a piece of the inner axis begins
// (the tokens' where they are the inner axis: at each step), and followed from there.
template <class R, int MATRIX, bool MN, bool VEC>
struct Source {
    static constexpr bool kSlope = R::kind == kGatherBack && MATRIX == kFeat;
    const uint16_t *row[kSmallVecs];   // at this thread's columns; NULL: past the last row
    uint32_t n;                        // elements of them that are there
    uint32_t width, col, first;        // of the matrix; this thread's columns and first row
    int64_t z_off;                     // bytes from an element to what act'(.) is taken of
    int buffer[kSmallVecs];            // bounds-checked builds
    Eight<VEC> v[kSmallVecs], u[kSlope ? kSmallVecs : 1];   // on their way, and what act'(.) is taken of

    __device__ __forceinline__ void begin(const LinearSmall &p, const Place (&at)[3])
    {
        const Place &t = at[kTokens], &d = at[kDim], &f = at[kFeatures];
        const bool by_d = MATRIX == kTok || (MATRIX == kW && R::w_by_feature);   // rows are dim long
        first = (MATRIX != kW ? t.all : R::w_by_feature ? f.at : d.at) + threadIdx.x / 8;
        col = (by_d ? d.at : f.at) + threadIdx.x % 8 * 8;
        rows(p, f.piece);
        n = col < width ? min(width - col, 8u) : 0;
        if (kSlope)
            z_off = reinterpret_cast<intptr_t>(p.z[f.piece]) - reinterpret_cast<intptr_t>(p.feat[f.piece]);
    }
    __device__ __forceinline__ void rows(const LinearSmall &p, uint32_t piece)
    {
#pragma unroll
        for (uint32_t i = 0; i < kSmallVecs; ++i) {
            const uint16_t *from = matrix_row<R, MATRIX>(p, piece, first + i * (kSmallThreads / 8), width, buffer[i]);
            row[i] = from ? from + col : nullptr;
        }
    }
    // The next 64 of the same piece.
    __device__ __forceinline__ void next(const LinearSmall &p, const Place (&at)[3])
    {
        if (!MN) {
            col += kSmallTile;
            n = col < width ? min(width - col, 8u) : 0;
#pragma unroll
            for (uint32_t i = 0; i < kSmallVecs; ++i)
                if (row[i]) row[i] += kSmallTile;
        } else {
            first += kSmallTile;
            if (MATRIX == kTok) {
                rows(p, 0);
                return;
            }
            const Place &f = at[kFeatures];
            const uint32_t have = MATRIX == kFeat ? p.tokens : R::w_by_feature ? p.f_len[f.piece] : p.dim;
#pragma unroll
            for (uint32_t i = 0; i < kSmallVecs; ++i)
                row[i] = first + i * (kSmallThreads / 8) < have ? row[i] + (uint64_t)kSmallTile * width : nullptr;
        }
    }
    // A step's vectors: on their way ...
    __device__ __forceinline__ void load(const LinearSmall &p, uint32_t piece)
    {
        (void)p, (void)piece;
#pragma unroll
        for (uint32_t i = 0; i < kSmallVecs; ++i)
            v[i].load(row[i], row[i] && n && LINEAR_OK(buffer[i], row[i], 2 * n) ? n : 0);
        if (!kSlope || p.act == DT_ACT_NONE) return;
#pragma unroll
        for (uint32_t i = 0; i < kSmallVecs; ++i) {
            const uint16_t *z = reinterpret_cast<const uint16_t *>(reinterpret_cast<intptr_t>(row[i]) + z_off);
            u[kSlope ? i : 0].load(z, row[i] && n && LINEAR_OK(kLinearPre + piece, z, 2 * n) ? n : 0);
        }
    }
    // ... and to shared memory; rest: what rounding left of the gradient before the activation.
    __device__ __forceinline__ void put(const LinearSmall &p, uint16_t *to, uint16_t *rest) const
    {
        (void)p, (void)rest;
        const uint32_t at_row = threadIdx.x / 8, at_col = threadIdx.x % 8 * 8;
#pragma unroll
        for (uint32_t i = 0; i < kSmallVecs; ++i) {
            uint32_t w[4];
            v[i].get(w);
            if (kSlope && p.act != DT_ACT_NONE) {
                uint32_t x[4];
                float g[8], f[8];
                u[kSlope ? i : 0].get(x);
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    g[j] = j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
                    f[j] = j & 1 ? bf16_hi(x[j / 2]) : bf16_lo(x[j / 2]);
                }
                times_slope(g, f, p.act);   // what is not there: 0 times the derivative at 0
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) {
                    w[j] = pack_bf16x2(g[2 * j], g[2 * j + 1]);
                    const float lo = bf16_lo(w[j]), hi = bf16_hi(w[j]);   // (of an infinity or NaN nothing is left)
                    x[j] = pack_bf16x2(fabsf(lo) < INFINITY ? g[2 * j] - lo : 0.0f, fabsf(hi) < INFINITY ? g[2 * j + 1] - hi : 0.0f);
                }
                *reinterpret_cast<uint4 *>(operand_at(rest, at_row + i * (kSmallThreads / 8), at_col)) =
                    make_uint4(x[0], x[1], x[2], x[3]);
            }
            *reinterpret_cast<uint4 *>(operand_at(to, at_row + i * (kSmallThreads / 8), at_col)) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

// Four 8 x 8 matrices of shared memory, a row's address to a lane.
template <bool TRANS>
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], const uint16_t *row)
{
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(smem_addr(row))
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(smem_addr(row))
                     : "memory");
}

__device__ __forceinline__ float4 cluster_load4(const float *here, uint32_t rank)
{
    float4 v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
                 "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(smem_addr(here)), "r"(rank)
                 : "memory");
    return v;
}

// Eight results to a row, or as many of them as there are.
__device__ __forceinline__ void small_store(const LinearSmall &p, uint16_t *to, const float (&v)[8], uint32_t n, int buffer)
{
    (void)p, (void)buffer;
    if (n == 8 && (reinterpret_cast<uintptr_t>(to) & 15) == 0) {
        if (LINEAR_OK(buffer, to, 16))
            *reinterpret_cast<uint4 *>(to) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                                        pack_bf16x2(v[6], v[7]));
        return;
    }
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
        if (j < n && LINEAR_OK(buffer, to + j, 2)) to[j] = f32_to_bf16(v[j]);
}

// v += the values of a row, as many as there are.
__device__ __forceinline__ void small_add(const LinearSmall &p, float (&v)[8], const uint16_t *from, uint32_t n, int buffer)
{
    (void)p, (void)buffer;
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
        if (j < n && LINEAR_OK(buffer, from + j, 2)) v[j] += bf16_to_f32(from[j]);
}

// Tile `tile` of a product, blocks [kb0, kb1) of its inner axis by this CTA, number `part` of
// the `parts` that share it.
template <class R, bool VEC>
__device__ __forceinline__ void small_tile(const LinearSmall &p, const LinearProduct &c, uint32_t tile, uint32_t part,
                                           uint32_t parts, SmallSmem<R::kind> &smem)
{
    constexpr int KIND = R::kind;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, wm = warp / 2 * 32, wn = warp % 2 * 32;
    const uint32_t kb0 = c.kblocks * part / parts, kb1 = c.kblocks * (part + 1) / parts;
    Place at[3] = {};
    at[R::m] = locate<R, R::m>(p, c, tile / c.nt, kSmallTile);
    at[R::n] = locate<R, R::n>(p, c, tile % c.nt, kSmallTile);
    const Place m = at[R::m], n = at[R::n];
    float sum[2][4][4] = {};
    Source<R, R::a, R::a_mn, VEC> source_a;
    Source<R, R::b, R::b_mn, VEC> source_b;
    uint32_t left = 0;   // steps of the present piece of the inner axis
    auto load = [&](uint32_t kb) {
        if (left == 0) {
            at[R::k] = locate<R, R::k>(p, c, kb, kSmallTile);
            left = (length<R, R::k>(p, at[R::k].piece) - at[R::k].at + kSmallTile - 1) / kSmallTile;
            source_a.begin(p, at);
            source_b.begin(p, at);
        } else {
            source_a.next(p, at);
            source_b.next(p, at);
        }
        --left;
        source_a.load(p, at[kFeatures].piece);
        source_b.load(p, at[kFeatures].piece);
    };
    if (kb0 < kb1) load(kb0);
    for (uint32_t kb = kb0; kb < kb1; ++kb) {
        auto &to = smem.operand[(kb - kb0) & 1];
        constexpr int kRest = KIND == kGatherBack ? 2 : 0;
        source_a.put(p, to[0], to[kRest]);
        source_b.put(p, to[1], nullptr);
        __syncthreads();   // (the step before last has been multiplied by all)
        if (kb + 1 < kb1) load(kb + 1);
        const uint32_t j = lane / 8, in = lane % 8;
#pragma unroll
        for (uint32_t k = 0; k < kSmallTile; k += 16) {
            uint32_t fa[2][4], fb[2][4];
#pragma unroll
            for (uint32_t i = 0; i < 2; ++i) {
                const uint32_t am = wm + i * 16 + (j & 1) * 8, ak = k + (j >> 1) * 8;
                const uint32_t bn = wn + i * 16 + (j >> 1) * 8, bk = k + (j & 1) * 8;
                load_matrices<R::a_mn>(fa[i], R::a_mn ? operand_at(to[0], ak + in, am) : operand_at(to[0], am + in, ak));
                load_matrices<R::b_mn>(fb[i], R::b_mn ? operand_at(to[1], bk + in, bn) : operand_at(to[1], bn + in, bk));
            }
            auto multiply = [&] {
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
                    for (uint32_t q = 0; q < 4; ++q) mma_16x8x16(sum[i][q], fa[i], fb[q / 2][q % 2 * 2], fb[q / 2][q % 2 * 2 + 1]);
            };
            multiply();
            if (KIND == kGatherBack && p.act != DT_ACT_NONE) {
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i) {
                    const uint32_t am = wm + i * 16 + (j & 1) * 8, ak = k + (j >> 1) * 8;
                    load_matrices<R::a_mn>(fa[i], R::a_mn ? operand_at(to[kRest], ak + in, am) : operand_at(to[kRest], am + in, ak));
                }
                multiply();
            }
        }
    }
    __syncthreads();
    // a lane holds rows g and g + 8 of columns 2 q and 2 q + 1 of each 16 x 8
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
            float *to = &smem.sum[wm + i * 16 + lane / 4][wn + q * 8 + lane % 4 * 2];
            to[0] = sum[i][q][0];
            to[1] = sum[i][q][1];
            to[8 * kSumPitch] = sum[i][q][2];
            to[8 * kSumPitch + 1] = sum[i][q][3];
        }
    __syncwarp();
    if (parts > 1) cluster_sync();
    else __syncthreads();
    const uint32_t rows = length<R, R::m>(p, m.piece) - m.at, cols = length<R, R::n>(p, n.piece) - n.at;
    constexpr int kOut = !is_back(KIND) ? kLinearY : R::second ? kLinearDw : kLinearDx;
    for (uint32_t o = part * kSmallThreads + threadIdx.x; o < kSmallTile * kSmallTile / 8; o += kSmallThreads * parts) {
        const uint32_t row = o / 8, e = o % 8 * 8;
        if (row >= rows || e >= cols) continue;
        const uint32_t there = min(cols - e, 8u);
        float v[8] = {};
        for (uint32_t k = 0; k < parts; ++k) {
            float4 lo, hi;
            if (parts > 1) {
                lo = cluster_load4(&smem.sum[row][e], k);
                hi = cluster_load4(&smem.sum[row][e + 4], k);
            } else {
                lo = *reinterpret_cast<const float4 *>(&smem.sum[row][e]);
                hi = *reinterpret_cast<const float4 *>(&smem.sum[row][e + 4]);
            }
            v[0] += lo.x, v[1] += lo.y, v[2] += lo.z, v[3] += lo.w, v[4] += hi.x, v[5] += hi.y, v[6] += hi.z, v[7] += hi.w;
        }
        const OutRow out = out_row<R>(p, c, m, n, row);
        if (!is_back(KIND) && p.biased) {
            const uint32_t r = KIND == kGather ? n.piece : 0;
            small_add(p, v, p.bias[r] + n.at + e, there, kLinearBias + r);
        }
        if (KIND == kReduce && p.residuals) small_add(p, v, p.residual[out.rank] + out.offset + e, there, kLinearResidual + out.rank);
        if (KIND == kGather && p.keep) small_store(p, p.pre[out.rank] + out.offset + e, v, there, kLinearPre + out.rank);
        if (KIND == kGather) activate(v, p.act);
        small_store(p, out.out + out.offset + e, v, there, kOut + out.rank);
    }
    __syncwarp();
    if (parts > 1) cluster_sync();   // no CTA leaves while another reads its sums
}

// 64 columns of the bias' gradient: eight threads across, 16 rows at a time, four of them
// under way for each thread.
template <class R>
__device__ __forceinline__ void small_sums(const LinearSmall &p, uint32_t strip, SmallSmem<R::kind> &smem)
{
    constexpr bool kFeature = R::kind == kGatherBack;
    constexpr int MATRIX = kFeature ? kFeat : kTok;
    Place at[3] = {};
    const Place col = kFeature ? locate<R, kFeatures>(p, p.product[1], strip, kSmallTile) : locate<R, kDim>(p, p.product[1], strip, kSmallTile);
    at[kFeature ? kFeatures : kDim] = col;
    float sum[8] = {};
    const uint32_t first = threadIdx.x / 8, e = col.at + threadIdx.x % 8 * 8;
    for (uint32_t row = first; row < p.tokens; row += 4 * (kSmallThreads / 8)) {
        Shifted w[4], u[4];
        uint32_t n[4];
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            uint32_t width;
            int buffer = 0;
            const uint16_t *from = matrix_row<R, MATRIX>(p, col.piece, row + k * (kSmallThreads / 8), width, buffer);
            n[k] = from && e < width ? min(width - e, 8u) : 0;
            w[k].load(from + e, n[k] && LINEAR_OK(buffer, from + e, 2 * n[k]) ? n[k] : 0);
            (void)buffer;
            if (kFeature && p.act != DT_ACT_NONE) {
                const uint16_t *z = p.z[col.piece] + (from - p.feat[col.piece]) + e;
                u[k].load(z, n[k] && LINEAR_OK(kLinearPre + col.piece, z, 2 * n[k]) ? n[k] : 0);
            }
        }
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            if (n[k] == 0) continue;
            uint32_t x[4];
            float g[8], v[8];
            w[k].get(x);
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) g[j] = j & 1 ? bf16_hi(x[j / 2]) : bf16_lo(x[j / 2]);
            if (kFeature && p.act != DT_ACT_NONE) {
                u[k].get(x);
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) v[j] = j & 1 ? bf16_hi(x[j / 2]) : bf16_lo(x[j / 2]);
                times_slope(g, v, p.act);
            }
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) sum[j] += g[j];
        }
    }
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) smem.sum[first][threadIdx.x % 8 * 8 + j] = sum[j];
    __syncthreads();
    if (threadIdx.x >= kSmallTile) return;
    float all = 0.0f;
#pragma unroll
    for (uint32_t k = 0; k < kSmallThreads / 8; ++k) all += smem.sum[k][threadIdx.x];
    const uint32_t width = kFeature ? p.f_len[col.piece] : p.dim, c = col.at + threadIdx.x;
    const uint32_t r = kFeature ? col.piece : 0;
    if (c < width && LINEAR_OK(kLinearDb + r, p.sums.out[r] + c, 2)) p.sums.out[r][c] = f32_to_bf16(all);
}

template <int KIND, int C, bool VEC>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kSmallThreads) linear_small_kernel(const __grid_constant__ LinearSmall p)
{
    using First = Roles<KIND, false, false>;
    using Second = Roles<KIND, is_back(KIND), false>;
    __shared__ __align__(16) SmallSmem<KIND> smem;
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    const uint32_t part = C > 1 ? cluster_rank() : 0;
    uint32_t cluster = blockIdx.x / C;
    auto run = [&](auto roles, const LinearProduct &c, bool shared) {
        const uint32_t tile = shared ? cluster : cluster * C + part;
        if (tile < c.mt * c.nt) small_tile<decltype(roles), VEC>(p, c, tile, shared ? part : 0, shared ? C : 1, smem);
    };
    if (cluster < p.clusters[0]) {
        run(First{}, p.product[0], p.shared[0]);
    } else if (is_back(KIND)) {
        cluster -= p.clusters[0];
        if (cluster < p.clusters[1]) {
            run(Second{}, p.product[1], p.shared[1]);
        } else {
            const uint32_t strip = (cluster - p.clusters[1]) * C + part;
            if (strip < p.strips) small_sums<Second>(p, strip, smem);
        }
    }
    DT_TL_END_BLOCK(DT_TL_LINEAR);
}

template <int KIND, int NT, bool VEC>
cudaError_t launch_few(const LinearFew &p, uint32_t ctas, cudaStream_t s)
{
    const dim3 grid(p.blocks * ctas), block(kThreads);
    switch (ctas) {
    case 8: return launch_kernel(linear_few_kernel<KIND, NT, VEC, 8>, grid, block, 0, s, false, p);
    case 4: return launch_kernel(linear_few_kernel<KIND, NT, VEC, 4>, grid, block, 0, s, false, p);
    case 2: return launch_kernel(linear_few_kernel<KIND, NT, VEC, 2>, grid, block, 0, s, false, p);
    default: return launch_kernel(linear_few_kernel<KIND, NT, VEC, 1>, grid, block, 0, s, false, p);
    }
}

template <int KIND>
cudaError_t launch_few(const LinearFew &p, bool vec, uint32_t ctas, cudaStream_t s)
{
    if (p.tokens <= 8) return vec ? launch_few<KIND, 1, true>(p, ctas, s) : launch_few<KIND, 1, false>(p, ctas, s);
    return vec ? launch_few<KIND, 2, true>(p, ctas, s) : launch_few<KIND, 2, false>(p, ctas, s);
}

template <int KIND, bool VEC>
cudaError_t launch_small(const LinearSmall &p, cudaStream_t s)
{
    const dim3 grid((p.clusters[0] + p.clusters[1] + (p.strips + p.ctas - 1) / p.ctas) * p.ctas), block(kSmallThreads);
    switch (p.ctas) {
    case 8: return launch_kernel(linear_small_kernel<KIND, 8, VEC>, grid, block, 0, s, false, p);
    case 4: return launch_kernel(linear_small_kernel<KIND, 4, VEC>, grid, block, 0, s, false, p);
    case 2: return launch_kernel(linear_small_kernel<KIND, 2, VEC>, grid, block, 0, s, false, p);
    default: return launch_kernel(linear_small_kernel<KIND, 1, VEC>, grid, block, 0, s, false, p);
    }
}

template <int KIND>
cudaError_t launch_small(const LinearSmall &p, bool vec, cudaStream_t s)
{
    return vec ? launch_small<KIND, true>(p, s) : launch_small<KIND, false>(p, s);
}

}  // namespace

DT_TL_BINDER(bind_timeline_linear_small)

cudaError_t launch_linear_small(const LinearSmall &p, LinearKind kind, bool vec, cudaStream_t s)
{
    switch (kind) {
    case kGather: return launch_small<kGather>(p, vec, s);
    case kGatherBack: return launch_small<kGatherBack>(p, vec, s);
    case kReduce: return launch_small<kReduce>(p, vec, s);
    default: return launch_small<kReduceBack>(p, vec, s);
    }
}

// Warps and CTAs that share a row of W: two steps of the inner axis to a warp at least,
// and as many CTAs as give the SMs two each.
cudaError_t launch_linear_few(LinearFew &p, LinearKind kind, bool vec, int device, cudaStream_t s)
{
    const uint32_t depth = few_depth(vec);
    uint64_t steps = 0, rows = 0;
    for (int r = 0; r < p.P; ++r) {
        if (kind == kGather) rows += (p.f_len[r] + kFewRows - 1) / kFewRows;
        else steps += (p.f_len[r] + depth - 1) / depth;
    }
    if (kind == kGather) steps = (p.dim + depth - 1) / depth;
    else rows = (p.dim + kFewRows - 1) / kFewRows;
    p.k_warps = 1;
    while (p.k_warps < kFewWarps && p.k_warps * 2 <= steps) p.k_warps *= 2;
    const uint32_t groups = kFewWarps / p.k_warps;
    p.blocks = 0;
    for (int r = 0; r < p.P; ++r)
        p.block_end[r] = p.blocks += kind == kGather ? (p.f_len[r] + groups * kFewRows - 1) / (groups * kFewRows) : 0;
    if (kind == kReduce) p.blocks = (uint32_t)((rows + groups - 1) / groups);
    uint32_t ctas = 1;
    while (ctas < 8 && p.blocks * ctas < 2u * sm_count(device) && (uint64_t)ctas * 4 * p.k_warps <= steps) ctas *= 2;
    return kind == kGather ? launch_few<kGather>(p, vec, ctas, s) : launch_few<kReduce>(p, vec, ctas, s);
}

}  // namespace dt
