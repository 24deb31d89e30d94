// Linear layers of a block whose tokens and features are both split over the
// ranks, and their gradients (LinearKind).
//
//   gathering   y_r  = act(X W_r^T + b_r)            X: all ranks' tokens
//               dx   = sum_r G_r W_r                 G_r = dy_r act'(pre_r)
//               dW_r = G_r^T X,  db_r = sum_tokens G_r
//   reducing    y    = sum_r H_r W_r^T + b + residual, each rank its own tokens
//               dH_r = Y W_r
//               dW_r = Y^T H_r,  db = sum_tokens Y       Y: all ranks' dy
//
// Every one of these is a product along one of three axes (tokens, columns of a
// token, features) of two of three matrices: the ranks' tokens, the ranks'
// features and the weights.  One persistent kernel serves all: tiles of 128 x
// bn outputs, or of 256 x bn for two CTAs of a cluster, operands brought by TMA
// into a ring of shared memory stages by one warp, multiplied by one warp's
// tcgen05.mma into tensor memory, and finished by eight or more warps that
// read the accumulator while the next tile's is made in the other half of tensor
// memory.  A backward call's two products are one launch, so that one's tiles
// fill what the other's leave of the last wave.
//
// The ranks are offsets and no more.  Along an output's axis a tile lies within
// one rank's piece; along the inner axis the ranks' pieces follow one another in
// blocks of 64 or 128, in the same accumulator: the gathered tokens and the partial sums
// of the ranks, which a gather and a reduction around a library's product would
// write and read, are never in memory, and the sum over the ranks is rounded once.
// Past a piece's end TMA fills in zeros.
//
// Sums are fp32.  The tensor cores add 16 products at a time, each aligned to the largest
// of them and the sum so far and cut off two bits below its last place: at most 2^-25 of
// the sum is lost to a term, n * 2^-25 to n of them (3.97 of 4 units of 2^-23 for 16 terms of
// 1.99 * 2^-25 beside a 1).  Terms of one sign, uniform from 0 to 1, lose n * 4.4e-9 to 5.3e-9 of
// their sum (16384, 65536 of them; 7e-5 of it at 16384), where results are rounded by up to
// 2^-8 of themselves; normal ones nothing that shows (rms 1.4e-11 n of the sum of magnitudes).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "dt_linear.cuh"

#include "dt_bounds.cuh"
#include "dt_device.cuh"
#include "dt_math.cuh"
#include "dt_tc.cuh"
#include "dt_tile.cuh"
#include "dt_timeline.cuh"

namespace dt {
namespace {

constexpr uint32_t kM = 128;                       // rows of a tile in a CTA
// Three stages of 128 rows and columns of A and B, or six of 64 columns (2048 tokens of
// 4096 to 16384 with four, five, six of them: 171, 157, 150 us).
// Forward tiles of up to 128 columns, whose products take less time than a stage takes to
// issue, have two such blocks to a stage (512 tokens of 4096 to 4096: 17.7 -> 14.7 us; wider
// tiles no faster, 512 of 4096 to 16384: 42.4 -> 45.3).
constexpr uint32_t kRingBytes = 192 * 1024;
constexpr uint32_t kMaxStages = 16;
constexpr uint32_t kTmemColumns = 512;             // two accumulators of 128 x 256 fp32
// Finishing warps, FW: eight, or 16 of gathering layers with a short inner axis and an
// activation, whose finish takes longer than the products, where each worker has several tiles
// (8192 tokens of 512 to 8192, gelu and what it is taken of: 106 us with eight, 100 with 16;
// without an activation 54 and 55; 1024 tokens of 1024 to 1024 with gelu 6.8 and 7.6).  Then
// one for TMA, one for the products, and backward two for the bias' gradient.
constexpr uint32_t kShortBlocks = 16;              // of 64: blocks of a short inner axis, at most
constexpr uint32_t kMostFinishWarps = 16, kSumWarps = 2;
__host__ __device__ constexpr int tc_threads(bool back, uint32_t fw) { return (fw + 2 + (back ? kSumWarps : 0)) * 32; }
constexpr uint32_t kStep = 32;                     // columns that a finishing warp takes at a time
constexpr uint32_t kStageOut = 32 * kStep * 2;     // its 32 rows of them in bf16
constexpr uint32_t kOutBytes = kMostFinishWarps * kStageOut;
constexpr uint32_t kBarBytes = 384, kBiasBytes = kMostFinishWarps * kStep * 2;
constexpr size_t kTcSmem = 1024 + kRingBytes + kOutBytes + kBarBytes + kBiasBytes;
static_assert(kTcSmem <= 227 * 1024, "shared memory above the per-block limit");
// Columns of tiles that are worked on together, rows fastest, so that the tiles in
// flight share few rows and columns and their operands come from L2 (2048 tokens of 4096
// to 16384: 16 columns, columns fastest 152 us, eight 142.5, rows fastest 141.5).
constexpr uint32_t kGroup = 8;

// Walks over the blocks of the inner axis, the blocks of one piece after the other.
template <class R>
struct Inner {
    Place at;            // of the piece's first block here
    uint32_t blocks;     // of it from there on, at most as many as are left
    uint32_t last;       // K steps of 16 in the piece's very last block
    bool ends;           // that one is among them
    uint32_t left;
    __device__ __forceinline__ Inner(const LinearParams &p, const LinearProduct &c, uint32_t kb0, uint32_t kb1)
        : at(locate<R, R::k>(p, c, kb0, R::depth)), left(kb1 - kb0)
    {
        take(p);
    }
    __device__ __forceinline__ void take(const LinearParams &p)
    {
        const uint32_t len = length<R, R::k>(p, at.piece) - at.at, all = (len + R::depth - 1) / R::depth;
        blocks = min(all, left);
        ends = all <= left;
        last = ((len - 1) % R::depth + 16) / 16;
        left -= blocks;
    }
    // The next piece that has something; false at the end.
    __device__ __forceinline__ bool next(const LinearParams &p)
    {
        if (left == 0) return false;
        while (length<R, R::k>(p, ++at.piece) == 0) {}
        at.at = 0;
        if (R::k == kTokens) at.all = p.t_first[at.piece];
        take(p);
        return true;
    }
};

struct Tile {
    bool second;
    uint32_t m, n, kb0, kb1, split;
};

__device__ __forceinline__ void place_tile(const LinearProduct &c, uint32_t i, Tile &t)
{
    const uint32_t per_split = c.mt * c.nt, all = kGroup * c.mt;
    t.split = 0, t.kb0 = 0, t.kb1 = c.kblocks;
    if (c.splits > 1) {   // at most 16 splits of 2^20 blocks
        t.split = i / per_split;
        i -= t.split * per_split;
        t.kb0 = c.kblocks * t.split / c.splits;
        t.kb1 = c.kblocks * (t.split + 1) / c.splits;
    }
    const uint32_t g = quotient(i, all, c.group_inverse);
    i -= g * all;
    const uint32_t n = quotient(i, c.mt, c.mt_inverse);
    t.n = g * kGroup + n;
    t.m = i - n * c.mt;
}

// The k-th tile of worker q (a CTA or a pair) of W; false when it has no more.
// First the tiles of the first product, one by one to the workers.  While the first `rest`
// workers still have one more of them, the others take `early` tiles of the second
// product each; then all take the rest of those in turn.
template <int KIND>
__device__ __forceinline__ bool next_tile(const LinearParams &p, uint32_t q, uint32_t W, uint32_t k, Tile &t)
{
    const uint32_t tiles = p.product[0].tiles;
    const uint32_t mine = q < tiles ? (tiles - q + W - 1) / W : 0;
    t.second = false;
    if (k < mine) {
        place_tile(p.product[0], q + k * W, t);
        return true;
    }
    if constexpr (!is_back(KIND)) return false;
    k -= mine;
    uint32_t i;
    const uint32_t others = W - p.rest;
    if (q >= p.rest && k < p.early) {
        i = q - p.rest + k * others;
    } else {
        if (q >= p.rest) k -= p.early;
        i = p.early * others + k * W + (q >= p.rest ? q - p.rest : q + others);
    }
    if (i >= p.product[1].tiles) return false;
    t.second = true;
    place_tile(p.product[1], i, t);
    return true;
}

// The map of an operand, and the column and row of its first box, at these places.
template <class R, int MATRIX>
__device__ __forceinline__ const CUtensorMap *operand(const LinearParams &p, const Place (&at)[3], uint32_t &col,
                                                      uint32_t &row)
{
    const Place &t = at[kTokens], &d = at[kDim], &f = at[kFeatures];
    if (MATRIX == kTok) {
        col = d.at;
        row = t.at;
        return &p.tok[t.piece];
    }
    if (MATRIX == kFeat) {
        col = f.at;
        row = t.all;
        return &p.feat[f.piece];
    }
    col = R::w_by_feature ? d.at : f.at;
    row = R::w_by_feature ? f.at : d.at;
    return &p.w[f.piece];
}

// From operand A's first box to its second: K-major boxes of few tokens' rows lie
// closer, MN-major ones are a fixed way apart.
__host__ __device__ constexpr uint32_t a_box_bytes(bool back, uint32_t rows)
{
    return back ? kBoxBytes : (rows * 128 + 1023) / 1024 * 1024;
}

// Boxes of 64 columns in a stage: one of a K-major operand, 64 deep, or as many as hold
// the columns of an MN-major one; backward, where one operand at least is MN-major, a
// K-major one has two.
__host__ __device__ constexpr uint32_t a_boxes(bool back) { return back ? 2 : 1; }
__host__ __device__ constexpr uint32_t b_boxes(bool back, uint32_t bn) { return back ? (bn + 63) / 64 : 1; }
__host__ __device__ constexpr uint32_t stage_size(bool back, uint32_t rows_t, uint32_t bn)
{
    return a_boxes(back) * a_box_bytes(back, rows_t) + (back ? b_boxes(back, bn) * kBoxBytes : bn * 128);
}

// A tile's loads.  A block of a stage is the boxes of A, 64 columns apart, and those of B; what it
// holds beside them is left over from earlier loads and reaches only rows of the
// accumulator that are not stored.  Maps and coordinates are worked out once for a
// piece of the inner axis: done for every stage they took the issuing thread longer
// (680 cycles) than the products take (2048 tokens of 4096 to 16384: 168 -> 162 us).
template <class R, int CG, class Wait>
__device__ __forceinline__ bool load_tile(const LinearParams &p, const LinearProduct &c, const Tile &t, uint32_t half,
                                          uint32_t ring, uint32_t block_bytes, uint32_t a_box, uint32_t full,
                                          uint32_t empty, const Wait &wait, uint32_t &s, uint32_t &round, uint32_t &n)
{
    constexpr bool kBack = R::b_mn;
    Place at[3] = {};
    at[R::m] = locate<R, R::m>(p, c, t.m * CG + half, kM);
    at[R::n] = locate<R, R::n>(p, c, t.n, p.bn);
    const uint32_t bn = p.bn / CG, boxes = b_boxes(kBack, bn), b_rows = kBack ? (R::b == kW ? R::depth : p.rows_t) : bn;
    const uint32_t bytes = CG * (a_boxes(kBack) * p.rows_t + boxes * b_rows) * 128, stages = p.stages;
    const uint32_t step = kBack ? 1 : p.step;
    Inner<R> k(p, c, t.kb0, t.kb1);
    do {
        at[R::k] = k.at;
        uint32_t a_col, a_row, b_col, b_row;
        const CUtensorMap *a_map = operand<R, R::a>(p, at, a_col, a_row), *b_map = operand<R, R::b>(p, at, b_col, b_row);
        (R::b_mn ? b_col : b_row) += half * bn;
        for (uint32_t i = 0; i < k.blocks; i += step, ++n) {
            if (!__all_sync(0xFFFFFFFFu, wait(empty + 8 * s, round ^ 1))) return false;
            const uint32_t bar = full + 8 * s, a = ring + s * step * block_bytes, b = a + a_boxes(kBack) * a_box;
            const bool two = step == 2 && i + 1 < k.blocks;
            if (elect_one()) {
                if (half == 0) mbar_expect_tx(bar, two ? 2 * bytes : bytes);
                tma_box<CG>(a, a_map, a_col, a_row, bar);
                if (a_boxes(kBack) == 2) tma_box<CG>(a + a_box, a_map, a_col + 64, a_row, bar);
                tma_box<CG>(b, b_map, b_col, b_row, bar);
                if (boxes == 2) tma_box<CG>(b + kBoxBytes, b_map, b_col + 64, b_row, bar);
                if (two) {   // (forward: K-major)
                    tma_box<CG>(a + block_bytes, a_map, a_col + R::depth, a_row, bar);
                    tma_box<CG>(b + block_bytes, b_map, b_col + R::depth, b_row, bar);
                }
            }
            (R::a_mn ? a_row : a_col) += step * R::depth;
            (R::b_mn ? b_row : b_col) += step * R::depth;
            if (++s == stages) s = 0, round ^= 1;
        }
    } while (k.next(p));
    return true;
}

// A stage's products.
template <class R, int CG>
__device__ __forceinline__ void multiply_stage(uint32_t acc, uint64_t a, uint64_t b, uint32_t desc, bool add, uint32_t steps,
                                               uint32_t a_box)
{
    // from a K step of 16 to the next: 16 rows of an MN-major box; 32 bytes of a
    // K-major one, and from its fourth to the next box, where a stage is that deep (B
    // is MN-major there)
    const uint32_t a_step = R::a_mn ? 16 * 128 : 32, a_next = R::a_mn ? 4 * a_step : a_box;
    const uint32_t b_step = R::b_mn ? 16 * 128 : 32, b_next = 4 * b_step;
#pragma unroll
    for (uint32_t j = 0; j < R::depth / 16; ++j)
        if (j < steps)
            mma_bf16<CG>(acc, a + ((j / 4 * a_next + j % 4 * a_step) >> 4), b + ((j / 4 * b_next + j % 4 * b_step) >> 4), desc,
                         add || j != 0);
}

// A tile's products.
template <class R, int CG, class Wait>
__device__ __forceinline__ bool multiply_tile(const LinearParams &p, const LinearProduct &c, const Tile &t, uint32_t acc,
                                              uint32_t ring, uint32_t block_bytes, uint32_t a_box, uint32_t full,
                                              uint32_t empty, const Wait &wait, uint32_t &s, uint32_t &round)
{
    const uint32_t desc = mma_desc(kM * CG, p.bn, R::a_mn, R::b_mn), stages = p.stages, step = R::b_mn ? 1 : p.step;
    const uint64_t a0 = smem_desc(ring, R::a_mn), b0 = smem_desc(ring + a_boxes(R::b_mn) * a_box, R::b_mn);
    Inner<R> k(p, c, t.kb0, t.kb1);
    bool add = false;
    do {
        for (uint32_t i = 0; i < k.blocks; i += step) {
            if (!__all_sync(0xFFFFFFFFu, wait(full + 8 * s, round))) return false;
            tc_fence_after();
            const uint32_t block = block_bytes >> 4, at = s * step * block;
            const uint32_t last = k.ends ? k.last : R::depth / 16;   // K steps of the piece's last block here
            const bool two = step == 2 && i + 1 < k.blocks;
            if (elect_one()) {
                if (i + 1 < k.blocks || last == R::depth / 16)
                    multiply_stage<R, CG>(acc, a0 + at, b0 + at, desc, add, R::depth / 16, a_box);
                else
                    multiply_stage<R, CG>(acc, a0 + at, b0 + at, desc, add, last, a_box);
                if (two)
                    multiply_stage<R, CG>(acc, a0 + at + block, b0 + at + block, desc, true,
                                          i + 2 < k.blocks ? R::depth / 16 : last, a_box);
                mma_commit<CG>(empty + 8 * s);
            }
            add = true;
            if (++s == stages) s = 0, round ^= 1;
        }
    } while (k.next(p));
    return true;
}

// A pointer of another lane.
__device__ __forceinline__ uint16_t *lane_pointer(uint16_t *v, uint32_t lane)
{
    return reinterpret_cast<uint16_t *>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(v), lane));
}

// The number of the buffer of another lane's row, which checks of bounds alone ask for
// (8192 tokens of 512 to 8192 with a bias: with these shuffles 63 us, 57.6 without).
__device__ __forceinline__ int lane_buffer(int buffer, uint32_t lane)
{
#ifdef DT_BOUNDS
    return __shfl_sync(0xFFFFFFFFu, buffer, lane);
#else
    return (void)lane, buffer;
#endif
}

// 16-byte chunk c (of four) of row r of a finishing warp's 32 x 64 bytes of shared
// memory: a thread writes its row, and four threads read a row, without bank conflicts.
__device__ __forceinline__ unsigned char *step_chunk(unsigned char *buf, uint32_t row, uint32_t c)
{
    return buf + row * 64 + ((c ^ (row >> 1 & 3)) << 4);
}

// A warp's rows between `buf` and memory, N elements of a row to a lane and as many
// rows at a time as that leaves lanes for.  row: where this lane's row begins, NULL
// where there is none.  Stores are marked as not soon read again, so that the operands
// stay in L2 (as above with gelu and what it is taken of: 155.7 -> 154.7 us).
template <int N, bool STORE>
__device__ __forceinline__ void move_rows(const LinearParams &p, unsigned char *buf, uint16_t *row, uint32_t cols, int buffer)
{
    using W = typename Words<N>::type;
    (void)p;
    constexpr uint32_t kLanes = kStep / N, kRows = 32 / kLanes;
    const uint32_t lane = threadIdx.x & 31, e = lane % kLanes * N, first = lane / kLanes;
#pragma unroll
    for (uint32_t k0 = 0; k0 < 32; k0 += 4 * kRows) {
        uint16_t *at[4];
        W v[4];
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            const uint32_t r = k0 + k * kRows + first;
            at[k] = lane_pointer(row, r);
            const int of = lane_buffer(buffer, r);
            if (!at[k] || e >= cols || !LINEAR_OK(of, at[k] + e, 2 * N)) at[k] = nullptr;
            (void)of;
            W *word = reinterpret_cast<W *>(step_chunk(buf, r, e >> 3) + (e & 7) * 2);
            if (at[k]) {
                if constexpr (STORE) __stcs(reinterpret_cast<W *>(at[k] + e), *word);
                else v[k] = *reinterpret_cast<const W *>(at[k] + e);
            }
        }
        if constexpr (!STORE) {
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
                if (at[k]) *reinterpret_cast<W *>(step_chunk(buf, k0 + k * kRows + first, e >> 3) + (e & 7) * 2) = v[k];
        }
    }
}

// The same for rows that begin at any element: an element to a lane, a row at a time,
// the loads of 16 rows under way together.
template <bool STORE>
__device__ __forceinline__ void move_rows_odd(const LinearParams &p, unsigned char *buf, uint16_t *row, uint32_t cols, int buffer)
{
    (void)p;
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll
    for (uint32_t r0 = 0; r0 < 32; r0 += 16) {
        uint16_t v[16];
#pragma unroll
        for (uint32_t k = 0; k < 16; ++k) {
            uint16_t *at = lane_pointer(row, r0 + k);
            const int of = lane_buffer(buffer, r0 + k);
            (void)of;
            const bool there = at && lane < cols && LINEAR_OK(of, at + lane, 2);
            v[k] = 0;
            if constexpr (STORE) {
                if (there) at[lane] = *reinterpret_cast<uint16_t *>(step_chunk(buf, r0 + k, lane >> 3) + (lane & 7) * 2);
            } else {
                if (there) v[k] = at[lane];
            }
        }
        if constexpr (!STORE)
#pragma unroll
            for (uint32_t k = 0; k < 16; ++k)
                *reinterpret_cast<uint16_t *>(step_chunk(buf, r0 + k, lane >> 3) + (lane & 7) * 2) = v[k];
    }
}

template <bool STORE>
__device__ __forceinline__ void move_rows(const LinearParams &p, unsigned char *buf, uint16_t *row, uint32_t cols,
                                          uint32_t align, int buffer)
{
    if (align == 8) move_rows<8, STORE>(p, buf, row, cols, buffer);
    else if (align == 4) move_rows<4, STORE>(p, buf, row, cols, buffer);
    else if (align == 2) move_rows<2, STORE>(p, buf, row, cols, buffer);
    else move_rows_odd<STORE>(p, buf, row, cols, buffer);
}

// This lane's row of 32 columns to memory by way of `buf`.
__device__ __forceinline__ void store_rows(const LinearParams &p, unsigned char *buf, const float (&v)[kStep], uint16_t *row,
                                           uint32_t cols, uint32_t align, int buffer)
{
    const uint32_t lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (uint32_t c = 0; c < kStep / 8; ++c)
        *reinterpret_cast<uint4 *>(step_chunk(buf, lane, c)) =
            make_uint4(pack_bf16x2(v[8 * c], v[8 * c + 1]), pack_bf16x2(v[8 * c + 2], v[8 * c + 3]),
                       pack_bf16x2(v[8 * c + 4], v[8 * c + 5]), pack_bf16x2(v[8 * c + 6], v[8 * c + 7]));
    __syncwarp();
    move_rows<true>(p, buf, row, cols, align, buffer);
}

// v += 32 bf16 values in four vectors.
template <class Vector>
__device__ __forceinline__ void add_vectors(float (&v)[kStep], const Vector &vector)
{
#pragma unroll
    for (uint32_t j = 0; j < kStep / 8; ++j) {
        const uint4 b = vector(j);
        const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
            const float2 f = add2(make_float2(v[8 * j + 2 * q], v[8 * j + 2 * q + 1]), make_float2(bf16_lo(w[q]), bf16_hi(w[q])));
            v[8 * j + 2 * q] = f.x, v[8 * j + 2 * q + 1] = f.y;
        }
    }
}

// What a step of 32 columns adds to its sums, on its way while the accumulator is waited
// for: the bias, a column to a lane, and, where rows are whole vectors, this lane's row
// of the residual.
struct Extra {
    uint16_t bias;
    uint4 residual[kStep / 8];
};

template <int KIND>
__device__ __forceinline__ void fetch(const LinearParams &p, const OutRow &o, bool there, const Place &n, uint32_t c,
                                      uint32_t cols, uint32_t align, Extra &x)
{
    if (!is_back(KIND) && p.biased) {
        // one bias for all ranks' tokens, or each rank's own for its features
        const uint32_t r = KIND == kGather ? n.piece : 0, lane = threadIdx.x & 31;
        const uint16_t *from = p.bias[r] + n.at + c + lane;
        x.bias = c + lane < cols && LINEAR_OK(kLinearBias + r, from, 2) ? *from : 0;
    }
    if (KIND == kReduce && p.residuals && align == 8) {
        const uint16_t *from = p.residual[o.rank] + o.offset + c;
#pragma unroll
        for (uint32_t j = 0; j < kStep / 8; ++j)
            x.residual[j] = there && c + 8 * j < cols && LINEAR_OK(kLinearResidual + o.rank, from + 8 * j, 16)
                                ? *reinterpret_cast<const uint4 *>(from + 8 * j)
                                : make_uint4(0, 0, 0, 0);
    }
}

// 32 sums of this lane's row, whose columns begin at column `c` of the tile: bias,
// residual, activation, and to memory.  `next` fetches what the next step adds.
template <int KIND, class R, class Next>
__device__ __forceinline__ void finish_row(const LinearParams &p, unsigned char *buf, unsigned char *biases,
                                           float (&v)[kStep], const Extra &x, const OutRow &o, bool there, uint32_t c,
                                           uint32_t cols, uint32_t align, const Next &next)
{
    const uint32_t lane = threadIdx.x & 31;
    if (!is_back(KIND) && p.biased) {
        __syncwarp();
        reinterpret_cast<uint16_t *>(biases)[lane] = x.bias;
        __syncwarp();
        add_vectors(v, [&](uint32_t j) { return reinterpret_cast<const uint4 *>(biases)[j]; });
    }
    if (KIND == kReduce && p.residuals) {
        if (align == 8) {
            add_vectors(v, [&](uint32_t j) { return x.residual[j]; });
        } else {
            uint16_t *from = there ? const_cast<uint16_t *>(p.residual[o.rank]) + o.offset + c : nullptr;
            __syncwarp();
            move_rows<false>(p, buf, from, cols, align, kLinearResidual + o.rank);
            __syncwarp();
            add_vectors(v, [&](uint32_t j) { return *reinterpret_cast<const uint4 *>(step_chunk(buf, lane, j)); });
        }
    }
    next();
    if (KIND == kGather && p.keep)
        store_rows(p, buf, v, there ? p.pre[o.rank] + o.offset + c : nullptr, cols, align, kLinearPre + o.rank);
    if (KIND == kGather) activate(v, p.act);
    constexpr int kOut = !is_back(KIND) ? kLinearY : R::k == kTokens ? kLinearDw : kLinearDx;
    store_rows(p, buf, v, there ? o.out + o.offset + c : nullptr, cols, align, kOut + o.rank);
}

// One tile's accumulator, by a warp whose 32 rows begin at row `quad` of the CTA's 128
// (number `unit` along the rows' axis) and which takes steps of 32 columns in turn, from `group` on.  `take` waits
// for the accumulator (false: it gave up), `give_back` hands it over as soon as the warp
// has read its part.
template <int KIND, uint32_t FW, class R, class Take, class GiveBack>
__device__ __forceinline__ bool finish_tile(const LinearParams &p, const LinearProduct &c, const Tile &t, uint32_t acc,
                                            uint32_t unit, uint32_t units, uint32_t quad, uint32_t group, unsigned char *buf,
                                            unsigned char *biases, const Take &take, const GiveBack &give_back)
{
    const Place m = locate<R, R::m>(p, c, unit, kM), n = locate<R, R::n>(p, c, t.n, p.bn);
    const uint32_t lane = threadIdx.x & 31, row = quad + lane, len = length<R, R::m>(p, m.piece);
    const uint32_t rows = m.at < len ? len - m.at : 0, cols = min(length<R, R::n>(p, n.piece) - n.at, p.bn);
    const bool there = row < rows;
    const bool none = group * kStep >= cols || quad >= rows;
    if (none) {
        if (!take()) return false;
        give_back();
        return true;
    }
    const OutRow o = c.splits > 1 ? OutRow{} : out_row<R>(p, c, m, n, there ? row : 0);
    // the rows of a warp may lie on several ranks, whose buffers are aligned alike (the host says how)
    const uint32_t align = c.align[R::m == kTokens && R::n == kDim ? 0 : o.rank];
    const uint64_t pitch = (uint64_t)c.nt * p.bn;
    float *part = c.acc + (((uint64_t)t.split * units + unit) * kM + quad) * pitch + t.n * p.bn;
    Extra x;
    if (c.splits == 1) fetch<KIND>(p, o, there, n, group * kStep, cols, align, x);
    if (!take()) return false;
    for (uint32_t b = group * kStep; b < cols; b += FW / 4 * kStep) {
        float v[kStep];
        tmem_load32(acc + b, v);
        if (b + FW / 4 * kStep >= cols) give_back();
        if (c.splits == 1) {
            finish_row<KIND, R>(p, buf, biases, v, x, o, there, b, min(cols - b, kStep), align, [&] {
                if (b + FW / 4 * kStep < cols) fetch<KIND>(p, o, there, n, b + FW / 4 * kStep, cols, align, x);
            });
            continue;
        }
        // fp32 sums: 16 columns at a time through shared memory, so that four threads
        // take a row's 64 bytes
#pragma unroll
        for (uint32_t h = 0; h < kStep; h += 16) {
            __syncwarp();
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
                *reinterpret_cast<float4 *>(step_chunk(buf, lane, j)) =
                    make_float4(v[h + 4 * j], v[h + 4 * j + 1], v[h + 4 * j + 2], v[h + 4 * j + 3]);
            __syncwarp();
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                const uint32_t r = 8 * j + lane / 4;
                float4 *to = reinterpret_cast<float4 *>(part + r * pitch + b + h + lane % 4 * 4);
                if (quad + r < rows && LINEAR_OK(kLinearWorkspace, to, 16))
                    *to = *reinterpret_cast<const float4 *>(step_chunk(buf, r, lane % 4));
            }
        }
    }
    return true;
}

// ---- the bias' gradient: column sums ---------------------------------------------

// 32 columns a warp, which walks down the rows four lanes to a row;
// warp `i` of `all` takes the groups of 32 columns i, i + all, ...
__device__ __forceinline__ void column_sums(const LinearParams &p, uint32_t i, uint32_t all)
{
    const LinearSums &c = p.sums;
    const uint32_t lane = threadIdx.x & 31;
    for (; i < c.groups; i += all) {
        int k = 0;
        uint32_t begin = 0;
        while (k + 1 < c.n && i >= c.group_end[k]) begin = c.group_end[k++];
        const uint32_t e = (i - begin) * 32 + lane % 4 * 8, cols = c.cols[k];
        const uint32_t n = e < cols ? min(cols - e, 8u) : 0;
        constexpr uint32_t kSumRows = 6;   // loads under way
        float sum[8] = {};
        for (int q = c.stacked ? 0 : k; q < (c.stacked ? c.sources : k + 1); ++q) {
            if (c.f32) {
                for (uint32_t first = lane / 4; first < c.rows[q]; first += 32) {
                    float v[4][8];
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) {
                        const float *from = static_cast<const float *>(c.src[q]) + (uint64_t)(first + 8 * j) * cols + e;
#pragma unroll
                        for (uint32_t z = 0; z < 8; ++z)
                            v[j][z] = first + 8 * j < c.rows[q] && z < n && LINEAR_OK(kLinearWorkspace, from + z, 4) ? from[z] : 0.0f;
                    }
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j)
#pragma unroll
                        for (uint32_t z = 0; z < 8; ++z) sum[z] += v[j][z];
                }
            } else {
                for (uint32_t first = lane / 4; first < c.rows[q]; first += 8 * kSumRows) {
                    Shifted v[kSumRows];
#pragma unroll
                    for (uint32_t j = 0; j < kSumRows; ++j) {
                        const uint16_t *from = static_cast<const uint16_t *>(c.src[q]) + (uint64_t)(first + 8 * j) * cols + e;
                        const bool there = first + 8 * j < c.rows[q] && n && LINEAR_OK(kLinearDy + q, from, 2 * n);
                        v[j].load(from, there ? n : 0);
                    }
#pragma unroll
                    for (uint32_t j = 0; j < kSumRows; ++j) {
                        uint32_t w[4];
                        v[j].get(w);
#pragma unroll
                        for (uint32_t z = 0; z < 8; ++z) sum[z] += z & 1 ? bf16_hi(w[z / 2]) : bf16_lo(w[z / 2]);
                    }
                }
            }
        }
#pragma unroll
        for (uint32_t o = 4; o < 32; o *= 2)
#pragma unroll
            for (int z = 0; z < 8; ++z) sum[z] += __shfl_xor_sync(0xFFFFFFFFu, sum[z], o);
        if (lane < 4)
#pragma unroll
            for (int z = 0; z < 8; ++z)
                if (e + z < cols && LINEAR_OK(kLinearDb + k, c.out[k] + e + z, 2)) c.out[k][e + z] = f32_to_bf16(sum[z]);
    }
}

template <int KIND, int CG, uint32_t FW>
__global__ void __cluster_dims__(CG, 1, 1) __launch_bounds__(tc_threads(is_back(KIND), FW), 1)
linear_kernel(const __grid_constant__ LinearParams p)
{
    using First = Roles<KIND, false>;
    using Second = Roles<KIND, is_back(KIND)>;
    constexpr bool kBack = is_back(KIND);
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const uint32_t ring = smem_addr(smem);
    unsigned char *out_buf = smem + kRingBytes;
    unsigned char *ctl = out_buf + kOutBytes;
    const uint32_t bars = smem_addr(ctl);
    const uint32_t full = bars, empty = bars + 8 * kMaxStages;         // stage loaded; stage consumed
    const uint32_t acc_full = bars + 16 * kMaxStages, acc_empty = acc_full + 16, drained = acc_empty + 16;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(ctl + kBarBytes - 8);
    volatile uint32_t *gave_up = tmem_slot + 1;
    static_assert(16 * kMaxStages + 40 <= kBarBytes - 8, "room for the barriers");
    // (the shuffle tells the compiler that a warp is one's whole)
    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t half = CG == 2 ? cluster_rank() : 0;                // of the tile's rows
    const uint32_t worker = blockIdx.x / CG, workers = gridDim.x / CG;

    DT_TL_BEGIN();
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < p.stages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (uint32_t s = 0; s < 2; ++s) {
            mbar_init(acc_full + 8 * s, 1);
            mbar_init(acc_empty + 8 * s, FW * CG);
        }
        mbar_init(drained, 1);
        *gave_up = 0;
        mbar_init_fence();
    }
    Tile t;
    const bool any = next_tile<KIND>(p, worker, workers, 0, t);
    if (warp == FW + 1) tmem_alloc<CG>(smem_addr(const_cast<uint32_t *>(tmem_slot)), kTmemColumns);
    tc_fence_before();
    __syncwarp();
    if (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
    pdl_begin();
    DT_TL_WAITED();
    const Waits wait{p.sink, gave_up};
    const uint32_t a_box = a_box_bytes(kBack, p.rows_t), block_bytes = stage_size(kBack, p.rows_t, p.bn / CG);

    // The loads' and the products' warps walk over them whole, and an elected lane issues:
    // issued by one lane of divergent code a stage of four products took 420 cycles, so 330
    // (512 tokens of 1024 to 4096: 9.9 -> 8.7 us).
    if (warp == FW) {
        uint32_t n = 0, s = 0, round = 0;   // loads issued; the next one's stage and its parity
        bool ok = any;
        for (uint32_t k = 1; ok; ok = ok && next_tile<KIND>(p, worker, workers, k++, t)) {
            if (kBack && t.second)
                ok = load_tile<Second, CG>(p, p.product[1], t, half, ring, block_bytes, a_box, full, empty, wait, s, round, n);
            else
                ok = load_tile<First, CG>(p, p.product[0], t, half, ring, block_bytes, a_box, full, empty, wait, s, round, n);
        }
        // leave nothing in flight: the stages are consumed or, where that
        // was given up, at least loaded (a pair's loads complete on its
        // first CTA's barriers, and neither CTA leaves before the other)
        if (lane == 0)
            for (uint32_t k = n > p.stages ? n - p.stages : 0; k < n; ++k) {
                const uint32_t at = k % p.stages, parity = (k / p.stages) & 1;
                if ((*gave_up || !wait(empty + 8 * at, parity)) && half == 0) wait(full + 8 * at, parity);
            }
        __syncwarp();
    } else if (warp == FW + 1) {
        if (half == 0) {
            uint32_t s = 0, round = 0;
            bool ok = true;
            bool more = any;
            for (uint32_t u = 0; ok && more; more = next_tile<KIND>(p, worker, workers, ++u, t)) {
                const uint32_t acc = tmem + (u & 1) * 256;
                if (!(ok = __all_sync(0xFFFFFFFFu, wait(acc_empty + 8 * (u & 1), ((u >> 1) & 1) ^ 1)))) break;
                tc_fence_after();
                if (kBack && t.second)
                    ok = multiply_tile<Second, CG>(p, p.product[1], t, acc, ring, block_bytes, a_box, full, empty, wait, s,
                                                   round);
                else
                    ok = multiply_tile<First, CG>(p, p.product[0], t, acc, ring, block_bytes, a_box, full, empty, wait, s,
                                                  round);
                if (ok && elect_one()) mma_commit<CG>(acc_full + 8 * (u & 1));
            }
            if (!ok) {   // the MMAs issued so far end before tensor memory is freed
                if (elect_one()) mma_commit<CG>(drained);
                wait(drained, 0);
            }
        }
        __syncwarp();
    } else if (kBack && warp >= FW + 2) {
        column_sums(p, blockIdx.x * kSumWarps + warp - FW - 2, gridDim.x * kSumWarps);
    } else {
        // Warps w, w + 4, ... read the same 32 rows (a warp reaches the tensor memory
        // lanes of its number modulo 4) and take columns in turn.
        const uint32_t quad = (warp & 3) * 32;   // first of this warp's rows in the CTA's
        unsigned char *buf = out_buf + warp * kStageOut, *biases = ctl + kBarBytes + warp * kStep * 2;
        bool more = any;
        for (uint32_t u = 0; more; more = next_tile<KIND>(p, worker, workers, ++u, t)) {
            const uint32_t acc = tmem + (u & 1) * 256 + ((warp & 3) * 32 << 16);
            auto take = [&] {
                const bool ok = wait(acc_full + 8 * (u & 1), (u >> 1) & 1);
                tc_fence_after();
                return !__any_sync(0xFFFFFFFFu, !ok);
            };
            auto give_back = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2) mbar_arrive_first(acc_empty + 8 * (u & 1));
                    else mbar_arrive(acc_empty + 8 * (u & 1));
                }
            };
            const bool ok = kBack && t.second
                                ? finish_tile<KIND, FW, Second>(p, p.product[1], t, acc, t.m * CG + half, p.product[1].mt * CG, quad,
                                                            warp >> 2, buf, biases, take, give_back)
                                : finish_tile<KIND, FW, First>(p, p.product[0], t, acc, t.m * CG + half, p.product[0].mt * CG, quad,
                                                           warp >> 2, buf, biases, take, give_back);
            if (!ok) break;
        }
    }
    tc_fence_before();
    __syncwarp();
    if (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    if (warp == FW + 1) tmem_free<CG>(tmem, kTmemColumns);
    DT_TL_END_BLOCK(DT_TL_LINEAR);
}

// The sums of a product's splits into one, four columns a thread, and what follows
// a sum.  A row of blocks to a row of the output.
template <int KIND, bool SECOND>
__global__ void __launch_bounds__(kThreads) linear_join_kernel(const __grid_constant__ LinearParams p)
{
    using R = Roles<KIND, SECOND>;
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    const LinearProduct &c = p.product[SECOND];
    const uint32_t pitch = c.nt * p.bn, col = (blockIdx.x * kThreads + threadIdx.x) * 4;
    if (col < pitch) {
        const Place m = locate<R, R::m>(p, c, blockIdx.y / kM, kM), n = locate<R, R::n>(p, c, col / p.bn, p.bn);
        const uint32_t row = blockIdx.y % kM, len = length<R, R::m>(p, m.piece), rows = m.at < len ? len - m.at : 0;
        const uint32_t e = col % p.bn, cols = length<R, R::n>(p, n.piece) - n.at;
        if (row < rows && e < cols) {
            const float4 *from = reinterpret_cast<const float4 *>(c.acc + (uint64_t)blockIdx.y * pitch + col);
            const uint64_t step = (uint64_t)gridDim.y * pitch / 4;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
            for (uint32_t k = 0; k < c.splits; ++k)
                if (LINEAR_OK(kLinearWorkspace, from + k * step, 16)) {
                    const float4 f = from[k * step];
                    v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
                }
            const OutRow o = out_row<R>(p, c, m, n, row);
            constexpr int kOut = !is_back(KIND) ? kLinearY : SECOND ? kLinearDw : kLinearDx;
            const uint32_t r = KIND == kGather ? n.piece : 0;
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                if (e + j >= cols) break;
                const uint64_t at = o.offset + e + j;
                if (!is_back(KIND) && p.biased && LINEAR_OK(kLinearBias + r, p.bias[r] + n.at + e + j, 2))
                    v[j] += bf16_to_f32(p.bias[r][n.at + e + j]);
                if (KIND == kReduce && p.residuals && LINEAR_OK(kLinearResidual + o.rank, p.residual[o.rank] + at, 2))
                    v[j] += bf16_to_f32(p.residual[o.rank][at]);
                if (KIND == kGather && p.keep && LINEAR_OK(kLinearPre + o.rank, p.pre[o.rank] + at, 2))
                    p.pre[o.rank][at] = f32_to_bf16(v[j]);
            }
            if (KIND == kGather) activate(v, p.act);
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                const uint64_t at = o.offset + e + j;
                if (e + j < cols && LINEAR_OK(kOut + o.rank, o.out + at, 2)) o.out[at] = f32_to_bf16(v[j]);
            }
        }
    }
    DT_TL_END_BLOCK(DT_TL_LINEAR);
}

// A strip of 256 columns of a chunk of rows to a block: 32 threads across, eight columns
// each, and eight rows at a time, two or four of them under way for each thread.
template <bool VEC, bool PRE>
__device__ __forceinline__ void prep_rows(const LinearPrep &p, const LinearPrepJob &job, uint32_t first, uint32_t end, uint32_t e,
                                          float (&sum)[8])
{
    constexpr uint32_t kBatch = !VEC && PRE ? 2 : 4;
    const uint32_t n = e < job.cols ? min(job.cols - e, 8u) : 0;
    auto load = [&](const uint16_t *base, uint32_t row, int buffer, Eight<VEC> &v) {
        (void)buffer;
        const uint16_t *at = base + (uint64_t)row * job.cols + e;
        v.load(at, row < end && n && LINEAR_OK(buffer, at, 2 * n) ? n : 0);
    };
#pragma unroll 1
    for (uint32_t row0 = first + threadIdx.x / 32; row0 < end; row0 += 8 * kBatch) {
        Eight<VEC> src[kBatch], pre[PRE ? kBatch : 1];
#pragma unroll
        for (uint32_t k = 0; k < kBatch; ++k) {
            load(job.src, row0 + 8 * k, job.src_buffer, src[k]);
            if (PRE) load(job.pre, row0 + 8 * k, job.pre_buffer, pre[PRE ? k : 0]);
        }
#pragma unroll
        for (uint32_t k = 0; k < kBatch; ++k) {
            const uint32_t row = row0 + 8 * k;
            if (row >= end) break;
            uint32_t w[4];
            src[k].get(w);
            if (PRE || job.sums) {
                float g[8];
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) g[j] = j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
                if (PRE) {
                    uint32_t u[4];
                    float z[8];
                    pre[PRE ? k : 0].get(u);
#pragma unroll
                    for (uint32_t j = 0; j < 8; ++j) z[j] = j & 1 ? bf16_hi(u[j / 2]) : bf16_lo(u[j / 2]);
                    times_slope(g, z, p.act);
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) w[j] = pack_bf16x2(g[2 * j], g[2 * j + 1]);
                }
#pragma unroll
                for (uint32_t j = 0; j < 8; j += 2) {
                    const float2 f = add2(make_float2(sum[j], sum[j + 1]), make_float2(g[j], g[j + 1]));
                    sum[j] = f.x, sum[j + 1] = f.y;
                }
            }
            uint4 *to = reinterpret_cast<uint4 *>(job.dst + (uint64_t)row * job.pitch + e);
            if (job.dst && e < job.pitch && LINEAR_OK(kLinearWorkspace, to, 16))
                *to = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

__global__ void __launch_bounds__(kThreads, 3) linear_prep_kernel(const __grid_constant__ LinearPrep p)
{
    __shared__ float part[8][kPrepCols + 4];
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    int k = 0;
    while (k + 1 < p.jobs && blockIdx.x >= p.job[k].block_end) ++k;
    const LinearPrepJob &job = p.job[k];
    const uint32_t block = blockIdx.x - (k ? p.job[k - 1].block_end : 0);
    const uint32_t strip = block % job.strips, chunk = block / job.strips;
    const uint32_t first = chunk * p.chunk_rows, end = min(first + p.chunk_rows, job.rows);
    const uint32_t t = threadIdx.x % 32, e = strip * kPrepCols + t * 8;
    float sum[8] = {};
    if (job.pre && job.vec) prep_rows<true, true>(p, job, first, end, e, sum);
    else if (job.pre) prep_rows<false, true>(p, job, first, end, e, sum);
    else if (job.vec) prep_rows<true, false>(p, job, first, end, e, sum);
    else prep_rows<false, false>(p, job, first, end, e, sum);
    if (job.sums) {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) part[threadIdx.x / 32][t * 8 + j] = sum[j];
        __syncthreads();
        const uint32_t c = strip * kPrepCols + threadIdx.x;
        float all = 0.0f;
#pragma unroll
        for (uint32_t r = 0; r < 8; ++r) all += part[r][threadIdx.x];
        float *to = job.sums + (uint64_t)chunk * job.cols + c;
        if (c < job.cols && LINEAR_OK(kLinearWorkspace, to, 4)) *to = all;
    }
    DT_TL_END_BLOCK(DT_TL_LINEAR);
}

template <int KIND, int CG, uint32_t FW>
cudaError_t launch_kind(LinearParams &p, int device, cudaStream_t s)
{
    static std::atomic<uint64_t> ready{0};   // devices whose shared memory limit is set
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (!(ready.load(std::memory_order_acquire) & bit) || !bit) {
        const cudaError_t e = cudaFuncSetAttribute(linear_kernel<KIND, CG, FW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)kTcSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    p.step = !is_back(KIND) && p.bn <= 128 ? 2 : 1;
    p.stages = std::min(kMaxStages, kRingBytes / (p.step * stage_size(is_back(KIND), p.rows_t, p.bn / CG)));
    return launch_kernel(linear_kernel<KIND, CG, FW>, dim3(p.workers * CG), dim3(tc_threads(is_back(KIND), FW)), kTcSmem, s,
                         false, p);
}

template <int KIND>
cudaError_t launch_kind(LinearParams &p, bool pairs, int device, cudaStream_t s)
{
    if constexpr (KIND == kGather)
        if (p.product[0].kblocks <= kShortBlocks && p.act != DT_ACT_NONE && p.product[0].tiles > 2 * p.workers)
            return pairs ? launch_kind<KIND, 2, 16>(p, device, s) : launch_kind<KIND, 1, 16>(p, device, s);
    return pairs ? launch_kind<KIND, 2, 8>(p, device, s) : launch_kind<KIND, 1, 8>(p, device, s);
}

template <int KIND, bool SECOND>
cudaError_t launch_join(const LinearParams &p, uint32_t high, cudaStream_t s)
{
    const LinearProduct &c = p.product[SECOND];
    return launch_kernel(linear_join_kernel<KIND, SECOND>, dim3((c.nt * p.bn / 4 + kThreads - 1) / kThreads, c.mt * high),
                         dim3(kThreads), 0, s, false, p);
}

}  // namespace

DT_TL_BINDER(bind_timeline_linear)

uint32_t linear_workers(bool pairs, int device) { return (uint32_t)std::max(1, sm_count(device) / (pairs ? 2 : 1)); }

// A finished tile costs a worker about a block of the inner axis more than its
// products.
constexpr uint32_t kTileCost = 1;

cudaError_t launch_linear(LinearParams &p, LinearKind kind, bool pairs, int device, cudaStream_t s)
{
    const uint32_t W = linear_workers(pairs, device);
    const LinearProduct &a = p.product[0], &b = p.product[1];
    const uint32_t second = is_back(kind) ? b.tiles : 0;
    p.workers = std::min(W, a.tiles + second);
    p.rest = p.early = 0;
    if (second && a.tiles % p.workers) {
        p.rest = a.tiles % p.workers;
        p.early = std::min((a.kblocks / a.splits + kTileCost) / (b.kblocks / b.splits + kTileCost), second / (p.workers - p.rest));
    }
    for (LinearProduct &c : p.product) {
        const uint64_t g = (uint64_t)kGroup * c.mt;
        c.group_inverse = g ? (uint32_t)((1ull << 32) / g + 1) : 0;
        c.mt_inverse = c.mt > 1 ? (uint32_t)((1ull << 32) / c.mt + 1) : 0;
    }
    switch (kind) {
    case kGather: return launch_kind<kGather>(p, pairs, device, s);
    case kGatherBack: return launch_kind<kGatherBack>(p, pairs, device, s);
    case kReduce: return launch_kind<kReduce>(p, pairs, device, s);
    default: return launch_kind<kReduceBack>(p, pairs, device, s);
    }
}

cudaError_t launch_linear_join(const LinearParams &p, LinearKind kind, int k, bool pairs, cudaStream_t s)
{
    const uint32_t high = pairs ? 2 * kM : kM;
    switch (kind) {
    case kGather: return launch_join<kGather, false>(p, high, s);
    case kGatherBack: return k ? launch_join<kGatherBack, true>(p, high, s) : launch_join<kGatherBack, false>(p, high, s);
    case kReduce: return launch_join<kReduce, false>(p, high, s);
    default: return k ? launch_join<kReduceBack, true>(p, high, s) : launch_join<kReduceBack, false>(p, high, s);
    }
}

cudaError_t launch_linear_prep(LinearPrep &p, cudaStream_t s)
{
    return launch_kernel(linear_prep_kernel, dim3(p.job[p.jobs - 1].block_end), dim3(kThreads), 0, s, false, p);
}

}  // namespace dt
