// Softmax cross entropy of tokens under a vocabulary whose rows are split over
// the ranks, without ever holding the logits, and its gradient.
//
//   l_tv = <h_t, w_v>      lse_t = log sum_v exp(l_tv)      loss_t = lse_t - l_t,target
//   g_tv = s (exp(l_tv - lse_t) - [v = target_t])    dh_t = sum_v g_tv w_v    dw_v = sum_t g_tv h_t
//
// Each of these is a product on the tensor cores, and one persistent kernel
// serves all (Mode): tiles of 128 x bn outputs, or of 256 x bn for two CTAs of
// a cluster, operands brought by TMA into a ring of shared memory stages by
// one thread, multiplied by one thread that issues tcgen05.mma into tensor
// memory, and finished by 8 or 16 warps that read the accumulator while the
// next tile's is being made in the other half of tensor memory.
//   kLse   logits; the finish reduces a tile's columns to a maximum and a
//          sum of exponentials for each token: 8 bytes for 256 logits.
//   kGrad  the same logits again (kGradLong: as sums of several accumulators);
//          the finish makes p - [target] and stores it as bf16 for a piece of
//          the vocabulary at a time.  That is the one
//          rounding on the way (2^-8 of each term at most, as the outputs'
//          own): the two products below need it in the operands' type.  The
//          scale s is applied to their fp32 sums.
//   kBack  dh, the piece's g times its rows of w, and dw, the piece's g
//          transposed times h, in one launch: a tile of dh takes as long as
//          many of dw, so the tiles of dw fill what dh leaves of the last wave.
//          dw is final for these rows of w.  dh over several pieces, or when
//          the vocabulary is split over blocks because there are few tokens,
//          stays in fp32 and is joined in a fixed order.  These sums, over a
//          piece of the vocabulary or all tokens, stay in one accumulator, which
//          cuts off up to 3e-8 of its value at each step of 16: 3e-4 of 131072
//          terms of one sign, where bf16 results are rounded by up to 4e-3.
// A pair of CTAs halves what each reads of B, so that L2 feeds a third less.
// It takes 256 rows of A, so up to 128 tokens a CTA works alone, on tiles of at
// most 128 columns, and loads only the rows there are of A: for one token 128
// KB of w are under way at a time, in eight stages, instead of 64 in four.
// A stage is 128 deep: four TMA boxes of 16 KB, which the
// copy engine serves faster than eight of 8 KB (2048 tokens of 32768 x 4096:
// 397 -> 328 us).
// Rank boundaries are no more than an offset: the ranks' rows are numbered
// through in units of 256 (the last unit of a rank is padded by zeros that TMA
// fills in), so the reductions over the ranks (of the maximum, the sum and dh)
// are the sums over units.
//
// Where dim is small the finish bounds the logits, not their products: below
// about 400 a tile of 256 x 256 takes the finishing warps 4000 cycles, half of
// which issue instructions (8192 tokens of 65536 x 256: 231 us, of which the
// products need 144).
//
// With n tokens the work is 2 n flops for each byte of w: below about 280
// tokens HBM bounds it, above it the tensor cores do.
#include <cudaTypedefs.h>

#include <algorithm>

#include "dt_ops.h"

#include "dt_bounds.cuh"
#include "dt_device.cuh"
#include "dt_math.cuh"
#include "dt_tc.cuh"
#include "dt_timeline.cuh"
#include "dt_vocab.h"

namespace dt {
namespace {

enum Mode { kLse, kGrad, kGradLong, kBack };

constexpr float kLog2e = 1.44269504088896340736f;

constexpr uint32_t kM = 128;                       // rows of a tile in a CTA
constexpr uint32_t kK = 128;                       // depth of a stage
constexpr uint32_t kRingBytes = 192 * 1024;        // three stages of 128 rows and columns of A and B
constexpr uint32_t kMaxStages = 8;
// The logits: blocks of the inner dimension whose sum the tensor cores make; the
// sums of further ones are added in registers.  The tensor cores round towards
// zero at every step of 16: whole sums of 4096 products came out 4e-6 of
// themselves too small, and losses 8e-7 off; with sums of 1024 that is 9e-7 and
// 2e-7, for 2% of the time (2048 tokens of 32768 x 4096: 332 -> 338 us).  The
// gradient's logits are summed alike, for up to 1% (2048 x 32768 x 4096: 977 ->
// 986 us): p is exp(l - lse), and with other logits than lse was made of, p - 1 of
// a confident token was mostly their difference (at 4096 columns, a logit of 17.5
// and p = 1 - 8e-5 1 - p came out 3.6 times as large; now 0.7% off, bf16's rounding
// and lse's own).
constexpr uint32_t kSumBlocks = 8;
constexpr uint32_t kTmemColumns = 512;             // two accumulators of 128 x 256 fp32
// Finishing warps: of logits that are only reduced 16, each with 64 columns of a
// tile in registers; else 8 with 128.  And one for TMA, one for the products,
// and the gradient's one for the tokens' count.
__host__ __device__ constexpr uint32_t finish_warps(int mode) { return mode == kLse ? 16 : 8; }
__host__ __device__ constexpr int tc_threads(int mode) { return (finish_warps(mode) + (mode == kGrad || mode == kGradLong ? 3 : 2)) * 32; }
constexpr uint32_t kJoins = 3;                     // tiles whose column groups' results there is room for
constexpr uint32_t kStageOut = 4096;               // a finishing warp's 32 rows x 128 bytes
constexpr uint32_t kBarBytes = 1024;
constexpr uint32_t kOutBytes = 8 * kStageOut;      // or kLse: 3 tiles x 4 column groups x 128 rows x 8 bytes
constexpr size_t kTcSmem = 1024 + kRingBytes + kOutBytes + kBarBytes;
static_assert(kTcSmem <= 227 * 1024, "shared memory above the per-block limit");

// Where a tile's operands and outputs are.
struct Tile {
    bool dw;             // kBack: a tile of dw, not of dh
    uint32_t m0, n0;     // first row and column of the output
    uint32_t kb0, kb1;   // blocks of 128 of the inner dimension
    uint32_t split;
    int r;               // rank and row there of the vocabulary rows that the tile covers (logits: n; dw: m)
    uint32_t vrow;
};

// n / d, where `inverse` is the least whole number above 2^32 / d (0 for 1): the
// product's high word is at most one too large.
__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t d, uint32_t inverse)
{
    if (d == 1) return n;
    const uint32_t q = __umulhi(n, inverse);
    return q * d > n ? q - 1 : q;
}

// The rank of a unit of 256 vocabulary rows, and the unit's first row there.
__device__ __forceinline__ int unit_rank(const VocabParams &p, uint32_t unit, uint32_t &row)
{
    int r = 0;
    uint32_t begin = 0;
    while (r + 1 < p.P && unit >= p.unit_end[r]) begin = p.unit_end[r++];
    row = (unit - begin) * kVocabUnit;
    return r;
}

// The k-th tile of worker q (a CTA or a pair) of W; false when it has no more.
// Logits: tile q + k W, columns in groups of 16, rows slowest within a group,
// so that the tiles in flight share few rows and columns and their operands
// come from L2.
// kBack: first the tiles of dh, one by one to the workers.  While the first
// dh_rest workers still have one more of them, the others take dw_early tiles
// of dw each; then all take the rest of dw in turn.
template <int MODE, int CG>
__device__ __forceinline__ bool next_tile(const VocabParams &p, uint32_t q, uint32_t W, uint32_t k, Tile &t)
{
    uint32_t i, width;
    t.dw = false;
    t.split = 0;
    t.r = 0;
    t.vrow = 0;
    if (MODE != kBack) {
        i = q + k * W;
        if (i >= p.tiles) return false;
        const uint32_t all = p.group * p.mt, g = quotient(i, all, p.per_group);
        i -= g * all;
        width = min(p.group, p.nt - g * p.group);
        const uint32_t m = quotient(i, width, width == p.group ? p.per_row : p.per_last);
        t.m0 = m * (kM * CG);
        t.n0 = (g * p.group + i - m * width) * p.bn;
        t.kb0 = 0;
        t.kb1 = p.kblocks;
        t.r = unit_rank(p, p.unit0 + t.n0 / kVocabUnit, t.vrow);
        t.vrow += t.n0 % kVocabUnit;
        return true;
    }
    const uint32_t mine = q < p.tiles ? (p.tiles - q + W - 1) / W : 0;   // tiles of dh
    if (k < mine) {
        i = q + k * W;
        const uint32_t per_split = p.mt * p.nt;
        t.split = i / per_split;
        i -= t.split * per_split;
        t.m0 = i / p.nt * (kM * CG);
        t.n0 = i % p.nt * p.bn;
        t.kb0 = (uint32_t)((uint64_t)p.kblocks * t.split / p.splits);
        t.kb1 = (uint32_t)((uint64_t)p.kblocks * (t.split + 1) / p.splits);
        return true;
    }
    k -= mine;
    const uint32_t others = W - p.dh_rest;
    if (q >= p.dh_rest && k < p.dw_early) {
        i = q - p.dh_rest + k * others;
    } else {
        if (q >= p.dh_rest) k -= p.dw_early;
        i = p.dw_early * others + k * W + (q >= p.dh_rest ? q - p.dh_rest : q + others);
    }
    if (i >= p.dw_tiles) return false;
    t.dw = true;
    t.m0 = i / p.nt * (kM * CG);
    t.n0 = i % p.nt * p.bn;
    t.kb0 = 0;
    t.kb1 = p.dw_kblocks;
    t.r = unit_rank(p, p.unit0 + t.m0 / kVocabUnit, t.vrow);
    t.vrow += t.m0 % kVocabUnit;
    return true;
}

// Vocabulary rows of rank r from `row` on that exist, at most `most`.
__device__ __forceinline__ uint32_t rows_left(const VocabParams &p, int r, uint32_t row, uint32_t most)
{
    return row >= p.rows[r] ? 0 : min(p.rows[r] - row, most);
}

// What a CTA's loads of a tile have in common, worked out once a tile.  The
// inner dimension is the column of a K-major operand and the row of an
// MN-major one.  An operand is two boxes of as many rows as its map says, but
// columns of B past the width of w or h are not loaded.  What a stage holds
// beside its boxes is left over from earlier loads and reaches only rows and
// columns of the accumulator that are not stored.
struct Loads {
    const CUtensorMap *a, *b;
    uint32_t nb, bytes;              // boxes of B; bytes of both CTAs
    uint32_t am, bn;                 // first row or column along M and N
};

template <int MODE, int CG>
__device__ __forceinline__ Loads tile_loads(const VocabParams &p, const Tile &t, uint32_t half)
{
    Loads l;
    const uint32_t bn = p.bn / CG;   // columns of B in a CTA
    l.am = t.m0 + half * kM;
    l.bn = half * bn;
    if (MODE != kBack) {
        l.a = &p.h;
        l.b = &p.w[p.packed ? 0 : t.r];
        l.bn += p.packed ? t.n0 : t.vrow;
        l.nb = 2;
        l.bytes = CG * 2 * (p.rows_h + p.rows_w) * 128;
    } else {
        l.a = &p.g;
        l.b = &p.h;
        l.bn += t.n0;
        l.nb = l.bn + 64 < p.dim ? 2 : 1;
        const uint32_t all = l.nb + (CG == 2 ? (t.n0 + (half ^ 1) * bn + 64 < p.dim ? 2 : 1) : 0);
        l.bytes = (CG * 2 * p.rows_g + all * (t.dw ? p.rows_h : p.rows_w)) * 128;
    }
    return l;
}

// a_box: from operand A's first box to its second.
template <int MODE, int CG>
__device__ __forceinline__ void load_stage(const VocabParams &p, const Tile &t, Loads &l, uint32_t half, uint32_t kb,
                                           uint32_t a, uint32_t a_box, uint32_t bar)
{
    const uint32_t b = a + 2 * a_box, k = kb * kK;
    if (half == 0) mbar_expect_tx(bar, l.bytes);
    if (MODE != kBack) {
        tma_box<CG>(a, l.a, k, l.am, bar);
        tma_box<CG>(b, l.b, k, l.bn, bar);
        tma_box<CG>(a + a_box, l.a, k + 64, l.am, bar);
        tma_box<CG>(b + p.rows_w * 128, l.b, k + 64, l.bn, bar);
        return;
    }
    uint32_t row = k;
    if (!t.dw) {
        tma_box<CG>(a, l.a, k, l.am, bar);
        tma_box<CG>(a + a_box, l.a, k + 64, l.am, bar);
        if (!p.packed) {
            const int r = unit_rank(p, p.unit0 + k / kVocabUnit, row);
            row += k % kVocabUnit;
            l.b = &p.w[r];
        } else {
            l.b = &p.w[0];
        }
    } else {
        tma_box<CG>(a, l.a, l.am, k, bar);
        tma_box<CG>(a + a_box, l.a, l.am + 64, k, bar);
    }
    tma_box<CG>(b, l.b, l.bn, row, bar);
    if (l.nb == 2) tma_box<CG>(b + kBoxBytes, l.b, l.bn + 64, row, bar);
}

// A finishing warp's 32 rows x 128 bytes in shared memory, 16-byte chunk c of
// row r at chunk c ^ (r mod 8): a thread writes its row, and eight threads
// read a row, without bank conflicts.
__device__ __forceinline__ uint4 *out_chunk(unsigned char *buf, uint32_t row, uint32_t c)
{
    return reinterpret_cast<uint4 *>(buf + row * 128 + ((c ^ (row & 7)) << 4));
}

#define VOCAB_OK(buffer, a, n) DT_IN_EXTENT(p, kBoundsVocab, (buffer), (a), (n))

// One instruction's worth of a row: N 16-bit elements.
template <int N> struct Words;
template <> struct Words<8> { using type = uint4; };
template <> struct Words<4> { using type = uint2; };
template <> struct Words<2> { using type = uint32_t; };

// A warp's rows from `buf` to memory, N elements of a row to a lane and as
// many rows at a time as that leaves lanes for.
template <int N>
__device__ __forceinline__ void store_rows(const VocabParams &p, const unsigned char *buf, uint16_t *out, uint64_t pitch,
                                           uint32_t rows, uint32_t cols, int buffer)
{
    using W = typename Words<N>::type;
    (void)p, (void)buffer;
    constexpr uint32_t kLanes = 64 / N, kRows = 32 / kLanes;
    const uint32_t lane = threadIdx.x & 31, e = lane % kLanes * N, first = lane / kLanes;
    if (e >= cols) return;
#pragma unroll 8
    for (uint32_t k = 0; k < 32; k += kRows) {
        const uint32_t row = k + first;
        const W v = *reinterpret_cast<const W *>(buf + row * 128 + ((((e >> 3) ^ row) & 7) << 4) + (e & 7) * 2);
        uint16_t *to = out + row * pitch + e;
        if (row < rows && VOCAB_OK(buffer, to, 2 * N)) *reinterpret_cast<W *>(to) = v;
    }
}

// The same for rows of an odd width, every other one of which starts between
// two words: a lane's word is then made of its neighbour's halves.  The first
// element of such a row, and a last one that no word takes, go afterwards, a
// row to a lane.
__device__ __forceinline__ void store_rows_odd(const VocabParams &p, const unsigned char *buf, uint16_t *out,
                                               uint64_t pitch, uint32_t rows, uint32_t cols, int buffer)
{
    (void)p, (void)buffer;
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t odd0 = (uint32_t)(reinterpret_cast<uintptr_t>(out) >> 1) & 1, odd_step = (uint32_t)pitch & 1;
    uint16_t *at = out + 2 * lane;
    uint32_t odd = odd0;
#pragma unroll 8
    for (uint32_t row = 0; row < 32; ++row, at += pitch, odd ^= odd_step) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(buf + row * 128 + ((((lane >> 2) ^ row) & 7) << 4) +
                                                               (lane & 3) * 4);
        const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, w, 1);
        uint16_t *to = at + odd;
        if (row < rows && 2 * lane + odd + 1 < cols && VOCAB_OK(buffer, to, 4))
            *reinterpret_cast<uint32_t *>(to) = odd ? __funnelshift_r(w, next, 16) : w;
    }
    if (lane >= rows) return;
    auto element = [&](uint32_t e) {
        const uint16_t v = *reinterpret_cast<const uint16_t *>(buf + lane * 128 + ((((e >> 3) ^ lane) & 7) << 4) + (e & 7) * 2);
        uint16_t *to = out + lane * pitch + e;
        if (VOCAB_OK(buffer, to, 2)) *to = v;
    };
    odd = odd0 ^ (odd_step & lane);
    if (odd) element(0);
    if ((cols - odd) & 1) element(cols - 1);
}

// 64 columns of bf16, packed two to a word: this thread's row into `buf`,
// then the warp's rows to memory in the widest words that their alignment
// allows (2 * align bytes).  Element by element a tile of dw 500 columns wide
// took 9700 cycles, against 1000 of its products.
__device__ __forceinline__ void store_rows_bf16(const VocabParams &p, unsigned char *buf, const uint32_t (&w)[32],
                                                uint16_t *out, uint64_t pitch, uint32_t rows, uint32_t cols,
                                                uint32_t align, int buffer)
{
    const uint32_t lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (uint32_t c = 0; c < 8; ++c)
        *out_chunk(buf, lane, c) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    __syncwarp();
    if (align == 8) store_rows<8>(p, buf, out, pitch, rows, cols, buffer);
    else if (align == 4) store_rows<4>(p, buf, out, pitch, rows, cols, buffer);
    else if (align == 2) store_rows<2>(p, buf, out, pitch, rows, cols, buffer);
    else store_rows_odd(p, buf, out, pitch, rows, cols, buffer);
}

// From operand A's first box to its second: K-major boxes of few tokens' rows
// lie closer, MN-major ones are a fixed way apart.
__host__ __device__ constexpr uint32_t a_box_bytes(bool back, uint32_t rows)
{
    return back ? kBoxBytes : (rows * 128 + 1023) / 1024 * 1024;
}

// A sum of exponentials relative to m, relative to `most` >= m.  No mass is
// left of minus infinities, but a NaN in a sum stays.
__device__ __forceinline__ float scaled(float m, float x, float most)
{
    return x * (m == -INFINITY ? 0.0f : exp2_fast((m - most) * kLog2e));
}

// A maximum and a sum relative to it, and another such pair, into one.
__device__ __forceinline__ void join(float &top, float &sum, float2 v)
{
    const float most = fmaxf(top, v.x);
    sum = scaled(top, sum, most) + scaled(v.x, v.y, most);
    top = most;
}

// The state of the pipeline's waits: a wait that runs out is recorded once,
// and every role then leaves its loop.
struct Waits {
    const ErrorSink &sink;
    volatile uint32_t *gave_up;
    // The timer is read only after 64 tries, each of which waits a while in the
    // hardware: reading it on every wait cost a fifth of the time (2048 tokens of 32768 x 4096: 501 -> 397 us).
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const
    {
        for (int k = 0; k < 64; ++k)
            if (mbar_try_wait(bar, parity)) return true;
        return slow(bar, parity);
    }
    __device__ __noinline__ bool slow(uint32_t bar, uint32_t parity) const
    {
        const uint64_t t0 = global_ns();
        do {
            for (int k = 0; k < 64; ++k)
                if (mbar_try_wait(bar, parity)) return true;
        } while (global_ns() - t0 <= sink.timeout_ns);
        *gave_up = 1;
        record_error(sink, DT_ERR_TIMEOUT, -1, blockIdx.x, 0);
        return false;
    }
};

template <int MODE, int CG>
__global__ void __cluster_dims__(CG, 1, 1) __launch_bounds__(tc_threads(MODE), 1)
vocab_kernel(const __grid_constant__ VocabParams p)
{
    constexpr uint32_t kFinishWarps = finish_warps(MODE);
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const uint32_t ring = smem_addr(smem);
    unsigned char *out_buf = smem + kRingBytes;
    unsigned char *ctl = out_buf + kOutBytes;
    const uint32_t bars = smem_addr(ctl);
    const uint32_t full = bars, empty = bars + 8 * kMaxStages;         // stage loaded; stage consumed
    const uint32_t acc_full = bars + 16 * kMaxStages, acc_empty = acc_full + 16, drained = acc_empty + 16;
    const uint32_t reduced = drained + 8;                              // kLse: the column groups' results are there,
    const uint32_t joined = reduced + 8 * kJoins;                      // and have been read
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(ctl + 256);
    volatile uint32_t *gave_up = tmem_slot + 1;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
            mbar_init(acc_empty + 8 * s, kFinishWarps * CG);
        }
        mbar_init(drained, 1);
        for (uint32_t s = 0; MODE == kLse && s < kJoins; ++s) {
            mbar_init(reduced + 8 * s, kFinishWarps - 4);
            mbar_init(joined + 8 * s, 4);
        }
        *gave_up = 0;
        mbar_init_fence();
    }
    if (warp == kFinishWarps) {
        if (lane < DT_MAX_RANKS && p.w_maps >> lane & 1) tma_prefetch_map(&p.w[lane]);
        if (lane == DT_MAX_RANKS) tma_prefetch_map(&p.h);
        if (MODE == kBack && lane == DT_MAX_RANKS + 1) tma_prefetch_map(&p.g);
    }
    if (warp == kFinishWarps + 1) tmem_alloc<CG>(smem_addr(const_cast<uint32_t *>(tmem_slot)), kTmemColumns);
    tc_fence_before();
    __syncwarp();
    if (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Tile t;
    pdl_begin();
    DT_TL_WAITED();
    const Waits wait{p.sink, gave_up};
    const uint32_t a_box = a_box_bytes(MODE == kBack, p.rows_h), stage_bytes = 2 * a_box + p.bn / CG * 256;

    if (warp == kFinishWarps) {
        if (lane == 0) {
            if (MODE == kLse && blockIdx.x == 0 && VOCAB_OK(kVocabWorkspace, p.ticket, 4)) *p.ticket = 0;   // for the kernel that joins the partial sums
            uint32_t n = 0, s = 0, round = 0;   // loads issued; the next one's stage and its parity
            bool ok = true;
            for (uint32_t k = 0; ok && next_tile<MODE, CG>(p, worker, workers, k, t); ++k) {
                Loads l = tile_loads<MODE, CG>(p, t, half);
                for (uint32_t kb = t.kb0; kb < t.kb1; ++kb, ++n) {
                    if (!(ok = wait(empty + 8 * s, round ^ 1))) break;
                    load_stage<MODE, CG>(p, t, l, half, kb, ring + s * stage_bytes, a_box, full + 8 * s);
                    if (++s == p.stages) s = 0, round ^= 1;
                }
            }
            // leave nothing in flight: the stages are consumed or, where that
            // was given up, at least loaded (a pair's loads complete on its
            // first CTA's barriers, and neither CTA leaves before the other)
            for (uint32_t k = n > p.stages ? n - p.stages : 0; k < n; ++k) {
                const uint32_t at = k % p.stages, parity = (k / p.stages) & 1;
                if ((*gave_up || !wait(empty + 8 * at, parity)) && half == 0) wait(full + 8 * at, parity);
            }
        }
        __syncwarp();
    } else if (warp == kFinishWarps + 1) {
        if (lane == 0 && half == 0) {
            uint32_t s = 0, round = 0, u = 0;   // u: accumulators handed over
            bool ok = true;
            for (uint32_t i = 0; ok && next_tile<MODE, CG>(p, worker, workers, i, t); ++i) {
                const bool a_mn = MODE == kBack && t.dw;
                constexpr bool b_mn = MODE == kBack;
                const uint32_t desc = mma_desc(kM * CG, p.bn, a_mn, b_mn);
                // from a K step of 16 to the next: 16 rows of an MN-major box;
                // 32 bytes of a K-major one, and from its fourth to the next box
                const uint32_t a_step = a_mn ? 16 * 128 : 32, a_next = a_mn ? 4 * a_step : a_box;
                const uint32_t b_step = b_mn ? 16 * 128 : 32, b_next = b_mn ? 4 * b_step : p.rows_w * 128;
                // K steps of 16 that the last block has
                const uint32_t inner = MODE != kBack ? p.dim : t.dw ? p.tokens : p.kblocks * kK;
                const uint32_t last = min((inner - (t.kb1 - 1) * kK + 15) / 16, 8u);
                for (uint32_t kb = t.kb0; ok && kb < t.kb1; ++u) {
                    const uint32_t first = kb, end = MODE != kBack ? min(kb + kSumBlocks, t.kb1) : t.kb1;
                    const uint32_t acc = tmem + (u & 1) * 256;
                    if (!(ok = wait(acc_empty + 8 * (u & 1), ((u >> 1) & 1) ^ 1))) break;
                    tc_fence_after();
                    for (; kb < end; ++kb) {
                        if (!(ok = wait(full + 8 * s, round))) break;
                        tc_fence_after();
                        const uint32_t at = ring + s * stage_bytes;
                        const uint64_t a = smem_desc(at, a_mn), b = smem_desc(at + 2 * a_box, b_mn);
                        const uint32_t steps = kb + 1 == t.kb1 ? last : 8;
#pragma unroll
                        for (uint32_t k = 0; k < 8; ++k)
                            if (k < steps)
                                mma_bf16<CG>(acc, a + ((k / 4 * a_next + k % 4 * a_step) >> 4),
                                             b + ((k / 4 * b_next + k % 4 * b_step) >> 4), desc, kb != first || k != 0);
                        mma_commit<CG>(empty + 8 * s);
                        if (++s == p.stages) s = 0, round ^= 1;
                    }
                    if (ok) mma_commit<CG>(acc_full + 8 * (u & 1));
                }
            }
            if (!ok) {   // the MMAs issued so far end before tensor memory is freed
                mma_commit<CG>(drained);
                wait(drained, 0);
            }
        }
        __syncwarp();
    } else if ((MODE == kGrad || MODE == kGradLong) && warp == kFinishWarps + 2) {
        // how many tokens count: a part of them to a CTA, 256 or more, which kBack adds.
        // (One warp for all tokens, whose loads waited for one another, outlasted the
        // tiles: 65536 tokens of 1000 x 64 910 us; this 355.)
        if (p.unit0 == 0 && blockIdx.x < p.kept_parts) {
            const uint32_t each = (p.tokens + p.kept_parts - 1) / p.kept_parts;
            const uint32_t begin = min(blockIdx.x * each, p.tokens), end = min(begin + each, p.tokens);
            uint32_t kept = 0;
            for (uint32_t first = begin; first < end; first += 256) {
                int32_t v[8];
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const uint32_t k = first + 32 * j + lane;
                    v[j] = k < end && VOCAB_OK(kVocabTargets, p.targets + k, 4) ? p.targets[k] : p.ignore;
                }
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const bool in = v[j] >= 0 && (uint32_t)v[j] < p.vocab;
                    if (v[j] != p.ignore && !in) record_error(p.sink, DT_ERR_INVALID, -1, (int)(first + 32 * j + lane), v[j]);
                    kept += v[j] != p.ignore && in;
                }
            }
            kept = __reduce_add_sync(0xFFFFFFFFu, kept);
            if (lane == 0 && VOCAB_OK(kVocabWorkspace, p.kept + blockIdx.x, 4)) p.kept[blockIdx.x] = kept;
        }
    } else {
        // Warps w, w + 4, ... read the same 32 rows (a warp reaches the tensor
        // memory lanes of its number modulo 4) and take an equal part of the
        // columns each, but for kLse at least 64.
        unsigned char *buf = out_buf + (MODE == kLse ? 0 : warp * kStageOut);
        float scale = 0.0f;
        if (MODE == kBack) {
            const float grad = p.grad && VOCAB_OK(kVocabGrad, p.grad, 4) ? *p.grad : 1.0f;
            uint32_t kept = 0;
#pragma unroll 4
            for (uint32_t k = lane; k < p.kept_parts; k += 32)
                if (VOCAB_OK(kVocabWorkspace, p.kept + k, 4)) kept += p.kept[k];
            kept = __reduce_add_sync(0xFFFFFFFFu, kept);
            scale = kept == 0 ? 0.0f : p.avg ? __fdiv_rn(grad, (float)kept) : grad;
            // for the kernel that joins dh's splits
            if (blockIdx.x == 0 && threadIdx.x == 0 && VOCAB_OK(kVocabWorkspace, p.scale, 4)) *p.scale = scale;
        }
        constexpr uint32_t kParts = kFinishWarps / 4;
        const uint32_t width = MODE == kLse || p.bn >= 128 ? p.bn / kParts : p.bn;
        const uint32_t c0 = (warp >> 2) * width, c1 = min(c0 + width, p.bn);
        bool late = false;
        uint32_t u = 0, j3 = 0, round = 0;   // accumulators taken over; kLse: the next tile's room for results, its parity
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
            ++u;
        };
        for (uint32_t i = 0; next_tile<MODE, CG>(p, worker, workers, i, t); ++i) {
            const uint32_t quad = half * kM + (warp & 3) * 32;   // first of this warp's rows in the tile
            const uint32_t row0 = t.m0 + quad, row = row0 + lane;
            // what does not depend on the accumulator, before the wait for it
            int32_t target = p.ignore;
            float lse = 0.0f;
            if (MODE != kBack && row < p.tokens) {
                if (VOCAB_OK(kVocabTargets, p.targets + row, 4)) target = p.targets[row];
                if (MODE != kLse && VOCAB_OK(kVocabLse, p.lse + row, 4)) lse = p.lse[row];
            }
            const uint32_t lanes = (warp & 3) * 32 << 16;   // of tensor memory
            uint32_t acc = tmem + (u & 1) * 256 + lanes;

            if (MODE != kBack) {
                const uint32_t valid = rows_left(p, t.r, t.vrow, p.bn);
                if (MODE == kLse) {
                    // the logits: one accumulator, or the sum of several.  A wait
                    // that runs out ends no loop here, as all warps meet below:
                    // there are just no more waits.
                    float v[64];
                    if (!late) late = !take();
#pragma unroll
                    for (uint32_t b = 0; b < 64; b += 32)
                        if (b < width) tmem_load32(acc + c0 + b, *reinterpret_cast<float(*)[32]>(v + b));
                    give_back();
                    for (uint32_t kb = t.kb0 + kSumBlocks; kb < t.kb1; kb += kSumBlocks) {
                        if (!late) late = !take();
                        acc = tmem + (u & 1) * 256 + lanes;
#pragma unroll
                        for (uint32_t b = 0; b < 64; b += 8) {
                            if (b >= width) continue;
                            float x[8];
                            tmem_load8(acc + c0 + b, x);
#pragma unroll
                            for (uint32_t j = 0; j < 8; ++j) v[b + j] += x[j];
                        }
                        give_back();
                    }
                    // four running values each, so that none waits for the one before
                    float tops[4];
                    float2 sums[4];
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) tops[j] = -INFINITY, sums[j] = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (uint32_t b = 0; b < 64; b += 16) {
                        if (b >= width) continue;
                        if (c0 + b + 16 > valid) {   // columns that are not there count for nothing
#pragma unroll
                            for (uint32_t j = 0; j < 16; ++j) v[b + j] = c0 + b + j < valid ? v[b + j] : -INFINITY;
                        }
#pragma unroll
                        for (uint32_t j = 0; j < 8; ++j) tops[j & 3] = max3(tops[j & 3], v[b + j], v[b + j + 8]);
                    }
                    float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    // v log2e - top2 is one fma, with top2 the rounded top * log2e: the sum comes
                    // out 2^rest too large, rest being what was rounded off, and is set right
                    // afterwards.  Relative to the maximum it is 1 at least, so that no loss is
                    // below zero.  From 2^30 on, where rest may be more than fp32 has powers for,
                    // it is as good as 1: other logits are 64 away, and the logarithm of how many
                    // are equal is less than half an ulp of them.
                    // (The distance first, then its scale: 8192 tokens of 65536 x 64 223 -> 244 us; this 226.)
                    const float from = top == -INFINITY ? 0.0f : top;   // no infinity from itself where all are -inf
                    const float top2 = from * kLog2e, rest = fmaf(from, kLog2e, -top2);
                    const float2 log2e2 = make_float2(kLog2e, kLog2e), down = make_float2(-top2, -top2);
#pragma unroll
                    for (uint32_t b = 0; b < 64; b += 16) {
                        if (b >= width) continue;
#pragma unroll
                        for (uint32_t j = 0; j < 16; j += 2) {
                            const float2 x = fma2(make_float2(v[b + j], v[b + j + 1]), log2e2, down);
                            sums[j / 2 & 3] = add2(sums[j / 2 & 3], make_float2(exp2_fast(x.x), exp2_fast(x.y)));
                        }
                    }
                    const float2 both = add2(add2(sums[0], sums[1]), add2(sums[2], sums[3]));
                    float sum = both.x + both.y;
                    const float right = fabsf(top) < 1073741824.0f ? sum * exp2_fast(-rest) : 1.0f;
                    sum = sum != sum ? sum : fmaxf(right, 1.0f);
                    // the column of this row's target in the tile, if it is there
                    const int64_t at = (int64_t)target - (int64_t)(p.first[t.r] + t.vrow);
                    const bool here = target != p.ignore && target >= 0 && at >= (int64_t)c0 && at < (int64_t)min(c1, valid);
                    if (__any_sync(0xFFFFFFFFu, here)) {
                        const uint32_t mine = (uint32_t)at - c0;
                        float logit = 0.0f;
#pragma unroll
                        for (uint32_t j = 0; j < 64; ++j)
                            if (j < width) logit = mine == j ? v[j] : logit;
                        if (here && row < p.tokens && VOCAB_OK(kVocabWorkspace, p.logit + row, 4)) p.logit[row] = logit;
                    }
                    // The four column groups' into one by the first warps; the others go on
                    // (with a barrier of them all a narrow head's tile took 12% longer), up to
                    // the tile whose results go where the first warps have yet to read: tensor
                    // memory lets them be two tiles ahead, so with room for three no warp waits.
                    // That order needs barriers of its own: the arrivals that give accumulators
                    // back release nothing (mbar_arrive_first).
                    float2(*red)[kM] = reinterpret_cast<float2(*)[kM]>(buf) + j3 * kParts;
                    const uint32_t in = (warp & 3) * 32 + lane;
                    if (warp >= 4) {
                        if (!late) late = __any_sync(0xFFFFFFFFu, !wait(joined + 8 * j3, round ^ 1));
                        red[warp >> 2][in] = make_float2(top, sum);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(reduced + 8 * j3);
                    } else {
                        if (!late) late = __any_sync(0xFFFFFFFFu, !wait(reduced + 8 * j3, round));
                        if (row < p.tokens) {
#pragma unroll
                            for (uint32_t q = 1; q < kParts; ++q) join(top, sum, red[q][in]);
                            const uint64_t part = (uint64_t)p.unit0 * (kVocabUnit / p.bn) + t.n0 / p.bn;
                            float2 *to = p.part + part * p.tokens + row;
                            if (VOCAB_OK(kVocabWorkspace, to, 8)) *to = make_float2(top, sum);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(joined + 8 * j3);
                    }
                    if (++j3 == kJoins) j3 = 0, round ^= 1;
                    continue;
                } else {
                    // the column of this row's target in the tile, if it is there
                    const int64_t at = (int64_t)target - (int64_t)(p.first[t.r] + t.vrow);
                    const bool here = target != p.ignore && target >= 0 && at >= (int64_t)c0 && at < (int64_t)min(c1, valid);
                    // the logits, summed as the loss sums them: of one accumulator 64 columns at a
                    // time below (8192 tokens of 65536 x 64: 655 us, 807 with all of them here)
                    constexpr bool kLong = MODE == kGradLong;
                    float v[kLong ? 128 : 64];
                    bool ok = take();
                    if constexpr (kLong) {
#pragma unroll
                        for (uint32_t b = 0; b < 128; b += 32)
                            if (c0 + b < c1) tmem_load32(acc + c0 + b, *reinterpret_cast<float(*)[32]>(v + b));
                        give_back();
                        for (uint32_t kb = t.kb0 + kSumBlocks; ok && kb < t.kb1; kb += kSumBlocks) {
                            ok = take();
                            acc = tmem + (u & 1) * 256 + lanes;
#pragma unroll
                            for (uint32_t b = 0; b < 128; b += 8) {
                                if (c0 + b >= c1) continue;
                                float x[8];
                                tmem_load8(acc + c0 + b, x);
#pragma unroll
                                for (uint32_t j = 0; j < 8; ++j) v[b + j] += x[j];
                            }
                            give_back();
                        }
                    }
                    if (!ok) break;
                    const bool keep = row < p.tokens && target != p.ignore && target >= 0 && (uint32_t)target < p.vocab;
                    const uint32_t col = here ? (uint32_t)at : 0xFFFFFFFFu;
                    const uint32_t rows = row0 < p.tokens ? min(p.tokens - row0, 32u) : 0;
                    const uint32_t mask = keep ? 0xFFFFFFFFu : 0u;   // of a row's results, two at a time
                    // the distance from lse first, which of a confident token is nearly all
                    // of its p - 1
                    const float2 down = make_float2(-lse, -lse), log2e2 = make_float2(kLog2e, kLog2e);
                    auto step = [&](uint32_t c, float *v) {   // 64 columns
                        uint32_t w[32];
                        // most steps have every column there and no row's target
                        const bool plain = c + 64 <= valid && !__any_sync(0xFFFFFFFFu, col - c < 64);
#pragma unroll
                        for (uint32_t q = 0; q < 64; q += 32) {
                            if constexpr (!kLong) tmem_load32(acc + c + q, *reinterpret_cast<float(*)[32]>(v + q));
#pragma unroll
                            for (uint32_t j = q; j < q + 32; j += 2) {
                                const float2 x = mul2(add2(make_float2(v[j], v[j + 1]), down), log2e2);
                                v[j] = exp2_fast(x.x);
                                v[j + 1] = exp2_fast(x.y);
                            }
                            if (!plain) {
#pragma unroll
                                for (uint32_t j = q; j < q + 32; ++j) {
                                    if (c + j == col) v[j] -= 1.0f;
                                    v[j] = c + j < valid ? v[j] : 0.0f;
                                }
                            }
#pragma unroll
                            for (uint32_t j = q; j < q + 32; j += 2) w[j / 2] = pack_bf16x2(v[j], v[j + 1]) & mask;
                        }
                        store_rows_bf16(p, buf, w, p.gbuf + (uint64_t)row0 * p.gpitch + t.n0 + c, p.gpitch, rows, 64, 8,
                                         kVocabG);
                    };
                    if constexpr (kLong) {
                        if (c0 < c1) step(c0, v);
                        if (c0 + 64 < c1) step(c0 + 64, v + 64);
                        continue;   // given back above
                    }
                    for (uint32_t c = c0; c < c1; c += 64) step(c, v);
                }
            } else if (!take()) {
                break;
            } else if (!t.dw) {
                // fp32 sums: 32 columns a step, through shared memory so that
                // eight threads take a row's line
                const uint32_t rows = row0 < p.tokens ? min(p.tokens - row0, 32u) : 0;
                float *part = p.acc + ((uint64_t)t.split * p.tokens + row0) * p.apitch + t.n0;
                for (uint32_t c = c0; c < c1 && t.n0 + c < p.dim; c += 32) {
                    float v[32];
                    tmem_load32(acc + c, v);
                    __syncwarp();
#pragma unroll
                    for (uint32_t q = 0; q < 8; ++q)
                        *out_chunk(buf, lane, q) =
                            make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                       __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]));
                    __syncwarp();
                    const uint32_t q = lane & 7, first = lane >> 3, e = t.n0 + c + 4 * q;
                    if (e >= p.dim) continue;
                    float4 f[8];   // rows first, first + 4, ... of the warp's 32
#pragma unroll
                    for (uint32_t k = 0; k < 8; ++k) f[k] = *reinterpret_cast<const float4 *>(out_chunk(buf, first + 4 * k, q));
                    float4 *at = reinterpret_cast<float4 *>(part + (uint64_t)first * p.apitch + c + 4 * q);
                    if (p.acc_in) {
#pragma unroll
                        for (uint32_t k = 0; k < 8; ++k)
                            if (first + 4 * k < rows && VOCAB_OK(kVocabWorkspace, at + (uint64_t)k * p.apitch, 16)) {
                                const float4 o = at[(uint64_t)k * p.apitch];
                                f[k].x += o.x, f[k].y += o.y, f[k].z += o.z, f[k].w += o.w;
                            }
                    }
                    if (!p.final) {
#pragma unroll
                        for (uint32_t k = 0; k < 8; ++k)
                            if (first + 4 * k < rows && VOCAB_OK(kVocabWorkspace, at + (uint64_t)k * p.apitch, 16))
                                at[(uint64_t)k * p.apitch] = f[k];
                        continue;
                    }
#pragma unroll
                    for (uint32_t k = 0; k < 8; ++k) {
                        if (first + 4 * k >= rows) continue;
                        uint16_t *to = p.dh + (uint64_t)(row0 + first + 4 * k) * p.dim + e;
                        const uint2 h = make_uint2(pack_bf16x2(f[k].x * scale, f[k].y * scale),
                                                   pack_bf16x2(f[k].z * scale, f[k].w * scale));
                        if (p.dh_vec) {
                            if (VOCAB_OK(kVocabDh, to, 8)) *reinterpret_cast<uint2 *>(to) = h;
                        } else {
                            const uint16_t x[4] = {(uint16_t)h.x, (uint16_t)(h.x >> 16), (uint16_t)h.y,
                                                   (uint16_t)(h.y >> 16)};
#pragma unroll
                            for (uint32_t j = 0; j < 4; ++j)
                                if (e + j < p.dim && VOCAB_OK(kVocabDh, to + j, 2)) to[j] = x[j];
                        }
                    }
                }
            } else {
                const uint32_t rows = rows_left(p, t.r, t.vrow + quad, 32);
                uint16_t *out = p.dw[t.r] + (uint64_t)(t.vrow + quad) * p.dim + t.n0;
                for (uint32_t c = c0; c < c1 && t.n0 + c < p.dim; c += 64) {
                    uint32_t w[32];
#pragma unroll
                    for (uint32_t q = 0; q < 2; ++q) {
                        float v[32];
                        tmem_load32(acc + c + 32 * q, v);
#pragma unroll
                        for (uint32_t j = 0; j < 16; ++j)
                            w[16 * q + j] = pack_bf16x2(v[2 * j] * scale, v[2 * j + 1] * scale);
                    }
                    store_rows_bf16(p, buf, w, out + c, p.dim, rows, min(p.dim - t.n0 - c, 64u), p.dw_align, kVocabDw + t.r);
                }
            }
            give_back();
        }
    }
    tc_fence_before();
    __syncwarp();
    if (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    if (warp == kFinishWarps + 1) tmem_free<CG>(tmem, kTmemColumns);
    DT_TL_END_BLOCK(DT_TL_VOCAB);
}

// Joins the partial maxima and sums of 32 tokens: thread (c, s) takes every
// 32nd of token c (loads of 32 tokens are whole lines), then warp c joins
// token c's 32 in a tree.  The block's sum of losses goes to memory, and the
// last block to finish adds the blocks' in block order.
constexpr int kTokens = 32, kSlices = 32;

__global__ void __launch_bounds__(kTokens *kSlices) vocab_finish_kernel(const __grid_constant__ VocabFinish p)
{
    __shared__ float2 part[kSlices][kTokens + 1];
    __shared__ float loss_of[kTokens];
    __shared__ uint32_t keeps[kTokens];
    __shared__ bool last;
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    const uint32_t lane = threadIdx.x % kTokens, warp = threadIdx.x / kTokens;
    const uint32_t t = blockIdx.x * kTokens + warp;   // the token that this warp finishes
    int32_t target = p.ignore;
    float logit = 0.0f;
    if (t < p.tokens) {
        if (VOCAB_OK(kVocabTargets, p.targets + t, 4)) target = p.targets[t];
        // nobody's where the target is not in the vocabulary: not used then
        if (VOCAB_OK(kVocabWorkspace, p.logit + t, 4)) logit = p.logit[t];
    }
    float top = -INFINITY, sum = 0.0f;
    const uint32_t column = blockIdx.x * kTokens + lane;
    if (column < p.tokens) {
#pragma unroll 4
        for (uint32_t k = warp; k < p.tiles; k += kSlices) {
            const float2 *from = p.part + (uint64_t)k * p.tokens + column;
            if (VOCAB_OK(kVocabWorkspace, from, 8)) join(top, sum, *from);
        }
    }
    part[warp][lane] = make_float2(top, sum);
    __syncthreads();
    const float2 v = part[lane][warp];
    float most = v.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    sum = scaled(v.x, v.y, most);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) {
        float loss = 0.0f;
        uint32_t kept = 0;
        if (t < p.tokens) {
            const float lse = most + logf(sum);
            if (target != p.ignore) {
                if (target >= 0 && (uint32_t)target < p.vocab) {
                    loss = lse - logit;
                    kept = 1;
                } else {
                    record_error(p.sink, DT_ERR_INVALID, -1, (int)t, target);
                }
            }
            if (p.lse && VOCAB_OK(kVocabLse, p.lse + t, 4)) p.lse[t] = lse;
            if (p.losses && VOCAB_OK(kVocabLosses, p.losses + t, 4)) p.losses[t] = loss;
        }
        loss_of[warp] = loss;
        keeps[warp] = kept;
    }
    __syncthreads();
    if (warp == 0 && p.loss) {
        // 32 losses in fp32; the blocks' sums, of which there may be many, in
        // 64 bits (a rare unit here, and slow: not for a single block)
        float sum32 = loss_of[lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum32 += __shfl_xor_sync(0xFFFFFFFFu, sum32, o);
        uint64_t kept = __reduce_add_sync(0xFFFFFFFFu, keeps[lane]);
        bool end = true;
        if (gridDim.x > 1) {
            if (lane == 0) {
                if (VOCAB_OK(kVocabWorkspace, p.block_sum + blockIdx.x, 4)) p.block_sum[blockIdx.x] = sum32;
                if (VOCAB_OK(kVocabWorkspace, p.block_kept + blockIdx.x, 4)) p.block_kept[blockIdx.x] = (uint32_t)kept;
                __threadfence();
                last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
            }
            __syncwarp();
            end = last;
            if (end) {
                __threadfence();
                double all = 0.0;
                kept = 0;
#pragma unroll 4
                for (uint32_t b = lane; b < gridDim.x; b += 32) {
                    if (VOCAB_OK(kVocabWorkspace, p.block_sum + b, 4)) all += __ldcg(p.block_sum + b);
                    if (VOCAB_OK(kVocabWorkspace, p.block_kept + b, 4)) kept += __ldcg(p.block_kept + b);
                }
                for (int o = 16; o > 0; o >>= 1) {
                    all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
                    kept += __shfl_xor_sync(0xFFFFFFFFu, kept, o);
                }
                sum32 = (float)all;
            }
        }
        if (end && lane == 0 && VOCAB_OK(kVocabLoss, p.loss, 4))
            *p.loss = kept == 0 ? 0.0f : p.avg ? __fdiv_rn(sum32, (float)kept) : sum32;
    }
    DT_TL_END_BLOCK(DT_TL_VOCAB);
}

// dh = s * (the sum of the splits), four elements a thread, 16 splits' loads
// under way at a time.
__global__ void __launch_bounds__(kThreads) vocab_join_kernel(const __grid_constant__ VocabParams p)
{
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    const uint32_t quads = p.apitch / 4;
    const uint64_t all = (uint64_t)p.tokens * quads, step = (uint64_t)gridDim.x * kThreads;
    for (uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += step) {
        const float scale = VOCAB_OK(kVocabWorkspace, p.scale, 4) ? *p.scale : 0.0f;
        const float4 *from = reinterpret_cast<const float4 *>(p.acc) + i;   // rows of quads, one split after the other
        float4 f = make_float4(0, 0, 0, 0);
        for (uint32_t k = 0; k < p.splits; k += 16) {
            float4 o[16];
#pragma unroll
            for (uint32_t j = 0; j < 16; ++j)
                o[j] = k + j < p.splits && VOCAB_OK(kVocabWorkspace, from + (k + j) * all, 16) ? from[(k + j) * all]
                                                                                             : make_float4(0, 0, 0, 0);
#pragma unroll
            for (uint32_t j = 0; j < 16; ++j) f.x += o[j].x, f.y += o[j].y, f.z += o[j].z, f.w += o[j].w;
        }
        const float v[4] = {f.x * scale, f.y * scale, f.z * scale, f.w * scale};
        const uint32_t row = (uint32_t)(i / quads), e = (uint32_t)(i - (uint64_t)row * quads) * 4;
        uint16_t *to = p.dh + (uint64_t)row * p.dim + e;
        if (p.dh_vec) {
            if (VOCAB_OK(kVocabDh, to, 8))
                *reinterpret_cast<uint2 *>(to) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        } else {
            for (uint32_t j = 0; j < 4 && e + j < p.dim; ++j)
                if (VOCAB_OK(kVocabDh, to + j, 2)) to[j] = f32_to_bf16(v[j]);
        }
    }
    DT_TL_END_BLOCK(DT_TL_VOCAB);
}

// Rows that TMA cannot address (a width that is not a multiple of 8, or a
// buffer off a 16-byte boundary), laid out again at a pitch of whole vectors:
// the hidden rows (`tokens` of them, in the call's first launch, else 0), then
// the vocabulary units [unit0, ...), whose rows past a rank's last are zeros.
// A warp takes a row; a lane makes a vector from the two aligned ones that its
// elements lie in, neither of which reaches past the 16-byte block of an
// element of its row.
__global__ void __launch_bounds__(kThreads) vocab_pack_kernel(const __grid_constant__ VocabPack p)
{
    DT_TL_BEGIN();
    pdl_begin();
    DT_TL_WAITED();
    const uint32_t vecs = p.pitch / 8, lane = threadIdx.x & 31, step = gridDim.x * (kThreads / 32);
    for (uint32_t i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < p.tokens + p.rows; i += step) {
        const bool h = i < p.tokens;
        const uint32_t row = h ? i : i - p.tokens;
        const uint16_t *base = p.hidden;
        uint32_t at = row, have = p.tokens;
        int r = -1;
        if (!h) {
            const uint32_t unit = p.unit0 + row / kVocabUnit;
            uint32_t begin = 0;
            r = 0;
#pragma unroll
            for (int q = 0; q + 1 < DT_MAX_RANKS; ++q)
                if (q + 1 < p.P && unit >= p.unit_end[q]) {
                    r = q + 1;
                    begin = p.unit_end[q];
                }
            at = (unit - begin) * kVocabUnit + row % kVocabUnit;
            have = p.src_rows[r];
            base = p.src[r];
        }
        uint4 *dst = reinterpret_cast<uint4 *>(h ? p.hidden_dst : p.dst) + (uint64_t)row * vecs;
        if (at >= have) {
            for (uint32_t k = lane; k < vecs; k += 32)
                if (VOCAB_OK(kVocabWorkspace, dst + k, 16)) dst[k] = make_uint4(0, 0, 0, 0);
            continue;
        }
        const uint16_t *src = base + (uint64_t)at * p.dim;
        const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(src) & 15, words = off / 4, bits = off % 4 * 8;
        const uint4 *blocks = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(src) & ~(uintptr_t)15);
#pragma unroll 4
        for (uint32_t k = lane; k < vecs; k += 32) {
            const uint32_t n = min(p.dim - 8 * k, 8u);   // elements of this vector
            uint32_t w[4] = {0, 0, 0, 0};
            if (VOCAB_OK(h ? (int)kVocabHidden : kVocabRows + r, src + 8 * k, 2 * n)) {
                const uint4 a = __ldg(blocks + k), b = off + 2 * n > 16 ? __ldg(blocks + k + 1) : make_uint4(0, 0, 0, 0);
                const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (uint32_t q = 0; q < 4; ++q) {
                    uint32_t lo = 0, hi = 0;   // words words + q and the next, by selection: no indexing of registers
#pragma unroll
                    for (uint32_t z = 0; z < 4; ++z) {
                        lo = words == z ? v[q + z] : lo;
                        hi = words == z ? (q + z + 1 < 8 ? v[q + z + 1] : 0u) : hi;
                    }
                    w[q] = __funnelshift_r(lo, hi, bits);
                    // elements past the row's end
                    if (2 * q >= n) w[q] = 0;
                    else if (2 * q + 1 >= n) w[q] &= 0xFFFFu;
                }
            }
            if (VOCAB_OK(kVocabWorkspace, dst + k, 16)) dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    DT_TL_END_BLOCK(DT_TL_VOCAB);
}

uint32_t tc_blocks(const VocabParams &p, int device)
{
    return std::min(p.workers, vocab_workers(p.pairs, device)) * (p.pairs ? 2 : 1);
}

template <int MODE, int CG>
cudaError_t launch_mode(VocabParams &p, int device, cudaStream_t s)
{
    static std::atomic<uint64_t> ready{0};   // devices whose shared memory limit is set
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (!(ready.load(std::memory_order_acquire) & bit) || !bit) {
        const cudaError_t e = cudaFuncSetAttribute(vocab_kernel<MODE, CG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)kTcSmem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    p.stages = std::min(kMaxStages, kRingBytes / (2 * a_box_bytes(MODE == kBack, p.rows_h) + p.bn / CG * 256));
    return launch_kernel(vocab_kernel<MODE, CG>, dim3(tc_blocks(p, device)), dim3(tc_threads(MODE)), kTcSmem, s, false, p);
}

template <int MODE>
cudaError_t launch_mode(VocabParams &p, int device, cudaStream_t s)
{
    return p.pairs ? launch_mode<MODE, 2>(p, device, s) : launch_mode<MODE, 1>(p, device, s);
}

unsigned elementwise_grid(uint64_t items, int device)
{
    const uint64_t want = (items + kThreads - 1) / kThreads, cap = (uint64_t)sm_count(device) * 16;
    return (unsigned)(want < cap ? (want ? want : 1) : cap);
}

}  // namespace

DT_TL_BINDER(bind_timeline_vocab)

uint32_t vocab_blocks(uint64_t inner) { return (uint32_t)((inner + kK - 1) / kK); }

uint32_t vocab_workers(bool pairs, int device) { return (uint32_t)std::max(1, sm_count(device) / (pairs ? 2 : 1)); }

cudaError_t launch_vocab_lse(VocabParams &p, int device, cudaStream_t s)
{
    p.workers = p.tiles;
    return launch_mode<kLse>(p, device, s);
}

cudaError_t launch_vocab_grad(VocabParams &p, int device, cudaStream_t s)
{
    p.workers = p.tiles;
    if (p.unit0 == 0) p.kept_parts = std::min(tc_blocks(p, device), (p.tokens + 255) / 256);
    return p.kblocks > kSumBlocks ? launch_mode<kGradLong>(p, device, s) : launch_mode<kGrad>(p, device, s);
}

// A finished tile costs a worker about a block of the inner dimension more than
// its products.
constexpr uint32_t kTileCost = 1;

cudaError_t launch_vocab_back(VocabParams &p, int device, cudaStream_t s)
{
    const uint32_t W = vocab_workers(p.pairs, device);
    p.workers = std::min(W, p.tiles + p.dw_tiles);
    p.dh_rest = p.tiles % p.workers;
    p.dw_early = 0;
    if (p.dh_rest) {
        const uint32_t others = p.workers - p.dh_rest;
        p.dw_early = std::min((p.kblocks / p.splits + kTileCost) / (p.dw_kblocks + kTileCost), p.dw_tiles / others);
    }
    return launch_mode<kBack>(p, device, s);
}

cudaError_t launch_vocab_finish(const VocabFinish &p, cudaStream_t s)
{
    return launch_kernel(vocab_finish_kernel, dim3(vocab_finish_blocks(p.tokens)), dim3(kTokens * kSlices), 0, s, false, p);
}

uint32_t vocab_finish_blocks(uint32_t tokens) { return (tokens + kTokens - 1) / kTokens; }

cudaError_t launch_vocab_join(const VocabParams &p, int device, cudaStream_t s)
{
    return launch_kernel(vocab_join_kernel, dim3(elementwise_grid((uint64_t)p.tokens * (p.apitch / 4), device)),
                         dim3(kThreads), 0, s, false, p);
}

cudaError_t launch_vocab_pack(const VocabPack &p, int device, cudaStream_t s)
{
    return launch_kernel(vocab_pack_kernel, dim3(elementwise_grid(((uint64_t)p.tokens + p.rows) * 32, device)),
                         dim3(kThreads), 0, s, false, p);
}

cudaError_t vocab_map(CUtensorMap *map, const void *base, uint64_t cols, uint64_t rows, uint64_t pitch, uint32_t box_rows)
{
    static std::atomic<void *> entry{nullptr};
    void *fn = entry.load(std::memory_order_acquire);
    if (!fn) {
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess) return e;
        if (found != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
        entry.store(fn, std::memory_order_release);
    }
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {pitch * 2};
    const cuuint32_t box[2] = {64, box_rows}, steps[2] = {1, 1};
    const CUresult r = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
        map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, steps,
        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace dt
