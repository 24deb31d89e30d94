// Parameter blocks and launchers of the linear layers over the ranks.  Not part
// of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dt.h"
#include "dt_internal.h"
#include "dt_ops.h"

namespace dt {

// What a launch computes.  With X [n, d] the ranks' tokens, W_r and f_r rank r's
// weights and features, G_r [n, f_r] and Y [n, d]:
//   kGather      y_r = act(X W_r^T + b_r)               W_r [f_r, d]
//   kGatherBack  dx = sum_r G_r W_r, dW_r = G_r^T X
//   kReduce      y = sum_r H_r W_r^T + b (+ residual)   W_r [d, f_r]
//   kReduceBack  dH_r = Y W_r, dW_r = Y^T H_r
enum LinearKind : int { kGather, kGatherBack, kReduce, kReduceBack };

// The three axes of these products: tokens, columns of a token, features.
enum LinearAxis : int { kTokens, kDim, kFeatures };

// Buffers, as bounds-checked builds number them: by rank from these on.
enum LinearBuffer : int {
    kLinearY, kLinearPre = DT_MAX_RANKS, kLinearDx = 2 * DT_MAX_RANKS, kLinearDw = 3 * DT_MAX_RANKS,
    kLinearDb = 4 * DT_MAX_RANKS, kLinearBias = 5 * DT_MAX_RANKS, kLinearResidual = 6 * DT_MAX_RANKS,
    kLinearX = 7 * DT_MAX_RANKS, kLinearW = 8 * DT_MAX_RANKS, kLinearDy = 9 * DT_MAX_RANKS,
    kLinearWorkspace = 10 * DT_MAX_RANKS, kLinearBuffers
};

// The depth of a stage, and of the blocks that the inner axis is cut into: 64, or where
// an operand's rows run along the inner axis 128, so that its boxes of 64 columns are
// not short.  Forward, more and shorter stages ride out the loads' latency.
__host__ __device__ constexpr uint32_t linear_depth(bool back) { return back ? 128 : 64; }

// One product of a launch: its tiles, splits of its inner axis, and outputs.
struct LinearProduct {
    uint32_t mt, nt, splits, tiles;    // tiles = mt * nt * splits
    uint32_t kblocks;                  // blocks of the inner axis
    uint32_t group_inverse, mt_inverse;   // for divisions by a group of tiles and by mt
    uint32_t f_end[DT_MAX_RANKS];      // the ranks' features and tokens in halves of 128 rows of a tile, its columns or
    uint32_t t_end[DT_MAX_RANKS];      // blocks, as their axis is cut here, numbered through: rank r's end at [r]
    uint16_t *out[DT_MAX_RANKS];
    uint32_t align[DT_MAX_RANKS];      // elements that the rows of out[r] (and pre[r], residual[r]) are a multiple of: 1, 2, 4, 8
    float *acc;                        // splits > 1: sums [splits][tiles' rows][tiles' columns]
};

// The bias' gradient: column sums of bf16 matrices, or of the floats that were summed
// over chunks of rows before, [rows, cols] each: of one matrix for each output, or of
// all of them (`stacked`) for the only one.
struct LinearSums {
    const void *src[DT_MAX_RANKS];
    uint16_t *out[DT_MAX_RANKS];
    uint32_t rows[DT_MAX_RANKS], cols[DT_MAX_RANKS];   // of the sources, of the outputs
    uint32_t group_end[DT_MAX_RANKS];  // groups of 32 columns, numbered through the outputs
    uint32_t groups;
    int32_t n, sources, stacked, f32;
};

// What every kernel of a call knows.
struct LinearCall {
    LinearProduct product[2];
    uint32_t f_len[DT_MAX_RANKS];
    uint32_t t_len[DT_MAX_RANKS], t_first[DT_MAX_RANKS];   // pieces of the token axis in the tokens' matrix
    uint32_t row_end[DT_MAX_RANKS];    // the ranks' tokens, numbered through
    int32_t P, t_pieces;
    int32_t f_pieces;                  // ranks up to the last that has features
    uint32_t tokens, dim;
    uint16_t *pre[DT_MAX_RANKS];
    const uint16_t *bias[DT_MAX_RANKS];
    const uint16_t *residual[DT_MAX_RANKS];
    int32_t act;
    int32_t keep, biased, residuals;   // pre, bias, residual are there
    LinearSums sums;                   // backward
    ErrorSink sink;
#ifdef DT_BOUNDS
    Extent extent[kLinearBuffers];
#endif
};

// The tensor core kernels (linear_kernel).
struct LinearParams : LinearCall {
    CUtensorMap tok[DT_MAX_RANKS];     // the ranks' tokens [t_len, dim] (one map when they are one matrix)
    CUtensorMap feat[DT_MAX_RANKS];    // [tokens, f_len]
    CUtensorMap w[DT_MAX_RANKS];       // [f_len, dim], or reducing [dim, f_len]
    uint32_t bn;                       // tile width, a multiple of 32: up to 256
    uint32_t stages, workers;
    uint32_t step;                     // forward: blocks of the inner axis to a stage, 1 or 2
    uint32_t rows_t, rows_w;           // of the maps' boxes
    uint32_t rest, early;              // the order of both products' tiles (next_tile)
};

// Small products, in place (linear_small_kernel): tiles of 64 x 64.
struct LinearSmall : LinearCall {
    const uint16_t *tok[DT_MAX_RANKS];     // the ranks' tokens
    const uint16_t *feat[DT_MAX_RANKS];    // [tokens, f_len]
    const uint16_t *weight[DT_MAX_RANKS];
    const uint16_t *z[DT_MAX_RANKS];       // gathering, backward: what act'(.) is taken of, where act is not none
    uint32_t ctas;                     // of a cluster: 1, 2, 4 or 8
    uint32_t shared[2];                // they share a tile's inner axis; else each has a tile
    uint32_t clusters[2];              // the first product's, and the second's after them; then those of the sums
    uint32_t strips;                   // of 64 columns of the bias' gradient
};
constexpr uint32_t kSmallTile = 64;

// What goes before the products: rows laid out again at a pitch that TMA can
// address, the gradient before the activation, and column sums for the bias'.
struct LinearPrepJob {
    const uint16_t *src;               // [rows, cols]
    const uint16_t *pre;               // NULL, or what act'(.) is taken of and src multiplied by
    uint16_t *dst;                     // NULL, or [rows, pitch]
    float *sums;                       // NULL, or [chunks of rows][cols]
    uint32_t rows, cols, pitch;
    uint32_t strips;                   // of kPrepCols columns
    uint32_t block_end;                // of the launch's blocks
    int32_t src_buffer, pre_buffer;    // numbers of LinearBuffer
    int32_t vec;                       // rows of src and pre are whole vectors
};
constexpr uint32_t kPrepCols = 256;
constexpr int kPrepJobs = 3 * DT_MAX_RANKS;
struct LinearPrep {
    LinearPrepJob job[kPrepJobs];
    uint32_t chunk_rows;               // of a block: a multiple of 32
    int32_t jobs, act;
    ErrorSink sink;
#ifdef DT_BOUNDS
    Extent extent[kLinearBuffers];
#endif
};

// Forward products of few tokens (linear_few_kernel).
struct LinearFew {
    const uint16_t *x[DT_MAX_RANKS];   // gathering: the ranks' tokens; reducing: the ranks' features
    const uint16_t *w[DT_MAX_RANKS];
    uint16_t *out[DT_MAX_RANKS], *pre[DT_MAX_RANKS];
    const uint16_t *bias[DT_MAX_RANKS], *residual[DT_MAX_RANKS];
    uint32_t f_len[DT_MAX_RANKS], row_end[DT_MAX_RANKS];
    uint32_t block_end[DT_MAX_RANKS];  // gathering: blocks of each rank's features, numbered through
    int32_t P;
    uint32_t tokens, dim, blocks;
    uint32_t k_warps;                  // warps of a block that share its rows' inner axis: 1, 2, 4 or 8
    int32_t act, keep, biased, residuals;
    ErrorSink sink;
#ifdef DT_BOUNDS
    Extent extent[kLinearBuffers];
#endif
};
constexpr uint32_t kFewTokens = 16;

cudaError_t launch_linear(LinearParams &p, LinearKind kind, bool pairs, int device, cudaStream_t s);
// The splits' sums into one, of product k.
cudaError_t launch_linear_join(const LinearParams &p, LinearKind kind, int k, bool pairs, cudaStream_t s);
// vec: every row that is read starts on a 16-byte boundary.
cudaError_t launch_linear_few(LinearFew &p, LinearKind kind, bool vec, int device, cudaStream_t s);
cudaError_t launch_linear_small(const LinearSmall &p, LinearKind kind, bool vec, cudaStream_t s);
cudaError_t launch_linear_prep(LinearPrep &p, cudaStream_t s);
// CTAs, or pairs of them, that run at once.
uint32_t linear_workers(bool pairs, int device);

}  // namespace dt
