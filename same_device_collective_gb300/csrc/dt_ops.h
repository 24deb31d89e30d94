// Parameter blocks and launchers of the layer norm and vocabulary loss
// kernels.  Not part of the C ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "dt.h"
#include "dt_internal.h"

namespace dt {

// ---- layer norm -------------------------------------------------------------
// Buffers, as bounds-checked builds number them: x r, dy 16 + r, y or dx 32 + r,
// mean 48 + r, rstd 64 + r, then these.
enum NormBuffer : int { kNormWeight = 5 * DT_MAX_RANKS, kNormBias, kNormDweight, kNormDbias, kNormWorkspace, kNormBuffers };

// The ranks' rows are numbered through: rank r has rows [row_end[r - 1],
// row_end[r]) of the call.
struct NormParams {
    const void *x[DT_MAX_RANKS];
    const void *dy[DT_MAX_RANKS];      // backward
    void *out[DT_MAX_RANKS];           // y, or dx
    float *mean[DT_MAX_RANKS];         // written by the forward pass (NULL: not wanted), read by the backward pass
    float *rstd[DT_MAX_RANKS];
    uint64_t row_end[DT_MAX_RANKS];
    const void *weight, *bias;         // NULL: 1, 0
    float *partial;                    // backward: [parts][2][cols] sums of dy * xhat and dy
    void *dweight, *dbias;             // NULL: not wanted
    uint64_t rows;
    uint32_t cols;
    uint32_t tpr;                      // threads that share a row, a multiple of 32
    uint32_t parts;                    // groups of them that walk over the rows; to the join, shares of dw and db
    // rings: chunks of up to chunk_rows rows of one rank (rank r's end at
    // chunk_end[r]); a stage holds a chunk of x, and backward of dy, in
    // array_bytes each, then of mean and rstd in stat_bytes each
    uint32_t chunk_rows, stages, stage_bytes, array_bytes, stat_bytes;
    uint64_t chunks;
    uint64_t chunk_end[DT_MAX_RANKS];  // rows in registers: the ranks' blocks in one row of `chunks` of them, or chunks 0
    int32_t P;
    int32_t weight_bf16;               // of both
    int32_t param_kind;                // how the forward kernel reads them
    float eps, inv_cols;
    float avg_scale;
    int32_t avg;                       // 0: sum; 1: divide the gradients by P
    int32_t avg_pow2;
    ErrorSink sink;
#ifdef DT_BOUNDS
    Extent extent[kNormBuffers];
#endif
};

// Bytes of partial sums that the backward pass of rows of `cols` elements
// writes at most on this device.
size_t norm_workspace(uint32_t cols, int device);
// vec: every row of every buffer starts on a 16-byte boundary
cudaError_t launch_norm(NormParams p, int dtype, bool vec, int device, cudaStream_t s);
cudaError_t launch_norm_backward(NormParams p, int dtype, bool vec, int device, cudaStream_t s);

#ifdef DT_TIMELINE
void bind_timeline_norm(const void *sink);
void bind_timeline_vocab(const void *sink);
#endif

}  // namespace dt
