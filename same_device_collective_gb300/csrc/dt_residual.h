// Parameter block and launchers of the residual norm.  Not part of the C ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "dt.h"
#include "dt_internal.h"
#include "dt_ops.h"

namespace dt {

// The matrices that a pass reads, row by row.
enum ResidualSource : int { kBranch, kX, kY = kX, kDz, kDy, kResidualSources };

// Buffers, as bounds-checked builds number them: branch r, x or y 16 + r, dz 32 + r,
// dy 48 + r, the first output 64 + r, the second 80 + r, the post norm's rstd 96 + r,
// the pre norm's 112 + r, then these.
enum ResidualBuffer : int {
    kResidualOut = kResidualSources * DT_MAX_RANKS,
    kResidualRstd = kResidualOut + 2 * DT_MAX_RANKS,
    kResidualPost = kResidualRstd + 2 * DT_MAX_RANKS, kResidualGate, kResidualPre, kResidualDpost, kResidualDgate,
    kResidualDpre, kResidualWorkspace, kResidualBuffers
};

// The ranks' rows are numbered through: rank r has rows [row_end[r - 1],
// row_end[r]) of the call.
struct ResidualParams {
    const void *src[kResidualSources][DT_MAX_RANKS];   // dy may be absent (NULL everywhere)
    void *out[2][DT_MAX_RANKS];        // y and z, or dx and dbranch
    float *rstd[2][DT_MAX_RANKS];      // of the post and the pre norm: written (NULL: not wanted), backward read
    const void *post, *gate, *pre;     // NULL: 1
    float *partial;                    // backward: [parts][2][cols] sums of d * h and dz * n
    void *dpost, *dgate, *dpre;        // NULL: not wanted
    uint64_t row_end[DT_MAX_RANKS];
    uint64_t rows;
    uint32_t cols;
    uint32_t tpr;                      // threads that share a row
    uint32_t parts;                    // groups of them that walk over the rows; to the join, shares of the sums
    // chunks of up to chunk_rows rows of one rank (rank r's end at chunk_end[r]); a stage
    // holds a chunk of each source in array_bytes, and backward of both rstd in stat_bytes
    uint32_t chunk_rows, stages, stage_bytes, array_bytes, stat_bytes;
    uint64_t chunks;
    uint64_t chunk_end[DT_MAX_RANKS];
    int32_t P;
    int32_t weight_bf16;               // of all three
    int32_t has_dy;
    float scale;                       // of the residual stream
    float eps, inv_cols;
    float avg_scale;
    int32_t avg, avg_pow2;             // divide the weights' gradients by P
    ErrorSink sink;
#ifdef DT_BOUNDS
    Extent extent[kResidualBuffers];
#endif
};

// Bytes of partial sums that the backward pass of rows of `cols` elements writes at
// most on this device.
size_t residual_workspace(uint32_t cols, int device);
// vec: every row of every buffer starts on a 16-byte boundary
cudaError_t launch_residual(ResidualParams p, int dtype, bool vec, int device, cudaStream_t s);
cudaError_t launch_residual_backward(ResidualParams p, int dtype, bool vec, int device, cudaStream_t s);

}  // namespace dt
