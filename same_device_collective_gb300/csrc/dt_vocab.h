// Parameter blocks and launchers of the vocabulary loss.  Not part of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "dt.h"
#include "dt_internal.h"

namespace dt {

// The ranks' vocabulary rows are numbered through in units of this many rows:
// rank r has units [unit_end[r - 1], unit_end[r]), its last one padded.
constexpr uint32_t kVocabUnit = 256;

// Buffers, as bounds-checked builds number them; then dweight 16 + r and the
// ranks' rows that are laid out again 32 + r.
enum VocabBuffer : int {
    kVocabG, kVocabDh, kVocabTargets, kVocabLse, kVocabLosses, kVocabLoss, kVocabGrad, kVocabWorkspace, kVocabHidden,
    kVocabDw = DT_MAX_RANKS, kVocabRows = 2 * DT_MAX_RANKS, kVocabBuffers = 3 * DT_MAX_RANKS
};

struct VocabParams {
    CUtensorMap h;                     // [tokens, dim]
    CUtensorMap g;                     // [tokens, gpitch]: a piece's p - [target]
    CUtensorMap w[DT_MAX_RANKS];       // rank r's rows; packed: w[0] holds the piece's units
    uint32_t unit_end[DT_MAX_RANKS];
    uint32_t rows[DT_MAX_RANKS];       // vocabulary rows of each rank
    uint32_t first[DT_MAX_RANKS];      // the vocabulary index of its first row
    uint32_t vocab;
    int32_t P;
    uint32_t packed;
    uint32_t unit0;                    // the piece's first unit
    uint32_t tokens, dim;
    uint32_t bn;                       // tile width: 64 or 128, of pairs 128 or 256
    uint32_t stages;
    uint32_t pairs;                    // two CTAs share a tile
    uint32_t workers;                  // CTAs or pairs that have a tile
    uint32_t mt, nt, splits, group;    // tiles of the logits or dh, splits of the inner dimension, tile order
    uint32_t per_group, per_row, per_last;   // inverses of group * mt, group and the last group's width (quotient)
    uint32_t kblocks;                  // blocks of the inner dimension
    uint32_t tiles;                    // mt * nt * splits
    uint32_t dw_tiles, dw_kblocks;     // the same of dw, whose tiles have the width of dh's
    uint32_t dh_rest, dw_early;        // the order of both (next_tile)
    uint32_t gpitch, apitch;
    uint32_t acc_in, final;            // dh: add to the sums so far; store the result
    uint32_t rows_h, rows_g, rows_w;   // of the maps' boxes
    uint32_t w_maps;                   // bit r: w[r] is a map
    uint32_t dh_vec;                   // rows of dh start on 8-byte boundaries
    uint32_t dw_align;                 // elements that rows of every dw are a multiple of, address and width: 1, 2, 4, 8
    int32_t ignore;
    int32_t avg;
    const int32_t *targets;
    const float *lse;
    const float *grad;
    float2 *part;                      // [tiles of the vocabulary][tokens]: maximum, sum of exponentials
    float *logit;                      // the target's logit of each token
    uint32_t *ticket;
    uint32_t *kept;                    // gradient: counted tokens, a part to a CTA of the first launch
    uint32_t kept_parts;
    float *scale;                      // gradient: grad, or grad / counted tokens
    uint16_t *gbuf;                    // [tokens, gpitch] bf16
    float *acc;                        // dh's sums [splits][tokens][apitch]
    uint16_t *dh;
    uint16_t *dw[DT_MAX_RANKS];
    ErrorSink sink;
#ifdef DT_BOUNDS
    Extent extent[kVocabBuffers];
#endif
};

struct VocabFinish {
    const float2 *part;
    const float *logit;
    const int32_t *targets;
    float *losses, *lse, *loss;        // each may be NULL
    float *block_sum;
    uint32_t *block_kept;
    uint32_t *ticket;
    uint32_t tokens, tiles, vocab;
    int32_t ignore, avg;
    ErrorSink sink;
#ifdef DT_BOUNDS
    Extent extent[kVocabBuffers];
#endif
};

struct VocabPack {
    const uint16_t *src[DT_MAX_RANKS];
    uint32_t src_rows[DT_MAX_RANKS];
    uint32_t unit_end[DT_MAX_RANKS];
    const uint16_t *hidden;
    uint16_t *hidden_dst, *dst;
    int32_t P;
    uint32_t unit0;
    uint32_t tokens, rows;             // hidden rows and vocabulary rows of this launch
    uint32_t dim, pitch;
    ErrorSink sink;
#ifdef DT_BOUNDS
    Extent extent[kVocabBuffers];
#endif
};

cudaError_t launch_vocab_lse(VocabParams &p, int device, cudaStream_t s);
cudaError_t launch_vocab_grad(VocabParams &p, int device, cudaStream_t s);
cudaError_t launch_vocab_back(VocabParams &p, int device, cudaStream_t s);
// CTAs, or pairs of them, that run at once.
uint32_t vocab_workers(bool pairs, int device);
cudaError_t launch_vocab_join(const VocabParams &p, int device, cudaStream_t s);
cudaError_t launch_vocab_finish(const VocabFinish &p, cudaStream_t s);
uint32_t vocab_finish_blocks(uint32_t tokens);
cudaError_t launch_vocab_pack(const VocabPack &p, int device, cudaStream_t s);
// Blocks of an inner dimension of `inner`.
uint32_t vocab_blocks(uint64_t inner);
// The tensor map of a row-major bf16 matrix, read in boxes of 64 columns.
cudaError_t vocab_map(CUtensorMap *map, const void *base, uint64_t cols, uint64_t rows, uint64_t pitch,
                      uint32_t box_rows);

}  // namespace dt
