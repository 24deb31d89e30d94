// C ABI entry points of the layer norm and the vocabulary loss: argument
// checks and launch planning.  They follow the collectives' conventions: every
// argument error is reported before anything is enqueued, device memory is the
// caller's, no call waits for the GPU and none throws.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "dt_group.h"
#include "dt_host.h"
#include "dt_ops.h"
#include "dt_vocab.h"

namespace {

using namespace dt::host;

constexpr size_t kMaxCols = (size_t)1 << 24;

bool float_dtype(int dtype) { return dtype == DT_F32 || dtype == DT_BF16; }

bool multiple(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// The buffers of a call.  Outputs may overlap nothing, but for an output and
// an input that carry the same tag (>= 0) and are the same buffer.
struct Buffers {
    Range in[5 * DT_MAX_RANKS], out[3 * DT_MAX_RANKS + 4];
    int nin = 0, nout = 0;

    void read(const void *p, size_t bytes, int tag = -1)
    {
        if (p && bytes) in[nin++] = Range{(uintptr_t)p, (uintptr_t)p + bytes, tag, 0};
    }
    void write(const void *p, size_t bytes, int tag = -1)
    {
        if (p && bytes) out[nout++] = Range{(uintptr_t)p, (uintptr_t)p + bytes, tag, 1};
    }
    bool clash() const
    {
        for (int o = 0; o < nout; ++o) {
            for (int k = o + 1; k < nout; ++k)
                if (overlaps(out[o], out[k])) return true;
            for (int i = 0; i < nin; ++i)
                if (overlaps(out[o], in[i]) && !(out[o].rank >= 0 && out[o].rank == in[i].rank && out[o].lo == in[i].lo))
                    return true;
        }
        return false;
    }
};

// Every rank's row count; false where the counts or the bytes of all rows pass
// what a size_t or a pointer can hold.
bool row_counts(int P, const size_t *rows, size_t rows_equal, size_t row_bytes, size_t *n, size_t *total)
{
    *total = 0;
    for (int r = 0; r < P; ++r) {
        n[r] = rows ? rows[r] : rows_equal;
        if (n[r] > SIZE_MAX / 64 / row_bytes) return false;
        *total += n[r];
        if (*total > SIZE_MAX / 64 / row_bytes) return false;
    }
    return true;
}

// What both passes of the layer norm check and set: x, the rows and the types.
dt_status norm_common(dt_group *g, const void *const *x, void *const *out, const size_t *rows, size_t rows_equal,
                      size_t cols, int dtype, int weight_dtype, const void *weight, dt::NormParams &p, size_t *n,
                      bool &vec)
{
    if (!x || !out || cols == 0 || cols > kMaxCols || !float_dtype(dtype) || !float_dtype(weight_dtype))
        return dtype == DT_I32 || weight_dtype == DT_I32 ? DT_ERR_UNSUPPORTED : DT_ERR_INVALID;
    const size_t es = elem_bytes(dtype), ws = elem_bytes(weight_dtype);
    size_t total = 0;
    if (!row_counts(g->P, rows, rows_equal, cols * es, n, &total)) return DT_ERR_INVALID;
    if (!multiple(weight, ws)) return DT_ERR_INVALID;
    memset(&p, 0, sizeof p);
    vec = cols * es % 16 == 0;
    uint64_t end = 0;
    for (int r = 0; r < g->P; ++r) {
        p.row_end[r] = end += n[r];
        if (n[r] == 0) continue;
        if (!x[r] || !out[r] || !multiple(x[r], es) || !multiple(out[r], es)) return DT_ERR_INVALID;
        p.x[r] = x[r];
        p.out[r] = out[r];
        dt::set_extent(p, r, x[r], n[r] * cols * es, false);
        dt::set_extent(p, 2 * DT_MAX_RANKS + r, out[r], n[r] * cols * es, true);
        vec = vec && aligned16(x[r]) && aligned16(out[r]);
    }
    p.rows = total;
    p.cols = (uint32_t)cols;
    p.inv_cols = 1.0f / (float)cols;
    p.P = g->P;
    p.weight = weight;
    p.weight_bf16 = weight_dtype == DT_BF16;
    p.sink = error_sink(g);
    dt::set_extent(p, dt::kNormWeight, weight, cols * ws, false);
    return DT_OK;
}

// ---- vocabulary loss --------------------------------------------------------

constexpr size_t kMaxTokens = (size_t)1 << 30, kMaxVocab = (size_t)1 << 30, kMaxDim = (size_t)1 << 20;
// A piece of the vocabulary: its p - [target], and its rows where they have to
// be laid out again, take at most this much.
constexpr uint64_t kPieceBytes = (uint64_t)512 << 20, kPackBytes = (uint64_t)128 << 20;
// Vocabulary tiles next to one another in the order of tiles: with 16, the
// 76 pairs of CTAs work on about 5 x 16 tiles of 256 x 256.
constexpr uint32_t kGroup = 16;

uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

// How a call is cut up, and where its parts of the workspace lie.  Sizes that
// the workspace query knows decide everything but `packed`.
struct VocabPlan {
    size_t rows[DT_MAX_RANKS];
    uint32_t units, pieces, piece;      // units of 256 rows; pieces of at most `piece` units
    bool pairs;                         // two CTAs share a tile
    uint32_t bn;                        // width of the logits' tiles
    uint32_t parts;                     // tiles, and partial sums, of a unit
    uint32_t pitch;                     // of rows laid out again
    uint32_t splits, apitch;
    bool packed;
    uint64_t part, logit, sums, kept, ticket, scale, g, acc, pack_h, pack_w, bytes;
};

// The wider of two tiles, unless the narrower one leaves the workers less to
// do one after the other; a tile costs about 64 columns more than it has.  82
// tiles of 128 for 152 SMs take less time than 164 of 64, but 128 of 64 less
// than 64 of 128.
uint32_t tile_width(uint64_t mt, uint64_t units, uint64_t workers, bool pairs)
{
    const uint32_t wide = pairs ? 256 : 128;
    auto cost = [&](uint32_t bn) { return (mt * units * (dt::kVocabUnit / bn) + workers - 1) / workers * (bn + 64); };
    return cost(wide / 2) < cost(wide) ? wide / 2 : wide;
}

bool vocab_plan(dt_group *g, const size_t *vocab, size_t vocab_equal, size_t tokens, size_t dim, bool back, bool packed,
                VocabPlan &v)
{
    if (tokens > kMaxTokens || dim == 0 || dim > kMaxDim) return false;
    size_t total = 0;
    v.units = 0;
    for (int r = 0; r < g->P; ++r) {
        v.rows[r] = vocab ? vocab[r] : vocab_equal;
        if (v.rows[r] > kMaxVocab || (total += v.rows[r]) > kMaxVocab) return false;
        v.units += (uint32_t)((v.rows[r] + dt::kVocabUnit - 1) / dt::kVocabUnit);
    }
    if (total == 0) return false;
    v.pairs = tokens > 128;
    const uint64_t workers = dt::vocab_workers(v.pairs, g->device), high = v.pairs ? 256 : 128;
    const uint64_t mt = (tokens + high - 1) / high;
    v.packed = packed;
    v.pitch = (uint32_t)up(dim, 8);
    const uint64_t pack_units = std::max<uint64_t>(1, kPackBytes / (dt::kVocabUnit * 2ull * v.pitch));
    uint64_t most = v.units;
    if (packed) most = std::min(most, pack_units);
    if (back && tokens) most = std::min(most, std::max<uint64_t>(1, kPieceBytes / (dt::kVocabUnit * 2ull * tokens)));
    v.pieces = (uint32_t)((v.units + most - 1) / most);
    v.piece = (v.units + v.pieces - 1) / v.pieces;
    v.pieces = (v.units + v.piece - 1) / v.piece;
    v.bn = tile_width(mt, v.piece, workers, v.pairs);
    v.parts = dt::kVocabUnit / v.bn;
    // few tokens: the vocabulary is split over the workers that dh's tiles leave idle
    v.apitch = (uint32_t)up(dim, 4);
    const uint64_t wide = v.pairs ? 256 : 128, across = (dim + wide - 1) / wide, tiles = mt * across;
    const uint64_t kblocks = dt::vocab_blocks(dt::kVocabUnit * (uint64_t)(v.units - (v.pieces - 1) * v.piece));
    v.splits = 1;
    if (back && tiles && tiles < workers)
        v.splits = (uint32_t)std::max<uint64_t>(1, std::min(workers / tiles, kblocks / 8));

    // tiles are counted in 32 bits
    if (mt * v.piece * 4 > 0x7FFFFFFF || tiles * v.splits + 2ull * v.piece * across > 0x7FFFFFFF) return false;

    uint64_t at = 0;
    auto take = [&at](uint64_t n) {
        const uint64_t from = at;
        at = up(at + n, 256);
        return from;
    };
    v.ticket = take(4);
    v.scale = take(4);
    v.part = v.logit = v.sums = v.kept = v.g = v.acc = 0;
    if (!back) {
        const uint64_t blocks = dt::vocab_finish_blocks((uint32_t)tokens);
        v.part = take((uint64_t)v.units * v.parts * tokens * sizeof(float2));
        v.logit = take(tokens * 4);
        v.sums = take(blocks * 4);
        v.kept = take(blocks * 4);
    } else {
        v.kept = take(workers * (v.pairs ? 2 : 1) * 4);
        v.g = take((uint64_t)v.piece * dt::kVocabUnit * 2 * tokens);
        if (v.splits > 1 || v.pieces > 1) v.acc = take((uint64_t)v.splits * tokens * v.apitch * 4);
    }
    v.pack_h = v.pack_w = 0;
    if (packed) {
        v.pack_h = take((uint64_t)tokens * v.pitch * 2);
        v.pack_w = take((uint64_t)v.piece * dt::kVocabUnit * 2 * v.pitch);
    }
    v.bytes = at;
    return true;
}

// Bytes for either form: a call finds out from its pointers whether rows have
// to be laid out again.
uint64_t vocab_bytes(dt_group *g, const size_t *vocab, size_t vocab_equal, size_t tokens, size_t dim, bool back)
{
    VocabPlan a, b;
    if (!vocab_plan(g, vocab, vocab_equal, tokens, dim, back, true, a)) return 0;
    if (dim % 8) return a.bytes;
    vocab_plan(g, vocab, vocab_equal, tokens, dim, back, false, b);
    return std::max(a.bytes, b.bytes);
}

// Checks what both passes share and fills in the parameters and the plan.
dt_status vocab_common(dt_group *g, const void *hidden, const void *const *weight, const size_t *vocab,
                       size_t vocab_equal, const int32_t *targets, size_t tokens, size_t dim, int dtype, int op,
                       int32_t ignore_index, void *workspace, size_t workspace_bytes, bool back, Buffers &b,
                       VocabPlan &v, dt::VocabParams &p)
{
    if (!valid_dtype(dtype) || !valid_op(op)) return DT_ERR_INVALID;
    if (dtype != DT_BF16 || (op != DT_SUM && op != DT_AVG)) return DT_ERR_UNSUPPORTED;
    if (!weight || !vocab_plan(g, vocab, vocab_equal, tokens, dim, back, false, v)) return DT_ERR_INVALID;
    if (tokens && (!hidden || !targets)) return DT_ERR_INVALID;
    if (!multiple(hidden, 2) || !multiple(targets, 4)) return DT_ERR_INVALID;
    bool in_place = dim % 8 == 0 && aligned16(hidden);
    b.read(hidden, tokens * dim * 2);
    b.read(targets, tokens * 4);
    memset(&p, 0, sizeof p);
    uint32_t unit = 0, first = 0;
    for (int r = 0; r < g->P; ++r) {
        p.unit_end[r] = unit += (uint32_t)((v.rows[r] + dt::kVocabUnit - 1) / dt::kVocabUnit);
        p.rows[r] = (uint32_t)v.rows[r];
        p.first[r] = first;
        first += (uint32_t)v.rows[r];
        if (v.rows[r] == 0) continue;
        if (!weight[r] || !multiple(weight[r], 2)) return DT_ERR_INVALID;
        in_place = in_place && aligned16(weight[r]);
        b.read(weight[r], v.rows[r] * dim * 2);
    }
    if (!in_place) vocab_plan(g, vocab, vocab_equal, tokens, dim, back, true, v);
    if (tokens && (!workspace || !multiple(workspace, 256) ||
                   workspace_bytes < vocab_bytes(g, vocab, vocab_equal, tokens, dim, back)))
        return DT_ERR_INVALID;
    b.write(workspace, workspace_bytes);
    p.vocab = first;
    p.P = g->P;
    p.packed = !in_place;
    p.tokens = (uint32_t)tokens;
    p.dim = (uint32_t)dim;
    p.ignore = ignore_index;
    p.avg = op == DT_AVG;
    p.targets = targets;
    p.sink = error_sink(g);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    p.ticket = reinterpret_cast<uint32_t *>(ws + v.ticket);
    p.scale = reinterpret_cast<float *>(ws + v.scale);
    p.kept = reinterpret_cast<uint32_t *>(ws + v.kept);
    p.part = reinterpret_cast<float2 *>(ws + v.part);
    p.logit = reinterpret_cast<float *>(ws + v.logit);
    p.gbuf = reinterpret_cast<uint16_t *>(ws + v.g);
    p.acc = reinterpret_cast<float *>(ws + v.acc);
    p.gpitch = v.piece * dt::kVocabUnit;
    p.apitch = v.apitch;
    dt::set_extent(p, dt::kVocabG, p.gbuf, back ? (uint64_t)tokens * p.gpitch * 2 : 0, false);
    dt::set_extent(p, dt::kVocabTargets, targets, tokens * 4, false);
    dt::set_extent(p, dt::kVocabWorkspace, workspace, v.bytes, false);
    return DT_OK;
}

// The tensor maps of the ranks' rows, or of a piece's rows laid out again, in
// boxes of rows_w rows, and of the hidden rows in boxes of rows_h.
cudaError_t vocab_maps(dt_group *g, const void *hidden, const void *const *weight, void *workspace, const VocabPlan &v,
                       dt::VocabParams &p, uint32_t rows_h, uint32_t rows_w)
{
    if (p.rows_h == rows_h && p.rows_w == rows_w) return cudaSuccess;   // as they are
    p.rows_h = rows_h;
    p.rows_w = rows_w;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    if (v.packed) {
        p.w_maps = 1;
        const cudaError_t e = dt::vocab_map(&p.h, ws + v.pack_h, p.dim, p.tokens, v.pitch, rows_h);
        if (e != cudaSuccess) return e;
        return dt::vocab_map(&p.w[0], ws + v.pack_w, p.dim, (uint64_t)v.piece * dt::kVocabUnit, v.pitch, rows_w);
    }
    cudaError_t e = dt::vocab_map(&p.h, hidden, p.dim, p.tokens, p.dim, rows_h);
    for (int r = 0; r < g->P && e == cudaSuccess; ++r) {
        if (p.rows[r] == 0) continue;
        p.w_maps |= 1u << r;
        e = dt::vocab_map(&p.w[r], weight[r], p.dim, p.rows[r], p.dim, rows_w);
    }
    return e;
}

// ... as the logits' tiles read them.
cudaError_t vocab_logit_maps(dt_group *g, const void *hidden, const void *const *weight, void *workspace,
                             const VocabPlan &v, dt::VocabParams &p)
{
    const uint32_t rows_h = v.pairs ? 128 : (uint32_t)up(p.tokens, 8);
    return vocab_maps(g, hidden, weight, workspace, v, p, rows_h, v.bn / (v.pairs ? 2 : 1));
}

// Where rows have to be laid out again: what the pieces' launches share.  The
// first one does the hidden rows too.
void vocab_prepare_pack(dt_group *g, const void *hidden, const void *const *weight, void *workspace, const VocabPlan &v,
                        const dt::VocabParams &p, dt::VocabPack &pack)
{
    if (!v.packed) return;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    memset(&pack, 0, sizeof pack);
    for (int r = 0; r < g->P; ++r) {
        pack.src[r] = static_cast<const uint16_t *>(weight[r]);
        pack.src_rows[r] = p.rows[r];
        pack.unit_end[r] = p.unit_end[r];
    }
    pack.hidden = static_cast<const uint16_t *>(hidden);
    pack.hidden_dst = reinterpret_cast<uint16_t *>(ws + v.pack_h);
    pack.dst = reinterpret_cast<uint16_t *>(ws + v.pack_w);
    pack.P = g->P;
    pack.dim = p.dim;
    pack.pitch = v.pitch;
    pack.sink = p.sink;
    for (int r = 0; r < g->P; ++r)
        dt::set_extent(pack, dt::kVocabRows + r, weight[r], (uint64_t)p.rows[r] * p.dim * 2, false);
    dt::set_extent(pack, dt::kVocabHidden, hidden, (uint64_t)p.tokens * p.dim * 2, false);
    dt::set_extent(pack, dt::kVocabWorkspace, workspace, v.bytes, false);
}

// The piece's first unit and, where needed, its rows laid out again.
cudaError_t vocab_piece(dt_group *g, const VocabPlan &v, uint32_t piece, dt::VocabParams &p, dt::VocabPack &pack,
                        uint32_t *units, cudaStream_t s)
{
    p.unit0 = piece * v.piece;
    *units = std::min(v.piece, v.units - p.unit0);
    if (!v.packed) return cudaSuccess;
    pack.unit0 = p.unit0;
    pack.tokens = piece == 0 ? p.tokens : 0;
    pack.rows = *units * dt::kVocabUnit;
    return dt::launch_vocab_pack(pack, g->device, s);
}

void logits_tiles(const VocabPlan &v, uint32_t units, dt::VocabParams &p)
{
    const uint32_t high = v.pairs ? 256 : 128;
    p.pairs = v.pairs;
    p.bn = v.bn;
    p.mt = (p.tokens + high - 1) / high;
    p.nt = units * (dt::kVocabUnit / v.bn);
    p.splits = 1;
    p.group = kGroup;
    p.kblocks = dt::vocab_blocks(p.dim);
    auto inverse = [](uint32_t d) { return (uint32_t)((1ull << 32) / d + 1); };
    p.per_group = inverse(p.group * p.mt);
    p.per_row = inverse(p.group);
    p.per_last = inverse((p.nt - 1) % p.group + 1);
    p.tiles = p.mt * p.nt;
}

}  // namespace

extern "C" {

dt_status dt_layer_norm(dt_group_t g, const void *const *x, const void *weight, const void *bias, void *const *y,
                        float *const *mean, float *const *rstd, const size_t *rows, size_t rows_equal, size_t cols,
                        float eps, int dtype, int weight_dtype, void *stream)
{
    DT_TRACE();
    if (!g) return DT_ERR_INVALID;
    std::lock_guard<std::mutex> lock(g->mu);
    dt_status st = take_device_error(g);
    if (st != DT_OK) return st;
    dt::NormParams p;
    size_t n[DT_MAX_RANKS];
    bool vec = false;
    st = norm_common(g, x, y, rows, rows_equal, cols, dtype, weight_dtype, weight, p, n, vec);
    if (st != DT_OK) return st;
    const size_t row_bytes = cols * elem_bytes(dtype), w_bytes = cols * elem_bytes(weight_dtype);
    if (!(eps >= 0.0f) || std::isinf(eps) || !multiple(bias, elem_bytes(weight_dtype))) return DT_ERR_INVALID;
    Buffers b;
    b.read(weight, w_bytes);
    b.read(bias, w_bytes);
    for (int r = 0; r < g->P; ++r) {
        if (n[r] == 0) continue;
        p.mean[r] = mean ? mean[r] : nullptr;
        p.rstd[r] = rstd ? rstd[r] : nullptr;
        if (!multiple(p.mean[r], 4) || !multiple(p.rstd[r], 4)) return DT_ERR_INVALID;
        b.read(x[r], n[r] * row_bytes, r);
        b.write(y[r], n[r] * row_bytes, r);
        b.write(p.mean[r], n[r] * 4);
        b.write(p.rstd[r], n[r] * 4);
        dt::set_extent(p, 3 * DT_MAX_RANKS + r, p.mean[r], n[r] * 4, true);
        dt::set_extent(p, 4 * DT_MAX_RANKS + r, p.rstd[r], n[r] * 4, true);
    }
    if (b.clash()) return DT_ERR_INVALID;
    if (p.rows == 0) return DT_OK;
    p.bias = bias;
    p.eps = eps;
    dt::set_extent(p, dt::kNormBias, bias, w_bytes, false);
    DeviceScope scope(g->device);
    if (!scope.ok) return DT_ERR_CUDA;
    return cuda_status(dt::launch_norm(p, dtype, vec, g->device, static_cast<cudaStream_t>(stream)));
}

dt_status dt_layer_norm_backward(dt_group_t g, const void *const *x, const void *const *dy, const void *weight,
                                 const float *const *mean, const float *const *rstd, void *const *dx, void *dweight,
                                 void *dbias, const size_t *rows, size_t rows_equal, size_t cols, int dtype,
                                 int weight_dtype, int op, void *workspace, size_t workspace_bytes, void *stream)
{
    DT_TRACE();
    if (!g) return DT_ERR_INVALID;
    std::lock_guard<std::mutex> lock(g->mu);
    dt_status st = take_device_error(g);
    if (st != DT_OK) return st;
    dt::NormParams p;
    size_t n[DT_MAX_RANKS];
    bool vec = false;
    st = norm_common(g, x, dx, rows, rows_equal, cols, dtype, weight_dtype, weight, p, n, vec);
    if (st != DT_OK) return st;
    if (!dy || !mean || !rstd || !valid_op(op)) return DT_ERR_INVALID;
    if (op != DT_SUM && op != DT_AVG) return DT_ERR_UNSUPPORTED;
    const size_t es = elem_bytes(dtype), ws = elem_bytes(weight_dtype);
    const bool sums = dweight || dbias;
    if (!multiple(dweight, ws) || !multiple(dbias, ws)) return DT_ERR_INVALID;
    if (sums && (!workspace || !aligned16(workspace) || workspace_bytes < dt::norm_workspace(p.cols, g->device)))
        return DT_ERR_INVALID;
    Buffers b;
    b.read(weight, cols * ws);
    for (int r = 0; r < g->P; ++r) {
        if (n[r] == 0) continue;
        if (!dy[r] || !mean[r] || !rstd[r] || !multiple(dy[r], es) || !multiple(mean[r], 4) || !multiple(rstd[r], 4))
            return DT_ERR_INVALID;
        p.dy[r] = dy[r];
        p.mean[r] = const_cast<float *>(mean[r]);
        p.rstd[r] = const_cast<float *>(rstd[r]);
        vec = vec && aligned16(dy[r]);
        b.read(x[r], n[r] * cols * es);
        b.read(dy[r], n[r] * cols * es, r);
        b.read(mean[r], n[r] * 4);
        b.read(rstd[r], n[r] * 4);
        b.write(dx[r], n[r] * cols * es, r);
        dt::set_extent(p, DT_MAX_RANKS + r, dy[r], n[r] * cols * es, false);
        dt::set_extent(p, 3 * DT_MAX_RANKS + r, mean[r], n[r] * 4, false);
        dt::set_extent(p, 4 * DT_MAX_RANKS + r, rstd[r], n[r] * 4, false);
    }
    b.write(dweight, cols * ws);
    b.write(dbias, cols * ws);
    if (sums) b.write(workspace, workspace_bytes);
    if (b.clash()) return DT_ERR_INVALID;
    if (p.rows == 0 && !sums) return DT_OK;
    p.dweight = dweight;
    p.dbias = dbias;
    dt::set_extent(p, dt::kNormDweight, dweight, cols * ws, true);
    dt::set_extent(p, dt::kNormDbias, dbias, cols * ws, true);
    dt::set_extent(p, dt::kNormWorkspace, workspace, workspace_bytes, false);
    p.partial = sums ? static_cast<float *>(workspace) : nullptr;
    p.avg = op == DT_AVG;
    p.avg_pow2 = (g->P & (g->P - 1)) == 0;
    p.avg_scale = p.avg_pow2 ? 1.0f / (float)g->P : 0.0f;
    DeviceScope scope(g->device);
    if (!scope.ok) return DT_ERR_CUDA;
    return cuda_status(dt::launch_norm_backward(p, dtype, vec, g->device, static_cast<cudaStream_t>(stream)));
}

size_t dt_layer_norm_workspace(dt_group_t g, size_t cols)
{
    if (!g || cols == 0 || cols > kMaxCols) return 0;
    return dt::norm_workspace((uint32_t)cols, g->device);
}

dt_status dt_vocab_loss(dt_group_t g, const void *hidden, const void *const *weight, const size_t *vocab,
                        size_t vocab_equal, const int32_t *targets, size_t tokens, size_t dim, int dtype, int op,
                        int32_t ignore_index, float *losses, float *lse, float *loss, void *workspace,
                        size_t workspace_bytes, void *stream)
{
    DT_TRACE();
    if (!g) return DT_ERR_INVALID;
    std::lock_guard<std::mutex> lock(g->mu);
    dt_status st = take_device_error(g);
    if (st != DT_OK) return st;
    Buffers b;
    VocabPlan v;
    dt::VocabParams p;
    dt::VocabPack pack;
    st = vocab_common(g, hidden, weight, vocab, vocab_equal, targets, tokens, dim, dtype, op, ignore_index, workspace,
                      workspace_bytes, false, b, v, p);
    if (st != DT_OK) return st;
    if (!multiple(losses, 4) || !multiple(lse, 4) || !multiple(loss, 4)) return DT_ERR_INVALID;
    b.write(losses, tokens * 4);
    b.write(lse, tokens * 4);
    b.write(loss, 4);
    if (b.clash()) return DT_ERR_INVALID;
    DeviceScope scope(g->device);
    if (!scope.ok) return DT_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tokens == 0) return loss ? cuda_status(cudaMemsetAsync(loss, 0, 4, s)) : DT_OK;

    vocab_prepare_pack(g, hidden, weight, workspace, v, p, pack);
    cudaError_t e = vocab_logit_maps(g, hidden, weight, workspace, v, p);
    for (uint32_t k = 0; k < v.pieces && e == cudaSuccess; ++k) {
        uint32_t units = 0;
        e = vocab_piece(g, v, k, p, pack, &units, s);
        logits_tiles(v, units, p);
        if (e == cudaSuccess) e = dt::launch_vocab_lse(p, g->device, s);
    }
    if (e != cudaSuccess) return cuda_status(e);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    dt::VocabFinish f;
    memset(&f, 0, sizeof f);
    f.part = p.part;
    f.logit = p.logit;
    f.targets = targets;
    f.losses = losses;
    f.lse = lse;
    f.loss = loss;
    f.block_sum = reinterpret_cast<float *>(ws + v.sums);
    f.block_kept = reinterpret_cast<uint32_t *>(ws + v.kept);
    f.ticket = p.ticket;
    f.tokens = p.tokens;
    f.tiles = v.units * v.parts;
    f.vocab = p.vocab;
    f.ignore = ignore_index;
    f.avg = p.avg;
    f.sink = p.sink;
    dt::set_extent(f, dt::kVocabTargets, targets, tokens * 4, false);
    dt::set_extent(f, dt::kVocabLse, lse, tokens * 4, true);
    dt::set_extent(f, dt::kVocabLosses, losses, tokens * 4, true);
    dt::set_extent(f, dt::kVocabLoss, loss, 4, true);
    dt::set_extent(f, dt::kVocabWorkspace, workspace, v.bytes, false);
    return cuda_status(dt::launch_vocab_finish(f, s));
}

dt_status dt_vocab_loss_backward(dt_group_t g, const void *hidden, const void *const *weight, const size_t *vocab,
                                 size_t vocab_equal, const int32_t *targets, const float *lse, const float *grad_loss,
                                 size_t tokens, size_t dim, int dtype, int op, int32_t ignore_index, void *dhidden,
                                 void *const *dweight, void *workspace, size_t workspace_bytes, void *stream)
{
    DT_TRACE();
    if (!g) return DT_ERR_INVALID;
    std::lock_guard<std::mutex> lock(g->mu);
    dt_status st = take_device_error(g);
    if (st != DT_OK) return st;
    Buffers b;
    VocabPlan v;
    dt::VocabParams p;
    dt::VocabPack pack;
    st = vocab_common(g, hidden, weight, vocab, vocab_equal, targets, tokens, dim, dtype, op, ignore_index, workspace,
                      workspace_bytes, true, b, v, p);
    if (st != DT_OK) return st;
    if (!dweight || !multiple(lse, 4) || !multiple(grad_loss, 4) || !multiple(dhidden, 2)) return DT_ERR_INVALID;
    if (tokens && (!lse || !dhidden)) return DT_ERR_INVALID;
    b.read(lse, tokens * 4);
    b.read(grad_loss, 4);
    b.write(dhidden, tokens * dim * 2);
    p.dh_vec = dim % 4 == 0 && multiple(dhidden, 8);
    p.dw_align = dim % 8 == 0 ? 8 : dim % 4 == 0 ? 4 : dim % 2 == 0 ? 2 : 1;
    for (int r = 0; r < g->P; ++r) {
        if (p.rows[r] == 0) continue;
        if (!dweight[r] || !multiple(dweight[r], 2)) return DT_ERR_INVALID;
        p.dw[r] = static_cast<uint16_t *>(dweight[r]);
        while (!multiple(dweight[r], 2 * p.dw_align)) p.dw_align /= 2;
        b.write(dweight[r], v.rows[r] * dim * 2);
        dt::set_extent(p, dt::kVocabDw + r, dweight[r], v.rows[r] * dim * 2, true);
    }
    if (b.clash()) return DT_ERR_INVALID;
    p.dh = static_cast<uint16_t *>(dhidden);
    p.lse = lse;
    p.grad = grad_loss;
    dt::set_extent(p, dt::kVocabDh, dhidden, tokens * dim * 2, true);
    dt::set_extent(p, dt::kVocabLse, lse, tokens * 4, false);
    dt::set_extent(p, dt::kVocabGrad, grad_loss, 4, false);
    DeviceScope scope(g->device);
    if (!scope.ok) return DT_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (tokens == 0) {
        for (int r = 0; r < g->P && e == cudaSuccess; ++r)
            if (p.rows[r]) e = cudaMemsetAsync(dweight[r], 0, v.rows[r] * dim * 2, s);
        return cuda_status(e);
    }

    vocab_prepare_pack(g, hidden, weight, workspace, v, p, pack);
    // few tokens: boxes of as many as there are, in whole K steps of 16
    p.rows_g = v.pairs ? 128 : (uint32_t)up(p.tokens, 16);
    e = dt::vocab_map(&p.g, p.gbuf, p.gpitch, p.tokens, p.gpitch, p.rows_g);
    for (uint32_t k = 0; k < v.pieces && e == cudaSuccess; ++k) {
        uint32_t units = 0;
        e = vocab_logit_maps(g, hidden, weight, workspace, v, p);
        if (e == cudaSuccess) e = vocab_piece(g, v, k, p, pack, &units, s);
        logits_tiles(v, units, p);
        if (e == cudaSuccess) e = dt::launch_vocab_grad(p, g->device, s);
        if (e != cudaSuccess) break;
        if (e == cudaSuccess) e = vocab_maps(g, hidden, weight, workspace, v, p, p.rows_g, 128);
        if (e != cudaSuccess) break;
        p.bn = v.pairs ? 256 : 128;
        p.nt = (p.dim + p.bn - 1) / p.bn;
        p.splits = v.splits;
        p.kblocks = dt::vocab_blocks(units * dt::kVocabUnit);
        p.tiles = p.mt * p.nt * p.splits;
        p.dw_tiles = units * (v.pairs ? 1 : 2) * p.nt;
        p.dw_kblocks = dt::vocab_blocks(p.tokens);
        p.acc_in = k > 0;
        p.final = v.splits == 1 && k + 1 == v.pieces;
        e = dt::launch_vocab_back(p, g->device, s);
    }
    if (e == cudaSuccess && v.splits > 1) e = dt::launch_vocab_join(p, g->device, s);
    return cuda_status(e);
}

size_t dt_vocab_loss_workspace(dt_group_t g, const size_t *vocab, size_t vocab_equal, size_t tokens, size_t dim,
                               int dtype, int backward)
{
    if (!g || dtype != DT_BF16) return 0;
    return (size_t)vocab_bytes(g, vocab, vocab_equal, tokens, dim, backward != 0);
}

}  // extern "C"
