// C ABI entry points of the linear layers over the ranks: argument checks and
// launch planning, by the conventions of the other calls (dt_ops.cpp).
#include <algorithm>
#include <cstring>

#include "dt_group.h"
#include "dt_host.h"
#include "dt_linear.h"

namespace {

using namespace dt::host;
using dt::LinearKind;

constexpr size_t kMaxTokens = (size_t)1 << 26, kMaxWidth = (size_t)1 << 22;

// How a call is cut up, and where its parts of the workspace lie.  The sizes
// decide all of it; which matrices are laid out again is seen from the pointers.
struct Plan {
    LinearKind kind;
    size_t n[DT_MAX_RANKS], f[DT_MAX_RANKS];
    size_t tokens, features, dim;
    bool pairs;                        // two CTAs share a tile
    uint32_t halves;                   // of 128 rows in a tile: 1 or 2, each within a rank's piece
    uint64_t chunk_rows, chunks;       // of rows, whose column sums the bias' gradient adds
    uint64_t tok, feat, w, sums, acc[2], bytes;
};

uint64_t tiles_of(uint64_t n, uint64_t size) { return (n + size - 1) / size; }

bool back(LinearKind k) { return k == dt::kGatherBack || k == dt::kReduceBack; }
bool gathers(LinearKind k) { return k == dt::kGather || k == dt::kGatherBack; }

// The tokens' pieces that a product's tiles or blocks of `size` are cut from: each
// rank's, or all of them as one.
uint64_t token_tiles(const Plan &v, bool pieces, uint64_t size)
{
    if (!pieces) return tiles_of(v.tokens, size);
    uint64_t t = 0;
    for (size_t k : v.n) t += tiles_of(k, size);
    return t;
}

uint64_t feature_tiles(const Plan &v, uint64_t size)
{
    uint64_t t = 0;
    for (size_t k : v.f) t += tiles_of(k, size);
    return t;
}

// Tiles across and down, and blocks of the inner axis, of a launch's products, with
// the tokens' matrix in pieces or as one; the splits that leave no worker idle.
struct Cut {
    uint32_t bn;
    uint64_t mt[2], nt[2], kblocks[2], splits[2];
    double us;                         // what it takes, about
    uint64_t acc_bytes(const Plan &v, int k) const { return splits[k] > 1 ? splits[k] * mt[k] * v.halves * 128 * nt[k] * bn * 4 : 0; }
};

// What a launch takes, in microseconds, as far as its cut decides it.  A stage takes the
// tensor cores as long as it has columns, and at least what its loads and products take to
// issue: forward, for 64 of the inner axis, 0.28, 0.22, 0.15 with 256, 192, 128 columns (512
// tokens of 4096 to 4096); backward, 128 deep, 0.67, 0.38, 0.32 with 256, 128, 64 (1024 tokens of it), where 64
// never paid (81 us, 49 with 128).  One CTA's loads take longer than a pair's.  A tile costs
// half a microsecond beside that and the last one's finish half of one for each 64 columns,
// and splits cost a second launch and their sums' way to L2 and back.
constexpr double kUsTile = 0.5, kUsFinish64 = 0.45, kUsJoin = 2.5, kJoinBytesPerUs = 8e6;

double stage_us(bool back, bool pairs, uint32_t bn)
{
    if (back) return pairs ? 0.2 + 0.47 * bn / 256 : 0.68;
    const double least = bn <= 128 ? 0.11 : 0.19;   // two blocks to a stage, or one
    return pairs ? std::max(least + 0.04, 0.28 * bn / 256) : least + 0.15 * bn / 256;
}

double join_cost(const Plan &v, const Cut &c)
{
    double us = 0.0;
    for (int k = 0; k < 2; ++k)
        if (c.splits[k] > 1) us += kUsJoin + 2.0 * c.acc_bytes(v, k) / kJoinBytesPerUs;
    return us;
}

bool cut(const dt_group *g, const Plan &v, bool pieces, Cut &best)
{
    const bool b = back(v.kind);
    const uint64_t workers = dt::linear_workers(v.pairs, g->device), depth = dt::linear_depth(b);
    const bool n_features = v.kind == dt::kGather || v.kind == dt::kReduceBack;
    Cut c;
    // the rows' axis of forward products is the tokens, which reducing are never in pieces
    c.mt[0] = tiles_of(token_tiles(v, pieces && n_features, 128), v.halves);
    c.kblocks[0] = n_features ? tiles_of(v.dim, depth) : feature_tiles(v, depth);
    c.mt[1] = c.nt[1] = c.kblocks[1] = 0;
    if (b) {
        c.mt[1] = tiles_of(gathers(v.kind) ? feature_tiles(v, 128) : tiles_of(v.dim, 128), v.halves);
        c.kblocks[1] = token_tiles(v, pieces, depth);
    }
    double least = 1e300;
    for (uint32_t bn = b && !v.pairs ? 128 : 256; bn >= (b ? 128u : 64u); bn -= b ? 64 : 32) {
        c.bn = bn;
        const double block_us = stage_us(b, v.pairs, bn);
        c.nt[0] = n_features ? feature_tiles(v, bn) : tiles_of(v.dim, bn);
        if (b) c.nt[1] = c.nt[0];
        for (int k = 0; k < 2; ++k)
            if (c.mt[k] * c.nt[k] > 0x7FFFFFFF / workers) return false;   // tiles are counted in 32 bits
        // splits of 512 at least; none where a join would have more rows of blocks than a grid can
        uint64_t most[2];
        for (int k = 0; k < 2; ++k)
            most[k] = c.mt[k] * v.halves * 128 > 65535
                          ? 1
                          : std::max<uint64_t>(1, std::min<uint64_t>(16, c.kblocks[k] * depth / 512));
        for (c.splits[0] = 1; c.splits[0] <= most[0]; ++c.splits[0])
            for (c.splits[1] = 1; c.splits[1] <= most[1]; ++c.splits[1]) {
                double unit[2], longest = 0.0, all = 0.0;
                uint64_t units = 0;
                for (int k = 0; k < (b ? 2 : 1); ++k) {
                    const uint64_t n = c.mt[k] * c.nt[k] * c.splits[k];
                    unit[k] = tiles_of(c.kblocks[k], c.splits[k]) * block_us + kUsTile;
                    longest = std::max(longest, unit[k]);
                    all += n * unit[k];
                    units += n;
                }
                // forward in whole waves; backward the second product's tiles fill the
                // first one's last wave
                const double us = (b ? std::max(all / workers, longest) : tiles_of(units, workers) * unit[0]) +
                                  tiles_of(bn, 64) * kUsFinish64 + join_cost(v, c);
                if (us >= least) continue;
                least = c.us = us;
                best = c;
            }
    }
    return true;
}

bool plan(const dt_group *g, LinearKind kind, const size_t *rows, size_t rows_equal, size_t dim, const size_t *features,
          size_t features_equal, Plan &v)
{
    if (dim == 0 || dim > kMaxWidth) return false;
    memset(&v, 0, sizeof v);
    v.kind = kind;
    v.dim = dim;
    uint64_t padded = 0;
    for (int r = 0; r < g->P; ++r) v.tokens += rows ? rows[r] : rows_equal;
    // few rows: more blocks; many: fewer partial sums
    v.chunk_rows = v.tokens <= 2048 ? 32 : 128;
    v.tokens = 0;
    for (int r = 0; r < g->P; ++r) {
        v.n[r] = rows ? rows[r] : rows_equal;
        v.f[r] = features ? features[r] : features_equal;
        if (v.n[r] > kMaxTokens || v.f[r] > kMaxWidth) return false;
        v.tokens += v.n[r];
        v.features += v.f[r];
        padded += up(v.f[r], 8);
        v.chunks += gathers(kind) ? 0 : tiles_of(v.n[r], v.chunk_rows);
    }
    if (v.tokens > kMaxTokens || v.features > kMaxWidth || v.features == 0) return false;
    if (gathers(kind)) v.chunks = tiles_of(v.tokens, v.chunk_rows);
    // Two CTAs to a tile share its operands, and wait for one another at its start and end:
    // forward products of a wave or less and short inner axes go without (512 tokens of 1024 to
    // 4096: 8.2 us, without 7.8; 300 of 512 to 2048: 5.8 and 5.1; 512 of 4096 to 4096: 14.7 and 16.4)
    const uint64_t inner = gathers(kind) ? dim : v.features, outer = gathers(kind) ? v.features : dim;
    v.pairs = v.tokens > 128 && (back(kind) || inner > 1024 || v.tokens * outer > (1ull << 21));
    v.halves = v.pairs ? 2 : 1;
    uint64_t at = 0;
    auto take = [&at](uint64_t n) {
        const uint64_t from = at;
        at = up(at + n, 256);
        return from;
    };
    if (kind != dt::kReduce) v.tok = take((uint64_t)v.tokens * up(dim, 8) * 2);
    if (kind != dt::kGather) v.feat = take((uint64_t)v.tokens * padded * 2);
    v.w = take(gathers(kind) ? (uint64_t)v.features * up(dim, 8) * 2 : (uint64_t)dim * padded * 2);
    if (back(kind)) v.sums = take(v.chunks * (gathers(kind) ? v.features : dim) * 4);
    Cut c[2];
    if (!cut(g, v, false, c[0]) || !cut(g, v, true, c[1])) return false;
    for (int k = 0; k < 2; ++k) v.acc[k] = take(std::max(c[0].acc_bytes(v, k), c[1].acc_bytes(v, k)));
    v.bytes = std::max<uint64_t>(at, 256);
    return true;
}

size_t workspace_bytes_of(dt_group_t g, LinearKind fwd, const size_t *rows, size_t rows_equal, size_t dim,
                          const size_t *features, size_t features_equal, int dtype, int backward)
{
    Plan v;
    const LinearKind kind = !backward ? fwd : fwd == dt::kGather ? dt::kGatherBack : dt::kReduceBack;
    if (!g || dtype != DT_BF16 || !plan(g, kind, rows, rows_equal, dim, features, features_equal, v)) return 0;
    return (size_t)v.bytes;
}

// Whether the bias' gradient is summed down all rows by the warps beside the products, or
// its rows are summed in chunks before them (a launch more): a warp's loads of 64 rows of
// 32 columns are about two microseconds under way beside the products' own, which should
// take half of the products' time at most (5000 tokens, 2000 columns: a walk of 79 steps
// beside products of 200 us).
bool sums_beside(const dt_group *g, const Plan &v)
{
    const uint64_t cols = gathers(v.kind) ? v.features : v.dim, warps = dt::linear_workers(v.pairs, g->device) * (v.pairs ? 4 : 2);
    const double walk = 2.0 * tiles_of(v.tokens, 64) * tiles_of(tiles_of(cols, 32), warps);
    return walk <= 4.0 + 2.0 * v.tokens * v.dim * v.features / 1.6e9;
}

// A call on its way: its plan, its buffers, and what goes before its products.
struct Call {
    dt_group *g;
    Plan v;
    Buffers b;
    unsigned char *ws;
    dt::LinearParams p;
    dt::LinearPrep prep;
    uint32_t pieces;                   // the tokens' matrix in the ranks' pieces (> 1), or as one
    bool in_pieces, again;             // which of these, and whether it is laid out again first
    const void *tok[DT_MAX_RANKS];     // its pieces as TMA reads them
    uint64_t tok_pitch;
};

template <typename Params>
void workspace_extent(Params &p, const Call &c)
{
    dt::set_extent(p, dt::kLinearWorkspace, c.ws, c.v.bytes, false);
}

// A buffer for each rank that has something, of `width` columns, and its alignment.
dt_status take_ranks(Call &c, const void *const *list, const size_t *n, const size_t *width, size_t equal, bool output,
                     int buffer, int tag = -1)
{
    for (int r = 0; r < c.g->P; ++r) {
        const size_t bytes = n[r] * (width ? width[r] : equal) * 2;
        if (bytes == 0) continue;
        if (!list || !list[r] || !multiple(list[r], 2)) return DT_ERR_INVALID;
        if (output) c.b.write(list[r], bytes, tag >= 0 ? tag + r : -1);
        else c.b.read(list[r], bytes, tag >= 0 ? tag + r : -1);
        dt::set_extent(c.p, buffer + r, list[r], bytes, output);
        dt::set_extent(c.prep, buffer + r, list[r], bytes, output);
    }
    return DT_OK;
}

uint32_t alignment(uint32_t least, const void *p, size_t width)
{
    while (width % least || !multiple(p, 2 * least)) least /= 2;
    return least;
}

// TMA, and loads of vectors, can read a matrix of rows of `width`.
bool addressable(const void *p, size_t width) { return width % 8 == 0 && aligned16(p); }

// A job of the launch before the products.
void add_job(Call &c, const void *src, const void *pre, void *dst, float *sums, size_t rows, size_t cols, size_t pitch,
             int src_buffer, int pre_buffer)
{
    if (rows == 0 || cols == 0) return;
    dt::LinearPrepJob &j = c.prep.job[c.prep.jobs];
    j.src = static_cast<const uint16_t *>(src);
    j.pre = static_cast<const uint16_t *>(pre);
    j.dst = static_cast<uint16_t *>(dst);
    j.sums = sums;
    j.rows = (uint32_t)rows;
    j.cols = (uint32_t)cols;
    j.pitch = (uint32_t)pitch;
    j.strips = (uint32_t)tiles_of(cols, dt::kPrepCols);
    j.block_end = (c.prep.jobs ? c.prep.job[c.prep.jobs - 1].block_end : 0) + j.strips * (uint32_t)tiles_of(rows, c.v.chunk_rows);
    j.src_buffer = src_buffer;
    j.pre_buffer = pre_buffer;
    j.vec = addressable(src, cols) && (!pre || addressable(pre, cols));
    ++c.prep.jobs;
}

// Checks what all calls share.
dt_status begin(Call &c, LinearKind kind, const size_t *rows, size_t rows_equal, size_t dim, const size_t *features,
                size_t features_equal, int dtype, void *workspace, size_t workspace_bytes)
{
    if (!valid_dtype(dtype)) return DT_ERR_INVALID;
    if (dtype != DT_BF16) return DT_ERR_UNSUPPORTED;
    if (!plan(c.g, kind, rows, rows_equal, dim, features, features_equal, c.v)) return DT_ERR_INVALID;
    memset(&c.p, 0, sizeof c.p);
    memset(&c.prep, 0, sizeof c.prep);
    c.ws = static_cast<unsigned char *>(workspace);
    if (c.v.tokens) {
        if (!workspace || !multiple(workspace, 256) || workspace_bytes < c.v.bytes) return DT_ERR_INVALID;
        c.b.write(workspace, workspace_bytes);
    }
    dt::LinearParams &p = c.p;
    uint32_t end = 0;
    for (int r = 0; r < c.g->P; ++r) {
        p.f_len[r] = (uint32_t)c.v.f[r];
        p.row_end[r] = end += (uint32_t)c.v.n[r];
        if (c.v.f[r]) p.f_pieces = r + 1;
    }
    p.P = c.g->P;
    p.tokens = (uint32_t)c.v.tokens;
    p.dim = (uint32_t)dim;
    c.prep.chunk_rows = (uint32_t)c.v.chunk_rows;
    p.sink = c.prep.sink = error_sink(c.g);
    workspace_extent(p, c);
    workspace_extent(c.prep, c);
    return DT_OK;
}

// What laying `bytes` out again takes before the products, in microseconds, in and out.
double again_us(double bytes) { return 3.0 + 2.0 * bytes / 4e6; }

// How the tokens' matrix is read: as one where the ranks' rows follow one another in
// memory, in the ranks' pieces where that takes no longer than laying them out again as one
// (77 tokens of 512 to 512 over 3 ranks: 5.7 us, in pieces 4.5).
void plan_tokens(Call &c, const void *const *x)
{
    const Plan &v = c.v;
    bool reads = true, follow = true, steps = true;
    const unsigned char *next = nullptr;
    uint64_t before = 0;
    for (int r = 0; r < c.g->P; ++r) {
        if (v.n[r] == 0) continue;
        reads = reads && addressable(x[r], v.dim);
        follow = follow && (!next || next == x[r]);
        next = static_cast<const unsigned char *>(x[r]) + v.n[r] * v.dim * 2;
        // as the inner axis, each piece but the last has to be whole steps of 16: a step's
        // other tokens would be the next rank's in the operand that is not in pieces
        // (times zero, but an infinity times zero is not zero)
        steps = steps && before % 16 == 0;
        before = v.n[r];
    }
    c.in_pieces = false;
    c.again = !(reads && follow);
    if (reads && !follow && (!back(v.kind) || steps)) {
        Cut one, pieces;
        cut(c.g, v, false, one);
        cut(c.g, v, true, pieces);
        c.in_pieces = pieces.us <= one.us + again_us(2.0 * v.tokens * v.dim);
        c.again = !c.in_pieces;
    }
}

// Its pieces, and what lays it out again.  sums: column sums of its rows are wanted.
void token_matrix(Call &c, const void *const *x, int buffer, float *sums)
{
    const Plan &v = c.v;
    uint32_t pieces = 0;
    c.tok_pitch = c.again ? up(v.dim, 8) : v.dim;
    uint64_t first = 0, chunk = 0;
    unsigned char *to = c.ws + v.tok;
    for (int r = 0; r < c.g->P; ++r) {
        if (v.n[r] == 0) continue;
        c.tok[pieces] = x[r];
        c.p.t_len[pieces++] = (uint32_t)v.n[r];
        if (c.again || sums)
            add_job(c, x[r], nullptr, c.again ? to + first * c.tok_pitch * 2 : nullptr, sums ? sums + chunk * v.dim : nullptr,
                    v.n[r], v.dim, c.tok_pitch, buffer + r, 0);
        chunk += tiles_of(v.n[r], v.chunk_rows);
        first += v.n[r];
    }
    if (c.again) c.tok[0] = to;
    if (!c.in_pieces) {
        pieces = 1;
        c.p.t_len[0] = c.p.tokens;
    }
    for (uint32_t k = 1; k < pieces; ++k) c.p.t_first[k] = c.p.t_first[k - 1] + c.p.t_len[k - 1];
    c.pieces = pieces;
    c.p.t_pieces = (int32_t)pieces;
}

// How small products are cut: CTAs of a cluster, and whether they share a tile's inner axis.
struct SmallCut {
    uint64_t mt[2], nt[2], kblocks[2], strips;
    uint32_t ctas, shared[2];
    double us;
};

// What they take, in microseconds: a launch, the longest CTA's round trips to memory, and
// in all so much for each step of a tile (measured at 17 to 1000 tokens of 100 to 1024,
// to 200 to 4096 features; rows at any element and an activation's derivative, whose two
// operands are two products, cost more: the gradient of 3 tokens of 164 to 4680 with gelu
// takes 26.6 us so and 11.4 in large tiles).
constexpr double kUsSmall = 5.0, kUsSmallStep = 0.45, kUsSmallSlope = 1.1, kUsSmallOdd = 0.35;

void small_cut(const dt_group *g, const Plan &v, bool sums, bool vec, bool slope, SmallCut &c)
{
    const bool b = back(v.kind), n_features = v.kind == dt::kGather || v.kind == dt::kReduceBack;
    const uint64_t tile = dt::kSmallTile, t = tiles_of(v.tokens, tile), d = tiles_of(v.dim, tile), f = feature_tiles(v, tile);
    c.mt[0] = t;
    c.nt[0] = c.nt[1] = n_features ? f : d;
    c.kblocks[0] = n_features ? d : f;
    c.mt[1] = b ? (gathers(v.kind) ? f : d) : 0;
    c.kblocks[1] = b ? t : 0;
    c.strips = sums ? (gathers(v.kind) ? f : d) : 0;
    uint64_t most = 0, steps = c.strips * t, longest = sums ? t : 0;
    for (int k = 0; k < 2; ++k) {
        c.shared[k] = c.kblocks[k] >= 4;
        if (c.shared[k]) most = std::max(most, c.kblocks[k]);
        steps += c.mt[k] * c.nt[k] * c.kblocks[k];
    }
    // two steps to a CTA at least; forward no more CTAs than SMs, which clusters of many
    // slow down (512 tokens of 512 to 512: 1, 2, 4, 8 CTAs 7.9, 8.5, 9.9, 12.6 us)
    c.ctas = 1;
    while (c.ctas < (b ? 8u : 4u) && c.ctas * 4 <= most &&
           (b || c.mt[0] * c.nt[0] * c.ctas * 2 <= dt::linear_workers(false, g->device)))
        c.ctas *= 2;
    for (int k = 0; k < 2; ++k) longest = std::max(longest, c.shared[k] ? tiles_of(c.kblocks[k], c.ctas) : c.kblocks[k]);
    const double step = b ? (slope ? 0.018 : 0.009) + (vec ? 0.0 : 0.004) : vec ? 0.0045 : 0.011;
    c.us = kUsSmall + std::max(longest * ((slope ? kUsSmallSlope : kUsSmallStep) + (vec ? 0.0 : kUsSmallOdd)), steps * step);
}

// What goes before the tensor core kernels' products, in microseconds: matrices that are
// laid out again, or (`written`) the ranks' features, which a job makes.
double prep_us(const Call &c, bool tok_again, const void *const *feat, const void *const *w, bool written)
{
    const Plan &v = c.v;
    double bytes = 0.0;
    bool feat_again = written, w_again = false;
    for (int r = 0; r < c.g->P; ++r) {
        if (feat && v.f[r]) feat_again = feat_again || !addressable(feat[r], v.f[r]);
        if (v.f[r]) w_again = w_again || !addressable(w[r], gathers(v.kind) ? v.dim : v.f[r]);
    }
    if (tok_again) bytes += 2.0 * v.tokens * v.dim;
    if (feat_again) bytes += (written ? 3.0 : 2.0) * v.tokens * v.features;
    if (w_again) bytes += 2.0 * v.features * v.dim;
    return bytes > 0.0 ? again_us(bytes) : 0.0;
}

// Small products where they are likely to take less time than the tensor core kernels':
// true where they were launched.  z: what act'(.) is taken of.
bool run_small(Call &c, const void *const *tok, const void *const *feat, const void *const *w, const void *const *z, int act,
               bool sums, bool written, cudaStream_t s, cudaError_t &e)
{
    const Plan &v = c.v;
    bool vec = true;
    for (int r = 0; r < c.g->P; ++r) {
        if (tok && v.n[r]) vec = vec && addressable(tok[r], v.dim);
        if (v.f[r] == 0) continue;
        if (feat) vec = vec && addressable(feat[r], v.f[r]) && (!z || addressable(z[r], v.f[r]));
        vec = vec && addressable(w[r], gathers(v.kind) ? v.dim : v.f[r]);
    }
    SmallCut t;
    small_cut(c.g, v, sums, vec, z != nullptr, t);
    Cut big;
    cut(c.g, v, tok && c.in_pieces, big);
    // A weight's gradient of few products: the large kernels' rounding of what stands before the
    // activation, which does not average out over them, is worth up to as much time again.  With
    // gelu, by this rule and without it: 4 tokens of 1024 to 4 x 256, results 1.65e-3 off by root
    // mean square and 2.4e-3, 8.7 and 8.6 us; where one rank's few features decide for all, 16
    // tokens of 1024 to 100 and 1000, 1.66e-3 and 2.4e-3, 13.4 and 9.4 us; 100 to 8 and 1000, the
    // same, 16.2 and 10.6.  (bf16 results alone are 1.66e-3 off.)
    bool near = false;
    for (int r = 0; r < c.g->P && written; ++r) near = near || (v.f[r] && v.f[r] * v.tokens < 2048);
    if (t.us >= (near ? 2.0 : 1.0) * (big.us + 3.0 + prep_us(c, tok && c.again, feat, w, written))) return false;
    dt::LinearSmall p;
    memset(&p, 0, sizeof p);
    static_cast<dt::LinearCall &>(p) = c.p;
    for (int r = 0; r < c.g->P; ++r) {
        p.tok[r] = tok ? static_cast<const uint16_t *>(tok[r]) : nullptr;
        p.feat[r] = feat ? static_cast<const uint16_t *>(feat[r]) : nullptr;
        p.weight[r] = static_cast<const uint16_t *>(w[r]);
        p.z[r] = z ? static_cast<const uint16_t *>(z[r]) : nullptr;
    }
    p.act = act;
    p.ctas = t.ctas;
    p.strips = (uint32_t)t.strips;
    uint32_t end = 0;
    for (int r = 0; r < c.g->P; ++r) {
        end += (uint32_t)tiles_of(v.f[r], dt::kSmallTile);
        p.product[0].f_end[r] = p.product[1].f_end[r] = end;
    }
    for (int k = 0; k < 2; ++k) {
        dt::LinearProduct &q = p.product[k];
        q.mt = (uint32_t)t.mt[k];
        q.nt = (uint32_t)t.nt[k];
        q.kblocks = (uint32_t)t.kblocks[k];
        p.shared[k] = t.shared[k];
        const uint32_t tiles = q.mt * q.nt;
        p.clusters[k] = t.shared[k] ? tiles : (tiles + t.ctas - 1) / t.ctas;
    }
    e = dt::launch_linear_small(p, v.kind, vec, s);
    return true;
}

// Whether few tokens' forward products go straight from memory to mma.sync: up to eight tokens
// until the weights are many times L2 (8 of 4096 to 16384, 134 MB: 27.9 us, in tensor core
// tiles 28.5; of 8192 to 28672, 470 MB: 77.5 and 73.5), up to 16, whose sums take registers
// from the loads in flight, while they are half of it (12 of 4096 to 8192: 12.7 and 13.9; to
// 16384: 32.7 and 29.0), and weights that TMA cannot read always.
bool few(const Call &c, const void *const *w)
{
    const Plan &v = c.v;
    if (v.tokens > dt::kFewTokens) return false;
    for (int r = 0; r < c.g->P; ++r)
        if (v.f[r] && !addressable(w[r], gathers(v.kind) ? v.dim : v.f[r])) return true;
    return 2.0 * v.features * v.dim <= (v.tokens <= 8 ? 256e6 : 72e6);
}

// The forward products of few tokens.
cudaError_t run_few(Call &c, const void *const *x, const void *const *w, cudaStream_t s)
{
    const Plan &v = c.v;
    const dt::LinearParams &p = c.p;
    dt::LinearFew f;
    memset(&f, 0, sizeof f);
    bool vec = true;
    const bool gather = v.kind == dt::kGather;
    for (int r = 0; r < c.g->P; ++r) {
        f.x[r] = static_cast<const uint16_t *>(x[r]);
        f.w[r] = static_cast<const uint16_t *>(w[r]);
        if (v.f[r]) vec = vec && addressable(w[r], gather ? v.dim : v.f[r]);
        if (gather ? v.n[r] : v.f[r]) vec = vec && addressable(x[r], gather ? v.dim : v.f[r]);
        f.out[r] = p.product[0].out[r];
        f.pre[r] = p.pre[r];
        f.bias[r] = p.bias[r];
        f.residual[r] = p.residual[r];
        f.f_len[r] = p.f_len[r];
        f.row_end[r] = p.row_end[r];
    }
    f.P = p.P;
    f.tokens = p.tokens;
    f.dim = p.dim;
    f.act = p.act;
    f.keep = p.keep;
    f.biased = p.biased;
    f.residuals = p.residuals;
    f.sink = p.sink;
#ifdef DT_BOUNDS
    memcpy(f.extent, p.extent, sizeof f.extent);
#endif
    return dt::launch_linear_few(f, v.kind, vec, c.g->device, s);
}

// A matrix for each rank, [rows, cols]: the map that reads it in place, or laid out
// again at `to`.
cudaError_t rank_matrix(Call &c, CUtensorMap *map, const void *src, size_t rows, size_t cols, unsigned char *&to, int buffer,
                        uint32_t box, bool written = false)
{
    if (rows == 0 || cols == 0) return cudaSuccess;
    const uint64_t pitch = up(cols, 8);
    unsigned char *dst = to;
    to += rows * pitch * 2;
    if (written) return dt::matrix_map(map, dst, cols, rows, pitch, box);
    if (addressable(src, cols)) return dt::matrix_map(map, src, cols, rows, cols, box);
    add_job(c, src, nullptr, dst, nullptr, rows, cols, pitch, buffer, 0);
    return dt::matrix_map(map, dst, cols, rows, pitch, box);
}

// The maps of all matrices, and the tiles.  feat: the ranks' [tokens, f] (written:
// a job before the products makes it in the workspace).
cudaError_t matrices(Call &c, const void *const *feat, int feat_buffer, bool written, const void *const *w)
{
    const Plan &v = c.v;
    dt::LinearParams &p = c.p;
    Cut t;
    cut(c.g, v, c.pieces > 1, t);
    const bool b = back(v.kind);
    p.bn = t.bn;
    // few tokens: boxes of as many as there are, in whole K steps of 16 where the
    // tokens are the inner axis
    p.rows_t = v.pairs ? 128 : (uint32_t)std::min<uint64_t>(128, up(v.tokens, b ? 16 : 8));
    p.rows_w = b ? 128 : t.bn / (v.pairs ? 2 : 1);
    cudaError_t e = cudaSuccess;
    if (v.kind != dt::kReduce)
        for (uint32_t k = 0; k < c.pieces && e == cudaSuccess; ++k)
            e = dt::matrix_map(&p.tok[k], c.tok[k], v.dim, p.t_len[k], c.tok_pitch, p.rows_t);
    unsigned char *to = c.ws + v.feat, *to_w = c.ws + v.w;
    for (int r = 0; r < c.g->P && e == cudaSuccess; ++r) {
        if (v.kind != dt::kGather)
            e = rank_matrix(c, &p.feat[r], feat[r], v.tokens, v.f[r], to, feat_buffer + r, p.rows_t, written);
        if (e == cudaSuccess)
            e = rank_matrix(c, &p.w[r], w[r], gathers(v.kind) ? v.f[r] : v.dim, gathers(v.kind) ? v.dim : v.f[r], to_w,
                            dt::kLinearW + r, p.rows_w);
    }
    for (int k = 0; k < (b ? 2 : 1); ++k) {
        dt::LinearProduct &q = p.product[k];
        q.mt = (uint32_t)t.mt[k];
        q.nt = (uint32_t)t.nt[k];
        q.kblocks = (uint32_t)t.kblocks[k];
        q.splits = (uint32_t)t.splits[k];
        q.tiles = q.mt * q.nt * q.splits;
        q.acc = reinterpret_cast<float *>(c.ws + v.acc[k]);
        // the size of a tile (its rows: of a half) or block along the features and the tokens here
        const bool n_features = v.kind == dt::kGather || v.kind == dt::kReduceBack;
        const uint64_t depth = dt::linear_depth(b), fs = n_features ? t.bn : k ? 128 : depth, ts = k ? depth : 128;
        uint32_t end = 0;
        for (int r = 0; r < c.g->P; ++r) q.f_end[r] = end += (uint32_t)tiles_of(v.f[r], fs);
        end = 0;
        for (uint32_t r = 0; r < c.pieces; ++r) q.t_end[r] = end += (uint32_t)tiles_of(p.t_len[r], ts);
    }
    return e;
}

// The launches of a call: what goes before, the products, and the splits' joins.
cudaError_t run(Call &c, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    if (c.prep.jobs) e = dt::launch_linear_prep(c.prep, s);
    if (e == cudaSuccess) e = dt::launch_linear(c.p, c.v.kind, c.v.pairs, c.g->device, s);
    for (int k = 0; k < 2 && e == cudaSuccess; ++k)
        if (c.p.product[k].splits > 1) e = dt::launch_linear_join(c.p, c.v.kind, k, c.v.pairs, s);
    return e;
}

cudaError_t zero_ranks(const dt_group *g, void *const *list, const size_t *n, const size_t *width, size_t equal, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    for (int r = 0; r < g->P && e == cudaSuccess; ++r) {
        const size_t bytes = n[r] * (width ? width[r] : equal) * 2;
        if (bytes) e = cudaMemsetAsync(list[r], 0, bytes, s);
    }
    return e;
}

bool valid_act(int act) { return act >= DT_ACT_NONE && act <= DT_ACT_SILU; }

}  // namespace

extern "C" {

dt_status dt_gather_linear(dt_group_t g, const void *const *x, const void *const *weight, const void *const *bias,
                           void *const *pre, void *const *y, const size_t *rows, size_t rows_equal, size_t dim,
                           const size_t *features, size_t features_equal, int dtype, int act, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    DT_TRACE();
    if (!g) return DT_ERR_INVALID;
    std::lock_guard<std::mutex> lock(g->mu);
    dt_status st = take_device_error(g);
    if (st != DT_OK) return st;
    Call c;
    c.g = g;
    st = begin(c, dt::kGather, rows, rows_equal, dim, features, features_equal, dtype, workspace, workspace_bytes);
    if (st != DT_OK) return st;
    if (!valid_act(act)) return DT_ERR_INVALID;
    const Plan &v = c.v;
    size_t n[DT_MAX_RANKS], one[DT_MAX_RANKS];
    std::fill(n, n + DT_MAX_RANKS, v.tokens);
    std::fill(one, one + DT_MAX_RANKS, (size_t)1);
    if ((st = take_ranks(c, x, v.n, nullptr, dim, false, dt::kLinearX)) != DT_OK) return st;
    if ((st = take_ranks(c, weight, v.f, nullptr, dim, false, dt::kLinearW)) != DT_OK) return st;
    if (bias && (st = take_ranks(c, bias, one, v.f, 0, false, dt::kLinearBias)) != DT_OK) return st;
    if (pre && (st = take_ranks(c, pre, n, v.f, 0, true, dt::kLinearPre)) != DT_OK) return st;
    if ((st = take_ranks(c, y, n, v.f, 0, true, dt::kLinearY)) != DT_OK) return st;
    if (c.b.clash()) return DT_ERR_INVALID;
    if (v.tokens == 0) return DT_OK;
    c.p.act = act;
    c.p.keep = pre != nullptr;
    c.p.biased = bias != nullptr;
    for (int r = 0; r < g->P; ++r) {
        if (v.f[r] == 0) continue;
        c.p.product[0].out[r] = static_cast<uint16_t *>(y[r]);
        c.p.pre[r] = pre ? static_cast<uint16_t *>(pre[r]) : nullptr;
        c.p.bias[r] = bias ? static_cast<const uint16_t *>(bias[r]) : nullptr;
        c.p.product[0].align[r] = alignment(alignment(8, y[r], v.f[r]), c.p.pre[r], v.f[r]);
    }
    DeviceScope scope(g->device);
    if (!scope.ok) return DT_ERR_CUDA;
    if (few(c, weight)) return cuda_status(run_few(c, x, weight, static_cast<cudaStream_t>(stream)));
    cudaError_t e = cudaSuccess;
    plan_tokens(c, x);
    if (run_small(c, x, nullptr, weight, nullptr, act, false, false, static_cast<cudaStream_t>(stream), e)) return cuda_status(e);
    token_matrix(c, x, dt::kLinearX, nullptr);
    e = matrices(c, nullptr, 0, false, weight);
    if (e == cudaSuccess) e = run(c, static_cast<cudaStream_t>(stream));
    return cuda_status(e);
}

dt_status dt_gather_linear_backward(dt_group_t g, const void *const *x, const void *const *weight, const void *const *pre,
                                    const void *const *dy, void *const *dx, void *const *dweight, void *const *dbias,
                                    const size_t *rows, size_t rows_equal, size_t dim, const size_t *features,
                                    size_t features_equal, int dtype, int act, void *workspace, size_t workspace_bytes,
                                    void *stream)
{
    DT_TRACE();
    if (!g) return DT_ERR_INVALID;
    std::lock_guard<std::mutex> lock(g->mu);
    dt_status st = take_device_error(g);
    if (st != DT_OK) return st;
    Call c;
    c.g = g;
    st = begin(c, dt::kGatherBack, rows, rows_equal, dim, features, features_equal, dtype, workspace, workspace_bytes);
    if (st != DT_OK) return st;
    if (!valid_act(act)) return DT_ERR_INVALID;
    if (act == DT_ACT_NONE) pre = nullptr;
    const Plan &v = c.v;
    size_t n[DT_MAX_RANKS], one[DT_MAX_RANKS];
    std::fill(n, n + DT_MAX_RANKS, v.tokens);
    std::fill(one, one + DT_MAX_RANKS, (size_t)1);
    if ((st = take_ranks(c, x, v.n, nullptr, dim, false, dt::kLinearX)) != DT_OK) return st;
    if ((st = take_ranks(c, weight, v.f, nullptr, dim, false, dt::kLinearW)) != DT_OK) return st;
    if (act != DT_ACT_NONE && (st = take_ranks(c, pre, n, v.f, 0, false, dt::kLinearPre)) != DT_OK) return st;
    if ((st = take_ranks(c, dy, n, v.f, 0, false, dt::kLinearDy)) != DT_OK) return st;
    if ((st = take_ranks(c, dx, v.n, nullptr, dim, true, dt::kLinearDx)) != DT_OK) return st;
    if ((st = take_ranks(c, dweight, v.f, nullptr, dim, true, dt::kLinearDw)) != DT_OK) return st;
    if (dbias && (st = take_ranks(c, dbias, one, v.f, 0, true, dt::kLinearDb)) != DT_OK) return st;
    if (c.b.clash()) return DT_ERR_INVALID;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceScope scope(g->device);
    if (!scope.ok) return DT_ERR_CUDA;
    if (v.tokens == 0) {
        cudaError_t e = zero_ranks(g, dweight, v.f, nullptr, dim, s);
        if (e == cudaSuccess && dbias) e = zero_ranks(g, dbias, one, v.f, 0, s);
        return cuda_status(e);
    }
    uint32_t tok_align = 8;
    for (int r = 0; r < g->P; ++r) {
        if (v.n[r]) {
            c.p.product[0].out[r] = static_cast<uint16_t *>(dx[r]);
            tok_align = alignment(tok_align, dx[r], dim);
        }
        if (v.f[r]) {
            c.p.product[1].out[r] = static_cast<uint16_t *>(dweight[r]);
            c.p.product[1].align[r] = alignment(8, dweight[r], dim);
        }
    }
    c.p.product[0].align[0] = tok_align;
    cudaError_t e = cudaSuccess;
    for (int r = 0; r < g->P; ++r) c.p.sums.out[r] = dbias ? static_cast<uint16_t *>(dbias[r]) : nullptr;
    plan_tokens(c, x);
    if (run_small(c, x, dy, weight, pre, act, dbias != nullptr, act != DT_ACT_NONE, s, e)) return cuda_status(e);
    c.prep.act = act;
    token_matrix(c, x, dt::kLinearX, nullptr);
    // G: dy itself where nothing is done to it and TMA can read it
    bool written = act != DT_ACT_NONE;
    for (int r = 0; r < g->P; ++r)
        if (v.f[r] && !addressable(dy[r], v.f[r])) written = true;
    // the bias' gradient: from dy, or from sums over chunks of the rows
    dt::LinearSums &sums = c.p.sums;
    const bool beside = !pre && sums_beside(g, v);
    float *part = reinterpret_cast<float *>(c.ws + v.sums);
    unsigned char *to = c.ws + v.feat;
    for (int r = 0; r < g->P; ++r) {
        const uint64_t pitch = up(v.f[r], 8);
        if (written || (dbias && !beside))
            add_job(c, dy[r], pre ? pre[r] : nullptr, written ? to : nullptr, dbias && !beside ? part : nullptr, v.tokens, v.f[r],
                    pitch, dt::kLinearDy + r, dt::kLinearPre + r);
        to += v.tokens * pitch * 2;
        if (!dbias) continue;
        sums.src[r] = beside ? dy[r] : part;
        sums.rows[r] = beside ? (uint32_t)v.tokens : (uint32_t)v.chunks;
        sums.cols[r] = (uint32_t)v.f[r];
        sums.group_end[r] = sums.groups += (uint32_t)tiles_of(v.f[r], 32);
        part += v.chunks * v.f[r];
    }
    sums.n = sums.sources = g->P;
    sums.f32 = !beside;
    e = matrices(c, dy, dt::kLinearDy, written, weight);
    if (e == cudaSuccess) e = run(c, s);
    return cuda_status(e);
}

size_t dt_gather_linear_workspace(dt_group_t g, const size_t *rows, size_t rows_equal, size_t dim, const size_t *features,
                                  size_t features_equal, int dtype, int backward)
{
    return workspace_bytes_of(g, dt::kGather, rows, rows_equal, dim, features, features_equal, dtype, backward);
}

dt_status dt_linear_reduce(dt_group_t g, const void *const *x, const void *const *weight, const void *bias,
                           const void *const *residual, void *const *y, const size_t *rows, size_t rows_equal, size_t dim,
                           const size_t *features, size_t features_equal, int dtype, void *workspace,
                           size_t workspace_bytes, void *stream)
{
    DT_TRACE();
    if (!g) return DT_ERR_INVALID;
    std::lock_guard<std::mutex> lock(g->mu);
    dt_status st = take_device_error(g);
    if (st != DT_OK) return st;
    Call c;
    c.g = g;
    st = begin(c, dt::kReduce, rows, rows_equal, dim, features, features_equal, dtype, workspace, workspace_bytes);
    if (st != DT_OK) return st;
    const Plan &v = c.v;
    size_t n[DT_MAX_RANKS], d[DT_MAX_RANKS];
    std::fill(n, n + DT_MAX_RANKS, v.tokens);
    std::fill(d, d + DT_MAX_RANKS, dim);
    if (!multiple(bias, 2)) return DT_ERR_INVALID;
    c.b.read(bias, dim * 2);
    dt::set_extent(c.p, dt::kLinearBias, bias, dim * 2, false);
    if ((st = take_ranks(c, x, n, v.f, 0, false, dt::kLinearX)) != DT_OK) return st;
    if ((st = take_ranks(c, weight, d, v.f, 0, false, dt::kLinearW)) != DT_OK) return st;
    // y may be the residual: a thread reads an element before it writes it
    if (residual && (st = take_ranks(c, residual, v.n, nullptr, dim, false, dt::kLinearResidual, 0)) != DT_OK) return st;
    if ((st = take_ranks(c, y, v.n, nullptr, dim, true, dt::kLinearY, 0)) != DT_OK) return st;
    if (c.b.clash()) return DT_ERR_INVALID;
    if (v.tokens == 0) return DT_OK;
    c.p.biased = bias != nullptr;
    c.p.bias[0] = static_cast<const uint16_t *>(bias);
    c.p.residuals = residual != nullptr;
    uint32_t align = 8;
    for (int r = 0; r < g->P; ++r) {
        if (v.n[r] == 0) continue;
        c.p.product[0].out[r] = static_cast<uint16_t *>(y[r]);
        c.p.residual[r] = residual ? static_cast<const uint16_t *>(residual[r]) : nullptr;
        align = alignment(alignment(align, y[r], dim), c.p.residual[r], dim);
    }
    c.p.product[0].align[0] = align;
    DeviceScope scope(g->device);
    if (!scope.ok) return DT_ERR_CUDA;
    if (few(c, weight)) return cuda_status(run_few(c, x, weight, static_cast<cudaStream_t>(stream)));
    cudaError_t e = cudaSuccess;
    if (run_small(c, nullptr, x, weight, nullptr, DT_ACT_NONE, false, false, static_cast<cudaStream_t>(stream), e))
        return cuda_status(e);
    c.pieces = 1;
    c.p.t_pieces = 1;
    c.p.t_len[0] = c.p.tokens;
    e = matrices(c, x, dt::kLinearX, false, weight);
    if (e == cudaSuccess) e = run(c, static_cast<cudaStream_t>(stream));
    return cuda_status(e);
}

dt_status dt_linear_reduce_backward(dt_group_t g, const void *const *x, const void *const *weight, const void *const *dy,
                                    void *const *dx, void *const *dweight, void *dbias, const size_t *rows,
                                    size_t rows_equal, size_t dim, const size_t *features, size_t features_equal, int dtype,
                                    void *workspace, size_t workspace_bytes, void *stream)
{
    DT_TRACE();
    if (!g) return DT_ERR_INVALID;
    std::lock_guard<std::mutex> lock(g->mu);
    dt_status st = take_device_error(g);
    if (st != DT_OK) return st;
    Call c;
    c.g = g;
    st = begin(c, dt::kReduceBack, rows, rows_equal, dim, features, features_equal, dtype, workspace, workspace_bytes);
    if (st != DT_OK) return st;
    const Plan &v = c.v;
    size_t n[DT_MAX_RANKS], d[DT_MAX_RANKS];
    std::fill(n, n + DT_MAX_RANKS, v.tokens);
    std::fill(d, d + DT_MAX_RANKS, dim);
    if ((st = take_ranks(c, x, n, v.f, 0, false, dt::kLinearX)) != DT_OK) return st;
    if ((st = take_ranks(c, weight, d, v.f, 0, false, dt::kLinearW)) != DT_OK) return st;
    if ((st = take_ranks(c, dy, v.n, nullptr, dim, false, dt::kLinearDy)) != DT_OK) return st;
    if ((st = take_ranks(c, dx, n, v.f, 0, true, dt::kLinearDx)) != DT_OK) return st;
    if ((st = take_ranks(c, dweight, d, v.f, 0, true, dt::kLinearDw)) != DT_OK) return st;
    if (!multiple(dbias, 2)) return DT_ERR_INVALID;
    c.b.write(dbias, dim * 2);
    dt::set_extent(c.p, dt::kLinearDb, dbias, dim * 2, true);
    if (c.b.clash()) return DT_ERR_INVALID;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeviceScope scope(g->device);
    if (!scope.ok) return DT_ERR_CUDA;
    if (v.tokens == 0) {
        cudaError_t e = zero_ranks(g, dweight, d, v.f, 0, s);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, dim * 2, s);
        return cuda_status(e);
    }
    for (int r = 0; r < g->P; ++r) {
        if (v.f[r] == 0) continue;
        c.p.product[0].out[r] = static_cast<uint16_t *>(dx[r]);
        c.p.product[1].out[r] = static_cast<uint16_t *>(dweight[r]);
        c.p.product[0].align[r] = alignment(8, dx[r], v.f[r]);
        c.p.product[1].align[r] = alignment(8, dweight[r], v.f[r]);
    }
    cudaError_t e = cudaSuccess;
    c.p.sums.out[0] = static_cast<uint16_t *>(dbias);
    plan_tokens(c, dy);
    if (run_small(c, dy, x, weight, nullptr, DT_ACT_NONE, dbias != nullptr, false, s, e)) return cuda_status(e);
    // the bias' gradient: from the ranks' dy, or from sums over chunks of the rows
    float *part = reinterpret_cast<float *>(c.ws + v.sums);
    const bool beside = sums_beside(g, v);
    token_matrix(c, dy, dt::kLinearDy, dbias && !beside ? part : nullptr);
    if (dbias) {
        dt::LinearSums &sums = c.p.sums;
        sums.cols[0] = (uint32_t)dim;
        sums.group_end[0] = sums.groups = (uint32_t)tiles_of(dim, 32);
        sums.n = sums.stacked = 1;
        sums.sources = beside ? g->P : 1;
        sums.f32 = !beside;
        sums.src[0] = part;
        sums.rows[0] = (uint32_t)v.chunks;
        for (int r = 0; r < g->P && beside; ++r) {
            sums.src[r] = dy[r];
            sums.rows[r] = (uint32_t)v.n[r];
        }
    }
    e = matrices(c, x, dt::kLinearX, false, weight);
    if (e == cudaSuccess) e = run(c, s);
    return cuda_status(e);
}

size_t dt_linear_reduce_workspace(dt_group_t g, const size_t *rows, size_t rows_equal, size_t dim, const size_t *features,
                                  size_t features_equal, int dtype, int backward)
{
    return workspace_bytes_of(g, dt::kReduce, rows, rows_equal, dim, features, features_equal, dtype, backward);
}

}  // extern "C"
