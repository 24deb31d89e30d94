// The linear layers' entry points with their launches taken out: what a call hands to the
// tensor core kernels, on the host alone.  Every tile's loads have to go through a tensor map
// that was made, the tiles have to cover every output once, and what a call lays out in the
// workspace lies within it and apart.  Prints what it saw; nothing is launched.
#include <cuda_runtime.h>

static cudaError_t no_get_device(int *d) { *d = 0; return cudaSuccess; }
static cudaError_t no_set_device(int) { return cudaSuccess; }
static cudaError_t no_memset(void *, int, size_t, cudaStream_t) { return cudaSuccess; }
#define cudaGetDevice no_get_device
#define cudaSetDevice no_set_device
#define cudaMemsetAsync no_memset

#include "dt_linear.cpp"
#include "dt_linear.cuh"

#include <cstdio>
#include <cstdlib>
#include <vector>

// What stands in a map's 128 bytes here; a map that was not made is zeros.
struct Map {
    uint64_t made, base, cols, rows, pitch, box;
};
constexpr uint64_t kMade = 0x5EED5EED5EED5EEDull;

static const unsigned char *workspace;
static size_t workspace_bytes;
static int launches, past_the_end, failures;

// What a call writes to its workspace before and between its products.
struct Part {
    uint64_t from, to;
};
static std::vector<Part> parts;

#define EXPECT(ok)                                                                    \
    do {                                                                              \
        if (!(ok) && ++failures <= 5) printf("line %d: %s\n", __LINE__, #ok);          \
    } while (0)

static void part(const void *from, uint64_t bytes)
{
    if (bytes) parts.push_back(Part{(uint64_t)from, (uint64_t)from + bytes});
}

static void check_parts()
{
    const uint64_t lo = (uint64_t)workspace, hi = lo + workspace_bytes;
    for (size_t i = 0; i < parts.size(); ++i) {
        EXPECT(parts[i].from >= lo && parts[i].to <= hi);
        for (size_t j = 0; j < i; ++j) EXPECT(parts[i].from >= parts[j].to || parts[j].from >= parts[i].to);
    }
}

// A map of the workspace reads what was laid out there, which may be several ranks' rows as one.
static void check_map(const Map &m)
{
    const uint64_t lo = (uint64_t)workspace, hi = lo + workspace_bytes, end = m.base + ((m.rows - 1) * m.pitch + m.cols) * 2;
    if (m.made != kMade || m.base + 1 <= lo || m.base >= hi) return;
    uint64_t at = m.base;
    for (size_t i = 0; i < parts.size() && at < end; ++i)
        if (parts[i].from <= at && at < parts[i].to) at = parts[i].to;
    EXPECT(at >= end);
}

static const Map &of(const CUtensorMap &m) { return reinterpret_cast<const Map &>(m); }

// The map that a matrix is read through at these places, and the first column and row there.
template <class R>
static const Map &operand(const dt::LinearParams &p, int matrix, const dt::Place (&at)[3], uint64_t &col, uint64_t &row)
{
    const dt::Place &t = at[dt::kTokens], &d = at[dt::kDim], &f = at[dt::kFeatures];
    col = matrix == dt::kTok ? d.at : matrix == dt::kFeat ? f.at : R::w_by_feature ? d.at : f.at;
    row = matrix == dt::kTok ? t.at : matrix == dt::kFeat ? t.all : R::w_by_feature ? f.at : d.at;
    return of(matrix == dt::kTok ? p.tok[t.piece] : matrix == dt::kFeat ? p.feat[f.piece] : p.w[f.piece]);
}

static bool sums_at(const void *from, uint64_t bytes)
{
    uint64_t at = (uint64_t)from;
    for (size_t i = 0; i < parts.size() && at < (uint64_t)from + bytes; ++i)
        if (parts[i].from <= at && at < parts[i].to) at = parts[i].to;
    return at >= (uint64_t)from + bytes;
}

template <class R>
static void walk(const dt::LinearParams &p, const dt::LinearProduct &c, bool pairs)
{
    const uint32_t halves = pairs ? 2 : 1;
    uint64_t rows = 0, cols = 0, deep = 0;
    EXPECT(c.mt && c.nt && c.kblocks && c.splits && c.splits <= c.kblocks && c.tiles == c.mt * c.nt * c.splits);
    for (uint32_t i = 0; i < c.mt * halves; ++i)
        for (uint32_t j = 0; j < c.nt; ++j)
            for (uint32_t k = 0; k < c.kblocks; ++k) {
                dt::Place at[3] = {};
                at[R::m] = dt::locate<R, R::m>(p, c, i, 128);
                at[R::n] = dt::locate<R, R::n>(p, c, j, p.bn);
                at[R::k] = dt::locate<R, R::k>(p, c, k, R::depth);
                const uint32_t m = dt::length<R, R::m>(p, at[R::m].piece), n = dt::length<R, R::n>(p, at[R::n].piece),
                               l = dt::length<R, R::k>(p, at[R::k].piece);
                for (int matrix : {R::a, R::b}) {
                    uint64_t col, row;
                    const Map &map = operand<R>(p, matrix, at, col, row);
                    EXPECT(map.made == kMade && map.base % 16 == 0 && map.pitch % 8 == 0 && col % 8 == 0);
                    EXPECT(map.box >= 1 && map.box <= 256 && map.cols >= 1 && map.rows >= 1);
                }
                EXPECT(at[R::n].at < n && at[R::k].at < l);
                if (at[R::m].at >= m) {
                    ++past_the_end;
                    EXPECT(i == c.mt * halves - 1);   // only the last half of all
                }
                if (j == 0 && k == 0) rows += at[R::m].at < m ? std::min<uint64_t>(128, m - at[R::m].at) : 0;
                if (i == 0 && k == 0) cols += std::min<uint64_t>(p.bn, n - at[R::n].at);
                if (i == 0 && j == 0) deep += std::min<uint64_t>(R::depth, l - at[R::k].at);
            }
    uint64_t features = 0;
    for (int r = 0; r < p.P; ++r) features += p.f_len[r];
    auto all = [&](int axis) { return axis == dt::kDim ? (uint64_t)p.dim : axis == dt::kTokens ? (uint64_t)p.tokens : features; };
    EXPECT(rows == all(R::m) && cols == all(R::n) && deep == all(R::k));
    if (c.splits > 1) part(c.acc, (uint64_t)c.splits * c.mt * halves * 128 * c.nt * p.bn * 4);
}

namespace dt {

cudaError_t matrix_map(CUtensorMap *map, const void *base, uint64_t cols, uint64_t rows, uint64_t pitch, uint32_t box_rows)
{
    reinterpret_cast<Map &>(*map) = Map{kMade, (uint64_t)base, cols, rows, pitch, box_rows};
    return cudaSuccess;
}
cudaError_t launch_linear(LinearParams &p, LinearKind kind, bool pairs, int, cudaStream_t)
{
    ++launches;
    for (int r = 0; r < p.P; ++r) {
        check_map(of(p.tok[r]));
        check_map(of(p.feat[r]));
        check_map(of(p.w[r]));
        if (p.sums.f32 && r < (p.sums.stacked ? 1 : p.sums.n) && p.sums.groups)   // sums of chunks are all there
            EXPECT(!p.sums.cols[r] || sums_at(p.sums.src[r], (uint64_t)p.sums.rows[r] * p.sums.cols[r] * 4));
    }
    switch (kind) {
    case kGather: walk<Roles<kGather, false>>(p, p.product[0], pairs); break;
    case kReduce: walk<Roles<kReduce, false>>(p, p.product[0], pairs); break;
    case kGatherBack:
        walk<Roles<kGatherBack, false>>(p, p.product[0], pairs);
        walk<Roles<kGatherBack, true>>(p, p.product[1], pairs);
        break;
    default:
        walk<Roles<kReduceBack, false>>(p, p.product[0], pairs);
        walk<Roles<kReduceBack, true>>(p, p.product[1], pairs);
    }
    check_parts();
    parts.clear();
    return cudaSuccess;
}
cudaError_t launch_linear_join(const LinearParams &, LinearKind, int, bool, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_linear_few(LinearFew &, LinearKind, bool, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_linear_small(const LinearSmall &, LinearKind, bool, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_linear_prep(LinearPrep &p, cudaStream_t)
{
    EXPECT(p.jobs >= 1 && p.jobs <= kPrepJobs && p.chunk_rows % 32 == 0);
    uint32_t blocks = 0;
    for (int k = 0; k < p.jobs; ++k) {
        const LinearPrepJob &j = p.job[k];
        const uint32_t chunks = (j.rows + p.chunk_rows - 1) / p.chunk_rows;
        EXPECT(j.rows && j.cols && j.pitch >= j.cols && j.pitch % 8 == 0 && j.strips == (j.cols + kPrepCols - 1) / kPrepCols);
        EXPECT(j.block_end - blocks == chunks * j.strips && (j.dst || j.sums));
        blocks = j.block_end;
        if (j.dst) part(j.dst, (uint64_t)j.rows * j.pitch * 2);
        if (j.sums) part(j.sums, (uint64_t)chunks * j.cols * 4);
    }
    return cudaSuccess;
}
uint32_t linear_workers(bool pairs, int) { return pairs ? 76 : 152; }

}  // namespace dt

// All four calls.  Addresses only: 4 GB of them to each buffer, `offset` bytes past a boundary.
static void call(int P, const size_t *rows, size_t dim, const size_t *features, size_t offset, int act)
{
    dt::DevError none = {};
    dt_group g;
    g.P = P;
    g.h_err = &none;
    const void *list[8][DT_MAX_RANKS];
    for (int k = 0; k < 8; ++k)
        for (int r = 0; r < P; ++r) list[k][r] = reinterpret_cast<const void *>(((uint64_t)(k * P + r + 1) << 32) + offset);
    void *const *out[3] = {const_cast<void *const *>(list[5]), const_cast<void *const *>(list[6]), const_cast<void *const *>(list[7])};
    void *ws = reinterpret_cast<void *>((uint64_t)1 << 44);
    workspace = static_cast<const unsigned char *>(ws);
    auto room = [&](bool gather, int back) {
        return workspace_bytes = gather ? dt_gather_linear_workspace(&g, rows, 0, dim, features, 0, DT_BF16, back)
                                        : dt_linear_reduce_workspace(&g, rows, 0, dim, features, 0, DT_BF16, back);
    };
    size_t n = room(true, 0);
    EXPECT(dt_gather_linear(&g, list[0], list[1], list[2], nullptr, out[0], rows, 0, dim, features, 0, DT_BF16, act, ws, n, nullptr) == DT_OK);
    n = room(true, 1);
    EXPECT(dt_gather_linear_backward(&g, list[0], list[1], act ? list[2] : nullptr, list[3], out[0], out[1], out[2], rows, 0, dim,
                                     features, 0, DT_BF16, act, ws, n, nullptr) == DT_OK);
    n = room(false, 0);
    EXPECT(dt_linear_reduce(&g, list[0], list[1], list[2][0], nullptr, out[0], rows, 0, dim, features, 0, DT_BF16, ws, n, nullptr) == DT_OK);
    n = room(false, 1);
    EXPECT(dt_linear_reduce_backward(&g, list[0], list[1], list[3], out[0], out[1], out[2][0], rows, 0, dim, features, 0, DT_BF16, ws, n,
                                     nullptr) == DT_OK);
}

int main()
{
    struct { size_t rows[4], dim, features[4]; } const shapes[] = {
        {{1024, 1024}, 512, {1100, 0}}, {{2000, 48, 0, 0}, 264, {1500, 700, 0, 0}}, {{100, 0, 33, 7}, 1024, {0, 2000, 72, 0}},
        {{300, 212, 0, 1}, 1030, {130, 0, 0, 0}}, {{0, 0, 0, 4000}, 136, {0, 0, 0, 1160}}, {{129, 0, 0, 0}, 4096, {0, 128, 0, 0}}};
    for (const auto &s : shapes)
        for (int P = 2; P <= 4; ++P)
            for (size_t offset : {0, 2})
                if (s.features[0] + s.features[1] + (P > 2 ? s.features[2] : 0) + (P > 3 ? s.features[3] : 0))
                    call(P, s.rows, s.dim, s.features, offset, P % 4);
    srand(1);
    for (int k = 0; k < 300; ++k) {
        const int P = 1 + rand() % DT_MAX_RANKS;
        size_t rows[DT_MAX_RANKS], features[DT_MAX_RANKS], all = 0;
        for (int r = 0; r < P; ++r) {
            rows[r] = rand() % 3 ? rand() % (4000 / P + 1) : rand() % 2 * 16;
            features[r] = rand() % 3 ? rand() % (4000 / P + 1) : 0;
            if (rand() % 2) features[r] = features[r] / 8 * 8;
            all += features[r];
        }
        if (!all) features[0] = 200;
        const size_t dim = rand() % 2 ? 8 + rand() % 150 * 8 : 1 + rand() % 1200;
        call(P, rows, dim, features, rand() % 3 ? 0 : 2, rand() % 4);
    }
    printf("%d launches, %d halves past the end, %d failures\n", launches, past_the_end, failures);
    return failures || !launches || !past_the_end;
}
