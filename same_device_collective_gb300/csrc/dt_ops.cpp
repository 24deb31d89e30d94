// C ABI entry points of the layer norm and the vocabulary loss: argument
// checks and launch planning.  They follow the collectives' conventions: every
// argument error is reported before anything is enqueued, device memory is the
// caller's, no call waits for the GPU and none throws.
#include <cmath>
#include <cstring>

#include "dt_group.h"
#include "dt_host.h"
#include "dt_ops.h"

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
        vec = vec && aligned16(x[r]) && aligned16(out[r]);
    }
    p.rows = total;
    p.cols = (uint32_t)cols;
    p.P = g->P;
    p.weight = weight;
    p.weight_bf16 = weight_dtype == DT_BF16;
    p.sink = error_sink(g);
    return DT_OK;
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
    }
    if (b.clash()) return DT_ERR_INVALID;
    if (p.rows == 0) return DT_OK;
    p.bias = bias;
    p.eps = eps;
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
    }
    b.write(dweight, cols * ws);
    b.write(dbias, cols * ws);
    if (sums) b.write(workspace, workspace_bytes);
    if (b.clash()) return DT_ERR_INVALID;
    if (p.rows == 0 && !sums) return DT_OK;
    p.dweight = dweight;
    p.dbias = dbias;
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

}  // extern "C"
