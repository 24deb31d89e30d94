// C ABI entry points of the residual norm: argument checks, by the conventions of the
// other calls (dt_ops.cpp).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "dt_group.h"
#include "dt_host.h"
#include "dt_residual.h"

namespace {

using namespace dt::host;

constexpr size_t kMaxCols = (size_t)1 << 24;

// What both passes check and set: the rows, the types and the weights.
struct Call {
    dt_group *g;
    dt::ResidualParams p;
    size_t n[DT_MAX_RANKS];
    size_t es, ws, cols;
    bool vec;
    Buffers b;

    dt_status begin(const size_t *rows, size_t rows_equal, size_t columns, int dtype, int weight_dtype, const void *post,
                    const void *gate, const void *pre, float scale)
    {
        if (!valid_dtype(dtype) || !valid_dtype(weight_dtype)) return DT_ERR_INVALID;
        if (!float_dtype(dtype) || !float_dtype(weight_dtype)) return DT_ERR_UNSUPPORTED;
        if (columns == 0 || columns > kMaxCols || !std::isfinite(scale)) return DT_ERR_INVALID;
        cols = columns;
        es = elem_bytes(dtype);
        ws = elem_bytes(weight_dtype);
        size_t total = 0;
        if (!row_counts(g->P, rows, rows_equal, cols * es, n, &total)) return DT_ERR_INVALID;
        memset(&p, 0, sizeof p);
        vec = cols * es % 16 == 0;
        uint64_t end = 0;
        for (int r = 0; r < g->P; ++r) p.row_end[r] = end += n[r];
        p.rows = total;
        p.cols = (uint32_t)cols;
        p.inv_cols = 1.0f / (float)cols;
        p.P = g->P;
        p.post = post;
        p.gate = gate;
        p.pre = pre;
        p.scale = scale;
        p.weight_bf16 = weight_dtype == DT_BF16;
        p.sink = error_sink(g);
        const void *const w[3] = {post, gate, pre};
        for (int k = 0; k < 3; ++k) {
            if (!multiple(w[k], ws)) return DT_ERR_INVALID;
            b.read(w[k], cols * ws);
            dt::set_extent(p, dt::kResidualPost + k, w[k], cols * ws, false);
        }
        return DT_OK;
    }
    // The ranks' matrices of rows; an output with tag t may be the input with that tag.
    dt_status source(int which, const void *const *list, int tag = -1)
    {
        for (int r = 0; r < g->P; ++r) {
            if (n[r] == 0) continue;
            if (!list || !list[r] || !multiple(list[r], es)) return DT_ERR_INVALID;
            p.src[which][r] = list[r];
            vec = vec && aligned16(list[r]);
            b.read(list[r], n[r] * cols * es, tag < 0 ? -1 : tag * DT_MAX_RANKS + r);
            dt::set_extent(p, which * DT_MAX_RANKS + r, list[r], n[r] * cols * es, false);
        }
        return DT_OK;
    }
    dt_status output(int which, void *const *list, int tag)
    {
        for (int r = 0; r < g->P; ++r) {
            if (n[r] == 0) continue;
            if (!list || !list[r] || !multiple(list[r], es)) return DT_ERR_INVALID;
            p.out[which][r] = list[r];
            vec = vec && aligned16(list[r]);
            b.write(list[r], n[r] * cols * es, tag * DT_MAX_RANKS + r);
            dt::set_extent(p, dt::kResidualOut + which * DT_MAX_RANKS + r, list[r], n[r] * cols * es, true);
        }
        return DT_OK;
    }
    dt_status rstds(int which, const float *const *list, bool written)
    {
        if (!list && written) return DT_OK;
        for (int r = 0; r < g->P; ++r) {
            if (n[r] == 0) continue;
            if (!list || (!list[r] && !written) || !multiple(list[r], 4)) return DT_ERR_INVALID;
            p.rstd[which][r] = const_cast<float *>(list[r]);
            if (written) b.write(list[r], n[r] * 4);
            else b.read(list[r], n[r] * 4);
            dt::set_extent(p, dt::kResidualRstd + which * DT_MAX_RANKS + r, list[r], n[r] * 4, written);
        }
        return DT_OK;
    }
};

}  // namespace

extern "C" {

dt_status dt_residual_norm(dt_group_t g, const void *const *x, const void *const *branch, const void *post_weight,
                           const void *gate, const void *pre_weight, float residual_scale, void *const *y, void *const *z,
                           float *const *rstd_post, float *const *rstd_pre, const size_t *rows, size_t rows_equal,
                           size_t cols, float eps, int dtype, int weight_dtype, void *stream)
{
    DT_TRACE();
    if (!g) return DT_ERR_INVALID;
    std::lock_guard<std::mutex> lock(g->mu);
    dt_status st = take_device_error(g);
    if (st != DT_OK) return st;
    Call c;
    c.g = g;
    st = c.begin(rows, rows_equal, cols, dtype, weight_dtype, post_weight, gate, pre_weight, residual_scale);
    if (st != DT_OK) return st;
    if (!(eps >= 0.0f) || std::isinf(eps)) return DT_ERR_INVALID;
    if ((st = c.source(dt::kX, x, 0)) != DT_OK || (st = c.source(dt::kBranch, branch, 1)) != DT_OK) return st;
    if ((st = c.output(0, y, 0)) != DT_OK || (st = c.output(1, z, 1)) != DT_OK) return st;
    if ((st = c.rstds(0, rstd_post, true)) != DT_OK || (st = c.rstds(1, rstd_pre, true)) != DT_OK) return st;
    if (c.b.clash()) return DT_ERR_INVALID;
    if (c.p.rows == 0) return DT_OK;
    c.p.eps = eps;
    DeviceScope scope(g->device);
    if (!scope.ok) return DT_ERR_CUDA;
    return cuda_status(dt::launch_residual(c.p, dtype, c.vec, g->device, static_cast<cudaStream_t>(stream)));
}

dt_status dt_residual_norm_backward(dt_group_t g, const void *const *branch, const void *const *y, const void *const *dy,
                                    const void *const *dz, const void *post_weight, const void *gate, const void *pre_weight,
                                    float residual_scale, const float *const *rstd_post, const float *const *rstd_pre,
                                    void *const *dx, void *const *dbranch, void *dpost_weight, void *dgate, void *dpre_weight,
                                    const size_t *rows, size_t rows_equal, size_t cols, int dtype, int weight_dtype, int op,
                                    void *workspace, size_t workspace_bytes, void *stream)
{
    DT_TRACE();
    if (!g) return DT_ERR_INVALID;
    std::lock_guard<std::mutex> lock(g->mu);
    dt_status st = take_device_error(g);
    if (st != DT_OK) return st;
    Call c;
    c.g = g;
    st = c.begin(rows, rows_equal, cols, dtype, weight_dtype, post_weight, gate, pre_weight, residual_scale);
    if (st != DT_OK) return st;
    if (!valid_op(op)) return DT_ERR_INVALID;
    if (op != DT_SUM && op != DT_AVG) return DT_ERR_UNSUPPORTED;
    const bool sums = dpost_weight || dgate || dpre_weight;
    if (!multiple(dpost_weight, c.ws) || !multiple(dgate, c.ws) || !multiple(dpre_weight, c.ws)) return DT_ERR_INVALID;
    if (sums && (!workspace || !aligned16(workspace) || workspace_bytes < dt::residual_workspace(c.p.cols, g->device)))
        return DT_ERR_INVALID;
    if ((st = c.source(dt::kBranch, branch)) != DT_OK || (st = c.source(dt::kY, y)) != DT_OK) return st;
    if (dy && (st = c.source(dt::kDy, dy, 0)) != DT_OK) return st;
    if ((st = c.source(dt::kDz, dz, 1)) != DT_OK) return st;
    if ((st = c.output(0, dx, 0)) != DT_OK || (st = c.output(1, dbranch, 1)) != DT_OK) return st;
    if ((st = c.rstds(0, rstd_post, false)) != DT_OK || (st = c.rstds(1, rstd_pre, false)) != DT_OK) return st;
    void *const grads[3] = {dpost_weight, dgate, dpre_weight};
    for (int k = 0; k < 3; ++k) {
        c.b.write(grads[k], cols * c.ws);
        dt::set_extent(c.p, dt::kResidualDpost + k, grads[k], cols * c.ws, true);
    }
    if (sums) c.b.write(workspace, workspace_bytes);
    if (c.b.clash()) return DT_ERR_INVALID;
    if (c.p.rows == 0 && !sums) return DT_OK;
    c.p.has_dy = dy != nullptr;
    c.p.dpost = dpost_weight;
    c.p.dgate = dgate;
    c.p.dpre = dpre_weight;
    c.p.partial = sums ? static_cast<float *>(workspace) : nullptr;
    dt::set_extent(c.p, dt::kResidualWorkspace, workspace, sums ? workspace_bytes : 0, false);
    c.p.avg = op == DT_AVG;
    c.p.avg_pow2 = (g->P & (g->P - 1)) == 0;
    c.p.avg_scale = c.p.avg_pow2 ? 1.0f / (float)g->P : 0.0f;
    DeviceScope scope(g->device);
    if (!scope.ok) return DT_ERR_CUDA;
    return cuda_status(dt::launch_residual_backward(c.p, dtype, c.vec, g->device, static_cast<cudaStream_t>(stream)));
}

size_t dt_residual_norm_workspace(dt_group_t g, size_t cols)
{
    if (!g || cols == 0 || cols > kMaxCols) return 0;
    return dt::residual_workspace((uint32_t)cols, g->device);
}

}  // extern "C"
