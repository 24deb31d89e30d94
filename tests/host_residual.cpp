// The residual norm's entry points with their launches taken out, for groups of 1 to 16
// ranks: what they register and refuse, on the host alone.  Prints "ok" at the end.
#include "dt_residual.cpp"

#include <cstdio>

namespace {

int launched;
dt::ResidualParams seen;

}  // namespace

namespace dt {

cudaError_t launch_residual(ResidualParams p, int, bool, int, cudaStream_t) { seen = p, ++launched; return cudaSuccess; }
cudaError_t launch_residual_backward(ResidualParams p, int, bool, int, cudaStream_t) { seen = p, ++launched; return cudaSuccess; }
size_t residual_workspace(uint32_t cols, int) { return (size_t)cols * 8; }

}  // namespace dt

extern "C" cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
extern "C" cudaError_t cudaSetDevice(int) { return cudaSuccess; }

namespace {

#define CHECK(ok)                                                        \
    do {                                                                 \
        if (!(ok)) {                                                     \
            printf("line %d: %s (P = %d)\n", __LINE__, #ok, P);          \
            return 1;                                                    \
        }                                                                \
    } while (0)

// A megabyte of addresses to each buffer; nothing is read or written.
struct Lists {
    float *at[DT_MAX_RANKS];
    Lists(int which)
    {
        for (int r = 0; r < DT_MAX_RANKS; ++r) at[r] = reinterpret_cast<float *>(((uintptr_t)which * DT_MAX_RANKS + r + 1) << 20);
    }
    operator const void *const *() const { return reinterpret_cast<const void *const *>(at); }
    operator void *const *() const { return reinterpret_cast<void *const *>(const_cast<float *const *>(at)); }
};

int run(int P)
{
    dt::DevError none = {};
    dt_group g;
    g.P = P;
    g.h_err = &none;
    const size_t rows = 3, cols = 8;
    float *const post = Lists(20).at[0], *const gate = Lists(20).at[1], *const pre = Lists(20).at[2];
    const Lists x(1), branch(2), y(3), z(4), dx(7), dbranch(8);
    auto forward = [&](const Lists &y_, const Lists &rpost, const Lists &rpre) {
        return dt_residual_norm(&g, x, branch, post, gate, pre, 1.0f, y_, z, rpost.at, rpre.at, nullptr, rows, cols, 1e-6f, DT_F32,
                                DT_F32, nullptr);
    };
    const Lists rpost(5), rpre(6);
    launched = 0;
    CHECK(forward(y, rpost, rpre) == DT_OK && launched == 1);
    for (int r = 0; r < P; ++r) {
        CHECK(seen.row_end[r] == rows * (r + 1) && seen.rstd[0][r] == rpost.at[r] && seen.rstd[1][r] == rpre.at[r]);
        CHECK(seen.src[dt::kX][r] == x.at[r] && seen.out[0][r] == y.at[r] && seen.out[1][r] == z.at[r]);
    }
    // the last of all outputs, over the first, over the one before it, and over an input
    for (float *over : {y.at[0], rpost.at[P - 1], x.at[P - 1], post}) {
        Lists bad(6);
        bad.at[P - 1] = over;
        CHECK(forward(y, rpost, bad) == DT_ERR_INVALID && launched == 1);
    }
    CHECK(forward(x, rpost, rpre) == DT_OK && launched == 2);   // in place

    const Lists dy(9), dz(10);
    auto backward = [&](const Lists &dbranch_, const Lists &rpre_, void *workspace) {
        return dt_residual_norm_backward(&g, branch, y, dy, dz, post, gate, pre, 1.0f, rpost.at, rpre_.at, dx, dbranch_,
                                         Lists(21).at[0], Lists(21).at[1], Lists(21).at[2], nullptr, rows, cols, DT_F32, DT_F32,
                                         DT_SUM, workspace, cols * 8, nullptr);
    };
    void *const ws = Lists(22).at[0];
    CHECK(backward(dbranch, rpre, ws) == DT_OK && launched == 3);
    for (int r = 0; r < P; ++r) CHECK(seen.rstd[1][r] == rpre.at[r] && seen.out[1][r] == dbranch.at[r] && seen.src[dt::kDy][r] == dy.at[r]);
    CHECK(backward(dbranch, rpre, dbranch.at[P - 1]) == DT_ERR_INVALID);
    Lists bad(6);
    bad.at[P - 1] = dbranch.at[P - 1];
    CHECK(backward(dbranch, bad, ws) == DT_ERR_INVALID && launched == 3);
    CHECK(backward(dz, rpre, ws) == DT_OK && launched == 4);    // in place
    return 0;
}

// A list of buffers that is full takes no more and lets no call through.
int full()
{
    const int P = 0;
    for (int outputs = 0; outputs < 2; ++outputs) {
        dt::host::Buffers b;
        int n = 0;
        for (; n < 16 * DT_MAX_RANKS && !b.clash(); ++n) {
            void *const p = reinterpret_cast<void *>(((uintptr_t)n + 1) << 20);
            if (outputs) b.write(p, 16);
            else b.read(p, 16);
        }
        CHECK(n < 16 * DT_MAX_RANKS && n > 3 * DT_MAX_RANKS);
    }
    return 0;
}

}  // namespace

int main()
{
    for (int P = 1; P <= DT_MAX_RANKS; ++P)
        if (run(P)) return 1;
    if (full()) return 1;
    printf("ok\n");
    return 0;
}
