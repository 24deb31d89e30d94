// Host helpers shared by the files that implement the C ABI: argument checks,
// the device scope of a call, status conversion, and the NVTX range that every
// public entry point opens in builds made with DT_NVTX=1.  Not part of the C
// ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "dt_group.h"

// Built with -DDT_NVTX (DT_NVTX=1 when building), every public entry point
// opens an NVTX range named after itself for profiler timelines.
#ifdef DT_NVTX
#include <nvtx3/nvToolsExt.h>
namespace dt {
namespace host {
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};
}  // namespace host
}  // namespace dt
#define DT_TRACE() dt::host::NvtxRange dt_nvtx_range_(__func__)
#else
#define DT_TRACE() ((void)0)
#endif

namespace dt {
namespace host {

inline size_t elem_bytes(int dtype) { return dtype == DT_BF16 ? 2 : 4; }
inline bool valid_dtype(int dtype) { return dtype == DT_F32 || dtype == DT_BF16 || dtype == DT_I32; }
inline bool valid_op(int op) { return op >= DT_SUM && op <= DT_SUM_STEPWISE; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Switch to the group's device for the duration of a call.
struct DeviceScope {
    int prev = -1;
    bool ok = true;
    explicit DeviceScope(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) { ok = false; return; }
        if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
    }
    ~DeviceScope()
    {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
    int rank;
    int kind;           // 0 input, 1 output
};

inline bool overlaps(const Range &a, const Range &b) { return a.lo < b.hi && b.lo < a.hi; }

// Status of a call that finds an error recorded by the device.
inline dt_status take_device_error(dt_group *g)
{
    if (g->poisoned) return DT_ERR_POISONED;
    const int code = static_cast<volatile DevError *>(g->h_err)->code;
    if (code != 0) {
        g->poisoned = true;
        g->poison_code = static_cast<dt_status>(code);
        return static_cast<dt_status>(code);
    }
    return DT_OK;
}

inline dt_status cuda_status(cudaError_t e)
{
    if (e == cudaSuccess) return DT_OK;
    if (e == cudaErrorMemoryAllocation) return DT_ERR_OOM;
    return DT_ERR_CUDA;
}

inline uint64_t timeout_ns(const dt_group *g) { return (uint64_t)g->timeout_ms * 1000000ull; }

inline ErrorSink error_sink(dt_group *g) { return ErrorSink{g->d_err, g->h_err_dev, timeout_ns(g)}; }

inline bool float_dtype(int dtype) { return dtype == DT_F32 || dtype == DT_BF16; }

inline bool multiple(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

inline uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

// The buffers of a call.  Outputs may overlap nothing, but for an output and
// an input that carry the same tag (>= 0) and are the same buffer.  The most
// that a call has: six lists of a buffer to a rank and three weights that the
// residual norm's gradient reads, four such lists that the norm writes.  A call
// with more clashes.
struct Buffers {
    static constexpr int kIn = 6 * DT_MAX_RANKS + 4, kOut = 4 * DT_MAX_RANKS + 4;
    Range in[kIn], out[kOut];
    int nin = 0, nout = 0;
    bool full = false;

    void read(const void *p, size_t bytes, int tag = -1)
    {
        if (!p || !bytes) return;
        if (nin == kIn) full = true;
        else in[nin++] = Range{(uintptr_t)p, (uintptr_t)p + bytes, tag, 0};
    }
    void write(const void *p, size_t bytes, int tag = -1)
    {
        if (!p || !bytes) return;
        if (nout == kOut) full = true;
        else out[nout++] = Range{(uintptr_t)p, (uintptr_t)p + bytes, tag, 1};
    }
    bool clash() const
    {
        if (full) return true;
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
inline bool row_counts(int P, const size_t *rows, size_t rows_equal, size_t row_bytes, size_t *n, size_t *total)
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

}  // namespace host
}  // namespace dt
