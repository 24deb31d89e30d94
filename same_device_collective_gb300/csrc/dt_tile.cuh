// Parts of the persistent tensor core kernels that do not depend on what they
// compute: the pipeline's bounded waits, a finishing warp's shared memory, and
// the index arithmetic of tiles.
#pragma once

#include <cstdint>

#include "dt_device.cuh"
#include "dt_internal.h"
#include "dt_tc.cuh"

namespace dt {

// n / d, where `inverse` is the least whole number above 2^32 / d (0 for 1): the
// product's high word is at most one too large.
__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t d, uint32_t inverse)
{
    if (d == 1) return n;
    const uint32_t q = __umulhi(n, inverse);
    return q * d > n ? q - 1 : q;
}

// A finishing warp's 32 rows x 128 bytes in shared memory, 16-byte chunk c of
// row r at chunk c ^ (r mod 8): a thread writes its row, and eight threads
// read a row, without bank conflicts.
__device__ __forceinline__ uint4 *out_chunk(unsigned char *buf, uint32_t row, uint32_t c)
{
    return reinterpret_cast<uint4 *>(buf + row * 128 + ((c ^ (row & 7)) << 4));
}

// One instruction's worth of a row: N 16-bit elements.
template <int N> struct Words;
template <> struct Words<8> { using type = uint4; };
template <> struct Words<4> { using type = uint2; };
template <> struct Words<2> { using type = uint32_t; };

// A try that may wait a microsecond in the hardware.  Without that hint a waiting
// thread tries again so often that the tensor cores' and the copies' own traffic with
// shared memory suffers (a linear layer of 2048 tokens, 4096 to 16384: 162 -> 152 us;
// with test_wait in a loop 190).
__device__ __forceinline__ bool mbar_try_wait_long(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// The state of the pipeline's waits: a wait that runs out is recorded once,
// and every role then leaves its loop.
struct Waits {
    const ErrorSink &sink;
    volatile uint32_t *gave_up;
    // The timer is read only after 64 tries, each of which waits a while in the
    // hardware: reading it on every wait cost a fifth of the time (2048 tokens of 32768 x 4096: 501 -> 397 us).
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const
    {
        for (int k = 0; k < 64; ++k)
            if (mbar_try_wait_long(bar, parity)) return true;
        return slow(bar, parity);
    }
    __device__ __noinline__ bool slow(uint32_t bar, uint32_t parity) const
    {
        const uint64_t t0 = global_ns();
        do {
            for (int k = 0; k < 64; ++k)
                if (mbar_try_wait_long(bar, parity)) return true;
        } while (global_ns() - t0 <= sink.timeout_ns);
        *gave_up = 1;
        record_error(sink, DT_ERR_TIMEOUT, -1, blockIdx.x, 0);
        return false;
    }
};

}  // namespace dt
