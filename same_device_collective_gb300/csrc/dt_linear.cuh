// What the kernels of the linear layers share: the axes and operands of a product, places
// along them, rows at any alignment, activations and where results go.
#pragma once

#include <cstdint>
#include <type_traits>

#include "dt_bounds.cuh"
#include "dt_linear.h"
#include "dt_math.cuh"
#include "dt_tc.cuh"

namespace dt {

#define LINEAR_OK(buffer, a, n) DT_IN_EXTENT(p, kBoundsLinear, (buffer), (a), (n))

__host__ __device__ constexpr bool is_back(int kind) { return kind == kGatherBack || kind == kReduceBack; }

// The matrices of a call.
enum Matrix : int { kTok, kFeat, kW };

// What the rows, columns and inner axis of a product are, and its operands.  An
// operand is MN-major where its rows run along the inner axis.
// PIECES: the token axis of the tokens' matrix is cut into pieces.
template <int KIND, bool SECOND, bool PIECES = true>
struct Roles {
    static constexpr int kind = KIND;
    static constexpr bool second = SECOND;
    static constexpr int m = !SECOND ? kTokens : KIND == kGatherBack ? kFeatures : kDim;
    static constexpr int n = KIND == kGather || KIND == kReduceBack ? kFeatures : kDim;
    static constexpr int k = SECOND ? kTokens : n == kFeatures ? kDim : kFeatures;
    static constexpr int a = KIND == kGather || KIND == kReduceBack ? kTok : kFeat;
    static constexpr int b = !SECOND ? kW : KIND == kGatherBack ? kTok : kFeat;
    static constexpr bool a_mn = SECOND, b_mn = is_back(KIND);
    static constexpr bool tok = PIECES && (a == kTok || b == kTok);   // the token axis is cut as the tokens' matrix is
    static constexpr uint32_t depth = linear_depth(is_back(KIND));   // of a stage
    static constexpr bool w_by_feature = KIND == kGather || KIND == kGatherBack;   // rows of W_r are features
};

// A place along an axis: the rank's piece, the place there, and overall (tokens).  A pair's
// second half may lie past the end of all: that is past the end of the last piece that has
// something, whose tensor map fills in zeros.
struct Place {
    uint32_t piece, at, all;
};

template <class R, int AXIS>
__host__ __device__ __forceinline__ Place locate(const LinearCall &p, const LinearProduct &c, uint32_t i, uint32_t unit)
{
    if constexpr (AXIS == kDim) {
        return Place{0, i * unit, 0};
    } else if constexpr (AXIS == kFeatures) {
        uint32_t r = 0, begin = 0;
        while ((int)r + 1 < p.f_pieces && i >= c.f_end[r]) begin = c.f_end[r++];
        return Place{r, (i - begin) * unit, 0};
    } else if (!R::tok) {
        return Place{0, i * unit, i * unit};
    } else {
        uint32_t r = 0, begin = 0;
        while ((int)r + 1 < p.t_pieces && i >= c.t_end[r]) begin = c.t_end[r++];
        const uint32_t at = (i - begin) * unit;
        return Place{r, at, p.t_first[r] + at};
    }
}

template <class R, int AXIS>
__host__ __device__ __forceinline__ uint32_t length(const LinearCall &p, uint32_t piece)
{
    return AXIS == kDim ? p.dim : AXIS == kFeatures ? p.f_len[piece] : R::tok ? p.t_len[piece] : p.tokens;
}

// 16 bytes where `there`, else zeros, without a branch: loads in branches wait for one
// another, as each is used before the next branch (rows at any element, a step of
// linear_small_kernel: 2.2 us, this 1.1).
__device__ __forceinline__ uint4 load_if(const void *from, bool there)
{
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
        "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(from), "r"((uint32_t)there));
    return v;
}

// Eight elements of a row from any element on, of which `n` are there (the others, and
// all of n = 0, come out as zeros).  load() fetches the aligned vectors that they lie in,
// neither of which reaches past the 16-byte block of one of them; get() puts them right.
struct Shifted {
    uint4 a, b;
    uint32_t off, n;
    __device__ __forceinline__ void load(const uint16_t *from, uint32_t count)
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(from);
        off = (uint32_t)at & 15;
        n = count;
        const uint4 *block = reinterpret_cast<const uint4 *>(at & ~(uintptr_t)15);
        a = load_if(block, n != 0);
        b = load_if(block + 1, n != 0 && off + 2 * n > 16);
    }
    __device__ __forceinline__ void get(uint32_t (&w)[4]) const
    {
        // by eight, four and two bytes
        const bool s8 = off & 8, s4 = off & 4;
        const uint32_t x[6] = {s8 ? a.z : a.x, s8 ? a.w : a.y, s8 ? b.x : a.z, s8 ? b.y : a.w, s8 ? b.z : b.x, s8 ? b.w : b.y};
        uint32_t y[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) y[i] = s4 ? x[i + 1] : x[i];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            w[i] = __funnelshift_r(y[i], y[i + 1], (off & 2) * 8);
            if (2 * i >= n) w[i] = 0;
            else if (2 * i + 1 >= n) w[i] &= 0xFFFFu;
        }
    }
};

// The same of rows that begin on 16-byte boundaries.
struct Whole {
    uint4 a;
    __device__ __forceinline__ void load(const uint16_t *from, uint32_t count) { a = load_if(from, count != 0); }
    __device__ __forceinline__ void get(uint32_t (&w)[4]) const { w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w; }
};
template <bool VEC>
using Eight = typename std::conditional<VEC, Whole, Shifted>::type;

__device__ constexpr float kTail[7] = {0.143713042f, 0.141772494f, 0.139719009f, 0.0265500601f, 0.180952892f, -0.179763854f, 0.0470560379f};

// The upper tail of the normal distribution at |v|, and exp(-v^2 / 2), two at a time.
// The tail is exp(-z^2 / 2) t (c0 + c1 t + ... + c6 t^6) with t = 1 / (1 + 0.36 z), the c
// a minimax fit of the relative error over t from 1 to z = 14: 1e-6 of itself off
// everywhere, where 1 - erf would have nothing left far out.  (Own fit; erfcf in its
// place is some 40 instructions, for every element.)
__device__ __forceinline__ float2 normal_tail(float2 v, float2 &bell)
{
    const float2 e = mul2(mul2(v, v), make_float2(-0.72134752044448170368f, -0.72134752044448170368f));
    bell = make_float2(exp2_fast(e.x), exp2_fast(e.y));
    const float2 d = fma2(make_float2(fabsf(v.x), fabsf(v.y)), make_float2(0.36f, 0.36f), make_float2(1.0f, 1.0f));
    const float2 t = make_float2(rcp_fast(d.x), rcp_fast(d.y));
    float2 s = make_float2(kTail[6], kTail[6]);
#pragma unroll
    for (int i = 5; i >= 0; --i) s = fma2(s, t, make_float2(kTail[i], kTail[i]));
    return mul2(mul2(s, t), bell);
}

// v times the normal distribution at v, from its tail: max(v, 0) - |v| tail.  An infinite
// |v| would make the product with a tail of zero no number; a NaN stays one.
__device__ __forceinline__ float gelu_of(float v, float q)
{
    float a;
    asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %1;\n\tmin.NaN.f32 %0, t, 0f7F7FFFFF;\n\t}" : "=f"(a) : "f"(v));
    return fmaf(-a, q, fmaxf(v, 0.0f));
}

// The normal distribution from its tail.
__device__ __forceinline__ float2 normal_of(float2 v, float2 q)
{
    return make_float2(v.x > 0.0f ? 1.0f - q.x : q.x, v.y > 0.0f ? 1.0f - q.y : q.y);
}

// 1 / (1 + exp(-v)).
__device__ __forceinline__ float2 logistic(float2 v)
{
    const float2 e = mul2(v, make_float2(-1.44269504088896340736f, -1.44269504088896340736f));
    return make_float2(rcp_fast(1.0f + exp2_fast(e.x)), rcp_fast(1.0f + exp2_fast(e.y)));
}

// The activation; a NaN stays one.
template <int ACT>
__device__ __forceinline__ float2 activate(float2 v)
{
    if (ACT == DT_ACT_RELU) return make_float2(v.x < 0.0f ? 0.0f : v.x, v.y < 0.0f ? 0.0f : v.y);
    if (ACT == DT_ACT_SILU) return mul2(v, logistic(v));
    if (ACT == DT_ACT_GELU) {
        float2 bell;
        const float2 q = normal_tail(v, bell);
        return make_float2(gelu_of(v.x, q.x), gelu_of(v.y, q.y));
    }
    return v;
}

// Its derivative.
template <int ACT>
__device__ __forceinline__ float2 slope(float2 v)
{
    if (ACT == DT_ACT_RELU) return make_float2(v.x > 0.0f ? 1.0f : 0.0f, v.y > 0.0f ? 1.0f : 0.0f);
    const float2 one = make_float2(1.0f, 1.0f);
    if (ACT == DT_ACT_SILU) {
        const float2 s = logistic(v), rest = fma2(s, make_float2(-1.0f, -1.0f), one);
        return mul2(s, fma2(v, rest, one));
    }
    if (ACT == DT_ACT_GELU) {
        float2 bell;
        const float2 q = normal_tail(v, bell);
        return fma2(mul2(v, make_float2(0.39894228040143267794f, 0.39894228040143267794f)), bell, normal_of(v, q));
    }
    return one;
}

// All of N values, so that the choice is made once.
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act)
{
    auto all = [&](auto of) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 a = activate<decltype(of)::value>(make_float2(v[j], v[j + 1]));
            v[j] = a.x, v[j + 1] = a.y;
        }
    };
    if (act == DT_ACT_RELU) all(std::integral_constant<int, DT_ACT_RELU>{});
    else if (act == DT_ACT_GELU) all(std::integral_constant<int, DT_ACT_GELU>{});
    else if (act == DT_ACT_SILU) all(std::integral_constant<int, DT_ACT_SILU>{});
}

// g[j] times the derivative at v[j].
template <int N>
__device__ __forceinline__ void times_slope(float (&g)[N], const float (&v)[N], int act)
{
    auto all = [&](auto of) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float2 a = mul2(make_float2(g[j], g[j + 1]), slope<decltype(of)::value>(make_float2(v[j], v[j + 1])));
            g[j] = a.x, g[j + 1] = a.y;
        }
    };
    if (act == DT_ACT_RELU) all(std::integral_constant<int, DT_ACT_RELU>{});
    else if (act == DT_ACT_GELU) all(std::integral_constant<int, DT_ACT_GELU>{});
    else if (act == DT_ACT_SILU) all(std::integral_constant<int, DT_ACT_SILU>{});
}

// Where row `row` (of the piece at.piece) of a product's output begins, its first
// element at column n.at of its tile; and the number of the buffer, by rank.
struct OutRow {
    uint16_t *out;
    uint64_t offset;   // elements from the buffer's start
    uint32_t rank;
};

template <class R>
__device__ __forceinline__ OutRow out_row(const LinearCall &p, const LinearProduct &c, const Place &m, const Place &n,
                                          uint32_t row)
{
    OutRow o;
    uint64_t at;
    if (R::m == kTokens && R::n == kDim) {       // a token's row on its rank
        const uint32_t t = m.all + row;
        uint32_t begin = 0;
        o.rank = 0;
        while ((int)o.rank + 1 < p.P && t >= p.row_end[o.rank]) begin = p.row_end[o.rank++];
        at = t - begin;
    } else if (R::m == kFeatures) {              // dW_r: a feature's row
        o.rank = m.piece;
        at = m.at + row;
    } else {                                     // a rank's features of a token, or of a column of W_r
        o.rank = n.piece;
        at = (R::m == kTokens ? m.all : m.at) + row;
    }
    o.offset = at * (R::n == kDim ? p.dim : p.f_len[n.piece]) + n.at;
    o.out = c.out[o.rank];
    return o;
}

}  // namespace dt
