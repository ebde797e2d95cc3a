/*
 * head_row.cuh — what the kernels that work on single heads of single tokens share (the norm and
 * rotation of queries and keys, its gradient, and the append to a paged cache): how the 32 lanes of
 * a warp divide rows of D elements, and the norm and rotation of one row.
 *
 * A row is one head of one token, D contiguous bf16 elements (D in {32, 64, 128}). D / 8 lanes hold
 * it, eight elements each, so a warp holds 32 / (D / 8) rows at a time. The eight elements are four
 * rotation pairs (A[u], B[u]), u = 0..3, so a rotation needs no exchange between lanes:
 *   half-split    lane l of the rotated part holds elements 4l..4l+3 and rot/2 + 4l..+3;
 *   interleaved   lane l holds elements 8l..8l+7, A the even ones and B the odd ones;
 *   behind rot    lane l holds elements 8l..8l+7 (A the first four), passed through.
 * Either way lane l < rot / 8 needs entries 4l..4l+3 of its position's row of the angle tables: one
 * 16-byte load of cos and one of sin. That is why rot is a multiple of 8.
 *
 * The position rotation and the norm are defined at attn_qk_norm_rope in attn.h.
 */
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace attn_b200 {

// n / d and n % d for 0 <= n < 2^31 by one multiplication: with s = ceil(log2 d) and
// m = ceil(2^(31+s) / d), m d - 2^(31+s) < d <= 2^s, so n m / 2^(31+s) is within n / 2^31 < 1 of n / d
// in units of 1/d and its floor is exact.
struct FastDiv {
    uint32_t d = 1, m = 0, s = 0;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div)
    {
        while ((1ull << s) < d)
            ++s;
        m = static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d);
    }
    __device__ __forceinline__ uint32_t quot(uint32_t n) const
    {
        return d == 1 ? n : static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> (31 + s));
    }
};

struct RopeTable {
    const float *cos, *sin;  // fp32 [max_pos][rot / 2]
    int rot, max_pos;
};

template <int D>
struct RowLanes {
    static constexpr int kLanes = D / 8;          // lanes of one row
    static constexpr int kRows = 32 / kLanes;     // rows a warp holds at a time
};

// First elements of the lane's two groups of four.
struct LaneElems {
    int e0, e1;
    bool rotated;
};

template <bool kInterleaved>
__device__ __forceinline__ LaneElems lane_elems(int l, int rot)
{
    LaneElems x;
    x.rotated = 8 * l < rot;
    const bool split = !kInterleaved && x.rotated;
    x.e0 = split ? 4 * l : 8 * l;
    x.e1 = split ? rot / 2 + 4 * l : 8 * l + 4;
    return x;
}

// The lane's eight elements as pairs.
struct Pairs {
    float A[4], B[4];
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <bool kInterleaved>
__device__ __forceinline__ Pairs unpack_pairs(uint2 g0, uint2 g1)
{
    Pairs x;
    if constexpr (kInterleaved) {
        x.A[0] = bf16_lo(g0.x), x.B[0] = bf16_hi(g0.x), x.A[1] = bf16_lo(g0.y), x.B[1] = bf16_hi(g0.y);
        x.A[2] = bf16_lo(g1.x), x.B[2] = bf16_hi(g1.x), x.A[3] = bf16_lo(g1.y), x.B[3] = bf16_hi(g1.y);
    } else {
        x.A[0] = bf16_lo(g0.x), x.A[1] = bf16_hi(g0.x), x.A[2] = bf16_lo(g0.y), x.A[3] = bf16_hi(g0.y);
        x.B[0] = bf16_lo(g1.x), x.B[1] = bf16_hi(g1.x), x.B[2] = bf16_lo(g1.y), x.B[3] = bf16_hi(g1.y);
    }
    return x;
}

__device__ __forceinline__ uint32_t pack_bf16_pair(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The inverse of unpack_pairs; fp32 -> bf16 to nearest even, the only rounding of a row's output.
template <bool kInterleaved>
__device__ __forceinline__ void pack_pairs(const Pairs &x, uint2 &g0, uint2 &g1)
{
    if constexpr (kInterleaved) {
        g0 = make_uint2(pack_bf16_pair(x.A[0], x.B[0]), pack_bf16_pair(x.A[1], x.B[1]));
        g1 = make_uint2(pack_bf16_pair(x.A[2], x.B[2]), pack_bf16_pair(x.A[3], x.B[3]));
    } else {
        g0 = make_uint2(pack_bf16_pair(x.A[0], x.A[1]), pack_bf16_pair(x.A[2], x.A[3]));
        g1 = make_uint2(pack_bf16_pair(x.B[0], x.B[1]), pack_bf16_pair(x.B[2], x.B[3]));
    }
}

// fp32 values of two groups of four consecutive elements (weights, coefficients) as pairs.
template <bool kInterleaved>
__device__ __forceinline__ Pairs arrange_pairs(float4 g0, float4 g1)
{
    Pairs x;
    if constexpr (kInterleaved) {
        x.A[0] = g0.x, x.B[0] = g0.y, x.A[1] = g0.z, x.B[1] = g0.w;
        x.A[2] = g1.x, x.B[2] = g1.y, x.A[3] = g1.z, x.B[3] = g1.w;
    } else {
        x.A[0] = g0.x, x.A[1] = g0.y, x.A[2] = g0.z, x.A[3] = g0.w;
        x.B[0] = g1.x, x.B[1] = g1.y, x.B[2] = g1.z, x.B[3] = g1.w;
    }
    return x;
}

// The lane's part of the norm's weight (bf16 [D]).
template <bool kInterleaved>
__device__ __forceinline__ Pairs load_weight(const __nv_bfloat16 *w, const LaneElems &le)
{
    return unpack_pairs<kInterleaved>(__ldg(reinterpret_cast<const uint2 *>(w + le.e0)),
                                      __ldg(reinterpret_cast<const uint2 *>(w + le.e1)));
}

// Sum over the lanes of a row; every lane of the row gets it. All 32 lanes of the warp take part.
template <int D>
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int o = RowLanes<D>::kLanes / 2; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float pairs_dot(const Pairs &x, const Pairs &y)
{
    float s = 0.f, t = 0.f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        s = fmaf(x.A[u], y.A[u], s);
        t = fmaf(x.B[u], y.B[u], t);
    }
    return s + t;
}

// (A, B) turned by the angles (c, s); backwards with s negated.
__device__ __forceinline__ void rotate_pairs(Pairs &x, float4 c4, float4 s4)
{
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const float a = x.A[u], b = x.B[u];
        x.A[u] = a * c[u] - b * s[u];
        x.B[u] = b * c[u] + a * s[u];
    }
}

// The angles of position `pos` for lane l; (1, 0) where there are none. An element behind rot is not
// put through rotate_pairs at all: an infinite neighbour times 0 would make it NaN.
__device__ __forceinline__ void load_angles(const RopeTable &t, int pos, int l, bool rotated, float4 &c, float4 &s)
{
    c = make_float4(1.f, 1.f, 1.f, 1.f);
    s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (rotated && pos >= 0 && pos < t.max_pos) {
        const size_t at = static_cast<size_t>(pos) * static_cast<size_t>(t.rot >> 1) + 4u * static_cast<unsigned>(l);
        c = __ldg(reinterpret_cast<const float4 *>(t.cos + at));
        s = __ldg(reinterpret_cast<const float4 *>(t.sin + at));
    }
}

}  // namespace attn_b200
