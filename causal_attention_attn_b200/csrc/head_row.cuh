/*
 * head_row.cuh — what the kernels that work on single heads of single tokens share (the norm and
 * rotation of queries and keys, its gradient, and the append to a paged cache): how the 32 lanes of
 * a warp divide rows of D elements, and the norm and rotation of one row.
 *
 * A row is one head of one token, D contiguous bf16 elements (D in {32, 64, 128}). D / 16 lanes hold
 * it, sixteen elements each in two 16-byte groups, so a warp holds 32 / (D / 16) rows at a time. The
 * sixteen elements are eight rotation pairs (A[u], B[u]), u = 0..7, so a rotation needs no exchange
 * between lanes:
 *   half-split    lane l of the rotated part holds elements 8l..8l+7 and rot/2 + 8l..+7;
 *   interleaved   lane l holds elements 16l..16l+15, A the even ones and B the odd ones;
 *   behind rot    lane l holds elements 16l..16l+15 (A the first eight), passed through.
 * Either way lane l < rot / 16 needs entries 8l..8l+7 of its position's row of the angle tables: two
 * 16-byte loads of cos and two of sin. That is why rot is a multiple of 16. (With eight elements to a
 * lane the kernels took up to twice as long: twice the index arithmetic and shuffles a byte.)
 *
 * Rows are worked on in pairs of neighbouring heads of one token, so that one load of the angles
 * serves two rows; a warp takes kRows pairs at a time (a unit) and copies the units ahead of it into
 * its own ring in shared memory with cp.async, each lane exactly the bytes that it will use itself:
 * no barrier, and the bytes in flight do not cost registers.
 *
 * The position rotation and the norm are defined at attn_qk_norm_rope in attn.h.
 */
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fast_div.h"
#include "sm100_ptx.cuh"

namespace attn_b200 {

struct RopeTable {
    const float *cos, *sin;  // fp32 [max_pos][rot / 2]
    int rot, max_pos;
    __device__ __forceinline__ bool has(int pos) const { return rot == 0 || (pos >= 0 && pos < max_pos); }
};

template <int D>
struct RowLanes {
    static constexpr int kLanes = D / 16;         // lanes of one row
    static constexpr int kRows = 32 / kLanes;     // rows a warp holds at a time
};

// First elements of the lane's two groups of eight.
struct LaneElems {
    int e0, e1;
    bool rotated;
};

template <bool kInterleaved>
__device__ __forceinline__ LaneElems lane_elems(int l, int rot)
{
    LaneElems x;
    x.rotated = 16 * l < rot;
    const bool split = !kInterleaved && x.rotated;
    x.e0 = split ? 8 * l : 16 * l;
    x.e1 = split ? rot / 2 + 8 * l : 16 * l + 8;
    return x;
}

// The lane's sixteen elements: as loaded (two groups), and as pairs.
struct RawRow {
    uint4 g0, g1;
};
struct Pairs {
    float A[8], B[8];
};

__device__ __forceinline__ RawRow load_row(const __nv_bfloat16 *x, const LaneElems &le)
{
    return RawRow{*reinterpret_cast<const uint4 *>(x + le.e0), *reinterpret_cast<const uint4 *>(x + le.e1)};
}

__device__ __forceinline__ RawRow zero_row() { return RawRow{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)}; }

__device__ __forceinline__ void store_row(__nv_bfloat16 *x, const LaneElems &le, const RawRow &r)
{
    *reinterpret_cast<uint4 *>(x + le.e0) = r.g0;
    *reinterpret_cast<uint4 *>(x + le.e1) = r.g1;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <bool kInterleaved>
__device__ __forceinline__ Pairs unpack_pairs(const RawRow &r)
{
    const uint32_t w[8] = {r.g0.x, r.g0.y, r.g0.z, r.g0.w, r.g1.x, r.g1.y, r.g1.z, r.g1.w};
    Pairs x;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        if constexpr (kInterleaved) {
            x.A[u] = bf16_lo(w[u]);
            x.B[u] = bf16_hi(w[u]);
        } else {
            x.A[u] = (u & 1) ? bf16_hi(w[u >> 1]) : bf16_lo(w[u >> 1]);
            x.B[u] = (u & 1) ? bf16_hi(w[4 + (u >> 1)]) : bf16_lo(w[4 + (u >> 1)]);
        }
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
__device__ __forceinline__ RawRow pack_pairs(const Pairs &x)
{
    uint32_t w[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        if constexpr (kInterleaved) {
            w[u] = pack_bf16_pair(x.A[u], x.B[u]);
            w[4 + u] = pack_bf16_pair(x.A[4 + u], x.B[4 + u]);
        } else {
            w[u] = pack_bf16_pair(x.A[2 * u], x.A[2 * u + 1]);
            w[4 + u] = pack_bf16_pair(x.B[2 * u], x.B[2 * u + 1]);
        }
    }
    return RawRow{make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7])};
}

// Element number, within the row, of A[u] and of B[u].
template <bool kInterleaved>
__device__ __forceinline__ int elem_a(const LaneElems &le, int u)
{
    return kInterleaved ? le.e0 + 2 * u : le.e0 + u;
}
template <bool kInterleaved>
__device__ __forceinline__ int elem_b(const LaneElems &le, int u)
{
    return kInterleaved ? le.e0 + 2 * u + 1 : le.e1 + u;
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
    float2 s = make_float2(0.f, 0.f), t = s;
#pragma unroll
    for (int u = 0; u < 8; u += 2) {
        s = __ffma2_rn(make_float2(x.A[u], x.A[u + 1]), make_float2(y.A[u], y.A[u + 1]), s);
        t = __ffma2_rn(make_float2(x.B[u], x.B[u + 1]), make_float2(y.B[u], y.B[u + 1]), t);
    }
    return (s.x + s.y) + (t.x + t.y);
}

// ---- the ring: slots of 16 bytes a lane, [slot][lane] -------------------------------------------

constexpr int kSlotBytes = 32 * 16;  // one 16-byte slot of every lane of a warp
constexpr int kRowSlots = 2, kAngleSlots = 4;

// 16 bytes to this lane's slot, zeros when `on` is false (then nothing is read). kReused: through L1,
// for what several warps read (the tables); otherwise past it.
template <bool kReused>
__device__ __forceinline__ void copy_slot(uint32_t dst, const void *src, bool on)
{
    const uint32_t n = on ? 16u : 0u;
    if constexpr (kReused)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Waits until at most kPending of this lane's latest groups are still in flight.
template <int kPending>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__device__ __forceinline__ uint4 read_slot(uint32_t src)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
    return v;
}

// A row: `x` must be a valid address of the tensor even when `on` is false (it is not read then).
__device__ __forceinline__ void copy_row(uint32_t dst, const __nv_bfloat16 *x, const LaneElems &le, bool on)
{
    copy_slot<false>(dst, x + le.e0, on);
    copy_slot<false>(dst + kSlotBytes, x + le.e1, on);
}

__device__ __forceinline__ RawRow read_row(uint32_t src) { return RawRow{read_slot(src), read_slot(src + kSlotBytes)}; }

// Entries 8l..8l+7 of row `pos` of the tables, cos then sin; only for a rotated lane and a pos they have.
__device__ __forceinline__ void copy_angles(uint32_t dst, const RopeTable &t, int pos, int l)
{
    const size_t at = static_cast<size_t>(pos) * static_cast<size_t>(t.rot >> 1) + 8u * static_cast<unsigned>(l);
    copy_slot<true>(dst, t.cos + at, true);
    copy_slot<true>(dst + kSlotBytes, t.cos + at + 4, true);
    copy_slot<true>(dst + 2 * kSlotBytes, t.sin + at, true);
    copy_slot<true>(dst + 3 * kSlotBytes, t.sin + at + 4, true);
}

// The angles of one position for a lane.
struct Angles {
    float c[8], s[8];
};

__device__ __forceinline__ Angles read_angles(uint32_t src)
{
    Angles a;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 v = read_slot(src + static_cast<uint32_t>(j) * kSlotBytes);
        float *to = (j < 2 ? a.c : a.s) + 4 * (j & 1);
        to[0] = __uint_as_float(v.x), to[1] = __uint_as_float(v.y), to[2] = __uint_as_float(v.z), to[3] = __uint_as_float(v.w);
    }
    return a;
}

// Two fp32 operations an instruction: the pairs' neighbours go together.
__device__ __forceinline__ float2 two(const float *x) { return make_float2(x[0], x[1]); }
__device__ __forceinline__ void put_two(float *x, float2 v) { x[0] = v.x, x[1] = v.y; }

// x <- x w.
__device__ __forceinline__ void mul_pairs(Pairs &x, const Pairs &w)
{
#pragma unroll
    for (int u = 0; u < 8; u += 2) {
        put_two(x.A + u, __fmul2_rn(two(x.A + u), two(w.A + u)));
        put_two(x.B + u, __fmul2_rn(two(x.B + u), two(w.B + u)));
    }
}

// x <- x r w.
__device__ __forceinline__ void scale_pairs(Pairs &x, float r, const Pairs &w)
{
    const float2 rr = make_float2(r, r);
#pragma unroll
    for (int u = 0; u < 8; u += 2) {
        put_two(x.A + u, __fmul2_rn(two(x.A + u), __fmul2_rn(rr, two(w.A + u))));
        put_two(x.B + u, __fmul2_rn(two(x.B + u), __fmul2_rn(rr, two(w.B + u))));
    }
}

// (A, B) turned by the angles; kBack: by their negatives. Only for a lane that is rotated: an element
// behind rot has no angle, and an infinite neighbour times sin 0 would make it NaN.
template <bool kBack>
__device__ __forceinline__ void rotate_pairs(Pairs &x, const Angles &t)
{
#pragma unroll
    for (int u = 0; u < 8; u += 2) {
        const float2 a = two(x.A + u), b = two(x.B + u), c = two(t.c + u), s = two(t.s + u);
        const float2 n = make_float2(-s.x, -s.y);
        put_two(x.A + u, __ffma2_rn(a, c, __fmul2_rn(b, kBack ? s : n)));
        put_two(x.B + u, __ffma2_rn(b, c, __fmul2_rn(a, kBack ? n : s)));
    }
}

}  // namespace attn_b200
