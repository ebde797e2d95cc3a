/*
 * norm_rope_sm100.cu — the norm and position rotation of queries and keys, head by head, in one
 * pass over them, and its gradient (attn_qk_norm_rope and attn_qk_norm_rope_bwd in attn.h).
 *
 * Forward, per row x (one head of one token, D elements):
 *   r = (mean(x^2) + eps)^(-1/2),  y = x r w,  z = R(pos) y.
 * Backward, given dz:
 *   dy = R(pos)^T dz,  g = w dy,  dx = r (g - x r^2 mean(g x)),  dw = sum over rows of dy x r.
 * Without weights there is no norm: z = R x and dx = R^T dz.
 *
 * Bound by memory: forward reads and writes each row once, backward reads two and writes one, with
 * about a dozen operations an element. So the design is about loads in flight and about instructions
 * per byte: a row lies in D / 8 lanes (head_row.cuh), each lane issues the loads of kIter rows before
 * it uses the first, and rows are numbered (token, head) so that consecutive rows of a warp mostly
 * share a token and its angles. The weight's gradient stays in registers over all rows of a warp,
 * then goes through shared memory to one partial per block; a second small kernel adds the
 * partials in a fixed order, so the result does not depend on timing (no atomics).
 */
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "head_row.cuh"
#include "kernels.h"

namespace attn_b200 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// One of q and k: its rows are numbered token * H + head, token = b * S + i.
struct Side {
    const __nv_bfloat16 *x, *w, *dz;
    __nv_bfloat16 *out;  // z, or dx
    TensorStrides xs, zs, os;
    FastDiv heads;
    int rows;   // B * S * H
    int units;  // warp-sized pieces of kRows * kIter rows
};

struct NormRopeParams {
    Side side[2];  // q, k
    RopeTable table;
    const int *positions;  // [B][S], or null: the row index
    FastDiv seq;           // S
    float eps;
    float *partials;  // backward: [block][2][D]
};

// A lane's place in one row.
struct RowAt {
    bool live;
    int pos;            // position of the rotation
    long long x, z, o;  // element offsets of the row
};

__device__ __forceinline__ RowAt locate_row(const NormRopeParams &p, const Side &sd, int row)
{
    RowAt r;
    r.live = row < sd.rows;
    const uint32_t n = r.live ? static_cast<uint32_t>(row) : 0u;
    const uint32_t tok = sd.heads.quot(n), h = n - tok * sd.heads.d;
    const uint32_t b = p.seq.quot(tok), i = tok - b * p.seq.d;
    r.pos = p.positions ? __ldg(p.positions + tok) : static_cast<int>(i);
    r.x = b * sd.xs.b + h * sd.xs.h + i * sd.xs.s;
    r.z = b * sd.zs.b + h * sd.zs.h + i * sd.zs.s;
    r.o = b * sd.os.b + h * sd.os.h + i * sd.os.s;
    return r;
}

// A plain load: the output may be the input (attn.h), so it is not read-only data.
__device__ __forceinline__ uint2 load_quad(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint2 *>(p); }

template <int D, bool kInterleaved, int kIter>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeParams p)
{
    using R = RowLanes<D>;
    const int lane = threadIdx.x & 31;
    const int l = lane & (R::kLanes - 1);
    const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const bool is_k = unit >= p.side[0].units;
    if (is_k && unit - p.side[0].units >= p.side[1].units)
        return;
    const Side &sd = p.side[is_k ? 1 : 0];
    const int row0 = (unit - (is_k ? p.side[0].units : 0)) * (R::kRows * kIter) + lane / R::kLanes;
    const LaneElems le = lane_elems<kInterleaved>(l, p.table.rot);

    RowAt at[kIter];
    uint2 g0[kIter], g1[kIter];
    float4 c[kIter], s[kIter];
#pragma unroll
    for (int k = 0; k < kIter; ++k) {
        at[k] = locate_row(p, sd, row0 + k * R::kRows);
        g0[k] = g1[k] = make_uint2(0u, 0u);
        if (at[k].live) {
            g0[k] = load_quad(sd.x + at[k].x + le.e0);
            g1[k] = load_quad(sd.x + at[k].x + le.e1);
        }
    }
#pragma unroll
    for (int k = 0; k < kIter; ++k)
        load_angles(p.table, at[k].pos, l, le.rotated && at[k].live, c[k], s[k]);
    const bool norm = sd.w != nullptr;
    Pairs w;
    if (norm)
        w = load_weight<kInterleaved>(sd.w, le);
#pragma unroll
    for (int k = 0; k < kIter; ++k) {
        Pairs x = unpack_pairs<kInterleaved>(g0[k], g1[k]);
        if (norm) {
            const float r = rsqrtf(row_sum<D>(pairs_dot(x, x)) * (1.f / D) + p.eps);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x.A[u] *= r * w.A[u];
                x.B[u] *= r * w.B[u];
            }
        }
        if (le.rotated)
            rotate_pairs(x, c[k], s[k]);
        uint2 o0, o1;
        pack_pairs<kInterleaved>(x, o0, o1);
        // A position without a row of the tables: a row of zeros.
        if (p.table.rot && (at[k].pos < 0 || at[k].pos >= p.table.max_pos))
            o0 = o1 = make_uint2(0u, 0u);
        if (at[k].live) {
            *reinterpret_cast<uint2 *>(sd.out + at[k].o + le.e0) = o0;
            *reinterpret_cast<uint2 *>(sd.out + at[k].o + le.e1) = o1;
        }
    }
}

template <int D, bool kInterleaved, int kIter>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(const NormRopeParams p)
{
    using R = RowLanes<D>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & (R::kLanes - 1);
    const LaneElems le = lane_elems<kInterleaved>(l, p.table.rot);
    __shared__ float red[kWarps][R::kRows][D];
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const Side &sd = p.side[side];
        const bool norm = sd.w != nullptr;
        Pairs w, dw;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            w.A[u] = w.B[u] = dw.A[u] = dw.B[u] = 0.f;
        if (norm)
            w = load_weight<kInterleaved>(sd.w, le);
        for (int unit = blockIdx.x * kWarps + warp; unit < sd.units; unit += gridDim.x * kWarps) {
            const int row0 = unit * (R::kRows * kIter) + lane / R::kLanes;
            RowAt at[kIter];
            uint2 g0[kIter], g1[kIter], d0[kIter], d1[kIter];
            float4 c[kIter], s[kIter];
            bool in[kIter];
#pragma unroll
            for (int k = 0; k < kIter; ++k) {
                at[k] = locate_row(p, sd, row0 + k * R::kRows);
                // A position without a row of the tables gave zeros, so its gradient is zero.
                in[k] = at[k].live && (!p.table.rot || (at[k].pos >= 0 && at[k].pos < p.table.max_pos));
                g0[k] = g1[k] = d0[k] = d1[k] = make_uint2(0u, 0u);
                if (in[k]) {
                    d0[k] = load_quad(sd.dz + at[k].z + le.e0);
                    d1[k] = load_quad(sd.dz + at[k].z + le.e1);
                    if (norm) {
                        g0[k] = load_quad(sd.x + at[k].x + le.e0);
                        g1[k] = load_quad(sd.x + at[k].x + le.e1);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kIter; ++k)
                load_angles(p.table, at[k].pos, l, le.rotated && at[k].live, c[k], s[k]);
#pragma unroll
            for (int k = 0; k < kIter; ++k) {
                Pairs dy = unpack_pairs<kInterleaved>(d0[k], d1[k]);
                if (le.rotated)
                    rotate_pairs(dy, c[k], make_float4(-s[k].x, -s[k].y, -s[k].z, -s[k].w));
                if (norm) {
                    const Pairs x = unpack_pairs<kInterleaved>(g0[k], g1[k]);
                    Pairs g;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        g.A[u] = dy.A[u] * w.A[u];
                        g.B[u] = dy.B[u] * w.B[u];
                    }
                    const float xx = row_sum<D>(pairs_dot(x, x)), gx = row_sum<D>(pairs_dot(g, x));
                    const float r = in[k] ? rsqrtf(xx * (1.f / D) + p.eps) : 0.f;
                    const float f = r * r * (gx * (1.f / D));
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        dw.A[u] = fmaf(dy.A[u], x.A[u] * r, dw.A[u]);
                        dw.B[u] = fmaf(dy.B[u], x.B[u] * r, dw.B[u]);
                        dy.A[u] = r * fmaf(-f, x.A[u], g.A[u]);
                        dy.B[u] = r * fmaf(-f, x.B[u], g.B[u]);
                    }
                }
                if (at[k].live) {
                    uint2 o0, o1;
                    pack_pairs<kInterleaved>(dy, o0, o1);
                    *reinterpret_cast<uint2 *>(sd.out + at[k].o + le.e0) = o0;
                    *reinterpret_cast<uint2 *>(sd.out + at[k].o + le.e1) = o1;
                }
            }
        }
        if (!p.partials)
            continue;
        // The block's partial: every lane's sums, in channel order, added in a fixed order.
        float *mine = red[warp][lane / R::kLanes];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if constexpr (kInterleaved) {
                mine[(u < 2 ? le.e0 : le.e1) + 2 * (u & 1)] = dw.A[u];
                mine[(u < 2 ? le.e0 : le.e1) + 2 * (u & 1) + 1] = dw.B[u];
            } else {
                mine[le.e0 + u] = dw.A[u];
                mine[le.e1 + u] = dw.B[u];
            }
        }
        __syncthreads();
        for (int d = threadIdx.x; d < D; d += kThreads) {
            float t = 0.f;
#pragma unroll
            for (int v = 0; v < kWarps; ++v)
#pragma unroll
                for (int j = 0; j < R::kRows; ++j)
                    t += red[v][j][d];
            p.partials[(static_cast<size_t>(blockIdx.x) * 2 + side) * D + d] = t;
        }
        __syncthreads();
    }
}

// dw[side][d] = the blocks' partials added up: one block per side and 32 channels, its 32 warps each
// over every 32nd partial, then the warps' sums in order.
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float *partials, int blocks, int D, float *dwq, float *dwk)
{
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int side = blockIdx.y, d = blockIdx.x * 32 + lane;
    float *dst = side ? dwk : dwq;
    if (!dst)
        return;
    float t = 0.f;
    for (int b = warp; b < blocks; b += 32)
        t += partials[(static_cast<size_t>(b) * 2 + side) * D + d];
    red[warp][lane] = t;
    __syncthreads();
    if (warp == 0) {
        t = 0.f;
#pragma unroll
        for (int v = 0; v < 32; ++v)
            t += red[v][lane];
        dst[d] = t;
    }
}

void fill_side(Side &sd, const NormRopeSide &a, int B, int S)
{
    sd.x = static_cast<const __nv_bfloat16 *>(a.x);
    sd.w = static_cast<const __nv_bfloat16 *>(a.w);
    sd.dz = static_cast<const __nv_bfloat16 *>(a.dz);
    sd.out = static_cast<__nv_bfloat16 *>(a.out);
    sd.xs = a.xs;
    sd.zs = a.zs;
    sd.os = a.os;
    sd.heads = FastDiv(static_cast<uint32_t>(a.H));
    sd.rows = B * S * a.H;
}

template <int D, bool kInterleaved>
cudaError_t launch(const NormRopeArgs &a, cudaStream_t stream)
{
    using R = RowLanes<D>;
    NormRopeParams p;
    fill_side(p.side[0], a.q, a.B, a.S);
    fill_side(p.side[1], a.k, a.B, a.S);
    p.table = RopeTable{a.cos, a.sin, a.rot_dim, a.max_pos};
    p.positions = a.positions;
    p.seq = FastDiv(static_cast<uint32_t>(a.S));
    p.eps = a.eps;
    p.partials = a.partials;
    auto units = [&](int iter) {
        const int per = R::kRows * iter;
        long long n = 0;
        for (Side &sd : p.side) {
            sd.units = static_cast<int>((static_cast<long long>(sd.rows) + per - 1) / per);
            n += sd.units;
        }
        return n;
    };
    if (!a.backward) {
        const long long n = units(4);
        norm_rope_kernel<D, kInterleaved, 4>
            <<<static_cast<unsigned>((n + kWarps - 1) / kWarps), kThreads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    const long long n = units(2);
    const long long want = (n + kWarps - 1) / kWarps;
    const int blocks = static_cast<int>(want < kNormRopeBwdBlocks ? want : kNormRopeBwdBlocks);
    norm_rope_bwd_kernel<D, kInterleaved, 2><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.partials)
        return e;
    weight_grad_kernel<<<dim3(D / 32, 2), 1024, 0, stream>>>(a.partials, blocks, D, a.dwq, a.dwk);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, cudaStream_t stream)
{
    switch (a.D) {
    case 32:
        return a.interleaved ? launch<32, true>(a, stream) : launch<32, false>(a, stream);
    case 64:
        return a.interleaved ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
    case 128:
        return a.interleaved ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
    default:
        return cudaErrorInvalidValue;
    }
}

}  // namespace attn_b200
