/*
 * append_sm100.cu — new tokens' keys and values written to their slots of a paged K/V cache, the
 * keys normalised and rotated on the way, and the same tokens' queries normalised and rotated for the
 * attention that follows (attn_append_paged and attn_append_paged_fp8 in attn.h). One kernel, so a
 * decode step needs one launch between its projection and its attention.
 *
 * Row arithmetic as in norm_rope_sm100.cu. With an e4m3 cache a key or value element x is stored as
 * the code nearest to x / coefficient (ties to even, saturating at +-448), from the fp32 value: a key
 * is rounded once, not to bf16 first.
 *
 * Bound by memory (each new row read and written once), and for a few tokens by the launch and one
 * chain of dependent loads: length, block-table entry, store. The rows of the inputs are loaded
 * before the chain's results are needed.
 */
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "head_row.cuh"
#include "kernels.h"

namespace attn_b200 {
namespace {

constexpr int kD = 128;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
using R = RowLanes<kD>;

enum Kind : int { kQ = 0, kK = 1, kV = 2 };

// The rows of q, k or v, numbered token * H + head, token = b * S + i.
struct Source {
    const __nv_bfloat16 *x, *w;
    TensorStrides xs;
    FastDiv heads;
    int rows, units;
};

struct AppendParams {
    Source src[3];
    __nv_bfloat16 *q_out;
    TensorStrides qos;
    void *pages[2];         // k, v
    const float *coef[2];   // e4m3: [Hkv][128]
    RopeTable table;
    const int *positions, *seq_lens, *new_lens, *block_table;
    FastDiv seq, page_size;
    int Hkv, num_pages, pages_per_seq;
    long long cap;  // slots of a block-table row
    float eps;
};

// Four consecutive elements' e4m3 codes, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

template <bool kInterleaved, bool kFp8, int kIter>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p)
{
    const int lane = threadIdx.x & 31;
    const int l = lane & (R::kLanes - 1);
    int unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
    int kind = kQ;
    while (kind <= kV && unit >= p.src[kind].units) {
        unit -= p.src[kind].units;
        ++kind;
    }
    if (kind > kV)
        return;
    const Source &sc = p.src[kind];
    const int row0 = unit * (R::kRows * kIter) + lane / R::kLanes;
    const LaneElems le = lane_elems<kInterleaved>(l, p.table.rot);

    struct At {
        bool row, live;  // a row of the input; of a token that is appended
        uint32_t b, i, h;
        long long pos;  // the token's slot in its sequence
        int rot_pos, page;
    } at[kIter];
    uint2 g0[kIter], g1[kIter];
    float4 c[kIter], s[kIter];
#pragma unroll
    for (int k = 0; k < kIter; ++k) {
        const int row = row0 + k * R::kRows;
        At &a = at[k];
        a.row = row < sc.rows;
        const uint32_t n = a.row ? static_cast<uint32_t>(row) : 0u;
        const uint32_t tok = sc.heads.quot(n);
        a.h = n - tok * sc.heads.d;
        a.b = p.seq.quot(tok);
        a.i = tok - a.b * p.seq.d;
        const __nv_bfloat16 *x = sc.x + a.b * sc.xs.b + a.h * sc.xs.h + a.i * sc.xs.s;
        g0[k] = g1[k] = make_uint2(0u, 0u);
        if (a.row) {
            g0[k] = *reinterpret_cast<const uint2 *>(x + le.e0);
            g1[k] = *reinterpret_cast<const uint2 *>(x + le.e1);
        }
        const long long S = p.seq.d;
        const long long fresh = p.new_lens ? min(max(static_cast<long long>(__ldg(p.new_lens + a.b)), 0LL), S) : S;
        a.pos = static_cast<long long>(__ldg(p.seq_lens + a.b)) - S + a.i;
        a.live = a.row && a.i >= S - fresh && a.pos >= 0 && a.pos < p.cap;
        a.rot_pos = p.positions ? __ldg(p.positions + tok) : static_cast<int>(a.live ? a.pos : 0);
        a.live = a.live && (p.table.rot == 0 || (a.rot_pos >= 0 && a.rot_pos < p.table.max_pos));
    }
#pragma unroll
    for (int k = 0; k < kIter; ++k) {
        At &a = at[k];
        a.page = -1;
        if (a.live)
            a.page = __ldg(p.block_table + static_cast<size_t>(a.b) * p.pages_per_seq +
                           p.page_size.quot(static_cast<uint32_t>(a.pos)));
        load_angles(p.table, a.rot_pos, l, kind != kV && le.rotated && a.live, c[k], s[k]);
    }
    const bool norm = sc.w != nullptr;
    Pairs w;
    if (norm)
        w = load_weight<kInterleaved>(sc.w, le);
#pragma unroll
    for (int k = 0; k < kIter; ++k) {
        At &a = at[k];
        a.live = a.live && a.page >= 0 && a.page < p.num_pages;
        Pairs x = unpack_pairs<kInterleaved>(g0[k], g1[k]);
        if (norm) {
            const float r = rsqrtf(row_sum<kD>(pairs_dot(x, x)) * (1.f / kD) + p.eps);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x.A[u] *= r * w.A[u];
                x.B[u] *= r * w.B[u];
            }
        }
        if (kind != kV && le.rotated)
            rotate_pairs(x, c[k], s[k]);
        uint2 o0, o1;
        pack_pairs<kInterleaved>(x, o0, o1);
        if (kind == kQ) {
            if (a.row) {
                __nv_bfloat16 *out = p.q_out + a.b * p.qos.b + a.h * p.qos.h + a.i * p.qos.s;
                const uint2 zero = make_uint2(0u, 0u);
                *reinterpret_cast<uint2 *>(out + le.e0) = a.live ? o0 : zero;
                *reinterpret_cast<uint2 *>(out + le.e1) = a.live ? o1 : zero;
            }
            continue;
        }
        if (!a.live)
            continue;
        const uint32_t slot = static_cast<uint32_t>(a.pos) - p.page_size.quot(static_cast<uint32_t>(a.pos)) * p.page_size.d;
        const size_t dst = ((static_cast<size_t>(a.page) * p.Hkv + a.h) * p.page_size.d + slot) * kD;
        if constexpr (kFp8) {
            const float *cf = p.coef[kind - kK] + a.h * kD;
            const Pairs f = arrange_pairs<kInterleaved>(__ldg(reinterpret_cast<const float4 *>(cf + le.e0)),
                                                        __ldg(reinterpret_cast<const float4 *>(cf + le.e1)));
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x.A[u] = x.A[u] / f.A[u];
                x.B[u] = x.B[u] / f.B[u];
            }
            uint8_t *out = static_cast<uint8_t *>(p.pages[kind - kK]) + dst;
            uint32_t w0, w1;
            if constexpr (kInterleaved) {
                w0 = e4m3x4(x.A[0], x.B[0], x.A[1], x.B[1]);
                w1 = e4m3x4(x.A[2], x.B[2], x.A[3], x.B[3]);
            } else {
                w0 = e4m3x4(x.A[0], x.A[1], x.A[2], x.A[3]);
                w1 = e4m3x4(x.B[0], x.B[1], x.B[2], x.B[3]);
            }
            *reinterpret_cast<uint32_t *>(out + le.e0) = w0;
            *reinterpret_cast<uint32_t *>(out + le.e1) = w1;
        } else {
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.pages[kind - kK]) + dst;
            *reinterpret_cast<uint2 *>(out + le.e0) = o0;
            *reinterpret_cast<uint2 *>(out + le.e1) = o1;
        }
    }
}

template <bool kInterleaved, bool kFp8>
cudaError_t launch(const AppendArgs &a, cudaStream_t stream)
{
    AppendParams p;
    const int heads[3] = {a.q ? a.Hq : 0, a.Hkv, a.Hkv};
    const void *x[3] = {a.q, a.k, a.v};
    const void *w[3] = {a.q_weight, a.k_weight, nullptr};
    const TensorStrides xs[3] = {a.qs, a.ks, a.vs};
    for (int i = 0; i < 3; ++i) {
        p.src[i].x = static_cast<const __nv_bfloat16 *>(x[i]);
        p.src[i].w = static_cast<const __nv_bfloat16 *>(w[i]);
        p.src[i].xs = xs[i];
        p.src[i].heads = FastDiv(static_cast<uint32_t>(heads[i] > 0 ? heads[i] : 1));
        p.src[i].rows = a.B * a.S * heads[i];
    }
    p.q_out = static_cast<__nv_bfloat16 *>(a.q_out);
    p.qos = a.qos;
    p.pages[0] = a.k_pages;
    p.pages[1] = a.v_pages;
    p.coef[0] = a.k_scale;
    p.coef[1] = a.v_scale;
    p.table = RopeTable{a.cos, a.sin, a.rot_dim, a.max_pos};
    p.positions = a.positions;
    p.seq_lens = a.seq_lens;
    p.new_lens = a.new_lens;
    p.block_table = a.block_table;
    p.seq = FastDiv(static_cast<uint32_t>(a.S));
    p.page_size = FastDiv(static_cast<uint32_t>(a.page_size));
    p.Hkv = a.Hkv;
    p.num_pages = a.num_pages;
    p.pages_per_seq = a.pages_per_seq;
    p.cap = static_cast<long long>(a.pages_per_seq) * a.page_size;
    p.eps = a.eps;
    constexpr int kIter = 4;
    long long units = 0;
    for (Source &sc : p.src) {
        sc.units = static_cast<int>((static_cast<long long>(sc.rows) + R::kRows * kIter - 1) / (R::kRows * kIter));
        units += sc.units;
    }
    append_kernel<kInterleaved, kFp8, kIter>
        <<<static_cast<unsigned>((units + kWarps - 1) / kWarps), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, cudaStream_t stream)
{
    if (a.k_scale)
        return a.interleaved ? launch<true, true>(a, stream) : launch<false, true>(a, stream);
    return a.interleaved ? launch<true, false>(a, stream) : launch<false, false>(a, stream);
}

}  // namespace attn_b200
