/*
 * merge_sm100.cu — merges the result of attention over one block of keys into a running result
 * over other keys: the log-sum-exp merge that Flash-Decoding uses for its key splits, here as a
 * kernel of its own for ring (context-parallel) attention, where the key blocks arrive one after
 * the other from the other ranks.
 *
 * Per row, with the accumulated (o_acc, lse_acc) and the part (o_part, lse_part), natural logs:
 *   M = max(lse_acc, lse_part),  w_a = e^(lse_acc - M),  w_p = e^(lse_part - M)
 *   o_acc <- (w_a o_acc + w_p o_part) / (w_a + w_p),  lse_acc <- M + ln(w_a + w_p)
 * An empty side (lse = -inf: no key yet) gets weight 0; when both are empty the row stays empty.
 *
 * Source (page title, section): "AI Infra 入门：RMSNorm、Softmax、Causal Mask、Sampling 的数学与底层
 * 优化", §3 (LSE paragraph: partial results over key splits combine through their LSEs).
 *
 * One warp per row; lane l owns D/32 consecutive elements (4 for D = 128). The accumulator is fp32
 * so that a chain of merges rounds once, when the bf16 output is written.
 */
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "kernels.h"

namespace attn_b200 {
namespace {

template <int E>  // elements per lane: D / 32
__global__ void __launch_bounds__(256) lse_merge_kernel(float *o_acc, float *lse_acc, const __nv_bfloat16 *o_part,
                                                        const float *lse_part, __nv_bfloat16 *o_out, long long rows)
{
    constexpr int D = 32 * E;
    const int lane = threadIdx.x & 31;
    const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
    for (long long row = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; row < rows;
         row += warps) {
        const float la = lse_acc[row];
        const float lp = lse_part[row];
        const float M = fmaxf(la, lp);
        float wa = 0.f, wp = 0.f;
        if (M != -INFINITY) {  // else both sides are empty
            wa = expf(la - M);  // e^-inf = 0 for an empty side
            wp = expf(lp - M);
        }
        const float sum = wa + wp;
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        float *acc = o_acc + row * D + lane * E;
        const __nv_bfloat16 *part = o_part + row * D + lane * E;
        float a[E], r[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            a[e] = acc[e];
#pragma unroll
        for (int e = 0; e < E; ++e)
            r[e] = sum > 0.f ? (wa * a[e] + wp * __bfloat162float(part[e])) * inv : a[e];
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = r[e];
        if (o_out) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                o_out[row * D + lane * E + e] = __float2bfloat16_rn(r[e]);
        }
        __syncwarp();  // every lane has read lse_acc[row] before it changes
        if (lane == 0)
            lse_acc[row] = sum > 0.f ? M + logf(sum) : M;
    }
}

}  // namespace

cudaError_t launch_lse_merge(float *o_acc, float *lse_acc, const void *o_part, const float *lse_part, void *o_out,
                             long long rows, int D, int sm_count, cudaStream_t stream)
{
    if (rows <= 0)
        return cudaSuccess;
    const long long want = (rows + 7) / 8;  // 8 warps (rows) per block
    const long long cap = static_cast<long long>(sm_count > 0 ? sm_count : 148) * 8;
    const unsigned grid = static_cast<unsigned>(want < cap ? want : cap);
    const auto *part = static_cast<const __nv_bfloat16 *>(o_part);
    auto *out = static_cast<__nv_bfloat16 *>(o_out);
    switch (D) {
    case 32:
        lse_merge_kernel<1><<<grid, 256, 0, stream>>>(o_acc, lse_acc, part, lse_part, out, rows);
        break;
    case 64:
        lse_merge_kernel<2><<<grid, 256, 0, stream>>>(o_acc, lse_acc, part, lse_part, out, rows);
        break;
    case 128:
        lse_merge_kernel<4><<<grid, 256, 0, stream>>>(o_acc, lse_acc, part, lse_part, out, rows);
        break;
    default:
        return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

namespace {

// Attention of one row of a shared-prefix decode from its parts: the segments of its list of prefix
// tiles (prefill_sm100.cu, decode_segment) and its own suffix, all fp32 with LSEs in log2 units:
//   M = max LSE_s,  O = sum 2^(LSE_s - M) O_s / W,  lse = (M + log2 W) ln 2,  W = sum 2^(LSE_s - M).
// One warp per row; the lanes look up the LSEs of 32 parts at a time, then each lane adds its four
// channels over the parts. Bound by reading the parts, which the kernels before left in L2; every part
// is read once. A row with no part (no prefix, no suffix) gives O = 0 and lse = -inf.
__global__ void __launch_bounds__(256) prefix_merge_kernel(const PrefixMergeArgs a)
{
    constexpr int kTile = 128, D = 128;
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(a.B) * a.Hq)
        return;
    const int b = static_cast<int>(row / a.Hq), h = static_cast<int>(row % a.Hq);
    const int tile = b / a.plan.tile_seqs;
    const int in_tile = (b - tile * a.plan.tile_seqs) * a.plan.group + h % a.plan.group;
    const long long list = static_cast<long long>(h / a.plan.group) * a.plan.tile_pairs + tile / 2;
    const int len = min(max(__ldg(a.prefix_len), 0), a.cap);
    const int tiles = (len + kTile - 1) / kTile;
    const long long total = a.plan.lists * tiles;
    const int ctas = a.plan.ctas;
    // The CTAs from the one that holds the list's first unit to the one that holds its last; with fewer
    // units than CTAs those between may hold none.
    int c0 = 0, n = 0;
    if (tiles > 0) {
        c0 = static_cast<int>(((list * tiles + 1) * ctas - 1) / total);
        n = static_cast<int>((((list + 1) * tiles) * ctas - 1) / total) - c0 + 1;
    }
    auto part_row = [&](int c) { return ((list + c) * 2 + (tile & 1)) * kTile + in_tile; };
    auto lse_of = [&](int k) {
        const int c = c0 + k;
        if (k >= n || total * c / ctas >= total * (c + 1) / ctas)
            return -INFINITY;
        return __ldg(a.part_lse + part_row(c));
    };
    const float suffix = a.o_suffix ? __ldg(a.lse_suffix + row) : -INFINITY;
    float M = suffix;
    for (int k = 0; k < n; k += 32)
        M = fmaxf(M, lse_of(k + lane));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float W = 0.f;
    // A NaN LSE (from NaN scores) must not look like an empty part: M drops NaN, so weigh by the part.
    auto weight = [&](float l) { return l == -INFINITY ? 0.f : exp2f(l - M); };
    if (suffix != -INFINITY) {
        const float w = weight(suffix);
        const float4 v = __ldg(reinterpret_cast<const float4 *>(a.o_suffix + row * D) + lane);
        acc = make_float4(w * v.x, w * v.y, w * v.z, w * v.w);
        W = w;
    }
    for (int k = 0; k < n; k += 32) {
        const float l = lse_of(k + lane);
        const unsigned some = __ballot_sync(0xffffffffu, l != -INFINITY);
        const float w = weight(l);
#pragma unroll 4
        for (int t = 0; t < min(32, n - k); ++t) {
            const float wt = __shfl_sync(0xffffffffu, w, t);
            if (!((some >> t) & 1u))
                continue;
            const float4 v = __ldg(reinterpret_cast<const float4 *>(a.part_o + part_row(c0 + k + t) * D) + lane);
            acc.x = fmaf(wt, v.x, acc.x);
            acc.y = fmaf(wt, v.y, acc.y);
            acc.z = fmaf(wt, v.z, acc.z);
            acc.w = fmaf(wt, v.w, acc.w);
            W += wt;
        }
    }
    const float inv = W == 0.f ? 0.f : 1.f / W;  // 0 only for a row without parts
    __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    uint2 out;
    out.x = *reinterpret_cast<uint32_t *>(&lo);
    out.y = *reinterpret_cast<uint32_t *>(&hi);
    reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + row * D)[lane] = out;
    if (lane == 0)
        a.lse[row] = W == 0.f ? -INFINITY : (M + log2f(W)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_prefix_merge(const PrefixMergeArgs &a, cudaStream_t stream)
{
    const long long rows = static_cast<long long>(a.B) * a.Hq;
    prefix_merge_kernel<<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace attn_b200
