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
#include "prefix_split.cuh"

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

// Attention of one row of a shared-prefix decode from its parts, all fp32 with LSEs in log2 units: the
// segments of its list of prefix tiles (prefill_sm100.cu, decode_segment) and its suffix, whole or in
// the pieces that the workers which shared its pair left (suffix_sm100.cuh).
//   M = max LSE_s,  O = sum 2^(LSE_s - M) O_s / W,  lse = (M + log2 W) ln 2,  W = sum 2^(LSE_s - M).
// kSplit warps take one row, each every kSplit-th part: lane i looks up where its i-th part lies and
// its LSE (before any O is read), then each lane adds its four channels over the warp's parts, eight reads
// in flight, and the warps' sums are joined in shared memory. Bound by the latency of that chain for few
// rows (four warps a row: see the launch), by reading the parts, still in L2, for many. Where the parts lie
// follows from the lengths alone and is computed before the wait for the kernel that writes them (kFind: the
// split of that kernel's grid too, from the same lengths). A row with no part (no prefix, no suffix) gives
// O = 0 and lse = -inf.
constexpr int kMergeWarps = 4;
constexpr int kMergeSplitRows = 1024;

template <int kSplit, bool kFind>
__global__ void __launch_bounds__(32 * kMergeWarps) prefix_merge_kernel(const PrefixMergeArgs a)
{
    constexpr int kTile = 128, D = 128;
    static_assert(kSplit == 1 || kSplit == kMergeWarps, "a row has a warp or a block");
    const int lane = threadIdx.x & 31, warp = kSplit == 1 ? 0 : threadIdx.x >> 5;
    const int row = kSplit == 1 ? blockIdx.x * kMergeWarps + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= a.B * a.Hq)
        return;
    const int b = a.by_hq.quot(row), h = row - b * a.Hq;

    const int tiles = (min(max(__ldg(a.prefix_len), 0), a.cap) + kTile - 1) / kTile;
    const int per = a.suffix.heads_per_pair, pairs = a.Hkv * a.suffix.head_groups;
    int before = 0, all = 0, own = 0;  // work of the sequences before b and of all, units of b
    if (a.o_suffix) {
        own = suffix_units(__ldg(a.seq_lens + b), a.suffix_cap);
        for (int i = lane; i < a.B; i += 32) {
            const int u = suffix_work(__ldg(a.seq_lens + i), a.suffix_cap);
            all += u;
            before += i < b ? u : 0;
        }
        before = __reduce_add_sync(0xffffffffu, before);
        all = __reduce_add_sync(0xffffffffu, all);
    }
    const int total = all * pairs;
    PrefixSplit split = a.fixed;
    if constexpr (kFind)
        split = split_prefix(a.plan, tiles, total, lane);
    // Prefix: the blocks from the one that holds the list's first KV tile to the one that holds its last.
    const int tile = a.by_tile_seqs.quot(b), part_of_heads = a.by_tile_group.quot(h);
    const int in_tile = (b - tile * a.plan.tile_seqs) * a.plan.group + h - part_of_heads * a.plan.group;
    const int pair = tile / 2, list = part_of_heads * a.plan.tile_pairs + pair;
    int c0 = 0, n_prefix = 0;
    if (split.per_last > 0) {
        c0 = part_of_heads * split.per_head(a.plan.tile_pairs) + pair * split.per_list;
        n_prefix = min(pair + 1 == a.plan.tile_pairs ? split.per_last : split.per_list, tiles);
    } else if (tiles > 0) {
        const EvenRange range(static_cast<unsigned>(a.plan.lists) * tiles, split.ctas);
        c0 = static_cast<int>(range.part_of(list * tiles));
        n_prefix = static_cast<int>(range.part_of((list + 1) * tiles - 1)) - c0 + 1;
    }
    // Suffix: its pair's units among all pairs' units, as suffix::run lays them.
    int s0 = 0, n_suffix = 0, in_pair = 0, first_piece = 0;
    if (own > 0) {
        const int g = a.by_group.quot(h), in_group = h - g * static_cast<int>(a.by_group.d), hg = a.by_pair.quot(in_group);
        in_pair = in_group - hg * per;
        const int start = before * pairs + (g * a.suffix.head_groups + hg) * (own + kSuffixPairUnits), first = start + kSuffixPairUnits;
        const EvenRange range(total, suffix_workers(total, a.plan.grid - split.ctas));
        s0 = static_cast<int>(range.part_of(first));
        n_suffix = static_cast<int>(range.part_of(first + own - 1)) - s0 + 1;
        // The first worker's piece is its last one unless its range starts with the pair.
        first_piece = static_cast<int>(range.begin(s0)) >= start ? 0 : 1;
    }
    const int n = n_prefix + n_suffix;

    // Where part k's O row and its LSE lie; null behind the last.
    auto find_part = [&](int k, const float **o, const float **lse) {
        *o = *lse = nullptr;
        if (k < n_prefix) {
            const long long r = (static_cast<long long>(list + c0 + k) * 2 + (tile & 1)) * kTile + in_tile;
            *o = a.part_o + r * D;
            *lse = a.part_lse + r;
        } else if (k < n && n_suffix == 1) {  // the whole pair
            *o = a.o_suffix + static_cast<size_t>(row) * D;
            *lse = a.lse_suffix + row;
        } else if (k < n) {
            const int i = k - n_prefix;
            const float *piece = a.pieces + (static_cast<size_t>(s0 + i) * 2 + (i == 0 ? first_piece : 0)) * suffix_piece(per);
            *o = piece + in_pair * D;
            *lse = piece + per * D + in_pair;
        }
    };
    const float *o, *lse;
    find_part(lane * kSplit + warp, &o, &lse);
    float M = -INFINITY, W = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int k = 0; k < n; k += 32 * kSplit) {
        if (k > 0)
            find_part(k + lane * kSplit + warp, &o, &lse);
        const float l = lse ? __ldcg(lse) : -INFINITY;
        const int parts = min(32, (n - k - warp + kSplit - 1) / kSplit);
        // Eight parts' rows at a time, the first eight sent for before their weights are known (16 at a time
        // took longer: fewer blocks fit an SM).
        constexpr int kFlight = 8;
        float4 v[kFlight];
        auto fetch = [&](int t) {
#pragma unroll
            for (int j = 0; j < kFlight; ++j) {
                const float *po = reinterpret_cast<const float *>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), min(t + j, 31)));
                v[j] = t + j < parts ? __ldcg(reinterpret_cast<const float4 *>(po) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        };
        fetch(0);
        float m = l;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
        const float new_m = fmaxf(M, m);
        const float keep = M == -INFINITY ? 0.f : exp2f(M - new_m);
        acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
        W *= keep;
        M = new_m;
        // fmaxf drops NaN: a part with a NaN LSE (from NaN scores) keeps a NaN weight.
        const float w = l == -INFINITY ? 0.f : exp2f(l - M);
        for (int t = 0; t < parts; t += kFlight) {
            if (t > 0)
                fetch(t);
#pragma unroll
            for (int j = 0; j < kFlight; ++j) {
                const float wt = __shfl_sync(0xffffffffu, w, min(t + j, 31)), u = t + j < parts ? wt : 0.f;
                if (u != 0.f) {  // a part of weight 0 may hold anything (all its scores -inf)
                    acc.x = fmaf(u, v[j].x, acc.x);
                    acc.y = fmaf(u, v[j].y, acc.y);
                    acc.z = fmaf(u, v[j].z, acc.z);
                    acc.w = fmaf(u, v[j].w, acc.w);
                    W += u;
                }
            }
        }
    }
    if constexpr (kSplit == 1) {
        const float inv = W == 0.f ? 0.f : 1.f / W;  // 0 only for a row without parts
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        uint2 out;
        out.x = *reinterpret_cast<const uint32_t *>(&lo);
        out.y = *reinterpret_cast<const uint32_t *>(&hi);
        reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + static_cast<size_t>(row) * D)[lane] = out;
        if (lane == 0)
            a.lse[row] = W == 0.f ? -INFINITY : (M + log2f(W)) * 0.6931471805599453f;
        return;
    }
    __shared__ float s_acc[kMergeWarps][D];
    __shared__ float s_m[kMergeWarps], s_w[kMergeWarps];
    *reinterpret_cast<float4 *>(&s_acc[warp][4 * lane]) = acc;
    if (lane == 0) {
        s_m[warp] = M;
        s_w[warp] = W;
    }
    __syncthreads();
    const int d = threadIdx.x;  // one channel each
    float top = s_m[0];
#pragma unroll
    for (int v = 1; v < kMergeWarps; ++v)
        top = fmaxf(top, s_m[v]);
    float sum = 0.f, out = 0.f;
#pragma unroll
    for (int v = 0; v < kMergeWarps; ++v) {
        // A warp without parts has M = -inf and sums 0 (or NaN, which stays).
        const float f = s_m[v] == top ? 1.f : exp2f(s_m[v] - top);
        sum = fmaf(f, s_w[v], sum);
        out = fmaf(f, s_acc[v][d], out);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // 0 only for a row without parts
    static_cast<__nv_bfloat16 *>(a.o)[static_cast<size_t>(row) * D + d] = __float2bfloat16_rn(out * inv);
    if (d == 0)
        a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_prefix_merge(const PrefixMergeArgs &args, cudaStream_t stream)
{
    PrefixMergeArgs a = args;
    a.by_hq = FastDiv(a.Hq);
    a.by_tile_seqs = FastDiv(a.plan.tile_seqs);
    a.by_tile_group = FastDiv(a.plan.group);
    a.by_group = FastDiv(a.Hq / a.Hkv);
    a.by_pair = FastDiv(a.suffix.heads_per_pair);
    static_assert(32 * kMergeWarps == 128, "one thread a channel");
    const int rows = a.B * a.Hq;
    // Four warps a row shorten the chain of a row's parts, one costs fewer blocks. Measured with either
    // behind 4,096 + 256 keys (about 18 parts a row), 32 query and 8 kv heads: 128 rows 12.2 us a call with four
    // and 14.5 with one, 768 rows 14.8 and 15.7, 1,024 rows 17.0 and 17.4, 1,280 rows 20.0 and 18.8, 4,096 rows
    // 47 and 37. (Rows of few parts, behind 512 keys, were faster with one at any count: 128 rows 9.6 and
    // 8.9, 1,024 rows 12.1 and 10.6.)
    const int split_blocks = rows, blocks = (rows + kMergeWarps - 1) / kMergeWarps;
    auto launch = [&](auto kernel, int grid) { return launch_behind(kernel, dim3(static_cast<unsigned>(grid)), 32 * kMergeWarps, stream, a); };
    if (rows <= kMergeSplitRows)
        return a.find ? launch(prefix_merge_kernel<kMergeWarps, true>, split_blocks)
                       : launch(prefix_merge_kernel<kMergeWarps, false>, split_blocks);
    return a.find ? launch(prefix_merge_kernel<1, true>, blocks) : launch(prefix_merge_kernel<1, false>, blocks);
}

}  // namespace attn_b200
