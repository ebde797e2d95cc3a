/*
 * suffix_sm100.cuh — the suffixes of a shared-prefix decode (attn_decode_prefix): one new token per
 * sequence over the sequence's own keys in a paged bf16 cache, head dim 128, results in fp32 for the
 * merge with the prefix (merge_sm100.cu).
 *
 * What it has to do is read every suffix's K and V once; the suffixes are many, short and of different
 * lengths. So the worker is one warp, not a CTA: a pair is one (sequence, kv head, up to 16 of its query
 * heads), its keys are units of 16, all pairs' units are laid end to end, two more before each pair for
 * what its start and end cost a warp, and cut evenly over the warps of the grid (EvenRange). Each warp
 * streams its units through a ring of its own by TMA and no warp waits for another, so the start and the
 * end of a pair are hidden behind the other eleven warps of the SM. (The CTA-wide paged decode kernel, whose
 * 128-key chunks pass through one softmax, took 53 us where this takes 31, for 125 sequences of up to 768
 * keys and 6 kv heads: it drains at every pair.)
 *
 * Per unit, K and V [16 keys][128] in shared memory (128-byte swizzle), heads in groups of eight:
 *   S^T = K Q^T       mma m16n8k16: A = K (ldmatrix), B = Q^T from registers; thread t holds keys t / 4
 *                     and t / 4 + 8 of heads 2 (t % 4) and + 1;
 *   softmax           online, base 2; the reference max moves only when a score passes it by 8; sums of
 *                     the fp32 weights (LSE) and of the bf16-rounded ones (normalises O) per thread;
 *   O^T += V^T P^T    mma m16n8k16: A = V^T (ldmatrix with transpose), B = the weights' 8 x 8 blocks
 *                     turned by movmatrix; O^T stays in registers, its columns are the thread's heads.
 * The products need a few per cent of the tensor core (8 heads: 4 flops a byte), so the warp-level
 * instructions do; memory bounds the kernel. mma.sync and not tcgen05 because a worker is one warp.
 *
 * A warp that holds a whole pair writes its result; pieces of pairs that several warps share go to the
 * workspace and the merge reads them there.
 */
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "sm100_ptx.cuh"
#include "tma_host.h"

namespace attn_b200 {
namespace suffix {

constexpr int kD = 128;
constexpr int kKeys = kSuffixUnitKeys;  // keys of a unit
constexpr int kWarps = kSuffixWarps;
constexpr int kStages = 2;  // (8 workers x 3, 6 x 4 and 4 x 6 were 2 to 18% slower over the longer suffixes)
constexpr int kBoxBytes = kKeys * 128;        // 16 keys x 64 dims
constexpr int kStageBytes = 4 * kBoxBytes;    // K dims 0-63, 64-127, then V
constexpr int kOffBar = kWarps * kStages * kStageBytes;
constexpr int kOffMisc = kOffBar + kWarps * kStages * 8;
constexpr int kOffStart = kOffMisc + 16;                    // where each sequence starts, and the end of all
constexpr int kOffUnits = kOffStart + 4 * (kPagedMaxBatch + 1);  // units before each sequence
constexpr int kOffLen = kOffUnits + 4 * (kPagedMaxBatch + 1);    // clamped lengths
constexpr int kSmem = kOffLen + 4 * kPagedMaxBatch + 1024;  // + alignment of the base
static_assert(kSmem <= 227 * 1024, "shared memory budget");
constexpr float kRescaleThreshold = 8.0f;
// Floor of the reference max: finite, so that a row of scores -inf has weights 0, not NaN, and at the end of
// fp32, below any finite score.
constexpr float kNoKeyMax = -3.4e38f;

struct SuffixParams {
    const __nv_bfloat16 *q;
    const int *seq_lens, *block_table;
    float *o, *lse, *pieces;
    int *status;
    int B, Hq, Hkv, group, head_groups, heads_per_pair;
    int num_pages, page_size, pages_per_seq, cap;
    float scale_log2;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// The transpose of an 8 x 8 matrix of 16-bit elements spread over the warp (two a thread).
__device__ __forceinline__ uint32_t turn8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A place in the sequence of all units: sequence, pair within it, unit within the pair.
struct Cursor {
    int b, pair, unit, units;
};

// The block's 32 kWarps threads; `cta` of `ctas` blocks that do this. kGroups: groups of eight query
// heads in a pair, 1 or 2.
template <int kGroups>
__device__ __forceinline__ void run(const CUtensorMap &tm_k, const CUtensorMap &tm_v, const SuffixParams &p, uint8_t *smem_raw,
                                    int cta, int ctas)
{
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc);
    int *start = reinterpret_cast<int *>(smem + kOffStart), *before = reinterpret_cast<int *>(smem + kOffUnits);
    int *len = reinterpret_cast<int *>(smem + kOffLen);
    const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp * kStages * kStageBytes);
    const uint32_t bar0 = smem_u32(smem) + kOffBar + static_cast<uint32_t>(warp * kStages * 8);
    const int pairs = p.Hkv * p.head_groups;  // of a sequence

    if (lane == 0) {
        for (int s = 0; s < kStages; ++s)
            mbar_init(bar0 + 8 * s, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (threadIdx.x == 0)
        *abort_flag = 0;
    for (int b = threadIdx.x; b < p.B; b += 32 * kWarps)
        len[b] = min(max(__ldg(p.seq_lens + b), 0), p.cap);
    __syncthreads();
    if (warp == 0) {  // exclusive sums of the sequences' units, with and without the pairs' own
        int places = 0, units = 0;
        for (int base = 0; base < p.B; base += 32) {
            const int b = base + lane;
            const int u = b < p.B ? pairs * ((len[b] + kKeys - 1) / kKeys) : 0, w = u > 0 ? u + pairs * kSuffixPairUnits : 0;
            int sum_w = w, sum_u = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum_w, o), z = __shfl_up_sync(0xffffffffu, sum_u, o);
                sum_w += lane >= o ? y : 0;
                sum_u += lane >= o ? z : 0;
            }
            if (b < p.B) {
                start[b] = places + sum_w - w;
                before[b] = units + sum_u - u;
            }
            places += __shfl_sync(0xffffffffu, sum_w, 31);
            units += __shfl_sync(0xffffffffu, sum_u, 31);
        }
        if (lane == 0) {
            start[p.B] = places;
            before[p.B] = units;
        }
    }
    __syncthreads();
    const int total = start[p.B];
    // Neighbouring ranges go to different SMs, so that few of them still use all.
    const int worker = warp * ctas + cta;
    const int workers = suffix_workers(total, ctas);
    if (worker >= workers)
        return;
    const EvenRange range(total, workers);

    // The first unit at or behind a place: even lanes find the range's begin, odd lanes its end.
    Cursor first{};
    int g0 = before[p.B];
    const int place = static_cast<int>(range.begin(worker + (lane & 1)));
    if (place < total) {
        int lo = 0, hi = p.B - 1;  // the last sequence that starts at or before it: it has units
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (start[mid] <= place)
                lo = mid;
            else
                hi = mid - 1;
        }
        first.b = lo;
        first.units = (len[lo] + kKeys - 1) / kKeys;
        const int w = place - start[lo];
        first.pair = w / (first.units + kSuffixPairUnits);
        first.unit = max(w - first.pair * (first.units + kSuffixPairUnits) - kSuffixPairUnits, 0);
        g0 = before[lo] + first.pair * first.units + first.unit;
    }
    const int n_units = __shfl_sync(0xffffffffu, g0, 1) - __shfl_sync(0xffffffffu, g0, 0);
    first.b = __shfl_sync(0xffffffffu, first.b, 0);
    first.pair = __shfl_sync(0xffffffffu, first.pair, 0);
    first.unit = __shfl_sync(0xffffffffu, first.unit, 0);
    first.units = __shfl_sync(0xffffffffu, first.units, 0);
    if (n_units == 0)
        return;
    auto next_pair = [&](Cursor &c) {
        c.unit = 0;
        if (++c.pair == pairs) {
            c.pair = 0;
            do {
                ++c.b;
            } while (c.b < p.B && len[c.b] == 0);
            c.units = c.b < p.B ? (len[c.b] + kKeys - 1) / kKeys : 0;
        }
    };

    // Copies: lane 0 keeps a cursor ahead of the one that computes, and the next unit's page with it.
    const uint64_t pol = l2_policy_evict_first();  // read once: the prefix's partials stay in L2 instead
    Cursor ahead = first;
    int issued = 0, page = 0, in_page = 0;
    auto look_up = [&]() {
        const int key = ahead.unit * kKeys, entry = key / p.page_size;
        in_page = key - entry * p.page_size;
        page = __ldg(p.block_table + static_cast<size_t>(ahead.b) * p.pages_per_seq + entry);  // not waited for here
    };
    auto issue = [&]() {  // lane 0
        const int s = issued % kStages;
        const uint32_t dst = ring + static_cast<uint32_t>(s * kStageBytes), bar = bar0 + 8 * s;
        const int kvh = ahead.pair / p.head_groups;
        if (page < 0 || page >= p.num_pages)
            page = p.num_pages;  // behind the last page: zeros
        mbar_arrive_expect_tx(bar, kStageBytes);
        tma_load_4d_hint(dst, &tm_k, bar, 0, in_page, kvh, page, pol);
        tma_load_4d_hint(dst + kBoxBytes, &tm_k, bar, 64, in_page, kvh, page, pol);
        tma_load_4d_hint(dst + 2 * kBoxBytes, &tm_v, bar, 0, in_page, kvh, page, pol);
        tma_load_4d_hint(dst + 3 * kBoxBytes, &tm_v, bar, 64, in_page, kvh, page, pol);
        if (++issued < n_units) {
            if (++ahead.unit == ahead.units)
                next_pair(ahead);
            look_up();
        }
    };
    if (lane == 0) {
        look_up();
        for (int s = 0; s < kStages && s < n_units; ++s)
            issue();
    }

    // ldmatrix rows: lane l gives a row of matrix l / 8. K: rows are keys, matrices (keys 0-7, 8-15) x
    // (dims 0-7, 8-15); V: rows are keys, matrices (dims 0-7, 8-15) x (keys 0-7, 8-15), read transposed.
    const int mat = lane >> 3, in8 = lane & 7;
    const int k_row = in8 + (mat & 1) * 8, k_chunk = mat >> 1;
    const int v_row = in8 + (mat >> 1) * 8, v_chunk = mat & 1;
    const uint32_t k_base = static_cast<uint32_t>(k_row * 128), v_base = static_cast<uint32_t>(2 * kBoxBytes + v_row * 128);

    Cursor cur = first;
    bool ok = true;
    for (int done = 0; ok && done < n_units;) {
        const int b = cur.b, kvh = cur.pair / p.head_groups, hg = cur.pair - kvh * p.head_groups;
        const int h0 = kvh * p.group + hg * p.heads_per_pair;
        const int heads = min(p.heads_per_pair, p.group - hg * p.heads_per_pair);
        const int seq_len = len[b];
        const int n = min(cur.units - cur.unit, n_units - done);
        const bool whole = n == cur.units;

        // Q^T: head t / 4 of each group of eight, dims 2 (t % 4), + 1, and those + 8, of every 16.
        uint32_t qf[kGroups][8][2];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int h = g * 8 + (lane >> 2);
            const uint32_t *row = reinterpret_cast<const uint32_t *>(p.q + (static_cast<size_t>(b) * p.Hq + h0 + min(h, heads - 1)) * kD);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    qf[g][ks][e] = h < heads ? __ldg(row + ks * 8 + e * 4 + (lane & 3)) : 0u;
        }
        float o[kGroups][8][4], m[kGroups][2], l[kGroups][2], lpv[kGroups][2];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
#pragma unroll
            for (int d = 0; d < 8; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[g][d][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[g][e] = kNoKeyMax;
                l[g][e] = lpv[g][e] = 0.f;
            }
        }
        for (int j = 0; j < n; ++j, ++done) {
            const int s = done % kStages;
            // Agreed by the warp: it gates warp-collective instructions.
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar0 + 8 * s, static_cast<uint32_t>(done / kStages) & 1u, abort_flag,
                                                         p.status, kSiteSuffix))))
                break;
            const uint32_t stage = ring + static_cast<uint32_t>(s * kStageBytes);
            const int valid = seq_len - (cur.unit + j) * kKeys;  // keys of this unit, if below 16
            if (valid < kKeys) {
                // Rows behind the last key hold what the cache holds there; their weights are 0, but
                // 0 * NaN is not.
                uint8_t *v = smem + warp * kStages * kStageBytes + s * kStageBytes + 2 * kBoxBytes;
                for (int i = lane; i < (kKeys - valid) * 16; i += 32) {
                    const int row = valid + (i >> 4), c = i & 15;
                    *reinterpret_cast<uint4 *>(v + (c >> 3) * kBoxBytes + row * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();  // before the next copy into this stage
                __syncwarp();
            }
            // S^T, two chains of four steps each.
            float sc[kGroups][2][4];
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[g][c][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                uint32_t a[4];
                const uint32_t chunk = static_cast<uint32_t>(((ks & 3) * 2 + k_chunk) ^ (k_row & 7));
                ldmatrix4(a, stage + (ks >> 2) * kBoxBytes + k_base + chunk * 16);
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
                    mma_bf16(sc[g][ks & 1], a, qf[g][ks][0], qf[g][ks][1]);
            }
            // Scores in log2 units; element e: key lane / 4 + 8 (e / 2), head 2 (lane % 4) + e % 2.
            float x[kGroups][4];
            bool need = false;
            float top[kGroups][2];
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[g][e] = (lane >> 2) + 8 * (e >> 1) < valid ? (sc[g][0][e] + sc[g][1][e]) * p.scale_log2 : -INFINITY;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[g][e] = fmaxf(x[g][e], x[g][e + 2]);
                    need = need || top[g][e] > m[g][e] + kRescaleThreshold;
                }
            }
            if (__any_sync(0xffffffffu, need)) {
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float t = top[g][e];
#pragma unroll
                        for (int sh = 4; sh < 32; sh <<= 1)
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, sh));
                        const float mn = fmaxf(m[g][e], t), alpha = ex2(m[g][e] - mn);
                        m[g][e] = mn;
                        l[g][e] *= alpha;
                        lpv[g][e] *= alpha;
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            o[g][d][e] *= alpha;
                            o[g][d][e + 2] *= alpha;
                        }
                    }
            }
            // Weights; their 8 x 8 blocks (keys 0-7, 8-15) turned into the product's B operand.
            uint32_t pb[kGroups][2];
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float p0 = ex2(x[g][2 * half] - m[g][0]), p1 = ex2(x[g][2 * half + 1] - m[g][1]);
                    const __nv_bfloat162 w = __floats2bfloat162_rn(p0, p1);
                    l[g][0] += p0;
                    l[g][1] += p1;
                    lpv[g][0] += __low2float(w);
                    lpv[g][1] += __high2float(w);
                    pb[g][half] = turn8x8(*reinterpret_cast<const uint32_t *>(&w));
                }
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                uint32_t a[4];
                const uint32_t chunk = static_cast<uint32_t>(((d & 3) * 2 + v_chunk) ^ (v_row & 7));
                ldmatrix4_trans(a, stage + (d >> 2) * kBoxBytes + v_base + chunk * 16);
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
                    mma_bf16(o[g][d], a, pb[g][0], pb[g][1]);
            }
            __syncwarp();  // every lane has read the stage
            if (lane == 0 && issued < n_units)
                issue();
        }
        if (!ok)
            break;

        // The pair's result, or this warp's piece of it: its first or its last.
        float *dst, *dst_lse;
        if (whole) {
            const size_t row = static_cast<size_t>(b) * p.Hq + h0;
            dst = p.o + row * kD;
            dst_lse = p.lse + row;
        } else {
            dst = p.pieces + (static_cast<size_t>(worker) * 2 + (done == n ? 0 : 1)) * suffix_piece(p.heads_per_pair);
            dst_lse = dst + p.heads_per_pair * kD;
        }
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int sh = 4; sh < 32; sh <<= 1) {
                    l[g][e] += __shfl_xor_sync(0xffffffffu, l[g][e], sh);
                    lpv[g][e] += __shfl_xor_sync(0xffffffffu, lpv[g][e], sh);
                }
                const int h = g * 8 + 2 * (lane & 3) + e;
                if (h < heads) {
                    const float inv = 1.f / lpv[g][e];
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        dst[h * kD + d * 16 + (lane >> 2)] = o[g][d][e] * inv;
                        dst[h * kD + d * 16 + (lane >> 2) + 8] = o[g][d][e + 2] * inv;
                    }
                    if ((lane >> 2) == 0)
                        dst_lse[h] = m[g][e] + log2f(l[g][e]);
                }
            }
        cur.unit += n;
        if (cur.unit == cur.units)
            next_pair(cur);
    }
    if (!ok && lane == 0) {
        // Let every copy already issued land before the CTA exits.
        for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i) {
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(bar0 + 8 * (i % kStages), static_cast<uint32_t>(i / kStages) & 1u) &&
                   global_timer_ns() - t0 < 100000000ull) {
            }
        }
    }
}

// Pages [num_pages][Hkv][page_size][D] as (dim, slot, kv head, page): boxes of 64 dims, 16 keys.
inline bool make_maps(PFN_cuTensorMapEncodeTiled_v12000 encode, const SuffixArgs &a, CUtensorMap *tk, CUtensorMap *tv, int *err)
{
    const Strides st{static_cast<long long>(a.Hkv) * a.page_size * kD, static_cast<long long>(a.page_size) * kD, kD};
    return make_map4(encode, tk, a.k_pages, 2, kD, a.page_size, a.Hkv, a.num_pages, st, 64, kKeys, CU_TENSOR_MAP_SWIZZLE_128B, err) &&
           make_map4(encode, tv, a.v_pages, 2, kD, a.page_size, a.Hkv, a.num_pages, st, 64, kKeys, CU_TENSOR_MAP_SWIZZLE_128B, err);
}

inline SuffixParams params(const SuffixArgs &a)
{
    SuffixParams p;
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.seq_lens = a.seq_lens;
    p.block_table = a.block_table;
    p.o = a.o;
    p.lse = a.lse;
    p.pieces = a.pieces;
    p.status = a.status;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.group = a.Hq / a.Hkv;
    p.head_groups = a.plan.head_groups;
    p.heads_per_pair = a.plan.heads_per_pair;
    p.num_pages = a.num_pages;
    p.page_size = a.page_size;
    p.pages_per_seq = a.pages_per_seq;
    p.cap = a.cap;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    return p;
}

}  // namespace suffix
}  // namespace attn_b200
