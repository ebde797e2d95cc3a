/*
 * prefix_split.cuh — how the blocks of a shared-prefix decode (attn_decode_prefix) are divided between
 * prefix and suffixes, and the prefix's among its lists of KV tiles.
 *
 * The first `ctas` blocks of the grid take the prefix, the rest the suffixes, side by side: the prefix is
 * bound by its softmax and tensor work, the suffixes by memory, and neither waits for the other (one behind
 * the other, 125 sequences of up to 768 keys behind 32,749 took 79 us instead of 65). A model of both
 * times, measured, says which split ends first, a tenth of the prefix's added so that of splits that end
 * alike it takes the one with the shorter prefix:
 *   prefix     4 us, and for each KV tile of a block 1.6 us, or 1.4 us in a list of one query tile;
 *   suffixes   4 us, and for each unit (16 keys' K and V, 8 KB) the root of the sum of the squares of what
 *              it takes the SMs, 0.074 us of one (0.098 us where a pair has two groups of heads), and what it
 *              takes the memory, 0.0007 us.
 * The prefix's blocks are divided one list at a time (a head's last list may hold one tile only and
 * then gets fewer), so that a block has one segment; or, where that fits badly, all lists laid end to end
 * are cut evenly and most blocks have two, 3 us more.
 *
 * The lengths are known on the device only. There the blocks work the split out, each for itself and all
 * alike, and one leaves it for the merge, which costs 3 us. So for calls that take no more than
 * kFixedSplitUs by their greatest lengths the host fixes the split from those. 32 sequences of up to 512
 * keys behind 4,096 take 20.0 us so and 23.2 by the device's split; when they hold a fifth of that, 19.4 and
 * 18.3. For 128 sequences, a longer call, the last two are 39.7 and 27.3.
 */
#pragma once

#include <cuda_runtime.h>

#include <cmath>

#include "kernels.h"

namespace attn_b200 {

__host__ __device__ __forceinline__ float about_quotient(float a, float b)
{
#ifdef __CUDA_ARCH__
    return __fdividef(a, b);
#else
    return a / b;
#endif
}

__host__ __device__ __forceinline__ float about_root(float x)
{
#ifdef __CUDA_ARCH__
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
#else
    return sqrtf(x);
#endif
}

// Candidate i of all splits, and its model time in us; infinity when there is none. Any split is right,
// so the times are rounded as it comes.
__host__ __device__ __forceinline__ float split_candidate(const PrefixPlan &p, int i, float tiles, float work, PrefixSplit *s)
{
    auto up = [](float n, int parts) { return ceilf(about_quotient(n, static_cast<float>(parts)) - 1e-3f); };
    const int most = p.grid - (work > 0.f ? 1 : 0);
    float us;
    if (i < 32) {  // end to end
        s->ctas = most * (i + 1) / 32 > 1 ? most * (i + 1) / 32 : 1;
        s->per_list = s->per_last = 0;
        us = 4.0f + 3.0f * up(static_cast<float>(p.lists), s->ctas) + 1.6f * up(tiles * static_cast<float>(p.lists), s->ctas);
    } else {  // a head's blocks: a share for each full list, the rest for the last (a single tile's: 0.8 of one)
        const int each = p.tile_pairs + i - 32;
        s->ctas = each * p.heads;
        if (s->ctas > most)
            return INFINITY;
        const int share = static_cast<int>(p.by_share.quot(p.odd ? 10 * each : each));
        s->per_list = p.tile_pairs == 1 ? 0 : share > 1 ? share : 1;
        s->per_last = each - (p.tile_pairs - 1) * s->per_list;
        us = 4.0f + fmaxf(s->per_list ? 1.6f * up(tiles, s->per_list) : 0.f, (p.odd ? 1.4f : 1.6f) * up(tiles, s->per_last));
    }
    const float own_us = about_quotient(p.suffix_unit_us, static_cast<float>(p.grid - s->ctas));
    return 0.1f * us + (work > 0.f ? fmaxf(us, 4.0f + work * about_root(own_us * own_us + 0.0007f * 0.0007f)) : us);
}

// The number of candidates, from the most blocks that one head can have.
__host__ __device__ __forceinline__ int split_candidates(const PrefixPlan &p)
{
    const int each = p.by_heads.quot(p.grid) - p.tile_pairs + 1;
    return 32 + (each > 0 ? each : 0);
}

// By a whole warp; every lane gets the result. `tiles`: KV tiles of the prefix, `work`: all suffixes' units,
// the pairs' own included.
__device__ __forceinline__ PrefixSplit split_prefix(const PrefixPlan &p, int tiles, int work, int lane)
{
    PrefixSplit mine{}, s;
    if (tiles == 0)
        return mine;
    float best = INFINITY;
    const int n = split_candidates(p);
    for (int i = lane; i < n; i += 32) {
        const float us = split_candidate(p, i, static_cast<float>(tiles), static_cast<float>(work), &s);
        if (us < best) {
            best = us;
            mine = s;
        }
    }
    const unsigned least = __reduce_min_sync(0xffffffffu, __float_as_uint(best));  // times are positive
    const int from = __ffs(__ballot_sync(0xffffffffu, __float_as_uint(best) == least)) - 1;
    s.ctas = __shfl_sync(0xffffffffu, mine.ctas, from);
    s.per_list = __shfl_sync(0xffffffffu, mine.per_list, from);
    s.per_last = __shfl_sync(0xffffffffu, mine.per_last, from);
    return s;
}

// Units of 16 keys of one suffix, and with what each pair counts on top.
__device__ __forceinline__ int suffix_units(int len, int cap)
{
    return (min(max(len, 0), cap) + kSuffixUnitKeys - 1) / kSuffixUnitKeys;
}
__device__ __forceinline__ int suffix_work(int len, int cap)
{
    const int u = suffix_units(len, cap);
    return u > 0 ? u + kSuffixPairUnits : 0;
}

}  // namespace attn_b200
