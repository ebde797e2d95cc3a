/*
 * prefix_split.cuh — how the blocks of a shared-prefix decode (attn_decode_prefix) are divided between
 * prefix and suffixes, and the prefix's among its lists of KV tiles.
 *
 * The first `ctas` blocks of the grid take the prefix, the rest the suffixes, side by side: the prefix is
 * bound by its softmax and tensor work, the suffixes by memory, and neither waits for the other (one behind
 * the other, 125 sequences of up to 768 keys behind 32,749 took 79 us instead of 63). A model of both
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
 * Of the splits that there can be, 32 are compared. The lengths are known on the device only: there a warp of
 * each block compares them, one a lane, and the merge does the same before it waits for the blocks, every
 * operation with its rounding named, so that all come to one choice. (32 prepared splits read from the
 * kernel's parameters took 2 to 4 us longer, the choice left in memory for the merge 1.5 us.) That takes 1 to
 * 1.5 us, so for short calls (kFixedSplitUs by the model) the host fixes the split, from the greatest lengths
 * that the call allows: 32 sequences of up to 512 keys behind 4,096, the first to be left to the device,
 * take 21.9 us with it and 20.7 with a fixed split, 18.7 and 19.4 when half as long; 128 of
 * them 55 either way, 36 and 41.
 */
#pragma once

#include <cuda_runtime.h>

#include <cmath>

#include "kernels.h"

namespace attn_b200 {

__host__ __device__ __forceinline__ float times(float a, float b)
{
#ifdef __CUDA_ARCH__
    return __fmul_rn(a, b);
#else
    return a * b;
#endif
}

__host__ __device__ __forceinline__ float plus(float a, float b)
{
#ifdef __CUDA_ARCH__
    return __fadd_rn(a, b);
#else
    return a + b;
#endif
}

// 1 / n and the square root, to a few units in the last place.
__host__ __device__ __forceinline__ float one_over(int n)
{
#ifdef __CUDA_ARCH__
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(__int2float_rn(n)));
    return y;
#else
    return 1.0f / static_cast<float>(n);
#endif
}

__host__ __device__ __forceinline__ float root(float x)
{
#ifdef __CUDA_ARCH__
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
#else
    return sqrtf(x);
#endif
}

// Split i of 32, and what it takes (us).
__host__ __device__ __forceinline__ float split_candidate(const PrefixPlan &p, int i, float tiles, float work, PrefixSplit *s)
{
    auto up = [](float n) { return ceilf(plus(n, -1e-3f)); };
    const int pairs = p.tile_pairs;
    float us;
    if (i < p.by_head) {  // a head's blocks: a share for each full list, the rest for the last (a single tile's: 0.8 of one)
        const int each = pairs + static_cast<int>(p.by_steps.quot(static_cast<unsigned>(p.steps * i)));
        const int share = static_cast<int>(p.by_share.quot(static_cast<unsigned>(p.odd ? 10 * each : each)));
        s->per_list = pairs == 1 ? 0 : share > 1 ? share : 1;
        s->per_last = each - (pairs - 1) * s->per_list;
        s->ctas = each * p.heads;
        const float full = s->per_list ? times(1.6f, up(times(tiles, one_over(s->per_list)))) : 0.f;
        us = plus(4.0f, fmaxf(full, times(p.odd ? 1.4f : 1.6f, up(times(tiles, one_over(s->per_last))))));
    } else {  // end to end
        const int ctas = static_cast<int>(p.by_rest.quot(static_cast<unsigned>(p.grid * (32 - i))));
        s->ctas = ctas > 1 ? ctas : 1;
        s->per_list = s->per_last = 0;
        const float lists = times(static_cast<float>(p.lists), one_over(s->ctas));
        us = plus(plus(4.0f, times(3.0f, up(lists))), times(1.6f, up(times(tiles, lists))));
    }
    float ends = us;
    if (work > 0.f) {
        const float own = times(p.suffix_unit_us, one_over(p.grid - s->ctas));  // infinite without a block for it
        ends = fmaxf(us, plus(4.0f, times(work, root(plus(times(own, own), 0.0007f * 0.0007f)))));
    }
    return plus(times(0.1f, us), ends);
}

// By a whole warp; every lane gets the choice. `tiles`: KV tiles of the prefix; `work`: all suffixes' units,
// the pairs' own included.
__device__ __forceinline__ PrefixSplit split_prefix(const PrefixPlan &p, int tiles, int work, int lane)
{
    PrefixSplit s;
    const unsigned us = __float_as_uint(split_candidate(p, lane, __int2float_rn(tiles), __int2float_rn(work), &s));  // positive
    const unsigned least = __reduce_min_sync(0xffffffffu, us);
    const int best = __ffs(__ballot_sync(0xffffffffu, us == least)) - 1;
    s.ctas = __shfl_sync(0xffffffffu, s.ctas, best);
    s.per_list = __shfl_sync(0xffffffffu, s.per_list, best);
    s.per_last = __shfl_sync(0xffffffffu, s.per_last, best);
    return tiles > 0 ? s : PrefixSplit{0, 0, 0};
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
