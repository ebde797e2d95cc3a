/*
 * fast_div.h — division of row and unit numbers by sizes that the host knows.
 */
#pragma once

#include <cstdint>

namespace attn_b200 {

// n / d and n % d for 0 <= n < 2^31 by one multiplication: with s = ceil(log2 d) and
// m = ceil(2^(31+s) / d), m d - 2^(31+s) < d <= 2^s, so n m / 2^(31+s) is above n / d by less than
// n / 2^31 < 1 in units of 1 / d, and its floor is exact.
struct FastDiv {
    uint32_t d = 1, m = 0, s = 0;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div)
    {
        while ((1ull << s) < d)
            ++s;
        m = static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d);
    }
    __host__ __device__ __forceinline__ uint32_t quot(uint32_t n) const
    {
        return d == 1 ? n : static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> (31 + s));
    }
};

}  // namespace attn_b200
