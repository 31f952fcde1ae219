// divide.cuh -- division of positions and slots by a page's size, known at the launch.
#pragma once

#include <cstdint>

namespace pkv {

// n / d for 0 <= n < 2^31 by one multiply-high (round-up reciprocal): with
// s = ceil(log2 d), mul = floor(2^32 (2^s - d) / d) + 1,
// n / d = (mulhi(n, mul) + n) >> s.
struct FastDiv {
    uint32_t mul, shift, d;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div) {
        shift = 0;
        while ((1ull << shift) < div) ++shift;
        mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - div)) / div + 1);
    }
    __device__ __forceinline__ uint32_t quot(uint32_t n) const {
        return (__umulhi(n, mul) + n) >> shift;
    }
};

}  // namespace pkv
