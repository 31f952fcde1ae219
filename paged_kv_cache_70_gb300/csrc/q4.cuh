// q4.cuh -- the row format of 4-bit K/V pools, shared by the kernels that
// write, read and attend over them.
//
// Pool: uint8 [num_blocks, Hkv, B, R], R = 5d/8 bytes per (token, KV head) row.
// The rows of one head in a page are contiguous (a page is [Hkv][B][R]), so one
// bulk copy brings a head's rows of a page into shared memory at row stride R:
// 80 bytes for d = 128, which spreads the rows of a tile over all banks.
// Row: d/2 bytes of codes, then for each of the NG = d/32 groups of 32 dims the
// scale s and the offset z, two bf16 in one 32-bit word (s in the low half).
// Value of code u in group g:  s_g (u - 8) + z_g.
// The 16-bit unit r * NG + g of the codes (r < 8) holds dims 32 g + 4 r .. + 3,
// lowest nibble first: a lane's chunk of the row (16 bytes for the scores, 8 for
// the output, d = 128) then holds the same number of dims of every group, which
// is what one lane of the tensor-core fragments takes.
#pragma once

#include "common.cuh"

namespace pkv {

constexpr int kQ4Group = 32;

__host__ __device__ constexpr int q4_row_bytes(int d) { return d / 2 + d / kQ4Group * 4; }

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
