// q8.cuh -- the format of 8-bit K/V pools, shared by the kernels that write, read and
// attend over them.
//
// Pool: e4m3 [num_blocks, Hkv, B, d]: the rows of one head in a page are contiguous,
// so that one tiled copy brings a piece of a page for several heads.  Scales: fp32
// [num_blocks, Hkv], one for each page and head; a value is its code times its scale.
#pragma once

#include "common.cuh"
#include "divide.cuh"

namespace pkv {

// codes (low byte first) of x and y, rounded to nearest even; NaN gives NaN, sizes past
// 448 give 448
__device__ __forceinline__ uint32_t e4m3x2(float x, float y) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
    return r;
}

// the four codes of a word as two pairs of fp16 (exact): codes 0, 1 and codes 2, 3
__device__ __forceinline__ void e4m3_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

}  // namespace pkv
