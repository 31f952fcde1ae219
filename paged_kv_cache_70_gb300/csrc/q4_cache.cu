// q4_cache.cu -- rows into and out of 4-bit K/V pools (format: q4.cuh).
//
// Write ("自己来实现一个", _update_paged_kv_cache_kernel, with a 4-bit cache
// dtype): for every token n with s = slot_mapping[n] >= 0 and every KV head, each
// group of 32 dims x of the row is stored as
//   s = bf16((hi - lo) / 15)   z = bf16((lo / 2 + hi / 2) + s / 2)
//   u = min(max(rint((x - z) * (1 / s)) + 8, 0), 15)
// with lo, hi the group's minimum and maximum and every operation rounded to
// fp32.  Values lie on both sides of z: u = 0 .. 15 spans z - 8s .. z + 7s, i.e.
// lo .. hi.  s below 2^-126 is stored as 0 with every value z.  A NaN makes lo
// and hi NaN and an infinity makes hi - lo infinite or NaN, so that such a group
// reads back as NaN instead of as a plausible number.
// Read: row n of the outputs is the values s (u - 8) + z at slot_mapping[n],
// rounded once to the output's type; zeros for a negative slot.
//
// Both move bytes: one warp per token and pool (grid.y: K, V), a lane per 8
// dims.  The four lanes of a group find lo and hi with two xor shuffles; two
// more shuffles exchange 16-bit code units between the groups of a head, so
// that the codes leave (and arrive) as whole 32-bit words, consecutive over the
// lanes.
//
// Measured (17,928 rows of 8 x 128, bf16, 96.4 MB of rows and codes): write 20.8 us,
// 4634 GB/s, bound by issue slots (79 % busy, 17 instructions per value for
// minimum, maximum, scaling, rounding and packing); its first form, with conversions,
// clamps and a division per value, took 27.  Read 16.7 us, 5780 GB/s (0.85 of the
// measured copy rate; 34,567 rows 30.7 us, 0.89), with a multiply and add per value in
// fp32 and a second rounding 17.0.
#include <algorithm>

#include "common.cuh"
#include "launch.h"
#include "q4.cuh"

namespace pkv {

namespace {

constexpr int kQ4Warps = 4;   // tokens per CTA

struct Q4Rows {
    const int32_t* slots;
    int64_t num_tokens;
    int64_t num_slots;
    FastDiv block;   // tokens per page
    int32_t hkv;
    unsigned int* err;
};

// lane's place in its 32-lane step: head row, group, chunk of 8 dims
template <int NG>
__device__ __forceinline__ void lane_place(int vec, int* head, int* g, int* c) {
    *head = vec / (4 * NG);
    *g = (vec / 4) % NG;
    *c = vec % 4;
}

// byte offset of head `h`'s row at `slot`
template <int NG>
__device__ __forceinline__ int64_t row_offset(const Q4Rows& a, int32_t page, int32_t at, int h) {
    return (((int64_t)page * a.hkv + h) * a.block.d + at) * q4_row_bytes(NG * kQ4Group);
}

// word w of lane (g, c) holds its 8 codes as two units (r = 2c low, 2c + 1 high).
// Exchange between the groups of a head: lane j of the NG lanes with the same
// c gets the j-th 32-bit word of chunk c of the row.
template <int NG>
__device__ __forceinline__ uint32_t units_to_words(uint32_t w, int lane, int g) {
    const int src = lane - 4 * g + 4 * (NG == 4 ? 2 * (g & 1) : 0);
    const uint32_t a = __shfl_sync(0xffffffffu, w, src);
    const uint32_t b = __shfl_sync(0xffffffffu, w, src + 4);
    return __byte_perm(a, b, (NG == 4 ? g >> 1 : g) ? 0x7632 : 0x5410);
}
// the inverse
template <int NG>
__device__ __forceinline__ uint32_t words_to_units(uint32_t w, int lane, int g) {
    const int src = lane - 4 * g + 4 * (NG == 4 ? g >> 1 : 0);
    const uint32_t a = __shfl_sync(0xffffffffu, w, src);
    const uint32_t b = __shfl_sync(0xffffffffu, w, src + (NG == 4 ? 8 : 4));
    return __byte_perm(a, b, (g & 1) ? 0x7632 : 0x5410);
}

template <bool F32>
struct Raw8 {
    uint4 a, b;  // b: fp32 only
};

template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t elem, Raw8<F32>& x) {
    if constexpr (F32) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + elem);
        x.a = __ldcs(p);
        x.b = __ldcs(p + 1);
    } else {
        x.a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem));
    }
}

template <bool F32>
__device__ __forceinline__ void widen8(const Raw8<F32>& r, float2* x) {
    if constexpr (F32) {
        x[0] = make_float2(__uint_as_float(r.a.x), __uint_as_float(r.a.y));
        x[1] = make_float2(__uint_as_float(r.a.z), __uint_as_float(r.a.w));
        x[2] = make_float2(__uint_as_float(r.b.x), __uint_as_float(r.b.y));
        x[3] = make_float2(__uint_as_float(r.b.z), __uint_as_float(r.b.w));
    } else {
        x[0] = make_float2(bf16lo(r.a.x), bf16hi(r.a.x));
        x[1] = make_float2(bf16lo(r.a.y), bf16hi(r.a.y));
        x[2] = make_float2(bf16lo(r.a.z), bf16hi(r.a.z));
        x[3] = make_float2(bf16lo(r.a.w), bf16hi(r.a.w));
    }
}

// minimum and maximum that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
    float y;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// x / 15 rounded to nearest, x >= 0: from a quotient that is off by an ulp at most,
// one step with the exact remainder and the rounded reciprocal gives the rounded
// quotient (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990, theorem on division).  An infinity stays.
__device__ __forceinline__ float div15(float x) {
    constexpr float kInv = 1.f / 15.f;
    const float q = __fmul_rn(x, kInv);
    const float y = __fmaf_rn(__fmaf_rn(-15.f, q, x), kInv, q);
    return q == INFINITY ? q : y;
}

// 1 / s rounded to nearest, for a bf16 s whose reciprocal is a normal number: the
// approximate instruction is off by an ulp at most, and one Newton step with the
// exact remainder gives the rounded reciprocal of any s whose significand is not all
// ones (Markstein, as above); eight bits followed by zeros are not.
__device__ __forceinline__ float reciprocal(float s) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
    return __fmaf_rn(y, __fmaf_rn(-s, y, 1.f), y);
}

template <int NG, bool F32, int U>
__global__ void __launch_bounds__(kQ4Warps * 32)
q4_write_kernel(const void* __restrict__ k, const void* __restrict__ v, const Q4Rows a,
                unsigned char* __restrict__ kc, unsigned char* __restrict__ vc) {
    PKV_DEPENDENT_PROLOGUE();
    constexpr int D = NG * kQ4Group;
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * kQ4Warps + (threadIdx.x >> 5);
    if (n >= a.num_tokens) return;
    const void* src = blockIdx.y ? v : k;
    unsigned char* pool = blockIdx.y ? vc : kc;
    const int vecs = a.hkv * (D / 8);  // lanes' worth of dims in a token's row
    const int64_t e0 = n * a.hkv * D;
    Raw8<F32> raw[U];
    auto load = [&](int v0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int vec = v0 + 32 * u + lane;
            raw[u].a = make_uint4(0, 0, 0, 0);
            raw[u].b = make_uint4(0, 0, 0, 0);
            if (vec < vecs) load8<F32>(src, e0 + (int64_t)vec * 8, raw[u]);
        }
    };
    // the row before its slot is known (a row that is not written wastes the load)
    const int32_t slot = __ldg(a.slots + n);
    load(0);
    if (slot < 0) return;
    if (slot >= a.num_slots) {
        if (lane == 0) flag_error(a.err, PKV_FLAG_BAD_SLOT);
        return;
    }
    const int32_t page = (int32_t)a.block.quot((uint32_t)slot);
    const int32_t at = slot - page * (int32_t)a.block.d;
    // a lane keeps its group and chunk; each step is 8 / NG heads further
    int head, g, c;
    lane_place<NG>(lane, &head, &g, &c);
    unsigned char* row = pool + row_offset<NG>(a, page, at, head);
    const int64_t row_step = (int64_t)(8 / NG) * a.block.d * q4_row_bytes(D);
    for (int v0 = 0; v0 < vecs; v0 += 32 * U) {
        if (v0 > 0) load(v0);
#pragma unroll
        for (int u = 0; u < U; ++u, row += row_step) {
            float2 x[4];
            widen8<F32>(raw[u], x);
            float lo = min_nan(x[0].x, x[0].y), hi = max_nan(x[0].x, x[0].y);
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                lo = min_nan(lo, x[i].x, x[i].y);
                hi = max_nan(hi, x[i].x, x[i].y);
            }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
                hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
            }
            // one rounding per operation (no contraction): the codes are the format's
            uint32_t sb = pack_bf16x2(div15(__fsub_rn(hi, lo)), 0.f);
            const bool usual = sb - 0x80u < 0x7F80u - 0x80u;  // 2^-126 <= s < infinity
            if (sb < 0x80u) sb = 0;
            const float s = __uint_as_float(sb << 16);
            const uint32_t zb =
                pack_bf16x2(0.f, __fadd_rn(__fadd_rn(0.5f * lo, 0.5f * hi), 0.5f * s));
            const float z = __uint_as_float(zb);
            const float inv = usual ? reciprocal(s) : 0.f;
            // (x - z) / s lies in about -8 .. 7 unless the rounding of s and z moved
            // an end by half a step: every operation is monotonic, so the ends tell
            // for the group.  rint(-8.5) is -8 and rint(7.5) is 8.
            const bool inside = __fmul_rn(__fsub_rn(lo, z), inv) >= -8.5f &&
                                __fmul_rn(__fsub_rn(hi, z), inv) < 7.5f;
            float2 q[4];
            const float2 z2 = make_float2(-z, -z), i2 = make_float2(inv, inv);
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = fmul2(fadd2(x[i], z2), i2);
            if (!__all_sync(0xffffffffu, inside)) {  // (a NaN becomes code 0)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    q[i] = make_float2(fminf(fmaxf(q[i].x, -8.f), 7.f),
                                       fminf(fmaxf(q[i].y, -8.f), 7.f));
            }
            // rint and the conversion by an addition: 2^23 + 2^22 + 8 + t rounds t to
            // a whole number, ties to even, and leaves code t + 8 in the low bits
            // (clamping to -8 .. 7 before it changes no code).  The bits above the
            // codes add up to a constant.
            uint32_t w = 0u - 0x4B400000u * 0x11111111u;
            const float2 magic = make_float2(12582920.f, 12582920.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                q[i] = fadd2(q[i], magic);
                w += (__float_as_uint(q[i].x) << (8 * i)) + (__float_as_uint(q[i].y) << (8 * i + 4));
            }
            w = units_to_words<NG>(w, lane, g);
            if (v0 + 32 * u + lane < vecs) {
                *reinterpret_cast<uint32_t*>(row + c * (4 * NG) + g * 4) = w;
                if (c == 0) *reinterpret_cast<uint32_t*>(row + D / 2 + g * 4) = sb | zb;
            }
        }
    }
}

template <int NG, bool F32, int U>
__global__ void __launch_bounds__(kQ4Warps * 32)
q4_read_kernel(const unsigned char* __restrict__ kc, const unsigned char* __restrict__ vc,
               const Q4Rows a, void* __restrict__ k, void* __restrict__ v) {
    PKV_DEPENDENT_PROLOGUE();
    constexpr int D = NG * kQ4Group;
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * kQ4Warps + (threadIdx.x >> 5);
    if (n >= a.num_tokens) return;
    const unsigned char* pool = blockIdx.y ? vc : kc;
    void* dst = blockIdx.y ? v : k;
    const int vecs = a.hkv * (D / 8);
    const int64_t e0 = n * a.hkv * D;
    const int32_t slot = __ldg(a.slots + n);
    const bool real = slot >= 0 && slot < a.num_slots;
    if (slot >= a.num_slots && lane == 0) flag_error(a.err, PKV_FLAG_BAD_SLOT);
    const int32_t page = real ? (int32_t)a.block.quot((uint32_t)slot) : 0;
    const int32_t at = real ? slot - page * (int32_t)a.block.d : 0;
    for (int v0 = 0; v0 < vecs; v0 += 32 * U) {
        uint32_t words[U], sz[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int vec = v0 + 32 * u + lane;
            words[u] = sz[u] = 0;
            if (vec < vecs && real) {
                int head, g, c;
                lane_place<NG>(vec, &head, &g, &c);
                const unsigned char* row = pool + row_offset<NG>(a, page, at, head);
                words[u] = *reinterpret_cast<const uint32_t*>(row + c * (4 * NG) + g * 4);
                sz[u] = *reinterpret_cast<const uint32_t*>(row + D / 2 + g * 4);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int vec = v0 + 32 * u + lane;
            const uint32_t w = words_to_units<NG>(words[u], lane, (vec / 4) % NG);
            if (vec >= vecs) continue;
            const int64_t e = e0 + (int64_t)vec * 8;
            // one fused multiply and add of the output's own type: one rounding
            if constexpr (F32) {
                const float s = bf16lo(sz[u]), z = bf16hi(sz[u]);
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] = fmaf((float)((w >> (4 * i)) & 15u) - 8.f, s, z);
                float4* o = reinterpret_cast<float4*>(static_cast<float*>(dst) + e);
                o[0] = make_float4(x[0], x[1], x[2], x[3]);
                o[1] = make_float4(x[4], x[5], x[6], x[7]);
            } else {
                const uint32_t ss = __byte_perm(sz[u], 0u, 0x1010), zz = __byte_perm(sz[u], 0u, 0x3232);
                uint32_t x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // bf16 128 + u of the byte's two codes, minus 136
                    const uint32_t y = w >> (8 * i);
                    x[i] = (y & 0xFu) | ((y << 12) & 0xF0000u) | 0x43004300u;
                    asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(x[i]) : "r"(0x43084308u));
                    asm("fma.rn.bf16x2 %0, %0, %1, %2;" : "+r"(x[i]) : "r"(ss), "r"(zz));
                }
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + e) =
                    make_uint4(x[0], x[1], x[2], x[3]);
            }
        }
    }
}

// the kernel `name` for a head dim, row type and 32-lane steps in flight per warp
// (as many as a row has, up to 4: 17,928 rows written and read 36.0 us with four, 37.3 with
// two, 41.7 with one)
#define PKV_Q4_KERNEL(name, d, f32, vecs)                                               \
    ((d) == 128 ? ((f32) ? PKV_Q4_STEPS(name, 4, true, vecs) : PKV_Q4_STEPS(name, 4, false, vecs)) \
                : ((f32) ? PKV_Q4_STEPS(name, 2, true, vecs) : PKV_Q4_STEPS(name, 2, false, vecs)))
#define PKV_Q4_STEPS(name, ng, f32, vecs) \
    ((vecs) <= 32 ? name<ng, f32, 1> : ((vecs) <= 64 ? name<ng, f32, 2> : name<ng, f32, 4>))

}  // namespace

cudaError_t launch_q4_write(const void* k, const void* v, int src_dtype, const int32_t* slots,
                            int64_t num_tokens, void* k_cache, void* v_cache, int hkv, int d,
                            int block_size, int64_t num_slots, unsigned int* err,
                            cudaStream_t stream) {
    if (num_tokens == 0) return cudaSuccess;
    const Q4Rows a{slots, num_tokens, num_slots, FastDiv((uint32_t)block_size), hkv, err};
    const dim3 grid((unsigned)((num_tokens + kQ4Warps - 1) / kQ4Warps), 2);
    const bool f32 = src_dtype == PKV_F32;
    auto kern = PKV_Q4_KERNEL(q4_write_kernel, d, f32, hkv * (d / 8));
    return launch_dependent(kern, grid, dim3(kQ4Warps * 32), 0, stream, k, v, a,
                            static_cast<unsigned char*>(k_cache),
                            static_cast<unsigned char*>(v_cache));
}

cudaError_t launch_q4_read(const void* k_cache, const void* v_cache, const int32_t* slots,
                           int64_t num_tokens, void* k, void* v, int dst_dtype, int hkv, int d,
                           int block_size, int64_t num_slots, unsigned int* err,
                           cudaStream_t stream) {
    if (num_tokens == 0) return cudaSuccess;
    const Q4Rows a{slots, num_tokens, num_slots, FastDiv((uint32_t)block_size), hkv, err};
    const dim3 grid((unsigned)((num_tokens + kQ4Warps - 1) / kQ4Warps), 2);
    const bool f32 = dst_dtype == PKV_F32;
    auto kern = PKV_Q4_KERNEL(q4_read_kernel, d, f32, hkv * (d / 8));
    return launch_dependent(kern, grid, dim3(kQ4Warps * 32), 0, stream,
                            static_cast<const unsigned char*>(k_cache),
                            static_cast<const unsigned char*>(v_cache), a, k, v);
}

}  // namespace pkv
