// rope.cuh -- the position rotation of a token's heads, as the write kernels apply it
// on the way into the cache and to the queries beside them.
//
// Row p of the table cos_sin [positions, rot] holds rot / 2 cosines c, then rot / 2
// sines s.  Dims (i, i + rot / 2) of a head, or (2i, 2i + 1) interleaved, become
//   x_a c_i - x_b s_i,   x_b c_i + x_a s_i     i < rot / 2;
// dims from rot on stay.  Every product and sum is rounded to fp32 by itself (no
// fused ones): the bits of a rotated row, and 8-bit codes made of it, are then those
// of any other program that computes the two products and the sum.
//
// A lane takes one unit of a head: two chunks of 8 dims that rotate with one another,
// chunks u and u + rot / 16 (interleaved: 2u and 2u + 1) for unit u < rot / 16, and
// two neighbouring ones of those behind rot.  Both forms then meet the cosines and
// sines 8u .. 8u + 7, and D / 16 lanes hold a head: no exchange between lanes, and a
// lane that keeps its unit from head to head loads them once per token.
#pragma once

#include "common.cuh"
#include "divide.cuh"

namespace pkv {

struct RopeTable {
    const float* cos_sin;   // [positions, rot], 16-byte aligned
    int32_t positions, rot;  // rot a multiple of 16; 0: no rotation
};

// the new tokens of a write call
struct NewTokens {
    const int32_t* seq;       // [num]; below 0: a padding row
    const int32_t* pos;       // [num]
    const int32_t* rope_pos;  // [num]
    const int32_t* table;     // [num_seqs, max_blocks]
    int64_t num, num_blocks;
    FastDiv block;            // by the page size
    int32_t num_seqs, max_blocks, hkv;
};

// Is there a row for a token at position p of sequence s, rotated by position rp?
// What is wrong is flagged (err may be null); a padding row is nothing wrong.
__device__ __forceinline__ bool token_ok(const NewTokens& t, const RopeTable& r, int32_t s,
                                         int32_t p, int32_t rp, unsigned int* err) {
    if (s < 0) return false;
    if (s >= t.num_seqs) {
        flag_error(err, PKV_FLAG_BAD_SEQ);
        return false;
    }
    if (p < 0 || (int32_t)t.block.quot((uint32_t)p) >= t.max_blocks ||
        (r.rot && (rp < 0 || rp >= r.positions))) {
        flag_error(err, PKV_FLAG_BAD_LENGTH);
        return false;
    }
    return true;
}

// the page of position p of sequence s, below 0 (flagged) if it is not in the pool
__device__ __forceinline__ int32_t token_page(const NewTokens& t, int32_t s, int32_t p,
                                              unsigned int* err) {
    const int32_t id = __ldg(t.table + (int64_t)s * t.max_blocks + t.block.quot((uint32_t)p));
    if (id >= 0 && id < t.num_blocks) return id;
    flag_error(err, PKV_FLAG_BAD_BLOCK);
    return -1;
}

template <bool F32>
struct RawUnit {
    uint4 a[F32 ? 2 : 1], b[F32 ? 2 : 1];  // chunks a and b
};

// first dims of a unit's two chunks
template <bool MIX>
__device__ __forceinline__ void unit_dims(int u, int rot, int* a, int* b) {
    const int h = rot >> 4;
    if (MIX || u >= h) {  // (unit u >= h: chunks 2h + 2(u - h) and the next)
        *a = 16 * u;
        *b = 16 * u + 8;
    } else {
        *a = 8 * u;
        *b = 8 * (u + h);
    }
}

template <bool F32>
__device__ __forceinline__ void load_unit(const void* head, int a, int b, RawUnit<F32>& x) {
    if constexpr (F32) {
        const float* p = static_cast<const float*>(head);
        x.a[0] = __ldcs(reinterpret_cast<const uint4*>(p + a));
        x.a[1] = __ldcs(reinterpret_cast<const uint4*>(p + a) + 1);
        x.b[0] = __ldcs(reinterpret_cast<const uint4*>(p + b));
        x.b[1] = __ldcs(reinterpret_cast<const uint4*>(p + b) + 1);
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(head);
        x.a[0] = __ldcs(reinterpret_cast<const uint4*>(p + a));
        x.b[0] = __ldcs(reinterpret_cast<const uint4*>(p + b));
    }
}

// x[0..7]: chunk a, x[8..15]: chunk b
template <bool F32>
__device__ __forceinline__ void widen_unit(const RawUnit<F32>& r, float* x) {
    if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[4 * i] = __uint_as_float(r.a[i].x);
            x[4 * i + 1] = __uint_as_float(r.a[i].y);
            x[4 * i + 2] = __uint_as_float(r.a[i].z);
            x[4 * i + 3] = __uint_as_float(r.a[i].w);
            x[8 + 4 * i] = __uint_as_float(r.b[i].x);
            x[8 + 4 * i + 1] = __uint_as_float(r.b[i].y);
            x[8 + 4 * i + 2] = __uint_as_float(r.b[i].z);
            x[8 + 4 * i + 3] = __uint_as_float(r.b[i].w);
        }
    } else {
        const uint32_t w[8] = {r.a[0].x, r.a[0].y, r.a[0].z, r.a[0].w,
                               r.b[0].x, r.b[0].y, r.b[0].z, r.b[0].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[2 * i] = bf16lo(w[i]);
            x[2 * i + 1] = bf16hi(w[i]);
        }
    }
}

struct UnitAngles {
    float c[8], s[8];
};

// of unit u < rot / 16 at a position inside the table
__device__ __forceinline__ void load_angles(const RopeTable& t, int32_t pos, int u,
                                            UnitAngles& y) {
    const float4* p = reinterpret_cast<const float4*>(t.cos_sin + (int64_t)pos * t.rot + 8 * u);
    const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + t.rot / 2);
    const float4 c0 = __ldg(p), c1 = __ldg(p + 1), s0 = __ldg(q), s1 = __ldg(q + 1);
    y.c[0] = c0.x; y.c[1] = c0.y; y.c[2] = c0.z; y.c[3] = c0.w;
    y.c[4] = c1.x; y.c[5] = c1.y; y.c[6] = c1.z; y.c[7] = c1.w;
    y.s[0] = s0.x; y.s[1] = s0.y; y.s[2] = s0.z; y.s[3] = s0.w;
    y.s[4] = s1.x; y.s[5] = s1.y; y.s[6] = s1.z; y.s[7] = s1.w;
}

// (Packed f32x2 products and sums would halve the instructions, but sums of packed products
// are compiled to fused ones, whatever rounding they ask for.)
template <bool MIX>
__device__ __forceinline__ void rotate_unit(float* x, const UnitAngles& t) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float& a = x[MIX ? 2 * i : i];
        float& b = x[MIX ? 2 * i + 1 : 8 + i];
        const float ra = __fsub_rn(__fmul_rn(a, t.c[i]), __fmul_rn(b, t.s[i]));
        b = __fadd_rn(__fmul_rn(b, t.c[i]), __fmul_rn(a, t.s[i]));
        a = ra;
    }
}

template <bool F32>
__device__ __forceinline__ void store_chunk(void* head, int dim, const float* x) {
    if constexpr (F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(head) + dim);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(head) + dim) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                       pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
}

// ---- the queries of a write call -------------------------------------------------
// Row n of q (fp32 or bf16 like the new rows) goes to q_out rotated, or as it is
// when the token is a padding row or its position lies outside the table.
struct RopeQuery {
    const void* q;
    void* out;
    int64_t stride, out_stride;  // elements from token to token
    int32_t heads;
    int32_t warps;               // per token
};

constexpr int kUnitRounds = 4;  // units a lane has in flight (fp32: half as many)
template <bool F32>
__host__ __device__ constexpr int unit_rounds() { return F32 ? kUnitRounds / 2 : kUnitRounds; }
// warps that take the `heads` heads of a token
template <bool F32>
__host__ __device__ constexpr int64_t unit_warps(int64_t heads, int d) {
    const int64_t per = 32 * unit_rounds<F32>();
    return (heads * (d / 16) + per - 1) / per;
}

// the w-th warp's units of a row of heads, loaded in `raw`, to the row at `dst`
template <int D, bool F32, bool OUT_F32, bool MIX>
__device__ __forceinline__ void move_units(void* dst, int heads, int w, int lane, bool turn,
                                           int rot, const RawUnit<F32>* raw,
                                           const UnitAngles& ang) {
    constexpr int U = D / 16, R = unit_rounds<F32>();
    const int u = lane % U;
    int a, b;
    unit_dims<MIX>(u, rot, &a, &b);
    const bool spin = turn && u < (rot >> 4);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int h = (w * R + i) * (32 / U) + lane / U;
        if (h >= heads) continue;
        float x[16];
        widen_unit<F32>(raw[i], x);
        if (spin) rotate_unit<MIX>(x, ang);
        void* head = static_cast<unsigned char*>(dst) + (int64_t)h * D * (OUT_F32 ? 4 : 2);
        store_chunk<OUT_F32>(head, a, x);
        store_chunk<OUT_F32>(head, b, x + 8);
    }
}
template <int D, bool F32, bool MIX>
__device__ __forceinline__ void load_units(const void* src, int heads, int w, int lane, int rot,
                                           RawUnit<F32>* raw) {
    constexpr int U = D / 16, R = unit_rounds<F32>();
    int a, b;
    unit_dims<MIX>(lane % U, rot, &a, &b);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int h = (w * R + i) * (32 / U) + lane / U;
        if (h < heads)
            load_unit<F32>(static_cast<const unsigned char*>(src) + (int64_t)h * D * (F32 ? 4 : 2),
                           a, b, raw[i]);
    }
}

// warp `w` of token n's queries; seq[n] < 0 marks a padding row
template <int D, bool F32, bool MIX>
__device__ __forceinline__ void query_warp(const RopeQuery& q, const RopeTable& t,
                                           const int32_t* seq, const int32_t* rope_pos, int64_t n,
                                           int w, int lane) {
    constexpr int U = D / 16, R = unit_rounds<F32>();
    const unsigned char* src = static_cast<const unsigned char*>(q.q) + n * q.stride * (F32 ? 4 : 2);
    unsigned char* dst = static_cast<unsigned char*>(q.out) + n * q.out_stride * (F32 ? 4 : 2);
    RawUnit<F32> raw[R];
    load_units<D, F32, MIX>(src, q.heads, w, lane, t.rot, raw);
    const int32_t p = __ldg(rope_pos + n);
    const bool turn = __ldg(seq + n) >= 0 && p >= 0 && p < t.positions;
    UnitAngles ang;
    if (turn && lane % U < (t.rot >> 4)) load_angles(t, p, lane % U, ang);
    move_units<D, F32, F32, MIX>(dst, q.heads, w, lane, turn, t.rot, raw, ang);
}

}  // namespace pkv
