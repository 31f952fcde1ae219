// q4_decode.cu -- paged decode (one query token per sequence) over a 4-bit cache.
//
//   out[b,h] = sum_j softmax_j(scale * q[b,h] . k_j) v_j,  j < cache_seqlens[b],
// with k_j, v_j the values of the 4-bit rows (format: q4.cuh), read through block
// table row b, merged by the online-softmax rule.
//
// One CTA per (sequence, query head); its warps take every fourth key and
// merge their states at the end.
#include "common.cuh"
#include "launch.h"
#include "q4.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 4;

struct Q4DecodeArgs {
    const void* q;
    const unsigned char* kc;
    const unsigned char* vc;
    const int32_t* table;
    const int32_t* seqlens;
    void* out;
    unsigned int* err;
    int64_t num_blocks;
    float qscale;  // scale * log2(e)
    int32_t max_blocks, hq, hkv, block_size;
};

template <int NG, bool F32>
__global__ void __launch_bounds__(kWarps * 32) q4_decode_kernel(const Q4DecodeArgs a) {
    PKV_DEPENDENT_PROLOGUE();
    constexpr int D = NG * kQ4Group, R = q4_row_bytes(D), UNITS = 8 * NG;
    __shared__ float so[kWarps][D], sm[kWarps], sl[kWarps];
    const int b = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kvh = h / (a.hq / a.hkv);
    const int64_t cap = (int64_t)a.max_blocks * a.block_size;
    int32_t L = a.seqlens[b];
    if (L < 0 || L > cap) {
        if (h == 0 && threadIdx.x == 0) flag_error(a.err, PKV_FLAG_BAD_LENGTH);
        L = L < 0 ? 0 : (int32_t)cap;
    }
    const int unit = lane < UNITS ? lane : 0;  // this lane's 4 dims
    const int g = unit % NG, dim = g * kQ4Group + 4 * (unit / NG);
    const int64_t qi = ((int64_t)b * a.hq + h) * D + dim;
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
    for (int i = 0; i < 4; ++i) {
        q[i] = F32 ? static_cast<const float*>(a.q)[qi + i]
                   : bf16lo(static_cast<const uint16_t*>(a.q)[qi + i]);
        q[i] = lane < UNITS ? q[i] * a.qscale : 0.f;
    }
    for (int32_t j = warp; j < L; j += kWarps) {
        const int32_t page = a.table[(int64_t)b * a.max_blocks + j / a.block_size];
        if (page < 0 || page >= a.num_blocks) {
            if (lane == 0) flag_error(a.err, PKV_FLAG_BAD_BLOCK);
            continue;
        }
        const int64_t row = (((int64_t)page * a.hkv + kvh) * a.block_size + j % a.block_size) * R;
        const uint16_t ku = *reinterpret_cast<const uint16_t*>(a.kc + row + 2 * unit);
        const uint32_t ks = *reinterpret_cast<const uint32_t*>(a.kc + row + D / 2 + 4 * g);
        const uint16_t vu = *reinterpret_cast<const uint16_t*>(a.vc + row + 2 * unit);
        const uint32_t vs = *reinterpret_cast<const uint32_t*>(a.vc + row + D / 2 + 4 * g);
        float s = 0.f;
        for (int i = 0; i < 4; ++i)
            s += q[i] * fmaf((float)((ku >> (4 * i)) & 15) - 8.f, bf16lo(ks), bf16hi(ks));
        if (lane >= UNITS) s = 0.f;
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        const float mn = fmaxf(m, s);
        const float c = m == -INFINITY ? 0.f : ex2(m - mn);
        const float p = s == -INFINITY ? 0.f : ex2(s - mn);  // a NaN score stays one
        l = l * c + p;
        for (int i = 0; i < 4; ++i)
            o[i] = o[i] * c +
                   p * fmaf((float)((vu >> (4 * i)) & 15) - 8.f, bf16lo(vs), bf16hi(vs));
        m = mn;
    }
    if (lane < UNITS)
        for (int i = 0; i < 4; ++i) so[warp][dim + i] = o[i];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
    for (int i = threadIdx.x; i < D; i += kWarps * 32) {
        float L1 = 0.f, acc = 0.f;
        for (int w = 0; w < kWarps; ++w) {
            const float c = sm[w] == -INFINITY ? 0.f : ex2(sm[w] - M);
            L1 += sl[w] * c;
            acc += so[w][i] * c;
        }
        acc = L1 == 0.f ? 0.f : acc / L1;
        const int64_t oi = ((int64_t)b * a.hq + h) * D + i;
        if (F32) static_cast<float*>(a.out)[oi] = acc;
        else static_cast<uint16_t*>(a.out)[oi] = f32_to_bf16_bits(acc);
    }
}

}  // namespace

bool plan_q4_decode(const DeviceInfo& dev, int32_t batch, int hq, int hkv, int d, int block_size,
                    int q_dtype, Q4DecodePlan* plan) {
    plan->ws_bytes = 0;
    return (d == 64 || d == 128) && batch <= kDecodeMaxBatch && hq <= 65535;
}

cudaError_t launch_q4_decode(const Q4DecodePlan& plan, const void* q, const void* k_cache,
                             const void* v_cache, const int32_t* table, int32_t max_blocks,
                             const int32_t* seqlens, int32_t batch, float scale, void* out,
                             void* workspace, int hq, int hkv, int d, int block_size,
                             int64_t num_blocks, int q_dtype, unsigned int* err,
                             cudaStream_t stream) {
    if (batch == 0) return cudaSuccess;
    const Q4DecodeArgs a{q, static_cast<const unsigned char*>(k_cache),
                         static_cast<const unsigned char*>(v_cache), table, seqlens, out, err,
                         num_blocks, scale * 1.4426950408889634f, max_blocks, hq, hkv, block_size};
    const bool f32 = q_dtype == PKV_F32;
    auto kern = d == 128 ? (f32 ? q4_decode_kernel<4, true> : q4_decode_kernel<4, false>)
                         : (f32 ? q4_decode_kernel<2, true> : q4_decode_kernel<2, false>);
    return launch_dependent(kern, dim3((unsigned)batch, (unsigned)hq), dim3(kWarps * 32), 0, stream,
                            a);
}

}  // namespace pkv
