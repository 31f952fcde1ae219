// split.cuh -- what the decode kernels over quantised pools share: the shares that
// the tiles of all sequences are cut into, warp-wide waits, tensor-core products from
// registers, and the kernel that merges the partial states of a split.
#pragma once

#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace pkv {

namespace {

// ---- the split's shares: tile t of sequence b sits at t + b + 1 on a line (a
// sequence's start counts as one tile) that is cut into equal parts
__device__ __forceinline__ int32_t share_len(int32_t total, int32_t batch, int ctas) {
    return max(1, (total + batch + ctas - 1) / ctas);
}
__device__ __forceinline__ int32_t share_first(const int32_t* tstart, int batch, int64_t x) {
    int lo = 0, hi = batch;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)tstart[mid + 1] + mid >= x) hi = mid; else lo = mid + 1;
    }
    if (lo >= batch) return tstart[batch];
    return (int32_t)max((int64_t)tstart[lo], x - lo - 1);
}

// the sequence of tile t
__device__ __forceinline__ int share_seq(const int32_t* tstart, int batch, int32_t t) {
    int lo = 0, hi = batch;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (tstart[mid + 1] <= t) lo = mid + 1; else hi = mid;
    }
    return lo;
}

__host__ __device__ constexpr size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }

__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}


__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
// a and b rounded to fp16; what was rounded off stays in them (REST)
template <bool REST>
__device__ __forceinline__ uint32_t take_f16x2(float& a, float& b) {
    const uint32_t y = pack_f16x2(a, b);
    if constexpr (REST) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y));
        a -= f.x;
        b -= f.y;
    }
    return y;
}

// ---- barriers by 32-bit shared address (computed once per warp)
__device__ __forceinline__ bool try_phase(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __noinline__ bool wait_phase_slow(uint32_t bar, uint32_t parity, unsigned int* err) {
    const uint64_t t0 = global_ns();
    while (!__all_sync(0xffffffffu, try_phase(bar, parity))) {
        if (global_ns() - t0 > kWaitLimitNs) {
            flag_error(err, PKV_FLAG_TIMEOUT);
            return false;
        }
    }
    return true;
}
// the whole warp waits for a phase; false (flagged) if it does not end in time
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, unsigned int* err) {
    if (__all_sync(0xffffffffu, try_phase(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_phase_slow(bar, parity, err));
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ---- combine ---------------------------------------------------------------------
// Merges the partial states of a (sequence, query head) and normalises.  W warps
// share one, each with every W-th piece, up to 8 in flight: a batch of one has as
// many pieces as CTAs, and 19 rounds of one warp took 15 us of a 21 us call.
struct SplitCombineArgs {
    const float* part_o;
    const float* part_ml;
    const int32_t* tstart;
    void* out;
    int32_t batch, hq, ctas;
    int32_t w;  // warps per (sequence, query head)
};
constexpr int kCombineWarps = 4;  // at least, per CTA
constexpr int kCombineLoads = 8;  // partial states in flight per warp
constexpr int kCombineMost = 16;  // warps of one (sequence, query head)

// the state (mo, lo, x) joins (M, L, acc)
template <int E>
__device__ __forceinline__ void join(float& M, float& L, float* acc, float mo, float lo,
                                     const float* x) {
    if (mo == -INFINITY) return;  // holds nothing
    const float mn = fmaxf(M, mo);
    const float ca = M == -INFINITY ? 0.f : ex2(M - mn), cb = ex2(mo - mn);
    L = L * ca + lo * cb;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * ca + x[e] * cb;
    M = mn;
}

template <int D, bool F32>
__global__ void __launch_bounds__(kCombineMost * 32) split_combine_kernel(const SplitCombineArgs a) {
    constexpr int E = D / 32;
    __shared__ float part[kCombineMost][32 * E + 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_cta = (blockDim.x >> 5) / a.w;  // (sequence, query head)s per CTA: 1 if w > 1
    const int rank = warp % a.w;
    const int64_t id = (int64_t)blockIdx.x * per_cta + warp / a.w;
    const bool live = id < (int64_t)a.batch * a.hq;
    const int b = live ? (int)(id / a.hq) : 0, h = live ? (int)(id % a.hq) : 0;
    // everything that the split stores is visible behind this wait only, its tile starts too
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int32_t ta = __ldcg(a.tstart + b), tb = __ldcg(a.tstart + b + 1);
    const int32_t len = share_len(__ldcg(a.tstart + a.batch), a.batch, a.ctas);
    const int c0 = (ta + b + 1) / len, c1 = tb > ta && live ? (tb + b) / len : c0 - 1;
    float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int base = c0 + rank; base <= c1; base += kCombineLoads * a.w) {
        float2 ml[kCombineLoads];
        float x[kCombineLoads][E];
#pragma unroll
        for (int i = 0; i < kCombineLoads; ++i) {
            const int piece = base + i * a.w;
            ml[i] = make_float2(-INFINITY, 0.f);
            if (piece <= c1) {
                const int64_t at = ((int64_t)piece + b) * a.hq + h;
                ml[i] = *reinterpret_cast<const float2*>(a.part_ml + at * 2);
                const float* p = a.part_o + at * D + lane * E;
                if constexpr (E == 4) {
                    const float4 y = *reinterpret_cast<const float4*>(p);
                    x[i][0] = y.x; x[i][1] = y.y; x[i][E - 2] = y.z; x[i][E - 1] = y.w;
                } else {
                    const float2 y = *reinterpret_cast<const float2*>(p);
                    x[i][0] = y.x; x[i][1] = y.y;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kCombineLoads; ++i) join<E>(M, L, acc, ml[i].x, ml[i].y, x[i]);
    }
    if (a.w > 1) {  // (then the CTA is one (sequence, query head))
#pragma unroll
        for (int e = 0; e < E; ++e) part[warp][e * 32 + lane] = acc[e];
        if (lane == 0) {
            part[warp][32 * E] = M;
            part[warp][32 * E + 1] = L;
        }
        __syncthreads();
        if (warp > 0) return;
        for (int w = 1; w < a.w; ++w) {
            float x[E];
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = part[w][e * 32 + lane];
            join<E>(M, L, acc, part[w][32 * E], part[w][32 * E + 1], x);
        }
    }
    if (!live) return;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int64_t at = id * D + lane * E;
    if constexpr (F32) {
        float* o = static_cast<float*>(a.out) + at;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = acc[e] * inv;
    } else {
        uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at);
#pragma unroll
        for (int e = 0; e < E; e += 2) o[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    }
}

cudaError_t launch_combine(int d, bool f32, const float* part_o, const float* part_ml,
                           const int32_t* tstart, void* out, int32_t batch, int hq, int ctas,
                           cudaStream_t stream) {
    // pieces of a sequence: about its share of the CTAs, and one at either end
    const int pieces = ctas / batch + 2;
    const int w = std::min(kCombineMost, (pieces + kCombineLoads - 1) / kCombineLoads);
    const SplitCombineArgs c{part_o, part_ml, tstart, out, batch, hq, ctas, w};
    auto kern = d == 128 ? (f32 ? split_combine_kernel<128, true> : split_combine_kernel<128, false>)
                         : (f32 ? split_combine_kernel<64, true> : split_combine_kernel<64, false>);
    const int per_cta = w > 1 ? 1 : kCombineWarps;
    const int64_t pairs = (int64_t)batch * hq;
    return launch_dependent(kern, dim3((unsigned)((pairs + per_cta - 1) / per_cta)),
                            dim3(per_cta * w * 32), 0, stream, c);
}

}  // namespace

}  // namespace pkv
