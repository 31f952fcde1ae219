// compact.cu -- compaction of cached tokens within their sequences' pages.
//
// For sequence b with keep list p_0, p_1, .., p_{n-1} (positions, p_i >= start + i:
// any ascending list), the K and V rows of position p_i move to position start +
// i, in place ("11. Paged attention 与 online softmax" §11.1 addressing; the
// pages behind the new end are free afterwards).  Used after tokens were
// evicted, or to keep the accepted path of a draft tree.
//
// In place without a second buffer: once the rows 0 .. i have been LOADED,
// writing destinations up to start + i cannot hit a source that is still to be
// read, because p_j >= start + j > start + i for j > i.  Tokens of a sequence therefore
// only need the order "a round's loads before its stores", and bytes of different
// columns of a row need no order at all: the rows are cut into column slices
// and one CTA walks one sequence's tokens for one slice of one pool, in rounds.
// Within a round all loads come before a barrier and all stores after it; the
// next round's loads are issued before this round's stores, so that they are
// in flight together.  No flags, no waits between CTAs, and the result does
// not depend on the order in which they run.
// HBM-bound: each moved row is read and written once; rows that stay where they
// are (p_i = start + i) are neither read nor written.
#include <algorithm>

#include "common.cuh"
#include "launch.h"

namespace pkv {

namespace {

constexpr int kCompactThreads = 256;
constexpr int kCompactUnroll = 4;  // rows in flight per thread and round

struct CompactArgs {
    unsigned char* pool[2];
    const int32_t* table;
    const int32_t* start;   // [batch] or null (0)
    const int32_t* keep;    // [total]
    const int32_t* cu;      // [batch + 1]
    int32_t* seqlens_out;   // [batch] or null
    unsigned int* err;
    int64_t page_bytes, token_bytes, head_bytes;  // strides of page, token, head
    int64_t num_blocks;
    int32_t max_blocks, block_size, total;
    int32_t vec_per_head;   // vectors that lie together; a token's row has `vecs` of them
    int32_t vecs;
    int32_t slice;          // vectors per slice
};

// one kept token of a round: byte offsets in the pool, -1 when nothing moves
struct Move {
    int64_t src, dst;
};

__device__ __forceinline__ Move find_move(const CompactArgs& a, const int32_t* row,
                                          const int32_t* list, int32_t i, int32_t n,
                                          int32_t start, bool report) {
    Move m{-1, -1};
    if (i >= n) return m;
    const int32_t p = list[i], to = start + i;
    if (p == to) return m;  // stays
    if (p < to || p >= (int64_t)a.max_blocks * a.block_size) {
        if (report) flag_error(a.err, PKV_FLAG_BAD_LENGTH);
        return m;
    }
    const int32_t sp = p / a.block_size, dp = to / a.block_size;
    const int32_t sb = row[sp], db = row[dp];
    if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks) {
        if (report) flag_error(a.err, PKV_FLAG_BAD_BLOCK);
        return m;
    }
    m.src = sb * a.page_bytes + (p - sp * a.block_size) * a.token_bytes;
    m.dst = db * a.page_bytes + (to - dp * a.block_size) * a.token_bytes;
    return m;
}

// grid (slices, batch, 2 pools)
template <typename Vec>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactArgs a) {
    PKV_DEPENDENT_PROLOGUE();
    const int b = blockIdx.y;
    const int32_t c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1);
    int32_t start = a.start ? __ldg(a.start + b) : 0;
    const bool first = blockIdx.x == 0 && blockIdx.z == 0;
    int32_t n = c1 - c0;
    if (c0 < 0 || c1 < c0 || c1 > a.total || start < 0 ||
        (int64_t)start + n > (int64_t)a.max_blocks * a.block_size) {
        if (first && threadIdx.x == 0) flag_error(a.err, PKV_FLAG_BAD_LENGTH);
        start = min(max(start, 0), a.max_blocks * a.block_size);
        n = 0;
    }
    if (first && threadIdx.x == 0 && a.seqlens_out) a.seqlens_out[b] = start + n;
    if (n == 0) return;
    const int32_t* list = a.keep + c0;
    const int32_t* row = a.table + (int64_t)b * a.max_blocks;
    unsigned char* pool = a.pool[blockIdx.z];
    // this thread's column of the slice and its first token of a round
    const int tokens = kCompactThreads / a.slice;  // tokens side by side
    const int tok = threadIdx.x / a.slice;
    const int32_t col = blockIdx.x * a.slice + threadIdx.x % a.slice;
    const bool live = tok < tokens && col < a.vecs;
    const int64_t off = live ? (int64_t)(col / a.vec_per_head) * a.head_bytes +
                                   (int64_t)(col % a.vec_per_head) * sizeof(Vec)
                             : 0;
    const int32_t step = tokens * kCompactUnroll;
    int64_t dst[kCompactUnroll], dst_next[kCompactUnroll];
    Vec x[kCompactUnroll], x_next[kCompactUnroll];
    auto load = [&](int32_t i0, int64_t* d, Vec* v) {
#pragma unroll
        for (int u = 0; u < kCompactUnroll; ++u) {
            d[u] = -1;
            if (!live) continue;
            const Move m = find_move(a, row, list, i0 + u * tokens + tok, n, start, first);
            if (m.src < 0) continue;
            d[u] = m.dst + off;
            v[u] = __ldcg(reinterpret_cast<const Vec*>(pool + m.src + off));
        }
    };
    load(0, dst, x);
    for (int32_t i0 = 0; i0 < n; i0 += step) {
        __syncthreads();  // every thread has read its rows of this round
        load(i0 + step, dst_next, x_next);
#pragma unroll
        for (int u = 0; u < kCompactUnroll; ++u) {
            if (dst[u] >= 0) *reinterpret_cast<Vec*>(pool + dst[u]) = x[u];
            dst[u] = dst_next[u];
            x[u] = x_next[u];
        }
    }
}

}  // namespace

cudaError_t launch_compact(const CompactLaunch& c, unsigned int* err, cudaStream_t stream) {
    CompactArgs a{};
    a.pool[0] = static_cast<unsigned char*>(c.k_cache);
    a.pool[1] = static_cast<unsigned char*>(c.v_cache);
    a.table = c.table;
    a.start = c.start;
    a.keep = c.keep;
    a.cu = c.cu_keep;
    a.seqlens_out = c.seqlens_out;
    a.err = err;
    a.page_bytes = c.page_bytes;
    a.token_bytes = c.token_bytes;
    a.head_bytes = c.head_bytes;
    a.num_blocks = c.num_blocks;
    a.max_blocks = c.max_blocks;
    a.block_size = c.block_size;
    a.total = c.total;
    // the widest vector that divides the pieces and the pools' alignment
    int vec = 16;
    while (vec > 2 && (c.piece_bytes % vec || !aligned(c.k_cache, vec) || !aligned(c.v_cache, vec)))
        vec /= 2;
    a.vec_per_head = (int32_t)(c.piece_bytes / vec);
    a.vecs = (int32_t)(a.vec_per_head * c.pieces);
    a.slice = std::min(a.vecs, 4);
    const dim3 grid((unsigned)((a.vecs + a.slice - 1) / a.slice), (unsigned)c.batch, 2);
    auto kern = vec == 16 ? compact_kernel<uint4>
                          : (vec == 8 ? compact_kernel<uint2>
                                      : (vec == 4 ? compact_kernel<uint32_t>
                                                  : compact_kernel<uint16_t>));
    return launch_dependent(kern, grid, dim3(kCompactThreads), 0, stream, a);
}

}  // namespace pkv
