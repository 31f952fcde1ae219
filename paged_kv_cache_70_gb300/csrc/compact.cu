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
// No flags, no waits between CTAs, and the result does not depend on the order in
// which they run.
//
// HBM-bound where the sequences are many: each moved row is read and written once;
// rows that stay where they are (p_i = start + i) are neither read nor written.  A round
// is a chain of four memory latencies (list entry, table entry, row, store), so a CTA
// keeps up to six rounds of rows in flight (cp.async into shared memory, each thread
// its own vectors), the table entries of the next round and the list entries of the one
// after: 80 KB of rows per CTA and two CTAs per SM.  Nothing joins the rounds of a
// sequence but their order, which bounds few sequences: those take narrower slices and
// more tokens per round (launch_typed).
// Measured: half of the tokens of 8 contexts of 16 K - 41 K (bf16, 8 heads, d = 128,
// 970.7 MB read and written) 185.5 us, 5230 GB/s (0.77 of the measured copy rate; the longest
// sequence ends last); 64 contexts up to 4 K 98 us, 5620 GB/s; one of 41 K 48 us.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "launch.h"
#include "q4.cuh"

namespace pkv {

namespace {

constexpr int kCompactUnroll = 2;  // rows of a round per thread
// A CTA's shape: threads, rounds in flight, tokens per round at most, CTAs per SM.
// A sequence's rounds are a chain, so a sequence takes as many rounds as its list has
// tokens per round, whatever the other SMs do: few sequences take narrow slices and
// many tokens per round.
struct LongLists {
    static constexpr int kThreads = 512, kDepth = 5, kTokens = 128, kCtas = 2;
};
struct FewLists {
    static constexpr int kThreads = 512, kDepth = 5, kTokens = 256, kCtas = 2;
};
struct TwoLists {
    static constexpr int kThreads = 512, kDepth = 3, kTokens = 512, kCtas = 2;
};
struct OneList {
    static constexpr int kThreads = 512, kDepth = 6, kTokens = 512, kCtas = 1;
};
// Short lists are one round, and many small CTAs start sooner.
struct ShortLists {
    static constexpr int kThreads = 128, kDepth = 1, kTokens = 32, kCtas = 8;
};
constexpr int32_t kNone = -0x7fffffff - 1;
constexpr int kAhead = 1;          // rounds between the steps of a lookup

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
    FastDiv block;          // by the page size
    int32_t max_blocks, total;
    int32_t vec_per_head;   // vectors that lie together; a token's row has `vecs` of them
    int32_t vecs;
    int32_t slice;          // vectors per slice
    int32_t tokens;         // side by side: threads / slice
};

// one kept token: byte offsets in the pool, -1 when nothing moves
struct Move {
    int64_t src, dst;
};

template <typename Vec>
__device__ __forceinline__ void copy_async(Vec* dst, const void* src) {
    if constexpr (sizeof(Vec) == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
                     : "memory");
    } else if constexpr (sizeof(Vec) >= 4) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src),
                     "n"(sizeof(Vec) >= 4 ? sizeof(Vec) : 4)
                     : "memory");
    } else {
        *dst = __ldcg(static_cast<const Vec*>(src));  // (no such copy of 2 bytes)
    }
}

// A sequence's list and start: the number kept; nothing (flagged by `report`) and a
// start within the table where they are out of range.
__device__ __forceinline__ int32_t kept(const CompactArgs& a, int b, bool report, int32_t& c0,
                                        int32_t& start) {
    c0 = __ldg(a.cu + b);
    const int32_t c1 = __ldg(a.cu + b + 1);
    start = a.start ? a.start[b] : 0;
    const int32_t cap = a.max_blocks * (int32_t)a.block.d;
    if (c0 >= 0 && c1 >= c0 && c1 <= a.total && start >= 0 && (int64_t)start + (c1 - c0) <= cap)
        return c1 - c0;
    if (report) flag_error(a.err, PKV_FLAG_BAD_LENGTH);
    start = min(max(start, 0), cap);
    return 0;
}

// The new lengths, after every CTA has read the starts: launched only where both are
// one array (a draft's lengths, moved on in place), one thread per sequence.
__global__ void __launch_bounds__(128) compact_lengths_kernel(const CompactArgs a, int32_t batch) {
    PKV_DEPENDENT_PROLOGUE();
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= batch) return;
    int32_t c0, start;
    const int32_t n = kept(a, b, false, c0, start);
    a.seqlens_out[b] = start + n;
}

// row ring, then lookup ring
template <typename Shape>
constexpr size_t ring_bytes() {
    return (size_t)Shape::kDepth * kCompactUnroll * Shape::kThreads * 16;
}
template <typename Shape>
constexpr size_t compact_smem() {
    return ring_bytes<Shape>() + (size_t)(Shape::kDepth + 2) * Shape::kTokens * sizeof(Move);
}

// grid (slices, batch, 2 pools)
template <typename Vec, typename Shape>
__global__ void __launch_bounds__(Shape::kThreads, Shape::kCtas) compact_kernel(const CompactArgs a) {
    PKV_DEPENDENT_PROLOGUE();
    constexpr int kDepth = Shape::kDepth, kThreads = Shape::kThreads, kTokens = Shape::kTokens;
    constexpr int kIndexRing = kDepth + 2;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, b = blockIdx.y;
    const bool report = blockIdx.x == 0 && blockIdx.z == 0;
    const int32_t cap = a.max_blocks * (int32_t)a.block.d;
    int32_t c0, start;
    const int32_t n = kept(a, b, report && tid == 0, c0, start);
    if (report && tid == 0 && a.seqlens_out) a.seqlens_out[b] = start + n;
    if (n == 0) return;
    const int32_t* list = a.keep + c0;
    const int32_t* row = a.table + (int64_t)b * a.max_blocks;
    unsigned char* pool = a.pool[blockIdx.z];
    Vec* ring = reinterpret_cast<Vec*>(smem);  // [round][u][thread]
    Move* moves = reinterpret_cast<Move*>(smem + ring_bytes<Shape>());
    // this thread's column of the slice and its first token of a round
    const int tok = tid / a.slice;
    const int32_t col = blockIdx.x * a.slice + tid % a.slice;
    const bool live = tok < a.tokens && col < a.vecs;
    const int64_t off = live ? (int64_t)(col / a.vec_per_head) * a.head_bytes +
                                   (int64_t)(col % a.vec_per_head) * sizeof(Vec)
                             : 0;
    const int step = a.tokens * kCompactUnroll;  // tokens per round
    const int rounds = (n + step - 1) / step;
    const bool indexer = tid < step;  // looks up token tid of each round

    // Three steps of a token's lookup, in rounds of their own so that each load has
    // time to arrive: the list entry, the two table entries, the offsets.
    auto entry = [&](int r) {
        const uint32_t i = (uint32_t)r * step + tid;
        return indexer && i < (uint32_t)n ? __ldg(list + i) : 0;
    };
    struct Pages {
        int32_t src, dst;
    };
    auto pages = [&](int r, int32_t& p) {  // makes p kNone where nothing moves
        Pages g{-1, -1};
        const uint32_t i = (uint32_t)r * step + tid;
        const int32_t to = start + (int32_t)i;
        if (!indexer || i >= (uint32_t)n || p == to) {  // no such token, or it stays
            p = kNone;
            return g;
        }
        if (p < to || p >= cap) {
            if (report) flag_error(a.err, PKV_FLAG_BAD_LENGTH);
            p = kNone;
            return g;
        }
        g.src = __ldg(row + a.block.quot((uint32_t)p));
        g.dst = __ldg(row + a.block.quot((uint32_t)to));
        return g;
    };
    auto offsets = [&](int r, int32_t p, const Pages& g) {
        if (!indexer) return;
        Move m{-1, -1};
        if (p != kNone) {
            const int32_t to = start + r * step + tid, B = (int32_t)a.block.d;
            if (g.src < 0 || g.src >= a.num_blocks || g.dst < 0 || g.dst >= a.num_blocks) {
                if (report) flag_error(a.err, PKV_FLAG_BAD_BLOCK);
            } else {
                const int32_t sp = (int32_t)a.block.quot((uint32_t)p), dp = (int32_t)a.block.quot((uint32_t)to);
                m.src = g.src * a.page_bytes + (int64_t)(p - sp * B) * a.token_bytes;
                m.dst = g.dst * a.page_bytes + (int64_t)(to - dp * B) * a.token_bytes;
            }
        }
        moves[r % kIndexRing * kTokens + tid] = m;
    };
    auto load = [&](int r) {  // (a group is closed for every round, also past the last)
        if (live && r < rounds) {
#pragma unroll
            for (int u = 0; u < kCompactUnroll; ++u) {
                const int64_t src = moves[r % kIndexRing * kTokens + u * a.tokens + tok].src;
                if (src >= 0)
                    copy_async(&ring[(r % kDepth * kCompactUnroll + u) * kThreads + tid],
                               pool + src + off);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // rounds ahead of the row loads: a table entry is looked up kAhead rounds
    // before its offsets are formed, a list entry kAhead before that
    int32_t p[kDepth + 2 * kAhead];
    Pages g[kDepth + kAhead];
#pragma unroll
    for (int r = 0; r < kDepth + 2 * kAhead; ++r) p[r] = entry(r);
#pragma unroll
    for (int r = 0; r < kDepth + kAhead; ++r) g[r] = pages(r, p[r]);
#pragma unroll
    for (int r = 0; r < kDepth; ++r) offsets(r, p[r], g[r]);
    int32_t pn[2 * kAhead];  // list entries of rounds r + kDepth ..
    Pages gn[kAhead];        // table entries of rounds r + kDepth ..
#pragma unroll
    for (int i = 0; i < 2 * kAhead; ++i) pn[i] = p[kDepth + i];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) gn[i] = g[kDepth + i];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kDepth; ++r) load(r);
    for (int r = 0; r < rounds; ++r) {
        offsets(r + kDepth, pn[0], gn[0]);
#pragma unroll
        for (int i = 0; i + 1 < kAhead; ++i) gn[i] = gn[i + 1];
        gn[kAhead - 1] = pages(r + kDepth + kAhead, pn[kAhead]);
#pragma unroll
        for (int i = 0; i + 1 < 2 * kAhead; ++i) pn[i] = pn[i + 1];
        pn[2 * kAhead - 1] = entry(r + kDepth + 2 * kAhead);
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
        __syncthreads();  // every thread has read its rows of this round
        if (live) {
#pragma unroll
            for (int u = 0; u < kCompactUnroll; ++u) {
                const int64_t dst = moves[r % kIndexRing * kTokens + u * a.tokens + tok].dst;
                if (dst >= 0)
                    *reinterpret_cast<Vec*>(pool + dst + off) =
                        ring[(r % kDepth * kCompactUnroll + u) * kThreads + tid];
            }
        }
        load(r + kDepth);
    }
}

// vectors per slice: as many as let a round hold the mean list, up to kTokens
template <typename Shape>
int slice_of(int vecs, int64_t mean) {
    constexpr int kRow = Shape::kThreads * kCompactUnroll;
    const int want = (int)std::min<int64_t>(Shape::kTokens, std::max<int64_t>(mean, 8));
    return std::max(std::min(vecs, kRow / want), kRow / Shape::kTokens);
}

template <typename Vec, typename Shape>
cudaError_t launch_shaped(int device, int64_t mean, int32_t batch, CompactArgs& a,
                          cudaStream_t stream) {
    a.slice = slice_of<Shape>(a.vecs, mean);
    a.tokens = std::min(Shape::kThreads / a.slice, Shape::kTokens / kCompactUnroll);
    const dim3 grid((unsigned)((a.vecs + a.slice - 1) / a.slice), (unsigned)batch, 2);
    auto kern = compact_kernel<Vec, Shape>;
    static std::atomic<uint64_t> set{0};  // the shared memory limit, once per device
    if (!(set.load(std::memory_order_relaxed) & (1ull << device))) {
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)compact_smem<Shape>());
        if (e != cudaSuccess) return e;
        set.fetch_or(1ull << device, std::memory_order_relaxed);
    }
    return launch_dependent(kern, grid, dim3(Shape::kThreads), compact_smem<Shape>(), stream, a);
}

// Lists of up to 32 tokens on average take the small CTAs: the accepted tokens of 64
// drafts took 3.5 us (bf16) against 3.8 (3.0 now).  Longer ones take the most tokens per round
// whose CTAs are all resident at once, or, of 256 per round, in two turns.  Half of the
// tokens of 1, 2, 4, 5, 6 and 8 contexts of 8 K - 40 K (bf16, 8 heads, d = 128), us:
//   OneList 48, 65, - | TwoLists 69, 58, 96 | FewLists 73, 73, 88, 129, 144, 173
//   LongLists 118, 96, 125, 155, 166, 181 (64 contexts up to 4 K: 98, FewLists 113)
// Narrower vectors have fewer slices' worth of bytes, and the rule is near the best of
// the four except where many slices of a 4-bit row are just too many at once.  Rule and
// best, us, 1, 2, 4, 6, 8 long contexts and 64 shorter ones: 4-bit rows, d = 64 (8-byte
// vectors) 47, 47, 59, 75, 136, 30 and 47, 47, 47, 74, 86, 30; 4-bit rows, d = 128
// (16-byte) 55, 56, 72, 97, 136, 48 and 54, 56, 62, 95, 110, 47; rows of 84 bytes
// (4-byte) 35, 36, 30, 35, 56, 18 and 35, 35, 30, 35, 50, 18; of 42 bytes (2-byte) 53,
// 54, 45, 53, 66, 23 and the same.
// The lists' lengths are on the device, so the rule has their mean only.  Half of one
// context of 41 K among 63 empty lists takes 115 - 129 (best 85), among 639 520 (best 421),
// and one list of 2048 among 639 empty ones 113 (the others 171 and more).
template <typename Vec>
cudaError_t launch_typed(const DeviceInfo& dev, int64_t mean, int32_t batch, CompactArgs& a,
                         cudaStream_t stream) {
    if (mean <= ShortLists::kTokens)
        return launch_shaped<Vec, ShortLists>(dev.device, mean, batch, a, stream);
    auto resident = [&](auto shape, int turns) {
        using Shape = decltype(shape);
        const int slice = slice_of<Shape>(a.vecs, mean);
        return (int64_t)((a.vecs + slice - 1) / slice) * batch * 2 <=
               (int64_t)dev.num_sms * Shape::kCtas * turns;
    };
    if (resident(OneList{}, 1))
        return launch_shaped<Vec, OneList>(dev.device, mean, batch, a, stream);
    if (resident(TwoLists{}, 1))
        return launch_shaped<Vec, TwoLists>(dev.device, mean, batch, a, stream);
    if (resident(FewLists{}, 2))
        return launch_shaped<Vec, FewLists>(dev.device, mean, batch, a, stream);
    return launch_shaped<Vec, LongLists>(dev.device, mean, batch, a, stream);
}

}  // namespace

cudaError_t launch_compact(const DeviceInfo& dev, const CompactLaunch& c, cudaStream_t stream) {
    CompactArgs a{};
    a.pool[0] = static_cast<unsigned char*>(c.k_cache);
    a.pool[1] = static_cast<unsigned char*>(c.v_cache);
    a.table = c.table;
    a.start = c.start;
    a.keep = c.keep;
    a.cu = c.cu_keep;
    a.seqlens_out = c.seqlens_out;
    a.err = dev.err;
    a.page_bytes = c.page_bytes;
    a.token_bytes = c.token_bytes;
    a.head_bytes = c.head_bytes;
    a.num_blocks = c.num_blocks;
    a.block = FastDiv((uint32_t)c.block_size);
    a.max_blocks = c.max_blocks;
    a.total = c.total;
    // the widest vector that divides the pieces and the pools' alignment
    int vec = 16;
    while (vec > 2 && (c.piece_bytes % vec || !aligned(c.k_cache, vec) || !aligned(c.v_cache, vec)))
        vec /= 2;
    a.vec_per_head = (int32_t)(c.piece_bytes / vec);
    a.vecs = (int32_t)(a.vec_per_head * c.pieces);
    // the starts' own array takes the lengths once every CTA has read it
    const bool in_place = c.seqlens_out && c.seqlens_out == c.start;
    CompactArgs lengths = a;
    if (in_place) a.seqlens_out = nullptr;
    const int64_t mean = ((int64_t)c.total + c.batch - 1) / c.batch;
    cudaError_t e;
    if (vec == 16) e = launch_typed<uint4>(dev, mean, c.batch, a, stream);
    else if (vec == 8) e = launch_typed<uint2>(dev, mean, c.batch, a, stream);
    else if (vec == 4) e = launch_typed<uint32_t>(dev, mean, c.batch, a, stream);
    else e = launch_typed<uint16_t>(dev, mean, c.batch, a, stream);
    if (e != cudaSuccess || !in_place) return e;
    return launch_dependent(compact_lengths_kernel, dim3((unsigned)((c.batch + 127) / 128)),
                            dim3(128), 0, stream, lengths, c.batch);
}

}  // namespace pkv
