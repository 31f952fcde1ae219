// q4_decode.cu -- paged decode (one query token per sequence) over a 4-bit cache.
//
//   out[b,h] = sum_j softmax_j(scale * q[b,h] . k_j) v_j,  j < cache_seqlens[b],
// with k_j, v_j the values s (u - 8) + z of the 4-bit rows (format: q4.cuh), read
// through block table row b and merged by the online-softmax rule ("11. Paged
// attention 与 online softmax" §11.1-§11.2).  Per group of 32 dims
//   score:   q . k_j = sum_g s_g(j) sum_{i in g} q_i (u_ji - 8) + z_g(j) sum_{i in g} q_i
//   output:  o_i     = sum_j p_j s_g(j) (u_ji - 8) + sum_j p_j z_g(j)
// so both are products of small whole numbers with 16-bit operands, and scales and
// offsets enter once per group, key and query instead of once per value.
//
// What bounds it: 160 bytes per key and KV head at d = 128 (K and V), 3.2 times
// fewer than bf16.  At HBM's rate an SM gets a key of one head every ~7 cycles; on
// the CUDA cores one query head alone would need 8 warp instructions of FMAs per
// key plus 16 for unpacking, and the queries of a group multiply the first.  So
// the products run on the tensor cores, from registers: a lane unpacks codes
// straight into the operand fragments of mma.m16n8k16 (one or two logic operations
// per PAIR of codes, code_pair below), keys (score) or dims (output) as the 16 rows
// and queries as the 8 columns.  tcgen05 would need the unpacked operand written to
// shared or tensor memory first, four times the bytes that came in, only to multiply
// it by 2 to 8 columns.
//
//  * Columns.  A group of QN = 2, 4 or 8 query heads (the next size up from
//    Hq / Hkv; more heads: several warps) shares the 8 columns with 8 / QN groups
//    of dims: column (g, q) holds query q with zeros outside group g, so one
//    accumulator tile keeps the groups' sums apart without a product for the
//    zeros that would not have been issued anyway.  The score tile is scaled per
//    group, summed over the groups by a reduce-scatter among the 4 lanes of a row
//    and each lane takes the exponential of its own share.
//  * Offsets.  sum (u - 8) x = sum u x - 8 sum x: the score's accumulator starts at
//    -8 sum q; for the output a product of the constant -8 with the weights runs
//    beside the others, in sums of its own that are added every kHold products, so
//    that nothing large is carried through a long sum.  With fp32 queries 8 is taken
//    off the operand instead (exactly), and queries and weights enter as two fp16
//    parts (22 bits), two products each.
//  * Weights are rounded to fp16 after the V scale is multiplied in, relative to the
//    largest V scale (2^-11 at most, below the 2^-8 of the bf16 output).  That scale is
//    a reference of the codes' sums alone: the weights themselves, their sum and the
//    offsets' sum p z are fp32 and relative to the maximum score only, so that neither
//    scales of 0 nor scales far apart reach them.
//  * Both references lag.  State and output are rescaled only when a score or a
//    V scale exceeds its reference by more than grow_by() or scale_grow() (one vote
//    per tile).
//  * Work split: the tiles of all sequences in one list, cut into equal contiguous
//    shares, one per CTA; each (CTA, sequence) piece leaves a partial state that a
//    second kernel merges.  Four producer warps bring tiles of K and V into a ring of
//    stages, one bulk copy per page piece and head; the other 12 (8 queries: 8) own
//    a (head, queries) and a share of the tile's keys each, and hold a stage for their
//    loads only.
//  * Keys of a page outside the pool are skipped and flagged; rows past the length
//    never enter: their scales count as 0 and their scores as -inf, whatever the
//    page holds there.  Every wait is time-limited.
//
// Measured (bf16 queries, device time of split and combine; of the measured copy rate):
//   8 sequences of 16 K - 41 K keys, 16 / 8 heads, d = 128, 303 MB   54.5 us  0.82
//   the same with 32 / 8 heads 67.0 us, 64 / 8 heads 93.7
//   64 sequences of 128 - 4096 keys, 16 / 8 heads, B = 16, 173 MB    38.6 us  0.66
//   8 x 16 K - 41 K keys, 16 / 8 heads, d = 64, 152 MB               42.0 us
//   one of 7777 keys, 32 / 4 heads, d = 64                            9.8 us
//   fp32 queries, 8 x 8 K - 20 K keys, 16 / 8 heads, d = 128         45.7 us
// 8 us of each are two launches, the plan, the first tile and the combine.  No pipe is
// full in any of the long ones (issue 55 - 60 %, ALU 49 - 55, tensor 18 - 33): three or
// four warps per scheduler wait for their own chains, so the time goes with the
// instructions executed, 31 million at 16 / 8 heads, 41 at 32 / 8 (2 % of them for
// spilled registers), 57 at 64 / 8, 26 at d = 64 and 27 with fp32 queries.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "launch.h"
#include "q4.cuh"
#include "split.cuh"

namespace pkv {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kHold = 16;         // 16-key products between additions of the offsets' sums
// A weight is 2^(score - maximum - kDown): sums of 2^31 keys' weights times any finite
// offset stay finite, and offsets down to 2^-78 keep their bits.  The references move
// when a score passes the maximum by 2^grow_by() or a V scale its bound by
// 2^scale_grow(): fp16 weights stay below 2^12 (bf16 queries; fp16 holds 11 bits of
// those down to 2^-14), or, moved up by 2^bias(), below 2^15 (fp32 queries, whose
// second part then has its bits for weights down to 2^-14 of the largest).
constexpr float kDown = 40.f;
template <bool F32>
__host__ __device__ constexpr float grow_by() { return F32 ? 2.f : 8.f; }
template <bool F32>
__host__ __device__ constexpr float scale_grow() { return F32 ? 1.f : 4.f; }
template <bool F32>
__host__ __device__ constexpr float bias() { return F32 ? 12.f : 0.f; }
constexpr int kProducers = 4;
constexpr int kMaxStages = 8;
constexpr int kHeader = 512;  // barriers and stage tags
constexpr size_t kStaticSmem = 1024;  // left for static shared memory

// Consumer warps: 12 with the 128 registers that 16 warps leave a thread, or 8 with
// 168 where 8 queries keep four column tiles (8 long contexts, 2 queries per KV head
// 53.8 us with 12 and 57.2 with 8; 8 queries 128 and 96, for spilled registers).  With
// 3 or 4 queries at d = 128 the 12 spill too, 76 bytes a thread (fp32 queries 104): 67.1
// us, and 67.6 with 8; fp32 queries over half the keys 55.6 and 52.3.
__host__ __device__ constexpr int consumers(int qn) { return qn == 8 ? 8 : 12; }
__host__ __device__ constexpr int threads(int qn) { return (consumers(qn) + kProducers) * 32; }

// 16-key products that a warp runs side by side (its share of a tile): two hide one
// another's latencies (8 long contexts 66.7 us with two and 79 with one, of an earlier
// form); with 8 queries they spill (121 us against 96).
template <int QN, bool F32>
__host__ __device__ constexpr int key_steps() { return QN == 8 ? 1 : 2; }

struct Q4DecodeArgs {
    const void* q;
    const unsigned char* kc;
    const unsigned char* vc;
    const int32_t* table;
    const int32_t* seqlens;
    float* part_o;     // [ctas + batch][hq][D]
    float* part_ml;    // [ctas + batch][hq][2]
    int32_t* tstart;   // [batch + 1]
    unsigned int* err;
    int64_t num_blocks;
    float qscale;  // scale * log2(e)
    int32_t max_blocks, batch, hq, hkv, block_size;
    int32_t hc;      // KV heads per CTA
    int32_t no;      // warps' worth of query heads per KV head
    int32_t wh;      // warps that share a head and its queries (part of a tile's keys each)
    int32_t stages;
    FastDiv block;   // by the page size
};

// One stage's description, written by the producer
struct Tag {
    uint32_t partial;  // fewer keys than the tile holds, or a bad page
    int32_t rows;      // keys
    int32_t bad;       // first key's position if a page was out of range, else -1
};

// a warp's merged state in shared memory: 8 NT output values, 2 maxima and 2 sums
// per lane
__host__ __device__ constexpr size_t state_bytes(int nt) { return (size_t)(8 * nt + 4) * 128; }

// d = a b + (c0, c1, c0, c1)
__device__ __forceinline__ void mma_from(float* d, const uint32_t* a, uint32_t b0, uint32_t b1,
                                         float c0, float c1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %11, %10, %11};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

// Codes 2i and 2i + 1 of both halves of x as operands, in units of code_unit().
//  * bf16 queries: a code in the low bits of an fp16's mantissa is a subnormal, so
//    fields of the word are operands as they are, without a shift (the upper bytes
//    come by a permutation): u0 and 16 u1 for the scores (score_pair), whose other
//    operands, q0 and q1 / 16, are exact; u0 and the byte of the two, u0 + 16 u1, for
//    the output (code_pair), one logic operation less for half of the pairs: there
//    both meet the same weights and the result takes u0 out again.  (The byte in the
//    scores as well, beside q0 - q1 / 16, took 0.4 us less at 8 long contexts and 2 less
//    with 4 queries per KV head, and fp16 does not hold that difference.)
//    The products are aligned by the operands' exponent fields, which overstate a
//    subnormal by up to 2^10, and cut 25 bits below the largest: about 2^-15 of the
//    largest weight, under the 2^-11 that the weights' own rounding leaves, and 2^-15
//    of the largest query for queries whose last bit is below that.
//  * EXACT (fp32 queries): 1024 + u, then minus 1024 + 8, gives the normal number
//    u0 - 8, and 1024 + 16 u, minus 1024 + 128, 16 (u1 - 8); the second parts of
//    queries and weights keep their bits.
template <bool EXACT>
__device__ __forceinline__ void code_pair(uint32_t x, int i, uint32_t& low, uint32_t& both) {
    if constexpr (EXACT) {
        const uint32_t y = i ? x >> 8 : x;
        low = (y & 0x000F000Fu) | 0x64006400u;
        both = (y & 0x00F000F0u) | 0x64006400u;
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(low) : "r"(0x64086408u));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(both) : "r"(0x64806480u));
    } else {
        both = i ? __byte_perm(x, 0u, 0x4341) : x & 0x00FF00FFu;
        low = both & 0x000F000Fu;
    }
}
template <bool EXACT>
__device__ __forceinline__ void score_pair(uint32_t x, int i, uint32_t& low, uint32_t& high) {
    if constexpr (EXACT) {
        code_pair<true>(x, i, low, high);
    } else {
        const uint32_t y = i ? __byte_perm(x, 0u, 0x4341) : x;
        low = y & 0x000F000Fu;
        high = y & 0x00F000F0u;
    }
}
template <bool EXACT>
__host__ __device__ constexpr float code_unit() { return EXACT ? 1.f : 1.f / 16777216.f; }

// where the 16 keys of a step sit: MMA row r + 8 half of the score product, and
// k index (2c, 2c+1, 2c+8, 2c+9 for i = 0..3) of the output product.  Chosen so
// that the lanes of one shared-memory access touch all banks once at row
// strides of 80 (d = 128) and 40 bytes (d = 64).
template <int NG>
__device__ __forceinline__ int score_key(int r, int half) {
    return NG == 4 ? (r >> 1) + 4 * (r & 1) + 8 * half : 4 * (r & 3) + (r >> 2) + 2 * half;
}
template <int NG>
__device__ __forceinline__ int output_key(int c, int i) {
    return NG == 4 ? 2 * c + (i & 1) + 8 * (i >> 1) : 4 * c + i;
}
// the (r, half) whose score_key is `key`
template <int NG>
__device__ __forceinline__ void score_row(int key, int* r, int* half) {
    if (NG == 4) {
        *half = key >> 3;
        *r = 2 * (key & 3) + ((key >> 2) & 1);
    } else {
        *half = (key >> 1) & 1;
        *r = (key >> 2) + 4 * (key & 1);
    }
}

template <int NG, int QN, bool F32>
__global__ void __launch_bounds__(threads(QN), 1)
q4_split_kernel(const Q4DecodeArgs a) {
    constexpr int WC = consumers(QN);
    constexpr int D = NG * kQ4Group, R = q4_row_bytes(D);
    constexpr int CPT = 8 / QN;                    // groups per column tile
    constexpr int NT = NG > CPT ? NG / CPT : 1;    // column tiles
    constexpr int PARTS = F32 ? 2 : 1;
    constexpr int NP = QN == 2 ? 1 : 2;            // queries a lane takes exponentials for
    constexpr int NV = QN == 8 ? 2 : 1;            // score rows a lane takes them for
    constexpr int KS = key_steps<QN, F32>();       // 16-key products side by side
    extern __shared__ __align__(128) unsigned char smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem);
    uint64_t* empty = full + kMaxStages;
    uint64_t* merge_bar = empty + kMaxStages;  // [2]
    Tag* tags = reinterpret_cast<Tag*>(smem + 256);
    int32_t* tstart = reinterpret_cast<int32_t*>(smem + kHeader);
    unsigned char* scratch = smem + kHeader + up((size_t)(a.batch + 1) * 4, 128);
    const int units = a.hc * a.no;  // (head, queries) of the CTA
    unsigned char* ring = scratch + (size_t)units * (a.wh - 1) * state_bytes(NT);
    __shared__ int32_t warp_sum[threads(QN) / 32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // A tile is the next T = KEYS * wh keys of a sequence: KEYS for each of the
    // wh warps of a head.
    constexpr int KEYS = 16 * KS;
    const int S = a.stages, T = KEYS * a.wh;
    const uint32_t half_bytes = (uint32_t)(a.hc * T * R);  // K (or V) of a stage
    const uint32_t stage_bytes = 2 * half_bytes;
    const int active = units * a.wh;  // consumer warps at work
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 2);  // a K and a V producer
            mbar_init(&empty[s], active);
        }
        mbar_init(&merge_bar[0], units * (a.wh - 1) + 1);
        mbar_init(&merge_bar[1], units);
        fence_barrier_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- plan: tile starts of the sequences (an exclusive scan of their tiles)
    const int64_t cap = (int64_t)a.max_blocks * a.block_size;
    const bool first_cta = blockIdx.x == 0 && blockIdx.y == 0;
    {
        constexpr int N = threads(QN);
        const int per = (a.batch + N - 1) / N;
        const int lo = tid * per, hi = min(lo + per, a.batch);
        int32_t sum = 0;
        for (int b = lo; b < hi; ++b) {
            const int32_t L = __ldg(a.seqlens + b);
            if (first_cta && (L < 0 || L > cap)) flag_error(a.err, PKV_FLAG_BAD_LENGTH);
            const int32_t n = (int32_t)min((int64_t)max(L, 0), cap);
            tstart[b + 1] = (n + T - 1) / T;
            sum += tstart[b + 1];
        }
        int32_t inc = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += y;
        }
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        int32_t run = inc - sum;
        for (int w = 0; w < warp; ++w) run += warp_sum[w];
        for (int b = lo; b < hi; ++b) {
            run += tstart[b + 1];
            tstart[b + 1] = run;
        }
        if (tid == 0) tstart[0] = 0;
        __syncthreads();
    }
    const int32_t total = tstart[a.batch];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (first_cta)  // for the combine, which reads them behind its wait
        for (int b = tid; b <= a.batch; b += blockDim.x) a.tstart[b] = tstart[b];
    const int32_t len = share_len(total, a.batch, gridDim.x);
    const int32_t t0 = share_first(tstart, a.batch, (int64_t)blockIdx.x * len);
    const int32_t t1 = share_first(tstart, a.batch, (int64_t)(blockIdx.x + 1) * len);
    if (t0 >= t1) return;
    const int head0 = blockIdx.y * a.hc;

    if (warp >= WC) {
        // ------------------------------ producers -----------------------------
        // Two pairs of warps take the tiles in turn, one warp of a pair K and the other
        // V: one tile costs a chain of ~2000 cycles (table entry, address, slot) and
        // ~60 more for each copy, whatever its size.  No more pairs than stages: a
        // warp then has seen its stage's last but one contents consumed (with its own
        // previous tile) before it waits for the last, which a wait on the phase's
        // parity alone could not tell apart.
#ifdef PKV_TEST_SPLIT_PRODUCER_IDLE
        return;  // test-only build: issue nothing, so the consumers' first wait runs out
#endif
        const bool is_v = (warp - WC) & 1;
        constexpr int prods = kProducers / 2;
        const uint64_t pol = l2_evict_first_policy();
        const uint32_t inv_hc = 65536u / a.hc + 1;  // i / hc for i < 512, hc <= 16
        const int64_t head_bytes = (int64_t)a.block_size * R;
        const int32_t tf = t0 + (warp - WC) / 2;
        if (tf >= t1) return;
        int b = share_seq(tstart, a.batch, tf);  // the sequence of tile t
        int32_t L = (int32_t)min((int64_t)max(__ldg(a.seqlens + b), 0), cap);
        // ids of a tile's first 32 pages, one tile ahead
        auto fetch = [&](int bb, int32_t p0, int32_t p1) {
            const int32_t pg = (int32_t)a.block.quot((uint32_t)p0) + lane;
            return (int64_t)pg * a.block_size < p1
                       ? __ldg(a.table + (int64_t)bb * a.max_blocks + pg) : -1;
        };
        int32_t p0 = (tf - tstart[b]) * T, p1 = min(L, p0 + T);
        int32_t next_page = fetch(b, p0, p1);
        int32_t last_k = -1;
        int s = tf - t0;      // stage and the times it was filled before
        uint32_t fills = 0;
        for (int32_t t = tf; t < t1; t += prods) {
            const int seq = b;
            const int32_t q0 = p0, q1 = p1;  // this tile's keys
            int32_t page = next_page;
            if (t + prods < t1) {  // the next tile's sequence and pages
                if (t + prods >= tstart[b + 1]) {
                    do ++b; while (tstart[b + 1] <= t + prods);
                    L = (int32_t)min((int64_t)max(__ldg(a.seqlens + b), 0), cap);
                }
                p0 = (t + prods - tstart[b]) * T;
                p1 = min(L, p0 + T);
                next_page = fetch(b, p0, p1);
            }
            const int32_t k = t - t0;
            const int32_t pg0 = (int32_t)a.block.quot((uint32_t)q0);
            const int np = (int32_t)a.block.quot((uint32_t)(q1 - 1)) - pg0 + 1;
            // the bytes that will arrive
            uint32_t bytes = 0;
            bool bad = false;
            for (int c0 = 0; c0 < np; c0 += 32) {
                const int32_t pg = pg0 + c0 + lane;
                if (c0 + lane < np) {
                    const int32_t id =
                        c0 == 0 ? page : __ldg(a.table + (int64_t)seq * a.max_blocks + pg);
                    const int32_t lo = max(q0, pg * a.block_size);
                    const int32_t hi = (int32_t)min((int64_t)q1, (int64_t)(pg + 1) * a.block_size);
                    if (id < 0 || id >= a.num_blocks) bad = true;
                    else bytes += (uint32_t)up((size_t)(hi - lo) * R, 16);
                }
            }
            bad = __any_sync(0xffffffffu, bad);
            bytes = __reduce_add_sync(0xffffffffu, bytes) * a.hc;
            bool ok = true;
            if (lane == 0) {
                ok = mbar_wait(&empty[s], (fills & 1) ^ 1, a.err);
                if (ok) {
                    if (bad) flag_error(a.err, PKV_FLAG_BAD_BLOCK);
                    if (!is_v)
                        tags[s] = Tag{bad || q1 - q0 < T, q1 - q0, bad ? q0 : -1};
                    mbar_arrive_expect_tx(&full[s], bytes);
                }
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            last_k = k;
            unsigned char* kd = ring + (size_t)s * 2 * half_bytes;
            for (int c0 = 0; c0 < np; c0 += 32) {
                if (c0 > 0) {
                    const int32_t pg = pg0 + c0 + lane;
                    page = c0 + lane < np ? __ldg(a.table + (int64_t)seq * a.max_blocks + pg) : -1;
                }
                const int n = min(32, np - c0) * a.hc;
                for (int i0 = 0; i0 < n; i0 += 32) {
                    const int i = min(i0 + lane, n - 1);
                    const int p = (int)((i * inv_hc) >> 16), h = i - p * a.hc;
                    const int32_t id = __shfl_sync(0xffffffffu, page, p);
                    if (i0 + lane >= n || id < 0 || id >= a.num_blocks) continue;
                    const int32_t pg = pg0 + c0 + p;
                    const int32_t lo = max(q0, pg * a.block_size);
                    const int32_t hi = (int32_t)min((int64_t)q1, (int64_t)(pg + 1) * a.block_size);
                    const int64_t src = ((int64_t)id * a.hkv + head0 + h) * head_bytes +
                                        (int64_t)(lo - pg * a.block_size) * R;
                    unsigned char* dst = kd + ((size_t)h * T + (lo - q0)) * R;
                    const uint32_t n16 = (uint32_t)up((size_t)(hi - lo) * R, 16);
                    bulk_g2s(is_v ? dst + half_bytes : dst, (is_v ? a.vc : a.kc) + src, n16,
                             &full[s], pol);
                }
            }
            __syncwarp();
            s += prods;
            if (s >= S) {
                s -= S;
                ++fills;
            }
        }
        // no copy may be in flight when the CTA exits (after a timeout the
        // consumers may have stopped waiting): wait for the fills that no later
        // one follows
        if (lane == 0)
            for (int32_t k = last_k; k >= 0 && k >= t1 - t0 - S; k -= prods)
                if (!mbar_wait(&full[k % S], (k / S) & 1, a.err)) break;
        return;
    }
    if (warp >= active) return;

    // ------------------------------- consumers --------------------------------
    const int unit = warp % units, rank = warp / units;
    const int hc = unit % a.hc, oct = unit / a.hc;
    const int r = lane >> 2, c = lane & 3;
    const int G = a.hq / a.hkv;
    const int q0 = oct * QN;                        // first query of this warp in its group
    const int nq = min(QN, G - q0);                 // queries it has
    const int qh0 = (head0 + hc) * G + q0;          // first query head
    const int my_q = r % QN;                        // query of this lane's column (n = r)

    // lanes that hold the weights of this lane's keys and query
    int src_lane[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int sr, half;
        score_row<NG>(output_key<NG>(c, i), &sr, &half);
        if (QN == 2) src_lane[i] = sr * 4 + half * 2 + my_q;
        else if (QN == 4) src_lane[i] = sr * 4 + half * 2 + (my_q >> 1);
        else src_lane[i] = sr * 4 + (my_q >> 1);
    }

    // One or two groups share a column tile's products (QN <= 4): the two 16-bit
    // halves of a code word then are two groups' codes, in columns of their own
    // (zeros meet the other half), and need no rearranging.  With 8 queries a tile
    // holds one group and a byte permutation brings its codes together.
    constexpr bool PAIR = QN < 8;
    const uint32_t half_shift = (r / QN) & 1 ? 16 : 0;  // this column's half
    uint32_t qf[PARTS][NG][4];  // score product's columns: 2 k-steps of 2 words per code word
    float qs[NT][2];            // sum of q over the group of columns 2c, 2c + 1, in units of code_unit()
    float start[NT][2];         // -8 times those: where a score product starts
    float cq[NP];               // from a product to log2 units, for this lane's queries
    constexpr int OT = PAIR ? NG : 2 * NG;  // output tiles of 16 rows
    float o[OT][4], ct[NT][4], zacc[NT], l[NP];
    // reference of the queries' weights, the same with -inf as 0, and the score
    // that makes it move; the V scale that makes the scales' reference move, and what
    // weights are multiplied by before their V scale (a power of two, like the former)
    float m[NP], mr[NP], lim[NP], slim = 0.f, wmul = 0.f;
    auto inverse = [](float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); };
    auto weight_scale = [&]() { return inverse(slim) * exp2f(kDown + bias<F32>() + scale_grow<F32>()); };
    auto settle = [&]() {
#pragma unroll
        for (int i = 0; i < OT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] += ct[(PAIR ? i / 2 * 2 : i / 2) / CPT][e];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) ct[j][e] = 0.f;
    };
    auto clear = [&]() {  // the state of a new piece
#pragma unroll
        for (int i = 0; i < OT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            zacc[j] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) ct[j][e] = 0.f;
        }
        slim = exp2f(scale_grow<F32>() - 60.f);
        wmul = weight_scale();
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            m[i] = lim[i] = -INFINITY;
            mr[i] = 0.f;
            l[i] = 0.f;
        }
    };
    auto load_queries = [&](int32_t seq) {
        float xs[NT][8];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int g_col = j * CPT + r / QN;  // the group of this lane's column
            float* x = xs[j];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.f;
            if (g_col < NG && my_q < nq) {
                const int64_t at = ((int64_t)seq * a.hq + qh0 + my_q) * D + g_col * 32 + c * 8;
                if constexpr (F32) {
                    const float4* p =
                        reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
                    const float4 u = __ldg(p), v = __ldg(p + 1);
                    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
                    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
                } else {
                    const uint4 w = __ldg(
                        reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at));
                    x[0] = bf16lo(w.x); x[1] = bf16hi(w.x); x[2] = bf16lo(w.y);
                    x[3] = bf16hi(w.y); x[4] = bf16lo(w.z); x[5] = bf16hi(w.z);
                    x[6] = bf16lo(w.w); x[7] = bf16hi(w.w);
                }
            }
        }
        // the query scaled by a power of two to below 2^12: fp16 then holds bf16
        // queries (and 1/16 of them) exactly down to 2^-24 of the largest, and two
        // parts hold 23 bits of fp32 ones
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(xs[j][e]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
#pragma unroll
        for (int off = 4 * QN; off < 32; off <<= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const int ex = (int)(__float_as_uint(mx) >> 23);
        const float up_q = __uint_as_float((uint32_t)min(max(265 - ex, 1), 252) << 23);
        const float down = a.qscale / code_unit<F32>() / up_q;
        if constexpr (QN == 2) {
            cq[0] = __shfl_sync(0xffffffffu, down, 4 * (c & 1));
        } else {
            const int n = QN == 4 ? 2 * (c & 1) : 2 * c;
            cq[0] = __shfl_sync(0xffffffffu, down, 4 * n);
            cq[NP - 1] = __shfl_sync(0xffffffffu, down, 4 * n + 4);
        }
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
            for (int w = 0; w < NG; ++w)
#pragma unroll
                for (int e = 0; e < 4; ++e) qf[part][w][e] = 0u;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int g_col = j * CPT + r / QN;
            float* x = xs[j];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= up_q;
            float sum = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
            sum *= code_unit<F32>();
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            qs[j][0] = __shfl_sync(0xffffffffu, sum, 8 * c);
            qs[j][1] = __shfl_sync(0xffffffffu, sum, 8 * c + 4);
            start[j][0] = F32 ? 0.f : -8.f * qs[j][0];
            start[j][1] = F32 ? 0.f : -8.f * qs[j][1];
#pragma unroll
            for (int e = 1; e < 8; e += 2) x[e] *= 0.0625f;  // (codes of odd dims count 16 times)
            if constexpr (PAIR) {
                // word (unit u of 2, pair of groups gp): dims 4u .. 4u + 3 of the
                // chunk, k-step e / 2, word e % 2
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float none = 0.f;
#pragma unroll
                        for (int part = 0; part < PARTS; ++part) {
                            const uint32_t w = take_f16x2<F32>(x[4 * u + e], none) << half_shift;
#pragma unroll
                            for (int gp = 0; gp < NG / 2; ++gp)
                                if (2 * gp / CPT == j && g_col >> 1 == gp)
                                    qf[part][u * (NG / 2) + gp][e] = w;
                        }
                    }
            } else {
#pragma unroll
                for (int part = 0; part < PARTS; ++part)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        qf[part][j][e] = take_f16x2<F32>(x[e], x[e + 4]);
            }
        }
    };
    // Where this lane's chunks sit in a head's rows of a stage (K: row of score
    // row r, V: row of its first key); other rows are constants away.
    constexpr int kHalfRow = (NG == 4 ? 8 : 2) * R;  // score row r + 8
    const int k_codes = score_key<NG>(r, 0) * R + 4 * NG * c;
    const int k_scale = score_key<NG>(r, 0) * R + D / 2 + 4 * (NT * CPT > NG ? (2 * c / QN) % NG : 2 * c / QN);
    const int v_codes = output_key<NG>(c, 0) * R + 2 * NG * r;
    const int v_scale = output_key<NG>(c, 0) * R + D / 2 + 4 * (NT * CPT > NG ? (r / QN) % NG : r / QN);
    const bool k_live = NT * CPT <= NG || 2 * c / QN < NG, v_live = NT * CPT <= NG || r / QN < NG;
    // scores of the step's keys in log2 units, for this lane's rows and queries,
    // and the V scales of its keys and columns
    auto scores = [&](const unsigned char* tile, float (&p)[KS][NV][NP],
                      uint32_t (&vsz)[KS][NT][4]) {
#pragma unroll
        for (int y = 0; y < KS; ++y) {
            const unsigned char* ks = tile + y * 16 * R;
            const unsigned char* vs = ks + half_bytes;
            uint32_t kw[2][NG], ksz[NT][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const unsigned char* at = ks + k_codes + h * kHalfRow;
                if constexpr (NG == 4) {
                    const uint4 w = *reinterpret_cast<const uint4*>(at);
                    kw[h][0] = w.x; kw[h][1] = w.y; kw[h][NG - 2] = w.z; kw[h][NG - 1] = w.w;
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(at);
                    kw[h][0] = w.x; kw[h][1] = w.y;
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    ksz[j][h] = *reinterpret_cast<const uint32_t*>(ks + k_scale + h * kHalfRow +
                                                                   4 * CPT * j);
                    if (!k_live) ksz[j][h] = 0u;
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    vsz[y][j][i] = *reinterpret_cast<const uint32_t*>(
                        vs + v_scale + output_key<NG>(0, i) * R + 4 * CPT * j);
                    if (!v_live) vsz[y][j][i] = 0u;
                }
            float sc[NT][4];
#pragma unroll
            for (int w = 0; w < NG; ++w) {
                uint32_t x[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (PAIR) x[h] = kw[h][w];
                    else x[h] = __byte_perm(kw[h][NG == 4 ? w >> 1 : 0], kw[h][NG == 4 ? 2 + (w >> 1) : 1],
                                            (w & 1) ? 0x7632 : 0x5410);
                }
                const int j = PAIR ? 2 * (w % (NG / 2)) / CPT : w;
                const bool opens = PAIR ? w < NG / 2 && (NT > 1 || w == 0) : true;  // tile j's first
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    uint32_t af[4];
                    score_pair<F32>(x[0], st, af[0], af[2]);
                    score_pair<F32>(x[1], st, af[1], af[3]);
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        const uint32_t b0 = qf[part][w][2 * st], b1 = qf[part][w][2 * st + 1];
                        if (opens && part == 0 && st == 0) {
                            mma_from(sc[j], af, b0, b1, start[j][0], start[j][1]);
                        } else {
                            mma(sc[j], af, b0, b1);
                        }
                    }
                }
            }
            // scale per group, sum over the groups
            float v[2][2];  // [row half][query 2c, 2c + 1]
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    v[h][i] = 0.f;
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        v[h][i] = fmaf(bf16lo(ksz[j][h]), sc[j][2 * h + i], v[h][i]);
                        v[h][i] = fmaf(bf16hi(ksz[j][h]), qs[j][i], v[h][i]);
                    }
                }
            if constexpr (QN == 8) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        p[y][NV == 2 ? h : 0][NP == 2 ? i : 0] = v[h][i] * cq[NP == 2 ? i : 0];
            } else {
                // lanes c and c ^ 2 hold other groups of the same queries: each
                // keeps one row half
                const bool up_half = c & 2;
                float w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float got = __shfl_xor_sync(0xffffffffu, up_half ? v[0][i] : v[1][i], 2);
                    w[i] = (up_half ? v[1][i] : v[0][i]) + got;
                }
                if constexpr (QN == 4) {
                    p[y][0][0] = w[0] * cq[0];
                    p[y][0][NP - 1] = w[1] * cq[NP - 1];
                } else {  // lanes c and c ^ 1: each keeps one query
                    const float got = __shfl_xor_sync(0xffffffffu, (c & 1) ? w[0] : w[1], 1);
                    p[y][0][0] = (((c & 1) ? w[1] : w[0]) + got) * cq[0];
                }
            }
        }
    };

    int merges = 0;
    const int32_t n_tiles = t1 - t0;
    uint32_t full_bar = smem_u32(full), empty_bar = smem_u32(empty);
    asm volatile("" : "+r"(full_bar), "+r"(empty_bar));  // (keep them)
    // this warp's keys in stage 0
    const unsigned char* keys0 = ring + (hc * T + rank * KEYS) * R;
    float p[KS][NV][NP];
    uint32_t vsz[KS][NT][4];
    clear();

    int s = 0;
    uint32_t phase = 0;    // of stage s
    int seq = share_seq(tstart, a.batch, t0) - 1;  // sequence of tile k
    int32_t next = 0;      // the tile that the next one begins with
    for (int32_t k = 0; k < n_tiles; ++k) {
        if (k == next) {  // (before the wait: the first queries come with the first tile)
            do ++seq; while (tstart[seq + 1] <= t0 + k);
            next = min(tstart[seq + 1] - t0, n_tiles);
            load_queries(seq);
        }
        if (!wait_phase(full_bar + 8 * s, phase, a.err)) break;
        const uint32_t partial = tags[s].partial;
        const unsigned char* tile = keys0 + s * stage_bytes;
        scores(tile, p, vsz);
        if (__builtin_expect(partial, 0)) {
            // keys that do not count: scores of -inf, scales of 0
            const Tag tag = tags[s];
            auto valid = [&](int key) {
                const int at = rank * KEYS + key;
                if (at >= tag.rows) return false;
                if (tag.bad < 0) return true;
                const int32_t id = __ldg(a.table + (int64_t)seq * a.max_blocks +
                                         (tag.bad + at) / a.block_size);
                return id >= 0 && id < a.num_blocks;
            };
#pragma unroll
            for (int y = 0; y < KS; ++y) {
#pragma unroll
                for (int h = 0; h < NV; ++h) {
                    const bool ok = valid(16 * y + score_key<NG>(r, QN == 8 ? h : c >> 1));
#pragma unroll
                    for (int i = 0; i < NP; ++i) p[y][h][i] = ok ? p[y][h][i] : -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool ok = valid(16 * y + output_key<NG>(c, i));
#pragma unroll
                    for (int j = 0; j < NT; ++j) vsz[y][j][i] = ok ? vsz[y][j][i] : 0u;
                }
            }
        }
        // The V words, and the stage is given back: it is held for its loads, not for
        // the arithmetic, which keeps the ring of three stages full.
        uint32_t vw[KS][4][2];
#pragma unroll
        for (int y = 0; y < KS; ++y)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const unsigned char* vr =
                    tile + half_bytes + v_codes + (16 * y + output_key<NG>(0, i)) * R;
                if constexpr (NG == 4) {
                    const uint2 x = *reinterpret_cast<const uint2*>(vr);
                    vw[y][i][0] = x.x;
                    vw[y][i][1] = x.y;
                } else {
                    vw[y][i][0] = *reinterpret_cast<const uint32_t*>(vr);
                }
            }
        const bool ends = k + 1 == next;
        __syncwarp();
        if (lane == 0) arrive(empty_bar + 8 * s);
        float smax = 0.f;
        bool grow = false;
#pragma unroll
        for (int y = 0; y < KS; ++y) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; i += 2)
                    smax = fmax3(smax, fabsf(bf16lo(vsz[y][j][i])),  // (of either sign)
                                 fabsf(bf16lo(vsz[y][j][i + 1])));
#pragma unroll
            for (int h = 0; h < NV; ++h)
#pragma unroll
                for (int i = 0; i < NP; ++i) grow |= p[y][h][i] > lim[i];
        }
        grow |= smax > slim;
        if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {  // move the reference to the running maximum
            // (an infinite scale makes its own group NaN, and is no reference for the others)
            smax = 0.f;
#pragma unroll
            for (int y = 0; y < KS; ++y)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = fabsf(bf16lo(vsz[y][j][i]));
                        smax = fmaxf(smax, x < INFINITY ? x : 0.f);
                    }
#pragma unroll
            for (int off = 1; off < 32; off <<= 1)
                smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, off));
            // the least power of two above the scales so far, 2^-60 at least
            constexpr int kGrow = (int)scale_grow<F32>();
            const int se = min(max((int)(__float_as_uint(smax) >> 23) - 126, -60), 126 - kGrow);
            const float was = slim;
            slim = fmaxf(slim, __uint_as_float((uint32_t)(se + kGrow + 127) << 23));
            wmul = weight_scale();
            const float fs = was * inverse(slim);
            float f[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int y = 0; y < KS; ++y)
#pragma unroll
                    for (int h = 0; h < NV; ++h) mx = fmaxf(mx, p[y][h][i]);
#pragma unroll
                for (int off = QN == 8 ? 4 : 2; off < 32; off <<= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                const float mn = fmaxf(m[i], mx + kDown);
                f[i] = m[i] == -INFINITY ? 0.f : ex2(m[i] - mn);
                m[i] = mn;
                mr[i] = mn == -INFINITY ? 0.f : mn;
                lim[i] = mn - kDown + grow_by<F32>();
                l[i] *= f[i];
            }
            // factors of this lane's columns 2c, 2c + 1 and of column r
            float f0, f1, fr;
            if constexpr (QN == 2) {
                f0 = __shfl_sync(0xffffffffu, f[0], lane & ~1);
                f1 = __shfl_sync(0xffffffffu, f[0], lane | 1);
                fr = my_q ? f1 : f0;
            } else {
                f0 = f[0];
                f1 = f[NP - 1];
                const float x0 = __shfl_sync(0xffffffffu, f0, (lane & ~3) | (my_q >> 1));
                const float x1 = __shfl_sync(0xffffffffu, f1, (lane & ~3) | (my_q >> 1));
                fr = (my_q & 1) ? x1 : x0;
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) zacc[j] *= fr;
            f0 *= fs;
            f1 *= fs;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                ct[j][0] *= f0;
                ct[j][1] *= f1;
                ct[j][2] *= f0;
                ct[j][3] *= f1;
            }
#pragma unroll
            for (int i = 0; i < OT; ++i) {
                o[i][0] *= f0;
                o[i][1] *= f1;
                o[i][2] *= f0;
                o[i][3] *= f1;
            }
        }
#pragma unroll
        for (int y = 0; y < KS; ++y) {
#pragma unroll
            for (int h = 0; h < NV; ++h)
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    p[y][h][i] = ex2(p[y][h][i] - mr[i]);
                    l[i] += p[y][h][i];
                }
            // the weights of this lane's 4 keys and query
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (QN == 2) {
                    w[i] = __shfl_sync(0xffffffffu, p[y][0][0], src_lane[i]);
                } else {
                    // (8 queries: key i's row half is i >> 1 in every lane)
                    const int h = QN == 8 && i >= 2 ? NV - 1 : 0;
                    const float x0 = __shfl_sync(0xffffffffu, p[y][h][0], src_lane[i]);
                    const float x1 = __shfl_sync(0xffffffffu, p[y][h][NP - 1], src_lane[i]);
                    w[i] = (my_q & 1) ? x1 : x0;
                }
            }
            float wm[4];  // for the codes
#pragma unroll
            for (int i = 0; i < 4; ++i) wm[i] = w[i] * wmul;
            // columns: a word per key (its weight in this column's half), or per two
            // keys
            constexpr int PW = PAIR ? 4 : 2;
            uint32_t pf[PARTS][NT][PW];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float ws[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ws[i] = wm[i] * bf16lo(vsz[y][j][i]);
                    zacc[j] = fmaf(w[i], bf16hi(vsz[y][j][i]), zacc[j]);
                }
                if constexpr (PAIR) {
#pragma unroll
                    for (int part = 0; part < PARTS; ++part)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float none = 0.f;
                            pf[part][j][i] = take_f16x2<F32>(ws[i], none) << half_shift;
                        }
                } else {
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) {
                        pf[part][j][0] = take_f16x2<F32>(ws[0], ws[1]);
                        pf[part][j][1] = take_f16x2<F32>(ws[2], ws[3]);
                    }
                }
                if constexpr (!F32) {
                    // -8 in rows r (u0), -8 - 128 in rows r + 8 (u0 + 16 u1)
                    const uint32_t off[4] = {0x80088008u, 0x80888088u, 0x80088008u, 0x80888088u};
#pragma unroll
                    for (int i = 0; i < PW; i += 2) mma(ct[j], off, pf[0][j][i], pf[0][j][i + 1]);
                }
            }
            if constexpr (PAIR) {
#pragma unroll
                for (int gp = 0; gp < NG / 2; ++gp)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int u = 0; u < 4; u += 2) {
                            uint32_t af[4];
                            code_pair<F32>(vw[y][u][gp], h, af[0], af[1]);
                            code_pair<F32>(vw[y][u + 1][gp], h, af[2], af[3]);
                            const int j = 2 * gp / CPT;
#pragma unroll
                            for (int part = 0; part < PARTS; ++part)
                                mma(o[2 * gp + h], af, pf[part][j][u], pf[part][j][u + 1]);
                        }
            } else {
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const uint32_t sel = (g & 1) ? 0x7632 : 0x5410;
                    const uint32_t xa = __byte_perm(vw[y][0][g >> 1], vw[y][1][g >> 1], sel);
                    const uint32_t xb = __byte_perm(vw[y][2][g >> 1], vw[y][3][g >> 1], sel);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t af[4];
                        code_pair<F32>(xa, h, af[0], af[1]);
                        code_pair<F32>(xb, h, af[2], af[3]);
#pragma unroll
                        for (int part = 0; part < PARTS; ++part)
                            mma(o[2 * g + h], af, pf[part][g][0], pf[part][g][1]);
                    }
                }
            }
        }
        if (!F32 && k % (kHold / KS) == 0) settle();
        if (++s == S) {
            s = 0;
            phase ^= 1;
        }
        if (!ends) continue;

        // ---- end of the piece: this warp's state, in output layout: dims 32 g +
        // 4 r .. + 3 of queries 2c, 2c + 1 (mod QN) for g = j CPT + 2c / QN
        if constexpr (!F32) settle();
#pragma unroll
        for (int i = 0; i < NP; ++i) {
#pragma unroll
            for (int off = QN == 8 ? 4 : 2; off < 32; off <<= 1)
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
            if (l[i] != l[i] && m[i] == -INFINITY) m[i] = 0.f;  // every score a NaN
        }
        float m2[2], l2[2], val[NT][2][4];
        if constexpr (QN == 2) {
            m2[0] = __shfl_sync(0xffffffffu, m[0], lane & ~1);
            m2[1] = __shfl_sync(0xffffffffu, m[0], lane | 1);
            l2[0] = __shfl_sync(0xffffffffu, l[0], lane & ~1);
            l2[1] = __shfl_sync(0xffffffffu, l[0], lane | 1);
        } else {
            m2[0] = m[0];
            m2[1] = m[NP - 1];
            l2[0] = l[0];
            l2[1] = l[NP - 1];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float z = zacc[j];
            z += __shfl_xor_sync(0xffffffffu, z, 1);
            z += __shfl_xor_sync(0xffffffffu, z, 2);
            const float z0 = __shfl_sync(0xffffffffu, z, 8 * c);
            const float z1 = __shfl_sync(0xffffffffu, z, 8 * c + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) val[j][0][e] = val[j][1][e] = 0.f;
#pragma unroll
            for (int gi = 0; gi < CPT; ++gi) {
                const int g = j * CPT + gi;
                if (g >= NG || gi != 2 * c / QN) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float u = inverse(wmul) / code_unit<F32>() / (e & 1 ? 16.f : 1.f);
                    const float* x = o[(PAIR ? g >> 1 : g) * 2 + (e >> 1)] + 2 * (e & 1);
                    const bool mixed = !F32 && (e & 1);  // holds its even neighbour too
                    val[j][0][e] = fmaf(x[0] - (mixed ? x[-2] : 0.f), u, z0);
                    val[j][1][e] = fmaf(x[1] - (mixed ? x[-1] : 0.f), u, z1);
                }
            }
        }
        clear();
        if (a.wh > 1) {  // the warps of this head and queries: rank 0 merges
            if (rank > 0) {
                if (merges > 0 &&
                    !__all_sync(0xffffffffu, mbar_wait(&merge_bar[1], (merges - 1) & 1, a.err)))
                    break;
                float* x = reinterpret_cast<float*>(
                    scratch + (size_t)((rank - 1) * units + unit) * state_bytes(NT));
                float4* y = reinterpret_cast<float4*>(x);
                y[lane] = make_float4(m2[0], m2[1], l2[0], l2[1]);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        y[(1 + 2 * j + i) * 32 + lane] = make_float4(val[j][i][0], val[j][i][1],
                                                                     val[j][i][2], val[j][i][3]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&merge_bar[0]);
            } else {
                if (unit == 0 && lane == 0) mbar_arrive(&merge_bar[0]);
                if (!__all_sync(0xffffffffu, mbar_wait(&merge_bar[0], merges & 1, a.err))) break;
                for (int wv = 1; wv < a.wh; ++wv) {
                    const float4* y = reinterpret_cast<const float4*>(
                        scratch + (size_t)((wv - 1) * units + unit) * state_bytes(NT));
                    const float4 st = y[lane];
                    const float mo[2] = {st.x, st.y}, lo[2] = {st.z, st.w};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float M = fmaxf(m2[i], mo[i]);
                        const float ca = m2[i] == -INFINITY ? 0.f : ex2(m2[i] - M);
                        const float cb = mo[i] == -INFINITY ? 0.f : ex2(mo[i] - M);
                        l2[i] = l2[i] * ca + lo[i] * cb;
                        m2[i] = M;
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const float4 x = y[(1 + 2 * j + i) * 32 + lane];
                            val[j][i][0] = val[j][i][0] * ca + x.x * cb;
                            val[j][i][1] = val[j][i][1] * ca + x.y * cb;
                            val[j][i][2] = val[j][i][2] * ca + x.z * cb;
                            val[j][i][3] = val[j][i][3] * ca + x.w * cb;
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&merge_bar[1]);
            }
            ++merges;
        }
        if (rank != 0) continue;
        const int64_t slot = (int64_t)blockIdx.x + seq;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int qi = (2 * c + i) % QN;
            if (qi >= nq) continue;
            const int64_t at = slot * a.hq + qh0 + qi;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int g = j * CPT + 2 * c / QN;
                if (g < NG)
                    *reinterpret_cast<float4*>(a.part_o + at * D + 32 * g + 4 * r) =
                        make_float4(val[j][i][0], val[j][i][1], val[j][i][2], val[j][i][3]);
            }
            if (r == 0 && 2 * c / QN == 0)
                *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(m2[i], l2[i]);
        }
    }
}

template <int NG, int QN, bool F32>
cudaError_t launch_split(const DeviceInfo& dev, const Q4DecodePlan& p, const Q4DecodeArgs& a,
                         cudaStream_t stream) {
    auto kern = q4_split_kernel<NG, QN, F32>;
    // the most shared memory a CTA may have, set once per device
    static std::atomic<uint64_t> set{0};
    const uint64_t bit = 1ull << dev.device;
    if (!(set.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
            (int)(dev.max_smem_optin - kStaticSmem));
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_dependent(kern, dim3(p.ctas, p.head_groups),
                            dim3(threads(QN)), p.smem_bytes, stream, a);
}

}  // namespace

bool plan_q4_decode(const DeviceInfo& dev, int32_t batch, int32_t max_blocks, int hq, int hkv,
                    int d, int block_size, int q_dtype, Q4DecodePlan* p) {
    if ((d != 64 && d != 128) || batch > kDecodeMaxBatch) return false;
    // positions, and a tile beyond, in 32 bits
    if ((double)max_blocks * block_size > 2147483647.0 - 4096) return false;
    // rows of 40 bytes: copies of a page piece start on 16 bytes when pages
    // hold an even number of rows
    if (d == 64 && block_size % 2) return false;
    const bool f32 = q_dtype == PKV_F32;
    const int G = hq / hkv;
    p->qn = G <= 2 ? 2 : (G <= 4 ? 4 : 8);
    const int wc = consumers(p->qn);
    p->no = (G + p->qn - 1) / p->qn;
    if (p->no > wc) return false;
    // KV heads per CTA: the most, up to 6 warps' worth, that keep four fifths of the
    // consumers at work; the warps left over share a head's keys.  (8 heads: 4 with 3
    // warps each, 38.2 us at 64 sequences and 53.8 at 8 long contexts; 2 heads with 6
    // warps, and more merges, 39.7 and 53.2; 8 heads with 1 warp, and 4 idle, 38.5 and
    // 57.3.)
    p->hc = 1;
    auto at_work = [&](int h) { return wc / (h * p->no) * (h * p->no); };
    for (int h = 1; h <= hkv && h * p->no <= std::max(6, p->no); ++h)
        if (hkv % h == 0 && (5 * at_work(h) >= 4 * wc || at_work(h) > at_work(p->hc))) p->hc = h;
    p->head_groups = hkv / p->hc;
    if (p->head_groups > 65535) return false;
    const int units = p->hc * p->no;
    p->wh = wc / units;
    p->tile = 16 * (p->qn == 8 ? key_steps<8, false>() : key_steps<2, false>()) * p->wh;
    const int R = q4_row_bytes(d);
    const int nt = std::max(1, d / kQ4Group * p->qn / 8);
    const size_t stage = (size_t)2 * p->hc * p->tile * R;
    const size_t fixed = kHeader + up((size_t)(batch + 1) * 4, 128) +
                         (size_t)units * (p->wh - 1) * state_bytes(nt);
    const size_t room = dev.max_smem_optin - kStaticSmem;
    if (room < fixed + 2 * stage) return false;
    p->stages = (int)std::min<size_t>(kMaxStages, (room - fixed) / stage);
    p->smem_bytes = fixed + p->stages * stage;
    // one CTA per SM, no more than there can be tiles
    const int64_t tiles = ((int64_t)max_blocks * block_size + p->tile - 1) / p->tile * batch;
    const int64_t most = std::max(1, dev.num_sms / p->head_groups);
    if (tiles + batch > 0x7fffffffLL - most) return false;  // the line of tiles is 32 bits long
    p->ctas = (int)std::max<int64_t>(1, std::min(most, tiles));
    const size_t slots = (size_t)most + batch;  // whatever the table's width is
    p->ws_bytes = up((size_t)(batch + 1) * 4, 256) + up(slots * hq * 2 * 4, 256) +
                  up(slots * hq * d * 4, 256);
    return true;
}

cudaError_t launch_q4_decode(const DeviceInfo& dev, const Q4DecodePlan& p, const void* q, const void* k_cache,
                             const void* v_cache, const int32_t* table, int32_t max_blocks,
                             const int32_t* seqlens, int32_t batch, float scale, void* out,
                             void* workspace, int hq, int hkv, int d, int block_size,
                             int64_t num_blocks, int q_dtype, unsigned int* err,
                             cudaStream_t stream) {
    if (batch == 0) return cudaSuccess;
    Q4DecodeArgs a{};
    a.q = q;
    a.kc = static_cast<const unsigned char*>(k_cache);
    a.vc = static_cast<const unsigned char*>(v_cache);
    a.table = table;
    a.seqlens = seqlens;
    const size_t slots = (size_t)p.ctas + batch;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    a.tstart = reinterpret_cast<int32_t*>(ws);
    ws += up((size_t)(batch + 1) * 4, 256);
    a.part_ml = reinterpret_cast<float*>(ws);
    ws += up(slots * hq * 2 * 4, 256);
    a.part_o = reinterpret_cast<float*>(ws);
    a.err = err;
    a.num_blocks = num_blocks;
    a.qscale = scale * kLog2e;
    a.max_blocks = max_blocks;
    a.batch = batch;
    a.hq = hq;
    a.hkv = hkv;
    a.block_size = block_size;
    a.hc = p.hc;
    a.no = p.no;
    a.wh = p.wh;
    a.block = FastDiv((uint32_t)block_size);
    a.stages = p.stages;
    const bool f32 = q_dtype == PKV_F32;
    cudaError_t e = cudaErrorInvalidValue;
#define PKV_Q4_CASE(NN, QQ, FF) \
    if (d == NN * kQ4Group && p.qn == QQ && f32 == FF) e = launch_split<NN, QQ, FF>(dev, p, a, stream);
    PKV_Q4_CASE(4, 2, false) PKV_Q4_CASE(4, 4, false) PKV_Q4_CASE(4, 8, false)
    PKV_Q4_CASE(4, 2, true) PKV_Q4_CASE(4, 4, true) PKV_Q4_CASE(4, 8, true)
    PKV_Q4_CASE(2, 2, false) PKV_Q4_CASE(2, 4, false) PKV_Q4_CASE(2, 8, false)
    PKV_Q4_CASE(2, 2, true) PKV_Q4_CASE(2, 4, true) PKV_Q4_CASE(2, 8, true)
#undef PKV_Q4_CASE
    if (e != cudaSuccess) return e;
    return launch_combine(d, f32, a.part_o, a.part_ml, a.tstart, out, batch, hq, p.ctas, stream);
}

}  // namespace pkv
