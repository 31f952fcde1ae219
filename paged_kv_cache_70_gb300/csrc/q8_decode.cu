// q8_decode.cu -- paged decode (one query token per sequence) over an 8-bit cache.
//
//   out[b,h] = sum_j softmax_j(scale * q[b,h] . k_j) v_j,  j < cache_seqlens[b],
// with k_j, v_j the e4m3 codes times their page's scale (format: q8.cuh), read through
// block table row b and merged by the online-softmax rule ("11. Paged attention 与
// online softmax" §11.1-§11.2).
//
// What bounds it: 2 d bytes per key and KV head (K and V).  At HBM's rate an SM gets a
// key of one head every 12 cycles at d = 128; on the CUDA cores each query head alone
// would need 8 warp instructions of FMAs per key.  So the products run on the tensor
// cores from registers: a lane turns codes into the fp16 operand fragments of
// mma.m16n8k16, two per instruction and exactly, with keys (score) or dims (output) as
// the 16 rows and 8 query heads as the columns.  tcgen05 takes e4m3 as it is, but
// then the queries and the weights have to be e4m3 as well: 4 bits of each.
//
//  * Columns: the query heads of one KV head, 8 per warp (fewer leave columns empty;
//    more: several warps).  Score rows are keys, so that each key's K scale
//    multiplies its row, and weights take their V scale before they are rounded to
//    fp16; an 8x8 transposition per 8 keys turns score tiles into weight operands.
//  * fp32 queries, and the weights that go with them, enter as two fp16 parts (22
//    bits), two products each.
//  * References, one of each per query, moved together when a vote of the warp asks for
//    it: the maximum score m of the weights p = 2^(score - m), and a power of two for
//    p times the V scale, which keeps the fp16 weights between kTarget and kLimit
//    whatever the scales are.
//  * Work split: the tiles of all sequences in one list, cut into equal contiguous
//    shares, one per CTA; each (CTA, sequence) piece leaves a partial state that a
//    second kernel merges (split.cuh).  Two pairs of producer warps bring tiles into
//    a ring of stages, one tiled copy per page piece for all heads of the CTA, 128-byte
//    swizzle (d = 64: 64-byte) so that a fragment's loads touch all banks once; the
//    other warps own a (head, 8 queries) and 16 of the tile's keys each and hold a
//    stage for their loads only.
//    Short sequences (plan_q8_decode) need no second kernel: a CTA takes one, or a
//    cluster shares one and its CTAs read each other's states.
//  * Keys of a page outside the pool are skipped and flagged; rows past the length
//    never enter: scores of -inf, V codes and scales of 0, whatever the page holds
//    there.  Every wait is time-limited.
//
// Measured (bf16 queries, a call among others; of the measured copy rate, 6696 GB/s):
//   8 sequences of 16 K - 41 K keys, 16 / 8 heads, d = 128, 485 MB     77.5 us  0.93
//   the same with 64 / 8 heads                                          78.8 us  0.92
//   64 sequences of 128 - 4096 keys, 16 / 8 heads, B = 16, 278 MB       50.8 us  0.82
//   one of 7777 keys, 32 / 4 heads, d = 64                               8.4 us
// From one to four times the long contexts the time grows by 6980 GB/s, above the copy
// rate.  What stands around the stream: ~5 us to the first copy (wait for the launch, plan,
// table), ~4 us that the SMs' last tiles lie apart, by chance, and ~4 us from the last tile
// to the end (merges, partial states, the second kernel).
#include <algorithm>
#include <atomic>
#include <numeric>

#include "common.cuh"
#include "launch.h"
#include "q8.cuh"
#include "split.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
// Weights are kept below kLimit (fp16 ends at 65504); a moved reference puts the
// largest at 2^kTarget .. 2^(kTarget + 1).  bf16: fp16's 11 bits for weights down to
// 2^-20 of the largest; fp32: the second part has its bits down to 2^-15 of it.
constexpr float kLimit = 32768.f;
template <bool F32>
__host__ __device__ constexpr int target() { return F32 ? 12 : 6; }
// the score's reference moves when a score passes it by 2^grow_by()
template <bool F32>
__host__ __device__ constexpr float grow_by() { return F32 ? 2.f : 8.f; }
constexpr int kProducers = 4;
constexpr int kMaxStages = 8;
constexpr int kMaxCluster = 16;  // (more than 8 have to be asked for)
constexpr int kHeader = 512;  // barriers and stage tags
constexpr size_t kStaticSmem = 1024;  // left for static shared memory
constexpr int kAlign = 1024;  // of the ring: the swizzle's period

// Consumer warps: 12 with the 128 registers that 16 warps leave a thread, 8 with 168
// for the second parts of fp32 queries.
template <bool F32>
__host__ __device__ constexpr int consumers() { return F32 ? 8 : 12; }
template <bool F32>
__host__ __device__ constexpr int threads() { return (consumers<F32>() + kProducers) * 32; }

struct Q8DecodeArgs {
    const void* q;
    const float* ks;
    const float* vs;
    const int32_t* table;
    const int32_t* seqlens;
    float* part_o;     // [ctas + batch][hq][D]
    float* part_ml;    // [ctas + batch][hq][2]
    int32_t* tstart;   // [batch + 1]
    void* out;         // WHOLE, CLUSTER
    unsigned int* err;
    int64_t num_blocks;
    float qscale;  // scale * log2(e)
    int32_t max_blocks, batch, hq, hkv, block_size;
    int32_t hc;      // KV heads per CTA
    int32_t no;      // warps' worth of query heads per KV head
    int32_t wh;      // warps that share a head and its queries (16 of a tile's keys each)
    int32_t piece;   // keys per copy
    int32_t stages;
    int32_t cluster;  // CTAs that share a sequence (CLUSTER)
    FastDiv block, tile;  // by the page size, and by a tile's keys
};

// One stage's description, written by the producer of its K
struct Tag {
    uint32_t partial;  // fewer keys than the tile holds, or a bad page
    int32_t rows;      // keys
    int32_t bad;       // first key's position if a page was out of range, else -1
};

// a warp's merged state in shared memory: D / 4 output values, 2 maxima and 2 sums per
// lane
__host__ __device__ constexpr size_t state_bytes(int d) { return (size_t)(d / 4 + 4) * 128; }

__device__ __forceinline__ void tile_copy(void* dst, const CUtensorMap* map, int y, int z,
                                          uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(smem_u32(bar)),
        "l"(policy)
        : "memory");
}

// transposes an 8x8 matrix of 16-bit values held by a warp, two per lane
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// 2^-i of 2^i, i in -126 .. 126
__device__ __forceinline__ float inverse(float x) {
    return __uint_as_float((254u << 23) - __float_as_uint(x));
}

// The key of MMA row r < 8 of a score tile (rows 8 .. 15: 8 more), and so of k index r
// of the output product.  A quarter of a warp loads 16 bytes of two rows and their
// four lanes (score), or of four rows 2c + i and two chunks (output): the rows are
// chosen so that under the swizzle these are 8 different chunks of the banks (d = 64,
// output: 16 half chunks of half a warp).
template <int D>
__device__ __forceinline__ int row_key(int r) {
    if (D == 128) return (r & 1) ? r ^ 4 : r;
    return (r & 4) | (r & 2 ? (r & 1) + 1 : (r & 1) * 3);
}
// what the swizzle adds to the address of a byte at `off` of the ring
template <int D>
__device__ __forceinline__ uint32_t swizzle(uint32_t off) {
    return D == 128 ? (off >> 3) & 0x70u : (off >> 3) & 0x30u;
}

// the word of shared memory that lies at `at` in CTA `cta` of the cluster
__device__ __forceinline__ uint32_t at_cta(uint32_t at, int cta) {
    uint32_t y;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"(at), "r"(cta));
    return y;
}
__device__ __forceinline__ float4 load_cluster(uint32_t at) {
    float4 y;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w) : "r"(at) : "memory");
    return y;
}
// all threads of the cluster that have not ended
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// What a CTA takes: its share of the line of all tiles, a sequence (and its heads), or
// its part of one that its cluster shares
enum Mode { SPLIT, WHOLE, CLUSTER };

template <int D, bool F32, Mode MODE>
__global__ void __launch_bounds__(threads<F32>(), 1)
q8_split_kernel(const Q8DecodeArgs a, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
    // one sequence, `own`, unless the tiles are SPLIT; part `part` of it
    constexpr bool ONE = MODE != SPLIT;
    const int own = MODE == CLUSTER ? blockIdx.x / a.cluster : ONE ? blockIdx.x : 0;
    const int part = MODE == CLUSTER ? blockIdx.x - own * a.cluster : 0;
    const int batch = ONE ? 1 : a.batch;
    const int32_t* const seqlens = a.seqlens + own;
    const int32_t* const table = a.table + (int64_t)own * a.max_blocks;
    constexpr int WC = consumers<F32>();
    constexpr int PARTS = F32 ? 2 : 1;
    constexpr int KW = D / 16;   // words of K codes per lane and row: 16-dim steps
    constexpr int VW = D / 32;   // words of V codes per lane and row
    constexpr int OT = D / 16;   // output tiles of 16 dims
    extern __shared__ __align__(128) unsigned char smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem);
    uint64_t* empty = full + kMaxStages;
    uint64_t* merge_bar = empty + kMaxStages;  // [2]
    Tag* tags = reinterpret_cast<Tag*>(smem + 256);
    int32_t* tstart = reinterpret_cast<int32_t*>(smem + kHeader);
    unsigned char* scratch = smem + kHeader + up((size_t)(batch + 1) * 4, 128);
    const int units = a.hc * a.no;  // (head, 8 queries) of the CTA
    const int S = a.stages, T = 16 * a.wh, P = a.piece;
    const int pieces = T / P;
    // scales [stage][piece][head]: K's and V's
    float* scales = reinterpret_cast<float*>(
        scratch + (size_t)units * (a.wh - (MODE == CLUSTER ? 0 : 1)) * state_bytes(D));
    unsigned char* ring = reinterpret_cast<unsigned char*>(scales) + (size_t)S * pieces * a.hc * 8;
    ring += (0u - smem_u32(ring)) % kAlign;
    __shared__ int32_t warp_sum[threads<F32>() / 32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t half_bytes = (uint32_t)(a.hc * T * D);  // K (or V) of a stage
    const int active = units * a.wh;  // consumer warps at work
    if (tid < S) {
        mbar_init(&full[tid], 2);  // a K and a V producer
        mbar_init(&empty[tid], active);
    } else if (tid == kMaxStages) {
        mbar_init(&merge_bar[0], units * (a.wh - 1) + 1);
        mbar_init(&merge_bar[1], units);
    }
    fence_barrier_init();
    if (tid >= WC * 32 && tid < WC * 32 + 64 && lane == 0)  // the producers' first K and V maps
        asm volatile("prefetch.tensormap [%0];" ::"l"(
                         reinterpret_cast<uint64_t>(tid == WC * 32 ? &kmap : &vmap))
                     : "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- plan: tile starts of the sequences (an exclusive scan of their tiles)
    const int64_t cap = (int64_t)a.max_blocks * a.block_size;
    const bool first_cta = (ONE ? part == 0 : blockIdx.x == 0) && blockIdx.y == 0;
    {
        // (what comes next, the table, is on its way meanwhile: 64 KB of it at most)
        const int64_t line = (int64_t)tid * 128;
        if (line < (int64_t)batch * a.max_blocks * 4)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                reinterpret_cast<const unsigned char*>(table) + line));
        auto tiles = [&](int b) {
            const int32_t L = __ldg(seqlens + b);
            if (first_cta && (L < 0 || L > cap)) flag_error(a.err, PKV_FLAG_BAD_LENGTH);
            const int32_t n = (int32_t)min((int64_t)max(L, 0), cap);
            return (int32_t)a.tile.quot((uint32_t)(n + T - 1));
        };
        auto scan = [&](int32_t x) {
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off) x += y;
            }
            return x;
        };
        if (ONE || batch <= 32) {  // one warp's work
            if (warp == 0) {
                const int32_t x = scan(lane < batch ? tiles(lane) : 0);
                if (lane < batch) tstart[lane + 1] = x;
                if (lane == 0) tstart[0] = 0;
            }
            __syncthreads();
        } else {
            constexpr int N = threads<F32>();
            const int per = (batch + N - 1) / N;
            const int lo = tid * per, hi = min(lo + per, batch);
            int32_t sum = 0;
            for (int b = lo; b < hi; ++b) {
                tstart[b + 1] = tiles(b);
                sum += tstart[b + 1];
            }
            const int32_t inc = scan(sum);
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
    }
    const int32_t total = tstart[batch];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int head0 = blockIdx.y * a.hc;
    int32_t t0 = 0, t1 = total;
    if constexpr (ONE) {
        if (total == 0) {  // no keys
            const int64_t at = ((int64_t)own * a.hq + head0 * (a.hq / a.hkv)) * D;
            uint32_t* const o = static_cast<uint32_t*>(a.out) + (F32 ? at : at / 2);
            const int words = part == 0 ? a.hc * (a.hq / a.hkv) * D / (F32 ? 1 : 2) : 0;
            for (int i = tid; i < words; i += blockDim.x) o[i] = 0u;
            return;
        }
        if constexpr (MODE == CLUSTER) {
            t0 = (int32_t)((int64_t)total * part / a.cluster);
            t1 = (int32_t)((int64_t)total * (part + 1) / a.cluster);
        }
    } else {
        if (first_cta)  // for the combine, which reads them behind its wait
            for (int b = tid; b <= batch; b += blockDim.x) a.tstart[b] = tstart[b];
        const int32_t len = share_len(total, batch, gridDim.x);
        t0 = share_first(tstart, batch, (int64_t)blockIdx.x * len);
        t1 = share_first(tstart, batch, (int64_t)(blockIdx.x + 1) * len);
        if (t0 >= t1) return;
    }

    if (warp >= WC) {
        // ------------------------------ producers -----------------------------
        // Two pairs of warps take the tiles in turn, one warp of a pair K and the other
        // V.  No more pairs than stages: a warp then has seen its stage's last but one
        // contents consumed (with its own previous tile) before it waits for the last,
        // which a wait on the phase's parity alone could not tell apart.
#ifdef PKV_TEST_SPLIT_PRODUCER_IDLE
        return;  // test-only build: issue nothing, so the consumers' first wait runs out
#endif
        const bool is_v = (warp - WC) & 1;
        const CUtensorMap* map = is_v ? &vmap : &kmap;
        const float* from = is_v ? a.vs : a.ks;
        constexpr int prods = kProducers / 2;
        const uint64_t pol = l2_evict_first_policy();
        const uint32_t inv_hc = 65536u / a.hc + 1;  // i / hc for i < 512, hc <= 16
        const int32_t tf = t0 + (warp - WC) / 2;
        if (tf >= t1) return;
        int b = share_seq(tstart, batch, tf);  // the sequence of tile t
        int32_t L = (int32_t)min((int64_t)max(__ldg(seqlens + b), 0), cap);
        // the page of this lane's piece of the 32 from piece c0 on
        auto fetch = [&](int bb, int32_t p0, int32_t p1, int c0) {
            const int32_t p = p0 + (c0 + lane) * P;
            return c0 + lane < pieces && p < p1
                       ? __ldg(table + (int64_t)bb * a.max_blocks + a.block.quot((uint32_t)p))
                       : -1;
        };
        int32_t p0 = (tf - tstart[b]) * T, p1 = min(L, p0 + T);
        int32_t next_page = fetch(b, p0, p1, 0);  // one tile ahead
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
                    L = (int32_t)min((int64_t)max(__ldg(seqlens + b), 0), cap);
                }
                p0 = (t + prods - tstart[b]) * T;
                p1 = min(L, p0 + T);
                next_page = fetch(b, p0, p1, 0);
            }
            const int32_t k = t - t0;
            const int np = (q1 - q0 + P - 1) / P;  // pieces that hold keys
            // how many of them arrive; the first round's scales
            int good = 0;
            for (int c0 = 0; c0 < np; c0 += 32) {
                const int32_t id = c0 == 0 ? page : fetch(seq, q0, q1, c0);
                good += __popc(__ballot_sync(0xffffffffu, c0 + lane < np && id >= 0 &&
                                                              id < a.num_blocks));
            }
            const bool bad = good < np;
            // the scale of this lane's (piece, head), the first 32 of them before the wait
            auto scale_of = [&](int32_t id32, int c0, int i0, int* at) {
                const int n = min(32, np - c0) * a.hc;
                const int i = min(i0 + lane, n - 1);
                const int p = (int)((i * inv_hc) >> 16), h = i - p * a.hc;
                const int32_t id = __shfl_sync(0xffffffffu, id32, p);
                const bool here = i0 + lane < n && id >= 0 && id < a.num_blocks;
                *at = here ? ((c0 + p) * a.hc + h) * 2 : -1;
                return here ? __ldg(from + (int64_t)id * a.hkv + head0 + h) : 0.f;
            };
            int first_at;
            const float first = scale_of(page, 0, 0, &first_at);
            bool ok = true;
            if (lane == 0) {
                ok = mbar_wait(&empty[s], (fills & 1) ^ 1, a.err);
                if (ok) {
                    if (bad) flag_error(a.err, PKV_FLAG_BAD_BLOCK);
                    if (!is_v) tags[s] = Tag{bad || q1 - q0 < T, q1 - q0, bad ? q0 : -1};
                }
            }
            __syncwarp();
            if (!__all_sync(0xffffffffu, ok)) break;
            last_k = k;
            // the copies first: the scales may still be on their way, and the barrier counts
            // bytes that arrive before they are expected
            unsigned char* dst = ring + (size_t)(2 * s + is_v) * half_bytes;
            for (int c0 = 0; c0 < np; c0 += 32) {
                const int32_t id = c0 == 0 ? page : fetch(seq, q0, q1, c0);
                if (c0 + lane < np && id >= 0 && id < a.num_blocks) {
                    const int32_t p = q0 + (c0 + lane) * P;
                    const int32_t pg = (int32_t)a.block.quot((uint32_t)p);
                    tile_copy(dst + (size_t)(c0 + lane) * a.hc * P * D, map,
                              p - pg * a.block_size, id * a.hkv + head0, &full[s], pol);
                }
            }
            float* to = scales + (size_t)s * pieces * a.hc * 2 + is_v;
            if (first_at >= 0) to[first_at] = first;
            if (np * a.hc > 32)
                for (int c0 = 0; c0 < np; c0 += 32) {
                    const int32_t id32 = c0 == 0 ? page : fetch(seq, q0, q1, c0);
                    for (int i0 = c0 == 0 ? 32 : 0; i0 < min(32, np - c0) * a.hc; i0 += 32) {
                        int at;
                        const float x = scale_of(id32, c0, i0, &at);
                        if (at >= 0) to[at] = x;
                    }
                }
            __syncwarp();
            if (lane == 0)
                mbar_arrive_expect_tx(&full[s], (uint32_t)good * a.hc * P * D);
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
    const int q0 = oct * 8;                         // first query of this warp in its group
    const int nq = min(8, G - q0);                  // queries it has
    const int qh0 = (head0 + hc) * G + q0;          // first query head

    // This lane's places in a stage's K (or V): rows r and r + 8 of the score tile with
    // chunk c, and k indices 2c + i, 2c + 8 + i of the output product with chunk r.
    auto place = [&](int key, int byte) {
        const int pc = key / P;
        const uint32_t off = (uint32_t)(((pc * a.hc + hc) * P + key - pc * P) * D);
        return (off + byte) ^ swizzle<D>(off);
    };
    uint32_t kat[2], vat[4], sat[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int key = 16 * rank + row_key<D>(r) + 8 * h;
        kat[h] = place(key, 16 * c);
        sat[h] = (uint32_t)(key / P * a.hc + hc) * 8;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        vat[i] = half_bytes +
                 place(16 * rank + row_key<D>(2 * c + (i & 1)) + 8 * (i >> 1), D / 8 * r);

    uint32_t qf[PARTS][KW][2];  // score product's columns
    float cq[2];                // from a product to log2 units, for queries 2c, 2c + 1
    float o[OT][4], l[2];
    // references of queries 2c, 2c + 1: of the scores, the same with -inf as 0, and the
    // score that makes it move; of the weights, and the largest weight that set it
    float m[2], mr[2], lim[2], wm[2], tm[2];
    auto clear = [&]() {  // the state of a new piece
#pragma unroll
        for (int i = 0; i < OT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[i] = lim[i] = -INFINITY;
            mr[i] = l[i] = tm[i] = 0.f;
            wm[i] = __uint_as_float(253u << 23);
        }
    };
    auto load_queries = [&](int32_t seq) {
        float x[KW][4];  // of query r: dims 16c + 4w .. + 3 (w >= 4: 64 more)
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[w][e] = 0.f;
        if (r < nq) {
#pragma unroll
            for (int w = 0; w < KW; w += F32 ? 1 : 2) {
                const int64_t at = ((int64_t)(ONE ? own : seq) * a.hq + qh0 + r) * D + 16 * c + (w & 3) * 4 +
                                   (w >= 4 ? 64 : 0);
                if constexpr (F32) {
                    const float4 u =
                        __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at));
                    x[w][0] = u.x; x[w][1] = u.y; x[w][2] = u.z; x[w][3] = u.w;
                } else {
                    const uint4 u = __ldg(
                        reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at));
                    x[w][0] = bf16lo(u.x); x[w][1] = bf16hi(u.x);
                    x[w][2] = bf16lo(u.y); x[w][3] = bf16hi(u.y);
                    x[w + 1][0] = bf16lo(u.z); x[w + 1][1] = bf16hi(u.z);
                    x[w + 1][2] = bf16lo(u.w); x[w + 1][3] = bf16hi(u.w);
                }
            }
        }
        // the query scaled by a power of two to 2^14 .. 2^15: fp16 then holds bf16
        // queries exactly down to 2^-31 of the largest, and two parts hold 22 bits of
        // fp32 ones
        float mx = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(x[w][e]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int ex = (int)(__float_as_uint(mx) >> 23);
        const float up_q = __uint_as_float((uint32_t)min(max(268 - ex, 1), 253) << 23);
        const float down = a.qscale * inverse(up_q);
        cq[0] = __shfl_sync(0xffffffffu, down, 8 * c);
        cq[1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[w][e] *= up_q;
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                qf[part][w][0] = take_f16x2<F32>(x[w][0], x[w][1]);
                qf[part][w][1] = take_f16x2<F32>(x[w][2], x[w][3]);
            }
        }
    };

    int merges = 0;
    // CLUSTER: where this head's and these queries' state of the CTA is left for the others
    float4* const left = reinterpret_cast<float4*>(
        scratch + (size_t)((a.wh - 1) * units + unit) * state_bytes(D));
    bool none = true;
    // (a store of 4 outputs of query 2c + i, D / 8 r + x first)
    auto store4 = [&](int i, int x, float4 y) {
        const int64_t at = ((int64_t)own * a.hq + qh0 + 2 * c + i) * D + D / 8 * r + x;
        if constexpr (F32)
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = y;
        else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
                make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    };
    const int32_t n_tiles = t1 - t0;
    uint32_t full_bar = smem_u32(full), empty_bar = smem_u32(empty);
    asm volatile("" : "+r"(full_bar), "+r"(empty_bar));  // (keep them)
    clear();

    int s = 0;
    uint32_t phase = 0;    // of stage s
    int seq = share_seq(tstart, batch, t0) - 1;  // sequence of tile k
    int32_t next = 0;      // the tile that the next one begins with
    for (int32_t k = 0; k < n_tiles; ++k) {
        if (k == next) {  // (before the wait: the first queries come with the first tile)
            do ++seq; while (tstart[seq + 1] <= t0 + k);
            next = min(tstart[seq + 1] - t0, n_tiles);
            load_queries(seq);
        }
        if (!wait_phase(full_bar + 8 * s, phase, a.err)) break;
        const uint32_t partial = tags[s].partial;
        const unsigned char* tile = ring + (size_t)s * 2 * half_bytes;
        const unsigned char* sc = reinterpret_cast<const unsigned char*>(scales) +
                                  (size_t)s * pieces * a.hc * 8;
        // scores of this lane's keys (rows r, r + 8) and queries (2c, 2c + 1)
        float2 ss[2];  // K scale, V scale
        uint32_t kw[2][KW];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ss[h] = *reinterpret_cast<const float2*>(sc + sat[h]);
#pragma unroll
            for (int x = 0; x < KW; x += 4) {
                const uint4 w = *reinterpret_cast<const uint4*>(tile + (kat[h] ^ (x ? 64u : 0u)));
                kw[h][x] = w.x; kw[h][x + 1] = w.y; kw[h][x + 2] = w.z; kw[h][x + 3] = w.w;
            }
        }
        float acc[2][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][e] = acc[1][e] = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            uint32_t af[4];
            e4m3_f16(kw[0][w], af[0], af[2]);
            e4m3_f16(kw[1][w], af[1], af[3]);
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
                mma(acc[w & 1], af, qf[part][w][0], qf[part][w][1]);
        }
        // the V words, and the stage is given back: it is held for its loads, not for
        // the arithmetic
        uint32_t vw[4][VW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (D == 128) {
                const uint4 w = *reinterpret_cast<const uint4*>(tile + vat[i]);
                vw[i][0] = w.x; vw[i][1] = w.y; vw[i][VW - 2] = w.z; vw[i][VW - 1] = w.w;
            } else {
                const uint2 w = *reinterpret_cast<const uint2*>(tile + vat[i]);
                vw[i][0] = w.x; vw[i][1] = w.y;
            }
        }
        float p[2][2];  // [key row][query]
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                p[h][i] = (acc[0][2 * h + i] + acc[1][2 * h + i]) * (cq[i] * ss[h].x);
        if (__builtin_expect(partial, 0)) {  // keys that do not count
            const Tag tag = tags[s];
            auto valid = [&](int key) {
                const int at = rank * 16 + key;
                if (at >= tag.rows) return false;
                if (tag.bad < 0) return true;
                const int32_t id = __ldg(table + (int64_t)seq * a.max_blocks +
                                         (tag.bad + at) / a.block_size);
                return id >= 0 && id < a.num_blocks;
            };
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (!valid(row_key<D>(r) + 8 * h)) {
                    p[h][0] = p[h][1] = -INFINITY;
                    ss[h].y = 0.f;
                }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (!valid(row_key<D>(2 * c + (i & 1)) + 8 * (i >> 1)))
#pragma unroll
                    for (int w = 0; w < VW; ++w) vw[i][w] = 0u;
        }
        const bool ends = k + 1 == next;
        __syncwarp();
        if (lane == 0) arrive(empty_bar + 8 * s);
        float w[2][2];
        bool grow = false;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x = p[h][i];
                const float e = ex2(x - mr[i]);
                w[h][i] = e * (ss[h].y * wm[i]);
                // (no number either: a weight of 0 times a scale that overflows here)
                grow |= x > lim[i] || !(fabsf(w[h][i]) <= kLimit);
                acc[h][i] = e;  // (scores stay in p: they are needed if the references move)
            }
        if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float mx = fmaxf(p[0][i], p[1][i]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                const float mn = fmaxf(m[i], mx);
                const float f = m[i] == -INFINITY ? 0.f : ex2(m[i] - mn);
                m[i] = mn;
                mr[i] = mn == -INFINITY ? 0.f : mn;
                lim[i] = mn + grow_by<F32>();
                l[i] *= f;
                // the largest weight with its V scale (those that are no numbers make
                // their own output NaN, and are no reference for others)
                float t = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    acc[h][i] = ex2(p[h][i] - mr[i]);
                    const float x = fabsf(acc[h][i] * ss[h].y);
                    t = fmaxf(t, x < INFINITY ? x : 0.f);
                }
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
                tm[i] = fmaxf(tm[i] * f, t);
                const float was = wm[i];
                const int te = (int)(__float_as_uint(tm[i]) >> 23);
                wm[i] = __uint_as_float((uint32_t)min(max(254 + target<F32>() - te, 1), 253) << 23);
                const float fo = f * inverse(was) * wm[i];
#pragma unroll
                for (int x = 0; x < OT; ++x) {
                    o[x][i] *= fo;
                    o[x][2 + i] *= fo;
                }
#pragma unroll
                // (in this order: scale and reference by themselves may pass fp32's range)
                for (int h = 0; h < 2; ++h) w[h][i] = acc[h][i] * ss[h].y * wm[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) l[i] += acc[0][i] + acc[1][i];
        uint32_t wf[PARTS][2];
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                wf[part][h] = transpose8(take_f16x2<F32>(w[h][0], w[h][1]));
#pragma unroll
        for (int x = 0; x < VW; ++x) {
            // codes of two keys side by side, two dims per word
            const uint32_t e0 = __byte_perm(vw[0][x], vw[1][x], 0x5140);
            const uint32_t e1 = __byte_perm(vw[0][x], vw[1][x], 0x7362);
            const uint32_t f0 = __byte_perm(vw[2][x], vw[3][x], 0x5140);
            const uint32_t f1 = __byte_perm(vw[2][x], vw[3][x], 0x7362);
            uint32_t af[4];
            e4m3_f16(e0, af[0], af[1]);
            e4m3_f16(f0, af[2], af[3]);
#pragma unroll
            for (int part = 0; part < PARTS; ++part) mma(o[2 * x], af, wf[part][0], wf[part][1]);
            e4m3_f16(e1, af[0], af[1]);
            e4m3_f16(f1, af[2], af[3]);
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
                mma(o[2 * x + 1], af, wf[part][0], wf[part][1]);
        }
        if (++s == S) {
            s = 0;
            phase ^= 1;
        }
        if (!ends) continue;

        // ---- end of the piece: this warp's state; output tile x holds dims
        // D / 8 r + 2x and + 2x + 1 of queries 2c, 2c + 1
        float val[2][D / 8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
            if (l[i] != l[i] && m[i] == -INFINITY) m[i] = 0.f;  // every score a NaN
            const float f = inverse(wm[i]);
#pragma unroll
            for (int x = 0; x < OT; ++x) {
                val[i][2 * x] = o[x][i] * f;
                val[i][2 * x + 1] = o[x][2 + i] * f;
            }
        }
        float m2[2] = {m[0], m[1]}, l2[2] = {l[0], l[1]};
        clear();
        if (a.wh > 1) {  // the warps of this head and queries: rank 0 merges
            if (rank > 0) {
                if (merges > 0 &&
                    !__all_sync(0xffffffffu, mbar_wait(&merge_bar[1], (merges - 1) & 1, a.err)))
                    break;
                float4* y = reinterpret_cast<float4*>(
                    scratch + (size_t)((rank - 1) * units + unit) * state_bytes(D));
                y[lane] = make_float4(m2[0], m2[1], l2[0], l2[1]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int x = 0; x < D / 8; x += 4)
                        y[(1 + i * (D / 32) + x / 4) * 32 + lane] =
                            make_float4(val[i][x], val[i][x + 1], val[i][x + 2], val[i][x + 3]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&merge_bar[0]);
            } else {
                if (unit == 0 && lane == 0) mbar_arrive(&merge_bar[0]);
                if (!__all_sync(0xffffffffu, mbar_wait(&merge_bar[0], merges & 1, a.err))) break;
                for (int wv = 1; wv < a.wh; ++wv) {
                    const float4* y = reinterpret_cast<const float4*>(
                        scratch + (size_t)((wv - 1) * units + unit) * state_bytes(D));
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
                        for (int x = 0; x < D / 8; x += 4) {
                            const float4 z = y[(1 + i * (D / 32) + x / 4) * 32 + lane];
                            val[i][x] = val[i][x] * ca + z.x * cb;
                            val[i][x + 1] = val[i][x + 1] * ca + z.y * cb;
                            val[i][x + 2] = val[i][x + 2] * ca + z.z * cb;
                            val[i][x + 3] = val[i][x + 3] * ca + z.w * cb;
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&merge_bar[1]);
            }
            ++merges;
        }
        if (rank != 0) continue;
        if constexpr (MODE == WHOLE) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (2 * c + i >= nq) continue;
                const float inv = l2[i] == 0.f ? 0.f : 1.f / l2[i];
#pragma unroll
                for (int x = 0; x < D / 8; x += 4)
                    store4(i, x, make_float4(val[i][x] * inv, val[i][x + 1] * inv,
                                             val[i][x + 2] * inv, val[i][x + 3] * inv));
            }
            continue;
        }
        if constexpr (MODE == CLUSTER) {
            left[lane] = make_float4(m2[0], m2[1], l2[0], l2[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int x = 0; x < D / 8; x += 4)
                    left[(1 + i * (D / 32) + x / 4) * 32 + lane] =
                        make_float4(val[i][x], val[i][x + 1], val[i][x + 2], val[i][x + 3]);
            none = false;
            continue;
        }
        const int64_t slot = (int64_t)blockIdx.x + seq;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (2 * c + i >= nq) continue;
            const int64_t at = slot * a.hq + qh0 + 2 * c + i;
#pragma unroll
            for (int x = 0; x < D / 8; x += 4)
                *reinterpret_cast<float4*>(a.part_o + at * D + D / 8 * r + x) =
                    make_float4(val[i][x], val[i][x + 1], val[i][x + 2], val[i][x + 3]);
            if (r == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(m2[i], l2[i]);
        }
    }
    if constexpr (MODE == CLUSTER) {
        // The parts' states, merged: piece q (4 values per lane) of a head and its queries by
        // the q-th CTA of the cluster.  Every warp that has work comes here, after a wait that
        // ran out too.
        if (rank == 0 && none) {  // no tile was this CTA's
            left[lane] = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
            for (int q = 0; q < D / 16; ++q) left[(1 + q) * 32 + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        cluster_sync();
        const uint32_t here = smem_u32(left + lane);
        for (int q = part + a.cluster * rank; q < D / 16; q += a.cluster * a.wh) {
            const int i = q / (D / 32);
            float M = -INFINITY, L = 0.f;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int j0 = 0; j0 < a.cluster; j0 += 8) {
                float4 y[8];
                float mj[8], lj[8], top = M;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    mj[j] = -INFINITY;
                    if (j0 + j >= a.cluster) continue;
                    const uint32_t there = at_cta(here, j0 + j);
                    const float4 st = load_cluster(there);
                    mj[j] = i ? st.y : st.x;
                    lj[j] = i ? st.w : st.z;
                    y[j] = load_cluster(there + (1 + q) * 512);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, mj[j]);
                const float f0 = M == -INFINITY ? 0.f : ex2(M - top);
                M = top;
                L *= f0;
                sum = make_float4(sum.x * f0, sum.y * f0, sum.z * f0, sum.w * f0);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (mj[j] == -INFINITY) continue;  // (no key)
                    const float f = ex2(mj[j] - M);
                    L += lj[j] * f;
                    sum.x += y[j].x * f;
                    sum.y += y[j].y * f;
                    sum.z += y[j].z * f;
                    sum.w += y[j].w * f;
                }
            }
            const float inv = L == 0.f ? 0.f : 1.f / L;
            if (2 * c + i < nq)
                store4(i, 4 * (q % (D / 32)),
                       make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv));
        }
        cluster_sync();  // (no CTA ends while its state is read)
    }
}

// How many clusters of n CTAs, each with an SM to itself, fit on the GPU (its SMs lie in
// groups of unequal size that no cluster spans).  Asked once per device and n.
int clusters_that_fit(const DeviceInfo& dev, int n) {
    static std::atomic<int> known[64][kMaxCluster + 1];  // 1 more than the answer
    std::atomic<int>& fit = known[dev.device & 63][n];
    if (const int k = fit.load(std::memory_order_relaxed)) return k - 1;
    auto kern = q8_split_kernel<128, false, CLUSTER>;
    const int smem = (int)(dev.max_smem_optin - kStaticSmem);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(threads<false>());
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)n, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int k = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&k, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    fit.store(k + 1, std::memory_order_relaxed);
    return k;
}

template <int D, bool F32, Mode MODE>
cudaError_t launch_split(const DeviceInfo& dev, const Q8DecodePlan& p, const Q8DecodeArgs& a,
                         const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
    auto kern = q8_split_kernel<D, F32, MODE>;
    // the most shared memory a CTA may have, set once per device
    static std::atomic<uint64_t> set{0};
    const uint64_t bit = 1ull << dev.device;
    if (!(set.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
            (int)(dev.max_smem_optin - kStaticSmem));
        if (e != cudaSuccess) return e;
        if (MODE == CLUSTER) {
            const cudaError_t f =
                cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (f != cudaSuccess) return f;
        }
        set.fetch_or(bit, std::memory_order_relaxed);
    }
    if (MODE == CLUSTER)
        return launch_clusters(kern, p.cluster, dim3(a.batch * p.cluster, p.head_groups),
                               dim3(threads<F32>()), p.smem_bytes, stream, a, kmap, vmap);
    return launch_dependent(kern, dim3(MODE == WHOLE ? a.batch : p.ctas, p.head_groups),
                            dim3(threads<F32>()), p.smem_bytes, stream, a, kmap, vmap);
}

// the pool as (dim, token, page and head), boxes of `piece` tokens of `hc` heads
bool pool_map(CUtensorMap* map, const void* pool, int64_t num_blocks, int hkv, int block_size,
              int d, int piece, int hc) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int64_t heads = std::max<int64_t>(num_blocks, 1) * hkv;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)block_size, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)d, (cuuint64_t)block_size * d};
    cuuint32_t box[3] = {(cuuint32_t)d, (cuuint32_t)piece, (cuuint32_t)hc};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(pool), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool plan_q8_decode(const DeviceInfo& dev, int32_t batch, int32_t max_blocks, int hq, int hkv,
                    int d, int block_size, int64_t num_blocks, int q_dtype, Q8DecodePlan* p) {
    if ((d != 64 && d != 128) || batch > kDecodeMaxBatch) return false;
    // positions, and a tile beyond, in 32 bits; pages and heads too (a copy's coordinate)
    if ((double)max_blocks * block_size > 2147483647.0 - 4096) return false;
    if ((double)num_blocks * hkv > 2147483647.0) return false;
    // rows of 64 bytes: copies land on 128 bytes when they hold an even number
    if (d == 64 && block_size % 2) return false;
    const bool f32 = q_dtype == PKV_F32;
    const int G = hq / hkv, wc = f32 ? consumers<true>() : consumers<false>();
    p->no = (G + 7) / 8;
    if (p->no > wc) return false;
    // KV heads per CTA: the most, up to 6 warps' worth, that keep four fifths of the
    // consumers at work; the warps left over share a head's keys
    p->hc = 1;
    auto at_work = [&](int h) { return wc / (h * p->no) * (h * p->no); };
    for (int h = 1; h <= hkv && h * p->no <= std::max(6, p->no); ++h)
        if (hkv % h == 0 && (5 * at_work(h) >= 4 * wc || at_work(h) > at_work(p->hc))) p->hc = h;
    // what follows from the heads of a CTA and from the CTAs of a cluster
    const size_t room = dev.max_smem_optin - kStaticSmem - kAlign;
    auto shape = [&](int hc, int cluster) {
        const int units = hc * p->no;
        p->hc = hc;
        p->cluster = cluster;
        p->head_groups = hkv / hc;
        p->wh = wc / units;
        p->tile = 16 * p->wh;
        p->piece = std::gcd(p->tile, block_size);
        const size_t stage = (size_t)2 * hc * p->tile * d;
        const size_t stage_scales = (size_t)p->tile / p->piece * hc * 8;
        const size_t fixed = kHeader + up((size_t)(batch + 1) * 4, 128) +
                             (size_t)units * (p->wh - (cluster > 1 ? 0 : 1)) * state_bytes(d);
        if (room < fixed + 2 * (stage + stage_scales)) return false;
        p->stages = (int)std::min<size_t>(kMaxStages, (room - fixed) / (stage + stage_scales));
        p->smem_bytes = fixed + p->stages * (stage + stage_scales) + kAlign;
        return true;
    };
    if (hkv / p->hc > 65535 || !shape(p->hc, 0)) return false;
    // one CTA per SM, no more than there can be tiles
    const int64_t tiles = ((int64_t)max_blocks * block_size + p->tile - 1) / p->tile * batch;
    const int64_t most = std::max(1, dev.num_sms / p->head_groups);
    if (tiles + batch > 0x7fffffffLL - most) return false;  // the line of tiles is 32 bits long
    p->ctas = (int)std::max<int64_t>(1, std::min(most, tiles));
    const size_t slots = (size_t)most + batch;  // whatever the table's width is
    p->ws_bytes = up((size_t)(batch + 1) * 4, 256) + up(slots * hq * 2 * 4, 256) +
                  up(slots * hq * d * 4, 256);
    // Sequences that the table keeps short enough need no second kernel: a cluster shares each
    // (and its heads), or one CTA takes it.
    const Q8DecodePlan split = *p;
    const double head_bytes = (double)max_blocks * block_size * 2 * d;  // a sequence's of one head
    // The clusters that put most SMs to work, all of them at once; 16 CTAs where 8 would have 40 KB
    // each or more (32 / 4 heads of 64, 8 and 16: 1000 keys 6.3 and 6.8 us, 6000 8.3 and 7.4).
    int hc = 1, cluster = 0;
    int64_t ctas = 0;
    for (int n = 2; n <= kMaxCluster; n *= 2) {
        const int64_t fit = clusters_that_fit(dev, n);
        for (int h = 1; h <= split.hc; ++h) {
            const int64_t m = (int64_t)batch * (hkv / h);
            if (hkv % h == 0 && m <= fit && m * n > ctas && (n <= 8 || head_bytes * h >= 320e3)) {
                hc = h;
                cluster = n;
                ctas = m * n;
            }
        }
    }
    // One CTA: up to 4 tiles, more where that puts most SMs to work, and no more than 150 KB where
    // there are SMs to share them.  At 16 / 8 heads, d = 128, 48 keys per tile, one CTA and a
    // cluster of 8 (4): one sequence of 20 keys 4.8 and 7.1 us, 140 6.6 and 7.3, 190 7.5 and 7.4;
    // 16 of 190 keys 7.7 and 7.2, 60 of 190 9.0 and (split) 14.1, of 700 23.5 and 23.7; at 4 / 1
    // heads one of 250 keys 7.0 and 7.0, 700 8.5 and 6.8.
    const int64_t whole = (int64_t)batch * split.head_groups;
    if (tiles <= (4 + 12 * whole / dev.num_sms) * batch && whole <= dev.num_sms &&
        (ctas < 4 * whole || head_bytes * split.hc <= 150e3)) {
        p->cluster = 1;
        return true;
    }
    // A cluster: where the second kernel costs more (1.6 us and the longer the more sequences it
    // has, or 70 KB and 3 KB each of what an SM streams) than SMs without work do.  The lengths
    // are not known here, and the figures are of sequences that fill the table; one long among
    // short ones is better split (one of 8000 and three of 100 keys 15.4 us, split 13.2).  At
    // 16 / 8 heads, d = 128, cluster and split: one sequence of 1000 keys
    // 7.3 and 8.5 us, 4000 9.1 and 9.1, 8000 12.1 and 10.4; 4 of 2000 9.5 and 10.9, of 16000 29.2
    // and 29.4; 16 of 300 7.9 and 10.0, of 2000 18.0 and 20.0; at 32 / 4 heads of 64 one of 12000
    // 8.8 and 9.8, of 16000 10.4 and 9.8, 16 of 1000 7.9 and 11.5.
    if (ctas == 0 ||
        head_bytes * hc / cluster * (1 - (double)ctas / dev.num_sms) > 70e3 + 3e3 * batch ||
        !shape(hc, cluster))
        *p = split;
    return true;
}

cudaError_t launch_q8_decode(const DeviceInfo& dev, const Q8DecodePlan& p, const void* q,
                             const void* k_cache, const void* v_cache, const float* k_scale,
                             const float* v_scale, const int32_t* table, int32_t max_blocks,
                             const int32_t* seqlens, int32_t batch, float scale, void* out,
                             void* workspace, int hq, int hkv, int d, int block_size,
                             int64_t num_blocks, int q_dtype, unsigned int* err,
                             cudaStream_t stream) {
    if (batch == 0) return cudaSuccess;
    Q8DecodeArgs a{};
    a.q = q;
    a.ks = k_scale;
    a.vs = v_scale;
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
    a.piece = p.piece;
    a.stages = p.stages;
    a.cluster = p.cluster;
    a.block = FastDiv((uint32_t)block_size);
    a.tile = FastDiv((uint32_t)p.tile);
    CUtensorMap kmap, vmap;
    if (!pool_map(&kmap, k_cache, num_blocks, hkv, block_size, d, p.piece, p.hc) ||
        !pool_map(&vmap, v_cache, num_blocks, hkv, block_size, d, p.piece, p.hc))
        return cudaErrorInvalidValue;
    a.out = out;
    const bool f32 = q_dtype == PKV_F32;
    cudaError_t e = cudaErrorInvalidValue;
#define PKV_Q8_CASE(DD, FF)                                                         \
    if (d == DD && f32 == FF)                                                       \
        e = p.cluster > 1 ? launch_split<DD, FF, CLUSTER>(dev, p, a, kmap, vmap, stream) \
            : p.cluster   ? launch_split<DD, FF, WHOLE>(dev, p, a, kmap, vmap, stream)   \
                          : launch_split<DD, FF, SPLIT>(dev, p, a, kmap, vmap, stream);
    PKV_Q8_CASE(128, false) PKV_Q8_CASE(128, true) PKV_Q8_CASE(64, false) PKV_Q8_CASE(64, true)
#undef PKV_Q8_CASE
    if (e != cudaSuccess || p.cluster) return e;
    return launch_combine(d, f32, a.part_o, a.part_ml, a.tstart, out, batch, hq, p.ctas, stream);
}

}  // namespace pkv
