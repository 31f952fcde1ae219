// q8_cache.cu -- rows into and out of 8-bit K/V pools (format: q8.cuh).
//
// Write: the new rows that fall into one page, with the largest finite magnitude a of a
// head's values among them (K after its rotation, rope.cuh), need the least power of
// two n >= 2^-100 with a <= 448 n.  If they begin the page, its scale is n; else it is
// s = max(n, the old scale, rounded up to a power of two), and the codes of the rows in
// front of them become e4m3(code * (old / s)): a shift of the exponent, which is exact
// until a code gets below 2^-6.  New codes are e4m3(x / s).  A power of two makes both
// divisions exact, so that a value is rounded once.  Tokens of one page follow one
// another in the list (a run), with rows that are not written between them or not; a run is
// found by its first token, which differs in sequence or page from the last one before it
// that has a place.
//
// What bounds it: bytes for long runs, the chain token -> page -> rows -> angles for
// single tokens.  A CTA looks at 256 tokens at once, one per thread, for one head of K or
// V, and takes every `parts`-th of the runs that begin among them: a warp each, or, runs
// of more rows than a warp holds, a team of two or of all.  Rows stay in shared memory
// from the load over the maximum to the store, so that they are read once (runs of more
// rows than a CTA holds: twice).  A thread copies there (cp.async) what it reads itself:
// no barrier but those of the maximum, and no registers for rows in flight.  Keys are put
// back rotated, bf16 ones in 16 bits that round to the same code.
//
// Measured: 16,729 tokens of 16 / 8 heads of 128, bf16, rotated, into pages of 256, 250 MB
// with the queries: 54 us (4630 GB/s, 0.69 of the measured copy rate; pages of 16 48 us, of
// 64 57).  The values alone, without rotation and queries, take 36 of them: CTAs that start
// together load together and then compute together, so that the time is the sum of both,
// and much of the instructions is not the arithmetic's.  A run that tokens without a place
// stand within is looked up row by row: with 5 % of them anywhere among these rows 97 us.
// 64 single tokens: 4 us beyond an empty graph, 256 8; 64 and 448 padding rows behind them 6.
// Read: row n of the outputs is code * scale at slot_mapping[n], in fp32 and then in the
// output's type; zeros for a negative slot.  34,567 rows of 8 x 128 to bf16, 212.5 MB: 33.0
// us, 6440 GB/s (0.96 of the measured copy rate).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "launch.h"
#include "q8.cuh"
#include "rope.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 8;  // per CTA of the write
// row steps that a CTA holds in shared memory, 8 KiB each (fp32: 16): 64 KiB, so that
// three CTAs share an SM
template <bool F32>
__host__ __device__ constexpr int most_steps() { return F32 ? 4 : 8; }
template <bool F32>
__host__ __device__ constexpr int step_bytes() { return kWarps * 32 * (F32 ? 64 : 32); }

struct Q8WriteArgs {
    const void* k;
    const void* v;
    int64_t k_stride, v_stride;  // elements from token to token
    NewTokens tok;
    unsigned char* kc;
    unsigned char* vc;
    float* ks;
    float* vs;
    RopeTable table;
    RopeQuery q;
    uint64_t kv_step;   // CTAs of K and V per CTA while there are any, in 2^-32
    uint32_t kv_ctas;   // the others take the queries
    int32_t steps;      // row steps held
    int32_t parts;      // CTAs that share the runs of kWarps * 32 tokens
    unsigned int* err;
};

// the least power of two n >= 2^-100 with a <= 448 n = 1.75 * 2^8 n
__device__ __forceinline__ float scale_for(float a) {
    const uint32_t b = __float_as_uint(a);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)max(e, 27) << 23);
}
// the least power of two >= a scale, NaN if it is none that a page may have
__device__ __forceinline__ float scale_up(float s) {
    if (!(s >= 0.f && s <= 8.507059173e37f)) return __uint_as_float(0x7fffffffu);  // 2^126
    return __uint_as_float((__float_as_uint(s) + 0x7fffffu) & 0x7f800000u);
}

// x and y cut to bf16, with the last bit set where something was cut off
__device__ __forceinline__ uint32_t odd_bf16x2(float x, float y) {
    const uint32_t lo = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x5410);
    const uint32_t hi = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
    uint32_t some;
    asm("min.u16x2 %0, %1, %2;" : "=r"(some) : "r"(lo), "r"(0x00010001u));
    return hi | some;
}

// the largest magnitude of 16 bf16, NaNs aside
__device__ __forceinline__ float largest_bf16(const uint4& a, const uint4& b) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %1;\n\tmax.bf16x2 %0, %0, t;\n\t}" : "+r"(m) : "r"(w[i]));
    return fmaxf(bf16lo(m), bf16hi(m));
}

// A thread's unit in shared memory: pieces of 16 bytes, kPiece apart, at `slot`
constexpr int kPiece = kWarps * 32 * 16;
template <bool F32>
__device__ __forceinline__ void stage_unit(uint32_t slot, const unsigned char* a,
                                           const unsigned char* b) {
    constexpr int C = F32 ? 4 : 2;
#pragma unroll
    for (int j = 0; j < C; ++j)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + j * kPiece),
                     "l"((j < C / 2 ? a : b) + (j % (C / 2)) * 16)
                     : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
    return w;
}
__device__ __forceinline__ void sts16(uint32_t at, uint4 w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w.x), "r"(w.y),
                 "r"(w.z), "r"(w.w)
                 : "memory");
}
template <bool F32>
__device__ __forceinline__ RawUnit<F32> staged_unit(uint32_t slot) {
    constexpr int C = F32 ? 4 : 2;
    RawUnit<F32> x;
#pragma unroll
    for (int j = 0; j < C; ++j) (j < C / 2 ? x.a[j % (C / 2)] : x.b[j % (C / 2)]) = lds16(slot + j * kPiece);
    return x;
}
template <bool F32>
__device__ __forceinline__ void restage_unit(uint32_t slot, const RawUnit<F32>& x) {
    constexpr int C = F32 ? 4 : 2;
#pragma unroll
    for (int j = 0; j < C; ++j) sts16(slot + j * kPiece, j < C / 2 ? x.a[j % (C / 2)] : x.b[j % (C / 2)]);
}

// four pairs, rotated; the largest magnitude
__device__ __forceinline__ float rotate4(float* a, float* b, const float4& c, const float4& s) {
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float r = __fsub_rn(__fmul_rn(a[i], cc[i]), __fmul_rn(b[i], ss[i]));
        b[i] = __fadd_rn(__fmul_rn(b[i], cc[i]), __fmul_rn(a[i], ss[i]));
        a[i] = r;
        m = fmax3(m, fabsf(a[i]), fabsf(b[i]));
    }
    return m;
}
// Half j of a unit's pairs, rotated in place (as rotate_unit does, in half the registers;
// bf16: to odd); the largest magnitude
template <bool F32, bool MIX>
__device__ __forceinline__ float rotate_half(RawUnit<F32>& x, int j, const float4& c,
                                             const float4& s) {
    float a[4], b[4], m;
    if constexpr (F32 && MIX) {  // pairs are neighbours, in chunk a (j = 0) or b
        uint4* const w = j ? x.b : x.a;
        float f[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[4 * i] = __uint_as_float(w[i].x);
            f[4 * i + 1] = __uint_as_float(w[i].y);
            f[4 * i + 2] = __uint_as_float(w[i].z);
            f[4 * i + 3] = __uint_as_float(w[i].w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = f[2 * i];
            b[i] = f[2 * i + 1];
        }
        m = rotate4(a, b, c, s);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = make_uint4(__float_as_uint(a[2 * i]), __float_as_uint(b[2 * i]),
                              __float_as_uint(a[2 * i + 1]), __float_as_uint(b[2 * i + 1]));
    } else if constexpr (F32) {  // piece j of chunk a with piece j of chunk b
        uint4 &u = x.a[j], &v = x.b[j];
        a[0] = __uint_as_float(u.x); a[1] = __uint_as_float(u.y);
        a[2] = __uint_as_float(u.z); a[3] = __uint_as_float(u.w);
        b[0] = __uint_as_float(v.x); b[1] = __uint_as_float(v.y);
        b[2] = __uint_as_float(v.z); b[3] = __uint_as_float(v.w);
        m = rotate4(a, b, c, s);
        u = make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]),
                       __float_as_uint(a[3]));
        v = make_uint4(__float_as_uint(b[0]), __float_as_uint(b[1]), __float_as_uint(b[2]),
                       __float_as_uint(b[3]));
    } else if constexpr (MIX) {
        uint4& u = j ? x.b[0] : x.a[0];
        a[0] = bf16lo(u.x); b[0] = bf16hi(u.x);
        a[1] = bf16lo(u.y); b[1] = bf16hi(u.y);
        a[2] = bf16lo(u.z); b[2] = bf16hi(u.z);
        a[3] = bf16lo(u.w); b[3] = bf16hi(u.w);
        m = rotate4(a, b, c, s);
        u = make_uint4(odd_bf16x2(a[0], b[0]), odd_bf16x2(a[1], b[1]), odd_bf16x2(a[2], b[2]),
                       odd_bf16x2(a[3], b[3]));
    } else {
        uint32_t &u0 = j ? x.a[0].z : x.a[0].x, &u1 = j ? x.a[0].w : x.a[0].y;
        uint32_t &v0 = j ? x.b[0].z : x.b[0].x, &v1 = j ? x.b[0].w : x.b[0].y;
        a[0] = bf16lo(u0); a[1] = bf16hi(u0); a[2] = bf16lo(u1); a[3] = bf16hi(u1);
        b[0] = bf16lo(v0); b[1] = bf16hi(v0); b[2] = bf16lo(v1); b[3] = bf16hi(v1);
        m = rotate4(a, b, c, s);
        u0 = odd_bf16x2(a[0], a[1]);
        u1 = odd_bf16x2(a[2], a[3]);
        v0 = odd_bf16x2(b[0], b[1]);
        v1 = odd_bf16x2(b[2], b[3]);
    }
    return m;
}
// the largest magnitude of a unit, NaNs aside
__device__ __forceinline__ float largest(const RawUnit<false>& x) {
    return largest_bf16(x.a[0], x.b[0]);
}
__device__ __forceinline__ float largest(const RawUnit<true>& r) {
    float x[16], m = 0.f;
    widen_unit<true>(r, x);
#pragma unroll
    for (int e = 0; e < 16; e += 2) m = fmax3(m, fabsf(x[e]), fabsf(x[e + 1]));
    return m;
}

// The runs (the tokens of one sequence on one page) that begin at tokens n0 .. n0 + 255, a
// CTA's window.  Tokens without a place (padding, a sequence or position past the table) are
// passed over: those in front of and behind them are one run, since two that had a page
// between them would both set its scale and shift its codes, at the same time.
constexpr int kWindow = kWarps * 32;
constexpr int kFar = 8 * kWindow;  // tokens that are looked at at once behind it
struct Runs {
    // tokens that begin a run, and that go on with the run of the one directly before them
    uint32_t starts[kWarps], goes_on[kWarps];
    // tokens behind the window: those that go on with its last run; others that have a place
    uint32_t behind[kFar / 32], other[kFar / 32];
    int32_t first[kWindow], page[kWindow];  // of each run (page below 0: not in the pool)
    int32_t len[kWindow];                   // tokens to its last, those passed over as well
    bool gaps[kWindow];                     // some were passed over
    bool open;                              // the last run may go on farther behind
    // where tokens are passed over: the window's, and which of them have a place
    int32_t seq[kWindow], pos[kWindow];
    uint32_t placed[kWarps];
};

// of `words`: how many bits from `at` on are set without a gap; the first one set from `at`
// on (N: none); the last one set below `end` (-1: none)
template <int N>
__device__ __forceinline__ int bits_from(const uint32_t* words, int at) {
    int end = at;
    while (end < N) {
        const uint32_t rest = ~words[end >> 5] >> (end & 31);
        if (rest) return end + __ffs(rest) - 1 - at;
        end = (end | 31) + 1;
    }
    return N - at;
}
template <int N>
__device__ __forceinline__ int first_from(const uint32_t* words, int at) {
    while (at < N) {
        const uint32_t rest = words[at >> 5] >> (at & 31);
        if (rest) return at + __ffs(rest) - 1;
        at = (at | 31) + 1;
    }
    return N;
}
__device__ __forceinline__ int last_below(const uint32_t* words, int end) {
    while (end > 0) {
        const uint32_t rest = words[(end - 1) >> 5] << (31 - ((end - 1) & 31));
        if (rest) return end - 1 - __clz(rest);
        end = (end - 1) & ~31;
    }
    return -1;
}

__device__ __forceinline__ int32_t block_of(const NewTokens& t, int32_t p) {
    return (int32_t)t.block.quot((uint32_t)max(p, 0));
}
__device__ __forceinline__ bool has_place(const NewTokens& t, int32_t s, int32_t p) {
    return s >= 0 && s < t.num_seqs && p >= 0 && block_of(t, p) < t.max_blocks;
}
// sequence and position of token m, -1 where there is none
__device__ __forceinline__ void load_token(const NewTokens& t, int64_t m, int32_t& s, int32_t& p) {
    s = p = -1;
    if (m >= 0 && m < t.num) {
        s = __ldg(t.seq + m);
        p = __ldg(t.pos + m);
    }
}
// how many runs begin in the window, and the number of the one that this thread's token would
// begin
__device__ __forceinline__ int count_runs(const Runs* w, int* k) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int total = 0;
    *k = __popc(w->starts[warp] & ((1u << lane) - 1));
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const int m = __popc(w->starts[i]);
        total += m;
        *k += i < warp ? m : 0;
    }
    return total;
}

// The same over the words of kFar tokens, by a warp: the first bit set of words ^ flip, and the
// last one set below `end`
__device__ __forceinline__ int first_of_far(const uint32_t* words, uint32_t flip) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kFar / 1024; ++i) {
        const uint32_t x = words[32 * i + lane] ^ flip;
        const uint32_t some = __ballot_sync(0xffffffffu, x != 0);
        if (some) {
            const int at = __ffs(some) - 1;
            return 1024 * i + 32 * at + __ffs(__shfl_sync(0xffffffffu, x, at)) - 1;
        }
    }
    return kFar;
}
__device__ __forceinline__ int last_of_far(const uint32_t* words, int end) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = kFar / 1024 - 1; i >= 0; --i) {
        const int left = end - 1024 * i - 32 * lane;  // bits of this lane's word below `end`
        uint32_t x = left > 0 ? words[32 * i + lane] : 0;
        if (left > 0 && left < 32) x &= (1u << left) - 1;
        const uint32_t some = __ballot_sync(0xffffffffu, x != 0);
        if (some) {
            const int at = 31 - __clz(some);
            return 1024 * i + 32 * at + 31 - __clz(__shfl_sync(0xffffffffu, x, at));
        }
    }
    return -1;
}

// Length and gaps of the window's last run, number `run`, that may go on behind the window.
// (Rare, as what follows: kept out of the registers of what runs every time.)
__device__ __noinline__ void follow_run(const NewTokens& t, int64_t n0, int run, Runs* w) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t from = n0 + w->first[run];
    const int32_t sl = __ldg(t.seq + from), bl = block_of(t, __ldg(t.pos + from));
    bool open = true;
    for (int64_t m = n0 + kWindow; open && m < t.num; m += kFar) {
        int32_t s[kFar / kWindow], p[kFar / kWindow];
#pragma unroll
        for (int i = 0; i < kFar / kWindow; ++i)
            load_token(t, m + i * kWindow + tid, s[i], p[i]);
#pragma unroll
        for (int i = 0; i < kFar / kWindow; ++i) {
            const bool has = has_place(t, s[i], p[i]);
            const bool on = has && s[i] == sl && block_of(t, p[i]) == bl;
            const uint32_t ons = __ballot_sync(0xffffffffu, on);
            const uint32_t others = __ballot_sync(0xffffffffu, has && !on);
            if (lane == 0) {
                w->behind[i * kWarps + warp] = ons;
                w->other[i * kWarps + warp] = others;
            }
        }
        __syncthreads();
        const int stop = first_of_far(w->other, 0u);
        open = stop == kFar;
        const int more = last_of_far(w->behind, stop) + 1;
        const bool gaps = first_of_far(w->behind, ~0u) < more;
        if (tid == 0 && more > 0) {
            if (from + w->len[run] < m || gaps) w->gaps[run] = true;
            w->len[run] = (int32_t)(m + more - from);
        }
        __syncthreads();
    }
}

// find_runs where a token with a place stands behind one without: a run goes on from the last
// token before that has one, however far that is.
__device__ __noinline__ int find_runs_over(const NewTokens& t, int64_t n0, unsigned int* err,
                                           Runs* w) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t s, p, s1, p1;  // this token, and the last before it
    load_token(t, n0 + tid, s, p);
    load_token(t, n0 - 1, s1, p1);
    const bool placed = has_place(t, s, p);
    w->seq[tid] = s;
    w->pos[tid] = p;
    const uint32_t mine = __ballot_sync(0xffffffffu, placed);
    if (lane == 0) w->placed[warp] = mine;
    __syncthreads();
    // (in front of the window: every warp for itself, 128 tokens at once)
    for (int64_t end = n0 - 1; end > 0 && !has_place(t, s1, p1); end -= 128) {
        int32_t ss[4], pp[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) load_token(t, end - 1 - 32 * i - lane, ss[i], pp[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t some = __ballot_sync(0xffffffffu, has_place(t, ss[i], pp[i]));
            if (some && !has_place(t, s1, p1)) {
                s1 = __shfl_sync(0xffffffffu, ss[i], __ffs(some) - 1);
                p1 = __shfl_sync(0xffffffffu, pp[i], __ffs(some) - 1);
            }
        }
    }
    const int at = last_below(w->placed, tid);
    if (at >= 0) {
        s1 = w->seq[at];
        p1 = w->pos[at];
    }
    const bool begins = placed && !(has_place(t, s1, p1) && s1 == s &&
                                    block_of(t, p1) == block_of(t, p));
    const int32_t page = begins ? token_page(t, s, p, err) : -1;
    const uint32_t starts = __ballot_sync(0xffffffffu, begins);
    if (lane == 0) w->starts[warp] = starts;
    __syncthreads();
    int k;
    const int total = count_runs(w, &k);
    if (begins) {
        const int end = last_below(w->placed, first_from<kWindow>(w->starts, tid + 1)) + 1;
        w->first[k] = tid;
        w->page[k] = page;
        w->len[k] = end - tid;
        w->gaps[k] = bits_from<kWindow>(w->placed, tid) < end - tid;
    }
    __syncthreads();
    if (total > 0) follow_run(t, n0, total - 1, w);
    return total;
}

// One thread looks at each token and at one behind the window; returns how many runs.
__device__ __forceinline__ int find_runs(const NewTokens& t, const RopeTable& table, int64_t n0,
                                         unsigned int* err, Runs* w) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t n = n0 + tid;
    int32_t s = -1, p = -1, rp = 0, s2 = -1, p2 = -1, sl = -1, pl = -1;
    if (n < t.num) {
        s = __ldg(t.seq + n);
        p = __ldg(t.pos + n);
        rp = __ldg(t.rope_pos + n);
    }
    if (n0 + kWindow < t.num) {  // the window's last token, and one behind it
        sl = __ldg(t.seq + n0 + kWindow - 1);
        pl = __ldg(t.pos + n0 + kWindow - 1);
        if (n + kWindow < t.num) {
            s2 = __ldg(t.seq + n + kWindow);
            p2 = __ldg(t.pos + n + kWindow);
        }
    }
    int32_t s1 = __shfl_up_sync(0xffffffffu, s, 1), p1 = __shfl_up_sync(0xffffffffu, p, 1);
    if (lane == 0) {
        s1 = n > 0 && n <= t.num ? __ldg(t.seq + n - 1) : -1;
        p1 = n > 0 && n <= t.num ? __ldg(t.pos + n - 1) : -1;
    }
    if (n < t.num) token_ok(t, table, s, p, rp, err);
    const bool placed = has_place(t, s, p);
    const bool on = placed && s1 == s && p1 >= 0 && block_of(t, p1) == block_of(t, p);
    const bool begins = placed && !on;
    int32_t page = -1;
    bool over = false;
    if (begins) {
        page = token_page(t, s, p, err);
        over = n > 0 && !has_place(t, s1, p1);
    }
    const uint32_t starts = __ballot_sync(0xffffffffu, begins);
    const uint32_t goes_on = __ballot_sync(0xffffffffu, on);
    const uint32_t behind = __ballot_sync(0xffffffffu, s2 >= 0 && s2 == sl && p2 >= 0 && pl >= 0 &&
                                                           block_of(t, p2) == block_of(t, pl));
    if (lane == 0) {
        w->starts[warp] = starts;
        w->goes_on[warp] = goes_on;
        w->behind[warp] = behind;
    }
    if (__syncthreads_or(over)) return find_runs_over(t, n0, err, w);
    int k;
    const int total = count_runs(w, &k);
    if (begins) {
        int len = 1 + bits_from<kWindow>(w->goes_on, tid + 1);
        if (tid + len == kWindow) len += bits_from<kWindow>(w->behind, 0);
        w->first[k] = tid;
        w->page[k] = page;
        w->len[k] = len;
        w->gaps[k] = false;
        if (k == total - 1) {  // does it end behind the window, with a token that has a place?
            const int end = tid + len;
            w->open = n0 + kWindow < t.num && n0 + end < t.num &&
                      (end < kWindow || end == 2 * kWindow ||
                       !has_place(t, __ldg(t.seq + n0 + end), __ldg(t.pos + n0 + end)));
        }
    }
    __syncthreads();
    if (total > 0 && w->open) follow_run(t, n0, total - 1, w);
    return total;
}

// `count` times 16 codes times `ratio`, every step-th from `first` on (rare: kept out of
// the registers of what runs every time; by one warp 29 us for the 255 rows of d = 128 in
// front of a token)
__device__ __noinline__ void rescale(unsigned char* codes, int64_t count, float ratio, int first,
                                     int step) {
    uint4* const w = reinterpret_cast<uint4*>(codes);
    for (int64_t i0 = first; i0 < count; i0 += step * 4) {
        uint4 c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i0 + step * i < count) c[i] = w[i0 + step * i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i0 + step * i >= count) continue;
            uint32_t* y = reinterpret_cast<uint32_t*>(&c[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t lo, hi;
                e4m3_f16(y[e], lo, hi);
                const float2 f = __half22float2(*reinterpret_cast<__half2*>(&lo));
                const float2 g = __half22float2(*reinterpret_cast<__half2*>(&hi));
                y[e] = e4m3x2(f.x * ratio, f.y * ratio) | e4m3x2(g.x * ratio, g.y * ratio) << 16;
            }
            w[i0 + step * i] = c[i];
        }
    }
}

// What a CTA writes: K or V of one head
struct Head {
    const unsigned char* rows;  // of the new tokens
    unsigned char* pool;        // at the head in page 0
    float* scales;
    int64_t stride;             // bytes from token to token
    int64_t page_bytes;
    uint32_t slot;              // this thread's place in the staging buffer
    int32_t rot;
    int u, da, db;              // this lane's unit and its chunks
};

// The run of `len` tokens from n on, in `page`, written by W warps of which this is the
// rank-th (W is 1, 2 or all of the CTA's); `gaps`: some of the tokens are passed over.
template <int D, bool F32, bool MIX, bool ROT, int W>
__device__ __forceinline__ void write_run(const Q8WriteArgs& a, const Head& hd, int64_t n,
                                          int32_t len, bool gaps, int32_t page, int rank,
                                          uint32_t* red) {
    constexpr int U = D / 16, RS = 32 / U;  // lanes per row, rows per step
    constexpr int step = W * RS;
    constexpr uint32_t kNext = (F32 ? 4 : 2) * kPiece;  // a thread's next slot
    const int lane = threadIdx.x & 31;
    const int cap = step * a.steps;                     // rows held
    const int32_t r0 = rank * RS + lane / U;            // this lane's first row
    const int32_t* const pos = a.tok.pos + n;
    const int32_t* const rope_pos = a.tok.rope_pos + n;
    const int32_t B = (int32_t)a.tok.block.d;
    const int32_t p = __ldg(pos);
    const int32_t p0 = (int32_t)a.tok.block.quot((uint32_t)p) * B;  // the page's first position
    const int32_t front = p - p0;                                   // rows in front of the run
    float* const sp = hd.scales + (int64_t)page * a.tok.hkv;
    const float old = front > 0 ? *sp : 0.f;
    const bool spins = ROT && hd.u < (hd.rot >> 4);

    // the largest of the warps'
    auto run_max = [&](uint32_t m) {
        m = __reduce_max_sync(0xffffffffu, m);
        if constexpr (W > 1) {
            auto meet = [&]() {
                if constexpr (W == kWarps) {
                    __syncthreads();
                } else {  // (barrier 0 is the CTA's)
                    const int bar = 1 + (threadIdx.x >> 5) / W;
                    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(W * 32) : "memory");
                }
            };
            meet();
            if (lane == 0) red[rank] = m;
            meet();
#pragma unroll
            for (int i = 0; i < W; ++i) m = max(m, red[i]);
        }
        return m;
    };
    // this lane's parts of the rows from base on
    auto fetch = [&](int32_t base) {
        const unsigned char* from = hd.rows + (n + base + r0) * hd.stride;
        uint32_t slot = hd.slot;
        for (int32_t r = base + r0; r < min(len, base + cap); r += step) {
            stage_unit<F32>(slot, from + hd.da * (F32 ? 4 : 2), from + hd.db * (F32 ? 4 : 2));
            from += step * hd.stride;
            slot += kNext;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int32_t rp0 = a.table.rot ? __ldg(rope_pos) : 0;
    fetch(0);
    // The usual run is one of consecutive positions, all of them in the table: then
    // nothing is looked up row by row.  (What follows is compiled for each kind by itself:
    // together, in the same registers, the usual ones took 3 to 6 us more of 60.)
    bool plain = !gaps && rp0 >= 0;
    for (int32_t r = r0; r < len; r += step) {
        plain &= __ldg(pos + r) - p == r;
        if (a.table.rot) {
            const int32_t rp = __ldg(rope_pos + r);
            plain &= rp - rp0 == r && rp < a.table.positions;
        }
    }
    auto rest = [&](auto by_row) {
        constexpr bool PLAIN = !decltype(by_row)::value;
        // the position that row r is rotated by (0 without a rotation), below 0: none, the
        // row is not written
        auto turn_of = [&](int32_t r) {
            if (PLAIN) return a.table.rot ? rp0 + r : 0;
            const int32_t pr = __ldg(pos + r);
            // (a token that is passed over)
            if (__ldg(a.tok.seq + n + r) != __ldg(a.tok.seq + n) || pr < p0 || pr - p0 >= B)
                return -1;
            if (!a.table.rot) return 0;
            const int32_t rp = __ldg(rope_pos + r);
            return rp < a.table.positions ? rp : -1;
        };
        // rotates the rows from base on in place (to odd where bf16 holds them: a further
        // rounding to 4 bits then gives what one rounding gives); the largest magnitude's
        // bits + 1
        auto rotate_rows = [&](int32_t base) {
            uint32_t top = 0, slot = hd.slot;
            asm volatile("cp.async.wait_all;" ::: "memory");
            #pragma unroll 1
            for (int32_t r = base + r0; r < min(len, base + cap); r += step, slot += kNext) {
                const int32_t rp = turn_of(r);
                if (rp < 0) continue;
                RawUnit<F32> x = staged_unit<F32>(slot);
                float m;  // (no maximum here takes notice of a NaN)
                if (spins) {
                    const float4* const c = reinterpret_cast<const float4*>(
                        a.table.cos_sin + (int64_t)rp * a.table.rot + 8 * hd.u);
                    const float4* const q = c + a.table.rot / 8;
                    m = rotate_half<F32, MIX>(x, 0, __ldg(c), __ldg(q));
                    m = fmaxf(m, rotate_half<F32, MIX>(x, 1, __ldg(c + 1), __ldg(q + 1)));
                    restage_unit<F32>(slot, x);
                } else {
                    m = largest(x);
                }
                top = max(top, __float_as_uint(m) + 1);
            }
            return top;
        };
        uint32_t top = 0;
        for (int32_t base = 0; base < len; base += cap) {
            if (base > 0) fetch(base);
            top = max(top, rotate_rows(base));
        }
        top = run_max(top);
        if (top == 0) return;  // no row to write
        const bool inf = top - 1 == 0x7f800000u;
        if (inf) {  // once more over the finite ones
            top = 1;
            for (int32_t base = 0; base < len; base += cap) {
                if (len > cap) {
                    fetch(base);
                    rotate_rows(base);
                }
                uint32_t slot = hd.slot;
#pragma unroll 1
                for (int32_t r = base + r0; r < min(len, base + cap); r += step, slot += kNext) {
                    float x[16];
                    if (turn_of(r) < 0) continue;
                    widen_unit<F32>(staged_unit<F32>(slot), x);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (fabsf(x[e]) < INFINITY) top = max(top, __float_as_uint(fabsf(x[e])) + 1);
                }
            }
            top = run_max(top);
        }
        float s = scale_for(__uint_as_float(top - 1));
        unsigned char* const head = hd.pool + page * hd.page_bytes;
        if (front > 0) {
            const float was = scale_up(old);
            s = was <= s ? s : was;  // (NaN stays)
            if (s != old) {
                const float ratio = old * __frcp_rn(s);
                rescale(head, (int64_t)front * (D / 16), ratio, rank * 32 + lane, W * 32);
            }
        }
        // (all warps of the run have read the old scale: they met in run_max)
        if (rank == 0 && lane == 0) *sp = s;
        const float inv = __frcp_rn(s);
        for (int32_t base = 0; base < len; base += cap) {
            if (len > cap) {
                fetch(base);
                rotate_rows(base);
            }
            uint32_t slot = hd.slot;
            #pragma unroll 1
            for (int32_t r = base + r0; r < min(len, base + cap); r += step, slot += kNext) {
                if (turn_of(r) < 0) continue;
                const int32_t at = PLAIN ? front + r : __ldg(pos + r) - p0;
                float x[16];
                widen_unit<F32>(staged_unit<F32>(slot), x);
                if (inf) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = fmaf(x[e], 0.f, x[e]);  // to NaN
                }
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 y = fmul2(make_float2(x[4 * e], x[4 * e + 1]), make_float2(inv, inv));
                    const float2 z = fmul2(make_float2(x[4 * e + 2], x[4 * e + 3]),
                                           make_float2(inv, inv));
                    w[e] = e4m3x2(y.x, y.y) | e4m3x2(z.x, z.y) << 16;
                }
                unsigned char* const to = head + (int64_t)at * D;
                if (hd.db == hd.da + 8) {
                    *reinterpret_cast<uint4*>(to + hd.da) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    *reinterpret_cast<uint2*>(to + hd.da) = make_uint2(w[0], w[1]);
                    *reinterpret_cast<uint2*>(to + hd.db) = make_uint2(w[2], w[3]);
                }
            }
        }
    };
    if (__all_sync(0xffffffffu, plain)) rest(std::false_type{});
    else rest(std::true_type{});
}

template <int D, bool F32, bool MIX, bool ROT, int TEAM>
__device__ __forceinline__ void write_runs(const Q8WriteArgs& a, uint32_t cta, Runs& runs,
                                           uint32_t* red) {
    constexpr int U = D / 16, RS = 32 / U;
    extern __shared__ __align__(16) unsigned char stage[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool is_v = cta & 1;
    const int h = (int)((cta >> 1) % (uint32_t)a.tok.hkv);
    const uint32_t rest = (cta >> 1) / (uint32_t)a.tok.hkv;
    const int part = (int)(rest % (uint32_t)a.parts);
    const int64_t n0 = (int64_t)(rest / (uint32_t)a.parts) * kWindow;
    Head hd;
    hd.rows = static_cast<const unsigned char*>(is_v ? a.v : a.k) + (int64_t)h * D * (F32 ? 4 : 2);
    hd.stride = (is_v ? a.v_stride : a.k_stride) * (F32 ? 4 : 2);
    hd.page_bytes = (int64_t)a.tok.hkv * a.tok.block.d * D;
    hd.pool = (is_v ? a.vc : a.kc) + (int64_t)h * a.tok.block.d * D;
    hd.scales = (is_v ? a.vs : a.ks) + h;
    hd.slot = smem_u32(stage) + threadIdx.x * 16;
    hd.rot = ROT ? a.table.rot : 0;
    hd.u = lane % U;
    unit_dims<MIX>(hd.u, hd.rot, &hd.da, &hd.db);
    // (one CTA of a window flags what is wrong with its tokens)
    const int total = find_runs(a.tok, a.table, n0, h == 0 && part == 0 && !is_v ? a.err : nullptr,
                                &runs);
    // every parts-th run, one per warp, then those of more rows than a warp holds, by teams
    for (int k = part + warp * a.parts; k < total; k += kWarps * a.parts)
        if (runs.page[k] >= 0 && (TEAM == 1 || runs.len[k] <= RS * a.steps))
            write_run<D, F32, MIX, ROT, 1>(a, hd, n0 + runs.first[k], runs.len[k], runs.gaps[k],
                                           runs.page[k], 0, nullptr);
    if constexpr (TEAM > 1) {
        const int team = TEAM == kWarps ? 0 : warp / TEAM, rank = TEAM == kWarps ? warp : warp % TEAM;
        for (int k = part + team * a.parts; k < total; k += kWarps / TEAM * a.parts)
            if (runs.page[k] >= 0 && runs.len[k] > RS * a.steps)
                write_run<D, F32, MIX, ROT, TEAM>(a, hd, n0 + runs.first[k], runs.len[k],
                                                  runs.gaps[k], runs.page[k], rank,
                                                  red + team * TEAM);
    }
}

// TEAM: warps that take a run of more rows than one holds
template <int D, bool F32, bool MIX, int TEAM>
__global__ void __launch_bounds__(kWarps * 32, 3) q8_write_kernel(const __grid_constant__ Q8WriteArgs a) {
    PKV_DEPENDENT_PROLOGUE();
    // CTAs of K and V lie among those of the queries, which fill the GPU behind them
    const uint32_t kv = (uint32_t)min((blockIdx.x * a.kv_step) >> 32, (uint64_t)a.kv_ctas);
    if (kv < a.kv_ctas && ((blockIdx.x + 1ull) * a.kv_step) >> 32 > kv) {
        __shared__ Runs runs;
        __shared__ uint32_t red[kWarps];
        if (a.table.rot && !(kv & 1)) write_runs<D, F32, MIX, true, TEAM>(a, kv, runs, red);
        else write_runs<D, F32, MIX, false, TEAM>(a, kv, runs, red);
        return;
    }
    const int64_t id = (int64_t)(blockIdx.x - kv) * kWarps + (threadIdx.x >> 5);
    const int64_t n = id / a.q.warps;
    if (n < a.tok.num)
        query_warp<D, F32, MIX>(a.q, a.table, a.tok.seq, a.tok.rope_pos, n,
                                (int)(id - n * a.q.warps), threadIdx.x & 31);
}

// ---- read -------------------------------------------------------------------------
constexpr int kReadWarps = 4;  // tokens per CTA
constexpr int kReadLoads = 4;  // 8-code chunks a lane has in flight

struct Q8ReadArgs {
    const unsigned char* kc;
    const unsigned char* vc;
    const float* ks;
    const float* vs;
    const int32_t* slots;
    void* k;
    void* v;
    int64_t num_tokens, num_slots;
    FastDiv block;
    int32_t hkv;
    unsigned int* err;
};

template <int D, bool F32>
__global__ void __launch_bounds__(kReadWarps * 32) q8_read_kernel(const Q8ReadArgs a) {
    PKV_DEPENDENT_PROLOGUE();
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * kReadWarps + (threadIdx.x >> 5);
    if (n >= a.num_tokens) return;
    const bool is_v = blockIdx.y;
    int32_t slot = __ldg(a.slots + n);
    if (slot >= a.num_slots) {
        if (lane == 0 && !is_v) flag_error(a.err, PKV_FLAG_BAD_SLOT);
        slot = -1;
    }
    const int64_t page = slot < 0 ? 0 : a.block.quot((uint32_t)slot);
    const int32_t at = slot < 0 ? 0 : slot - (int32_t)page * (int32_t)a.block.d;
    const unsigned char* const pool = is_v ? a.vc : a.kc;
    const float* const scales = (is_v ? a.vs : a.ks) + page * a.hkv;
    unsigned char* const out = static_cast<unsigned char*>(is_v ? a.v : a.k) +
                               n * a.hkv * D * (F32 ? 4 : 2);
    const int chunks = a.hkv * (D / 8);
    for (int c0 = lane; c0 < chunks; c0 += 32 * kReadLoads) {
        uint2 w[kReadLoads];
        float s[kReadLoads];
#pragma unroll
        for (int i = 0; i < kReadLoads; ++i) {
            const int c = c0 + 32 * i;
            w[i] = make_uint2(0u, 0u);
            s[i] = 0.f;
            if (c < chunks && slot >= 0) {
                const int h = c / (D / 8);
                w[i] = __ldcs(reinterpret_cast<const uint2*>(
                    pool + ((page * a.hkv + h) * a.block.d + at) * D + c % (D / 8) * 8));
                s[i] = __ldg(scales + h);
            }
        }
#pragma unroll
        for (int i = 0; i < kReadLoads; ++i) {
            const int c = c0 + 32 * i;
            if (c >= chunks) continue;
            float x[8];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t lo, hi;
                e4m3_f16(e ? w[i].y : w[i].x, lo, hi);
                const float2 f = __half22float2(*reinterpret_cast<__half2*>(&lo));
                const float2 g = __half22float2(*reinterpret_cast<__half2*>(&hi));
                x[4 * e] = f.x * s[i];
                x[4 * e + 1] = f.y * s[i];
                x[4 * e + 2] = g.x * s[i];
                x[4 * e + 3] = g.y * s[i];
            }
            store_chunk<F32>(out, 8 * c, x);
        }
    }
}

template <int D, bool F32, bool MIX, int TEAM>
cudaError_t launch_write(const DeviceInfo& dev, const Q8WriteArgs& a, int64_t ctas, size_t smem,
                         cudaStream_t stream) {
    auto kern = q8_write_kernel<D, F32, MIX, TEAM>;
    // the most shared memory a CTA may have, set once per device
    static std::atomic<uint64_t> set{0};
    const uint64_t bit = 1ull << dev.device;
    if (!(set.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 most_steps<F32>() * step_bytes<F32>());
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_relaxed);
    }
    return launch_dependent(kern, dim3((unsigned)ctas), dim3(kWarps * 32), smem, stream, a);
}

}  // namespace

cudaError_t launch_q8_write(const DeviceInfo& dev, const RopeWriteLaunch& r, float* k_scale,
                            float* v_scale, cudaStream_t stream) {
    if (r.num_tokens == 0) return cudaSuccess;
    const bool f32 = r.src_dtype == PKV_F32, mix = r.interleaved != 0;
    Q8WriteArgs a{};
    a.k = r.k;
    a.v = r.v;
    a.k_stride = r.k_stride;
    a.v_stride = r.v_stride;
    a.tok = NewTokens{r.token_seq, r.token_pos, r.rope_pos ? r.rope_pos : r.token_pos, r.table,
                      r.num_tokens, r.num_blocks, FastDiv((uint32_t)r.block_size), r.num_seqs,
                      r.max_blocks, r.hkv};
    a.kc = static_cast<unsigned char*>(r.k_cache);
    a.vc = static_cast<unsigned char*>(r.v_cache);
    a.ks = k_scale;
    a.vs = v_scale;
    a.table = RopeTable{r.cos_sin, r.positions, r.rot};
    // steps that a page's rows take of one warp
    const int rows = 32 / (r.d / 16), most = f32 ? most_steps<true>() : most_steps<false>();
    a.steps = (int32_t)std::min<int64_t>(most, ((int64_t)r.block_size + rows - 1) / rows);
    const size_t smem = (size_t)a.steps * (f32 ? step_bytes<true>() : step_bytes<false>());
    // CTAs that share a window: as many as fill the GPU, but no fewer tokens than warps
    const int64_t windows = (r.num_tokens + kWindow - 1) / kWindow;
    const int64_t fill = 3 * dev.num_sms / (windows * r.hkv * 2);
    a.parts = (int32_t)std::max<int64_t>(
        1, std::min<int64_t>(fill, (std::min<int64_t>(r.num_tokens, kWindow) + kWarps - 1) / kWarps));
    const int64_t kv_ctas = windows * a.parts * r.hkv * 2;
    int64_t ctas = kv_ctas;
    if (r.q) {
        const int32_t w = (int32_t)(f32 ? unit_warps<true>(r.hq, r.d) : unit_warps<false>(r.hq, r.d));
        a.q = RopeQuery{r.q, r.q_out, r.q_stride, r.q_out_stride, r.hq, w};
        ctas += (r.num_tokens * w + kWarps - 1) / kWarps;
    }
    if (ctas > 0x7fffffff) return cudaErrorNotSupported;
    a.kv_ctas = (uint32_t)kv_ctas;
    const uint64_t even = (((uint64_t)kv_ctas << 32) + ctas - 1) / ctas;
    a.kv_step = std::min(2 * even, (uint64_t)1 << 32);
    a.err = r.err;
    // a page's rows are a warp's, two warps', or all warps' (16,729 tokens of 16 / 8 heads in
    // pages of 64: 56 us by twos, 65 by all; of 128: 77 by twos, 57 by all)
    const int64_t held = (int64_t)a.steps * rows;
    const int team = r.block_size <= held ? 1 : (r.block_size <= 2 * held ? 2 : 8);
    cudaError_t e = cudaErrorInvalidValue;
#define PKV_Q8_CASE(DD, FF, MM) \
    if (r.d == DD && f32 == FF && mix == MM) \
        e = team == 1 ? launch_write<DD, FF, MM, 1>(dev, a, ctas, smem, stream) \
            : team == 2 ? launch_write<DD, FF, MM, 2>(dev, a, ctas, smem, stream) \
                        : launch_write<DD, FF, MM, 8>(dev, a, ctas, smem, stream);
    PKV_Q8_CASE(64, false, false) PKV_Q8_CASE(64, false, true)
    PKV_Q8_CASE(64, true, false) PKV_Q8_CASE(64, true, true)
    PKV_Q8_CASE(128, false, false) PKV_Q8_CASE(128, false, true)
    PKV_Q8_CASE(128, true, false) PKV_Q8_CASE(128, true, true)
#undef PKV_Q8_CASE
    return e;
}

cudaError_t launch_q8_read(const void* k_cache, const void* v_cache, const float* k_scale,
                           const float* v_scale, const int32_t* slots, int64_t num_tokens,
                           void* k, void* v, int dst_dtype, int hkv, int d, int block_size,
                           int64_t num_slots, unsigned int* err, cudaStream_t stream) {
    if (num_tokens == 0) return cudaSuccess;
    const Q8ReadArgs a{static_cast<const unsigned char*>(k_cache),
                       static_cast<const unsigned char*>(v_cache), k_scale, v_scale, slots, k, v,
                       num_tokens, num_slots, FastDiv((uint32_t)block_size), hkv, err};
    const bool f32 = dst_dtype == PKV_F32;
    auto kern = d == 128 ? (f32 ? q8_read_kernel<128, true> : q8_read_kernel<128, false>)
                         : (f32 ? q8_read_kernel<64, true> : q8_read_kernel<64, false>);
    const int64_t ctas = (num_tokens + kReadWarps - 1) / kReadWarps;
    return launch_dependent(kern, dim3((unsigned)ctas, 2), dim3(kReadWarps * 32), 0, stream, a);
}

}  // namespace pkv
