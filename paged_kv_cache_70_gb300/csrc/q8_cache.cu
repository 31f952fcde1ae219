// q8_cache.cu -- rows into and out of 8-bit K/V pools (format: q8.cuh).
//
// Write: the new rows that fall into one page, with the largest finite magnitude a of a
// head's values among them (K after its rotation, rope.cuh), need the least power of
// two n >= 2^-100 with a <= 448 n.  If they begin the page, its scale is n; else it is
// s = max(n, the old scale, rounded up to a power of two), and the codes of the rows in
// front of them become e4m3(code * (old / s)): a shift of the exponent, which is exact
// until a code gets below 2^-6.  New codes are e4m3(x / s).  A power of two makes both
// divisions exact, so that a value is rounded once.  Tokens of one page follow one
// another in the list (a run); a run is found by its first token, which differs from
// the token before it in sequence or page.
//
// What bounds it: bytes for long runs, the chain token -> page -> old scale -> rows for
// single tokens.  A (run, head) is held by wr warps in registers from the load over the
// maximum to the store, so that rows are read once: 4 rows (d = 64: 8) per warp and
// step, 8 steps (fp32: 4); only runs of more rows than that are read twice.  The
// CTAs take `window` tokens each, as few as fill the GPU: one CTA per token would be
// mostly CTAs in which no run begins.
// Read: row n of the outputs is code * scale at slot_mapping[n], rounded once to the
// output's type; zeros for a negative slot.
#include <algorithm>

#include "launch.h"
#include "q8.cuh"
#include "rope.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 8;  // per CTA of the write
template <bool F32>
__host__ __device__ constexpr int row_steps() { return F32 ? 4 : 8; }  // that a warp holds

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
    int64_t kv_ctas;    // the CTAs behind them take the queries
    int32_t wr;         // warps per (run, head)
    int32_t groups;     // of kWarps / wr heads
    int32_t window;     // tokens whose runs a CTA takes
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

template <int D, bool F32, bool MIX>
__device__ __forceinline__ void write_runs(const Q8WriteArgs& a) {
    constexpr int U = D / 16, RS = 32 / U;  // lanes per row, rows per step
    constexpr int S = row_steps<F32>();
    __shared__ uint32_t red[2][kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool is_v = blockIdx.x & 1;
    const int64_t id = blockIdx.x >> 1;
    const int64_t n0 = id / a.groups * a.window;
    const int64_t n1 = min(n0 + a.window, a.tok.num);
    const int group = (int)(id % a.groups);
    const int team = warp / a.wr, rank = warp % a.wr;
    const int h = group * (kWarps / a.wr) + team;
    const bool has = h < a.tok.hkv;
    const bool reports = group == 0 && !is_v && warp == 0;  // flags what is wrong with tokens
    const int32_t B = (int32_t)a.tok.block.d;
    unsigned char* const pool = is_v ? a.vc : a.kc;
    float* const scales = is_v ? a.vs : a.ks;
    const int rot = is_v ? 0 : a.table.rot;
    const int u = lane % U;
    int da, db;
    unit_dims<MIX>(u, rot, &da, &db);
    const bool spins = u < (rot >> 4);
    const unsigned char* const rows =
        static_cast<const unsigned char*>(is_v ? a.v : a.k) + (int64_t)h * D * (F32 ? 4 : 2);
    const int64_t stride = (is_v ? a.v_stride : a.k_stride) * (F32 ? 4 : 2);
    int turn = 0;  // of `red`

    // the largest of the team's
    auto team_max = [&](uint32_t m) {
        m = __reduce_max_sync(0xffffffffu, m);
        if (a.wr == 1) return m;
        if (lane == 0) red[turn][warp] = m;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(a.wr * 32) : "memory");
        for (int i = 0; i < a.wr; ++i) m = max(m, red[turn][team * a.wr + i]);
        turn ^= 1;
        return m;
    };

    // the run of `len` tokens from n on, on one page of B positions from `p0` on, the
    // first of them at p
    auto write_run = [&](int64_t n, int32_t len, int32_t page, int32_t p0, int32_t p) {
        const int32_t front = p - p0;  // rows of the page in front of the run
        float* const sp = scales + (int64_t)page * a.tok.hkv + h;
        const float old = has && front > 0 ? *sp : 0.f;
        const int cap = a.wr * RS * S;
        RawUnit<F32> raw[S];
        auto row = [&](int32_t base, int i) { return base + (i * a.wr + rank) * RS + lane / U; };
        auto load = [&](int32_t base) {
#pragma unroll
            for (int i = 0; i < S; ++i)
                if (row(base, i) < len && has)
                    load_unit<F32>(rows + (n + row(base, i)) * stride, da, db, raw[i]);
        };
        // this lane's part of row r, rotated, and its place in the page; below 0: none
        auto value = [&](int32_t r, const RawUnit<F32>& w, float* x) {
            if (r >= len || !has) return -1;
            UnitAngles ang;
            if (a.table.rot) {
                const int32_t rp = __ldg(a.tok.rope_pos + n + r);
                if (rp < 0 || rp >= a.table.positions) return -1;
                if (spins) load_angles(a.table, rp, u, ang);
            }
            widen_unit<F32>(w, x);
            if (spins) rotate_unit<MIX>(x, ang);
            return __ldg(a.tok.pos + n + r) - p0;
        };
        uint32_t top = 0;  // the largest magnitude's bits + 1
        for (int32_t base = 0; base < len; base += cap) {
            load(base);
#pragma unroll
            for (int i = 0; i < S; ++i) {
                float x[16];
                if (value(row(base, i), raw[i], x) < 0) continue;
                float m = 0.f;
                // (x + 0 x is NaN for an infinity, and fmaxf takes no notice of NaN)
#pragma unroll
                for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(fmaf(x[e], 0.f, x[e])));
                top = max(top, __float_as_uint(m) + 1);
            }
        }
        top = team_max(top);
        if (top == 0) return;  // no row to write
        float s = scale_for(__uint_as_float(top - 1));
        unsigned char* const head = pool + ((int64_t)page * a.tok.hkv + h) * B * D;
        if (front > 0) {
            const float was = scale_up(old);
            s = was <= s ? s : was;  // (NaN stays)
            if (s != old) {
                const float ratio = old * __frcp_rn(s);
                uint4* const w = reinterpret_cast<uint4*>(head);
                for (int64_t i = rank * 32 + lane; i < (int64_t)front * (D / 16);
                     i += a.wr * 32) {
                    uint4 c = w[i];
                    uint32_t* y = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t lo, hi;
                        e4m3_f16(y[e], lo, hi);
                        const float2 f = __half22float2(*reinterpret_cast<__half2*>(&lo));
                        const float2 g = __half22float2(*reinterpret_cast<__half2*>(&hi));
                        y[e] = e4m3x2(f.x * ratio, f.y * ratio) |
                               e4m3x2(g.x * ratio, g.y * ratio) << 16;
                    }
                    w[i] = c;
                }
            }
        }
        // (the team has read the old scale: it met in team_max)
        if (rank == 0 && lane == 0) *sp = s;
        const float inv = __frcp_rn(s);
        for (int32_t base = 0; base < len; base += cap) {
            if (len > cap) load(base);
#pragma unroll
            for (int i = 0; i < S; ++i) {
                float x[16];
                const int32_t at = value(row(base, i), raw[i], x);
                if (at < 0) continue;
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = fmaf(x[e], 0.f, x[e] * inv);  // inf: NaN
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = e4m3x2(x[4 * e], x[4 * e + 1]) |
                           e4m3x2(x[4 * e + 2], x[4 * e + 3]) << 16;
                unsigned char* const to = head + (int64_t)at * D;
                *reinterpret_cast<uint2*>(to + da) = make_uint2(w[0], w[1]);
                *reinterpret_cast<uint2*>(to + db) = make_uint2(w[2], w[3]);
            }
        }
    };

    for (int64_t base = n0; base < n1; base += 32) {
        // runs that begin at one of these tokens
        const int64_t n = base + lane;
        int32_t s = -1, p = 0;
        bool starts = false;
        if (n < n1) {
            s = __ldg(a.tok.seq + n);
            p = __ldg(a.tok.pos + n);
            const int32_t rp = __ldg(a.tok.rope_pos + n);
            const int32_t s1 = n > 0 ? __ldg(a.tok.seq + n - 1) : -1;
            const int32_t p1 = n > 0 ? __ldg(a.tok.pos + n - 1) : -1;
            token_ok(a.tok, a.table, s, p, rp, reports ? a.err : nullptr);
            starts = s >= 0 && s < a.tok.num_seqs && p >= 0 &&
                     (int32_t)a.tok.block.quot((uint32_t)p) < a.tok.max_blocks &&
                     (s1 != s || p1 < 0 ||
                      a.tok.block.quot((uint32_t)p1) != a.tok.block.quot((uint32_t)p));
        }
        uint32_t found = __ballot_sync(0xffffffffu, starts);
        while (found) {
            const int bit = __ffs(found) - 1;
            found &= found - 1;
            const int32_t rs = __shfl_sync(0xffffffffu, s, bit);
            const int32_t rp = __shfl_sync(0xffffffffu, p, bit);
            const int32_t page = token_page(a.tok, rs, rp, reports && lane == 0 ? a.err : nullptr);
            if (page < 0) continue;
            const int32_t pg = (int32_t)a.tok.block.quot((uint32_t)rp);
            // the tokens behind it on the same page: 128 at a time where a page can
            // hold more than 32
            int32_t len = 1;
            for (bool more = true; more;) {
                bool same[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t t = base + bit + len + 32 * i + lane;
                    same[i] = false;
                    if ((i == 0 || B > 32) && t < a.tok.num) {
                        const int32_t ts = __ldg(a.tok.seq + t), tp = __ldg(a.tok.pos + t);
                        same[i] = ts == rs && tp >= 0 &&
                                  (int32_t)a.tok.block.quot((uint32_t)tp) == pg;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (!more || (i > 0 && B <= 32)) continue;
                    const uint32_t m = __ballot_sync(0xffffffffu, same[i]);
                    more = m == 0xffffffffu;
                    len += more ? 32 : __ffs(~m) - 1;
                }
            }
            write_run(base + bit, len, page, pg * B, rp);
        }
    }
}

template <int D, bool F32, bool MIX>
__global__ void __launch_bounds__(kWarps * 32, 2) q8_write_kernel(const Q8WriteArgs a) {
    PKV_DEPENDENT_PROLOGUE();
    if (blockIdx.x < a.kv_ctas) {
        write_runs<D, F32, MIX>(a);
        return;
    }
    const int64_t id = (int64_t)(blockIdx.x - a.kv_ctas) * kWarps + (threadIdx.x >> 5);
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
    // warps that hold a page's rows of a head, up to a CTA's
    const int per = 32 / (r.d / 16) * (f32 ? row_steps<true>() : row_steps<false>());
    a.wr = 1;
    while (a.wr < kWarps && a.wr * per < r.block_size) a.wr *= 2;
    const int heads = kWarps / a.wr;
    a.groups = (r.hkv + heads - 1) / heads;
    const double all = (double)r.num_tokens * a.groups * 2;
    a.window = (int32_t)std::min(64.0, std::max(1.0, all / (32.0 * dev.num_sms)));
    a.kv_ctas = (r.num_tokens + a.window - 1) / a.window * a.groups * 2;
    int64_t ctas = a.kv_ctas;
    if (r.q) {
        const int32_t w = (int32_t)(f32 ? unit_warps<true>(r.hq, r.d) : unit_warps<false>(r.hq, r.d));
        a.q = RopeQuery{r.q, r.q_out, r.q_stride, r.q_out_stride, r.hq, w};
        ctas += (r.num_tokens * w + kWarps - 1) / kWarps;
    }
    if (ctas > 0x7fffffff) return cudaErrorNotSupported;
    a.err = r.err;
    cudaError_t e = cudaErrorInvalidValue;
    auto go = [&](auto kern) {
        e = launch_dependent(kern, dim3((unsigned)ctas), dim3(kWarps * 32), 0, stream, a);
    };
#define PKV_Q8_CASE(DD, FF, MM) \
    if (r.d == DD && f32 == FF && mix == MM) go(q8_write_kernel<DD, FF, MM>);
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
