// rope_write.cu -- the cache write of new K/V rows with the position rotation on the
// way (format and arithmetic of the rotation: rope.cuh): keys are rotated and written
// with the values to the slots of their positions ("11. Paged attention 与 online
// softmax" §11.1), the queries of the same tokens are rotated beside them.
//
// What bounds it: bytes.  A token's q, K and V are read and written once and its row
// of the table is read; 6 operations per two rotated values are nothing beside that.
// Alone, a rotation would read and write q and K once more: 1.5 times the bytes of
// the whole call at 16 / 8 heads.  One warp moves up to 16 heads (fp32: 8) of 128 dims
// of one token's q, K or V, every load of it in flight before the first is needed and
// before the slot is known; a small batch then spreads over 3 to 4 warps per token.
//
// Measured: 16,729 tokens of 16 / 8 heads of 128, bf16, the columns of one projection, into
// pages of 256, 282.8 MB: 45.6 us, 6205 GB/s (0.93 of the measured copy rate).  2430 tokens
// of 16 / 8 heads of 64 in fp32 into bf16 pools, 36.2 MB: 7.8 us.  64 tokens: 4.1 us a
// call among others, what the host takes to make it.
#include "common.cuh"
#include "launch.h"
#include "rope.cuh"

namespace pkv {

namespace {

constexpr int kWarps = 4;  // per CTA

struct RopeWriteArgs {
    const void* k;
    const void* v;
    int64_t k_stride, v_stride;  // elements from token to token
    NewTokens tok;
    int32_t* slots_out;
    void* kc;
    void* vc;
    RopeTable table;
    RopeQuery q;
    int32_t kv_warps;  // per token, of K (and of V)
    unsigned int* err;
};

template <int D, bool F32, bool OUT_F32, bool MIX>
__global__ void __launch_bounds__(kWarps * 32) rope_write_kernel(const RopeWriteArgs a) {
    PKV_DEPENDENT_PROLOGUE();
    constexpr int U = D / 16, R = unit_rounds<F32>();
    const int lane = threadIdx.x & 31;
    const int per = 2 * a.kv_warps + a.q.warps;
    const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t n = id / per;
    if (n >= a.tok.num) return;
    const int job = (int)(id - n * per);
    if (job >= 2 * a.kv_warps) {
        query_warp<D, F32, MIX>(a.q, a.table, a.tok.seq, a.tok.rope_pos, n, job - 2 * a.kv_warps,
                                lane);
        return;
    }
    const bool is_v = job >= a.kv_warps;
    const int w = is_v ? job - a.kv_warps : job;
    const unsigned char* src = static_cast<const unsigned char*>(is_v ? a.v : a.k) +
                               n * (is_v ? a.v_stride : a.k_stride) * (F32 ? 4 : 2);
    RawUnit<F32> raw[R];
    load_units<D, F32, MIX>(src, a.tok.hkv, w, lane, a.table.rot, raw);
    UnitAngles ang;
    const int32_t rp = __ldg(a.tok.rope_pos + n);
    if (!is_v && rp >= 0 && rp < a.table.positions && lane % U < (a.table.rot >> 4))
        load_angles(a.table, rp, lane % U, ang);
    // one lane of a token flags what is wrong with it and stores its slot
    const bool first = job == 0 && lane == 0;
    const int32_t p = __ldg(a.tok.pos + n), s = __ldg(a.tok.seq + n);
    int32_t page = -1;
    if (token_ok(a.tok, a.table, s, p, rp, first ? a.err : nullptr))
        page = token_page(a.tok, s, p, first ? a.err : nullptr);
    const int32_t B = (int32_t)a.tok.block.d;
    const int32_t at = p - (int32_t)a.tok.block.quot((uint32_t)p) * B;
    if (first && a.slots_out) a.slots_out[n] = page < 0 ? -1 : page * B + at;
    if (page < 0) return;
    const int64_t row = ((int64_t)page * B + at) * a.tok.hkv * D * (OUT_F32 ? 4 : 2);
    move_units<D, F32, OUT_F32, MIX>(static_cast<unsigned char*>(is_v ? a.vc : a.kc) + row,
                                     a.tok.hkv, w, lane, !is_v, a.table.rot, raw, ang);
}

}  // namespace

cudaError_t launch_rope_write(const RopeWriteLaunch& r, cudaStream_t stream) {
    if (r.num_tokens == 0) return cudaSuccess;
    const bool f32 = r.src_dtype == PKV_F32, out_f32 = r.cache_dtype == PKV_F32;
    const bool mix = r.interleaved != 0;
    auto warps = [&](int heads) {
        return (int32_t)(f32 ? unit_warps<true>(heads, r.d) : unit_warps<false>(heads, r.d));
    };
    RopeWriteArgs a{};
    a.k = r.k;
    a.v = r.v;
    a.k_stride = r.k_stride;
    a.v_stride = r.v_stride;
    a.tok = NewTokens{r.token_seq, r.token_pos, r.rope_pos ? r.rope_pos : r.token_pos, r.table,
                      r.num_tokens, r.num_blocks, FastDiv((uint32_t)r.block_size), r.num_seqs,
                      r.max_blocks, r.hkv};
    a.slots_out = r.slots_out;
    a.kc = r.k_cache;
    a.vc = r.v_cache;
    a.table = RopeTable{r.cos_sin, r.positions, r.rot};
    a.kv_warps = warps(r.hkv);
    if (r.q) a.q = RopeQuery{r.q, r.q_out, r.q_stride, r.q_out_stride, r.hq, warps(r.hq)};
    a.err = r.err;
    const int64_t all = r.num_tokens * (2 * (int64_t)a.kv_warps + a.q.warps);
    const int64_t ctas = (all + kWarps - 1) / kWarps;
    if (ctas > 0x7fffffff) return cudaErrorNotSupported;
    cudaError_t e = cudaErrorInvalidValue;
    auto go = [&](auto kern) {
        e = launch_dependent(kern, dim3((unsigned)ctas), dim3(kWarps * 32), 0, stream, a);
    };
#define PKV_ROPE_CASE(DD, FF, OO, MM) \
    if (r.d == DD && f32 == FF && out_f32 == OO && mix == MM) go(rope_write_kernel<DD, FF, OO, MM>);
#define PKV_ROPE_TYPES(DD, MM)                                             \
    PKV_ROPE_CASE(DD, false, false, MM) PKV_ROPE_CASE(DD, false, true, MM) \
    PKV_ROPE_CASE(DD, true, false, MM) PKV_ROPE_CASE(DD, true, true, MM)
    PKV_ROPE_TYPES(64, false) PKV_ROPE_TYPES(64, true)
    PKV_ROPE_TYPES(128, false) PKV_ROPE_TYPES(128, true)
#undef PKV_ROPE_TYPES
#undef PKV_ROPE_CASE
    return e;
}

}  // namespace pkv
