// q8_api.cu -- the extern "C" entry points of the cache write with the position
// rotation and of 8-bit K/V pools (declared in include/pagedkv.h): argument checks and
// dispatch.
#include "common.cuh"
#include "launch.h"

using pkv::DeviceInfo;
using pkv::aligned;
using pkv::elt_size;

namespace {

int cuda_status(cudaError_t e) {
    if (e == cudaErrorNotSupported) return PKV_ERR_UNSUPPORTED;  // a grid past its limits
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// tokens of a call: their places in it are counted in 32 bits
constexpr int64_t kMaxTokens = 1 << 30;

// the geometry of a call whose kernels take head_dim 64 or 128; dtype has been looked at
int check_heads(const pkv_geom* g) {
    pkv_geom as = *g;  // the checks every pool shares
    as.dtype = PKV_BF16;
    const int st = pkv::check_geom(&as);
    if (st != PKV_OK) return st;
    if (g->head_dim != 64 && g->head_dim != 128) return PKV_ERR_UNSUPPORTED;
    // a token's rows are counted in 32 bits
    return (int64_t)g->num_heads * g->head_dim > (1 << 30) ? PKV_ERR_UNSUPPORTED : PKV_OK;
}

int check_q8_geom(const pkv_geom* g) {
    if (!g || g->dtype != PKV_Q8) return PKV_ERR_INVALID;
    return check_heads(g);
}

// rows of `elt`-byte values, `stride` of them from token to token, in 16-byte pieces
bool rows_ok(const void* p, int64_t stride, int elt) {
    return p && aligned(p, 16) && stride >= 0 && stride * elt % 16 == 0;
}

// what both writes check and fill in alike; rope may be null where `plain` is allowed
int fill(pkv::RopeWriteLaunch* r, const void* k, int64_t k_stride, const void* v,
         int64_t v_stride, int32_t kv_dtype, const pkv_rope* rope, bool plain,
         const int32_t* block_table, int32_t max_blocks_per_seq, int32_t num_seqs,
         const int32_t* token_seq, const int32_t* token_pos, int64_t num_tokens, void* k_cache,
         void* v_cache, const pkv_geom* g) {
    const int elt = elt_size(kv_dtype);
    if (!elt || num_tokens < 0 || max_blocks_per_seq < 0 || num_seqs < 0 || (!rope && !plain))
        return PKV_ERR_INVALID;
    if (num_tokens > kMaxTokens) return PKV_ERR_UNSUPPORTED;
    if (rope && (rope->rotary_dim < 16 || rope->rotary_dim > g->head_dim ||
                 rope->rotary_dim % 16 || rope->num_positions < 0))
        return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    if (!rows_ok(k, k_stride, elt) || !rows_ok(v, v_stride, elt) || !token_seq || !token_pos ||
        !k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return PKV_ERR_INVALID;
    if (num_seqs > 0 && max_blocks_per_seq > 0 && !block_table) return PKV_ERR_INVALID;
    r->k = k;
    r->v = v;
    r->src_dtype = kv_dtype;
    r->k_stride = k_stride;
    r->v_stride = v_stride;
    r->token_seq = token_seq;
    r->token_pos = token_pos;
    r->num_tokens = num_tokens;
    r->table = block_table;
    r->num_seqs = num_seqs;
    r->max_blocks = max_blocks_per_seq;
    if (rope) {
        if (!rope->cos_sin || !aligned(rope->cos_sin, 16)) return PKV_ERR_INVALID;
        r->cos_sin = rope->cos_sin;
        r->positions = rope->num_positions;
        r->rot = rope->rotary_dim;
        r->interleaved = rope->interleaved;
        r->rope_pos = rope->positions;
        if (rope->q) {
            if (!rows_ok(rope->q, rope->q_stride, elt) ||
                !rows_ok(rope->q_out, rope->q_out_stride, elt) ||
                rope->q_out_stride < (int64_t)g->num_heads * g->head_dim)
                return PKV_ERR_INVALID;
            // in place: a row must not land on another token's
            if (rope->q == rope->q_out && rope->q_stride != rope->q_out_stride && num_tokens > 1)
                return PKV_ERR_INVALID;
            r->q = rope->q;
            r->q_out = rope->q_out;
            r->q_stride = rope->q_stride;
            r->q_out_stride = rope->q_out_stride;
        }
    }
    r->k_cache = k_cache;
    r->v_cache = v_cache;
    r->cache_dtype = g->dtype;
    r->hq = g->num_heads;
    r->hkv = g->num_kv_heads;
    r->d = g->head_dim;
    r->block_size = g->block_size;
    r->num_blocks = g->num_blocks;
    return PKV_OK;
}

}  // namespace

extern "C" {

int paged_kv_write_rope(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                        int32_t kv_dtype, const pkv_rope* rope, const int32_t* block_table,
                        int32_t max_blocks_per_seq, int32_t num_seqs, const int32_t* token_seq,
                        const int32_t* token_pos, int64_t num_tokens, int32_t* slot_mapping_out,
                        void* k_cache, void* v_cache, const pkv_geom* geom, cudaStream_t stream) {
    if (!geom || !elt_size(geom->dtype)) return PKV_ERR_INVALID;
    int st = check_heads(geom);
    if (st != PKV_OK) return st;
    pkv::RopeWriteLaunch r{};
    st = fill(&r, k, k_stride, v, v_stride, kv_dtype, rope, false, block_table, max_blocks_per_seq,
              num_seqs, token_seq, token_pos, num_tokens, k_cache, v_cache, geom);
    if (st != PKV_OK || num_tokens == 0) return st;
    DeviceInfo dev;
    if (pkv::current_device_info(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    r.slots_out = slot_mapping_out;
    r.err = dev.err;
    return cuda_status(pkv::launch_rope_write(r, stream));
}

int paged_kv_write_q8(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                      int32_t kv_dtype, const pkv_rope* rope, const int32_t* block_table,
                      int32_t max_blocks_per_seq, int32_t num_seqs, const int32_t* token_seq,
                      const int32_t* token_pos, int64_t num_tokens, void* k_cache, void* v_cache,
                      float* k_scale, float* v_scale, const pkv_geom* geom, cudaStream_t stream) {
    int st = check_q8_geom(geom);
    if (st != PKV_OK) return st;
    pkv::RopeWriteLaunch r{};
    st = fill(&r, k, k_stride, v, v_stride, kv_dtype, rope, true, block_table, max_blocks_per_seq,
              num_seqs, token_seq, token_pos, num_tokens, k_cache, v_cache, geom);
    if (st != PKV_OK || num_tokens == 0) return st;
    if (!k_scale || !v_scale) return PKV_ERR_INVALID;
    DeviceInfo dev;
    if (pkv::current_device_info(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    r.err = dev.err;
    return cuda_status(pkv::launch_q8_write(dev, r, k_scale, v_scale, stream));
}

int paged_kv_read_q8(const void* k_cache, const void* v_cache, const float* k_scale,
                     const float* v_scale, const int32_t* slot_mapping, int64_t num_tokens,
                     void* k_out, void* v_out, int32_t kv_dtype, const pkv_geom* geom,
                     cudaStream_t stream) {
    const int st = check_q8_geom(geom);
    if (st != PKV_OK) return st;
    if (!elt_size(kv_dtype) || num_tokens < 0) return PKV_ERR_INVALID;
    if (num_tokens > kMaxTokens) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (!k_out || !v_out || !slot_mapping || !k_cache || !v_cache || !k_scale || !v_scale)
        return PKV_ERR_INVALID;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16))
        return PKV_ERR_INVALID;
    DeviceInfo dev;
    if (pkv::current_device_info(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    return cuda_status(pkv::launch_q8_read(
        k_cache, v_cache, k_scale, v_scale, slot_mapping, num_tokens, k_out, v_out, kv_dtype,
        geom->num_kv_heads, geom->head_dim, geom->block_size, geom->num_blocks * geom->block_size,
        dev.err, stream));
}

size_t paged_decode_q8_workspace_size(int32_t batch, int32_t q_dtype, const pkv_geom* geom) {
    if (check_q8_geom(geom) != PKV_OK || batch < 0 || !elt_size(q_dtype)) return 0;
    DeviceInfo dev;
    if (pkv::current_device_info(&dev) != cudaSuccess) return 0;
    pkv::Q8DecodePlan plan;
    if (!pkv::plan_q8_decode(dev, batch, 0, geom->num_heads, geom->num_kv_heads, geom->head_dim,
                             geom->block_size, geom->num_blocks, q_dtype, &plan))
        return 0;
    return plan.ws_bytes;
}

int paged_decode_q8(const void* q, int32_t q_dtype, const void* k_cache, const void* v_cache,
                    const float* k_scale, const float* v_scale, const int32_t* block_table,
                    int32_t max_blocks_per_seq, const int32_t* cache_seqlens, int32_t batch,
                    float scale, void* out, void* workspace, size_t workspace_bytes,
                    const pkv_geom* geom, cudaStream_t stream) {
    const int st = check_q8_geom(geom);
    if (st != PKV_OK) return st;
    if (!elt_size(q_dtype) || batch < 0 || max_blocks_per_seq < 0) return PKV_ERR_INVALID;
    if (batch == 0) return PKV_OK;
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !cache_seqlens || !out ||
        (max_blocks_per_seq > 0 && !block_table))
        return PKV_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
        return PKV_ERR_INVALID;
    DeviceInfo dev;
    if (pkv::current_device_info(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    pkv::Q8DecodePlan plan;
    if (!pkv::plan_q8_decode(dev, batch, max_blocks_per_seq, geom->num_heads, geom->num_kv_heads,
                             geom->head_dim, geom->block_size, geom->num_blocks, q_dtype, &plan))
        return PKV_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < plan.ws_bytes || !aligned(workspace, 256))
        return PKV_ERR_WORKSPACE;
    return cuda_status(pkv::launch_q8_decode(
        dev, plan, q, k_cache, v_cache, k_scale, v_scale, block_table, max_blocks_per_seq,
        cache_seqlens, batch, scale, out, workspace, geom->num_heads, geom->num_kv_heads,
        geom->head_dim, geom->block_size, geom->num_blocks, q_dtype, dev.err, stream));
}

}  // extern "C"
