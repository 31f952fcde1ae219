// q4_api.cu -- the extern "C" entry points of 4-bit K/V pools and of cache
// compaction (declared in include/pagedkv.h): argument checks and dispatch.
#include "common.cuh"
#include "launch.h"
#include "q4.cuh"

using pkv::DeviceInfo;
using pkv::aligned;
using pkv::elt_size;

namespace {

// batch int32 values at a and at b share some, but are not one array
bool straddle(const int32_t* a, const int32_t* b, int64_t n) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x != y && (x < y ? y - x : x - y) < (uintptr_t)n * sizeof(int32_t);
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA; }

// the geometry of a call on 4-bit pools (geom->dtype PKV_Q4)
int check_q4_geom(const pkv_geom* g) {
    if (!g || g->dtype != PKV_Q4) return PKV_ERR_INVALID;
    pkv_geom as = *g;  // the checks every pool shares
    as.dtype = PKV_BF16;
    const int st = pkv::check_geom(&as);
    if (st != PKV_OK) return st;
    return g->head_dim == 64 || g->head_dim == 128 ? PKV_OK : PKV_ERR_UNSUPPORTED;
}

// the write and the read count a token's row in 32 bits, 8 values at a time
bool row_too_long(const pkv_geom* g) { return (int64_t)g->num_kv_heads * g->head_dim > (1 << 30); }

// rows' worth of grid: one warp per token, 4 tokens per CTA
constexpr int64_t kMaxTokens = (int64_t)4 * 0x7fffffff;

}  // namespace

extern "C" {

int paged_kv_write_q4(const void* k, const void* v, int32_t kv_dtype, const int32_t* slot_mapping,
                      int64_t num_tokens, void* k_cache, void* v_cache, const pkv_geom* geom,
                      cudaStream_t stream) {
    const int st = check_q4_geom(geom);
    if (st != PKV_OK) return st;
    if (!elt_size(kv_dtype) || num_tokens < 0 || num_tokens > kMaxTokens) return PKV_ERR_INVALID;
    if (row_too_long(geom)) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_mapping || !k_cache || !v_cache) return PKV_ERR_INVALID;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return PKV_ERR_INVALID;
    DeviceInfo dev;
    if (pkv::current_device_info(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    return cuda_status(pkv::launch_q4_write(k, v, kv_dtype, slot_mapping, num_tokens, k_cache,
                                            v_cache, geom->num_kv_heads, geom->head_dim,
                                            geom->block_size,
                                            geom->num_blocks * geom->block_size, dev.err, stream));
}

int paged_kv_read_q4(const void* k_cache, const void* v_cache, const int32_t* slot_mapping,
                     int64_t num_tokens, void* k_out, void* v_out, int32_t kv_dtype,
                     const pkv_geom* geom, cudaStream_t stream) {
    const int st = check_q4_geom(geom);
    if (st != PKV_OK) return st;
    if (!elt_size(kv_dtype) || num_tokens < 0 || num_tokens > kMaxTokens) return PKV_ERR_INVALID;
    if (row_too_long(geom)) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (!k_out || !v_out || !slot_mapping || !k_cache || !v_cache) return PKV_ERR_INVALID;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16))
        return PKV_ERR_INVALID;
    DeviceInfo dev;
    if (pkv::current_device_info(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    return cuda_status(pkv::launch_q4_read(k_cache, v_cache, slot_mapping, num_tokens, k_out,
                                           v_out, kv_dtype, geom->num_kv_heads, geom->head_dim,
                                           geom->block_size,
                                           geom->num_blocks * geom->block_size, dev.err, stream));
}

size_t paged_decode_q4_workspace_size(int32_t batch, int32_t q_dtype, const pkv_geom* geom) {
    if (check_q4_geom(geom) != PKV_OK || batch < 0 || !elt_size(q_dtype)) return 0;
    DeviceInfo dev;
    if (pkv::current_device_info(&dev) != cudaSuccess) return 0;
    pkv::Q4DecodePlan plan;
    if (!pkv::plan_q4_decode(dev, batch, 0, geom->num_heads, geom->num_kv_heads, geom->head_dim,
                             geom->block_size, q_dtype, &plan))
        return 0;
    return plan.ws_bytes;
}

int paged_decode_q4(const void* q, int32_t q_dtype, const void* k_cache, const void* v_cache,
                    const int32_t* block_table, int32_t max_blocks_per_seq,
                    const int32_t* cache_seqlens, int32_t batch, float scale, void* out,
                    void* workspace, size_t workspace_bytes, const pkv_geom* geom,
                    cudaStream_t stream) {
    const int st = check_q4_geom(geom);
    if (st != PKV_OK) return st;
    if (!elt_size(q_dtype) || batch < 0 || max_blocks_per_seq < 0) return PKV_ERR_INVALID;
    if (batch == 0) return PKV_OK;
    if (!q || !k_cache || !v_cache || !block_table || !cache_seqlens || !out)
        return PKV_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
        return PKV_ERR_INVALID;
    DeviceInfo dev;
    if (pkv::current_device_info(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    pkv::Q4DecodePlan plan;
    if (!pkv::plan_q4_decode(dev, batch, max_blocks_per_seq, geom->num_heads, geom->num_kv_heads,
                             geom->head_dim, geom->block_size, q_dtype, &plan))
        return PKV_ERR_UNSUPPORTED;
    if (plan.ws_bytes &&
        (!workspace || workspace_bytes < plan.ws_bytes || !aligned(workspace, 256)))
        return PKV_ERR_WORKSPACE;
    return cuda_status(pkv::launch_q4_decode(
        dev, plan, q, k_cache, v_cache, block_table, max_blocks_per_seq, cache_seqlens, batch, scale,
        out, workspace, geom->num_heads, geom->num_kv_heads, geom->head_dim, geom->block_size,
        geom->num_blocks, q_dtype, dev.err, stream));
}

int paged_kv_compact(void* k_cache, void* v_cache, const int32_t* block_table,
                     int32_t max_blocks_per_seq, const int32_t* start, const int32_t* keep,
                     int32_t total_keep, const int32_t* cu_keep, int32_t batch,
                     int32_t* seqlens_out, const pkv_geom* geom, cudaStream_t stream) {
    if (!geom) return PKV_ERR_INVALID;
    const int st = geom->dtype == PKV_Q4 ? check_q4_geom(geom) : pkv::check_geom(geom);
    if (st != PKV_OK) return st;
    if (batch < 0 || max_blocks_per_seq < 0 || total_keep < 0) return PKV_ERR_INVALID;
    if (batch == 0) return PKV_OK;
    if (batch > 65535) return PKV_ERR_UNSUPPORTED;  // one grid row per sequence
    if (straddle(start, seqlens_out, batch)) return PKV_ERR_INVALID;
    if (!cu_keep || (total_keep > 0 && (!keep || !block_table || !k_cache || !v_cache)))
        return PKV_ERR_INVALID;
    // positions are int32
    if ((double)max_blocks_per_seq * geom->block_size > 2147483647.0) return PKV_ERR_UNSUPPORTED;
    const bool q4 = geom->dtype == PKV_Q4;
    const int align = q4 ? 16 : elt_size(geom->dtype);
    if (!aligned(k_cache, align) || !aligned(v_cache, align)) return PKV_ERR_INVALID;
    pkv::CompactLaunch c{};
    c.k_cache = k_cache;
    c.v_cache = v_cache;
    c.table = block_table;
    c.start = start;
    c.keep = keep;
    c.cu_keep = cu_keep;
    c.seqlens_out = seqlens_out;
    c.num_blocks = geom->num_blocks;
    c.max_blocks = max_blocks_per_seq;
    c.block_size = geom->block_size;
    c.batch = batch;
    c.total = total_keep;
    if (q4) {  // [block][head][token][row]
        c.pieces = geom->num_kv_heads;
        c.piece_bytes = pkv::q4_row_bytes(geom->head_dim);
        c.token_bytes = c.piece_bytes;
        c.head_bytes = c.piece_bytes * geom->block_size;
    } else {  // [block][token][heads and dims]
        c.pieces = 1;
        c.piece_bytes = (int64_t)geom->num_kv_heads * geom->head_dim * elt_size(geom->dtype);
        c.token_bytes = c.piece_bytes;
        c.head_bytes = 0;
    }
    c.page_bytes = c.pieces * c.piece_bytes * geom->block_size;
    if (c.pieces * c.piece_bytes > (1 << 24)) return PKV_ERR_UNSUPPORTED;
    // pools that share rows: K's moves and V's, in no order, would move some twice
    const uintptr_t kp = reinterpret_cast<uintptr_t>(k_cache);
    const uintptr_t vp = reinterpret_cast<uintptr_t>(v_cache);
    const uintptr_t pool_bytes = (uintptr_t)(geom->num_blocks * c.page_bytes);
    if (total_keep > 0 && (kp < vp ? vp - kp : kp - vp) < pool_bytes)
        return PKV_ERR_INVALID;
    DeviceInfo dev;
    if (pkv::current_device_info(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    return cuda_status(pkv::launch_compact(dev, c, stream));
}

}  // extern "C"
