/*
 * pagedkv.h -- C ABI of the GB300 (sm_103a) paged KV-cache attention library
 * (libpagedkv.so).
 *
 * The library implements the data-parallel hot path of paged attention:
 *   - the slot_mapping KV-cache write (new K/V rows scattered into the paged
 *     pool, negative slots skipped);
 *   - one-query-per-sequence decode that reads K/V through a block table and
 *     merges blocks with the online-softmax rule (split over the keys of long
 *     sequences, partial states merged by the same rule);
 *   - causal varlen prefill over cu_seqlens_q / cu_seqlens_k that reads the
 *     paged prior context (prefix cache / chunked prefill) on the tensor cores.
 *
 * Sources: "11. Paged attention 与 online softmax" (dilfish.github.io), §11.1
 * block table and offset equation, §11.2 boxed merge equation;
 * "从零开始写Qwen3（六）PagedAttention" (mlqm.cn), sections "fast-attn 库的使用"
 * (the varlen / kvcache call shapes and their parameters) and "自己来实现一个"
 * (the slot_mapping write kernel); "Sayfalı dikkat" (Hugging Face transformers
 * docs), varlen path (cu_seq_lens) and decode path (block_table, cache_seqlens).
 *
 * Conventions shared by every call
 * --------------------------------
 * Memory.  Every pointer argument is a DEVICE pointer unless stated otherwise
 * (pkv_geom is read on the host).  The caller owns every buffer; the library
 * allocates no device memory.  Calls are asynchronous on `stream` and never
 * synchronise the host, except paged_error_flags.
 * Ordering.  Work enqueued on `stream` before a call completes before the
 * call reads anything, and work enqueued after it sees all of its results,
 * as for any stream-ordered launch.  The library's kernels are launched as
 * programmatic dependents of the kernel before them and let the next kernel
 * launch early (programmatic dependent launch).  This matters only to a
 * caller kernel that is itself launched after a call with the
 * programmatic-stream-serialization attribute: it may start before the call's
 * kernels finish, and must execute griddepcontrol.wait
 * (cudaGridDependencySynchronize) before it reads their results.
 * Layouts (row-major, contiguous):
 *   K/V pools  [num_blocks, block_size, num_kv_heads, head_dim]; the element
 *              offset of logical position p of a sequence whose block-table row
 *              is t is (t[p / B] * B + p % B) * kvDim, kvDim = Hkv * head_dim.
 *   block_table [rows, max_blocks_per_seq] int32; entries past a sequence's
 *              length are never read and may hold -1.
 *   q / out    decode [batch, Hq, head_dim]; prefill [total_q, Hq, head_dim].
 *   index arrays are int32.
 * GQA: query head h reads KV head h / (Hq / Hkv).
 * dtype: q, out and both pools share pkv_geom.dtype.
 * Return codes: PKV_OK, or a negative PKV_ERR_* (no work is enqueued then).
 * Device-side checks: an out-of-range block id, slot or sequence length found
 * while a kernel runs is skipped (never dereferenced) and recorded in a
 * per-device error word read by paged_error_flags.
 */
#ifndef PAGEDKV_H
#define PAGEDKV_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
/* PKV_Q4, PKV_Q8: 4-bit and 8-bit pools, for the calls that name them ("4-bit pools",
 * "8-bit pools" below) */
typedef enum pkv_dtype { PKV_F32 = 0, PKV_BF16 = 1, PKV_Q4 = 2, PKV_Q8 = 3 } pkv_dtype;

/* status codes */
#define PKV_OK 0
#define PKV_ERR_INVALID (-1)     /* null pointer, bad size, Hq % Hkv != 0, misaligned */
#define PKV_ERR_UNSUPPORTED (-2) /* valid but not implemented (dtype/head_dim/GQA combo) */
#define PKV_ERR_WORKSPACE (-3)   /* workspace missing or smaller than the *_workspace_size */
#define PKV_ERR_CUDA (-4)        /* a CUDA runtime call or kernel launch failed */
#define PKV_ERR_NO_SPACE (-5)    /* block manager: not enough free blocks (nothing changed) */

/* device error-word bits (paged_error_flags) */
#define PKV_FLAG_BAD_BLOCK (1u << 0)   /* block-table entry outside [0, num_blocks) */
#define PKV_FLAG_BAD_SLOT (1u << 1)    /* slot_mapping entry >= num_blocks * block_size */
#define PKV_FLAG_BAD_LENGTH (1u << 2)  /* length < 0 or beyond max_blocks_per_seq * B */
#define PKV_FLAG_BAD_SEQ (1u << 3)     /* token sequence index >= num_seqs */
#define PKV_FLAG_TIMEOUT (1u << 4)     /* a pipeline wait gave up (kernel returned early) */

/* Geometry of one paged pool (one layer's K pool and V pool). */
typedef struct pkv_geom {
    int32_t num_heads;    /* Hq, query heads */
    int32_t num_kv_heads; /* Hkv, KV heads; Hq % Hkv == 0 */
    int32_t head_dim;     /* d */
    int32_t block_size;   /* B, tokens per physical block (page) */
    int64_t num_blocks;   /* physical blocks in each pool */
    int32_t dtype;        /* pkv_dtype of q, out and the pools */
} pkv_geom;

/*
 * paged_build_slot_mapping -- address translation for the new tokens of a step.
 * ("11. Paged attention 与 online softmax" §11.1: logical block p / B, slot
 * p mod B, phys = table[p / B]; "自己来实现一个": the per-token index is
 * computed once and reused by every layer.)
 *   slot_mapping[n] = block_table[s][p / B] * B + p % B with s = token_seq[n],
 *   p = token_pos[n]; token_seq[n] < 0 marks a padding row -> -1.
 *   block_table [num_seqs, max_blocks_per_seq]; token_seq, token_pos,
 *   slot_mapping [num_tokens].  Out-of-range s, p or table entries give -1 and
 *   set PKV_FLAG_BAD_SEQ / _BAD_LENGTH / _BAD_BLOCK.
 */
int paged_build_slot_mapping(const int32_t* block_table, int32_t max_blocks_per_seq,
                             int32_t num_seqs, const int32_t* token_seq,
                             const int32_t* token_pos, int64_t num_tokens, int32_t block_size,
                             int32_t* slot_mapping, cudaStream_t stream);

/*
 * paged_kv_write -- the slot_mapping cache write ("自己来实现一个",
 * _update_paged_kv_cache_kernel).  For every token n with s = slot_mapping[n]
 * >= 0: k_cache[s*kvDim + j] = cast(k[n*kvDim + j]) and likewise for v,
 * j < kvDim; s < 0 writes nothing.  k, v [num_tokens, Hkv, d] of kv_dtype; the
 * pools of geom->dtype.  fp32 -> bf16 rounds to nearest even; equal dtypes
 * copy bits.  Duplicate non-negative slots are a caller error (the surviving
 * row is unspecified).  s >= num_blocks*B is skipped and sets PKV_FLAG_BAD_SLOT.
 */
int paged_kv_write(const void* k, const void* v, int32_t kv_dtype, const int32_t* slot_mapping,
                   int64_t num_tokens, void* k_cache, void* v_cache, const pkv_geom* geom,
                   cudaStream_t stream);

/*
 * paged_kv_write_positions -- paged_build_slot_mapping and paged_kv_write in
 * one launch: token n's slot is block_table[s][p / B] * B + p % B with
 * s = token_seq[n], p = token_pos[n] ("11. Paged attention 与 online softmax"
 * §11.1; "自己来实现一个" computes it once per step for every layer), and its
 * K and V rows are written there as paged_kv_write does.  The slots are also
 * stored in slot_mapping_out [num_tokens] when it is not NULL, so that the
 * other layers of the step can call paged_kv_write with them.  token_seq[n] < 0
 * marks a padding row (slot -1, nothing written).  Out-of-range s, p or table
 * entries give slot -1 (nothing written) and set PKV_FLAG_BAD_SEQ /
 * _BAD_LENGTH / _BAD_BLOCK; a slot >= num_blocks * B sets PKV_FLAG_BAD_SLOT.
 * Arguments as for the two calls it replaces.
 */
int paged_kv_write_positions(const void* k, const void* v, int32_t kv_dtype,
                             const int32_t* block_table, int32_t max_blocks_per_seq,
                             int32_t num_seqs, const int32_t* token_seq,
                             const int32_t* token_pos, int64_t num_tokens,
                             int32_t* slot_mapping_out, void* k_cache, void* v_cache,
                             const pkv_geom* geom, cudaStream_t stream);

/*
 * paged_decode_workspace_size -- bytes of device scratch paged_decode needs for
 * `batch` sequences on the CURRENT device (the split plan depends on its SM
 * count).  Returns 0 for invalid arguments.  There is no max_seqlen_k
 * argument: the keys of all sequences are cut into one share per CTA, so the
 * scratch holds (CTAs + batch) partial states whatever the lengths are, and
 * the lengths themselves are device data the host need not know.  On the
 * tensor-core path (below) it adds c partial states per (sequence, query
 * head), c = min(32, ceil(SMs / (batch * Hkv))).
 */
size_t paged_decode_workspace_size(int32_t batch, const pkv_geom* geom);

/*
 * paged_decode -- paged attention of one query token per sequence ("Sayfalı
 * dikkat" decode path; "11. Paged attention 与 online softmax" §11.1-§11.2).
 * Sequence b attends over exactly cache_seqlens[b] keys (positions 0 ..
 * cache_seqlens[b]-1, read through block_table row b), i.e. the new token's
 * K/V must already have been written with paged_kv_write.
 *   out[b,h,:] = sum_j softmax_j(scale * q[b,h,:] . k_j) v_j  over those keys,
 *   0 when cache_seqlens[b] == 0.
 * The keys of all sequences are cut into shares, one per CTA (equal once each
 * sequence start is counted as one tile of keys); each CTA keeps the (m, l, o)
 * online-softmax state of its share and a second kernel merges the shares of
 * each sequence with the same rule and normalises.
 * Tensor-core path: bf16 with G = Hq/Hkv >= 4 (and dividing 128), and block
 * sizes the shared-prefix pass takes (multiples of 128, or divisors of 128 of
 * at least 8).  There the keys of each sequence are attended on the tensor
 * cores in c chunks of ceil(max_blocks_per_seq * B / c) keys rounded up to
 * 128, one work item per (sequence, KV head, chunk) with the G query heads as
 * rows of one MMA tile (keys past the length in the last page are masked, and
 * their V rows zeroed in shared memory); the same second kernel merges the
 * chunks' states (two launches, no split).
 * Supported: head_dim 64 or 128; fp32 or bf16; G = Hq/Hkv in {1, 2, 4, 8, 16,
 * 32} (from 8 up, G/4 warps per KV head, 4 query heads each, share its K/V
 * tiles); with s = 8 / max(1, G/4) KV heads per CTA, Hkv divides s or is a
 * multiple of s; any block_size >= 1; batch <= 4096.
 * Like its workspace-size call it takes no max_seqlen_k: nothing in the launch
 * depends on the longest sequence.
 * workspace: device scratch of at least paged_decode_workspace_size(batch, geom)
 * bytes, 256-byte aligned, contents irrelevant on entry; it must not be used by
 * another call that runs concurrently.
 */
int paged_decode(const void* q, const void* k_cache, const void* v_cache,
                 const int32_t* block_table, int32_t max_blocks_per_seq,
                 const int32_t* cache_seqlens, int32_t batch, float scale, void* out,
                 void* workspace, size_t workspace_bytes, const pkv_geom* geom,
                 cudaStream_t stream);

/*
 * paged_decode_append -- paged_decode with the in-place append of the new
 * token ("Sayfalı dikkat" decode path: the flash_attn_with_kvcache call takes
 * the new k and v, writes them into the cache and attends over them together
 * with the cached keys).  cache_seqlens[b] counts the keys cached BEFORE this
 * step.  For every sequence b:
 *   - k_new[b], v_new[b] ([batch, Hkv, d], the cache dtype) are written at
 *     position cache_seqlens[b] (slot = block_table[b][L / B] * B + L % B);
 *   - out[b,h] = attention of q[b,h] over the cache_seqlens[b] cached keys
 *     and the new key (cache_seqlens[b] + 1 keys in all).
 * The caller advances cache_seqlens afterwards.  The new key is scored from
 * k_new directly (not read back from the cache) and written after the cached
 * keys have been read.  Supported, workspace and errors as paged_decode (same
 * workspace size); a position past max_blocks_per_seq * B or a bad table
 * entry skips that write and sets PKV_FLAG_BAD_LENGTH / _BAD_BLOCK.
 */
int paged_decode_append(const void* q, const void* k_new, const void* v_new, void* k_cache,
                        void* v_cache, const int32_t* block_table, int32_t max_blocks_per_seq,
                        const int32_t* cache_seqlens, int32_t batch, float scale, void* out,
                        void* workspace, size_t workspace_bytes, const pkv_geom* geom,
                        cudaStream_t stream);

/*
 * paged_varlen_prefill_workspace_size -- bytes of device scratch
 * paged_varlen_prefill needs (0 when it needs none).  Returns 0 for invalid
 * arguments as well.
 */
size_t paged_varlen_prefill_workspace_size(int32_t batch, int32_t max_seqlen_q,
                                           const pkv_geom* geom);

/*
 * paged_varlen_prefill -- causal varlen prefill over a paged cache
 * ("从零开始写Qwen3（六）PagedAttention", "fast-attn 库的使用": prefix cache and
 * chunked prefill read the cache through block_table; "Sayfalı dikkat" varlen
 * path).  Request r owns query rows [cu_seqlens_q[r], cu_seqlens_q[r+1]) of q
 * and keys 0 .. k_len-1, k_len = cu_seqlens_k[r+1] - cu_seqlens_k[r], read
 * through block_table row r (the new tokens' K/V must already be written).
 * With causal != 0 query i of a request with q_len queries sees key j iff
 * j <= i + k_len - q_len (bottom-right alignment: the queries are the last
 * q_len positions); a row that sees no key outputs 0.
 * max_seqlen_q / max_seqlen_k are host-side upper bounds of the per-request
 * lengths (they size the launch).  q, out [total_q, Hq, d].
 * Contiguous mode ("从零开始写Qwen3（六）PagedAttention", "一个小细节": without
 * a prefix cache the varlen call reads packed K/V): block_table == NULL makes
 * k_cache / v_cache packed arrays [rows, Hkv, d] with rows = geom->num_blocks
 * * geom->block_size (any factorisation, e.g. block_size 1), and request r's
 * keys are rows cu_seqlens_k[r] .. cu_seqlens_k[r+1]-1; max_blocks_per_seq is
 * ignored.  Keys past row `rows` are flagged PKV_FLAG_BAD_LENGTH.
 * Supported: bf16, head_dim 64 or 128, Hq/Hkv in {1, 2, 4, 8, ...}; paged
 * mode: a block_size that is a multiple of 128 or divides 128 and is >= 8.
 */
int paged_varlen_prefill(const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t batch,
                         int32_t max_seqlen_q, int32_t max_seqlen_k, const int32_t* block_table,
                         int32_t max_blocks_per_seq, int32_t causal, float scale, void* out,
                         void* workspace, size_t workspace_bytes, const pkv_geom* geom,
                         cudaStream_t stream);

/*
 * paged_decode_shared_prefix -- paged_decode for batches whose sequences come
 * in groups that share the physical blocks of a common prefix ("11. Paged
 * attention 与 online softmax" §11.3 block sharing; the prefix cache of
 * "结合nanovllm的FlashAttention和PagedAttention主要原理概述" 题目6), reading each
 * shared block once per group instead of once per sequence.
 *   group_cu [n_groups + 1] (device): group g is sequences group_cu[g] ..
 *   group_cu[g+1]-1 of the batch (group_cu[0] = 0, group_cu[n_groups] =
 *   batch: the batch is ordered by group; a sequence sharing nothing is a
 *   group of one with prefix 0).  group_prefix_len [n_groups] (device): the
 *   leading keys every sequence of group g holds in the same physical blocks,
 *   a multiple of block_size and at most each member's cache_seqlens; the
 *   prefix blocks are read through the table row of the group's first
 *   sequence.  max_group_size: a host-side bound of the group sizes.
 * The result is paged_decode's (same arguments and layouts otherwise): the
 * prefix part is the attention of the group's queries over the prefix keys
 * (one pass over them, on the tensor cores), the rest the decode of each
 * sequence's own keys, merged with §11.2's boxed rule.
 * Supported: bf16, head_dim 64 or 128, Hq/Hkv and Hkv as for paged_decode,
 * block_size a multiple of 128 or a divisor of 128 (>= 8).
 * workspace: at least
 * paged_decode_shared_prefix_workspace_size(batch, geom) bytes, 256-byte
 * aligned.  A prefix length that is negative, longer than a member's keys or
 * not a multiple of block_size sets PKV_FLAG_BAD_LENGTH.
 */
size_t paged_decode_shared_prefix_workspace_size(int32_t batch, const pkv_geom* geom);
int paged_decode_shared_prefix(const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_table, int32_t max_blocks_per_seq,
                               const int32_t* cache_seqlens, int32_t batch,
                               const int32_t* group_cu, const int32_t* group_prefix_len,
                               int32_t n_groups, int32_t max_group_size, float scale, void* out,
                               void* workspace, size_t workspace_bytes, const pkv_geom* geom,
                               cudaStream_t stream);

/*
 * paged_mixed_step -- one continuous-batching step in one call: prefill
 * requests and decode sequences over the same pools ("从零开始写Qwen3（六）
 * PagedAttention", "fast-attn 库的使用": the varlen call for prefill, the
 * kvcache call for decode; "11. Paged attention 与 online softmax" §11.3 for
 * groups sharing a prefix).  In order on `stream`:
 *   1. the prefill requests' new K/V rows are written at prefill_slots
 *      (paged_kv_write; negative slots skipped);
 *   2. causal varlen prefill of the prefill requests (paged_varlen_prefill);
 *   3. decode of the decode sequences with the in-place append
 *      (paged_decode_append), through the shared-prefix path when n_groups > 0
 *      (paged_decode_shared_prefix semantics).
 * Parts with a zero count are skipped.  The decode kernels are launched as
 * programmatic dependents of the prefill kernel, which they do not read: they
 * start on SMs the prefill leaves free instead of after it.  Arguments mean
 * what they mean in the single calls; all pointers in the struct are DEVICE
 * pointers.  Supported as the single calls; with a prefill part or groups:
 * bf16 and head_dim 64 or 128.  workspace: at least
 * paged_mixed_step_workspace_size(decode_batch, geom) bytes, 256-byte aligned.
 */
typedef struct pkv_mixed_step {
    /* prefill requests */
    const void* prefill_k_new;   /* [prefill_new_tokens, Hkv, d] */
    const void* prefill_v_new;
    const int32_t* prefill_slots; /* [prefill_new_tokens] */
    int64_t prefill_new_tokens;
    const void* prefill_q;        /* [total_q, Hq, d] */
    const int32_t* cu_seqlens_q;  /* [prefill_batch + 1] */
    const int32_t* cu_seqlens_k;
    int32_t prefill_batch;
    int32_t max_seqlen_q;
    int32_t max_seqlen_k;
    const int32_t* prefill_table; /* [prefill_batch, prefill_max_blocks] */
    int32_t prefill_max_blocks;
    void* prefill_out;            /* [total_q, Hq, d] */
    /* decode sequences (in-place append) */
    const void* decode_q;         /* [decode_batch, Hq, d] */
    const void* decode_k_new;     /* [decode_batch, Hkv, d] */
    const void* decode_v_new;
    const int32_t* decode_table;  /* [decode_batch, decode_max_blocks] */
    int32_t decode_max_blocks;
    const int32_t* decode_seqlens; /* keys cached before the step */
    int32_t decode_batch;
    const int32_t* group_cu;      /* [n_groups + 1], or NULL with n_groups 0 */
    const int32_t* group_prefix_len;
    int32_t n_groups;
    int32_t max_group_size;
    void* decode_out;             /* [decode_batch, Hq, d] */
    float scale;
} pkv_mixed_step;

size_t paged_mixed_step_workspace_size(int32_t decode_batch, const pkv_geom* geom);
int paged_mixed_step(const pkv_mixed_step* step, void* k_cache, void* v_cache, void* workspace,
                     size_t workspace_bytes, const pkv_geom* geom, cudaStream_t stream);

/*
 * paged_mixed_step_one_launch -- paged_mixed_step's result from ONE kernel
 * launch (plus a 16-byte memset of its counters): the prefill rows' write, the
 * shared-prefix and causal-prefill work items on the tensor cores, the decode
 * split and the combine with the append run as CTAs of one grid, in that
 * order of block index; a CTA that needs earlier results (a prefill item the
 * write, a combine CTA the prefix items and the split) waits until their
 * counters are complete (time-limited: PKV_FLAG_TIMEOUT).  Same arguments,
 * workspace and errors as paged_mixed_step.  It takes full steps (prefill
 * rows, prefill requests and grouped decode sequences) in bf16, head_dim 128,
 * with 2 query heads per KV head and at most 8 KV heads; any other step is done
 * by paged_mixed_step.  paged_mixed_step is faster on GB300 (each phase keeps
 * its own CTA shape there); this form is for callers that need a single
 * kernel launch.
 */
int paged_mixed_step_one_launch(const pkv_mixed_step* step, void* k_cache, void* v_cache,
                                void* workspace, size_t workspace_bytes, const pkv_geom* geom,
                                cudaStream_t stream);

/*
 * paged_decode_noalloc -- paged_decode for callers that cannot allocate device
 * memory.  The pages have no counterpart: this is a deployment variant of
 * paged_decode that takes no workspace.
 * Some callers cannot hand the library a scratch buffer: a plugin whose host
 * framework owns every device allocation and offers no workspace hook, or a
 * serving loop that must not call cudaMalloc because it can synchronise the
 * device and stall other streams.  This call allocates nothing (no cudaMalloc,
 * no cudaFree, no allocating library routine); its split-KV scratch is a fixed
 * device array of PKV_NOALLOC_SCRATCH_BYTES inside the library, which every
 * GPU that loads the library holds until the process exits.
 *   - Same arguments, layouts, results and support matrix as paged_decode,
 *     minus workspace / workspace_bytes.  It always takes the CUDA-core split
 *     (never paged_decode's tensor-core path), whose scratch is the array.
 *   - Returns PKV_ERR_WORKSPACE when the split needs more scratch than the
 *     array holds.  That scratch is about
 *     (SMs + batch) * Hq * (head_dim + 2) * 4 bytes, so the limit is
 *     batch <= PKV_NOALLOC_SCRATCH_BYTES / (Hq * (head_dim + 2) * 4) - SMs:
 *     about 850 sequences for Hq=16, head_dim=128 on a 152-SM GPU.
 *   - All calls share the one array, and it keeps the previous call's contents
 *     (nothing in it needs to start at zero).  Calls that overlap on the GPU
 *     race on it: order them on one stream or with events.
 *   - Set-up: the first call on each device looks up the array's device
 *     address (cudaGetSymbolAddress) with that device current.  Under lazy
 *     module loading (the CUDA default) that lookup also loads the module that
 *     holds the array, which may allocate and synchronise.  A call with
 *     batch 0 does this set-up alone (and nothing else): make it once per
 *     device at initialisation, before any stream capture, or run with
 *     CUDA_MODULE_LOADING=EAGER.  The looked-up address is cached; after
 *     cudaDeviceReset the library must not be used on that device again.
 */
#define PKV_NOALLOC_SCRATCH_BYTES (8u << 20)
int paged_decode_noalloc(const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* block_table, int32_t max_blocks_per_seq,
                         const int32_t* cache_seqlens, int32_t batch, float scale, void* out,
                         const pkv_geom* geom, cudaStream_t stream);

/*
 * paged_error_flags -- read (and with clear != 0, reset) the device error word
 * of the current device: an OR of PKV_FLAG_* bits set by kernels since the
 * last clear.  *flags (host pointer) receives the word.
 * This call SYNCHRONISES with the device (it copies the word to the host with
 * cudaMemcpy), unlike every other call here: use it between steps, not on a
 * latency-critical path.  It replaces a plain int-returning "last error"
 * call: the word is a set of independent flag bits, so it is returned through
 * a pointer beside the status, and reading without clearing is possible.
 */
int paged_error_flags(uint32_t* flags, int32_t clear);

/*
 * Block manager (host side) and block copies -- "11. Paged attention 与 online
 * softmax" §11.3 (block sharing, copy-on-write, reference counts and the free
 * stack) and "结合nanovllm的FlashAttention和PagedAttention主要原理概述" 题目6
 * (prefix cache: chained block hashes, a hit shares the block, release in
 * reverse block order).
 *
 * A pkv_block_manager owns the bookkeeping of one pool of num_blocks blocks of
 * block_size tokens and the sequences that hold them; it makes no CUDA call and
 * is not thread-safe (callers serialise).  Every pointer of the paged_bm_*
 * calls is a HOST pointer.
 *   - refs[b] = the number of sequence block tables that contain block b; a
 *     block with refs 0 is on the free stack (top = block 0 at creation; a
 *     released block is pushed on top, allocation pops the top).
 *   - Only full blocks are shared by lookup.  The cache key of block i of a
 *     token sequence is (the physical block of block i-1, or -1; the block's
 *     block_size token ids), compared in full: two sequences share their
 *     leading full blocks exactly as far as their tokens agree.
 *   - PKV_ERR_NO_SPACE leaves the manager unchanged.
 */
typedef struct pkv_block_manager pkv_block_manager;

/* a manager of num_blocks (< 2^31) blocks of block_size (>= 1) tokens */
int paged_bm_create(int64_t num_blocks, int32_t block_size, pkv_block_manager** out);
int paged_bm_destroy(pkv_block_manager* bm);

/* New sequence holding tokens[0 .. n_tokens): its leading full blocks that are
 * cached are shared (refs +1), the rest are allocated (refs 1) and the full
 * ones cached.  *seq_out: the sequence id; *cached_tokens_out (may be NULL):
 * tokens in shared blocks, i.e. tokens whose K/V are already in the pool. */
int paged_bm_allocate(pkv_block_manager* bm, const int64_t* tokens, int64_t n_tokens,
                      int64_t* seq_out, int64_t* cached_tokens_out);

/* New sequence with the same tokens and blocks as `seq` (every block refs +1). */
int paged_bm_fork(pkv_block_manager* bm, int64_t seq, int64_t* child_out);

/* One more token for `seq`.  A full last block gets a new block after it; a
 * partial last block that is shared (refs > 1) is replaced by a new block the
 * sequence owns and *cow_src_out / *cow_dst_out name the block whose contents
 * must be copied first (paged_copy_blocks) -- otherwise both are -1.  A block
 * that the token fills enters the cache. */
int paged_bm_append(pkv_block_manager* bm, int64_t seq, int64_t token, int32_t* cow_src_out,
                    int32_t* cow_dst_out);

/* The bookkeeping of paged_kv_compact for `seq`: it keeps its tokens below
 * `start` and, of the others, those at the positions keep[0 .. n_keep)
 * (strictly ascending, in [start, length)).  Blocks behind the new end are
 * released, in reverse order.  A shared block that rows move into is replaced
 * by a new block: the *n_cow_out pairs (cow_src_out[i], cow_dst_out[i]) must be
 * copied first (paged_copy_blocks).  table_out [table_capacity, at least the
 * present table's length] receives the present table with those replacements:
 * pass it to paged_kv_compact, in stream order before any write into the
 * released blocks.  Blocks that rows move into leave the prefix cache and never
 * enter it again (their tokens no longer say what they hold), nor do the
 * sequence's later blocks; a last block that is partial now leaves it too.
 * PKV_ERR_INVALID (a capacity too small: *n_cow_out says how many pairs there
 * are) and PKV_ERR_NO_SPACE change nothing. */
int paged_bm_compact(pkv_block_manager* bm, int64_t seq, int64_t start, const int32_t* keep,
                     int64_t n_keep, int32_t* table_out, int32_t table_capacity,
                     int32_t* cow_src_out, int32_t* cow_dst_out, int32_t cow_capacity,
                     int32_t* n_cow_out);

/* Release a sequence: its blocks in reverse order, refs -1 each; a block at 0
 * leaves the cache and is pushed on the free stack. */
int paged_bm_free(pkv_block_manager* bm, int64_t seq);

/* The sequence's block table (host int32 array of `capacity` entries);
 * *n_blocks_out receives its length (also when capacity is too small, which
 * returns PKV_ERR_INVALID). */
int paged_bm_block_table(const pkv_block_manager* bm, int64_t seq, int32_t* table_out,
                         int32_t capacity, int32_t* n_blocks_out);
int paged_bm_seq_len(const pkv_block_manager* bm, int64_t seq, int64_t* len_out);
int paged_bm_ref_count(const pkv_block_manager* bm, int32_t block, int32_t* ref_out);

/* The free stack, bottom first, into stack_out[capacity] (NULL: count only);
 * *n_out receives the number of free blocks. */
int paged_bm_free_blocks(const pkv_block_manager* bm, int32_t* stack_out, int64_t capacity,
                         int64_t* n_out);

/*
 * paged_copy_blocks -- the copies a copy-on-write needs (§11.3: the old
 * contents go into the new block before the write).  For i < n_pairs, block
 * dst[i] of both pools becomes a bitwise copy of block src[i] (block_size *
 * kvDim elements of geom->dtype).  src, dst: DEVICE int32 arrays; a dst block
 * must not also be a src block or appear twice (the result is unspecified
 * then).  An id outside [0, num_blocks) skips the pair and sets
 * PKV_FLAG_BAD_BLOCK.
 */
int paged_copy_blocks(void* k_cache, void* v_cache, const int32_t* src, const int32_t* dst,
                      int32_t n_pairs, const pkv_geom* geom, cudaStream_t stream);

/*
 * 4-bit pools -- K and V held in 4 bits per value ("Sayfalı dikkat": the cache
 * is what bounds the batch; here it takes 5 bits per value with its scales
 * instead of 16).  geom->dtype is PKV_Q4 in every call below, head_dim 64 or 128.
 * Layout:
 *   pools  uint8 [num_blocks, num_kv_heads, block_size, R], R = 5 * head_dim / 8
 *          bytes per (token, KV head) row: the row of (block, token t, head h)
 *          is at ((block * Hkv + h) * B + t) * R.  Slots, block tables and
 *          lengths mean what they mean for the other pools (slot = block * B + t).
 *   row    head_dim / 2 bytes of codes, then for each of the NG = head_dim / 32
 *          groups of 32 dims a scale s and an offset z, both bf16 (s first).
 *          The 16-bit unit r * NG + g of the codes (r < 8, little-endian) holds
 *          the 4-bit codes u of dims 32 g + 4 r .. 32 g + 4 r + 3, lowest bits
 *          first.  The value of code u in group g is s_g * (u - 8) + z_g; s_g may have
 *          either sign (paged_kv_write_q4 stores none below 0).
 * A page is copied by paged_copy_blocks with a geom whose pages have the same
 * number of bytes (e.g. one head, block_size 1, head_dim Hkv * B * R / 2, bf16).
 */

/*
 * paged_kv_write_q4 -- paged_kv_write into 4-bit pools: for every token n with
 * slot_mapping[n] >= 0 its rows k[n], v[n] ([num_tokens, Hkv, d] of kv_dtype,
 * PKV_F32 or PKV_BF16) are stored at that slot.  Per group with minimum lo and
 * maximum hi:
 *   s = bf16((hi - lo) / 15)        z = bf16((lo / 2 + hi / 2) + s / 2)
 *   u = min(max(rint((x - z) * (1 / s)) + 8, 0), 15)
 * every operation in fp32 with one rounding, so that the stored bytes are the
 * same on every run.  s below 2^-126 is stored as 0 (every value reads as z).  A
 * value is off by at most s / 2 plus what the bf16 rounding of s and z leaves
 * at the ends of the range (2^-8 of |lo| + |hi|).  A group that holds a NaN or
 * an infinity, or spans more than fp32 holds, reads back as NaN.  Duplicate
 * slots, negative slots and slots past the pool as in paged_kv_write.  k, v and
 * the pools 16-byte aligned; num_kv_heads * head_dim up to 2^30, here and in
 * paged_kv_read_q4 (PKV_ERR_UNSUPPORTED).
 */
int paged_kv_write_q4(const void* k, const void* v, int32_t kv_dtype, const int32_t* slot_mapping,
                      int64_t num_tokens, void* k_cache, void* v_cache, const pkv_geom* geom,
                      cudaStream_t stream);

/*
 * paged_kv_read_q4 -- rows of 4-bit pools as values: row n of k_out and v_out
 * ([num_tokens, Hkv, d] of kv_dtype, rounded once) holds what slot_mapping[n]
 * stores; a negative slot gives a row of zeros, and so does a slot past the pool
 * (PKV_FLAG_BAD_SLOT).  The same slot may appear more than once.  With the slots
 * of all keys of a step's requests (paged_build_slot_mapping) this yields the
 * packed K/V that paged_varlen_prefill takes with block_table == NULL: prompts
 * over a 4-bit cache.  k_out, v_out and the pools 16-byte aligned.
 */
int paged_kv_read_q4(const void* k_cache, const void* v_cache, const int32_t* slot_mapping,
                     int64_t num_tokens, void* k_out, void* v_out, int32_t kv_dtype,
                     const pkv_geom* geom, cudaStream_t stream);

/*
 * paged_decode_q4 -- paged_decode over 4-bit pools: one query per sequence (q,
 * out [batch, Hq, d] of q_dtype, PKV_F32 or PKV_BF16), cache_seqlens[b] keys
 * each, read through block_table row b; 0 when cache_seqlens[b] == 0.  The
 * values are used as stored (4-bit codes, bf16 scales); scores, softmax
 * statistics and sums are fp32.
 * Supported: any Hq / Hkv up to 64; head_dim 128 with any block_size, 64 with an
 * even one; batch <= 4096; max_blocks_per_seq * block_size up to 2^31 - 4097, and
 * below 2^34 for the whole batch.
 * Rounding: bf16 queries enter the scores exactly (products of those below 2^-7 of
 * the largest are cut at 2^-14 of it, per unit of code); each weight is multiplied by its
 * V scale and rounded to fp16 (11 bits; those below 2^-14 of the largest to 2^-25 of
 * it), below the output's own rounding.  With fp32 queries, queries and weights keep
 * 22 bits or more.  Queries and K up to 1e30 in magnitude (a query is scaled to fp16's
 * range, and what that leaves for K and the scale is fp32's).  V may have any finite
 * size; its scales count to 2^-85 absolutely and to 2^-25 of the largest scale that a
 * head's keys hold, so that groups of V that span less lose them.  A NaN or infinite
 * query, or a NaN key, makes its own heads' output NaN; a group of V that holds no
 * numbers, its own 32 dims.
 * workspace: paged_decode_q4_workspace_size(batch, q_dtype, geom) bytes, 256-byte
 * aligned, contents irrelevant on entry, as for paged_decode; it must not be used
 * by another call that runs concurrently.  A length below 0 or past the table
 * counts as the nearest valid one (PKV_FLAG_BAD_LENGTH); keys of a bad page are
 * skipped (PKV_FLAG_BAD_BLOCK).
 */
size_t paged_decode_q4_workspace_size(int32_t batch, int32_t q_dtype, const pkv_geom* geom);
int paged_decode_q4(const void* q, int32_t q_dtype, const void* k_cache, const void* v_cache,
                    const int32_t* block_table, int32_t max_blocks_per_seq,
                    const int32_t* cache_seqlens, int32_t batch, float scale, void* out,
                    void* workspace, size_t workspace_bytes, const pkv_geom* geom,
                    cudaStream_t stream);

/*
 * paged_kv_compact -- keep selected tokens of each sequence, moved together in
 * place (token eviction; the accepted path of a draft tree), after which the
 * pages behind the new length can be released.  Any pool: PKV_F32, PKV_BF16 or
 * PKV_Q4.  Sequence b keeps its positions below start[b] (start == NULL: 0) as
 * they are, and of the others those in keep[cu_keep[b] .. cu_keep[b+1]-1]: the
 * K and V rows of the i-th of them move to position start[b] + i, through
 * block_table row b ([batch, max_blocks_per_seq]).  The i-th entry of a list
 * must be >= start[b] + i, which any ascending list is.  cu_keep [batch + 1]
 * starts at 0 and ends at total_keep, the length of keep.  seqlens_out [batch] (may be
 * NULL) receives start[b] + (number kept), for the next decode; it may be the
 * lengths' own array (no lengths are read), or `start` itself (which then moves
 * on in place: with one call per layer, in the last one only), but may overlap
 * no input otherwise.  The two pools may not overlap.
 * Rows at and behind the new end keep their old contents.  The pages written
 * must belong to one sequence only (copy shared ones first, paged_copy_blocks).
 * An entry below start[b] + i or past the table sets PKV_FLAG_BAD_LENGTH, and a
 * bad table entry PKV_FLAG_BAD_BLOCK; that row is not moved.  A start below 0,
 * bounds outside keep, or a new length past the table set PKV_FLAG_BAD_LENGTH,
 * and nothing of that sequence is moved.
 */
int paged_kv_compact(void* k_cache, void* v_cache, const int32_t* block_table,
                     int32_t max_blocks_per_seq, const int32_t* start, const int32_t* keep,
                     int32_t total_keep, const int32_t* cu_keep, int32_t batch,
                     int32_t* seqlens_out, const pkv_geom* geom, cudaStream_t stream);

/*
 * Position rotation of new tokens -- what the writes below apply to keys on their way
 * into the cache and to the queries of the same tokens.  The dims (i, i + R / 2) of a
 * head (interleaved != 0: (2 i, 2 i + 1)), i < R / 2 with R = rotary_dim, of a token
 * at position p become
 *   x_a c - x_b s,  x_b c + x_a s   with c = cos_sin[p][i], s = cos_sin[p][R / 2 + i];
 * dims from R on stay as they are.  Every product and sum is rounded to fp32, the result
 * once more to the type that it is stored in.
 *   cos_sin    DEVICE fp32 [num_positions, R], 16-byte aligned: R / 2 cosines, then R / 2
 *              sines of each position (of whatever frequencies and scaling the model has)
 *   rotary_dim a multiple of 16, 16 .. head_dim
 *   positions  DEVICE int32 [num_tokens], the position each token is rotated by, or NULL:
 *              token_pos.  They differ where tokens were evicted from the cache
 *              (paged_kv_compact) and the rotation goes on counting them.
 *   q          the tokens' queries [num_tokens, Hq, d] of kv_dtype, or NULL; q_out, which
 *              may be q itself with q's stride, receives them rotated.  The row of a
 *              padding token, or of one whose position is outside the table, is passed on
 *              as it is.
 *   q_stride, q_out_stride   elements from token to token; equal where q_out is q
 */
typedef struct pkv_rope {
    const float* cos_sin;
    int32_t num_positions;
    int32_t rotary_dim;
    int32_t interleaved;
    const int32_t* positions;
    const void* q;
    int64_t q_stride;
    void* q_out;
    int64_t q_out_stride;
} pkv_rope;

/*
 * paged_kv_write_rope -- paged_kv_write_positions with the position rotation on the way
 * ("11. Paged attention 与 online softmax" §11.1; "自己来实现一个"): K rows are rotated
 * and written, V rows written as they are, and the queries rotated, in one launch.
 * Tokens, block_table, slot_mapping_out and flags as in paged_kv_write_positions, but
 * for a table entry outside the pool, which sets PKV_FLAG_BAD_BLOCK; a token whose
 * rotation's position is outside cos_sin is not written (PKV_FLAG_BAD_LENGTH).
 * k, v [num_tokens, Hkv, d] with k_stride and v_stride elements from token to token (the
 * columns of one projection's output, for instance).  The strides in bytes and every
 * address are multiples of 16.  Supported: fp32 and bf16 rows into fp32 and bf16 pools
 * (geom->dtype), head_dim 64 or 128, Hq * d and num_tokens up to 2^30.
 */
int paged_kv_write_rope(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                        int32_t kv_dtype, const pkv_rope* rope, const int32_t* block_table,
                        int32_t max_blocks_per_seq, int32_t num_seqs, const int32_t* token_seq,
                        const int32_t* token_pos, int64_t num_tokens, int32_t* slot_mapping_out,
                        void* k_cache, void* v_cache, const pkv_geom* geom, cudaStream_t stream);

/*
 * 8-bit pools -- K and V as e4m3 codes with a scale for each block and KV head ("Sayfalı
 * dikkat": the cache is what bounds the batch; half of bf16's bytes).  geom->dtype is
 * PKV_Q8 in every call below, head_dim 64 or 128.
 * Layout:
 *   pools  e4m3 [num_blocks, num_kv_heads, block_size, head_dim]
 *   scales fp32 [num_blocks, num_kv_heads], one array for K and one for V; a value is
 *          its code times its block's and head's scale.  The write makes scales powers
 *          of two; the read and the decode take any finite ones.
 * A page is copied by paged_copy_blocks with a geom whose pages have the same number of
 * bytes (e.g. one head, block_size 1, head_dim Hkv * B * d / 2, bf16), its scales by a
 * second call (one head, block_size 1, head_dim Hkv, fp32).  paged_kv_compact does not
 * take these pools: it moves bytes, and a token's codes would have to be shifted to the
 * scale of the page that it comes to.
 */

/*
 * paged_kv_write_q8 -- the tokens' K and V rows into 8-bit pools at their positions, K
 * rotated first where rope is not NULL (then also the queries, as above).  Arguments and
 * flags as in paged_kv_write_rope.
 * The tokens of a call that lie in one page of one sequence follow one another, in
 * ascending positions; rows that are not written (padding, a sequence or position past the
 * table) may stand between them, a token of another sequence or page may not.
 * With a the largest finite magnitude among their values of a head
 * they need the least power of two n >= 2^-100 with a <= 448 n.  If they begin the page
 * (the first of them is at a multiple of block_size) its scale becomes s = n, whatever
 * it was.  Else s = max(n, the least power of two >= the old scale), and where that
 * differs from the old scale the codes of the rows in front of them become
 * e4m3(code * (old / s)).  The new codes are e4m3(x / s), rounded to nearest even.
 * Every value is then within 2^-4 of itself or 2^-10 s of what was written (the larger),
 * and 2^-10 s more for each time that the scale grew afterwards; sizes from 2^128 - 2^123
 * on round to 2^128, which reads as infinite.  Rows behind the tokens
 * keep their codes.  A NaN or an infinity is stored as a NaN of its own.  An old scale
 * below 0, above 2^126 or NaN makes the page's scale NaN.  The pages written must
 * belong to one sequence only (copy shared ones first, paged_copy_blocks).
 */
int paged_kv_write_q8(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                      int32_t kv_dtype, const pkv_rope* rope, const int32_t* block_table,
                      int32_t max_blocks_per_seq, int32_t num_seqs, const int32_t* token_seq,
                      const int32_t* token_pos, int64_t num_tokens, void* k_cache, void* v_cache,
                      float* k_scale, float* v_scale, const pkv_geom* geom, cudaStream_t stream);

/*
 * paged_kv_read_q8 -- rows of 8-bit pools as values: row n of k_out and v_out
 * ([num_tokens, Hkv, d] of kv_dtype) holds what slot_mapping[n] stores, code times scale
 * in fp32 and rounded to kv_dtype (exact in both for scales that are powers of two, but
 * for what lies below the type's range); a negative slot gives a row of zeros, and so does
 * a slot past the pool (PKV_FLAG_BAD_SLOT).  The same slot may appear more than once.
 * With the slots of all keys of a step's requests (paged_build_slot_mapping) this yields
 * the packed K/V that paged_varlen_prefill takes with block_table == NULL: prompts over an
 * 8-bit cache.
 * k_out, v_out and the pools 16-byte aligned; Hkv * d and num_tokens up to 2^30.
 */
int paged_kv_read_q8(const void* k_cache, const void* v_cache, const float* k_scale,
                     const float* v_scale, const int32_t* slot_mapping, int64_t num_tokens,
                     void* k_out, void* v_out, int32_t kv_dtype, const pkv_geom* geom,
                     cudaStream_t stream);

/*
 * paged_decode_q8 -- paged_decode over 8-bit pools: one query per sequence (q, out
 * [batch, Hq, d] of q_dtype, PKV_F32 or PKV_BF16), cache_seqlens[b] keys each, read
 * through block_table row b; 0 when cache_seqlens[b] == 0.  block_table may be NULL where
 * max_blocks_per_seq is 0.  Codes and scales are used
 * as stored; scores, softmax statistics and sums are fp32.
 * Supported: any Hq / Hkv up to 64; head_dim 128 with any block_size (multiples of 8
 * are fastest), 64 with an even one; batch <= 4096; num_blocks * Hkv below 2^31;
 * max_blocks_per_seq * block_size up to 2^31 - 4097, and below 2^34 for the whole batch.
 * Rounding: bf16 queries enter the scores exactly (down to 2^-31 of the largest value of
 * the query); each weight is multiplied by its V scale and rounded to fp16 (11 bits; those
 * below 2^-20 of the largest of a head's to 2^-31 of it), below the output's own
 * rounding.  With fp32 queries, queries and weights keep 22 bits.  Scores and values have
 * fp32's range; V scales may lie as far apart as that allows.  A NaN or infinite
 * query, or a NaN key, makes its own heads' output NaN, and so does a V scale that is no
 * number; a NaN code of V makes its own dim NaN.
 * workspace: paged_decode_q8_workspace_size(batch, q_dtype, geom) bytes, 256-byte
 * aligned, contents irrelevant on entry, as for paged_decode; it must not be used by
 * another call that runs concurrently.  A length below 0 or past the table counts as
 * the nearest valid one (PKV_FLAG_BAD_LENGTH); keys of a bad page are skipped
 * (PKV_FLAG_BAD_BLOCK).
 */
size_t paged_decode_q8_workspace_size(int32_t batch, int32_t q_dtype, const pkv_geom* geom);
int paged_decode_q8(const void* q, int32_t q_dtype, const void* k_cache, const void* v_cache,
                    const float* k_scale, const float* v_scale, const int32_t* block_table,
                    int32_t max_blocks_per_seq, const int32_t* cache_seqlens, int32_t batch,
                    float scale, void* out, void* workspace, size_t workspace_bytes,
                    const pkv_geom* geom, cudaStream_t stream);

/* paged_status_string -- static text for a PKV_* status code. */
const char* paged_status_string(int status);

#ifdef __cplusplus
}
#endif
#endif /* PAGEDKV_H */
