/*
 * pa.h -- C ABI of libpa.so: paged KV-cache decode attention for GB300 (sm_103a).
 *
 * The KV cache of every sequence is stored in fixed-size physical blocks of
 * block_size (B) tokens.  Logical token t of sequence s lives in physical block
 * block_tables[s][t / B], at row t % B of that block (daiw.org "Paged Attention",
 * section 直觉 and 定义; aiqz.cc "vLLM PagedAttention engine", section 分页存储设计,
 * N_i = ceil(S_i / B) and BlockTable_i[j]).  Attention itself is ordinary softmax
 * attention over the logical sequence; only the way K/V addresses are found changes
 * (chenyuan1125 "vllm-pagedattention", section 页表真正解开的，是逻辑连续和物理连续).
 *
 * Layouts (all row-major, all device memory unless stated otherwise):
 *   q             [num_seqs, num_q_heads, head_dim]              fp16 or bf16
 *   out           [num_seqs, num_q_heads, head_dim]              same dtype as q
 *   k_cache       [num_blocks, num_kv_heads, block_size, head_dim] same dtype
 *   v_cache       [num_blocks, num_kv_heads, block_size, head_dim] same dtype
 *   block_tables  [num_seqs, max_blocks_per_seq] int32; entries past ceil(ctx/B) unread
 *   context_lens  [num_seqs] int32, the number of tokens each query attends to
 *   key, value    [num_tokens, num_kv_heads, head_dim]            same dtype
 *   slot_mapping  [num_tokens] int64, slot = block * B + row; negative = skip
 *   block_mapping [num_pairs, 2] int32, (src, dst) block ids
 * Query head h reads kv head h / (num_q_heads / num_kv_heads): contiguous groups (GQA).
 *
 * Supported shapes: head_dim in {64, 128}; block_size in {8, 16, 32};
 * num_q_heads a multiple of num_kv_heads.  Every pointer to q, out, caches, key and
 * value must be 16-byte aligned.
 *
 * Ownership: the caller owns every buffer.  The library allocates no device memory;
 * pa_decode's scratch is the caller's `workspace`.  Device calls are asynchronous on
 * `stream` (NULL = the legacy default stream) and return before the GPU work ends.
 *
 * Status codes: every int-returning call returns PA_OK (0) or a negative PA_ERR_*.
 * Argument errors are found on the host before anything is launched.  Errors that
 * only the device can see (a block id outside the pool, a context length < 1 or
 * > max_blocks_per_seq * B, a slot beyond the pool, a bad copy pair) make the kernel
 * skip that work item -- decode writes zeros for the affected sequence -- and set a
 * bit in a per-device error word that pa_get_device_error reads.  No kernel traps.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* PA_FP8_E4M3 names FP8 K/V blocks; it is accepted only where a call handles caches
 * alone (pa_copy_blocks, pa_swap_blocks).  The FP8 decode and cache write take the
 * 16-bit type of q / out / key / value instead.  PA_FP32 names probabilities
 * (pa_verify_drafts alone). */
typedef enum { PA_FP16 = 0, PA_BF16 = 1, PA_FP8_E4M3 = 2, PA_FP32 = 3 } pa_dtype;

enum {
  PA_OK = 0,
  PA_ERR_ARG = -1,            /* null pointer, unsupported shape or dtype, misalignment */
  PA_ERR_WORKSPACE = -2,      /* workspace missing or smaller than pa_decode_workspace_size */
  PA_ERR_CUDA = -3,           /* a CUDA runtime call failed (launch, attribute, copy) */
  PA_ERR_POOL_EXHAUSTED = -4, /* not enough free blocks; the pool is unchanged */
  PA_ERR_UNKNOWN_SEQ = -5,    /* sequence id not live (or already live, for a new id) */
  PA_ERR_WRONG_TIER = -6      /* sequence swapped out where a resident one is needed, or
                                 resident where a swapped-out one is needed */
};

/* Bits of the per-device error word (pa_get_device_error). */
#define PA_DEVERR_BAD_BLOCK   0x1u  /* decode: a used block-table entry is outside [0, num_blocks) */
#define PA_DEVERR_BAD_CONTEXT 0x2u  /* decode: context length < 1 or > max_blocks_per_seq * B */
#define PA_DEVERR_BAD_SLOT    0x4u  /* reshape_and_cache: slot >= num_blocks * B */
#define PA_DEVERR_BAD_PAIR    0x8u  /* copy_blocks / swap_blocks: a block id outside its pool */
#define PA_DEVERR_TIMEOUT     0x10u /* a bounded wait gave up (about 1 s; prefill pipeline, decode
                                         split-KV merge): output invalid */
#define PA_DEVERR_NO_BLOCKS   0x20u /* build_step: fewer free blocks than the step needs */
#define PA_DEVERR_BAD_PROBS   0x40u /* verify_drafts: a row of probabilities none of which is above 2^-55 */

/*
 * pa_reshape_and_cache -- write each new token's K and V rows into its cache slot.
 *
 * A new token's K/V row goes into the free slot of its sequence's last block; when
 * that block is full a fresh block from the free pool is appended to the table first
 * (chenyuan1125 "vllm-pagedattention", section 页表真正解开的…; horeb.top "vLLM
 * PagedAttention：大模型推理的显存管理革命", section 分配策略).  The host chooses the
 * slots (pa_pool_append_slot); this call only moves the bytes:
 *   k_cache[slot / B, h, slot % B, :] = key[i, h, :]   (and v_cache from value)
 * for every token i whose slot_mapping[i] >= 0.  Two tokens naming the same slot in
 * one call give an undefined winner.  Slots >= num_blocks * B are skipped and flagged
 * (PA_DEVERR_BAD_SLOT).  num_tokens == 0 is a no-op.
 */
int pa_reshape_and_cache(const void* key, const void* value, void* k_cache, void* v_cache,
                         const int64_t* slot_mapping, int num_tokens, int num_blocks,
                         int num_kv_heads, int head_dim, int block_size, pa_dtype dtype,
                         cudaStream_t stream);

/*
 * pa_decode -- single-query (decode) attention over paged K/V.
 *
 * For every sequence s and query head h (kv head g = h / G):
 *   z_t = scale * <q[s,h,:], K_s[t,g,:]>,  t < context_lens[s]
 *   out[s,h,:] = sum_t softmax(z)_t * V_s[t,g,:]
 * where K_s[t] = k_cache[block_tables[s][t / B], :, t % B, :] (same for V).  Scores,
 * the softmax and the weighted sum run block by block through the table
 * (daiw.org "Paged Attention", section 定义, Attention 内核; chenyuan1125, section
 * 页表真正解开的…).  Accumulation is fp32; the output is rounded to nearest-even.
 *
 * Work is split into equal shares of K/V stages (16 tokens; 32 over FP8 / INT4 blocks),
 * one share per SM, so a long sequence may be cut into pieces; the SM that finishes a
 * pair's last outstanding piece merges them with a log-sum-exp reduction (split-KV)
 * inside the same kernel, in a fixed order.  Cut points depend only on logical token
 * positions and the batch's context lengths, never on where blocks sit, so permuting
 * physical blocks (and the table with them) gives bit-identical output.
 *
 * workspace: device scratch of at least pa_decode_workspace_size(...) bytes for the
 * split pieces and their arrival counters, 16-byte aligned, owned by the caller.  Its
 * contents between calls do not matter: a counter left by another call (or never
 * written) is recognised by a tag that differs from call to call, and each merge leaves
 * its counter at zero, so calls replayed from a captured CUDA graph, which repeat their
 * tag, start from zero too.  Concurrent pa_decode calls must not share a workspace.
 * Returns PA_ERR_WORKSPACE if it is NULL or too small.  num_seqs == 0 is a no-op.
 *
 * Ordering: a launch is a programmatic dependent of the kernel before it in the stream.
 * It reads context_lens and block_tables (to plan its work) while that kernel drains,
 * and q, the caches and the workspace only after it has finished.  So block_tables and
 * context_lens must not be written by the kernel immediately before it in the stream
 * when that kernel lets its dependents start early (pa_build_step, the one kernel of this
 * library that writes tables, lets none start early; a plain copy or a kernel without
 * programmatic launch is always safe).  The same
 * holds for every decode entry point below.
 */
int pa_decode(const void* q, const void* k_cache, const void* v_cache,
              const int32_t* block_tables, int max_blocks_per_seq,
              const int32_t* context_lens, int num_seqs, int num_q_heads, int num_kv_heads,
              int head_dim, int block_size, int num_blocks, float scale, void* out,
              void* workspace, size_t workspace_bytes, pa_dtype dtype, cudaStream_t stream);

/*
 * FP8 KV blocks.  Paging does not reduce the bytes the cache needs; quantising the cached
 * K/V does (daiw.org "Paged Attention", section 量化, callout; horeb.top, section 生态现状:
 * serving engines store KV in FP8 or INT4).  Format: each cache element is an E4M3 code
 * (1 sign, 4 exponent bits with bias 7, 3 mantissa bits; exponent field 0 = subnormals
 * m * 2^-9; no infinities; S.1111.111 is NaN; largest finite 448), in the same
 * [num_blocks][Hkv][B][d] layout, one byte per element.  One float32 scale per cache: a
 * code c means decode(c) * k_scale in the K cache and decode(c) * v_scale in the V cache.
 * Scales are the caller's (calibrated or fixed); both must be finite and > 0.
 */
/* Quantising cache write: k_cache[slot / B, h, slot % B, :] = E4M3(key[i, h, :] / k_scale)
 * (V likewise), the division in IEEE float32, rounding to nearest-even, magnitudes above
 * 448 clamped to 448.  key / value are fp16 or bf16 (`dtype`); other rules as
 * pa_reshape_and_cache. */
int pa_reshape_and_cache_fp8(const void* key, const void* value, void* k_cache, void* v_cache,
                             const int64_t* slot_mapping, int num_tokens, int num_blocks,
                             int num_kv_heads, int head_dim, int block_size, float k_scale,
                             float v_scale, pa_dtype dtype, cudaStream_t stream);
/* pa_decode over FP8 blocks: z_t = scale * k_scale * <q, decode(K codes)>, out = v_scale *
 * sum_t softmax(z)_t decode(V codes).  q and out are fp16 or bf16 (`dtype`).  The codes
 * are widened to f16 exactly and multiplied on the tensor cores in f16 (bf16 queries are
 * rounded to f16 for that product); accumulation fp32.  Same workspace, error and
 * determinism rules as pa_decode; there is no fused cache write for FP8 blocks. */
int pa_decode_fp8(const void* q, const void* k_cache, const void* v_cache,
                  const int32_t* block_tables, int max_blocks_per_seq,
                  const int32_t* context_lens, int num_seqs, int num_q_heads, int num_kv_heads,
                  int head_dim, int block_size, int num_blocks, float scale, float k_scale,
                  float v_scale, void* out, void* workspace, size_t workspace_bytes,
                  pa_dtype dtype, cudaStream_t stream);

/* One FP8 decode step in one call and one launch: each sequence's newest token (key_new /
 * value_new [num_seqs][Hkv][d], fp16 or bf16) is quantised with the arithmetic of
 * pa_reshape_and_cache_fp8 by the warp that computes the sequence's last stage, attended
 * from there and stored at position context_lens[s] - 1 through the table; caches and
 * output equal pa_reshape_and_cache_fp8 + pa_decode_fp8 bit for bit.  (A sequence whose
 * newest slot is invalid writes nothing; the decode flags it.) */
int pa_decode_append_fp8(const void* q, const void* key_new, const void* value_new,
                         void* k_cache, void* v_cache, const int32_t* block_tables,
                         int max_blocks_per_seq, const int32_t* context_lens, int num_seqs,
                         int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                         int num_blocks, float scale, float k_scale, float v_scale, void* out,
                         void* workspace, size_t workspace_bytes, pa_dtype dtype,
                         cudaStream_t stream);

/*
 * INT4 KV blocks (the other quantised format horeb.top, section 生态现状, names).  The
 * pages give no INT4 format; this one is symmetric integer quantisation with one scale
 * per cached row:
 *   codes   [num_blocks][Hkv][B][d/2] uint8: two 4-bit codes per byte, element 2i in the
 *           low nibble of byte i, each stored as u = c + 8 for a code c in [-7, 7];
 *   scales  [num_blocks][Hkv][B] float32, one per (block, kv head, row), K and V apart.
 * A row (one token of one kv head) means the values c_i * s.  All arrays 16-byte aligned,
 * owned by the caller.
 */
/* Quantising cache write: for each token i with slot = slot_mapping[i] >= 0 and each kv
 * head h, the row x = key[i, h, :] gets s = max_j |x_j| / 7 and c_j = x_j / s (both IEEE
 * float32 divisions) rounded to nearest-even and clamped to [-7, 7] (s = 0 and c = 0 for
 * an all-zero row); likewise value.  Inputs are finite fp16 or bf16 (`dtype`); other
 * rules as pa_reshape_and_cache. */
int pa_reshape_and_cache_int4(const void* key, const void* value, void* k_codes, void* v_codes,
                              float* k_scales, float* v_scales, const int64_t* slot_mapping,
                              int num_tokens, int num_blocks, int num_kv_heads, int head_dim,
                              int block_size, pa_dtype dtype, cudaStream_t stream);
/* pa_decode over INT4 blocks: z_t = scale * sK_t * <q, cK_t>, out = sum_t softmax(z)_t *
 * sV_t * cV_t.  q and out are fp16 or bf16 (`dtype`).  The codes are widened to f16
 * exactly and multiplied on the tensor cores in f16 (bf16 queries rounded to f16); each
 * token's K scale multiplies its fp32 scores, and each token's V scale multiplies its
 * softmax weight before that weight is rounded to f16 for P V (so V rows need
 * max|v| < 7 * 65504, and rows with max|v| below about 4e-4 lose precision to f16
 * subnormals).  Same workspace, error and determinism rules as pa_decode. */
int pa_decode_int4(const void* q, const void* k_codes, const void* v_codes, const float* k_scales,
                   const float* v_scales, const int32_t* block_tables, int max_blocks_per_seq,
                   const int32_t* context_lens, int num_seqs, int num_q_heads, int num_kv_heads,
                   int head_dim, int block_size, int num_blocks, float scale, void* out,
                   void* workspace, size_t workspace_bytes, pa_dtype dtype, cudaStream_t stream);
/* One INT4 decode step in one call and one launch: each sequence's newest token (key_new /
 * value_new [num_seqs][Hkv][d]) is quantised with the arithmetic of
 * pa_reshape_and_cache_int4 by the warp that computes its last stage, attended from there
 * and stored (codes and scales) at position context_lens[s] - 1 through the table; equal to
 * pa_reshape_and_cache_int4 + pa_decode_int4 bit for bit (a sequence whose newest slot is
 * invalid writes nothing and the decode flags it). */
int pa_decode_append_int4(const void* q, const void* key_new, const void* value_new,
                          void* k_codes, void* v_codes, float* k_scales, float* v_scales,
                          const int32_t* block_tables, int max_blocks_per_seq,
                          const int32_t* context_lens, int num_seqs, int num_q_heads,
                          int num_kv_heads, int head_dim, int block_size, int num_blocks,
                          float scale, void* out, void* workspace, size_t workspace_bytes,
                          pa_dtype dtype, cudaStream_t stream);
/* pa_copy_blocks for INT4 blocks: the codes and the scales of each pair (two launches). */
int pa_copy_blocks_int4(void* k_codes, void* v_codes, float* k_scales, float* v_scales,
                        const int32_t* block_mapping, int num_pairs, int num_blocks,
                        int num_kv_heads, int head_dim, int block_size, cudaStream_t stream);
/* pa_swap_blocks for INT4 blocks: codes and scales move together between two pools (one
 * of them may be pinned host memory); the same pair rules. */
int pa_swap_blocks_int4(const void* src_k, const void* src_v, const float* src_ks,
                        const float* src_vs, void* dst_k, void* dst_v, float* dst_ks,
                        float* dst_vs, const int32_t* block_mapping, int num_pairs,
                        int src_num_blocks, int dst_num_blocks, int num_kv_heads, int head_dim,
                        int block_size, cudaStream_t stream);

/*
 * pa_build_step -- block tables and slots of one step from request lengths, on the GPU.
 *
 * The host pool (pa_pool_*) plans blocks one request at a time.  This call plans a whole step
 * where the lengths already are, so that decode steps can follow one another, or a captured
 * graph replay, with no round trip to the host.  Request s has context_lens[s] tokens in this
 * step, query_lens[s] of them new.  With old_s = ceil((c_s - q_s) / B) and need_s =
 * ceil(c_s / B) - old_s (aiqz.cc, section 分页存储设计, N_i = ceil(S_i / B)), o_s the sum of
 * need over the requests before s, and N_s the sum of their new tokens:
 *   block_tables[s][old_s + k] = free_blocks[free_start[0] + o_s + k],   k < need_s
 *   slot_mapping[N_s + i] = block_tables[s][p / B] * B + p % B,          p = c_s - q_s + i
 *   query_start[s] = N_s,   query_start[num_seqs] = N,   free_next[0] = free_start[0] + sum need
 * Blocks leave the head of the list in request order, as from the host pool's free list.
 * On top of the host pool the list is a reserve: the table of blocks that pa_pool_allocate gives an
 * id of its own.  The pool counts them as that id's until pa_pool_free takes them all back, whichever
 * requests hold them by then; fork, prefix caching and swap planning know the pool's ids alone.
 * slot_mapping entries N .. num_slots - 1 are -1 (a padded batch: the cache writes skip
 * them).  Other table entries are left as they were; the old_s entries of a request are read.
 * A request may have no new tokens (q_s = 0) and no context.  A tail block shared with
 * another sequence must have been copied first (pa_copy_blocks*).
 *
 * Device: query_lens, context_lens [num_seqs], free_blocks [num_free], free_start [1],
 * block_tables [num_seqs][max_blocks_per_seq], query_start [num_seqs + 1], free_next [1],
 * all int32; slot_mapping [num_slots] int64.  free_next must not be free_start (a loop
 * alternates two cells) and no output may overlap an input.
 *
 * A step that needs more blocks than free_blocks holds behind free_start[0]
 * (PA_DEVERR_NO_BLOCKS; also a free_start[0] outside [0, num_free]), or more slots than
 * num_slots (PA_DEVERR_BAD_SLOT), changes no table, sets every slot to -1 and free_next to
 * free_start; query_start is written all the same (clipped to 2^31 - 1).  An impossible
 * request (negative length, q_s > c_s, c_s > max_blocks_per_seq * B) gets no blocks, slots
 * -1 for its max(q_s, 0) tokens, and PA_DEVERR_BAD_CONTEXT; a block id outside [0,
 * num_blocks) gives slots -1 and PA_DEVERR_BAD_BLOCK, and is not written into a table.
 * num_seqs == 0 writes query_start[0] = 0, free_next and the slots.
 * The launch waits for the kernel before it and lets none after it start early, so the
 * tables it writes may be read by any call that follows it in the stream.
 */
int pa_build_step(const int32_t* query_lens, const int32_t* context_lens, int num_seqs,
                  const int32_t* free_blocks, int num_free, const int32_t* free_start,
                  int32_t* block_tables, int max_blocks_per_seq, int block_size, int num_blocks,
                  int64_t* slot_mapping, int num_slots, int32_t* query_start, int32_t* free_next,
                  cudaStream_t stream);

/*
 * FP8 KV blocks with a scale for each (block, kv head).  The caches hold E4M3 codes as above,
 *   k_cache, v_cache    [num_blocks][Hkv][B][d]
 *   k_scales, v_scales  [num_blocks][Hkv] float32
 * and a code c of kv head h in block b means decode(c) * scales[b][h].  Nothing has to be
 * calibrated: the cache write chooses each scale from the data.  The scales it stores are
 * powers of two 2^e, -100 <= e <= 120; a floating-point code loses nothing by that.  Other
 * finite positive scales (a cache made elsewhere) are read as they are.  Codes 16-byte,
 * scales 4-byte aligned, all owned by the caller.
 */
/* Cache write of each sequence's newest tokens.  Sequence s owns rows query_start[s] ..
 * query_start[s+1]-1 of key / value [num_tokens][Hkv][d] (fp16 or bf16, `dtype`), its positions
 * c - q .. c - 1 (c = context_lens[s], q = their number): one row for a decode step, a prompt
 * or a chunk of one otherwise, mixed freely.  Rows from query_start[num_seqs] on (a padded
 * batch) are not read.  For each block that these positions touch, kv head h, and K and V
 * apart:
 *   amax = the largest finite |x| of the new rows, e = the smallest integer with
 *   amax <= 448 * 2^e, held in [-100, 120];  S = 2^e if the call writes the block's row 0,
 *   else max(2^e, scales[b][h]);
 *   earlier rows of the block, where S > scales[b][h]: code := E4M3(decode(code) *
 *   scales[b][h] / S) (for powers of two exact, but where the result is subnormal);
 *   new rows: code = E4M3(x / S), rounding to nearest-even, magnitudes above 448 S (only
 *   infinities) clamped, NaN kept.  scales[b][h] = S.  (Where an earlier scale that is no
 *   power of two stays, x is multiplied by its rounded reciprocal.)
 * Rows of a touched block behind the last new one are left as they were.  A touched block
 * must belong to one sequence of the call (copy-on-write first), and its rows before c - q
 * must have been written by this call's kind.  A sequence with an impossible span
 * (query_start decreasing or beyond num_tokens, q > c, c > max_blocks_per_seq * B) writes
 * nothing: PA_DEVERR_BAD_CONTEXT; a block id out of range is skipped: PA_DEVERR_BAD_BLOCK.
 * A launch is a programmatic dependent of the kernel before it; it reads everything only
 * after that kernel has finished. */
int pa_append_fp8_block(const void* key, const void* value, void* k_cache, void* v_cache,
                        float* k_scales, float* v_scales, const int32_t* block_tables,
                        int max_blocks_per_seq, const int32_t* context_lens,
                        const int32_t* query_start, int num_seqs, int num_tokens, int num_blocks,
                        int num_kv_heads, int head_dim, int block_size, pa_dtype dtype,
                        cudaStream_t stream);
/* pa_decode over those blocks: z_t = scale * sK_t * <q, decode(K codes_t)>, out = sum_t
 * softmax(z)_t * sV_t * decode(V codes_t), sK_t and sV_t the scales of token t's block.  q and
 * out are fp16 or bf16 (`dtype`).  The codes are widened to f16 exactly and multiplied on the
 * tensor cores in f16; bf16 queries, those of a kv head together, are brought to the type's upper
 * range by a power of two, so that queries of any size can be used: f16 loses 2^-39 of the
 * largest of them at most.  The K scale multiplies the fp32 scores, the V scale the softmax
 * weights before they are rounded to f16, relative to the largest product of a weight and its V
 * scale: f16 loses 2^-25 of that at most, so a block of large values with next to no weight
 * costs the others no precision.  Accumulation fp32;
 * outputs past the type's largest value are clamped to it (a cached 65504 is held as 65536).
 * Same workspace, ordering, error and determinism rules as pa_decode. */
int pa_decode_fp8_block(const void* q, const void* k_cache, const void* v_cache,
                        const float* k_scales, const float* v_scales, const int32_t* block_tables,
                        int max_blocks_per_seq, const int32_t* context_lens, int num_seqs,
                        int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                        int num_blocks, float scale, void* out, void* workspace,
                        size_t workspace_bytes, pa_dtype dtype, cudaStream_t stream);
/* pa_prefill over those blocks: the arguments and rules of pa_prefill with K and V the values
 * decode(code) * scale of each token's block, and two more: num_tokens, the rows of q and out
 * (a sequence whose span lies outside them gets PA_DEVERR_BAD_CONTEXT and nothing is read
 * or written for it; rows behind the last sequence are not touched), and scale > 0;
 * num_q_heads <= 65536.
 * Products run in f16 over the codes, widened exactly, and bf16 rows of q brought to the type's
 * upper range by a power of two; K's scales multiply the fp32 scores, V's the softmax weights before
 * they are rounded to f16, relative to the largest such product of the keys that the token attends
 * to; accumulation fp32; outputs clamped as by pa_decode_fp8_block.  So a key that a token does
 * not attend to changes none of its output's bits, whatever its codes and scales, and one that it
 * attends to with next to no weight costs the others no precision.  Write the sequences' new tokens first
 * (pa_append_fp8_block). */
int pa_prefill_fp8_block(const void* q, const void* k_cache, const void* v_cache,
                         const float* k_scales, const float* v_scales,
                         const int32_t* block_tables, int max_blocks_per_seq,
                         const int32_t* context_lens, const int32_t* query_start, int num_seqs,
                         int num_tokens, int max_query_len, int num_q_heads, int num_kv_heads,
                         int head_dim, int block_size, int num_blocks, float scale, void* out,
                         pa_dtype dtype, cudaStream_t stream);
/* pa_copy_blocks for those blocks: codes and scales of each pair, in one launch. */
int pa_copy_blocks_fp8_block(void* k_cache, void* v_cache, float* k_scales, float* v_scales,
                             const int32_t* block_mapping, int num_pairs, int num_blocks,
                             int num_kv_heads, int head_dim, int block_size,
                             cudaStream_t stream);
/* pa_swap_blocks for those blocks: codes and scales move together between two pools (one of
 * them may be pinned host memory), in one launch; the same pair rules. */
int pa_swap_blocks_fp8_block(const void* src_k, const void* src_v, const float* src_ks,
                             const float* src_vs, void* dst_k, void* dst_v, float* dst_ks,
                             float* dst_vs, const int32_t* block_mapping, int num_pairs,
                             int src_num_blocks, int dst_num_blocks, int num_kv_heads,
                             int head_dim, int block_size, cudaStream_t stream);

/*
 * pa_prefill -- causal multi-query attention of each sequence's newest tokens over its
 * paged context (a prompt from scratch, or a chunk of one).
 *
 * Sequence s owns query rows query_start[s] .. query_start[s+1]-1 of q: its newest
 * q_len_s = query_start[s+1] - query_start[s] tokens, at positions ctx_s - q_len_s ..
 * ctx_s - 1, whose K/V rows are already in the cache (write them first with
 * pa_reshape_and_cache).  The token at position p attends to positions 0 .. p:
 *   out[row, h, :] = sum_{t <= p} softmax(scale * <q[row, h, :], K_s[t, h / G, :]>) V_s[t, h / G, :]
 * with K_s[t] = k_cache[block_tables[s][t / B], :, t % B, :] (horeb.top "vLLM
 * PagedAttention：大模型推理的显存管理革命", section 分配策略: a prompt is allotted its
 * blocks at prefill; daiw.org "Paged Attention", section 回顾与衔接: the attention kernel
 * reads the block table).  Accumulation is fp32, the output rounded to nearest-even.
 *
 * q, out: [query_start[num_seqs], Hq, d] device, 16-byte aligned; query_start: int32
 * [num_seqs + 1] device, non-decreasing from 0; max_query_len: host bound on q_len_s
 * (the launch covers it; larger q_len_s are not computed).  Requires Hq / Hkv <= 64.
 * A sequence whose context is invalid (ctx < 1, ctx > T * B, or q_len_s > ctx_s) gets
 * zeros and PA_DEVERR_BAD_CONTEXT; a block id out of range gives zeros for the query
 * block that reads it and PA_DEVERR_BAD_BLOCK.  Uses no workspace.  A launch is a
 * programmatic dependent of the kernel before it in the stream.
 */
int pa_prefill(const void* q, const void* k_cache, const void* v_cache,
               const int32_t* block_tables, int max_blocks_per_seq,
               const int32_t* context_lens, const int32_t* query_start, int num_seqs,
               int max_query_len, int num_q_heads, int num_kv_heads, int head_dim,
               int block_size, int num_blocks, float scale, void* out, pa_dtype dtype,
               cudaStream_t stream);

/*
 * A decoding step that checks drafted tokens.  Each sequence feeds its last token and some
 * drafted ones through the model at once; the calls below are the step's own work on paged
 * caches: positions and the cache write (pa_rotary_append), attention of those few tokens over the
 * long context (pa_decode_drafts), and the verdict on the drafts (pa_verify_drafts), whose
 * context_next are the next step's lengths on the GPU.  pa_cross is the same attention without a
 * mask, over an encoder's states.
 *
 * Common to them: sequence s owns rows query_start[s] .. query_start[s+1]-1 of the step's
 * tensors (num_tokens rows in all), q_s of them.  query_start [num_seqs + 1] and context_lens
 * [num_seqs] are int32 device arrays.  A sequence with an impossible span (query_start negative,
 * decreasing or beyond num_tokens) is not read or written, and gets PA_DEVERR_BAD_CONTEXT.  Rows
 * behind the last sequence (a padded batch) are left as they were.  A launch is a programmatic
 * dependent of the kernel before it and reads everything only after that kernel has finished.
 */
/* Turns per token of `n` angles (radians per token, host), as pa_rotary and pa_rotary_append take
 * them: freqs_out[i] = radians[i] / 2 pi in units of 2^-64, rounded, whole turns dropped (host;
 * the caller copies them to the device).  |radians[i]| <= 10^6, else PA_ERR_ARG. */
int pa_rotary_frequencies(const double* radians, int n, uint64_t* freqs_out);
/*
 * pa_rotary_append -- rotary positions of a step's new tokens, and their cache write.
 *
 * Row i of sequence s is at position p = context_lens[s] - q_s + i (context_lens count the
 * step's tokens).  Pair j < rotary_dim / 2 of a head's first rotary_dim values is
 * (x_j, x_{j + rotary_dim / 2}), or (x_2j, x_{2j+1}) if interleaved, and becomes
 *   (a cos t - b sin t, b cos t + a sin t) * amplitude,   t = p * freqs[j] turns,
 * in fp32, rounded to nearest-even; a head's other values are copied.  q's rows go to q_out; key's
 * turned rows and value's rows go through the block table into the caches, at row p % B of block
 * block_tables[s][p / B].  Positions are exact at any distance.
 *
 * q [num_tokens][Hq][d], key, value [num_tokens][Hkv][d], q_out as q: fp16 or bf16, heads
 * contiguous, rows *_stride values apart (a multiple of 8, at least the row), so that they may be
 * slices of one projection; bases 16-byte aligned.  q_out may be q itself, with q's stride.  rotary_dim: a
 * multiple of 16 up to d.  freqs [rotary_dim / 2] device, 8-byte aligned.
 * A sequence with q_s > context_lens[s] or a context beyond its table is skipped
 * (PA_DEVERR_BAD_CONTEXT); where the block id is out of range K and V are skipped
 * (PA_DEVERR_BAD_BLOCK), q is turned all the same.  No two rows may share a slot
 * (copy-on-write first).
 */
int pa_rotary_append(const void* q, int64_t q_stride, const void* key, int64_t key_stride,
                     const void* value, int64_t value_stride, void* q_out, int64_t q_out_stride,
                     void* k_cache, void* v_cache, const int32_t* block_tables,
                     int max_blocks_per_seq, const int32_t* context_lens,
                     const int32_t* query_start, const uint64_t* freqs, int rotary_dim,
                     int interleaved, float amplitude, int num_seqs, int num_tokens,
                     int num_blocks, int num_q_heads, int num_kv_heads, int head_dim,
                     int block_size, pa_dtype dtype, cudaStream_t stream);
/* The same without the cache write, for caches of other formats: turned keys go to key_out, rows
 * key_out_stride apart (which may be key itself, with its stride). */
int pa_rotary(const void* q, int64_t q_stride, const void* key, int64_t key_stride, void* q_out,
              int64_t q_out_stride, void* key_out, int64_t key_out_stride,
              const int32_t* context_lens, const int32_t* query_start, const uint64_t* freqs,
              int rotary_dim, int interleaved, float amplitude, int num_seqs, int num_tokens,
              int num_q_heads, int num_kv_heads, int head_dim, pa_dtype dtype,
              cudaStream_t stream);
/*
 * pa_decode_drafts -- causal attention of each sequence's newest tokens over its paged context,
 * as pa_prefill, with the keys of a sequence split over the SMs: for a few tokens per sequence
 * (drafts to be checked, the end of a prompt) over contexts of any length.  64 contexts of 2048, 32 / 8
 * heads of 128: 1 row each 91 us (pa_prefill 135), 16 rows 97 (139), 64 rows 126 (142), 256 rows 411 (446); whole
 * prompts are pa_prefill's (8 of 2048: 274 us, here 313).
 *
 * q, out [num_tokens][Hq][d]; row i of sequence s is at position context_lens[s] - q_s + i, attends
 * to positions up to its own, and its K/V rows are already in the cache (pa_rotary_append).
 * scale > 0; Hq / Hkv <= 128; Hq <= 65536.  Accumulation fp32; weights are rounded to the type of q for the
 * product with V, as in pa_prefill; fp16 ones keep what is above 2^-31 of a row's largest.  Scores, scaled or not, may be of any size that fp32 holds (a row's largest has the
 * weight 1).  V may hold magnitudes up to 2^100.  A key that a row does not attend to changes none
 * of its bits, whatever it holds, NaN and infinities among it.
 * The cuts depend on query_start, context_lens, max_blocks_per_seq, num_tokens and the head shape
 * alone, never on where blocks sit.
 * A sequence with rows and an invalid context (ctx < 1, ctx > T * B, q_s > ctx) gets zeros and
 * PA_DEVERR_BAD_CONTEXT; a block id out of range gives zeros for the query tile that reads it
 * and PA_DEVERR_BAD_BLOCK.
 * workspace: device scratch of at least pa_split_workspace_size(...) bytes, 16-byte aligned, owned
 * by the caller; its contents between calls do not matter.  Calls that may overlap must not share
 * one.  PA_ERR_WORKSPACE if it is missing or too small.  num_seqs or num_tokens of 0: a no-op.
 */
int pa_decode_drafts(const void* q, const void* k_cache, const void* v_cache,
                     const int32_t* block_tables, int max_blocks_per_seq,
                     const int32_t* context_lens, const int32_t* query_start, int num_seqs,
                     int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                     int block_size, int num_blocks, float scale, void* out, void* workspace,
                     size_t workspace_bytes, pa_dtype dtype, cudaStream_t stream);
/*
 * pa_cross -- attention of each sequence's rows to all context_lens[s] cached tokens: a decoder's
 * tokens (one, or a whole prompt) over an encoder's states of another length, whose K/V rows lie
 * in paged blocks (written once with pa_reshape_and_cache; shared by forks like any blocks).
 * Where every sequence has one row and a state at least, pa_decode computes the same and is faster (64
 * rows over 100..1500 states, 16 heads of 64: 42 us, here 49).
 * Arguments and rules of pa_decode_drafts, but: no mask; q_s and context_lens[s] are independent;
 * a context of 0 gives zeros and no error (ctx < 0 or > T * B: zeros and PA_DEVERR_BAD_CONTEXT).
 */
int pa_cross(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
             int max_blocks_per_seq, const int32_t* context_lens, const int32_t* query_start,
             int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
             int block_size, int num_blocks, float scale, void* out, void* workspace,
             size_t workspace_bytes, pa_dtype dtype, cudaStream_t stream);
/* Bytes of workspace pa_decode_drafts and pa_cross need on the current device: it depends on
 * its SM count and head_dim alone (152 SMs, head_dim 128: 41 MB). */
size_t pa_split_workspace_size(int num_q_heads, int num_kv_heads, int head_dim);
/*
 * pa_verify_drafts -- which drafted tokens stay, and the token after them.
 *
 * tokens [num_tokens] int32 are the step's inputs: a sequence's row 0 is its last token, rows 1 ..
 * q_s - 1 its drafts.  target_probs [num_tokens][V] is the model's distribution after each row,
 * draft_probs the same of the model that drafted: row i is what the draft in row i + 1 was drawn
 * from (a sequence's last row is not read); NULL where each draft was certain (looked up, or the
 * draft model's first choice).  Rows are *_stride values apart; fp32, fp16 or bf16 (`dtype`, both
 * alike), in [0, 1] (what is negative or no number counts as 0, above 1 as 1); a row need not sum
 * to 1.  uniforms [num_tokens] float32 in [0, 1).
 *   Draft i + 1 is accepted while uniforms[i] * draft[i][x] < target[i][x], x = tokens[i + 1] (rows of
 *   the sequence; draft 1 where NULL; probabilities as they count, and uniforms[i] alike: below 0 and
 *   NaN as 0, above 1 as 1).  A token outside [0, V) is refused.
 *   At the first refusal, row a: weights max(target[a] - draft[a], 0) (NULL: target[a] without x);
 *   where all of them are zero, target[a].  With every draft accepted, a = q_s - 1: target[a].
 *   The sampled token is the smallest t whose running sum of weights exceeds
 *   uniforms[q_s - 1] times their sum.  For weights and sums, target and draft values are whole
 *   units of 2^-54, each rounded to nearest (from 2^-31 on fp32 loses nothing; 2^-55 and less is 0, so a row
 *   or a rest of nothing but such values counts as all zero), and sums are exact: the token depends on no
 *   order of addition.  (A number outside [0, 1): below 0 and NaN sample as 0, 1 and more the last
 *   token that has a weight.)
 * out_tokens [num_tokens]: rows 0 .. a - 1 the accepted drafts, row a the sampled token, -1 behind
 * it.  emitted[s] = a + 1.  context_next[s] = context_lens[s] - q_s + emitted[s]: the tokens whose
 * K/V rows stay (context_lens count the step's tokens; the next step adds its own); it may be
 * context_lens itself, but not overlap it otherwise.  A sequence without rows: 0 and context_lens[s].
 * A row a without a probability above 2^-55: -1 there, emitted[s] = a, PA_DEVERR_BAD_PROBS.  An impossible
 * span or context_lens[s] < q_s: 0, context_lens[s], PA_DEVERR_BAD_CONTEXT.  V <= 2^20; out_tokens
 * must not overlap tokens.  The launch lets none after it
 * start early, so the lengths it writes may be read by any call that follows it in the stream.
 * Blocks that a rejected draft had opened stay in the request's table (every call reads
 * ceil(ctx / B) entries); pa_pool_truncate gives them back to the host pool.
 */
int pa_verify_drafts(const int32_t* tokens, const void* target_probs, int64_t target_stride,
                     const void* draft_probs, int64_t draft_stride, const float* uniforms,
                     const int32_t* query_start, const int32_t* context_lens, int num_seqs,
                     int num_tokens, int vocab_size, int32_t* out_tokens, int32_t* emitted,
                     int32_t* context_next, pa_dtype dtype, cudaStream_t stream);

/*
 * pa_decode_append -- one whole decode step in one kernel: the cache write of every
 * sequence's newest token followed by pa_decode over contexts that include it.
 *
 * key_new, value_new: [num_seqs, Hkv, d] device, row s = the token just produced by
 * sequence s, at its position ctx_s - 1, so its slot is
 * block_tables[s][(ctx_s - 1) / B] * B + (ctx_s - 1) % B (the slot formula of
 * pa_reshape_and_cache; chenyuan1125, section 页表真正解开的…: the new token goes into the
 * last block's free slot, then attention reads the context through the table).
 * Results -- out and both caches -- are bit-identical to pa_reshape_and_cache of those rows
 * into those slots followed by pa_decode with the same arguments.  The attention takes the
 * newest row from key_new/value_new, and the cache row is stored during the same kernel,
 * so that slot must not lie inside another sequence's context in the same call (true once
 * copy-on-write has given every written last block a single owner).  A sequence whose
 * context length or newest block id is invalid writes nothing and is flagged as in
 * pa_decode.  Other arguments, errors and the workspace are pa_decode's.
 */
int pa_decode_append(const void* q, const void* key_new, const void* value_new, void* k_cache,
                     void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
                     const int32_t* context_lens, int num_seqs, int num_q_heads,
                     int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
                     void* out, void* workspace, size_t workspace_bytes, pa_dtype dtype,
                     cudaStream_t stream);

/*
 * pa_decode_fixed_scratch -- pa_decode for callers that cannot allocate device memory.
 *
 * The pages have no counterpart to this call; it exists for library users.  Some callers
 * may not call cudaMalloc at all -- a server that gave nearly all HBM to the KV block pool
 * up front, or a host framework that owns every device buffer -- and so cannot supply
 * pa_decode's workspace.  This call takes the same arguments minus the workspace and uses
 * a fixed 32 MiB scratch array built into the library instead (held on every GPU that
 * loads the library until the process exits).  It allocates nothing.
 *   - Every call on a device shares that scratch and leaves its contents behind; nothing in
 *     it needs to start at zero.  Calls whose GPU work overlaps (unordered streams) race on
 *     it and give undefined output.
 *   - The first call on a device looks up the scratch's device address there; make that
 *     first call before any stream capture begins.
 *   - A device and head shape needing more than 32 MiB of decode scratch (more than about
 *     250 SMs at 16 query heads per kv head and head_dim 128) gets PA_ERR_WORKSPACE and
 *     nothing is launched.
 *   - q must be device memory of the current device (the scratch is per device); a q
 *     elsewhere gets PA_ERR_ARG.  Other errors are pa_decode's.
 */
int pa_decode_fixed_scratch(const void* q, const void* k_cache, const void* v_cache,
                            const int32_t* block_tables, int max_blocks_per_seq,
                            const int32_t* context_lens, int num_seqs, int num_q_heads,
                            int num_kv_heads, int head_dim, int block_size, int num_blocks,
                            float scale, void* out, pa_dtype dtype, cudaStream_t stream);

/*
 * pa_decode_timeline -- diagnostics: time the phases of 16-bit decode launches.
 *
 * The pages have no counterpart; it exists to measure where a launch's time goes.  While
 * a buffer is set, every decode launch made by this host thread (pa_decode,
 * pa_decode_append, pa_decode_fixed_scratch) runs a copy of the kernel in which lane 0 of
 * each warp writes three %globaltimer readings (ns) into the buffer.  That works for
 * 16-bit blocks at head_dim 128 with at most 8 query heads per kv head.  Launches made
 * without a buffer run the kernel without that code.  The layout is [cta][warp][k]
 * unsigned long long with 8 warps a CTA, and k is:
 *   0  the programmatic wait on the previous kernel released,
 *   1  the warp's streaming done (before the cut pieces are counted in),
 *   2  its end (after any merge).
 * A CTA with no work writes nothing, so zero the buffer first.  buffer is device memory of
 * at least SM count x 8 x 3 x 8 bytes (29 184 bytes on 152 SMs).  While a buffer is set,
 * a decode launch returns PA_ERR_ARG and launches nothing if the buffer is smaller than
 * that, if the blocks are FP8 or INT4, or if the shape is another one.  NULL clears the
 * setting.  The caller owns the buffer, and outputs are unaffected.  Returns PA_ERR_ARG
 * for a non-null buffer that is not 8-byte aligned.
 */
int pa_decode_timeline(void* buffer, size_t bytes);

/* Bytes of workspace pa_decode needs on the current device for these head counts.
 * It depends on the device's SM count and the head shape only, not on the batch
 * (152 SMs: 5.1 MB for 32 query / 8 kv heads at head_dim 128, at most about 20 MB). */
size_t pa_decode_workspace_size(int num_q_heads, int num_kv_heads, int head_dim);

/*
 * pa_copy_blocks -- copy whole physical blocks (every kv head, every row) of both
 * caches: k_cache[dst] = k_cache[src], v_cache[dst] = v_cache[src] for each pair.
 *
 * This is the copy behind copy-on-write: a branch that must write into a last block
 * still shared with other sequences first copies it, then remaps and writes; full old
 * blocks stay shared (chenyuan1125, section 一块内存，如何安全地属于多条序列; horeb.top,
 * section 内存共享：写时复制).  block_mapping is device memory.  Pairs must not alias
 * (distinct dst, no dst also a src); pa_check_block_mapping checks a host copy.  A pair
 * with an id outside [0, num_blocks) is skipped and flagged (PA_DEVERR_BAD_PAIR).
 */
int pa_copy_blocks(void* k_cache, void* v_cache, const int32_t* block_mapping, int num_pairs,
                   int num_blocks, int num_kv_heads, int head_dim, int block_size,
                   pa_dtype dtype, cudaStream_t stream);

/*
 * pa_swap_blocks -- copy whole blocks from one pool to another:
 *   dst_k[d] = src_k[s], dst_v[d] = src_v[s]  for each pair (s, d) of block_mapping.
 *
 * This moves a preempted request's blocks to CPU memory (swap-out) and back (swap-in);
 * the block table is what makes the move a plain block copy (aiqz.cc "vLLM
 * PagedAttention engine", section 连续批处理：随到随走的新秩序).  pa_pool_swap_out /
 * pa_pool_swap_in plan the pairs.
 *
 * Pools: src [src_num_blocks, Hkv, B, d], dst [dst_num_blocks, Hkv, B, d], same dtype.
 * Each of the five pointers may be device memory or page-locked host memory registered
 * with CUDA (cudaHostAlloc, cudaMallocHost, cudaHostRegister; a pinned torch tensor):
 * the GPU reads and writes host memory directly (over NVLink-C2C on GB300), so one
 * kernel launch moves every pair.  Anything else (pageable host memory) is PA_ERR_ARG.
 * block_mapping is int32 [num_pairs, 2].  Destination ids must be distinct and the two
 * pools must not overlap.  A pair with an id outside its pool is skipped and flagged
 * (PA_DEVERR_BAD_PAIR).  num_pairs == 0 is a no-op.
 */
int pa_swap_blocks(const void* src_k, const void* src_v, void* dst_k, void* dst_v,
                   const int32_t* block_mapping, int num_pairs, int src_num_blocks,
                   int dst_num_blocks, int num_kv_heads, int head_dim, int block_size,
                   pa_dtype dtype, cudaStream_t stream);

/* Host-side check of a copy_blocks pair list (host memory): PA_OK, or PA_ERR_ARG when an
 * id is outside [0, num_blocks), a dst repeats, or a dst is also a src. */
int pa_check_block_mapping(const int32_t* host_block_mapping, int num_pairs, int num_blocks);

/* Synchronise `stream`, then read and clear the current device's error word. */
int pa_get_device_error(cudaStream_t stream, uint32_t* flags_out);

/* Human-readable name of a status code (static string). */
const char* pa_status_string(int status);

/*
 * Host block pool: free list, reference counts, fork and copy-on-write planning.
 *
 * Blocks leave the head of an ordered free list and return to its tail (aiqz.cc,
 * section Python 演示).  Prefill takes ceil(n / B) blocks; decode takes a new block
 * every B tokens; a finished sequence returns its blocks (horeb.top, section 分配策略).
 * A block shared by several sequences is reclaimed only when its reference count
 * reaches zero (daiw.org "Paged Attention", section 量化).  When a sequence must write
 * into a partly filled last block whose count is above one, the pool plans a copy: it
 * takes a new block, moves this sequence's table entry to it and returns the (src, dst)
 * pair, which the caller copies with pa_copy_blocks before writing (chenyuan1125,
 * section 一块内存…).  An operation that cannot get every block it needs changes
 * nothing and returns PA_ERR_POOL_EXHAUSTED (daiw.org, section 速查卡: an exhausted pool
 * rejects new requests instead of failing).  Host memory only; not thread-safe.
 *
 * A second pool of CPU blocks (pa_pool_create_tiered) backs preemption: a group of
 * resident sequences is swapped out whole and later swapped back in (aiqz.cc, section
 * 连续批处理：随到随走的新秩序).  Each distinct block of the group's tables (sequences in
 * the order given, tables in order, first appearance) takes one block from the head of
 * the other pool's free list and carries the group's references to it; the old block
 * loses them and, at zero, returns to its pool's tail in that order.  The tables are
 * rewritten to the new ids.  A swapped-out sequence can be freed or swapped in; grow,
 * fork and pa_pool_slots return PA_ERR_WRONG_TIER.
 */
typedef struct pa_pool pa_pool;

/* initial_free_order: NULL for 0..num_blocks-1, else a permutation of it (host).
 * Returns NULL on a bad argument or allocation failure. */
pa_pool* pa_pool_create(int num_blocks, int block_size, const int32_t* initial_free_order);
/* The same with a CPU pool of num_cpu_blocks (>= 0) blocks, free order cpu_free_order
 * (NULL for 0..num_cpu_blocks-1, else a permutation of it). */
pa_pool* pa_pool_create_tiered(int num_blocks, int block_size, const int32_t* initial_free_order,
                               int num_cpu_blocks, const int32_t* cpu_free_order);
void pa_pool_destroy(pa_pool* pool);
/* Prefill: a new sequence holding n_tokens tokens in ceil(n_tokens / B) blocks. */
int pa_pool_allocate(pa_pool* pool, int64_t seq_id, int n_tokens);
/* Reserve the next token's slot.  Returns 0, or 1 when a copy is planned (then
 * *cow_src, *cow_dst name the blocks to copy before writing), or a negative error. */
int pa_pool_append_slot(pa_pool* pool, int64_t seq_id, int64_t* slot_out, int32_t* cow_src,
                        int32_t* cow_dst);
/* The child shares every block of the parent (reference counts + 1). */
int pa_pool_fork(pa_pool* pool, int64_t parent_id, int64_t child_id);
/* Keep the sequence's first n_tokens tokens (0 <= n_tokens <= its length), those of rejected drafts
 * say given up: its table keeps ceil(n / B) blocks, the others lose a reference and, at zero, go to
 * the free-list tail in table order.  A last block that keeps fewer tokens than its digest names
 * loses the digest (later tokens are written over the rest).  PA_ERR_ARG for n_tokens out of
 * range, PA_ERR_WRONG_TIER for a sequence swapped out. */
int pa_pool_truncate(pa_pool* pool, int64_t seq_id, int n_tokens);
/* End a sequence; blocks whose count reaches zero go to the free-list tail in table order. */
int pa_pool_free(pa_pool* pool, int64_t seq_id);
/* Copy up to `cap` table entries into out; returns the table length or an error. */
int pa_pool_block_table(const pa_pool* pool, int64_t seq_id, int32_t* out, int cap);
/* Tokens held by the sequence, or an error. */
int pa_pool_context_len(const pa_pool* pool, int64_t seq_id);
/* Slots of logical tokens [first, first + count) of the sequence (all < context_len). */
int pa_pool_slots(const pa_pool* pool, int64_t seq_id, int first, int count, int64_t* slots_out);
int pa_pool_num_free(const pa_pool* pool);
/* Copy up to `cap` free-list entries, head first; returns the free-list length. */
int pa_pool_free_list(const pa_pool* pool, int32_t* out, int cap);
/* Reference count of a block, or PA_ERR_ARG for an id outside the pool. */
int pa_pool_refcount(const pa_pool* pool, int32_t block);
/* Swap a group of n distinct resident sequences out to the CPU pool.  Writes the
 * (device block, CPU block) pairs to pairs_out [cap][2] and returns their number, or an
 * error (PA_ERR_ARG for a repeated id or cap too small, PA_ERR_UNKNOWN_SEQ,
 * PA_ERR_WRONG_TIER, PA_ERR_POOL_EXHAUSTED); on error nothing changes.  The caller then
 * copies the pairs with pa_swap_blocks (device pool -> CPU pool). */
int pa_pool_swap_out(pa_pool* pool, const int64_t* seq_ids, int n, int32_t* pairs_out, int cap);
/* The mirror image: (CPU block, device block) pairs, copied CPU pool -> device pool. */
int pa_pool_swap_in(pa_pool* pool, const int64_t* seq_ids, int n, int32_t* pairs_out, int cap);
/* 1 if the sequence is swapped out, 0 if resident, or PA_ERR_UNKNOWN_SEQ. */
int pa_pool_is_swapped(const pa_pool* pool, int64_t seq_id);
int pa_pool_num_free_cpu(const pa_pool* pool);
int pa_pool_cpu_free_list(const pa_pool* pool, int32_t* out, int cap);
int pa_pool_cpu_refcount(const pa_pool* pool, int32_t block);

/*
 * Automatic prefix caching.  A full block is named by its parent's digest, its tokens and
 * the request's extra keys, so a prompt that starts with blocks already in the pool
 * reuses their K/V and skips that part of prefill (chenyuan1125, section
 * 一块内存，如何安全地属于多条序列); `extra` (a tenant's cache salt, an adapter id, ...)
 * keeps requests that must not share apart (same page, section 分页不是免费午餐).
 * Digest of full block i (SHA-256, FIPS 180-4; integers little-endian):
 *   SHA-256(digest_{i-1} || B as u32 || tokens[iB .. iB+B-1] as i32 || extra_len as u32
 *           || extra),   digest_{-1} = 32 zero bytes.
 * The lookup walks the prompt's full blocks in order and stops at the first miss.  A hit
 * adds a reference to the cached block (taking it out of the free list if its count was
 * zero); the rest of the prompt gets blocks from the head of the free list, and each full
 * block among them is registered under its digest unless the digest already names a
 * block.  A cached block at count zero stays cached in the free list, so the free-list
 * order is the eviction order; any block taken from the head loses its digest.  Partly
 * filled blocks and blocks filled by decode are not registered.
 */
/* Prefill with prefix caching: a new sequence holding tokens[0 .. n_tokens-1] (host
 * int32).  *cached_tokens_out (may be NULL) receives the number of leading tokens whose
 * K/V the reused blocks already hold (a multiple of B); the caller computes and writes
 * the rest.  Errors as pa_pool_allocate; on error nothing changes. */
int pa_pool_allocate_prefix(pa_pool* pool, int64_t seq_id, const int32_t* tokens, int n_tokens,
                            const uint8_t* extra, int extra_len, int* cached_tokens_out);
/* A scheduler step's prompts in one call: requests r = 0..n-1 with ids seq_ids[r], tokens
 * tokens[token_start[r] .. token_start[r+1]-1] and extra bytes extras[extra_start[r] ..
 * extra_start[r+1]-1] (extras NULL: none), placed in order exactly as n calls of
 * pa_pool_allocate_prefix would.  The digest chains of different requests are computed in
 * parallel on a small pool of host threads (the library's own; batch calls are serialised
 * on it).  Outputs: cached_out[n]; slots_out (may be NULL) the slots of every request's
 * uncached tokens, request after request (what pa_reshape_and_cache takes for the new
 * rows); tables_out (may be NULL) [n][table_width] block tables padded with 0.
 * token_start and extra_start must start at 0 or above and never decrease.  A negative
 * start, a decreasing offset, a span longer than INT_MAX or a table wider than
 * table_width is PA_ERR_ARG before anything changes.  On a later error the requests
 * before the failing one stay allocated: *n_done (may be NULL) says how many. */
/* The table width a batch of n requests needs (tokens token_start[r] .. token_start[r+1]-1
 * each): the largest number of blocks one of them takes, ceil(tokens / B); PA_ERR_ARG for
 * a negative start or a decreasing offset. */
int pa_pool_table_width(const pa_pool* pool, int n, const int64_t* token_start);
int pa_pool_allocate_prefix_batch(pa_pool* pool, int n, const int64_t* seq_ids,
                                  const int32_t* tokens, const int64_t* token_start,
                                  const uint8_t* extras, const int64_t* extra_start,
                                  int* cached_out, int64_t* slots_out, int32_t* tables_out,
                                  int table_width, int* n_done);
/* The same placement from digests computed earlier (pa_prefix_block_hashes when a request
 * arrives, say, so that hashing stays off the scheduling step): request r holds
 * n_tokens[r] tokens, and `digests` holds the 32-byte digests of every request's
 * n_tokens[r] / B full blocks, request after request.  Results equal
 * pa_pool_allocate_prefix_batch on the tokens those digests came from. */
int pa_pool_allocate_hashed_batch(pa_pool* pool, int n, const int64_t* seq_ids,
                                  const int32_t* n_tokens, const uint8_t* digests,
                                  int* cached_out, int64_t* slots_out, int32_t* tables_out,
                                  int table_width, int* n_done);
/* pa_pool_free of n sequences in order; stops at the first error. */
int pa_pool_free_batch(pa_pool* pool, const int64_t* seq_ids, int n);
/* Number of blocks registered under a digest (in use or waiting in the free list). */
int pa_pool_num_cached(const pa_pool* pool);
/* 1 and the block's 32-byte digest, 0 if the block has none, or PA_ERR_ARG. */
int pa_pool_block_digest(const pa_pool* pool, int32_t block, uint8_t* digest_out);
/* The digests of the n_tokens / B full blocks of a token list into digests_out
 * [cap][32]; returns their number (pure host function). */
int pa_prefix_block_hashes(const int32_t* tokens, int n_tokens, int block_size,
                           const uint8_t* extra, int extra_len, uint8_t* digests_out, int cap);
/* SHA-256 of `len` bytes (FIPS 180-4) into digest_out[32]. */
int pa_sha256(const void* data, size_t len, uint8_t* digest_out);

#ifdef __cplusplus
}
#endif
#endif /* PA_H_ */
