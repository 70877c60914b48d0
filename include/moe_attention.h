/*
 * moe_attention.h — C ABI of the attention operators that stand beside the MoE layer (moe_prefill.h) in a transformer
 * block: attention over whole prompts, block tables and slot maps, the write into an 8-bit paged cache, and decode
 * attention over that cache. NVIDIA GB300 (sm_103a), one GPU. The functions live in libmoe_prefill.so.
 *
 * Conventions.
 *   - Status codes, moe_prefill_last_error() and their meaning are those of moe_prefill.h. Arguments are checked before
 *     any device use; a call with nothing to do (no tokens, no requests) returns MOE_OK.
 *   - All pointers are device pointers; calls enqueue work on `stream` (NULL: the default stream) and do not synchronise.
 *     No device memory is allocated.
 *   - dtype: MOE_ATTN_BF16 or MOE_ATTN_F16, the type of q, k, v and out. Strides are in elements; the head dimension is
 *     dense. Rows of q, k, v and out start on 16-byte boundaries (pointers 16-byte aligned, strides multiples of 8).
 *   - n_heads is a multiple of n_kv_heads; query head h reads kv head h / (n_heads / n_kv_heads).
 *     head_dim is 64, 128 or 256.
 *   - Scores, softmax statistics and accumulators are float32. The probabilities enter the second product rounded to the
 *     operands' type (decode: to f16), unnormalised; the sum that divides them is taken before that rounding. Where that
 *     type is f16 they are scaled up first, so that a probability keeps f16's 11 bits down to 2^-21 (decode: 2^-29) of the
 *     row's largest; below that it is off by up to 2^-32 (2^-40) of the largest. Decode takes its queries as f16, each row
 *     scaled by a power of two: exact down to 2^-28 of the row's largest.
 *   - Values in places that the mask hides (later keys, other sequences, slots past a request's length) have no
 *     influence, NaN and infinities included.
 *   - Lengths, offsets, block ids and slots on the device are not trusted: what lies outside the buffers is left out.
 */
#ifndef MOE_ATTENTION_H_
#define MOE_ATTENTION_H_

#include <stddef.h>
#include <stdint.h>

#include "moe_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MOE_ATTN_BF16 = 0, MOE_ATTN_F16 = 1 };

/*
 * Causal attention over packed sequences. Sequence b owns query rows cu_q[b] .. cu_q[b+1]-1 and key rows
 * cu_k[b] .. cu_k[b+1]-1 (int32 [n_seqs+1], ascending from 0). Its queries are the last ones of its keys: query i (of
 * q_len) sees keys 0 .. i + k_len - q_len, so k_len = q_len is a whole prompt and k_len > q_len a chunk after a prefix. A
 * query that sees no key (k_len < q_len) gets zeros and lse = -inf. Rows of out and lse that belong to no sequence (from
 * cu_q[n_seqs] on) are not written.
 *   out[t][h] = sum_j softmax_j(scale * q[t][h] . k[j][h']) v[j][h'],   lse[h][t] = ln sum_j exp(scale * q . k_j)
 * A row's output does not depend on how the prompt is cut into chunks, nor on the other sequences of the call, to the last
 * bit as long as the values are finite. Where a value that it does not see is not, a row may be computed another way,
 * which moves its last bits. A channel in which a row sees a NaN or an infinity is not finite. out must not overlap the
 * inputs.
 * Limits: n_seqs, total_q and total_k up to 2^30, (total_q + n_seqs) * n_heads below 2^31. Rows of q, k and v must be
 * apart (strides above 0); the head stride of k and v may be 0, one head's rows for all. Rows of out must be at least
 * head_dim apart.
 */
typedef struct {
  const void* q;        /* [total_q][n_heads][head_dim] */
  const void* k;        /* [total_k][n_kv_heads][head_dim] */
  const void* v;        /* [total_k][n_kv_heads][head_dim] */
  void* out;            /* [total_q][n_heads][head_dim] */
  float* lse;           /* [n_heads][total_q] or NULL */
  const int32_t* cu_q;  /* [n_seqs + 1] */
  const int32_t* cu_k;  /* [n_seqs + 1] */
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head; /* strides in elements */
  int32_t n_seqs, total_q, total_k, n_heads, n_kv_heads, head_dim, dtype;
  float scale;
} moe_attn_prefill_args;

moe_status moe_attn_prefill(const moe_attn_prefill_args* args, void* stream);

/*
 * Waits for `stream`, then reports and clears the device's error word of moe_attn_prefill: MOE_ERR_DEVICE_TIMEOUT when a
 * wait inside a kernel since the last check gave up (nothing of its CTA had advanced for 2 s; the outputs it was for are
 * then undefined), else MOE_OK.
 */
moe_status moe_attn_check(void* stream);

/*
 * Block tables and slot maps of a step, from the requests' lengths. Request b holds ctx_lens[b] cached tokens in the
 * blocks block_table[b][0 .. ceil(ctx/block_size)-1] and gets new_lens[b] tokens in this step (negative lengths count
 * as 0). The blocks it needs beyond those it holds are taken from free_blocks in order, request after request:
 *   block_table[b][i]   the new entries; entries past the request's last block become -1
 *   cu_new[n+1]         exclusive sum of new_lens: the step's tokens are packed request after request
 *   kv_lens[n]          ctx + new
 *   slot_map[max_tokens]   token -> block * block_size + offset (int64); -1 past the last token, and for tokens whose
 *                       block does not exist (free_blocks exhausted, or past max_blocks)
 *   positions[max_tokens]  token -> its position in the request; -1 past the last token
 *   used[1]             blocks needed beyond those held (more than n_free: the pool was too small)
 * Lengths, sums and positions stop at 2^31 - 1; slots do not. Calling it again with the same arguments gives the same
 * outputs. n_requests <= 16384.
 */
typedef struct {
  const int32_t* ctx_lens;     /* [n_requests] */
  const int32_t* new_lens;     /* [n_requests] */
  const int32_t* free_blocks;  /* [n_free] */
  int32_t* block_table;        /* [n_requests][max_blocks], row stride table_stride */
  int32_t* cu_new;             /* [n_requests + 1] */
  int32_t* kv_lens;            /* [n_requests] */
  int64_t* slot_map;           /* [max_tokens] */
  int32_t* positions;          /* [max_tokens] */
  int32_t* used;               /* [1] */
  int64_t table_stride;
  int32_t n_requests, n_free, max_blocks, block_size, max_tokens;
} moe_kv_assign_args;

moe_status moe_kv_assign(const moe_kv_assign_args* args, void* stream);

/*
 * The 8-bit paged cache: codes [num_blocks][n_kv_heads][block_size][head_dim] e4m3 and one float32 scale for each
 * (block, kv head), for K and for V; a stored value is code * scale. block_size is 16, 32, 64 or 128; the codes start
 * on 16-byte boundaries.
 *
 * moe_kv_append writes the tokens of k and v at slot_map[t] (block * block_size + offset; slots outside the cache, such
 * as -1, are skipped). Tokens of one block follow one another in the call, in ascending offsets. The scale of a block is
 * the smallest power of two (from 2^-40 to 2^40) that brings its largest magnitude to 448 or less; a
 * power of two costs e4m3 no precision. Where the first token written to a block has offset 0 the block is taken as new;
 * otherwise its scale only grows, and the codes it holds are rewritten for the new scale (multiplied by a power of two,
 * rounded to nearest even). NaN stays NaN and takes no part in the scale, nor do infinities, which saturate.
 */
typedef struct {
  const void* k;            /* [n_tokens][n_kv_heads][head_dim] */
  const void* v;
  const int64_t* slot_map;  /* [n_tokens] */
  void* k_codes;
  void* v_codes;
  float* k_scale;           /* [num_blocks][n_kv_heads] */
  float* v_scale;
  int64_t k_token, k_head, v_token, v_head; /* strides in elements */
  int32_t n_tokens, n_kv_heads, head_dim, dtype, block_size, num_blocks;
} moe_kv_append_args;

moe_status moe_kv_append(const moe_kv_append_args* args, void* stream);

/*
 * Attention of one query token a request over the cache: request b attends to its first kv_lens[b] slots (at most
 * max_blocks * block_size), in the blocks block_table[b][..]; slots whose block id lies outside the cache are left out. No
 * slot: zeros and lse = -inf. Rows of out must be at least head_dim apart. Scales may be any normal float32 values from
 * 2^-40 to 2^40; a V scale of 0 leaves its block out. The cache is split over the GPU by the requests' lengths and the
 * pieces are joined in a fixed order: the same call gives the same bytes.
 * workspace: moe_attn_decode_workspace() bytes, 16-byte aligned, needs no initialisation; calls that overlap on the GPU
 * need one each.
 */
typedef struct {
  const void* q;               /* [n_requests][n_heads][head_dim] */
  const void* k_codes;
  const void* v_codes;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;  /* [n_requests][max_blocks], row stride table_stride */
  const int32_t* kv_lens;      /* [n_requests] */
  void* out;                   /* [n_requests][n_heads][head_dim] */
  float* lse;                  /* [n_requests][n_heads] or NULL */
  void* workspace;
  size_t workspace_bytes;
  int64_t q_token, q_head, out_token, out_head, table_stride; /* strides in elements */
  int32_t n_requests, n_heads, n_kv_heads, head_dim, dtype, block_size, num_blocks, max_blocks;
  float scale;
} moe_attn_decode_args;

size_t moe_attn_decode_workspace(int32_t n_requests, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim);
moe_status moe_attn_decode(const moe_attn_decode_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTENTION_H_ */
