/*
 * shn_kv.h — C ABI of the paged INT8 KV cache of libshn.so: where the tokens of a batch of requests
 * go, writing and reading the pages, and attention that reads them.
 *
 * The cache holds what the codec's KV tensors hold (shn.h): INT8 values with one float32 scale per
 * group of head_dim values, cut into pages so that requests of different lengths share one buffer.
 * A page is [kv_heads][page_tokens][head_dim] contiguous bytes with its scales in the same order, so
 * a page (or a run of pages) is a codec segment as it is, and shn_decode_bf16 with
 * log2_group = log2(head_dim) reads its stream.
 *
 * Conventions are those of shn.h: caller-owned memory, asynchronous on `stream`, on the device that is
 * current for the calling thread; errors the host can see are returned and nothing is enqueued; errors
 * only the device can see (a page id outside the cache, more tokens than a buffer holds) go to the
 * status word at the start of the caller's workspace (d_work), which every call sets (0: no error, and what
 * stood in the workspace before does not matter); of several requests or tokens that are wrong it names the
 * first. A workspace serves one call at a time: calls whose GPU work may overlap (other streams, replays of
 * other graphs) need one each. Everything can be captured into a CUDA
 * graph: lengths, tables and counts are read on the device, the host arguments are sizes of buffers.
 * Results do not depend on timing: the same inputs give the same bits.
 *
 * Token t of request r lies in page block_table[r][t / page_tokens], at t % page_tokens. A slot is
 * page * page_tokens + t % page_tokens; a negative slot means "none" (padding of a captured batch).
 * Values: bfloat16 activations (uint16_t here), INT8 cache, float32 scales. Query head j reads key head
 * j / (q_heads / kv_heads).
 */
#ifndef SHN_KV_H
#define SHN_KV_H

#include "shn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace of every call here but shn_kv_attn_shared, 256-byte aligned. */
#define SHN_KV_WORKSPACE_BYTES 256u

/* One layer's cache. All four pointers are 16-byte aligned. */
typedef struct shn_kv_cache {
  int8_t* d_k;           /* [n_pages][kv_heads][page_tokens][head_dim] */
  int8_t* d_v;
  float* d_k_scale;      /* [n_pages][kv_heads][page_tokens] */
  float* d_v_scale;
  uint32_t n_pages;      /* n_pages * page_tokens < 2^31 */
  uint32_t kv_heads;     /* 1 .. 1024 */
  uint32_t page_tokens;  /* a power of two, 16 .. 1024 */
  uint32_t head_dim;     /* 64 or 128 (SHN_ERR_UNSUPPORTED otherwise) */
} shn_kv_cache;

/* SHN_OK if c describes a cache these calls accept, else SHN_ERR_INVALID_ARG or SHN_ERR_UNSUPPORTED.
 * Host only, no CUDA call. */
int shn_kv_check_cache(const shn_kv_cache* c);

/*
 * Block tables and slot maps of one step, from the requests' lengths.
 *
 * Request r holds d_ctx_len[r] tokens in the first ceil(ctx / page_tokens) pages of its table row and
 * takes d_new_len[r] more (>= 0). Pages that are missing come from d_free_pages[*d_free_head ...], in
 * request order, and are written into the row behind the ones it has.
 *  d_block_table  device, [n_reqs][max_blocks], read and extended
 *  d_free_pages   device, [n_free]; d_free_head: index of the first page not taken yet; d_free_next: receives
 *                 that index after this call (may be d_free_head itself)
 *  d_cu_new       device, [n_reqs + 1]: exclusive sum of the new tokens
 *  d_kv_len       device, [n_reqs]: ctx + new
 *  d_positions, d_slots  device, [max_tokens]: position and slot of each new token, requests one after
 *                 another; behind the last token position 0 and slot -1
 * Outputs overlap neither each other nor inputs, but for d_free_next (d_kv_len that is d_ctx_len or d_new_len is refused).
 * A page that is shared with another request must not be extended: let shared prefixes end with a page.
 * Device errors: SHN_ERR_CAPACITY (more than max_tokens new tokens, a row of more than max_blocks pages,
 * too few free pages), SHN_ERR_INVALID_ARG (a negative length, a head outside [0, n_free]). After these no
 * page is taken, the table is as it was, d_cu_new and d_kv_len are 0, d_positions 0 and d_slots -1.
 * SHN_ERR_INVALID_ARG also for a negative page id, or one whose slots pass 2^31 (its tokens get slot -1);
 * detail = the request.
 */
int shn_kv_plan(const int32_t* d_ctx_len, const int32_t* d_new_len, uint32_t n_reqs, uint32_t page_tokens,
                int32_t* d_block_table, uint32_t max_blocks, const int32_t* d_free_pages, uint32_t n_free,
                const int32_t* d_free_head, int32_t* d_free_next, int32_t* d_cu_new, int32_t* d_kv_len,
                int32_t* d_positions, int32_t* d_slots, uint32_t max_tokens, void* d_work, size_t work_bytes,
                void* stream);

/*
 * What a step's projections give, into the cache: optional RMS norm of every query and key head,
 * optional rotation by the token's position, then the query as bfloat16 and key and value quantised into
 * the token's slot. Per head row x of head_dim values, all in float32:
 *   y = x * rsqrt(mean(x^2) + eps) * weight                         (where a weight is given)
 *   the first rot_dim values turned by the angles of row position of the table (where one is given):
 *     pairs = 0: (y_i, y_{i + rot/2}) by angle i;  pairs = 1: (y_2i, y_2i+1) by angle i:
 *     (a, b) -> (a cos - b sin, b cos + a sin)
 *   query: bfloat16(y);  key, and value with y = x: scale = max(|y|max, 1e-30) / 127,
 *     int8 = round_half_even(y / scale) in [-127, 127]. A row with an infinity or NaN gets that as its scale, so
 *     that it reads as values that are not finite.
 *  d_q, d_k, d_v  device, [n_tokens][heads][head_dim], heads contiguous, tokens *_stride values apart (a
 *                 multiple of 8); 16-byte aligned. d_q may be NULL (q_heads 0: keys and values only).
 *  d_q_out        device, [n_tokens][q_heads][head_dim], tokens q_out_stride values apart; may be d_q with the same
 *                 stride. A token whose slot is negative still has its query done.
 *  d_q_weight, d_k_weight  device bfloat16 [head_dim], or NULL for no norm
 *  d_cos_sin      device float32 [n_positions][rot_dim]: rot_dim/2 cosines, then rot_dim/2 sines; 16-byte aligned;
 *                 rot_dim a multiple of 16 up to head_dim. NULL (rot_dim 0): no rotation, d_positions may be NULL.
 * Slots of one call are distinct: of two tokens with one slot, which bytes stay is not defined.
 * Device errors: SHN_ERR_INVALID_ARG for a position outside the table or a slot outside the cache (detail = the
 * token): nothing of that token is written.
 */
int shn_kv_store(const uint16_t* d_q, uint64_t q_stride, uint32_t q_heads, const uint16_t* d_k, uint64_t k_stride,
                 const uint16_t* d_v, uint64_t v_stride, uint32_t n_tokens, const int32_t* d_positions,
                 const int32_t* d_slots, const uint16_t* d_q_weight, const uint16_t* d_k_weight, float eps,
                 const float* d_cos_sin, uint32_t n_positions, uint32_t rot_dim, uint32_t pairs,
                 const shn_kv_cache* cache, uint16_t* d_q_out, uint64_t q_out_stride, void* d_work,
                 size_t work_bytes, void* stream);

/*
 * Rows of the cache as bfloat16(int8 * scale), the values shn_decode_bf16 gives for the same bytes.
 *  d_slots  device, [n_tokens], in any order, repeats allowed; the rows of a negative slot are left as they were
 *  d_k_out, d_v_out  device, [n_tokens][kv_heads][head_dim], tokens *_stride values apart (a multiple of 8),
 *           16-byte aligned; either may be NULL
 * Device errors: SHN_ERR_INVALID_ARG for a slot outside the cache (detail = the token; its rows stay).
 */
int shn_kv_load(const shn_kv_cache* cache, const int32_t* d_slots, uint32_t n_tokens, uint16_t* d_k_out,
                uint64_t k_stride, uint16_t* d_v_out, uint64_t v_stride, void* d_work, size_t work_bytes,
                void* stream);

/*
 * Causal attention of packed prompts over the cache. Request r has the queries
 * [d_cu_q[r], d_cu_q[r + 1]) and d_kv_len[r] tokens in its pages, of which the last ones are its queries' own
 * (stored before): query i of n sees the tokens 0 .. kv_len - n + i. Per query and head, in float32:
 *   s_j = softmax_scale * (q . k_j);  out = sum_j softmax(s)_j v_j, k_j and v_j = int8 * scale
 * A query that sees nothing (kv_len < n) gives zeros. Rows of d_out behind d_cu_q[n_reqs] stay as they were.
 *  d_q, d_out  device, [n_tokens][q_heads][head_dim] bfloat16, tokens *_stride values apart (a multiple of 8),
 *              16-byte aligned; they do not overlap (one that is the other is refused)
 *  q_heads     a multiple of kv_heads, at most 64 * kv_heads
 * Arithmetic: queries and keys enter the products exactly (parts of a query 2^-32 of the largest of its block of 256 rows
 * aside), scores, their scalings, the softmax and the sums are float32. At most three things are rounded to fp16, by 2^-11
 * of themselves: a weight, its token's value scale (relative to the largest of 32 tokens) and the scale's product with the INT8
 * value. What fp16 cannot hold adds up over the tokens: a query that sees n tokens, whose largest value scale is s, is exact to
 * (n 2^-30 + 2^-24) 127 s besides. Tokens that a query does not see have no part in either, whatever stands there.
 * Tokens whose value scale is not finite (or 1e36 and more) make the rows that see them NaN and leave the others alone, and so
 * does what stands behind a sequence's end in its last page.
 * Device errors: SHN_ERR_INVALID_ARG for a page id outside the cache (detail = the request; that page counts as zeros),
 * a d_kv_len that the table row cannot hold (taken as what it holds) or a d_cu_q that decreases or leaves
 * [0, n_tokens] (those queries are left out; what rows hold that are then in two ranges is not defined);
 * SHN_ERR_TIMEOUT if a wait inside a kernel gave up (a quarter of a second; the result is not complete).
 */
int shn_kv_attn_prompt(const uint16_t* d_q, uint64_t q_stride, uint32_t n_tokens, uint32_t q_heads,
                       const shn_kv_cache* cache, const int32_t* d_block_table, uint32_t max_blocks,
                       const int32_t* d_cu_q, const int32_t* d_kv_len, uint32_t n_reqs, float softmax_scale,
                       uint16_t* d_out, uint64_t out_stride, void* d_work, size_t work_bytes, void* stream);

/*
 * Attention of one query per request (a decoding step) for requests whose first *d_prefix_len tokens
 * are the same: those are read once for all queries. Query r sees the tokens 0 .. d_kv_len[r] - 1; the first
 * min(kv_len, prefix_len) of them lie in d_prefix_pages (in order), the others in the request's own table
 * row, which is indexed by the token's position as everywhere (so the pages of the prefix may stand there too,
 * but are not read). With *d_prefix_len = 0 this is plain decoding attention. kv_len 0 gives zeros.
 *  d_prefix_pages  device, [n_prefix_pages] (NULL if n_prefix_pages is 0); d_prefix_len: device, one value
 *  d_work          shn_kv_attn_shared_workspace_bytes, 256-byte aligned; what holds n_reqs requests holds fewer too
 *                  (same cache shape and q_heads)
 * Other arguments and device errors as shn_kv_attn_prompt; *d_prefix_len that the pages cannot hold is taken as what they
 * hold (SHN_ERR_INVALID_ARG). Arithmetic: as there for a large prefix (many query rows, room for many tokens in d_prefix_pages); for a
 * smaller one and for the requests' own tokens only the product of weight and value scale is rounded to fp16 (2^-11, and
 * n 2^-30 127 s), and parts of a query below 2^-25 of its largest are lost. The parts of a row meet in float32 before they are divided
 * by the sum of the weights: a sum of weights times values above 3.4e38 is infinite. A token whose value scale is not finite makes
 * the rows that see it NaN or infinite.
 * Which kernel a call takes is chosen by the sizes on the host, n_reqs, n_prefix_pages and max_blocks: a captured step with room for
 * far more tokens than it has takes what suits the room.
 */
size_t shn_kv_attn_shared_workspace_bytes(const shn_kv_cache* cache, uint32_t n_reqs, uint32_t q_heads);
int shn_kv_attn_shared(const uint16_t* d_q, uint64_t q_stride, uint32_t n_reqs, uint32_t q_heads,
                       const shn_kv_cache* cache, const int32_t* d_prefix_pages, uint32_t n_prefix_pages,
                       const int32_t* d_prefix_len, const int32_t* d_block_table, uint32_t max_blocks,
                       const int32_t* d_kv_len, float softmax_scale, uint16_t* d_out, uint64_t out_stride,
                       void* d_work, size_t work_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SHN_KV_H */
