/* Attention over a paged KV cache held in 8 bits (e4m3) with one fp32 scale for each
 * block of tokens and head, and the store that fills such a cache.
 *
 * Cache. K and V are e4m3 codes [num_slots, kv_heads, dim]; a slot is
 * page * page_size + offset, the slot that topk_select_paged writes. Scales are
 * [num_slots / block_tokens, kv_heads]: a code c of slot s and head h stands for
 * c * scale[s / block_tokens, h]. block_tokens divides page_size, so a block lies
 * inside one page.
 *
 * Store (kv8_store). For the new tokens of one block and head, with a the largest
 * finite magnitude among them, the block's scale becomes the least power of two
 * s = 2^e, e >= -120, with a <= 448 * 2^e; where the block has earlier tokens (the
 * run of new tokens does not start at the block's first position) it becomes the
 * larger of that and the scale the block has, and where it grows the earlier tokens'
 * codes are rounded again as codes of the new scale. Codes are rounded to nearest
 * even and saturate at +-448 (an infinity stores 448 of its sign, a NaN stores NaN).
 * A power of two costs a floating code no precision and makes the growth of a scale
 * exact except for codes that become subnormal.
 *
 * Attention (kv8_attention, kv8_attention_selected). For query row t and query head
 * i, reading key head h = i / (q_heads / kv_heads):
 *   x(p) = sm_scale * sum_d q(t, i, d) * k(p, h, d),
 *   lse(t, i) = log sum_p exp(x(p)),  out(t, i) = sum_p exp(x(p) - lse) * v(p, h).
 * kv8_attention takes p over positions [0, lens[t]) through a block table, for decode
 * steps and for verify steps of up to 8 query rows per request; kv8_attention_selected
 * takes p over a list of slots per query row (the out_slots of topk_select_paged),
 * skipping negative ones. A row that attends to nothing gives out 0 and lse -infinity.
 * What lies at positions that a row does not attend to, NaN codes and scales among it,
 * never reaches its result. Scales must be >= 0. Scores, softmax statistics and sums are
 * fp32; the weights exp(..) are rounded to fp16 relative to the row's largest weight *
 * value scale. A weight, or weight * value scale, below 2^-120 of the row's largest weight
 * may count as 0. The result does not depend on the run (no floating-point atomics).
 */
#ifndef KV8_ATTENTION_H
#define KV8_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* kv8_stream_t; /* identical to cudaStream_t */

/* Types of q / out and of the tokens to store. */
enum { KV8_BF16 = 0, KV8_FP16 = 1 };

/* Host-side return codes (negative: nothing was enqueued). */
enum {
  KV8_OK = 0,
  KV8_ERR_NULL = -1,      /* a required pointer is NULL (with rows / tokens > 0) */
  KV8_ERR_SHAPE = -2,     /* rows, tokens, max_len or k < 0, dim not 64 or 128, kv_heads < 1,
                             q_heads not a multiple of kv_heads or more than 16 times it,
                             group_rows outside [1, 8], dtype unknown, page_size < 1,
                             block_tokens not a positive multiple of 16, page_size not a
                             multiple of block_tokens, num_slots < 0, >= 2^31 or not a
                             multiple of page_size (of block_tokens for the selected form),
                             n_tables < 1, table_ld < 1, a row stride below the row or not
                             a multiple of 8, slots_ld < k, sm_scale not finite, more
                             than 2^33 pairs of a group and a key head; of the shared form
                             n_sets outside [0, KV8_MAX_SETS], max_prefix < 0 or
                             (rows + group_rows) * (q_heads / kv_heads) >= 2^31 */
  KV8_ERR_ALIGN = -3,     /* q, out, k, v, caches or workspace not 16-byte aligned, or
                             another array not 4-byte aligned */
  KV8_ERR_CUDA = -4,      /* a launch or a device query failed */
  KV8_ERR_WORKSPACE = -5  /* workspace smaller than kv8_attention_workspace_bytes, or for the shared
                             form kv8_attention_shared_workspace_bytes, whatever its bounds */
};

/* Device status bits, OR-ed into *status. */
enum {
  KV8_STATUS_LEN = 1,          /* a length < 0 or > max_len: the row attends to nothing */
  KV8_STATUS_TABLE_WIDTH = 2,  /* a position's page is past table_ld: row attends to
                                  nothing / token not stored */
  KV8_STATUS_TABLE_ENTRY = 4,  /* negative page entry: position skipped / not stored */
  KV8_STATUS_SLOT = 8,         /* slot >= num_slots: position skipped / not stored */
  KV8_STATUS_TABLE_ROW = 16,   /* table row outside [0, n_tables): rows attend to nothing /
                                  token not stored */
  KV8_STATUS_POSITION = 32,    /* kv8_store: a negative position: token not stored */
  KV8_STATUS_SETS = 64,        /* kv8_attention_shared: set_starts falls or leaves [0, groups]: no
                                  prefix is read once for several rows; or a prefix length
                                  outside [0, max_prefix]: that set's is not */
  KV8_STATUS_TIMEOUT = 128     /* kv8_attention_shared: a wait inside the kernel ran out (200 ms of
                                  wall time): rows and heads whose prefix it was to give are NaN
                                  in out and lse, the others are right */
};

/* Quantises `tokens` tokens into the cache. One launch.
 *   k, v         device bf16 / fp16 bits [tokens, ld], head h at columns [h * dim, ..);
 *                16-byte aligned, ld >= kv_heads * dim, a multiple of 8
 *   positions    device int32 [tokens]: position of each token in its request
 *   token_table  device int32 [tokens]: block-table row of each token's request
 *   block_table  device int32 [n_tables, table_ld]: page ids
 *   caches       device uint8 [num_slots, kv_heads, dim], 16-byte aligned
 *   scales       device float32 [num_slots / block_tokens, kv_heads]
 *   status       device int32 [1] or NULL: KV8_STATUS_* bits OR-ed in
 * Tokens of one request are consecutive and at consecutive positions. A run of them
 * inside one block is an append: the block's positions after the run are taken to
 * hold nothing. Two runs in the same block in one call race. Pages shared by several
 * rows must be made single first (kvpages_reserve). */
int kv8_store(const uint16_t* k, int64_t k_ld, const uint16_t* v, int64_t v_ld, int dtype,
              int tokens, int kv_heads, int dim, const int32_t* positions,
              const int32_t* token_table, const int32_t* block_table, int n_tables,
              int64_t table_ld, int page_size, int block_tokens, uint8_t* k_cache,
              uint8_t* v_cache, float* k_scale, float* v_scale, int64_t num_slots,
              int32_t* status, kv8_stream_t stream);

/* Bytes of workspace that any attention call with these heads, dim and group_rows (1
 * for the selected form) needs on the current device, whatever its rows and lengths.
 * Queries the device. Negative: a KV8_ERR_* code. */
int64_t kv8_attention_workspace_bytes(int q_heads, int kv_heads, int dim, int group_rows);

/* Attention through a block table. Two launches.
 *   q            device bf16 / fp16 [rows, q_ld], head i at columns [i * dim, ..)
 *   lens         device int32 [rows]: row t attends to positions [0, lens[t])
 *   max_len      bound on every length
 *   group_rows   G in [1, 8]: rows g*G .. g*G + G - 1 (the last group may be shorter)
 *                share one block-table row, and their keys are read once for all
 *   group_table  device int32 [ceil(rows / G)] or NULL (group g uses row g)
 *   block_table  device int32 [n_tables, table_ld]; entries past a length are not read
 *   out          device, q's type [rows, out_ld], 16-byte aligned; may not overlap q
 *   lse          device float32 [rows, q_heads] or NULL
 *   workspace    device, 16-byte aligned; what it holds before and after is of no account.
 *                One workspace serves one stream at a time, and its two launches belong
 *                together: host threads that share one enqueue their calls one after another. */
int kv8_attention(const void* q, int64_t q_ld, int dtype, int rows, int q_heads, int kv_heads,
                  int dim, float sm_scale, const int32_t* lens, int max_len, int group_rows,
                  const int32_t* group_table, const int32_t* block_table, int n_tables,
                  int64_t table_ld, int page_size, int block_tokens, const uint8_t* k_cache,
                  const uint8_t* v_cache, const float* k_scale, const float* v_scale,
                  int64_t num_slots, void* out, int64_t out_ld, float* lse, void* workspace,
                  int64_t ws_bytes, int32_t* status, kv8_stream_t stream);

/* Attention over a list of slots per query row. Two launches. Arguments as above, and
 *   slots        device int32 [rows, slots_ld]: k slots per row; negative ones are
 *                skipped; a slot given twice counts twice */
int kv8_attention_selected(const void* q, int64_t q_ld, int dtype, int rows, int q_heads,
                           int kv_heads, int dim, float sm_scale, const int32_t* slots, int k,
                           int64_t slots_ld, int block_tokens, const uint8_t* k_cache,
                           const uint8_t* v_cache, const float* k_scale, const float* v_scale,
                           int64_t num_slots, void* out, int64_t out_ld, float* lse,
                           void* workspace, int64_t ws_bytes, int32_t* status,
                           kv8_stream_t stream);

/* Bytes of workspace of a kv8_attention_shared call with these heads, dim and group_rows and at
 * most `rows` query rows on the current device. Queries the device. Negative: a KV8_ERR_* code. */
int64_t kv8_attention_shared_workspace_bytes(int rows, int q_heads, int kv_heads, int dim,
                                             int group_rows);

/* kv8_attention for batches whose requests share prefixes (samples of one prompt, requests
 * behind one system prompt): the result is kv8_attention's, but positions that a set of
 * groups shares are read once for the whole set, as one product of all its query rows.
 * Four launches. Arguments as above, and
 *   set_starts   device int32 [n_sets + 1], rising, within [0, groups]: set s is the groups
 *                set_starts[s] .. set_starts[s + 1] - 1; groups of no set share nothing
 *   n_sets       at most KV8_MAX_SETS
 *   prefix_lens  device int32 [n_sets]: positions p < prefix_lens[s] hold the same keys and
 *                values in the block-table rows of all groups of set s (kvpages_shared finds
 *                them). They are read through the row of the set's first group that has keys, as
 *                far as they lie below the least length > 0 of the set's rows. A set of one
 *                such group, or less than 128 positions, is left to the rows' own pass
 *   max_prefix   bound on every prefix length. Where (groups - 1) * max_prefix positions are less
 *                than 256 MB of keys and values, sharing saves no time: the call is
 *                kv8_attention's (two launches), and sets and prefixes are not looked at. A loose
 *                bound, or many groups of no set, cost two launches more (about 25 us)
 *   workspace    of kv8_attention_shared_workspace_bytes; the four launches belong together
 * Numbers are held as in kv8_attention; where value scales of a prefix lie within 2^8 of its
 * first one, weights keep 2^-31 of the row's largest weight * value scale, else each row's
 * weights are taken relative to its own largest. A value scale that is infinite makes the rows
 * that see it NaN. (rows + group_rows) * (q_heads / kv_heads) < 2^31. */
#define KV8_MAX_SETS 1024
int kv8_attention_shared(const void* q, int64_t q_ld, int dtype, int rows, int q_heads,
                         int kv_heads, int dim, float sm_scale, const int32_t* lens, int max_len,
                         int group_rows, const int32_t* group_table, const int32_t* set_starts,
                         int n_sets, const int32_t* prefix_lens, int max_prefix,
                         const int32_t* block_table, int n_tables, int64_t table_ld,
                         int page_size, int block_tokens, const uint8_t* k_cache,
                         const uint8_t* v_cache, const float* k_scale, const float* v_scale,
                         int64_t num_slots, void* out, int64_t out_ld, float* lse,
                         void* workspace, int64_t ws_bytes, int32_t* status,
                         kv8_stream_t stream);

/* Test entry: kv8_attention_shared with a CTA (skip_cta >= 0; -1 = none) of the prefixes' pass
 * whose keys and values never come, so that its waits run out: the call ends after 200 ms with
 * KV8_STATUS_TIMEOUT and NaN for the rows and heads of that CTA. */
int kv8_attention_shared_test(const void* q, int64_t q_ld, int dtype, int rows, int q_heads,
                              int kv_heads, int dim, float sm_scale, const int32_t* lens,
                              int max_len, int group_rows, const int32_t* group_table,
                              const int32_t* set_starts, int n_sets, const int32_t* prefix_lens,
                              int max_prefix, const int32_t* block_table, int n_tables,
                              int64_t table_ld, int page_size, int block_tokens,
                              const uint8_t* k_cache, const uint8_t* v_cache,
                              const float* k_scale, const float* v_scale, int64_t num_slots,
                              void* out, int64_t out_ld, float* lse, void* workspace,
                              int64_t ws_bytes, int32_t* status, kv8_stream_t stream,
                              int skip_cta);

#ifdef __cplusplus
}
#endif

#endif /* KV8_ATTENTION_H */
