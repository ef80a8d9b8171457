// Entry points of the attention over the 8-bit paged KV cache through block tables and over
// selected slots (include/kv8_attention.h); the kernels are in kv8_attention.cuh.
#include "kv8_attention.cuh"

extern "C" int64_t kv8_attention_workspace_bytes(int q_heads, int kv_heads, int dim,
                                                 int group_rows) {
  if (!heads_ok(q_heads, kv_heads, dim, group_rows)) return KV8_ERR_SHAPE;
  const int sms = sm_count(current_device());
  if (sms < 0) return KV8_ERR_CUDA;
  const int rows = padded_rows(group_rows * (q_heads / kv_heads));
  const int64_t most = (int64_t)sms * (rows <= 16 ? 12 : 2);  // CTAs of any variant for these rows
  const int64_t ctas = most < kMaxCtas ? most : kMaxCtas;
  return kMaxCtas * (int64_t)sizeof(Shared) + ctas * 2 * rows * (dim + 4) * 4;
}

extern "C" int kv8_attention(const void* q, int64_t q_ld, int dtype, int rows, int q_heads,
                             int kv_heads, int dim, float sm_scale, const int32_t* lens,
                             int max_len, int group_rows, const int32_t* group_table,
                             const int32_t* block_table, int n_tables, int64_t table_ld,
                             int page_size, int block_tokens, const uint8_t* k_cache,
                             const uint8_t* v_cache, const float* k_scale, const float* v_scale,
                             int64_t num_slots, void* out, int64_t out_ld, float* lse,
                             void* workspace, int64_t ws_bytes, int32_t* status,
                             kv8_stream_t stream) {
  if (max_len < 0 || n_tables < 1 || table_ld < 1 || page_size < 1 || block_tokens < 16 ||
      page_size % block_tokens || num_slots % page_size)
    return KV8_ERR_SHAPE;
  const int err = check_common(q, q_ld, dtype, rows, q_heads, kv_heads, dim, sm_scale,
                               group_rows, block_tokens, k_cache, v_cache, k_scale, v_scale,
                               num_slots, out, out_ld, lse, workspace, status);
  if (err || rows == 0) return err;
  if (!lens || !block_table) return KV8_ERR_NULL;
  if (!aligned(lens, 4) || !aligned(group_table, 4) || !aligned(block_table, 4))
    return KV8_ERR_ALIGN;
  Params p = common(q, q_ld, rows, q_heads, kv_heads, sm_scale, block_tokens, k_cache, v_cache,
                    k_scale, v_scale, num_slots, out, out_ld, lse, status);
  p.lens = lens;
  p.max_len = max_len;
  p.group_rows = group_rows;
  p.group_table = group_table;
  p.block_table = block_table;
  p.n_tables = n_tables;
  p.table_ld = table_ld;
  p.page_size = page_size;
  p.page_shift = shift_of(page_size);
  return run<false>(p, dim, dtype, workspace, ws_bytes, (cudaStream_t)stream);
}

extern "C" int kv8_attention_selected(const void* q, int64_t q_ld, int dtype, int rows,
                                      int q_heads, int kv_heads, int dim, float sm_scale,
                                      const int32_t* slots, int k, int64_t slots_ld,
                                      int block_tokens, const uint8_t* k_cache,
                                      const uint8_t* v_cache, const float* k_scale,
                                      const float* v_scale, int64_t num_slots, void* out,
                                      int64_t out_ld, float* lse, void* workspace,
                                      int64_t ws_bytes, int32_t* status, kv8_stream_t stream) {
  if (k < 0 || slots_ld < k) return KV8_ERR_SHAPE;
  const int err = check_common(q, q_ld, dtype, rows, q_heads, kv_heads, dim, sm_scale, 1,
                               block_tokens, k_cache, v_cache, k_scale, v_scale, num_slots, out,
                               out_ld, lse, workspace, status);
  if (err || rows == 0) return err;
  if (k > 0 && !slots) return KV8_ERR_NULL;
  if (!aligned(slots, 4)) return KV8_ERR_ALIGN;
  Params p = common(q, q_ld, rows, q_heads, kv_heads, sm_scale, block_tokens, k_cache, v_cache,
                    k_scale, v_scale, num_slots, out, out_ld, lse, status);
  p.slots = slots;
  p.slots_ld = slots_ld;
  p.max_len = k;
  p.group_rows = 1;
  return run<true>(p, dim, dtype, workspace, ws_bytes, (cudaStream_t)stream);
}
