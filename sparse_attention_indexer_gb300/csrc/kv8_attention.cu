// Attention over the 8-bit paged KV cache (formulas and rules in include/kv8_attention.h).
//
// One CTA per query row and query head; its warps take the keys in turn with a running
// maximum and sum each, and meet in shared memory. Lane l holds channels l * dim / 32 ...
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "kv8_attention.h"

namespace {

constexpr int kWarps = 8;

struct Params {
  const uint16_t* q;
  int64_t q_ld;
  int q_heads, kv_heads;
  float scale;  // sm_scale * log2(e)
  const int32_t* lens;
  int max_len;
  int group_rows;
  const int32_t* group_table;
  const int32_t* block_table;
  int n_tables;
  int64_t table_ld;
  int page_size;
  const int32_t* slots;  // the selected form: slots[row * slots_ld + i], i < max_len
  int64_t slots_ld;
  int block;
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  int64_t num_slots;
  uint16_t* out;
  int64_t out_ld;
  float* lse;
  int32_t* status;
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int DIM, bool FP16, bool SELECTED>
__global__ void __launch_bounds__(kWarps * 32) kv8_attention_kernel(Params p) {
  constexpr int E = DIM / 32;
  const int row = blockIdx.x, head = blockIdx.y, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int h = head / (p.q_heads / p.kv_heads);
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][DIM];
  int err = 0, len = p.max_len, table = 0;
  if (!SELECTED) {
    len = p.lens[row];
    const int g = row / p.group_rows;
    table = p.group_table ? p.group_table[g] : g;
    if (len < 0 || len > p.max_len) {
      err |= KV8_STATUS_LEN;
      len = 0;
    } else if (table < 0 || table >= p.n_tables) {
      err |= KV8_STATUS_TABLE_ROW;
      len = 0;
    } else if (((int64_t)len + p.page_size - 1) / p.page_size > p.table_ld) {
      err |= KV8_STATUS_TABLE_WIDTH;
      len = 0;
    }
  }
  float q[E], o[E], m = -INFINITY, l = 0.0f;
  for (int i = 0; i < E; ++i) {
    const uint16_t b = p.q[row * p.q_ld + (int64_t)head * DIM + lane * E + i];
    q[i] = FP16 ? __half2float(__ushort_as_half(b)) : __uint_as_float((uint32_t)b << 16);
    o[i] = 0.0f;
  }
  for (int i = warp; i < len; i += kWarps) {
    int64_t slot;
    if (SELECTED) {
      slot = p.slots[row * p.slots_ld + i];
      if (slot < 0) continue;
    } else {
      const int32_t page = p.block_table[table * p.table_ld + i / p.page_size];
      if (page < 0) {
        err |= KV8_STATUS_TABLE_ENTRY;
        continue;
      }
      slot = (int64_t)page * p.page_size + i % p.page_size;
    }
    if (slot >= p.num_slots) {
      err |= KV8_STATUS_SLOT;
      continue;
    }
    const int64_t at = (slot * p.kv_heads + h) * DIM + lane * E;
    const int64_t sc = (slot / p.block) * p.kv_heads + h;
    float x = 0.0f;
    for (int e = 0; e < E; ++e)
      x += q[e] * __half2float(__half(__nv_cvt_fp8_to_halfraw(p.k[at + e], __NV_E4M3)));
    x = warp_sum(x) * p.scale * p.k_scale[sc];
    const float top = fmaxf(m, x);
    const float keep = m == -INFINITY ? 0.0f : exp2f(m - top);
    const float w = x == -INFINITY ? 0.0f : exp2f(x - top);
    const float sv = p.v_scale[sc];
    m = top;
    l = l * keep + w;
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * keep +
             w * sv * __half2float(__half(__nv_cvt_fp8_to_halfraw(p.v[at + e], __NV_E4M3)));
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  __syncthreads();
  if (tid < DIM) {
    float top = -INFINITY, sum = 0.0f, val = 0.0f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
    for (int w = 0; w < kWarps; ++w) {
      const float f = s_m[w] == -INFINITY ? 0.0f : exp2f(s_m[w] - top);
      sum += s_l[w] * f;
      if (f != 0.0f) val += s_o[w][tid] * f;
    }
    val = sum == 0.0f ? 0.0f : val / sum;
    p.out[row * p.out_ld + (int64_t)head * DIM + tid] =
        FP16 ? __half_as_ushort(__float2half_rn(val))
             : __bfloat16_as_ushort(__float2bfloat16_rn(val));
    if (tid == 0 && p.lse)
      p.lse[(int64_t)row * p.q_heads + head] =
          sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
  }
  if (err && lane == 0 && p.status) atomicOr(p.status, err);
}

bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) % a) == 0; }

bool heads_ok(int q_heads, int kv_heads, int dim, int group_rows) {
  return kv_heads >= 1 && q_heads >= kv_heads && q_heads % kv_heads == 0 && q_heads <= 65535 &&
         q_heads / kv_heads <= 16 && (dim == 64 || dim == 128) && group_rows >= 1 &&
         group_rows <= 8;
}

// What both forms check of the arguments that they share.
int check_common(const void* q, int64_t q_ld, int dtype, int rows, int q_heads, int kv_heads,
                 int dim, float sm_scale, int group_rows, int block_tokens,
                 const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                 const float* v_scale, int64_t num_slots, void* out, int64_t out_ld,
                 const float* lse, void* workspace, const int32_t* status) {
  if ((dtype != KV8_BF16 && dtype != KV8_FP16) || rows < 0 ||
      !heads_ok(q_heads, kv_heads, dim, group_rows) || block_tokens < 16 || block_tokens % 16 ||
      num_slots < 0 || num_slots >= (int64_t(1) << 31) || num_slots % block_tokens ||
      q_ld < (int64_t)q_heads * dim || (q_ld & 7) || out_ld < (int64_t)q_heads * dim ||
      (out_ld & 7) || !std::isfinite(sm_scale))
    return KV8_ERR_SHAPE;
  if (rows == 0) return KV8_OK;
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !out || !workspace)
    return KV8_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(workspace, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
      !aligned(lse, 4) || !aligned(status, 4))
    return KV8_ERR_ALIGN;
  return KV8_OK;
}

template <bool SELECTED>
int launch(const Params& p, int rows, int dim, int dtype, cudaStream_t s) {
  const dim3 grid((unsigned)rows, (unsigned)p.q_heads);
  if (dim == 128) {
    if (dtype == KV8_FP16)
      kv8_attention_kernel<128, true, SELECTED><<<grid, kWarps * 32, 0, s>>>(p);
    else
      kv8_attention_kernel<128, false, SELECTED><<<grid, kWarps * 32, 0, s>>>(p);
  } else {
    if (dtype == KV8_FP16)
      kv8_attention_kernel<64, true, SELECTED><<<grid, kWarps * 32, 0, s>>>(p);
    else
      kv8_attention_kernel<64, false, SELECTED><<<grid, kWarps * 32, 0, s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? KV8_OK : KV8_ERR_CUDA;
}

}  // namespace

extern "C" int64_t kv8_attention_workspace_bytes(int q_heads, int kv_heads, int dim,
                                                 int group_rows) {
  if (!heads_ok(q_heads, kv_heads, dim, group_rows)) return KV8_ERR_SHAPE;
  return 16;
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
  const int64_t need = kv8_attention_workspace_bytes(q_heads, kv_heads, dim, group_rows);
  if (need < 0) return (int)need;
  if (ws_bytes < need) return KV8_ERR_WORKSPACE;
  const Params p{(const uint16_t*)q, q_ld,     q_heads,    kv_heads,    sm_scale * 1.44269504f,
                 lens,               max_len,  group_rows, group_table, block_table,
                 n_tables,           table_ld, page_size,  nullptr,     0,
                 block_tokens,       k_cache,  v_cache,    k_scale,     v_scale,
                 num_slots,          (uint16_t*)out, out_ld, lse,       status};
  return launch<false>(p, rows, dim, dtype, (cudaStream_t)stream);
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
  const int64_t need = kv8_attention_workspace_bytes(q_heads, kv_heads, dim, 1);
  if (need < 0) return (int)need;
  if (ws_bytes < need) return KV8_ERR_WORKSPACE;
  const Params p{(const uint16_t*)q, q_ld,     q_heads,  kv_heads,  sm_scale * 1.44269504f,
                 nullptr,            k,        1,        nullptr,   nullptr,
                 1,                  0,        block_tokens, slots, slots_ld,
                 block_tokens,       k_cache,  v_cache,  k_scale,   v_scale,
                 num_slots,          (uint16_t*)out, out_ld, lse,   status};
  return launch<true>(p, rows, dim, dtype, (cudaStream_t)stream);
}
