// Store into the 8-bit paged KV cache: one power-of-two scale per (block of tokens, head)
// and e4m3 codes (the rule is stated in include/kv8_attention.h).
//
// Work split. A run is a maximal stretch of consecutive tokens of the call that lie in one
// block; run x head x {K, V} is one CTA's work, since its scale needs every token of the
// run and, where the block has earlier tokens, their old scale and codes. The first token
// of a run is found from its neighbour (same table row, position one less, same block), so
// the launch needs no lengths from the host: CTA c looks at tokens [c * chunk, (c + 1) *
// chunk) and serves the runs that start there.
//
// A row of dim 16-bit values is one 16-byte load per lane of dim / 8 lanes. The run's rows
// stay in registers between the maximum and the rounding, so each input byte is read once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kv8_attention.h"

namespace {

constexpr int kThreads = 128;
constexpr int kHold = 8;        // rows a thread keeps in registers
constexpr int kMaxChunk = 128;  // tokens whose run starts one CTA looks for

struct Params {
  const uint16_t* x[2];  // K, V
  int64_t ld[2];
  int tokens;
  int heads;
  const int32_t* positions;
  const int32_t* token_table;
  const int32_t* block_table;
  int n_tables;
  int64_t table_ld;
  int page_size;
  int block;
  uint8_t* cache[2];
  float* scale[2];
  int64_t num_slots;
  int32_t* status;
  int chunk;
};

// Whether token t starts a run: it does not continue token t - 1 inside one block.
__device__ __forceinline__ bool starts_run(const Params& p, int t) {
  if (t == 0) return true;
  const int pos = __ldg(p.positions + t), prev = __ldg(p.positions + t - 1);
  return pos <= 0 || prev != pos - 1 || pos % p.block == 0 ||
         __ldg(p.token_table + t) != __ldg(p.token_table + t - 1);
}

template <bool FP16>
__device__ __forceinline__ float2 widen(uint32_t w) {
  if (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// The least power of two s = 2^e, e >= -120, with a <= 448 s. With a = f 2^E, f in [1, 2):
// 448 = 1.75 * 2^8, so e = E - 8 where f <= 1.75 and E - 7 above. From the bits, so exact.
__device__ __forceinline__ float least_scale(float a) {
  const uint32_t b = __float_as_uint(a);
  int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(e, -120);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

template <bool FP16>
__device__ __forceinline__ float amax8(const uint4& v, float a) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = widen<FP16>(w[i]);
    const float x = fabsf(f.x), y = fabsf(f.y);
    a = fmaxf(a, x < INFINITY ? x : 0.0f);  // finite magnitudes only
    a = fmaxf(a, y < INFINITY ? y : 0.0f);
  }
  return a;
}

// x / s as codes. A power of two divides exactly by its reciprocal; a scale that the cache
// came with may be any number and takes the division.
template <bool FP16>
__device__ __forceinline__ uint2 codes8(const uint4& v, float s, float inv, bool pow2) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = widen<FP16>(w[i]);
    c[i] = pow2 ? e4m3x2(f.x * inv, f.y * inv) : e4m3x2(__fdiv_rn(f.x, s), __fdiv_rn(f.y, s));
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ uint32_t rescale4(uint32_t c, float r) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    out |= e4m3x2(f.x * r, f.y * r) << (16 * i);
  }
  return out;
}

template <int DIM, bool FP16>
__global__ void __launch_bounds__(kThreads) kv8_store_kernel(Params p) {
  constexpr int kLanes = DIM / 8;                // lanes of one token's row
  constexpr int kRows = kThreads / kLanes;       // rows per pass
  __shared__ int s_first[kMaxChunk];
  __shared__ int s_runs, s_len;
  __shared__ float s_max[kThreads / 32];
  const int tid = threadIdx.x;
  const int head = blockIdx.y, kv = blockIdx.z;
  const int t0 = blockIdx.x * p.chunk;

  if (p.chunk == 1) {
    if (!starts_run(p, t0)) return;  // the same for every thread
    if (tid == 0) {
      s_runs = 1;
      s_first[0] = t0;
    }
  } else {
    if (tid == 0) s_runs = 0;
    __syncthreads();
    if (tid < p.chunk && t0 + tid < p.tokens && starts_run(p, t0 + tid))
      s_first[atomicAdd(&s_runs, 1)] = t0 + tid;  // the order does not matter
  }
  __syncthreads();
  const int runs = s_runs;

  for (int r = 0; r < runs; ++r) {
    const int t = s_first[r];
    const int pos = __ldg(p.positions + t), row = __ldg(p.token_table + t);
    int err = 0;
    int64_t slot = -1;
    if (pos < 0) {
      err = KV8_STATUS_POSITION;
    } else if (row < 0 || row >= p.n_tables) {
      err = KV8_STATUS_TABLE_ROW;
    } else if ((int64_t)(pos / p.page_size) >= p.table_ld) {
      err = KV8_STATUS_TABLE_WIDTH;
    } else {
      const int32_t page = __ldg(p.block_table + (int64_t)row * p.table_ld + pos / p.page_size);
      slot = (int64_t)page * p.page_size + pos % p.page_size;
      if (page < 0) err = KV8_STATUS_TABLE_ENTRY;
      else if (slot >= p.num_slots) err = KV8_STATUS_SLOT;
    }
    if (err) {  // holds for the whole run: its tokens share the page
      if (tid == 0 && p.status) atomicOr(p.status, err);
      continue;
    }
    const int off = pos % p.block;
    // length of the run
    if (tid == 0) s_len = min(p.block - off, p.tokens - t);
    __syncthreads();
    for (int i = 1 + tid; i < min(p.block - off, p.tokens - t); i += kThreads)
      if (starts_run(p, t + i)) atomicMin(&s_len, i);
    __syncthreads();
    const int n = s_len;

    const int lane = tid % kLanes, sub = tid / kLanes;
    const uint16_t* src = p.x[kv] + (int64_t)t * p.ld[kv] + (int64_t)head * DIM + lane * 8;
    uint4 hold[kHold];
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
      const int i = j * kRows + sub;
      if (i < n) hold[j] = __ldg(reinterpret_cast<const uint4*>(src + (int64_t)i * p.ld[kv]));
    }
#pragma unroll
    for (int j = 0; j < kHold; ++j)
      if (j * kRows + sub < n) a = amax8<FP16>(hold[j], a);
    for (int i = kHold * kRows + sub; i < n; i += kRows)
      a = amax8<FP16>(__ldg(reinterpret_cast<const uint4*>(src + (int64_t)i * p.ld[kv])), a);
#pragma unroll
    for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (tid % 32 == 0) s_max[tid / 32] = a;
    __syncthreads();
    a = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));

    float* scale_at = p.scale[kv] + (slot / p.block) * p.heads + head;
    const float least = least_scale(a);
    float s = least;
    float before = 0.0f;
    if (off) {
      before = *scale_at;
      s = fmaxf(before, least);
    }
    const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0 && s >= 0x1p-120f;
    const float inv = __fdiv_rn(1.0f, s);
    uint8_t* dst = p.cache[kv] + (slot * p.heads + head) * DIM + lane * 8;
    const int64_t step = (int64_t)p.heads * DIM;
    __syncthreads();  // every thread has read the old scale
    if (off && s > before) {
      const float ratio = __fdiv_rn(before, s);
      for (int i = sub; i < off; i += kRows) {
        uint2* at = reinterpret_cast<uint2*>(dst + (int64_t)(i - off) * step);
        const uint2 c = *at;
        *at = make_uint2(rescale4(c.x, ratio), rescale4(c.y, ratio));
      }
    }
    if (tid == 0) *scale_at = s;
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
      const int i = j * kRows + sub;
      if (i < n)
        *reinterpret_cast<uint2*>(dst + (int64_t)i * step) = codes8<FP16>(hold[j], s, inv, pow2);
    }
    for (int i = kHold * kRows + sub; i < n; i += kRows)
      *reinterpret_cast<uint2*>(dst + (int64_t)i * step) = codes8<FP16>(
          __ldg(reinterpret_cast<const uint4*>(src + (int64_t)i * p.ld[kv])), s, inv, pow2);
    // s_len, s_max are written again only after the barriers of the next run
  }
}

bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) % a) == 0; }

}  // namespace

extern "C" int kv8_store(const uint16_t* k, int64_t k_ld, const uint16_t* v, int64_t v_ld,
                         int dtype, int tokens, int kv_heads, int dim, const int32_t* positions,
                         const int32_t* token_table, const int32_t* block_table, int n_tables,
                         int64_t table_ld, int page_size, int block_tokens, uint8_t* k_cache,
                         uint8_t* v_cache, float* k_scale, float* v_scale, int64_t num_slots,
                         int32_t* status, kv8_stream_t stream) {
  if ((dtype != KV8_BF16 && dtype != KV8_FP16) || tokens < 0 || kv_heads < 1 ||
      kv_heads > 65535 || (dim != 64 && dim != 128) || n_tables < 1 || table_ld < 1 ||
      page_size < 1 || block_tokens < 16 || block_tokens % 16 || page_size % block_tokens ||
      num_slots < 0 || num_slots >= (int64_t(1) << 31) || num_slots % page_size ||
      k_ld < (int64_t)kv_heads * dim || (k_ld & 7) || v_ld < (int64_t)kv_heads * dim ||
      (v_ld & 7))
    return KV8_ERR_SHAPE;
  if (tokens == 0) return KV8_OK;
  if (!k || !v || !positions || !token_table || !block_table || !k_cache || !v_cache ||
      !k_scale || !v_scale)
    return KV8_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(positions, 4) || !aligned(token_table, 4) || !aligned(block_table, 4) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(status, 4))
    return KV8_ERR_ALIGN;
  // A CTA per token finds the runs of a decode step at once; for a prefill most tokens start
  // no run, and a CTA per block of tokens launches as many CTAs as there is work.
  int chunk = 1;
  if ((int64_t)tokens * kv_heads * 2 > 16384)
    chunk = block_tokens < kMaxChunk ? block_tokens : kMaxChunk;
  Params p{{k, v},   {k_ld, v_ld}, tokens,    kv_heads,     positions,        token_table,
           block_table, n_tables,  table_ld,  page_size,    block_tokens,     {k_cache, v_cache},
           {k_scale, v_scale},     num_slots, status,       chunk};
  const dim3 grid((unsigned)((tokens + (int64_t)chunk - 1) / chunk), (unsigned)kv_heads, 2);
  cudaStream_t s = (cudaStream_t)stream;
  if (dim == 128) {
    if (dtype == KV8_FP16) kv8_store_kernel<128, true><<<grid, kThreads, 0, s>>>(p);
    else kv8_store_kernel<128, false><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (dtype == KV8_FP16) kv8_store_kernel<64, true><<<grid, kThreads, 0, s>>>(p);
    else kv8_store_kernel<64, false><<<grid, kThreads, 0, s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? KV8_OK : KV8_ERR_CUDA;
}
