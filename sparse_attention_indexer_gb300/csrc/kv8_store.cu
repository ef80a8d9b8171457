// Store into the 8-bit paged KV cache: one power-of-two scale per (block of tokens, head)
// and e4m3 codes (the rule is stated in include/kv8_attention.h).
//
// Work split. A run is a maximal stretch of consecutive tokens of the call that lie in one
// block; (run, head, K or V) is a unit of work, a warp's, since its scale needs every token of
// the run and, where the block has earlier tokens, their old scale and codes. The first token
// of a run is found from its neighbour (same table row, position one less, same block), so
// the launch needs no lengths from the host: CTA (c, y) looks at tokens [c * chunk, (c + 1) *
// chunk), and its warps serve the runs that start there for the four units of share y.
//
// Bound by HBM for a prefill (6 bytes per element moved), by the chain of loads (positions,
// page, values) for a decode step. A warp asks for all rows of its unit at once with cp.async,
// 16 bytes to a lane: they stay in shared memory between the maximum and the rounding, so that each
// input byte is read once, and no warp waits for another after the marks of the starts are made.
// (With the rows in registers, half as many bytes were on their way: 41 us for 20487 tokens of 8
// heads of 128, against 34 us, 3.7 TB/s, here; 64 tokens of 64 sequences take 6.4 us.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kv8_attention.h"

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxChunk = 128;  // tokens whose run starts one CTA looks for
constexpr int kWindow = 384;    // tokens from a CTA's first whose marks it keeps

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
  int hold;  // rows of a unit that stay in shared memory
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

// Magnitudes of two 16-bit values order like their bits without the sign: running maxima of the
// lower and the upper halves, infinities and NaN among them.
__device__ __forceinline__ uint32_t max8(const uint4& v, uint32_t m) {
  m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
  m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
  return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}

// The same over the finite values alone.
template <bool FP16>
__device__ __forceinline__ uint32_t max8_finite(const uint4& v, uint32_t m) {
  constexpr uint32_t kInf = FP16 ? 0x7C007C00u : 0x7F807F80u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = w[i] & 0x7FFF7FFFu;
    m = __vmaxu2(m, x & ~__vcmpgeu2(x, kInf));
  }
  return m;
}

// x / s as codes. A power of two divides exactly by its reciprocal; a scale that the cache
// came with may be any number and takes the division.
template <bool FP16>
__device__ __forceinline__ uint2 codes8(const uint4& v, float inv) {
  const float2 a = widen<FP16>(v.x), b = widen<FP16>(v.y), c = widen<FP16>(v.z),
               d = widen<FP16>(v.w);
  return make_uint2(e4m3x2(a.x * inv, a.y * inv) | (e4m3x2(b.x * inv, b.y * inv) << 16),
                    e4m3x2(c.x * inv, c.y * inv) | (e4m3x2(d.x * inv, d.y * inv) << 16));
}

template <bool FP16>
__device__ __forceinline__ uint2 codes8_div(const uint4& v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = widen<FP16>(w[i]);
    c[i] = e4m3x2(__fdiv_rn(f.x, s), __fdiv_rn(f.y, s));
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

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int DIM, bool FP16>
__global__ void __launch_bounds__(kThreads) kv8_store_kernel(const __grid_constant__ Params p) {
  constexpr int kLanes = DIM / 8;       // lanes of one token's row
  constexpr int kRows = 32 / kLanes;    // rows a warp loads at a time
  extern __shared__ __align__(16) uint4 s_rows[];
  __shared__ uint8_t s_start[kWindow];
  __shared__ int s_first[kMaxChunk];
  __shared__ int s_runs;
  const int tid = threadIdx.x, warp = tid >> 5;
  const int t0 = blockIdx.x * p.chunk;

  if (tid == 0) s_runs = 0;
  const int window = min(min(p.chunk + p.block, kWindow), p.tokens - t0);
#pragma unroll
  for (int i = 0; i < kWindow / kThreads; ++i) {
    const int x = i * kThreads + tid;
    if (x < window) s_start[x] = starts_run(p, t0 + x);
  }
  __syncthreads();
  if (tid < p.chunk && tid < window && s_start[tid])
    s_first[atomicAdd(&s_runs, 1)] = t0 + tid;  // the order does not matter
  __syncthreads();
  const int runs = s_runs;

  const int u = blockIdx.y * kWarps + warp;  // unit: head u / 2, K or V
  if (u >= 2 * p.heads) return;
  const int head = u >> 1, kv = u & 1;
  const int lane = tid % kLanes, sub = (tid & 31) / kLanes;
  uint4* rows = s_rows + (int64_t)warp * p.hold * kLanes;
  const int64_t ld = p.ld[kv];
  const int64_t step = (int64_t)p.heads * DIM;

  for (int r = 0; r < runs; ++r) {
    const int t = s_first[r];
    const int pos = __ldg(p.positions + t), row = __ldg(p.token_table + t);
    // length of the run: up to the next start, the block's end or the last token
    const int off = pos > 0 ? pos % p.block : 0;
    int n = min(p.block - off, p.tokens - t);
    for (int i0 = 1; i0 < n; i0 += 32) {
      const int i = i0 + (tid & 31), x = t - t0 + i;
      const bool start = i < n && (x < window ? s_start[x] != 0 : starts_run(p, t + i));
      const uint32_t m = __ballot_sync(0xffffffffu, start);
      if (m) n = i0 + __ffs(m) - 1;
    }

    const uint16_t* src = p.x[kv] + t * ld + (int64_t)head * DIM + lane * 8;
    const int held = min(n, p.hold);
    for (int i = sub; i < held; i += kRows)
      copy16((uint32_t)__cvta_generic_to_shared(rows + i * kLanes + lane), src + i * ld);
    asm volatile("cp.async.commit_group;" ::: "memory");
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
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (err) {  // holds for the whole run: its tokens share the page
      if (tid % 32 == 0 && p.status) atomicOr(p.status, err);
      continue;
    }
    // each lane reads back what it copied itself
    float* scale_at = p.scale[kv] + (slot / p.block) * p.heads + head;
    const float before = off ? *scale_at : 0.0f;
    const int rest = held + (sub + kRows - held % kRows) % kRows;  // this lane's first beyond
    auto row_at = [&](int i) { return __ldg(reinterpret_cast<const uint4*>(src + i * ld)); };
    uint32_t top = 0;
#pragma unroll 8
    for (int i = sub; i < held; i += kRows) top = max8(rows[i * kLanes + lane], top);
    for (int i = rest; i < n; i += kRows) top = max8(row_at(i), top);
    top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
    if (top >= (FP16 ? 0x7C00u : 0x7F80u)) {  // not finite: once more without what is not
      top = 0;
      for (int i = sub; i < held; i += kRows) top = max8_finite<FP16>(rows[i * kLanes + lane], top);
      for (int i = rest; i < n; i += kRows) top = max8_finite<FP16>(row_at(i), top);
      top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
    }
    const float a = widen<FP16>(top).x;

    const float s = off ? fmaxf(before, least_scale(a)) : least_scale(a);
    const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0 && s >= 0x1p-120f;
    const float inv = __fdiv_rn(1.0f, s);
    uint8_t* dst = p.cache[kv] + (slot * p.heads + head) * DIM + lane * 8;
    if (off && s > before) {
      const float ratio = __fdiv_rn(before, s);
      for (int i = sub; i < off; i += kRows) {
        uint2* at = reinterpret_cast<uint2*>(dst + (int64_t)(i - off) * step);
        const uint2 c = *at;
        *at = make_uint2(rescale4(c.x, ratio), rescale4(c.y, ratio));
      }
    }
    __syncwarp();  // every lane has read the old scale
    if (tid % 32 == 0) *scale_at = s;
    if (pow2) {
#pragma unroll 8
      for (int i = sub; i < held; i += kRows)
        *reinterpret_cast<uint2*>(dst + i * step) = codes8<FP16>(rows[i * kLanes + lane], inv);
    } else {
      for (int i = sub; i < held; i += kRows)
        *reinterpret_cast<uint2*>(dst + i * step) = codes8_div<FP16>(rows[i * kLanes + lane], s);
    }
    for (int i = rest; i < n; i += kRows)
      *reinterpret_cast<uint2*>(dst + i * step) =
          pow2 ? codes8<FP16>(row_at(i), inv) : codes8_div<FP16>(row_at(i), s);
  }
}

template <int DIM, bool FP16>
int launch(const Params& p, dim3 grid, cudaStream_t s) {
  const size_t bytes = (size_t)kWarps * p.hold * DIM * 2;
  const auto kernel = kv8_store_kernel<DIM, FP16>;
  if (bytes > 40960 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            kWarps * 8192 * 2) != cudaSuccess)
    return KV8_ERR_CUDA;
  kernel<<<grid, kThreads, bytes, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? KV8_OK : KV8_ERR_CUDA;
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
      kv_heads > 32767 || (dim != 64 && dim != 128) || n_tables < 1 || table_ld < 1 ||
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
  // no run, and a CTA per block of tokens launches as many CTAs as there is work. Runs of a
  // decode step are a few tokens, those of a prefill a block: 16 KB a warp hold 64 rows of 128.
  int chunk = 1, hold = 8;
  if ((int64_t)tokens * kv_heads * 2 > 16384) {
    chunk = block_tokens < kMaxChunk ? block_tokens : kMaxChunk;
    hold = block_tokens < 8192 / dim ? block_tokens : 8192 / dim;
  }
  const Params p{{k, v},   {k_ld, v_ld}, tokens,    kv_heads,     positions,        token_table,
                 block_table, n_tables,  table_ld,  page_size,    block_tokens,
                 {k_cache, v_cache},     {k_scale, v_scale},      num_slots, status, chunk, hold};
  const dim3 grid((unsigned)((tokens + (int64_t)chunk - 1) / chunk),
                  (unsigned)((2 * kv_heads + kWarps - 1) / kWarps));
  cudaStream_t s = (cudaStream_t)stream;
  if (dim == 128)
    return dtype == KV8_FP16 ? launch<128, true>(p, grid, s) : launch<128, false>(p, grid, s);
  return dtype == KV8_FP16 ? launch<64, true>(p, grid, s) : launch<64, false>(p, grid, s);
}
