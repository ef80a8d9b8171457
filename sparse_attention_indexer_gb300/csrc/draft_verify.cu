// Verification of drafted tokens (rules in include/draft_verify.h).
//
// A request reads two probabilities per draft for the tests and then one row (the bonus
// row) or two (target and draft of the refused position) of the vocabulary: bound by HBM for
// a batch, by latency for one request. A cluster of C CTAs takes a request; every CTA decides
// the tests for itself (a few loads), each warp sums a slice of the weights in steps of 256
// tokens, 8 consecutive 32s, all loads of a step on their way together, and keeps the sum of
// each step in shared memory. The slices' sums meet through distributed shared memory; the
// warp whose slice holds the drawn point finds the step from the sums kept, and reads this
// step alone again. Sums are 64-bit integers, so the split of the row does not show in the
// result.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "draft_verify.h"

namespace cg = cooperative_groups;

namespace {

constexpr int kStep = 8;      // tokens of a lane in a step
constexpr int kRecords = 64;  // sums of steps that a warp keeps

struct Params {
  const float* target;
  int64_t target_req, target_row;
  const float* draft;
  int64_t draft_req, draft_row;
  const int32_t* tokens;
  const int32_t* n_drafts;
  const float* uniforms;
  int drafts;
  int vocab;
  int32_t* out_tokens;
  int32_t* kept;
  int32_t* status;
};

__device__ __forceinline__ float checked_prob(float x, int* err) {
  if (__float_as_uint(x) > 0x3F800000u && !(x == 0.0f)) {  // above 1, negative or NaN
    *err |= VERIFY_STATUS_PROB;
    return x > 1.0f ? 1.0f : 0.0f;
  }
  return x;
}

__device__ __forceinline__ float checked_uniform(float u, int* err) {
  if (!(u >= 0.0f && u < 1.0f)) {
    *err |= VERIFY_STATUS_UNIFORM;
    return u >= 1.0f ? 0x1.fffffep-1f : 0.0f;
  }
  return u;
}

// A probability in [0, 1] in units of 2^-60, rounded down: its 24 significant bits, shifted. In
// integer operations, as the conversion to 64 bits is slow: 45 us against MEASURED for 64 requests.
__device__ __forceinline__ uint64_t units(float x) {
  const uint32_t b = __float_as_uint(x);
  const uint32_t e = (b >> 23) & 0xFF, m = (b << 8) | 0x80000000u;
  const uint32_t s = 130 - e;  // m * 2^32 >> s; 3 for 1.0
  const uint32_t lo = s <= 32 ? __funnelshift_rc(0, m, s) : s < 64 ? m >> (s - 32) : 0;
  const uint32_t hi = s < 32 ? m >> s : 0;
  return ((uint64_t)hi << 32) | lo;  // a subnormal is below the last bit
}

// max(p - q, 0) in those units; a non-negative q >= p gives 0.
__device__ __forceinline__ uint64_t weight(float p, float q) {
  const uint64_t a = units(p), b = units(q);
  return a > b ? a - b : 0;
}

enum Row { kBonus, kRefused, kRefusedPoint };

// The weights of tokens v0 + 32 i + lane, i < kStep; 0 past `end`. Tokens past it read the
// row's last one instead, so that no load waits for a condition.
__device__ __forceinline__ void step_weights(const float* p, const float* q, Row row, int point,
                                             int v0, int end, uint64_t (&w)[kStep], int* err) {
  const int lane = threadIdx.x & 31;
  float a[kStep], b[kStep];
#pragma unroll
  for (int i = 0; i < kStep; ++i) a[i] = __ldg(p + min(v0 + i * 32 + lane, end - 1));
  if (row == kRefused) {
#pragma unroll
    for (int i = 0; i < kStep; ++i) b[i] = __ldg(q + min(v0 + i * 32 + lane, end - 1));
#pragma unroll
    for (int i = 0; i < kStep; ++i) w[i] = weight(checked_prob(a[i], err), checked_prob(b[i], err));
  } else {
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      w[i] = units(checked_prob(a[i], err));
      if (row == kRefusedPoint && v0 + i * 32 + lane == point) w[i] = 0;
    }
  }
#pragma unroll
  for (int i = 0; i < kStep; ++i)
    if (v0 + i * 32 + lane >= end) w[i] = 0;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) draft_verify_kernel(Params p) {
  constexpr int kWarps = THREADS / 32;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int req = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int s_kept;
  __shared__ uint64_t s_sum[kWarps];
  __shared__ uint64_t s_high[kWarps];
  __shared__ uint64_t s_cta[2];  // read by the cluster: the sum, and that of its upper halves
  __shared__ uint64_t s_step[kWarps][kRecords];
  int err = 0;

  const int n = p.n_drafts ? __ldg(p.n_drafts + req) : p.drafts;
  int32_t* out = p.out_tokens + (int64_t)req * (p.drafts + 1);
  if (n < 0 || n > p.drafts) {  // the same for the whole cluster
    if (rank == 0) {
      if (tid <= p.drafts) out[tid] = -1;
      if (tid == 0) {
        p.kept[req] = 0;
        if (p.status) atomicOr(p.status, VERIFY_STATUS_COUNT);
      }
    }
    return;
  }
  const float* uni = p.uniforms + (int64_t)req * (p.drafts + 1);
  const float* target = p.target + (int64_t)req * p.target_req;
  const float* draft = p.draft ? p.draft + (int64_t)req * p.draft_req : nullptr;
  const int32_t* tok = p.tokens + (int64_t)req * p.drafts;

  // the tests: one lane per draft (at most 31)
  if (warp == 0) {
    bool keep = false;
    int e = 0;
    if (lane < n) {
      const int t = __ldg(tok + lane);
      if (t < 0 || t >= p.vocab) {
        e = VERIFY_STATUS_TOKEN;
      } else {
        const float pt = checked_prob(__ldg(target + lane * p.target_row + t), &e);
        const float qt = draft ? checked_prob(__ldg(draft + lane * p.draft_row + t), &e) : 1.0f;
        const float u = checked_uniform(__ldg(uni + lane), &e);
        keep = (double)u * (double)qt < (double)pt;  // 24 + 24 bits: the product is exact
      }
    }
    const uint32_t refused = ~__ballot_sync(0xffffffffu, keep);
    const int a = min(n, __ffs(refused) - 1);
    if (lane <= a) err |= e;  // what lies behind the first refusal is not looked at
    if (lane == 0) s_kept = a;
  }
  __syncthreads();
  const int kept = s_kept;
  const float* prow = target + kept * p.target_row;
  const float* qrow = draft && kept < n ? draft + kept * p.draft_row : nullptr;
  const int point = kept < n ? __ldg(tok + kept) : -1;
  Row row = kept == n ? kBonus : qrow ? kRefused : kRefusedPoint;

  // slices: CTA, then warp, each a whole number of steps; a record sums `each` steps
  constexpr int kTokens = 32 * kStep;
  const int parts = ranks * kWarps;
  const int64_t stride = (int64_t)parts * kTokens;
  const int steps = (int)((p.vocab + stride - 1) / stride);
  const int each = (steps + kRecords - 1) / kRecords;
  const int64_t begin64 = ((int64_t)rank * kWarps + warp) * steps * kTokens;
  const int begin = (int)min(begin64, (int64_t)p.vocab);
  const int end = (int)min(begin64 + (int64_t)steps * kTokens, (int64_t)p.vocab);

  // A row that sums to 16 or more would wrap the sums: the upper halves tell
  uint64_t total = 0, before = 0, high = 0;
  for (int round = 0; round < 2; ++round) {
    uint64_t sum = 0, record = 0, upper = 0;
    int v0 = begin;
    for (int i = 0; v0 < end; ++i, v0 += kTokens) {
      uint64_t w[kStep], x = 0;
      step_weights(prow, qrow, row, point, v0, end, w, &err);
#pragma unroll
      for (int k = 0; k < kStep; ++k) x += w[k];
      upper += x >> 32;
      x = warp_sum(x);
      sum += x;
      record += x;
      if (i % each == each - 1 || v0 + kTokens >= end) {
        if (lane == 0) s_step[warp][i / each] = record;
        record = 0;
      }
    }
    upper = warp_sum(upper);
    if (lane == 0) {
      s_sum[warp] = sum;
      s_high[warp] = upper;
    }
    __syncthreads();
    if (warp == 0) {
      const uint64_t c = warp_sum(lane < kWarps ? s_sum[lane] : 0);
      const uint64_t d = warp_sum(lane < kWarps ? s_high[lane] : 0);
      if (lane == 0) {
        s_cta[0] = c;
        s_cta[1] = d;
      }
    }
    cluster.sync();
    total = before = high = 0;
    for (int r = 0; r < ranks; ++r) {
      const uint64_t* c = cluster.map_shared_rank(s_cta, r);
      if (r < rank) before += c[0];
      total += c[0];
      high += c[1];
    }
    if (total || high || row == kBonus) break;
    row = kBonus;  // nothing is left of p - q: draw from p itself
    cluster.sync();
  }

  const float r = checked_uniform(__ldg(uni + p.drafts), &err);
  const uint64_t at = __umul64hi(total, __float2ull_rz(r * 0x1p64f));  // floor(r * total)
  const bool lost = high >= uint64_t(15) << 28;
  if (lost || total > (uint64_t(1) << 63)) err |= VERIFY_STATUS_PROB;
  for (int w = 0; w < warp; ++w) before += s_sum[w];
  const uint64_t mine = s_sum[warp];
  // the warp whose range holds the point: before <= at < before + mine
  if (total && !lost && at >= before && at - before < mine) {
    uint64_t run = before;
    int i = 0;
    while (run + s_step[warp][i] <= at) run += s_step[warp][i++];  // ends: run + mine > at
    int ignored = 0;
    for (int v0 = begin + i * each * kTokens;; v0 += kTokens) {
      uint64_t w[kStep];
      step_weights(prow, qrow, row, point, v0, end, w, &ignored);
      int token = -1;
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        uint64_t x = w[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, run + x > at);
        if (past && token < 0) token = v0 + k * 32 + __ffs(past) - 1;
        run += __shfl_sync(0xffffffffu, x, 31);
      }
      if (token >= 0 || v0 + kTokens >= end) {
        if (lane == 0) out[kept] = token;
        break;
      }
    }
  }
  if (rank == 0) {
    if (tid <= p.drafts && tid != kept) out[tid] = tid < kept ? __ldg(tok + tid) : -1;
    if (tid == 0) {
      p.kept[req] = kept;
      if (lost) {
        out[kept] = -1;
      } else if (total == 0) {
        out[kept] = -1;
        err |= VERIFY_STATUS_EMPTY;
      }
    }
  }
  if (err && p.status) atomicOr(p.status, err);
  cluster.sync();  // no CTA leaves while another still reads its sum
}

bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) % a) == 0; }

}  // namespace

extern "C" int draft_verify(const float* target, int64_t target_req, int64_t target_row,
                            const float* draft, int64_t draft_req, int64_t draft_row,
                            const int32_t* tokens, const int32_t* n_drafts,
                            const float* uniforms, int reqs, int drafts, int vocab,
                            int32_t* out_tokens, int32_t* kept, int32_t* status,
                            verify_stream_t stream) {
  if (reqs < 0 || reqs > (1 << 27) || drafts < 0 || drafts > VERIFY_MAX_DRAFTS || vocab < 1 ||
      vocab > (1 << 30) || target_req < 0 || (drafts > 0 && target_row < vocab) ||
      (draft && drafts > 0 && (draft_req < 0 || draft_row < vocab)))
    return VERIFY_ERR_SHAPE;
  if (reqs == 0) return VERIFY_OK;
  if (!target || (drafts > 0 && !tokens) || !uniforms || !out_tokens || !kept)
    return VERIFY_ERR_NULL;
  if (!aligned(target, 4) || !aligned(draft, 4) || !aligned(tokens, 4) || !aligned(n_drafts, 4) ||
      !aligned(uniforms, 4) || !aligned(out_tokens, 4) || !aligned(kept, 4) ||
      !aligned(status, 4))
    return VERIFY_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return VERIFY_ERR_CUDA;
  // CTAs per request: up to 8 while they all run at once (1024 threads to an SM) and a warp has
  // a step to sum. Few requests take CTAs of 512 threads, more of them smaller ones, which
  // spread evenly: 64 requests of 100K tokens 256 x 512 threads MEASURED, 512 x 256 MEASURED.
  const int threads = (int64_t)reqs * 8 <= 2 * sms ? 512 : 256;
  int c = 8;
  while (c > 1 && ((int64_t)reqs * c * threads > (int64_t)1024 * sms ||
                   vocab <= c / 2 * threads * kStep))
    c >>= 1;
  const Params p{target,   target_req, target_row, draft, draft_req,  draft_row, tokens,
                 n_drafts, uniforms,   drafts,     vocab, out_tokens, kept,      status};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(reqs * c));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, threads == 512 ? draft_verify_kernel<512> : draft_verify_kernel<256>, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? VERIFY_OK : VERIFY_ERR_CUDA;
}
