// Verification of drafted tokens (rules in include/draft_verify.h).
//
// A request reads two probabilities per draft for the tests and then one row (the bonus
// row) or two (target and draft of the refused position) of the vocabulary: bound by HBM for
// a batch, by latency for one request. A cluster of C CTAs takes a request; every CTA decides
// the tests for itself (a few loads), each sums its slice of the weights, the slices' sums
// meet through distributed shared memory, and the CTA, then the warp, whose range holds the
// drawn point reads its part again (from L2) to find the token. Sums are 64-bit integers, so the split
// of the row does not show in the result.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "draft_verify.h"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

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
  if (!(x >= 0.0f && x <= 1.0f)) {
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

// A probability in units of 2^-60. x * 2^60 is exact, the conversion drops what is below.
__device__ __forceinline__ uint64_t units(float x) { return __float2ull_rz(x * 0x1p60f); }

// max(p - q, 0) in those units; a non-negative q >= p gives 0.
__device__ __forceinline__ uint64_t weight(float p, float q) {
  const uint64_t a = units(p), b = units(q);
  return a > b ? a - b : 0;
}

enum Row { kBonus, kRefused, kRefusedPoint };

__device__ __forceinline__ uint64_t weight_at(const float* p, const float* q, Row row, int point,
                                              int v, int* err) {
  const float a = checked_prob(__ldg(p + v), err);
  if (row == kRefused) return weight(a, checked_prob(__ldg(q + v), err));
  if (row == kRefusedPoint && v == point) return 0;
  return units(a);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__global__ void __launch_bounds__(kThreads) draft_verify_kernel(Params p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int req = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int s_kept;
  __shared__ uint64_t s_sum[kWarps];
  __shared__ uint64_t s_cta;  // read by the cluster
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

  // slices: CTA, then warp, each a whole number of 32s
  const int per_warp = ((p.vocab + ranks * kWarps - 1) / (ranks * kWarps) + 31) & ~31;
  const int64_t begin64 = ((int64_t)rank * kWarps + warp) * per_warp;
  const int begin = (int)min(begin64, (int64_t)p.vocab);
  const int end = (int)min(begin64 + per_warp, (int64_t)p.vocab);

  uint64_t total = 0, before = 0;
  for (int round = 0; round < 2; ++round) {
    uint64_t sum = 0;
#pragma unroll 8
    for (int v = begin + lane; v < end; v += 32) sum += weight_at(prow, qrow, row, point, v, &err);
    sum = warp_sum(sum);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (tid == 0) {
      uint64_t c = 0;
      for (int w = 0; w < kWarps; ++w) c += s_sum[w];
      s_cta = c;
    }
    cluster.sync();
    total = before = 0;
    for (int r = 0; r < ranks; ++r) {
      const uint64_t c = *cluster.map_shared_rank(&s_cta, r);
      if (r < rank) before += c;
      total += c;
    }
    if (total || row == kBonus) break;
    row = kBonus;  // nothing is left of p - q: draw from p itself
    cluster.sync();
  }

  const float r = checked_uniform(__ldg(uni + p.drafts), &err);
  const uint64_t at = __umul64hi(total, __float2ull_rz(r * 0x1p64f));  // floor(r * total)
  if (total > (uint64_t(1) << 63)) err |= VERIFY_STATUS_PROB;
  for (int w = 0; w < warp; ++w) before += s_sum[w];
  const uint64_t mine = s_sum[warp];
  // the warp whose range holds the point: before <= at < before + mine
  if (total && at >= before && at - before < mine) {
    uint64_t run = before;
    int ignored = 0;
    for (int v0 = begin; v0 < end; v0 += 32) {
      const int v = v0 + lane;
      uint64_t x = v < end ? weight_at(prow, qrow, row, point, v, &ignored) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, run + x > at);
      if (past) {
        if (lane == 0) out[kept] = v0 + __ffs(past) - 1;
        break;
      }
      run += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  if (rank == 0) {
    if (tid <= p.drafts && tid != kept) out[tid] = tid < kept ? __ldg(tok + tid) : -1;
    if (tid == 0) {
      p.kept[req] = kept;
      if (total == 0) {
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
  // CTAs per request: up to 8 while the batch leaves SMs idle and a CTA keeps 4096 tokens
  int c = 8;
  while (c > 1 && ((int64_t)reqs * c > 2 * sms || vocab / c < 4096)) c >>= 1;
  const Params p{target,   target_req, target_row, draft, draft_req,  draft_row, tokens,
                 n_drafts, uniforms,   drafts,     vocab, out_tokens, kept,      status};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(reqs * c));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, draft_verify_kernel, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? VERIFY_OK : VERIFY_ERR_CUDA;
}
