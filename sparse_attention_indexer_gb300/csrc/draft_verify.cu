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

// A probability in [0, 1] as a whole number of 2^-60, in three signed digits of 20 bits: adding
// 1.5 * 2^k rounds to the sum's last place (2^-20, 2^-40, 2^-60) and leaves the digit in its
// bits, and the differences are exact. Ten operations, seven of them on the wide fp32 pipe: 64
// requests of 100003 tokens take 26 us; with conversions to 64-bit integers, or shifts, 39 us.
struct Digits {
  int a, b, c;
};

__device__ __forceinline__ Digits digits(float x) {
  constexpr float k1 = 0x1.8p3f, k2 = 0x1.8p-17f, k3 = 0x1.8p-37f;
  const float t1 = x + k1;
  const float r1 = x - (t1 - k1);
  const float t2 = r1 + k2;
  const float t3 = (r1 - (t2 - k2)) + k3;
  return {__float_as_int(t1) - __float_as_int(k1), __float_as_int(t2) - __float_as_int(k2),
          __float_as_int(t3) - __float_as_int(k3)};
}

__device__ __forceinline__ uint64_t value(const Digits& d) {
  return ((uint64_t)(int64_t)d.a << 40) + ((uint64_t)(int64_t)d.b << 20) + (uint64_t)(int64_t)d.c;
}

// floor(r * total) for r in [0, 1): the significand times total, 88 bits, moved down by the exponent.
__device__ __forceinline__ uint64_t drawn_point(float r, uint64_t total) {
  const uint32_t b = __float_as_uint(r), e = b >> 23;
  const uint64_t m = (b & 0x7FFFFFu) | (e ? 0x800000u : 0u);  // r = m * 2^-down
  const int down = 150 - (int)max(e, 1u);                     // 24 .. 149
  const uint64_t low = m * total, high = __umul64hi(m, total);
  if (down >= 88) return 0;
  return down >= 64 ? high >> (down - 64) : (high << (64 - down)) | (low >> down);
}

enum Row { kBonus, kRefused, kRefusedPoint };

// The weights of tokens v0 + 32 i + lane, i < kStep, in digits; 0 past `end`. Loads past it
// read the row's last token instead, so that none waits for a condition.
__device__ __forceinline__ void step_weights(const float* p, const float* q, Row row, int point,
                                             int v0, int end, Digits (&w)[kStep], int* err) {
  const int v = v0 + (threadIdx.x & 31);
  const bool whole = v0 + 32 * kStep <= end;
  float a[kStep], b[kStep];
  bool bad = false;  // above 1, negative or NaN (or -0)
#pragma unroll
  for (int i = 0; i < kStep; ++i) a[i] = __ldg(p + (whole ? v + i * 32 : min(v + i * 32, end - 1)));
  if (row == kRefused) {
#pragma unroll
    for (int i = 0; i < kStep; ++i)
      b[i] = __ldg(q + (whole ? v + i * 32 : min(v + i * 32, end - 1)));
#pragma unroll
    for (int i = 0; i < kStep; ++i) bad |= __float_as_uint(b[i]) > 0x3F800000u;
  } else {
#pragma unroll
    for (int i = 0; i < kStep; ++i) b[i] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kStep; ++i) bad |= __float_as_uint(a[i]) > 0x3F800000u;
  if (bad) {
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      a[i] = checked_prob(a[i], err);
      b[i] = checked_prob(b[i], err);
    }
  }
  if (!whole || (row == kRefusedPoint && point >= v0 && point < v0 + 32 * kStep)) {
#pragma unroll
    for (int i = 0; i < kStep; ++i)
      if (v + i * 32 >= end || (row == kRefusedPoint && v + i * 32 == point)) a[i] = 0.0f;
  }
  if (row == kRefused) {
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      // max(p - q, 0): the rounding keeps the order, so p <= q gives 0
      const bool more = a[i] > b[i];
      const Digits x = digits(more ? a[i] : 0.0f), y = digits(more ? b[i] : 0.0f);
      w[i] = {x.a - y.a, x.b - y.b, x.c - y.c};
    }
  } else {
#pragma unroll
    for (int i = 0; i < kStep; ++i) w[i] = digits(a[i]);
  }
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// More CTAs than 1024 threads to an SM would not run at once.
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

  // A row that sums to 16 or more wraps the sums: the upper halves tell
  uint64_t total = 0, before = 0, high = 0;
  for (int round = 0; round < 2; ++round) {
    uint64_t sum = 0, record = 0, upper = 0;
    int v0 = begin;
    for (int i = 0; v0 < end; ++i, v0 += kTokens) {
      Digits w[kStep], d = {0, 0, 0};
      step_weights(prow, qrow, row, point, v0, end, w, &err);
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        d.a += w[k].a;
        d.b += w[k].b;
        d.c += w[k].c;
      }
      uint64_t x = value(d);
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
  const uint64_t at = drawn_point(r, total);
  // 15 or more: a sum below 16 is in `total` as it is; of one above, the upper halves of at most
  // 2^27 partial sums, each less than one too low, leave more than 15 * 2^28
  const bool lost = high >= uint64_t(15) << 28 || total >= uint64_t(15) << 60;
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
      Digits w[kStep];
      step_weights(prow, qrow, row, point, v0, end, w, &ignored);
      int token = -1;
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        uint64_t x = value(w[k]);
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
  // a step to sum. Few requests take CTAs of 512 threads, so that one request has 4096; more of
  // them take CTAs of 256, eight to a request still, which spread more evenly over the SMs.
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
