// Sampling by temperature, top-k, top-p and min-p (rules in include/token_sample.h).
//
// A cluster of CTAs takes a row. The logits are read from memory once and kept in shared memory
// (each thread rereads what it wrote, in 16-byte pieces); a row too long for that is read again
// for every pass, mostly from L2. The passes: the maximum; the threshold of top-k and of top-p,
// a logit and how many tokens that tie with it are kept; the kept weights of every warp's
// range, from which the warp that holds the drawn point is found, which scans its range alone.
// Sums are 64-bit integers, so neither the split nor the order shows in the result.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>

#include "token_sample.h"

namespace cg = cooperative_groups;

namespace {

constexpr int kMaxCluster = 8;

struct Params {
  const void* logits;
  int64_t ld;
  int vocab;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int param_rows;
  const float* uniforms;
  int32_t* tokens;
  float* probs;
  int64_t probs_ld;
  int32_t* status;
  int steps;  // of a warp
};

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T lowest();
template <>
__device__ __forceinline__ float lowest() { return -INFINITY; }
template <>
__device__ __forceinline__ __half lowest() { return __ushort_as_half(0xFC00); }
template <>
__device__ __forceinline__ __nv_bfloat16 lowest() { return __ushort_as_bfloat16(0xFF80); }

// 16 bytes of logits.
template <typename T>
struct __align__(16) Piece {
  static constexpr int kN = 16 / sizeof(T);
  T x[kN];
};

// Rises with the logit; the two zeros are one value.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// P(f) * 2^24 and n of a z < 41: the weight is (P << 16) >> n. The header's steps, none fused.
__device__ __forceinline__ uint64_t weight_of(float z) {
  if (!(z < 41.0f)) return 0;
  const float n = floorf(z), f = z - n;
  float y = 0x1.c946d2p-14f;
  y = __fadd_rn(__fmul_rn(y, f), -0x1.4e2aeap-10f);
  y = __fadd_rn(__fmul_rn(y, f), 0x1.39e3fcp-7f);
  y = __fadd_rn(__fmul_rn(y, f), -0x1.c6948ep-5f);
  y = __fadd_rn(__fmul_rn(y, f), 0x1.ebfacp-3f);
  y = __fadd_rn(__fmul_rn(y, f), -0x1.62e42cp-1f);
  y = __fadd_rn(__fmul_rn(y, f), 1.0f);
  return ((uint64_t)(uint32_t)(y * 0x1p24f) << 16) >> (int)n;
}

// floor (or ceil) of r * total, r in [0, 1): the significand times total, 88 bits, moved down.
__device__ __forceinline__ uint64_t part_of(float r, uint64_t total, bool up) {
  const uint32_t b = __float_as_uint(r), e = b >> 23;
  const uint64_t m = (b & 0x7FFFFFu) | (e ? 0x800000u : 0u);  // r = m * 2^-down
  const int down = 150 - (int)max(e, 1u);                     // 24 .. 149
  const uint64_t low = m * total, high = __umul64hi(m, total);
  uint64_t whole;
  bool rest;
  if (down >= 88) {
    whole = 0;
    rest = (low | high) != 0;
  } else if (down >= 64) {
    whole = high >> (down - 64);
    rest = low != 0 || (high & ((uint64_t(1) << (down - 64)) - 1)) != 0;
  } else {
    whole = (high << (64 - down)) | (low >> down);
    rest = (low & ((uint64_t(1) << down) - 1)) != 0;
  }
  return whole + (up && rest ? 1 : 0);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename T, int THREADS, bool STAGED>
__global__ void __launch_bounds__(THREADS) token_sample_kernel(const __grid_constant__ Params p) {
  constexpr int kWarps = THREADS / 32, kN = Piece<T>::kN;
  extern __shared__ __align__(16) uint8_t s_stage[];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int64_t row = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ uint64_t s_a[kWarps], s_b[kWarps];
  __shared__ uint64_t s_cta[2][2];  // read by the cluster, in turn
  int turn = 0, err = 0;

  // ---- the row's settings
  const int64_t of = row / p.param_rows;
  float temp = p.temperature ? __ldg(p.temperature + of) : 1.0f;
  int top_k = p.top_k ? __ldg(p.top_k + of) : 0;
  float top_p = p.top_p ? __ldg(p.top_p + of) : 1.0f;
  float min_p = p.min_p ? __ldg(p.min_p + of) : 0.0f;
  if (!(temp >= 0.0f && temp <= FLT_MAX)) {
    temp = 1.0f;
    err |= SAMPLE_STATUS_PARAM;
  }
  if (top_p != top_p) {
    top_p = 1.0f;
    err |= SAMPLE_STATUS_PARAM;
  }
  if (!(min_p <= 1.0f)) {
    min_p = 0.0f;
    err |= SAMPLE_STATUS_PARAM;
  }
  const float scale = fminf(__fdiv_rn(0x1.715476p0f, temp), FLT_MAX);
  const uint64_t least = min_p > 0.0f ? (uint64_t)ceil((double)min_p * 0x1p40) : 0;

  // ---- pieces: step s of this warp's range, lane by lane. Piece boundaries are those of
  // memory, so a row that starts off a boundary has a first piece that begins before it.
  const T* logits = reinterpret_cast<const T*>(p.logits) + row * p.ld;
  const int ahead = (int)((reinterpret_cast<uintptr_t>(logits) & 15) / sizeof(T));
  const int64_t first = ((int64_t)rank * kWarps + warp) * p.steps * (32 * kN) + lane * kN - ahead;
  Piece<T>* const stage = reinterpret_cast<Piece<T>*>(s_stage) + (int64_t)warp * p.steps * 32 + lane;
  auto read = [&](int s) {
    const int64_t v = first + (int64_t)s * (32 * kN);
    Piece<T> x;
    if (v >= 0 && v + kN <= p.vocab) {
      *reinterpret_cast<uint4*>(&x) = __ldg(reinterpret_cast<const uint4*>(logits + v));
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        x.x[i] = v + i >= 0 && v + i < p.vocab ? logits[v + i] : lowest<T>();
    }
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (to_float(x.x[i]) != to_float(x.x[i])) {
        x.x[i] = lowest<T>();
        err |= SAMPLE_STATUS_NAN;
      }
    return x;
  };
  const int steps = (int)min((int64_t)p.steps,
                             max((int64_t)0, ((int64_t)p.vocab - first + lane * kN + 32 * kN - 1) / (32 * kN)));

  // ---- the sums of a and b over the cluster
  auto reduce = [&](uint64_t& a, uint64_t& b) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (lane == 0) {
      s_a[warp] = a;
      s_b[warp] = b;
    }
    __syncthreads();
    if (warp == 0) {
      a = warp_sum(lane < kWarps ? s_a[lane] : 0);
      b = warp_sum(lane < kWarps ? s_b[lane] : 0);
      if (lane == 0) {
        s_cta[turn][0] = a;
        s_cta[turn][1] = b;
      }
    }
    cluster.sync();
    a = b = 0;
    if (lane < ranks) {
      const uint64_t* c = cluster.map_shared_rank(s_cta[turn], lane);
      a = c[0];
      b = c[1];
    }
    a = warp_sum(a);
    b = warp_sum(b);
    turn ^= 1;
  };

  // ---- the maximum
  float top = -INFINITY;
  for (int s = 0; s < steps; ++s) {
    const Piece<T> x = read(s);
    if (STAGED) stage[s * 32] = x;
#pragma unroll
    for (int i = 0; i < kN; ++i) top = fmaxf(top, to_float(x.x[i]));
  }
  auto piece = [&](int s) { return STAGED ? stage[s * 32] : read(s); };
  {
    const uint32_t k = __reduce_max_sync(0xffffffffu, key_of(top));
    if (lane == 0) s_a[warp] = k;
    __syncthreads();
    if (warp == 0) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, lane < kWarps ? (uint32_t)s_a[lane] : 0u);
      if (lane == 0) s_cta[turn][0] = m;
    }
    cluster.sync();
    const uint32_t m = __reduce_max_sync(
        0xffffffffu, lane < ranks ? (uint32_t)*cluster.map_shared_rank(s_cta[turn], lane) : 0u);
    turn ^= 1;
    top = __uint_as_float(m & 0x80000000u ? m & 0x7FFFFFFFu : ~m);
  }
  const bool none = top == -INFINITY;
  if (none) err |= SAMPLE_STATUS_EMPTY;
  const bool greedy = temp == 0.0f;
  auto z_of = [&](float x) { return x == top ? 0.0f : __fmul_rn(__fsub_rn(top, x), scale); };

  // ---- thresholds: kept are the tokens above `cut` and the first `ties` of those that have it
  uint32_t cut = 0;
  uint64_t ties = 0;
  // the largest key with F(key) >= target, F(key) the count or the weight of the tokens from
  // it on; `above` becomes F(key + 1)
  auto search = [&](bool count, uint64_t target, uint64_t& above) {
    uint32_t key = 0;
    above = 0;
    for (uint32_t bit = 0x80000000u; bit; bit >>= 1) {
      uint64_t a = 0, b = 0;
      for (int s = 0; s < steps; ++s) {
        const Piece<T> x = piece(s);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const float y = to_float(x.x[i]);
          if (key_of(y) >= (key | bit)) {
            const uint64_t w = weight_of(z_of(y));
            a += count ? (w != 0) : w;
          }
        }
      }
      reduce(a, b);
      if (a >= target) key |= bit;
      else above = a;
    }
    return key;
  };
  if (greedy || none) {
    cut = key_of(top);
    ties = none ? 0 : 1;
  } else {
    // the weights of all tokens, and how many weigh something: only these can be kept
    uint64_t total = 0, some = 0;
    const bool by_p = top_p < 1.0f;
    if (by_p || top_k > 0) {
      for (int s = 0; s < steps; ++s) {
        const Piece<T> x = piece(s);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const uint64_t w = weight_of(z_of(to_float(x.x[i])));
          total += w;
          some += w != 0;
        }
      }
      reduce(total, some);
    }
    if (top_k > 0 && top_k < some) {
      uint64_t above;
      cut = search(true, top_k, above);
      ties = top_k - above;
      if (by_p) {
        total = 0;
        for (int s = 0; s < steps; ++s) {
          const Piece<T> x = piece(s);
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const float y = to_float(x.x[i]);
            if (key_of(y) > cut) total += weight_of(z_of(y));
          }
        }
        uint64_t ignored = 0;
        reduce(total, ignored);
        total += ties * weight_of(z_of(__uint_as_float(cut & 0x80000000u ? cut & 0x7FFFFFFFu : ~cut)));
      }
    }
    if (by_p) {
      const uint64_t target = top_p > 0.0f ? max(part_of(top_p, total, true), uint64_t(1)) : 1;
      uint64_t above;
      cut = search(false, target, above);
      const uint64_t w = weight_of(z_of(__uint_as_float(cut & 0x80000000u ? cut & 0x7FFFFFFFu : ~cut)));
      ties = (target - above + w - 1) / w;
    }
  }
  const uint64_t tie_weight =
      greedy || none ? uint64_t(1) << 40
                     : weight_of(z_of(__uint_as_float(cut & 0x80000000u ? cut & 0x7FFFFFFFu : ~cut)));
  if (tie_weight < least && !greedy) ties = 0;
  // the weight of a token above the cut
  auto strict = [&](float y) {
    const uint64_t w = key_of(y) > cut ? weight_of(z_of(y)) : 0;
    return w >= least ? w : 0;
  };

  // ---- kept weights of this warp's range: those above the cut, and how many have it
  uint64_t sum = 0, tied = 0;
  for (int s = 0; s < steps; ++s) {
    const Piece<T> x = piece(s);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float y = to_float(x.x[i]);
      sum += strict(y);
      tied += key_of(y) == cut && y > -INFINITY;
    }
  }
  sum = warp_sum(sum);
  tied = warp_sum(tied);
  __syncthreads();
  if (lane == 0) {
    s_a[warp] = sum;
    s_b[warp] = tied;
  }
  __syncthreads();
  if (warp == 0) {
    const uint64_t a = warp_sum(lane < kWarps ? s_a[lane] : 0), b = warp_sum(lane < kWarps ? s_b[lane] : 0);
    if (lane == 0) {
      s_cta[turn][0] = a;
      s_cta[turn][1] = b;
    }
  }
  cluster.sync();
  uint64_t before = 0, ties_before = 0, total = 0, ties_total = 0;
  for (int r = 0; r < ranks; ++r) {
    const uint64_t* c = cluster.map_shared_rank(s_cta[turn], r);
    const uint64_t a = c[0], b = c[1];
    if (r < rank) {
      before += a;
      ties_before += b;
    }
    total += a;
    ties_total += b;
  }
  for (int w = 0; w < warp; ++w) {
    before += s_a[w];
    ties_before += s_b[w];
  }
  before += min(ties_before, ties) * tie_weight;
  total += min(ties_total, ties) * tie_weight;
  const uint64_t mine = sum + (min(ties_before + tied, ties) - min(ties_before, ties)) * tie_weight;

  // ---- the token
  if (p.tokens) {
    float u = __ldg(p.uniforms + row);
    if (!(u >= 0.0f && u < 1.0f)) {
      u = u >= 1.0f ? 0x1.fffffep-1f : 0.0f;
      err |= SAMPLE_STATUS_UNIFORM;
    }
    const uint64_t at = part_of(u, total, false);
    if (total && at >= before && at - before < mine) {
      uint64_t run = before, seen = ties_before;
      for (int s = 0; s < steps; ++s) {
        const Piece<T> x = piece(s);
        uint64_t w[kN], lane_sum = 0;
        int lane_ties = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i) lane_ties += key_of(to_float(x.x[i])) == cut;
        int scan = lane_ties;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, scan, o);
          if (lane >= o) scan += y;
        }
        uint64_t rank_of = seen + scan - lane_ties;
        seen += __shfl_sync(0xffffffffu, scan, 31);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const float y = to_float(x.x[i]);
          if (key_of(y) == cut) w[i] = rank_of++ < ties ? tie_weight : 0;
          else w[i] = strict(y);
          lane_sum += w[i];
        }
        uint64_t incl = lane_sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, run + incl > at);
        if (past) {
          if (lane == __ffs(past) - 1) {
            uint64_t here = run + incl - lane_sum;
            int i = 0;
            while (here + w[i] <= at) here += w[i++];
            p.tokens[row] = (int32_t)(first + (int64_t)s * (32 * kN) + i);
          }
          break;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (none && rank == 0 && tid == 0) p.tokens[row] = -1;
  }

  // ---- the probabilities
  if (p.probs) {
    float* out = p.probs + row * p.probs_ld;
    const double share = total ? 1.0 / (double)total : 0.0;
    const float f = (float)(share * 0x1p40);  // 2^-40 of a weight times it: no subnormal factor
    uint64_t seen = ties_before;
    for (int s = 0; s < steps; ++s) {
      const Piece<T> x = piece(s);
      const int64_t v = first + (int64_t)s * (32 * kN);
      int lane_ties = 0;
#pragma unroll
      for (int i = 0; i < kN; ++i) lane_ties += key_of(to_float(x.x[i])) == cut;
      int scan = lane_ties;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += y;
      }
      uint64_t rank_of = seen + scan - lane_ties;
      seen += __shfl_sync(0xffffffffu, scan, 31);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float y = to_float(x.x[i]);
        uint64_t w;
        if (key_of(y) == cut) w = rank_of++ < ties ? tie_weight : 0;
        else w = strict(y);
        if (v + i >= 0 && v + i < p.vocab) out[v + i] = (float)w * 0x1p-40f * f;
      }
    }
  }
  if (err && p.status) atomicOr(p.status, err);
  cluster.sync();  // no CTA leaves while another still reads its sums
}

bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) % a) == 0; }

constexpr int kMaxDevices = 64;

int current_device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev < kMaxDevices ? dev : -1;
}

// SMs of a device, or < 0; asked for once.
int sm_count(int dev) {
  static std::atomic<int> known[kMaxDevices];
  if (dev < 0) return -1;
  int sms = known[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
    known[dev].store(sms, std::memory_order_relaxed);
  }
  return sms;
}

constexpr int kMaxStage = 200 * 1024;  // bytes of a CTA's logits

template <typename T, int THREADS, bool STAGED>
int launch(const Params& p, int rows, int ranks, int stage, int dev, cudaStream_t s) {
  const auto kernel = token_sample_kernel<T, THREADS, STAGED>;
  if (STAGED) {
    static std::atomic<uint64_t> ready;
    if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxStage) !=
          cudaSuccess)
        return SAMPLE_ERR_CUDA;
      ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * ranks);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = STAGED ? stage : 0;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? SAMPLE_OK : SAMPLE_ERR_CUDA;
}

template <typename T>
int run(Params& p, int rows, int dev, int sms, cudaStream_t s) {
  constexpr int kThreads = 256;
  constexpr int kPass = kThreads * Piece<T>::kN;  // logits of a step of a CTA
  int ranks = kMaxCluster;
  while (ranks > 1 && p.vocab <= ranks / 2 * kPass) ranks >>= 1;
  // a row that starts off a 16-byte boundary covers up to kN - 1 places more
  const int64_t places = (int64_t)p.vocab + Piece<T>::kN - 1;
  p.steps = (int)((places + (int64_t)ranks * kPass - 1) / ((int64_t)ranks * kPass));
  const int64_t stage = (int64_t)p.steps * kThreads * 16;
  if (stage <= kMaxStage) return launch<T, kThreads, true>(p, rows, ranks, (int)stage, dev, s);
  return launch<T, kThreads, false>(p, rows, ranks, 0, dev, s);
}

}  // namespace

extern "C" int token_sample(const void* logits, int64_t ld, int dtype, int rows, int vocab,
                            const float* temperature, const int32_t* top_k, const float* top_p,
                            const float* min_p, int param_rows, const float* uniforms,
                            int32_t* tokens, float* probs, int64_t probs_ld, int32_t* status,
                            sample_stream_t stream) {
  if (rows < 0 || rows > (1 << 27) || vocab < 1 || vocab > (1 << 22) || ld < vocab ||
      param_rows < 1 || (dtype != SAMPLE_BF16 && dtype != SAMPLE_FP16 && dtype != SAMPLE_FP32) ||
      (probs && probs_ld < vocab))
    return SAMPLE_ERR_SHAPE;
  if (rows == 0) return SAMPLE_OK;
  if (!logits || (tokens && !uniforms) || (!tokens && !probs)) return SAMPLE_ERR_NULL;
  if (!aligned(logits, dtype == SAMPLE_FP32 ? 4 : 2) || !aligned(temperature, 4) ||
      !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(uniforms, 4) ||
      !aligned(tokens, 4) || !aligned(probs, 4) || !aligned(status, 4))
    return SAMPLE_ERR_ALIGN;
  const int dev = current_device(), sms = sm_count(dev);
  if (sms < 0) return SAMPLE_ERR_CUDA;
  Params p{logits,   ld,     vocab, temperature, top_k,  top_p, min_p, param_rows,
           uniforms, tokens, probs, probs_ld,    status, 0};
  if (dtype == SAMPLE_FP32) return run<float>(p, rows, dev, sms, (cudaStream_t)stream);
  if (dtype == SAMPLE_FP16) return run<__half>(p, rows, dev, sms, (cudaStream_t)stream);
  return run<__nv_bfloat16>(p, rows, dev, sms, (cudaStream_t)stream);
}
