// Sampling by temperature, top-k, top-p and min-p (rules in include/token_sample.h).
//
// A cluster of up to 8 CTAs takes a row. The logits are read from memory once and kept in shared
// memory (each thread rereads what it wrote, in 16-byte pieces); a row too long for that is read
// again for every pass, mostly from L2. The passes:
//   - the maximum;
//   - the thresholds of top-k and top-p, a logit and how many tokens that tie with it are kept.
//     Tokens are counted (their weights added up, in three digits) in bins of 1/32 of z, 16 of z at
//     a time, which most rows need once; every CTA finds the bin that holds the threshold, its
//     tokens (with top-k all before it too, where they fit) go to the first CTA, and that searches
//     their keys bit by bit from registers;
//   - the kept weights of every warp's range, from which the warp that holds the drawn point is
//     found, which goes through its range alone;
//   - the probabilities, from the weights of the pass before where the logits are fp32.
// Sums are 64-bit integers, so neither the split nor the order shows in the result.
//
// Bound by instructions, about 110 a logit with top-p, and by cluster barriers: 256 rows of 131072 fp32
// logits with probabilities 279 us (0.96 TB/s), 64 rows of 100003 in bf16 68 us; one row by its
// eight cluster barriers, 32 us. Where the bin of a threshold holds more than 2048 tokens (flat
// rows, one value in many places) all search it bit by bit: 64 rows of 131072 fp32 normal logits
// with top-p 119 us at T = 1, 603 at T = 5, 715 at T = 20, of two values 413. (A search bit by bit over all logits in place of the bins: 1436, 440 and 296 us;
// weights one by one in place of two to an operation, lists searched from shared memory: 435,
// 112, 61.) Few rows take CTAs of 512 threads, more of them 256, three to an SM.
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
constexpr int kBins = 512;   // of 16 in z: 1 / 32 of a power of two
constexpr int kAtOnce = 4;   // pieces
constexpr int kList = 4 * kBins;  // tokens that one CTA searches, in the place of the bins

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

// Two floats to an operation, rounded to nearest each; products and sums are not fused.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// a * b + c with two roundings: the sum as 1 * (a * b) + c, since ptxas fuses mul.rn.f32x2 and
// add.rn.f32x2 into one operation (3.2 of 8.4 million pairs of f then have other weights).
__device__ __forceinline__ uint64_t mul_add2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(mul2(a, b)), "l"(pack2(1.0f, 1.0f)), "l"(c));
  return d;
}

// The weights of two z in [0, 41], by the header's steps (41 gives 0). Neither floor nor weight
// is converted: z + 2^23 rounded down has floor(z) in its low bits, and P in [1/2, 1] has its 24
// bits in its significand: the weight is (significand << 17) >> (n + 1), or >> n where P is 1.
__device__ __forceinline__ void weights2(float z0, float z1, uint64_t& w0, uint64_t& w1) {
  const float t0 = __fadd_rd(z0, 0x1p23f), t1 = __fadd_rd(z1, 0x1p23f);
  const uint64_t n = add2(pack2(t0, t1), pack2(-0x1p23f, -0x1p23f));
  const float2 nf = unpack2(n);
  const uint64_t f = pack2(z0 - nf.x, z1 - nf.y);
  auto both = [](float c) { return pack2(c, c); };
  uint64_t y = both(0x1.c946d2p-14f);
  y = mul_add2(y, f, both(-0x1.4e2aeap-10f));
  y = mul_add2(y, f, both(0x1.39e3fcp-7f));
  y = mul_add2(y, f, both(-0x1.c6948ep-5f));
  y = mul_add2(y, f, both(0x1.ebfacp-3f));
  y = mul_add2(y, f, both(-0x1.62e42cp-1f));
  y = mul_add2(y, f, both(1.0f));
  const float2 p = unpack2(y);
  auto whole = [](float p, float t) {
    const uint32_t b = __float_as_uint(p);
    const int down = (int)(__float_as_uint(t) & 63) + 127 - (int)(b >> 23);
    return ((uint64_t)((b & 0x7FFFFFu) | 0x800000u) << 17) >> down;
  };
  w0 = whole(p.x, t0);
  w1 = whole(p.y, t1);
}
__device__ __forceinline__ uint64_t weight_of(float z) {
  uint64_t a, b;
  weights2(fminf(z, 41.0f), 41.0f, a, b);
  return a;
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
__global__ void __launch_bounds__(THREADS, 768 / THREADS) token_sample_kernel(const __grid_constant__ Params p) {
  constexpr int kWarps = THREADS / 32, kN = Piece<T>::kN;
  extern __shared__ __align__(16) uint8_t s_stage[];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int64_t row = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ uint64_t s_a[kWarps], s_b[kWarps];
  __shared__ uint64_t s_cta[2][2];  // read by the cluster, in turn
  __shared__ uint32_t s_bins[4][kBins];  // weights in digits of 13, 13 and 14 bits; tokens
  __shared__ uint32_t s_n;
  uint32_t* const s_list = &s_bins[0][0];
  __shared__ uint64_t s_found[5];
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
    const int64_t v0 = v - lane * kN;  // of the warp
    Piece<T> x;
    if (v0 >= 0 && v0 + 32 * kN <= p.vocab) {
      *reinterpret_cast<uint4*>(&x) = __ldg(reinterpret_cast<const uint4*>(logits + v));
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        x.x[i] = v + i >= 0 && v + i < p.vocab ? logits[v + i] : lowest<T>();
    }
    return x;
  };
  auto clean = [&](Piece<T>& x) {  // a NaN is -infinity
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kN; ++i) bad |= to_float(x.x[i]) != to_float(x.x[i]);
    if (bad) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (to_float(x.x[i]) != to_float(x.x[i])) x.x[i] = lowest<T>();
      err |= SAMPLE_STATUS_NAN;
    }
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

  if (tid == 0) s_n = 0;
  // ---- the maximum
  float top = -INFINITY;
  for (int s = 0; s < steps; s += kAtOnce) {  // their loads on their way together
    Piece<T> x[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) x[u] = read(s + u);
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      clean(x[u]);
      if (STAGED && s + u < steps) stage[(s + u) * 32] = x[u];
#pragma unroll
      for (int i = 0; i < kN; ++i) top = fmaxf(top, to_float(x[u].x[i]));
    }
  }
  auto piece = [&](int s) {
    if (STAGED) return stage[s * 32];
    Piece<T> x = read(s);
    clean(x);
    return x;
  };
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
  // z, 41 where it is more
  auto z_of = [&](float x) {
    return x == top ? 0.0f : fminf(__fmul_rn(__fsub_rn(top, x), scale), 41.0f);
  };
  const bool infinite = top == INFINITY;  // the only largest logit whose difference to itself is not 0
  const uint64_t top2 = pack2(top, top), scale2 = pack2(scale, scale);
  auto z2_of = [&](float a, float b, float& z0, float& z1) {
    const float2 z = unpack2(mul2(add2(top2, pack2(-a, -b)), scale2));
    z0 = infinite && a == top ? 0.0f : fminf(z.x, 41.0f);
    z1 = infinite && b == top ? 0.0f : fminf(z.y, 41.0f);
  };

  // ---- thresholds: kept are the tokens above `cut` and the first `ties` of those that have it
  uint32_t cut = 0;
  uint64_t ties = 0;
  auto logit_of = [](uint32_t key) { return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key); };
  auto each = [&](auto&& f) {  // f(logit, z, logit, z)
#pragma unroll 2
    for (int s = 0; s < steps; ++s) {
      const Piece<T> x = piece(s);
#pragma unroll
      for (int i = 0; i < kN; i += 2) {
        const float a = to_float(x.x[i]), b = to_float(x.x[i + 1]);
        float z0, z1;
        z2_of(a, b, z0, z1);
        f(a, z0, b, z1);
      }
    }
  };
  // Which bin of z, in the order of the tokens, brings the count (or weight) of the tokens up to
  // and with it to `target`, which all tokens together reach: rounds of 16 in z, most rows need
  // one. `before` becomes the count (weight) of the bins before it, `inside` its tokens.
  bool used = false;  // the bins: others may still be reading them
  // While the first round passes over the tokens it sums up all weights for a target that
  // depends on them (target(sum)).
  auto find_bin = [&](bool count, auto&& target_of_all, uint64_t& before, uint64_t& inside,
                      uint64_t& target) {
    before = 0;
    uint64_t all_weights = 0, some = 0;
    for (int round = 0;; ++round) {
      if (used) cluster.sync();
      used = true;
      for (int b = tid; b < kBins * 4; b += THREADS) s_bins[b / kBins][b % kBins] = 0;
      if (tid == 0) s_found[0] = ~uint64_t(0);
      __syncthreads();
      const float z0 = round * 16.0f;
      auto put = [&](float z, uint64_t w) {
        const int b = (int)((z - z0) * (kBins / 16));
        if (!count) {
          const uint32_t d0 = (uint32_t)w & 0x1FFFu, d1 = (uint32_t)(w >> 13) & 0x1FFFu;
          const uint32_t d2 = (uint32_t)(w >> 26);
          if (d0) atomicAdd(&s_bins[0][b], d0);
          if (d1) atomicAdd(&s_bins[1][b], d1);
          if (d2) atomicAdd(&s_bins[2][b], d2);
        }
        atomicAdd(&s_bins[3][b], 1u);
      };
      each([&](float, float za, float, float zb) {
        const bool ina = za >= z0 && za < z0 + 16.0f, inb = zb >= z0 && zb < z0 + 16.0f;
        if (count) {  // a weight of 0 is no token: z may pass 40 without one
          if (ina && (za < 40.0f || weight_of(za))) put(za, 0);
          if (inb && (zb < 40.0f || weight_of(zb))) put(zb, 0);
        } else if (round == 0 || ina || inb) {
          uint64_t wa, wb;
          weights2(za, zb, wa, wb);
          all_weights += wa + wb;
          if (ina && wa) put(za, wa);
          if (inb && wb) put(zb, wb);
        }
      });
      if (round == 0) {
        if (!count) reduce(all_weights, some);
        target = target_of_all(all_weights);
      }
      cluster.sync();
      // every CTA finds it for itself: thread t sums bins t * kEach ..
      constexpr int kEach = kBins / THREADS;
      uint64_t value[kEach], mine = 0;
      uint32_t tokens[kEach];
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int b = tid * kEach + e;
        uint64_t a[4] = {};
        for (int r = 0; r < ranks; ++r) {
          const uint32_t* h = cluster.map_shared_rank(&s_bins[0][0], r);
#pragma unroll
          for (int d = 0; d < 4; ++d)
            if (d == 3 || !count) a[d] += h[d * kBins + b];
        }
        tokens[e] = (uint32_t)a[3];
        value[e] = count ? a[3] : a[0] + (a[1] << 13) + (a[2] << 26);
        mine += value[e];
      }
      uint64_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s_a[warp] = incl;
      __syncthreads();
      uint64_t at = before + incl - mine, all = before;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at += s_a[w];
        all += s_a[w];
      }
      if (at < target && target <= at + mine) {
        int e = 0;
        while (at + value[e] < target) at += value[e++];
        s_found[0] = round * kBins + tid * kEach + e;
        s_found[1] = at;
        s_found[2] = tokens[e];
      }
      __syncthreads();
      const uint64_t found = s_found[0];
      if (found != ~uint64_t(0)) {
        before = s_found[1];
        inside = s_found[2];
        return (int)found;
      }
      if (round == 2) return -1;  // a count that all tokens do not reach
      before = all;
    }
  };
  // whether a token's z lies in bins [b0, b1], as find_bin counts them
  auto low_z = [](int b) { return b * (16.0f / kBins); };
  auto inside_of = [&](float z, float z0, float z1) {
    return z >= z0 && z < z1 && (z < 40.0f || weight_of(z) != 0);
  };
  // The largest key among the tokens of bins [b0, b1] with F(key) >= target, F(key) the count or the
  // weight of these tokens from it on; `above` becomes F(key + 1). They are gathered by the
  // first CTA where they fit its list; else all CTAs search them where they are. One list may be
  // searched twice: for a count k, then for a share of the weight of the first k.
  auto gather = [&](int b0, int b1) {
    cluster.sync();  // all have read the bins
    uint32_t* const n = cluster.map_shared_rank(&s_n, 0);
    uint32_t* const list = cluster.map_shared_rank(s_list, 0);
    const float z0 = low_z(b0), z1 = low_z(b1 + 1);
    auto put = [&](float y) {
      const uint32_t at = atomicAdd(n, 1u);
      if (at < kList) list[at] = key_of(y);
    };
    each([&](float a, float za, float b, float zb) {
      if (inside_of(za, z0, z1)) put(a);
      if (inside_of(zb, z0, z1)) put(b);
    });
    cluster.sync();
  };
  // ---- searches: bit by bit from the top, with `sum` to add up over the tokens
  // (bits of `low` and `high`, the least and the largest key, that are the same need no search)
  auto search = [&](auto&& sum, uint64_t target, uint64_t& above, uint32_t low = 0,
                    uint32_t high = 0xFFFFFFFFu) {
    const int bits = 32 - __clz(low ^ high);
    uint32_t key = bits == 32 ? 0 : high >> bits << bits;
    above = 0;
    for (uint32_t bit = bits ? 1u << (bits - 1) : 0u; bit; bit >>= 1) {
      const uint64_t a = sum(key | bit);
      if (a >= target) key |= bit;
      else above = a;
    }
    return key;
  };
  // Lists are searched from registers, kList / THREADS tokens and their weights to a thread (`at`: the
  // thread's place, `stride`: the threads).
  uint32_t lk[kList / THREADS];
  uint64_t lw[kList / THREADS];
  auto take_list = [&](int n, int at, int stride) {
#pragma unroll
    for (int e = 0; e < kList / THREADS; ++e) {
      const int i = e * stride + at;
      lk[e] = i < n ? s_list[i] : 0;
      lw[e] = i < n ? weight_of(z_of(logit_of(lk[e]))) : 0;
    }
  };
  auto in_list = [&](bool count) {  // by the first CTA alone
    return [&, count](uint32_t key) {
      uint64_t a = 0;
#pragma unroll
      for (int e = 0; e < kList / THREADS; ++e)
        if (lk[e] >= key) a += count ? 1 : lw[e];
      a = warp_sum(a);
      __syncthreads();
      if (lane == 0) s_a[warp] = a;
      __syncthreads();
      a = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) a += s_a[w];
      return a;
    };
  };
  // Short ones by every warp for itself: no barriers.
  constexpr int kShort = 32 * (kList / THREADS);
  auto in_warp = [&](bool count) {
    return [&, count](uint32_t key) {
      uint64_t a = 0;
#pragma unroll
      for (int e = 0; e < kList / THREADS; ++e)
        if (lk[e] >= key) a += count ? 1 : lw[e];
      return count ? (uint64_t)__reduce_add_sync(0xffffffffu, (uint32_t)a) : warp_sum(a);
    };
  };
  auto ends = [&](int n, uint32_t& low, uint32_t& high) {  // of the list
    low = 0xFFFFFFFFu;
    high = 0;
    for (int i = tid; i < n; i += THREADS) {
      low = min(low, s_list[i]);
      high = max(high, s_list[i]);
    }
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    __syncthreads();
    if (lane == 0) s_a[warp] = (uint64_t)low << 32 | high;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
      low = min(low, (uint32_t)(s_a[w] >> 32));
      high = max(high, (uint32_t)s_a[w]);
    }
  };
  auto everywhere = [&](bool count, int b0, int b1) {  // by all
    return [&, count, b0, b1](uint32_t key) {
      uint64_t a = 0, b = 0;
      const float z0 = low_z(b0), z1 = low_z(b1 + 1);
      auto add = [&](float y, float z) {
        if (key_of(y) >= key && inside_of(z, z0, z1)) a += count ? 1 : weight_of(z);
      };
      each([&](float x, float zx, float y, float zy) {
        add(x, zx);
        add(y, zy);
      });
      reduce(a, b);
      return a;
    };
  };
  auto share = [&] {  // what the first CTA found
    if (rank == 0 && tid == 0) {
      s_found[3] = cut;
      s_found[4] = ties;
    }
    cluster.sync();
    const uint64_t* f = cluster.map_shared_rank(s_found, 0);
    cut = (uint32_t)f[3];
    ties = f[4];
  };
  auto weight_at = [&](uint32_t key) { return weight_of(z_of(logit_of(key))); };
  auto target_of = [&](uint64_t total) {
    return top_p > 0.0f ? max(part_of(top_p, total, true), uint64_t(1)) : uint64_t(1);
  };
  if (greedy || none) {
    cut = key_of(top);
    ties = none ? 0 : 1;
  } else {
    const bool by_p = top_p < 1.0f;
    bool by_k = top_k > 0 && top_k < p.vocab;
    uint64_t total = 0;
    bool done = false;
    if (by_k) {
      uint64_t before = 0, inside = 0, k;
      const int b = find_bin(true, [&](uint64_t) { return (uint64_t)top_k; }, before, inside, k);
      by_k = b >= 0;
      if (by_k) {
      const bool all = before + inside <= kList;  // all that top-k can keep fit the list
      uint64_t above = 0;
      if (inside <= kList) {
        gather(all ? 0 : b, b);
        if (rank == 0) {
          const int n = (int)(all ? before + inside : inside);
          uint32_t low, high;
          ends(n, low, high);
          auto solve = [&](auto&& counts, auto&& weights) {
            cut = search(counts, all ? (uint64_t)top_k : top_k - before, above, low, high);
            ties = top_k - above - (all ? 0 : before);
            if (all && by_p) {
              uint64_t w = weight_at(cut);
              const uint64_t target = target_of(weights(cut + 1) + ties * w);
              cut = search(weights, target, above, low, high);
              w = weight_at(cut);
              ties = (target - above + w - 1) / w;
            }
          };
          if (n <= kShort) {
            take_list(n, lane, 32);
            solve(in_warp(true), in_warp(false));
          } else {
            take_list(n, tid, THREADS);
            solve(in_list(true), in_list(false));
          }
        }
        share();
        done = all;
      } else {
        cut = search(everywhere(true, b, b), top_k - before, above);
        ties = top_k - before - above;
      }
      if (!done && by_p) {  // the weight of the first k
        total = 0;
        auto add = [&](float y, float z) {
          if (key_of(y) > cut) total += weight_of(z);
        };
        each([&](float x, float zx, float y, float zy) {
          add(x, zx);
          add(y, zy);
        });
        uint64_t ignored = 0;
        reduce(total, ignored);
        total += ties * weight_at(cut);
      }
      }
    }
    if (by_p && !done) {
      uint64_t before = 0, inside = 0, above = 0, target;
      const int b = find_bin(
          false, [&](uint64_t all) { return target_of(by_k ? total : all); }, before, inside, target);
      if (inside <= kList) {
        if (tid == 0) s_n = 0;  // before all meet in the gathering
        gather(b, b);
        if (rank == 0) {
          uint32_t low, high;
          ends((int)inside, low, high);
          if (inside <= kShort) {
            take_list((int)inside, lane, 32);
            cut = search(in_warp(false), target - before, above, low, high);
          } else {
            take_list((int)inside, tid, THREADS);
            cut = search(in_list(false), target - before, above, low, high);
          }
          const uint64_t w = weight_at(cut);
          ties = (target - before - above + w - 1) / w;
        }
        share();
      } else {
        cut = search(everywhere(false, b, b), target - before, above);
        const uint64_t w = weight_at(cut);
        ties = (target - before - above + w - 1) / w;
      }
    }
  }
  const uint64_t tie_weight =
      greedy || none ? uint64_t(1) << 40
                     : weight_at(cut);
  if (tie_weight < least && !greedy) ties = 0;
  const float border = cut ? logit_of(cut) : -INFINITY;
  // the weights of the tokens of a piece that are above the cut; 0 of others
  auto strict = [&](const Piece<T>& x, uint64_t (&w)[kN]) {
#pragma unroll
    for (int i = 0; i < kN; i += 2) {
      const float a = to_float(x.x[i]), b = to_float(x.x[i + 1]);
      w[i] = w[i + 1] = 0;
      if (a > border || b > border) {
        float z0, z1;
        z2_of(a, b, z0, z1);
        weights2(z0, z1, w[i], w[i + 1]);
        if (!(a > border) || w[i] < least) w[i] = 0;
        if (!(b > border) || w[i + 1] < least) w[i + 1] = 0;
      }
    }
  };
  // fp32 logits that are kept in shared memory give way to their weights (an fp32 number holds one
  // exactly; kTie stands for a tie) in the pass that needs them first
  constexpr bool kInPlace = STAGED && sizeof(T) == 4;
  constexpr float kTie = -1.0f;
  bool replaced = false;
  auto ties_of = [&](const Piece<T>& x) {
    int n = 0;
    if (kInPlace && replaced) {
#pragma unroll
      for (int i = 0; i < kN; ++i) n += to_float(x.x[i]) == kTie;
      return n;
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) n += to_float(x.x[i]) == border;
    return border > -INFINITY ? n : 0;
  };
  // the weights of a piece that are kept, the ties in the order of the tokens behind `seen` of them
  auto kept = [&](const Piece<T>& x, uint64_t& seen, uint64_t (&w)[kN]) {
    if (kInPlace) {
#pragma unroll
      for (int i = 0; i < kN; ++i) w[i] = to_float(x.x[i]) > 0.0f ? (uint64_t)to_float(x.x[i]) : 0;
    } else {
      strict(x, w);
    }
    const int mine = ties_of(x);
    if (!__any_sync(0xffffffffu, mine)) return;
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += y;
    }
    uint64_t rank_of = seen + scan - mine;
    seen += __shfl_sync(0xffffffffu, scan, 31);
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (to_float(x.x[i]) == (kInPlace ? kTie : border)) w[i] = rank_of++ < ties ? tie_weight : 0;
  };

  // ---- kept weights of this warp's range: those above the cut, and how many have it
  uint64_t sum = 0, tied = 0;
  for (int s = 0; s < steps; ++s) {
    const Piece<T> x = piece(s);
    uint64_t w[kN];
    strict(x, w);
#pragma unroll
    for (int i = 0; i < kN; ++i) sum += w[i];
    tied += ties_of(x);
    if constexpr (kInPlace) {
      Piece<T> y;
#pragma unroll
      for (int i = 0; i < kN; ++i)
        y.x[i] = border > -INFINITY && x.x[i] == border ? kTie : (float)w[i];
      stage[s * 32] = y;
    }
  }
  replaced = kInPlace;
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
        kept(x, seen, w);
#pragma unroll
        for (int i = 0; i < kN; ++i) lane_sum += w[i];
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
      float prob[kN];
      bool tie = !kInPlace;
      if constexpr (kInPlace) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          prob[i] = x.x[i] * 0x1p-40f * f;
          tie |= x.x[i] == kTie;
        }
      }
      if (__any_sync(0xffffffffu, tie)) {
        uint64_t w[kN];
        kept(x, seen, w);
#pragma unroll
        for (int i = 0; i < kN; ++i) prob[i] = (float)w[i] * 0x1p-40f * f;
      }
      if (v >= 0 && v + kN <= p.vocab && (reinterpret_cast<uintptr_t>(out + v) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < kN; i += 4)
          __stcs(reinterpret_cast<float4*>(out + v + i),
                 make_float4(prob[i], prob[i + 1], prob[i + 2], prob[i + 3]));
      } else {
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (v + i >= 0 && v + i < p.vocab) out[v + i] = prob[i];
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

template <typename T, int kThreads>
int run(Params& p, int rows, int dev, cudaStream_t s) {
  constexpr int kPass = kThreads * Piece<T>::kN;  // logits of a step of a CTA
  int ranks = kMaxCluster;
  while (ranks > 1 && p.vocab <= ranks / 2 * kPass) ranks >>= 1;
  // a row that starts off a 16-byte boundary covers up to kN - 1 places more
  const bool off = !aligned(p.logits, 16) || (rows > 1 && p.ld % Piece<T>::kN);
  const int64_t places = (int64_t)p.vocab + (off ? Piece<T>::kN - 1 : 0);
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
  if (rows < 0 || rows > (1 << 27) || vocab < 1 || vocab > (1 << 20) || ld < vocab ||
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
  // CTAs of 512 threads while each has an SM, so that few rows take less time each
  const bool few = (int64_t)rows * kMaxCluster <= sms;
  const cudaStream_t s = (cudaStream_t)stream;
  if (dtype == SAMPLE_FP32)
    return few ? run<float, 512>(p, rows, dev, s) : run<float, 256>(p, rows, dev, s);
  if (dtype == SAMPLE_FP16)
    return few ? run<__half, 512>(p, rows, dev, s) : run<__half, 256>(p, rows, dev, s);
  return few ? run<__nv_bfloat16, 512>(p, rows, dev, s) : run<__nv_bfloat16, 256>(p, rows, dev, s);
}
