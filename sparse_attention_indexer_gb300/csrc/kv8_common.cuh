// What the kernels of the attention over the 8-bit cache share: arguments, the even split of
// the tiles over the CTAs, the parts of shared units and the launch that joins them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "kv8_attention.h"

namespace kv8 {

constexpr int kMaxCtas = 2048;
constexpr float kNone = -3e38f;  // maximum of a row that has no key yet: finite, so that no difference
                                 // of two of them is NaN

// A unit whose parts CTAs first .. last have; last < 0: none, or one CTA has it whole. Kept by
// unit where there are at most kMaxCtas units, else by the unit's first CTA.
struct __align__(16) Shared {
  int32_t g, h, first, last;
};

struct Params {
  const uint16_t* q;
  int64_t q_ld;
  int q_heads, kv_heads;
  float scale;  // sm_scale * log2(e)
  int rows;
  const int32_t* lens;
  int max_len;
  int group_rows;
  const int32_t* group_table;
  const int32_t* block_table;
  int n_tables;
  int64_t table_ld;
  int page_size;
  int page_shift;  // log2 where a power of two, else -1
  const int32_t* slots;  // the selected form: slots[row * slots_ld + i], i < max_len
  int64_t slots_ld;
  int block;
  int block_shift;
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  int64_t num_slots;
  uint16_t* out;
  int64_t out_ld;
  float* lse;
  int32_t* status;
  int halves;      // parts that a unit's rows come in (64 each where more than one)
  Shared* shared;  // workspace: the shared unit that starts in each CTA
  float* parts;    // workspace: two partial results per CTA
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16 / 4 bytes to shared memory, zeros where !in (the source is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

__device__ __forceinline__ uint4 ldmatrix_trans(uint32_t a) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

// Four e4m3 codes as fp16, exactly: lo the two lower, hi the two upper.
__device__ __forceinline__ void widen4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of fp16 (lane 4 r + c: row r, columns 2 c, 2 c + 1) transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 0xFF in each byte that is a NaN code.
__device__ __forceinline__ uint32_t nan_codes(uint32_t c) {
  return __vcmpeq4(c & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}

// ------------------------------------------------------------------ lengths
// Keys that group g attends to at most: the largest length of its rows that pass the checks;
// len_of(row) is 0 for one that does not. `err` collects what is wrong.
__device__ __forceinline__ int row_len(const Params& p, int row, int table, int* err) {
  const int len = __ldg(p.lens + row);
  if (len < 0 || len > p.max_len) {
    *err |= KV8_STATUS_LEN;
    return 0;
  }
  if (table < 0 || table >= p.n_tables) {
    *err |= KV8_STATUS_TABLE_ROW;
    return 0;
  }
  if ((int64_t)len > p.table_ld * p.page_size) {
    *err |= KV8_STATUS_TABLE_WIDTH;
    return 0;
  }
  return len;
}

__device__ __forceinline__ int group_len(const Params& p, int g, int* err) {
  const int table = p.group_table ? __ldg(p.group_table + g) : g;
  int len = 0;
  const int64_t r0 = (int64_t)g * p.group_rows;
  for (int i = 0; i < p.group_rows && r0 + i < p.rows; ++i)
    len = max(len, row_len(p, (int)(r0 + i), table, err));
  return len;
}

// A unit has at least one tile, so that rows without keys are written too.
template <int KEYS>
__device__ __forceinline__ int tiles_of(int len) {
  return max(1, (int)(((uint32_t)len + KEYS - 1) / KEYS));
}

// A CTA's tiles [w0, w1) of the `all` that n CTAs share, and the unit of the first: group g, sub s
// (a key head, or a part of its rows), the group's length and the unit's first tile.
struct Range {
  int64_t all, n, w0, w1, first;
  int g, s, len;
};

// Every thread of the CTA calls this; the first 128 look at the lengths. Each group has `subs`
// units. A CTA gets at least `least` tiles, but a unit is not split where there are CTAs enough
// for one each. CTA 0 adds what is wrong with the rows to *err.
template <int KEYS>
__device__ __forceinline__ Range locate(const Params& p, int groups, int subs, int least, int* err) {
  __shared__ int64_t s_sum[4], s_first;
  __shared__ int s_group;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Range r = {};
  const int per = (groups + 127) / 128;
  const int64_t g0 = tid < 128 ? min((int64_t)groups, (int64_t)tid * per) : groups;
  const int64_t g1 = min((int64_t)groups, g0 + per);
  int64_t mine = 0;
  int bad = 0;
  for (int64_t i = g0; i < g1; ++i) mine += tiles_of<KEYS>(group_len(p, (int)i, &bad));
  if (blockIdx.x == 0) *err |= bad;
  int64_t before = mine, total = 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  if (warp < 4 && lane == 31) s_sum[warp] = before;
  __syncthreads();
  before -= mine;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t x = s_sum[i];
    if (i < warp) before += x;
    total += x;
  }
  r.all = total * subs;
  r.n = min((int64_t)gridDim.x, max((int64_t)groups * subs, (r.all + least - 1) / least));
  const int64_t me = blockIdx.x;
  r.w0 = me * r.all / r.n;
  r.w1 = me < r.n ? (me + 1) * r.all / r.n : r.w0;
  if (tid < 128 && r.w0 < r.w1 && r.w0 >= before * subs && r.w0 < (before + mine) * subs) {
    int ignored = 0;
    int64_t i = g0, at = before * subs;
    for (;; ++i) {
      const int64_t here = (int64_t)tiles_of<KEYS>(group_len(p, (int)i, &ignored)) * subs;
      if (r.w0 < at + here) break;
      at += here;
    }
    s_group = (int)i;
    s_first = at;
  }
  __syncthreads();
  if (r.w0 < r.w1) {
    int ignored = 0;
    r.g = s_group;
    r.len = group_len(p, r.g, &ignored);
    const int tiles = tiles_of<KEYS>(r.len);
    r.s = (int)((r.w0 - s_first) / tiles);
    r.first = s_first + (int64_t)r.s * tiles;
  }
  return r;
}

// A part of a unit in the workspace: ROWS x DIM sums, then {m, m + d, sum} per row.
template <int DIM, int ROWS>
struct Part {
  static constexpr int kStat = ROWS * DIM;
  static constexpr int kFloats = ROWS * (DIM + 4);
};

// Channels [N * c, N * c + N) of row r of unit (g, h): v relative to 2^topv over l relative to
// 2^top, and with c == 0 the row's lse.
template <int DIM, bool FP16, int N>
__device__ __forceinline__ void write_row(const Params& p, int g, int h, int r, int c,
                                          const float* v, float top, float topv, float l) {
  const int ratio = p.q_heads / p.kv_heads;
  const int64_t row = (int64_t)g * p.group_rows + r / ratio;
  if (row >= p.rows) return;
  const int head = h * ratio + r % ratio;
  const bool none = l == 0.0f;  // no key: one that counts adds 1 to l, a NaN makes it NaN
  const float f = none ? 0.0f : exp2f(topv - top) / l;
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float x = none ? 0.0f : v[2 * i] * f, y = none ? 0.0f : v[2 * i + 1] * f;
    if (FP16) {
      w[i] = pack_half(x, y);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  uint16_t* dst = p.out + row * p.out_ld + (int64_t)head * DIM + c * N;
  if (N == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[N / 2 - 1]);
  else *reinterpret_cast<uint32_t*>(dst) = w[0];
  if (c == 0 && p.lse)
    p.lse[row * p.q_heads + head] = none ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
}

// Joins the parts of the shared units: CTA (i, y) the rows y, y + gridDim.y, .. of entry i. The
// warps take a row's parts in turn, each lane 16th .. of its channels, and meet in shared memory in
// the order of the warps.
constexpr int kJoinWarps = 8;

template <int DIM, bool FP16, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32)
kv8_join_kernel(const __grid_constant__ Params p) {
  using Q = Part<DIM, ROWS>;
  constexpr int kVec = DIM / 32;  // channels of a lane
  __shared__ float s_v[kJoinWarps][DIM];
  __shared__ float s_st[kJoinWarps][3];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Shared u = p.shared[blockIdx.x];
  if (u.last < 0) return;
  // the rows of this entry: all of them, or one half
  const int r0 = u.h % p.halves * ROWS;
  const int live = min(p.group_rows * (p.q_heads / p.kv_heads) - r0, ROWS);
  const int parts = u.last - u.first + 1;
  // the first CTA's part is its second one, the others' are their first
  auto part = [&](int c) {
    return p.parts + (2 * (int64_t)(u.first + c) + (c == 0)) * Q::kFloats;
  };
  for (int r = blockIdx.y; r < live; r += gridDim.y) {
    float top = -INFINITY, topv = -INFINITY, l = 0.0f, v[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = 0.0f;
    for (int c0 = warp; c0 < parts; c0 += 4 * kJoinWarps) {
      float4 st[4];
      float y[4][kVec];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + k * kJoinWarps;
        if (c < parts) {
          const float* q = part(c);
          st[k] = __ldcg(reinterpret_cast<const float4*>(q + Q::kStat + r * 4));
          const float* src = q + r * DIM + lane * kVec;
          if (kVec == 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
            y[k][0] = x.x;
            y[k][1] = x.y;
            y[k][kVec - 2] = x.z;
            y[k][kVec - 1] = x.w;
          } else {
            const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
            y[k][0] = x.x;
            y[k][1] = x.y;
          }
        } else {
          st[k] = make_float4(-INFINITY, -INFINITY, 0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < kVec; ++i) y[k][i] = 0.0f;
        }
      }
      float nt = top, nv = topv;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        nt = fmaxf(nt, st[k].x);
        nv = fmaxf(nv, st[k].y);
      }
      const float ut = nt == -INFINITY ? 0.0f : nt, uv = nv == -INFINITY ? 0.0f : nv;
      l *= exp2_fast(top - ut);
      const float keep = exp2_fast(topv - uv);
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] *= keep;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        l += st[k].z * exp2_fast(st[k].x - ut);
        const float f = exp2_fast(st[k].y - uv);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] += y[k][i] * f;
      }
      top = nt;
      topv = nv;
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) s_v[warp][lane * kVec + i] = v[i];
    if (lane == 0) {
      s_st[warp][0] = top;
      s_st[warp][1] = topv;
      s_st[warp][2] = l;
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int w = 1; w < kJoinWarps; ++w) {
        top = fmaxf(top, s_st[w][0]);
        topv = fmaxf(topv, s_st[w][1]);
      }
      const float ut = top == -INFINITY ? 0.0f : top, uv = topv == -INFINITY ? 0.0f : topv;
      l = 0.0f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) {
        l += s_st[w][2] * exp2_fast(s_st[w][0] - ut);
        const float f = exp2_fast(s_st[w][1] - uv);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] += s_v[w][lane * kVec + i] * f;
      }
      write_row<DIM, FP16, kVec>(p, u.g, u.h / p.halves, r0 + r, lane, v, top, topv, l);
    }
    __syncthreads();
  }
}

// Launches the join behind the launch whose parts it reads: `units` of them, or by CTA.
template <int DIM, bool FP16, int ROWS>
int launch_join(const Params& p, int64_t units, int grid, cudaStream_t s) {
  const int live = p.group_rows * (p.q_heads / p.kv_heads);
  const int entries = units > kMaxCtas ? grid : (int)units;
  const int rows = 4096 / entries < 1 ? 1 : 4096 / entries;
  const int most = live < ROWS ? live : ROWS;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)entries, (unsigned)(most < rows ? most : rows));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_join_kernel<DIM, FP16, ROWS>, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KV8_OK : KV8_ERR_CUDA;
}

constexpr int kMaxDevices = 64;

// The current device, or < 0.
inline int current_device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev < kMaxDevices ? dev : -1;
}

// SMs of a device, or < 0; asked for once.
inline int sm_count(int dev) {
  static std::atomic<int> known[kMaxDevices];
  if (dev < 0) return -1;
  int sms = known[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
    known[dev].store(sms, std::memory_order_relaxed);
  }
  return sms;
}

// Kernels on the 5th-generation tensor cores for more than 32 rows to a unit of 128 channels
// (kv8_wide.cu).
int launch_wide(Params& p, bool fp16, int dev, cudaStream_t s);

}  // namespace kv8
