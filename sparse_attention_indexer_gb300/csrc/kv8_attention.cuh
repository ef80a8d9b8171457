// Attention over the 8-bit paged KV cache (formulas and rules in include/kv8_attention.h): the
// kernels and their launch, for kv8_attention.cu and kv8_shared.cu.
//
// Bound by HBM: a decode step reads 2 * dim bytes per key and head and does 4 * dim * M
// operations on them, M = query rows of the group * query heads per key head (1 .. 128).
//
// Work split. A unit is a (group of query rows, key head): its M query rows attend to the
// same keys. The units' tiles of 32 keys are laid end to end, and CTA i of N takes the tiles
// [i * W / N, (i + 1) * W / N) of the W there are, whatever the lengths: the loads are even
// for one long row and for a ragged batch alike, with no plan from the host. A unit that
// several CTAs share leaves its parts in the workspace, and a second, small launch joins them
// in the order of the CTAs. (The last CTA to arrive joining its unit alone took 250 of 334 us
// for 56 rows to a unit of 80K keys: 38 parts of 28 KB through one SM.)
//
// A tile. The W warps of a CTA (four, or one) form groups that take a segment's tiles in turn, WM
// warps to a group, each with NT * 8 of the M rows. A group keeps kStages tiles of codes and scales
// in flight with cp.async (a key that is masked or missing is filled with zeros and its
// score set to -inf, so what lies there never enters). Products run on mma.sync m16n8k16
// fp16 with fp32 accumulators, keys and channels on its 16 rows and query rows on its 8
// columns: the 8 query heads of a key head fill it, where query rows on the 16 would leave
// half of the products, the weights and the registers of the sums idle (52 against 40 us for
// one row of 64 heads over 80000 keys on 8 key heads, 4.1 TB/s; 32 ragged rows of 857K keys in
// all 429 against 387 us, 5.7 TB/s). Up to 16 rows three CTAs of two stages fit an SM, which
// beats two of three stages by 6 %; from there on the products and the weights bound the kernel
// (56 rows: 98 us, 40 % of the tensor pipe).
//   - q . k: an fp16 times an e4m3 (widened, exact) product is exact. Rows of bf16 q are
//     brought to [2^14, 2^15) by a power of two, which fp16 then holds exactly but for
//     channels 2^-38 below the row's largest. The channels may be summed in any order, so
//     lane t of a quad takes 16 contiguous bytes of a key, one shared-memory load for four
//     mma steps, and the query fragments are laid out to match.
//   - p . v: ldmatrix.trans hands each lane pairs of channels of two keys; one byte
//     permutation sorts them into the fragments of the even and the odd channels, which
//     are rows g and g + 8 of a product of 16 channels. The weights turn from keys x rows
//     into rows x keys by movmatrix.
//   - the value scale of a block is folded into its weights before these are rounded to
//     fp16: w' = 2^(x - m) * sv * 2^-d, m the row's maximum, which is raised only when an x
//     passes it by 4 (in most tiles none does, and no lane asks another). While the scales
//     met so far lie within 2^8 of each other, one d for all rows keeps the row's largest w'
//     in [1, 2^13), and fp16 holds what is 2^-24 of it; else (a scale of 0 counts as the
//     least) d is chosen per row so that the largest w' is about 1. Where a tile has one key
//     and one value scale, they come out of the sums. fp16 is what the products take in one
//     pass: the rounding, 2^-11 of a weight at most, has no direction. It leaves bf16 outputs
//     as far from the exact ones as fp32 weights do (relative error 1.7e-3), fp16 outputs of
//     32 ragged rows at 3.1e-4 in place of 2.1e-4. Maxima, sums and joins are fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "kv8_attention.h"

namespace {

constexpr int kKeys = 32;   // keys of a tile
constexpr float kNone = -3e38f;  // maximum of a row that has no key yet: finite, so that no difference
                                 // of two of them is NaN
constexpr float kSlack = 4.0f;   // log2 by which a row may pass its maximum before that is raised
constexpr int kMaxCtas = 2048;

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
  // the form that leaves a shared prefix out: positions of each group that it starts behind, and
  // what each row has of them (kv8_shared.cu)
  const int32_t* start;
  const float* before;
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

// ------------------------------------------------------------------ layout in shared memory
template <int DIM, int NT, int WM, int W>
struct Smem {
  static constexpr int kGroups = W / WM;
  static constexpr int kRows = 8 * NT * WM;
  // tiles in flight per warp group, CTAs per SM
  static constexpr int kStages = WM == 4 ? 6 : NT <= 2 ? 2 : 3;
  static constexpr int kCtas = W == 1 ? (DIM == 64 ? 12 : NT == 1 ? 11 : 10) : NT <= 2 ? 3 : 2;
  static constexpr int kTile = kKeys * DIM;        // bytes of the K (or V) codes of a tile
  static constexpr int kRing = kGroups * kStages * 2 * kTile;
  static constexpr int kLd = DIM + 4;  // floats between the rows of the warps' sums
  static constexpr int kJoin = kGroups * kRows * kLd * 4;  // these sums, over the ring
  static constexpr int kQ = kRing > kJoin ? kRing : kJoin;
  static constexpr int kScale = kQ + kRows * DIM * 2;
  static constexpr int kMask = kScale + kGroups * kStages * 2 * kKeys * 4;
  static constexpr int kStat = kMask + ((kGroups * kStages * 4 + 15) & ~15);  // m, m + d, sum
  static constexpr int kMul = kStat + kGroups * kRows * 3 * 4;
  static constexpr int kLen = kMul + kRows * 4;
  static constexpr int kTotal = kLen + kRows * 4;
};

// A row of codes is DIM / 16 pieces of 16 bytes, permuted so that both the reads of q . k (4
// pieces of each of 8 keys) and those of p . v (one piece of 8 keys) meet every bank once.
template <int DIM>
__device__ __forceinline__ int piece_at(int key, int piece) {
  if (DIM == 128) return key * 128 + ((piece ^ (key & 7)) << 4);
  return (key >> 1) * 128 + ((((key & 1) * 4 + piece) ^ ((key >> 1) & 3)) << 4);
}

// ------------------------------------------------------------------ lengths
// The length of a row, 0 where it does not pass the checks; `err` collects what is wrong.
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

// What of a length of group g lies behind the shared prefix.
template <bool TAIL>
__device__ __forceinline__ int behind(const Params& p, int g, int len) {
  return TAIL ? max(0, len - __ldg(p.start + g)) : len;
}

// Keys that group g attends to at most (behind the shared prefix): its rows' largest length.
template <bool TAIL>
__device__ __forceinline__ int group_len(const Params& p, int g, int* err) {
  const int table = p.group_table ? __ldg(p.group_table + g) : g;
  int len = 0;
  const int64_t r0 = (int64_t)g * p.group_rows;
  for (int i = 0; i < p.group_rows && r0 + i < p.rows; ++i)
    len = max(len, row_len(p, (int)(r0 + i), table, err));
  return behind<TAIL>(p, g, len);
}

// A unit has at least one tile, so that rows without keys are written too.
__device__ __forceinline__ int tiles_of(int len) {
  return max(1, (int)(((uint32_t)len + kKeys - 1) / kKeys));
}

// What a unit counts when the work is divided: its tiles, and behind a shared prefix, where most
// units are short, kUnitTiles for its start and end, which take as long (queries, the first
// loads, the join of its warps, the prefix's part). 64 requests of 64-4096 tokens of their own on 8
// key heads: 70 us with tiles alone, 48 with 3 more, 37 with 8, 33 with 16.
constexpr int kUnitTiles = 16;
template <bool TAIL>
__device__ __forceinline__ int span_of(int len) {
  return tiles_of(len) + (TAIL ? kUnitTiles : 0);
}

// 0xFF in each byte that is a NaN code.
__device__ __forceinline__ uint32_t nan_codes(uint32_t c) {
  return __vcmpeq4(c & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}

// The prefix's part of a row and head, in p.before: DIM sums, then {m, m + d, sum}. Adds it.
template <int DIM, int N>
__device__ __forceinline__ void add_prefix(const float* x, int c, float (&v)[N], float& top,
                                           float& topv, float& l) {
  const float pl = __ldg(x + DIM + 2);
  if (pl == 0.0f) return;
  const float pt = __ldg(x + DIM), pv = __ldg(x + DIM + 1);
  const float nt = fmaxf(top, pt), nv = fmaxf(topv, pv);
  l = l * exp2f(top - nt) + pl * exp2f(pt - nt);
  const float keep = exp2f(topv - nv), add = exp2f(pv - nv);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = v[i] * keep + __ldg(x + c * N + i) * add;
  top = nt;
  topv = nv;
}

// A part of a unit in the workspace: ROWS x DIM sums, then {m, m + d, sum} per row.
template <int DIM, int ROWS>
struct Part {
  static constexpr int kStat = ROWS * DIM;
  static constexpr int kFloats = ROWS * (DIM + 4);
};

// Channels [N * c, N * c + N) of row r of unit (g, h): v relative to 2^topv over l relative to
// 2^top, and with c == 0 the row's lse.
template <int DIM, bool FP16, bool TAIL, int N>
__device__ __forceinline__ void write_row(const Params& p, int g, int h, int r, int c,
                                          float (&v)[N], float top, float topv, float l) {
  const int ratio = p.q_heads / p.kv_heads;
  const int64_t row = (int64_t)g * p.group_rows + r / ratio;
  if (row >= p.rows) return;
  const int head = h * ratio + r % ratio;
  if (TAIL && __ldg(p.start + g) > 0)
    add_prefix<DIM, N>(p.before + (row * p.q_heads + head) * (DIM + 4), c, v, top, topv, l);
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

// ------------------------------------------------------------------ kernel
template <int DIM, bool FP16, bool SELECTED, bool TAIL, int NT, int WM, int W>
__global__ void __launch_bounds__(W * 32, Smem<DIM, NT, WM, W>::kCtas)
kv8_attention_kernel(const __grid_constant__ Params p) {
  using L = Smem<DIM, NT, WM, W>;
  constexpr int kWarps = W, kThreads = W * 32;
  constexpr int kGroups = L::kGroups, kRows = L::kRows, kStages = L::kStages;
  constexpr int kPieces = DIM / 16;   // 16-byte pieces of a row of codes
  constexpr int kSteps = DIM / 16;    // mma steps of q . k
  extern __shared__ __align__(128) uint8_t smem[];
  asm volatile("griddepcontrol.launch_dependents;");  // the join, which waits for this launch
  __shared__ int64_t s_sum[kWarps];
  __shared__ int64_t s_first;
  __shared__ int s_group;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kg = warp / WM, wm = warp % WM;
  const int quad = lane >> 2, t = lane & 3;
  const int ratio = p.q_heads / p.kv_heads;
  const int groups = SELECTED ? p.rows : (p.rows + p.group_rows - 1) / p.group_rows;
  const int live = (SELECTED ? 1 : p.group_rows) * ratio;  // rows of a unit, <= kRows
  int err = 0;

  // ---- this CTA's tiles [w0, w1) and the unit of the first
  int64_t all, first_tile = 0;  // tiles of the launch; first tile of the unit at hand
  int g = 0, h = 0, len = p.max_len;
  int64_t w0, w1;
  // CTAs that take part: each gets a tile for each of its warp groups, and a unit is not split
  // where there are CTAs enough for one each
  int64_t n = gridDim.x;
  const int64_t units = (int64_t)groups * p.kv_heads;
  const int64_t me = blockIdx.x;
  if (SELECTED) {
    const int64_t tiles = tiles_of(len);
    all = tiles * groups * p.kv_heads;
    n = min(n, max(units, (all + kGroups - 1) / kGroups));
    w0 = me * all / n;
    w1 = me < n ? (me + 1) * all / n : w0;
    const int64_t u = w0 / tiles;
    g = (int)(u / p.kv_heads);
    h = (int)(u % p.kv_heads);
    first_tile = u * tiles;
  } else {
    const int per = (groups + kThreads - 1) / kThreads;
    const int64_t g0 = min((int64_t)groups, (int64_t)tid * per);
    const int64_t g1 = min((int64_t)groups, g0 + per);
    int64_t mine = 0;
    if (p.group_rows == 1) {  // all loads of eight rows on their way at once
#pragma unroll 8
      for (int64_t i = g0; i < g1; ++i)
        mine += span_of<TAIL>(behind<TAIL>(
            p, (int)i,
            row_len(p, (int)i, p.group_table ? __ldg(p.group_table + i) : (int)i, &err)));
    } else {
#pragma unroll 2
      for (int64_t i = g0; i < g1; ++i) mine += span_of<TAIL>(group_len<TAIL>(p, (int)i, &err));
    }
    if (me) err = 0;  // CTA 0 reports for all
    int64_t before = mine, total = 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += x;
    }
    if (lane == 31) s_sum[warp] = before;
    __syncthreads();
    before -= mine;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int64_t x = s_sum[i];
      if (i < warp) before += x;
      total += x;
    }
    all = total * p.kv_heads;
    n = min(n, max(units, (all + kGroups - 1) / kGroups));
    w0 = me * all / n;
    w1 = me < n ? (me + 1) * all / n : w0;
    if (w0 < w1 && w0 >= before * p.kv_heads && w0 < (before + mine) * p.kv_heads) {
      int ignored = 0;
      int64_t i = g0, at = before * p.kv_heads;
      for (; i + 1 < g1; ++i) {
        const int64_t here = (int64_t)span_of<TAIL>(group_len<TAIL>(p, (int)i, &ignored)) * p.kv_heads;
        if (w0 < at + here) break;
        at += here;
      }
      s_group = (int)i;
      s_first = at;
    }
    __syncthreads();
    if (w0 < w1) {
      int ignored = 0;
      g = s_group;
      first_tile = s_first;
      len = group_len<TAIL>(p, g, &ignored);
      const int span = span_of<TAIL>(len);
      h = (int)((w0 - first_tile) / span);
      first_tile += (int64_t)h * span;
    }
  }

  const uint32_t ring = smem_u32(smem) + kg * kStages * 2 * L::kTile;
  const uint32_t scales = smem_u32(smem + L::kScale) + kg * kStages * 2 * kKeys * 4;
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem + L::kMask) + kg * kStages;
  float* s_stat = reinterpret_cast<float*>(smem + L::kStat);
  float* s_mul = reinterpret_cast<float*>(smem + L::kMul);
  int* s_len = reinterpret_cast<int*>(smem + L::kLen);

  Shared mine = {0, 0, 0, -1};
  int64_t w = w0;
  while (w < w1) {
    const int tiles = tiles_of(len), span = span_of<TAIL>(len);
    const int span1 = (int)min((int64_t)span, w1 - first_tile);
    const int tile0 = max(0, (int)(w - first_tile) - (span - tiles));
    const int tile1 = span1 - (span - tiles);
    if (TAIL && tile1 <= 0) break;  // the range ends in what stands for the unit's start
    const int table = SELECTED ? 0 : p.group_table ? __ldg(p.group_table + g) : g;
    const int start = TAIL ? __ldg(p.start + g) : 0;  // positions of the prefix

    // ---- keys of a tile: this lane's key is tile * 32 + lane
    auto slot_of = [&](int tile) -> int {
      const int64_t i = (int64_t)tile * kKeys + lane;
      if (tile >= tile1 || i >= len) return -1;
      int64_t slot;
      if (SELECTED) {
        slot = __ldg(p.slots + g * p.slots_ld + i);
        if (slot < 0) return -1;
      } else {
        const int pos = (int)i + start;
        const int pg = p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page_size;
        const int32_t page = __ldg(p.block_table + table * p.table_ld + pg);
        if (page < 0) {
          err |= KV8_STATUS_TABLE_ENTRY;
          return -1;
        }
        slot = (int64_t)page * p.page_size + (pos - pg * p.page_size);
      }
      if (slot >= p.num_slots) {
        err |= KV8_STATUS_SLOT;
        return -1;
      }
      return (int)slot;
    };
    auto issue = [&](int stage, int slot) {
      const uint32_t k_at = ring + stage * 2 * L::kTile, v_at = k_at + L::kTile;
      constexpr int kKeysPerPass = 32 / kPieces;
      constexpr int kPasses = kKeys / kKeysPerPass / WM;
      const int piece = lane % kPieces;
#pragma unroll
      for (int j = 0; j < kPasses; ++j) {
        const int key = (j * WM + wm) * kKeysPerPass + lane / kPieces;
        const int s = __shfl_sync(0xffffffffu, slot, key);
        const int64_t off = ((int64_t)max(s, 0) * p.kv_heads + h) * DIM + piece * 16;
        const int at = piece_at<DIM>(key, piece);
        copy16(k_at + at, p.k + off, s >= 0);
        copy16(v_at + at, p.v + off, s >= 0);
      }
      if (wm == 0) {
        const int sl = max(slot, 0);
        const int b = p.block_shift >= 0 ? sl >> p.block_shift : sl / p.block;
        const int64_t off = (int64_t)b * p.kv_heads + h;
        const uint32_t at = scales + (stage * 2 * kKeys + lane) * 4;
        copy4(at, p.k_scale + off, slot >= 0);
        copy4(at + kKeys * 4, p.v_scale + off, slot >= 0);
        const uint32_t in = __ballot_sync(0xffffffffu, slot >= 0);
        if (lane == 0) masks[stage] = in;
      }
    };

    // ---- first tiles on their way
    int next = tile0 + kg;  // the tile that is issued next
    int slot = slot_of(next);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      issue(i, slot);
      copy_commit();
      next += kGroups;
      slot = slot_of(next);
    }

    // ---- queries: row r of the unit is row r / ratio of the group, head r % ratio of h's
    for (int x = tid; x < kRows * kPieces; x += kThreads) {
      const int r = x / kPieces, c = x % kPieces;  // 16 channels from 16 c
      const int64_t row = (int64_t)g * (SELECTED ? 1 : p.group_rows) + r / ratio;
      const bool in = r < live && row < p.rows;
      uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (in) {
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + row * p.q_ld + (int64_t)(h * ratio + r % ratio) * DIM + c * 16);
        v[0] = __ldg(src);
        v[1] = __ldg(src + 1);
      }
      uint32_t wds[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
      float mul = p.scale;
      if (!FP16) {
        uint32_t top = 0;  // largest magnitude bits of the row
#pragma unroll
        for (int i = 0; i < 8; ++i)
          top = max(top, max(wds[i] & 0x7FFFu, (wds[i] >> 16) & 0x7FFFu));
#pragma unroll
        for (int o = kPieces / 2; o; o >>= 1)
          top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // 2^up brings the row's largest magnitude into [2^14, 2^15)
        const int e = (int)(top >> 7);  // biased exponent
        const int up = e == 255 || top == 0 ? 0 : min(126, 14 - (e - 127));
        const float f = __uint_as_float((uint32_t)(up + 127) << 23);
        mul *= __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          wds[i] = pack_half(__uint_as_float(wds[i] << 16) * f,
                             __uint_as_float(wds[i] & 0xFFFF0000u) * f);
      }
      // fragments of two steps: lane (r % 8) * 4 + t holds channels 16 t + 4 s .. of 64
      const int half = c >> 2, tt = c & 3;
      uint4* dst = reinterpret_cast<uint4*>(smem + L::kQ) +
                   ((r >> 3) * (kSteps / 2) + half * 2) * 32 + (r & 7) * 4 + tt;
      dst[0] = make_uint4(wds[0], wds[1], wds[2], wds[3]);
      dst[32] = make_uint4(wds[4], wds[5], wds[6], wds[7]);
      if (c == 0) {
        int ignored = 0;
        s_mul[r] = mul;
        // only rows that end before the unit's keys do need the comparison with their length
        s_len[r] = !in || SELECTED
                       ? INT32_MAX
                       : behind<TAIL>(p, g, row_len(p, (int)row, table, &ignored));
      }
    }
    __syncthreads();

    // this thread's query rows: row0 + i * 8 + 2 t + b
    const int row0 = wm * 8 * NT;
    int least = INT32_MAX;  // where the unit's first row ends
#pragma unroll
    for (int i = 0; i < (kRows + 31) / 32; ++i)
      if (i * 32 + lane < kRows) least = min(least, s_len[i * 32 + lane]);
    least = __reduce_min_sync(0xffffffffu, least);
    float mul[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b) mul[i][b] = s_mul[row0 + i * 8 + 2 * t + b];
    const uint32_t q_at = smem_u32(smem + L::kQ) + wm * NT * (kSteps / 2) * 512 + lane * 16;
    uint4 qf[NT <= 2 ? NT : 1][kSteps / 2];  // few enough to stay in registers
    if (NT <= 2) {
#pragma unroll
      for (int i = 0; i < (NT <= 2 ? NT : 1); ++i)
#pragma unroll
        for (int st = 0; st < kSteps / 2; ++st) qf[i][st] = lds128(q_at + (i * (kSteps / 2) + st) * 512);
    }
    float o[NT][kPieces][4];
    // m: a maximum of x, not more than kSlack below the running one; o is relative to
    // 2^(m + d), sum to 2^m
    float m[NT][2], d[NT][2], sum[NT][2];
    uint32_t sv_top = 0, sv_low = 255;  // largest and least exponent of the value scales so far
    float d_all = 0.0f;                 // d, while all rows have the same
    bool d_own = false;                 // they have not
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][j][c] = 0.0f;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        m[i][b] = kNone;
        d[i][b] = sum[i][b] = 0.0f;
      }
    }
    auto group_sync = [&] {
      if (WM == 1) __syncwarp();
      else asm volatile("bar.sync %0, %1;" ::"r"(1 + kg), "n"(32 * WM) : "memory");
    };

    int stage = 0;
    for (int tile = tile0 + kg; tile < tile1; tile += kGroups) {
      copy_wait<kStages - 2>();
      // the group's warps see this tile, and are done with the one that the next copy replaces
      group_sync();
      issue(stage == 0 ? kStages - 1 : stage - 1, slot);
      copy_commit();
      next += kGroups;
      slot = slot_of(next);

      const uint32_t k_at = ring + stage * 2 * L::kTile, v_at = k_at + L::kTile;
      // scores: s[i][j][2 c + b] is key 16 j + 8 c + quad, row 8 i + 2 t + b
      float s[NT][2][4];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[i][j][c] = 0.0f;
#pragma unroll
      for (int half = 0; half < DIM / 64; ++half) {
        uint32_t kr[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 x = lds128(k_at + piece_at<DIM>(j * 8 + quad, half * 4 + t));
          kr[j][0] = x.x;
          kr[j][1] = x.y;
          kr[j][2] = x.z;
          kr[j][3] = x.w;
        }
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) {
          uint4 q[NT];
#pragma unroll
          for (int i = 0; i < NT; ++i)
            q[i] = NT <= 2 ? qf[NT <= 2 ? i : 0][half * 2 + s2]
                           : lds128(q_at + (i * (kSteps / 2) + half * 2 + s2) * 512);
#pragma unroll
          for (int s1 = 0; s1 < 2; ++s1)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t a0, a1, a2, a3;
              widen4(kr[2 * j][s2 * 2 + s1], a0, a2);
              widen4(kr[2 * j + 1][s2 * 2 + s1], a1, a3);
#pragma unroll
              for (int i = 0; i < NT; ++i)
                mma(s[i][j], a0, a1, a2, a3, s1 ? q[i].z : q[i].x, s1 ? q[i].w : q[i].y);
            }
        }
      }

      // ---- scores to weights: x = acc * mul * key scale (log2 units)
      const uint32_t in = masks[stage];
      const float* sc = reinterpret_cast<const float*>(smem + L::kScale) +
                        (kg * kStages + stage) * 2 * kKeys;
      const float ks0 = sc[0], vs0 = sc[kKeys];
      bool same;  // one key scale and one value scale
      {
        // exponents of the scales of the values; a 0 counts as the least: where the heaviest key's
        // scale is 0, the row's largest weight * scale may lie any distance below the maximum
        const float v = sc[kKeys + lane];
        const bool some = (in >> lane) & 1;
        const uint32_t e = (__float_as_uint(v) & 0x7FFFFFFFu) >> 23;
        sv_top = max(sv_top, __reduce_max_sync(0xffffffffu, some ? e : 0u));
        sv_low = min(sv_low, __reduce_min_sync(0xffffffffu, some ? e : 255u));
        same = !SELECTED && __all_sync(0xffffffffu, sc[lane] == ks0 && v == vs0);
      }
      const bool near = sv_top <= sv_low + 8 || sv_low == 255;
      // some row of the unit ends inside this tile or before it
      const bool ragged = (int64_t)(tile + 1) * kKeys > least;
      const bool masked = ragged || in != 0xffffffffu;
      // the plain tile: the scales come out of the sums, and x is not needed to find its maximum
      const bool plain = same && !masked && near && vs0 > 0.0f && ks0 >= 0.0f && p.scale >= 0.0f;
      // d: 2^8 below the largest scale while all of them lie within 2^8, so that the row's
      // largest weight * scale is 2^d times a number in [1, 2^9) (2^kSlack more between two
      // updates); 2^d and its reciprocal stay in range
      const float d_near = sv_low == 255 ? 0.0f : (float)max((int)sv_top - 127 - 8, -120);
      float vs[2][2];
      float tm[NT][2];
      if (plain) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            tm[i][b] = fmaxf(fmaxf(s[i][0][b], s[i][0][2 + b]), fmaxf(s[i][1][b], s[i][1][2 + b])) *
                       (mul[i][b] * ks0);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float ks = sc[j * 16 + c * 8 + quad];
            vs[j][c] = sc[kKeys + j * 16 + c * 8 + quad];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int b = 0; b < 2; ++b) s[i][j][2 * c + b] *= mul[i][b] * ks;
          }
        if (masked) {
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const int end = s_len[row0 + i * 8 + 2 * t + b];
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const int at = j * 16 + c * 8 + quad;
                  if (!((in >> at) & 1) || (int64_t)tile * kKeys + at >= end)
                    s[i][j][2 * c + b] = -INFINITY;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int b = 0; b < 2; ++b)  // NaN is no maximum
            tm[i][b] = fmaxf(fmaxf(s[i][0][b], s[i][0][2 + b]), fmaxf(s[i][1][b], s[i][1][2 + b]));
      }
      bool update = !near || d_own || d_near != d_all;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b) update |= tm[i][b] > m[i][b] + kSlack;
      if (__any_sync(0xffffffffu, update)) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          float keep[2];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float top = tm[i][b], dn = d_near;
#pragma unroll
            for (int x = 4; x <= 16; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            top = fmaxf(top, m[i][b]);
            if (!near) {  // what makes the row's largest weight * scale 1
              float tv = -INFINITY;
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  tv = fmaxf(tv, s[i][j][2 * c + b] + log2_fast(vs[j][c]));
#pragma unroll
              for (int x = 4; x <= 16; x <<= 1) tv = fmaxf(tv, __shfl_xor_sync(0xffffffffu, tv, x));
              // 2^(m + d) is the largest so far (the first time a bound below it): d is no whole
              // number, as one would let m + d rise with every rise of m
              const float was = m[i][b] > kNone ? m[i][b] + d[i][b] : -INFINITY;
              dn = tv <= was && top == m[i][b] ? d[i][b] : fmaxf(tv, was) - top;
              dn = fminf(fmaxf(dn, -120.0f), 126.0f);
            }
            const float drop = exp2_fast(m[i][b] - top);
            sum[i][b] *= drop;
            keep[b] = dn == d[i][b] ? drop : exp2_fast((m[i][b] - top) + (d[i][b] - dn));
            m[i][b] = top;
            d[i][b] = dn;
          }
#pragma unroll
          for (int j = 0; j < kPieces; ++j) {
            o[i][j][0] *= keep[0];
            o[i][j][1] *= keep[1];
            o[i][j][2] *= keep[0];
            o[i][j][3] *= keep[1];
          }
        }
        d_all = d_near;
        d_own = !near;
      }
      uint32_t pb[NT][2][2];
      if (plain) {
        // w' = 2^(x - m + log2(vs 2^-d)) at once; the sum of the weights is that of the w' / (vs 2^-d)
        const float f = vs0 * exp2_fast(-d_all), lf = log2_fast(f), back = 1.0f / f;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float c0 = mul[i][0] * ks0, c1 = mul[i][1] * ks0;
          const float z0 = lf - m[i][0], z1 = lf - m[i][1];
          float add0 = 0.0f, add1 = 0.0f;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float w0 = exp2_fast(fmaf(s[i][j][2 * c], c0, z0));
              const float w1 = exp2_fast(fmaf(s[i][j][2 * c + 1], c1, z1));
              add0 += w0;
              add1 += w1;
              pb[i][j][c] = transpose8(pack_half(w0, w1));
            }
          sum[i][0] = fmaf(add0, back, sum[i][0]);
          sum[i][1] = fmaf(add1, back, sum[i][1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          float w2[2][2][2];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float f = exp2_fast(-d[i][b]);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float e = exp2_fast(s[i][j][2 * c + b] - m[i][b]);
                sum[i][b] += e;
                w2[j][c][b] = e * vs[j][c] * f;  // in this order: f may be large where e is 0
                // a key outside the row weighs 0, whatever the scale of its block is
                if (masked && s[i][j][2 * c + b] == -INFINITY) w2[j][c][b] = 0.0f;
              }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              pb[i][j][c] = transpose8(pack_half(w2[j][c][0], w2[j][c][1]));
        }
      }

      // ---- a NaN code must not reach the rows that end before it (0 * NaN is NaN in a
      // product). Only a tile in which a row ends can hold one that some rows see and others do
      // not: there the rows that see it become NaN here, and the code a zero.
      if (ragged) {
        uint32_t nan = 0;
#pragma unroll
        for (int j = 0; j < L::kTile / 512; ++j) {
          const uint4 c = lds128(v_at + (j * 32 + lane) * 16);
          nan |= nan_codes(c.x) | nan_codes(c.y) | nan_codes(c.z) | nan_codes(c.w);
        }
        if (__any_sync(0xffffffffu, nan != 0)) {
          for (int key = 0; key < kKeys; ++key) {
            const int64_t pos = (int64_t)tile * kKeys + key;
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {  // this thread's channels: 16 c + 2 quad ..
              uint16_t codes;
              asm volatile("ld.shared.u16 %0, [%1];"
                           : "=h"(codes)
                           : "r"(v_at + piece_at<DIM>(key, c) + 2 * quad));
              const uint32_t bad = nan_codes(codes);
#pragma unroll
              for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int b = 0; b < 2; ++b)
                  if (pos < s_len[row0 + i * 8 + 2 * t + b]) {
                    if (bad & 1) o[i][c][b] = NAN;
                    if (bad & 256) o[i][c][2 + b] = NAN;
                  }
            }
          }
          group_sync();
#pragma unroll 1
          for (int j = wm; j < L::kTile / 512; j += WM) {
            const uint32_t at = v_at + (j * 32 + lane) * 16;
            const uint4 c = lds128(at);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                         "r"(c.x & ~nan_codes(c.x)), "r"(c.y & ~nan_codes(c.y)),
                         "r"(c.z & ~nan_codes(c.z)), "r"(c.w & ~nan_codes(c.w))
                         : "memory");
          }
          group_sync();
        }
      }

      // ---- values times weights: o[i][c][2 e + b] is channel 16 c + 2 quad + e, row 8 i + 2 t + b
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const int key = kk * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
        for (int cp = 0; cp < kPieces / 2; ++cp) {
          const uint4 r = ldmatrix_trans(v_at + piece_at<DIM>(key, cp * 2 + (lane >> 4)));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // bytes: (key 2t, channels 2 quad, 2 quad + 1), (key 2t + 1, the same)
            uint32_t a0, a1, a2, a3;
            widen4(__byte_perm(e ? r.z : r.x, 0, 0x3120), a0, a1);
            widen4(__byte_perm(e ? r.w : r.y, 0, 0x3120), a2, a3);
#pragma unroll
            for (int i = 0; i < NT; ++i)
              mma(o[i][cp * 2 + e], a0, a1, a2, a3, pb[i][kk][0], pb[i][kk][1]);
          }
        }
      }
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    copy_wait<0>();
    __syncthreads();  // the ring is free: it takes the warps' sums

    // ---- join the warp groups
    float* s_sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        float x = sum[i][b];
#pragma unroll
        for (int y = 4; y <= 16; y <<= 1) x += __shfl_xor_sync(0xffffffffu, x, y);
        const int r = kg * kRows + row0 + i * 8 + 2 * t + b;
        if (quad == 0) {
          s_stat[r * 3] = m[i][b];
          s_stat[r * 3 + 1] = m[i][b] + d[i][b];
          s_stat[r * 3 + 2] = x;
        }
#pragma unroll
        for (int c = 0; c < kPieces; ++c)
          *reinterpret_cast<float2*>(s_sums + r * L::kLd + 16 * c + 2 * quad) =
              make_float2(o[i][c][b], o[i][c][2 + b]);
      }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == tiles;
    // the CTA that has the unit's first tile keeps its part in its second place (its first may
    // hold the end of the unit before); the others theirs in their first
    float* part = p.parts + (2 * me + (tile0 == 0)) * Part<DIM, kRows>::kFloats;
    for (int x = tid; x < live * (DIM / 4); x += kThreads) {
      const int r = x / (DIM / 4), c4 = x % (DIM / 4);
      float top = -INFINITY, topv = -INFINITY, l = 0.0f;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        top = fmaxf(top, s_stat[(k * kRows + r) * 3]);
        topv = fmaxf(topv, s_stat[(k * kRows + r) * 3 + 1]);
      }
      const float ut = top == -INFINITY ? 0.0f : top, uv = topv == -INFINITY ? 0.0f : topv;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        const float* st = s_stat + (k * kRows + r) * 3;
        l += st[2] * exp2_fast(st[0] - ut);
        const float f = exp2_fast(st[1] - uv);
        const float4 y =
            *reinterpret_cast<const float4*>(s_sums + (k * kRows + r) * L::kLd + c4 * 4);
        v[0] += y.x * f;
        v[1] += y.y * f;
        v[2] += y.z * f;
        v[3] += y.w * f;
      }
      if (whole) {
        write_row<DIM, FP16, TAIL, 4>(p, g, h, r, c4, v, top, topv, l);
      } else {
        reinterpret_cast<float4*>(part)[r * (DIM / 4) + c4] =
            make_float4(v[0], v[1], v[2], v[3]);
        if (c4 == 0) {
          float* st = part + Part<DIM, kRows>::kStat + r * 4;
          st[0] = top;
          st[1] = topv;
          st[2] = l;
        }
      }
    }
    if (tile0 == 0) {
      const Shared u = {g, h, (int32_t)me,
                        whole ? -1 : (int32_t)(((first_tile + span) * n - 1) / all)};
      if (units > kMaxCtas) mine = whole ? mine : u;
      else if (tid == 0) p.shared[(int64_t)g * p.kv_heads + h] = u;
    }
    __syncthreads();  // the shared arrays are free for the next unit

    // ---- next unit
    w = first_tile + span1;
    if (tile1 == tiles) {
      first_tile += span;
      if (++h == p.kv_heads) {
        h = 0;
        ++g;
        int ignored = 0;
        if (!SELECTED && w < w1) len = group_len<TAIL>(p, g, &ignored);
      }
    }
  }
  if (tid == 0 && units > kMaxCtas) p.shared[me] = mine;
  if (err && p.status) atomicOr(p.status, err);
}

// Joins the parts of the shared units: CTA (i, y) a share of the rows of entry i. A unit of few
// parts gives a row to a warp, which sums all of them; of many, the warps take a row's
// parts in turn and meet in shared memory, in the order of the warps.
constexpr int kJoinWarps = 8;

// Adds parts c0, c0 + step, .. (< parts) of row r to (top, topv, l, v); `part` gives their address.
template <int DIM, int ROWS, typename F>
__device__ __forceinline__ void add_parts(F&& part, int c0, int step, int parts, int r, float& top,
                                          float& topv, float& l, float (&v)[DIM / 32]) {
  constexpr int kVec = DIM / 32;  // channels of a lane
  const int lane = threadIdx.x & 31;
  for (; c0 < parts; c0 += 4 * step) {
    float4 st[4];
    float y[4][kVec];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c0 + k * step;
      if (c < parts) {
        const float* q = part(c);
        st[k] = __ldcg(reinterpret_cast<const float4*>(q + Part<DIM, ROWS>::kStat + r * 4));
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
    l *= exp2_fast(top - nt);  // the first part makes both finite
    const float keep = exp2_fast(topv - nv);
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] *= keep;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      l += st[k].z * exp2_fast(st[k].x - nt);
      const float f = exp2_fast(st[k].y - nv);
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] += y[k][i] * f;
    }
    top = nt;
    topv = nv;
  }
}

template <int DIM, bool FP16, bool TAIL, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32)
kv8_join_kernel(const __grid_constant__ Params p) {
  using Q = Part<DIM, ROWS>;
  constexpr int kVec = DIM / 32;
  __shared__ float s_v[kJoinWarps][DIM];
  __shared__ float s_st[kJoinWarps][3];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Shared u = p.shared[blockIdx.x];
  if (u.last < 0) return;
  const int live = p.group_rows * (p.q_heads / p.kv_heads);
  const int share = (live + gridDim.y - 1) / gridDim.y;
  const int r0 = blockIdx.y * share, r1 = min(live, r0 + share);
  const int parts = u.last - u.first + 1;
  // the first CTA's part is its second one, the others' are their first
  auto part = [&](int c) {
    return p.parts + (2 * (int64_t)(u.first + c) + (c == 0)) * Q::kFloats;
  };
  if (share > 1 && parts <= 2 * kJoinWarps) {
    for (int r = r0 + warp; r < r1; r += kJoinWarps) {
      float top = -INFINITY, topv = -INFINITY, l = 0.0f, v[kVec] = {};
      add_parts<DIM, ROWS>(part, 0, 1, parts, r, top, topv, l, v);
      write_row<DIM, FP16, TAIL, kVec>(p, u.g, u.h, r, lane, v, top, topv, l);
    }
    return;
  }
  for (int r = r0; r < r1; ++r) {
    float top = -INFINITY, topv = -INFINITY, l = 0.0f, v[kVec] = {};
    add_parts<DIM, ROWS>(part, warp, kJoinWarps, parts, r, top, topv, l, v);
#pragma unroll
    for (int i = 0; i < kVec; ++i) s_v[warp][lane * kVec + i] = v[i];
    if (lane == 0) {
      s_st[warp][0] = top;
      s_st[warp][1] = topv;
      s_st[warp][2] = l;
    }
    __syncthreads();
    if (warp == 0) {  // has a part, so its maxima are finite
#pragma unroll
      for (int w = 1; w < kJoinWarps; ++w) {
        top = fmaxf(top, s_st[w][0]);
        topv = fmaxf(topv, s_st[w][1]);
      }
      l = 0.0f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) {
        l += s_st[w][2] * exp2_fast(s_st[w][0] - top);
        const float f = exp2_fast(s_st[w][1] - topv);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] += s_v[w][lane * kVec + i] * f;
      }
      write_row<DIM, FP16, TAIL, kVec>(p, u.g, u.h, r, lane, v, top, topv, l);
    }
    __syncthreads();
  }
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

constexpr int kMaxDevices = 64;

// The current device, or < 0.
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

// Rows that the variant for a unit of `live` rows pads to.
int padded_rows(int live) {
  return live <= 8 ? 8 : live <= 16 ? 16 : live <= 32 ? 32 : live <= 64 ? 64 : 128;
}

int shift_of(int x) {
  if (x & (x - 1)) return -1;
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

template <int DIM, bool FP16, bool SELECTED, bool TAIL, int NT, int WM, int W>
int launch(const Params& p, int dev, cudaStream_t s) {
  using L = Smem<DIM, NT, WM, W>;
  constexpr int kThreads = W * 32;
  const auto kernel = kv8_attention_kernel<DIM, FP16, SELECTED, TAIL, NT, WM, W>;
  const auto join = kv8_join_kernel<DIM, FP16, TAIL, L::kRows>;
  // once on a device; both with the largest share of shared memory: a change of it between
  // them would cost time
  static std::atomic<uint64_t> ready;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal) !=
            cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100) !=
            cudaSuccess ||
        cudaFuncSetAttribute(join, cudaFuncAttributePreferredSharedMemoryCarveout, 100) !=
            cudaSuccess)
      return KV8_ERR_CUDA;
    ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  const int sms = sm_count(dev);
  // a tile for each warp group of a CTA, where there is that little work
  const int64_t groups = ((int64_t)p.rows + p.group_rows - 1) / p.group_rows;
  const int64_t units = groups * p.kv_heads;
  const int64_t tiles = p.max_len < kKeys ? 1 : ((int64_t)p.max_len + kKeys - 1) / kKeys;
  if (units > (int64_t(1) << 33)) return KV8_ERR_SHAPE;
  const int64_t want = units * ((tiles + L::kGroups - 1) / L::kGroups);
  const int64_t most = sms * L::kCtas < kMaxCtas ? sms * L::kCtas : kMaxCtas;
  const int grid = (int)(want < most ? want : most);
  kernel<<<(unsigned)grid, kThreads, L::kTotal, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return KV8_ERR_CUDA;
  // the join is launched while the first kernel runs and waits for its end
  const int live = p.group_rows * (p.q_heads / p.kv_heads);
  const int entries = units > kMaxCtas ? grid : (int)units;
  // a CTA per row where that launches few or a unit has many parts on average, else one for each
  // 8 rows: 448 rows of 8 parts 20.9 against 22.5 us (7 x 2048 slots), 2048 rows of 1-2
  // parts 79 against 75.6 us (64 x 2048 slots)
  const bool each = (int64_t)entries * live <= 1024 || grid / entries > 2 * kJoinWarps;
  const int rows = each ? live : (live + kJoinWarps - 1) / kJoinWarps;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)entries, (unsigned)rows);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, join, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KV8_OK : KV8_ERR_CUDA;
}

// Up to 16 rows to a unit: four warps to a CTA, or, where there is a unit for every warp of the
// device, one. Then a warp passes from unit to unit without waiting for three others: 2048 rows
// of 200-400 keys and 8 key heads 345 against 299 us, 8192 of 20-40 keys 819 against 590 us.
template <int DIM, bool FP16, bool SELECTED, bool TAIL, int NT>
int launch_few(const Params& p, int dev, cudaStream_t s) {
  const int64_t groups = ((int64_t)p.rows + p.group_rows - 1) / p.group_rows;
  if (groups * p.kv_heads >= (int64_t)sm_count(dev) * Smem<DIM, NT, 1, 1>::kCtas)
    return launch<DIM, FP16, SELECTED, TAIL, NT, 1, 1>(p, dev, s);
  return launch<DIM, FP16, SELECTED, TAIL, NT, 1, 4>(p, dev, s);
}

template <int DIM, bool FP16, bool SELECTED, bool TAIL>
int launch_rows(const Params& p, int live, int dev, cudaStream_t s) {
  const int rows = padded_rows(live);
  if (rows == 8) return launch_few<DIM, FP16, SELECTED, TAIL, 1>(p, dev, s);
  if (rows == 16) return launch_few<DIM, FP16, SELECTED, TAIL, 2>(p, dev, s);
  if constexpr (!SELECTED) {  // the selected form has at most 16 rows to a unit
    if (rows == 32) return launch<DIM, FP16, false, TAIL, 4, 1, 4>(p, dev, s);
    if (rows == 64) return launch<DIM, FP16, false, TAIL, 4, 2, 4>(p, dev, s);
    return launch<DIM, FP16, false, TAIL, 4, 4, 4>(p, dev, s);
  }
  return KV8_ERR_SHAPE;
}

Params common(const void* q, int64_t q_ld, int rows, int q_heads, int kv_heads, float sm_scale,
              int block_tokens, const uint8_t* k_cache, const uint8_t* v_cache,
              const float* k_scale, const float* v_scale, int64_t num_slots, void* out,
              int64_t out_ld, float* lse, int32_t* status) {
  Params p = {};
  p.q = (const uint16_t*)q;
  p.q_ld = q_ld;
  p.rows = rows;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.scale = sm_scale * 1.44269504088896341f;
  p.block = block_tokens;
  p.block_shift = shift_of(block_tokens);
  p.k = k_cache;
  p.v = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.num_slots = num_slots;
  p.out = (uint16_t*)out;
  p.out_ld = out_ld;
  p.lse = lse;
  p.status = status;
  return p;
}

// Fills in the workspace and launches the variant for these sizes.
template <bool SELECTED, bool TAIL = false>
int run(Params& p, int dim, int dtype, void* workspace, int64_t ws_bytes, cudaStream_t s) {
  const int64_t need =
      kv8_attention_workspace_bytes(p.q_heads, p.kv_heads, dim, SELECTED ? 1 : p.group_rows);
  if (need < 0) return (int)need;
  if (ws_bytes < need) return KV8_ERR_WORKSPACE;
  const int dev = current_device();
  if (sm_count(dev) < 0) return KV8_ERR_CUDA;
  p.shared = reinterpret_cast<Shared*>(workspace);
  p.parts = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) +
                                     kMaxCtas * sizeof(Shared));
  const int live = p.group_rows * (p.q_heads / p.kv_heads);
  if (dim == 128)
    return dtype == KV8_FP16 ? launch_rows<128, true, SELECTED, TAIL>(p, live, dev, s)
                             : launch_rows<128, false, SELECTED, TAIL>(p, live, dev, s);
  return dtype == KV8_FP16 ? launch_rows<64, true, SELECTED, TAIL>(p, live, dev, s)
                           : launch_rows<64, false, SELECTED, TAIL>(p, live, dev, s);
}

}  // namespace
