// Attention over the 8-bit paged KV cache for more than 32 query rows to a key head (verify steps
// of grouped heads), on the 5th-generation tensor cores: tcgen05.mma of e4m3 codes as they lie in
// the cache, accumulators in tensor memory. Formulas and rules in include/kv8_attention.h, the
// split of the tiles over the CTAs in kv8_common.cuh.
//
// With M rows the products are 4 * 128 * M operations for 256 bytes of codes. On mma.sync the
// codes are widened by every warp that needs them and M = 56 rows took 98 us for 80K keys where
// the bytes take 24. Here nothing is widened: a tile of 128 keys goes from HBM to shared memory
// in the 128-byte swizzle and is an operand of both products.
//   - S[key, row] = K[128 keys, 128] . Q[rows, 128]^T, keys on the 128 lanes of tensor
//     memory. Q is e4m3 too, in pieces stacked along N: q = q0 + q1 / 32 (+ q2 / 1024 for fp16),
//     each piece the rounding to 4 significant bits of what the one before left. The row's
//     largest magnitude lies in [2^7, 2^8), so two pieces hold a bf16, and three an fp16, to
//     2^-22 of it.
//   - O^T[channel, row] = V^T[128, keys] . W[keys, rows]: V in its own order is the transposed
//     operand. The weights w' are rounded to fp16 and split into three pieces the same way,
//     stacked along N with an accumulator each: O = O0 + O1 / 32 + O2 / 1024.
//   - w' = 2^(x + log2 sv - B), the value scale folded in, B a reference per row raised (and O
//     and the sums rescaled) only when a w' would pass 2^8; the largest w' of a row then
//     lies in [2^4, 2^8], and what lies below 2^-20 of 1 is lost. The sum of weights is kept in
//     fp32, unrounded: sum of w' / sv. A thread of the weights is a key, so its scales and
//     its mask are its own, and no row needs a reduction until the end of a unit.
//
// Warp roles (13 warps): 0 .. 7 make the weights, warp w for keys 32 (w % 4) .. + 31 and half
// w / 4 of the rows; 8 .. 11 copy the tiles with cp.async (32 keys each, zeros where a key is
// masked or missing), three tiles on their way; one lane of warp 12 issues the products: those
// of the next tile's scores before those of this tile's values, so that the tensor cores work
// while the weights are made. Every wait is bounded; one that expires sets a flag that ends all
// others, the control flow runs on to its end, and the status tells.
#include "kv8_common.cuh"

namespace kv8 {
namespace {

constexpr int kDim = 128;
constexpr int kTileKeys = 128;
constexpr int kRows = 64;      // rows of a unit (one half of up to 128)
constexpr int kRing = 4;       // tiles in shared memory
constexpr int kDepth = 3;      // tiles on their way
constexpr int kSoftThreads = 256;
constexpr int kLoadThreads = 128;
constexpr int kWideThreads = 512;  // 16 warps, the last three idle: registers move by warpgroups
constexpr int kTileBytes = kTileKeys * kDim;  // codes of K or V: 16 KB
constexpr int kPieceBytes = kTileKeys * kRows;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 192;  // scores in columns [0, 192), sums in [192, 384)
constexpr uint64_t kWaitNs = 200ull * 1000 * 1000;
constexpr float kPass = 256.0f;  // a weight above this raises the reference
constexpr float kHead = 4.0f;    // log2 of a row's largest weight after that

// shared memory, base aligned to 1024 bytes
constexpr int kQOff = kRing * 2 * kTileBytes;
constexpr int kPOff = kQOff + 3 * kRows * kDim;
constexpr int kScaleOff = kPOff + 3 * kPieceBytes;       // [kRing][2][128]
constexpr int kMaskOff = kScaleOff + kRing * 2 * kTileKeys * 4;  // [kRing][4]
constexpr int kMulOff = kMaskOff + kRing * 16;           // [64] each
constexpr int kLenOff = kMulOff + kRows * 4;
constexpr int kBOff = kLenOff + kRows * 4;
constexpr int kKeepOff = kBOff + kRows * 4;
constexpr int kMaxOff = kKeepOff + kRows * 4;            // [4][64]
constexpr int kSumOff = kMaxOff + 4 * kRows * 4;         // [4][64]
constexpr int kNanOff = kSumOff + 4 * kRows * 4;         // [64][4]: a bit per channel
constexpr int kBarOff = kNanOff + kRows * 16;
constexpr int kSmemBytes = kBarOff + 256 + 1024;

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(100000u)
      : "memory");
  return ok != 0;
}

// Waits for the phase of parity `parity`, for at most kWaitNs or until another wait expired.
__device__ __forceinline__ void bar_wait(uint32_t bar, uint32_t parity, volatile int* expired) {
  if (bar_try(bar, parity)) return;
  const uint64_t t0 = now_ns();
  while (!bar_try(bar, parity)) {
    if (*expired) return;
    if (now_ns() - t0 > kWaitNs) {
      *expired = 1;
      return;
    }
  }
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}

__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor: D fp32 (bits 4-5), A and B e4m3 (0 in bits 7-12), transposed A and B in
// bits 15 and 16, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
__host__ __device__ constexpr uint32_t idesc(int n, bool transposed) {
  return (1u << 4) | (transposed ? 3u << 15 : 0u) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

// Matrix descriptor: start >> 4, leading and stride byte offsets >> 4, version 1, swizzle mode (2:
// 128 bytes, 4: 64 bytes). Operands along K: rows of 128 bytes, `stride` from one group of 8
// to the next. Transposed operands: rows (keys) of one swizzle width, `stride` from 8
// keys to the next 8, `lead` from one width of channels or rows to the next.
__device__ __forceinline__ uint64_t mdesc(uint32_t addr, uint32_t lead, uint32_t stride,
                                          uint64_t swizzle) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(stride >> 4) << 32) | ((uint64_t)1 << 46) | (swizzle << 61);
}

// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_load_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
      ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(at)
      : "memory");
}

// Barrier of the 8 weight warps.
__device__ __forceinline__ void soft_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory");
}
__device__ __forceinline__ bool soft_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(kSoftThreads)
      : "memory");
  return r != 0;
}

// Two numbers to e4m3 (a in the lower byte), and back.
__device__ __forceinline__ uint32_t to_e4m3(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3(uint32_t c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3);
  return __half22float2(__half2(h));
}

// a, b (at most 256 in magnitude) as codes of the pieces: x = p0 + p1 / 32 + p2 / 1024.
__device__ __forceinline__ void pieces(float a, float b, uint32_t (&p)[3]) {
  p[0] = to_e4m3(a, b);
  const float2 f = from_e4m3(p[0]);
  const float a1 = (a - f.x) * 32.0f, b1 = (b - f.y) * 32.0f;  // exact
  p[1] = to_e4m3(a1, b1);
  const float2 g = from_e4m3(p[1]);
  p[2] = to_e4m3((a1 - g.x) * 32.0f, (b1 - g.y) * 32.0f);
}

// The same of two fp16 (non-negative, at most 256): the differences are exact in fp16 too, two at
// an operation.
__device__ __forceinline__ uint32_t half_to_e4m3(__half2 x) {
  return (uint32_t)__nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE,
                                              __NV_E4M3);
}
__device__ __forceinline__ __half2 half_from_e4m3(uint32_t c) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3));
}
__device__ __forceinline__ void pieces(__half2 x, uint32_t (&p)[3]) {
  const __half2 up = __float2half2_rn(32.0f);
  p[0] = half_to_e4m3(x);
  const __half2 x1 = __hmul2(__hsub2(x, half_from_e4m3(p[0])), up);
  p[1] = half_to_e4m3(x1);
  const __half2 x2 = __hmul2(__hsub2(x1, half_from_e4m3(p[1])), up);
  p[2] = half_to_e4m3(x2);
}

// The next segment of a CTA's range: tiles [tile0, tile1) of a unit of `tiles`.
struct Segment {
  int tile0, tile1, tiles;
};

struct Walk {
  Range r;
  int64_t w;
  __device__ __forceinline__ bool more() const { return w < r.w1; }
  __device__ __forceinline__ Segment segment() const {
    const int tiles = tiles_of<kTileKeys>(r.len);
    return {(int)(w - r.first), (int)min((int64_t)tiles, r.w1 - r.first), tiles};
  }
  __device__ __forceinline__ void next(const Params& p, const Segment& s, int subs) {
    w = r.first + s.tile1;
    if (s.tile1 == s.tiles) {
      r.first += s.tiles;
      if (++r.s == subs) {
        r.s = 0;
        ++r.g;
        int ignored = 0;
        if (w < r.w1) r.len = group_len(p, r.g, &ignored);
      }
    }
  }
};

template <bool FP16>
__global__ void __launch_bounds__(kWideThreads, 1)
kv8_wide_kernel(const __grid_constant__ Params p) {
  constexpr int kQPieces = FP16 ? 3 : 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_expired;
  uint8_t* const sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t base = smem_u32(sm);
  const uint32_t bars = base + kBarOff;
  const uint32_t b_full = bars;                   // [kRing] copies of a tile (128 threads)
  const uint32_t b_empty = bars + 8 * kRing;      // [kRing] both products of a tile done
  const uint32_t b_scores = bars + 16 * kRing;    // scores in tensor memory
  const uint32_t b_read = b_scores + 8;           // scores read (256 threads)
  const uint32_t b_weights = b_read + 8;          // weights in shared memory (256)
  const uint32_t b_values = b_weights + 8;        // product with the values done
  const uint32_t b_query = b_values + 8;          // queries of a segment staged (256)
  const uint32_t b_sums = b_query + 8;            // sums of a segment read (256)
  const uint32_t b_done = b_sums + 8;             // every product done
  volatile uint32_t* const tmem_slot = reinterpret_cast<volatile uint32_t*>(sm + kBarOff + 192);
  volatile int* const expired = &s_expired;
  asm volatile("griddepcontrol.launch_dependents;");  // the join, which waits for this launch

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_expired = 0;
    for (int i = 0; i < kRing; ++i) {
      bar_init(b_full + 8 * i, kLoadThreads);
      bar_init(b_empty + 8 * i, 1);
    }
    bar_init(b_scores, 1);
    bar_init(b_read, kSoftThreads);
    bar_init(b_weights, kSoftThreads);
    bar_init(b_values, 1);
    bar_init(b_query, kSoftThreads);
    bar_init(b_sums, kSoftThreads);
    bar_init(b_done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(const_cast<uint32_t*>(tmem_slot))),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int ratio = p.q_heads / p.kv_heads;
  const int groups = (p.rows + p.group_rows - 1) / p.group_rows;
  const int subs = p.kv_heads * p.halves;
  int err = 0;
  Walk walk;
  walk.r = locate<kTileKeys>(p, groups, subs, 1, &err);
  walk.w = walk.r.w0;
  const int64_t units = (int64_t)groups * subs;
  Shared mine = {0, 0, 0, -1};

  // 512 threads of 128 registers: 256 of 184 and 256 of 72
  if (warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ---------------------------------------------------------------- copies
    const int lw = warp - 8;
    int it = 0, done = 0;
    for (; walk.more();) {
      const Segment sg = walk.segment();
      const int h = walk.r.s / p.halves, len = walk.r.len;
      const int table = p.group_table ? __ldg(p.group_table + walk.r.g) : walk.r.g;
      auto slot_of = [&](int tile) -> int {
        const int64_t i = (int64_t)tile * kTileKeys + lw * 32 + lane;
        if (tile >= sg.tile1 || i >= len) return -1;
        const int pos = (int)i;
        const int pg = p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page_size;
        const int32_t page = __ldg(p.block_table + table * p.table_ld + pg);
        if (page < 0) {
          err |= KV8_STATUS_TABLE_ENTRY;
          return -1;
        }
        const int64_t slot = (int64_t)page * p.page_size + (pos - pg * p.page_size);
        if (slot >= p.num_slots) {
          err |= KV8_STATUS_SLOT;
          return -1;
        }
        return (int)slot;
      };
      int slot = slot_of(sg.tile0);
      for (int tile = sg.tile0; tile < sg.tile1; ++tile) {
        const int stage = it % kRing;
        if (it >= kRing) bar_wait(b_empty + 8 * stage, (it / kRing - 1) & 1, expired);
        const uint32_t k_at = base + stage * 2 * kTileBytes + lw * 32 * kDim, v_at = k_at + kTileBytes;
        const int piece = lane & 7;
        const int64_t row = ((int64_t)max(slot, 0) * p.kv_heads + h) * kDim;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int key = j * 4 + (lane >> 3);
          const int64_t off = __shfl_sync(0xffffffffu, row, key) + piece * 16;
          const bool in = __shfl_sync(0xffffffffu, slot, key) >= 0;
          const int at = key * kDim + ((piece ^ (key & 7)) << 4);
          copy16(k_at + at, p.k + off, in);
          copy16(v_at + at, p.v + off, in);
        }
        const int sl = max(slot, 0);
        const int b = p.block_shift >= 0 ? sl >> p.block_shift : sl / p.block;
        const int64_t off = (int64_t)b * p.kv_heads + h;
        const uint32_t s_at = base + kScaleOff + (stage * 2 * kTileKeys + lw * 32 + lane) * 4;
        copy4(s_at, p.k_scale + off, slot >= 0);
        copy4(s_at + kTileKeys * 4, p.v_scale + off, slot >= 0);
        copy_commit();
        const uint32_t in = __ballot_sync(0xffffffffu, slot >= 0);
        if (lane == 0) reinterpret_cast<uint32_t*>(sm + kMaskOff)[stage * 4 + lw] = in;
        slot = slot_of(tile + 1);
        ++it;
        if (it - done >= kDepth) {
          copy_wait<kDepth - 1>();
          fence_async();
          bar_arrive(b_full + 8 * (done % kRing));
          ++done;
        }
      }
      walk.next(p, sg, subs);
    }
    copy_wait<0>();
    fence_async();
    for (; done < it; ++done) bar_arrive(b_full + 8 * (done % kRing));
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // ---------------------------------------------------------------- products
    if (warp == 12 && lane == 0) {
      constexpr uint32_t kScores = idesc(kRows * kQPieces, false);
      constexpr uint32_t kValues = idesc(kRows * 3, true);
      int it = 0, seg = 0;
      auto scores = [&](int i) {
        const int stage = i % kRing;
        bar_wait(b_full + 8 * stage, (i / kRing) & 1, expired);
        if (i > 0) bar_wait(b_read, (i - 1) & 1, expired);
        if (*expired) return;
        tc_fence_after();
        const uint64_t a = mdesc(base + stage * 2 * kTileBytes, 16, 1024, 2);
        const uint64_t b = mdesc(base + kQOff, 16, 1024, 2);
#pragma unroll
        for (int k = 0; k < kDim / 32; ++k)  // 32 bytes on along a row
          tc_mma(tmem, a + 2 * k, b + 2 * k, kScores, k > 0);
        tc_commit(b_scores);
      };
      for (; walk.more(); ++seg) {
        const Segment sg = walk.segment();
        bar_wait(b_query, seg & 1, expired);
        for (int tile = sg.tile0; tile < sg.tile1; ++tile, ++it) {
          if (tile == sg.tile0) scores(it);
          if (tile + 1 < sg.tile1) scores(it + 1);
          bar_wait(b_weights, it & 1, expired);
          if (tile == sg.tile0 && seg > 0) bar_wait(b_sums, (seg - 1) & 1, expired);
          if (*expired) continue;
          tc_fence_after();
          const int stage = it % kRing;
          const uint64_t a = mdesc(base + stage * 2 * kTileBytes + kTileBytes, 16, 1024, 2);
          const uint64_t b = mdesc(base + kPOff, kPieceBytes, 512, 4);
#pragma unroll
          for (int k = 0; k < kTileKeys / 32; ++k)  // 32 keys on
            tc_mma(tmem + kOCol, a + k * (32 * kDim >> 4), b + k * (32 * kRows >> 4), kValues,
                   k > 0 || tile > sg.tile0);
          tc_commit(b_values);
          tc_commit(b_empty + 8 * stage);
        }
        walk.next(p, sg, subs);
      }
      tc_commit(b_done);
      bar_wait(b_done, 0, expired);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    // ---------------------------------------------------------------- weights
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const int c0 = half * 32;  // this thread's rows: c0 .. c0 + 31
    const int key = quarter * 32 + lane;
    float* const s_mul = reinterpret_cast<float*>(sm + kMulOff);
    int* const s_len = reinterpret_cast<int*>(sm + kLenOff);
    float* const s_b = reinterpret_cast<float*>(sm + kBOff);
    float* const s_keep = reinterpret_cast<float*>(sm + kKeepOff);
    float* const s_max = reinterpret_cast<float*>(sm + kMaxOff);
    float* const s_sum = reinterpret_cast<float*>(sm + kSumOff);
    uint32_t* const s_nan = reinterpret_cast<uint32_t*>(sm + kNanOff);
    int it = 0;
    for (; walk.more();) {
      const Segment sg = walk.segment();
      const int h = walk.r.s / p.halves, r0 = walk.r.s % p.halves * kRows;
      const int live = min(p.group_rows * ratio - r0, kRows);
      const int table = p.group_table ? __ldg(p.group_table + walk.r.g) : walk.r.g;
      // ---- queries in pieces
#pragma unroll
      for (int x = tid; x < kRows * 8; x += kSoftThreads) {
        const int r = x >> 3, c = x & 7;  // 16 channels from 16 c
        const int64_t row = (int64_t)walk.r.g * p.group_rows + (r0 + r) / ratio;
        const bool in = r < live && row < p.rows;
        uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (in) {
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + row * p.q_ld + (int64_t)(h * ratio + (r0 + r) % ratio) * kDim + c * 16);
          v[0] = __ldg(src);
          v[1] = __ldg(src + 1);
        }
        const uint32_t wds[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
        float f[16];
        uint32_t top = 0;  // bits of the largest magnitude
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (FP16) {
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&wds[i]));
            f[2 * i] = y.x;
            f[2 * i + 1] = y.y;
          } else {
            f[2 * i] = __uint_as_float(wds[i] << 16);
            f[2 * i + 1] = __uint_as_float(wds[i] & 0xFFFF0000u);
          }
          top = max(top, max(__float_as_uint(fabsf(f[2 * i])), __float_as_uint(fabsf(f[2 * i + 1]))));
        }
#pragma unroll
        for (int o = 4; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // 2^up brings the row's largest magnitude into [2^7, 2^8)
        const int e = (int)(top >> 23);
        const int up = top == 0 ? 0 : min(126, 7 - (e - 127));
        const float g = e == 255 ? 0.0f : __uint_as_float((uint32_t)(up + 127) << 23);
        uint32_t q[3][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t pc[3];
          pieces(e == 255 ? 0.0f : f[2 * i] * g, e == 255 ? 0.0f : f[2 * i + 1] * g, pc);
#pragma unroll
          for (int k = 0; k < 3; ++k)
            q[k][i >> 1] = i & 1 ? q[k][i >> 1] | (pc[k] << 16) : pc[k];
        }
#pragma unroll
        for (int k = 0; k < kQPieces; ++k)
          *reinterpret_cast<uint4*>(sm + kQOff + (k * kRows + r) * kDim + ((c ^ (r & 7)) << 4)) =
              make_uint4(q[k][0], q[k][1], q[k][2], q[k][3]);
        if (c == 0) {
          int ignored = 0;
          // a row that is not finite gives NaN
          s_mul[r] = e == 255 ? NAN : p.scale * __uint_as_float((uint32_t)(127 - up) << 23);
          // only rows that end before the unit's keys do need the comparison with their length
          s_len[r] = in ? row_len(p, (int)row, table, &ignored) : INT32_MAX;
          s_b[r] = kNone;
        }
      }
      if (tid < kRows * 4) s_nan[tid] = 0;
      fence_async();
      soft_sync();
      bar_arrive(b_query);
      const int least =
          __reduce_min_sync(0xffffffffu, min(s_len[lane], s_len[32 + lane]));  // where a row ends

      float sum[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) sum[c] = 0.0f;
      for (int tile = sg.tile0; tile < sg.tile1; ++tile, ++it) {
        const int stage = it % kRing;
        bar_wait(b_scores, it & 1, expired);
        bar_wait(b_full + 8 * stage, (it / kRing) & 1, expired);
        __syncwarp();
        tc_fence_after();
        const uint32_t in = reinterpret_cast<const uint32_t*>(sm + kMaskOff)[stage * 4 + quarter];
        const float* sc = reinterpret_cast<const float*>(sm + kScaleOff) + stage * 2 * kTileKeys;
        const float ks = sc[key], sv = sc[kTileKeys + key];
        const bool valid = (in >> lane) & 1;
        // values of scale 0 weigh nothing but count in the sum: they pass through it at 2^-60
        const bool zero = sv == 0.0f;
        const float lv = zero ? -60.0f : log2_fast(sv);
        const float back = zero ? 0x1p60f : sv > 0.0f && sv < INFINITY ? 1.0f / sv : 1.0f;
        const bool ragged = (int64_t)(tile + 1) * kTileKeys > least;
        // x, the log2 of the weights (with the value scale, without the reference)
        auto scores = [&](float (&x)[32]) {
          uint32_t a[32];
          tmem_load(lanes + c0, a);
          tmem_load(lanes + kRows + c0, reinterpret_cast<uint32_t(&)[32]>(x));
          tmem_load_wait();
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c] = fmaf(x[c], 1.0f / 32, __uint_as_float(a[c]));
          if (FP16) {
            tmem_load(lanes + 2 * kRows + c0, a);
            tmem_load_wait();
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c] = fmaf(__uint_as_float(a[c]), 1.0f / 1024, x[c]);
          }
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 m = *reinterpret_cast<const float4*>(s_mul + c0 + c);
            x[c] = fmaf(x[c] * ks, m.x, lv);
            x[c + 1] = fmaf(x[c + 1] * ks, m.y, lv);
            x[c + 2] = fmaf(x[c + 2] * ks, m.z, lv);
            x[c + 3] = fmaf(x[c + 3] * ks, m.w, lv);
          }
          if (ragged || in != 0xffffffffu) {
            const int64_t pos = (int64_t)tile * kTileKeys + key;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!valid || pos >= s_len[c0 + c]) x[c] = -INFINITY;
          }
        };
        bool freed = tile == sg.tile0;  // the product before has read its weights
        float w[32];
        // Once in most tiles. Where a weight would pass kPass, a second time with new references for
        // the rows where one does (the scores are read again, which costs no registers meanwhile).
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          scores(w);
          if (pass == 1) {
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const int bits = __float_as_int(w[c]);
              const int top = __reduce_max_sync(0xffffffffu, bits ^ ((bits >> 31) & 0x7fffffff));
              if (lane == c)
                s_max[quarter * kRows + c0 + c] = __int_as_float(top ^ ((top >> 31) & 0x7fffffff));
            }
            soft_sync();
            if (tid < kRows) {
              const float top = fmaxf(fmaxf(s_max[tid], s_max[kRows + tid]),
                                      fmaxf(s_max[2 * kRows + tid], s_max[3 * kRows + tid]));
              const float b = s_b[tid], to = exp2_fast(top - b) > kPass ? top - kHead : b;
              s_keep[tid] = exp2_fast(b - to);
              s_b[tid] = to;
            }
            soft_sync();
            if (!freed) {
              bar_wait(b_values, (it - 1) & 1, expired);
              __syncwarp();
              freed = true;
              tc_fence_after();
#pragma unroll 1
              for (int k = 0; k < 3; ++k) {
                const uint32_t at = lanes + kOCol + k * kRows + c0;
                uint32_t v[32];
                tmem_load(at, v);
                tmem_load_wait();
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  v[c] = __float_as_uint(__uint_as_float(v[c]) * s_keep[c0 + c]);
                tmem_store(at, v);
              }
              asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            }
#pragma unroll
            for (int c = 0; c < 32; ++c) sum[c] *= s_keep[c0 + c];
          }
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 b = *reinterpret_cast<const float4*>(s_b + c0 + c);
            w[c] = exp2_fast(w[c] - b.x);
            w[c + 1] = exp2_fast(w[c + 1] - b.y);
            w[c + 2] = exp2_fast(w[c + 2] - b.z);
            w[c + 3] = exp2_fast(w[c + 3] - b.w);
          }
          if (pass == 1) break;
          float most = 0.0f;
#pragma unroll
          for (int c = 0; c < 32; ++c) most = fmaxf(most, w[c]);
          if (!soft_any(most > kPass)) break;
        }
        tc_fence_before();
        bar_arrive(b_read);
#pragma unroll
        for (int c = 0; c < 32; ++c) sum[c] = fmaf(w[c], back, sum[c]);
        if (__any_sync(0xffffffffu, zero)) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (zero) w[c] = 0.0f;
        }
        // ---- the weights' pieces: 16 rows are 16 bytes of a piece
        uint32_t code[3][8];
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          uint32_t lo[3], hi[3];
          pieces(__floats2half2_rn(w[c], w[c + 1]), lo);
          pieces(__floats2half2_rn(w[c + 2], w[c + 3]), hi);
#pragma unroll
          for (int k = 0; k < 3; ++k) code[k][c >> 2] = __byte_perm(lo[k], hi[k], 0x5410);
        }
        if (!freed) {
          bar_wait(b_values, (it - 1) & 1, expired);
          __syncwarp();
        }
        uint8_t* const at = sm + kPOff + key * kRows;
        const int turn = (key >> 1) & 3;
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint4*>(at + k * kPieceBytes + (((half * 2 + i) ^ turn) << 4)) =
                make_uint4(code[k][4 * i], code[k][4 * i + 1], code[k][4 * i + 2], code[k][4 * i + 3]);
        // ---- a NaN code must not reach the rows that end before it (0 * NaN is NaN in a
        // product): where a row ends, the rows that see one are marked, and it becomes 0
        if (ragged && half == 0 && valid) {
          const int64_t pos = (int64_t)tile * kTileKeys + key;
          uint8_t* const v_row = sm + stage * 2 * kTileBytes + kTileBytes + key * kDim;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint4* const v_at = reinterpret_cast<uint4*>(v_row + ((c ^ (key & 7)) << 4));
            const uint4 v = *v_at;
            const uint32_t n[4] = {nan_codes(v.x), nan_codes(v.y), nan_codes(v.z), nan_codes(v.w)};
            if (!(n[0] | n[1] | n[2] | n[3])) continue;
            *v_at = make_uint4(v.x & ~n[0], v.y & ~n[1], v.z & ~n[2], v.w & ~n[3]);
            uint32_t bits = 0;  // of channels 16 c .. + 15
#pragma unroll
            for (int i = 0; i < 16; ++i) bits |= ((n[i >> 2] >> (8 * (i & 3))) & 1) << i;
            for (int r = 0; r < live; ++r)
              if (pos < s_len[r]) atomicOr(s_nan + r * 4 + (c >> 1), bits << (16 * (c & 1)));
          }
        }
        fence_async();
        tc_fence_before();
        bar_arrive(b_weights);
      }

      // ---- end of the segment: sums of the weights, then the products
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        float y = sum[c];
#pragma unroll
        for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (lane == c) s_sum[quarter * kRows + c0 + c] = y;
      }
      bar_wait(b_values, (it - 1) & 1, expired);
      __syncwarp();
      tc_fence_after();
      float o[32];
      {
        uint32_t a[32], b[32];
        tmem_load(lanes + kOCol + c0, a);
        tmem_load(lanes + kOCol + kRows + c0, b);
        tmem_load_wait();
#pragma unroll
        for (int c = 0; c < 32; ++c)
          o[c] = fmaf(__uint_as_float(b[c]), 1.0f / 32, __uint_as_float(a[c]));
        tmem_load(lanes + kOCol + 2 * kRows + c0, a);
        tmem_load_wait();
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] = fmaf(__uint_as_float(a[c]), 1.0f / 1024, o[c]);
      }
      tc_fence_before();
      bar_arrive(b_sums);
      soft_sync();
      const bool whole = sg.tile0 == 0 && sg.tile1 == sg.tiles;
      const int channel = quarter * 32 + lane;  // of this thread
      using P = Part<kDim, kRows>;
      float* const part = p.parts + (2 * (int64_t)blockIdx.x + (sg.tile0 == 0)) * P::kFloats;
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const int r = c0 + c;
        if (r >= live) break;
        float v = o[c];
        if ((s_nan[r * 4 + quarter] >> lane) & 1) v = NAN;
        const float l = (s_sum[r] + s_sum[kRows + r]) + (s_sum[2 * kRows + r] + s_sum[3 * kRows + r]);
        if (whole) {
          const int64_t row = (int64_t)walk.r.g * p.group_rows + (r0 + r) / ratio;
          if (row >= p.rows) continue;
          const int head = h * ratio + (r0 + r) % ratio;
          const float y = l == 0.0f ? 0.0f : v / l;
          p.out[row * p.out_ld + (int64_t)head * kDim + channel] =
              FP16 ? __half_as_ushort(__float2half_rn(y))
                   : __bfloat16_as_ushort(__float2bfloat16_rn(y));
          if (channel == 0 && p.lse)
            p.lse[row * p.q_heads + head] =
                l == 0.0f ? -INFINITY : (s_b[r] + log2f(l)) * 0.69314718055994531f;
        } else {
          part[r * kDim + channel] = v;
          if (channel == 0)
            *reinterpret_cast<float4*>(part + P::kStat + r * 4) = make_float4(s_b[r], s_b[r], l, 0.0f);
        }
      }
      if (sg.tile0 == 0) {
        const Shared u = {walk.r.g, walk.r.s, (int32_t)blockIdx.x,
                          whole ? -1 : (int32_t)(((walk.r.first + sg.tiles) * walk.r.n - 1) / walk.r.all)};
        if (units > kMaxCtas) mine = whole ? mine : u;
        else if (tid == 0) p.shared[(int64_t)walk.r.g * subs + walk.r.s] = u;
      }
      soft_sync();  // the shared arrays serve the next segment
      walk.next(p, sg, subs);
    }
    if (tid == 0 && units > kMaxCtas) p.shared[blockIdx.x] = mine;
  }
  if (err && p.status) atomicOr(p.status, err);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && s_expired && p.status) atomicOr(p.status, KV8_STATUS_TIMEOUT);
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                 : "memory");
}

template <bool FP16>
int launch(const Params& p, int dev, cudaStream_t s) {
  const auto kernel = kv8_wide_kernel<FP16>;
  const auto join = kv8_join_kernel<kDim, FP16, kRows>;
  static std::atomic<uint64_t> ready;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) !=
            cudaSuccess ||
        cudaFuncSetAttribute(join, cudaFuncAttributePreferredSharedMemoryCarveout, 100) !=
            cudaSuccess)
      return KV8_ERR_CUDA;
    ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  const int sms = sm_count(dev);
  const int64_t groups = ((int64_t)p.rows + p.group_rows - 1) / p.group_rows;
  const int64_t units = groups * p.kv_heads * p.halves;
  const int64_t tiles =
      p.max_len < kTileKeys ? 1 : ((int64_t)p.max_len + kTileKeys - 1) / kTileKeys;
  if (units > (int64_t(1) << 33)) return KV8_ERR_SHAPE;
  const int64_t want = units * tiles;
  const int64_t most = sms < kMaxCtas ? sms : kMaxCtas;
  const int grid = (int)(want < most ? want : most);
  kernel<<<(unsigned)grid, kWideThreads, kSmemBytes, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return KV8_ERR_CUDA;
  return launch_join<kDim, FP16, kRows>(p, units, grid, s);
}

}  // namespace

int launch_wide(Params& p, bool fp16, int dev, cudaStream_t s) {
  p.halves = (p.group_rows * (p.q_heads / p.kv_heads) + kRows - 1) / kRows;
  return fp16 ? launch<true>(p, dev, s) : launch<false>(p, dev, s);
}

}  // namespace kv8
