// Attention of requests that share prefixes over the 8-bit paged cache (rules in
// include/kv8_attention.h).
//
// A set's requests read the same keys below its prefix length, so that all their query rows on
// a key head are one product with them: 4 * dim operations a key for each of M = requests * rows
// * (query heads / key heads) rows, and 2 * dim bytes a key once. From M of about 256 on the
// tensor cores bound it, below that HBM. What lies behind the prefix is each request's own and is
// read by the kernel of kv8_attention.cuh, which starts behind the prefix and adds what the
// rows have of it.
//
// Launches: the prefixes' parts (below); the join of the parts of units that several CTAs
// share; the rows' own positions; the join of those.
//
// Prefix kernel. One CTA to an SM. A unit is (set, key head, 256 of the set's query rows) and
// its steps are tiles of 128 keys; the steps of all units are laid end to end and divided
// evenly over the CTAs, from the lengths on the device. Two streams of 128 rows run in a CTA,
// so that the products of one overlap the softmax of the other: they take the same keys for
// different rows, or, where only 128 rows are left, the tiles of even and odd number for the
// same rows (their sums are joined at the end).
//   - Warps 8-15 bring codes from the pages into a ring by cp.async, widen them to fp16 (exact)
//     and store them in the 128-byte swizzle; keys as they lie (K-major), values as they lie
//     too, as the transposed (MN-major) operand.
//   - Warps 0-3 and 4-7 are the two streams, a thread to a row. The first thread of each issues
//     its tcgen05.mma (kind::f16): S = Q K^T into tensor memory, and O += P V with the weights P
//     read from tensor memory. All take the scores from there and put weights back over them
//     as fp16; the next scores wait until O += P V has read them (1 % of the time). O stays in
//     tensor memory; a row's reference is raised, and its O rescaled, only when sixteen of its
//     weights together pass 2^15. It is set 2^7 below the row's largest, so that fp16 holds
//     weights down to 2^-31 of it.
//   - Scales belong to 16 keys at least (block_tokens): key scales multiply the scores, value
//     scales join the exponent, relative to the first of the segment, and come out of the
//     row's sum again. Where they lie more than 2^8 apart, sums and weights get references
//     of their own and an exponential each.
// Measured: 64 requests behind 32768 positions, 64 / 8 heads of 128, 105 us (69 Gflop, 650
// TFLOP/s): a stream takes 5500 cycles for 128 keys, where the products of both streams are 2048;
// within a stream scores, weights and sums of a tile follow one another. 8 requests behind 80000
// positions 78 us (2.1 TB/s), half of a stream's rows empty. Start and end take 9 us.
//
// Every mbarrier wait is bounded; one that runs out sets KV8_STATUS_TIMEOUT and ends the CTA's
// work after its products in flight. Instead of the sums of all its units that are not finished
// the CTA then writes NaN, which the join and the rows' own pass carry into out and lse: what an
// earlier call left in these places of the workspace would give numbers like any other.
#include <cfloat>

#include "kv8_attention.cuh"

namespace {

constexpr int kTile = 128;      // keys of a tile, rows of a stream
constexpr int kWidenWarps = 8;  // behind the eight of the streams
constexpr int kPThreads = 256 + 32 * kWidenWarps;
constexpr int kPRows = 2 * kTile;
constexpr int kLeast = 128;     // positions of the least prefix that is read for all
// Bytes of keys and values that sharing has to save by the caller's bounds, (groups - 1) *
// max_prefix positions: below, the rows' own pass reads the prefixes again, mostly from L2, and is
// done before two launches more would be (one set on 8 key heads of 128, 64 tokens of their own, rows'
// own pass against this: 8 requests of 8192 positions 33 / 38 us, 117 MB; 4 of 32768 49 / 60,
// 201 MB; 8 of 32768 82 / 61, 470 MB; 32 of 8192 82 / 58, 520 MB; on 2 key heads 32 of 32768 81 / 62,
// 520 MB). The bounds count all groups and the longest prefix: where two requests of a batch share
// 512 positions under a bound of 32768, the call takes about 25 us more than kv8_attention's (64 of
// 4096 tokens 142 / 116, 256 of 512 141 / 117).
constexpr double kWorth = 256e6;
constexpr float kRaise = 11.0f, kBelow = 7.0f;  // log2: a reference is raised from here, to there
constexpr float kMost = 32768.0f;  // of 16 weights together: 2^15, which is 2^kRaise for the largest
constexpr uint64_t kWaitNs = 200ull * 1000 * 1000;

// A unit whose parts CTAs first .. last have (last < 0: none).
struct __align__(16) Split {
  int32_t g0, h;        // first group of the set, key head
  int32_t row0, row1;   // its rows, counted over the set's groups, rows and heads
  int32_t first, last;
  int32_t pad[2];
};

struct Prefix {
  Params p;
  const int32_t* set_starts;
  int n_sets;
  const int32_t* prefix_lens;
  int max_prefix;
  int groups;
  int32_t* start;    // [groups] (written): positions that a group has from its set
  float* before;     // [rows * q_heads][dim + 4] (written)
  Split* splits;     // [CTAs] (written): the split unit that starts in each
  float* parts;      // two parts of kPRows rows for each CTA
  int skip;          // a CTA whose keys and values never come (tests), or -1
};

// What the softmax needs to know of a tile; sixteen keys of it have one scale.
struct __align__(16) Meta {
  float ks[8];    // key scales
  float dl[8];    // log2(value scale) - ref
  float inv[8];   // 2^-dl
  float ref;      // log2 of the segment's first value scale
  uint32_t in;    // sixteens that have a page
  int32_t end;    // keys of the tile below the prefix length
  int32_t wide;   // value scales more than 2^8 from the first, in this tile or one before
};

template <int DIM>
struct PSmem {
  static constexpr int kBlocks = DIM / 64;             // 64 channels of fp16: 128 bytes of a row
  static constexpr int kOperand = kBlocks * kTile * 128;  // bytes of 128 rows of fp16
  static constexpr int kHalf = kTile * DIM;            // codes of a tile's keys (or values)
  static constexpr int kK = 2 * kOperand;              // two tiles, behind the two of queries
  static constexpr int kV = kK + 2 * kOperand;         // one
  static constexpr int kRaw = kV + kOperand;           // codes on their way: kSlots halves, and
  static constexpr int kSlots = 3;                     // kMoreSlots over the second queries'
  static constexpr int kMoreSlots = 2;                 // place where there is one tile of them
  static constexpr int kMeta = kRaw + kSlots * kHalf;
  static constexpr int kBars = kMeta + 4 * (int)sizeof(Meta);
  static constexpr int kMul = kBars + 256;
  static constexpr int kStart = kMul + kPRows * 4;
  static constexpr int kEff = kStart + (KV8_MAX_SETS + 4) * 4;
  static constexpr int kLead = kEff + KV8_MAX_SETS * 4;
  static constexpr int kTotal = kLead + KV8_MAX_SETS * 4 + 1024;  // base brought to 1024 bytes
  // before the first segment, over keys and values
  static constexpr int kCum = kK;                      // int64 [sets + 1]
  static constexpr int kLast = kCum + (KV8_MAX_SETS + 2) * 8;
  static_assert(kLast + KV8_MAX_SETS * 4 <= kMeta, "over keys, values and codes");
  static constexpr int kLd = DIM + 4;  // floats between rows where the streams' sums meet
  static_assert(kK + 2 * kTile * kLd * 4 <= kMeta, "the sums fit over keys, values and codes");
  static_assert(kMoreSlots * kHalf <= kOperand, "halves over the second queries");
  static_assert(kTotal <= 227 * 1024, "shared memory of an SM");
};

// ------------------------------------------------------------------ PTX
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
      : "r"(bar), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}
// Waits for the phase of this parity, unless the CTA gave up or kWaitNs pass: then it gives up.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* quit) {
  if (bar_try(bar, parity)) return true;
  const uint64_t t0 = now_ns();
  while (!bar_try(bar, parity)) {
    if (*quit) return false;
    if (now_ns() - t0 > kWaitNs) {
      *quit = 1;
      return false;
    }
  }
  return true;
}
// The same, whether the CTA gave up or not.
__device__ __forceinline__ void bar_wait_through(uint32_t bar, uint32_t parity, volatile int* quit) {
  const uint64_t t0 = now_ns();
  while (!bar_try(bar, parity))
    if (now_ns() - t0 > kWaitNs) {
      *quit = 1;
      return;
    }
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// What this thread wrote to shared memory is seen by the tensor cores after the next barrier.
__device__ __forceinline__ void proxy_fence() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Arrives on `bar` once every product this thread issued before has finished.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}
// D[tmem] (+)= A[smem] . B[smem], fp16 x fp16 -> fp32.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of kind::f16: D fp32 (bits 4-5 = 1), A and B fp16 (0 in bits 7-9 and
// 10-12), B transposed (MN-major) in bit 16, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}
// Shared-memory descriptor in the 128-byte swizzle: start >> 4 in bits 0-13, leading offset
// >> 4 in bits 16-29 (between blocks of 64 of an MN-major operand; unused for a K-major one),
// stride offset >> 4 in bits 32-45 (1024 bytes between groups of 8 rows), version 1 in bits
// 46-47, swizzle mode 2 in bits 61-63.
__device__ __forceinline__ uint64_t sdesc(uint32_t at, uint32_t leading) {
  return (uint64_t)((at & 0x3FFFFu) >> 4) | ((uint64_t)(leading >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Two floats to an operation.
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Tensor memory: this warp's 32 lanes x N columns from `at`, one row of them to a thread.
__device__ __forceinline__ void tmem_ld(uint32_t at, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(at)
      : "memory");
}

__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&v)[64]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x64.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, "
      "%33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, "
      "%49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63, %64};"
      :
      : "r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
        "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
        "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]),
        "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(v[32]), "r"(v[33]), "r"(v[34]),
        "r"(v[35]), "r"(v[36]), "r"(v[37]), "r"(v[38]), "r"(v[39]), "r"(v[40]), "r"(v[41]),
        "r"(v[42]), "r"(v[43]), "r"(v[44]), "r"(v[45]), "r"(v[46]), "r"(v[47]), "r"(v[48]),
        "r"(v[49]), "r"(v[50]), "r"(v[51]), "r"(v[52]), "r"(v[53]), "r"(v[54]), "r"(v[55]),
        "r"(v[56]), "r"(v[57]), "r"(v[58]), "r"(v[59]), "r"(v[60]), "r"(v[61]), "r"(v[62]),
        "r"(v[63])
      : "memory");
}

__device__ __forceinline__ void tmem_st(uint32_t at, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      :
      : "r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]),
        "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]),
        "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]),
        "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
        "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t at, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15])
      : "r"(at)
      : "memory");
}

__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8};"
      :
      : "r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
        "r"(v[7])
      : "memory");
}
// The same in two steps: the registers are not to be touched before the wait, which is for all
// loads of the thread.
__device__ __forceinline__ void tmem_ld_start(uint32_t at, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15])
      : "r"(at)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_wait(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ------------------------------------------------------------------ a segment
// What a CTA does of one unit at a time; written by its first thread. The roles are functions of
// their own, so that each has the registers to itself.
struct __align__(16) Segment {
  const int32_t* table;  // block-table row through which the prefix is read
  float* part;           // where the sums go if the unit is split
  int32_t g0, h;         // first group of the set, key head
  int32_t row0, rows;    // first row of the unit; rows of the set on a key head
  int32_t eff;           // positions of the prefix
  int32_t tile0, tile1;
  int32_t two;           // two streams of rows, else of keys
  int32_t whole;         // the CTA has all of the unit
  int32_t count[2];      // tiles of each stream
  uint32_t tiles_done, turns[2], parity;  // of the segments before: the barriers' counters

  // query row and head of a row of the unit
  __device__ __forceinline__ int64_t row_at(const Params& p, int ratio, int r) const {
    return (int64_t)g0 * p.group_rows + (row0 + r) / ratio;
  }
  __device__ __forceinline__ int head_at(int ratio, int r) const {
    return h * ratio + (row0 + r) % ratio;
  }
  __device__ __forceinline__ bool has_row(const Params& p, int ratio, int r) const {
    return row0 + r < rows && row_at(p, ratio, r) < p.rows;
  }
};

// Warps 0-7: the queries, as kv8_attention.cuh brings them to fp16; a negative scale turns their sign.
template <int DIM, bool FP16>
__device__ __noinline__ void load_queries(const Prefix& P, const Segment& g, uint32_t base,
                                          float* s_mul) {
  using L = PSmem<DIM>;
  constexpr int kPieces = DIM / 16;
  const Params& p = P.p;
  const int tid = threadIdx.x, ratio = p.q_heads / p.kv_heads;
  for (int x = tid; x < (g.two ? kPRows : kTile) * kPieces; x += 256) {
    const int r = x / kPieces, c = x % kPieces;  // 16 channels from 16 c
    uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (g.has_row(p, ratio, r)) {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + g.row_at(p, ratio, r) * p.q_ld +
                                                        (int64_t)g.head_at(ratio, r) * DIM + c * 16);
      v[0] = __ldg(src);
      v[1] = __ldg(src + 1);
    }
    uint32_t wds[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    float mul = fabsf(p.scale);
    if (!FP16) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        top = max(top, max(wds[i] & 0x7FFFu, (wds[i] >> 16) & 0x7FFFu));
#pragma unroll
      for (int o = kPieces / 2; o; o >>= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = (int)(top >> 7);
      const int up = e == 255 || top == 0 ? 0 : min(126, 14 - (e - 127));
      const float f = __uint_as_float((uint32_t)(up + 127) << 23);
      mul *= __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        wds[i] = pack_half(__uint_as_float(wds[i] << 16) * f,
                           __uint_as_float(wds[i] & 0xFFFF0000u) * f);
    }
    const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) wds[i] ^= flip;
    const uint32_t at = base + (r / kTile) * L::kOperand + (c >> 2) * (kTile * 128) +
                        (r % kTile) * 128;
    const int c0 = (c & 3) * 2, sw = r & 7;
    sts128(at + ((c0 ^ sw) << 4), wds[0], wds[1], wds[2], wds[3]);
    sts128(at + (((c0 + 1) ^ sw) << 4), wds[4], wds[5], wds[6], wds[7]);
    if (c == 0) s_mul[r] = mul;
  }
  proxy_fence();
}

// Warps 8-15: codes of the segment's tiles into shared memory as fp16, and the tiles' scales.
// Returns status bits.
template <int DIM>
__device__ __noinline__ int widen_tiles(const Prefix& P, const Segment& g, uint32_t base, Meta* meta,
                                        uint32_t bars, volatile int* quit) {
  using L = PSmem<DIM>;
  constexpr int kPieces = DIM / 16;  // 16-byte pieces of a row of codes
  const Params& p = P.p;
  const uint32_t k_full = bars, k_empty = bars + 16, v_full = bars + 32, v_empty = bars + 48;
  const uint32_t m_full = bars + 64;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tile0 = g.tile0, tile1 = g.tile1, eff = g.eff, h = g.h;
  const int32_t* const table = g.table;
  const uint32_t tiles_done = g.tiles_done;
  int err = 0;
  const int ww = warp - 8;
  constexpr int kKeysWarp = 32 / kPieces, kKeysPass = kWidenWarps * kKeysWarp, kPasses = kTile / kKeysPass;
  // 8 lanes that store together meet every bank once: 4 pieces of an even and an odd key
  const int piece = DIM == 128 ? (lane & 3) + 4 * ((lane >> 3) & 1) : lane & 3;
  const int key0 = ww * kKeysWarp +
                   (DIM == 128 ? ((lane >> 2) & 1) + 2 * (lane >> 4) : lane >> 2);
  const int c0 = (piece & 3) * 2;
  // Halves of tiles come by cp.async into a ring, each thread the pieces that it widens, so that
  // no thread waits for another's: keys 0, keys 1, values 0, keys 2, values 1, .. . (Loads into
  // registers go through what shared memory leaves of the L1 cache, 28 KB, which bounds what is on
  // its way.) Slots and scales come four tiles at a time, a lane for each sixteen keys.
  const int tiles = tile1 - tile0, halves = 2 * tiles;
  const int ring = g.two ? L::kSlots : L::kSlots + L::kMoreSlots;
  const uint32_t mine = (threadIdx.x - 256) * 16;
  auto place = [&](int slot) {
    return base + mine + (slot < L::kSlots ? L::kRaw + slot * L::kHalf
                                           : L::kOperand + (slot - L::kSlots) * L::kHalf);
  };
  // half x: values or keys, and of which tile
  auto values_at = [&](int x) { return x > 0 && ((x & 1) == 0 || x == halves - 1); };
  auto tile_at = [&](int x) { return values_at(x) ? (x - 1) >> 1 : (x + 1) >> 1; };
  // first slot of this lane's sixteen keys of tiles tile0 + 4 * batch .. + 3, or -1
  auto slots_of = [&](int batch) -> int {
    const int64_t tile = tile0 + 4 * (int64_t)batch + (lane >> 3);
    const int64_t pos64 = tile * kTile + (lane & 7) * 16;
    if (tile >= tile1 || pos64 >= eff) return -1;
    const int pos = (int)pos64;
    const int pg = p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page_size;
    const int32_t page = __ldg(table + pg);
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
  int slots_k = slots_of(0), slots_next = slots_of(1), slots_v = slots_k;
  float ks = 0.0f, vs = 1.0f, ks_next = 0.0f, vs_next = 1.0f;
  int at = -1, at_next = -1;  // slots of the scales
  auto scales = [&] {
    at_next = slots_k;
    if (ww == 0 && slots_k >= 0) {
      const int b = p.block_shift >= 0 ? slots_k >> p.block_shift : slots_k / p.block;
      ks_next = __ldg(p.k_scale + (int64_t)b * p.kv_heads + h);
      vs_next = __ldg(p.v_scale + (int64_t)b * p.kv_heads + h);
    }
  };
  scales();
  const int stride = p.kv_heads * DIM;
  const uint8_t *const from_k = p.k + h * DIM + piece * 16, *const from_v = p.v + h * DIM + piece * 16;
  auto load = [&](int x, int slot) {  // x rises call by call
    if (x < halves) {
      const bool values = values_at(x);
      const int tile = tile_at(x);
      if (tile > 0 && (tile & 3) == 0) {
        if (values) {
          slots_v = slots_k;
        } else {
          slots_k = slots_next;
          slots_next = slots_of((tile >> 2) + 1);
          scales();
        }
      }
      const uint8_t* from = values ? from_v : from_k;
      const int here = values ? slots_v : slots_k;
      const int lane0 = (tile & 3) * 8, left = eff - (tile0 + tile) * kTile;
      const uint32_t to = place(slot);
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int key = i * kKeysPass + key0;
        const int s = __shfl_sync(0xffffffffu, here, lane0 + (key >> 4));
        copy16(to + i * (512 * kWidenWarps), from + (int64_t)(max(s, 0) + (key & 15)) * stride, s >= 0 && key < left);
      }
    }
    copy_commit();
  };
  float ref = 0.0f, lv = 0.0f;
  bool found = false, wide = false;
#pragma unroll 1
  for (int x = 0; x < ring; ++x) load(x, x);
  int slot = 0;
#pragma unroll 1
  for (int x = 0; x < halves; ++x) {
    const bool values = values_at(x);
    const int tile = tile_at(x);
    const uint32_t t = tiles_done + tile;
    const uint32_t empty = values ? v_empty : k_empty + 8 * (t & 1);
    const uint32_t turn = values ? t : t >> 1;
    if (g.two) copy_wait<L::kSlots - 1>();
    else copy_wait<L::kSlots + L::kMoreSlots - 1>();
    if (!__all_sync(0xffffffffu, bar_wait(empty, (turn & 1) ^ 1, quit))) break;
    const uint32_t from = place(slot);
    const uint32_t to = base + (values ? L::kV : L::kK + (t & 1) * L::kOperand) +
                        (piece >> 2) * (kTile * 128);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int key = i * kKeysPass + key0;
      const uint4 c = lds128(from + i * (512 * kWidenWarps));
      uint32_t y[8];
      widen4(c.x, y[0], y[1]);
      widen4(c.y, y[2], y[3]);
      widen4(c.z, y[4], y[5]);
      widen4(c.w, y[6], y[7]);
      sts128(to + key * 128 + ((c0 ^ (key & 7)) << 4), y[0], y[1], y[2], y[3]);
      sts128(to + key * 128 + (((c0 + 1) ^ (key & 7)) << 4), y[4], y[5], y[6], y[7]);
    }
    proxy_fence();
    __syncwarp();
    if (lane == 0) {
      // values: to the stream that takes them. (One barrier for both would let a stream that
      // skips a tile take its phase for that of the tile before.)
      if (!values) bar_arrive(k_full + 8 * (t & 1));
      if (values && (g.two || (tile & 1) == 0)) bar_arrive(v_full);
      if (values && (g.two || (tile & 1) == 1)) bar_arrive(v_full + 8);
    }
    load(x + ring, slot);
    slot = slot == ring - 1 ? 0 : slot + 1;
    if (ww == 0 && !values) {
      // scales; those of four tiles before were read before this tile's place was free
      if ((tile & 3) == 0) {
        ks = ks_next;
        vs = vs_next;
        at = at_next;
        lv = log2f(vs);
      }
      const int lane0 = (tile & 3) * 8;
      const bool in = (lane & 24) == lane0 && at >= 0;
      const uint32_t fit = __ballot_sync(0xffffffffu, in && vs > 0.0f && vs <= FLT_MAX);
      if (!found && fit) {
        ref = __shfl_sync(0xffffffffu, lv, __ffs(fit) - 1);
        found = true;
      }
      wide |= __any_sync(0xffffffffu, in && !(fabsf(lv - ref) <= 8.0f));
      const uint32_t have = __ballot_sync(0xffffffffu, in) >> lane0;
      Meta& d = meta[t & 3];
      if ((lane & 24) == lane0) {
        d.ks[lane & 7] = in ? ks : 0.0f;
        d.dl[lane & 7] = in ? lv - ref : 0.0f;
        d.inv[lane & 7] = in ? exp2f(ref - lv) : 1.0f;
      }
      if (lane == 0) {
        d.ref = ref;
        d.in = have & 0xFFu;
        d.end = min(kTile, eff - (tile0 + tile) * kTile);
        d.wide = wide;
      }
      __syncwarp();
      if (lane == 0) bar_arrive(m_full + 8 * (t & 3));
    }
  }
  copy_wait<0>();
  return err;
}

// Warps 0-3 and 4-7: the streams' products and softmax, and the sums of their rows at the end.
template <int DIM>
__device__ __noinline__ void stream_rows(const Prefix& P, const Segment& g, uint32_t base,
                                         uint8_t* smem, uint32_t bars, uint32_t tmem,
                                         volatile int* quit) {
  using L = PSmem<DIM>;
  const Params& p = P.p;
  const uint32_t k_full = bars, k_empty = bars + 16, v_full = bars + 32, v_empty = bars + 48;
  const uint32_t m_full = bars + 64, s_full = bars + 96, p_ready = bars + 112, done = bars + 128;
  const uint32_t summed = bars + 136;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ratio = p.q_heads / p.kv_heads;
  const Meta* const meta = reinterpret_cast<const Meta*>(smem + L::kMeta);
  const float* const s_mul = reinterpret_cast<const float*>(smem + L::kMul);
  const bool two = g.two != 0;
  const uint32_t tiles_done = g.tiles_done;
  const int b = warp >> 2;                 // stream
  const int count = g.count[b];
  const uint32_t turns = g.turns[b];
  const int r = (warp & 3) * 32 + lane;    // row of the stream
  const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  const uint32_t t_s = t_lane + b * kTile, t_o = t_lane + 2 * kTile + b * DIM;
  const float mul = s_mul[two ? b * kTile + r : r];
  // Products of this stream, issued by its first thread: the scores of its turn j, and the
  // sums of its turn j once its four warps have their weights in place. Keys and values are
  // given back by both streams, by one of them twice where it alone had them. Scores go where the
  // weights of the turn before lie, which its sums' product reads: products with different
  // accumulators are not ordered, so they wait for it.
  constexpr uint32_t kIdS = idesc_f16(kTile, kTile, false), kIdO = idesc_f16(kTile, DIM, true);
  auto tile_at = [&](int j) { return tiles_done + (uint32_t)(two ? j : 2 * j + b); };
  auto issue_scores = [&](int j) {
    const uint32_t t = tile_at(j), st = t & 1;
    if (!bar_wait(k_full + 8 * st, (t >> 1) & 1, quit) ||
        (j > 0 && !bar_wait(summed + 8 * b, (turns + j - 1) & 1, quit)))
      return;
    tc_fence_after();
    const uint32_t q = base + (two ? b : 0) * L::kOperand, k = base + L::kK + st * L::kOperand;
#pragma unroll
    for (int i = 0; i < DIM / 16; ++i) {
      const uint32_t off = (i >> 2) * (kTile * 128) + (i & 3) * 32;
      mma_ss(tmem + b * kTile, sdesc(q + off, 16), sdesc(k + off, 16), kIdS, i > 0);
    }
    tc_commit(s_full + 8 * b);
    tc_commit(k_empty + 8 * st);
    if (!two) tc_commit(k_empty + 8 * st);
  };
  auto issue_sums = [&](int j) {
    if (!bar_wait(p_ready + 8 * b, (turns + j) & 1, quit) ||
        !bar_wait(v_full + 8 * b, (turns + j) & 1, quit))
      return;
    tc_fence_after();
    const uint32_t v = base + L::kV;
#pragma unroll
    for (int i = 0; i < kTile / 16; ++i)
      mma_ts(tmem + 2 * kTile + b * DIM, tmem + b * kTile + i * 8,
             sdesc(v + i * 2048, kTile * 128), kIdO, j > 0 || i > 0);
    tc_commit(summed + 8 * b);
    tc_commit(v_empty);
    if (!two) tc_commit(v_empty);
  };
  const bool first = (tid & 127) == 0;
  if (first && count > 0) issue_scores(0);
  __syncwarp();
  // mo: the reference of o where scales lie far apart, else m
  float m = kNone, mo = kNone, l = 0.0f, ref = 0.0f;
  bool ok = true;
  for (int j = 0; j < count; ++j) {
    const uint32_t t = tile_at(j);
    ok = bar_wait(s_full + 8 * b, (turns + j) & 1, quit) &&
         bar_wait(m_full + 8 * (t & 3), (t >> 2) & 1, quit);
    if (!__all_sync(0xffffffffu, ok)) break;
    tc_fence_after();
    // The loops over parts of a row stay rolled: their code has to stay in the instruction
    // cache beside that of the other roles
    const Meta& d = meta[t & 3];
    ref = d.ref;
    if (d.in != 0xFFu || d.end != kTile) {  // keys that are not there
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t have = (d.in >> (2 * c) & 1 ? 0xFFFFu : 0u) | (d.in >> (2 * c + 1) & 1 ? 0xFFFF0000u : 0u);
        const int left = d.end - c * 32;
        if (left < 32) have &= left <= 0 ? 0u : (1u << left) - 1;
        float v[32];
        tmem_ld(t_s + c * 32, v);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!(have >> i & 1)) v[i] = -INFINITY;
        tmem_st(t_s + c * 32, v);
      }
      tmem_st_wait();
    }
    // a score times this is x; never 0, which would make a masked -infinity NaN
    auto factor = [&](float ks) {
      const float a = mul * ks;
      return a == 0.0f ? FLT_MIN : a;
    };
    // references raised to kBelow below the maxima tm and to, sums with them
    auto raise = [&](float tm, float to, bool apart) {
      const bool up = tm > m + kRaise;
      const float top = up ? tm - kBelow : m;
      const float topo = !apart ? top : to > mo + kRaise ? to - kBelow : mo;
      l *= exp2_fast(m - top);
      const float keep = exp2_fast(mo - topo);
      m = top;
      mo = topo;
      if (j == 0) return;
      // the products of the tile before are finished: so are this tile's scores
#pragma unroll 1
      for (int c = 0; c < DIM / 32; ++c) {
        float o[32];
        tmem_ld(t_o + c * 32, o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= keep;
        tmem_st(t_o + c * 32, o);
      }
    };
    if (!d.wide) {
      // The weights by the reference as it is. If sixteen of them pass kMost, some score lies 2^kRaise
      // above it (as one of the first tile does): then the maxima are looked for, the references
      // raised and the weights taken again. Otherwise no maximum is needed.
      uint32_t w[64];
      float add;
      for (int again = j == 0;; ++again) {
        if (again > 0) {
          float tm = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            float v[16];
            tmem_ld(t_s + c * 16, v);
            float x = v[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) x = fmaxf(x, v[i]);
            tm = fmaxf(tm, fmaf(x, factor(d.ks[c]), d.dl[c]));
          }
          raise(tm, tm, false);
        }
        add = 0.0f;
        bool past = false;
        float v[2][16];
        tmem_ld_start(t_s, v[0]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float a = factor(d.ks[c]), z = d.dl[c] - m;
          const uint64_t a2 = pack2(a, a), z2 = pack2(z, z);
          uint64_t sum = pack2(0.0f, 0.0f);
          tmem_ld_wait(v[c & 1]);
          if (c < 7) tmem_ld_start(t_s + (c + 1) * 16, v[(c + 1) & 1]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 x = unpack2(fma2(pack2(v[c & 1][2 * i], v[c & 1][2 * i + 1]), a2, z2));
            const float e0 = exp2_fast(x.x), e1 = exp2_fast(x.y);
            sum = add2(sum, pack2(e0, e1));
            w[8 * c + i] = pack_half(e0, e1);
          }
          const float2 both = unpack2(sum);
          const float s16 = both.x + both.y;
          past |= s16 > kMost;
          add = fmaf(s16, d.inv[c], add);
        }
        if (again > 0 || !__any_sync(0xffffffffu, past)) break;
      }
      l += add;
      mo = m;
      tmem_st(t_s, w);
    } else {
      float tm = -INFINITY, to = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        float v[16];
        tmem_ld(t_s + c * 16, v);
        float x = v[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) x = fmaxf(x, v[i]);
        x *= factor(d.ks[c]);
        tm = fmaxf(tm, x);
        to = fmaxf(to, x + d.dl[c]);
      }
      if (__any_sync(0xffffffffu, tm > m + kRaise || to > mo + kRaise)) raise(tm, to, true);
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        const float a = factor(d.ks[c]), z = d.dl[c] - mo;
        float v[16];
        tmem_ld(t_s + c * 16, v);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          l += exp2_fast(fmaf(v[2 * i], a, -m)) + exp2_fast(fmaf(v[2 * i + 1], a, -m));
          w[i] = pack_half(exp2_fast(fmaf(v[2 * i], a, z)), exp2_fast(fmaf(v[2 * i + 1], a, z)));
        }
        tmem_st(t_s + c * 8, w);
      }
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) bar_arrive(p_ready + 8 * b);
    if (first) {
      issue_sums(j);
      if (j + 1 < count) issue_scores(j + 1);
    }
    __syncwarp();
  }
  if (first) tc_commit(done);  // all products issued above
  bar_wait_through(done, g.parity, quit);
  __syncwarp();
  tc_fence_after();
  // ---- the rows' sums, through shared memory (keys and values are done with), so that a warp
  // writes a row at a time: a thread that writes its own row takes 15 us here
  float* const meet = reinterpret_cast<float*>(smem + L::kK) + b * kTile * L::kLd;
#pragma unroll 1
  for (int c = 0; c < DIM / 32; ++c) {
    float o[32];
    if (count > 0) {
      tmem_ld(t_o + c * 32, o);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float4*>(meet + r * L::kLd + c * 32 + 4 * i) =
          make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  }
  *reinterpret_cast<float4*>(meet + r * L::kLd + DIM) = make_float4(m, mo + ref, l, 0.0f);
  // this warp's rows: its own 32, or 16 of those that the streams have together
  if (two) __syncwarp();
  else asm volatile("bar.sync 1, 256;" ::: "memory");
  const int n = two ? 32 : 16;
  const int r0 = two ? (warp & 3) * 32 : warp * 16;
  const float* const s0 =
      reinterpret_cast<const float*>(smem + L::kK) + (two ? b * kTile * L::kLd : 0) + r0 * L::kLd;
  const float* const s1 = s0 + kTile * L::kLd;  // the other stream's
  float f0 = 1.0f, f1 = 0.0f;
  float* dst = nullptr;  // of row r0 + lane; null: there is none
  if (lane < n) {
    const int ur = two ? b * kTile + r0 + lane : r0 + lane;
    if (g.has_row(p, ratio, ur)) {
      const int64_t row = g.row_at(p, ratio, ur);
      const int gr = (int)(row / p.group_rows);
      int ignored = 0;
      // a row of length 0 attends to nothing, the prefix neither
      const bool on =
          row_len(p, (int)row, p.group_table ? __ldg(p.group_table + gr) : gr, &ignored) > 0;
      dst = g.whole ? P.before + (row * p.q_heads + g.head_at(ratio, ur)) * (DIM + 4)
                    : g.part + ur * DIM;
      float4 st = *reinterpret_cast<const float4*>(s0 + lane * L::kLd + DIM);
      if (!two) {
        const float4 x = *reinterpret_cast<const float4*>(s1 + lane * L::kLd + DIM);
        const float top = fmaxf(st.x, x.x), topv = fmaxf(st.y, x.y);
        f0 = exp2_fast(st.y - topv);
        f1 = exp2_fast(x.y - topv);
        st.z = st.z * exp2_fast(st.x - top) + x.z * exp2_fast(x.x - top);
        st.x = top;
        st.y = topv;
      }
      if (!on) {
        st = make_float4(kNone, kNone, 0.0f, 0.0f);
        f0 = -1.0f;  // marks it
      }
      float* const stat = g.whole ? dst + DIM : g.part + Part<DIM, kPRows>::kStat + ur * 4;
      *reinterpret_cast<float4*>(stat) = st;
    }
  }
  constexpr int kLanes = DIM / 4;  // of a row
  const int sub = lane / kLanes, c4 = lane % kLanes;
#pragma unroll 4
  for (int i = 0; i < n; i += 32 / kLanes) {
    const int k = i + sub;
    float* const to = reinterpret_cast<float*>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), k));
    const float a = __shfl_sync(0xffffffffu, f0, k), c = __shfl_sync(0xffffffffu, f1, k);
    float4 x = *reinterpret_cast<const float4*>(s0 + k * L::kLd + c4 * 4);
    if (!two) {
      const float4 y = *reinterpret_cast<const float4*>(s1 + k * L::kLd + c4 * 4);
      x = make_float4(x.x * a + y.x * c, x.y * a + y.y * c, x.z * a + y.z * c, x.w * a + y.w * c);
    }
    if (a < 0.0f) x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (to) *reinterpret_cast<float4*>(to + c4 * 4) = x;
  }
}

// All warps, in a CTA that gave up: NaN for the unit's sums of weights, of which every row of it
// becomes NaN.
template <int DIM>
__device__ __noinline__ void void_rows(const Prefix& P, const Segment& g) {
  const Params& p = P.p;
  const int ratio = p.q_heads / p.kv_heads;
  for (int r = threadIdx.x; r < (g.two ? kPRows : kTile); r += kPThreads) {
    if (!g.has_row(p, ratio, r)) continue;
    const int64_t row = g.row_at(p, ratio, r);
    float* const stat = g.whole ? P.before + (row * p.q_heads + g.head_at(ratio, r)) * (DIM + 4) + DIM
                                : g.part + Part<DIM, kPRows>::kStat + r * 4;
    const int gr = (int)(row / p.group_rows);
    int ignored = 0;
    const bool on =  // as in stream_rows
        row_len(p, (int)row, p.group_table ? __ldg(p.group_table + gr) : gr, &ignored) > 0;
    *reinterpret_cast<float4*>(stat) = make_float4(kNone, kNone, on ? NAN : 0.0f, 0.0f);
  }
}

// ------------------------------------------------------------------ kernel
template <int DIM, bool FP16>
__global__ void __launch_bounds__(kPThreads, 1)
kv8_prefix_kernel(const __grid_constant__ Prefix P) {
  using L = PSmem<DIM>;
  const Params& p = P.p;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  Meta* const meta = reinterpret_cast<Meta*>(smem + L::kMeta);
  float* const s_mul = reinterpret_cast<float*>(smem + L::kMul);
  int64_t* const s_cum = reinterpret_cast<int64_t*>(smem + L::kCum);
  int* const s_start = reinterpret_cast<int*>(smem + L::kStart);
  int* const s_eff = reinterpret_cast<int*>(smem + L::kEff);
  int* const s_lead = reinterpret_cast<int*>(smem + L::kLead);
  int* const s_last = reinterpret_cast<int*>(smem + L::kLast);
  __shared__ uint32_t s_tmem;
  __shared__ Segment seg;
  __shared__ int s_quit, s_bad;
  volatile int* const quit = &s_quit;

  const uint32_t bars = base + L::kBars;
  // keys in place [2] and their places free [2], values in place for each stream [2] and their place
  // free, a tile's scales [4], a stream's scores [2] and weights [2], a segment's products, a
  // stream's sums [2]
  const uint32_t k_full = bars, k_empty = bars + 16, v_full = bars + 32, v_empty = bars + 48;
  const uint32_t m_full = bars + 64, s_full = bars + 96, p_ready = bars + 112, done = bars + 128;
  const uint32_t summed = bars + 136;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ratio = p.q_heads / p.kv_heads;
  int err = 0;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(k_full + 8 * i, kWidenWarps);
      bar_init(v_full + 8 * i, kWidenWarps);
      bar_init(k_empty + 8 * i, 2);
      bar_init(s_full + 8 * i, 1);
      bar_init(p_ready + 8 * i, 4);
      bar_init(summed + 8 * i, 1);
    }
    for (int i = 0; i < 4; ++i) bar_init(m_full + 8 * i, 1);
    bar_init(v_empty, 2);
    bar_init(done, 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_quit = s_bad = 0;
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s_tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // ---- the sets: where they start, and what of their prefixes is read for all
  for (int s = tid; s <= P.n_sets; s += kPThreads) s_start[s] = __ldg(P.set_starts + s);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  for (int s = tid; s < P.n_sets; s += kPThreads) {
    const int a = s_start[s], b = s_start[s + 1];
    int pre = __ldg(P.prefix_lens + s);
    if (a < 0 || b < a || b > P.groups) s_bad = 1;
    if (pre < 0 || pre > P.max_prefix) {
      err |= KV8_STATUS_SETS;
      pre = 0;
    }
    s_eff[s] = pre;
    s_lead[s] = INT32_MAX;
    s_last[s] = -1;
  }
  __syncthreads();
  const bool bad = s_bad != 0;
  if (bad) err |= KV8_STATUS_SETS;
  // the set of a group, or -1
  auto set_of = [&](int g) {
    if (bad || g < s_start[0] || g >= s_start[P.n_sets]) return -1;
    int lo = 0, hi = P.n_sets;  // s_start[lo] <= g < s_start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_start[mid] <= g) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  for (int r = tid; r < p.rows; r += kPThreads) {
    const int g = r / p.group_rows, s = set_of(g);
    int ignored = 0;  // the rows' own pass reports
    const int len = row_len(p, r, p.group_table ? __ldg(p.group_table + g) : g, &ignored);
    if (s < 0 || len == 0) continue;
    atomicMin(s_eff + s, len);
    atomicMin(s_lead + s, g);
    atomicMax(s_last + s, g);
  }
  __syncthreads();
  // rows of a set on one key head; its steps on one: pairs of 128 rows take a tile to a step,
  // 128 rows left over two
  auto rows_of = [&](int s) { return (s_start[s + 1] - s_start[s]) * p.group_rows * ratio; };
  auto tiles_in = [&](int s) { return (int)(((uint32_t)s_eff[s] + kTile - 1) / kTile); };
  auto steps_of = [&](int s) -> int64_t {
    const int m = (rows_of(s) + kTile - 1) / kTile, t = tiles_in(s);
    return (int64_t)(m >> 1) * t + (m & 1) * ((t + 1) >> 1);
  };
  for (int s = tid; s < P.n_sets; s += kPThreads)
    if (bad || s_last[s] <= s_lead[s] || s_eff[s] < kLeast) s_eff[s] = 0;
  __syncthreads();
  if (warp == 0) {  // s_cum[s]: steps of the sets before s
    int64_t run = 0;
    for (int s0 = 0; s0 < P.n_sets; s0 += 32) {
      const int64_t mine = s0 + lane < P.n_sets ? steps_of(s0 + lane) * p.kv_heads : 0;
      int64_t x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (s0 + lane < P.n_sets) s_cum[s0 + lane] = run + x - mine;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) s_cum[P.n_sets] = run;
  }
  for (int g = blockIdx.x * kPThreads + tid; g < P.groups; g += gridDim.x * kPThreads) {
    const int s = set_of(g);
    P.start[g] = s < 0 ? 0 : s_eff[s];
  }
  __syncthreads();

  // ---- this CTA's steps
  const int64_t all = s_cum[P.n_sets];
  const int64_t n = max((int64_t)1, min((int64_t)gridDim.x, (all + 1) / 2));
  const int64_t me = blockIdx.x;
  const int64_t w0 = me < n ? me * all / n : all, w1 = me < n ? (me + 1) * all / n : all;
  int set = 0;  // the set of the steps at hand, and the steps before it
  while (set + 1 < P.n_sets && s_cum[set + 1] <= w0) ++set;
  int64_t before = s_cum[set];
  __syncthreads();  // s_cum gives way to keys
  Split mine = {0, 0, 0, 0, 0, -1, {0, 0}};
  uint32_t tiles_done = 0, turns[2] = {0, 0}, segments = 0;
  bool gave_up = false;
  for (int64_t w = w0; w < w1;) {
    // ---- the segment: a unit's steps [i0, i1) of `steps`
    for (int64_t of_set; (of_set = steps_of(set) * p.kv_heads) <= w - before; ++set) before += of_set;
    const int tiles = tiles_in(set), rows = rows_of(set);
    const int pairs = ((rows + kTile - 1) / kTile) >> 1;
    const int64_t per_head = steps_of(set);
    const int64_t rel = w - before;
    const int h = (int)(rel / per_head);
    const int64_t in_head = rel - h * per_head;
    const int pair = (int)min(in_head / tiles, (int64_t)pairs);
    const bool two = pair < pairs;
    const int steps = two ? tiles : (tiles + 1) >> 1;
    const int i0 = (int)(in_head - (int64_t)pair * tiles);
    const int i1 = (int)min((int64_t)steps, i0 + (w1 - w));
    const int tile0 = two ? i0 : 2 * i0, tile1 = two ? i1 : min(2 * i1, tiles);
    const int count0 = two ? i1 - i0 : (tile1 - tile0 + 1) >> 1;
    const int count1 = two ? i1 - i0 : (tile1 - tile0) >> 1;
    const bool whole = i0 == 0 && i1 == steps;
    if (tid == 0) {
      const int lead = s_lead[set];
      seg.table = p.block_table +
                  (int64_t)(p.group_table ? __ldg(p.group_table + lead) : lead) * p.table_ld;
      seg.part = P.parts + (2 * me + (i0 == 0)) * Part<DIM, kPRows>::kFloats;
      seg.g0 = s_start[set];
      seg.h = h;
      seg.row0 = pair * kPRows;
      seg.rows = rows;
      seg.eff = s_eff[set];
      seg.tile0 = tile0;
      seg.tile1 = tile1;
      seg.two = two;
      seg.whole = whole;
      seg.count[0] = count0;
      seg.count[1] = count1;
      seg.tiles_done = tiles_done;
      seg.turns[0] = turns[0];
      seg.turns[1] = turns[1];
      seg.parity = segments & 1;
      if (i0 == 0 && !whole)  // for the join
        mine = {seg.g0, h, seg.row0, min(rows, seg.row0 + (two ? kPRows : kTile)), (int32_t)me,
                (int32_t)(((w + steps) * n - 1) / all), {0, 0}};
    }
    __syncthreads();
    if (gave_up) {
      // no unit is begun any more
    } else if (warp >= 8) {
      if (me != P.skip) err |= widen_tiles<DIM>(P, seg, base, meta, bars, quit);
    } else {  // while the first codes are on their way
      load_queries<DIM, FP16>(P, seg, base, s_mul);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      stream_rows<DIM>(P, seg, base, smem, bars, tmem, quit);
    }
    tiles_done += (uint32_t)(tile1 - tile0);
    turns[0] += (uint32_t)count0;
    turns[1] += (uint32_t)count1;
    ++segments;
    w += i1 - i0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    gave_up = *quit;  // no thread waits before the next unit's barrier: all see the same
    if (gave_up) {
      void_rows<DIM>(P, seg);
      __syncthreads();
    }
  }
  if (tid == 0) {
    P.splits[me] = mine;
    if (s_quit) err |= KV8_STATUS_TIMEOUT;
  }
  if (err && p.status) atomicOr(p.status, err);
  if (warp == 8)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
}

// Joins the parts of the split units: CTA (i, y) a share of the rows of entry i, a warp to a row.
template <int DIM>
__global__ void __launch_bounds__(kJoinWarps * 32)
kv8_prefix_join_kernel(const __grid_constant__ Prefix P) {
  constexpr int kVec = DIM / 32;
  const Params& p = P.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Split u = P.splits[blockIdx.x];
  if (u.last < 0) return;
  const int ratio = p.q_heads / p.kv_heads;
  auto part = [&](int c) {
    return P.parts + (2 * (int64_t)(u.first + c) + (c == 0)) * Part<DIM, kPRows>::kFloats;
  };
  for (int r = blockIdx.y * kJoinWarps + warp; r < u.row1 - u.row0; r += gridDim.y * kJoinWarps) {
    const int64_t row = (int64_t)u.g0 * p.group_rows + (u.row0 + r) / ratio;
    if (row >= p.rows) return;
    float top = -INFINITY, topv = -INFINITY, l = 0.0f, v[kVec] = {};
    add_parts<DIM, kPRows>(part, 0, 1, u.last - u.first + 1, r, top, topv, l, v);
    float* dst = P.before + (row * p.q_heads + u.h * ratio + (u.row0 + r) % ratio) * (DIM + 4);
#pragma unroll
    for (int i = 0; i < kVec; ++i) dst[lane * kVec + i] = v[i];
    if (lane == 0) *reinterpret_cast<float4*>(dst + DIM) = make_float4(top, topv, l, 0.0f);
  }
}

// Workspace behind that of the rows' own pass.
struct SharedWork {
  int64_t start, splits, parts, before, total;
};

SharedWork shared_work(int64_t own, int sms, int64_t rows, int q_heads, int dim, int group_rows) {
  auto up = [](int64_t x) { return (x + 255) & ~int64_t(255); };
  SharedWork w;
  w.start = up(own);
  w.splits = up(w.start + (rows + group_rows - 1) / group_rows * 4);
  w.parts = up(w.splits + sms * (int64_t)sizeof(Split));
  w.before = up(w.parts + (int64_t)sms * 2 * kPRows * (dim + 4) * 4);
  w.total = up(w.before + rows * q_heads * (dim + 4) * 4);
  return w;
}

template <int DIM, bool FP16>
int launch_prefix(const Prefix& P, int dev, cudaStream_t s) {
  const auto kernel = kv8_prefix_kernel<DIM, FP16>;
  const auto join = kv8_prefix_join_kernel<DIM>;
  constexpr int kBytes = PSmem<DIM>::kTotal;
  static std::atomic<uint64_t> ready;
  if (!(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) !=
            cudaSuccess ||
        cudaFuncSetAttribute(join, cudaFuncAttributePreferredSharedMemoryCarveout, 100) !=
            cudaSuccess)
      return KV8_ERR_CUDA;
    ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  const int grid = sm_count(dev);
  kernel<<<(unsigned)grid, kPThreads, kBytes, s>>>(P);
  if (cudaGetLastError() != cudaSuccess) return KV8_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, kPRows / kJoinWarps);  // a row to a warp
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, join, P);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KV8_OK : KV8_ERR_CUDA;
}

}  // namespace

extern "C" int64_t kv8_attention_shared_workspace_bytes(int rows, int q_heads, int kv_heads,
                                                        int dim, int group_rows) {
  if (rows < 0) return KV8_ERR_SHAPE;
  const int64_t own = kv8_attention_workspace_bytes(q_heads, kv_heads, dim, group_rows);
  if (own < 0) return own;
  const int sms = sm_count(current_device());
  if (sms < 0) return KV8_ERR_CUDA;
  return shared_work(own, sms, rows, q_heads, dim, group_rows).total;
}

namespace {

int attention_shared(
    const void* q, int64_t q_ld, int dtype, int rows, int q_heads, int kv_heads, int dim,
    float sm_scale, const int32_t* lens, int max_len, int group_rows, const int32_t* group_table,
    const int32_t* set_starts, int n_sets, const int32_t* prefix_lens, int max_prefix,
    const int32_t* block_table, int n_tables, int64_t table_ld, int page_size, int block_tokens,
    const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale, const float* v_scale,
    int64_t num_slots, void* out, int64_t out_ld, float* lse, void* workspace, int64_t ws_bytes,
    int32_t* status, kv8_stream_t stream, int skip_cta) {
  if (max_len < 0 || n_tables < 1 || table_ld < 1 || page_size < 1 || block_tokens < 16 ||
      page_size % block_tokens || num_slots % page_size || n_sets < 0 || n_sets > KV8_MAX_SETS ||
      max_prefix < 0)
    return KV8_ERR_SHAPE;
  const int err = check_common(q, q_ld, dtype, rows, q_heads, kv_heads, dim, sm_scale,
                               group_rows, block_tokens, k_cache, v_cache, k_scale, v_scale,
                               num_slots, out, out_ld, lse, workspace, status);
  if (err || rows == 0) return err;
  if (((int64_t)rows + group_rows) * (q_heads / kv_heads) >= (int64_t(1) << 31)) return KV8_ERR_SHAPE;
  if (!lens || !block_table || (n_sets && (!set_starts || !prefix_lens))) return KV8_ERR_NULL;
  if (!aligned(lens, 4) || !aligned(group_table, 4) || !aligned(block_table, 4) ||
      !aligned(set_starts, 4) || !aligned(prefix_lens, 4))
    return KV8_ERR_ALIGN;
  const int64_t own = kv8_attention_workspace_bytes(q_heads, kv_heads, dim, group_rows);
  if (own < 0) return (int)own;
  const int dev = current_device(), sms = sm_count(dev);
  if (sms < 0) return KV8_ERR_CUDA;
  const SharedWork at = shared_work(own, sms, rows, q_heads, dim, group_rows);
  if (ws_bytes < at.total) return KV8_ERR_WORKSPACE;
  const int groups = (int)(((int64_t)rows + group_rows - 1) / group_rows);
  if (n_sets == 0 || max_prefix < kLeast ||
      (double)(groups - 1) * max_prefix * kv_heads * 2.0 * dim < kWorth)
    return kv8_attention(q, q_ld, dtype, rows, q_heads, kv_heads, dim, sm_scale, lens, max_len,
                         group_rows, group_table, block_table, n_tables, table_ld, page_size,
                         block_tokens, k_cache, v_cache, k_scale, v_scale, num_slots, out, out_ld,
                         lse, workspace, own, status, stream);
  Params p = common(q, q_ld, rows, q_heads, kv_heads, sm_scale, block_tokens, k_cache, v_cache,
                    k_scale, v_scale, num_slots, out, out_ld, lse, status);
  p.lens = lens;
  p.max_len = max_len;
  p.group_rows = group_rows;
  p.group_table = group_table;
  p.block_table = block_table;
  p.n_tables = n_tables;
  p.table_ld = table_ld;
  p.page_size = page_size;
  p.page_shift = shift_of(page_size);
  cudaStream_t s = (cudaStream_t)stream;
  char* const ws = reinterpret_cast<char*>(workspace);
  Prefix P = {};
  P.p = p;
  P.set_starts = set_starts;
  P.n_sets = n_sets;
  P.prefix_lens = prefix_lens;
  P.max_prefix = max_prefix;
  P.groups = groups;
  P.start = reinterpret_cast<int32_t*>(ws + at.start);
  P.splits = reinterpret_cast<Split*>(ws + at.splits);
  P.parts = reinterpret_cast<float*>(ws + at.parts);
  P.before = reinterpret_cast<float*>(ws + at.before);
  P.skip = skip_cta;
  const int code = dim == 128 ? dtype == KV8_FP16 ? launch_prefix<128, true>(P, dev, s)
                                                  : launch_prefix<128, false>(P, dev, s)
                   : dtype == KV8_FP16 ? launch_prefix<64, true>(P, dev, s)
                                       : launch_prefix<64, false>(P, dev, s);
  if (code) return code;
  p.start = P.start;
  p.before = P.before;
  return run<false, true>(p, dim, dtype, workspace, own, s);
}

}  // namespace

extern "C" int kv8_attention_shared(
    const void* q, int64_t q_ld, int dtype, int rows, int q_heads, int kv_heads, int dim,
    float sm_scale, const int32_t* lens, int max_len, int group_rows, const int32_t* group_table,
    const int32_t* set_starts, int n_sets, const int32_t* prefix_lens, int max_prefix,
    const int32_t* block_table, int n_tables, int64_t table_ld, int page_size, int block_tokens,
    const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale, const float* v_scale,
    int64_t num_slots, void* out, int64_t out_ld, float* lse, void* workspace, int64_t ws_bytes,
    int32_t* status, kv8_stream_t stream) {
  return attention_shared(q, q_ld, dtype, rows, q_heads, kv_heads, dim, sm_scale, lens, max_len,
                          group_rows, group_table, set_starts, n_sets, prefix_lens, max_prefix,
                          block_table, n_tables, table_ld, page_size, block_tokens, k_cache,
                          v_cache, k_scale, v_scale, num_slots, out, out_ld, lse, workspace,
                          ws_bytes, status, stream, -1);
}

extern "C" int kv8_attention_shared_test(
    const void* q, int64_t q_ld, int dtype, int rows, int q_heads, int kv_heads, int dim,
    float sm_scale, const int32_t* lens, int max_len, int group_rows, const int32_t* group_table,
    const int32_t* set_starts, int n_sets, const int32_t* prefix_lens, int max_prefix,
    const int32_t* block_table, int n_tables, int64_t table_ld, int page_size, int block_tokens,
    const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale, const float* v_scale,
    int64_t num_slots, void* out, int64_t out_ld, float* lse, void* workspace, int64_t ws_bytes,
    int32_t* status, kv8_stream_t stream, int skip_cta) {
  return attention_shared(q, q_ld, dtype, rows, q_heads, kv_heads, dim, sm_scale, lens, max_len,
                          group_rows, group_table, set_starts, n_sets, prefix_lens, max_prefix,
                          block_table, n_tables, table_ld, page_size, block_tokens, k_cache,
                          v_cache, k_scale, v_scale, num_slots, out, out_ld, lse, workspace,
                          ws_bytes, status, stream, skip_cta);
}
