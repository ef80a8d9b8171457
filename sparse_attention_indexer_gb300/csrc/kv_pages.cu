// Ownership and data of cache pages: reserve, fork, free, compact, copy (rules in
// include/kv_pages.h).
//
// Two kinds of work. The tables and counts are a few integers per page: fork and free are
// one CTA per row with integer atomics on the counts (their results do not depend on the
// order), reserve and compact need the free ids in order and take one CTA for that (the
// plan), which scans the counts 16 bytes a thread. The data is a list of (source, destination)
// pages that the plan writes to the workspace, and one copy kernel moves it: HBM-bound, every
// byte read once and written once, 32 KB of a plane's page to a CTA at a time with 128 bytes of each
// thread on their way (1251 pages of 139 KB: 60 us, 5.8 TB/s; 66 us with 16 KB and a CTA for each
// small plane). The plan of a pool of 16384 pages takes 8 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "kv_pages.h"

namespace {

constexpr int kCopyThreads = 256;
constexpr int kItemBytes = 32768;  // one CTA's unit of copy work
constexpr int kSmallBytes = 2048;  // planes up to this size a page share one unit, a warp each
constexpr int kPlanThreads = 1024;
constexpr int kRowThreads = 256;

// The planes above kSmallBytes first.
struct Planes {
  int n, large;
  char* base[KVPAGES_MAX_PLANES];
  int64_t bytes[KVPAGES_MAX_PLANES];
  int32_t first[KVPAGES_MAX_PLANES + 1];  // items of a page before each large plane
  int items;                              // of a page: the small planes are the last one
};

// Workspace: counts[16] | need[n] | offset[n] | pair_src[m] | pair_dst[m] | free[P] |
// item_row[P] | item_col[P], all int32, m = max(n, P / 2 + 1).
struct Work {
  int32_t *counts, *need, *offset, *src, *dst, *free, *row, *col;
};

__host__ __device__ inline int64_t pair_cap(int64_t n, int64_t pages) {
  return n > pages / 2 + 1 ? n : pages / 2 + 1;
}

Work layout(void* ws, int64_t n, int64_t pages) {
  int32_t* w = reinterpret_cast<int32_t*>(ws);
  const int64_t m = pair_cap(n, pages);
  Work r;
  r.counts = w;
  r.need = w + 16;
  r.offset = r.need + n;
  r.src = r.offset + n;
  r.dst = r.src + m;
  r.free = r.dst + m;
  r.row = r.free + pages;
  r.col = r.row + pages;
  return r;
}

__device__ __forceinline__ void report(int32_t* status, int bit) {
  if (status) atomicOr(status, bit);
}

// ------------------------------------------------------------------ copy
// Items are handed out round-robin: item = pair * p.items + j, j running over the planes' pieces
// of kItemBytes.
__device__ __forceinline__ bool by_16(const void* base, int64_t bytes) {
  return ((reinterpret_cast<uintptr_t>(base) | (uintptr_t)bytes) & 15) == 0;
}

__device__ __forceinline__ void copy_item(const Planes& p, int64_t src, int64_t dst, int j) {
  if (j == p.first[p.large]) {  // the small planes
    const int lane = threadIdx.x & 31;
    for (int i = p.large + (threadIdx.x >> 5); i < p.n; i += kCopyThreads / 32) {
      const int n = (int)p.bytes[i];
      const char* s = p.base[i] + src * n;
      char* d = p.base[i] + dst * n;
      if (by_16(p.base[i], n)) {
        for (int o = lane * 16; o < n; o += 512)
          *reinterpret_cast<uint4*>(d + o) = *reinterpret_cast<const uint4*>(s + o);
      } else {
        for (int o = lane * 4; o < n; o += 128)
          *reinterpret_cast<uint32_t*>(d + o) = *reinterpret_cast<const uint32_t*>(s + o);
      }
    }
    return;
  }
  int lo = 0, hi = p.large;  // the plane whose items hold j
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.first[mid] <= j) lo = mid;
    else hi = mid;
  }
  const int64_t bytes = p.bytes[lo];
  const int64_t at = (int64_t)(j - p.first[lo]) * kItemBytes;
  const int n = (int)(bytes - at < kItemBytes ? bytes - at : kItemBytes);
  const char* s = p.base[lo] + src * bytes + at;
  char* d = p.base[lo] + dst * bytes + at;
  if (by_16(p.base[lo], bytes)) {
    constexpr int kVec = kItemBytes / 16 / kCopyThreads;
    uint4 v[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int o = (i * kCopyThreads + threadIdx.x) * 16;
      if (o < n) v[i] = __ldcs(reinterpret_cast<const uint4*>(s + o));
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int o = (i * kCopyThreads + threadIdx.x) * 16;
      if (o < n) __stcs(reinterpret_cast<uint4*>(d + o), v[i]);
    }
  } else {
    for (int o = threadIdx.x * 4; o < n; o += kCopyThreads * 4)
      *reinterpret_cast<uint32_t*>(d + o) = *reinterpret_cast<const uint32_t*>(s + o);
  }
}

__global__ void __launch_bounds__(kCopyThreads)
copy_pairs_kernel(const __grid_constant__ Planes p, const int32_t* src, const int32_t* dst, int n,
                  int num_pages, int32_t* status) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the plan, where there is one
  const int64_t per = p.items;
  for (int64_t item = blockIdx.x; item < n * per; item += gridDim.x) {
    const int64_t i = item / per;
    const int j = (int)(item - i * per);
    const int32_t a = src[i], b = dst[i];
    if (a < 0 && b < 0) continue;
    if (a < 0 || b < 0 || a >= num_pages || b >= num_pages) {
      if (j == 0 && threadIdx.x == 0) report(status, KVPAGES_STATUS_PAGE);
      continue;
    }
    copy_item(p, a, b, j);
  }
}

// ------------------------------------------------------------------ fork and free
__global__ void __launch_bounds__(kRowThreads)
fork_kernel(const int32_t* parents, const int32_t* children, const int32_t* lens,
            int32_t* table, int n_tables, int64_t ld, int page_size, int32_t* refs, int num_pages,
            int32_t* status) {
  const int i = blockIdx.x;
  const int from = parents[i], to = children[i], len = lens[i];
  if (from < 0 || from >= n_tables || to < 0 || to >= n_tables) {
    if (threadIdx.x == 0) report(status, KVPAGES_STATUS_ROW);
    return;
  }
  const int64_t pages = len <= 0 ? 0 : ((int64_t)len + page_size - 1) / page_size;
  if (len < 0 || pages > ld) {
    if (threadIdx.x == 0) report(status, KVPAGES_STATUS_LEN);
    return;
  }
  const int32_t* a = table + from * ld;
  int32_t* b = table + to * ld;
  int held = 0;
  for (int64_t c = threadIdx.x; c < ld; c += kRowThreads) held |= b[c] >= 0;
  if (__syncthreads_or(held)) {
    if (threadIdx.x == 0) report(status, KVPAGES_STATUS_CHILD);
    return;
  }
  for (int64_t c = threadIdx.x; c < pages; c += kRowThreads) {
    int32_t e = a[c];
    if (e >= num_pages) {
      report(status, KVPAGES_STATUS_PAGE);
      e = -1;
    }
    b[c] = e;
    if (e >= 0) atomicAdd(refs + e, 1);
  }
}

__global__ void __launch_bounds__(kRowThreads)
free_kernel(const int32_t* rows, const int32_t* keep, int32_t* table, int n_tables, int64_t ld,
            int page_size, int32_t* refs, int num_pages, int32_t* status) {
  const int i = blockIdx.x;
  const int row = rows[i], len = keep ? keep[i] : 0;
  if (row < 0 || row >= n_tables) {
    if (threadIdx.x == 0) report(status, KVPAGES_STATUS_ROW);
    return;
  }
  const int64_t pages = len <= 0 ? 0 : ((int64_t)len + page_size - 1) / page_size;
  if (len < 0) {
    if (threadIdx.x == 0) report(status, KVPAGES_STATUS_LEN);
    return;
  }
  int32_t* a = table + row * ld;
  for (int64_t c = pages + threadIdx.x; c < ld; c += kRowThreads) {
    const int32_t e = a[c];
    if (e < 0) continue;
    a[c] = -1;
    if (e >= num_pages) {
      report(status, KVPAGES_STATUS_PAGE);
    } else if (atomicSub(refs + e, 1) <= 0) {
      atomicAdd(refs + e, 1);
      report(status, KVPAGES_STATUS_REFS);
    }
  }
}

// ------------------------------------------------------------------ plans (one CTA)
// Exclusive prefix of v over the CTA's threads; *total gets the sum. Two barriers; the
// shared array may be used again after the next call's first barrier.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* s_warp, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  T before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const T t = s_warp[w];
    if (w < warp) before += t;
    sum += t;
  }
  *total = sum;
  return before + x - v;
}

// A round of a scan over the pages: warp w looks at 512 of them, its lanes at 4 consecutive
// ones of each quarter k, so that loads and stores of 16 bytes to a lane are contiguous.
constexpr int kQuarters = 4;
constexpr int kRound = kPlanThreads * 4 * kQuarters;

__device__ __forceinline__ int64_t first_of(int64_t round, int k) {
  return round + (threadIdx.x >> 5) * (128 * kQuarters) + k * 128 + (threadIdx.x & 31) * 4;
}

// The counts of pages [first, first + 4), -1 past the end.
__device__ __forceinline__ int4 load_counts(const int32_t* refs, int64_t first, int num_pages) {
  if (first + 4 <= num_pages && (reinterpret_cast<uintptr_t>(refs) & 15) == 0)
    return *reinterpret_cast<const int4*>(refs + first);
  int4 v = make_int4(-1, -1, -1, -1);
  if (first < num_pages) v.x = refs[first];
  if (first + 1 < num_pages) v.y = refs[first + 1];
  if (first + 2 < num_pages) v.z = refs[first + 2];
  if (first + 3 < num_pages) v.w = refs[first + 3];
  return v;
}

// Of the flagged pages of a round (flags[k]: 4 bits), how many come before this lane's of each
// quarter; *total gets their number. The quarters' counts are scanned together, a byte each
// (at most 128 to a warp).
__device__ __forceinline__ void ranks(const uint32_t (&flags)[kQuarters], int (&before)[kQuarters],
                                      int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t mine = 0;
#pragma unroll
  for (int k = 0; k < kQuarters; ++k) mine |= (uint32_t)__popc(flags[k]) << (8 * k);
  uint32_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  const uint32_t all = __shfl_sync(0xffffffffu, x, 31);
  x -= mine;
  int sum = 0;
#pragma unroll
  for (int k = 0; k < kQuarters; ++k) {
    before[k] = sum + (int)((x >> (8 * k)) & 0xFF);
    sum += (int)((all >> (8 * k)) & 0xFF);
  }
  __syncthreads();
  if (lane == 0) s_warp[warp] = sum;
  __syncthreads();
  // every warp sums the warps before it
  const int w = s_warp[lane];
  int upto = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  *total = __shfl_sync(0xffffffffu, upto, 31);
  const int base = __shfl_sync(0xffffffffu, upto - w, warp);
#pragma unroll
  for (int k = 0; k < kQuarters; ++k) before[k] += base;
}

// Pages of [old, new) that row `row` needs, lane by lane in order. `page(c, rank)` is
// called for each needed column c with its rank; returns their number. Whole warp.
template <typename F>
__device__ __forceinline__ int row_needs(const int32_t* a, int64_t first, int64_t last,
                                         const int32_t* refs, int num_pages, int32_t* status,
                                         F&& page) {
  const int lane = threadIdx.x & 31;
  int total = 0;
  for (int64_t c0 = first; c0 < last; c0 += 32) {
    const int64_t c = c0 + lane;
    bool need = false;
    if (c < last) {
      const int32_t e = a[c];
      if (e >= num_pages) report(status, KVPAGES_STATUS_PAGE);
      else need = e < 0 || refs[e] > 1;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, need);
    if (need) page(c, total + __popc(m & ((1u << lane) - 1)));
    total += __popc(m);
  }
  return total;
}

__global__ void __launch_bounds__(kPlanThreads)
reserve_plan_kernel(const int32_t* rows, const int32_t* old_lens, const int32_t* new_lens, int n,
                    int32_t* table, int n_tables, int64_t ld, int page_size, int32_t* refs,
                    int num_pages, Work w, int32_t* status) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ int64_t s_warp64[kPlanThreads / 32];
  __shared__ int32_t s_free[2 * kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // the pages of row i's span; [0, 0) where there is none
  auto span = [&](int i, int64_t* first, int64_t* last) {
    *first = *last = 0;
    const int row = rows[i], a = old_lens[i], b = new_lens[i];
    if (row < 0 || row >= n_tables) return (int)KVPAGES_STATUS_ROW;
    const int64_t end = ((int64_t)b + page_size - 1) / page_size;
    if (a < 0 || b < a || end > ld) return (int)KVPAGES_STATUS_LEN;
    if (b > a) {
      *first = a / page_size;
      *last = end;
    }
    return 0;
  };
  // The lowest free ids in order, `store(k, id)` for the k-th, until `total` are found.
  auto find_free = [&](int64_t total, auto&& store) {
    int found = 0;
    for (int64_t p0 = 0; p0 < num_pages && found < total; p0 += kRound) {
      uint32_t flags[kQuarters];
#pragma unroll
      for (int k = 0; k < kQuarters; ++k) {
        const int4 r = load_counts(refs, first_of(p0, k), num_pages);
        flags[k] = (r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3;
      }
      int before[kQuarters], sum;
      ranks(flags, before, s_warp, &sum);
#pragma unroll
      for (int k = 0; k < kQuarters; ++k) {
        int at = found + before[k];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (flags[k] >> i & 1) store(at++, (int32_t)(first_of(p0, k) + i));
      }
      found += sum;
    }
    __syncthreads();
    return found;
  };

  // Decode and verify steps: a row to a thread, two pages to a row at most. What a row needs stays
  // in its thread's registers and the free ids in shared memory, so that tables and counts
  // are read once (free, fork and reserve of 8 rows: 18.9 us, 21.5 us by the way below).
  if (n <= kPlanThreads) {
    int64_t first = 0, last = 0;
    int bad = 0;
    if (tid < n) bad = span(tid, &first, &last);
    if (__syncthreads_and(last - first <= 2)) {
      if (bad) report(status, bad);
      int32_t* const a = table + (first < last ? rows[tid] * ld : 0);
      const int64_t old = tid < n ? old_lens[tid] : 0;
      int32_t was[2];
      bool need[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        need[k] = false;
        if (first + k < last) {
          was[k] = a[first + k];
          if (was[k] >= num_pages) report(status, KVPAGES_STATUS_PAGE);
          else need[k] = was[k] < 0 || refs[was[k]] > 1;
        }
      }
      const int mine = need[0] + need[1];
      int total;
      int at = block_scan(mine, s_warp, &total);
      const int found = find_free(total, [&](int k, int32_t id) {
        if (k < 2 * kPlanThreads) s_free[k] = id;
      });
      int32_t from = -1, to = -1;
      if (mine && at + mine > found) {
        report(status, KVPAGES_STATUS_NO_PAGE);
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (!need[k]) continue;
          const int32_t id = s_free[at++];
          if (was[k] >= 0) {
            atomicSub(refs + was[k], 1);
            if ((first + k) * page_size < old) {  // only the page of position old - 1
              from = was[k];
              to = id;
            }
          }
          a[first + k] = id;
          refs[id] = 1;
        }
      }
      if (tid < n) {
        w.src[tid] = from;
        w.dst[tid] = to;
      }
      return;
    }
  }

  // 1: how many pages each row needs
  for (int i = warp; i < n; i += kPlanThreads / 32) {
    int64_t first, last;
    const int err = span(i, &first, &last);
    if (err && lane == 0) report(status, err);
    const int need = row_needs(table + (first < last ? rows[i] * ld : 0), first, last, refs,
                               num_pages, status, [](int64_t, int) {});
    if (lane == 0) w.need[i] = need;
  }
  __syncthreads();
  // 2: offsets in the order of the rows, held at INT_MAX where they would pass it (no row
  // behind that point can be served)
  int64_t total = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int64_t v = i0 + tid < n ? w.need[i0 + tid] : 0;
    int64_t sum;
    const int64_t before = block_scan(v, s_warp64, &sum);
    if (i0 + tid < n) w.offset[i0 + tid] = (int32_t)min(total + before, (int64_t)INT32_MAX);
    total += sum;
  }
  // 3: the lowest free ids, until there are enough
  const int found = find_free(total, [&](int k, int32_t id) { w.free[k] = id; });
  // 4: the list of needed pages of the rows that can be served (nothing is changed yet: the
  // needs of one row read counts that serving another changes)
  for (int i = warp; i < n; i += kPlanThreads / 32) {
    const int need = w.need[i], off = w.offset[i];
    int64_t first, last;
    span(i, &first, &last);
    if (lane == 0) w.src[i] = w.dst[i] = -1;
    if (need == 0) continue;
    if ((int64_t)off + need > found) {
      if (lane == 0) report(status, KVPAGES_STATUS_NO_PAGE);
      continue;
    }
    row_needs(table + rows[i] * ld, first, last, refs, num_pages, nullptr,
              [&](int64_t c, int rank) {
                w.row[off + rank] = i;
                w.col[off + rank] = (int32_t)c;
              });
  }
  // the served rows are a prefix of those with needs: the items are [0, served)
  __syncthreads();
  int served = 0;
  for (int i = tid; i < n; i += kPlanThreads)
    if ((int64_t)w.offset[i] + w.need[i] <= found)
      served = max(served, w.offset[i] + w.need[i]);
  __shared__ int s_served;
  if (tid == 0) s_served = 0;
  __syncthreads();
  atomicMax(&s_served, served);
  __syncthreads();
  served = s_served;
  // 5: hand the pages out
  for (int x = tid; x < served; x += kPlanThreads) {
    const int i = w.row[x], c = w.col[x], id = w.free[x];
    int32_t* at = table + rows[i] * ld + c;
    const int32_t was = *at;
    if (was >= 0) {
      atomicSub(refs + was, 1);
      if ((int64_t)c * page_size < old_lens[i]) {  // only the page of position old - 1
        w.src[i] = was;
        w.dst[i] = id;
      }
    }
    *at = id;
    refs[id] = 1;
  }
}

__global__ void __launch_bounds__(kPlanThreads)
compact_plan_kernel(int32_t* refs, int num_pages, Work w, int32_t* new_ids, int32_t* counts) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int s_warp[kPlanThreads / 32];
  const int tid = threadIdx.x;
  int mine = 0;
  for (int64_t p0 = 0; p0 < num_pages; p0 += kRound)
#pragma unroll
    for (int k = 0; k < kQuarters; ++k) {
      const int4 r = load_counts(refs, first_of(p0, k), num_pages);
      mine += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
    }
  int live;
  block_scan(mine, s_warp, &live);
  int holes = 0, movers = 0;
  for (int64_t p0 = 0; p0 < num_pages; p0 += kRound) {
    uint32_t hole[kQuarters], mover[kQuarters];
#pragma unroll
    for (int k = 0; k < kQuarters; ++k) {
      const int64_t first = first_of(p0, k);
      const int4 v = load_counts(refs, first, num_pages);
      const int32_t r[4] = {v.x, v.y, v.z, v.w};
      int32_t id[4];
      hole[k] = mover[k] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = first + i < num_pages, used = r[i] > 0;
        id[i] = used ? (int32_t)(first + i) : -1;
        if (in && used && first + i >= live) mover[k] |= 1u << i;
        if (in && !used && first + i < live) hole[k] |= 1u << i;
      }
      if (first + 4 <= num_pages && (reinterpret_cast<uintptr_t>(new_ids) & 15) == 0) {
        *reinterpret_cast<int4*>(new_ids + first) = make_int4(id[0], id[1], id[2], id[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (first + i < num_pages) new_ids[first + i] = id[i];
      }
    }
    int before[kQuarters], sum;
    ranks(hole, before, s_warp, &sum);
#pragma unroll
    for (int k = 0; k < kQuarters; ++k) {
      int at = holes + before[k];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (hole[k] >> i & 1) w.dst[at++] = (int32_t)(first_of(p0, k) + i);
    }
    holes += sum;
    ranks(mover, before, s_warp, &sum);
#pragma unroll
    for (int k = 0; k < kQuarters; ++k) {
      int at = movers + before[k];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (mover[k] >> i & 1) w.src[at++] = (int32_t)(first_of(p0, k) + i);
    }
    movers += sum;
  }
  __syncthreads();
#pragma unroll 4
  for (int i = tid; i < movers; i += kPlanThreads) {  // as many holes as movers
    const int a = w.src[i], b = w.dst[i];
    new_ids[a] = b;
    refs[b] = refs[a];
    refs[a] = 0;
  }
  if (tid == 0) {
    w.counts[0] = movers;
    if (counts) {
      counts[0] = live;
      counts[1] = movers;
    }
  }
}

// The data of the moved pages, and every table entry's new id.
__global__ void __launch_bounds__(kCopyThreads)
compact_move_kernel(const __grid_constant__ Planes p, Work w, int num_pages, int32_t* table,
                    int64_t entries, const int32_t* new_ids, int32_t* status) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the plan
  const int64_t per = p.items;
  const int64_t items = (int64_t)w.counts[0] * per;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t i = item / per;
    copy_item(p, w.src[i], w.dst[i], (int)(item - i * per));
  }
  for (int64_t c = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; c < entries;
       c += (int64_t)gridDim.x * kCopyThreads) {
    const int32_t e = table[c];
    if (e < 0) continue;
    if (e >= num_pages) {
      report(status, KVPAGES_STATUS_PAGE);
      continue;
    }
    const int32_t to = new_ids[e];
    if (to < 0) report(status, KVPAGES_STATUS_REFS);
    else if (to != e) table[c] = to;
  }
}

// ------------------------------------------------------------------ host
bool aligned(const void* q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) % a) == 0; }

int copy_grid(int64_t items) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return -1;
  const int64_t most = (int64_t)sms * 8;
  return (int)(items < 1 ? 1 : items < most ? items : most);
}

int make_planes(const kvpages_plane* planes, int n, Planes* p) {
  if (n < 0 || n > KVPAGES_MAX_PLANES) return KVPAGES_ERR_SHAPE;
  if (n > 0 && !planes) return KVPAGES_ERR_NULL;
  for (int i = 0; i < n; ++i) {
    if (planes[i].page_bytes < 4 || (planes[i].page_bytes & 3)) return KVPAGES_ERR_SHAPE;
    if (!planes[i].base) return KVPAGES_ERR_NULL;
    if (!aligned(planes[i].base, 4)) return KVPAGES_ERR_ALIGN;
  }
  p->n = n;
  int64_t items = 0;
  int at = 0;
  for (int small = 0; small < 2; ++small) {
    for (int i = 0; i < n; ++i) {
      if ((planes[i].page_bytes <= kSmallBytes) != (small == 1)) continue;
      p->base[at] = reinterpret_cast<char*>(planes[i].base);
      p->bytes[at] = planes[i].page_bytes;
      p->first[at] = (int32_t)items;
      ++at;
      if (!small) items += (planes[i].page_bytes + kItemBytes - 1) / kItemBytes;
      if (items > (int64_t(1) << 30)) return KVPAGES_ERR_SHAPE;
    }
    if (!small) {
      p->large = at;
      p->first[at] = (int32_t)items;
    }
  }
  p->first[p->large] = (int32_t)items;
  p->items = (int)items + (p->large < n);
  return KVPAGES_OK;
}

bool table_ok(int n, int n_tables, int64_t ld, int page_size, int num_pages) {
  return n >= 0 && n_tables >= 1 && ld >= 1 && ld < (int64_t(1) << 31) && page_size >= 1 &&
         num_pages >= 0;
}

// A launch that may be set up while the plan before it still runs; the kernel waits for its end.
template <typename... Args, typename... Given>
int launch_after(void (*kernel)(Args...), int grid, cudaStream_t s, Given... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Args>(args)...);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KVPAGES_OK : KVPAGES_ERR_CUDA;
}

int launched() { return cudaGetLastError() == cudaSuccess ? KVPAGES_OK : KVPAGES_ERR_CUDA; }

}  // namespace

extern "C" size_t kvpages_workspace_bytes(int n, int num_pages) {
  if (n < 0 || num_pages < 0) return 0;
  const size_t ints = 16 + 2 * (size_t)n + 2 * (size_t)pair_cap(n, num_pages) +
                      3 * (size_t)num_pages;
  return (ints * 4 + 255) & ~size_t(255);
}

extern "C" int kvpages_reserve(const int32_t* rows, const int32_t* old_lens,
                               const int32_t* new_lens, int n, int32_t* block_table,
                               int n_tables, int64_t table_ld, int page_size, int32_t* refs,
                               int num_pages, const kvpages_plane* planes, int n_planes,
                               void* workspace, size_t ws_bytes, int32_t* status,
                               kvpages_stream_t stream) {
  if (!table_ok(n, n_tables, table_ld, page_size, num_pages)) return KVPAGES_ERR_SHAPE;
  Planes p;
  const int err = make_planes(planes, n_planes, &p);
  if (err) return err;
  if (n == 0) return KVPAGES_OK;
  if (!rows || !old_lens || !new_lens || !block_table || (num_pages && !refs) || !workspace)
    return KVPAGES_ERR_NULL;
  if (!aligned(rows, 4) || !aligned(old_lens, 4) || !aligned(new_lens, 4) ||
      !aligned(block_table, 4) || !aligned(refs, 4) || !aligned(status, 4) ||
      !aligned(workspace, 16))
    return KVPAGES_ERR_ALIGN;
  if (ws_bytes < kvpages_workspace_bytes(n, num_pages)) return KVPAGES_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  const Work w = layout(workspace, n, num_pages);
  const int64_t items = (int64_t)n * p.items;
  const int grid = copy_grid(items);
  if (grid < 0) return KVPAGES_ERR_CUDA;
  reserve_plan_kernel<<<1, kPlanThreads, 0, s>>>(rows, old_lens, new_lens, n, block_table,
                                                 n_tables, table_ld, page_size, refs, num_pages,
                                                 w, status);
  const int code = launched();
  if (code || items == 0) return code;
  return launch_after(copy_pairs_kernel, grid, s, p, w.src, w.dst, n, num_pages, nullptr);
}

extern "C" int kvpages_fork(const int32_t* parents, const int32_t* children, const int32_t* lens,
                            int n, int32_t* block_table, int n_tables, int64_t table_ld,
                            int page_size, int32_t* refs, int num_pages, int32_t* status,
                            kvpages_stream_t stream) {
  if (!table_ok(n, n_tables, table_ld, page_size, num_pages)) return KVPAGES_ERR_SHAPE;
  if (n == 0) return KVPAGES_OK;
  if (!parents || !children || !lens || !block_table || (num_pages && !refs))
    return KVPAGES_ERR_NULL;
  if (!aligned(parents, 4) || !aligned(children, 4) || !aligned(lens, 4) ||
      !aligned(block_table, 4) || !aligned(refs, 4) || !aligned(status, 4))
    return KVPAGES_ERR_ALIGN;
  fork_kernel<<<n, kRowThreads, 0, (cudaStream_t)stream>>>(parents, children, lens, block_table,
                                                          n_tables, table_ld, page_size, refs,
                                                          num_pages, status);
  return launched();
}

extern "C" int kvpages_free(const int32_t* rows, const int32_t* keep_lens, int n,
                            int32_t* block_table, int n_tables, int64_t table_ld, int page_size,
                            int32_t* refs, int num_pages, int32_t* status,
                            kvpages_stream_t stream) {
  if (!table_ok(n, n_tables, table_ld, page_size, num_pages)) return KVPAGES_ERR_SHAPE;
  if (n == 0) return KVPAGES_OK;
  if (!rows || !block_table || (num_pages && !refs)) return KVPAGES_ERR_NULL;
  if (!aligned(rows, 4) || !aligned(keep_lens, 4) || !aligned(block_table, 4) ||
      !aligned(refs, 4) || !aligned(status, 4))
    return KVPAGES_ERR_ALIGN;
  free_kernel<<<n, kRowThreads, 0, (cudaStream_t)stream>>>(rows, keep_lens, block_table, n_tables,
                                                          table_ld, page_size, refs, num_pages,
                                                          status);
  return launched();
}

extern "C" int kvpages_compact(int32_t* block_table, int n_tables, int64_t table_ld,
                               int32_t* refs, int num_pages, const kvpages_plane* planes,
                               int n_planes, int32_t* new_ids, int32_t* counts, void* workspace,
                               size_t ws_bytes, int32_t* status, kvpages_stream_t stream) {
  if (!table_ok(0, n_tables, table_ld, 1, num_pages)) return KVPAGES_ERR_SHAPE;
  Planes p;
  const int err = make_planes(planes, n_planes, &p);
  if (err) return err;
  if (!block_table || !workspace || (num_pages && (!refs || !new_ids))) return KVPAGES_ERR_NULL;
  if (!aligned(block_table, 4) || !aligned(refs, 4) || !aligned(new_ids, 4) ||
      !aligned(counts, 4) || !aligned(status, 4) || !aligned(workspace, 16))
    return KVPAGES_ERR_ALIGN;
  if (ws_bytes < kvpages_workspace_bytes(0, num_pages)) return KVPAGES_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  const Work w = layout(workspace, 0, num_pages);
  const int64_t entries = (int64_t)n_tables * table_ld;
  const int64_t items = (int64_t)(num_pages / 2 + 1) * p.items;
  const int grid = copy_grid(items > entries / kCopyThreads ? items : entries / kCopyThreads);
  if (grid < 0) return KVPAGES_ERR_CUDA;
  compact_plan_kernel<<<1, kPlanThreads, 0, s>>>(refs, num_pages, w, new_ids, counts);
  const int code = launched();
  if (code) return code;
  return launch_after(compact_move_kernel, grid, s, p, w, num_pages, block_table, entries, new_ids,
                      status);
}

extern "C" int kvpages_copy(const int32_t* src, const int32_t* dst, int n, int num_pages,
                            const kvpages_plane* planes, int n_planes, int32_t* status,
                            kvpages_stream_t stream) {
  if (n < 0 || num_pages < 0) return KVPAGES_ERR_SHAPE;
  Planes p;
  const int err = make_planes(planes, n_planes, &p);
  if (err) return err;
  const int64_t items = (int64_t)n * p.items;
  if (items == 0) return KVPAGES_OK;
  if (!src || !dst) return KVPAGES_ERR_NULL;
  if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(status, 4)) return KVPAGES_ERR_ALIGN;
  const int grid = copy_grid(items);
  if (grid < 0) return KVPAGES_ERR_CUDA;
  copy_pairs_kernel<<<grid, kCopyThreads, 0, (cudaStream_t)stream>>>(p, src, dst, n, num_pages,
                                                                     status);
  return launched();
}
