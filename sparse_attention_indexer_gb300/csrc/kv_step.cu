// The places of a step's new tokens, and the prefix that block tables share (rules in
// include/kv_pages.h).
//
// Both are integer look-ups, bound by the latency of a few dependent loads where they are small
// and by what they write or read where they are large.
//
// step: every CTA sums the requests' counts for itself (4096 at a time, 16 to a thread, kept as
// running sums in shared memory) and fills its own range of tokens, each token finding its
// request by bisection: one launch, no plan, and the same work for one long prompt as for a
// thousand single tokens. 512 requests of 2.1 million tokens (34 MB written): 27 us; a token at a
// time to a thread in place of four 33; 64 tokens 6 us.
//
// shared: a cluster of 8 CTAs takes a set. An item is 512 columns of one member's row, compared
// with the same columns of the set's first live row; 256 warps take the items in turn and the
// least column that differs is joined through distributed shared memory. 8 rows of 1250 pages
// 4 us; 16 sets of 1028 rows in all 11 us (18 with 64 warps to a set).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kv_pages.h"

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kEach = 16;                   // requests of a thread in a round
constexpr int kRound = kThreads * kEach;    // requests of a round
constexpr int kSpan = 1024;                 // tokens that a CTA's range is a multiple of
constexpr int kAtOnce = 4;                  // tokens of a thread whose loads are on their way together
constexpr int kCluster = 8;
constexpr int kSetThreads = 1024;
constexpr int kColumns = 512;               // table columns of an item

__device__ __forceinline__ void report(int32_t* status, int bits) {
  if (bits && status) atomicOr(status, bits);
}

struct Step {
  const int32_t *rows, *old_lens, *new_lens;
  int n;
  const int32_t* table;
  int n_tables;
  int64_t ld;
  int page;
  int num_pages;
  int tokens;
  int32_t *positions, *token_table, *slots, *lens, *starts;
  int32_t* status;
  int span;  // tokens of a CTA
  int page_shift;  // log2 of a page that is a power of two, else -1
};

// Tokens of request i; 0 where it fails a check.
__device__ __forceinline__ int64_t count_of(const Step& p, int i, int* err) {
  const int row = __ldg(p.rows + i), a = __ldg(p.old_lens + i), b = __ldg(p.new_lens + i);
  if (row < 0 || row >= p.n_tables) {
    *err |= KVPAGES_STATUS_ROW;
    return 0;
  }
  if (a < 0 || b < a || (int64_t)b > p.ld * p.page) {
    *err |= KVPAGES_STATUS_LEN;
    return 0;
  }
  return b - a;
}

__global__ void __launch_bounds__(kThreads) step_kernel(const __grid_constant__ Step p) {
  __shared__ int32_t s_start[kRound + 1];  // running sums before each request, at most `tokens`
  __shared__ int64_t s_warp[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t first = (int64_t)blockIdx.x * p.span;
  const int64_t last = min(first + p.span, (int64_t)p.tokens);
  int64_t sum = 0;  // tokens of the requests of earlier rounds
  int err = 0;
  for (int i0 = 0; i0 < p.n && (sum < last || blockIdx.x == 0); i0 += kRound) {
    const int here = min(p.n - i0, kRound);
    int64_t mine[kEach], total = 0;
    int bad = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int i = tid * kEach + j;
      const int64_t c = i < here ? count_of(p, i0 + i, &bad) : 0;
      mine[j] = total;
      total += c;
    }
    if (blockIdx.x == 0) err |= bad;  // one CTA reports for all
    int64_t before = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += x;
    }
    __syncthreads();  // the round before is done with the sums
    if (lane == 31) s_warp[warp] = before;
    __syncthreads();
    before += sum - total;
    int64_t end = sum;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_warp[w];
      end += s_warp[w];
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int i = tid * kEach + j;
      if (i < here) {
        const int32_t at = (int32_t)min(before + mine[j], (int64_t)p.tokens);
        s_start[i] = at;
        if (blockIdx.x == 0) p.starts[i0 + i] = at;
      }
    }
    if (tid == 0) s_start[here] = (int32_t)min(end, (int64_t)p.tokens);
    __syncthreads();
    // tokens of this round inside the CTA's range
    const int64_t t1 = min(last, (int64_t)s_start[here]);
    for (int64_t t0 = max(first, min(sum, (int64_t)p.tokens)) + tid; t0 < t1;
         t0 += kThreads * kAtOnce) {
      int of[kAtOnce], row[kAtOnce], pos[kAtOnce], col[kAtOnce], page[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int64_t t = min(t0 + u * kThreads, t1 - 1);  // places past the end repeat the last
        int lo = 0, hi = here;  // s_start[lo] <= t < s_start[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_start[mid] <= t) lo = mid;
          else hi = mid;
        }
        of[u] = lo;
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        row[u] = __ldg(p.rows + i0 + of[u]);
        pos[u] = __ldg(p.old_lens + i0 + of[u]);
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        pos[u] += (int)(min(t0 + u * kThreads, t1 - 1) - s_start[of[u]]);
        col[u] = p.page_shift >= 0 ? pos[u] >> p.page_shift : pos[u] / p.page;
        page[u] = __ldg(p.table + row[u] * p.ld + col[u]);
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int64_t t = t0 + u * kThreads;
        if (t >= t1) break;
        int slot = -1;
        if (page[u] < 0) err |= KVPAGES_STATUS_NO_PAGE;
        else if (page[u] >= p.num_pages) err |= KVPAGES_STATUS_PAGE;
        else slot = page[u] * p.page + (pos[u] - col[u] * p.page);
        p.positions[t] = pos[u];
        p.token_table[t] = row[u];
        p.slots[t] = slot;
        p.lens[t] = pos[u] + 1;
      }
    }
    sum = end;
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.starts[p.n] = (int32_t)min(sum, (int64_t)p.tokens);
    if (sum > p.tokens) err |= KVPAGES_STATUS_TOKENS;
  }
  // places behind the last token
  for (int64_t t = max(first, sum) + tid; t < last; t += kThreads) {
    p.positions[t] = p.token_table[t] = p.slots[t] = -1;
    p.lens[t] = 0;
  }
  report(p.status, err);
}

struct Sets {
  const int32_t *rows, *lens, *starts;
  int n;
  const int32_t* table;
  int n_tables;
  int64_t ld;
  int page;
  int num_pages;
  int32_t* prefix;
  int32_t* status;
};

__global__ void __launch_bounds__(kSetThreads) shared_kernel(const __grid_constant__ Sets p) {
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ int s_lead, s_least, s_live, s_bad, s_col;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster.block_rank();
  const int set = blockIdx.x / kCluster;
  int a = __ldg(p.starts + set), b = __ldg(p.starts + set + 1);
  int err = 0;
  if (tid == 0) {
    s_lead = s_least = INT32_MAX;
    s_live = s_bad = 0;
  }
  __syncthreads();
  if (a < 0 || b < a || b > p.n) {
    err |= KVPAGES_STATUS_LEN;
    a = b = 0;
  }
  // ---- the set's live rows
  for (int i = a + tid; i < b; i += kSetThreads) {
    const int row = __ldg(p.rows + i), len = __ldg(p.lens + i);
    if (len == 0) continue;
    int bad = 0;
    if (row < 0 || row >= p.n_tables) bad = KVPAGES_STATUS_ROW;
    else if (len < 0 || (int64_t)len > p.ld * p.page) bad = KVPAGES_STATUS_LEN;
    if (bad) {
      err |= bad;
      s_bad = 1;
    } else {
      atomicMin(&s_lead, i);
      atomicMin(&s_least, len);
      atomicAdd(&s_live, 1);
    }
  }
  __syncthreads();
  const bool any = s_live > 1 && !s_bad;
  const int cols = any ? s_least / p.page : 0;
  if (tid == 0) s_col = cols;
  __syncthreads();
  // ---- the least column in which a live row differs from the first one
  if (any) {
    const int32_t* lead = p.table + __ldg(p.rows + s_lead) * p.ld;
    const int per = (cols + kColumns - 1) / kColumns;
    const int64_t items = (int64_t)(b - a) * per;
    for (int64_t item = (int64_t)warp * kCluster + rank; item < items; item += kSetThreads / 32 * kCluster) {
      const int i = a + (int)(item / per);
      const int c0 = (int)(item % per) * kColumns + lane;
      if (__ldg(p.lens + i) == 0) continue;
      const int32_t* row = p.table + __ldg(p.rows + i) * p.ld;
      int32_t x[kColumns / 32], y[kColumns / 32];
#pragma unroll
      for (int j = 0; j < kColumns / 32; ++j) {
        const int c = c0 + j * 32;
        x[j] = c < cols ? __ldg(lead + c) : 0;
        y[j] = c < cols ? __ldg(row + c) : 0;
      }
      int col = INT32_MAX;
#pragma unroll
      for (int j = kColumns / 32 - 1; j >= 0; --j) {
        if (x[j] != y[j] || x[j] < 0 || x[j] >= p.num_pages) {
          if (c0 + j * 32 < cols) col = c0 + j * 32;
        }
      }
      col = __reduce_min_sync(0xffffffffu, col);
      if (lane == 0 && col < cols) atomicMin(&s_col, col);
    }
  }
  cluster.sync();
  if (rank == 0 && tid < 32) {
    int col = tid < kCluster ? *cluster.map_shared_rank(&s_col, tid) : INT32_MAX;
    col = __reduce_min_sync(0xffffffffu, col);
    if (tid == 0) p.prefix[set] = col * p.page;
  }
  cluster.sync();  // no CTA leaves while its column is read
  if (rank == 0) report(p.status, err);
}

bool aligned(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 3) == 0; }

bool table_ok(int n, int n_tables, int64_t ld, int page_size, int num_pages) {
  return n >= 0 && n_tables >= 1 && ld >= 1 && ld < (int64_t(1) << 31) && page_size >= 1 &&
         num_pages >= 0 && (int64_t)num_pages * page_size < (int64_t(1) << 31);
}

}  // namespace

extern "C" int kvpages_step(const int32_t* rows, const int32_t* old_lens, const int32_t* new_lens,
                            int n, const int32_t* block_table, int n_tables, int64_t table_ld,
                            int page_size, int num_pages, int tokens, int32_t* positions,
                            int32_t* token_table, int32_t* slots, int32_t* lens, int32_t* starts,
                            int32_t* status, kvpages_stream_t stream) {
  if (!table_ok(n, n_tables, table_ld, page_size, num_pages) || tokens < 0)
    return KVPAGES_ERR_SHAPE;
  if (!starts || (n && (!rows || !old_lens || !new_lens || !block_table)) ||
      (tokens && (!positions || !token_table || !slots || !lens)))
    return KVPAGES_ERR_NULL;
  if (!aligned(rows) || !aligned(old_lens) || !aligned(new_lens) || !aligned(block_table) ||
      !aligned(positions) || !aligned(token_table) || !aligned(slots) || !aligned(lens) ||
      !aligned(starts) || !aligned(status))
    return KVPAGES_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return KVPAGES_ERR_CUDA;
  const int64_t spans = ((int64_t)tokens + kSpan - 1) / kSpan;
  const int64_t most = (int64_t)sms * 8;
  const int64_t each = spans <= most ? 1 : (spans + most - 1) / most;
  const int grid = spans ? (int)((spans + each - 1) / each) : 1;
  int shift = -1;
  for (int i = 0; i < 31; ++i)
    if (page_size == 1 << i) shift = i;
  const Step p{rows,   old_lens,  new_lens,    n,     block_table, n_tables, table_ld, page_size, num_pages,
               tokens, positions, token_table, slots, lens,        starts,   status,   (int)(each * kSpan), shift};
  step_kernel<<<grid, kThreads, 0, (cudaStream_t)stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? KVPAGES_OK : KVPAGES_ERR_CUDA;
}

extern "C" int kvpages_shared(const int32_t* rows, const int32_t* lens, int n,
                              const int32_t* set_starts, int n_sets, const int32_t* block_table,
                              int n_tables, int64_t table_ld, int page_size, int num_pages,
                              int32_t* prefix_lens, int32_t* status, kvpages_stream_t stream) {
  if (!table_ok(n, n_tables, table_ld, page_size, num_pages) || n_sets < 0 || n_sets > (1 << 27))
    return KVPAGES_ERR_SHAPE;
  if (n_sets == 0) return KVPAGES_OK;
  if (!set_starts || !prefix_lens || (n && (!rows || !lens || !block_table)))
    return KVPAGES_ERR_NULL;
  if (!aligned(rows) || !aligned(lens) || !aligned(set_starts) || !aligned(block_table) ||
      !aligned(prefix_lens) || !aligned(status))
    return KVPAGES_ERR_ALIGN;
  const Sets p{rows, lens, set_starts, n, block_table, n_tables, table_ld, page_size, num_pages,
               prefix_lens, status};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)n_sets * kCluster);
  cfg.blockDim = dim3(kSetThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kCluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, shared_kernel, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? KVPAGES_OK : KVPAGES_ERR_CUDA;
}
