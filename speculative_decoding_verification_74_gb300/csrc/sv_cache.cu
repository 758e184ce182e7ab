// The paged key/value cache: page bookkeeping (reserve, fork, release, and the pages that a commit
// gives back) and the rows that are written, moved or copied (append, commit, fork).
//
// Pages are handed out lowest number first, so the tables do not depend on the order in which
// threads run.  A page's state is its reference count alone: there is no free list to keep in step.
//
// Measured (GB300): a turn of 64 trees of up to 16 nodes in 32 layers (8 heads of 128) 63 us: reserve 4 us, append 45 us
// (its bytes copied: 40 us), commit 10 us; 16 prompts to 48 beams (the partly filled pages of 32 layers copied) 72 us (59
// us).  The rows are bound by memory; the bookkeeping by the latency of one CTA's scans, and small calls by their launches
// (a turn of four requests: three launches, 11 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "sv_device.cuh"
#include "sv_ops.h"
#include "sv_pages.cuh"

namespace sv {

sv_status check_cache(const sv_cache* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr || c->page_refs == nullptr)
    return set_error(SV_ERR_INVALID_ARG, "cache, its pools or page_refs is NULL");
  if (!aligned16(c->k) || !aligned16(c->v)) return set_error(SV_ERR_INVALID_ARG, "cache pools are not 16-byte aligned");
  if (c->layers < 1 || c->pages < 1 || c->pages > SV_MAX_PAGES)
    return set_error(SV_ERR_INVALID_ARG, "layers=%d pages=%d", c->layers, c->pages);
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
    return set_error(SV_ERR_INVALID_ARG, "page_size=%d: a power of two in [8, 1024] is needed", c->page_size);
  if (c->kv_heads < 1 || c->kv_heads > 1024) return set_error(SV_ERR_INVALID_ARG, "kv_heads=%d outside [1, 1024]", c->kv_heads);
  if (c->head_dim != 64 && c->head_dim != 128) return set_error(SV_ERR_INVALID_ARG, "head_dim=%d: 64 or 128", c->head_dim);
  const int64_t st[4] = {c->layer_stride, c->page_stride, c->slot_stride, c->head_stride};
  for (int i = 0; i < 4; ++i)
    if (st[i] < 8 || (st[i] & 7) != 0)
      return set_error(SV_ERR_INVALID_ARG, "cache stride %lld: multiples of 8 elements are needed", (long long)st[i]);
  return SV_OK;
}

sv_status check_table(const int32_t* page_table, int table_width, const int32_t* seq_len, int B) {
  if (B < 0 || B > SV_MAX_BATCH) return set_error(SV_ERR_INVALID_ARG, "B=%d outside [0, %d]", B, SV_MAX_BATCH);
  if (B == 0) return SV_OK;
  if (page_table == nullptr || seq_len == nullptr) return set_error(SV_ERR_INVALID_ARG, "page_table / seq_len is NULL");
  if (table_width < 1 || table_width > SV_MAX_TABLE_WIDTH)
    return set_error(SV_ERR_INVALID_ARG, "table_width=%d outside [1, %d]", table_width, SV_MAX_TABLE_WIDTH);
  return SV_OK;
}

namespace {

// ---- reserve ---------------------------------------------------------------------------------
__global__ void __launch_bounds__(kPageThreads) reserve_kernel(Pool p, int32_t* table, int width, const int32_t* seq_len,
                                                               const int32_t* extra, int B, int32_t* out_ok,
                                                               uint32_t* status) {
  __shared__ int buf[33];
  __shared__ int32_t held[SV_MAX_BATCH];        // first entry to fill
  __shared__ int32_t begin[SV_MAX_BATCH + 1];   // pages that the rows before lack
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = warp; i < B; i += kPageThreads / 32) {
    const int64_t len = seq_len[i], more = extra[i];
    const int64_t need = (len + more + (int64_t(1) << p.shift) - 1) >> p.shift;
    int lack = 0, first = 0;
    if (len < 0 || more < 0 || need > width) {
      if (lane == 0) atomicOr(status, SV_DEV_BAD_SEQ);
      lack = -1;  // not served
    } else {
      first = static_cast<int>(need);
      // the held entries come first; those before the length's page need no look unless the row
      // is short of pages for the slots that it already has
      int64_t e0 = len >> p.shift;
      if (e0 > 0 && table[static_cast<int64_t>(i) * width + e0 - 1] < 0) e0 = 0;
      for (; e0 < need; e0 += 32) {
        const int64_t e = e0 + lane;
        const unsigned none = __ballot_sync(0xFFFFFFFFu, e < need && table[static_cast<int64_t>(i) * width + e] < 0);
        if (none != 0) {
          first = static_cast<int>(e0) + __ffs(none) - 1;
          break;
        }
      }
      lack = static_cast<int>(need) - first;
    }
    if (lane == 0) {
      held[i] = first;
      begin[i] = lack;
    }
  }
  __syncthreads();
  int lack[kPerThread], sum = 0;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int i = threadIdx.x * kPerThread + j;
    lack[j] = i < B ? begin[i] : 0;
    sum += max(lack[j], 0);
  }
  int total, found;
  int at = block_scan(sum, buf, &total);  // total <= SV_MAX_BATCH * table_width, below 2^32; see the host check
  const int rank = block_scan(count_free(p), buf, &found);
  int served = 0;  // pages that go to served rows: those rows come first
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int i = threadIdx.x * kPerThread + j;
    if (i < B) {
      const int n = max(lack[j], 0);
      const bool ok = lack[j] == 0 || (lack[j] > 0 && n <= found - at);
      begin[i] = at;
      if (ok && n > 0) served = at + n;
      if (!ok && lack[j] > 0) atomicOr(status, SV_DEV_OUT_OF_PAGES);
      if (out_ok != nullptr) out_ok[i] = ok;
      if (i == B - 1) begin[B] = at + n;
      at += n;
    }
  }
  served = __reduce_max_sync(0xFFFFFFFFu, served);
  __syncthreads();
  if (lane == 0) buf[warp] = served;
  __syncthreads();
  served = buf[0];
  for (int w = 1; w < kPageThreads / 32; ++w) served = max(served, buf[w]);
  take_free(p, rank, served, [&](int r, int page) {
    int lo = 0, hi = B;  // the row with begin[lo] <= r < begin[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (begin[mid] <= r) lo = mid; else hi = mid;
    }
    table[static_cast<int64_t>(lo) * width + held[lo] + (r - begin[lo])] = page;
    p.refs[page] = 1;
  });
}

// ---- fork ------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kPageThreads) fork_kernel(Pool p, int32_t* table, int width, int rows, int32_t* seq_len,
                                                            const int32_t* src, const int32_t* dst, int n,
                                                            int32_t* out_ok, uint32_t* status) {
  __shared__ int buf[33];
  __shared__ int32_t to[SV_MAX_BATCH];    // dst rows, then the pair that gets free page r
  __shared__ int32_t len[SV_MAX_BATCH];   // slots to share, -1 = pair left out
  pdl_wait();
  for (int j = threadIdx.x; j < n; j += kPageThreads) to[j] = dst[j];
  __syncthreads();
  for (int j = threadIdx.x; j < n; j += kPageThreads) {
    const int a = src[j], b = to[j];
    int64_t l = -1;
    if (a >= 0 && a < rows && b >= 0 && b < rows && a != b) {
      l = seq_len[a];
      if (l > (static_cast<int64_t>(width) << p.shift) || table[static_cast<int64_t>(b) * width] >= 0) l = -1;
      for (int h = 0; h < n && l >= 0; ++h)
        if (h != j && to[h] == b) l = -1;  // every pair of a row named twice is left out
    }
    if (l < 0) atomicOr(status, SV_DEV_BAD_SEQ);
    len[j] = l < 0 ? -1 : static_cast<int32_t>(l);
  }
  __syncthreads();
  // a row that lacks a page for a slot of its own has nothing to copy there: one warp per pair looks its entries through
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j = warp; j < n; j += kPageThreads / 32) {
    if (len[j] <= 0) continue;
    const int32_t* from = table + static_cast<int64_t>(src[j]) * width;
    const int held = ((len[j] - 1) >> p.shift) + 1;
    bool lacks = false;
#pragma unroll 4
    for (int e = lane; e < held; e += 32) lacks |= static_cast<uint32_t>(from[e]) >= static_cast<uint32_t>(p.pages);
    if (__any_sync(0xFFFFFFFFu, lacks) && lane == 0) {
      atomicOr(status, SV_DEV_BAD_PAGE);
      len[j] = -1;
    }
  }
  __syncthreads();
  const int part_mask = (1 << p.shift) - 1;
  int split[kPerThread], sum = 0;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int i = threadIdx.x * kPerThread + j;
    split[j] = i < n && len[i] > 0 && (len[i] & part_mask) != 0;
    sum += split[j];
  }
  int total, found;
  int at = block_scan(sum, buf, &total);
  const int rank = block_scan(count_free(p), buf, &found);
  int ok[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int i = threadIdx.x * kPerThread + j;
    ok[j] = i < n && len[i] >= 0 && (!split[j] || at < found);
    if (i < n) {
      if (len[i] >= 0 && !ok[j]) {
        atomicOr(status, SV_DEV_OUT_OF_PAGES);
        len[i] = -1;
      }
      if (out_ok != nullptr) out_ok[i] = ok[j];
      if (ok[j]) seq_len[to[i]] = len[i];
    }
    if (split[j]) at += 1;
  }
  __syncthreads();
  // new pages first (free pages have count 0, and sharing only raises counts above 0)
  int32_t* pair_of = to;  // the dst rows are read from the argument from here on
  {
    int r = at;
#pragma unroll
    for (int j = kPerThread - 1; j >= 0; --j)
      if (split[j]) {
        --r;
        pair_of[r] = ok[j] ? static_cast<int>(threadIdx.x) * kPerThread + j : -1;
      }
  }
  __syncthreads();
  take_free(p, rank, min(total, found), [&](int r, int page) {
    const int i = pair_of[r];
    if (i >= 0) {
      table[static_cast<int64_t>(dst[i]) * width + (len[i] >> p.shift)] = page;
      p.refs[page] = 1;
    }
  });
  __syncthreads();
  // the full pages are shared: one warp per pair
  for (int i = warp; i < n; i += kPageThreads / 32) {
    const int full = len[i] < 0 ? 0 : len[i] >> p.shift;
    const int32_t* from = table + static_cast<int64_t>(len[i] < 0 ? 0 : src[i]) * width;
    int32_t* row = table + static_cast<int64_t>(len[i] < 0 ? 0 : dst[i]) * width;
    for (int e = lane; e < full; e += 32) {
      const int page = from[e];
      atomicAdd(p.refs + page, 1);
      row[e] = page;
    }
  }
}

__global__ void __launch_bounds__(kPageThreads) release_kernel(Pool p, int32_t* table, int width, int rows,
                                                               int32_t* seq_len, const int32_t* seqs, int n,
                                                               uint32_t* status) {
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int j = warp; j < n; j += kPageThreads / 32) {
    const int i = seqs[j];
    if (i < 0 || i >= rows) {
      if (lane == 0) atomicOr(status, SV_DEV_BAD_SEQ);
      continue;
    }
    release_entries(p, table + static_cast<int64_t>(i) * width, 0, width, status);
    if (lane == 0) seq_len[i] = 0;
  }
}

// ---- reorder ---------------------------------------------------------------------------------
// marks after plan_kernel: the free page that row j gets for its partly filled last page (>= 0), or
constexpr int32_t kKeeps = -1;    // row j takes its source row's entries as they are
constexpr int32_t kShares = -2;   // it shares the full pages, there is nothing else
constexpr int32_t kEmpties = -3;  // it names no source
constexpr int32_t kFailed = -4;   // in marks[0 .. rows): nothing changes

constexpr size_t kPlanSmem = 200 << 10;  // shared memory that a plan may take

// What becomes of every row, and the pages: one CTA.  Shared memory: five ints per row, and with kWhole the table, which is then
// rewritten here too (without it by gather_kernel).
template <bool kWhole>
__global__ void __launch_bounds__(kPageThreads) plan_kernel(Pool p, int32_t* table, int width, int rows, int32_t* seq_len,
                                                            const int32_t* src, int32_t* out_ok, int32_t* marks,
                                                            uint32_t* status) {
  extern __shared__ int32_t per_row[];
  int32_t *from = per_row, *len = per_row + rows, *first = per_row + 2 * rows, *pair_of = per_row + 3 * rows, *mark = per_row + 4 * rows;
  int32_t* old = per_row + 5 * rows;
  __shared__ int buf[33];
  __shared__ uint32_t wrong;
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) wrong = 0;
  for (int j = threadIdx.x; j < rows; j += kPageThreads) {
    from[j] = src[j];
    len[j] = seq_len[j];
    first[j] = INT_MAX;  // the first row that names row j: INT_MAX = none
  }
  if constexpr (kWhole)
    for (int x = threadIdx.x; x < rows * width; x += kPageThreads) old[x] = table[x];
  const int32_t* entries = kWhole ? old : table;
  const int free_pages = count_free(p);
  __syncthreads();
  for (int j = threadIdx.x; j < rows; j += kPageThreads) {
    const int s = from[j];
    if (s < -1 || s >= rows) atomicOr(&wrong, SV_DEV_BAD_SEQ);
    else if (s >= 0) atomicMin(first + s, s == j ? -1 : j);  // the row itself comes before all others
  }
  __syncthreads();
  bool drops = false;  // some row's pages are given back
  for (int j = warp; j < rows; j += kPageThreads / 32) {
    const int32_t* row = entries + static_cast<int64_t>(j) * width;
    if (first[j] == INT_MAX) {
      drops |= row[0] >= 0;
      continue;
    }
    const int64_t held = (static_cast<int64_t>(len[j]) + (1 << p.shift) - 1) >> p.shift;
    if (len[j] < 0 || held > width) {
      if (lane == 0) atomicOr(&wrong, SV_DEV_BAD_SEQ);
      continue;
    }
    bool lacks = false;
#pragma unroll 4
    for (int e = lane; e < held; e += 32) lacks |= static_cast<uint32_t>(row[e]) >= static_cast<uint32_t>(p.pages);
    if (__any_sync(0xFFFFFFFFu, lacks) && lane == 0) atomicOr(&wrong, SV_DEV_BAD_PAGE);
  }
  drops = __syncthreads_or(drops);
  uint32_t problem = wrong;
  int total = 0;
  int split[kPerThread], at = 0;
  if (problem == 0) {
    // the pages of rows that no row names are given back first (their table rows are rewritten later)
    auto each_entry = [&](auto f) {
      for (int j = warp; j < rows; j += kPageThreads / 32) {
        if (first[j] != INT_MAX) continue;
        const int32_t* row = entries + static_cast<int64_t>(j) * width;
        for (int e0 = 0; e0 < width; e0 += 32) {
          const int page = e0 + lane < width ? row[e0 + lane] : -1;
          if (page >= 0) f(page);
          if (__any_sync(0xFFFFFFFFu, page < 0)) break;
        }
      }
    };
    // (counts may fall below 0 here, where a page is named more often than it is counted: so that all can be taken back)
    bool too_often = false;
    if (drops) {
      each_entry([&](int page) { too_often |= page >= p.pages || atomicSub(p.refs + page, 1) <= 0; });
      too_often = __syncthreads_or(too_often);
    }
    const int part_mask = (1 << p.shift) - 1;
    int sum = 0;
#pragma unroll
    for (int x = 0; x < kPerThread; ++x) {
      const int j = threadIdx.x * kPerThread + x;
      const int s = j < rows ? from[j] : -1;
      split[x] = s >= 0 && first[s] != (s == j ? -1 : j) && (len[s] & part_mask) != 0;
      sum += split[x];
    }
    at = block_scan(sum, buf, &total);
    int found, rank = 0;
    if (total == 0) {
      found = 0;
    } else {
      rank = block_scan(drops ? count_free<true>(p) : free_pages, buf, &found);
    }
    if (total > found) problem = SV_DEV_OUT_OF_PAGES;
    if (too_often || (problem != 0 && drops)) {
      each_entry([&](int page) {
        if (page >= p.pages) return;
        if (problem != 0) atomicAdd(p.refs + page, 1);
        else atomicMax(p.refs + page, 0);
      });
      if (threadIdx.x == 0 && too_often) atomicOr(status, SV_DEV_BAD_PAGE);
      __syncthreads();
    }
    if (problem == 0 && total > 0) {
#pragma unroll
      for (int x = 0; x < kPerThread; ++x)
        if (split[x]) pair_of[at++] = threadIdx.x * kPerThread + x;
      __syncthreads();
      take_free(p, rank, total, [&](int r, int page) {
        (kWhole ? mark : marks)[pair_of[r]] = page;
        p.refs[page] = 1;
      });
    }
  }
#pragma unroll
  for (int x = 0; x < kPerThread; ++x) {
    const int j = threadIdx.x * kPerThread + x;
    if (j >= rows) continue;
    const int s = from[j];
    int32_t* its = (kWhole ? mark : marks) + j;
    if (problem != 0) {
      *its = kFailed;
    } else {
      if (s < 0) *its = kEmpties;
      else if (!split[x]) *its = first[s] == (s == j ? -1 : j) ? kKeeps : kShares;
      seq_len[j] = s < 0 ? 0 : len[s];
    }
  }
  if (threadIdx.x == 0) {
    if (problem != 0) atomicOr(status, problem);
    if (out_ok != nullptr) out_ok[0] = problem == 0;
  }
  if constexpr (kWhole) {
    __syncthreads();
    for (int j = warp; j < rows; j += kPageThreads / 32) {
      const int what = mark[j], s = from[j], full = what == kFailed || what == kEmpties ? 0 : len[s] >> p.shift;
      if (lane == 0) marks[j] = what >= 0 ? old[s * width + full] : what;
      if (what == kFailed || (what == kKeeps && s == j)) continue;
      for (int e = lane; e < width; e += 32) {
        int32_t page = -1;
        if (what == kKeeps) {
          page = old[s * width + e];
        } else if (what != kEmpties && e < full) {
          page = old[s * width + e];
          atomicAdd(p.refs + page, 1);
        } else if (what >= 0 && e == full) {
          page = what;
        }
        table[static_cast<int64_t>(j) * width + e] = page;
      }
    }
  }
}

// The table rows, `columns` entries of every row to a CTA: all are read before any is written.
__global__ void __launch_bounds__(kRowThreads) gather_kernel(Pool p, int32_t* table, int width, int rows,
                                                             const int32_t* seq_len, const int32_t* src, int32_t* marks,
                                                             int columns) {
  extern __shared__ int32_t old[];  // [rows][columns]
  pdl_wait();
  if (marks[0] == kFailed) return;
  const int c0 = blockIdx.x * columns, n = min(columns, width - c0);
  const int items = rows * columns;
  bool some = false;
  for (int x = threadIdx.x; x < items; x += kRowThreads) {
    const int j = x / columns, c = x - j * columns;
    const int32_t page = c < n ? table[static_cast<int64_t>(j) * width + c0 + c] : -1;
    some |= page >= 0;
    old[x] = page;
  }
  if (__syncthreads_or(some) == 0) return;  // (a row's held entries come first: past the longest row there are none)
  for (int x = threadIdx.x; x < items; x += kRowThreads) {
    const int j = x / columns, c = x - j * columns, e = c0 + c;
    if (c >= n) continue;
    const int mark = marks[j];
    int32_t page = -1;
    if (mark != kEmpties) {
      const int s = src[j], full = seq_len[j] >> p.shift;
      page = old[s * columns + c];
      if (mark != kKeeps) {
        if (e < full) {
          atomicAdd(p.refs + page, 1);
        } else if (e == full && mark >= 0) {
          // rows of this CTA alone look at this mark from here on: a partly filled page lies in one column
          const int32_t source = page;
          page = mark;
          marks[j] = source;
        } else {
          page = -1;
        }
      }
    }
    table[static_cast<int64_t>(j) * width + e] = page;
  }
}

// ---- rows ------------------------------------------------------------------------------------
// Where the 16-byte piece `e` of a token's keys (or values) lies within its slot.
struct RowShape {
  int64_t layer_stride, page_stride, slot_stride, head_stride;
  int32_t pieces;      // kv_heads * head_dim / 8
  int32_t dim_shift;   // head_dim / 8 = 1 << dim_shift
  int32_t shift, pages;
};
__device__ __forceinline__ int64_t piece_offset(const RowShape& r, int e) {
  const int h = e >> r.dim_shift, d = e & ((1 << r.dim_shift) - 1);
  return static_cast<int64_t>(h) * r.head_stride + d * 8;
}
// Element offset of a slot within a layer, or -1.
__device__ __forceinline__ int64_t slot_offset(const RowShape& r, const int32_t* row, int width, int64_t slot) {
  const int64_t e = slot >> r.shift;
  if (e >= width) return -1;
  const int page = row[e];
  if (page < 0 || page >= r.pages) return -1;
  return page * r.page_stride + (slot & ((1 << r.shift) - 1)) * r.slot_stride;
}

struct AppendParams {
  RowShape r;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  int64_t new_layer_stride, new_row_stride, n_rows;
  const int32_t *table, *seq_len, *node_offsets;
  int32_t width, B, layers;
  uint32_t* status;
};

// One CTA per (new row, group of layers): thread x copies pieces x, x + 256, ... of [layer][k, v][piece].
__global__ void __launch_bounds__(kRowThreads) append_kernel(AppendParams a) {
  pdl_wait();
  const int64_t row = blockIdx.x;
  __shared__ int64_t where;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < a.B; i += kRowThreads)
      if (a.node_offsets[i] < 0 || a.node_offsets[i + 1] < a.node_offsets[i] || a.node_offsets[i + 1] > a.n_rows)
        atomicOr(a.status, SV_DEV_BAD_NODES);
  if (threadIdx.x < 32) {
    const int lo = request_of_row(a.node_offsets, a.B, row);
    if (threadIdx.x == 0) {
      const int64_t first = a.node_offsets[lo], last = a.node_offsets[lo + 1], len = a.seq_len[lo];
      where = -1;
      if (first >= 0 && last <= a.n_rows && row >= first && row < last) {
        where = len < 0 ? -1 : slot_offset(a.r, a.table + static_cast<int64_t>(lo) * a.width, a.width, len + (row - first));
        if (where < 0) atomicOr(a.status, len < 0 ? SV_DEV_BAD_SEQ : SV_DEV_BAD_PAGE);
      }
    }
  }
  __syncthreads();
  if (where < 0) return;
  const int per_layer = 2 * a.r.pieces;
  const int64_t items = static_cast<int64_t>(a.layers) * per_layer;
  const int64_t step = static_cast<int64_t>(gridDim.y) * kRowThreads;
#pragma unroll 4
  for (int64_t x = static_cast<int64_t>(blockIdx.y) * kRowThreads + threadIdx.x; x < items; x += step) {
    const int layer = static_cast<int>(x / per_layer);
    int e = static_cast<int>(x - static_cast<int64_t>(layer) * per_layer);
    const bool second = e >= a.r.pieces;
    e -= second ? a.r.pieces : 0;
    const int4 data = __ldg(reinterpret_cast<const int4*>((second ? a.v_new : a.k_new) + layer * a.new_layer_stride +
                                                          row * a.new_row_stride) + e);
    *reinterpret_cast<int4*>((second ? a.v : a.k) + layer * a.r.layer_stride + where + piece_offset(a.r, e)) = data;
  }
}

struct CommitParams {
  RowShape r;
  Pool pool;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  int32_t* table;
  const int32_t *seq_len, *node_offsets, *path, *accept_len;
  int32_t* out_len;
  int32_t width, B, Nmax, layers;
  uint32_t* status;
  int32_t* arrived;  // [B] CTAs of a request that are done with its table row (zero between calls)
};

constexpr int kMoveBatch = 8;  // nodes whose pieces a thread holds at once

// grid (groups of layers, B).  A thread moves one piece of every accepted node, in path order: node
// path[j] >= j + 1, so a slot that is written was read before, or is never read.  The request's CTA that finishes
// last gives back the pages past the new length: by then none of them reads the table row any more.
__global__ void __launch_bounds__(kRowThreads) commit_kernel(CommitParams a) {
  extern __shared__ int64_t moves[];  // [2 * Nmax]: source, destination offsets (-1 = stays)
  __shared__ int bad, last_one;
  pdl_wait();
  const int i = blockIdx.y;
  const int64_t len = a.seq_len[i];
  const int32_t* row = a.table + static_cast<int64_t>(i) * a.width;
  const int nodes = a.node_offsets[i + 1] - a.node_offsets[i];
  int n = a.accept_len[i];
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  const bool wrong = len < 0 || nodes < 0 || nodes > a.Nmax || n > (nodes > 0 ? nodes - 1 : 0) ||
                     len + nodes > (static_cast<int64_t>(a.width) << a.r.shift);
  const int keep = wrong || nodes == 0 ? -1 : n;
  for (int j = threadIdx.x; j < keep; j += kRowThreads) {
    const int node = a.path[static_cast<int64_t>(i) * a.Nmax + j];
    const int before = j > 0 ? a.path[static_cast<int64_t>(i) * a.Nmax + j - 1] : 0;
    if (node <= before || node >= nodes) {
      bad = 1;
    } else {
      const int64_t from = slot_offset(a.r, row, a.width, len + node), to = slot_offset(a.r, row, a.width, len + 1 + j);
      const bool stays = node == j + 1 || from < 0 || to < 0;
      if ((from < 0 || to < 0) && blockIdx.x == 0) atomicOr(a.status, SV_DEV_BAD_PAGE);
      moves[2 * j] = stays ? -1 : from;
      moves[2 * j + 1] = to;
    }
  }
  // node 0 stays, but in a slot that has a page
  if (keep >= 0 && blockIdx.x == 0 && threadIdx.x == kRowThreads - 1 && slot_offset(a.r, row, a.width, len) < 0)
    atomicOr(a.status, SV_DEV_BAD_PAGE);
  __syncthreads();
  const bool invalid = wrong || bad != 0;
  if (invalid && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, SV_DEV_BAD_SEQ);
  if (!invalid) {
    const int per_layer = 2 * a.r.pieces;
    const int64_t items = static_cast<int64_t>(a.layers) * per_layer;
    for (int64_t x = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; x < items;
         x += static_cast<int64_t>(gridDim.x) * kRowThreads) {
      const int layer = static_cast<int>(x / per_layer);
      int e = static_cast<int>(x - static_cast<int64_t>(layer) * per_layer);
      const bool second = e >= a.r.pieces;
      e -= second ? a.r.pieces : 0;
      __nv_bfloat16* base = (second ? a.v : a.k) + layer * a.r.layer_stride + piece_offset(a.r, e);
      for (int j0 = 0; j0 < keep; j0 += kMoveBatch) {
        int4 data[kMoveBatch];
#pragma unroll
        for (int j = 0; j < kMoveBatch; ++j)
          if (j0 + j < keep && moves[2 * (j0 + j)] >= 0) data[j] = *reinterpret_cast<const int4*>(base + moves[2 * (j0 + j)]);
#pragma unroll
        for (int j = 0; j < kMoveBatch; ++j)
          if (j0 + j < keep && moves[2 * (j0 + j)] >= 0) *reinterpret_cast<int4*>(base + moves[2 * (j0 + j) + 1]) = data[j];
      }
    }
  }
  __syncthreads();  // every thread has read what it needs of the row
  if (threadIdx.x == 0) {
    __threadfence();
    last_one = atomicAdd(a.arrived + i, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (last_one && threadIdx.x < 32) {
    const int64_t now = invalid || nodes == 0 || n < 0 ? len : len + 1 + n;
    if (!invalid)
      release_entries(a.pool, a.table + static_cast<int64_t>(i) * a.width,
                      static_cast<int>((now + (int64_t(1) << a.r.shift) - 1) >> a.r.shift), a.width, a.status);
    if (threadIdx.x == 0) {
      a.out_len[i] = static_cast<int32_t>(now);
      a.arrived[i] = 0;
    }
  }
}

struct CopyParams {
  RowShape r;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  const int32_t *table, *seq_len, *src, *dst;
  int32_t width, layers;
  const int32_t* done;  // [n] pairs that were forked; after a reorder (src NULL), the pages to copy from
};

// grid (pieces of [layer][k, v][slot][piece], pairs): the used slots of each forked pair's last page.  I: an unsigned type
// that counts a pair's pieces (64-bit divisions per piece cost more than its copy).
constexpr int kInFlight = 4;
template <typename I>
__global__ void __launch_bounds__(kRowThreads) fork_rows_kernel(CopyParams a) {
  pdl_wait();
  int32_t from, to;
  const int part = copied_slots(a.src, a.dst, a.done, a.table, a.width, a.seq_len, a.r.shift, blockIdx.y, &from, &to);
  if (part == 0) return;
  const I pieces = static_cast<I>(a.r.pieces), per_side = part * pieces, items = static_cast<I>(a.layers) * 2 * per_side;
  const I step = static_cast<I>(gridDim.x) * kRowThreads;
  for (I x0 = static_cast<I>(blockIdx.x) * kRowThreads + threadIdx.x; x0 < items; x0 += kInFlight * step) {
    int4 w[kInFlight];
    __nv_bfloat16* at[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const I x = x0 + u * step;
      at[u] = nullptr;
      if (x >= items) continue;
      const I side = x / per_side, y = x - side * per_side, slot = y / pieces;
      at[u] = ((side & 1) ? a.v : a.k) + static_cast<int64_t>(side >> 1) * a.r.layer_stride + static_cast<int64_t>(slot) * a.r.slot_stride +
              piece_offset(a.r, static_cast<int>(y - slot * pieces));
      w[u] = *reinterpret_cast<const int4*>(at[u] + from * a.r.page_stride);
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u)
      if (at[u] != nullptr) *reinterpret_cast<int4*>(at[u] + to * a.r.page_stride) = w[u];
  }
}

// Copies of `items` pieces per pair, in one wave of eight CTAs an SM (half as many again 73.5 us against 72.0 for 16 prompts to 48 beams).
cudaError_t copy_rows(const CopyParams& a, int page_size, int n, void* stream) {
  const int64_t items = static_cast<int64_t>(a.layers) * 2 * page_size * a.r.pieces;
  const int64_t groups = std::min<int64_t>(std::max(1, 8 * 152 / n), (items + 4 * kRowThreads - 1) / (4 * kRowThreads));
  const auto kernel = items <= INT_MAX ? fork_rows_kernel<uint32_t> : fork_rows_kernel<uint64_t>;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(std::max<int64_t>(1, groups)), n), kRowThreads, 0, stream,
                          SV_KERNEL_CACHE_ROWS, 1, a);
}

RowShape row_shape(const sv_cache* c) {
  RowShape r;
  r.layer_stride = c->layer_stride;
  r.page_stride = c->page_stride;
  r.slot_stride = c->slot_stride;
  r.head_stride = c->head_stride;
  r.pieces = c->kv_heads * c->head_dim / 8;
  r.dim_shift = log2_of(c->head_dim / 8);
  r.shift = log2_of(c->page_size);
  r.pages = c->pages;
  return r;
}

CopyParams copy_params(const sv_cache* c, const int32_t* table, int width, const int32_t* seq_len) {
  CopyParams a = {};
  a.r = row_shape(c);
  a.k = static_cast<__nv_bfloat16*>(c->k);
  a.v = static_cast<__nv_bfloat16*>(c->v);
  a.table = table;
  a.seq_len = seq_len;
  a.width = width;
  a.layers = c->layers;
  return a;
}

Pool pool_of(const sv_cache* c) { return Pool{c->page_refs, c->pages, log2_of(c->page_size)}; }

}  // namespace

cudaError_t reserve_pages(const Pool& p, int32_t* table, int width, const int32_t* seq_len, const int32_t* extra, int B,
                          int32_t* out_ok, void* ws, void* stream) {
  return launch_dependent(reserve_kernel, dim3(1), kPageThreads, 0, stream, SV_KERNEL_CACHE_PAGES, 1, p, table, width, seq_len,
                          extra, B, out_ok, status_of(ws));
}
cudaError_t fork_pages(const Pool& p, int32_t* table, int width, int rows, int32_t* seq_len, const int32_t* src,
                       const int32_t* dst, int n, int32_t* done, void* ws, void* stream) {
  return launch_dependent(fork_kernel, dim3(1), kPageThreads, 0, stream, SV_KERNEL_CACHE_PAGES, 1, p, table, width, rows,
                          seq_len, src, dst, n, done, status_of(ws));
}
cudaError_t release_pages(const Pool& p, int32_t* table, int width, int rows, int32_t* seq_len, const int32_t* seqs, int n,
                          void* ws, void* stream) {
  return launch_dependent(release_kernel, dim3(1), kPageThreads, 0, stream, SV_KERNEL_CACHE_PAGES, 1, p, table, width, rows,
                          seq_len, seqs, n, status_of(ws));
}
cudaError_t reorder_pages(const Pool& p, int32_t* table, int width, int rows, int32_t* seq_len, const int32_t* src,
                          int32_t* out_ok, void* ws, void* stream) {
  // a table that fits into shared memory is rewritten by the CTA that plans (256 rows of up to 58 pages 27 us
  // with it, 46 without; up to 127 pages 39 and 56; four of 9 8.2 and 10.2)
  const size_t per_row = sizeof(int32_t) * 5 * rows, table_bytes = sizeof(int32_t) * rows * static_cast<size_t>(width);
  const bool whole = per_row + table_bytes <= kPlanSmem;
  cudaError_t e = whole ? allow_smem<plan_kernel<true>>(kPlanSmem) : allow_smem<plan_kernel<false>>(sizeof(int32_t) * 5 * SV_MAX_BATCH);
  if (e != cudaSuccess) return e;
  e = launch_dependent(whole ? plan_kernel<true> : plan_kernel<false>, dim3(1), kPageThreads, per_row + (whole ? table_bytes : 0),
                       stream, SV_KERNEL_CACHE_PAGES, 1, p, table, width, rows,
                       seq_len, src, out_ok, marks_of(ws), status_of(ws));
  if (e != cudaSuccess || whole) return e;
  // a CTA holds its columns of every row in at most 32 KB (64 KB for 4096 rows)
  const int columns = std::min(std::max(4, 8192 / rows), std::max(width, 1));
  const size_t bytes = sizeof(int32_t) * columns * rows;
  e = allow_smem<gather_kernel>(sizeof(int32_t) * 4 * SV_MAX_BATCH);
  if (e != cudaSuccess) return e;
  return launch_dependent(gather_kernel, dim3((width + columns - 1) / columns), kRowThreads, bytes, stream,
                          SV_KERNEL_CACHE_PAGES, 1, p, table, width, rows, seq_len, src, marks_of(ws), columns);
}

}  // namespace sv

using namespace sv;

extern "C" {

sv_status sv_cache_reserve(const sv_cache* c, int32_t* page_table, int table_width, const int32_t* seq_len,
                           const int32_t* extra, int B, int32_t* out_ok, void* ws, size_t ws_bytes, void* stream) {
  sv_status s;
  if ((s = check_cache(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, B)) != SV_OK) return s;
  if (B == 0) return SV_OK;
  if (extra == nullptr) return set_error(SV_ERR_INVALID_ARG, "extra is NULL");
  if (static_cast<int64_t>(B) * table_width > INT_MAX)
    return set_error(SV_ERR_INVALID_ARG, "B * table_width = %lld exceeds 2^31 - 1", (long long)B * table_width);
  if ((s = check_workspace(ws, ws_bytes, SV_CACHE_WORKSPACE_BYTES)) != SV_OK) return s;
  return launch_status(reserve_pages(pool_of(c), page_table, table_width, seq_len, extra, B, out_ok, ws, stream), "reserve");
}

sv_status sv_cache_append(const sv_cache* c, int layer, int layers, const int32_t* page_table, int table_width,
                          const int32_t* seq_len, const int32_t* node_offsets, int64_t n_rows, const void* k_new,
                          const void* v_new, int64_t new_layer_stride, int64_t new_row_stride, int B, void* ws,
                          size_t ws_bytes, void* stream) {
  sv_status s;
  if ((s = check_cache(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, B)) != SV_OK) return s;
  if (layer < 0 || layers < 0 || layer > c->layers - layers)
    return set_error(SV_ERR_INVALID_ARG, "layers [%d, %d) outside the cache's %d", layer, layer + layers, c->layers);
  if (n_rows < 0 || n_rows > INT_MAX) return set_error(SV_ERR_INVALID_ARG, "n_rows=%lld", (long long)n_rows);
  if (B == 0 || layers == 0 || n_rows == 0) return SV_OK;
  if (node_offsets == nullptr || k_new == nullptr || v_new == nullptr)
    return set_error(SV_ERR_INVALID_ARG, "node_offsets / k_new / v_new is NULL");
  if (!aligned16(k_new) || !aligned16(v_new) || (new_layer_stride & 7) != 0 || (new_row_stride & 7) != 0 ||
      new_row_stride < static_cast<int64_t>(c->kv_heads) * c->head_dim || new_layer_stride < 0)
    return set_error(SV_ERR_INVALID_ARG, "k_new / v_new: 16-byte aligned rows of kv_heads * head_dim elements are needed");
  if ((s = check_workspace(ws, ws_bytes, SV_CACHE_WORKSPACE_BYTES)) != SV_OK) return s;
  AppendParams a = {};
  a.r = row_shape(c);
  a.k = static_cast<__nv_bfloat16*>(c->k) + layer * c->layer_stride;
  a.v = static_cast<__nv_bfloat16*>(c->v) + layer * c->layer_stride;
  a.k_new = static_cast<const __nv_bfloat16*>(k_new);
  a.v_new = static_cast<const __nv_bfloat16*>(v_new);
  a.new_layer_stride = new_layer_stride;
  a.new_row_stride = new_row_stride;
  a.n_rows = n_rows;
  a.table = page_table;
  a.seq_len = seq_len;
  a.node_offsets = node_offsets;
  a.width = table_width;
  a.B = B;
  a.layers = layers;
  a.status = status_of(ws);
  // about four pieces a thread
  const int64_t items = static_cast<int64_t>(layers) * 2 * a.r.pieces;
  const int64_t groups = std::min<int64_t>(64, (items + 4 * kRowThreads - 1) / (4 * kRowThreads));
  return launch_status(launch_dependent(append_kernel, dim3(static_cast<unsigned>(n_rows), static_cast<unsigned>(groups)),
                                        kRowThreads, 0, stream, SV_KERNEL_CACHE_ROWS, 1, a),
                       "append");
}

sv_status sv_cache_commit(const sv_cache* c, int32_t* page_table, int table_width, const int32_t* seq_len,
                          const int32_t* node_offsets, const int32_t* path, const int32_t* accept_len, int B, int Nmax,
                          int32_t* out_len, void* ws, size_t ws_bytes, void* stream) {
  sv_status s;
  if ((s = check_cache(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, B)) != SV_OK) return s;
  if (Nmax < 1 || Nmax > SV_MAX_DRAFT + 1) return set_error(SV_ERR_INVALID_ARG, "Nmax=%d outside [1, %d]", Nmax, SV_MAX_DRAFT + 1);
  if (B == 0) return SV_OK;
  if (node_offsets == nullptr || path == nullptr || accept_len == nullptr || out_len == nullptr)
    return set_error(SV_ERR_INVALID_ARG, "node_offsets / path / accept_len / out_len is NULL");
  if ((s = check_workspace(ws, ws_bytes, SV_CACHE_WORKSPACE_BYTES)) != SV_OK) return s;
  CommitParams a = {};
  a.r = row_shape(c);
  a.pool = pool_of(c);
  a.k = static_cast<__nv_bfloat16*>(c->k);
  a.v = static_cast<__nv_bfloat16*>(c->v);
  a.table = page_table;
  a.seq_len = seq_len;
  a.node_offsets = node_offsets;
  a.path = path;
  a.accept_len = accept_len;
  a.out_len = out_len;
  a.width = table_width;
  a.B = B;
  a.Nmax = Nmax;
  a.layers = c->layers;
  a.status = status_of(ws);
  a.arrived = arrived_of(ws);
  const int64_t items = static_cast<int64_t>(c->layers) * 2 * a.r.pieces;
  const int64_t groups = std::min<int64_t>(64, (items + kRowThreads - 1) / kRowThreads);
  return launch_status(launch_dependent(commit_kernel, dim3(static_cast<unsigned>(groups), B), kRowThreads,
                                        sizeof(int64_t) * 2 * Nmax, stream, SV_KERNEL_CACHE_ROWS, 1, a),
                       "commit");
}

sv_status sv_cache_fork(const sv_cache* c, int32_t* page_table, int table_width, int rows, int32_t* seq_len,
                        const int32_t* src, const int32_t* dst, int n, int32_t* out_ok, void* ws, size_t ws_bytes,
                        void* stream) {
  sv_status s;
  if ((s = check_cache(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, rows)) != SV_OK) return s;
  if (n < 0 || n > SV_MAX_BATCH) return set_error(SV_ERR_INVALID_ARG, "n=%d outside [0, %d]", n, SV_MAX_BATCH);
  if (n == 0) return SV_OK;
  if (rows == 0 || src == nullptr || dst == nullptr) return set_error(SV_ERR_INVALID_ARG, "rows, src or dst is missing");
  if ((s = check_workspace(ws, ws_bytes, SV_CACHE_WORKSPACE_BYTES)) != SV_OK) return s;
  int32_t* done = out_ok != nullptr ? out_ok : marks_of(ws);
  const cudaError_t e = fork_pages(pool_of(c), page_table, table_width, rows, seq_len, src, dst, n, done, ws, stream);
  if (e != cudaSuccess) return launch_status(e, "fork");
  CopyParams a = copy_params(c, page_table, table_width, seq_len);
  a.src = src;
  a.dst = dst;
  a.done = done;
  return launch_status(copy_rows(a, c->page_size, n, stream), "fork rows");
}

sv_status sv_cache_release(const sv_cache* c, int32_t* page_table, int table_width, int rows, int32_t* seq_len,
                           const int32_t* seqs, int n, void* ws, size_t ws_bytes, void* stream) {
  sv_status s;
  if ((s = check_cache(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, rows)) != SV_OK) return s;
  if (n < 0 || n > SV_MAX_BATCH) return set_error(SV_ERR_INVALID_ARG, "n=%d outside [0, %d]", n, SV_MAX_BATCH);
  if (n == 0) return SV_OK;
  if (rows == 0 || seqs == nullptr) return set_error(SV_ERR_INVALID_ARG, "rows or seqs is missing");
  if ((s = check_workspace(ws, ws_bytes, SV_CACHE_WORKSPACE_BYTES)) != SV_OK) return s;
  return launch_status(release_pages(pool_of(c), page_table, table_width, rows, seq_len, seqs, n, ws, stream), "release");
}

sv_status sv_cache_reorder(const sv_cache* c, int32_t* page_table, int table_width, int rows, int32_t* seq_len,
                           const int32_t* src, int32_t* out_ok, void* ws, size_t ws_bytes, void* stream) {
  sv_status s;
  if ((s = check_cache(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, rows)) != SV_OK) return s;
  if (rows == 0) return SV_OK;
  if (src == nullptr) return set_error(SV_ERR_INVALID_ARG, "src is NULL");
  if ((s = check_workspace(ws, ws_bytes, SV_CACHE_WORKSPACE_BYTES)) != SV_OK) return s;
  const cudaError_t e = reorder_pages(pool_of(c), page_table, table_width, rows, seq_len, src, out_ok, ws, stream);
  if (e != cudaSuccess) return launch_status(e, "reorder");
  CopyParams a = copy_params(c, page_table, table_width, seq_len);
  a.done = marks_of(ws);
  return launch_status(copy_rows(a, c->page_size, rows, stream), "reorder rows");
}

}  // extern "C"
