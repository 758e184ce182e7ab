// Page bookkeeping shared by the bf16 and the 4-bit cache: reference counts, free pages, table rows.
#pragma once
#include <cuda_runtime.h>

#include "sv_ops.h"

namespace sv {

// A pool's pages, whatever they hold.
struct Pool {
  int32_t* refs;
  int32_t pages, shift;  // page_size = 1 << shift
};

// The calls that only move pages (sv_cache.cu), arguments as in sv.h and checked by the caller; rows are copied by the caller.
cudaError_t reserve_pages(const Pool& p, int32_t* table, int width, const int32_t* seq_len, const int32_t* extra, int B,
                          int32_t* out_ok, void* ws, void* stream);
// done[j] = 1 where pair j was forked
cudaError_t fork_pages(const Pool& p, int32_t* table, int width, int rows, int32_t* seq_len, const int32_t* src,
                       const int32_t* dst, int n, int32_t* done, void* ws, void* stream);
cudaError_t release_pages(const Pool& p, int32_t* table, int width, int rows, int32_t* seq_len, const int32_t* seqs, int n,
                          void* ws, void* stream);
// Afterwards marks_of(ws)[j] is the page that row j's partly filled last page is copied from, negative = nothing to copy.
cudaError_t reorder_pages(const Pool& p, int32_t* table, int width, int rows, int32_t* seq_len, const int32_t* src,
                          int32_t* out_ok, void* ws, void* stream);

inline uint32_t* status_of(void* ws) { return static_cast<uint32_t*>(ws); }
// commit's arrival counters (zero between calls), and fork's marks or reorder's pages
inline int32_t* arrived_of(void* ws) { return reinterpret_cast<int32_t*>(static_cast<unsigned char*>(ws) + SV_STATUS_BYTES); }
inline int32_t* marks_of(void* ws) { return arrived_of(ws) + SV_MAX_BATCH; }
inline int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

namespace {

constexpr int kPageThreads = 1024;
constexpr int kRowThreads = 256;
constexpr int kPerThread = SV_MAX_BATCH / kPageThreads;  // rows per thread of the bookkeeping CTA

// Sum over the CTA before this thread (exclusive), and the total.  buf: 33 ints of shared memory.
__device__ __forceinline__ int block_scan(int v, int* buf, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // buf may still be read from a scan before
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int n = blockDim.x >> 5;
    int w = lane < n ? buf[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, w, d);
      if (lane >= d) w += y;
    }
    if (lane < n) buf[lane] = w;
    if (lane == 31) buf[32] = w;
  }
  __syncthreads();
  *total = buf[32];
  return x - v + (warp > 0 ? buf[warp - 1] : 0);
}

// Thread t owns pages [t n, (t + 1) n), n a multiple of 4: one scan gives every free page its
// rank in page order.  16-byte loads, four in flight.
__device__ __forceinline__ int pages_per_thread(int pages) {
  return ((pages + kPageThreads - 1) / kPageThreads + 3) & ~3;
}
// kBelow: while pages are given back tentatively, counts below 0 are those of free pages too.
template <bool kBelow = false>
__device__ __forceinline__ int count_free(const Pool& p) {
  auto is_free = [](int refs) { return kBelow ? refs <= 0 : refs == 0; };
  const int n = pages_per_thread(p.pages);
  const int64_t first = static_cast<int64_t>(threadIdx.x) * n;
  const int64_t last = min(first + n, static_cast<int64_t>(p.pages));
  int free_pages = 0;
  if ((reinterpret_cast<uintptr_t>(p.refs) & 15u) == 0) {
#pragma unroll 4
    for (int64_t g = first; g < last; g += 4) {
      if (g + 4 <= last) {
        const int4 r = *reinterpret_cast<const int4*>(p.refs + g);
        free_pages += is_free(r.x) + is_free(r.y) + is_free(r.z) + is_free(r.w);
      } else {
        for (int64_t h = g; h < last; ++h) free_pages += is_free(p.refs[h]);
      }
    }
  } else {
    for (int64_t g = first; g < last; ++g) free_pages += is_free(p.refs[g]);
  }
  return free_pages;
}

// Calls take(rank, page) for this thread's free pages of rank < wanted, in page order.
template <typename F>
__device__ __forceinline__ void take_free(const Pool& p, int rank, int wanted, F take) {
  const int n = pages_per_thread(p.pages);
  const int64_t first = static_cast<int64_t>(threadIdx.x) * n;
  const int64_t last = min(first + n, static_cast<int64_t>(p.pages));
  for (int64_t g = first; g < last && rank < wanted; ++g)
    if (p.refs[g] == 0) {
      take(rank, static_cast<int>(g));
      ++rank;
    }
}

// Gives back one reference of a page; a page that nothing holds is reported and left at 0.
__device__ __forceinline__ void give_back(const Pool& p, int page, uint32_t* status) {
  if (page >= p.pages || atomicSub(p.refs + page, 1) <= 0) {
    if (page < p.pages) atomicAdd(p.refs + page, 1);
    atomicOr(status, SV_DEV_BAD_PAGE);
  }
}

// Entries of one row from `from` on that hold a page, given back by one warp (the held entries of a
// row come first, so the row is read up to the first entry that holds none).
__device__ __forceinline__ void release_entries(const Pool& p, int32_t* row, int from, int width, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  for (int e0 = from; e0 < width; e0 += 32) {
    const int e = e0 + lane;
    const int page = e < width ? row[e] : -1;
    if (page >= 0 && atomicExch(row + e, -1) >= 0) give_back(p, page, status);
    if (__any_sync(0xFFFFFFFFu, page < 0)) break;
  }
}

// Used slots of the partly filled last page that pair (or, with src NULL, row) j copies, and the pages; 0 = nothing to copy.
// done: after a fork, 0 where a pair was left out; after a reorder, the pages to copy from.
__device__ __forceinline__ int copied_slots(const int32_t* src, const int32_t* dst, const int32_t* done, const int32_t* table,
                                            int width, const int32_t* seq_len, int shift, int j, int32_t* from, int32_t* to) {
  const int mark = done[j];
  if (src != nullptr ? mark == 0 : mark < 0) return 0;
  const int row = src != nullptr ? dst[j] : j;
  const int len = seq_len[row], part = len & ((1 << shift) - 1), e0 = len >> shift;
  if (part == 0) return 0;
  *from = src != nullptr ? table[static_cast<int64_t>(src[j]) * width + e0] : mark;
  *to = table[static_cast<int64_t>(row) * width + e0];  // (both name pages: the kernel before has seen to it)
  return part;
}

}  // namespace
}  // namespace sv
