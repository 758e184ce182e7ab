// What the attention kernels over a bf16 and over a 4-bit cache share: the line of work that all (row tile, cache tile) pairs of
// a batch lie on, bounded waits, and the outputs of requests that turned out bad.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "sv_device.cuh"
#include "sv_ops.h"

namespace sv {
namespace {

constexpr int kMaxCtas = 152;              // SMs of the GPU: one CTA each
constexpr int kSmemMax = 232448;           // shared memory that a CTA can have

struct alignas(16) Job {  // a row tile that several CTAs worked on: parts of CTAs `first` to `last`
  int32_t valid, request, head, mtile, rows, first, last, pad;
};

struct Line {  // what the line of work follows from
  const int32_t *seq_len, *node_offsets;
  int64_t n_rows;
  int32_t B, Nmax, width, shift, window, sinks;
  int32_t group;       // query heads of a key/value head
  int32_t tile_rows;   // rows (nodes times group) of a row tile
  int32_t extra;       // places before a row tile's cache tiles
};
struct Marks {
  uint32_t* status;
  int32_t* any_bad;   // [2]: some request is bad; CTAs of the join that are done with that
  uint8_t* bad;       // [SV_MAX_BATCH] requests whose outputs become 0
};
struct Outputs {
  __nv_bfloat16* out;
  float* lse;
  int64_t out_row_stride, out_head_stride;
  int32_t q_heads;
};

// ---- the line of work ------------------------------------------------------------------------------
// T: slots of a cache tile.  A request's part: its cache tiles are [0, sink_tiles) and [near_tile, ...).
struct Request {
  int64_t first;       // its first query row
  int32_t len, nodes;
  int32_t sink_tiles, near_tile, tiles;  // tiles = cache tiles that some node sees
  int32_t mtiles;      // row tiles per key/value head
  uint32_t bad;        // SV_DEV_* bits
};
template <int T>
__device__ __forceinline__ Request request_of(const Line& a, int i) {
  Request r = {};
  const int64_t first = a.node_offsets[i], last = a.node_offsets[i + 1];
  const int64_t len = a.seq_len[i], nodes = last - first;
  r.first = first;
  if (first < 0 || nodes < 0 || nodes > a.Nmax || last > a.n_rows) {
    r.bad = SV_DEV_BAD_NODES;
    return r;
  }
  if (nodes == 0) return r;
  if (len < 0 || len + nodes > (static_cast<int64_t>(a.width) << a.shift)) {
    r.bad = SV_DEV_BAD_SEQ;
    return r;
  }
  r.len = static_cast<int32_t>(len);
  r.nodes = static_cast<int32_t>(nodes);
  const int all = static_cast<int>((len + nodes + T - 1) / T);
  if (a.window > 0) {
    const int lo = max(0, r.len - a.window + 1);
    r.near_tile = lo / T;
    r.sink_tiles = min(static_cast<int>((static_cast<int64_t>(min(a.sinks, lo)) + T - 1) / T), r.near_tile);
  }
  r.tiles = r.sink_tiles + all - r.near_tile;
  r.mtiles = (r.nodes * a.group + a.tile_rows - 1) / a.tile_rows;
  return r;
}

// A stretch of cache tiles [kv0, kv1) of one row tile.
struct Segment {
  Request r;
  int32_t request, head, mtile, kv0, kv1;
  uint32_t begin, next;  // places of the line: the row tile's first, and the one after this stretch
};
// (a: in shared memory; a kernel parameter passed by reference is read through global memory, 0.3 us a field)
template <int T>
__device__ __forceinline__ Segment segment_at_here(const Line& a, const uint32_t* before, uint32_t t, uint32_t end) {
  int lo = 0, hi = a.B;  // the last request whose tiles begin at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= t) lo = mid; else hi = mid;
  }
  Segment s;
  s.request = lo;
  s.r = request_of<T>(a, lo);
  const uint32_t places = s.r.tiles + a.extra, local = t - before[lo], unit = local / places, at = local - unit * places;
  const uint32_t to = min(places, at + (end - t));
  s.begin = t - at;
  s.next = s.begin + to;
  s.kv0 = max(static_cast<int>(at) - a.extra, 0);
  s.kv1 = max(static_cast<int>(to) - a.extra, 0);  // (kv0: the part ends among the places before the tiles)
  s.head = static_cast<int>(unit / s.r.mtiles);   // a head's row tiles are neighbours: they share its tiles in L2
  s.mtile = static_cast<int>(unit - static_cast<uint32_t>(s.head) * s.r.mtiles);
  return s;
}
template <int T>
__device__ __noinline__ Segment segment_at_call(const Line& a, const uint32_t* before, uint32_t t, uint32_t end) {
  return segment_at_here<T>(a, before, t, end);
}
// kHere: in line, for kernels whose warpgroups share out their registers (those may call nothing); otherwise a function, as code
// that runs once in a while keeps the rest out of the instruction cache.
template <int T, bool kHere = false>
__device__ __forceinline__ Segment segment_at(const Line& a, const uint32_t* before, uint32_t t, uint32_t end) {
  if constexpr (kHere) return segment_at_here<T>(a, before, t, end);
  else return segment_at_call<T>(a, before, t, end);
}
template <int T>
__device__ __forceinline__ int tile_slot(const Request& r, int j) {
  return (j < r.sink_tiles ? j : r.near_tile + (j - r.sink_tiles)) * T;
}
// The line in n parts as equal as can be: the first `longer` have a place more.  (32-bit arithmetic: a 64-bit division is
// a page of code, and at a call's start code comes from behind the instruction cache.)
struct Parts {
  uint32_t length, longer;
  __device__ __forceinline__ Parts(uint32_t total, uint32_t n) : length(total / n), longer(total - length * n) {}
  __device__ __forceinline__ uint32_t begin(uint32_t c) const { return c * length + min(c, longer); }
  // the part that holds place `at`
  __device__ __forceinline__ int of(uint32_t at) const {
    const uint32_t first = longer * (length + 1);
    return static_cast<int>(at < first ? at / (length + 1) : longer + (at - first) / length);
  }
};
// Bits [lo, hi) of a 32-bit word whose bit 0 stands for position `at`.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int at) {
  const int a = max(lo - at, 0), b = min(hi - at, 32);
  if (b <= a) return 0u;
  return (b == 32 ? 0xFFFFFFFFu : (1u << b) - 1u) & ~((1u << a) - 1u);
}

// Bounded wait (about 2 s), polling: the waits between products and softmax are a fraction of a microsecond each, and
// a suspended try_wait oversleeps them.  The loop is not inlined: with it at every wait the kernel's code does not
// stay in the instruction cache.
__device__ __forceinline__ bool still_waiting_here(uint64_t* began, volatile int32_t* dead, uint32_t* status) {
  const uint64_t now = globaltimer_ns();
  if (*began == 0) *began = now;
  if (!*dead && now - *began <= kWaitLimitNs) return true;
  atomicOr(status, SV_DEV_TIMEOUT);
  *dead = 1;
  return false;
}
__device__ __noinline__ bool still_waiting_call(uint64_t* began, volatile int32_t* dead, uint32_t* status) {
  return still_waiting_here(began, dead, status);
}
template <bool kHere = false>
__device__ __forceinline__ bool still_waiting(uint64_t* began, volatile int32_t* dead, uint32_t* status) {
  if constexpr (kHere) return still_waiting_here(began, dead, status);
  else return still_waiting_call(began, dead, status);
}
template <bool kHere>
__device__ __forceinline__ bool wait_slow_here(uint64_t* bar, uint32_t parity, volatile int32_t* dead, uint32_t* status) {
  uint64_t began = 0;
#pragma unroll 1
  for (uint32_t it = 1;; ++it) {
    if (it >= 16) __nanosleep(40);
    if (mbar_test_wait(bar, parity)) return true;
    if ((it & 255u) == 0 && !still_waiting<kHere>(&began, dead, status)) return false;
  }
}
__device__ __noinline__ bool wait_slow_call(uint64_t* bar, uint32_t parity, volatile int32_t* dead, uint32_t* status) {
  return wait_slow_here<false>(bar, parity, dead, status);
}
template <bool kHere = false>
__device__ __forceinline__ bool wait_or_leave(uint64_t* bar, uint32_t parity, volatile int32_t* dead, uint32_t* status) {
  if (mbar_test_wait(bar, parity)) return true;
  if constexpr (kHere) return wait_slow_here<true>(bar, parity, dead, status);
  else return wait_slow_call(bar, parity, dead, status);
}
// The same by a whole warp: every lane gets the same answer.
template <bool kHere = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int32_t* dead, uint32_t* status) {
  return __all_sync(0xFFFFFFFFu, wait_or_leave<kHere>(bar, parity, dead, status));
}

__device__ __forceinline__ void mark_bad(const Marks& a, int request, uint32_t bits) {
  a.bad[request] = 1;
  *a.any_bad = 1;
  atomicOr(a.status, bits);
}

// By the last kernel of a call, all its CTAs: the outputs of bad requests become 0 (lse -inf), and the marks are cleared for the next call.
template <int D, int kThreads>
__device__ __forceinline__ void clear_bad(const Line& line, const Marks& marks, const Outputs& a) {
  if (*marks.any_bad != 0) {
    const int blocks = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
    for (int i = me; i < line.B; i += blocks) {
      if (!marks.bad[i]) continue;
      const int64_t first = max(int64_t(0), static_cast<int64_t>(line.node_offsets[i]));
      const int64_t last = min(line.n_rows, static_cast<int64_t>(line.node_offsets[i + 1]));
      for (int64_t row = first; row < last; ++row) {
        for (int x = threadIdx.x; x < a.q_heads * (D / 8); x += kThreads)
          *reinterpret_cast<uint4*>(a.out + row * a.out_row_stride + (x / (D / 8)) * a.out_head_stride + (x % (D / 8)) * 8) =
              make_uint4(0, 0, 0, 0);
        if (a.lse != nullptr)
          for (int x = threadIdx.x; x < a.q_heads; x += kThreads) a.lse[row * a.q_heads + x] = -INFINITY;
      }
    }
    // the last CTA clears the marks for the next call
    __shared__ int last_one;
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      last_one = atomicAdd(marks.any_bad + 1, 1) == blocks - 1;
    }
    __syncthreads();
    if (last_one) {
      for (int i = threadIdx.x; i < line.B; i += kThreads) marks.bad[i] = 0;
      if (threadIdx.x == 0) {
        marks.any_bad[0] = 0;
        marks.any_bad[1] = 0;
      }
    }
  }
}

}  // namespace
}  // namespace sv
