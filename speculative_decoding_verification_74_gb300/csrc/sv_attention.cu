// sv_tree_attention: a token tree's queries against a paged cache.
//
// Rows and tiles.  The query heads that share a key/value head, for as many nodes as fit into 128 rows (the height of
// a tcgen05 product), form a row tile; the cache is read in tiles of 128 slots.  For a row tile, with c = scale
// log2(e) and running maximum m:
//   S = Q K^T          [128 x 128], accumulated in tensor memory
//   P = 2^(c S - m)    bf16, written back to tensor memory over S
//   O = O + P V        in tensor memory
// and at the end o = O / (sum of the rounded P), lse = (m + log2 sum P) ln 2.  O is scaled by 2^(m - m') only when some
// row's maximum has grown by more than 8 (P stays below 2^8, so float32 sums and bf16's range are far from their ends).
//
// Work split.  All (row tile, cache tile) pairs of the batch lie on one line, and before each row tile a few places for what
// beginning and ending it costs; CTA c of C takes the c-th part of the line (a persistent CTA per SM), in segments:
// stretches of one row tile.  A row tile that crosses CTAs leaves partial (O, m, sums) in the workspace, and join_kernel
// adds them.  So one long context and many short ones load the SMs alike.
//
// Few rows.  A row of S belongs to one lane of tensor memory, and a quarter of its lanes to one of the SM's four
// schedulers.  So a tile of at most 64 (32) rows is multiplied with Q's rows two (four) times over, one copy per half (quarter)
// of the lanes, and each copy takes the exponentials of its half (quarter) of the slots; P is 0 elsewhere.  The copies' (O,
// m, sums) are added at the end of a segment, like those of the two groups.
//
// Pairs of heads.  With 64 dimensions a slot of one head is 128 bytes, and the next lies kv_heads * 128 bytes on: too short
// a piece for memory's pace (4.5 of 6.8 TB/s measured).  So two neighbouring heads make one tile of 128 dimensions: Q's rows
// of the first in the lower half of the (copy's) rows and the lower 64 dimensions, those of the second in the upper ones,
// zeros elsewhere; of O each row's own 64 columns count.  The products do the work of 128 dimensions on as many bytes.
//
// Measured (GB300, 32 query and 8 key/value heads of 128, graph replay; a copy of the cache's bytes in brackets): 64 requests
// of one token over 6k to 8k slots 281 to 287 us (275), 64 trees of up to 16 nodes over 512 to 4096 slots 113 us (92), four
// chains of 17 over 99k to 131k slots 286 to 293 us (278); a window of 1024 with 16 heads of 64, 33 trees 38 us (19); four
// requests of one token and up to 130 slots 10.9 us.  Long contexts are bound by memory.  A row tile's masked tiles and
// end cost about 4 us besides its tiles (1.5 us each), which short contexts feel; a call's launches, first tile and join
// about 11 us.
//
// Roles in a CTA: warps 0 and 11 copy K and V page by page through a ring of stages (TMA; one warp alone needs
// 1.1 us a tile for it); one thread of warp 1 issues the products; warp 10 brings each segment's description, parents and
// Q; two groups of four warps take the tiles in turn (a thread has a row), each with its own S and O, so one group's
// exponentials run beside the other's products.  P is rounded to bf16, the products' type; o is divided by the sum of
// the rounded P, so its weights add up to 1, and lse takes the sum before rounding.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "sv_device.cuh"
#include "sv_ops.h"

namespace sv {
namespace {

constexpr int kTile = 128;                 // rows of Q, and slots of the cache, in a tile
constexpr int kGroupThreads = 128;
constexpr int kSoftThreads = 2 * kGroupThreads;
constexpr int kThreads = 128 + kSoftThreads;
constexpr int kWarpK = 0, kWarpMma = 1, kWarpQ = 10, kWarpV = 11;  // 2 to 9: the two groups
constexpr int kHalfBytes = kTile * 128;    // 128 slots of 64 bf16: one swizzled column block
constexpr int kTmemColumns = 512;
// Tensor memory by group: S at columns 0 and 128, O from 256 on.  With 128 dimensions P lies over S, so a group's next
// S waits for its product P V; with 64 there is room for P, and S only waits until the softmax has read it.
template <int D>
struct Columns {
  static constexpr bool kOwnP = D == 64;
  static __device__ __forceinline__ constexpr uint32_t s(uint32_t g) { return g * 128; }
  static __device__ __forceinline__ constexpr uint32_t o(uint32_t g) { return 256 + g * D; }
  static __device__ __forceinline__ constexpr uint32_t p(uint32_t g) { return kOwnP ? 384 + g * 64 : g * 128; }
};
constexpr float kLazyGrowth = 8.0f;        // log2 units by which a maximum may grow without a rescale of O
constexpr int kJoinRows = 16;              // rows per CTA of the join
// What a row tile costs besides its cache tiles, in those: its masked tiles and its end, about 4 us against 1.5 a tile
// (64 trees over 512 to 4096 slots 126 us at 0, 114 at 2, 3 and 4; the window's 33 trees 55.5, 40.7, 40.6 and 41.2).
constexpr int kExtra = 3;
constexpr int kMixFloat4 = 768;            // (a fifth stage still fits)
constexpr int kMaxStages = 12;
constexpr int kMaxCtas = 152;              // SMs of the GPU: one CTA each
constexpr int kSmemMax = 232448;           // shared memory that a CTA can have

struct alignas(16) Job {  // a row tile that several CTAs worked on: parts of CTAs `first` to `last`
  int32_t valid, request, head, mtile, rows, first, last, pad;
};

struct Line {  // what the line of work follows from
  const int32_t *seq_len, *node_offsets;
  int64_t n_rows;
  int32_t B, Nmax, width, shift, window, sinks;
  int32_t tile_nodes;  // nodes of a row tile
  int32_t extra;       // places before a row tile's cache tiles
};
struct AttendParams : Line {
  int64_t out_row_stride, out_head_stride;
  const int32_t *table, *parent;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
  int32_t* any_bad;   // [2]: some request is bad; CTAs of the join that are done with that
  uint8_t* bad;       // [SV_MAX_BATCH] requests whose outputs become 0
  Job* jobs;          // [grid]
  float* parts;       // [2 grid] partial results
  int32_t pages, q_heads, kv_heads, group;
  int32_t units;       // key/value heads, or pairs of them
  int32_t half_rows;   // rows of a copy that one head takes
  uint32_t over_group; // ceil(2^16 / group)
  int32_t stages;
  float scale;
};

// Floats of one partial result: O as [D / 4][128 rows][4], then m and the two sums per row.
template <int D>
constexpr int part_floats() { return kTile * D + 3 * kTile; }

// ---- tcgen05 -----------------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t* dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "n"(kTmemColumns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(kTmemColumns));
}
__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Arrives on `bar` when every product issued so far by this thread is complete.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// D[128 x N] (+)= A B, A and B in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Shared-memory matrix descriptor, 128-byte swizzle: start address, leading and stride byte offsets.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(stride >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// Instruction descriptor: float32 accumulator, bf16 operands, M = 128.
constexpr uint32_t instr_desc(int n, bool b_rows_are_k) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_rows_are_k ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(kTile >> 4) << 24);
}

// True in one thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

#define SV_R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define SV_I8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
// 32 columns of this warp's 32 rows: lane r holds row r.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : SV_R8(x, 0), SV_R8(x, 8), SV_R8(x, 16), SV_R8(x, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::SV_I8(x, 0),
      SV_I8(x, 8), SV_I8(x, 16), SV_I8(x, 24), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// After the wait, loaded registers may be used: the empty statements keep their uses behind it.
template <int N>
__device__ __forceinline__ void tmem_loaded(uint32_t (&x)[N]) {
  tmem_wait_load();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(x[i]));
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : SV_R8(x, 0), SV_R8(x, 8)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_load8(uint32_t addr, uint32_t* x) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : SV_R8(x, 0) : "r"(addr));
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::SV_I8(x, 0),
      SV_I8(x, 8), "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---- the line of work ------------------------------------------------------------------------------
// A request's part: its cache tiles are [0, sink_tiles) and [near_tile, ...).
struct Request {
  int64_t first;       // its first query row
  int32_t len, nodes;
  int32_t sink_tiles, near_tile, tiles;  // tiles = cache tiles that some node sees
  int32_t mtiles;      // row tiles per key/value head
  uint32_t bad;        // SV_DEV_* bits
};
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
  const int all = static_cast<int>((len + nodes + kTile - 1) / kTile);
  if (a.window > 0) {
    const int lo = max(0, r.len - a.window + 1);
    r.near_tile = lo / kTile;
    r.sink_tiles = min(static_cast<int>((static_cast<int64_t>(min(a.sinks, lo)) + kTile - 1) / kTile), r.near_tile);
  }
  r.tiles = r.sink_tiles + all - r.near_tile;
  r.mtiles = (r.nodes + a.tile_nodes - 1) / a.tile_nodes;
  return r;
}

// A stretch of cache tiles [kv0, kv1) of one row tile.
struct Segment {
  Request r;
  int32_t request, head, mtile, kv0, kv1;
  uint32_t begin, next;  // places of the line: the row tile's first, and the one after this stretch
};
// (a: in shared memory; a kernel parameter passed by reference is read through global memory, 0.3 us a field)
__device__ __noinline__ Segment segment_at(const Line& a, const uint32_t* before, uint32_t t, uint32_t end) {
  int lo = 0, hi = a.B;  // the last request whose tiles begin at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= t) lo = mid; else hi = mid;
  }
  Segment s;
  s.request = lo;
  s.r = request_of(a, lo);
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
__device__ __forceinline__ int tile_slot(const Request& r, int j) {
  return (j < r.sink_tiles ? j : r.near_tile + (j - r.sink_tiles)) * kTile;
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
// row / group for row < 128, group <= 128: over = ceil(2^16 / group).
__device__ __forceinline__ int over_group(int row, uint32_t over) { return static_cast<int>((row * over) >> 16); }

// Bits [lo, hi) of a 32-bit word whose bit 0 stands for position `at`.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int at) {
  const int a = max(lo - at, 0), b = min(hi - at, 32);
  if (b <= a) return 0u;
  return (b == 32 ? 0xFFFFFFFFu : (1u << b) - 1u) & ~((1u << a) - 1u);
}

// The part of shared memory with a fixed size; then come the tiles before each request [B], the parents of two segments'
// trees [2][Nmax] and, 1024-byte aligned, Q and the ring.
struct Smem {
  Line line;
  Segment seg[2];              // by the segment's parity
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t q_full[2];          // by the segment's parity: its Q and description are there
  uint64_t q_free;             // once per segment: its last S is complete
  uint64_t seg_free[2];        // every softmax thread is done with a description
  uint64_t s_full[2], p_full[2], pv_done[2];  // by group
  uint64_t sums_full, o_free;  // once per segment: the groups' sums are there; every thread has read O
  uint64_t mix_full[2], mix_free[2];  // by group: copies' columns written, read
  float m[2][2][kTile], l[2][2][kTile], lr[2][2][kTile];  // by the segment's parity and group
  float4 mix[2][kMixFloat4];   // by group: columns that the copies exchange, four columns of all rows together
  uint32_t scan[kThreads / 32];
  uint32_t tmem;
  volatile int32_t dead;       // a wait ran out: everyone leaves
};

// Bounded wait (about 2 s), polling: the waits between products and softmax are a fraction of a microsecond each, and
// a suspended try_wait oversleeps them.  The loop is not inlined: with it at every wait the kernel's code does not
// stay in the instruction cache.
__device__ __noinline__ bool still_waiting(uint64_t* began, volatile int32_t* dead, uint32_t* status) {
  const uint64_t now = globaltimer_ns();
  if (*began == 0) *began = now;
  if (!*dead && now - *began <= kWaitLimitNs) return true;
  atomicOr(status, SV_DEV_TIMEOUT);
  *dead = 1;
  return false;
}
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int32_t* dead, uint32_t* status) {
  uint64_t began = 0;
  for (uint32_t it = 1;; ++it) {
    if (it >= 16) __nanosleep(40);
    if (mbar_test_wait(bar, parity)) return true;
    if ((it & 255u) == 0 && !still_waiting(&began, dead, status)) return false;
  }
}
__device__ __forceinline__ bool wait_or_leave(uint64_t* bar, uint32_t parity, volatile int32_t* dead, uint32_t* status) {
  return mbar_test_wait(bar, parity) || wait_slow(bar, parity, dead, status);
}
// The same by a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int32_t* dead, uint32_t* status) {
  return __all_sync(0xFFFFFFFFu, wait_or_leave(bar, parity, dead, status));
}

__device__ __forceinline__ void mark_bad(const AttendParams& a, int request, uint32_t bits) {
  a.bad[request] = 1;
  *a.any_bad = 1;
  atomicOr(a.status, bits);
}

// A place in the ring of stages and the parity of its present round.
struct Ring {
  uint32_t stage = 0, parity = 0;
  __device__ __forceinline__ void step(uint32_t stages) {
    if (++stage == stages) {
      stage = 0;
      parity ^= 1;
    }
  }
};

template <int D, bool kPair, int kCopies>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const AttendParams a, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map) {
  constexpr int W = kPair ? 2 * D : D;  // dimensions of a tile
  using Col = Columns<W>;
  constexpr int kHalves = W / 64;
  constexpr int kHalfRows = kTile / kCopies / (kPair ? 2 : 1);
  constexpr int kStageBytes = kHalves * kHalfBytes;
  extern __shared__ unsigned char dyn[];
  __shared__ Smem sm;
  uint32_t* before = reinterpret_cast<uint32_t*>(dyn);           // [B]
  int32_t* parents = reinterpret_cast<int32_t*>(dyn) + a.B;      // [2][Nmax]
  unsigned char* q_buf = dyn + 4 * (a.B + 2 * a.Nmax);
  q_buf += (1024u - (smem_u32(q_buf) & 1023u)) & 1023u;
  unsigned char* ring = q_buf + kHalves * kHalfBytes;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // (known to be the same in all lanes)
  if (tid == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.q_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.seg_free[i], kSoftThreads);
      mbar_init(&sm.mix_full[i], kGroupThreads);
      mbar_init(&sm.mix_free[i], kGroupThreads);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], kGroupThreads);
      mbar_init(&sm.pv_done[i], 1);
    }
    mbar_init(&sm.sums_full, kSoftThreads);
    mbar_init(&sm.o_free, kSoftThreads);
    sm.dead = 0;
    sm.line = a;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if constexpr (kPair) {  // the other head's dimensions: never written again
    for (int i = tid; i < kHalves * kHalfBytes / 16; i += kThreads) reinterpret_cast<uint4*>(q_buf)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (warp == kWarpMma) tmem_alloc(&sm.tmem);
  pdl_wait();
  pdl_trigger();
  // tiles before each request
  uint32_t total;
  {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int i0 = min(a.B, tid * per), i1 = min(a.B, i0 + per);
    uint32_t sum = 0;
    for (int i = i0; i < i1; ++i) {
      const Request r = request_of(a, i);
      if (r.bad != 0 && blockIdx.x == 0) mark_bad(a, i, r.bad);
      before[i] = sum;
      sum += static_cast<uint32_t>(r.tiles + a.extra) * r.mtiles * a.units;
    }
    uint32_t x = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) sm.scan[warp] = x;
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    uint32_t at = x - sum;
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += sm.scan[w];
      total += sm.scan[w];
    }
    for (int i = i0; i < i1; ++i) before[i] += at;
    __syncthreads();
  }
  const uint32_t tmem = sm.tmem;
  // with fewer places than CTAs the last CTAs have none
  const Parts parts(total, max(1u, min(gridDim.x, total)));
  const uint32_t t0 = min(parts.begin(blockIdx.x), total), t1 = min(parts.begin(blockIdx.x + 1), total);
  Segment opening = {};
  if (t0 < t1) opening = segment_at(sm.line, before, t0, t1);
  const bool some = opening.kv0 < opening.kv1;
  // a part's stretches but the first begin a row tile; the last may hold none of its cache tiles
  auto stretch_at = [&](uint32_t t) { return t == t0 ? some : t + a.extra < t1; };
  const uint32_t stages = a.stages;
  uint32_t loaded = 0, segments = 0;  // stages and Q's that were asked for

  if (warp == kWarpK || warp == kWarpV) {
    // ---- copies -----------------------------------------------------------------------------------
    const int box_shift = min(7, a.shift), box = 1 << box_shift;  // slots per copy: a page, or 128 slots of one
    const int chunks = kTile >> box_shift;
    bool go = true;
    const uint32_t second = warp == kWarpV;  // K's and V's stages alternate
    const CUtensorMap* map = second ? &v_map : &k_map;
    Ring at;
    if (second) at.step(stages);
    loaded = second;
    // page numbers of 32 copies at a time (a copy's page: lane = its number in the block), one block ahead
    auto pages_of = [&](const Segment& s, int block) {
      const int64_t slot = (static_cast<int64_t>(block) * 32 + lane) << box_shift;
      return slot < s.r.len + s.r.nodes ? a.table[static_cast<int64_t>(s.request) * a.width + (slot >> a.shift)] : -1;
    };
    Segment s = {}, next = {};  // the next segment and its first pages are looked up while the ring is full
    int block = 0, page_now = -1, page_next = -1, next_block = 0, next_now = -1;
    if (some) {
      s = opening;
      block = tile_slot(s.r, s.kv0) >> (box_shift + 5);
      page_now = pages_of(s, block);
    }
    for (uint32_t t = t0; stretch_at(t) && go;) {
      const int end = s.r.len + s.r.nodes, lo = a.window > 0 ? max(0, s.r.len - a.window + 1) : 0;
      const uint32_t after = s.next;
      page_next = pages_of(s, block + 1);
      for (int j = s.kv0; j < s.kv1 && go; ++j) {
        const int s0 = tile_slot(s.r, j);
        const int need = s0 >> (box_shift + 5);
        if (need != block) {
          page_now = need == block + 1 ? page_next : pages_of(s, need);
          block = need;
          page_next = pages_of(s, block + 1);
        }
        // lane x < chunks copies the x-th page's part; a page without a visible slot is left out
        const int slot = s0 + (lane << box_shift);
        int page = __shfl_sync(0xFFFFFFFFu, page_now, ((s0 >> box_shift) + lane) & 31);
        const bool wanted = lane < chunks && slot < end && (a.window <= 0 || slot < a.sinks || slot + box > lo);
        if (wanted && (page < 0 || page >= a.pages)) {
          mark_bad(a, s.request, SV_DEV_BAD_PAGE);
          page = a.pages;  // outside the tensor: the copy fills zeros
        }
        const int bytes = __popc(__ballot_sync(0xFFFFFFFFu, wanted)) * kHalves * box * 128;
        if (loaded >= stages) go = warp_wait(&sm.empty[at.stage], at.parity ^ 1, &sm.dead, a.status);
        if (!go) break;
        if (lane == 0) mbar_arrive_expect_tx(&sm.full[at.stage], bytes);
        __syncwarp();
        if (wanted) {
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            tma_load_4d(ring + at.stage * kStageBytes + h * kHalfBytes + (lane << box_shift) * 128, map, kPair ? 0 : h * 64,
                        kPair ? 2 * s.head + h : s.head,
                        slot & ((1 << a.shift) - 1), page, &sm.full[at.stage]);
        }
        loaded += 2;
        at.step(stages);
        at.step(stages);
        if (j == max(s.kv0, s.kv1 - 2) && stretch_at(after)) {
          next = segment_at(sm.line, before, after, t1);
          next_block = tile_slot(next.r, next.kv0) >> (box_shift + 5);
          next_now = pages_of(next, next_block);
        }
      }
      t = after;
      s = next;
      block = next_block;
      page_now = next_now;
    }
  } else if (warp == kWarpQ) {
    // ---- segments: description, parents, Q --------------------------------------------------------
    constexpr int rows_apart = kTile / kCopies;
    for (uint32_t t = t0; stretch_at(t); ++segments) {
      const Segment s = t == t0 ? opening : segment_at(sm.line, before, t, t1);
      const int b = segments & 1;
      if (segments >= 2 && !warp_wait(&sm.seg_free[b], ((segments >> 1) - 1) & 1, &sm.dead, a.status)) break;
      if (a.parent != nullptr)
        for (int x = lane; x < s.r.nodes; x += 32) parents[b * a.Nmax + x] = a.parent[s.r.first + x];
      if (lane == 0) sm.seg[b] = s;
      if (segments >= 1 && !warp_wait(&sm.q_free, (segments - 1) & 1, &sm.dead, a.status)) break;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_expect_tx(&sm.q_full[b], kCopies * kHalves * a.tile_nodes * a.group * 128);
        for (int copy = 0; copy < kCopies; ++copy)
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            tma_load_3d(q_buf + h * kHalfBytes + (copy * rows_apart + (kPair ? h * kHalfRows : 0)) * 128, &q_map,
                        kPair ? 0 : h * 64, (kPair ? 2 * s.head + h : s.head) * a.group,
                        static_cast<int>(s.r.first) + s.mtile * a.tile_nodes, &sm.q_full[b]);
      }
      t = s.next;
    }
  } else if (warp == kWarpMma) {
    // ---- products ---------------------------------------------------------------------------------
    // The whole warp runs the loop, so counters and descriptors stay in uniform registers, which tcgen05.mma takes its
    // operands from; one elected thread issues.
    if (some) {
      const bool elected = elect_one();
      auto ready = [](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity)); };
      constexpr uint32_t kDescS = instr_desc(kTile, false), kDescO = instr_desc(W, true);
      bool more = true;                   // S's are left
      // descriptors by addition: their low words count 16-byte units of shared memory
      const uint64_t q_desc0 = smem_desc(smem_u32(q_buf), 16, 1024), k_desc0 = smem_desc(smem_u32(ring), 16, 1024),
                     v_desc0 = smem_desc(smem_u32(ring), kHalfBytes, 1024);
      Ring ks, vs;  // K's and V's stages alternate
      vs.step(stages);
      uint32_t s_seg = 0, p_seg = 0;      // segments of the next S and the next P V
      int s_left = 0, p_tiles = 0, p_j = 0;
      uint32_t n = 0, i = 0;  // tiles of the next S and the next P V: whichever is ready is issued, so neither waits
                              // behind the other's barriers
      uint32_t idle = 0;
      uint64_t began = 0;
      while (more || i < n) {
        bool issued = false;
        if (more) {
          if (s_left == 0 && ready(&sm.q_full[s_seg & 1], (s_seg >> 1) & 1))
            s_left = __shfl_sync(0xFFFFFFFFu, sm.seg[s_seg & 1].kv1 - sm.seg[s_seg & 1].kv0, 0);
          // the group's S was last read by the softmax, or by the product P V, of tile n - 2
          if (s_left > 0 && ready(&sm.full[ks.stage], ks.parity) &&
              (n < 2 || ready(Col::kOwnP ? &sm.p_full[n & 1] : &sm.pv_done[n & 1], ((n - 2) >> 1) & 1))) {
            tc_after_sync();
            const uint64_t k_desc = k_desc0 + ks.stage * (kStageBytes >> 4);
            const uint32_t d = tmem + Col::s(n & 1);
            --s_left;
            if (elected) {
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_ss(d, q_desc0 + h * (kHalfBytes >> 4) + 2 * k, k_desc + h * (kHalfBytes >> 4) + 2 * k, kDescS, h + k > 0);
              tc_commit(&sm.s_full[n & 1]);
              tc_commit(&sm.empty[ks.stage]);
              if (s_left == 0) tc_commit(&sm.q_free);
            }
            ks.step(stages);
            ks.step(stages);
            if (s_left == 0) more = stretch_at(__shfl_sync(0xFFFFFFFFu, sm.seg[s_seg & 1].next, 0));
            s_seg += s_left == 0;
            ++n;
            issued = true;
          }
        }
        if (i < n) {
          if (p_j == p_tiles) {
            p_tiles = __shfl_sync(0xFFFFFFFFu, sm.seg[p_seg & 1].kv1 - sm.seg[p_seg & 1].kv0, 0);
            p_j = 0;
            ++p_seg;
          }
          // (at a segment's first tile both groups' O of the segment before have been read)
          if (ready(&sm.p_full[i & 1], (i >> 1) & 1) && ready(&sm.full[vs.stage], vs.parity) &&
              (p_j > 0 || p_seg < 2 || ready(&sm.o_free, (p_seg - 2) & 1))) {
            tc_after_sync();
            const uint64_t v_desc = v_desc0 + vs.stage * (kStageBytes >> 4);
            const uint32_t d = tmem + Col::o(i & 1), p = tmem + Col::p(i & 1);
            const uint32_t more = p_j > 1;
            if (elected) {
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k) mma_ts(d, p + 8 * k, v_desc + k * (2048 >> 4), kDescO, k > 0 ? 1u : more);
              tc_commit(&sm.pv_done[i & 1]);
              tc_commit(&sm.empty[vs.stage]);
            }
            vs.step(stages);
            vs.step(stages);
            ++p_j;
            ++i;
            issued = true;
          }
        }
        idle = issued ? 0 : idle + 1;
        if ((idle & 1023u) == 1023u && !__all_sync(0xFFFFFFFFu, still_waiting(&began, &sm.dead, a.status))) break;
        if (issued) began = 0;
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: thread r of a group has row r of the tile: row `row_in` of copy `copy` -----------
    const int group = (warp - 2) >> 2;
    const int r = (warp & 3) * 32 + lane;
    constexpr int rows_apart = kTile / kCopies;
    const int row_in = r & (rows_apart - 1), copy = r / rows_apart;
    const int half = kPair ? row_in / kHalfRows : 0, local = row_in & (kHalfRows - 1);  // its head of the pair, its row there
    constexpr int kWide = kCopies == 4 ? 32 : 64;           // slots whose scores are in registers at once
    constexpr int kSteps = kTile / kCopies / kWide;          // of a copy's slots: 2 with one copy, else 1
    const int slot0 = copy * (kTile / kCopies);              // first slot of a tile that this thread's copy takes
    const uint32_t my = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_addr = my + Col::s(group), o_addr = my + Col::o(group), p_addr = my + Col::p(group);
    float4* mix = sm.mix[group];
    const float c = a.scale * 1.44269504088896341f;
    if (tid == 64) a.jobs[blockIdx.x].valid = 0;
    uint32_t n0 = 0, seg = 0, mixes = 0, frees = 0;  // the segment's first tile in this CTA's count
    for (uint32_t t = t0; stretch_at(t); ++seg) {
      const int b = seg & 1;
      if (!warp_wait(&sm.q_full[b], (seg >> 1) & 1, &sm.dead, a.status)) break;
      const Segment& s = sm.seg[b];
      const int32_t* tree = parents + b * a.Nmax;
      auto parent_of = [&](int node) { return a.parent != nullptr ? tree[node] : node - 1; };
      const int rows = min(a.tile_nodes, s.r.nodes - s.mtile * a.tile_nodes) * a.group;
      const bool active = (((warp & 3) * 32) & (kHalfRows - 1)) < rows;  // some row of this warp exists
      const bool exists = local < rows;
      const int local_node = exists ? over_group(local, a.over_group) : 0, node = s.mtile * a.tile_nodes + local_node;
      const int len = s.r.len, end = len + s.r.nodes;
      const int lo = a.window > 0 ? max(0, len - a.window + 1) : 0;  // before it (and past the sinks) no node sees a slot
      int depth = 0;
      if (a.window > 0) {
        if (a.parent == nullptr) depth = node;
        else
          for (int p = node; p > 0; ++depth) {
            const int up = tree[p];
            if (up < 0 || up >= p) break;  // reported where the node's own tile is masked
            p = up;
          }
      }
      const int near = a.window > 0 ? len + depth - a.window + 1 : 0;  // first position of the window
      const int tiles = s.kv1 - s.kv0;
      float m = -INFINITY, l = 0.0f, lr = 0.0f;  // maximum, sum of P, sum of the rounded P
      bool left = false;
      for (int j = (group + n0) & 1; j < tiles; j += 2) {
        const uint32_t n = n0 + j;
        if (left = !warp_wait(&sm.s_full[group], (n >> 1) & 1, &sm.dead, a.status); left) break;
        tc_after_sync();
        const int s0 = tile_slot(s.r, s.kv0 + j);
        const bool whole = s0 + kTile <= len && (a.window <= 0 || s0 + kTile <= a.sinks || s0 >= len + s.r.nodes - a.window);
        if (!whole && (s0 + kTile > end || (a.window > 0 && s0 < lo && s0 + kTile > a.sinks))) {
          // slots that no node sees may hold anything: 0 times it has to be 0
          const uint32_t v = 2 * n + 1, st = v % stages;
          if (left = !warp_wait(&sm.full[st], (v / stages) & 1, &sm.dead, a.status); left) break;
          const int slot = s0 + r;
          if (slot >= end || (slot < lo && slot >= a.sinks)) {
#pragma unroll 4
            for (int x = 0; x < W / 8; ++x)
              *reinterpret_cast<uint4*>(ring + st * kStageBytes + (x >> 3) * kHalfBytes + r * 128 + ((x + r) & 7) * 16) = make_uint4(0, 0, 0, 0);  // (neighbours in different banks)
          }
          fence_proxy_async_smem();
        }
        if (active) {
          // With one copy S is read in two halves, the first half twice (for the maximum and for P); P's columns
          // lie over columns that were read before.
          uint32_t x[kWide];
          float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int k = 0; k < kSteps; ++k) {
            const int col = slot0 + k * kWide;
#pragma unroll
            for (int i = 0; i < kWide; i += 32) tmem_load32(s_addr + col + i, x + i);
            uint32_t see[kWide / 32];
            if (!whole) {
#pragma unroll
              for (int w = 0; w < kWide / 32; ++w)
                see[w] = range_bits(near, len, s0 + col + 32 * w) | (a.window > 0 ? range_bits(0, min(a.sinks, len), s0 + col + 32 * w) : 0u);
              if (s0 + col + kWide > len && exists) {
                int d = depth;
                for (int up = node;; --d) {
                  const int bit = len + up - s0 - col;
                  if (bit >= 0 && bit < kWide && (a.window <= 0 || len + d >= near || len + d < a.sinks)) {
                    if (kWide == 32 || bit < 32) see[0] |= 1u << (bit & 31);
                    else see[kWide / 32 - 1] |= 1u << (bit & 31);
                  }
                  if (up <= 0 || bit < 0) break;
                  const int p = parent_of(up);
                  if (p < 0 || p >= up) {
                    mark_bad(a, s.request, SV_DEV_BAD_PARENT);
                    break;
                  }
                  up = p;
                }
              }
            }
            tmem_loaded(x);
            if (!whole) {
#pragma unroll
              for (int i = 0; i < kWide; ++i)
                if (!((see[i >> 5] >> (i & 31)) & 1u)) x[i] = 0xFF800000u;
              if (kSteps > 1 && k == 0) {  // masked, for the second reading
#pragma unroll
                for (int i = 0; i < kWide; i += 32) tmem_store32(s_addr + col + i, x + i);
              }
            }
#pragma unroll
            for (int i = 0; i < kWide; i += 8)  // four chains, three operands a step
#pragma unroll
              for (int e = 0; e < 4; ++e)
                top4[e] = fmaxf(fmaxf(top4[e], __uint_as_float(x[i + e])), __uint_as_float(x[i + 4 + e]));
          }
          if (!whole) tmem_wait_store();
          const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * c;  // c > 0
          if (j < 2) {
            m = top;
          } else {
            const bool grow = top > m + kLazyGrowth || (m == -INFINITY && top > -INFINITY);
            if (__any_sync(0xFFFFFFFFu, grow)) {
              const float keep = grow ? (m == -INFINITY ? 0.0f : ex2_approx(m - top)) : 1.0f;
              if (grow) m = top;
              l *= keep;
              lr *= keep;
              // the group's O is complete up to its tile before
              if (left = !warp_wait(&sm.pv_done[group], ((n - 2) >> 1) & 1, &sm.dead, a.status); left) break;
              tc_after_sync();
#pragma unroll 1
              for (int i = 0; i < W; i += 16) {
                uint32_t o[16];
                tmem_load16(o_addr + i, o);
                tmem_loaded(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                tmem_store16(o_addr + i, o);
              }
            }
          }
          if (Col::kOwnP && j >= 2) {  // the product of the group's tile before has read P
            if (left = !warp_wait(&sm.pv_done[group], ((n - 2) >> 1) & 1, &sm.dead, a.status); left) break;
            tc_after_sync();
          }
          const float off = m == -INFINITY ? 0.0f : -m;
          const f32x2 c2 = f2_pack(c, c), off2 = f2_pack(off, off);
          f32x2 sum[2] = {0, 0}, sumr[2] = {0, 0};
          [[maybe_unused]] uint32_t later[kSteps > 1 ? 32 : 1];
#pragma unroll 1
          for (int k = kSteps - 1; k >= 0; --k) {  // the last step's scores are still there
            const int col = slot0 + k * kWide;
            if (k < kSteps - 1) {
#pragma unroll
              for (int i = 0; i < kWide; i += 32) tmem_load32(s_addr + col + i, x + i);
              tmem_loaded(x);
            }
#pragma unroll
            for (int i = 0; i < kWide; i += 2) {
              float e0, e1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), c2, off2), e0, e1);
              e0 = ex2_approx(e0);
              e1 = ex2_approx(e1);
              const uint32_t w = pack_bf16(e0, e1);
              sum[(i >> 1) & 1] = f2_add(sum[(i >> 1) & 1], f2_pack(e0, e1));
              sumr[(i >> 1) & 1] = f2_add(sumr[(i >> 1) & 1], f2_pack(bf16_lo(w), bf16_hi(w)));
              x[i >> 1] = w;
            }
            if constexpr (kSteps > 1) {
              if (k > 0) {  // this half's P lies over the half of S that is still to be read
#pragma unroll
                for (int i = 0; i < 32; ++i) later[i] = x[i];
              } else {
                tmem_store32(p_addr, x);
                tmem_store32(p_addr + 32, later);
              }
            } else if constexpr (kWide == 64) {
              tmem_store32(p_addr + col / 2, x);
            } else {
              tmem_store16(p_addr + col / 2, x);
            }
          }
          if constexpr (kCopies > 1) {
            uint32_t zero[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) zero[i] = 0;
#pragma unroll 1
            for (int k = 0; k < 4; ++k)
              if (32 * k < slot0 || 32 * k >= slot0 + kTile / kCopies) tmem_store16(p_addr + 16 * k, zero);
          }
          float e0, e1;
          f2_unpack(f2_add(sum[0], sum[1]), e0, e1);
          l += e0 + e1;
          f2_unpack(f2_add(sumr[0], sumr[1]), e0, e1);
          lr += e0 + e1;
          tmem_wait_store();
        }
        tc_before_sync();
        mbar_arrive(&sm.p_full[group]);
      }
      if (left) break;
      // ---- the segment's end: the sums of groups and copies, then half of the columns per group --------
      sm.m[b][group][r] = m;
      sm.l[b][group][r] = l;
      sm.lr[b][group][r] = lr;
      mbar_arrive(&sm.sums_full);
      if (!warp_wait(&sm.sums_full, seg & 1, &sm.dead, a.status)) break;
      float top = -INFINITY, sum = 0.0f, sumr = 0.0f;
      for (int x = row_in; x < kTile; x += rows_apart) top = fmaxf(top, fmaxf(sm.m[b][0][x], sm.m[b][1][x]));
      for (int x = row_in; x < kTile; x += rows_apart)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float w = sm.m[b][g][x] == -INFINITY ? 0.0f : ex2_approx(sm.m[b][g][x] - top);
          sum += w * sm.l[b][g][x];
          sumr += w * sm.lr[b][g][x];
        }
      const bool complete = s.kv0 == 0 && s.kv1 == s.r.tiles;
      // Every row sees its own node's slot, so a sum that is not above 0 is that of a row without a softmax: NaN among its
      // scores (which the maximum passes over), or nothing but -inf.  Its outputs are NaN; the parts' sums tell the join.
      const float inv = !complete ? 1.0f : sumr > 0.0f ? 1.0f / sumr : NAN;
      // (a group without a tile in the segment has m = -inf: its O is not used, whatever it holds)
      const float w0 = (sm.m[b][0][r] == -INFINITY ? 0.0f : ex2_approx(sm.m[b][0][r] - top)) * inv;
      const float w1 = (sm.m[b][1][r] == -INFINITY ? 0.0f : ex2_approx(sm.m[b][1][r] - top)) * inv;
      const int head = ((kPair ? 2 * s.head + half : s.head) - local_node) * a.group + local;  // (of an existing row)
      float* part = a.parts + static_cast<int64_t>(2 * blockIdx.x + (s.kv0 == 0)) * part_floats<D>();
      // four columns of this thread's row: to the output, or to this CTA's partial result
      __nv_bfloat16* out_row = a.out + (s.r.first + node) * a.out_row_stride +
                               head * a.out_head_stride - (kPair ? half * D : 0);
      float* part_row = part + row_in * 4 - (kPair ? half * D * kTile : 0);
      auto emit4 = [&](int column, float4 v) {
        if (complete) *reinterpret_cast<uint2*>(out_row + column) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        else *reinterpret_cast<float4*>(part_row + column * kTile) = v;
      };
      if (group == 0 && copy == 0 && exists) {
        if (!complete) {
          part[kTile * D + row_in] = top;
          part[kTile * D + kTile + row_in] = sum;
          part[kTile * D + 2 * kTile + row_in] = sumr;
        } else if (a.lse != nullptr) {
          a.lse[(s.r.first + node) * a.q_heads + head] = (top + log2f(sum)) * 0.693147180559945309f;
        }
      }
      if (tid == 64 && s.kv0 == 0 && !complete) {
        // the CTA in which the row tile ends
        const uint32_t ends = s.begin + a.extra + s.r.tiles - 1;
        const Job job = {1, s.request, s.head, s.mtile, rows, static_cast<int32_t>(blockIdx.x), parts.of(ends), 0};
        a.jobs[blockIdx.x] = job;
      }
      // the last tile of each parity: its product is the last into that group's O
      const uint32_t last = n0 + tiles - 1;
      bool ok = warp_wait(&sm.pv_done[last & 1], (last >> 1) & 1, &sm.dead, a.status);
      if (ok && tiles > 1) ok = warp_wait(&sm.pv_done[(last - 1) & 1], ((last - 1) >> 1) & 1, &sm.dead, a.status);
      if (!ok) break;
      tc_after_sync();
      // P of this thread's columns from `column` on, both groups' O's together
      auto read_o = [&](int column, auto& f) {
        constexpr int P = sizeof(f) / sizeof(float);
        uint32_t x[P], y[P];
        if constexpr (P == 16) {
          tmem_load16(my + Col::o(0) + column, x);
          tmem_load16(my + Col::o(1) + column, y);
        } else {
          tmem_load8(my + Col::o(0) + column, x);
          tmem_load8(my + Col::o(1) + column, y);
        }
        tmem_loaded(x);
        tmem_loaded(y);
#pragma unroll
        for (int e = 0; e < P; ++e)
          f[e] = (w0 != 0.0f ? w0 * __uint_as_float(x[e]) : 0.0f) + (w1 != 0.0f ? w1 * __uint_as_float(y[e]) : 0.0f);
      };
      const int col0 = group * (W / 2), col1 = col0 + W / 2;
      const bool writes = exists && (!kPair || half == group);
      if constexpr (kCopies == 1) {
        if (active) {
#pragma unroll 1
          for (int i = col0; i < col1; i += 16) {
            float f[16];
            read_o(i, f);
            if (writes) {
#pragma unroll
              for (int q = 0; q < 4; ++q) emit4(i + 4 * q, make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]));
            }
          }
        }
      } else {
        // The copies' sum through shared memory: in a round every copy takes P columns, to which the others send theirs.
        // Rounds of as many columns as fit: each costs 0.8 us, most of it latency.  (Loops, not unrolled: this code runs
        // once a segment and comes from behind the instruction cache.)
        const int kept_rows = (rows + 7) & ~7;
        auto mixed = [&](auto width) {
          constexpr int P = decltype(width)::value;
#pragma unroll 1
          for (int i0 = col0; i0 < col1; i0 += kCopies * P) {
            float f[P];
            if (active) {
#pragma unroll 1
              for (int o = 1; o < kCopies; ++o) {
                const int to = (copy + o) % kCopies;
                read_o(i0 + to * P, f);
                float4* at = mix + (to * (kCopies - 1) + o - 1) * (P / 4) * kept_rows + local;
                if (writes) {
#pragma unroll
                  for (int q = 0; q < P / 4; ++q) at[q * kept_rows] = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
                }
              }
              read_o(i0 + copy * P, f);
            }
            mbar_arrive(&sm.mix_full[group]);
            if (!warp_wait(&sm.mix_full[group], mixes & 1, &sm.dead, a.status)) return false;
            ++mixes;
            if (writes) {
              const float4* from = mix + copy * (kCopies - 1) * (P / 4) * kept_rows + local;
#pragma unroll
              for (int q = 0; q < P / 4; ++q) {
                float4 v = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
#pragma unroll
                for (int o = 0; o < kCopies - 1; ++o) {
                  const float4 w = from[(o * (P / 4) + q) * kept_rows];
                  v.x += w.x;
                  v.y += w.y;
                  v.z += w.z;
                  v.w += w.w;
                }
                emit4(i0 + copy * P + 4 * q, v);
              }
            }
            if (i0 + kCopies * P < col1) {  // the buffer is written again
              mbar_arrive(&sm.mix_free[group]);
              if (!warp_wait(&sm.mix_free[group], frees & 1, &sm.dead, a.status)) return false;
              ++frees;
            }
          }
          return true;
        };
        // (kept_rows copies (copies - 1) P floats; a half of 32 columns goes over four copies by 8)
        static_assert(64 * 2 * 16 <= 4 * kMixFloat4 && 16 * 4 * 3 * 16 <= 4 * kMixFloat4 && 32 * 4 * 3 * 8 <= 4 * kMixFloat4, "mix");
        using Sixteen = std::integral_constant<int, 16>;
        using Eight = std::integral_constant<int, 8>;
        if constexpr (kCopies == 2) left = !mixed(Sixteen());
        else if constexpr (W == 64) left = !mixed(Eight());
        else left = kept_rows <= 16 ? !mixed(Sixteen()) : !mixed(Eight());
      }
      if (left) break;
      tc_before_sync();
      t = s.next;
      mbar_arrive(&sm.o_free);
      mbar_arrive(&sm.seg_free[b]);
      n0 += tiles;
    }
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  if (sm.dead) {  // copies in flight land before the CTA leaves
    if (warp == kWarpK || warp == kWarpV)  // its last fills: every second place of the ring's line
      for (uint32_t x = loaded > stages + 1 ? loaded - ((stages + 1) & ~1u) : (warp == kWarpV); x < loaded; x += 2)
        mbar_wait(&sm.full[x % stages], (x / stages) & 1, a.status);
    if (warp == kWarpQ && segments > 0) mbar_wait(&sm.q_full[(segments - 1) & 1], ((segments - 1) >> 1) & 1, a.status);
    __syncthreads();
  }
  if (warp == kWarpMma) tmem_free(tmem);
}

// Adds the partial results of row tile `jobs[x]`: with M = max m_i, o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// grid (CTAs of the attention, row groups); a thread has four columns of a row.  Then the outputs of bad requests become 0.
template <int D>
__global__ void __launch_bounds__(kJoinRows * D / 4) join_kernel(const AttendParams a) {
  constexpr int kJoinThreads = kJoinRows * D / 4;
  pdl_wait();
  const Job job = a.jobs[blockIdx.x];
  const int heads = a.kv_heads / a.units, piece = threadIdx.x / kJoinRows;
  int local = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows;
  if (job.valid != 0 && local < heads * job.rows && !a.bad[job.request]) {
    const int half = local >= job.rows;
    local -= half * job.rows;
    const int r = half * a.half_rows + local;
    const int n = job.last - job.first + 1;
    // part i > 0 is its CTA's first, part 0 its CTA's second
    const float* first = a.parts + static_cast<int64_t>(2 * job.first + 1) * part_floats<D>();
    const float* others = a.parts + static_cast<int64_t>(2 * job.first) * part_floats<D>();
    float M = -INFINITY, L = 0.0f, R = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = 0; i < n; ++i) M = fmaxf(M, (i == 0 ? first : others + static_cast<int64_t>(2 * i) * part_floats<D>())[kTile * D + r]);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float* part = i == 0 ? first : others + static_cast<int64_t>(2 * i) * part_floats<D>();
      const float m = part[kTile * D + r];
      const float w = m == -INFINITY ? 0.0f : ex2_approx(m - M);
      const float4 v = *reinterpret_cast<const float4*>(part + (piece * kTile + r) * 4);
      L += w * part[kTile * D + kTile + r];
      R += w * part[kTile * D + 2 * kTile + r];
      o[0] += w * v.x;
      o[1] += w * v.y;
      o[2] += w * v.z;
      o[3] += w * v.w;
    }
    const float inv = R > 0.0f ? 1.0f / R : NAN;  // (not above 0: NaN among the row's scores, or nothing but -inf)
    const int node = job.mtile * a.tile_nodes + local / a.group, head = (heads * job.head + half) * a.group + local % a.group;
    const int64_t row = a.node_offsets[job.request] + node;
    uint2 w;
    w.x = pack_bf16(o[0] * inv, o[1] * inv);
    w.y = pack_bf16(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2*>(a.out + row * a.out_row_stride + head * a.out_head_stride + piece * 4) = w;
    if (piece == 0 && a.lse != nullptr) a.lse[row * a.q_heads + head] = (M + log2f(L)) * 0.693147180559945309f;
  }
  if (*a.any_bad != 0) {
    const int blocks = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
    for (int i = me; i < a.B; i += blocks) {
      if (!a.bad[i]) continue;
      const int64_t first = max(int64_t(0), static_cast<int64_t>(a.node_offsets[i]));
      const int64_t last = min(a.n_rows, static_cast<int64_t>(a.node_offsets[i + 1]));
      for (int64_t row = first; row < last; ++row) {
        for (int x = threadIdx.x; x < a.q_heads * (D / 8); x += kJoinThreads)
          *reinterpret_cast<uint4*>(a.out + row * a.out_row_stride + (x / (D / 8)) * a.out_head_stride + (x % (D / 8)) * 8) =
              make_uint4(0, 0, 0, 0);
        if (a.lse != nullptr)
          for (int x = threadIdx.x; x < a.q_heads; x += kJoinThreads) a.lse[row * a.q_heads + x] = -INFINITY;
      }
    }
    // the last CTA clears the marks for the next call
    __shared__ int last_one;
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      last_one = atomicAdd(a.any_bad + 1, 1) == blocks - 1;
    }
    __syncthreads();
    if (last_one) {
      for (int i = threadIdx.x; i < a.B; i += kJoinThreads) a.bad[i] = 0;
      if (threadIdx.x == 0) {
        a.any_bad[0] = 0;
        a.any_bad[1] = 0;
      }
    }
  }
}

// ---- host --------------------------------------------------------------------------------------------
struct Layout {
  size_t bad, jobs, parts, total;
};
Layout layout_of(int ctas, int head_dim) {
  Layout L;
  L.bad = SV_STATUS_BYTES;
  L.jobs = L.bad + SV_MAX_BATCH;
  L.parts = (L.jobs + sizeof(Job) * ctas + 255) & ~size_t(255);
  L.total = L.parts + sizeof(float) * (head_dim == 128 ? part_floats<128>() : part_floats<64>()) * 2 * ctas;
  return L;
}
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// The pool of one layer as (dimension, head, slot, page); a copy takes 64 dimensions of one head's slots in a
// page (or 128 of them).
bool encode_pool(CUtensorMap* map, const sv_cache* c, const void* base) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->head_dim), static_cast<cuuint64_t>(c->kv_heads),
                              static_cast<cuuint64_t>(c->page_size), static_cast<cuuint64_t>(c->pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c->head_stride) * 2, static_cast<cuuint64_t>(c->slot_stride) * 2,
                                 static_cast<cuuint64_t>(c->page_stride) * 2};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(std::min(kTile, c->page_size)), 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The query rows as (dimension, head, row); a copy takes 64 dimensions of a head group's rows of a tile.
bool encode_queries(CUtensorMap* map, const void* q, int64_t row_stride, int64_t head_stride, int head_dim, int heads,
                    int64_t rows, int group, int tile_nodes) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2, static_cast<cuuint64_t>(row_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(tile_nodes)};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kPair, int kCopies>
cudaError_t launch_attention(AttendParams& a, const CUtensorMap& q_map, const CUtensorMap& k_map, const CUtensorMap& v_map,
                             int ctas, void* stream) {
  // the ring gets what Q, the tables and the fixed part leave of the shared memory: at least 4 stages
  constexpr int kStageBytes = (kPair ? 2 : 1) * D / 64 * kHalfBytes;
  const int fixed = 4 * (a.B + 2 * a.Nmax) + 1024 + kStageBytes;
  const int room = kSmemMax - static_cast<int>(sizeof(Smem)) - 64 - fixed;
  a.stages = std::min(kMaxStages, room / kStageBytes);
  const size_t dyn = static_cast<size_t>(fixed) + static_cast<size_t>(a.stages) * kStageBytes;
  cudaError_t e = allow_smem<attend_kernel<D, kPair, kCopies>>(kSmemMax - sizeof(Smem) - 64);
  if (e != cudaSuccess) return e;
  e = launch_dependent(attend_kernel<D, kPair, kCopies>, dim3(ctas), kThreads, dyn, stream, SV_KERNEL_ATTENTION, 1, a, q_map, k_map, v_map);
  if (e != cudaSuccess) return e;
  const int groups = ((kPair ? 2 : 1) * a.tile_nodes * a.group + kJoinRows - 1) / kJoinRows;
  return launch_dependent(join_kernel<D>, dim3(ctas, groups), kJoinRows * D / 4, 0, stream, SV_KERNEL_ATTENTION_JOIN, 1, a);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t sv_attention_workspace_size(const sv_cache* c, int q_heads) {
  if (check_cache(c) != SV_OK || q_heads < 1 || q_heads % c->kv_heads != 0 || q_heads / c->kv_heads > kTile) return 0;
  return layout_of(kMaxCtas, c->head_dim).total;
}

sv_status sv_tree_attention(const sv_cache* c, int layer, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                            int q_heads, const int32_t* page_table, int table_width, const int32_t* seq_len,
                            const int32_t* node_offsets, int64_t n_rows, const int32_t* parent, int B, int Nmax,
                            float scale, int window, int sinks, void* out, int64_t out_row_stride,
                            int64_t out_head_stride, float* out_lse, void* ws, size_t ws_bytes, void* stream) {
  sv_status s;
  if ((s = check_cache(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, B)) != SV_OK) return s;
  if (layer < 0 || layer >= c->layers) return set_error(SV_ERR_INVALID_ARG, "layer=%d outside [0, %d)", layer, c->layers);
  if (q_heads < 1 || q_heads % c->kv_heads != 0 || q_heads / c->kv_heads > kTile)
    return set_error(SV_ERR_INVALID_ARG, "q_heads=%d: 1 to %d times kv_heads=%d are needed", q_heads, kTile, c->kv_heads);
  if (Nmax < 1 || Nmax > SV_MAX_DRAFT + 1) return set_error(SV_ERR_INVALID_ARG, "Nmax=%d outside [1, %d]", Nmax, SV_MAX_DRAFT + 1);
  if (n_rows < 0 || n_rows > static_cast<int64_t>(SV_MAX_BATCH) * (SV_MAX_DRAFT + 1))
    return set_error(SV_ERR_INVALID_ARG, "n_rows=%lld", (long long)n_rows);
  if (!(scale > 0.0f) || std::isinf(scale)) return set_error(SV_ERR_INVALID_ARG, "scale must be finite and positive");
  if (window < 0 || sinks < 0) return set_error(SV_ERR_INVALID_ARG, "window=%d sinks=%d: must be >= 0", window, sinks);
  if (B == 0 || n_rows == 0) return SV_OK;
  if (q == nullptr || out == nullptr || node_offsets == nullptr)
    return set_error(SV_ERR_INVALID_ARG, "q / out / node_offsets is NULL");
  if (!aligned16(q) || !aligned16(out) || ((q_row_stride | q_head_stride | out_row_stride | out_head_stride) & 7) != 0 ||
      q_head_stride < c->head_dim || out_head_stride < c->head_dim || q_row_stride < 0 || out_row_stride < 0)
    return set_error(SV_ERR_INVALID_ARG, "q / out: 16-byte aligned rows of head_dim elements are needed");
  if ((s = check_workspace(ws, ws_bytes, sv_attention_workspace_size(c, q_heads))) != SV_OK) return s;
  // two heads at a time where they lie side by side and all nodes' rows of both fit into a tile (else a tile would be
  // read once for each of their row tiles; 64 contexts of 8192, 16 heads of 64, one node: 322 us against 504 one by one; the window's 33 trees 41 against 50)
  const int group = q_heads / c->kv_heads;
  const bool pair = c->head_dim == 64 && c->head_stride == 64 && c->kv_heads % 2 == 0 && 2 * Nmax * group <= kTile;
  const int tile_nodes = std::min(kTile / group, Nmax);
  // the line of work is counted in 32 bits
  const int64_t tiles = ((static_cast<int64_t>(table_width) * c->page_size + kTile - 1) / kTile + 1 + kExtra) *
                        ((Nmax + tile_nodes - 1) / tile_nodes);
  if (tiles > INT_MAX || tiles * c->kv_heads > INT_MAX || tiles * c->kv_heads * B > INT_MAX)
    return set_error(SV_ERR_INVALID_ARG, "B=%d requests of up to %lld tiles a head are too many for one call", B, (long long)tiles);
  const size_t offset = static_cast<size_t>(layer) * c->layer_stride * 2;
  CUtensorMap q_map, k_map, v_map;
  if (!encode_queries(&q_map, q, q_row_stride, q_head_stride, c->head_dim, q_heads, n_rows, group, tile_nodes))
    return set_error(SV_ERR_CUDA, "the query rows' strides or sizes cannot be described to the copy engine");
  if (!encode_pool(&k_map, c, static_cast<const unsigned char*>(c->k) + offset) ||
      !encode_pool(&v_map, c, static_cast<const unsigned char*>(c->v) + offset))
    return set_error(SV_ERR_CUDA, "the cache's strides or sizes cannot be described to the copy engine");
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return launch_status(e, "device");
  const int ctas = std::min(sms, kMaxCtas);
  const Layout L = layout_of(kMaxCtas, c->head_dim);
  unsigned char* w = static_cast<unsigned char*>(ws);
  AttendParams a = {};
  a.out_row_stride = out_row_stride;
  a.out_head_stride = out_head_stride;
  a.table = page_table;
  a.seq_len = seq_len;
  a.node_offsets = node_offsets;
  a.parent = parent;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = out_lse;
  a.status = reinterpret_cast<uint32_t*>(w);
  a.any_bad = reinterpret_cast<int32_t*>(w) + 1;
  a.bad = w + L.bad;
  a.jobs = reinterpret_cast<Job*>(w + L.jobs);
  a.parts = reinterpret_cast<float*>(w + L.parts);
  a.n_rows = n_rows;
  a.width = table_width;
  a.B = B;
  a.Nmax = Nmax;
  a.pages = c->pages;
  a.shift = 0;
  while ((1 << a.shift) < c->page_size) ++a.shift;
  a.q_heads = q_heads;
  a.kv_heads = c->kv_heads;
  a.units = pair ? c->kv_heads / 2 : c->kv_heads;
  a.group = group;
  a.tile_nodes = tile_nodes;
  a.over_group = (65536 + group - 1) / group;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale;
  // as many copies of a row tile as its height leaves room for (window's 33 trees, 32 rows: 41 us with four, 43 with two, 45
  // with one; 64 trees of 64 rows: 114 with two, 121 with one; 64 contexts of 1000, 4 rows: 57, 58, 60)
  const int tile_rows = tile_nodes * group * (pair ? 2 : 1), copies = tile_rows <= 32 ? 4 : tile_rows <= 64 ? 2 : 1;
  a.half_rows = kTile / copies / (pair ? 2 : 1);
  a.extra = kExtra;
  const auto launch = pair                 ? (copies == 4   ? launch_attention<64, true, 4>
                                              : copies == 2 ? launch_attention<64, true, 2>
                                                            : launch_attention<64, true, 1>)
                      : c->head_dim == 128 ? (copies == 4   ? launch_attention<128, false, 4>
                                              : copies == 2 ? launch_attention<128, false, 2>
                                                            : launch_attention<128, false, 1>)
                                           : (copies == 4   ? launch_attention<64, false, 4>
                                              : copies == 2 ? launch_attention<64, false, 2>
                                                            : launch_attention<64, false, 1>);
  return launch_status(launch(a, q_map, k_map, v_map, ctas, stream), "attention");
}

}  // extern "C"
