// sv_tree_attention: a token tree's queries against a paged cache.
//
// Rows and tiles.  A request's query rows of one key/value head (its nodes times the query heads that
// share the head) form tiles of 128 rows, the height of a tcgen05 product; the cache is read in tiles of
// 128 slots.  For a tile of rows, with c = scale log2(e) and running maximum m:
//   S = Q K^T          [128 x 128], accumulated in tensor memory
//   P = 2^(c S - m)    bf16, written back to tensor memory over S
//   O = O + P V        in tensor memory; l = l + row sums of P (float32, before P's rounding)
// and at the end o = O / l, lse = (m + log2 l) ln 2.  O is scaled by 2^(m - m') only when some row's maximum has
// grown by more than 8 (P stays below 2^8, so float32 sums and bf16's range are far from their ends).
//
// Work split.  All (row tile, cache tile) pairs of the batch lie on one line; CTA c of C takes the c-th part of
// it (a persistent CTA per SM).  A row tile whose line part crosses CTAs leaves partial (O, m, l) in the workspace,
// and join_kernel adds them.  So one long context and many short ones load the SMs alike.
//
// Roles in a CTA: warp 0 copies tiles (TMA, page by page, through a ring of stages); one thread of warp 1 issues the
// products; warps 2 to 5 own a row per thread: they load Q, turn S into P and read O.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "sv_device.cuh"
#include "sv_ops.h"

namespace sv {
namespace {

constexpr int kTile = 128;                 // rows of Q, and slots of the cache, in a tile
constexpr int kSoftThreads = 128;
constexpr int kThreads = 64 + kSoftThreads;
constexpr int kHalfBytes = kTile * 128;    // 128 slots of 64 bf16: one swizzled column block
constexpr int kTmemColumns = 512;
constexpr int kColS = 0, kColO = 256;      // S / P buffers at columns 0 and 128, O at 256
constexpr float kLazyGrowth = 8.0f;        // log2 units by which a maximum may grow without a rescale of O
constexpr int kJoinRows = 16;              // rows per CTA of the join

// Stages of 32 KB (D = 128) or 16 KB: five tiles' halves in flight keep about 160 KB on the way per SM.
template <int D>
struct Shape {
  static constexpr int kHalves = D / 64;
  static constexpr int kStageBytes = kHalves * kHalfBytes;
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kQBytes = kHalves * kHalfBytes;
};

struct alignas(16) Job {  // a row tile that several CTAs worked on: parts of CTAs `first` to `last`
  int32_t valid, request, head, mtile, rows, first, last, pad;
};

struct AttendParams {
  const __nv_bfloat16* q;
  int64_t q_row_stride, q_head_stride, out_row_stride, out_head_stride;
  const int32_t *table, *seq_len, *node_offsets, *parent;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
  int32_t* any_bad;   // [2]: some request is bad; CTAs of the join that are done with that
  uint8_t* bad;       // [SV_MAX_BATCH] requests whose outputs become 0
  Job* jobs;          // [grid]
  float* parts;       // [2 grid] partial results
  int64_t n_rows;
  int32_t width, B, Nmax, pages, shift, q_heads, kv_heads, group, window, sinks;
  float scale;
};

// Floats of one partial result: O as [D / 4][128 rows][4], then m and l per row.
template <int D>
constexpr int part_floats() { return kTile * D + 2 * kTile; }

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
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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
__device__ __forceinline__ Request request_of(const AttendParams& a, int i) {
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
  r.mtiles = (r.nodes * a.group + kTile - 1) / kTile;
  return r;
}

// A stretch of cache tiles [kv0, kv1) of one row tile.
struct Segment {
  Request r;
  int32_t request, head, mtile, kv0, kv1;
};
__device__ __forceinline__ Segment segment_at(const AttendParams& a, const uint32_t* before, uint32_t t, uint32_t end) {
  int lo = 0, hi = a.B;  // the last request whose tiles begin at or before t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= t) lo = mid; else hi = mid;
  }
  Segment s;
  s.request = lo;
  s.r = request_of(a, lo);
  const uint32_t local = t - before[lo], unit = local / static_cast<uint32_t>(s.r.tiles);
  s.kv0 = static_cast<int>(local - unit * s.r.tiles);
  s.kv1 = static_cast<int>(min(static_cast<uint32_t>(s.r.tiles), s.kv0 + (end - t)));
  s.head = static_cast<int>(unit / s.r.mtiles);   // a head's row tiles are neighbours: they share its tiles in L2
  s.mtile = static_cast<int>(unit - static_cast<uint32_t>(s.head) * s.r.mtiles);
  return s;
}
__device__ __forceinline__ int tile_slot(const Request& r, int j) {
  return (j < r.sink_tiles ? j : r.near_tile + (j - r.sink_tiles)) * kTile;
}
__device__ __forceinline__ uint32_t part_begin(uint32_t total, uint32_t c, uint32_t n) {
  return static_cast<uint32_t>(static_cast<uint64_t>(total) * c / n);
}

// Bits [lo, hi) of a 32-bit word whose bit 0 stands for position `at`.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int at) {
  const int a = max(lo - at, 0), b = min(hi - at, 32);
  if (b <= a) return 0u;
  return (b == 32 ? 0xFFFFFFFFu : (1u << b) - 1u) & ~((1u << a) - 1u);
}

template <int D>
struct Smem {
  alignas(1024) unsigned char q[Shape<D>::kQBytes];
  alignas(1024) unsigned char stage[Shape<D>::kStages][Shape<D>::kStageBytes];
  alignas(16) uint64_t full[Shape<D>::kStages];
  uint64_t empty[Shape<D>::kStages];
  uint64_t s_full[2], p_full[2], pv_done, q_full;
  uint32_t tmem;
  volatile int32_t dead;       // a wait ran out: everyone leaves
  uint32_t scan[kThreads / 32 + 1];
  int32_t parent[SV_MAX_DRAFT + 1];
  uint32_t before[1];          // [B + 1] tiles of the requests before
};

__device__ __forceinline__ bool wait_or_leave(uint64_t* bar, uint32_t parity, volatile int32_t* dead, uint32_t* status) {
  if (*dead) return false;
  if (mbar_wait(bar, parity, status)) return true;
  *dead = 1;
  return false;
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const AttendParams a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  using Sh = Shape<D>;
  extern __shared__ unsigned char dyn[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < Sh::kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], kSoftThreads);
    }
    mbar_init(&sm.pv_done, 1);
    mbar_init(&sm.q_full, kSoftThreads);
    sm.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == 1) tmem_alloc(&sm.tmem);
  pdl_wait();
  pdl_trigger();
  // tiles before each request
  uint32_t total;
  {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int i0 = tid * per, i1 = min(a.B, i0 + per);
    uint32_t sum = 0;
    for (int i = i0; i < i1; ++i) {
      const Request r = request_of(a, i);
      if (r.bad != 0 && blockIdx.x == 0) mark_bad(a, i, r.bad);
      sm.before[i] = sum;
      sum += static_cast<uint32_t>(r.tiles) * r.mtiles * a.kv_heads;
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
    for (int i = i0; i < i1; ++i) sm.before[i] += at;
    __syncthreads();
  }
  const uint32_t tmem = sm.tmem;
  // every part holds a tile: with fewer tiles than CTAs the last CTAs have none
  const uint32_t parts = min(gridDim.x, total);
  const uint32_t t0 = blockIdx.x < parts ? part_begin(total, blockIdx.x, parts) : total;
  const uint32_t t1 = blockIdx.x < parts ? part_begin(total, blockIdx.x + 1, parts) : total;
  uint32_t loaded = 0;  // stages that the producer filled

  if (warp == 0) {
    // ---- copies -----------------------------------------------------------------------------------
    const int box = min(kTile, 1 << a.shift), chunks = kTile / box;  // pages (or one part of a page) per tile
    bool go = true;
    for (uint32_t t = t0; t < t1 && go;) {
      const Segment s = segment_at(a, sm.before, t, t1);
      const int end = s.r.len + s.r.nodes, lo = a.window > 0 ? max(0, s.r.len - a.window + 1) : 0;
      const int32_t* row = a.table + static_cast<int64_t>(s.request) * a.width;
      for (int j = s.kv0; j < s.kv1 && go; ++j) {
        const int s0 = tile_slot(s.r, j);
        // lane x < chunks looks its page up; a page without a visible slot is left out
        int page = -1;
        bool wanted = false;
        if (lane < chunks) {
          const int at = s0 + lane * box;
          wanted = at < end && (a.window <= 0 || at < a.sinks || at + box > lo);
          if (wanted) {
            page = row[at >> a.shift];
            if (page < 0 || page >= a.pages) {
              mark_bad(a, s.request, SV_DEV_BAD_PAGE);
              page = a.pages;  // outside the tensor: the copy fills zeros
            }
          }
        }
        const int bytes = __popc(__ballot_sync(0xFFFFFFFFu, wanted)) * Sh::kHalves * box * 128;
        for (int kv = 0; kv < 2; ++kv, ++loaded) {
          const uint32_t st = loaded % Sh::kStages, round = loaded / Sh::kStages;
          if (round > 0) go = warp_wait(&sm.empty[st], (round - 1) & 1, &sm.dead, a.status);
          if (!go) break;
          if (lane == 0) mbar_arrive_expect_tx(&sm.full[st], bytes);
          __syncwarp();
          if (wanted) {
#pragma unroll
            for (int h = 0; h < Sh::kHalves; ++h)
              tma_load_4d(sm.stage[st] + h * kHalfBytes + lane * box * 128, kv ? &v_map : &k_map, h * 64, s.head,
                          (s0 + lane * box) & ((1 << a.shift) - 1), page, &sm.full[st]);
          }
        }
      }
      t += s.kv1 - s.kv0;
    }
  } else if (warp == 1) {
    // ---- products ---------------------------------------------------------------------------------
    if (lane == 0) {
      constexpr uint32_t kDescS = instr_desc(kTile, false), kDescO = instr_desc(D, true);
      const uint32_t q_addr = smem_u32(sm.q);
      auto scores = [&](uint32_t n) {  // S of the n-th tile of this CTA
        const uint32_t st = (2 * n) % Sh::kStages, round = (2 * n) / Sh::kStages;
        if (!wait_or_leave(&sm.full[st], round & 1, &sm.dead, a.status)) return;
        tc_after_sync();
        const uint32_t k_addr = smem_u32(sm.stage[st]);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k / 4) * kHalfBytes + (k % 4) * 32;
          mma_ss(tmem + kColS + (n & 1) * kTile, smem_desc(q_addr + off, 16, 1024), smem_desc(k_addr + off, 16, 1024), kDescS, k > 0);
        }
        tc_commit(&sm.s_full[n & 1]);
        tc_commit(&sm.empty[st]);
      };
      uint32_t n = 0, seg = 0;
      for (uint32_t t = t0; t < t1 && !sm.dead; ++seg) {
        const Segment s = segment_at(a, sm.before, t, t1);
        const int tiles = s.kv1 - s.kv0;
        if (!wait_or_leave(&sm.q_full, seg & 1, &sm.dead, a.status)) break;
        // S's buffer of tile n was last read by the product P V of tile n - 2 (and the barrier can
        // only be asked about its latest phase)
        if (n >= 1 && !wait_or_leave(&sm.pv_done, (n - 1) & 1, &sm.dead, a.status)) break;
        scores(n);
        for (int j = 0; j < tiles && !sm.dead; ++j, ++n) {
          if (j + 1 < tiles) {
            if (n >= 1 && !wait_or_leave(&sm.pv_done, (n - 1) & 1, &sm.dead, a.status)) break;
            scores(n + 1);
          }
          const uint32_t st = (2 * n + 1) % Sh::kStages, round = (2 * n + 1) / Sh::kStages;
          if (!wait_or_leave(&sm.full[st], round & 1, &sm.dead, a.status)) break;
          if (!wait_or_leave(&sm.p_full[n & 1], (n >> 1) & 1, &sm.dead, a.status)) break;
          tc_after_sync();
          const uint32_t v_addr = smem_u32(sm.stage[st]);
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            mma_ts(tmem + kColO, tmem + kColS + (n & 1) * kTile + k * 8, smem_desc(v_addr + k * 2048, kHalfBytes, 1024), kDescO,
                   j > 0 || k > 0);
          tc_commit(&sm.pv_done);
          tc_commit(&sm.empty[st]);
        }
        t += tiles;
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: thread r has row r of the tile ---------------------------------------------------
    const int r = (warp & 3) * 32 + lane;
    const uint32_t my = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const float c = a.scale * 1.44269504088896341f;
    uint32_t n = 0;
    // Q's rows of a segment, in the swizzled layout of its product, and the tree's parents
    auto load_q = [&](const Segment& s) {
      const int rows = min(kTile, s.r.nodes * a.group - s.mtile * kTile);
      // neighbouring threads take neighbouring 16-byte pieces of a row
      for (int x = tid - 64; x < rows * (D / 8); x += kSoftThreads) {
        const int row = x / (D / 8), piece = x % (D / 8);
        const int at = s.mtile * kTile + row, node = at / a.group, g = at - node * a.group;
        const uint4 v = *reinterpret_cast<const uint4*>(a.q + (s.r.first + node) * a.q_row_stride +
                                                        (s.head * a.group + g) * a.q_head_stride + piece * 8);
        *reinterpret_cast<uint4*>(sm.q + (piece >> 3) * kHalfBytes + row * 128 + (((piece & 7) ^ (row & 7)) << 4)) = v;
      }
      if (a.parent != nullptr)
        for (int x = tid - 64; x < s.r.nodes; x += kSoftThreads) sm.parent[x] = a.parent[s.r.first + x];
      fence_proxy_async_smem();
      mbar_arrive(&sm.q_full);
    };
    auto parent_of = [&](int node) { return a.parent != nullptr ? sm.parent[node] : node - 1; };
    Segment s;
    if (r == 0) a.jobs[blockIdx.x].valid = 0;
    if (t0 < t1) {
      s = segment_at(a, sm.before, t0, t1);
      load_q(s);
    }
    uint32_t seg = 0;
    for (uint32_t t = t0; t < t1; ++seg) {
      if (!warp_wait(&sm.q_full, seg & 1, &sm.dead, a.status)) break;  // the parents are there for every thread
      const int rows = min(kTile, s.r.nodes * a.group - s.mtile * kTile);
      const bool active = (warp & 3) * 32 < rows;  // some row of this warp exists
      const int at = s.mtile * kTile + r;
      const int node = r < rows ? at / a.group : 0;
      const int len = s.r.len, end = len + s.r.nodes;
      const int lo = a.window > 0 ? max(0, len - a.window + 1) : 0;  // before it (and past the sinks) no node sees a slot
      // depth, and a check of the path
      int depth = 0;
      if (r < rows)
        for (int p = node; p > 0; ++depth) {
          const int up = parent_of(p);
          if (up < 0 || up >= p) {
            mark_bad(a, s.request, SV_DEV_BAD_PARENT);
            break;
          }
          p = up;
        }
      const int near = a.window > 0 ? len + depth - a.window + 1 : 0;  // first position of the window
      float m = -INFINITY, l = 0.0f;
      for (int j = s.kv0; j < s.kv1; ++j, ++n) {
        if (!warp_wait(&sm.s_full[n & 1], (n >> 1) & 1, &sm.dead, a.status)) break;
        tc_after_sync();
        const int s0 = tile_slot(s.r, j);
        const bool whole = s0 + kTile <= len && (a.window <= 0 || s0 + kTile <= a.sinks || s0 >= len + s.r.nodes - a.window);
        if (!whole && (s0 + kTile > end || (a.window > 0 && s0 < lo && s0 + kTile > a.sinks))) {
          // slots that no node sees may hold anything: 0 times it has to be 0
          const uint32_t v = 2 * n + 1, st = v % Sh::kStages;
          if (!warp_wait(&sm.full[st], (v / Sh::kStages) & 1, &sm.dead, a.status)) break;
          const int slot = s0 + r;
          if (slot >= end || (slot < lo && slot >= a.sinks)) {
#pragma unroll
            for (int x = 0; x < D / 8; ++x)
              *reinterpret_cast<uint4*>(sm.stage[st] + (x >> 3) * kHalfBytes + r * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (active) {
          uint32_t x[kTile];
          const uint32_t s_addr = my + kColS + (n & 1) * kTile;
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_load32(s_addr + 32 * i, x + 32 * i);
          tmem_wait_load();
          if (!whole) {
            uint32_t see[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int p = s0 + 32 * w;
              see[w] = range_bits(near, len, p) | (a.window > 0 ? range_bits(0, min(a.sinks, len), p) : 0u);
            }
            if (s0 + kTile > len && r < rows) {
              int d = depth;
              for (int up = node;; --d) {
                const int b = len + up - s0;
                if (b >= 0 && b < kTile && (len + d >= near || len + d < a.sinks)) {
#pragma unroll
                  for (int w = 0; w < 4; ++w)
                    if ((b >> 5) == w) see[w] |= 1u << (b & 31);
                }
                if (up <= 0 || d <= 0 || b < 0) break;
                up = parent_of(up);
              }
            }
#pragma unroll
            for (int i = 0; i < kTile; ++i)
              if (!((see[i >> 5] >> (i & 31)) & 1u)) x[i] = 0xFF800000u;
          }
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < kTile; ++i) top = fmaxf(top, __uint_as_float(x[i]));
          top *= c;  // c > 0
          const bool grow = top > m + kLazyGrowth || (m == -INFINITY && top > -INFINITY);
          if (j == s.kv0) {
            m = top;
          } else if (__any_sync(0xFFFFFFFFu, grow)) {
            const float keep = grow ? (m == -INFINITY ? 0.0f : ex2_approx(m - top)) : 1.0f;
            if (grow) m = top;
            l *= keep;
            // O is complete up to the tile before
            if (!warp_wait(&sm.pv_done, (n - 1) & 1, &sm.dead, a.status)) break;
            tc_after_sync();
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              uint32_t o[32];
              tmem_load32(my + kColO + 32 * i, o);
              tmem_wait_load();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
              tmem_store32(my + kColO + 32 * i, o);
            }
          }
          const float off = m == -INFINITY ? 0.0f : -m;
          float sum0 = 0.0f, sum1 = 0.0f;
          const f32x2 c2 = f2_pack(c, c), off2 = f2_pack(off, off);
#pragma unroll
          for (int i = 0; i < kTile; i += 2) {
            float e0, e1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), c2, off2), e0, e1);
            e0 = ex2_approx(e0);
            e1 = ex2_approx(e1);
            sum0 += e0;
            sum1 += e1;
            x[i >> 1] = pack_bf16(e0, e1);
          }
          l += sum0 + sum1;
          tmem_store32(s_addr, x);
          tmem_store32(s_addr + 32, x + 32);
          tmem_wait_store();
        }
        tc_before_sync();
        mbar_arrive(&sm.p_full[n & 1]);
      }
      // the next segment's Q can go in: every product with this one's is complete
      const Segment done = s;
      t += s.kv1 - s.kv0;
      // every thread has arrived with its last tile: none still reads the parents
      if (!warp_wait(&sm.p_full[(n - 1) & 1], ((n - 1) >> 1) & 1, &sm.dead, a.status)) break;
      if (t < t1) {
        s = segment_at(a, sm.before, t, t1);
        load_q(s);
      }
      if (!warp_wait(&sm.pv_done, (n - 1) & 1, &sm.dead, a.status)) break;
      tc_after_sync();
      const bool complete = done.kv0 == 0 && done.kv1 == done.r.tiles;
      if (active) {
        if (complete) {
          const float inv = l > 0.0f ? 1.0f / l : 0.0f;
          const int g = at - node * a.group;
          const int64_t row = done.r.first + node;
          const int head = done.head * a.group + g;
          __nv_bfloat16* out = a.out + row * a.out_row_stride + head * a.out_head_stride;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            tmem_load32(my + kColO + 32 * i, o);
            tmem_wait_load();
            if (r < rows) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint4 w;
                w.x = pack_bf16(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                w.y = pack_bf16(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
                w.z = pack_bf16(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv);
                w.w = pack_bf16(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv);
                *reinterpret_cast<uint4*>(out + 32 * i + e) = w;
              }
            }
          }
          if (r < rows && a.lse != nullptr) a.lse[row * a.q_heads + head] = (m + log2f(l)) * 0.693147180559945309f;
        } else {
          float* part = a.parts + static_cast<int64_t>(2 * blockIdx.x + (done.kv0 == 0)) * part_floats<D>();
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t o[32];
            tmem_load32(my + kColO + 32 * i, o);
            tmem_wait_load();
            if (r < rows) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<uint4*>(part + ((8 * i + e / 4) * kTile + r) * 4) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
          if (r < rows) {
            part[kTile * D + r] = m;
            part[kTile * D + kTile + r] = l;
          }
        }
      }
      tc_before_sync();
      if (r == 0 && done.kv0 == 0 && !complete) {
        // the CTA in which the row tile ends
        const uint32_t last = t - 1 + (done.r.tiles - done.kv1);
        uint32_t e = static_cast<uint32_t>(static_cast<uint64_t>(last) * parts / total);
        while (part_begin(total, e + 1, parts) <= last) ++e;
        Job job = {1, done.request, done.head, done.mtile, rows, static_cast<int32_t>(blockIdx.x), static_cast<int32_t>(e), 0};
        a.jobs[blockIdx.x] = job;
      }
    }
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  if (sm.dead && warp == 0)  // copies in flight land before the CTA leaves
    for (uint32_t x = loaded > Sh::kStages ? loaded - Sh::kStages : 0; x < loaded; ++x)
      mbar_wait(&sm.full[x % Sh::kStages], (x / Sh::kStages) & 1, a.status);
  if (warp == 1) tmem_free(tmem);
}

// Adds the partial results of row tile `jobs[x]`: with M = max m_i, o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// grid (CTAs of the attention, row groups).  Then the outputs of bad requests become 0.
template <int D>
__global__ void __launch_bounds__(128) join_kernel(const AttendParams a) {
  pdl_wait();
  const Job job = a.jobs[blockIdx.x];
  const int row0 = blockIdx.y * kJoinRows;
  if (job.valid != 0 && row0 < job.rows && !a.bad[job.request]) {
    constexpr int kPieces = D / 4;
    const int n = job.last - job.first + 1;
    for (int x = threadIdx.x; x < kJoinRows * kPieces; x += 128) {
      const int r = row0 + x % kJoinRows, piece = x / kJoinRows;
      if (r >= job.rows) continue;
      float M = -INFINITY, L = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int i = 0; i < n; ++i) {
        const float* part = a.parts + static_cast<int64_t>(2 * (job.first + i) + (i == 0)) * part_floats<D>();
        M = fmaxf(M, part[kTile * D + r]);
      }
      for (int i = 0; i < n; ++i) {
        const float* part = a.parts + static_cast<int64_t>(2 * (job.first + i) + (i == 0)) * part_floats<D>();
        const float m = part[kTile * D + r];
        const float w = m == -INFINITY ? 0.0f : ex2_approx(m - M);
        const float4 v = *reinterpret_cast<const float4*>(part + (piece * kTile + r) * 4);
        L += w * part[kTile * D + kTile + r];
        o[0] += w * v.x;
        o[1] += w * v.y;
        o[2] += w * v.z;
        o[3] += w * v.w;
      }
      const float inv = L > 0.0f ? 1.0f / L : 0.0f;
      const int at = job.mtile * kTile + r, node = at / a.group, head = job.head * a.group + (at - node * a.group);
      const int64_t row = a.node_offsets[job.request] + node;
      uint2 w;
      w.x = pack_bf16(o[0] * inv, o[1] * inv);
      w.y = pack_bf16(o[2] * inv, o[3] * inv);
      *reinterpret_cast<uint2*>(a.out + row * a.out_row_stride + head * a.out_head_stride + piece * 4) = w;
      if (piece == 0 && a.lse != nullptr) a.lse[row * a.q_heads + head] = (M + log2f(L)) * 0.693147180559945309f;
    }
  }
  if (*a.any_bad != 0) {
    const int blocks = gridDim.x * gridDim.y, me = blockIdx.y * gridDim.x + blockIdx.x;
    for (int i = me; i < a.B; i += blocks) {
      if (!a.bad[i]) continue;
      const int64_t first = max(int64_t(0), static_cast<int64_t>(a.node_offsets[i]));
      const int64_t last = min(a.n_rows, static_cast<int64_t>(a.node_offsets[i + 1]));
      for (int64_t row = first; row < last; ++row) {
        for (int x = threadIdx.x; x < a.q_heads * (D / 8); x += 128)
          *reinterpret_cast<uint4*>(a.out + row * a.out_row_stride + (x / (D / 8)) * a.out_head_stride + (x % (D / 8)) * 8) =
              make_uint4(0, 0, 0, 0);
        if (a.lse != nullptr)
          for (int x = threadIdx.x; x < a.q_heads; x += 128) a.lse[row * a.q_heads + x] = -INFINITY;
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
      for (int i = threadIdx.x; i < a.B; i += 128) a.bad[i] = 0;
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
constexpr int kMaxCtas = 152;  // SMs of the GPU: one CTA each

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

template <int D>
cudaError_t launch_attention(const AttendParams& a, const CUtensorMap& k_map, const CUtensorMap& v_map, int ctas, void* stream) {
  const size_t dyn = sizeof(Smem<D>) + sizeof(uint32_t) * a.B + 1024;
  cudaError_t e = cudaFuncSetAttribute(attend_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(dyn));
  if (e != cudaSuccess) return e;
  e = launch_dependent(attend_kernel<D>, dim3(ctas), kThreads, dyn, stream, SV_KERNEL_ATTENTION, 1, a, k_map, v_map);
  if (e != cudaSuccess) return e;
  const int groups = (std::min(kTile, a.Nmax * a.group) + kJoinRows - 1) / kJoinRows;
  return launch_dependent(join_kernel<D>, dim3(ctas, groups), 128, 0, stream, SV_KERNEL_ATTENTION_JOIN, 1, a);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t sv_attention_workspace_size(const sv_cache* c, int q_heads) {
  if (check_cache(c) != SV_OK || q_heads < 1 || q_heads % c->kv_heads != 0) return 0;
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
  if (q_heads < 1 || q_heads % c->kv_heads != 0)
    return set_error(SV_ERR_INVALID_ARG, "q_heads=%d is no multiple of kv_heads=%d", q_heads, c->kv_heads);
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
  // the line of work is counted in 32 bits
  const int64_t tiles = ((static_cast<int64_t>(table_width) * c->page_size + kTile - 1) / kTile + 1) *
                        ((static_cast<int64_t>(Nmax) * (q_heads / c->kv_heads) + kTile - 1) / kTile);
  if (tiles > INT_MAX || tiles * c->kv_heads > INT_MAX || tiles * c->kv_heads * B > INT_MAX)
    return set_error(SV_ERR_INVALID_ARG, "B=%d requests of up to %lld tiles a head are too many for one call", B, (long long)tiles);
  const size_t offset = static_cast<size_t>(layer) * c->layer_stride * 2;
  CUtensorMap k_map, v_map;
  if (!encode_pool(&k_map, c, static_cast<const unsigned char*>(c->k) + offset) ||
      !encode_pool(&v_map, c, static_cast<const unsigned char*>(c->v) + offset))
    return set_error(SV_ERR_CUDA, "the cache's strides or sizes cannot be described to the copy engine");
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return launch_status(e, "device");
  const int ctas = std::min(sms, kMaxCtas);
  const Layout L = layout_of(kMaxCtas, c->head_dim);
  unsigned char* w = static_cast<unsigned char*>(ws);
  AttendParams a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_row_stride = q_row_stride;
  a.q_head_stride = q_head_stride;
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
  a.group = q_heads / c->kv_heads;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale;
  return launch_status(c->head_dim == 128 ? launch_attention<128>(a, k_map, v_map, ctas, stream)
                                          : launch_attention<64>(a, k_map, v_map, ctas, stream),
                       "attention");
}

}  // extern "C"
