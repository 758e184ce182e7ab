// sv_tree_attention4: a token tree's queries against a paged cache held in 4 bits.
//
// A warp holds a row tile of 8 or 16 rows (query heads that share a key/value head, times nodes) and goes over its share of the
// cache in chunks of 32 slots.  With c = scale k_scale log2(e) and running maximum m:
//   S' = K Q' [32 x rows];  P' = 2^(c S' - m) in float16;  O' = O' + V' P' [D x rows], all sums in float32
// (' = transposed) and at the end o = v_scale O / sum P, lse = (m + log2 sum P) ln 2.  The cache is the 16-row operand of the
// 16 x 8 x 16 products and the queries the 8-column one, so few rows waste little: one decoded token has 4 or 8.
//
// Exactness.  A code times its e4m3 scale has at most six significant bits and lies in [2^-10, 2688]: it is a float16 without
// rounding.  A query row is scaled by a power of two so that its largest element lies in [2^14, 2^15); elements down to 2^-28
// of it keep all bits of their bf16.  So the products are those of the stored values, in float32 sums.  P is rounded to
// float16 (half a step is 2^-12 of it; below 2^-14, of a maximum between 2^kBias and 2^(kBias + kLazyGrowth), 2^-25).
//
// Layout.  The chunk is one contiguous copy (36 D bytes) per page, by the warp itself, through a ring of its own: no barrier
// is shared between warps.  In a group of eight slots a lane's codes are 16 (8 for D = 64) neighbouring bytes, in lane order: for K
// the slot lane / 4 and a quarter of its dimensions, whose order in the product is free as long as Q's is the same; for V two
// neighbouring slots and an eighth of the dimensions.  So codes go from shared memory to the fragments through registers
// only: per pair of elements a conversion and a multiplication by the scales.  P' comes out of the first product with a slot's
// rows in a lane and goes into the second with a row's slots: 8 x 8 blocks are transposed by movmatrix.
//
// Work split.  All (row tile, chunk) pairs of the batch lie on one line, and before each row tile a few places for what
// beginning and ending it costs; every warp of the grid takes an equal part of the line, in segments: stretches of one row
// tile.  Warps share nothing but the SM, so one's loads of Q and results run beside another's products.  A row tile that
// crosses warps leaves partial results in the workspace, which join4_kernel adds.
//
// Measured (GB300, 32 query and 8 key/value heads of 128, graph replay; a copy of the bytes read in brackets): 64 requests of one
// token over 6k to 8k slots 110 us (77), four of up to 130 slots 14.4 us; a window of 1024 with 16 heads of 64, 33 trees of up to
// 16 nodes 44 us (6).  A chunk takes 640 instructions, of them 256 that turn codes into products' operands; with 16 warps of 128
// registers 62% of the issue slots are used and as much of the memory's pace.  Short calls are latency: two launches, the line's
// scan, a row tile's chain.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "sv_decode4.cuh"
#include "sv_device.cuh"
#include "sv_line.cuh"
#include "sv_ops.h"

namespace sv {
namespace {

constexpr int kChunk = 32;                // slots that a warp takes at a time
// Row tiles of N columns of eight.  Warps: as many as the registers leave room for, so that their latencies overlap.
template <int N>
struct Tile4 {
  static constexpr int kRows = 8 * N;
  static constexpr int kWarps = N == 1 ? 16 : 8;
  static constexpr int kThreads = 32 * kWarps;
};
constexpr int kMaxWarps = 16;
constexpr float kLazyGrowth4 = 8.0f;      // log2 units by which a maximum may grow without a rescale of O
constexpr float kBias = 4.0f;             // P is 2^kBias at the maximum that it is scaled to
// Places of the line for a row tile's beginning and end, in chunks (the window's 33 trees 62 us at 1, 50 at 2, 43 at 4, 42 at 8; 64
// contexts of 100 to 1000 30.9, 30.8, 30.8, 32.3).
constexpr int kExtra4 = 4;
constexpr int kMaxStages4 = 4;
// Rows above which tiles of 128 rows take the call (32 requests of 1000 to 8000 slots: 16 rows 64 us here, 100 there; 24 rows 110
// and 100, 48 rows 157 and 101).
constexpr int kTilesFrom = 16;

struct Attend4Params : Line, Marks, Outputs {
  const __nv_bfloat16* q;
  int64_t q_row_stride, q_head_stride;
  const unsigned char* pool;     // of the layer
  int64_t page_stride, head_stride;
  const int32_t *table, *parent;
  int32_t* n_jobs;    // [2] row tiles to join; CTAs of the join that are done (both zero between calls)
  Job* jobs;          // [warps of the grid]
  float* parts;       // [2 warps of the grid] partial results
  int32_t pages, kv_heads, stages;
  float scale;        // with k_scale
  float v_scale;
};

// Floats of one partial result: O [rows][D], then m and the sum per row.
template <int D, int N>
constexpr int part4_floats() { return 8 * N * (D + 2); }

constexpr int kQueue = kMaxStages4 + 2;   // segments between a warp's copies and its products: one per chunk in flight, and the ends

struct Smem4 {
  Line line;
  uint64_t full[kMaxWarps][kMaxStages4];
  Segment queue[kMaxWarps][kQueue];
  uint32_t scan[kMaxWarps];
  volatile int32_t dead;       // a wait ran out: the launch finishes on what it holds
};

// D += A B: 16 x 16 by 16 x 8.
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The transpose of an 8 x 8 block: lane 4 i + j has elements 2 j and 2 j + 1 of row i.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
}
// Over the lanes of the same lane % 4.
__device__ __forceinline__ float column_max(float x) {
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
  return x;
}
__device__ __forceinline__ float column_sum(float x) {
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
  return x;
}

template <int D, int N>
__global__ void __launch_bounds__(Tile4<N>::kThreads, 1) attend4_kernel(const Attend4Params a) {
  constexpr int kRows = Tile4<N>::kRows, kWarps = Tile4<N>::kWarps, kThreads4 = Tile4<N>::kThreads;
  constexpr int kGroupBytes = 9 * D;                       // eight slots
  constexpr int kChunkBytes = kChunk / 8 * kGroupBytes;
  constexpr int kSteps = D / 16;                           // products over the dimensions
  constexpr int kWords = D / 32;                           // words of a lane's codes in a group: 4 or 2
  constexpr int kDimTiles = D / 16;                        // 16-row tiles of O'
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ Smem4 sm;
  uint32_t* before = reinterpret_cast<uint32_t*>(dyn + static_cast<size_t>(kWarps) * a.stages * kChunkBytes);  // [B]
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int g = lane >> 2, t4 = lane & 3;
  // (a barrier a thread: by one thread they take 2 us)
  for (int i = tid; i < kWarps * kMaxStages4; i += kThreads4) mbar_init(&sm.full[i / kMaxStages4][i % kMaxStages4], 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  fence_proxy_async_smem();
  if (tid == 0) {
    sm.dead = 0;
    sm.line = a;
  }
  pdl_wait();
  pdl_trigger();
  // places of the line before each request
  uint32_t total;
  {
    const int per = (a.B + kThreads4 - 1) / kThreads4;
    const int i0 = min(a.B, tid * per), i1 = min(a.B, i0 + per);
    uint32_t sum = 0;
    for (int i = i0; i < i1; ++i) {
      const Request r = request_of<kChunk>(a, i);
      if (r.bad != 0 && blockIdx.x == 0) mark_bad(a, i, r.bad);
      before[i] = sum;
      sum += static_cast<uint32_t>(r.tiles + a.extra) * r.mtiles * a.kv_heads;
    }
    uint32_t x = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) sm.scan[warp] = x;
    __syncthreads();
    uint32_t at = x - sum;
    total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += sm.scan[w];
      total += sm.scan[w];
    }
    for (int i = i0; i < i1; ++i) before[i] += at;
    __syncthreads();
  }
  // parts are dealt out CTA by CTA: with fewer places than warps every SM has some
  const uint32_t me = warp * gridDim.x + blockIdx.x;
  const Parts parts(total, max(1u, min(gridDim.x * kWarps, total)));
  const uint32_t t0 = min(parts.begin(me), total), t1 = min(parts.begin(me + 1), total);

  // ---- copies: this warp's chunks in the order of the line -------------------------------------------
  unsigned char* ring = dyn + static_cast<size_t>(warp) * a.stages * kChunkBytes;
  const int piece_shift = min(5, a.shift);                   // slots per copy: a page, or 32 slots of one
  const bool copies = lane < (kChunk >> piece_shift);        // this lane copies the lane-th piece
  uint32_t asked = 0, used = 0;                              // chunks that were asked for, and used
  uint32_t ask_stage = 0, use_stage = 0, use_parity = 0;
  uint32_t ask_t = t0, found = 0;                            // place of the next segment to look for, segments found
  Segment load = {};
  int load_j = 0, load_end = 0, block = -1, page_now = -1;   // pages of 32 entries at a time
  // Finds the next chunk to ask for: false = there is none in this part.
  auto settle = [&]() {
    if (load_j < load_end) return true;
    while (ask_t < t1) {
      load = segment_at<kChunk>(sm.line, before, ask_t, t1);
      ask_t = load.next;
      if (load.kv0 >= load.kv1) continue;                    // (only places before a row tile's chunks)
      if (lane == 0) sm.queue[warp][found % kQueue] = load;
      ++found;
      // its rows of Q, before its chunks: loads behind a ring's copies wait for all of them
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int row = load.mtile * kRows + 8 * n + g;
        if (row < load.r.nodes * a.group) {
          const int node = row / a.group;
          const __nv_bfloat16* q = a.q + (load.r.first + node) * a.q_row_stride + (load.head * a.group + row - node * a.group) * a.q_head_stride + t4 * (D / 4);
          asm volatile("prefetch.global.L1 [%0];" ::"l"(q));
        }
      }
      load_j = load.kv0;
      load_end = load.kv1;
      block = -1;
      return true;
    }
    return false;
  };
  bool more = settle();
  bool page_there = false;
  const unsigned char* page_at = nullptr;
  // page numbers of 32 entries from a multiple of 32 on
  auto pages_from = [&](int entry) {
    if ((entry >> 5) == block) return;
    block = entry >> 5;
    const int e = 32 * block + lane;
    page_now = (static_cast<int64_t>(e) << a.shift) < load.r.len + load.r.nodes ? a.table[static_cast<int64_t>(load.request) * a.width + e] : -1;
  };
  auto ask = [&]() {
    const int s0 = tile_slot<kChunk>(load.r, load_j);
    constexpr int kUnit = kGroupBytes / 8;                    // bytes of a slot
    uint64_t* bar = &sm.full[warp][ask_stage];
    if (a.shift >= 5) {  // one copy, of a page that is looked up where it begins, or where the chunk does not follow the last one
      const int in_page = s0 & ((1 << a.shift) - 1);
      if (in_page == 0 || block < 0 || load_j == load.r.sink_tiles) {
        const int entry = s0 >> a.shift;
        pages_from(entry);
        const int page = __shfl_sync(0xFFFFFFFFu, page_now, entry & 31);
        page_there = page >= 0 && page < a.pages;
        if (!page_there) mark_bad(a, load.request, SV_DEV_BAD_PAGE);
        page_at = a.pool + page * a.page_stride + load.head * a.head_stride;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, page_there ? kChunkBytes : 0);
        if (page_there) bulk_g2s(ring + ask_stage * kChunkBytes, page_at + in_page * kUnit, kChunkBytes, bar);
      }
      __syncwarp();
    } else {
      const int entry = s0 >> a.shift, slot = s0 + (lane << piece_shift);
      pages_from(entry);
      const int page = __shfl_sync(0xFFFFFFFFu, page_now, (entry + lane) & 31);
      bool wanted = copies && slot < load.r.len + load.r.nodes;
      if (a.window > 0) wanted = wanted && (slot < a.sinks || slot + (1 << piece_shift) > load.r.len - a.window + 1);
      if (wanted && (page < 0 || page >= a.pages)) {
        mark_bad(a, load.request, SV_DEV_BAD_PAGE);
        wanted = false;
      }
      const int bytes = (__popc(__ballot_sync(0xFFFFFFFFu, wanted)) << piece_shift) * kUnit;
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      if (wanted)
        bulk_g2s(ring + ask_stage * kChunkBytes + (lane << piece_shift) * kUnit,
                 a.pool + page * a.page_stride + load.head * a.head_stride + (slot & ((1 << a.shift) - 1)) * kUnit,
                 kUnit << piece_shift, bar);
    }
    ask_stage = ask_stage + 1 == static_cast<uint32_t>(a.stages) ? 0 : ask_stage + 1;
    ++asked;
    ++load_j;
    more = settle();
  };
  while (more && asked < static_cast<uint32_t>(a.stages)) ask();

  // ---- row tiles --------------------------------------------------------------------------------------
  for (uint32_t seg = 0; seg < found; ++seg) {  // (a segment is found before the one before it ends)
    __syncwarp();
    const Segment s = sm.queue[warp][seg % kQueue];
    const int len = s.r.len, end = len + s.r.nodes;
    const int first_row = s.mtile * kRows, rows = min(kRows, s.r.nodes * a.group - first_row);
    // Q': this lane has a quarter of row g of each column of eight, scaled by a power of two
    uint32_t q[N][kSteps][2];
    float c[N][2];                     // from here on this lane has rows 2 t4 and 2 t4 + 1 of each column of eight
    int node[N][2], depth[N][2], near[N][2];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int local = 8 * n + g, row = first_row + local;
      uint4 w[D / 32];
      if (local < rows) {
        const int its_node = row / a.group;
        const uint4* from = reinterpret_cast<const uint4*>(a.q + (s.r.first + its_node) * a.q_row_stride +
                                                           (s.head * a.group + row - its_node * a.group) * a.q_head_stride + t4 * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) w[i] = __ldg(from + i);
      } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) w[i] = make_uint4(0, 0, 0, 0);
      }
      const uint32_t* p = reinterpret_cast<const uint32_t*>(w);
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) top = fmaxf(top, fmaxf(fabsf(bf16_lo(p[i])), fabsf(bf16_hi(p[i]))));
      top = quad_max(top);
      // 2^up brings the largest element into [2^14, 2^15); rows below 2^-100 stay below it
      const int up = 14 - max(static_cast<int>((__float_as_uint(top) >> 23) & 0xFF) - 127, -100);
      const float by = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
      // (not 0, however small the scale: masked scores are -inf)
      const float its_c = fmaxf(a.scale * 1.44269504088896341f * __uint_as_float(static_cast<uint32_t>(127 - up) << 23), 1e-37f);
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) q[n][k][i] = pack_f16(bf16_lo(p[2 * k + i]) * by, bf16_hi(p[2 * k + i]) * by);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        c[n][e] = __shfl_sync(0xFFFFFFFFu, its_c, 4 * (2 * t4 + e));
        const int other = 8 * n + 2 * t4 + e;
        node[n][e] = other < rows ? (first_row + other) / a.group : -1;
        depth[n][e] = near[n][e] = 0;
        if (a.window > 0 && other < rows) {
          if (a.parent == nullptr) depth[n][e] = node[n][e];
          else
            for (int x = node[n][e]; x > 0; ++depth[n][e]) {
              const int up_node = a.parent[s.r.first + x];
              if (up_node < 0 || up_node >= x) break;  // reported where the node's own chunk is masked
              x = up_node;
            }
          near[n][e] = len + depth[n][e] - a.window + 1;
        }
      }
    }
    float o[kDimTiles][N][4];
#pragma unroll
    for (int i = 0; i < kDimTiles; ++i)
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][n][e] = 0.0f;
    float m[N][2], l[N][2];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = -INFINITY;
        l[n][e] = 0.0f;
      }
    for (int j = s.kv0; j < s.kv1; ++j) {
      const int s0 = tile_slot<kChunk>(s.r, j);
      warp_wait(&sm.full[warp][use_stage], use_parity, &sm.dead, a.status);
      const unsigned char* chunk = ring + use_stage * kChunkBytes;
      float p[2][N][4];  // sixteen slots each: this lane has slots g and g + 8 of them
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) p[h][n][e] = 0.0f;
        uint32_t w[2][kWords], sc[2][2];  // of both groups of eight: codes and scales of slot g's quarter t4
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const unsigned char* group = chunk + (2 * h + u) * kGroupBytes;
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(group + lane * 16);
            w[u][0] = v.x;
            w[u][1] = v.y;
            w[u][2] = v.z;
            w[u][3] = v.w;
            const uint32_t two = decode_scales(*reinterpret_cast<const uint16_t*>(group + 4 * D + lane * 2));
            sc[u][0] = __byte_perm(two, two, 0x1010);
            sc[u][1] = __byte_perm(two, two, 0x3232);
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(group + lane * 8);
            w[u][0] = v.x;
            w[u][1] = v.y;
            const uint32_t one = decode_scales(group[4 * D + lane]);
            sc[u][0] = sc[u][1] = __byte_perm(one, one, 0x1010);
          }
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          uint32_t x0[4], x1[4];
          decode8(w[0][i], x0);
          decode8(w[1][i], x1);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t ka[4] = {mul_f16x2(x0[2 * k], sc[0][i / 2]), mul_f16x2(x1[2 * k], sc[1][i / 2]),
                                    mul_f16x2(x0[2 * k + 1], sc[0][i / 2]), mul_f16x2(x1[2 * k + 1], sc[1][i / 2])};
#pragma unroll
            for (int n = 0; n < N; ++n) mma16(p[h][n], ka, q[n][2 * i + k][0], q[n][2 * i + k][1]);
          }
        }
      }
      const bool whole = s0 + kChunk <= len && (a.window <= 0 || s0 + kChunk <= a.sinks || s0 >= end - a.window);
      uint32_t live = 0xFFFFFFFFu;  // slots that may be seen by some node: the others may hold anything
      if (!whole) {
        const int lo = a.window > 0 ? max(0, len - a.window + 1) : 0;
        live = range_bits(lo, end, s0) | (a.window > 0 ? range_bits(0, min(a.sinks, end), s0) : 0u);
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t see = 0;
            if (node[n][e] >= 0) {
              see = range_bits(near[n][e], len, s0) | (a.window > 0 ? range_bits(0, min(a.sinks, len), s0) : 0u);
              if (s0 + kChunk > len) {
                int d = depth[n][e];
                for (int at = node[n][e];; --d) {
                  const int bit = len + at - s0;
                  if (bit >= 0 && bit < kChunk && (a.window <= 0 || len + d >= near[n][e] || len + d < a.sinks)) see |= 1u << bit;
                  if (at <= 0 || bit < 0) break;
                  const int up_node = a.parent != nullptr ? a.parent[s.r.first + at] : at - 1;
                  if (up_node < 0 || up_node >= at) {
                    mark_bad(a, s.request, SV_DEV_BAD_PARENT);
                    break;
                  }
                  at = up_node;
                }
              }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int u = 0; u < 2; ++u)
                if (!((see >> (16 * h + 8 * u + g)) & 1u)) p[h][n][2 * u + e] = -INFINITY;
          }
      }
      float top[N][2];
      bool grows = false;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[n][e] = fmaxf(fmaxf(p[0][n][e], p[0][n][2 + e]), fmaxf(p[1][n][e], p[1][n][2 + e])) * c[n][e];  // c > 0
          grows |= top[n][e] > m[n][e] + kLazyGrowth4;  // (m = -inf: some slot is seen)
        }
      if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float now = fmaxf(m[n][e], column_max(top[n][e]));
            const float keep = m[n][e] == -INFINITY ? 0.0f : ex2_approx(m[n][e] - now);
            m[n][e] = now;
            l[n][e] *= keep;
#pragma unroll
            for (int i = 0; i < kDimTiles; ++i) {
              o[i][n][e] *= keep;
              o[i][n][2 + e] *= keep;
            }
          }
      }
      uint32_t pb[2][N][2];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float off[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) off[e] = m[n][e] == -INFINITY ? 0.0f : kBias - m[n][e];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[h][n][e] = ex2_approx(fmaf(p[h][n][e], c[n][e & 1], off[e & 1]));
            l[n][e & 1] += p[h][n][e];
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) pb[h][n][u] = transpose8(pack_f16(p[h][n][2 * u], p[h][n][2 * u + 1]));
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // sixteen slots: this lane has pair t4 of both groups, and eighth g of the dimensions
        uint32_t even[2][kWords / 2], odd[2][kWords / 2], by[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const unsigned char* group = chunk + (2 * h + u) * kGroupBytes + 4 * D + D / 2;
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(group + lane * 16);
            even[u][0] = v.x;
            even[u][1] = v.y;
            odd[u][0] = v.z;
            odd[u][1] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(group + lane * 8);
            even[u][0] = v.x;
            odd[u][0] = v.y;
          }
          by[u] = decode_scales(*reinterpret_cast<const uint16_t*>(group + 4 * D + (D == 128 ? lane * 2 : (g >> 1) * 8 + t4 * 2)));
          if (!whole) {  // 0 times what an unseen slot holds has to be 0
            const uint32_t bits = live >> (16 * h + 8 * u + 2 * t4);
            by[u] &= ((bits & 1u) ? 0xFFFFu : 0u) | ((bits & 2u) ? 0xFFFF0000u : 0u);
          }
        }
#pragma unroll
        for (int i = 0; i < kWords / 2; ++i) {
          uint32_t v[2][2][4];  // [group][dimension's parity]: pairs of slots
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            decode8((even[u][i] & 0x0F0F0F0Fu) | ((odd[u][i] << 4) & 0xF0F0F0F0u), v[u][0]);
            decode8(((even[u][i] >> 4) & 0x0F0F0F0Fu) | (odd[u][i] & 0xF0F0F0F0u), v[u][1]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // dimensions 8 i + 2 e in the tile's rows g, and the next ones in its rows g + 8
            const uint32_t va[4] = {mul_f16x2(v[0][0][e], by[0]), mul_f16x2(v[0][1][e], by[0]), mul_f16x2(v[1][0][e], by[1]),
                                    mul_f16x2(v[1][1][e], by[1])};
#pragma unroll
            for (int n = 0; n < N; ++n) mma16(o[4 * i + e][n], va, pb[h][n][0], pb[h][n][1]);
          }
        }
      }
      ++used;
      use_stage = use_stage + 1 == static_cast<uint32_t>(a.stages) ? 0 : use_stage + 1;
      use_parity ^= use_stage == 0;
      __syncwarp();  // every lane has read the stage
      if (more) ask();
    }
    // ---- the segment's end -----------------------------------------------------------------------------
    const bool complete = s.kv0 == 0 && s.kv1 == s.r.tiles;
    float* part = a.parts + static_cast<int64_t>(2 * me + (s.kv0 == 0)) * part4_floats<D, N>();
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] = column_sum(l[n][e]);
        const int r = 8 * n + 2 * t4 + e;
        if (r >= rows) continue;
        const int head = s.head * a.group + (first_row + r - node[n][e] * a.group);
        // this lane's eighth of the dimensions
        if (complete) {
          // Every row sees its own node's slot, so a sum that is not above 0 is that of a row without a softmax (NaN among its
          // scores, or nothing but -inf): its outputs are NaN.
          const float inv = l[n][e] > 0.0f ? a.v_scale / l[n][e] : NAN;
          uint4* to = reinterpret_cast<uint4*>(a.out + (s.r.first + node[n][e]) * a.out_row_stride + head * a.out_head_stride + g * (D / 8));
#pragma unroll
          for (int i = 0; i < kDimTiles; i += 4)
            to[i / 4] = make_uint4(pack_bf16x2(o[i][n][e] * inv, o[i][n][2 + e] * inv), pack_bf16x2(o[i + 1][n][e] * inv, o[i + 1][n][2 + e] * inv),
                                   pack_bf16x2(o[i + 2][n][e] * inv, o[i + 2][n][2 + e] * inv), pack_bf16x2(o[i + 3][n][e] * inv, o[i + 3][n][2 + e] * inv));
          if (g == 0 && a.lse != nullptr)
            a.lse[(s.r.first + node[n][e]) * a.q_heads + head] = (m[n][e] - kBias + log2f(l[n][e])) * 0.693147180559945309f;
        } else {
#pragma unroll
          for (int i = 0; i < kDimTiles; i += 2)
            *reinterpret_cast<float4*>(part + r * D + g * (D / 8) + 2 * i) =
                make_float4(o[i][n][e], o[i][n][2 + e], o[i + 1][n][e], o[i + 1][n][2 + e]);
          if (g == 0) {
            part[kRows * D + r] = m[n][e];
            part[kRows * D + kRows + r] = l[n][e];
          }
        }
      }
    if (lane == 0 && s.kv0 == 0 && !complete) {
      const uint32_t ends = s.begin + a.extra + s.r.tiles - 1;  // the part in which the row tile ends
      const Job job = {1, s.request, s.head, s.mtile, rows, static_cast<int32_t>(me), parts.of(ends), 0};
      a.jobs[atomicAdd(a.n_jobs, 1)] = job;
    }
  }
  // (after a wait that ran out: no copy may be in flight when the CTA leaves)
  for (; used < asked; ++used) {
    mbar_wait(&sm.full[warp][use_stage], use_parity, a.status);
    use_stage = use_stage + 1 == static_cast<uint32_t>(a.stages) ? 0 : use_stage + 1;
    use_parity ^= use_stage == 0;
  }
}

// Adds the partial results of row tile `jobs[x]`: with M = max m_i, o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.  A thread
// has four columns of a row and every kJoinGroups-th part (long contexts over few row tiles leave dozens).  Then the outputs
// of bad requests become 0.
constexpr int kJoinGroups = 2;
template <int D, int N>
__global__ void __launch_bounds__(kJoinGroups * 8 * N * D / 4) join4_kernel(const Attend4Params a) {
  constexpr int kRows = Tile4<N>::kRows, kPieces = kRows * D / 4;
  __shared__ float4 other_o[kPieces];
  __shared__ float other_l[kRows];
  pdl_wait();
  const int n_jobs = *a.n_jobs;
  for (int x = blockIdx.x; x < n_jobs; x += gridDim.x) {
    const Job job = a.jobs[x];
    const int half = threadIdx.x / kPieces, at = threadIdx.x - half * kPieces, r = at / (D / 4), i = at % (D / 4) * 4;
    const bool mine = r < job.rows && !a.bad[job.request];
    const int n = job.last - job.first + 1;
    // part x > 0 is its warp's first, part 0 its warp's second
    auto part_of = [&](int y) { return a.parts + static_cast<int64_t>(2 * (job.first + y) + (y == 0)) * part4_floats<D, N>(); };
    float M = -INFINITY, L = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (mine) {
#pragma unroll 8
      for (int y = 0; y < n; ++y) M = fmaxf(M, part_of(y)[kRows * D + r]);
#pragma unroll 4
      for (int y = half; y < n; y += kJoinGroups) {
        const float* part = part_of(y);
        const float m = part[kRows * D + r], l = part[kRows * D + kRows + r];
        const float4 v = *reinterpret_cast<const float4*>(part + r * D + i);
        // (a part that saw nothing of the row has m = -inf and sums of 0; one whose scores are NaN has NaN sums)
        const float w = m == -INFINITY ? (l == 0.0f ? 0.0f : NAN) : ex2_approx(m - M);
        L += w * l;
        o.x += w * v.x;
        o.y += w * v.y;
        o.z += w * v.z;
        o.w += w * v.w;
      }
    }
    if (half == 1) {
      other_o[at] = o;
      if (i == 0) other_l[r] = L;
    }
    __syncthreads();
    if (half == 0 && mine) {
      const float4 v = other_o[at];
      L += other_l[r];
      const float inv = L > 0.0f ? a.v_scale / L : NAN;
      const int row = job.mtile * kRows + r, node = row / a.group, head = job.head * a.group + row - node * a.group;
      const int64_t to = a.node_offsets[job.request] + node;
      *reinterpret_cast<uint2*>(a.out + to * a.out_row_stride + head * a.out_head_stride + i) =
          make_uint2(pack_bf16x2((o.x + v.x) * inv, (o.y + v.y) * inv), pack_bf16x2((o.z + v.z) * inv, (o.w + v.w) * inv));
      if (i == 0 && a.lse != nullptr) a.lse[to * a.q_heads + head] = (M - kBias + log2f(L)) * 0.693147180559945309f;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0 && atomicAdd(a.n_jobs + 1, 1) == static_cast<int>(gridDim.x) - 1) {  // every CTA has read the count
    a.n_jobs[0] = 0;
    a.n_jobs[1] = 0;
  }
  clear_bad<D, kJoinGroups * kPieces>(a, a, a);
}

// ---- host --------------------------------------------------------------------------------------------
struct Layout4 {
  size_t bad, jobs, parts, total;
};
Layout4 layout4_of(int head_dim) {
  // 16 warps of 8 rows, or 8 of 16: the same floats
  static_assert(Tile4<1>::kWarps * part4_floats<128, 1>() == Tile4<2>::kWarps * part4_floats<128, 2>(), "parts");
  Layout4 L;
  L.bad = SV_STATUS_BYTES;
  L.jobs = L.bad + SV_MAX_BATCH;
  L.parts = (L.jobs + sizeof(Job) * kMaxWarps * kMaxCtas + 255) & ~size_t(255);
  L.total = L.parts + sizeof(float) * (head_dim == 128 ? part4_floats<128, 1>() : part4_floats<64, 1>()) * 2 * Tile4<1>::kWarps * kMaxCtas;
  return L;
}

template <int D, int N>
cudaError_t launch_attention4(Attend4Params& a, int ctas, void* stream) {
  using T = Tile4<N>;
  constexpr int kChunkBytes = kChunk / 8 * 9 * D;
  const int room = kSmemMax - static_cast<int>(sizeof(Smem4)) - 128 - 4 * a.B;
  a.stages = std::min(kMaxStages4, room / (T::kWarps * kChunkBytes));  // at least 2
  const size_t dyn = 4 * static_cast<size_t>(a.B) + static_cast<size_t>(T::kWarps) * a.stages * kChunkBytes;
  cudaError_t e = allow_smem<attend4_kernel<D, N>>(kSmemMax - sizeof(Smem4) - 128);
  if (e != cudaSuccess) return e;
  e = launch_dependent(attend4_kernel<D, N>, dim3(ctas), T::kThreads, dyn, stream, SV_KERNEL_ATTENTION, 1, a);
  if (e != cudaSuccess) return e;
  // row tiles to join: at most all, and at most a part's worth each
  const int64_t row_tiles = static_cast<int64_t>(a.B) * a.kv_heads * ((static_cast<int64_t>(a.Nmax) * a.group + T::kRows - 1) / T::kRows);
  const int joins = static_cast<int>(std::min<int64_t>(row_tiles, 8 * ctas));
  return launch_dependent(join4_kernel<D, N>, dim3(joins), kJoinGroups * T::kRows * D / 4, 0, stream, SV_KERNEL_ATTENTION_JOIN, 1, a);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t sv_attention4_workspace_size(const sv_cache4* c, int q_heads) {
  if (check_cache4(c) != SV_OK) return 0;
  if (q_heads < 1 || q_heads % c->kv_heads != 0 || q_heads / c->kv_heads > 128) {
    set_error(SV_ERR_INVALID_ARG, "q_heads=%d: 1 to 128 times kv_heads=%d are needed", q_heads, c->kv_heads);
    return 0;
  }
  return std::max(layout4_of(c->head_dim).total, attention4_tiles_workspace(c->head_dim));
}

sv_status sv_tree_attention4(const sv_cache4* c, int layer, const void* q, int64_t q_row_stride, int64_t q_head_stride,
                             int q_heads, const int32_t* page_table, int table_width, const int32_t* seq_len,
                             const int32_t* node_offsets, int64_t n_rows, const int32_t* parent, int B, int Nmax,
                             float scale, int window, int sinks, void* out, int64_t out_row_stride,
                             int64_t out_head_stride, float* out_lse, void* ws, size_t ws_bytes, void* stream) {
  sv_status s;
  if ((s = check_cache4(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, B)) != SV_OK) return s;
  if (layer < 0 || layer >= c->layers) return set_error(SV_ERR_INVALID_ARG, "layer=%d outside [0, %d)", layer, c->layers);
  if (q_heads < 1 || q_heads % c->kv_heads != 0 || q_heads / c->kv_heads > 128)
    return set_error(SV_ERR_INVALID_ARG, "q_heads=%d: 1 to 128 times kv_heads=%d are needed", q_heads, c->kv_heads);
  if (Nmax < 1 || Nmax > SV_MAX_DRAFT + 1) return set_error(SV_ERR_INVALID_ARG, "Nmax=%d outside [1, %d]", Nmax, SV_MAX_DRAFT + 1);
  if (n_rows < 0 || n_rows > static_cast<int64_t>(SV_MAX_BATCH) * (SV_MAX_DRAFT + 1))
    return set_error(SV_ERR_INVALID_ARG, "n_rows=%lld", (long long)n_rows);
  if (!(scale > 0.0f) || std::isinf(scale) || !(scale * c->k_scale > 0.0f) || std::isinf(scale * c->k_scale))
    return set_error(SV_ERR_INVALID_ARG, "scale, and its product with k_scale, must be finite and positive");
  if (window < 0 || sinks < 0) return set_error(SV_ERR_INVALID_ARG, "window=%d sinks=%d: must be >= 0", window, sinks);
  if (B == 0 || n_rows == 0) return SV_OK;
  if (q == nullptr || out == nullptr || node_offsets == nullptr)
    return set_error(SV_ERR_INVALID_ARG, "q / out / node_offsets is NULL");
  if (!aligned16(q) || !aligned16(out) || ((q_row_stride | q_head_stride | out_row_stride | out_head_stride) & 7) != 0 ||
      q_head_stride < c->head_dim || out_head_stride < c->head_dim || q_row_stride < 0 || out_row_stride < 0)
    return set_error(SV_ERR_INVALID_ARG, "q / out: 16-byte aligned rows of head_dim elements are needed");
  if ((s = check_workspace(ws, ws_bytes, sv_attention4_workspace_size(c, q_heads))) != SV_OK) return s;
  const int group = q_heads / c->kv_heads;
  // the line of work is counted in 32 bits
  // (16 rows as two tiles of eight: 64 contexts of 6k to 8k 195 us against 158, codes decoded twice)
  const int rows = Nmax * group <= 8 ? 8 : 16;
  const int64_t tiles = ((static_cast<int64_t>(table_width) * c->page_size + kChunk - 1) / kChunk + 1 + kExtra4) *
                        ((static_cast<int64_t>(Nmax) * group + rows - 1) / rows);
  if (tiles > INT_MAX || tiles * c->kv_heads > INT_MAX || tiles * c->kv_heads * B > INT_MAX)
    return set_error(SV_ERR_INVALID_ARG, "B=%d requests of up to %lld tiles a head are too many for one call", B, (long long)tiles);
  // more rows than a warp's tile holds: decoding once for up to 128 rows
  if (Nmax * group > kTilesFrom)
    return attention4_tiles(c, layer, q, q_row_stride, q_head_stride, q_heads, page_table, table_width, seq_len, node_offsets, n_rows,
                            parent, B, Nmax, scale, window, sinks, out, out_row_stride, out_head_stride, out_lse, ws, stream);
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return launch_status(e, "device");
  const int ctas = std::min(sms, kMaxCtas);
  const Layout4 L = layout4_of(c->head_dim);
  unsigned char* w = static_cast<unsigned char*>(ws);
  Attend4Params a = {};
  a.out_row_stride = out_row_stride;
  a.out_head_stride = out_head_stride;
  a.table = page_table;
  a.seq_len = seq_len;
  a.node_offsets = node_offsets;
  a.parent = parent;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = out_lse;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_row_stride = q_row_stride;
  a.q_head_stride = q_head_stride;
  a.pool = static_cast<const unsigned char*>(c->pool) + layer * c->layer_stride;
  a.page_stride = c->page_stride;
  a.head_stride = c->head_stride;
  a.status = reinterpret_cast<uint32_t*>(w);
  a.any_bad = reinterpret_cast<int32_t*>(w) + 1;
  a.n_jobs = reinterpret_cast<int32_t*>(w) + 3;
  a.bad = w + L.bad;
  a.jobs = reinterpret_cast<Job*>(w + L.jobs);
  a.parts = reinterpret_cast<float*>(w + L.parts);
  a.n_rows = n_rows;
  a.width = table_width;
  a.B = B;
  a.Nmax = Nmax;
  a.pages = c->pages;
  while ((1 << a.shift) < c->page_size) ++a.shift;
  a.q_heads = q_heads;
  a.kv_heads = c->kv_heads;
  a.group = group;
  a.tile_rows = rows;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale * c->k_scale;
  a.v_scale = c->v_scale;
  a.extra = kExtra4;
  const auto launch = c->head_dim == 128 ? (rows == 8 ? launch_attention4<128, 1> : launch_attention4<128, 2>)
                                         : (rows == 8 ? launch_attention4<64, 1> : launch_attention4<64, 2>);
  return launch_status(launch(a, ctas, stream), "attention");
}

}  // extern "C"
