// sv_tree_attention4: a token tree's queries against a paged cache held in 4 bits.
//
// A warp holds a row tile: 16 rows (query heads that share a key/value head, times nodes) as fragments of the 16 x 8 x 16
// products of two-byte floats, and goes over its share of the cache in chunks of 32 slots.  With c = scale k_scale log2(e) and
// running maximum m:
//   S = Q K^T [16 x 32];  P = 2^(c S - m) in float16;  O = O + P V [16 x D], all sums in float32
// and at the end o = v_scale O / sum P, lse = (m + log2 sum P) ln 2.
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
// only: per pair of elements a conversion and a multiplication by the scales.
//
// Work split.  All (row tile, cache tile of 128 slots) pairs lie on one line, cut into equal parts, one per CTA; a part's
// stretches of row tiles are shared by the CTA's warps chunk by chunk, whose partial results are added in shared memory; a
// row tile that crosses CTAs leaves partial results in the workspace, which join4_kernel adds.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "sv_device.cuh"
#include "sv_line.cuh"
#include "sv_ops.h"

namespace sv {
namespace {

constexpr int kRows = 16;                 // rows of a row tile
constexpr int kChunk = 32;                // slots that a warp takes at a time
constexpr int kWarps = 8;
constexpr int kThreads4 = 32 * kWarps;
constexpr float kLazyGrowth4 = 8.0f;      // log2 units by which a maximum may grow without a rescale of O
constexpr float kBias = 4.0f;             // P is 2^kBias at the maximum that it is scaled to
constexpr int kExtra4 = 2;                // places of the line for a row tile's beginning and end
constexpr int kMaxStages4 = 8;

struct Attend4Params : Line, Marks, Outputs {
  const __nv_bfloat16* q;
  int64_t q_row_stride, q_head_stride;
  const unsigned char* pool;     // of the layer
  int64_t page_stride, head_stride;
  const int32_t *table, *parent;
  Job* jobs;          // [grid]
  float* parts;       // [2 grid] partial results
  int32_t pages, kv_heads, stages;
  float scale;        // with k_scale
  float v_scale;
};

// Floats of one partial result: O [16][D], then m and the sum per row.
template <int D>
constexpr int part4_floats() { return kRows * D + 2 * kRows; }

struct Smem4 {
  Line line;
  uint64_t full[kWarps][kMaxStages4];
  float m[kWarps][kRows], l[kWarps][kRows];
  uint32_t scan[kWarps];
  volatile int32_t dead;       // a wait ran out: the launch finishes on what it holds
};

// D += A B: 16 x 16 by 16 x 8.
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four bytes of two codes each: pairs of float16, the low half's code first.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t decode_scales(uint16_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
  return h;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
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
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
  return x + __shfl_xor_sync(0xFFFFFFFFu, x, 2);
}

// First slot of the segment's x-th chunk.
__device__ __forceinline__ int chunk_slot(const Segment& s, int x) {
  constexpr int per = kTile / kChunk;
  return tile_slot(s.r, s.kv0 + x / per) + (x % per) * kChunk;
}
// Whether some node sees a slot of [slot, slot + n).
__device__ __forceinline__ bool seen_by_some(const Line& a, const Request& r, int slot, int n) {
  const int lo = a.window > 0 ? max(0, r.len - a.window + 1) : 0;
  return slot < r.len + r.nodes && (a.window <= 0 || slot < a.sinks || slot + n > lo);
}

// A warp's chunks in the order of the line: its place, and where the next one is.
struct Walk {
  Segment s;
  uint32_t t;      // place of the line where the segment begins
  int x, n;        // chunk, chunks of the segment
};

template <int D>
__global__ void __launch_bounds__(kThreads4, 1) attend4_kernel(const Attend4Params a) {
  constexpr int kGroupBytes = 9 * D;                       // eight slots
  constexpr int kChunkBytes = kChunk / 8 * kGroupBytes;
  constexpr int kSteps = D / 16;                           // products over the dimensions
  constexpr int kWords = D / 32;                           // words of a lane's codes in a group: 4 or 2
  constexpr int kEighth = D / 8;                           // 8-column tiles of O
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ Smem4 sm;
  float* mix = reinterpret_cast<float*>(dyn);                                  // [kWarps][kRows][D + 4]
  unsigned char* rings = dyn + sizeof(float) * kWarps * kRows * (D + 4);
  uint32_t* before = reinterpret_cast<uint32_t*>(rings + static_cast<size_t>(kWarps) * a.stages * kChunkBytes);  // [B]
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int g = lane >> 2, t4 = lane & 3;
  if (tid == 0) {
    for (int w = 0; w < kWarps; ++w)
      for (int i = 0; i < a.stages; ++i) mbar_init(&sm.full[w][i], 1);
    sm.dead = 0;
    sm.line = a;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
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
      const Request r = request_of(a, i);
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
  // with fewer places than CTAs the last CTAs have none
  const Parts parts(total, max(1u, min(gridDim.x, total)));
  const uint32_t t0 = min(parts.begin(blockIdx.x), total), t1 = min(parts.begin(blockIdx.x + 1), total);
  if (tid == 0) a.jobs[blockIdx.x].valid = 0;

  // ---- copies ---------------------------------------------------------------------------------------
  unsigned char* ring = rings + static_cast<size_t>(warp) * a.stages * kChunkBytes;
  const int piece_shift = min(5, a.shift), piece = 1 << piece_shift;  // slots per copy: a page, or 32 slots of one
  // The next chunk of this warp that some node sees, from w.x on; false = there is none in this CTA's part.
  auto settle = [&](Walk& w) {
    for (;;) {
      while (w.x < w.n && !seen_by_some(sm.line, w.s.r, chunk_slot(w.s, w.x), kChunk)) w.x += kWarps;
      if (w.x < w.n) return true;
      if (w.s.next >= t1) return false;
      w.t = w.s.next;
      w.s = segment_at(sm.line, before, w.t, t1);
      w.n = (w.s.kv1 - w.s.kv0) * (kTile / kChunk);
      w.x = warp;
    }
  };
  uint32_t asked = 0, used = 0;      // chunks that were asked for, and used
  Walk load = {};
  bool more = t0 < t1;
  if (more) {
    load.t = t0;
    load.s = segment_at(sm.line, before, t0, t1);
    load.n = (load.s.kv1 - load.s.kv0) * (kTile / kChunk);
    load.x = warp;
  }
  auto page_of = [&](const Walk& w) {  // lane x < 32 / piece: the page of the chunk's x-th piece
    const int64_t slot = chunk_slot(w.s, w.x) + (lane << piece_shift);
    return lane < (kChunk >> piece_shift) && seen_by_some(sm.line, w.s.r, static_cast<int>(slot), piece)
               ? a.table[static_cast<int64_t>(w.s.request) * a.width + (slot >> a.shift)]
               : INT_MIN;              // (left out)
  };
  int page_now = INT_MIN;
  if (more) more = settle(load);
  if (more) page_now = page_of(load);
  auto ask = [&]() {
    const uint32_t stage = asked % a.stages;
    const int slot = chunk_slot(load.s, load.x) + (lane << piece_shift);
    int page = page_now;
    bool wanted = page != INT_MIN;
    if (wanted && (page < 0 || page >= a.pages)) {
      mark_bad(a, load.s.request, SV_DEV_BAD_PAGE);
      wanted = false;
    }
    const int bytes = __popc(__ballot_sync(0xFFFFFFFFu, wanted)) * (piece >> 3) * kGroupBytes;
    if (lane == 0) mbar_arrive_expect_tx(&sm.full[warp][stage], bytes);
    __syncwarp();
    if (wanted)
      bulk_g2s(ring + stage * kChunkBytes + (lane << piece_shift >> 3) * kGroupBytes,
               a.pool + page * a.page_stride + load.s.head * a.head_stride + ((slot & ((1 << a.shift) - 1)) >> 3) * kGroupBytes,
               (piece >> 3) * kGroupBytes, &sm.full[warp][stage]);
    ++asked;
    load.x += kWarps;
    more = settle(load);
    if (more) page_now = page_of(load);
  };
  while (more && asked < static_cast<uint32_t>(a.stages)) ask();

  // ---- row tiles --------------------------------------------------------------------------------------
  for (uint32_t t = t0; t < t1;) {
    const Segment s = segment_at(sm.line, before, t, t1);
    const uint32_t after = s.next;
    if (s.kv0 >= s.kv1) {  // the part begins or ends among the places before a row tile's cache tiles
      t = after;
      continue;
    }
    const int len = s.r.len, end = len + s.r.nodes;
    const int first_row = s.mtile * kRows, rows = min(kRows, s.r.nodes * a.group - first_row);
    // this lane's rows: g and g + 8
    int node[2], head[2], depth[2] = {0, 0}, near[2] = {0, 0};
    float c[2];
    uint32_t q[kSteps][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int local = g + 8 * h, row = first_row + local;
      const bool exists = local < rows;
      node[h] = exists ? row / a.group : -1;
      head[h] = exists ? s.head * a.group + row - node[h] * a.group : 0;
      uint4 w[D / 32];
      if (exists) {
        const uint4* from = reinterpret_cast<const uint4*>(a.q + (s.r.first + node[h]) * a.q_row_stride + head[h] * a.q_head_stride + t4 * (D / 4));
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
      c[h] = fmaxf(a.scale * 1.44269504088896341f * __uint_as_float(static_cast<uint32_t>(127 - up) << 23), 1e-37f);
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        q[k][h] = pack_f16(bf16_lo(p[2 * k]) * by, bf16_hi(p[2 * k]) * by);
        q[k][2 + h] = pack_f16(bf16_lo(p[2 * k + 1]) * by, bf16_hi(p[2 * k + 1]) * by);
      }
      if (a.window > 0 && exists) {
        if (a.parent == nullptr) depth[h] = node[h];
        else
          for (int x = node[h]; x > 0; ++depth[h]) {
            const int up_node = a.parent[s.r.first + x];
            if (up_node < 0 || up_node >= x) break;  // reported where the node's own chunk is masked
            x = up_node;
          }
        near[h] = len + depth[h] - a.window + 1;
      }
    }
    float o[kEighth][4];
#pragma unroll
    for (int i = 0; i < kEighth; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const int chunks = (s.kv1 - s.kv0) * (kTile / kChunk);
    for (int x = warp; x < chunks; x += kWarps) {
      const int s0 = chunk_slot(s, x);
      if (!seen_by_some(sm.line, s.r, s0, kChunk)) continue;
      const uint32_t stage = used % a.stages;
      warp_wait(&sm.full[warp][stage], (used / a.stages) & 1, &sm.dead, a.status);
      const unsigned char* chunk = ring + stage * kChunkBytes;
      float p[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {  // eight slots: this lane has slot g's quarter t4
        const unsigned char* group = chunk + u * kGroupBytes;
        uint32_t w[kWords];
        if constexpr (D == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(group + lane * 16);
          w[0] = v.x;
          w[1] = v.y;
          w[2] = v.z;
          w[3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(group + lane * 8);
          w[0] = v.x;
          w[1] = v.y;
        }
        uint32_t sc[2];  // of the quarter's first and last sixteen dimensions (D = 64: of all its sixteen)
        if constexpr (D == 128) {
          const uint32_t two = decode_scales(*reinterpret_cast<const uint16_t*>(group + 4 * D + lane * 2));
          sc[0] = __byte_perm(two, two, 0x1010);
          sc[1] = __byte_perm(two, two, 0x3232);
        } else {
          const uint32_t one = decode_scales(group[4 * D + lane]);
          sc[0] = sc[1] = __byte_perm(one, one, 0x1010);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) p[u][e] = 0.0f;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          uint32_t h[4];
          decode8(w[i], h);
          const uint32_t by = sc[i / 2];
          mma16(p[u], q[2 * i], mul_f16x2(h[0], by), mul_f16x2(h[1], by));
          mma16(p[u], q[2 * i + 1], mul_f16x2(h[2], by), mul_f16x2(h[3], by));
        }
      }
      const bool whole = s0 + kChunk <= len && (a.window <= 0 || s0 + kChunk <= a.sinks || s0 >= end - a.window);
      uint32_t live = 0xFFFFFFFFu;  // slots that may be seen by some node: the others may hold anything
      if (!whole) {
        const int lo = a.window > 0 ? max(0, len - a.window + 1) : 0;
        live = range_bits(lo, end, s0) | (a.window > 0 ? range_bits(0, min(a.sinks, end), s0) : 0u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t see = 0;
          if (node[h] >= 0) {
            see = range_bits(near[h], len, s0) | (a.window > 0 ? range_bits(0, min(a.sinks, len), s0) : 0u);
            if (s0 + kChunk > len) {
              int d = depth[h];
              for (int at = node[h];; --d) {
                const int bit = len + at - s0;
                if (bit >= 0 && bit < kChunk && (a.window <= 0 || len + d >= near[h] || len + d < a.sinks)) see |= 1u << bit;
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
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!((see >> (8 * u + 2 * t4 + e)) & 1u)) p[u][2 * h + e] = -INFINITY;
        }
      }
      float top[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(fmaxf(fmaxf(p[0][2 * h], p[0][2 * h + 1]), fmaxf(p[1][2 * h], p[1][2 * h + 1])),
                       fmaxf(fmaxf(p[2][2 * h], p[2][2 * h + 1]), fmaxf(p[3][2 * h], p[3][2 * h + 1]))) * c[h];  // c > 0
      }
      if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + kLazyGrowth4 || top[1] > m[1] + kLazyGrowth4)) {  // (m = -inf: some slot is seen)
        float keep[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float now = fmaxf(m[h], quad_max(top[h]));
          keep[h] = m[h] == -INFINITY ? 0.0f : ex2_approx(m[h] - now);
          m[h] = now;
          l[h] *= keep[h];
        }
#pragma unroll
        for (int i = 0; i < kEighth; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= keep[e >> 1];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float off = m[h] == -INFINITY ? 0.0f : kBias - m[h];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            p[u][2 * h + e] = ex2_approx(fmaf(p[u][2 * h + e], c[h], off));
            l[h] += p[u][2 * h + e];
          }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // sixteen slots: this lane has pair t4 of both groups, and eighth g of the dimensions
        const uint32_t pa[4] = {pack_f16(p[2 * k][0], p[2 * k][1]), pack_f16(p[2 * k][2], p[2 * k][3]),
                                pack_f16(p[2 * k + 1][0], p[2 * k + 1][1]), pack_f16(p[2 * k + 1][2], p[2 * k + 1][3])};
        uint32_t b[2][kEighth];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const unsigned char* group = chunk + (2 * k + u) * kGroupBytes + 4 * D + D / 2;
          uint32_t even[kWords / 2], odd[kWords / 2];
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(group + lane * 16);
            even[0] = v.x;
            even[1] = v.y;
            odd[0] = v.z;
            odd[1] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(group + lane * 8);
            even[0] = v.x;
            odd[0] = v.y;
          }
          uint32_t by = decode_scales(*reinterpret_cast<const uint16_t*>(group + 4 * D + (D == 128 ? lane * 2 : (g >> 1) * 8 + t4 * 2)));
          if (!whole) {  // 0 times what an unseen slot holds has to be 0
            const uint32_t bits = live >> (8 * (2 * k + u) + 2 * t4);
            by &= ((bits & 1u) ? 0xFFFFu : 0u) | ((bits & 2u) ? 0xFFFF0000u : 0u);
          }
#pragma unroll
          for (int i = 0; i < kWords / 2; ++i) {
            uint32_t h[4];
            decode8((even[i] & 0x0F0F0F0Fu) | ((odd[i] << 4) & 0xF0F0F0F0u), h);
#pragma unroll
            for (int e = 0; e < 4; ++e) b[u][8 * i + 2 * e] = mul_f16x2(h[e], by);
            decode8(((even[i] >> 4) & 0x0F0F0F0Fu) | (odd[i] & 0xF0F0F0F0u), h);
#pragma unroll
            for (int e = 0; e < 4; ++e) b[u][8 * i + 2 * e + 1] = mul_f16x2(h[e], by);
          }
        }
#pragma unroll
        for (int i = 0; i < kEighth; ++i) mma16(o[i], pa, b[0][i], b[1][i]);
      }
      ++used;
      __syncwarp();  // every lane has read the stage
      if (more) ask();
    }
    // ---- the segment's end: the warps' results together ----------------------------------------------
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] = quad_sum(l[h]);
      if (t4 == 0) {
        sm.m[warp][g + 8 * h] = m[h];
        sm.l[warp][g + 8 * h] = l[h];
      }
#pragma unroll
      for (int col = 0; col < 2; ++col)  // columns i of eighths 2 t4 and 2 t4 + 1
#pragma unroll
        for (int i = 0; i < kEighth; i += 4)
          *reinterpret_cast<float4*>(mix + (warp * kRows + g + 8 * h) * (D + 4) + (2 * t4 + col) * kEighth + i) =
              make_float4(o[i][2 * h + col], o[i + 1][2 * h + col], o[i + 2][2 * h + col], o[i + 3][2 * h + col]);
    }
    __syncthreads();
    {
      constexpr int kPer = kThreads4 / kRows;  // threads of a row
      const int r = tid / kPer, at = tid % kPer;
      const bool complete = s.kv0 == 0 && s.kv1 == s.r.tiles;
      float top = -INFINITY, sum = 0.0f, w[kWarps];
#pragma unroll
      for (int x = 0; x < kWarps; ++x) top = fmaxf(top, sm.m[x][r]);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        // (a warp that saw nothing of the row has m = -inf and sums of 0; one whose scores are NaN has NaN sums)
        w[x] = sm.m[x][r] == -INFINITY ? (sm.l[x][r] == 0.0f ? 0.0f : NAN) : ex2_approx(sm.m[x][r] - top);
        sum += w[x] == 0.0f ? 0.0f : w[x] * sm.l[x][r];
      }
      const int row = first_row + r, its_node = row / a.group, its_head = s.head * a.group + row - its_node * a.group;
      // Every row sees its own node's slot, so a sum that is not above 0 is that of a row without a softmax: its outputs are NaN.
      const float inv = complete ? (sum > 0.0f ? a.v_scale / sum : NAN) : 1.0f;
      if (r < rows) {
        float* part = a.parts + static_cast<int64_t>(2 * blockIdx.x + (s.kv0 == 0)) * part4_floats<D>();
#pragma unroll
        for (int i = 4 * at; i < D; i += 4 * kPer) {
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int x = 0; x < kWarps; ++x) {
            const float4 y = *reinterpret_cast<const float4*>(mix + (x * kRows + r) * (D + 4) + i);
            if (w[x] == 0.0f) continue;
            v.x += w[x] * y.x;
            v.y += w[x] * y.y;
            v.z += w[x] * y.z;
            v.w += w[x] * y.w;
          }
          if (complete)
            *reinterpret_cast<uint2*>(a.out + (s.r.first + its_node) * a.out_row_stride + its_head * a.out_head_stride + i) =
                make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
          else
            *reinterpret_cast<float4*>(part + r * D + i) = v;
        }
        if (at == 0) {
          if (!complete) {
            part[kRows * D + r] = top;
            part[kRows * D + kRows + r] = sum;
          } else if (a.lse != nullptr) {
            a.lse[(s.r.first + its_node) * a.q_heads + its_head] = (top - kBias + log2f(sum)) * 0.693147180559945309f;
          }
        }
      }
      if (tid == 0 && s.kv0 == 0 && !complete) {
        const uint32_t ends = s.begin + a.extra + s.r.tiles - 1;  // the CTA in which the row tile ends
        const Job job = {1, s.request, s.head, s.mtile, rows, static_cast<int32_t>(blockIdx.x), parts.of(ends), 0};
        a.jobs[blockIdx.x] = job;
      }
    }
    __syncthreads();
    t = after;
  }
  // (after a wait that ran out: no copy may be in flight when the CTA leaves)
  for (; used < asked; ++used) mbar_wait(&sm.full[warp][used % a.stages], (used / a.stages) & 1, a.status);
}

// Adds the partial results of row tile `jobs[x]`: with M = max m_i, o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i; a thread
// has four columns of a row.  Then the outputs of bad requests become 0.
template <int D>
__global__ void __launch_bounds__(kRows * D / 4) join4_kernel(const Attend4Params a) {
  pdl_wait();
  const Job job = a.jobs[blockIdx.x];
  const int r = threadIdx.x / (D / 4), i = threadIdx.x % (D / 4) * 4;
  if (job.valid != 0 && r < job.rows && !a.bad[job.request]) {
    const int n = job.last - job.first + 1;
    // part x > 0 is its CTA's first, part 0 its CTA's second
    auto part_of = [&](int x) { return a.parts + static_cast<int64_t>(2 * (job.first + x) + (x == 0)) * part4_floats<D>(); };
    float M = -INFINITY, L = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int x = 0; x < n; ++x) M = fmaxf(M, part_of(x)[kRows * D + r]);
#pragma unroll 4
    for (int x = 0; x < n; ++x) {
      const float* part = part_of(x);
      const float m = part[kRows * D + r], l = part[kRows * D + kRows + r];
      const float w = m == -INFINITY ? (l == 0.0f ? 0.0f : NAN) : ex2_approx(m - M);
      if (w == 0.0f) continue;
      const float4 v = *reinterpret_cast<const float4*>(part + r * D + i);
      L += w * l;
      o.x += w * v.x;
      o.y += w * v.y;
      o.z += w * v.z;
      o.w += w * v.w;
    }
    const float inv = L > 0.0f ? a.v_scale / L : NAN;
    const int row = job.mtile * kRows + r, node = row / a.group, head = job.head * a.group + row - node * a.group;
    const int64_t at = a.node_offsets[job.request] + node;
    *reinterpret_cast<uint2*>(a.out + at * a.out_row_stride + head * a.out_head_stride + i) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (i == 0 && a.lse != nullptr) a.lse[at * a.q_heads + head] = (M - kBias + log2f(L)) * 0.693147180559945309f;
  }
  clear_bad<D, kRows * D / 4>(a, a, a);
}

// ---- host --------------------------------------------------------------------------------------------
struct Layout4 {
  size_t bad, jobs, parts, total;
};
Layout4 layout4_of(int head_dim) {
  Layout4 L;
  L.bad = SV_STATUS_BYTES;
  L.jobs = L.bad + SV_MAX_BATCH;
  L.parts = (L.jobs + sizeof(Job) * kMaxCtas + 255) & ~size_t(255);
  L.total = L.parts + sizeof(float) * (head_dim == 128 ? part4_floats<128>() : part4_floats<64>()) * 2 * kMaxCtas;
  return L;
}

template <int D>
cudaError_t launch_attention4(Attend4Params& a, int ctas, void* stream) {
  constexpr int kChunkBytes = kChunk / 8 * 9 * D;
  const int fixed = static_cast<int>(sizeof(float)) * kWarps * kRows * (D + 4) + 4 * a.B;
  const int room = kSmemMax - static_cast<int>(sizeof(Smem4)) - 128 - fixed;
  a.stages = std::min(kMaxStages4, room / (kWarps * kChunkBytes));  // at least 3
  const size_t dyn = static_cast<size_t>(fixed) + static_cast<size_t>(kWarps) * a.stages * kChunkBytes;
  cudaError_t e = allow_smem<attend4_kernel<D>>(kSmemMax - sizeof(Smem4) - 128);
  if (e != cudaSuccess) return e;
  e = launch_dependent(attend4_kernel<D>, dim3(ctas), kThreads4, dyn, stream, SV_KERNEL_ATTENTION, 1, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(join4_kernel<D>, dim3(ctas), kRows * D / 4, 0, stream, SV_KERNEL_ATTENTION_JOIN, 1, a);
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
  return layout4_of(c->head_dim).total;
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
  const int64_t tiles = ((static_cast<int64_t>(table_width) * c->page_size + kTile - 1) / kTile + 1 + kExtra4) *
                        ((static_cast<int64_t>(Nmax) * group + kRows - 1) / kRows);
  if (tiles > INT_MAX || tiles * c->kv_heads > INT_MAX || tiles * c->kv_heads * B > INT_MAX)
    return set_error(SV_ERR_INVALID_ARG, "B=%d requests of up to %lld tiles a head are too many for one call", B, (long long)tiles);
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
  a.tile_rows = kRows;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale * c->k_scale;
  a.v_scale = c->v_scale;
  a.extra = kExtra4;
  return launch_status(c->head_dim == 128 ? launch_attention4<128>(a, ctas, stream) : launch_attention4<64>(a, ctas, stream), "attention");
}

}  // extern "C"
