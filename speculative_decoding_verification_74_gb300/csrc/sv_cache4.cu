// The paged key/value cache held in 4 bits: new rows quantised (append), moved (commit) and copied (fork, reorder).  The page
// bookkeeping is that of the bf16 cache.
//
// A head's page lies in groups of eight slots, 9 D bytes each: key codes, key scales, value codes, value scales, in the order
// in which a warp of the attention reads them (see sv.h).  So 32 slots of one head are one contiguous copy of 36 D bytes.
//
// Measured (GB300, graph replay; a copy of the bytes in brackets): a turn of 64 trees of up to 16 nodes in 32 layers (8 heads of
// 128) 59 us (26): append 40, which quantising's 200 instructions for sixteen elements and the lookup of each row's place bound,
// commit 10, reserve 4; 64 rows reordered in 32 layers 16 us (4): the plan 8, the copies 6.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "sv_device.cuh"
#include "sv_ops.h"
#include "sv_pages.cuh"

namespace sv {

sv_status check_cache4(const sv_cache4* c) {
  if (c == nullptr || c->pool == nullptr || c->page_refs == nullptr)
    return set_error(SV_ERR_INVALID_ARG, "cache, its pool or page_refs is NULL");
  if (!aligned16(c->pool)) return set_error(SV_ERR_INVALID_ARG, "the cache's pool is not 16-byte aligned");
  if (c->layers < 1 || c->pages < 1 || c->pages > SV_MAX_PAGES)
    return set_error(SV_ERR_INVALID_ARG, "layers=%d pages=%d", c->layers, c->pages);
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
    return set_error(SV_ERR_INVALID_ARG, "page_size=%d: a power of two in [8, 1024] is needed", c->page_size);
  if (c->kv_heads < 1 || c->kv_heads > 1024) return set_error(SV_ERR_INVALID_ARG, "kv_heads=%d outside [1, 1024]", c->kv_heads);
  if (c->head_dim != 64 && c->head_dim != 128) return set_error(SV_ERR_INVALID_ARG, "head_dim=%d: 64 or 128", c->head_dim);
  const int64_t head_bytes = static_cast<int64_t>(c->page_size) * 9 * c->head_dim / 8;
  const int64_t st[3] = {c->layer_stride, c->page_stride, c->head_stride};
  for (int64_t s : st)
    if (s < head_bytes || (s & 15) != 0)
      return set_error(SV_ERR_INVALID_ARG, "cache strides must be multiples of 16 and at least the %lld bytes of a head's page", (long long)head_bytes);
  for (float g : {c->k_scale, c->v_scale})
    if (!(g > 0.0f) || std::isinf(g) || std::isinf(1.0f / g) || 1.0f / g == 0.0f)
      return set_error(SV_ERR_INVALID_ARG, "k_scale and v_scale must be finite and positive, and their reciprocals too");
  return SV_OK;
}

namespace {

struct Shape4 {
  int64_t layer_stride, page_stride, head_stride;
  int32_t heads, dim, shift, pages;
};
// Byte offset of a slot's group within a layer (its place in the group is slot & 7), or -1.
__device__ __forceinline__ int64_t group_offset(const Shape4& r, const int32_t* row, int width, int64_t slot) {
  const int64_t e = slot >> r.shift;
  if (e >= width) return -1;
  const int page = row[e];
  if (page < 0 || page >= r.pages) return -1;
  return page * r.page_stride + ((slot & ((1 << r.shift) - 1)) >> 3) * (9 * r.dim);
}
// Places in a group: the eight dimensions from 8 x on of slot i, and their scale.
template <int D>
__device__ __forceinline__ int code_place(bool value, int i, int x) {
  constexpr int kEighth = D / 8;  // dimensions: 8 or 16
  const int e = 8 * x / kEighth;
  return value ? 4 * D + D / 2 + (4 * e + (i >> 1)) * kEighth + (i & 1) * (kEighth / 2) + (8 * x) % kEighth / 2 : i * (D / 2) + 4 * x;
}
template <int D>
__device__ __forceinline__ int scale_place(bool value, int i, int x) {
  return value ? 8 * D + D / 2 + (x >> 1) * 8 + i : 4 * D + i * (D / 16) + (x >> 1);
}

// t / s of eight values as e2m1, the first in the low half of the first byte.
__device__ __forceinline__ uint32_t codes_of(const float* r) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]));
  return w;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The e4m3 nearest to v >= 0, at most 448.
__device__ __forceinline__ uint8_t scale_of(float v) {
  uint16_t w;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(w) : "f"(0.0f), "f"(v));
  return static_cast<uint8_t>(w & 0xFF);
}
__device__ __forceinline__ float scale_value(uint8_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFF)));
}

struct Append4Params {
  Shape4 r;
  unsigned char* pool;
  const __nv_bfloat16 *k_new, *v_new;
  int64_t new_layer_stride, new_row_stride, n_rows;
  const int32_t *table, *seq_len, *node_offsets;
  int32_t width, B, layers;
  float k_inverse, v_inverse;
  uint32_t* status;
};

// One CTA per (new row, part of the layers): a thread quantises sixteen dimensions of [layer][k, v][head] at a time, about four
// times, the next ones' loads in flight; the first are asked for before the row's place is known.
template <int D>
__global__ void __launch_bounds__(kRowThreads) append4_kernel(Append4Params a) {
  pdl_wait();
  const int64_t row = blockIdx.x;
  constexpr int kScales = D / 16;                          // sixteens of a head
  const uint32_t per_side = a.r.heads * kScales, items = 2 * a.layers * per_side, step = gridDim.y * kRowThreads;
  // item x is sixteen e of side (layer; k or v)
  uint32_t x = blockIdx.y * kRowThreads + threadIdx.x, side = x / per_side, e = x - side * per_side;
  const uint32_t step_side = step / per_side, step_e = step - step_side * per_side;
  uint4 next[2] = {};
  auto fetch = [&](uint32_t its_side, uint32_t its_e) {
    const uint4* from = reinterpret_cast<const uint4*>(((its_side & 1) ? a.v_new : a.k_new) + (its_side >> 1) * a.new_layer_stride + row * a.new_row_stride) + 2 * its_e;
    next[0] = __ldg(from);
    next[1] = __ldg(from + 1);
  };
  if (x < items) fetch(side, e);
  __shared__ int64_t where;
  __shared__ int place;
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
        where = len < 0 ? -1 : group_offset(a.r, a.table + static_cast<int64_t>(lo) * a.width, a.width, len + (row - first));
        place = static_cast<int>((len + (row - first)) & 7);
        if (where < 0 && blockIdx.y == 0) atomicOr(a.status, len < 0 ? SV_DEV_BAD_SEQ : SV_DEV_BAD_PAGE);
      }
    }
  }
  __syncthreads();
  if (where < 0) return;
  bool wrong = false;
  for (; x < items; x += step) {
    const uint4 w[2] = {next[0], next[1]};
    const uint32_t layer = side >> 1;
    const bool value = side & 1;
    const int head = e / kScales, part = e % kScales;
    side += step_side;
    e += step_e;
    if (e >= per_side) {
      e -= per_side;
      ++side;
    }
    if (x + step < items) fetch(side, e);
    float t[16], top = 0.0f;
    const float inverse = value ? a.v_inverse : a.k_inverse;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t pair = reinterpret_cast<const uint32_t*>(w)[i];
      t[2 * i] = __fmul_rn(bf16_lo(pair), inverse);
      t[2 * i + 1] = __fmul_rn(bf16_hi(pair), inverse);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max_nan(top, fabsf(t[i]));
    wrong |= !(top <= 3.402823466e38f);
    const uint8_t scale = scale_of(fminf(__fmul_rn(top, 1.0f / 6.0f), 448.0f));
    // t / s, s known to four bits: with 1 / s as a pair of floats, fma(t, high, t low) is the correctly rounded quotient
    // (Brisebarre, Muller and Raina 2004; checked for all significands of s and t)
    const float by = scale_value(scale), high = by > 0.0f ? 1.0f / by : 0.0f, low = __fmul_rn(fmaf(-high, by, 1.0f), high);
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = fmaf(t[i], high, __fmul_rn(t[i], low));
    if (by == 0.0f) {
#pragma unroll
      for (int i = 0; i < 16; ++i) t[i] = 0.0f;
    }
    unsigned char* group = a.pool + layer * a.r.layer_stride + where + head * a.r.head_stride;
    const uint32_t codes[2] = {codes_of(t), codes_of(t + 8)};
    unsigned char* to = group + code_place<D>(value, place, 2 * part);
    if (D == 64 && value) {  // (two eighths of the dimensions)
      *reinterpret_cast<uint32_t*>(to) = codes[0];
      *reinterpret_cast<uint32_t*>(group + code_place<D>(value, place, 2 * part + 1)) = codes[1];
    } else {
      *reinterpret_cast<uint2*>(to) = make_uint2(codes[0], codes[1]);
    }
    group[scale_place<D>(value, place, 2 * part)] = scale;
  }
  if (wrong) atomicOr(a.status, SV_DEV_BAD_VALUE);
}

struct Commit4Params {
  Shape4 r;
  Pool pages;
  unsigned char* pool;
  int32_t* table;
  const int32_t *seq_len, *node_offsets, *path, *accept_len;
  int32_t* out_len;
  int32_t width, B, Nmax, layers;
  uint32_t* status;
  int32_t* arrived;  // [B] CTAs of a request that are done with its table row (zero between calls)
};

constexpr int kMoveBatch = 8;  // nodes whose pieces a thread holds at once

// grid (parts of the layers, B).  A thread moves eight dimensions of every accepted node, and with the first eight of sixteen
// their scale, in path order: node path[j] >= j + 1, so a slot that is written was read before, or is never read.  The
// request's CTA that finishes last gives back the pages past the new length.
template <int D>
__global__ void __launch_bounds__(kRowThreads) commit4_kernel(Commit4Params a) {
  extern __shared__ int64_t moves[];  // [2 * Nmax]: 8 * group offset + place of source and destination (-1 = stays)
  __shared__ int bad, last_one;
  pdl_wait();
  const int i = blockIdx.y;
  const int64_t len = a.seq_len[i];
  const int32_t* row = a.table + static_cast<int64_t>(i) * a.width;
  const int nodes = a.node_offsets[i + 1] - a.node_offsets[i];
  const int n = a.accept_len[i];
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
      const int64_t from = group_offset(a.r, row, a.width, len + node), to = group_offset(a.r, row, a.width, len + 1 + j);
      const bool stays = node == j + 1 || from < 0 || to < 0;
      if ((from < 0 || to < 0) && blockIdx.x == 0) atomicOr(a.status, SV_DEV_BAD_PAGE);
      moves[2 * j] = stays ? -1 : 8 * from + ((len + node) & 7);
      moves[2 * j + 1] = 8 * to + ((len + 1 + j) & 7);
    }
  }
  // node 0 stays, but in a slot that has a page
  if (keep >= 0 && blockIdx.x == 0 && threadIdx.x == kRowThreads - 1 && group_offset(a.r, row, a.width, len) < 0)
    atomicOr(a.status, SV_DEV_BAD_PAGE);
  __syncthreads();
  const bool invalid = wrong || bad != 0;
  if (invalid && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.status, SV_DEV_BAD_SEQ);
  if (!invalid) {
    constexpr int parts = D / 8;
    const int per_layer = 2 * a.r.heads * parts;
    const int64_t items = static_cast<int64_t>(a.layers) * per_layer;
    for (int64_t x = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; x < items;
         x += static_cast<int64_t>(gridDim.x) * kRowThreads) {
      const int layer = static_cast<int>(x / per_layer);
      int e = static_cast<int>(x - static_cast<int64_t>(layer) * per_layer);
      const bool value = e >= per_layer / 2;
      e -= value ? per_layer / 2 : 0;
      const int head = e / parts, part = e - head * parts;
      const bool scales = (part & 1) == 0;
      unsigned char* base = a.pool + layer * a.r.layer_stride + head * a.r.head_stride;
      for (int j0 = 0; j0 < keep; j0 += kMoveBatch) {
        uint32_t codes[kMoveBatch];
        unsigned char scale[kMoveBatch];
#pragma unroll
        for (int j = 0; j < kMoveBatch; ++j)
          if (j0 + j < keep && moves[2 * (j0 + j)] >= 0) {
            const int64_t m = moves[2 * (j0 + j)];
            const unsigned char* group = base + (m >> 3);
            codes[j] = *reinterpret_cast<const uint32_t*>(group + code_place<D>(value, m & 7, part));
            if (scales) scale[j] = group[scale_place<D>(value, m & 7, part)];
          }
#pragma unroll
        for (int j = 0; j < kMoveBatch; ++j)
          if (j0 + j < keep && moves[2 * (j0 + j)] >= 0) {
            const int64_t m = moves[2 * (j0 + j) + 1];
            unsigned char* group = base + (m >> 3);
            *reinterpret_cast<uint32_t*>(group + code_place<D>(value, m & 7, part)) = codes[j];
            if (scales) group[scale_place<D>(value, m & 7, part)] = scale[j];
          }
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
      release_entries(a.pages, a.table + static_cast<int64_t>(i) * a.width,
                      static_cast<int>((now + (int64_t(1) << a.r.shift) - 1) >> a.r.shift), a.width, a.status);
    if (threadIdx.x == 0) {
      a.out_len[i] = static_cast<int32_t>(now);
      a.arrived[i] = 0;
    }
  }
}

struct Copy4Params {
  Shape4 r;
  unsigned char* pool;
  const int32_t *table, *seq_len, *src, *dst, *done;  // see copied_slots
  int32_t width, layers;
};

// grid (parts of [layer][head], pairs): the groups of eight used slots of each copied last page, one contiguous piece per layer
// and head, which a warp copies (no division per 16 bytes: 16 requests of four beams 20 us -> 15).
constexpr int kInFlight = 4;
__global__ void __launch_bounds__(kRowThreads) copy4_kernel(Copy4Params a) {
  pdl_wait();
  int32_t from, to;
  const int part = copied_slots(a.src, a.dst, a.done, a.table, a.width, a.seq_len, a.r.shift, blockIdx.y, &from, &to);
  if (part == 0) return;
  const int pieces = ((part + 7) >> 3) * 9 * a.r.dim / 16, lane = threadIdx.x & 31;
  const uint32_t places = static_cast<uint32_t>(a.layers) * a.r.heads, step = gridDim.x * (kRowThreads / 32);
  for (uint32_t x = blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32; x < places; x += step) {
    const uint32_t layer = x / a.r.heads;
    unsigned char* base = a.pool + layer * a.r.layer_stride + (x - layer * a.r.heads) * a.r.head_stride;
    const int4* source = reinterpret_cast<const int4*>(base + from * a.r.page_stride);
    int4* target = reinterpret_cast<int4*>(base + to * a.r.page_stride);
    for (int i0 = lane; i0 < pieces; i0 += 32 * kInFlight) {
      int4 w[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u)
        if (i0 + 32 * u < pieces) w[u] = source[i0 + 32 * u];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u)
        if (i0 + 32 * u < pieces) target[i0 + 32 * u] = w[u];
    }
  }
}

Shape4 shape_of(const sv_cache4* c) {
  return Shape4{c->layer_stride, c->page_stride, c->head_stride, c->kv_heads, c->head_dim, log2_of(c->page_size), c->pages};
}
Pool pool_of(const sv_cache4* c) { return Pool{c->page_refs, c->pages, log2_of(c->page_size)}; }

// The copies after fork_pages (src and dst given) or reorder_pages.
cudaError_t copy_rows(const sv_cache4* c, const int32_t* table, int width, const int32_t* seq_len, const int32_t* src,
                      const int32_t* dst, const int32_t* done, int n, void* stream) {
  Copy4Params a = {};
  a.r = shape_of(c);
  a.pool = static_cast<unsigned char*>(c->pool);
  a.table = table;
  a.seq_len = seq_len;
  a.src = src;
  a.dst = dst;
  a.done = done;
  a.width = width;
  a.layers = c->layers;
  const int64_t places = static_cast<int64_t>(c->layers) * c->kv_heads;
  const int64_t groups = std::min<int64_t>(std::max(1, 16 * 152 / n), (places + kRowThreads / 32 - 1) / (kRowThreads / 32));
  return launch_dependent(copy4_kernel, dim3(static_cast<unsigned>(std::max<int64_t>(1, groups)), n), kRowThreads, 0, stream,
                          SV_KERNEL_CACHE_ROWS, 1, a);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

sv_status sv_cache4_reserve(const sv_cache4* c, int32_t* page_table, int table_width, const int32_t* seq_len,
                            const int32_t* extra, int B, int32_t* out_ok, void* ws, size_t ws_bytes, void* stream) {
  sv_status s;
  if ((s = check_cache4(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, B)) != SV_OK) return s;
  if (B == 0) return SV_OK;
  if (extra == nullptr) return set_error(SV_ERR_INVALID_ARG, "extra is NULL");
  if (static_cast<int64_t>(B) * table_width > INT_MAX)
    return set_error(SV_ERR_INVALID_ARG, "B * table_width = %lld exceeds 2^31 - 1", (long long)B * table_width);
  if ((s = check_workspace(ws, ws_bytes, SV_CACHE_WORKSPACE_BYTES)) != SV_OK) return s;
  return launch_status(reserve_pages(pool_of(c), page_table, table_width, seq_len, extra, B, out_ok, ws, stream), "reserve");
}

sv_status sv_cache4_append(const sv_cache4* c, int layer, int layers, const int32_t* page_table, int table_width,
                           const int32_t* seq_len, const int32_t* node_offsets, int64_t n_rows, const void* k_new,
                           const void* v_new, int64_t new_layer_stride, int64_t new_row_stride, int B, void* ws,
                           size_t ws_bytes, void* stream) {
  sv_status s;
  if ((s = check_cache4(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, B)) != SV_OK) return s;
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
  Append4Params a = {};
  a.r = shape_of(c);
  a.pool = static_cast<unsigned char*>(c->pool) + layer * c->layer_stride;
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
  a.k_inverse = 1.0f / c->k_scale;
  a.v_inverse = 1.0f / c->v_scale;
  a.status = status_of(ws);
  const int64_t items = static_cast<int64_t>(layers) * 2 * c->kv_heads * (c->head_dim / 16);
  if (items > INT_MAX) return set_error(SV_ERR_INVALID_ARG, "layers=%d: too many for one call", layers);
  const int64_t groups = std::min<int64_t>(64, (items + 4 * kRowThreads - 1) / (4 * kRowThreads));
  return launch_status(launch_dependent(c->head_dim == 128 ? append4_kernel<128> : append4_kernel<64>, dim3(static_cast<unsigned>(n_rows), static_cast<unsigned>(groups)),
                                        kRowThreads, 0, stream, SV_KERNEL_CACHE_ROWS, 1, a),
                       "append");
}

sv_status sv_cache4_commit(const sv_cache4* c, int32_t* page_table, int table_width, const int32_t* seq_len,
                           const int32_t* node_offsets, const int32_t* path, const int32_t* accept_len, int B, int Nmax,
                           int32_t* out_len, void* ws, size_t ws_bytes, void* stream) {
  sv_status s;
  if ((s = check_cache4(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, B)) != SV_OK) return s;
  if (Nmax < 1 || Nmax > SV_MAX_DRAFT + 1) return set_error(SV_ERR_INVALID_ARG, "Nmax=%d outside [1, %d]", Nmax, SV_MAX_DRAFT + 1);
  if (B == 0) return SV_OK;
  if (node_offsets == nullptr || path == nullptr || accept_len == nullptr || out_len == nullptr)
    return set_error(SV_ERR_INVALID_ARG, "node_offsets / path / accept_len / out_len is NULL");
  if ((s = check_workspace(ws, ws_bytes, SV_CACHE_WORKSPACE_BYTES)) != SV_OK) return s;
  Commit4Params a = {};
  a.r = shape_of(c);
  a.pages = pool_of(c);
  a.pool = static_cast<unsigned char*>(c->pool);
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
  const int64_t items = static_cast<int64_t>(c->layers) * 2 * c->kv_heads * (c->head_dim / 8);
  const int64_t groups = std::min<int64_t>(64, (items + 4 * kRowThreads - 1) / (4 * kRowThreads));
  return launch_status(launch_dependent(c->head_dim == 128 ? commit4_kernel<128> : commit4_kernel<64>, dim3(static_cast<unsigned>(groups), B), kRowThreads,
                                        sizeof(int64_t) * 2 * Nmax, stream, SV_KERNEL_CACHE_ROWS, 1, a),
                       "commit");
}

sv_status sv_cache4_fork(const sv_cache4* c, int32_t* page_table, int table_width, int rows, int32_t* seq_len,
                         const int32_t* src, const int32_t* dst, int n, int32_t* out_ok, void* ws, size_t ws_bytes,
                         void* stream) {
  sv_status s;
  if ((s = check_cache4(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, rows)) != SV_OK) return s;
  if (n < 0 || n > SV_MAX_BATCH) return set_error(SV_ERR_INVALID_ARG, "n=%d outside [0, %d]", n, SV_MAX_BATCH);
  if (n == 0) return SV_OK;
  if (rows == 0 || src == nullptr || dst == nullptr) return set_error(SV_ERR_INVALID_ARG, "rows, src or dst is missing");
  if ((s = check_workspace(ws, ws_bytes, SV_CACHE_WORKSPACE_BYTES)) != SV_OK) return s;
  int32_t* done = out_ok != nullptr ? out_ok : marks_of(ws);
  const cudaError_t e = fork_pages(pool_of(c), page_table, table_width, rows, seq_len, src, dst, n, done, ws, stream);
  if (e != cudaSuccess) return launch_status(e, "fork");
  return launch_status(copy_rows(c, page_table, table_width, seq_len, src, dst, done, n, stream), "fork rows");
}

sv_status sv_cache4_release(const sv_cache4* c, int32_t* page_table, int table_width, int rows, int32_t* seq_len,
                            const int32_t* seqs, int n, void* ws, size_t ws_bytes, void* stream) {
  sv_status s;
  if ((s = check_cache4(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, rows)) != SV_OK) return s;
  if (n < 0 || n > SV_MAX_BATCH) return set_error(SV_ERR_INVALID_ARG, "n=%d outside [0, %d]", n, SV_MAX_BATCH);
  if (n == 0) return SV_OK;
  if (rows == 0 || seqs == nullptr) return set_error(SV_ERR_INVALID_ARG, "rows or seqs is missing");
  if ((s = check_workspace(ws, ws_bytes, SV_CACHE_WORKSPACE_BYTES)) != SV_OK) return s;
  return launch_status(release_pages(pool_of(c), page_table, table_width, rows, seq_len, seqs, n, ws, stream), "release");
}

sv_status sv_cache4_reorder(const sv_cache4* c, int32_t* page_table, int table_width, int rows, int32_t* seq_len,
                            const int32_t* src, int32_t* out_ok, void* ws, size_t ws_bytes, void* stream) {
  sv_status s;
  if ((s = check_cache4(c)) != SV_OK || (s = check_table(page_table, table_width, seq_len, rows)) != SV_OK) return s;
  if (rows == 0) return SV_OK;
  if (src == nullptr) return set_error(SV_ERR_INVALID_ARG, "src is NULL");
  if ((s = check_workspace(ws, ws_bytes, SV_CACHE_WORKSPACE_BYTES)) != SV_OK) return s;
  const cudaError_t e = reorder_pages(pool_of(c), page_table, table_width, rows, seq_len, src, out_ok, ws, stream);
  if (e != cudaSuccess) return launch_status(e, "reorder");
  return launch_status(copy_rows(c, page_table, table_width, seq_len, nullptr, nullptr, marks_of(ws), rows, stream), "reorder rows");
}

}  // extern "C"
