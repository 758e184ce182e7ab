// sv_tree_attention: a token tree's queries against a paged cache.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "sv_device.cuh"
#include "sv_ops.h"

namespace sv {
namespace {

constexpr int kWarps = 8;

struct AttendParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int64_t page_stride, slot_stride, head_stride;
  int64_t q_row_stride, q_head_stride, out_row_stride, out_head_stride;
  const int32_t *table, *seq_len, *node_offsets, *parent;
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
  int64_t n_rows;
  int32_t width, B, Nmax, pages, shift, q_heads, group, window, sinks;
  float scale;
};

// One CTA per (row, query head); each warp takes every eighth slot, lanes split the head's dimensions.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) attend_kernel(AttendParams a) {
  constexpr int kPer = D / 32;
  __shared__ uint32_t seen[32];  // bit c: node c is on the path
  __shared__ int depth, invalid, request;
  __shared__ float wm[kWarps], wl[kWarps], wo[kWarps][D];
  pdl_wait();
  const int64_t row = blockIdx.x;
  const int h = blockIdx.y, g = h / a.group, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < 32) {
    const int i = request_of_row(a.node_offsets, a.B, row);
    seen[lane] = 0;
    __syncwarp();
    if (lane == 0) {
      request = i;
      const int64_t first = a.node_offsets[i], last = a.node_offsets[i + 1], len = a.seq_len[i];
      uint32_t bad = 0;
      if (first < 0 || row < first || row >= last || last > a.n_rows || last - first > a.Nmax) bad |= SV_DEV_BAD_NODES;
      else if (len < 0 || len + (last - first) > (static_cast<int64_t>(a.width) << a.shift)) bad |= SV_DEV_BAD_SEQ;
      int d = 0;
      if (bad == 0) {
        int c = static_cast<int>(row - first);
        seen[c >> 5] |= 1u << (c & 31);
        while (c > 0) {
          const int up = a.parent != nullptr ? a.parent[first + c] : c - 1;
          if (up < 0 || up >= c) {
            bad |= SV_DEV_BAD_PARENT;
            break;
          }
          c = up;
          seen[c >> 5] |= 1u << (c & 31);
          ++d;
        }
        for (int64_t e = 0; e << a.shift < len + (last - first); ++e) {
          const int page = a.table[static_cast<int64_t>(i) * a.width + e];
          if (page < 0 || page >= a.pages) bad |= SV_DEV_BAD_PAGE;
        }
      }
      depth = d;
      invalid = bad != 0;
      if (bad != 0) atomicOr(a.status, bad);
    }
  }
  __syncthreads();
  __nv_bfloat16* out = a.out + row * a.out_row_stride + h * a.out_head_stride;
  if (invalid) {
    for (int d = threadIdx.x; d < D; d += kWarps * 32) out[d] = __float2bfloat16(0.0f);
    if (threadIdx.x == 0 && a.lse != nullptr) a.lse[row * a.q_heads + h] = -INFINITY;
    return;
  }
  const int64_t len = a.seq_len[request], slots = len + (a.node_offsets[request + 1] - a.node_offsets[request]);
  const int64_t first_near = a.window > 0 ? len + depth - a.window + 1 : 0;  // first position inside the window
  float q[kPer], o[kPer], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int d = 0; d < kPer; ++d) {
    q[d] = __bfloat162float(a.q[row * a.q_row_stride + h * a.q_head_stride + lane * kPer + d]);
    o[d] = 0.0f;
  }
  for (int64_t s = warp; s < slots; s += kWarps) {
    int64_t position = s;
    if (s >= len) {
      const int c = static_cast<int>(s - len);
      if (!(seen[c >> 5] >> (c & 31) & 1u)) continue;
      int d = 0;  // ancestors before c
      for (int w = 0; w <= (c >> 5); ++w) d += __popc(w == (c >> 5) ? seen[w] & ((1u << (c & 31)) - 1u) : seen[w]);
      position = len + d;
    }
    if (position < first_near && position >= a.sinks) continue;
    const int64_t at = a.table[static_cast<int64_t>(request) * a.width + (s >> a.shift)] * a.page_stride +
                       (s & ((1 << a.shift) - 1)) * a.slot_stride + g * a.head_stride + lane * kPer;
    float x = 0.0f;
#pragma unroll
    for (int d = 0; d < kPer; ++d) x += q[d] * __bfloat162float(a.k[at + d]);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, w);
    x *= a.scale;
    const float m2 = fmaxf(m, x), keep = expf(m - m2), e = expf(x - m2);
    l = l * keep + e;
#pragma unroll
    for (int d = 0; d < kPer; ++d) o[d] = o[d] * keep + e * __bfloat162float(a.v[at + d]);
    m = m2;
  }
  if (lane == 0) {
    wm[warp] = m;
    wl[warp] = l;
  }
#pragma unroll
  for (int d = 0; d < kPer; ++d) wo[warp][lane * kPer + d] = o[d];
  __syncthreads();
  float M = -INFINITY, L = 0.0f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w]);
  for (int w = 0; w < kWarps; ++w)
    if (wl[w] > 0.0f) L += wl[w] * expf(wm[w] - M);
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float x = 0.0f;
    for (int w = 0; w < kWarps; ++w)
      if (wl[w] > 0.0f) x += wo[w][d] * expf(wm[w] - M);
    out[d] = __float2bfloat16(x / L);
  }
  if (threadIdx.x == 0 && a.lse != nullptr) a.lse[row * a.q_heads + h] = M + logf(L);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t sv_attention_workspace_size(const sv_cache* c, int q_heads) {
  if (check_cache(c) != SV_OK || q_heads < 1 || q_heads % c->kv_heads != 0) return 0;
  return SV_STATUS_BYTES;
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
  AttendParams a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(c->k) + layer * c->layer_stride;
  a.v = static_cast<const __nv_bfloat16*>(c->v) + layer * c->layer_stride;
  a.page_stride = c->page_stride;
  a.slot_stride = c->slot_stride;
  a.head_stride = c->head_stride;
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
  a.status = static_cast<uint32_t*>(ws);
  a.n_rows = n_rows;
  a.width = table_width;
  a.B = B;
  a.Nmax = Nmax;
  a.pages = c->pages;
  a.shift = 0;
  while ((1 << a.shift) < c->page_size) ++a.shift;
  a.q_heads = q_heads;
  a.group = q_heads / c->kv_heads;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale;
  const dim3 grid(static_cast<unsigned>(n_rows), q_heads);
  return launch_status(c->head_dim == 128
                           ? launch_dependent(attend_kernel<128>, grid, kWarps * 32, 0, stream, SV_KERNEL_ATTENTION, 1, a)
                           : launch_dependent(attend_kernel<64>, grid, kWarps * 32, 0, stream, SV_KERNEL_ATTENTION, 1, a),
                       "attention");
}

}  // extern "C"
