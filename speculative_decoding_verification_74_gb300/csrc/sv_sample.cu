// sv_sample_rows: draws from logit rows with temperature, top-k, top-p and min-p.
//
// One thread-block cluster per row; each CTA keeps a contiguous slice of the row in shared memory,
// so the row is read from memory once.  Weights are integers (multiples of 2^-40), so every sum
// is exact and the result does not depend on how the row is split.  The filters keep a prefix of
// the order (x desc, index asc): the boundary logit is found by a radix descent on the
// order-preserving integer image of x, 8 bits a step, with histograms of counts and weights that the
// cluster's CTAs add up through distributed shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>

#include "sv_device.cuh"
#include "sv_ops.h"

namespace sv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 256;
constexpr int kMaxCluster = 8;
constexpr int kPieces = 4;  // bulk copies (and barriers) per slice

struct SampleParams {
  const void* logits;
  int64_t row_stride;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* uniforms;
  int32_t* out_tokens;
  float* out_probs;
  void* out_rows;
  int64_t out_stride;
  uint32_t* status;
  int32_t R, V, M, slice;  // slice: elements per CTA, a multiple of 8
};

// What the cluster's CTAs read from one another.
struct Shared {
  uint64_t weight[kBins];
  uint32_t count[kBins];
  uint64_t z;          // kept weights of the slice
  float top;           // largest logit of the slice
  uint64_t bar[kPieces];
  uint64_t seg[kWarps];
  uint32_t ties[kWarps];
  uint64_t scan_w[kWarps];
  uint32_t scan_c[kWarps];
  // result of a descent step
  uint32_t bin, above_c, here_c;
  uint64_t above_w, here_w;
  uint32_t cut;        // first tie (vocabulary index) that is left out
  float red[kWarps];
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
// Address of a peer CTA's copy of a shared-memory object.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t peer_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t peer_u64(const void* p, uint32_t rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Integer image of x: a larger logit has a larger key, -0 and +0 the same.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ float exponent_of(float x, float top, float steep) {
  return __fmul_rn(__fsub_rn(x, top), steep);
}
// 2^y as a multiple of 2^-40.
__device__ __forceinline__ uint64_t weight_of(float y) { return __float2ull_rn(ex2_approx(y) * 0x1p40f); }

// floor(total * part / 2^24), part <= 2^24, total < 2^62.
__device__ __forceinline__ uint64_t share_of(uint64_t total, uint32_t part) {
  return (total >> 24) * part + (((total & 0xFFFFFFu) * part) >> 24);
}

template <int DT>
struct Vec {
  static constexpr int kElems = DT == SV_BF16 ? 8 : 4;
  float x[kElems];
  __device__ __forceinline__ explicit Vec(const uint4& w) {
    if constexpr (DT == SV_BF16) {
      x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
      x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
    } else {
      x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
    }
  }
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// One slice of a row in shared memory: 16-byte vectors, the first `phase` elements and those past
// the slice padded with -inf.
template <int DT>
struct Slice {
  static constexpr int kElems = Vec<DT>::kElems;
  using Elem = typename std::conditional<DT == SV_BF16, uint16_t, uint32_t>::type;
  unsigned char* data;
  int phase, n, vecs;
  int64_t first;  // vocabulary index of element 0 of the slice

  __device__ __forceinline__ uint4 vec(int i) const { return lds128(data + static_cast<size_t>(i) * 16); }
  __device__ __forceinline__ int index(int vec, int e) const { return static_cast<int>(first) + vec * kElems + e - phase; }
};

// Radix descent over the whole row for the boundary of a prefix of (x desc): the smallest prefix whose count
// reaches `want` (by count) or whose weight does.  Returns the boundary key, the count and weight above
// it, and how often the key occurs (in the row, and in the CTAs before this one).
struct Boundary {
  uint32_t key, above_c, equal_c, equal_before, equal_here;
  uint64_t above_w;
};
template <int DT, bool kByWeight>
__device__ Boundary descend(const Slice<DT>& s, Shared& sh, uint64_t want, float top, float steep) {
  constexpr int kLevels = DT == SV_BF16 ? 2 : 4;
  const uint32_t cs = cluster_size(), rank = cluster_rank();
  uint32_t prefix = 0, above_c = 0;
  uint64_t above_w = 0;
  Boundary b = {};
  for (int level = 0; level < kLevels; ++level) {
    const int shift = 24 - 8 * level;
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
      sh.count[i] = 0;
      sh.weight[i] = 0;
    }
    __syncthreads();
    for (int v = threadIdx.x; v < s.vecs; v += kThreads) {
      const Vec<DT> x(s.vec(v));
#pragma unroll
      for (int e = 0; e < Vec<DT>::kElems; ++e) {
        const uint32_t key = key_of(x.x[e]);
        if (x.x[e] != -INFINITY && (level == 0 || (key >> (shift + 8)) == prefix)) {
          const uint32_t bin = (key >> shift) & 255u;
          atomicAdd(&sh.count[bin], 1u);
          if (kByWeight) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.weight[bin]), weight_of(exponent_of(x.x[e], top, steep)));
        }
      }
    }
    cluster_sync();  // every slice's histogram is complete
    // thread t of the first 256 takes bin 255 - t: a scan over threads goes from large to small logits
    const int bin = kBins - 1 - static_cast<int>(threadIdx.x);
    uint32_t c = 0;
    uint64_t w = 0;
    if (bin >= 0)
      for (uint32_t r = 0; r < cs; ++r) {
        c += peer_u32(&sh.count[bin], r);
        if (kByWeight) w += peer_u64(&sh.weight[bin], r);
      }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t ci = c;
    uint64_t wi = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t cu = __shfl_up_sync(0xFFFFFFFFu, ci, d);
      const uint64_t wu = __shfl_up_sync(0xFFFFFFFFu, wi, d);
      if (lane >= d) {
        ci += cu;
        wi += wu;
      }
    }
    if (lane == 31) {
      sh.scan_c[warp] = ci;
      sh.scan_w[warp] = wi;
    }
    if (threadIdx.x == 0) sh.bin = 0xFFFFFFFFu;
    __syncthreads();
    for (int i = 0; i < warp; ++i) {
      ci += sh.scan_c[i];
      wi += sh.scan_w[i];
    }
    ci += above_c;
    wi += above_w;
    const bool reaches = bin >= 0 && c > 0 && (kByWeight ? wi >= want && wi - w < want : ci >= want && ci - c < want);
    if (reaches) {
      sh.bin = bin;
      sh.above_c = ci - c;
      sh.above_w = wi - w;
      sh.here_c = c;
    }
    __syncthreads();
    if (sh.bin == 0xFFFFFFFFu) {  // fewer than `want`: everything is kept (the caller's want is at most the total by weight)
      b.key = 0;
      cluster_sync();
      return b;
    }
    above_c = sh.above_c;
    above_w = sh.above_w;
    prefix = level == 0 ? sh.bin : (prefix << 8) | sh.bin;
    if (level == kLevels - 1) {
      b.equal_c = sh.here_c;
      b.equal_here = sh.count[sh.bin];
      for (uint32_t r = 0; r < rank; ++r) b.equal_before += peer_u32(&sh.count[sh.bin], r);
    }
    cluster_sync();  // the peers have read this histogram
  }
  // bf16 keys: the low half of a key is 0x8000 or more exactly for negative logits (all ones), else 0
  b.key = DT == SV_BF16 ? ((prefix << 16) | ((prefix & 0x8000u) ? 0u : 0xFFFFu)) : prefix;
  b.above_c = above_c;
  b.above_w = above_w;
  return b;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) sample_kernel(SampleParams p) {
  using Elem = typename Slice<DT>::Elem;
  constexpr int kElems = Vec<DT>::kElems;
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ Shared sh;
  const uint32_t cs = cluster_size(), rank = cluster_rank();
  const int64_t row = blockIdx.x / cs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Elem* x_row = static_cast<const Elem*>(p.logits) + row * p.row_stride;
  Slice<DT> s;
  s.data = dyn;
  s.first = static_cast<int64_t>(rank) * p.slice;
  s.n = static_cast<int>(max(int64_t(0), min(static_cast<int64_t>(p.slice), p.V - s.first)));
  const Elem* src = x_row + s.first;
  s.phase = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15u) / sizeof(Elem));
  s.vecs = s.n > 0 ? (s.phase + s.n + kElems - 1) / kElems : 0;
  if (tid == 0) {
    for (int i = 0; i < kPieces; ++i) mbar_init(&sh.bar[i], 1);
    fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_wait();
  // whole 16-byte vectors by bulk copy, the row's ragged ends element by element
  const int v0 = s.phase > 0 ? 1 : 0, v1 = (s.phase + s.n) / kElems;
  const int per_piece = v1 > v0 ? (v1 - v0 + kPieces - 1) / kPieces : 0;
  if (tid == 0)
    for (int i = 0; i < kPieces; ++i) {
      const int a = min(v1, v0 + i * per_piece), b = min(v1, a + per_piece);
      if (b > a) {
        mbar_arrive_expect_tx(&sh.bar[i], (b - a) * 16);
        bulk_g2s(dyn + a * 16, reinterpret_cast<const unsigned char*>(src - s.phase) + static_cast<int64_t>(a) * 16, (b - a) * 16, &sh.bar[i]);
      } else {
        mbar_arrive(&sh.bar[i]);
      }
    }
  const Elem none = DT == SV_BF16 ? static_cast<Elem>(0xFF80u) : static_cast<Elem>(0xFF800000u);
  for (int i = tid; i < s.vecs * kElems; i += kThreads) {
    if (i >= v0 * kElems && v1 > v0 && i < v1 * kElems) {
      i += ((v1 * kElems - i - 1) / kThreads) * kThreads;  // skip the copied vectors
      continue;
    }
    const int e = i - s.phase;
    reinterpret_cast<Elem*>(dyn)[i] = e >= 0 && e < s.n ? src[e] : none;
  }
  float T = p.temperature[row];
  const int k_in = p.top_k != nullptr ? p.top_k[row] : 0;
  const float p_in = p.top_p != nullptr ? p.top_p[row] : 1.0f;
  const float q_in = p.min_p != nullptr ? p.min_p[row] : 0.0f;
  uint32_t bad = 0;
  if (!(T >= 0.0f) || T == INFINITY) bad |= SV_DEV_BAD_TEMPERATURE;
  if (k_in < 0 || !(p_in > 0.0f && p_in <= 1.0f) || !(q_in >= 0.0f && q_in <= 1.0f)) bad |= SV_DEV_BAD_FILTER;
  for (int j = 0; j < p.M; ++j) {
    const float u = p.uniforms[row * p.M + j];
    if (!(u >= 0.0f && u < 1.0f)) bad |= SV_DEV_BAD_FILTER;
  }
  __syncthreads();
  for (int i = 0; i < kPieces; ++i) mbar_wait(&sh.bar[i], 0, p.status);
  // ---- the largest logit --------------------------------------------------------------------
  float top = -INFINITY;
  for (int v = tid; v < s.vecs; v += kThreads) {
    const Vec<DT> x(s.vec(v));
#pragma unroll
    for (int e = 0; e < kElems; ++e) top = max_nan(top, x.x[e]);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  if (lane == 0) sh.red[warp] = top;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) top = max_nan(top, sh.red[w]);
    sh.top = top;
  }
  cluster_sync();
  top = -INFINITY;
  for (uint32_t r = 0; r < cs; ++r) top = max_nan(top, __uint_as_float(peer_u32(&sh.top, r)));
  if (!(top < INFINITY)) bad |= SV_DEV_BAD_LOGIT;
  const bool empty = top == -INFINITY;
  if (bad != 0 || empty) {  // the same in every CTA of the cluster
    if (bad != 0 && rank == 0 && tid == 0) atomicOr(p.status, bad);
    if (rank == 0)
      for (int j = tid; j < p.M; j += kThreads) {
        p.out_tokens[row * p.M + j] = -1;
        if (p.out_probs != nullptr) p.out_probs[row * p.M + j] = bad != 0 ? NAN : 0.0f;
      }
    if (p.out_rows != nullptr)
      for (int i = tid; i < s.n; i += kThreads) static_cast<Elem*>(p.out_rows)[row * p.out_stride + s.first + i] = none;
    cluster_sync();  // no CTA leaves while a peer may still read its shared memory
    return;
  }
  const bool greedy = T == 0.0f;
  const float steep = greedy ? 1.0f : fminf(__fdiv_rn(1.44269504088896341f, T), FLT_MAX);
  const int k = greedy ? 1 : (k_in == 0 ? p.V : k_in);
  const float least = greedy ? -INFINITY : log2f(q_in);
  const uint32_t p24 = greedy ? 1u << 24 : static_cast<uint32_t>(rintf(p_in * 16777216.0f));
  // ---- the filters' boundary ----------------------------------------------------------------
  Boundary b = {};          // key 0: every logit lies above
  uint32_t ties_kept = 0;   // how many of the boundary's equals are kept, lowest indexes first
  uint64_t total = 0;
  if (k < p.V) {
    b = descend<DT, false>(s, sh, k, top, steep);
    ties_kept = b.key == 0 ? 0 : k - b.above_c;
  }
  const bool nucleus = !greedy && p_in < 1.0f;
  if (nucleus) {
    // W: weights of the top-k
    uint64_t w = 0;
    for (int v = tid; v < s.vecs; v += kThreads) {
      const Vec<DT> x(s.vec(v));
#pragma unroll
      for (int e = 0; e < kElems; ++e)
        if (key_of(x.x[e]) > b.key) w += weight_of(exponent_of(x.x[e], top, steep));
    }
    w = warp_sum(w);
    if (lane == 0) sh.seg[warp] = w;
    __syncthreads();
    if (tid == 0) {
      uint64_t z = 0;
      for (int i = 0; i < kWarps; ++i) z += sh.seg[i];
      sh.z = z;
    }
    cluster_sync();
    for (uint32_t r = 0; r < cs; ++r) total += peer_u64(&sh.z, r);
    if (b.key != 0) total += static_cast<uint64_t>(ties_kept) * weight_of(exponent_of(logit_of_key(b.key), top, steep));
    cluster_sync();
    const uint64_t limit = max(share_of(total, p24), uint64_t(1));
    b = descend<DT, true>(s, sh, limit, top, steep);
    const uint64_t each = weight_of(exponent_of(logit_of_key(b.key), top, steep));
    ties_kept = each == 0 ? 0 : static_cast<uint32_t>((limit - b.above_w + each - 1) / each);
  }
  // ties of this slice that are kept: those before vocabulary index `cut`
  uint32_t cut = 0xFFFFFFFFu;
  {
    const uint32_t quota = ties_kept > b.equal_before ? min(ties_kept - b.equal_before, b.equal_here) : 0;
    if (b.key == 0) {
      cut = 0;
    } else if (quota == 0) {
      cut = 0;
    } else if (quota < b.equal_here) {
      // the quota-th tie of the slice, in order: warps own contiguous runs of vectors
      const int run = (s.vecs + kWarps - 1) / kWarps;
      const int a = min(s.vecs, warp * run), z = min(s.vecs, a + run);
      uint32_t c = 0;
      for (int v = a + lane; v < z; v += 32) {
        const Vec<DT> x(s.vec(v));
#pragma unroll
        for (int e = 0; e < kElems; ++e) c += key_of(x.x[e]) == b.key;
      }
      c = __reduce_add_sync(0xFFFFFFFFu, c);
      if (lane == 0) sh.ties[warp] = c;
      __syncthreads();
      uint32_t before = 0;
      for (int i = 0; i < warp; ++i) before += sh.ties[i];
      if (before < quota && before + c >= quota) {
        for (int v0r = a; v0r < z; v0r += 32) {
          const int v = v0r + lane;
          uint32_t mask = 0;
          if (v < z) {
            const Vec<DT> x(s.vec(v));
#pragma unroll
            for (int e = 0; e < kElems; ++e) mask |= (key_of(x.x[e]) == b.key ? 1u : 0u) << e;
          }
          uint32_t incl = __popc(mask);
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += u;
          }
          const uint32_t excl = incl - __popc(mask);
          if (before + excl < quota && before + incl >= quota) {
            uint32_t left = quota - before - excl;  // the left-th set bit of mask
            while (--left > 0) mask &= mask - 1;
            sh.cut = static_cast<uint32_t>(s.index(v, __ffs(mask) - 1)) + 1;
          }
          before += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
      }
      __syncthreads();
      cut = sh.cut;
    }
  }
  // kept weight of an element (0 = cut or no weight)
  auto keeps = [&](float x, int index) {
    const uint32_t key = key_of(x);
    return x != -INFINITY && (key > b.key || (key == b.key && static_cast<uint32_t>(index) < cut)) &&
           exponent_of(x, top, steep) >= least;
  };
  // ---- kept weights by warp runs, the row's total, the draws -----------------------------------
  const int run = (s.vecs + kWarps - 1) / kWarps;
  const int run_a = min(s.vecs, warp * run), run_z = min(s.vecs, run_a + run);
  {
    uint64_t w = 0;
    for (int v = run_a + lane; v < run_z; v += 32) {
      const Vec<DT> x(s.vec(v));
      float kept[kElems];
#pragma unroll
      for (int e = 0; e < kElems; ++e) {
        const bool keep = keeps(x.x[e], s.index(v, e));
        kept[e] = keep ? x.x[e] : -INFINITY;
        if (keep) w += weight_of(exponent_of(x.x[e], top, steep));
      }
      if (p.out_rows != nullptr) {
        Elem* out = static_cast<Elem*>(p.out_rows) + row * p.out_stride;
#pragma unroll
        for (int e = 0; e < kElems; ++e) {
          const int64_t i = s.index(v, e);
          if (i >= s.first && i < s.first + s.n)
            out[i] = DT == SV_BF16 ? static_cast<Elem>(__float_as_uint(kept[e]) >> 16) : static_cast<Elem>(__float_as_uint(kept[e]));
        }
      }
    }
    w = warp_sum(w);
    if (lane == 0) sh.seg[warp] = w;
    __syncthreads();
    if (tid == 0) {
      uint64_t z = 0;
      for (int i = 0; i < kWarps; ++i) z += sh.seg[i];
      sh.z = z;
    }
  }
  cluster_sync();
  uint64_t before = 0, z = 0, mine = 0;
  for (uint32_t r = 0; r < cs; ++r) {
    const uint64_t zr = peer_u64(&sh.z, r);
    if (r < rank) before += zr;
    if (r == rank) mine = zr;
    z += zr;
  }
  for (int j = warp; j < p.M; j += kWarps) {
    const uint32_t u24 = static_cast<uint32_t>(p.uniforms[row * p.M + j] * 16777216.0f);
    uint64_t t = share_of(z, u24);
    if (t < before || t >= before + mine) continue;  // another CTA's
    t -= before;
    int seg = 0;
    while (seg < kWarps - 1 && t >= sh.seg[seg]) t -= sh.seg[seg++];
    const int a = min(s.vecs, seg * run), b_end = min(s.vecs, a + run);
    for (int vb = a; vb < b_end; vb += 32) {
      const int v = vb + lane;
      uint64_t each[kElems], sum = 0;
#pragma unroll
      for (int e = 0; e < kElems; ++e) each[e] = 0;
      if (v < b_end) {
        const Vec<DT> x(s.vec(v));
#pragma unroll
        for (int e = 0; e < kElems; ++e) {
          if (keeps(x.x[e], s.index(v, e))) each[e] = weight_of(exponent_of(x.x[e], top, steep));
          sum += each[e];
        }
      }
      uint64_t incl = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += u;
      }
      const uint64_t all = __shfl_sync(0xFFFFFFFFu, incl, 31);
      if (t < all) {
        if (t < incl && t >= incl - sum) {
          uint64_t left = t - (incl - sum);
          int e = 0;
#pragma unroll
          for (int i = 0; i < kElems - 1; ++i)
            if (e == i && left >= each[i]) {
              left -= each[i];
              e = i + 1;
            }
          uint64_t w = 0;
#pragma unroll
          for (int i = 0; i < kElems; ++i) w = e == i ? each[i] : w;
          p.out_tokens[row * p.M + j] = s.index(v, e);
          if (p.out_probs != nullptr) p.out_probs[row * p.M + j] = __fdiv_rn(__ull2float_rn(w), __ull2float_rn(z));
        }
        break;
      }
      t -= all;
    }
  }
  cluster_sync();  // no CTA leaves while a peer may still read its shared memory
}

template <int DT>
cudaError_t launch_sample(SampleParams p, void* stream) {
  constexpr int kElt = DT == SV_BF16 ? 2 : 4;
  int cs = 1;  // slices of about 32 KB: a row's CTAs share its passes
  while (cs < kMaxCluster && static_cast<int64_t>(p.V) * kElt > cs * 32768) cs *= 2;
  p.slice = ((p.V + cs - 1) / cs + 7) & ~7;
  const size_t dyn = static_cast<size_t>(p.slice) * kElt + 32;
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(dyn));
  if (e != cudaSuccess) return e;
  return launch_dependent(sample_kernel<DT>, dim3(static_cast<unsigned>(p.R) * cs), kThreads, dyn, stream, SV_KERNEL_SAMPLE, cs, p);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status sv_sample_rows(const void* logits, int64_t row_stride, sv_dtype dt, int R, int V,
                                    const float* temperature, const int32_t* top_k, const float* top_p,
                                    const float* min_p, const float* uniforms, int M, int32_t* out_tokens,
                                    float* out_probs, void* out_rows, int64_t out_stride, void* ws, size_t ws_bytes,
                                    void* stream) {
  if (dt != SV_BF16 && dt != SV_F32) return set_error(SV_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
  if (R < 0 || R > SV_MAX_SAMPLE_ROWS) return set_error(SV_ERR_INVALID_ARG, "R=%d outside [0, %d]", R, SV_MAX_SAMPLE_ROWS);
  if (V < 1 || V > SV_MAX_SAMPLE_VOCAB) return set_error(SV_ERR_INVALID_ARG, "V=%d outside [1, %d]", V, SV_MAX_SAMPLE_VOCAB);
  if (M < 0 || M > SV_MAX_SAMPLE_DRAWS) return set_error(SV_ERR_INVALID_ARG, "M=%d outside [0, %d]", M, SV_MAX_SAMPLE_DRAWS);
  if (R == 0 || (M == 0 && out_rows == nullptr)) return SV_OK;
  const uintptr_t elt = dt == SV_BF16 ? 2 : 4;
  if (logits == nullptr || temperature == nullptr) return set_error(SV_ERR_INVALID_ARG, "logits / temperature is NULL");
  if (M > 0 && (uniforms == nullptr || out_tokens == nullptr))
    return set_error(SV_ERR_INVALID_ARG, "uniforms / out_tokens is NULL");
  if ((reinterpret_cast<uintptr_t>(logits) % elt) != 0 || (reinterpret_cast<uintptr_t>(out_rows) % elt) != 0)
    return set_error(SV_ERR_INVALID_ARG, "rows are not aligned to their element size");
  if (row_stride < V || (out_rows != nullptr && out_stride < V))
    return set_error(SV_ERR_INVALID_ARG, "row stride below V = %d", V);
  if (out_rows == logits && out_stride != row_stride)
    return set_error(SV_ERR_INVALID_ARG, "rows cut in place keep their stride");
  sv_status st = check_workspace(ws, ws_bytes, SV_STATUS_BYTES);
  if (st != SV_OK) return st;
  SampleParams p = {};
  p.logits = logits;
  p.row_stride = row_stride;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.uniforms = uniforms;
  p.out_tokens = out_tokens;
  p.out_probs = out_probs;
  p.out_rows = out_rows;
  p.out_stride = out_stride;
  p.status = static_cast<uint32_t*>(ws);
  p.R = R;
  p.V = V;
  p.M = M;
  return launch_status(dt == SV_BF16 ? launch_sample<SV_BF16>(p, stream) : launch_sample<SV_F32>(p, stream), "sample");
}
