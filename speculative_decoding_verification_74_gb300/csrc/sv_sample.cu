// sv_sample_rows: draws from logit rows with temperature, top-k, top-p and min-p.
//
// One thread-block cluster per row; each CTA keeps a contiguous slice of the row in shared memory, so the row is
// read from memory once.  Weights are integers (multiples of 2^-40), so every sum is exact and the result does not
// depend on how the row is split.  The filters keep a prefix of the order (x desc, index asc):
//   1. a bound below the prefix's end, from little work:
//        top-k   each thread's largest logit stands for a group; a CTA publishes a few order statistics of its groups'
//                maxima (rounded down to one of 512 steps), and the largest of them above which the CTAs together
//                vouch for k logits is the bound
//        top-p   logits whose weight is below (1 - p) W / V add up to less than (1 - p) W
//        min-p   its own threshold
//   2. the logits at or above the bound are listed in vocabulary order;
//   3. up to 2048 of them are gathered by the cluster's first CTA, sorted, and summed up: the prefix's end, its weight
//      and the draws follow from scans of that list.  The other CTAs are done.
// Longer lists (flat rows under top-p alone, large k) stay with their CTAs (cut_wide): a histogram of the listed logits
// (512 steps between bound and top; counts, and weights in three 14-bit limbs, which 32-bit atomics add without
// overflow), summed over the cluster, gives the step that holds the boundary, and that step's logits are exchanged and
// ranked by every CTA.  Where a step holds more logits than the exchange takes (long runs of equals), the boundary is
// found by a radix descent on the integer image of x instead.
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
constexpr int kSteps = kThreads;        // histogram steps: one per thread
constexpr int kMaxCluster = 8;
constexpr int kPieces = 4;              // bulk copies (and barriers) per slice
constexpr int kListPerWarp = 384;       // listed logits per warp; a warp with more walks its run instead
constexpr int kExchange = kThreads;     // logits of one step that the cluster exchanges: one per thread
constexpr int kLimb = 14;
constexpr int kGather = 2048;           // logits that one CTA sorts
constexpr int kGatherK = 1024;          // largest k that goes that way
constexpr int kRanks = 8;               // order statistics of a CTA's groups that it publishes

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

// Per-CTA state; the parts that peers read are written before a cluster barrier.
struct Shared {
  union {
    uint64_t gather[kGather];          // this CTA's listed logits: integer image << 32 | ~index; the first CTA's: everybody's
    struct {                           // cut_wide
      uint32_t limb[3][kSteps];
      uint32_t all[kExchange];         // the cluster's keys of the exchanged step
      uint64_t all_w[kExchange];
      uint32_t mine[kExchange];        // this CTA's
    };
  };
  uint32_t count[kSteps];
  uint16_t list[kWarps][kListPerWarp];
  uint64_t z;                          // a sum of the slice
  float top;                           // largest logit of the slice
  float rank_at[kRanks];               // a logit at or below the ranks()[j]-th largest group maximum
  uint32_t mine_n;                     // logits in `gather` (more than kGather: too many), or of the exchanged step
  uint64_t bar[kPieces];
  uint64_t seg[kWarps];
  uint32_t ties[kWarps];
  uint64_t scan_w[kWarps];
  uint32_t scan_c[kWarps];
  uint32_t from[kMaxCluster + 1];      // where each CTA's logits begin in the cluster's list
  uint32_t step, above_c, here_c;      // the step that holds a boundary
  uint64_t above_w;
  uint32_t key, key_above_c, key_equal_c;
  uint64_t key_above_w;
  uint32_t equal_before, equal_here;
  uint32_t cut;                        // first equal (vocabulary index) that is left out; entries of the sorted prefix
  float red[2][kWarps];
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
__device__ __forceinline__ float peer_f32(const void* p, uint32_t rank) { return __uint_as_float(peer_u32(p, rank)); }
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

// A running sum of weights, for up to 4096 terms: adding 1.5 2^3 leaves 2^y rounded to a multiple of 2^-20 in the
// low bits, adding 1.5 2^-17 to what is left does the same for 2^-40; both images are summed as integers.
struct WeightSum {
  uint32_t hi = 0, lo = 0, n = 0;
  __device__ __forceinline__ void add(float y) {
    const float e = ex2_approx(y);
    const float t = __fadd_rn(e, 12.0f);
    const float rest = __fsub_rn(e, __fsub_rn(t, 12.0f));
    hi += __float_as_uint(t);
    lo += __float_as_uint(__fadd_rn(rest, 0x1.8p-17f));
    ++n;
  }
  __device__ __forceinline__ uint64_t total() const {
    const uint32_t h = hi - n * __float_as_uint(12.0f);
    const int32_t l = static_cast<int32_t>(lo - n * __float_as_uint(0x1.8p-17f));
    return (static_cast<uint64_t>(h) << 20) + static_cast<uint64_t>(static_cast<int64_t>(l));
  }
};

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
// the slice padded with -inf.  A warp owns a contiguous run of vectors.
template <int DT>
struct Slice {
  static constexpr int kElems = Vec<DT>::kElems;
  using Elem = typename std::conditional<DT == SV_BF16, uint16_t, uint32_t>::type;
  unsigned char* data;
  int phase, n, vecs;
  int run_a, run_z;  // this warp's vectors
  int64_t first;     // vocabulary index of element 0 of the slice

  __device__ __forceinline__ uint4 vec(int i) const { return lds128(data + static_cast<size_t>(i) * 16); }
  // by position in the padded slice
  __device__ __forceinline__ float at(int pos) const {
    if constexpr (DT == SV_BF16) return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(data)[pos]) << 16);
    else return reinterpret_cast<const float*>(data)[pos];
  }
  __device__ __forceinline__ int index_of(int pos) const { return static_cast<int>(first) + pos - phase; }
};

// Boundary of a prefix of the order (x desc): the smallest one whose count, or weight, reaches what is asked for.
// key 0: none, everything lies above.
struct Boundary {
  uint32_t key, above_c, equal_c, equal_before, equal_here;
  uint64_t above_w;
};

// Adds a weight to a histogram step in limbs.
__device__ __forceinline__ void add_limbs(Shared& sh, int step, uint64_t w) {
  const uint32_t mask = (1u << kLimb) - 1u;
  const uint32_t a = static_cast<uint32_t>(w) & mask, b = static_cast<uint32_t>(w >> kLimb) & mask,
                 c = static_cast<uint32_t>(w >> (2 * kLimb));
  if (a) atomicAdd(&sh.limb[0][step], a);
  if (b) atomicAdd(&sh.limb[1][step], b);
  if (c) atomicAdd(&sh.limb[2][step], c);
}
__device__ __forceinline__ uint64_t limbs_of(uint64_t a, uint64_t b, uint64_t c) { return a + (b << kLimb) + (c << (2 * kLimb)); }

__device__ __forceinline__ void clear_histogram(Shared& sh) {
  const int t = threadIdx.x;
  sh.count[t] = sh.limb[0][t] = sh.limb[1][t] = sh.limb[2][t] = 0;
}

// Sum over the threads before this one (exclusive) of a 64-bit value.
__device__ uint64_t block_scan(Shared& sh, uint64_t v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 31) sh.scan_w[warp] = x;
  __syncthreads();
  uint64_t before = x - v;
  for (int w = 0; w < warp; ++w) before += sh.scan_w[w];
  return before;
}

// The cluster's count and weight of one histogram step.
__device__ __noinline__ void merged_step(const Shared& sh, int step, bool weights, uint32_t* c, uint64_t* w) {
  const uint32_t cs = cluster_size();
  uint32_t n = 0;
  uint64_t l0 = 0, l1 = 0, l2 = 0;
  for (uint32_t r = 0; r < cs; ++r) {
    n += peer_u32(&sh.count[step], r);
    if (weights) {
      l0 += peer_u32(&sh.limb[0][step], r);
      l1 += peer_u32(&sh.limb[1][step], r);
      l2 += peer_u32(&sh.limb[2][step], r);
    }
  }
  *c = n;
  *w = limbs_of(l0, l1, l2);
}

// Finds the first thread, in thread order, at which base + the running sum of c (or w) reaches `want`; writes
// step = its index, above_c / above_w = the sums before it, here_c to shared memory; step = 0xFFFFFFFF if none does.
template <bool kByWeight>
__device__ __noinline__ void find_step(Shared& sh, uint32_t c, uint64_t w, uint64_t want, uint32_t base_c, uint64_t base_w) {
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
  __syncthreads();
  if (lane == 31) {
    sh.scan_c[warp] = ci;
    sh.scan_w[warp] = wi;
  }
  if (threadIdx.x == 0) sh.step = 0xFFFFFFFFu;
  __syncthreads();
  ci += base_c;
  wi += base_w;
  for (int i = 0; i < warp; ++i) {
    ci += sh.scan_c[i];
    wi += sh.scan_w[i];
  }
  if (c > 0 && (kByWeight ? wi >= want && wi - w < want : ci >= want && ci - c < want)) {
    sh.step = threadIdx.x;
    sh.above_c = ci - c;
    sh.above_w = wi - w;
    sh.here_c = c;
  }
  __syncthreads();
}

// Radix descent over the whole row, 8 bits of the key a level.
template <int DT, bool kByWeight>
__device__ __noinline__ Boundary descend(const Slice<DT>& s, Shared& sh, uint64_t want, float top, float steep) {
  constexpr int kLevels = DT == SV_BF16 ? 2 : 4;
  const uint32_t rank = cluster_rank();
  uint32_t prefix = 0, above_c = 0;
  uint64_t above_w = 0;
  Boundary b = {};
  for (int level = 0; level < kLevels; ++level) {
    const int shift = 24 - 8 * level;
    clear_histogram(sh);
    __syncthreads();
    for (int v = threadIdx.x; v < s.vecs; v += kThreads) {
      const Vec<DT> x(s.vec(v));
#pragma unroll
      for (int e = 0; e < Vec<DT>::kElems; ++e) {
        const uint32_t key = key_of(x.x[e]);
        if (x.x[e] != -INFINITY && (level == 0 || (key >> (shift + 8)) == prefix)) {
          const uint32_t step = 255u - ((key >> shift) & 255u);  // large logits first
          atomicAdd(&sh.count[step], 1u);
          if (kByWeight) add_limbs(sh, step, weight_of(exponent_of(x.x[e], top, steep)));
        }
      }
    }
    cluster_sync();  // every slice's histogram is complete
    uint32_t c;
    uint64_t w;
    merged_step(sh, threadIdx.x, kByWeight, &c, &w);
    find_step<kByWeight>(sh, c, w, want, above_c, above_w);
    if (sh.step == 0xFFFFFFFFu) {  // fewer than `want`: everything is kept
      cluster_sync();
      return b;
    }
    above_c = sh.above_c;
    above_w = sh.above_w;
    const uint32_t digit = 255u - sh.step;
    prefix = level == 0 ? digit : (prefix << 8) | digit;
    if (level == kLevels - 1) {
      b.equal_c = sh.here_c;
      b.equal_here = sh.count[sh.step];
      for (uint32_t r = 0; r < rank; ++r) b.equal_before += peer_u32(&sh.count[sh.step], r);
    }
    cluster_sync();  // the peers have read this histogram
  }
  // a bf16 key's low half is all ones for a negative logit, else 0
  b.key = DT == SV_BF16 ? ((prefix << 16) | ((prefix & 0x8000u) ? 0u : 0xFFFFu)) : prefix;
  b.above_c = above_c;
  b.above_w = above_w;
  return b;
}

// Calls f(position, x) for this warp's logits at or above `bound`, in vocabulary order and by whole warps: lanes
// without one get position -1.  listed >= 0: from the warp's list.
template <int DT, typename F>
__device__ __forceinline__ void for_candidates(const Slice<DT>& s, const Shared& sh, int listed, float bound, F f) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (listed >= 0) {
    for (int i = lane; i - lane < listed; i += 32) {
      const int pos = i < listed ? sh.list[warp][i] : -1;
      f(pos, pos >= 0 ? s.at(pos) : -INFINITY);
    }
  } else {
    for (int p0 = s.run_a * Slice<DT>::kElems; p0 < s.run_z * Slice<DT>::kElems; p0 += 32) {
      const int pos = p0 + lane;
      const float x = pos < s.run_z * Slice<DT>::kElems ? s.at(pos) : -INFINITY;
      const bool in = x >= bound && x != -INFINITY;
      if (__any_sync(0xFFFFFFFFu, in)) f(in ? pos : -1, in ? x : -INFINITY);
    }
  }
}

// Steps of the candidates' histogram: equal widths between the top and the bound, the last one open.
struct Scale {
  float top, inv;
  static __device__ __forceinline__ Scale over(float top, float range) {
    return {top, range > 0.0f ? fminf(static_cast<float>(kSteps - 1) / range, FLT_MAX) : 0.0f};
  }
  __device__ __forceinline__ int step(float x) const {
    return static_cast<int>(fminf(__fmul_rn(__fsub_rn(top, x), inv), static_cast<float>(kSteps - 1)));
  }
};

// The logits of one step, exchanged over the cluster and ranked: the boundary by count or weight, given the sums
// above the step.
template <int DT, bool kByWeight>
__device__ __noinline__ Boundary rank_step(const Slice<DT>& s, Shared& sh, int listed, float bound, const Scale& scale, int step,
                              uint64_t want, uint32_t above_c, uint64_t above_w, float top, float steep) {
  const uint32_t cs = cluster_size(), rank = cluster_rank();
  const int tid = threadIdx.x;
  if (tid == 0) {
    sh.mine_n = 0;
    sh.equal_before = sh.equal_here = 0;
  }
  __syncthreads();
  for_candidates<DT>(s, sh, listed, bound, [&](int pos, float x) {
    if (pos >= 0 && scale.step(x) == step) sh.mine[atomicAdd(&sh.mine_n, 1u)] = key_of(x);
  });
  cluster_sync();
  if (tid <= static_cast<int>(cs)) {
    uint32_t n = 0;
    for (int r = 0; r < tid; ++r) n += peer_u32(&sh.mine_n, r);
    sh.from[tid] = n;
  }
  __syncthreads();
  const uint32_t n = sh.from[cs];
  uint32_t key = 0;
  uint64_t w = 0;
  if (tid < static_cast<int>(n)) {
    uint32_t r = 0;
    while (sh.from[r + 1] <= static_cast<uint32_t>(tid)) ++r;
    key = peer_u32(&sh.mine[tid - sh.from[r]], r);
    w = weight_of(exponent_of(logit_of_key(key), top, steep));
    sh.all[tid] = key;
    sh.all_w[tid] = w;
  }
  __syncthreads();
  if (tid < static_cast<int>(n)) {
    uint32_t more = 0, equal = 0;
    uint64_t more_w = 0;
    for (uint32_t i = 0; i < n; ++i) {
      const uint32_t k = sh.all[i];
      more += k > key;
      equal += k == key;
      if (kByWeight) more_w += k > key ? sh.all_w[i] : 0;
    }
    const bool here = kByWeight ? above_w + more_w < want && above_w + more_w + equal * w >= want
                                : above_c + more < want && above_c + more + equal >= want;
    if (here) {  // every holder of the key writes the same
      if (!kByWeight)
        for (uint32_t i = 0; i < n; ++i) more_w += sh.all[i] > key ? sh.all_w[i] : 0;
      sh.key = key;
      sh.key_above_c = above_c + more;
      sh.key_above_w = above_w + more_w;
      sh.key_equal_c = equal;
      if (tid < static_cast<int>(sh.from[rank])) atomicAdd(&sh.equal_before, 1u);
      else if (tid < static_cast<int>(sh.from[rank + 1])) atomicAdd(&sh.equal_here, 1u);
    }
  }
  __syncthreads();
  Boundary b;
  b.key = sh.key;
  b.above_c = sh.key_above_c;
  b.above_w = sh.key_above_w;
  b.equal_c = sh.key_equal_c;
  b.equal_before = sh.equal_before;
  b.equal_here = sh.equal_here;
  return b;
}

// Sum of one value per thread over the cluster (one cluster barrier; a second one before sh.z may be written again).
__device__ __noinline__ uint64_t cluster_total(Shared& sh, uint64_t v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_sum(v);
  if (lane == 0) sh.seg[warp] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    uint64_t z = 0;
    for (int i = 0; i < kWarps; ++i) z += sh.seg[i];
    sh.z = z;
  }
  cluster_sync();
  uint64_t total = 0;
  for (uint32_t r = 0; r < cluster_size(); ++r) total += peer_u64(&sh.z, r);
  return total;
}

// What a row asks for, the same in every CTA of its cluster.
struct Ask {
  const SampleParams* p;
  void* out_row;       // this slice's part of the cut row, or NULL
  int64_t row;
  float top, steep, least, bound;
  uint64_t total;      // W, where it is known
  int k;
  uint32_t p24;
  bool by_count, nucleus, floor_on;
};

// Up to 128 KB of shared memory is on its way at once: waits of microseconds, not inlined.
__device__ __noinline__ void wait_piece(uint64_t* bar, uint32_t* status) { mbar_wait(bar, 0, status); }

// Draws from the weights of `gather` (vocabulary order) at or above `last`, whose sum is z; thread t looks at its run
// of `per` entries.
__device__ __forceinline__ void draw_gathered(Shared& sh, const Ask& ask, const uint64_t* g, int n, uint64_t last, uint64_t z) {
  const int per = (n + kThreads - 1) / kThreads;
  const int a = min(n, static_cast<int>(threadIdx.x) * per), b = min(n, a + per);
  auto weight = [&](int i) {
    return g[i] >= last ? weight_of(exponent_of(logit_of_key(static_cast<uint32_t>(g[i] >> 32)), ask.top, ask.steep)) : 0;
  };
  uint64_t sum = 0;
  for (int i = a; i < b; ++i) sum += weight(i);
  const uint64_t before = block_scan(sh, sum);
  const SampleParams& p = *ask.p;
  for (int j = 0; j < p.M; ++j) {
    const uint64_t t = share_of(z, static_cast<uint32_t>(p.uniforms[ask.row * p.M + j] * 16777216.0f));
    if (t < before || t >= before + sum) continue;
    uint64_t at = before;
    for (int i = a; i < b; ++i) {
      const uint64_t w = weight(i);
      if (t < at + w) {
        p.out_tokens[ask.row * p.M + j] = static_cast<int32_t>(~static_cast<uint32_t>(g[i]));
        if (p.out_probs != nullptr) p.out_probs[ask.row * p.M + j] = __fdiv_rn(__ull2float_rn(w), __ull2float_rn(z));
        break;
      }
      at += w;
    }
  }
}

// Step 3 in the cluster's first CTA, which holds the n gathered logits in vocabulary order; `sorted`: room for as many
// (a power of two, at most kGather).
template <int DT>
__device__ __noinline__ void finish_gathered(Shared& sh, const Ask& ask, int n, uint64_t* sorted) {
  const int tid = threadIdx.x;
  int size = 32;
  while (size < n) size *= 2;
  for (int i = tid; i < size; i += kThreads) sorted[i] = i < n ? sh.gather[i] : 0;
  __syncthreads();
  // bitonic, descending: by logit, then by index
#pragma unroll 1
  for (int block = 2; block <= size; block *= 2)
#pragma unroll 1
    for (int stride = block / 2; stride > 0; stride /= 2) {
      for (int i = tid; i < size / 2; i += kThreads) {
        const int lo = 2 * i - (i & (stride - 1)), hi = lo + stride;
        const uint64_t x = sorted[lo], y = sorted[hi];
        if ((x < y) == ((lo & block) == 0)) {
          sorted[lo] = y;
          sorted[hi] = x;
        }
      }
      // a warp's pairs of a stride up to 32 lie in 64 entries that only this warp touches until the next longer stride
      if (stride > 32 || (stride == 1 && block >= 64)) __syncthreads(); else __syncwarp();
    }
  __syncthreads();
  const int per = (n + kThreads - 1) / kThreads;
  const int a = min(n, tid * per), b = min(n, a + per);
  auto exponent = [&](int i) { return exponent_of(logit_of_key(static_cast<uint32_t>(sorted[i] >> 32)), ask.top, ask.steep); };
  // how many entries are kept: the top-k, the top-p of their weight, those above min-p
  int kept = ask.by_count ? min(ask.k, n) : n;
  uint64_t sum = 0;
  for (int i = a; i < min(b, kept); ++i) sum += weight_of(exponent(i));
  const uint64_t before = block_scan(sh, sum);
  uint64_t total = ask.total;
  if (ask.by_count) {
    __syncthreads();
    if (tid == kThreads - 1) sh.z = before + sum;
    __syncthreads();
    total = sh.z;
  }
  if (tid == 0) sh.cut = kept;
  __syncthreads();
  if (ask.nucleus || ask.floor_on) {
    const uint64_t limit = ask.nucleus ? max(share_of(total, ask.p24), uint64_t(1)) : ~uint64_t(0);
    uint64_t at = before;
    for (int i = a; i < min(b, kept); ++i) {
      const float y = exponent(i);
      if (at >= limit || y < ask.least) {  // the first entry of this thread that is left out
        atomicMin(&sh.cut, static_cast<uint32_t>(i));
        break;
      }
      at += weight_of(y);
    }
    __syncthreads();
  }
  kept = static_cast<int>(sh.cut);
  const uint64_t last = sorted[kept - 1];  // (the largest logit is always kept)
  uint64_t mine = 0;
  for (int i = a; i < min(b, kept); ++i) mine += weight_of(exponent(i));
  mine = warp_sum(mine);
  if ((tid & 31) == 0) sh.seg[tid >> 5] = mine;
  __syncthreads();
  uint64_t z = 0;
  for (int w = 0; w < kWarps; ++w) z += sh.seg[w];
  if (ask.out_row != nullptr) {  // the first CTA's part begins the row
    using Elem = typename Slice<DT>::Elem;
    Elem* out = static_cast<Elem*>(ask.out_row);
    for (int i = tid; i < kept; i += kThreads) {
      const uint32_t bits = __float_as_uint(logit_of_key(static_cast<uint32_t>(sorted[i] >> 32)));
      out[~static_cast<uint32_t>(sorted[i])] = DT == SV_BF16 ? static_cast<Elem>(bits >> 16) : static_cast<Elem>(bits);
    }
  }
  draw_gathered(sh, ask, sh.gather, n, last, z);
}

// Steps 3 and 4 with the lists where they are.
template <int DT>
__device__ __noinline__ void cut_wide(const Slice<DT>& s, Shared& sh, const Ask& ask, int listed) {
  using Elem = typename Slice<DT>::Elem;
  constexpr int kElems = Slice<DT>::kElems;
  const SampleParams& p = *ask.p;
  const uint32_t cs = cluster_size(), rank = cluster_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float top = ask.top, steep = ask.steep, bound = ask.bound;
  uint64_t total = ask.total;
  Boundary b = {};
  uint32_t ties_kept = 0;  // how many of the boundary's equals are kept, lowest indexes first
  if (ask.by_count || ask.nucleus) {
    clear_histogram(sh);
    const Scale scale = Scale::over(top, bound == -INFINITY ? 64.0f / steep : __fsub_rn(top, bound));
    __syncthreads();
    for_candidates<DT>(s, sh, listed, bound, [&](int pos, float x) {
      if (pos >= 0) {
        const int step = scale.step(x);
        atomicAdd(&sh.count[step], 1u);
        if (ask.nucleus) add_limbs(sh, step, weight_of(exponent_of(x, top, steep)));
      }
    });
    cluster_sync();
    uint32_t c;
    uint64_t w;
    merged_step(sh, tid, ask.nucleus, &c, &w);
    bool found = true, crowded = false;
    if (ask.by_count) {
      find_step<false>(sh, c, w, ask.k, 0, 0);
      found = sh.step != 0xFFFFFFFFu;  // else fewer than k logits: all are kept
      crowded = found && sh.here_c > kExchange;
      const int step = sh.step;
      const uint32_t above_c = sh.above_c;
      const uint64_t above_w = sh.above_w;
      cluster_sync();  // the peers have read the histogram (the exchange's arrays are beside it)
      if (crowded) b = descend<DT, false>(s, sh, ask.k, top, steep);
      else if (found) b = rank_step<DT, false>(s, sh, listed, bound, scale, step, ask.k, above_c, above_w, top, steep);
      ties_kept = found ? ask.k - b.above_c : 0;
    }
    if (ask.nucleus) {
      if (ask.by_count) {
        // W: what lies above the boundary, and its kept equals
        if (found && !crowded) {
          total = b.above_w;
        } else {
          WeightSum sum;
          for (int v = s.run_a + lane; v < s.run_z; v += 32) {
            const Vec<DT> x(s.vec(v));
#pragma unroll
            for (int e = 0; e < kElems; ++e)
              if (key_of(x.x[e]) > b.key) sum.add(exponent_of(x.x[e], top, steep));
          }
          total = cluster_total(sh, sum.total());
        }
        if (found) total += static_cast<uint64_t>(ties_kept) * weight_of(exponent_of(logit_of_key(b.key), top, steep));
      }
      const uint64_t limit = max(share_of(total, ask.p24), uint64_t(1));
      if (crowded) {
        b = descend<DT, true>(s, sh, limit, top, steep);
      } else {
        find_step<true>(sh, c, w, limit, 0, 0);
        const int step = sh.step;
        const uint32_t here_c = sh.here_c, above_c = sh.above_c;
        const uint64_t above_w = sh.above_w;
        const bool inside = sh.step != 0xFFFFFFFFu;
        cluster_sync();  // the peers have read the histogram, or the keys exchanged before
        // (a bound at min-p's threshold may lie above the boundary: then everything above the bound is kept)
        if (inside ? here_c > kExchange : !ask.floor_on) b = descend<DT, true>(s, sh, limit, top, steep);
        else if (inside) b = rank_step<DT, true>(s, sh, listed, bound, scale, step, limit, above_c, above_w, top, steep);
        else b = Boundary{};
      }
      if (b.key != 0) {
        const uint64_t each = weight_of(exponent_of(logit_of_key(b.key), top, steep));
        ties_kept = each == 0 ? 0 : static_cast<uint32_t>((limit - b.above_w + each - 1) / each);
      }
    }
  }
  // equals of this slice that are kept: those before vocabulary index `cut`
  uint32_t cut = 0xFFFFFFFFu;
  {
    const uint32_t quota = ties_kept > b.equal_before ? min(ties_kept - b.equal_before, b.equal_here) : 0;
    if (b.key == 0 || quota == 0) {
      cut = 0;
    } else if (quota < b.equal_here) {
      uint32_t c = 0;
      for_candidates<DT>(s, sh, listed, bound, [&](int pos, float x) { c += pos >= 0 && key_of(x) == b.key; });
      c = __reduce_add_sync(0xFFFFFFFFu, c);
      if (lane == 0) sh.ties[warp] = c;
      __syncthreads();
      uint32_t before = 0;
      for (int i = 0; i < warp; ++i) before += sh.ties[i];
      if (before < quota && before + c >= quota)
        for_candidates<DT>(s, sh, listed, bound, [&](int pos, float x) {
          const bool equal = pos >= 0 && key_of(x) == b.key;
          const uint32_t set = __ballot_sync(0xFFFFFFFFu, equal);
          if (equal && before + __popc(set & ((1u << lane) - 1u)) == quota - 1) sh.cut = static_cast<uint32_t>(s.index_of(pos)) + 1;
          before += __popc(set);
        });
      __syncthreads();
      cut = sh.cut;
    }
  }
  auto keeps = [&](int pos, float x) {
    const uint32_t key = key_of(x);
    return (key > b.key || (key == b.key && static_cast<uint32_t>(s.index_of(pos)) < cut)) && exponent_of(x, top, steep) >= ask.least;
  };
  // kept weights by warp, the row's total, the kept logits
  Elem* out_row = static_cast<Elem*>(ask.out_row);
  uint64_t w = 0;
  for_candidates<DT>(s, sh, listed, bound, [&](int pos, float x) {
    if (pos >= 0 && keeps(pos, x)) {
      w += weight_of(exponent_of(x, top, steep));
      if (out_row != nullptr) out_row[pos - s.phase] = reinterpret_cast<const Elem*>(s.data)[pos];
    }
  });
  w = warp_sum(w);
  cluster_sync();  // sh.z may be written again
  if (lane == 0) sh.seg[warp] = w;
  __syncthreads();
  if (tid == 0) {
    uint64_t z = 0;
    for (int i = 0; i < kWarps; ++i) z += sh.seg[i];
    sh.z = z;
  }
  cluster_sync();
  uint64_t before = 0, z = 0, mine = 0;
  for (uint32_t r = 0; r < cs; ++r) {
    const uint64_t zr = peer_u64(&sh.z, r);
    if (r < rank) before += zr;
    if (r == rank) mine = zr;
    z += zr;
  }
  // the draws: the CTA that holds a draw's crossing, its warp, its logit
  for (int j = 0; j < p.M; ++j) {
    const uint32_t u24 = static_cast<uint32_t>(p.uniforms[ask.row * p.M + j] * 16777216.0f);
    uint64_t t = share_of(z, u24);
    if (t < before || t >= before + mine) continue;
    t -= before;
    uint64_t ahead = 0;
    for (int i = 0; i < warp; ++i) ahead += sh.seg[i];
    if (t < ahead || t >= ahead + sh.seg[warp]) continue;  // the warp that owns the run draws
    t -= ahead;
    bool open = true;
    for_candidates<DT>(s, sh, listed, bound, [&](int pos, float x) {
      if (!open) return;
      const uint64_t we = pos >= 0 && keeps(pos, x) ? weight_of(exponent_of(x, top, steep)) : 0;
      uint64_t incl = we;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += u;
      }
      const uint64_t all = __shfl_sync(0xFFFFFFFFu, incl, 31);
      if (t < all) {
        if (t < incl && t >= incl - we) {
          p.out_tokens[ask.row * p.M + j] = s.index_of(pos);
          if (p.out_probs != nullptr) p.out_probs[ask.row * p.M + j] = __fdiv_rn(__ull2float_rn(we), __ull2float_rn(z));
        }
        open = false;
      }
      t -= all;
    });
  }
  cluster_sync();  // no CTA leaves while a peer may still read its shared memory
}

// No filter: every logit's weight.  A lane sums a contiguous stretch of its warp's run (an odd number of vectors, so
// that a quarter warp's 16-byte loads fall on different banks): a draw then looks into one lane's stretch.
template <int DT>
__device__ __noinline__ void draw_all(const Slice<DT>& s, Shared& sh, const Ask& ask) {
  using Elem = typename Slice<DT>::Elem;
  constexpr int kElems = Slice<DT>::kElems;
  const SampleParams& p = *ask.p;
  const uint32_t cs = cluster_size(), rank = cluster_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int stretch = (s.run_z - s.run_a + 31) / 32 | 1;
  const int va = min(s.run_z, s.run_a + lane * stretch), vz = min(s.run_z, va + stretch);
  WeightSum sum;
  for (int v = va; v < vz; ++v) {
    const Vec<DT> x(s.vec(v));
#pragma unroll
    for (int e = 0; e < kElems; ++e) sum.add(exponent_of(x.x[e], ask.top, ask.steep));
  }
  if (ask.out_row != nullptr)
    for (int pos = s.run_a * kElems + lane; pos < s.run_z * kElems; pos += 32)
      if (pos >= s.phase && pos < s.phase + s.n)
        static_cast<Elem*>(ask.out_row)[pos - s.phase] = reinterpret_cast<const Elem*>(s.data)[pos];
  const uint64_t w = sum.total();
  uint64_t incl = w;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += u;
  }
  if (lane == 31) sh.seg[warp] = incl;
  __syncthreads();
  if (tid == 0) {
    uint64_t z = 0;
    for (int i = 0; i < kWarps; ++i) z += sh.seg[i];
    sh.z = z;
  }
  cluster_sync();
  uint64_t before = 0, z = 0;
  for (uint32_t r = 0; r < cs; ++r) {
    const uint64_t zr = peer_u64(&sh.z, r);
    if (r < rank) before += zr;
    z += zr;
  }
  for (int i = 0; i < warp; ++i) before += sh.seg[i];
  for (int j = 0; j < p.M; ++j) {
    const uint64_t t0 = share_of(z, static_cast<uint32_t>(p.uniforms[ask.row * p.M + j] * 16777216.0f));
    if (t0 < before || t0 >= before + sh.seg[warp]) continue;
    const uint64_t t = t0 - before;
    const uint32_t owner = __ballot_sync(0xFFFFFFFFu, t >= incl - w && t < incl);
    const int from = __ffs(owner) - 1;
    uint64_t left = t - __shfl_sync(0xFFFFFFFFu, incl - w, from);
    const int first = (s.run_a + from * stretch) * kElems, last = min(s.run_z, s.run_a + (from + 1) * stretch) * kElems;
    for (int base = first; base < last; base += 32) {
      const int pos = base + lane;
      const uint64_t we = pos < last ? weight_of(exponent_of(s.at(pos), ask.top, ask.steep)) : 0;
      uint64_t in = we;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, in, d);
        if (lane >= d) in += u;
      }
      const uint64_t all = __shfl_sync(0xFFFFFFFFu, in, 31);
      if (left < all) {
        if (left < in && left >= in - we) {
          p.out_tokens[ask.row * p.M + j] = s.index_of(pos);
          if (p.out_probs != nullptr) p.out_probs[ask.row * p.M + j] = __fdiv_rn(__ull2float_rn(we), __ull2float_rn(z));
        }
        break;
      }
      left -= all;
    }
  }
  cluster_sync();  // no CTA leaves while a peer may still read its shared memory
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
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
  const int run = (s.vecs + kWarps - 1) / kWarps;
  s.run_a = min(s.vecs, warp * run);
  s.run_z = min(s.vecs, s.run_a + run);
  if (tid == 0) {
    for (int i = 0; i < kPieces; ++i) mbar_init(&sh.bar[i], 1);
    fence_proxy_async_smem();
  }
  sh.count[tid] = 0;
  __syncthreads();
  pdl_wait();
  // whole 16-byte vectors by bulk copy, the slice's ragged ends element by element
  const int v0 = s.phase > 0 ? 1 : 0, v1 = (s.phase + s.n) / kElems;
  const int per_piece = max(1, v1 > v0 ? (v1 - v0 + kPieces - 1) / kPieces : 0);
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
  // the ragged ends: at most two vectors
  if (tid < 2 * kElems) {
    const int v = tid < kElems ? 0 : s.vecs - 1;
    const int pos = v * kElems + (tid % kElems);
    if (s.vecs > 0 && (tid < kElems || s.vecs > 1) && !(v >= v0 && v < v1)) {
      const int e = pos - s.phase;
      reinterpret_cast<Elem*>(dyn)[pos] = e >= 0 && e < s.n ? src[e] : none;
    }
  }
  Ask ask;
  const float T = p.temperature[row];
  const int k_in = p.top_k != nullptr ? p.top_k[row] : 0;
  const float p_in = p.top_p != nullptr ? p.top_p[row] : 1.0f;
  const float q_in = p.min_p != nullptr ? p.min_p[row] : 0.0f;
  uint32_t bad = 0;
  if (!(T >= 0.0f) || T == INFINITY) bad |= SV_DEV_BAD_TEMPERATURE;
  if (k_in < 0 || !(p_in > 0.0f && p_in <= 1.0f) || !(q_in >= 0.0f && q_in <= 1.0f)) bad |= SV_DEV_BAD_FILTER;
  bool bad_uniform = false;
  for (int j = tid; j < p.M; j += kThreads) {
    const float u = p.uniforms[row * p.M + j];
    bad_uniform |= !(u >= 0.0f && u < 1.0f);
  }
  const bool greedy = T == 0.0f;
  ask.p = &p;
  ask.row = row;
  ask.total = 0;
  ask.steep = greedy ? 1.0f : fminf(__fdiv_rn(1.44269504088896341f, T), FLT_MAX);
  ask.k = greedy ? 1 : (k_in == 0 ? p.V : k_in);
  ask.by_count = ask.k < p.V;
  ask.nucleus = !greedy && p_in < 1.0f;
  ask.floor_on = !greedy && q_in > 0.0f;
  ask.least = ask.floor_on ? log2f(q_in) : -INFINITY;  // of y
  ask.p24 = static_cast<uint32_t>(rintf(p_in * 16777216.0f));
  // The cut row is -inf but for what is kept: filled while the logits are on their way (a row cut in place only
  // after they have arrived), and the kept logits follow at the end.
  Elem* out_row = p.out_rows != nullptr ? static_cast<Elem*>(p.out_rows) + row * p.out_stride + s.first : nullptr;
  ask.out_row = out_row;
  const bool in_place = p.out_rows == p.logits;
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1) {
      if (__syncthreads_or(bad_uniform)) bad |= SV_DEV_BAD_FILTER;
      if (!in_place) break;
      // every copy of the slice has landed before its place is overwritten
      for (int i = 0; i < kPieces; ++i) wait_piece(&sh.bar[i], p.status);
      __syncthreads();
    }
    if (out_row != nullptr && in_place == (pass == 1)) {
      const int head = min(s.n, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(out_row) & 15u)) & 15u) / sizeof(Elem)));
      const int vecs = (s.n - head) / kElems;
      const uint32_t w = DT == SV_BF16 ? 0xFF80FF80u : 0xFF800000u;
      for (int i = tid; i < vecs; i += kThreads) reinterpret_cast<uint4*>(out_row + head)[i] = make_uint4(w, w, w, w);
      for (int i = tid; i < s.n - vecs * kElems; i += kThreads) out_row[i < head ? i : i + vecs * kElems] = none;
    }
  }
  // ---- the largest logit, of the slice and of each thread's group -------------------------------
  // a warp waits for the copies that hold its run only
  for (int i = 0; i < kPieces; ++i) {
    const int a = v0 + i * per_piece;
    if (a < s.run_z && min(v1, a + per_piece) > s.run_a) wait_piece(&sh.bar[i], p.status);
  }
  float group = -INFINITY;
#pragma unroll 4
  for (int v = s.run_a + lane; v < s.run_z; v += 32) {
    const Vec<DT> x(s.vec(v));
#pragma unroll
    for (int e = 0; e < kElems; ++e) group = max_nan(group, x.x[e]);
  }
  float top = group, low = group == -INFINITY ? INFINITY : group;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, d));
  }
  if (lane == 0) {
    sh.red[0][warp] = top;
    sh.red[1][warp] = low;
  }
  __syncthreads();
  {
    top = lane < kWarps ? sh.red[0][lane] : -INFINITY;
    low = lane < kWarps ? sh.red[1][lane] : INFINITY;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, d));
    }
  }
  if (tid == 0) sh.top = top;
  // ---- 1. a bound ---------------------------------------------------------------------------------
  // the CTA vouches for ranks(j) logits at or above rank_at[j]: from an even share of k to all of it
  auto rank_of = [&](int j) { return static_cast<uint32_t>(ceilf(static_cast<float>(ask.k) * exp2f(-3.0f + 3.0f * j / (kRanks - 1)))); };
  if (ask.by_count) {
    if (tid < kRanks) sh.rank_at[tid] = -INFINITY;
    const Scale groups = Scale::over(top, __fsub_rn(top, low));
    if (group > -INFINITY && top < INFINITY) atomicAdd(&sh.count[groups.step(group)], 1u);
    __syncthreads();
    const uint32_t c = sh.count[tid];
    const uint32_t before = static_cast<uint32_t>(block_scan(sh, c));
#pragma unroll
    for (int j = 0; j < kRanks; ++j) {
      const uint32_t want = rank_of(j);
      // a step's lower end, a little lower than the roundings of step() may put it
      if (before < want && before + c >= want)
        sh.rank_at[j] = groups.inv > 0.0f ? __fsub_rd(top, __fmul_ru(static_cast<float>(tid + 1) / groups.inv, 1.00001f)) : top;
    }
  }
  cluster_sync();
  top = lane < static_cast<int>(cs) ? peer_f32(&sh.top, lane) : -INFINITY;
#pragma unroll
  for (int d = kMaxCluster / 2; d > 0; d >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  top = __shfl_sync(0xFFFFFFFFu, top, 0);
  ask.top = top;
  if (!(top < INFINITY)) bad |= SV_DEV_BAD_LOGIT;
  if (bad != 0 || top == -INFINITY) {  // the same in every CTA of the cluster
    if (bad != 0 && rank == 0 && tid == 0) atomicOr(p.status, bad);
    if (rank == 0)
      for (int j = tid; j < p.M; j += kThreads) {
        p.out_tokens[row * p.M + j] = -1;
        if (p.out_probs != nullptr) p.out_probs[row * p.M + j] = bad != 0 ? NAN : 0.0f;
      }
    cluster_sync();  // no CTA leaves while a peer may still read its shared memory
    return;
  }
  if (!ask.by_count && !ask.nucleus && !ask.floor_on) {
    draw_all<DT>(s, sh, ask);
    return;
  }
  float bound = -INFINITY;
  if (ask.by_count) {
    // the largest published logit above which the CTAs together vouch for k: lane l tries the l-th and the (l + 32)-th
    // (CTA, order statistic)
    if (warp == 0) {
      float at[2];
      int sure[2] = {0, 0};
      for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        at[h] = i < static_cast<int>(cs) * kRanks ? peer_f32(&sh.rank_at[i % kRanks], i / kRanks) : -INFINITY;
      }
      const int mine = static_cast<int>(rank_of(lane % kRanks));
      for (uint32_t r = 0; r < cs; ++r) {
        int most[2] = {0, 0};
        for (int j = 0; j < kRanks; ++j) {
          const int i = r * kRanks + j;
          const float v = __shfl_sync(0xFFFFFFFFu, i < 32 ? at[0] : at[1], i & 31);
          const int vouched = __shfl_sync(0xFFFFFFFFu, mine, j);
          if (v >= at[0]) most[0] = vouched;
          if (v >= at[1]) most[1] = vouched;
        }
        sure[0] += most[0];
        sure[1] += most[1];
      }
      for (int h = 0; h < 2; ++h)
        if (at[h] > -INFINITY && sure[h] >= ask.k) bound = fmaxf(bound, at[h]);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) bound = fmaxf(bound, __shfl_xor_sync(0xFFFFFFFFu, bound, d));
      if (lane == 0) sh.red[0][0] = bound;
    }
    __syncthreads();
    bound = sh.red[0][0];
  } else if (ask.nucleus) {
    WeightSum sum;
#pragma unroll 2
    for (int v = s.run_a + lane; v < s.run_z; v += 32) {
      const Vec<DT> x(s.vec(v));
#pragma unroll
      for (int e = 0; e < kElems; ++e) sum.add(exponent_of(x.x[e], top, ask.steep));
    }
    ask.total = cluster_total(sh, sum.total());
    // V weights of at most this (and half a unit of rounding each) stay below (1 - p) W; 1e-3 covers ex2 and log2
    const float each = static_cast<float>(ask.total) * (static_cast<float>((1u << 24) - ask.p24) * 0x1p-24f) / static_cast<float>(p.V) - 0.5f;
    if (each > 0.0f) bound = __fadd_rd(top, __fdiv_rd(log2f(each) - 40.0f - 1e-3f, ask.steep));
  }
  // Below min-p's threshold nothing is kept.  The boundary may then lie below the bound: it is not found, and everything
  // above the bound is kept.  Only the top-k's own weight needs all of the top-k.
  if (ask.floor_on && !(ask.by_count && ask.nucleus)) bound = fmaxf(bound, __fadd_rd(top, __fdiv_rd(ask.least * 1.000001f, ask.steep)));
  if (!(bound < top)) bound = bound >= top ? top : -INFINITY;
  ask.bound = bound;
  // ---- 2. the logits at or above the bound, by warp and in order -------------------------------
  int n = 0;
#pragma unroll 1
  for (int vb = s.run_a; vb < s.run_z; vb += 32) {
    const int v = vb + lane;
    uint32_t mask = 0;
    if (v < s.run_z) {
      const Vec<DT> x(s.vec(v));
#pragma unroll
      for (int e = 0; e < kElems; ++e) mask |= (x.x[e] >= bound && x.x[e] != -INFINITY ? 1u : 0u) << e;
    }
    if (__any_sync(0xFFFFFFFFu, mask != 0)) {
      const int c = __popc(mask);
      int incl = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += u;
      }
      int at = n + incl - c;
      n += __shfl_sync(0xFFFFFFFFu, incl, 31);
      if (n <= kListPerWarp)
        for (uint32_t m = mask; m != 0; m &= m - 1) sh.list[warp][at++] = static_cast<uint16_t>(v * kElems + __ffs(m) - 1);
    }
  }
  const int listed = n <= kListPerWarp ? n : -1;
  // ---- 3. gathered by the first CTA, if they are few -----------------------------------------------
  const bool few = __syncthreads_and(listed >= 0) && (!ask.by_count || ask.k <= kGatherK);
  if (lane == 0) sh.ties[warp] = n;
  __syncthreads();
  uint32_t at = 0, all = 0;
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) at += sh.ties[i];
    all += sh.ties[i];
  }
  const bool fits = few && all <= kGather;
  if (fits)
    for (int i = lane; i < listed; i += 32) {
      const int pos = sh.list[warp][i];
      sh.gather[at + i] = static_cast<uint64_t>(key_of(s.at(pos))) << 32 | static_cast<uint32_t>(~s.index_of(pos));
    }
  if (tid == 0) sh.mine_n = fits ? all : kGather + 1;
  cluster_sync();
  uint32_t gathered = 0;
  for (uint32_t r = 0; r < cs; ++r) gathered += peer_u32(&sh.mine_n, r);
  if (gathered > kGather) {  // the same in every CTA
    cluster_sync();          // everyone has read the counts
    cut_wide<DT>(s, sh, ask, listed);
    return;
  }
  if (rank == 0) {
    uint32_t to = all;
    for (uint32_t r = 1; r < cs; ++r) {
      const uint32_t m = peer_u32(&sh.mine_n, r);
      for (uint32_t i = tid; i < m; i += kThreads) sh.gather[to + i] = peer_u64(&sh.gather[i], r);
      to += m;
    }
  }
  cluster_sync();  // the first CTA has everything: the others leave
  if (rank == 0) finish_gathered<DT>(sh, ask, static_cast<int>(gathered), reinterpret_cast<uint64_t*>(dyn));
}

template <int DT>
cudaError_t launch_sample(SampleParams p, void* stream) {
  constexpr int kElt = DT == SV_BF16 ? 2 : 4;
  int cs = 1;  // slices of about 32 KB: a row's CTAs share its passes
  while (cs < kMaxCluster && static_cast<int64_t>(p.V) * kElt > cs * 32768) cs *= 2;
  p.slice = ((p.V + cs - 1) / cs + 7) & ~7;
  const size_t dyn = std::max(static_cast<size_t>(p.slice) * kElt + 32, sizeof(uint64_t) * kGather);  // (the sort's room too)
  const cudaError_t e = allow_smem<sample_kernel<DT>>(dyn);
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
