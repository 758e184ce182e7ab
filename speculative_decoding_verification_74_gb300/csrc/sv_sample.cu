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
//   3. up to 2048 of them are gathered by the cluster's first CTA, which finds the prefix's end and draws; the other CTAs
//      are done.  Up to 128 are ranked by counting; more go into a histogram (512 steps between bound and top; counts,
//      and weights in three 14-bit limbs, which 32-bit atomics add without overflow), whose step that holds the end
//      is ranked; a step of more than 128 (long runs of equals) is sorted out by sorting the list.
// Longer lists (flat rows under top-p alone, large k) stay with their CTAs (cut_wide): a histogram of counts, summed over
// the cluster, gives the step that holds the boundary (for top-p by the weight of each step's middle, then checked
// against the exact weights of the steps around it), and that step's logits are exchanged and ranked by every CTA.
// Where a step holds more logits than the exchange takes, the boundary is found by a radix descent on the integer image
// of x instead.
//
// Many rows with a top-k or min-p: the latency of a cluster's steps, not memory, bounds the above.  Such rows go another
// way: maxima_kernel streams them once and keeps the largest logit of every 128 bytes; select_kernel (a CTA per row) takes
// the bound from these maxima, reads again only the 128-byte groups that reach it (about k of them; for top-p without
// top-k the whole row, for W) and goes on with step 3.  Rows that it leaves (neither filter, bad input, too long a list)
// are listed for the clusters, which take them in turn.
//
// Measured (GB300, 151936 logits a row; a copy of the same bytes takes 97.5 us for 1088 float32 rows): 1088 rows float32
// plain 297 us, greedy 313 us, top-k 50 163 us (maxima 100, select 55), min-p alone 155 us, top-p 0.9 alone 720 us (peaked
// rows) to 1230 us (flat ones); mixed filters with the cut rows written 377 to 396 us (maxima with the cut rows' -inf 200, 195
// being their copy's; select 80; clusters for the 50 rows with top-p alone 95).  64 rows bf16: plain 15 us, top-k 50 18
// us, top-p alone 54 to 60 us, mixed 39 to 63 us by the rows.  Four rows of 32000: 6.3 to 6.7 us, the latency of one launch
// and its barriers.
// What bounds it now: with few rows the chain of barriers and passes of the slowest row (a flat row under top-p alone
// takes six passes over its slices and ten cluster barriers: 34 us by itself), with many the reading.
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
constexpr int kExchange = 2 * kThreads; // logits of one step that the cluster exchanges: two per thread
constexpr int kLimb = 14;
constexpr int kGather = 2048;           // logits that one CTA sorts
constexpr int kGatherK = 1024;          // largest k that goes that way
constexpr int kTries = 8;               // estimates of the step that holds a top-p boundary, before a radix descent
constexpr int kRanks = 8;               // order statistics of a CTA's groups that it publishes
constexpr int kShort = 128;             // a gathered list this short is ranked by counting, a longer one sorted

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
  int32_t* left;           // [1 + R] the rows that select_kernel leaves to the clusters, after their number; or NULL: all
  float* maxima;           // [R][groups]
  int32_t R, V, M, slice;  // slice: elements per CTA, a multiple of 8
  int32_t groups, segments;
};

// Per-CTA state; the parts that peers read are written before a cluster barrier.
struct Shared {
  union {
    uint64_t gather[kGather];          // this CTA's listed logits: integer image << 32 | ~index; the first CTA's: everybody's
    struct {                           // cut_wide
      uint32_t limb[3][kSteps];
      uint32_t mine[kExchange];        // this CTA's keys of the exchanged step
      uint64_t all_w[kExchange];       // the cluster's, sorted; weights
    };
  };
  uint32_t count[kSteps];
  uint16_t list[kWarps][kListPerWarp];
  uint64_t z;                          // a sum of the slice
  uint32_t top;                        // image of the slice's largest logit
  float rank_at[kRanks];               // a logit at or below the rank_n[j]-th largest group maximum
  float rank_all[kMaxCluster * kRanks];  // the cluster's
  uint32_t rank_n[kRanks];
  uint32_t bound;                      // image of the bound, 0 = none
  uint32_t mine_n;                     // logits in `gather` (more than kGather: too many), or of the exchanged step
  SampleParams params;                 // for functions that are not inlined: a kernel parameter behind a pointer is read
                                       // through global memory
  uint64_t bar[kPieces];
  uint64_t seg[kWarps];
  uint32_t ties[kWarps];
  uint64_t scan_w[kWarps];
  uint32_t scan_c[kWarps];
  uint32_t from[kMaxCluster + 1];      // where each CTA's logits begin in the cluster's list
  uint32_t step, above_c, here_c;      // the step that holds a boundary
  uint64_t above_w;
  uint32_t key, key_above_c;
  uint64_t key_above_w;
  uint64_t end[2];                     // the prefix's last logit, and the weight up to it
  uint32_t cut;                        // first equal (vocabulary index) that is left out; entries of the sorted prefix
  uint32_t red[2][kWarps];
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// cluster_sync in two halves.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
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
// low bits, adding 1.5 2^-17 to what is left does the same for 2^-40; both images are summed as integers.  Two logits
// at a time in packed arithmetic, each half rounded like the scalar operation.  A logit of -inf adds nothing.
__device__ __forceinline__ f32x2 f2_mul(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
struct WeightSum {
  uint32_t hi = 0, lo = 0;
  f32x2 minus_top, steep;
  __device__ __forceinline__ WeightSum(float top, float s) : minus_top(f2_pack(-top, -top)), steep(f2_pack(s, s)) {}
  __device__ __forceinline__ void add(float x0, float x1) {
    float y0, y1, t0, t1, r0, r1;
    f2_unpack(f2_mul(f2_add(f2_pack(x0, x1), minus_top), steep), y0, y1);
    const f32x2 e = f2_pack(ex2_approx(y0), ex2_approx(y1));
    const f32x2 t = f2_add(e, f2_pack(12.0f, 12.0f));
    f2_unpack(t, t0, t1);
    const f32x2 high = f2_add(t, f2_pack(-12.0f, -12.0f));
    float h0, h1;
    f2_unpack(high, h0, h1);
    f2_unpack(f2_add(f2_add(e, f2_pack(-h0, -h1)), f2_pack(0x1.8p-17f, 0x1.8p-17f)), r0, r1);
    hi += __float_as_uint(t0) + __float_as_uint(t1);
    lo += __float_as_uint(r0) + __float_as_uint(r1);
  }
  // after n additions (of two)
  __device__ __forceinline__ uint64_t total(uint32_t n) const {
    const uint32_t h = hi - 2 * n * __float_as_uint(12.0f);
    const int32_t l = static_cast<int32_t>(lo - 2 * n * __float_as_uint(0x1.8p-17f));
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
// The cluster's sum of one value per CTA, by every warp for itself: a lane per CTA (reads of peers one after the other take
// 0.25 us each).
__device__ __forceinline__ uint64_t peers_sum(const uint64_t* value) {
  const uint32_t r = threadIdx.x % kMaxCluster;
  uint64_t v = r < cluster_size() ? peer_u64(value, r) : 0;
#pragma unroll
  for (int d = kMaxCluster / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
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

// This warp's weights of the logits above `last` (each lane its share; any order).
template <int DT>
__device__ __forceinline__ uint64_t weights_above(const Slice<DT>& s, float last, float top, float steep) {
  const int lane = threadIdx.x & 31;
  WeightSum sum(top, steep);
  uint32_t n = 0;
#pragma unroll 2
  for (int v = s.run_a + lane; v < s.run_z; v += 32, ++n) {
    const Vec<DT> x(s.vec(v));
#pragma unroll
    for (int e = 0; e < Vec<DT>::kElems; e += 2)
      sum.add(x.x[e] > last ? x.x[e] : -INFINITY, x.x[e + 1] > last ? x.x[e + 1] : -INFINITY);
  }
  return sum.total(n * (Vec<DT>::kElems / 2));
}

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

// Sum over the threads before this one (exclusive).
__device__ uint32_t block_scan32(Shared& sh, uint32_t v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 31) sh.scan_c[warp] = x;
  __syncthreads();
  const uint32_t ahead = lane < warp ? sh.scan_c[lane] : 0;  // (warp <= 16: the lanes cover it)
  return x - v + __reduce_add_sync(0xFFFFFFFFu, ahead);
}
// The same for 64 bits.
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
  uint32_t n = 0, part[kMaxCluster];
  uint64_t l0 = 0, l1 = 0, l2 = 0;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) part[r] = r < cs ? peer_u32(&sh.count[step], r) : 0;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) n += part[r];
  if (weights)
    for (uint32_t r = 0; r < cs; ++r) {
      l0 += peer_u32(&sh.limb[0][step], r);
      l1 += peer_u32(&sh.limb[1][step], r);
      l2 += peer_u32(&sh.limb[2][step], r);
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

// Steps of the candidates' histogram: equal widths between the top and the bound, the last one open.
struct Scale {
  float top, inv;
  static __device__ __forceinline__ Scale over(float top, float range) {
    return {top, range > 0.0f ? fminf(static_cast<float>(kSteps - 1) / range, FLT_MAX) : 0.0f};
  }
  // a logit surely above the steps from `step` on, and one surely below those up to it (step() rounds a little)
  __device__ __forceinline__ float above(int step) const {
    return inv > 0.0f && step > 0 ? __fadd_ru(top, __fmul_ru(-(step / inv), 0.99999f)) : INFINITY;
  }
  __device__ __forceinline__ float below(int step) const {
    return inv > 0.0f && step < kSteps - 1 ? __fadd_rd(top, __fmul_rd(-((step + 1) / inv), 1.00001f)) : -INFINITY;
  }
  // A logit at or below every one of the steps up to `step`, a little lower than the roundings of step() may put it; `range`
  // as given to over().  A range past the largest float (finite logits of 2e38 beside -2e38) leaves one step for all:
  // its lower end is not known.
  __device__ __forceinline__ float lower_end(int step, float range) const {
    return inv > 0.0f ? __fsub_rd(top, __fmul_ru(static_cast<float>(step + 1) / inv, 1.00001f)) : range > 0.0f ? -INFINITY : top;
  }
  __device__ __forceinline__ int step(float x) const {
    return static_cast<int>(fminf(__fmul_rn(__fsub_rn(top, x), inv), static_cast<float>(kSteps - 1)));
  }
};

// Bitonic sort, descending, of `size` (a power of two) entries.
__device__ __noinline__ void sort_descending(uint64_t* x, int size) {
#pragma unroll 1
  for (int block = 2; block <= size; block *= 2)
#pragma unroll 1
    for (int stride = block / 2; stride > 0; stride /= 2) {
      for (int i = threadIdx.x; i < size / 2; i += kThreads) {
        const int lo = 2 * i - (i & (stride - 1)), hi = lo + stride;
        const uint64_t a = x[lo], b = x[hi];
        if ((a < b) == ((lo & block) == 0)) {
          x[lo] = b;
          x[hi] = a;
        }
      }
      // a warp's pairs of a stride up to 32 lie in 64 entries that only this warp touches until the next longer stride
      if (stride > 32 || (stride == 1 && block >= 64)) __syncthreads(); else __syncwarp();
    }
  __syncthreads();
}

// Adds the marked logits of vector v (a lane's bits) to the warp's list, in order; n: how many it has, or would have.
template <int kElems>
__device__ __forceinline__ void list_marked(Shared& sh, int& n, uint32_t marked, int v) {
  const int lane = threadIdx.x & 31, c = __popc(marked);
  int incl = c;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += u;
  }
  int at = n + incl - c;
  n += __shfl_sync(0xFFFFFFFFu, incl, 31);
  if (n <= kListPerWarp)
    for (uint32_t m = marked; m != 0; m &= m - 1) sh.list[threadIdx.x >> 5][at++] = static_cast<uint16_t>(v * kElems + __ffs(m) - 1);
}

// The logits of one step, exchanged over the cluster and ranked: the boundary by count or weight, given the sums
// above the step, and how many logits the warp has listed among which they are (-1: none).
template <int DT, bool kByWeight>
__device__ __noinline__ Boundary rank_step(const Slice<DT>& s, Shared& sh, float bound, const Scale& scale, int step, uint64_t want,
                              uint32_t above_c, uint64_t above_w, float top, float steep, int listed) {
  const uint32_t cs = cluster_size(), rank = cluster_rank();
  const int tid = threadIdx.x;
  if (tid == 0) sh.mine_n = 0;
  __syncthreads();
  const float hi = scale.above(step), lo = fmaxf(scale.below(step), bound);
  auto exchange = [&](float x) {
    if (x >= lo && x <= hi && x != -INFINITY && scale.step(x) == step) sh.mine[atomicAdd(&sh.mine_n, 1u)] = key_of(x);
  };
#pragma unroll 1
  for (int i = tid & 31; i < listed; i += 32) exchange(s.at(sh.list[tid >> 5][i]));
  if (listed < 0)
#pragma unroll 2
  for (int v = s.run_a + (tid & 31); v < s.run_z; v += 32) {
    const Vec<DT> x(s.vec(v));
#pragma unroll
    for (int e = 0; e < Vec<DT>::kElems; ++e) exchange(x.x[e]);
  }
  cluster_sync();
  if (tid < 32) {
    uint32_t n = tid > 0 && tid <= static_cast<int>(cs) ? peer_u32(&sh.mine_n, tid - 1) : 0;
#pragma unroll
    for (int d = 1; d <= kMaxCluster; d <<= 1) {
      const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, n, d);
      if (tid >= d) n += u;
    }
    if (tid <= kMaxCluster) sh.from[tid] = n;  // (the same from cs on)
  }
  __syncthreads();
  const int n = static_cast<int>(sh.from[cs]);
  uint32_t key[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = tid + j * kThreads;
    key[j] = 0;  // (a logit's image is never 0)
    if (i < n) {
      uint32_t r = 0;
      while (sh.from[r + 1] <= static_cast<uint32_t>(i)) ++r;
      key[j] = peer_u32(&sh.mine[i - sh.from[r]], r);
    }
    sh.all_w[i] = key[j];
  }
  __syncthreads();
  int size = 32;
  while (size < n) size *= 2;
  sort_descending(sh.all_w, size);
  // thread t has the 2t-th largest and the next; runs of equals are one boundary
  uint32_t mine[2];
  uint64_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    mine[j] = static_cast<uint32_t>(sh.all_w[2 * tid + j]);
    w[j] = mine[j] != 0 ? weight_of(exponent_of(logit_of_key(mine[j]), top, steep)) : 0;
  }
  uint64_t at[2];
  at[0] = above_w + block_scan(sh, w[0] + w[1]);
  at[1] = at[0] + w[0];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (mine[j] != 0 && (kByWeight ? at[j] < want && at[j] + w[j] >= want : above_c + 2 * tid + j + 1 == want)) sh.key = mine[j];
  __syncthreads();
  Boundary b;
  b.key = sh.key;
  b.equal_c = b.equal_before = b.equal_here = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = 2 * tid + j;
    if (mine[j] == b.key && (i == 0 || static_cast<uint32_t>(sh.all_w[i - 1]) != b.key)) {
      sh.key_above_c = above_c + i;
      sh.key_above_w = at[j];
    }
    const int own = tid + j * kThreads;
    const bool equal = key[j] == b.key;
    b.equal_c += __syncthreads_count(equal);
    b.equal_before += __syncthreads_count(equal && own < static_cast<int>(sh.from[rank]));
    b.equal_here += __syncthreads_count(equal && own >= static_cast<int>(sh.from[rank]) && own < static_cast<int>(sh.from[rank + 1]));
  }
  b.above_c = sh.key_above_c;
  b.above_w = sh.key_above_w;
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
  return peers_sum(&sh.z);
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

// The row's parameters; SV_DEV_* bits of those that are out of range.
__device__ __forceinline__ uint32_t read_ask(const SampleParams& p, int64_t row, Ask& ask) {
  const float T = p.temperature[row];
  const int k_in = p.top_k != nullptr ? p.top_k[row] : 0;
  const float p_in = p.top_p != nullptr ? p.top_p[row] : 1.0f;
  const float q_in = p.min_p != nullptr ? p.min_p[row] : 0.0f;
  uint32_t bad = 0;
  if (!(T >= 0.0f) || T == INFINITY) bad |= SV_DEV_BAD_TEMPERATURE;
  if (k_in < 0 || !(p_in > 0.0f && p_in <= 1.0f) || !(q_in >= 0.0f && q_in <= 1.0f)) bad |= SV_DEV_BAD_FILTER;
  const bool greedy = T == 0.0f;
  ask.row = row;
  ask.total = 0;
  ask.steep = greedy ? 1.0f : fminf(__fdiv_rn(1.44269504088896341f, T), FLT_MAX);
  ask.k = greedy ? 1 : (k_in == 0 ? p.V : k_in);
  ask.by_count = ask.k < p.V;
  ask.nucleus = !greedy && p_in < 1.0f;
  ask.floor_on = !greedy && q_in > 0.0f;
  ask.least = ask.floor_on ? log2f(q_in) : -INFINITY;  // of y
  ask.p24 = static_cast<uint32_t>(rintf(p_in * 16777216.0f));
  return bad;
}
// Rows for maxima_kernel and select_kernel: their prefix's end follows from few logits (and W, which top-p alone needs).
__device__ __forceinline__ bool by_maxima(const Ask& ask, uint32_t bad) {
  return bad == 0 && (ask.by_count ? ask.k <= kGatherK : ask.floor_on);
}
// Top-p alone: V weights below this logit (and half a unit of rounding each) stay below (1 - p) W; 1e-3 covers ex2 and
// log2.
__device__ __forceinline__ float nucleus_bound(const Ask& ask, int V) {
  const float each = static_cast<float>(ask.total) * (static_cast<float>((1u << 24) - ask.p24) * 0x1p-24f) / static_cast<float>(V) - 0.5f;
  return each > 0.0f ? __fadd_rd(ask.top, __fdiv_rd(log2f(each) - 40.0f - 1e-3f, ask.steep)) : -INFINITY;
}

// Min-p: no logit below this one reaches the threshold.  An exponent is rounded twice (a part in 2^23), and one that
// underflows to a multiple of 2^-149: at q = 1 all those that round to -0 reach 0.
__device__ __forceinline__ float floor_bound(const Ask& ask) {
  return __fadd_rd(ask.top, __fdiv_rd(__fmaf_rd(ask.least, 1.000001f, -0x1p-148f), ask.steep));
}

__device__ __forceinline__ Scale scale_of(const Ask& ask) {
  return Scale::over(ask.top, ask.bound == -INFINITY ? 64.0f / ask.steep : __fsub_rn(ask.top, ask.bound));
}

// Up to 128 KB of shared memory is on its way at once: waits of microseconds, not inlined.
__device__ __noinline__ void wait_piece(uint64_t* bar, uint32_t parity, uint32_t* status) { mbar_wait(bar, parity, status); }

// Step 3 for at most kShort gathered logits: thread t has the t-th, counts those before it in the order, and adds
// their weights.
template <int DT>
__device__ __noinline__ void finish_short(Shared& sh, const Ask& ask, int n, uint64_t* weights) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t g = 0, w = 0;
  float y = -INFINITY;
  if (tid < n) {
    g = sh.gather[tid];
    y = exponent_of(logit_of_key(static_cast<uint32_t>(g >> 32)), ask.top, ask.steep);
    w = weight_of(y);
    weights[tid] = w;
  }
  __syncthreads();
  uint32_t more = 0;
  uint64_t above = 0;
  if (warp * 32 < n)
#pragma unroll 4
    for (int i = 0; i < n; ++i)
      if (sh.gather[i] > g) {
        ++more;
        above += weights[i];
      }
  const bool in_k = tid < n && (!ask.by_count || more < static_cast<uint32_t>(ask.k));
  uint64_t total = ask.total;
  if (ask.by_count && ask.nucleus) {  // the top-k's weight
    const uint64_t part = warp_sum(in_k ? w : 0);
    if (lane == 0) sh.scan_w[warp] = part;
    __syncthreads();
    total = 0;
    for (int i = 0; i < kShort / 32; ++i) total += sh.scan_w[i];
  }
  const bool keep = in_k && (!ask.nucleus || above < max(share_of(total, ask.p24), uint64_t(1))) && y >= ask.least;
  if (keep && ask.out_row != nullptr) {
    using Elem = typename Slice<DT>::Elem;
    const uint32_t bits = __float_as_uint(logit_of_key(static_cast<uint32_t>(g >> 32)));
    static_cast<Elem*>(ask.out_row)[~static_cast<uint32_t>(g)] = DT == SV_BF16 ? static_cast<Elem>(bits >> 16) : static_cast<Elem>(bits);
  }
  if (!keep) w = 0;
  // draws: the list is in vocabulary order
  uint64_t incl = w;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += u;
  }
  if (lane == 31) sh.seg[warp] = incl;
  __syncthreads();
  uint64_t before = incl - w, z = 0;
  for (int i = 0; i < kShort / 32; ++i) {
    if (i < warp) before += sh.seg[i];
    z += sh.seg[i];
  }
  const SampleParams& p = *ask.p;
  if (w != 0)
    for (int j = 0; j < p.M; ++j) {
      const uint64_t t = share_of(z, static_cast<uint32_t>(p.uniforms[ask.row * p.M + j] * 16777216.0f));
      if (t >= before && t < before + w) {
        p.out_tokens[ask.row * p.M + j] = static_cast<int32_t>(~static_cast<uint32_t>(g));
        if (p.out_probs != nullptr) p.out_probs[ask.row * p.M + j] = __fdiv_rn(__ull2float_rn(w), __ull2float_rn(z));
      }
    }
}

// Among the gathered logits of one histogram step: the entry up to which the prefix goes, by count (the want-th
// of all) or by weight (the one that makes the weight reach want), and the weight up to it inclusive; `few` has room
// for kShort, `weights` for all.
struct End {
  uint64_t entry, weight;
};
template <bool kByWeight>
__device__ __noinline__ End end_in_step(Shared& sh, const Ask& ask, const Scale& scale, int n, uint64_t want, uint64_t* sorted) {
  const int tid = threadIdx.x;
  const uint32_t step = sh.step;
  const uint32_t here = sh.here_c, above_c = sh.above_c;
  const uint64_t above_w = sh.above_w;
  __syncthreads();
  auto weight = [&](uint64_t g) { return weight_of(exponent_of(logit_of_key(static_cast<uint32_t>(g >> 32)), ask.top, ask.steep)); };
  if (here > kShort) {  // many equals: sort everything (rare)
    int size = 32;
    while (size < n) size *= 2;
    for (int i = tid; i < size; i += kThreads) sorted[i] = i < n ? sh.gather[i] : 0;
    __syncthreads();
    sort_descending(sorted, size);
    const int per = (n + kThreads - 1) / kThreads, a = min(n, tid * per), b = min(n, a + per);
    uint64_t sum = 0;
    for (int i = a; i < b; ++i) sum += weight(sorted[i]);
    uint64_t at = block_scan(sh, sum);
    for (int i = a; i < b; ++i) {
      const uint64_t w = weight(sorted[i]);
      if (kByWeight ? at < want && at + w >= want : i + 1 == static_cast<int>(want)) {
        sh.end[0] = sorted[i];
        sh.end[1] = at + w;
      }
      at += w;
    }
    __syncthreads();
  } else {
    if (tid == 0) sh.mine_n = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t g = sh.gather[i];
      if (scale.step(logit_of_key(static_cast<uint32_t>(g >> 32))) == static_cast<int>(step)) sorted[atomicAdd(&sh.mine_n, 1u)] = g;
    }
    __syncthreads();
    if (tid < static_cast<int>(here)) {
      const uint64_t g = sorted[tid], w = weight(g);
      uint32_t more = above_c;
      uint64_t at = above_w;
      for (uint32_t i = 0; i < here; ++i)
        if (sorted[i] > g) {
          ++more;
          at += weight(sorted[i]);
        }
      if (kByWeight ? at < want && at + w >= want : more + 1 == want) {
        sh.end[0] = g;
        sh.end[1] = at + w;
      }
    }
    __syncthreads();
  }
  const End end = {sh.end[0], sh.end[1]};
  __syncthreads();
  return end;
}

// Step 3 in the cluster's first CTA, which holds the n > kShort gathered logits in vocabulary order (the histogram's limbs
// and the ends lie in `more`, and so does room for sorting).
template <int DT>
__device__ __noinline__ void finish_gathered(Shared& sh, const Ask& ask, int n, uint64_t* more) {
  const int tid = threadIdx.x;
  uint32_t* limb = reinterpret_cast<uint32_t*>(more + kGather);  // [3][kSteps]
  const Scale scale = scale_of(ask);
  uint64_t last = 0;
  if (ask.by_count || ask.nucleus) {
    sh.count[tid] = 0;
    for (int l = 0; l < 3; ++l) limb[l * kSteps + tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const float x = logit_of_key(static_cast<uint32_t>(sh.gather[i] >> 32));
      const int step = scale.step(x);
      const uint64_t w = weight_of(exponent_of(x, ask.top, ask.steep));
      atomicAdd(&sh.count[step], 1u);
      for (int l = 0; l < 3; ++l) {
        const uint32_t part = static_cast<uint32_t>(w >> (l * kLimb)) & ((1u << kLimb) - 1u);
        if (part) atomicAdd(&limb[l * kSteps + step], part);
      }
    }
    __syncthreads();
    const uint32_t c = sh.count[tid];
    const uint64_t w = limbs_of(limb[tid], limb[kSteps + tid], limb[2 * kSteps + tid]);
    uint64_t total = ask.total;
    if (ask.by_count) {
      find_step<false>(sh, c, w, ask.k, 0, 0);
      if (sh.step != 0xFFFFFFFFu) {
        const End end = end_in_step<false>(sh, ask, scale, n, ask.k, more);
        last = end.entry;
        total = end.weight;
      } else {  // fewer than k logits: all are kept
        __syncthreads();
        const uint64_t before = block_scan(sh, w);
        if (tid == kThreads - 1) sh.z = before + w;
        __syncthreads();
        total = sh.z;
      }
    }
    if (ask.nucleus) {
      const uint64_t limit = max(share_of(total, ask.p24), uint64_t(1));
      find_step<true>(sh, c, w, limit, 0, 0);
      if (sh.step != 0xFFFFFFFFu) last = max(last, end_in_step<true>(sh, ask, scale, n, limit, more).entry);
    }
  }
  // the kept logits are those at or above `last` and min-p's threshold; thread t has a run of the list
  const int per = (n + kThreads - 1) / kThreads;
  const int a = min(n, tid * per), b = min(n, a + per);
  auto weight = [&](int i) {
    const uint64_t g = sh.gather[i];
    const float y = exponent_of(logit_of_key(static_cast<uint32_t>(g >> 32)), ask.top, ask.steep);
    return g >= last && y >= ask.least ? weight_of(y) : 0;
  };
  uint64_t sum = 0;
  for (int i = a; i < b; ++i) {
    sum += weight(i);
    if (ask.out_row != nullptr) {  // the first CTA's part begins the row
      const uint64_t g = sh.gather[i];
      const float x = logit_of_key(static_cast<uint32_t>(g >> 32));
      using Elem = typename Slice<DT>::Elem;
      if (g >= last && exponent_of(x, ask.top, ask.steep) >= ask.least)
        static_cast<Elem*>(ask.out_row)[~static_cast<uint32_t>(g)] =
            DT == SV_BF16 ? static_cast<Elem>(__float_as_uint(x) >> 16) : static_cast<Elem>(__float_as_uint(x));
    }
  }
  const uint64_t before = block_scan(sh, sum);
  if (tid == kThreads - 1) sh.z = before + sum;
  __syncthreads();
  const uint64_t z = sh.z;
  const SampleParams& p = *ask.p;
  for (int j = 0; j < p.M; ++j) {
    const uint64_t t = share_of(z, static_cast<uint32_t>(p.uniforms[ask.row * p.M + j] * 16777216.0f));
    if (t < before || t >= before + sum) continue;
    uint64_t at = before;
    for (int i = a; i < b; ++i) {
      const uint64_t w = weight(i);
      if (t < at + w) {
        p.out_tokens[ask.row * p.M + j] = static_cast<int32_t>(~static_cast<uint32_t>(sh.gather[i]));
        if (p.out_probs != nullptr) p.out_probs[ask.row * p.M + j] = __fdiv_rn(__ull2float_rn(w), __ull2float_rn(z));
        break;
      }
      at += w;
    }
  }
}

// Kept weights, the row's total, the draws and the kept logits, with every slice where it is.  A logit is kept if it lies
// above the boundary, or equals it and has an index below `cut`.  A lane sums a
// contiguous stretch of its warp's run (an odd number of vectors, so that a quarter warp's 16-byte loads fall on
// different banks): a draw then looks into one lane's stretch.
template <int DT, bool kAll>
__device__ __noinline__ void draw_slices(const Slice<DT>& s, Shared& sh, const Ask& ask, uint32_t boundary, uint32_t cut) {
  using Elem = typename Slice<DT>::Elem;
  constexpr int kElems = Slice<DT>::kElems;
  const SampleParams& p = *ask.p;
  const uint32_t cs = cluster_size(), rank = cluster_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int stretch = (s.run_z - s.run_a + 31) / 32 | 1;
  const int va = min(s.run_z, s.run_a + lane * stretch), vz = min(s.run_z, va + stretch);
  const float last = kAll || boundary == 0 ? -INFINITY : logit_of_key(boundary);
  // (logits compare as their images do: -0 and +0 are one value in both)
  auto kept = [&](float x, int pos) {
    return kAll || x > last || (x == last && x != -INFINITY && static_cast<uint32_t>(s.index_of(pos)) < cut) ? x : -INFINITY;
  };
  // the cut row: a warp's vectors side by side, those without a kept logit left as they are
  if (Elem* out_row = static_cast<Elem*>(ask.out_row); out_row != nullptr) {
    const bool aligned = ((reinterpret_cast<uintptr_t>(out_row) - s.phase * sizeof(Elem)) & 15u) == 0;
#pragma unroll 1
    for (int v = s.run_a + lane; v < s.run_z; v += 32) {
      uint4 w = s.vec(v);
      const Vec<DT> x(w);
      Elem* raw = reinterpret_cast<Elem*>(&w);
      uint32_t keep = 0;
#pragma unroll
      for (int e = 0; e < kElems; ++e) keep |= (kept(x.x[e], v * kElems + e) != -INFINITY ? 1u : 0u) << e;
      if (keep == 0) continue;
      const int at = v * kElems - s.phase;
      if (aligned && at >= 0 && at + kElems <= s.n) {
#pragma unroll
        for (int e = 0; e < kElems; ++e)
          if (!((keep >> e) & 1u)) raw[e] = DT == SV_BF16 ? static_cast<Elem>(0xFF80u) : static_cast<Elem>(0xFF800000u);
        *reinterpret_cast<uint4*>(out_row + at) = w;
      } else {
#pragma unroll
        for (int e = 0; e < kElems; ++e)
          if ((keep >> e) & 1u) out_row[at + e] = raw[e];
      }
    }
  }
  WeightSum sum(ask.top, ask.steep);
  uint32_t adds = 0;
#pragma unroll 2
  for (int v = va; v < vz; ++v, ++adds) {
    const Vec<DT> x(s.vec(v));
#pragma unroll
    for (int e = 0; e < kElems; e += 2) {
      const float x0 = kept(x.x[e], v * kElems + e), x1 = kept(x.x[e + 1], v * kElems + e + 1);
      sum.add(x0, x1);
    }
  }
  const uint64_t w = sum.total(adds * (kElems / 2));
  uint64_t incl = w;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += u;
  }
  __syncthreads();  // (no peer still reads sh.z: a cluster barrier lies between cluster_total and here)
  if (lane == 31) sh.seg[warp] = incl;
  __syncthreads();
  if (tid == 0) {
    uint64_t z = 0;
    for (int i = 0; i < kWarps; ++i) z += sh.seg[i];
    sh.z = z;
  }
  cluster_sync();
  const uint32_t peer = lane % kMaxCluster;
  const uint64_t zr = peer < cs ? peer_u64(&sh.z, peer) : 0;
  uint64_t z = zr, before = peer < rank ? zr : 0;
#pragma unroll
  for (int d = kMaxCluster / 2; d > 0; d >>= 1) {
    z += __shfl_xor_sync(0xFFFFFFFFu, z, d);
    before += __shfl_xor_sync(0xFFFFFFFFu, before, d);
  }
  cluster_arrive();  // this CTA has read its peers' sums
  for (int i = 0; i < warp; ++i) before += sh.seg[i];
  for (int j = 0; j < p.M; ++j) {
    const uint64_t t0 = share_of(z, static_cast<uint32_t>(p.uniforms[ask.row * p.M + j] * 16777216.0f));
    if (t0 < before || t0 >= before + sh.seg[warp]) continue;
    const uint64_t t = t0 - before;
    const uint32_t owner = __ballot_sync(0xFFFFFFFFu, t >= incl - w && t < incl);
    const int from = __ffs(owner) - 1;
    uint64_t left = t - __shfl_sync(0xFFFFFFFFu, incl - w, from);
    const int first = (s.run_a + from * stretch) * kElems, end = min(s.run_z, s.run_a + (from + 1) * stretch) * kElems;
    for (int base = first; base < end; base += 32) {
      const int pos = base + lane;
      const uint64_t we = pos < end ? weight_of(exponent_of(kept(s.at(pos), pos), ask.top, ask.steep)) : 0;
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
  cluster_wait();  // no CTA leaves while a peer may still read its shared memory
}

// The cluster's exact weight of the steps before `step` - 1, and of `step` - 1, `step` and `step` + 1 (turn: 0 and 1 in
// turn, so a call's sums are not written while a peer reads the call's before).  Returns how many
// logits the warp has listed that may lie in these three, or -1 for too many.
template <int DT>
__device__ __noinline__ int weights_around(const Slice<DT>& s, Shared& sh, const Ask& ask, const Scale& scale, int step,
                                           uint32_t turn, uint64_t (&out)[4]) {
  constexpr int kElems = Vec<DT>::kElems;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // surely above: the packed sum; surely below: nothing; the few between are listed and weighed by their step (in
  // registers: atomics on four addresses would queue up)
  const float hi = scale.above(step - 1), lo = fmaxf(scale.below(step + 1), ask.bound);
  WeightSum sum(ask.top, ask.steep);
  uint32_t adds = 0;
  int n = 0;
#pragma unroll 2
  for (int vb = s.run_a; vb < s.run_z; vb += 32) {
    const int v = vb + lane;
    uint32_t between = 0;
    if (v < s.run_z) {
      const Vec<DT> x(s.vec(v));
#pragma unroll
      for (int e = 0; e < kElems; e += 2) {
        sum.add(x.x[e] > hi ? x.x[e] : -INFINITY, x.x[e + 1] > hi ? x.x[e + 1] : -INFINITY);
        between |= (x.x[e] >= lo && x.x[e] <= hi ? 1u : 0u) << e | (x.x[e + 1] >= lo && x.x[e + 1] <= hi ? 2u : 0u) << e;
      }
      ++adds;
    }
    if (__any_sync(0xFFFFFFFFu, between != 0)) list_marked<kElems>(sh, n, between, v);
  }
  uint64_t part[4] = {0, 0, 0, 0};
  auto weigh = [&](float x) {
    const int d = scale.step(x) - step + 1;
    const uint64_t w = weight_of(exponent_of(x, ask.top, ask.steep));  // (0 for -inf)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[i] += (i == 0 ? d < 0 : d == i - 1) ? w : 0;
  };
  __syncwarp();
  if (n <= kListPerWarp) {
#pragma unroll 1
    for (int i = lane; i < n; i += 32) weigh(s.at(sh.list[warp][i]));
  } else {
#pragma unroll 1
    for (int pos = s.run_a * kElems + lane; pos < s.run_z * kElems; pos += 32) {
      const float x = s.at(pos);
      if (x >= lo && x <= hi) weigh(x);
    }
  }
  const uint64_t high = warp_sum(sum.total(adds * (Vec<DT>::kElems / 2)));
  uint64_t* sums_at = sh.all_w + (turn & 1) * 4 * (kWarps + 1);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t t = warp_sum(part[i]) + (i == 0 ? high : 0);
    if (lane == 0) sums_at[4 * warp + i] = t;
  }
  __syncthreads();
  if (tid < 4) {
    uint64_t t = 0;
    for (int w = 0; w < kWarps; ++w) t += sums_at[4 * w + tid];
    sums_at[4 * kWarps + tid] = t;
  }
  cluster_sync();
  static_assert(4 * kMaxCluster == 32, "a lane per CTA and value");
  uint64_t sums = peers_sum(&sums_at[4 * kWarps + lane / kMaxCluster]);
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = __shfl_sync(0xFFFFFFFFu, sums, i * kMaxCluster);
  return n <= kListPerWarp ? n : -1;
}

// The image of the smallest logit whose exponent reaches `least` (<= 0): min-p's threshold, exactly.
__device__ __noinline__ uint32_t floor_key(float top, float steep, float least) {
  uint32_t lo = key_of(-INFINITY), hi = key_of(top);  // lo does not reach it, hi does
  while (hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (exponent_of(logit_of_key(mid), top, steep) >= least) hi = mid; else lo = mid;
  }
  return hi;
}

// The cluster's counts of the logits at or above the bound: thread t's step.
template <int DT>
__device__ __noinline__ uint32_t count_steps(const Slice<DT>& s, Shared& sh, const Ask& ask) {
  const Scale scale = scale_of(ask);
  const float bound = ask.bound;
  sh.count[threadIdx.x] = 0;
  __syncthreads();
#pragma unroll 2
  for (int v = s.run_a + (threadIdx.x & 31); v < s.run_z; v += 32) {
    const Vec<DT> x(s.vec(v));
#pragma unroll
    for (int e = 0; e < Vec<DT>::kElems; ++e)
      if (x.x[e] >= bound && x.x[e] != -INFINITY) atomicAdd(&sh.count[scale.step(x.x[e])], 1u);
  }
  cluster_sync();
  uint32_t c;
  uint64_t none;
  merged_step(sh, threadIdx.x, false, &c, &none);
  return c;
}

// Step 3 for long lists; c: this thread's step of the histogram.
template <int DT>
__device__ __noinline__ void cut_wide(const Slice<DT>& s, Shared& sh, const Ask& ask, uint32_t c) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float top = ask.top, steep = ask.steep, bound = ask.bound;
  uint64_t total = ask.total;
  Boundary b = {};
  uint32_t ties_kept = 0;  // how many of the boundary's equals are kept, lowest indexes first
  if (ask.by_count || ask.nucleus) {
    const Scale scale = scale_of(ask);
    // a step's weight by its middle, in units of 2^-30: good to a part in a few hundred
    const float middle = scale.inv > 0.0f ? -(tid + 0.5f) / scale.inv * steep : 0.0f;
    const uint64_t about = static_cast<uint64_t>(static_cast<float>(c) * ex2_approx(middle) * 0x1p30f);
    uint64_t near[4];
    int listed = -1;
    bool by_radix = false;
    if (ask.by_count) {
      find_step<false>(sh, c, 0, ask.k, 0, 0);
      const uint32_t step = sh.step, here = sh.here_c, above_c = sh.above_c;
      cluster_sync();  // the peers have read the histogram
      if (step != 0xFFFFFFFFu) {
        by_radix = here > kExchange;
        uint64_t above_w = 0;
        if (ask.nucleus) {
          listed = weights_around<DT>(s, sh, ask, scale, step, 0, near);
          above_w = near[0] + near[1];
        }
        if (by_radix) b = descend<DT, false>(s, sh, ask.k, top, steep);
        else b = rank_step<DT, false>(s, sh, bound, scale, step, ask.k, above_c, above_w, top, steep, listed);
        ties_kept = ask.k - b.above_c;
      }  // else fewer than k logits: all are kept
      if (ask.nucleus) {  // W: what lies above the boundary, and its kept equals
        if (step != 0xFFFFFFFFu && !by_radix) {
          total = b.above_w;
        } else {
          total = cluster_total(sh, weights_above<DT>(s, b.key == 0 ? -INFINITY : logit_of_key(b.key), top, steep));
        }
        if (step != 0xFFFFFFFFu) total += static_cast<uint64_t>(ties_kept) * weight_of(exponent_of(logit_of_key(b.key), top, steep));
      }
    }
    if (ask.nucleus) {
      const uint64_t limit = max(share_of(total, ask.p24), uint64_t(1));
      if (by_radix) cluster_sync();  // the peers have read the last histogram (else weights_around's barrier sees to it)
      // The step whose weight makes the sum reach the limit, about; it is weighed with its neighbours, exactly, and if it
      // is not one of them, the estimate is set right there and another step chosen (few heavy logits make it that far
      // off).
      const uint64_t ahead = by_radix ? 0 : block_scan(sh, about);
      uint64_t want = max(limit >> 10, uint64_t(1));
      bool inside = false, all = false;
      uint64_t above_w = 0;
      int step = kSteps - 1;
#pragma unroll 1
      for (int tries = 0; tries < kTries && !by_radix && !inside && !all; ++tries) {
        const int last = step;
        const bool below = tries > 0 && near[0] >= limit;  // the boundary lies before the weighed steps
        if (tid == 0) sh.step = kSteps - 1;
        __syncthreads();
        if (ahead < want && ahead + about >= want) sh.step = tid;
        __syncthreads();
        step = sh.step;
        if (tries > 0) step = below ? min(step, last - 3) : max(step, last + 3);
        step = max(0, min(step, kSteps - 1));
        listed = weights_around<DT>(s, sh, ask, scale, step, tries, near);
        above_w = near[0];
        int in = step - 1;
        for (int i = 1; i < 4 && !inside; ++i) {
          if (above_w < limit && above_w + near[i] >= limit) inside = true;
          else {
            above_w += near[i];
            ++in;
          }
        }
        // a bound at min-p's threshold may lie above the boundary: then everything above the bound is kept (and so it is
        // where the descent finds the boundary below the bound)
        all = !inside && step == kSteps - 1 && above_w < limit;
        if (tid == max(step - 1, 0)) sh.above_w = ahead;
        __syncthreads();
        want = max(static_cast<int64_t>((limit >> 10) + sh.above_w - (near[0] >> 10)), int64_t(1));
        if (inside) step = in;
      }
      uint32_t here = 0;
      if (inside) {
        // how many logits the step holds, from the thread that has it
        if (tid == step) sh.here_c = c;
        __syncthreads();
        here = sh.here_c;
      }
      if (inside && here <= kExchange) b = rank_step<DT, true>(s, sh, bound, scale, step, limit, 0, above_w, top, steep, listed);
      else if (!all) b = descend<DT, true>(s, sh, limit, top, steep);
      if (b.key != 0) {
        const uint64_t each = weight_of(exponent_of(logit_of_key(b.key), top, steep));
        ties_kept = each == 0 ? 0 : static_cast<uint32_t>((limit - b.above_w + each - 1) / each);
      }
    }
  }
  // equals of this slice that are kept: those before vocabulary index `cut`
  uint32_t cut = 0xFFFFFFFFu;
  const uint32_t quota = ties_kept > b.equal_before ? min(ties_kept - b.equal_before, b.equal_here) : 0;
  if (b.key == 0 || quota == 0) {
    cut = 0;
  } else if (quota < b.equal_here) {
    const float last = logit_of_key(b.key);
    uint32_t c = 0;
#pragma unroll 2
    for (int v = s.run_a + lane; v < s.run_z; v += 32) {
      const Vec<DT> x(s.vec(v));
#pragma unroll
      for (int e = 0; e < Vec<DT>::kElems; ++e) c += x.x[e] == last;
    }
    c = __reduce_add_sync(0xFFFFFFFFu, c);
    if (lane == 0) sh.ties[warp] = c;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < warp; ++i) before += sh.ties[i];
    if (before < quota && before + c >= quota)
      for (int vb = s.run_a; vb < s.run_z && before < quota; vb += 32) {
        uint32_t mask = 0;
        if (vb + lane < s.run_z) {
          const Vec<DT> x(s.vec(vb + lane));
#pragma unroll
          for (int e = 0; e < Vec<DT>::kElems; ++e) mask |= (x.x[e] == last ? 1u : 0u) << e;
        }
        uint32_t incl = __popc(mask);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
          if (lane >= d) incl += u;
        }
        const uint32_t excl = incl - __popc(mask);
        if (before + excl < quota && before + incl >= quota) {
          for (uint32_t left = quota - before - excl; left > 1; --left) mask &= mask - 1;
          sh.cut = static_cast<uint32_t>(s.index_of((vb + lane) * Vec<DT>::kElems + __ffs(mask) - 1)) + 1;
        }
        before += __shfl_sync(0xFFFFFFFFu, incl, 31);
      }
    __syncthreads();
    cut = sh.cut;
  }
  // min-p as a boundary of its own: everything above the logit just below its threshold
  uint32_t last = b.key;
  if (ask.floor_on) {
    const uint32_t under = floor_key(top, steep, ask.least) - 1;
    if (under > last) {
      last = under;
      cut = 0;
    }
  }
  draw_slices<DT, false>(s, sh, ask, last, cut);
}

// One row by the cluster; `parity` of the copies' barriers.
template <int DT>
__device__ __forceinline__ void sample_row(const SampleParams& p, int64_t row, unsigned char* dyn, Shared& sh, uint32_t parity) {
  using Elem = typename Slice<DT>::Elem;
  constexpr int kElems = Vec<DT>::kElems;
  const uint32_t cs = cluster_size(), rank = cluster_rank();
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
  sh.count[tid] = 0;
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
  uint32_t bad = read_ask(p, row, ask);
  ask.p = &sh.params;
  bool bad_uniform = false;
  for (int j = tid; j < p.M; j += kThreads) {
    const float u = p.uniforms[row * p.M + j];
    bad_uniform |= !(u >= 0.0f && u < 1.0f);
  }
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
      for (int i = 0; i < kPieces; ++i) wait_piece(&sh.bar[i], parity, p.status);
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
    if (a < s.run_z && min(v1, a + per_piece) > s.run_a) wait_piece(&sh.bar[i], parity, p.status);
  }
  float group = -INFINITY;
#pragma unroll 4
  for (int v = s.run_a + lane; v < s.run_z; v += 32) {
    const Vec<DT> x(s.vec(v));
#pragma unroll
    for (int e = 0; e < kElems; ++e) group = max_nan(group, x.x[e]);
  }
  // reductions on integer images (a NaN's lies above that of +inf)
  const uint32_t none_key = key_of(-INFINITY), inf_key = key_of(INFINITY);
  {
    const uint32_t key = key_of(group);
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, key);
    const uint32_t lo = __reduce_min_sync(0xFFFFFFFFu, key > none_key ? key : 0xFFFFFFFFu);
    if (lane == 0) {
      sh.red[0][warp] = hi;
      sh.red[1][warp] = lo;
    }
  }
  __syncthreads();
  const uint32_t top_key = __reduce_max_sync(0xFFFFFFFFu, sh.red[0][lane & (kWarps - 1)]);
  const uint32_t low_key = __reduce_min_sync(0xFFFFFFFFu, sh.red[1][lane & (kWarps - 1)]);
  if (tid == 0) sh.top = top_key;
  // ---- 1. a bound ---------------------------------------------------------------------------------
  // the CTA vouches for rank_n[j] logits at or above rank_at[j]: from an even share of k to all of it
  if (ask.by_count && ask.k > 1) {  // (one: the largest is the bound)
    if (tid < kRanks) {
      sh.rank_at[tid] = -INFINITY;
      sh.rank_n[tid] = static_cast<uint32_t>(ceilf(static_cast<float>(ask.k) * exp2f(-3.0f + 3.0f * tid / (kRanks - 1))));
    }
    if (tid == 0) sh.bound = 0;
    const float own = logit_of_key(top_key);
    const bool counts = top_key < inf_key && low_key != 0xFFFFFFFFu;
    const float range = counts ? __fsub_rn(own, logit_of_key(low_key)) : 0.0f;
    const Scale groups = Scale::over(own, range);
    if (counts && group > -INFINITY) atomicAdd(&sh.count[groups.step(group)], 1u);
    __syncthreads();
    const uint32_t c = sh.count[tid];
    const uint32_t before = block_scan32(sh, c);
    if (c > 0) {
      const float at = groups.lower_end(tid, range);
#pragma unroll 1
      for (int j = 0; j < kRanks; ++j) {
        const uint32_t want = sh.rank_n[j];
        if (before < want && before + c >= want) sh.rank_at[j] = at;
      }
    }
  }
  cluster_sync();
  const uint32_t row_top = __reduce_max_sync(0xFFFFFFFFu, lane < static_cast<int>(cs) ? peer_u32(&sh.top, lane) : 0u);
  const float top = logit_of_key(row_top);
  ask.top = top;
  if (row_top >= inf_key) bad |= SV_DEV_BAD_LOGIT;
  if (bad != 0 || row_top <= none_key) {  // the same in every CTA of the cluster
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
    draw_slices<DT, true>(s, sh, ask, 0, 0);
    return;
  }
  float bound = -INFINITY;
  if (ask.by_count && ask.k == 1) {
    bound = top;
  } else if (ask.by_count) {
    // the largest published logit above which the CTAs together vouch for k: thread t asks CTA t % 8 about the
    // (t / 8)-th published one
    if (tid < kMaxCluster * kRanks)
      sh.rank_all[tid] = tid < static_cast<int>(cs) * kRanks ? peer_f32(&sh.rank_at[tid % kRanks], tid / kRanks) : -INFINITY;
    __syncthreads();
    const float at = sh.rank_all[tid / kMaxCluster];
    uint32_t sure = 0;
#pragma unroll 1
    for (int j = 0; j < kRanks; ++j)
      if (sh.rank_all[(tid % kMaxCluster) * kRanks + j] >= at) sure = sh.rank_n[j];
    sure += __shfl_xor_sync(0xFFFFFFFFu, sure, 1);
    sure += __shfl_xor_sync(0xFFFFFFFFu, sure, 2);
    sure += __shfl_xor_sync(0xFFFFFFFFu, sure, 4);
    const uint32_t good = __reduce_max_sync(0xFFFFFFFFu, at > -INFINITY && sure >= static_cast<uint32_t>(ask.k) ? key_of(at) : 0u);
    if (lane == 0 && good != 0) atomicMax(&sh.bound, good);
    __syncthreads();
    if (sh.bound != 0) bound = logit_of_key(sh.bound);
  } else if (ask.nucleus) {
    ask.total = cluster_total(sh, weights_above<DT>(s, -INFINITY, top, ask.steep));
    bound = nucleus_bound(ask, p.V);
  }
  // Below min-p's threshold nothing is kept.  The boundary may then lie below the bound: it is not found, and everything
  // above the bound is kept.  Only the top-k's own weight needs all of the top-k.
  if (ask.floor_on && !(ask.by_count && ask.nucleus)) bound = fmaxf(bound, floor_bound(ask));
  if (!(bound < top)) bound = bound >= top ? top : -INFINITY;  // (a NaN: no bound)
  ask.bound = bound;
  if (ask.nucleus && !ask.by_count) {  // top-p alone: its list may be long, which the counts tell for less than listing
    const uint32_t c = count_steps<DT>(s, sh, ask);
    const uint32_t before = block_scan32(sh, c);
    if (tid == kThreads - 1) sh.here_c = before + c;
    __syncthreads();
    const uint32_t all = sh.here_c;
    if (all > kGather) {
      cut_wide<DT>(s, sh, ask, c);
      return;
    }
  }
  // ---- 2. the logits at or above the bound, by warp and in order -------------------------------
  int n = 0;
#pragma unroll 2
  for (int vb = s.run_a; vb < s.run_z; vb += 32) {
    const int v = vb + lane;
    uint32_t mask = 0;
    if (v < s.run_z) {
      const Vec<DT> x(s.vec(v));
#pragma unroll
      for (int e = 0; e < kElems; ++e) mask |= (x.x[e] >= bound && x.x[e] != -INFINITY ? 1u : 0u) << e;
    }
    if (__any_sync(0xFFFFFFFFu, mask != 0)) list_marked<kElems>(sh, n, mask, v);
  }
  const int listed = n <= kListPerWarp ? n : -1;
  // ---- 3. gathered by the first CTA, if they are few -----------------------------------------------
  const bool few = __syncthreads_and(listed >= 0) && (!ask.by_count || ask.k <= kGatherK);
  if (lane == 0) sh.ties[warp] = n;
  __syncthreads();
  const uint32_t warp_n = lane < kWarps ? sh.ties[lane] : 0;
  const uint32_t at = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? warp_n : 0), all = __reduce_add_sync(0xFFFFFFFFu, warp_n);
  const bool fits = few && all <= kGather;
  if (fits)
    for (int i = lane; i < listed; i += 32) {
      const int pos = sh.list[warp][i];
      sh.gather[at + i] = static_cast<uint64_t>(key_of(s.at(pos))) << 32 | static_cast<uint32_t>(~s.index_of(pos));
    }
  if (tid == 0) sh.mine_n = fits ? all : kGather + 1;
  cluster_sync();
  const uint32_t peer_n = lane < static_cast<int>(cs) ? peer_u32(&sh.mine_n, lane) : 0;
  const uint32_t gathered = __reduce_add_sync(0xFFFFFFFFu, peer_n);
  if (gathered > kGather) {  // the same in every CTA
    cluster_sync();          // everyone has read the counts
    cut_wide<DT>(s, sh, ask, count_steps<DT>(s, sh, ask));
    return;
  }
  if (rank == 0) {
    uint32_t from = peer_n;  // where lane l's CTA's logits end in the list
#pragma unroll
    for (int d = 1; d < kMaxCluster; d <<= 1) {
      const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, from, d);
      if (lane >= d) from += u;
    }
    for (uint32_t i0 = all; i0 < gathered; i0 += kThreads) {
      const uint32_t i = i0 + tid;
      uint32_t r = 0, begin = 0;
#pragma unroll
      for (int l = 0; l < kMaxCluster - 1; ++l) {
        const uint32_t end = __shfl_sync(0xFFFFFFFFu, from, l);
        if (i >= end && l + 1 < static_cast<int>(cs)) {
          r = l + 1;
          begin = end;
        }
      }
      if (i < gathered) sh.gather[i] = peer_u64(&sh.gather[i - begin], r);
    }
  }
  cluster_sync();  // the first CTA has everything: the others leave
  if (rank == 0) {
    if (gathered <= kShort) finish_short<DT>(sh, ask, static_cast<int>(gathered), reinterpret_cast<uint64_t*>(dyn));
    else finish_gathered<DT>(sh, ask, static_cast<int>(gathered), reinterpret_cast<uint64_t*>(dyn));
  }
}

// A cluster per row, or (kListed) resident clusters for the rows that select_kernel has left, in turn.
template <int DT, bool kListed>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ Shared sh;
  const int cluster = blockIdx.x / cluster_size(), clusters = gridDim.x / cluster_size();
  if (threadIdx.x == 0) {
    sh.params = p;
    for (int i = 0; i < kPieces; ++i) mbar_init(&sh.bar[i], 1);
    fence_proxy_async_smem();
  }
  __syncthreads();
  pdl_wait();
  if (!kListed) {
    sample_row<DT>(p, cluster, dyn, sh, 0);
    return;
  }
  const int rows = p.left[0];
  uint32_t parity = 0;
#pragma unroll 1
  for (int i = cluster; i < rows; i += clusters) {  // (a row's end has synchronised the cluster)
    sample_row<DT>(p, p.left[1 + i], dyn, sh, parity);
    parity ^= 1;
    __syncthreads();
    fence_proxy_async_smem();  // the next row's copies overwrite what this one has read and written
  }
}

// ---- many rows: maxima of 128-byte groups, then a CTA per row ----------------------------------------
constexpr int kMaxThreads = 256;
constexpr int kMaxLoads = 4;                             // 16-byte loads of a thread at a time, and as many in flight
constexpr int kSegmentVecs = kMaxThreads * kMaxLoads;    // 16 KB of a row
constexpr int kMaxCtas = 4;                              // per SM
constexpr int kGroupVecs = 8;
constexpr int kSumLoads = 4;                             // the same, where a CTA sums a whole row
constexpr int kSelectCtas = 3;                           // per SM
// Where the maxima pay, in bytes of logits (mixed filters / top-k 50, by maxima against by clusters; bf16 rows): 39 MB
// 105 / 29 against 74 / 37 us, 78 MB 126 / 40 against 113 / 69, 155 MB 162 / 70 against 179 / 125.
constexpr int64_t kStreamBytes = 64 << 20;

// N vectors of 16 bytes of a row, from v on and kMaxThreads or kThreads (`apart`) from each other; vectors lie on 16-byte
// boundaries, and outside the row is -inf.  The loads of whole vectors are all in flight before the (at most two) ragged
// ones are put together.
template <int DT, int N>
__device__ __forceinline__ void row_vecs(const typename Slice<DT>::Elem* x_row, int phase, int V, int v, int apart, uint4 (&w)[N]) {
  using Elem = typename Slice<DT>::Elem;
  constexpr int kElems = Vec<DT>::kElems;
  constexpr uint32_t kNone = DT == SV_BF16 ? 0xFF80FF80u : 0xFF800000u;
  const uint4* vecs = reinterpret_cast<const uint4*>(x_row - phase);
  const int whole_a = phase > 0 ? 1 : 0, whole_z = (phase + V) / kElems, all = (phase + V + kElems - 1) / kElems;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int u = v + i * apart;
    w[i] = make_uint4(kNone, kNone, kNone, kNone);
    if (u >= whole_a && u < whole_z) w[i] = __ldg(vecs + u);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int u = v + i * apart;
    if (u < all && (u < whole_a || u >= whole_z)) {
      Elem* e = reinterpret_cast<Elem*>(&w[i]);
#pragma unroll
      for (int x = 0; x < kElems; ++x) {
        const int at = u * kElems - phase + x;
        if (at >= 0 && at < V) e[x] = x_row[at];
      }
    }
  }
}

// Resident CTAs take 16 KB segments of rows in turn, the next one's loads in flight while one's maxima are taken.  Bound by
// memory: nothing but loads, maxima and one float per 128 bytes written (and the cut row's -inf).
template <int DT>
__global__ void __launch_bounds__(kMaxThreads, kMaxCtas) maxima_kernel(const SampleParams p) {
  using Elem = typename Slice<DT>::Elem;
  constexpr int kElems = Vec<DT>::kElems;
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) p.left[0] = 0;
  const uint32_t items = static_cast<uint32_t>(p.R) * p.segments;
  auto wanted = [&](uint32_t item) {
    Ask ask;
    return item < items && by_maxima(ask, read_ask(p, item / p.segments, ask));
  };
  auto load = [&](uint32_t item, uint4 (&w)[kMaxLoads]) {
    const uint32_t row = item / p.segments;
    const Elem* x_row = static_cast<const Elem*>(p.logits) + row * p.row_stride;
    const int phase = static_cast<int>((reinterpret_cast<uintptr_t>(x_row) & 15u) / sizeof(Elem));
    row_vecs<DT>(x_row, phase, p.V, static_cast<int>(item - row * p.segments) * kSegmentVecs + static_cast<int>(threadIdx.x), kMaxThreads, w);
  };
  uint4 w[kMaxLoads], w_next[kMaxLoads];
  uint32_t item = blockIdx.x;
  bool want = wanted(item), want_next = wanted(item + gridDim.x);
  if (want) load(item, w);
#pragma unroll 1
  for (; item < items; item += gridDim.x) {
    if (want_next) load(item + gridDim.x, w_next);
    const bool want_later = wanted(item + 2 * gridDim.x);
    const uint32_t row = item / p.segments;
    const int segment = static_cast<int>(item - row * p.segments);
    if (want && p.out_rows != nullptr) {  // (never the rows themselves: those are left to the clusters)
      const int e0 = segment * kSegmentVecs * kElems;
      const int n = max(0, min(kSegmentVecs * kElems, p.V - e0));
      Elem* out = static_cast<Elem*>(p.out_rows) + row * p.out_stride + e0;
      const Elem none = DT == SV_BF16 ? static_cast<Elem>(0xFF80u) : static_cast<Elem>(0xFF800000u);
      const int head = min(n, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(out) & 15u)) & 15u) / sizeof(Elem)));
      const int whole = (n - head) / kElems;
      const uint32_t ninf = DT == SV_BF16 ? 0xFF80FF80u : 0xFF800000u;
      for (int i = threadIdx.x; i < whole; i += kMaxThreads) reinterpret_cast<uint4*>(out + head)[i] = make_uint4(ninf, ninf, ninf, ninf);
      for (int i = threadIdx.x; i < n - whole * kElems; i += kMaxThreads) out[i < head ? i : i + whole * kElems] = none;
    }
    if (want) {
#pragma unroll
      for (int i = 0; i < kMaxLoads; ++i) {
        const Vec<DT> x(w[i]);
        float m = x.x[0];
#pragma unroll
        for (int e = 1; e < kElems; ++e) m = max_nan(m, x.x[e]);
#pragma unroll
        for (int d = 1; d < kGroupVecs; d <<= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        const int g = (segment * kSegmentVecs + i * kMaxThreads + threadIdx.x) / kGroupVecs;
        if ((threadIdx.x & (kGroupVecs - 1)) == 0 && g < p.groups) p.maxima[row * static_cast<int64_t>(p.groups) + g] = m;
      }
    }
#pragma unroll
    for (int i = 0; i < kMaxLoads; ++i) w[i] = w_next[i];
    want = want_next;
    want_next = want_later;
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads, kSelectCtas) select_kernel(const SampleParams p) {
  using Elem = typename Slice<DT>::Elem;
  constexpr int kElems = Vec<DT>::kElems;
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ Shared sh;
  uint64_t* more = reinterpret_cast<uint64_t*>(dyn);                                     // step 3's room
  float* maxima = reinterpret_cast<float*>(dyn + sizeof(uint64_t) * kGather + sizeof(uint32_t) * 3 * kSteps);
  uint16_t* groups = &sh.list[0][0];
  constexpr int kMost = kWarps * kListPerWarp;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x;
  sh.count[tid] = 0;
  if (tid == 0) sh.params = p;
  pdl_wait();
  Ask ask;
  const uint32_t bad = read_ask(p, row, ask);
  ask.p = &sh.params;
  bool bad_uniform = false;
  for (int j = tid; j < p.M; j += kThreads) {
    const float u = p.uniforms[row * p.M + j];
    bad_uniform |= !(u >= 0.0f && u < 1.0f);
  }
  const bool mine = !__syncthreads_or(bad_uniform) && by_maxima(ask, bad);
  const Elem* x_row = static_cast<const Elem*>(p.logits) + row * p.row_stride;
  const int phase = static_cast<int>((reinterpret_cast<uintptr_t>(x_row) & 15u) / sizeof(Elem));
  const int vecs = (phase + p.V + kElems - 1) / kElems, n_groups = (vecs + kGroupVecs - 1) / kGroupVecs;
  const uint32_t none_key = key_of(-INFINITY), inf_key = key_of(INFINITY);
  uint32_t hi = 0, lo = 0xFFFFFFFFu;
  if (mine)
#pragma unroll 4
    for (int g = tid; g < n_groups; g += kThreads) {
      const float m = p.maxima[row * p.groups + g];
      maxima[g] = m;
      const uint32_t key = key_of(m);
      hi = max(hi, key);
      if (key > none_key) lo = min(lo, key);
    }
  hi = __reduce_max_sync(0xFFFFFFFFu, hi);
  lo = __reduce_min_sync(0xFFFFFFFFu, lo);
  if (lane == 0) {
    sh.red[0][warp] = hi;
    sh.red[1][warp] = lo;
  }
  __syncthreads();
  const uint32_t top_key = __reduce_max_sync(0xFFFFFFFFu, sh.red[0][lane & (kWarps - 1)]);
  const uint32_t low_key = __reduce_min_sync(0xFFFFFFFFu, sh.red[1][lane & (kWarps - 1)]);
  if (!mine || top_key >= inf_key || top_key <= none_key) {
    if (tid == 0) p.left[1 + atomicAdd(p.left, 1)] = static_cast<int>(row);  // (in any order: rows do not depend on it)
    return;
  }
  const float top = logit_of_key(top_key);
  ask.top = top;
  // the bound: the k-th largest maximum has k logits at or above it
  float bound = ask.k == 1 ? top : -INFINITY;
  if (ask.by_count && ask.k > 1) {
    const float range = __fsub_rn(top, logit_of_key(low_key));
    const Scale scale = Scale::over(top, range);
    for (int g = tid; g < n_groups; g += kThreads)
      if (maxima[g] > -INFINITY) atomicAdd(&sh.count[scale.step(maxima[g])], 1u);
    __syncthreads();
    find_step<false>(sh, sh.count[tid], 0, ask.k, 0, 0);
    if (sh.step != 0xFFFFFFFFu) bound = scale.lower_end(sh.step, range);
  }
  if (ask.nucleus && !ask.by_count) {  // W, over the whole row (its second reading)
    WeightSum sum(top, ask.steep);
    uint32_t adds = 0;
#pragma unroll 1
    for (int v = tid; v < vecs; v += kSumLoads * kThreads) {
      uint4 w[kSumLoads];
      row_vecs<DT>(x_row, phase, p.V, v, kThreads, w);
#pragma unroll
      for (int i = 0; i < kSumLoads; ++i) {
        const Vec<DT> x(w[i]);
#pragma unroll
        for (int e = 0; e < kElems; e += 2) sum.add(x.x[e], x.x[e + 1]);
      }
      adds += kSumLoads;
    }
    const uint64_t w = warp_sum(sum.total(adds * (kElems / 2)));
    if (lane == 0) sh.seg[warp] = w;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) ask.total += sh.seg[i];
    bound = nucleus_bound(ask, p.V);
  }
  if (ask.floor_on && !(ask.by_count && ask.nucleus)) bound = fmaxf(bound, floor_bound(ask));
  if (!(bound < top)) bound = bound >= top ? top : -INFINITY;  // (a NaN: no bound)
  ask.bound = bound;
  ask.out_row = p.out_rows != nullptr ? static_cast<Elem*>(p.out_rows) + row * p.out_stride : nullptr;
  // the groups that reach it, in order: thread t looks at a stretch
  const int per = (n_groups + kThreads - 1) / kThreads, a = min(n_groups, tid * per), b = min(n_groups, a + per);
  uint32_t c = 0;
  for (int g = a; g < b; ++g) c += maxima[g] >= bound && maxima[g] > -INFINITY;
  uint32_t at = block_scan32(sh, c);
  if (tid == kThreads - 1) sh.here_c = at + c;
  for (int g = a; g < b; ++g)
    if (maxima[g] >= bound && maxima[g] > -INFINITY) {
      if (at < kMost) groups[at] = static_cast<uint16_t>(g);
      ++at;
    }
  __syncthreads();
  const int listed = static_cast<int>(sh.here_c);
  __syncthreads();
  // their logits at or above the bound, in order: eight threads a group
  int n = 0;
  bool too_many = listed > kMost;
  for (int g0 = 0; g0 < listed && !too_many; g0 += kThreads / kGroupVecs) {
    const int g = g0 + tid / kGroupVecs;
    const int v = g < listed ? groups[g] * kGroupVecs + tid % kGroupVecs : vecs;
    uint32_t mask = 0;
    uint4 w[1];
    row_vecs<DT>(x_row, phase, p.V, v, 0, w);
    const Vec<DT> x(w[0]);
    if (v < vecs)
#pragma unroll
      for (int e = 0; e < kElems; ++e) mask |= (x.x[e] >= bound && x.x[e] != -INFINITY ? 1u : 0u) << e;
    const uint32_t count = __popc(mask);
    uint32_t to = n + block_scan32(sh, count);
    if (tid == kThreads - 1) sh.here_c = to + count;
    __syncthreads();
    n = static_cast<int>(sh.here_c);
    too_many = n > kGather;
    if (!too_many)
#pragma unroll
      for (int e = 0; e < kElems; ++e)
        if ((mask >> e) & 1u) sh.gather[to++] = static_cast<uint64_t>(key_of(x.x[e])) << 32 | static_cast<uint32_t>(~(v * kElems + e - phase));
    __syncthreads();
  }
  if (too_many) {
    if (tid == 0) p.left[1 + atomicAdd(p.left, 1)] = static_cast<int>(row);
    return;
  }
  if (n <= kShort) finish_short<DT>(sh, ask, n, more);
  else finish_gathered<DT>(sh, ask, n, more);
}

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }
int groups_of(int V) { return (V + 2 * 4) / (4 * kGroupVecs) + 1; }  // float32 rows have the most

template <int DT>
cudaError_t launch_sample(SampleParams p, void* stream) {
  constexpr int kElt = DT == SV_BF16 ? 2 : 4;
  // CTAs per row: slices of at most 78 KB (two CTAs an SM), and smaller ones while all rows' CTAs are on the GPU at
  // once (two of 512 threads an SM)
  int cs = 1, sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int64_t bytes = static_cast<int64_t>(p.V) * kElt;
  while (cs < kMaxCluster && (bytes > cs * 79872 || (bytes > cs * 16384 && 2 * static_cast<int64_t>(cs) * p.R <= 2 * sms))) cs *= 2;
  p.slice = ((p.V + cs - 1) / cs + 7) & ~7;
  const size_t dyn = std::max(static_cast<size_t>(p.slice) * kElt + 32, sizeof(uint64_t) * kGather + sizeof(uint32_t) * 3 * kSteps);  // (the first CTA's room too)
  if (p.left != nullptr) {
    p.segments = ((p.V + 2 * (16 / kElt)) / (16 / kElt) + kSegmentVecs) / kSegmentVecs;
    const int64_t items = static_cast<int64_t>(p.R) * p.segments;
    e = launch_dependent(maxima_kernel<DT>, dim3(static_cast<unsigned>(std::min<int64_t>(items, kMaxCtas * sms))), kMaxThreads, 0, stream, SV_KERNEL_SAMPLE, 1, p);
    if (e != cudaSuccess) return e;
    const size_t room = sizeof(uint64_t) * kGather + sizeof(uint32_t) * 3 * kSteps + sizeof(float) * p.groups;
    if ((e = allow_smem<select_kernel<DT>>(room)) != cudaSuccess) return e;
    e = launch_dependent(select_kernel<DT>, dim3(p.R), kThreads, room, stream, SV_KERNEL_SAMPLE, 1, p);
    if (e != cudaSuccess) return e;
    if ((e = allow_smem<sample_kernel<DT, true>>(dyn)) != cudaSuccess) return e;
    const int clusters = std::min(p.R, std::max(1, 2 * sms / cs));
    return launch_dependent(sample_kernel<DT, true>, dim3(static_cast<unsigned>(clusters) * cs), kThreads, dyn, stream, SV_KERNEL_SAMPLE, cs, p);
  }
  if ((e = allow_smem<sample_kernel<DT, false>>(dyn)) != cudaSuccess) return e;
  return launch_dependent(sample_kernel<DT, false>, dim3(static_cast<unsigned>(p.R) * cs), kThreads, dyn, stream, SV_KERNEL_SAMPLE, cs, p);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t sv_sample_workspace_size(int R, int V) {
  if (R < 0 || R > SV_MAX_SAMPLE_ROWS || V < 1 || V > SV_MAX_SAMPLE_VOCAB) return 0;
  return SV_STATUS_BYTES + round256(sizeof(int32_t) * (1 + R)) + sizeof(float) * static_cast<size_t>(R) * groups_of(V);
}

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
  sv_status st = check_workspace(ws, ws_bytes, sv_sample_workspace_size(R, V));
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
  p.groups = groups_of(V);
  p.maxima = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + SV_STATUS_BYTES + round256(sizeof(int32_t) * (1 + R)));
  // by the maxima where rows may have a top-k or min-p and there is enough to stream; rows cut in place are not: their
  // logits are needed again after the fill
  if ((top_k != nullptr || min_p != nullptr) && static_cast<int64_t>(R) * V * static_cast<int64_t>(elt) >= kStreamBytes && out_rows != logits)
    p.left = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(ws) + SV_STATUS_BYTES);
  return launch_status(dt == SV_BF16 ? launch_sample<SV_BF16>(p, stream) : launch_sample<SV_F32>(p, stream), "sample");
}
