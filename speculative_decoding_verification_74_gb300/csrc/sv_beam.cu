// sv_beam_select: one step of beam search, the K best of all beams' continuations.
//
// rows_kernel reads every row of logits once; a row is cut into parts, a CTA each.  A warp takes every eighth piece of its CTA's
// part, 2 KB held in registers, the next ones in flight, and keeps
//   the sum of exp(x - ref) for a reference near the part's maximum: float32 terms, compensated sums;
//   each lane's largest logit of each piece, in shared memory.
// Then the CTA finds a bound that at least K of its threads' largest logits, and few more, are at or above (bisection, a barrier
// that counts per step): the part's K best logits are at or above it too.  The pieces' lanes that reach it are read again (64 bytes each), and their logits
// at or above the bound are ranked by counting.  Parts with too many of those (long runs of equals, or too few finite maxima for a
// bound) are scanned in order instead, by one warp with a sorted list into which batches of candidates are merged.
//
// merge_kernel, a CTA per request, gives each row A = score - log sum exp(x - m), m its largest logit, so that a candidate's total
// is A + (x - m) (m apart: next to a large one the rest would be lost).  A bisection on totals in float32 leaves little more
// than K candidates, which are ranked by counting on totals in 64 bits.  The float32 terms leave A uncertain by up to 2^-19: 2^-22
// of ex2, the roundings of a term's exponent and of its lane's reference (half a step of numbers below 8, or of up to log2 V for
// terms that are as many as they are small, times ln 2: 2^-21 each), a piece's plain sum (ten steps of 2^-24), logf and exp2f
// (2^-23 each); the pieces' compensated sums add next to nothing.  So where neighbours of different beams in the order lie within
// kNear of each other, or the K-th and any candidate past the cut do, their rows are summed again with terms in pairs of floats,
// and the ranking is repeated.  With this the order is that of the exact totals where those of two beams differ by 2^-25 (each
// term is off by 2^-30 of itself and 2^-45, V of them by 2^-27), and that of beams where they are equal.
//
// Measured (GB300, graph replay; a copy of the logits in brackets): 256 requests of four rows of 151936, K = 8, float32 123 us (92),
// bf16 77 (46); of 64 requests of 16 beams a quarter with one beam only, K = 32, bf16 62 (35: rows of missing beams are not read);
// 64 rows float32 20 us (6), four rows of 32000 bf16 14 to 16 us.  Of the 77, the stream takes 55, looking for candidates 12, all
// CTAs at about the same time, and the merge 10.  Where two beams' totals lie near each other (one request of 32 candidates in
// 300), summing their rows again takes another 55 to 80 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>

#include "sv_device.cuh"
#include "sv_ops.h"

namespace sv {
namespace {

constexpr int kThreads = 256;
constexpr int kRowCtas = 3;                    // CTAs of the rows' kernel on an SM (784 rows bf16 61 us; with 4 64, with 2 75)
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;                       // 16-byte vectors of a piece per lane
constexpr int kPiece = 32 * kVecs;             // vectors of a piece
constexpr int kBatch = 64;                     // candidates that wait for the list
constexpr int kMaxParts = 32;                  // parts of a row: a lane each in the merge
constexpr float kLog2e = 1.44269504088896341f;
// How far a logit may lie above a sum's reference: exponents of the largest terms stay below 8, so that half a step of them is
// 2^-22.  (64 requests of 16 beams 61.3 us with 30 and 8, 61.6 with 5, 61.8 with 3.)
constexpr float kRefSlack = 5.0f;
constexpr float kFarRef = 0x1p12f;             // references past this are subtracted from the logits themselves
constexpr int kFraction = 40;                  // fractional bits of a part's sum
constexpr int kMergeThreads = 512;
constexpr double kNear = 0x1p-18;              // totals of two beams nearer than this are told apart by exact sums

struct Entry {  // a candidate: entries of -inf are none
  float x;
  int32_t token;
};
struct Part {   // of a row: largest logit, sum of 2^((x - m) log2 e) in units of 2^-kFraction
  uint64_t sum;
  float m;
  uint32_t bad;
};

struct BeamParams {
  const void* logits;
  int64_t row_stride;
  const float* scores;
  const int32_t* finished;
  float* out_scores;
  int32_t *out_rows, *out_tokens;
  Part* parts;       // [rows][P]
  Entry* entries;    // [rows][P][K]
  uint32_t* status;
  int32_t W, V, K, P, pad, rows;
};

template <int DT>
struct Elem;
template <>
struct Elem<SV_BF16> {
  static constexpr int kPerVec = 8, kBytes = 2;
  static constexpr uint32_t kNone = 0xFF80FF80u;
};
template <>
struct Elem<SV_F32> {
  static constexpr int kPerVec = 4, kBytes = 4;
  static constexpr uint32_t kNone = 0xFF800000u;
};
template <int DT>
__device__ __forceinline__ float element(const uint4 (&w)[kVecs], int i, int j) {
  const uint32_t* p = reinterpret_cast<const uint32_t*>(&w[i]);
  if constexpr (DT == SV_BF16) return (j & 1) ? bf16_hi(p[j >> 1]) : bf16_lo(p[j >> 1]);
  else return __uint_as_float(p[j]);
}

// One of a vector's elements, j known at run time only.
template <int DT>
__device__ __forceinline__ float element_at(const uint4& w, int j) {
  if constexpr (DT == SV_BF16) {
    const uint32_t pair = j < 4 ? (j < 2 ? w.x : w.y) : (j < 6 ? w.z : w.w);
    return (j & 1) ? bf16_hi(pair) : bf16_lo(pair);
  } else {
    return __uint_as_float(j < 2 ? (j < 1 ? w.x : w.y) : (j < 3 ? w.z : w.w));
  }
}
// Its largest element (NaN passed over).
template <int DT>
__device__ __forceinline__ float vec_max(const uint4& w) {
  if constexpr (DT == SV_BF16) {
    uint32_t a, b;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w.x), "r"(w.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w.z), "r"(w.w));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return fmaxf(bf16_lo(a), bf16_hi(a));
  } else {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
}
// The largest of a lane's elements of a piece.
template <int DT>
__device__ __forceinline__ float piece_max(const uint4 (&w)[kVecs]) {
  if constexpr (DT == SV_BF16) {
    uint32_t m[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int i = 1; i < kVecs; ++i) {
      asm("max.bf16x2 %0, %0, %1;" : "+r"(m[0]) : "r"(w[i].x));
      asm("max.bf16x2 %0, %0, %1;" : "+r"(m[1]) : "r"(w[i].y));
      asm("max.bf16x2 %0, %0, %1;" : "+r"(m[2]) : "r"(w[i].z));
      asm("max.bf16x2 %0, %0, %1;" : "+r"(m[3]) : "r"(w[i].w));
    }
    return vec_max<DT>(make_uint4(m[0], m[1], m[2], m[3]));
  } else {
    float m = vec_max<DT>(w[0]);
#pragma unroll
    for (int i = 1; i < kVecs; ++i) m = fmaxf(m, vec_max<DT>(w[i]));
    return m;
  }
}

// At least K of a piece's logits are at or above it: every lane's vectors are groups, and at least K groups' largest logits are.
// Found by bisection between the smallest and the largest of them, until little more than K are.
__device__ __forceinline__ float group_bound(const float (&high)[kVecs], float mine, int K) {
  float low = mine, top = mine;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) low = fminf(low, high[i]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, d));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  }
  low = fmaxf(low, -FLT_MAX);          // (all groups are at or above it, or it is no bound at all)
  float over = top;
#pragma unroll 1
  for (int step = 0; step < 10; ++step) {
    const float mid = 0.5f * low + 0.5f * over;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) n += __popc(__ballot_sync(0xFFFFFFFFu, high[i] >= mid));
    if (n >= K) {
      low = mid;
      if (n <= K + (K >> 2)) break;
    } else {
      over = mid;
    }
  }
  return fmaxf(low, -FLT_MAX);         // (a piece of nothing but -inf)
}

// A row as 16-byte vectors: `lead` elements of the first lie before the row.
struct Row {
  const unsigned char* base;
  int lead, vecs, V;
};
template <int DT>
__device__ __forceinline__ Row row_of(const BeamParams& a, int64_t row) {
  using E = Elem<DT>;
  const unsigned char* p = static_cast<const unsigned char*>(a.logits) + row * a.row_stride * E::kBytes;
  Row r;
  r.lead = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / E::kBytes);
  r.base = p - r.lead * E::kBytes;
  r.vecs = (r.lead + a.V + E::kPerVec - 1) / E::kPerVec;
  r.V = a.V;
  return r;
}
// A vector that holds elements outside the row: those are -inf.
template <int DT>
__device__ __noinline__ uint4 edge_vec(const Row& r, int vec) {
  using E = Elem<DT>;
  uint32_t w[4];
  for (int i = 0; i < 4; ++i) w[i] = E::kNone;
  for (int j = 0; j < E::kPerVec; ++j) {
    const int v = vec * E::kPerVec + j - r.lead;
    if (v < 0 || v >= r.V) continue;
    const unsigned char* p = r.base + (static_cast<int64_t>(vec) * E::kPerVec + j) * E::kBytes;
    if constexpr (DT == SV_BF16) {
      const uint32_t x = __ldg(reinterpret_cast<const uint16_t*>(p));
      w[j >> 1] = (j & 1) ? (w[j >> 1] & 0xFFFFu) | (x << 16) : (w[j >> 1] & 0xFFFF0000u) | x;
    } else {
      w[j] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int DT>
__device__ __forceinline__ uint4 load_vec(const Row& r, int vec) {
  using E = Elem<DT>;
  const int last = (r.lead + r.V) % E::kPerVec != 0 ? r.vecs - 1 : r.vecs;  // vectors from here on are not whole
  uint4 w;
  if (vec >= (r.lead != 0 ? 1 : 0) && vec < last) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "l"(r.base + static_cast<int64_t>(vec) * 16));
  } else {
    w = vec < r.vecs ? edge_vec<DT>(r, vec) : make_uint4(E::kNone, E::kNone, E::kNone, E::kNone);
  }
  return w;
}
template <int DT>
__device__ __forceinline__ void load_piece(const Row& r, int piece, uint4 (&w)[kVecs]) {
#pragma unroll
  for (int i = 0; i < kVecs; ++i) w[i] = load_vec<DT>(r, piece * kPiece + i * 32 + static_cast<int>(threadIdx.x & 31));
}

// Floats as integers in their order; 0 is below them all.
__device__ __forceinline__ uint32_t float_key(float t) {
  const uint32_t b = __float_as_uint(t + 0.0f);  // (-0 equals 0)
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float float_of_key(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k); }
// A key that at least `want` threads' keys are at or above, at most `enough` where they differ; `least` where fewer are above that.
// Every thread of the CTA calls it; most: the largest key; guess: where to look first.
template <int kThreadsOfCta>
__device__ __forceinline__ uint32_t lower_bound_of(uint32_t key, uint32_t least, uint32_t most, uint32_t guess, int want, int enough) {
  static_assert(kThreadsOfCta >= SV_MAX_BEAM_CANDIDATES + 1, "a thread for each");
  if (most <= least) return least;
  uint32_t low = least, over = most + 1;
  for (uint32_t mid = guess;;) {
    if (mid <= low || mid >= over) mid = low + ((over - low) >> 1);
    const int n = __syncthreads_count(key >= mid);
    if (n >= want) {
      low = mid;
      if (n <= enough) return low;
    } else {
      over = mid;
    }
    if (over - low <= 1) return low;
    mid = 0;
  }
}
// Order of candidates as an integer: larger x first, then the lower token.
__device__ __forceinline__ uint64_t order_key(float x, int token) {
  return (static_cast<uint64_t>(float_key(x)) << 32) | ~static_cast<uint32_t>(token);
}
__device__ __forceinline__ float logit_of(uint64_t key) { return float_of_key(static_cast<uint32_t>(key >> 32)); }
__device__ __forceinline__ Entry entry_of(uint64_t key) { return Entry{logit_of(key), static_cast<int32_t>(~static_cast<uint32_t>(key))}; }
// The next float above x (x finite or -inf).
__device__ __forceinline__ float above(float x) {
  if (x == 0.0f) return __uint_as_float(1u);
  const uint32_t b = __float_as_uint(x);
  return __uint_as_float((b & 0x80000000u) ? b - 1 : b + 1);
}

// Shared memory of a scan.
struct Scan {
  uint4 piece[kPiece];                       // a piece whose candidates are looked for
  uint64_t list[2][SV_MAX_BEAM_CANDIDATES];  // keys, best first; the halves in turn
  uint64_t batch[kBatch], sorted[32];
  int32_t from, listed, waiting;             // the list's half and length, the batch's length
};

// How many of keys[0 .. n) (best first) are better than `key`.
__device__ __forceinline__ int better(const uint64_t* keys, int n, uint64_t key) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (keys[mid] > key) lo = mid + 1; else hi = mid;
  }
  return lo;
}
// Merges the batch's first n <= 32 keys into list[from][0 .. listed); returns the list's new length, in the other half.
__device__ __noinline__ int merge_batch(Scan& sh, int from, int listed, int n, int K) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  const uint64_t key = lane < n ? sh.batch[lane] : 0;
  int rank = 0;
#pragma unroll 8
  for (int j = 0; j < n; ++j) rank += sh.batch[j] > key;
  if (lane < n) sh.sorted[rank] = key;
  __syncwarp();
  uint64_t* to = sh.list[from ^ 1];
  for (int i = lane; i < listed; i += 32) {
    const uint64_t k = sh.list[from][i];
    const int at = i + better(sh.sorted, n, k);
    if (at < K) to[at] = k;
  }
  if (lane < n) {
    const int at = rank + better(sh.list[from], listed, key);
    if (at < K) to[at] = key;
  }
  __syncwarp();
  return min(K, listed + n);
}
// The batch's first 32 into the list.
__device__ __noinline__ void flush_batch(Scan& sh, int K) {
  const int lane = threadIdx.x & 31, n = min(sh.waiting, 32), left = sh.waiting - n;
  const int listed = merge_batch(sh, sh.from, sh.listed, n, K);
  const uint64_t later = lane < left ? sh.batch[32 + lane] : 0;
  __syncwarp();
  if (lane < left) sh.batch[lane] = later;
  if (lane == 0) {
    sh.from ^= 1;
    sh.listed = listed;
    sh.waiting = left;
  }
  __syncwarp();
}
// The candidates of the piece in shared memory, whose vector v is at row vector first_vec + v: those at or above `bound` (until K
// are listed also at or above the piece's own bound).  Returns the bound of the pieces after it.
template <int DT>
__device__ __noinline__ float scan_piece(Scan& sh, int first_vec, int lead, float bound, int K) {
  using E = Elem<DT>;
  const int lane = threadIdx.x & 31;
  float high[kVecs], mine = -INFINITY;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    high[i] = vec_max<DT>(sh.piece[i * 32 + lane]);
    mine = fmaxf(mine, high[i]);
  }
  float least = sh.listed < K ? fmaxf(bound, group_bound(high, mine, K)) : bound;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    // the lanes whose vectors reach it, one by one: its elements go to as many lanes
    uint32_t lanes = __ballot_sync(0xFFFFFFFFu, high[i] >= least);
    while (lanes != 0) {
      const int vec = i * 32 + __ffs(lanes) - 1;
      lanes &= lanes - 1;
      const float x = element_at<DT>(sh.piece[vec], lane & (E::kPerVec - 1));
      const bool takes = lane < E::kPerVec && x >= least;
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, takes);
      const int waiting = sh.waiting;
      if (takes) sh.batch[waiting + __popc(who & ((1u << lane) - 1u))] = order_key(x, (first_vec + vec) * E::kPerVec + lane - lead);
      __syncwarp();
      if (lane == 0) sh.waiting = waiting + __popc(who);
      __syncwarp();
      if (waiting + __popc(who) >= 32) {
        flush_batch(sh, K);
        if (sh.listed == K) least = fmaxf(least, logit_of(sh.list[sh.from][K - 1]));  // no logit below the K-th counts
      }
    }
  }
  if (sh.waiting > 0 && sh.listed < K) flush_batch(sh, K);
  return sh.listed == K ? above(logit_of(sh.list[sh.from][K - 1])) : -FLT_MAX;  // an equal logit further on comes after it
}

// A sum of exp(x - ref): terms 2^(k x - k ref), the product with k = log2 e exact but for one rounding; Kahan's sum.
struct Sum {
  float ref = 0.0f, sum = 0.0f, lost = 0.0f;
  bool begun = false;                  // ref is a logit's
};
template <int DT>
__device__ __forceinline__ void add_piece(Sum& a, const uint4 (&w)[kVecs], float mine) {
  using E = Elem<DT>;
  if (mine > (a.begun ? a.ref + kRefSlack : -INFINITY)) {
    const float by = a.begun ? exp2f((a.ref - mine) * kLog2e) : 0.0f;
    a.sum *= by;
    a.lost *= by;
    a.ref = mine;
    a.begun = true;
  }
  // Up to kFarRef, k ref is off by 2^-12 at most, and 2^rest = 1 + rest ln 2 to 2^-26.  Past it (masks of large numbers, logits far
  // from 0) the difference comes first, rounded once more; nothing of k ref is left then.
  const bool far = __any_sync(0xFFFFFFFFu, fabsf(a.ref) > kFarRef);
  const float off = far ? 0.0f : -a.ref * kLog2e, rest = far ? 0.0f : fmaf(-a.ref, kLog2e, -off);  // off + rest = -k ref
  const f32x2 k2 = f2_pack(kLog2e, kLog2e), off2 = f2_pack(off, off);
  f32x2 s[2] = {0, 0};
  if (far) {
    const f32x2 less = f2_pack(-a.ref, -a.ref);
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int j = 0; j < E::kPerVec; j += 2)
        s[(j >> 1) & 1] = f2_add(s[(j >> 1) & 1], f2_exp2_offset(f2_add(f2_pack(element<DT>(w, i, j), element<DT>(w, i, j + 1)), less), k2, off2));
  } else {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int j = 0; j < E::kPerVec; j += 2)
        s[(j >> 1) & 1] = f2_add(s[(j >> 1) & 1], f2_exp2_offset(f2_pack(element<DT>(w, i, j), element<DT>(w, i, j + 1)), k2, off2));
  }
  float s0, s1;
  f2_unpack(f2_add(s[0], s[1]), s0, s1);
  const float terms = fmaf(s0 + s1, rest * 0.693147181f, s0 + s1);
  const float y = terms - a.lost, now = a.sum + y;
  a.lost = (now - a.sum) - y;
  a.sum = now;
}

constexpr int kGroups = 512;                   // lanes of pieces that are read again (of K = 128 about 250)
constexpr int kFound = 1024;                   // their logits that are ranked
// Shared memory of a CTA; then the maxima [pieces of the part][32].
struct Shared {
  union {
    Scan scan;
    struct {
      uint64_t key[kFound];
      int32_t group[kGroups];
    } few;
  };
  unsigned long long sum;
  float top[kWarps];
  int n_groups, n_found;
};

template <int DT>
__global__ void __launch_bounds__(kThreads, kRowCtas) rows_kernel(const BeamParams a) {
  using E = Elem<DT>;
  extern __shared__ __align__(16) unsigned char dyn[];
  Shared& sh = *reinterpret_cast<Shared*>(dyn);
  float* maxima = reinterpret_cast<float*>(dyn + sizeof(Shared));
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t id = blockIdx.x, row = id / a.P;
  const int part = static_cast<int>(id - row * a.P), K = a.K;
  const float score = a.scores[row];
  if (!(fabsf(score) <= FLT_MAX) || (a.finished != nullptr && a.finished[row] != 0)) return;  // (the merge looks at neither)
  const Row r = row_of<DT>(a, row);
  const int pieces = (r.vecs + kPiece - 1) / kPiece;
  const int p0 = static_cast<int>(static_cast<int64_t>(pieces) * part / a.P), p1 = static_cast<int>(static_cast<int64_t>(pieces) * (part + 1) / a.P);
  if (tid == 0) {
    sh.sum = 0;
    sh.n_groups = sh.n_found = 0;
  }
  float top = -INFINITY;
  Sum total;
  {
    uint4 w[kVecs], next[kVecs];
    auto step = [&](const uint4 (&x)[kVecs], int piece) {
      const float mine = piece_max<DT>(x);
      top = fmaxf(top, mine);
      maxima[(piece - p0) * 32 + lane] = mine;
      add_piece<DT>(total, x, mine);
    };
    int piece = p0 + warp;
    if (piece < p1) load_piece<DT>(r, piece, w);
    for (; piece < p1; piece += 2 * kWarps) {
      if (piece + kWarps < p1) load_piece<DT>(r, piece + kWarps, next);
      step(w, piece);
      if (piece + kWarps >= p1) break;
      if (piece + 2 * kWarps < p1) load_piece<DT>(r, piece + 2 * kWarps, w);
      step(next, piece + kWarps);
    }
  }
  // the sum, relative to the part's largest logit; a NaN or +inf logit leaves one that is not finite
  float high = top;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) high = fmaxf(high, __shfl_xor_sync(0xFFFFFFFFu, high, d));
  if (lane == 0) sh.top[warp] = high;
  const bool bad = __syncthreads_or(!(fabsf(total.sum) <= FLT_MAX) || high == INFINITY);
#pragma unroll
  for (int x = 0; x < kWarps; ++x) high = fmaxf(high, sh.top[x]);
  uint64_t units = 0;
  if (!bad && total.begun)
    units = __float2ull_rn((total.sum - total.lost) * exp2f((total.ref - high) * kLog2e) * static_cast<float>(1ull << kFraction));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) units += __shfl_xor_sync(0xFFFFFFFFu, units, d);
  if (lane == 0 && units != 0) atomicAdd(&sh.sum, static_cast<unsigned long long>(units));
  // the bound: at least K threads' largest logits are at or above it, or it is the lowest there is
  const float bound = float_of_key(lower_bound_of<kThreads>(float_key(top), float_key(-FLT_MAX), float_key(high), float_key(high - 8.0f), K, K + (K >> 2)));
  const int groups = (p1 - p0) * 32;
  for (int x = tid; x < groups; x += kThreads)
    if (maxima[x] >= bound) {
      const int at = atomicAdd(&sh.n_groups, 1);
      if (at < kGroups) sh.few.group[at] = x;
    }
  __syncthreads();
  const int n_groups = sh.n_groups;
  if (n_groups <= kGroups) {
    for (int x = tid; x < n_groups * kVecs; x += kThreads) {
      const int g = sh.few.group[x / kVecs], vec = (p0 + (g >> 5)) * kPiece + (x % kVecs) * 32 + (g & 31);
      const uint4 v = load_vec<DT>(r, vec);
      if (vec_max<DT>(v) >= bound)
#pragma unroll
        for (int j = 0; j < E::kPerVec; ++j) {
          const float e = element_at<DT>(v, j);
          if (e >= bound) {
            const int at = atomicAdd(&sh.n_found, 1);
            if (at < kFound) sh.few.key[at] = order_key(e, vec * E::kPerVec + j - r.lead);
          }
        }
    }
  }
  __syncthreads();
  const int n = n_groups <= kGroups ? sh.n_found : INT_MAX;
  Entry* out = a.entries + id * K;
  if (n <= kFound) {
    for (int x = tid; x < n; x += kThreads) {
      const uint64_t key = sh.few.key[x];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) rank += sh.few.key[j] > key;
      if (rank < K) out[rank] = entry_of(key);
    }
    for (int x = n + tid; x < K; x += kThreads) out[x] = Entry{-INFINITY, -1};
  } else if (warp == 0) {
    Scan& scan = sh.scan;
    if (lane == 0) scan.from = scan.listed = scan.waiting = 0;
    __syncwarp();
    float least = bound;
    for (int piece = p0; piece < p1; ++piece) {
      if (!__any_sync(0xFFFFFFFFu, maxima[(piece - p0) * 32 + lane] >= least)) continue;
      uint4 w[kVecs];
      load_piece<DT>(r, piece, w);
#pragma unroll
      for (int i = 0; i < kVecs; ++i) scan.piece[i * 32 + lane] = w[i];
      __syncwarp();
      least = fmaxf(bound, scan_piece<DT>(scan, piece * kPiece, r.lead, least, K));
      __syncwarp();
    }
    while (scan.waiting > 0) flush_batch(scan, K);
    for (int i = lane; i < K; i += 32) out[i] = i < scan.listed ? entry_of(scan.list[scan.from][i]) : Entry{-INFINITY, -1};
  }
  if (tid == 0) a.parts[id] = Part{sh.sum, high, bad};
}

// ---- merge -----------------------------------------------------------------------------------------
__device__ __forceinline__ f32x2 f2_all(float x) { return f2_pack(x, x); }
__device__ __forceinline__ f32x2 f2_less(f32x2 a, f32x2 b) { return f2_fma(b, f2_all(-1.0f), a); }  // a - b

// A sum of 2^((x - m) log2 e), x <= m, in units of 2^-44: each term from pairs of floats (Dekker's and Knuth's exact sums and
// products), off by about 2^-30 of itself and half a unit, and then rounded to whole units, so that the sum does not depend on
// its order.  Two logits at a time in packed arithmetic (two rows
// of 151936 by one CTA 78 us; one logit at a time, converted to integers by instructions, 158).
struct ExactSum {
  static constexpr float kHigh = 3.0f, kLow = 1.5f * 0x1p-21f;  // a sum with these is a multiple of 2^-22, of 2^-44
  uint32_t high = 0, low = 0;                                   // their bits added up
  uint32_t pairs = 0;
  __device__ __forceinline__ void add(f32x2 x, f32x2 m) {
    constexpr float k = kLog2e, k_low = 1.92596299e-8f, ln2 = 0.693147182f, ln2_low = -1.90465421e-9f, whole = 0x1.8p23f;
    const f32x2 s = f2_less(x, m), b = f2_less(s, x), err = f2_less(f2_less(x, f2_less(s, b)), f2_add(m, b));  // x - m = s + err
    const f32x2 np = f2_mul(s, f2_all(-k));
    const f32x2 e = f2_fma(err, f2_all(k), f2_fma(s, f2_all(k_low), f2_fma(s, f2_all(k), np)));  // (x - m) log2 e = e - np
    const f32x2 nm = f2_less(f2_all(whole), np);                 // its whole part n above `whole`
    const f32x2 f = f2_less(f2_less(f2_all(whole), nm), np);     // and the rest
    // the exponent's fraction times ln 2: t + u
    const f32x2 t = f2_mul(f, f2_all(ln2)), nt = f2_mul(f, f2_all(-ln2));
    const f32x2 u = f2_fma(e, f2_all(ln2), f2_fma(f, f2_all(ln2_low), f2_fma(f, f2_all(ln2), nt)));
    const f32x2 q = f2_mul(t, t), q_low = f2_fma(f2_add(t, t), u, f2_fma(t, t, f2_mul(t, nt)));
    f32x2 rest = f2_fma(t, f2_all(1.0f / 40320.0f), f2_all(1.0f / 5040.0f));  // Taylor's series from t^3 / 6 on
    rest = f2_fma(t, rest, f2_all(1.0f / 720.0f));
    rest = f2_fma(t, rest, f2_all(1.0f / 120.0f));
    rest = f2_fma(t, rest, f2_all(1.0f / 24.0f));
    rest = f2_mul(f2_mul(f2_fma(t, rest, f2_all(1.0f / 6.0f)), q), t);
    const f32x2 c = f2_add(t, f2_all(1.0f)), c_low = f2_less(t, f2_add(c, f2_all(-1.0f)));
    const f32x2 half = f2_mul(q, f2_all(0.5f)), d = f2_add(c, half), d_low = f2_less(half, f2_less(d, c));
    // (u times e^t: 1 and t, which is in q_low, and t^2 / 2 and the rest)
    const f32x2 parts = f2_add(f2_add(c_low, d_low), f2_add(f2_fma(f2_all(0.5f), q_low, f2_fma(u, f2_add(half, rest), u)), rest));
    const f32x2 main = f2_add(d, parts), l = f2_less(parts, f2_less(main, d));
    float n0, n1, p0, p1, d0, d1, l0, l1;
    f2_unpack(nm, n0, n1);
    f2_unpack(np, p0, p1);
    const f32x2 unit = f2_pack(__uint_as_float((__float_as_uint(n0) << 23) + 0x3F800000u), __uint_as_float((__float_as_uint(n1) << 23) + 0x3F800000u));
    f2_unpack(f2_mul(main, unit), d0, d1);
    f2_unpack(f2_mul(l, unit), l0, l1);
    const f32x2 v = f2_pack(p0 < 45.0f ? d0 : 0.0f, p1 < 45.0f ? d1 : 0.0f), v_low = f2_pack(p0 < 45.0f ? l0 : 0.0f, p1 < 45.0f ? l1 : 0.0f);
    const f32x2 at_high = f2_add(v, f2_all(kHigh));
    const f32x2 at_low = f2_add(f2_add(f2_less(v, f2_add(at_high, f2_all(-kHigh))), v_low), f2_all(kLow));
    high += static_cast<uint32_t>(at_high) + static_cast<uint32_t>(at_high >> 32);
    low += static_cast<uint32_t>(at_low) + static_cast<uint32_t>(at_low >> 32);
    ++pairs;
  }
  __device__ __forceinline__ uint64_t units() const {
    const uint32_t h = high - 2 * pairs * __float_as_uint(kHigh), l = low - 2 * pairs * __float_as_uint(kLow);
    return (static_cast<uint64_t>(h) << 22) + static_cast<int64_t>(static_cast<int32_t>(l));
  }
};

constexpr int kRanked = 512;      // candidates that are ranked by counting: one a thread,
constexpr int kFew = 128;         // or with a quarter of the others to a thread
struct MergeShared {
  double A[SV_MAX_BEAMS];         // what is added to a beam's x - m
  float score[SV_MAX_BEAMS];      // (out_scores may lie over the scores)
  float m[SV_MAX_BEAMS], high[SV_MAX_BEAMS], low[SV_MAX_BEAMS];  // and A as a pair of floats
  uint8_t exact[SV_MAX_BEAMS];    // A is not to be summed again
  uint8_t live[SV_MAX_BEAMS];     // the beam's logits count
  uint8_t asked[SV_MAX_BEAMS];
  uint64_t key[kRanked], out_key[SV_MAX_BEAM_CANDIDATES + 1];
  uint64_t what[kRanked], out_what[SV_MAX_BEAM_CANDIDATES + 1];
  unsigned long long sum;
  uint32_t bad;
  int again, n, counts[32], rank[kFew];
  uint32_t tops[32];
};

// Totals as integers in their order; 0 is below them all.
__device__ __forceinline__ uint64_t total_key(double t) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(t + 0.0));
  return (b >> 63) ? ~b : b | (uint64_t(1) << 63);
}
__device__ __forceinline__ double total_of_key(uint64_t k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? k & ~(uint64_t(1) << 63) : ~k));
}

// high + low + (x - m), rounded once or twice: the rounding of each sum is kept (Knuth's exact sum).  Sums below float32's range
// are its lowest number.
__device__ __forceinline__ float about_total(float high, float low, float x, float m) {
  const float d = x - m, b = d - x, d_low = (x - (d - b)) - (m + b);
  const float t = high + d, c = t - high;
  const float total = t + (((high - (t - c)) + (d - c)) + (low + d_low));
  return total >= -FLT_MAX ? total : -FLT_MAX;  // (what was lost of an infinite sum is NaN)
}

// What stands for a candidate, in the order of equal totals, the larger first: the lower beam, of its candidates the larger logit
// (a total may have lost what tells two of a beam's logits apart), then the lower token.
constexpr int kTokenBits = 18, kBeamAt = kTokenBits + 32;
constexpr uint32_t kTokenMask = (1u << kTokenBits) - 1u;
__device__ __forceinline__ uint64_t standing(int beam, float x, int token) {
  return static_cast<uint64_t>(SV_MAX_BEAMS - 1 - beam) << kBeamAt | static_cast<uint64_t>(float_key(x)) << kTokenBits | (kTokenMask - static_cast<uint32_t>(token));
}
__device__ __forceinline__ int beam_of(uint64_t what) { return SV_MAX_BEAMS - 1 - static_cast<int>(what >> kBeamAt); }
__device__ __forceinline__ int token_of(uint64_t what) { return static_cast<int>(kTokenMask - (static_cast<uint32_t>(what) & kTokenMask)); }

template <int DT>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const BeamParams a) {
  using E = Elem<DT>;
  extern __shared__ uint32_t about[];  // [W][P][K] the totals in float32, as integers (0 = none)
  __shared__ MergeShared sh;
  pdl_wait();
  const int request = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = static_cast<int64_t>(request) * a.W;
  const int K = a.K, W = a.W, P = a.P, lists = W * P;
  static_assert(SV_MAX_SAMPLE_VOCAB <= 1 << kTokenBits && SV_MAX_BEAMS <= 1 << (64 - kBeamAt), "what stands for a candidate");
  if (tid == 0) sh.bad = 0;
  __syncthreads();
  for (int w = warp; w < W; w += kMergeThreads / 32) {  // one sum of the parts'
    const float score = a.scores[row0 + w];
    if (!(score < INFINITY) && lane == 0) atomicOr(&sh.bad, 1u);
    const bool lives = fabsf(score) <= FLT_MAX && (a.finished == nullptr || a.finished[row0 + w] == 0);
    const Part part = lives && lane < P ? a.parts[(row0 + w) * P + lane] : Part{0, -INFINITY, 0};
    if (__any_sync(0xFFFFFFFFu, part.bad != 0) && lane == 0) atomicOr(&sh.bad, 1u);
    float m = part.m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    float sum = part.m == -INFINITY ? 0.0f : __ull2float_rn(part.sum) * exp2f((part.m - m) * kLog2e);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if (lane == 0) {
      sh.score[w] = score;
      // log of the sum: its exponent's share exact, the fraction's to float32
      const int e = (__float_as_int(sum) >> 23) - 127;
      const float fraction = __int_as_float((__float_as_int(sum) & 0x7FFFFF) | 0x3F800000);
      sh.A[w] = !lives || m == -INFINITY ? static_cast<double>(score)
                                         : static_cast<double>(score) - ((e - kFraction) * 0.69314718055994530942 + static_cast<double>(logf(fraction)));
      sh.m[w] = lives ? m : 0.0f;
      sh.live[w] = lives;
      sh.exact[w] = !lives || m == -INFINITY;  // (a finished beam's total is its score; the others have no candidates)
    }
  }
  __syncthreads();
  if (sh.bad != 0) {
    for (int k = tid; k < K; k += kMergeThreads) {
      a.out_scores[static_cast<int64_t>(request) * K + k] = NAN;
      a.out_rows[static_cast<int64_t>(request) * K + k] = -1;
      a.out_tokens[static_cast<int64_t>(request) * K + k] = -1;
    }
    if (tid == 0) atomicOr(a.status, SV_DEV_BAD_LOGIT);
    return;
  }
  const Entry* entries = a.entries + row0 * P * K;
  // f(list, place, beam) for this thread's candidates: a warp takes a list, or as many short ones as it has lanes for
  const int places = min(32, 1 << (32 - __clz(K - 1))), per_warp = 32 / places;  // (K = 1: 1)
  auto each = [&](auto f) {
#pragma unroll 4
    for (int l0 = warp * per_warp; l0 < lists; l0 += kMergeThreads / 32 * per_warp) {
      const int l = l0 + lane / places;
      if (l < lists)
        for (int i = lane & (places - 1); i < K; i += places) f(l, i, l / P);
    }
  };
  // A candidate: its total, and what stands for it
  auto candidate = [&](int l, int i, int w, uint64_t* key, uint64_t* what) {
    const double A = sh.A[w];
    if (sh.live[w]) {
      const Entry e = entries[l * K + i];
      *key = total_key(A + (static_cast<double>(e.x) - sh.m[w]));
      *what = standing(w, e.x, e.token);
    } else {
      *key = total_key(A);
      *what = standing(w, 0.0f, 0);
    }
  };
  // two beams whose totals nearly agree: their rows are to be summed again, unless that is done
  auto settled = [&](int beam, int other) { return beam == other || (sh.exact[beam] && sh.exact[other]); };
  auto ask = [&](int beam, int other) {
    if (settled(beam, other)) return;
    if (!sh.exact[beam]) sh.asked[beam] = 1;
    if (!sh.exact[other]) sh.asked[other] = 1;
    sh.again = 1;
  };
  for (;;) {
    if (tid < SV_MAX_BEAMS) sh.asked[tid] = 0;
    if (tid == 0) {
      sh.again = 0;
      sh.n = 0;
    }
    if (tid < W) {
      sh.high[tid] = static_cast<float>(sh.A[tid]);
      sh.low[tid] = fabsf(sh.high[tid]) <= FLT_MAX ? static_cast<float>(sh.A[tid] - sh.high[tid]) : 0.0f;
    }
    __syncthreads();
    // totals in float32: off by a step or so, which the bound leaves room for
    uint32_t top = 0;
    int mine = 0;
    each([&](int l, int i, int w) {
      uint32_t key = 0;
      if (sh.live[w]) {
        const Entry e = entries[l * K + i];
        // a part whose part before has K logits at or above this one adds none: they come first
        const bool late = l != w * P && entries[l * K - 1].x >= e.x;
        if (e.token >= 0 && !late) key = float_key(about_total(sh.high[w], sh.low[w], e.x, sh.m[w]));
      } else if (l == w * P && i == 0 && sh.A[w] > -INFINITY) {
        key = float_key(sh.high[w]);
      }
      about[l * K + i] = key;
      top = max(top, key);
      mine += key != 0;
    });
    const uint32_t top_of_warp = __reduce_max_sync(0xFFFFFFFFu, top);
    const int there_of_warp = __reduce_add_sync(0xFFFFFFFFu, mine);
    if (lane == 0) {
      sh.tops[warp] = top_of_warp;
      sh.counts[warp] = there_of_warp;
    }
    __syncthreads();
    const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, lane < kMergeThreads / 32 ? sh.tops[lane] : 0u);
    const int there = __reduce_add_sync(0xFFFFFFFFu, lane < kMergeThreads / 32 ? sh.counts[lane] : 0);
    const int want = min(K + 1, there);
    // the bound: `want` threads' best totals are at or above it, and few more where totals differ; a few steps of float32 below
    uint32_t low = there <= kFew ? 1 : lower_bound_of<kMergeThreads>(top, 1, best, float_key(float_of_key(best) - 8.0f), K + 1, K + 1 + (K >> 2));
    // a thread may have several: further by counting all
    auto count_from = [&](uint32_t bound) {
      int n = 0;
      each([&](int l, int i, int) { n += about[l * K + i] >= bound; });
      n = __reduce_add_sync(0xFFFFFFFFu, n);
      __syncthreads();
      if (lane == 0) sh.counts[warp] = n;
      __syncthreads();
      return __reduce_add_sync(0xFFFFFFFFu, lane < kMergeThreads / 32 ? sh.counts[lane] : 0);
    };
    if (there > kFew) {
      uint32_t over = best + 1;
      for (int n = count_from(low); n > kFew - 16 && over - low > 1;) {
        const uint32_t mid = low + ((over - low) >> 1);
        const int at_mid = count_from(mid);
        if (at_mid >= want) {
          low = mid;
          n = at_mid;
        } else {
          over = mid;
        }
      }
    }
    // totals in float32 may be off by a few steps, and whatever may come before the K-th once its row is summed again counts too
    if (low > float_key(-FLT_MAX)) low = float_key(float_of_key(low) - static_cast<float>(2.0 * kNear));
    low = low > 16 ? low - 16 : 1;
    __syncthreads();
    each([&](int l, int i, int w) {
      if (about[l * K + i] < low) return;
      const int at = atomicAdd(&sh.n, 1);
      if (at < kRanked) candidate(l, i, w, &sh.key[at], &sh.what[at]);
    });
    __syncthreads();
    const int n = sh.n;
    if (n <= kFew) {
      const int i = tid & (kFew - 1), part = tid / kFew;
      if (tid < kFew) sh.rank[tid] = 0;
      __syncthreads();
      if (i < n) {
        const uint64_t key = sh.key[i];
        const uint64_t what = sh.what[i];
        int rank = 0;
#pragma unroll 4
        for (int j = part; j < n; j += kMergeThreads / kFew) rank += sh.key[j] > key || (sh.key[j] == key && sh.what[j] > what);
        atomicAdd(&sh.rank[i], rank);
      }
      __syncthreads();
      if (tid < n && sh.rank[tid] <= K) {
        sh.out_key[sh.rank[tid]] = sh.key[tid];
        sh.out_what[sh.rank[tid]] = sh.what[tid];
      }
    } else if (n <= kRanked) {
      if (tid < n) {
        const uint64_t key = sh.key[tid];
        const uint64_t what = sh.what[tid];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) rank += sh.key[j] > key || (sh.key[j] == key && sh.what[j] > what);
        if (rank <= K) {
          sh.out_key[rank] = key;
          sh.out_what[rank] = what;
        }
      }
    } else {  // long runs of equals: one by one, the (K + 1)-th of another beam than the K-th
      uint64_t before = ~uint64_t(0);
      uint64_t before_what = 0;
      for (int k = 0; k < want; ++k) {
        uint64_t best_key = 0;
        uint64_t best_what = 0;
        const int last = k == K ? beam_of(before_what) : -1;  // past the cut: the best of a beam that the K-th's is to be told from
        each([&](int l, int i, int w) {
          if (about[l * K + i] < low || (last >= 0 && settled(last, w))) return;
          uint64_t key, what;
          candidate(l, i, w, &key, &what);
          if ((key < before || (key == before && what < before_what)) && (key > best_key || (key == best_key && what > best_what))) {
            best_key = key;
            best_what = what;
          }
        });
        sh.key[tid] = best_key;
        sh.what[tid] = best_what;
        for (int d = kMergeThreads / 2; d > 0; d >>= 1) {
          __syncthreads();
          if (tid < d && (sh.key[tid + d] > sh.key[tid] || (sh.key[tid + d] == sh.key[tid] && sh.what[tid + d] > sh.what[tid]))) {
            sh.key[tid] = sh.key[tid + d];
            sh.what[tid] = sh.what[tid + d];
          }
        }
        __syncthreads();
        before = sh.key[0];
        before_what = sh.what[0];
        if (tid == 0) {
          sh.out_key[k] = before;
          sh.out_what[k] = before_what;
        }
        __syncthreads();
      }
    }
    __syncthreads();
    // candidates past the cut, of other beams than the K-th's (more than kRanked: found one by one)
    if (want > K && n <= kRanked && tid < n) {
      const uint64_t key = sh.key[tid], last_key = sh.out_key[K - 1], what = sh.what[tid], last_what = sh.out_what[K - 1];
      if ((key < last_key || (key == last_key && what < last_what)) && total_of_key(last_key) - total_of_key(key) < kNear)
        ask(beam_of(last_what), beam_of(what));
    }
    for (int k = tid; k < K; k += kMergeThreads) {
      const bool some = k < want;
      const uint64_t key = some ? sh.out_key[k] : 0;
      const uint64_t what = some ? sh.out_what[k] : 0;
      const int beam = beam_of(what);
      const int64_t at = static_cast<int64_t>(request) * K + k;
      a.out_scores[at] = some ? static_cast<float>(total_of_key(key)) : -INFINITY;
      a.out_rows[at] = some ? static_cast<int32_t>(row0) + beam : -1;
      a.out_tokens[at] = !some ? -1 : sh.live[beam] ? token_of(what) : a.pad;
      if (k + 1 < want && total_of_key(key) - total_of_key(sh.out_key[k + 1]) < kNear) ask(beam, beam_of(sh.out_what[k + 1]));
    }
    __syncthreads();
    if (sh.again == 0) return;
    // the rows in question once more
    for (int w = 0; w < W; ++w) {
      if (!sh.asked[w]) continue;
      if (tid == 0) sh.sum = 0;
      __syncthreads();
      const Row r = row_of<DT>(a, row0 + w);
      const float m = sh.m[w];
      ExactSum exact;
      uint4 next = tid < r.vecs ? load_vec<DT>(r, tid) : make_uint4(0, 0, 0, 0);
#pragma unroll 1
      for (int v = tid; v < r.vecs; v += kMergeThreads) {
        const uint4 x = next;
        if (v + kMergeThreads < r.vecs) next = load_vec<DT>(r, v + kMergeThreads);
        const uint32_t* p = reinterpret_cast<const uint32_t*>(&x);
#pragma unroll
        for (int j = 0; j < 4; j += DT == SV_BF16 ? 1 : 2)
          exact.add(DT == SV_BF16 ? f2_pack(bf16_lo(p[j]), bf16_hi(p[j])) : f2_pack(__uint_as_float(p[j]), __uint_as_float(p[j + 1])), f2_all(m));
      }
      uint64_t sum = exact.units();
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
      if (lane == 0) atomicAdd(&sh.sum, static_cast<unsigned long long>(sum));
      __syncthreads();
      if (tid == 0) {
        sh.A[w] = static_cast<double>(sh.score[w]) - log(static_cast<double>(sh.sum) * 0x1p-44);
        sh.exact[w] = 1;
      }
      __syncthreads();
    }
  }
}

// ---- host --------------------------------------------------------------------------------------------
// Parts of a row: as many as give every CTA that fits on the GPU one, each of a piece per warp at least.
constexpr int kCtas = kRowCtas * 152;
int most_parts(int V) {
  const int pieces = (V + 7 + kPiece * 4 - 1) / (kPiece * 4);  // (of float32: the most there are)
  return std::max(1, std::min(kMaxParts, pieces / kWarps));
}
int parts_of(int rows, int V) { return std::max(1, std::min(most_parts(V), kCtas / rows)); }
// ... and as many as the merge's shared memory has room for.
constexpr int kMerged = 8192;     // candidates of a request's beams and parts: more take longer to merge than a row's further parts save
int parts_of(int rows, int V, int W, int K) { return std::max(1, std::min(parts_of(rows, V), kMerged / (W * K))); }
struct BeamLayout {
  size_t parts, entries, total;
};
// Sizes for the most parts that any number of rows up to this one has: a workspace serves every call of no more rows, vocabulary
// and candidates.
BeamLayout layout_of(int rows, int V, int K) {
  const size_t n = std::max(static_cast<size_t>(rows), std::min<size_t>(kCtas, static_cast<size_t>(rows) * most_parts(V)));
  BeamLayout L;
  L.parts = SV_STATUS_BYTES;
  L.entries = L.parts + ((sizeof(Part) * n + 255) & ~size_t(255));
  L.total = L.entries + ((sizeof(Entry) * n * K + 255) & ~size_t(255));
  return L;
}
bool valid_sizes(int rows, int V, int K) {
  return rows >= 0 && rows <= SV_MAX_BEAM_ROWS && V >= 1 && V <= SV_MAX_SAMPLE_VOCAB && K >= 1 && K <= SV_MAX_BEAM_CANDIDATES;
}

template <int DT>
cudaError_t launch_beam(const BeamParams& a, int B, void* stream) {
  constexpr int kPerPiece = kPiece * Elem<DT>::kPerVec;
  auto bytes = [](int V, int P) {  // a part's pieces, rounded up
    const int pieces = (V + Elem<DT>::kPerVec - 1 + kPerPiece - 1) / kPerPiece;
    return sizeof(Shared) + sizeof(float) * 32 * ((pieces + P - 1) / P);
  };
  cudaError_t e = allow_smem<rows_kernel<DT>>(bytes(SV_MAX_SAMPLE_VOCAB, 1));
  if (e != cudaSuccess) return e;
  e = launch_dependent(rows_kernel<DT>, dim3(static_cast<unsigned>(a.rows) * a.P), kThreads, bytes(a.V, a.P), stream, SV_KERNEL_BEAM, 1, a);
  if (e != cudaSuccess) return e;
  e = allow_smem<merge_kernel<DT>>(4 * kMerged);
  if (e != cudaSuccess) return e;
  return launch_dependent(merge_kernel<DT>, dim3(B), kMergeThreads, 4 * static_cast<size_t>(a.W) * a.P * a.K, stream, SV_KERNEL_BEAM_MERGE, 1, a);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t sv_beam_workspace_size(int rows, int V, int K) { return valid_sizes(rows, V, K) ? layout_of(std::max(rows, 1), V, K).total : 0; }

sv_status sv_beam_select(const void* logits, int64_t row_stride, sv_dtype dt, int B, int W, int V, const float* scores,
                         const int32_t* finished, int pad, int K, float* out_scores, int32_t* out_rows,
                         int32_t* out_tokens, void* ws, size_t ws_bytes, void* stream) {
  if (dt != SV_BF16 && dt != SV_F32) return set_error(SV_ERR_INVALID_ARG, "dt=%d", static_cast<int>(dt));
  if (B < 0 || W < 1 || W > SV_MAX_BEAMS) return set_error(SV_ERR_INVALID_ARG, "B=%d W=%d: B >= 0 and W in [1, %d] are needed", B, W, SV_MAX_BEAMS);
  if (static_cast<int64_t>(B) * W > SV_MAX_BEAM_ROWS || !valid_sizes(B * W, V, K))
    return set_error(SV_ERR_INVALID_ARG, "B * W=%lld V=%d K=%d: at most %d, %d and %d", (long long)B * W, V, K, SV_MAX_BEAM_ROWS,
                     SV_MAX_SAMPLE_VOCAB, SV_MAX_BEAM_CANDIDATES);
  if (pad < 0) return set_error(SV_ERR_INVALID_ARG, "pad=%d: must be >= 0", pad);
  if (B == 0) return SV_OK;
  if (logits == nullptr || scores == nullptr || out_scores == nullptr || out_rows == nullptr || out_tokens == nullptr)
    return set_error(SV_ERR_INVALID_ARG, "logits / scores / out_scores / out_rows / out_tokens is NULL");
  if ((reinterpret_cast<uintptr_t>(logits) & (dt == SV_BF16 ? 1u : 3u)) != 0)
    return set_error(SV_ERR_INVALID_ARG, "logits are not aligned to their element size");
  if (row_stride < V) return set_error(SV_ERR_INVALID_ARG, "row_stride=%lld is less than V=%d", (long long)row_stride, V);
  const sv_status s = check_workspace(ws, ws_bytes, sv_beam_workspace_size(B * W, V, K));
  if (s != SV_OK) return s;
  const BeamLayout L = layout_of(B * W, V, K);
  unsigned char* w = static_cast<unsigned char*>(ws);
  BeamParams a = {};
  a.logits = logits;
  a.row_stride = row_stride;
  a.scores = scores;
  a.finished = finished;
  a.out_scores = out_scores;
  a.out_rows = out_rows;
  a.out_tokens = out_tokens;
  a.parts = reinterpret_cast<Part*>(w + L.parts);
  a.entries = reinterpret_cast<Entry*>(w + L.entries);
  a.status = reinterpret_cast<uint32_t*>(w);
  a.W = W;
  a.V = V;
  a.K = K;
  a.P = parts_of(B * W, V, W, K);
  a.pad = pad;
  a.rows = B * W;
  return launch_status(dt == SV_BF16 ? launch_beam<SV_BF16>(a, B, stream) : launch_beam<SV_F32>(a, B, stream), "beam select");
}

}  // extern "C"
