// sv_beam_select: one step of beam search, the K best of all beams' continuations.
//
// rows_kernel reads every row of logits once.  A row is cut into parts, one CTA each; a CTA takes its part in pieces of 16 KB
// held in registers, the next one in flight, and keeps
//   the sum of exp(x - ref) for a reference near the part's maximum: float32 terms, compensated sums;
//   a list of candidates for the part's K largest logits.  A bound below the K-th largest lets few of them in: at first the
//   smallest of G >= K groups' largest logits (a group is some threads' logits: K groups have a logit at or above it),
//   later the K-th largest so far, and then only logits above it (an equal one further on comes after it).
// Candidates are ranked by counting.  Pieces with more candidates than the list takes (long runs of equals) are worked off by
// K rounds of a maximum.
//
// merge_kernel, a CTA per request, merges a row's parts, gives each row A = score - log sum exp(x - m), m its largest logit, and merges the
// beams by A + (x - m), all in 64 bits (m apart: next to a large one the rest would be lost), best first.  The float32 terms leave A uncertain by up to about 2^-19 (each term by 2^-22 of ex2
// and a few 2^-24 |y|, y its exponent; of E|y| <= log2 V; compensated sums add next to nothing).  So where the best two beams' totals
// lie within kNear of each other, their rows are summed again with terms in pairs of floats (about 2^-30), and the
// merge starts over: with this the order is that of the exact totals, down to 2^-29.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>

#include "sv_device.cuh"
#include "sv_ops.h"

namespace sv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;                       // 16-byte vectors of a piece per thread
constexpr int kPiece = kThreads * kVecs;       // vectors of a piece
constexpr int kList = 1024;                    // candidates of a part
constexpr int kKeep = 256;                     // listed candidates above which the list is cut to the K best
constexpr int kMaxParts = 32;                  // parts of a row: a lane each in the merge
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kRefSlack = 30.0f;             // how far a logit may lie above a sum's reference
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
  int32_t W, V, K, P, pad, groups;
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
__device__ __forceinline__ void load_piece(const Row& r, int piece, uint4 (&w)[kVecs]) {
  using E = Elem<DT>;
  const int last = (r.lead + r.V) % E::kPerVec != 0 ? r.vecs - 1 : r.vecs;  // vectors from here on are not whole
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int vec = piece * kPiece + i * kThreads + static_cast<int>(threadIdx.x);
    if (vec >= (r.lead != 0 ? 1 : 0) && vec < last) {
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                   : "l"(r.base + static_cast<int64_t>(vec) * 16));
    } else {
      w[i] = vec < r.vecs ? edge_vec<DT>(r, vec) : make_uint4(E::kNone, E::kNone, E::kNone, E::kNone);
    }
  }
}

// Order of candidates as an integer: larger x first, then the lower token.
__device__ __forceinline__ uint64_t order_key(float x, int token) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // (-0 equals 0)
  const uint32_t k = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return (static_cast<uint64_t>(k) << 32) | ~static_cast<uint32_t>(token);
}
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t hi = static_cast<uint32_t>(k >> 32), top = __reduce_max_sync(0xFFFFFFFFu, hi);
  const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, hi == top ? static_cast<uint32_t>(k) : 0u);
  return (static_cast<uint64_t>(top) << 32) | lo;
}
// The next float above x (x finite or -inf).
__device__ __forceinline__ float above(float x) {
  if (x == 0.0f) return __uint_as_float(1u);
  const uint32_t b = __float_as_uint(x);
  return __uint_as_float((b & 0x80000000u) ? b - 1 : b + 1);
}

struct Shared {
  Entry list[2][kList];
  float lowest[kWarps], top[kWarps];
  uint64_t best[kWarps];
  unsigned long long sum;
  int n;
};

// The K best of list[from][0 .. n), in order, into the other half; fewer than K are followed by none.
__device__ __forceinline__ void rank_list(Shared& sh, int from, int n, int K) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Entry e = sh.list[from][i];
    const uint64_t key = order_key(e.x, e.token);
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const Entry o = sh.list[from][j];
      rank += order_key(o.x, o.token) > key;
    }
    if (rank < K) sh.list[from ^ 1][rank] = e;
  }
  for (int i = n + threadIdx.x; i < K; i += kThreads) sh.list[from ^ 1][i] = Entry{-INFINITY, -1};
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 3) rows_kernel(const BeamParams a) {
  using E = Elem<DT>;
  __shared__ Shared sh;
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x / a.P;
  const int part = static_cast<int>(blockIdx.x - row * a.P), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float score = a.scores[row];
  if (!(fabsf(score) <= FLT_MAX) || (a.finished != nullptr && a.finished[row] != 0)) return;  // (the merge looks at neither)
  const Row r = row_of<DT>(a, row);
  const int pieces = (r.vecs + kPiece - 1) / kPiece;
  const int p0 = static_cast<int>(static_cast<int64_t>(pieces) * part / a.P), p1 = static_cast<int>(static_cast<int64_t>(pieces) * (part + 1) / a.P);
  const int K = a.K;
  if (tid == 0) {
    sh.n = 0;
    sh.sum = 0;
  }
  uint4 w[kVecs], next[kVecs];
  if (p0 < p1) load_piece<DT>(r, p0, w);
  float bound = 0.0f;                  // candidates are at or above it
  float ref = -INFINITY, sum = 0.0f, lost = 0.0f, top = -INFINITY;
  int from = 0, listed = 0;            // the list's half, and its length before this piece
  bool first = true;
  for (int piece = p0; piece < p1; ++piece) {
    if (piece + 1 < p1) load_piece<DT>(r, piece + 1, next);
    float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int j = 0; j < E::kPerVec; j += 2) {
        t0 = fmaxf(t0, element<DT>(w, i, j));
        t1 = fmaxf(t1, element<DT>(w, i, j + 1));
      }
    const float mine = fmaxf(t0, t1);
    top = fmaxf(top, mine);
    auto group_bound = [&]() {  // at least K of this piece's logits are at or above it
      float g = mine;
      for (int d = 1; d < kThreads / a.groups; d <<= 1) g = fmaxf(g, __shfl_xor_sync(0xFFFFFFFFu, g, d));
      float low = g, high = g;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, d));
        high = fmaxf(high, __shfl_xor_sync(0xFFFFFFFFu, high, d));
      }
      if (lane == 0) {
        sh.lowest[warp] = low;
        sh.top[warp] = high;
      }
      __syncthreads();
      low = sh.lowest[0];
      high = sh.top[0];
      for (int x = 1; x < kWarps; ++x) {
        low = fminf(low, sh.lowest[x]);
        high = fmaxf(high, sh.top[x]);
      }
      __syncthreads();
      ref = ref == -INFINITY ? high : ref;
      return fmaxf(low, -FLT_MAX);  // (-inf is no candidate)
    };
    if (first) bound = group_bound();
    // the sum
    if (mine > ref + kRefSlack || (ref == -INFINITY && mine > -INFINITY)) {
      const float by = ref == -INFINITY ? 0.0f : exp2f((ref - mine) * kLog2e);
      sum *= by;
      lost *= by;
      ref = mine;
    }
    {
      const float at = ref == -INFINITY ? 0.0f : ref;  // (nothing but -inf so far: terms of 0)
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int j = 0; j < E::kPerVec; ++j) s[j & 3] += ex2_approx((element<DT>(w, i, j) - at) * kLog2e);
      const float y = ((s[0] + s[1]) + (s[2] + s[3])) - lost, now = sum + y;  // Kahan's compensated sum
      lost = (now - sum) - y;
      sum = now;
    }
    // the candidates
    auto collect = [&]() {
      if (!(mine >= bound)) return;
      int n = 0;
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int j = 0; j < E::kPerVec; ++j) n += element<DT>(w, i, j) >= bound;
      int at = atomicAdd(&sh.n, n);
      if (at + n > kList) return;
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int j = 0; j < E::kPerVec; ++j) {
          const float x = element<DT>(w, i, j);
          if (x >= bound) sh.list[from][at++] = Entry{x, (piece * kPiece + i * kThreads + tid) * E::kPerVec + j - r.lead};
        }
    };
    collect();
    int n = 0;
    if (__syncthreads_or(mine >= bound)) {
      n = sh.n;
      if (n > kList && !first) {  // a bound from this piece's own groups
        __syncthreads();
        if (tid == 0) sh.n = listed;
        bound = fmaxf(bound, group_bound());
        collect();
        __syncthreads();
        n = sh.n;
      }
      if (n > kList) {  // the piece's K best, one by one
        uint64_t before = ~uint64_t(0);
        n = listed;
        for (int k = 0; k < K; ++k) {
          uint64_t best = 0;
#pragma unroll
          for (int i = 0; i < kVecs; ++i)
#pragma unroll
            for (int j = 0; j < E::kPerVec; ++j) {
              const float x = element<DT>(w, i, j);
              const uint64_t key = order_key(x, (piece * kPiece + i * kThreads + tid) * E::kPerVec + j - r.lead);
              if (x >= bound && key < before && key > best) best = key;
            }
          best = warp_max(best);
          __syncthreads();
          if (lane == 0) sh.best[warp] = best;
          __syncthreads();
          for (int x = 0; x < kWarps; ++x) best = max(best, sh.best[x]);
          if (best == 0) break;
          before = best;
          if (tid == 0) {
            const uint32_t b = static_cast<uint32_t>(best >> 32);
            sh.list[from][n] = Entry{__uint_as_float((b & 0x80000000u) ? b & 0x7FFFFFFFu : ~b), static_cast<int32_t>(~static_cast<uint32_t>(best))};
          }
          ++n;
        }
        __syncthreads();
      }
      if (n > kKeep || (n >= K && (first || n >= 2 * K))) {
        rank_list(sh, from, n, K);
        from ^= 1;
        n = K;
        __syncthreads();
        bound = above(sh.list[from][K - 1].x);
      }
      if (tid == 0) sh.n = n;
      listed = n;
      __syncthreads();
    }
    first = first && listed < K;   // (until K are listed every logit counts: the bound is -FLT_MAX or this piece's own)
    if (first) bound = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) w[i] = next[i];
  }
  __syncthreads();
  rank_list(sh, from, listed, K);
  // the sum, relative to the part's largest logit
  float high = top;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) high = fmaxf(high, __shfl_xor_sync(0xFFFFFFFFu, high, d));
  if (lane == 0) sh.top[warp] = high;
  __syncthreads();
  high = sh.top[0];
  for (int x = 1; x < kWarps; ++x) high = fmaxf(high, sh.top[x]);
  // a NaN or +inf logit leaves a sum that is not finite
  const bool bad = __syncthreads_or(!(fabsf(sum) <= FLT_MAX) || high == INFINITY);
  if (!bad && ref > -INFINITY) {
    atomicAdd(&sh.sum, __float2ull_rn((sum - lost) * exp2f((ref - high) * kLog2e) * static_cast<float>(1ull << kFraction)));
  }
  __syncthreads();
  const int64_t at = row * a.P + part;
  if (tid == 0) a.parts[at] = Part{sh.sum, high, bad};
  for (int i = tid; i < K; i += kThreads) a.entries[at * K + i] = sh.list[from ^ 1][i];
}

// ---- merge -----------------------------------------------------------------------------------------
// 2^((x - m) log2 e) in units of 2^-44, from pairs of floats (Dekker's and Knuth's exact sums and products): off by about
// 2^-30 of itself and half a unit.
__device__ __forceinline__ uint64_t exact_weight(float x, float m) {
  const float s = x - m, b = s - x, err = (x - (s - b)) - (m + b);            // x - m = s + err
  const float p = s * kLog2e;
  const float e = fmaf(err, kLog2e, fmaf(s, 1.92596299e-8f, fmaf(s, kLog2e, -p)));  // (x - m) log2 e = p + e
  if (!(p > -45.0f)) return 0;
  const float n = rintf(p), f = p - n;
  const float t = f * 0.693147182f;                                           // the exponent's fraction times ln 2: t + u
  const float u = fmaf(e, 0.693147182f, fmaf(f, -1.90465421e-9f, fmaf(f, 0.693147182f, -t)));
  const float q = t * t, q_low = fmaf(2.0f * t, u, fmaf(t, t, -q));
  float rest = fmaf(t, 1.0f / 40320.0f, 1.0f / 5040.0f);                      // Taylor's series from t^3 / 6 on
  rest = fmaf(t, rest, 1.0f / 720.0f);
  rest = fmaf(t, rest, 1.0f / 120.0f);
  rest = fmaf(t, rest, 1.0f / 24.0f);
  rest = fmaf(t, rest, 1.0f / 6.0f) * q * t;
  const float c = 1.0f + t, c_low = t - (c - 1.0f);
  const float d = c + 0.5f * q, d_low = 0.5f * q - (d - c);
  const float low = (c_low + d_low) + (fmaf(0.5f, q_low, u) + rest);
  const float unit = __uint_as_float(static_cast<uint32_t>(127 + 44 + static_cast<int>(n)) << 23);
  return __float2ull_rn(d * unit) + static_cast<uint64_t>(__float2ll_rn(low * unit));
}

struct MergeShared {
  double A[SV_MAX_BEAMS];         // what is added to a beam's x - m
  float m[SV_MAX_BEAMS];
  uint8_t exact[SV_MAX_BEAMS];    // A is not to be summed again
  uint8_t asked[SV_MAX_BEAMS];
  unsigned long long sum;
  uint32_t bad;
  int again;
};

// Totals as integers in their order.
__device__ __forceinline__ uint64_t total_key(double t) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(t + 0.0));
  return (b >> 63) ? ~b : b | (uint64_t(1) << 63);
}
__device__ __forceinline__ double total_of_key(uint64_t k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? k & ~(uint64_t(1) << 63) : ~k));
}

template <int DT>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const BeamParams a) {
  using E = Elem<DT>;
  extern __shared__ Entry lists[];  // [W][K]
  __shared__ MergeShared sh;
  pdl_wait();
  const int request = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = static_cast<int64_t>(request) * a.W;
  const int K = a.K, W = a.W, P = a.P;
  if (tid == 0) sh.bad = 0;
  __syncthreads();
  // a row's parts: one list, one sum
  for (int w = warp; w < W; w += kMergeThreads / 32) {
    const int64_t row = row0 + w;
    const float score = a.scores[row];
    const bool done = a.finished != nullptr && a.finished[row] != 0;
    Entry* list = lists + w * K;
    if (!(score < INFINITY)) {
      if (lane == 0) atomicOr(&sh.bad, 1u);
    }
    if (done || !(fabsf(score) <= FLT_MAX)) {
      for (int i = lane; i < K; i += 32) list[i] = i == 0 && done && score > -INFINITY ? Entry{0.0f, a.pad} : Entry{-INFINITY, -1};
      if (lane == 0) {
        sh.A[w] = score;
        sh.m[w] = 0.0f;
        sh.exact[w] = 1;
      }
      continue;
    }
    Part part = lane < P ? a.parts[row * P + lane] : Part{0, -INFINITY, 0};
    if (__any_sync(0xFFFFFFFFu, part.bad != 0) && lane == 0) atomicOr(&sh.bad, 1u);
    float m = part.m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    double sum = part.m == -INFINITY ? 0.0 : static_cast<double>(part.sum) * exp2f((part.m - m) * kLog2e);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if (lane == 0) {
      sh.A[w] = static_cast<double>(score) - log(sum * (1.0 / static_cast<double>(1ull << kFraction)));
      sh.m[w] = m;
      sh.exact[w] = m == -INFINITY;  // (no candidates)
    }
    const Entry* from = a.entries + row * P * K;
    if (P == 1) {
      for (int i = lane; i < K; i += 32) list[i] = from[i];
      continue;
    }
    // heads of the parts' lists; the one after is on its way
    from += static_cast<int64_t>(lane) * K;
    const Entry none = {-INFINITY, -1};
    Entry head = lane < P ? from[0] : none, after = lane < P && K > 1 ? from[1] : none;
    int taken = 0;
    for (int k = 0; k < K; ++k) {
      const uint64_t key = head.token < 0 ? 0 : order_key(head.x, head.token);
      const uint64_t best = warp_max(key);
      if (best == 0) {
        for (int i = k + lane; i < K; i += 32) list[i] = none;
        break;
      }
      if (key == best) {
        list[k] = head;
        head = after;
        ++taken;
        after = taken + 1 < K ? from[taken + 1] : none;
      }
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
  for (;;) {
    if (tid < SV_MAX_BEAMS) sh.asked[tid] = 0;
    if (tid == 0) sh.again = 0;
    __syncthreads();
    if (warp == 0) {  // lane l has the lists of beams l and l + 32
      int taken[2] = {0, 0};
      uint64_t key[2];
      auto fetch = [&](int h) {
        const int w = lane + 32 * h;
        const Entry e = w < W && taken[h] < K ? lists[w * K + taken[h]] : Entry{-INFINITY, -1};
        key[h] = e.token < 0 ? 0 : total_key(sh.A[w] + (static_cast<double>(e.x) - sh.m[w]));
      };
      fetch(0);
      fetch(1);
      for (int k = 0; k < K; ++k) {
        const uint64_t mine = max(key[0], key[1]), best = warp_max(mine);
        int beam = -1;
        if (best != 0) {
          beam = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, key[0] == best ? lane : key[1] == best ? lane + 32 : INT_MAX));
          // the best of the other beams
          const uint64_t rest = warp_max(max(beam == lane ? 0 : key[0], beam == lane + 32 ? 0 : key[1]));
          if (rest != 0 && total_of_key(best) - total_of_key(rest) < kNear) {
            const double least = total_of_key(best) - kNear;
            bool ask = false;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (key[h] != 0 && total_of_key(key[h]) > least && !sh.exact[lane + 32 * h]) {
                sh.asked[lane + 32 * h] = 1;
                ask = true;
              }
            if (__any_sync(0xFFFFFFFFu, ask) && lane == 0) sh.again = 1;
          }
        }
        if (lane == (beam & 31) || (beam < 0 && lane == 0)) {
          const int64_t at = static_cast<int64_t>(request) * K + k;
          a.out_scores[at] = beam < 0 ? -INFINITY : static_cast<float>(total_of_key(best));
          a.out_rows[at] = beam < 0 ? -1 : static_cast<int32_t>(row0) + beam;
          a.out_tokens[at] = beam < 0 ? -1 : lists[beam * K + taken[beam >> 5]].token;
          if (beam >= 0) {
            ++taken[beam >> 5];
            if (beam < 32) fetch(0);
            else fetch(1);
          }
        }
        __syncwarp();
      }
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
      uint64_t sum = 0;
      const unsigned char* x = r.base + r.lead * E::kBytes;
#pragma unroll 4
      for (int v = tid; v < a.V; v += kMergeThreads) sum += exact_weight(load_logit<DT>(x, v), m);
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
      if (lane == 0) atomicAdd(&sh.sum, static_cast<unsigned long long>(sum));
      __syncthreads();
      if (tid == 0) {
        sh.A[w] = static_cast<double>(a.scores[row0 + w]) - log(static_cast<double>(sh.sum) * 0x1p-44);
        sh.exact[w] = 1;
      }
      __syncthreads();
    }
  }
}

// ---- host --------------------------------------------------------------------------------------------
// Parts of a row: as many as give every CTA that fits on the GPU one, each of a piece at least.
int parts_of(int rows, int V) {
  const int pieces = (V + 7 + kPiece * 4 - 1) / (kPiece * 4);  // (of float32: the most there are)
  return std::max(1, std::min({kMaxParts, pieces, (2 * 152 + rows - 1) / rows}));
}
struct BeamLayout {
  size_t parts, entries, total;
};
BeamLayout layout_of(int rows, int V, int K) {
  const size_t n = static_cast<size_t>(rows) * parts_of(rows, V);
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
  cudaError_t e = launch_dependent(rows_kernel<DT>, dim3(static_cast<unsigned>(B) * a.W * a.P), kThreads, 0, stream, SV_KERNEL_BEAM, 1, a);
  if (e != cudaSuccess) return e;
  e = allow_smem<merge_kernel<DT>>(sizeof(Entry) * SV_MAX_BEAMS * SV_MAX_BEAM_CANDIDATES);
  if (e != cudaSuccess) return e;
  return launch_dependent(merge_kernel<DT>, dim3(B), kMergeThreads, sizeof(Entry) * a.W * a.K, stream, SV_KERNEL_BEAM_MERGE, 1, a);
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
  a.P = parts_of(B * W, V);
  a.pad = pad;
  a.groups = 8;  // a power of two, at least K (at most a group to two threads)
  while (a.groups < K) a.groups *= 2;
  return launch_status(dt == SV_BF16 ? launch_beam<SV_BF16>(a, B, stream) : launch_beam<SV_F32>(a, B, stream), "beam select");
}

}  // extern "C"
