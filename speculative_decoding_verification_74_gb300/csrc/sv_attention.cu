// sv_tree_attention: a token tree's queries against a paged cache.
//
// Rows and tiles.  The query heads that share a key/value head, for as many nodes as fit into 128 rows (the height of
// a tcgen05 product), form a row tile; the cache is read in tiles of 128 slots.  For a row tile, with c = scale
// log2(e) and running maximum m:
//   S = Q K^T          [128 x 128], accumulated in tensor memory
//   P = 2^(c S - m)    bf16, written back to tensor memory over S
//   O = O + P V        in tensor memory
// and at the end o = O / (sum of the rounded P), lse = (m + log2 sum P) ln 2.  O is scaled by 2^(m - m') only when some
// row's maximum has grown by more than 8 (P stays below 2^8, so float32 sums and bf16's range are far from their ends).
//
// Work split.  All (row tile, cache tile) pairs of the batch lie on one line, and before each row tile a few places for what
// beginning and ending it costs; CTA c of C takes the c-th part of the line (a persistent CTA per SM), in segments:
// stretches of one row tile.  A row tile that crosses CTAs leaves partial (O, m, sums) in the workspace, and join_kernel
// adds them.  So one long context and many short ones load the SMs alike.
//
// Few rows.  A row of S belongs to one lane of tensor memory, and a quarter of its lanes to one of the SM's four
// schedulers.  So a tile of at most 64 (32) rows is multiplied with Q's rows two (four) times over, one copy per half (quarter)
// of the lanes, and each copy takes the exponentials of its half (quarter) of the slots; P is 0 elsewhere.  The copies' (O,
// m, sums) are added at the end of a segment, like those of the two groups.
//
// Pairs of heads.  With 64 dimensions a slot of one head is 128 bytes, and the next lies kv_heads * 128 bytes on: too short
// a piece for memory's pace (4.5 of 6.8 TB/s measured).  So two neighbouring heads make one tile of 128 dimensions: Q's rows
// of the first in the lower half of the (copy's) rows and the lower 64 dimensions, those of the second in the upper ones,
// zeros elsewhere; of O each row's own 64 columns count.  The products do the work of 128 dimensions on as many bytes.
//
// Measured (GB300, 32 query and 8 key/value heads of 128; a copy of the cache's bytes in brackets; one call after the other, and a
// graph of one call replayed, whose start takes some 4 us): 64 requests of one token over 6k to 8k slots 279 and 289 us (275), 64
// trees of up to 16 nodes over 512 to 4096 slots 112 and 117 us (92), four chains of 17 over 99k to 131k slots 283 and 295 us
// (278); a window of 1024 with 16 heads of 64, 33 trees 39 and 43 us (19); four requests of one token and up to 130 slots 11.8 and
// 14.4 us.  Long contexts are bound by memory.  A row tile's masked tiles and
// end cost about 4 us besides its tiles (1.5 us each), which short contexts feel; a call's launches, first tile and join
// about 11 us.
//
// Roles in a CTA: warps 0 and 11 copy K and V page by page through a ring of stages (TMA; one warp alone needs
// 1.1 us a tile for it); one thread of warp 1 issues the products; warp 10 brings each segment's description, parents and
// Q; two groups of four warps take the tiles in turn (a thread has a row), each with its own S and O, so one group's
// exponentials run beside the other's products.  P is rounded to bf16, the products' type; o is divided by the sum of
// the rounded P, so its weights add up to 1, and lse takes the sum before rounding.
//
// A cache in 4 bits (kFour) with more rows than sv_attention4.cu's tiles: one warp copies a tile's codes into a ring of their
// own, and four more warps turn them into the stages' K and V, as float16 (exact: a code times its scale has six bits), and Q
// into float16 rows scaled by powers of two.  S and P V are issued by two warps; the one that brings Q finds the segments for all.
// The rest is the same, with P in float16, 2^7 to 2^15 at a row's maximum.  Whole warpgroups share out the registers.
// Measured (graph replay, bytes in 4 bits in brackets): 64 trees 108 us (28), four chains 250 us (78; their products padded to 128
// rows 126).  A tile takes 1.2 us however few its bytes: a warp's decoding 2100 clocks of 2300, the softmax of a group 1900, the
// products 1100, and half of the issue slots are used; a row tile's beginning and end 6 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "sv_decode4.cuh"
#include "sv_device.cuh"
#include "sv_line.cuh"
#include "sv_ops.h"

namespace sv {
namespace {

constexpr int kTile = 128;                 // rows of Q, and slots of the cache, in a tile
constexpr int kGroupThreads = 128;
constexpr int kSoftThreads = 2 * kGroupThreads;
// Warps: the two groups of the softmax are four consecutive ones each.
template <bool kFour>
struct Warps {  // a cache in bf16
  static constexpr int kThreads = 128 + kSoftThreads, kSoft = 2, kK = 0, kMma = 1, kQ = 10, kV = 11, kDecode = 99, kPv = 99;
  static constexpr int kSegments = 2;      // descriptions held at once
};
template <>
struct Warps<true> {  // in 4 bits: whole warpgroups, which share out the registers
  static constexpr int kThreads = 256 + kSoftThreads, kSoft = 4, kK = 2, kMma = 0, kQ = 1, kV = 99, kDecode = 12, kPv = 3;
  static constexpr int kSegments = 4;
};
constexpr int kHalfBytes = kTile * 128;    // 128 slots of 64 bf16: one swizzled column block
constexpr int kTmemColumns = 512;
// Tensor memory by group: S at columns 0 and 128, O from 256 on.  With 128 dimensions P lies over the upper half of S (which is
// read first), so a group's next S waits for its product P V; with 64 there is room for P, and S only waits until the softmax
// has read it.
template <int D>
struct Columns {
  static constexpr bool kOwnP = D == 64;
  static __device__ __forceinline__ constexpr uint32_t s(uint32_t g) { return g * 128; }
  static __device__ __forceinline__ constexpr uint32_t o(uint32_t g) { return 256 + g * D; }
  static __device__ __forceinline__ constexpr uint32_t p(uint32_t g) { return kOwnP ? 384 + g * 64 : g * 128 + 64; }
};
constexpr float kLazyGrowth = 8.0f;        // log2 units by which a maximum may grow without a rescale of O
// In 4 bits P is float16: m lies this far below the maximum, so P is 2^kBias there, 2^(kBias + kLazyGrowth) at most (float16 ends
// at 2^16), and the many small weights beside a large one, which float16 has no bits for below 2^-25, are kept down to 2^-32 of it.
constexpr float kBias = 7.0f;
constexpr int kJoinRows = 16;              // rows per CTA of the join
// What a row tile costs besides its cache tiles, in those: its masked tiles and its end, about 4 us against 1.5 a tile
// (64 trees over 512 to 4096 slots 126 us at 0, 114 at 2, 3 and 4; the window's 33 trees 55.5, 40.7, 40.6 and 41.2).
constexpr int kExtra = 3;
constexpr int kMixFloat4 = 768;            // (a fifth stage of 128 dimensions still fits)
constexpr int kMixFloat4Of4 = 512;         // in 4 bits: at most two copies
// A cache in 4 bits: one warp copies a tile's codes into a ring of their own, and four decode them, each a quarter of its slots,
// eight at a time.  (Sixteen: 64 trees 123 us against 113; the roles' code together has to fit into the instruction cache.)
constexpr int kRawSlots = 8;
constexpr int kMaxRaw = 2;                 // (beside four stages four chains over 131k take 260 us; with 1 323, with 2 and three stages 313, 3 and three 330)
constexpr int kMaxStages = 12;
struct AttendParams : Line, Marks, Outputs {
  const int32_t *table, *parent;
  Job* jobs;          // [grid]
  float* parts;       // [2 grid] partial results
  int32_t pages, kv_heads;
  int32_t tile_nodes;  // nodes of a row tile
  int32_t units;       // key/value heads, or pairs of them
  int32_t half_rows;   // rows of a copy that one head takes
  uint32_t over_group; // ceil(2^16 / group)
  int32_t stages;
  float scale;         // with the cache's k_scale
  float v_scale;
  // a cache in 4 bits: the layer's pool, and the places of the codes' ring
  const unsigned char* pool;
  int64_t page_stride, head_stride;
  int32_t raw_stages;
};

// Floats of one partial result: O as [D / 4][128 rows][4], then m and the two sums per row.
template <int D>
constexpr int part_floats() { return kTile * D + 3 * kTile; }

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
// Instruction descriptor: float32 accumulator, bf16 (or float16) operands, M = 128.
constexpr uint32_t instr_desc(int n, bool b_rows_are_k, bool f16 = false) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_rows_are_k ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(kTile >> 4) << 24);
}

// True in one thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
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
// After the wait, loaded registers may be used: the empty statements keep their uses behind it.
template <int N>
__device__ __forceinline__ void tmem_loaded(uint32_t (&x)[N]) {
  tmem_wait_load();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(x[i]));
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : SV_R8(x, 0), SV_R8(x, 8)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_load8(uint32_t addr, uint32_t* x) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : SV_R8(x, 0) : "r"(addr));
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::SV_I8(x, 0),
      SV_I8(x, 8), "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void lds64(uint32_t at, uint32_t& a, uint32_t& b) {
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
// Registers of this warpgroup's threads from here on.
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// row / group for row < 128, group <= 128: over = ceil(2^16 / group).
__device__ __forceinline__ int over_group(int row, uint32_t over) { return static_cast<int>((row * over) >> 16); }

// The part of shared memory with a fixed size; then come the tiles before each request [B], the parents of some segments'
// trees [kSegments][Nmax] and, 1024-byte aligned, Q and the ring.
static_assert(kMaxRaw == 2 && kMaxStages <= 32, "the barriers' threads");
template <bool kFour>
struct Smem {
  Line line;
  Segment seg[Warps<kFour>::kSegments];             // segments' descriptions in turn
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t raw_full[kFour ? kMaxRaw : 1], raw_empty[kFour ? kMaxRaw : 1];  // a tile's codes are there, are decoded
  uint64_t q_raw[2];           // in 4 bits, by the segment's parity: its Q is there in bf16
  uint64_t q_full[2];          // by the segment's parity: its Q and description are there
  uint64_t q_free;             // once per segment: its last S is complete
  uint64_t seg_there[kFour ? Warps<kFour>::kSegments : 1];  // in 4 bits: a description is there
  uint64_t seg_free[Warps<kFour>::kSegments];  // every softmax thread is done with a description
  uint64_t s_full[2], p_full[2], pv_done[2];  // by group
  uint64_t sums_full, o_free;  // once per segment: the groups' sums are there; every thread has read O
  uint64_t mix_full[2], mix_free[2];  // by group: copies' columns written, read
  float m[2][2][kTile], l[2][2][kTile], lr[2][2][kTile];  // by the segment's parity and group
  float q_size[kFour ? 2 : 1][kFour ? kTile : 1];  // by the segment's parity: what a row of Q was divided by
  float4 mix[2][kFour ? kMixFloat4Of4 : kMixFloat4];   // by group: columns that the copies exchange, four columns of all rows together
  uint32_t scan[Warps<kFour>::kThreads / 32];
  uint32_t tmem;
  volatile int32_t dead;       // a wait ran out: everyone leaves
};

// A place in the ring of stages and the parity of its present round.
struct Ring {
  uint32_t stage = 0, parity = 0;
  __device__ __forceinline__ void step(uint32_t stages) {
    if (++stage == stages) {
      stage = 0;
      parity ^= 1;
    }
  }
};

template <int D, bool kPair, int kCopies, bool kFour>
__global__ void __launch_bounds__(Warps<kFour>::kThreads, 1)
    attend_kernel(const AttendParams a, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map) {
  constexpr int W = kPair ? 2 * D : D;  // dimensions of a tile
  using Col = Columns<W>;
  using Role = Warps<kFour>;
  constexpr int kThreads = Role::kThreads;
  constexpr int kHalves = W / 64;
  constexpr int kHalfRows = kTile / kCopies / (kPair ? 2 : 1);
  constexpr int kStageBytes = kHalves * kHalfBytes;
  extern __shared__ unsigned char dyn[];
  __shared__ Smem<kFour> sm;
  uint32_t* before = reinterpret_cast<uint32_t*>(dyn);           // [B]
  int32_t* parents = reinterpret_cast<int32_t*>(dyn) + a.B;      // [segments' descriptions][Nmax]
  unsigned char* q_buf = dyn + 4 * (a.B + Role::kSegments * a.Nmax);
  q_buf += (1024u - (smem_u32(q_buf) & 1023u)) & 1023u;
  unsigned char* ring = q_buf + kHalves * kHalfBytes;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // (known to be the same in all lanes)
  // (a few barriers a thread: by one thread they take 1 to 2 us)
  if (tid < a.stages) {
    mbar_init(&sm.full[tid], kFour ? 128 : 1);
    mbar_init(&sm.empty[tid], 1);
  } else if (tid >= 32 && tid < 34) {
    const int i = tid - 32;
    mbar_init(&sm.q_raw[i], 1);
    mbar_init(&sm.q_full[i], kFour ? 128 : 1);
    mbar_init(&sm.mix_full[i], kGroupThreads);
    mbar_init(&sm.mix_free[i], kGroupThreads);
  } else if (tid >= 64 && tid < 66) {
    const int i = tid - 64;
    mbar_init(&sm.s_full[i], 1);
    mbar_init(&sm.p_full[i], kGroupThreads);
    mbar_init(&sm.pv_done[i], 1);
    if constexpr (kFour) {
      mbar_init(&sm.raw_full[i], 1);
      mbar_init(&sm.raw_empty[i], 4);
    }
  } else if (tid == 96) {
    mbar_init(&sm.q_free, 1);
    mbar_init(&sm.sums_full, kSoftThreads);
    mbar_init(&sm.o_free, kSoftThreads);
  } else if (tid >= 97 && tid < 97 + Role::kSegments) {
    mbar_init(&sm.seg_free[tid - 97], kSoftThreads);
    if constexpr (kFour) mbar_init(&sm.seg_there[tid - 97], 1);
  }
  if (tid < 128) {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (tid == 0) {
    sm.dead = 0;
    sm.line = a;
  }
  if constexpr (kPair) {  // the other head's dimensions: never written again
    for (int i = tid; i < kHalves * kHalfBytes / 16; i += kThreads) reinterpret_cast<uint4*>(q_buf)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (warp == Role::kMma) tmem_alloc(&sm.tmem);
  pdl_wait();
  pdl_trigger();
  // tiles before each request
  uint32_t total;
  {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int i0 = min(a.B, tid * per), i1 = min(a.B, i0 + per);
    uint32_t sum = 0;
    for (int i = i0; i < i1; ++i) {
      const Request r = request_of<kTile>(a, i);
      if (r.bad != 0 && blockIdx.x == 0) mark_bad(a, i, r.bad);
      before[i] = sum;
      sum += static_cast<uint32_t>(r.tiles + a.extra) * r.mtiles * a.units;
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
    for (int i = i0; i < i1; ++i) before[i] += at;
    __syncthreads();
  }
  const uint32_t tmem = sm.tmem;
  // with fewer places than CTAs the last CTAs have none
  const Parts parts(total, max(1u, min(gridDim.x, total)));
  const uint32_t t0 = min(parts.begin(blockIdx.x), total), t1 = min(parts.begin(blockIdx.x + 1), total);
  Segment opening = {};
  if (t0 < t1) opening = segment_at<kTile, kFour>(sm.line, before, t0, t1);
  const bool some = opening.kv0 < opening.kv1;
  // a part's stretches but the first begin a row tile; the last may hold none of its cache tiles
  auto stretch_at = [&](uint32_t t) { return t == t0 ? some : t + a.extra < t1; };
  const uint32_t stages = a.stages;
  uint32_t loaded = 0, segments = 0;  // stages and Q's that were asked for

  // In 4 bits only one warp finds the segments, and the others read its descriptions (code that is in line for every role does
  // not fit into the instruction cache).  k: the segment's number in this CTA.
  constexpr int kSegMask = Role::kSegments - 1;
  [[maybe_unused]] auto described = [&](uint32_t k, Segment* s) {
    if (k == 0) {
      *s = opening;
      return true;
    }
    if (!warp_wait<kFour>(&sm.seg_there[k & kSegMask], (k / Role::kSegments) & 1, &sm.dead, a.status)) return false;
    *s = sm.seg[k & kSegMask];
    return true;
  };

  [[maybe_unused]] auto copies = [&]() {
    // ---- copies -----------------------------------------------------------------------------------
    const int box_shift = min(7, a.shift), box = 1 << box_shift;  // slots per copy: a page, or 128 slots of one
    const int chunks = kTile >> box_shift;
    bool go = true;
    const uint32_t second = warp == Role::kV;  // K's and V's stages alternate (in 4 bits they come together)
    const CUtensorMap* map = second ? &v_map : &k_map;
    const uint32_t places = kFour ? a.raw_stages : stages;
    Ring at;
    if (second) at.step(stages);
    loaded = second;
    // page numbers of 32 copies at a time (a copy's page: lane = its number in the block), one block ahead
    auto pages_of = [&](const Segment& s, int block) {
      const int64_t slot = (static_cast<int64_t>(block) * 32 + lane) << box_shift;
      return slot < s.r.len + s.r.nodes ? a.table[static_cast<int64_t>(s.request) * a.width + (slot >> a.shift)] : -1;
    };
    Segment s = {}, next = {};  // the next segment and its first pages are looked up while the ring is full
    int block = 0, page_now = -1, page_next = -1, next_block = 0, next_now = -1;
    [[maybe_unused]] uint32_t segment = 0;
    if (some) {
      s = opening;
      block = tile_slot<kTile>(s.r, s.kv0) >> (box_shift + 5);
      page_now = pages_of(s, block);
    }
    for (uint32_t t = t0; stretch_at(t) && go;) {
      const int end = s.r.len + s.r.nodes, lo = a.window > 0 ? max(0, s.r.len - a.window + 1) : 0;
      const uint32_t after = s.next;
      page_next = pages_of(s, block + 1);
      for (int j = s.kv0; j < s.kv1 && go; ++j) {
        const int s0 = tile_slot<kTile>(s.r, j);
        const int need = s0 >> (box_shift + 5);
        if (need != block) {
          page_now = need == block + 1 ? page_next : pages_of(s, need);
          block = need;
          page_next = pages_of(s, block + 1);
        }
        // lane x < chunks copies the x-th page's part; a page without a visible slot is left out
        const int slot = s0 + (lane << box_shift);
        int page = __shfl_sync(0xFFFFFFFFu, page_now, ((s0 >> box_shift) + lane) & 31);
        const bool wanted = lane < chunks && slot < end && (a.window <= 0 || slot < a.sinks || slot + box > lo);
        if (wanted && (page < 0 || page >= a.pages)) {
          mark_bad(a, s.request, SV_DEV_BAD_PAGE);
          page = a.pages;  // outside the tensor: the copy fills zeros
        }
        if constexpr (kFour) {
          constexpr int kHeads = kPair ? 2 : 1, kSlotBytes = 9 * D / 8;
          const bool there = wanted && page < a.pages;
          const int bytes = __popc(__ballot_sync(0xFFFFFFFFu, there)) * kHeads * box * kSlotBytes;
          if (loaded >= places) go = warp_wait<kFour>(&sm.raw_empty[at.stage], at.parity ^ 1, &sm.dead, a.status);
          if (!go) break;
          if (lane == 0) mbar_arrive_expect_tx(&sm.raw_full[at.stage], bytes);
          __syncwarp();
          if (there) {
#pragma unroll
            for (int h = 0; h < kHeads; ++h)
              bulk_g2s(ring + stages * kStageBytes + (at.stage * kHeads + h) * kTile * kSlotBytes + (lane << box_shift) * kSlotBytes,
                       a.pool + page * a.page_stride + (kHeads * s.head + h) * a.head_stride + (slot & ((1 << a.shift) - 1)) * kSlotBytes,
                       box * kSlotBytes, &sm.raw_full[at.stage]);
          }
          ++loaded;
          at.step(places);
        } else {
          const int bytes = __popc(__ballot_sync(0xFFFFFFFFu, wanted)) * kHalves * box * 128;
          if (loaded >= stages) go = warp_wait<kFour>(&sm.empty[at.stage], at.parity ^ 1, &sm.dead, a.status);
          if (!go) break;
          if (lane == 0) mbar_arrive_expect_tx(&sm.full[at.stage], bytes);
          __syncwarp();
          if (wanted) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              tma_load_4d(ring + at.stage * kStageBytes + h * kHalfBytes + (lane << box_shift) * 128, map, kPair ? 0 : h * 64,
                          kPair ? 2 * s.head + h : s.head,
                          slot & ((1 << a.shift) - 1), page, &sm.full[at.stage]);
          }
          loaded += 2;
          at.step(stages);
          at.step(stages);
        }
        if (j == max(s.kv0, s.kv1 - 2) && stretch_at(after)) {
          if constexpr (kFour) {
            if (go = described(++segment, &next); !go) break;
          } else {
            next = segment_at<kTile>(sm.line, before, after, t1);
          }
          next_block = tile_slot<kTile>(next.r, next.kv0) >> (box_shift + 5);
          next_now = pages_of(next, next_block);
        }
      }
      t = after;
      s = next;
      block = next_block;
      page_now = next_now;
    }
  };
  auto queries = [&]() {
    // ---- segments: description, parents, Q --------------------------------------------------------
    constexpr int rows_apart = kTile / kCopies;
    // the k-th segment's description, once the softmax is done with the one that lay there
    auto describe = [&](uint32_t k, const Segment& s) {
      const uint32_t slot = k & kSegMask;
      if (k >= Role::kSegments && !warp_wait<kFour>(&sm.seg_free[slot], (k / Role::kSegments - 1) & 1, &sm.dead, a.status)) return false;
      if (a.parent != nullptr)
        for (int x = lane; x < s.r.nodes; x += 32) parents[slot * a.Nmax + x] = a.parent[s.r.first + x];
      if (lane == 0) sm.seg[slot] = s;
      return true;
    };
    [[maybe_unused]] uint32_t told = 0, tell_t = t0;
    for (uint32_t t = t0; stretch_at(t); ++segments) {
      Segment s;
      if constexpr (kFour) {  // descriptions run one ahead of Q, but for the first
        bool go = true;
        while (go && told < segments + (segments > 0 ? 2 : 1) && stretch_at(tell_t)) {
          const Segment one = told == 0 ? opening : segment_at<kTile, kFour>(sm.line, before, tell_t, t1);
          go = describe(told, one);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.seg_there[told & kSegMask]);
          ++told;
          tell_t = one.next;
        }
        if (!go) break;
        s = sm.seg[segments & kSegMask];
        // what belongs to Q is there twice: every softmax thread has to be done with the segment before the last one
        if (segments >= 2 && !warp_wait<kFour>(&sm.seg_free[(segments - 2) & kSegMask], ((segments - 2) / Role::kSegments) & 1, &sm.dead, a.status)) break;
      } else {
        s = t == t0 ? opening : segment_at<kTile>(sm.line, before, t, t1);
        if (!describe(segments, s)) break;
      }
      if (segments >= 1 && !warp_wait<kFour>(&sm.q_free, (segments - 1) & 1, &sm.dead, a.status)) break;
      __syncwarp();
      if (lane == 0) {
        uint64_t* there = kFour ? &sm.q_raw[segments & 1] : &sm.q_full[segments & 1];
        mbar_arrive_expect_tx(there, kCopies * kHalves * a.tile_nodes * a.group * 128);
        for (int copy = 0; copy < kCopies; ++copy)
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            tma_load_3d(q_buf + h * kHalfBytes + (copy * rows_apart + (kPair ? h * kHalfRows : 0)) * 128, &q_map,
                        kPair ? 0 : h * 64, (kPair ? 2 * s.head + h : s.head) * a.group,
                        static_cast<int>(s.r.first) + s.mtile * a.tile_nodes, there);
      }
      t = s.next;
    }
  };
  // ---- products -----------------------------------------------------------------------------------
  // The whole warp runs these loops, so counters and descriptors stay in uniform registers, which tcgen05.mma takes its
  // operands from; one elected thread issues.  Descriptors go by addition: their low words count 16-byte units of shared memory.
  constexpr uint32_t kDescS = instr_desc(kTile, false, kFour), kDescO = instr_desc(W, true, kFour);
  const uint64_t q_desc0 = smem_desc(smem_u32(q_buf), 16, 1024), k_desc0 = smem_desc(smem_u32(ring), 16, 1024),
                 v_desc0 = smem_desc(smem_u32(ring), kHalfBytes, 1024);
  // S of tile n from a stage of K; the segment's last one frees Q
  auto issue_s = [&](bool elected, uint32_t n, uint32_t stage, bool last) {
    tc_after_sync();
    const uint64_t k_desc = k_desc0 + stage * (kStageBytes >> 4);
    const uint32_t d = tmem + Col::s(n & 1);
    if (elected) {
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss(d, q_desc0 + h * (kHalfBytes >> 4) + 2 * k, k_desc + h * (kHalfBytes >> 4) + 2 * k, kDescS, h + k > 0);
      tc_commit(&sm.s_full[n & 1]);
      tc_commit(&sm.empty[stage]);
      if (last) tc_commit(&sm.q_free);
    }
  };
  // P V of tile i, the segment's j-th, from a stage of V
  auto issue_pv = [&](bool elected, uint32_t i, uint32_t stage, int j) {
    tc_after_sync();
    const uint64_t v_desc = v_desc0 + stage * (kStageBytes >> 4);
    const uint32_t d = tmem + Col::o(i & 1), p = tmem + Col::p(i & 1);
    const uint32_t more = j > 1;
    if (elected) {
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k) mma_ts(d, p + 8 * k, v_desc + k * (2048 >> 4), kDescO, k > 0 ? 1u : more);
      tc_commit(&sm.pv_done[i & 1]);
      tc_commit(&sm.empty[stage]);
    }
  };
  auto ready = [](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity)); };
  [[maybe_unused]] auto products = [&]() {
    if (some) {
      const bool elected = elect_one();
      bool more = true;                   // S's are left
      Ring ks, vs;  // K's and V's stages alternate
      vs.step(stages);
      uint32_t s_seg = 0, p_seg = 0;      // segments of the next S and the next P V
      int s_left = 0, p_tiles = 0, p_j = 0;
      uint32_t n = 0, i = 0;  // tiles of the next S and the next P V: whichever is ready is issued, so neither waits
                              // behind the other's barriers
      uint32_t idle = 0;
      uint64_t began = 0;
      while (more || i < n) {
        bool issued = false;
        if (more) {
          if (s_left == 0 && ready(&sm.q_full[s_seg & 1], (s_seg >> 1) & 1))
            s_left = __shfl_sync(0xFFFFFFFFu, sm.seg[s_seg & 1].kv1 - sm.seg[s_seg & 1].kv0, 0);
          // The group's S was last read by the softmax, or by the product P V, of tile n - 2.  Parities tell a stage's fills apart
          // only while the one before has been seen: with an odd number of stages that is a tile's V, whose product comes first.
          if (s_left > 0 && 2 * i + stages > 2 * n && ready(&sm.full[ks.stage], ks.parity) &&
              (n < 2 || ready(Col::kOwnP ? &sm.p_full[n & 1] : &sm.pv_done[n & 1], ((n - 2) >> 1) & 1))) {
            --s_left;
            issue_s(elected, n, ks.stage, s_left == 0);
            ks.step(stages);
            ks.step(stages);
            if (s_left == 0) more = stretch_at(__shfl_sync(0xFFFFFFFFu, sm.seg[s_seg & 1].next, 0));
            s_seg += s_left == 0;
            ++n;
            issued = true;
          }
        }
        if (i < n) {
          if (p_j == p_tiles) {
            p_tiles = __shfl_sync(0xFFFFFFFFu, sm.seg[p_seg & 1].kv1 - sm.seg[p_seg & 1].kv0, 0);
            p_j = 0;
            ++p_seg;
          }
          // (at a segment's first tile both groups' O of the segment before have been read)
          if (ready(&sm.p_full[i & 1], (i >> 1) & 1) && ready(&sm.full[vs.stage], vs.parity) &&
              (p_j > 0 || p_seg < 2 || ready(&sm.o_free, (p_seg - 2) & 1))) {
            issue_pv(elected, i, vs.stage, p_j);
            vs.step(stages);
            vs.step(stages);
            ++p_j;
            ++i;
            issued = true;
          }
        }
        idle = issued ? 0 : idle + 1;
        if ((idle & 1023u) == 1023u && !__all_sync(0xFFFFFFFFu, still_waiting<kFour>(&began, &sm.dead, a.status))) break;
        if (issued) began = 0;
      }
    }
    __syncwarp();
  };
  // In 4 bits two warps issue, one S and one P V, each behind its own barriers (four chains 260 us by one warp, 250 by two).  With
  // an odd ring S waits for the product of two tiles before even where S itself could go: its stage may have held that tile's V.
  [[maybe_unused]] auto half_of_products = [&](auto of_values) {
    constexpr bool kPv = decltype(of_values)::value;
    if (some) {
      const bool elected = elect_one();
      // (by polling: a sleeping warp wakes late)
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        uint64_t began = 0;
        bool there = true;
        for (uint32_t it = 1; there && !mbar_test_wait(bar, parity); ++it)
          if ((it & 1023u) == 0) there = still_waiting<kFour>(&began, &sm.dead, a.status);
        return __all_sync(0xFFFFFFFFu, there) != 0;
      };
      Ring at;
      if (kPv) at.step(stages);
      uint32_t n = 0, seg = 0;
      bool go = true;
      for (uint32_t t = t0; go && stretch_at(t); ++seg) {
        if (go = wait(&sm.q_full[seg & 1], (seg >> 1) & 1); !go) break;
        const Segment& s = sm.seg[seg & kSegMask];
        const int tiles = __shfl_sync(0xFFFFFFFFu, s.kv1 - s.kv0, 0);
        t = __shfl_sync(0xFFFFFFFFu, s.next, 0);
        for (int j = 0; j < tiles && go; ++j, ++n) {
          if constexpr (kPv) {  // (at a segment's first tile both groups' O of the segment before have been read)
            go = (j > 0 || seg == 0 || wait(&sm.o_free, (seg - 1) & 1)) && wait(&sm.p_full[n & 1], (n >> 1) & 1) && wait(&sm.full[at.stage], at.parity);
            if (go) issue_pv(elected, n, at.stage, j);
          } else {
            go = (n < 2 || wait(Col::kOwnP && (stages & 1) == 0 ? &sm.p_full[n & 1] : &sm.pv_done[n & 1], ((n - 2) >> 1) & 1)) && wait(&sm.full[at.stage], at.parity);
            if (go) issue_s(elected, n, at.stage, j + 1 == tiles);
          }
          at.step(stages);
          at.step(stages);
        }
      }
    }
    __syncwarp();
  };
  [[maybe_unused]] auto decode = [&]() {
    // ---- decoding: codes times scales into the stages, as float16 (exact: six bits) -----------------------
    // And Q: each row is scaled by a power of two so that its largest element lies in [2^14, 2^15), where elements down to
    // 2^-28 of it keep all bits of their bf16.
    if constexpr (kFour) {
      constexpr int kHeads = kPair ? 2 : 1, kGroupBytes = 9 * D, kHeadBytes = kTile / 8 * kGroupBytes;
      constexpr int kWords = D / 32;   // words of a lane's codes in a group of eight slots
      constexpr int kAll = kHeads * (kRawSlots / 8);  // groups of a chunk: [head][group]
      const int quarter = warp - Role::kDecode, chunk0 = quarter * 32, g = lane >> 2, t4 = lane & 3;
      const uint32_t raw = smem_u32(ring) + stages * kStageBytes + chunk0 / 8 * kGroupBytes;
      // Where this lane's codes lie in a group, and where its 16-byte pieces (eight dimensions of a slot) go: piece i of a lane at
      // `to` ^ 16 i.  Half of the lanes take their two 8-byte halves the other way round, so that eight neighbouring lanes' pieces
      // lie in different banks.
      // keys: slot g, a quarter of its dimensions; values: slots 2 t4 and 2 t4 + 1, an eighth of the dimensions
      const uint32_t k_flip = D == 128 && (t4 & 2) ? 1u : 0u, v_flip = D == 128 && (g & 1) ? 1u : 0u;
      const uint32_t k_piece = t4 * kWords, v_piece = g * (kWords / 2);
      const uint32_t k_to = (k_piece >> 3) * kHalfBytes + (chunk0 + g) * 128 + (((k_piece ^ g) & 7) ^ (2 * k_flip)) * 16;
      const uint32_t v_to = (v_piece >> 3) * kHalfBytes + (chunk0 + 2 * t4 + v_flip) * 128 + ((v_piece ^ (2 * t4 + v_flip)) & 7) * 16;
      const uint32_t v_to2 = (v_piece >> 3) * kHalfBytes + (chunk0 + 2 * t4 + (v_flip ^ 1)) * 128 + ((v_piece ^ (2 * t4 + (v_flip ^ 1))) & 7) * 16;
      const uint32_t k_low = k_flip ? 0x3232 : 0x1010, k_high = k_flip ? 0x1010 : 0x3232;  // selectors of the scales
      const uint32_t v_low = v_flip ? 0x3232 : 0x1010, v_high = v_flip ? 0x1010 : 0x3232;
      Ring codes;
      Ring at;
      uint32_t filled = 0, seg = 0;
      bool go = true;
      auto convert = [&](int b) {
        constexpr int kLanes = W / 8, kAtOnce = 32 / kLanes;  // lanes of a row, rows at once
#pragma unroll 2
        for (int x = 0; x < 32; x += kAtOnce) {
          const int row = chunk0 + x + lane / kLanes, y = lane & (kLanes - 1);
          uint4* at = reinterpret_cast<uint4*>(q_buf + (y >> 3) * kHalfBytes + row * 128 + ((y ^ row) & 7) * 16);
          const uint4 v = *at;
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
          float top = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(bf16_lo(in[i])), fabsf(bf16_hi(in[i]))));
#pragma unroll
          for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
          const int up = 14 - max(static_cast<int>((__float_as_uint(top) >> 23) & 0xFF) - 127, -100);
          const float by = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
          if (y == 0) sm.q_size[b][row] = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
          uint32_t out[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) out[i] = pack_f16(bf16_lo(in[i]) * by, bf16_hi(in[i]) * by);
          *at = make_uint4(out[0], out[1], out[2], out[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(&sm.q_full[b]);
      };
      for (uint32_t t = t0; stretch_at(t) && go;) {
        Segment s;
        if (go = described(seg, &s); !go) break;
        const int end = s.r.len + s.r.nodes, lo = a.window > 0 ? max(0, s.r.len - a.window + 1) : 0;
        for (int j = s.kv0; j < s.kv1 && go; ++j) {
          const int s0 = tile_slot<kTile>(s.r, j) + chunk0;
          uint32_t live = 0xFFFFFFFFu;  // this quarter's slots that some node may see: the others may hold anything
          if (s0 + 32 > end || (a.window > 0 && s0 < lo && s0 + 32 > a.sinks))
            live = range_bits(lo, end, s0) | (a.window > 0 ? range_bits(0, min(a.sinks, end), s0) : 0u);
#pragma unroll
          for (int value = 0; value < 2; ++value) {
            if (filled >= stages) go = warp_wait<kFour>(&sm.empty[at.stage], at.parity ^ 1, &sm.dead, a.status);
            if (!go) break;
            const uint32_t stage = smem_u32(ring) + at.stage * kStageBytes;
            if (value == 0) go = warp_wait<kFour>(&sm.raw_full[codes.stage], codes.parity, &sm.dead, a.status);
            // a chunk's codes and scales are read before the one before it is stored: loads do not pass stores by themselves
            uint32_t w[kAll][kWords], two[kAll], next_w[kAll][kWords], next_two[kAll];
            auto fetch = [&](int c) {
#pragma unroll
              for (int x = 0; x < kAll; ++x) {
                const int head = x / (kRawSlots / 8), u = x % (kRawSlots / 8);
                const uint32_t group = raw + (codes.stage * kHeads + head) * kHeadBytes + (c * (kRawSlots / 8) + u) * kGroupBytes + (value ? 4 * D + D / 2 : 0);
                if constexpr (D == 128) {
                  const uint32_t at_codes = group + lane * 16 + (value ? v_flip : k_flip) * 8;
                  lds64(at_codes, next_w[x][0], next_w[x][1]);
                  lds64(at_codes ^ 8, next_w[x][2], next_w[x][3]);
                  next_two[x] = lds16(group + 4 * D + lane * 2);
                } else {
                  lds64(group + lane * 8, next_w[x][0], next_w[x][1]);
                  next_two[x] = value ? lds16(group + 4 * D + (g >> 1) * 8 + t4 * 2) : lds8(group + 4 * D + lane);
                }
              }
            };
            fetch(0);
#pragma unroll 1
            for (int c = 0; c < 32 / kRawSlots; ++c) {
#pragma unroll
              for (int x = 0; x < kAll; ++x) {
                two[x] = next_two[x];
#pragma unroll
                for (int i = 0; i < kWords; ++i) w[x][i] = next_w[x][i];
              }
              if (c + 1 < 32 / kRawSlots) fetch(c + 1);
#pragma unroll
              for (int x = 0; x < kAll; ++x) {
                const int head = x / (kRawSlots / 8), u = x % (kRawSlots / 8);
                const uint32_t to = stage + head * kHalfBytes + (c * kRawSlots + u * 8) * 128;
                uint32_t by = decode_scales(static_cast<uint16_t>(two[x]));
                if (value == 1 && live != 0xFFFFFFFFu) {
                  const uint32_t bits = live >> (c * kRawSlots + u * 8 + 2 * t4);
                  by &= ((bits & 1u) ? 0xFFFFu : 0u) | ((bits & 2u) ? 0xFFFF0000u : 0u);
                }
                const uint32_t low = __byte_perm(by, by, D == 64 && value == 0 ? 0x1010 : value ? v_low : k_low);
                const uint32_t high = D == 64 && value == 0 ? low : __byte_perm(by, by, value ? v_high : k_high);
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                  uint32_t h[4];
                  decode8(w[x][i], h);
#pragma unroll
                  for (int e = 0; e < 4; ++e) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[e]) : "r"(2 * i < kWords ? low : high));
                  constexpr int kHalf = kWords / 2;
                  const uint32_t place = value == 0 ? to + (k_to ^ (16 * i)) : i < kHalf ? to + (v_to ^ (16 * i)) : to + (v_to2 ^ (16 * (i - kHalf)));
                  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(place), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
                }
              }
            }
            if (value == 1) {  // the codes are done with
              __syncwarp();
              if (lane == 0) mbar_arrive(&sm.raw_empty[codes.stage]);
              codes.step(a.raw_stages);
            }
            fence_proxy_async_smem();
            mbar_arrive(&sm.full[at.stage]);
            ++filled;
            at.step(stages);
          }
          // (behind the segment's first stages: Q comes when the segment before has had its last S)
          if (j == s.kv0 && go) {
            go = warp_wait<kFour>(&sm.q_raw[seg & 1], (seg >> 1) & 1, &sm.dead, a.status);
            convert(seg & 1);
          }
        }
        ++seg;
        t = s.next;
      }
    }
  };
  auto softmax = [&]() {
    // ---- softmax: thread r of a group has row r of the tile: row `row_in` of copy `copy` -----------
    const int group = (warp - Role::kSoft) >> 2;
    const int r = (warp & 3) * 32 + lane;
    constexpr int rows_apart = kTile / kCopies;
    const int row_in = r & (rows_apart - 1), copy = r / rows_apart;
    const int half = kPair ? row_in / kHalfRows : 0, local = row_in & (kHalfRows - 1);  // its head of the pair, its row there
    // slots whose scores are in registers at once (in 4 bits with two copies 64 trees 113 us with 64, 109 with 32: less code; four
    // chains, one copy, 250 and 264)
    constexpr int kWide = kCopies == 4 || (kFour && kCopies == 2) ? 32 : 64;
    constexpr int kSteps = kTile / kCopies / kWide;          // of a copy's slots
    const int slot0 = copy * (kTile / kCopies);              // first slot of a tile that this thread's copy takes
    const uint32_t my = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_addr = my + Col::s(group), o_addr = my + Col::o(group), p_addr = my + Col::p(group);
    float4* mix = sm.mix[group];
    float c = a.scale * 1.44269504088896341f;
    if (tid == 32 * Role::kSoft) a.jobs[blockIdx.x].valid = 0;
    uint32_t n0 = 0, seg = 0, mixes = 0, frees = 0;  // the segment's first tile in this CTA's count
    for (uint32_t t = t0; stretch_at(t); ++seg) {
      const int b = seg & 1;
      if (!warp_wait<kFour>(&sm.q_full[b], (seg >> 1) & 1, &sm.dead, a.status)) break;
      if constexpr (kFour) c = fmaxf(a.scale * 1.44269504088896341f * sm.q_size[b][r], 1e-37f);  // (not 0: masked scores are -inf)
      const Segment& s = sm.seg[seg & kSegMask];
      const int32_t* tree = parents + (seg & kSegMask) * a.Nmax;
      auto parent_of = [&](int node) { return a.parent != nullptr ? tree[node] : node - 1; };
      const int rows = min(a.tile_nodes, s.r.nodes - s.mtile * a.tile_nodes) * a.group;
      const bool active = (((warp & 3) * 32) & (kHalfRows - 1)) < rows;  // some row of this warp exists
      const bool exists = local < rows;
      const int local_node = exists ? over_group(local, a.over_group) : 0, node = s.mtile * a.tile_nodes + local_node;
      const int len = s.r.len, end = len + s.r.nodes;
      const int lo = a.window > 0 ? max(0, len - a.window + 1) : 0;  // before it (and past the sinks) no node sees a slot
      int depth = 0;
      if (a.window > 0) {
        if (a.parent == nullptr) depth = node;
        else
          for (int p = node; p > 0; ++depth) {
            const int up = tree[p];
            if (up < 0 || up >= p) break;  // reported where the node's own tile is masked
            p = up;
          }
      }
      const int near = a.window > 0 ? len + depth - a.window + 1 : 0;  // first position of the window
      const int tiles = s.kv1 - s.kv0;
      float m = -INFINITY, l = 0.0f, lr = 0.0f;  // maximum, sum of P, sum of the rounded P
      bool left = false;
      for (int j = (group + n0) & 1; j < tiles; j += 2) {
        const uint32_t n = n0 + j;
        if (left = !warp_wait<kFour>(&sm.s_full[group], (n >> 1) & 1, &sm.dead, a.status); left) break;
        tc_after_sync();
        const int s0 = tile_slot<kTile>(s.r, s.kv0 + j);
        const bool whole = s0 + kTile <= len && (a.window <= 0 || s0 + kTile <= a.sinks || s0 >= len + s.r.nodes - a.window);
        if (!kFour && !whole && (s0 + kTile > end || (a.window > 0 && s0 < lo && s0 + kTile > a.sinks))) {
          // slots that no node sees may hold anything: 0 times it has to be 0
          const uint32_t v = 2 * n + 1, st = v % stages;
          if (left = !warp_wait<kFour>(&sm.full[st], (v / stages) & 1, &sm.dead, a.status); left) break;
          const int slot = s0 + r;
          if (slot >= end || (slot < lo && slot >= a.sinks)) {
#pragma unroll 4
            for (int x = 0; x < W / 8; ++x)
              *reinterpret_cast<uint4*>(ring + st * kStageBytes + (x >> 3) * kHalfBytes + r * 128 + ((x + r) & 7) * 16) = make_uint4(0, 0, 0, 0);  // (neighbours in different banks)
          }
          fence_proxy_async_smem();
        }
        if (active) {
          // With one copy S is read in two halves, the first half twice (for the maximum and for P); P's columns
          // lie over the second half.
          uint32_t x[kWide];
          float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int k = 0; k < kSteps; ++k) {
            const int col = slot0 + k * kWide;
#pragma unroll
            for (int i = 0; i < kWide; i += 32) tmem_load32(s_addr + col + i, x + i);
            uint32_t see[kWide / 32];
            if (!whole) {
#pragma unroll
              for (int w = 0; w < kWide / 32; ++w)
                see[w] = range_bits(near, len, s0 + col + 32 * w) | (a.window > 0 ? range_bits(0, min(a.sinks, len), s0 + col + 32 * w) : 0u);
              if (s0 + col + kWide > len && exists) {
                int d = depth;
                for (int up = node;; --d) {
                  const int bit = len + up - s0 - col;
                  if (bit >= 0 && bit < kWide && (a.window <= 0 || len + d >= near || len + d < a.sinks)) {
                    if (kWide == 32 || bit < 32) see[0] |= 1u << (bit & 31);
                    else see[kWide / 32 - 1] |= 1u << (bit & 31);
                  }
                  if (up <= 0 || bit < 0) break;
                  const int p = parent_of(up);
                  if (p < 0 || p >= up) {
                    mark_bad(a, s.request, SV_DEV_BAD_PARENT);
                    break;
                  }
                  up = p;
                }
              }
            }
            tmem_loaded(x);
            if (!whole) {
#pragma unroll
              for (int i = 0; i < kWide; ++i)
                if (!((see[i >> 5] >> (i & 31)) & 1u)) x[i] = 0xFF800000u;
              if (k + 1 < kSteps) {  // masked, for the second reading
#pragma unroll
                for (int i = 0; i < kWide; i += 32) tmem_store32(s_addr + col + i, x + i);
              }
            }
#pragma unroll
            for (int i = 0; i < kWide; i += 8)  // four chains, three operands a step
#pragma unroll
              for (int e = 0; e < 4; ++e)
                top4[e] = fmaxf(fmaxf(top4[e], __uint_as_float(x[i + e])), __uint_as_float(x[i + 4 + e]));
          }
          if (!whole) tmem_wait_store();
          const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * c;  // c > 0
          const float now = kFour ? top - kBias : top;
          if (j < 2) {
            m = now;
          } else {
            const bool grow = now > m + kLazyGrowth || (m == -INFINITY && now > -INFINITY);
            if (__any_sync(0xFFFFFFFFu, grow)) {
              const float keep = grow ? (m == -INFINITY ? 0.0f : ex2_approx(m - now)) : 1.0f;
              if (grow) m = now;
              l *= keep;
              lr *= keep;
              // the group's O is complete up to its tile before
              if (left = !warp_wait<kFour>(&sm.pv_done[group], ((n - 2) >> 1) & 1, &sm.dead, a.status); left) break;
              tc_after_sync();
#pragma unroll 1
              for (int i = 0; i < W; i += 16) {
                uint32_t o[16];
                tmem_load16(o_addr + i, o);
                tmem_loaded(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                tmem_store16(o_addr + i, o);
              }
            }
          }
          if (Col::kOwnP && j >= 2) {  // the product of the group's tile before has read P
            if (left = !warp_wait<kFour>(&sm.pv_done[group], ((n - 2) >> 1) & 1, &sm.dead, a.status); left) break;
            tc_after_sync();
          }
          const float off = m == -INFINITY ? 0.0f : -m;
          const f32x2 c2 = f2_pack(c, c), off2 = f2_pack(off, off);
          f32x2 sum[2] = {0, 0}, sumr[2] = {0, 0};
#pragma unroll 1
          for (int k = kSteps - 1; k >= 0; --k) {  // the last step's scores are still there
            const int col = slot0 + k * kWide;
            if (k < kSteps - 1) {
#pragma unroll
              for (int i = 0; i < kWide; i += 32) tmem_load32(s_addr + col + i, x + i);
              tmem_loaded(x);
            }
#pragma unroll
            for (int i = 0; i < kWide; i += 2) {
              float e0, e1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), c2, off2), e0, e1);
              e0 = ex2_approx(e0);
              e1 = ex2_approx(e1);
              // (a float16 is off by 2^-12 of itself, below 2^-14 by 2^-25: o is divided by the sum before rounding)
              const uint32_t w = kFour ? pack_f16(e0, e1) : pack_bf16(e0, e1);
              sum[(i >> 1) & 1] = f2_add(sum[(i >> 1) & 1], f2_pack(e0, e1));
              if (!kFour) sumr[(i >> 1) & 1] = f2_add(sumr[(i >> 1) & 1], f2_pack(bf16_lo(w), bf16_hi(w)));
              x[i >> 1] = w;
            }
            if constexpr (kWide == 64) {
              tmem_store32(p_addr + col / 2, x);
            } else {
              tmem_store16(p_addr + col / 2, x);
            }
          }
          if constexpr (kCopies > 1) {
            uint32_t zero[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) zero[i] = 0;
#pragma unroll 1
            for (int k = 0; k < 4; ++k)
              if (32 * k < slot0 || 32 * k >= slot0 + kTile / kCopies) tmem_store16(p_addr + 16 * k, zero);
          }
          float e0, e1;
          f2_unpack(f2_add(sum[0], sum[1]), e0, e1);
          l += e0 + e1;
          if (!kFour) f2_unpack(f2_add(sumr[0], sumr[1]), e0, e1);
          lr += e0 + e1;
          tmem_wait_store();
        }
        tc_before_sync();
        mbar_arrive(&sm.p_full[group]);
      }
      if (left) break;
      // ---- the segment's end: the sums of groups and copies, then half of the columns per group --------
      sm.m[b][group][r] = m;
      sm.l[b][group][r] = l;
      sm.lr[b][group][r] = lr;
      mbar_arrive(&sm.sums_full);
      if (!warp_wait<kFour>(&sm.sums_full, seg & 1, &sm.dead, a.status)) break;
      float top = -INFINITY, sum = 0.0f, sumr = 0.0f;
      for (int x = row_in; x < kTile; x += rows_apart) top = fmaxf(top, fmaxf(sm.m[b][0][x], sm.m[b][1][x]));
      for (int x = row_in; x < kTile; x += rows_apart)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float w = sm.m[b][g][x] == -INFINITY ? 0.0f : ex2_approx(sm.m[b][g][x] - top);
          sum += w * sm.l[b][g][x];
          sumr += w * sm.lr[b][g][x];
        }
      const bool complete = s.kv0 == 0 && s.kv1 == s.r.tiles;
      // Every row sees its own node's slot, so a sum that is not above 0 is that of a row without a softmax: NaN among its
      // scores (which the maximum passes over), or nothing but -inf.  Its outputs are NaN; the parts' sums tell the join.
      const float inv = !complete ? 1.0f : sumr > 0.0f ? a.v_scale / sumr : NAN;
      // (a group without a tile in the segment has m = -inf: its O is not used, whatever it holds)
      const float w0 = (sm.m[b][0][r] == -INFINITY ? 0.0f : ex2_approx(sm.m[b][0][r] - top)) * inv;
      const float w1 = (sm.m[b][1][r] == -INFINITY ? 0.0f : ex2_approx(sm.m[b][1][r] - top)) * inv;
      const int head = ((kPair ? 2 * s.head + half : s.head) - local_node) * a.group + local;  // (of an existing row)
      float* part = a.parts + static_cast<int64_t>(2 * blockIdx.x + (s.kv0 == 0)) * part_floats<D>();
      // four columns of this thread's row: to the output, or to this CTA's partial result
      __nv_bfloat16* out_row = a.out + (s.r.first + node) * a.out_row_stride +
                               head * a.out_head_stride - (kPair ? half * D : 0);
      float* part_row = part + row_in * 4 - (kPair ? half * D * kTile : 0);
      auto emit4 = [&](int column, float4 v) {
        if (complete) *reinterpret_cast<uint2*>(out_row + column) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        else *reinterpret_cast<float4*>(part_row + column * kTile) = v;
      };
      if (group == 0 && copy == 0 && exists) {
        if (!complete) {
          part[kTile * D + row_in] = top;
          part[kTile * D + kTile + row_in] = sum;
          part[kTile * D + 2 * kTile + row_in] = sumr;
        } else if (a.lse != nullptr) {
          a.lse[(s.r.first + node) * a.q_heads + head] = (top + log2f(sum)) * 0.693147180559945309f;
        }
      }
      if (tid == 32 * Role::kSoft && s.kv0 == 0 && !complete) {
        // the CTA in which the row tile ends
        const uint32_t ends = s.begin + a.extra + s.r.tiles - 1;
        const Job job = {1, s.request, s.head, s.mtile, rows, static_cast<int32_t>(blockIdx.x), parts.of(ends), 0};
        a.jobs[blockIdx.x] = job;
      }
      // the last tile of each parity: its product is the last into that group's O
      const uint32_t last = n0 + tiles - 1;
      bool ok = warp_wait<kFour>(&sm.pv_done[last & 1], (last >> 1) & 1, &sm.dead, a.status);
      if (ok && tiles > 1) ok = warp_wait<kFour>(&sm.pv_done[(last - 1) & 1], ((last - 1) >> 1) & 1, &sm.dead, a.status);
      if (!ok) break;
      tc_after_sync();
      // P of this thread's columns from `column` on, both groups' O's together
      auto read_o = [&](int column, auto& f) {
        constexpr int P = sizeof(f) / sizeof(float);
        uint32_t x[P], y[P];
        if constexpr (P == 16) {
          tmem_load16(my + Col::o(0) + column, x);
          tmem_load16(my + Col::o(1) + column, y);
        } else {
          tmem_load8(my + Col::o(0) + column, x);
          tmem_load8(my + Col::o(1) + column, y);
        }
        tmem_loaded(x);
        tmem_loaded(y);
#pragma unroll
        for (int e = 0; e < P; ++e)
          f[e] = (w0 != 0.0f ? w0 * __uint_as_float(x[e]) : 0.0f) + (w1 != 0.0f ? w1 * __uint_as_float(y[e]) : 0.0f);
      };
      const int col0 = group * (W / 2), col1 = col0 + W / 2;
      const bool writes = exists && (!kPair || half == group);
      if constexpr (kCopies == 1) {
        if (active) {
#pragma unroll 1
          for (int i = col0; i < col1; i += 16) {
            float f[16];
            read_o(i, f);
            if (writes) {
#pragma unroll
              for (int q = 0; q < 4; ++q) emit4(i + 4 * q, make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]));
            }
          }
        }
      } else {
        // The copies' sum through shared memory: in a round every copy takes P columns, to which the others send theirs.
        // Rounds of as many columns as fit: each costs 0.8 us, most of it latency.  (Loops, not unrolled: this code runs
        // once a segment and comes from behind the instruction cache.)
        const int kept_rows = (rows + 7) & ~7;
        auto mixed = [&](auto width) {
          constexpr int P = decltype(width)::value;
#pragma unroll 1
          for (int i0 = col0; i0 < col1; i0 += kCopies * P) {
            float f[P];
            if (active) {
#pragma unroll 1
              for (int o = 1; o < kCopies; ++o) {
                const int to = (copy + o) % kCopies;
                read_o(i0 + to * P, f);
                float4* at = mix + (to * (kCopies - 1) + o - 1) * (P / 4) * kept_rows + local;
                if (writes) {
#pragma unroll
                  for (int q = 0; q < P / 4; ++q) at[q * kept_rows] = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
                }
              }
              read_o(i0 + copy * P, f);
            }
            mbar_arrive(&sm.mix_full[group]);
            if (!warp_wait<kFour>(&sm.mix_full[group], mixes & 1, &sm.dead, a.status)) return false;
            ++mixes;
            if (writes) {
              const float4* from = mix + copy * (kCopies - 1) * (P / 4) * kept_rows + local;
#pragma unroll
              for (int q = 0; q < P / 4; ++q) {
                float4 v = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
#pragma unroll
                for (int o = 0; o < kCopies - 1; ++o) {
                  const float4 w = from[(o * (P / 4) + q) * kept_rows];
                  v.x += w.x;
                  v.y += w.y;
                  v.z += w.z;
                  v.w += w.w;
                }
                emit4(i0 + copy * P + 4 * q, v);
              }
            }
            if (i0 + kCopies * P < col1) {  // the buffer is written again
              mbar_arrive(&sm.mix_free[group]);
              if (!warp_wait<kFour>(&sm.mix_free[group], frees & 1, &sm.dead, a.status)) return false;
              ++frees;
            }
          }
          return true;
        };
        // (kept_rows copies (copies - 1) P floats; a half of 32 columns goes over four copies by 8)
        static_assert(64 * 2 * 16 <= 4 * kMixFloat4 && 16 * 4 * 3 * 16 <= 4 * kMixFloat4 && 32 * 4 * 3 * 8 <= 4 * kMixFloat4, "mix");
        static_assert(!kFour || (kCopies <= 2 && 64 * 2 * 16 <= 4 * kMixFloat4Of4), "mix");
        using Sixteen = std::integral_constant<int, 16>;
        using Eight = std::integral_constant<int, 8>;
        if constexpr (kCopies == 2) left = !mixed(Sixteen());
        else if constexpr (W == 64) left = !mixed(Eight());
        else left = kept_rows <= 16 ? !mixed(Sixteen()) : !mixed(Eight());
      }
      if (left) break;
      tc_before_sync();
      t = s.next;
      mbar_arrive(&sm.o_free);
      mbar_arrive(&sm.seg_free[seg & kSegMask]);
      n0 += tiles;
    }
  };
  if constexpr (kFour) {
    if (warp < Role::kSoft) {  // 128 registers a thread at launch: 4 * 128 >= 72 + 2 * 168 + 104
      fewer_registers<72>();
      if (warp == Role::kMma) half_of_products(std::false_type());
      else if (warp == Role::kPv) half_of_products(std::true_type());
      else if (warp == Role::kQ) queries();
      else if (warp == Role::kK) copies();
    } else if (warp < Role::kDecode) {
      more_registers<168>();
      softmax();
    } else {
      fewer_registers<104>();
      decode();
    }
  } else {
    if (warp == Role::kK || warp == Role::kV) copies();
    else if (warp == Role::kQ) queries();
    else if (warp == Role::kMma) products();
    else softmax();
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  if (sm.dead) {  // copies in flight land before the CTA leaves
    if (kFour && warp == Role::kK)
      for (uint32_t x = loaded > static_cast<uint32_t>(a.raw_stages) ? loaded - a.raw_stages : 0; x < loaded; ++x)
        mbar_wait(&sm.raw_full[x % a.raw_stages], (x / a.raw_stages) & 1, a.status);
    if (!kFour && (warp == Role::kK || warp == Role::kV))  // its last fills: every second place of the ring's line
      for (uint32_t x = loaded > stages + 1 ? loaded - ((stages + 1) & ~1u) : (warp == Role::kV); x < loaded; x += 2)
        mbar_wait(&sm.full[x % stages], (x / stages) & 1, a.status);
    if (warp == Role::kQ && segments > 0)
      mbar_wait(kFour ? &sm.q_raw[(segments - 1) & 1] : &sm.q_full[(segments - 1) & 1], ((segments - 1) >> 1) & 1, a.status);
    __syncthreads();
  }
  if (warp == Role::kMma) tmem_free(tmem);
}

// Adds the partial results of row tile `jobs[x]`: with M = max m_i, o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// grid (CTAs of the attention, row groups); a thread has four columns of a row.  Then the outputs of bad requests become 0.
template <int D>
__global__ void __launch_bounds__(kJoinRows * D / 4) join_kernel(const AttendParams a) {
  constexpr int kJoinThreads = kJoinRows * D / 4;
  pdl_wait();
  const Job job = a.jobs[blockIdx.x];
  const int heads = a.kv_heads / a.units, piece = threadIdx.x / kJoinRows;
  int local = blockIdx.y * kJoinRows + threadIdx.x % kJoinRows;
  if (job.valid != 0 && local < heads * job.rows && !a.bad[job.request]) {
    const int half = local >= job.rows;
    local -= half * job.rows;
    const int r = half * a.half_rows + local;
    const int n = job.last - job.first + 1;
    // part i > 0 is its CTA's first, part 0 its CTA's second
    const float* first = a.parts + static_cast<int64_t>(2 * job.first + 1) * part_floats<D>();
    const float* others = a.parts + static_cast<int64_t>(2 * job.first) * part_floats<D>();
    float M = -INFINITY, L = 0.0f, R = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = 0; i < n; ++i) M = fmaxf(M, (i == 0 ? first : others + static_cast<int64_t>(2 * i) * part_floats<D>())[kTile * D + r]);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float* part = i == 0 ? first : others + static_cast<int64_t>(2 * i) * part_floats<D>();
      const float m = part[kTile * D + r];
      const float w = m == -INFINITY ? 0.0f : ex2_approx(m - M);
      const float4 v = *reinterpret_cast<const float4*>(part + (piece * kTile + r) * 4);
      L += w * part[kTile * D + kTile + r];
      R += w * part[kTile * D + 2 * kTile + r];
      o[0] += w * v.x;
      o[1] += w * v.y;
      o[2] += w * v.z;
      o[3] += w * v.w;
    }
    const float inv = R > 0.0f ? a.v_scale / R : NAN;  // (not above 0: NaN among the row's scores, or nothing but -inf)
    const int node = job.mtile * a.tile_nodes + local / a.group, head = (heads * job.head + half) * a.group + local % a.group;
    const int64_t row = a.node_offsets[job.request] + node;
    uint2 w;
    w.x = pack_bf16(o[0] * inv, o[1] * inv);
    w.y = pack_bf16(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2*>(a.out + row * a.out_row_stride + head * a.out_head_stride + piece * 4) = w;
    if (piece == 0 && a.lse != nullptr) a.lse[row * a.q_heads + head] = (M + log2f(L)) * 0.693147180559945309f;
  }
  clear_bad<D, kJoinThreads>(a, a, a);
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

// The query rows as (dimension, head, row); a copy takes 64 dimensions of a head group's rows of a tile.
bool encode_queries(CUtensorMap* map, const void* q, int64_t row_stride, int64_t head_stride, int head_dim, int heads,
                    int64_t rows, int group, int tile_nodes) {
  const EncodeTiled fn = encode_tiled();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2, static_cast<cuuint64_t>(row_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(tile_nodes)};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kPair, int kCopies, bool kFour>
cudaError_t launch_attention(AttendParams& a, const CUtensorMap& q_map, const CUtensorMap& k_map, const CUtensorMap& v_map,
                             int ctas, void* stream) {
  // the ring gets what Q, the tables and the fixed part leave of the shared memory: at least 4 stages (in 4 bits 3, behind
  // the codes' rings)
  constexpr int kStageBytes = (kPair ? 2 : 1) * D / 64 * kHalfBytes;
  constexpr int kRawBytes = kFour ? (kPair ? 2 : 1) * kTile / 8 * 9 * D : 0;
  constexpr int kStatic = sizeof(Smem<kFour>) + 64;
  int fixed = 4 * (a.B + Warps<kFour>::kSegments * a.Nmax) + 1024 + kStageBytes;
  if (kFour) {
    a.raw_stages = std::min(kMaxRaw, (kSmemMax - kStatic - fixed - 3 * kStageBytes) / std::max(kRawBytes, 1));
    fixed += a.raw_stages * kRawBytes;
  }
  a.stages = std::min(kMaxStages, (kSmemMax - kStatic - fixed) / kStageBytes);
  // With an even number of stages K and V keep to their own.  Where S does not wait for the product P V of two tiles before (tiles
  // of 64 dimensions), the V warp could otherwise take an earlier emptying of a stage for its K's.  Pairs of heads, whose S waits,
  // go by it too: a fifth stage is no gain there (33 trees, window 1024: 42.5 us with 4, 43.0 with 5).
  if (Columns<D>::kOwnP && a.stages > 3) a.stages &= ~1;
  const size_t dyn = static_cast<size_t>(fixed) + static_cast<size_t>(a.stages) * kStageBytes;
  cudaError_t e = allow_smem<attend_kernel<D, kPair, kCopies, kFour>>(kSmemMax - kStatic);
  if (e != cudaSuccess) return e;
  e = launch_dependent(attend_kernel<D, kPair, kCopies, kFour>, dim3(ctas), Warps<kFour>::kThreads, dyn, stream,
                       SV_KERNEL_ATTENTION, 1, a, q_map, k_map, v_map);
  if (e != cudaSuccess) return e;
  const int groups = ((kPair ? 2 : 1) * a.tile_nodes * a.group + kJoinRows - 1) / kJoinRows;
  return launch_dependent(join_kernel<D>, dim3(ctas, groups), kJoinRows * D / 4, 0, stream, SV_KERNEL_ATTENTION_JOIN, 1, a);
}

}  // namespace

size_t attention4_tiles_workspace(int head_dim) { return layout_of(kMaxCtas, head_dim).total; }
sv_status attention4_tiles(const sv_cache4* c, int layer, const void* q, int64_t q_row_stride, int64_t q_head_stride, int q_heads,
                           const int32_t* page_table, int table_width, const int32_t* seq_len, const int32_t* node_offsets,
                           int64_t n_rows, const int32_t* parent, int B, int Nmax, float scale, int window, int sinks, void* out,
                           int64_t out_row_stride, int64_t out_head_stride, float* out_lse, void* ws, void* stream) {
  const int group = q_heads / c->kv_heads;
  const bool pair = c->head_dim == 64 && c->kv_heads % 2 == 0 && 2 * Nmax * group <= kTile;
  const int tile_nodes = std::min(kTile / group, Nmax);
  CUtensorMap q_map;
  if (!encode_queries(&q_map, q, q_row_stride, q_head_stride, c->head_dim, q_heads, n_rows, group, tile_nodes))
    return set_error(SV_ERR_CUDA, "the query rows' strides or sizes cannot be described to the copy engine");
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return launch_status(e, "device");
  const int ctas = std::min(sms, kMaxCtas);
  const Layout L = layout_of(kMaxCtas, c->head_dim);
  unsigned char* w = static_cast<unsigned char*>(ws);
  AttendParams a = {};
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
  while ((1 << a.shift) < c->page_size) ++a.shift;
  a.q_heads = q_heads;
  a.kv_heads = c->kv_heads;
  a.units = pair ? c->kv_heads / 2 : c->kv_heads;
  a.group = group;
  a.tile_nodes = tile_nodes;
  a.tile_rows = tile_nodes * group;
  a.over_group = (65536 + group - 1) / group;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale * c->k_scale;
  a.v_scale = c->v_scale;
  a.pool = static_cast<const unsigned char*>(c->pool) + layer * c->layer_stride;
  a.page_stride = c->page_stride;
  a.head_stride = c->head_stride;
  const int copies = tile_nodes * group * (pair ? 2 : 1) <= 64 ? 2 : 1;
  a.half_rows = kTile / copies / (pair ? 2 : 1);
  a.extra = kExtra;
  const auto launch = pair                 ? (copies == 2 ? launch_attention<64, true, 2, true> : launch_attention<64, true, 1, true>)
                      : c->head_dim == 128 ? (copies == 2 ? launch_attention<128, false, 2, true> : launch_attention<128, false, 1, true>)
                                           : (copies == 2 ? launch_attention<64, false, 2, true> : launch_attention<64, false, 1, true>);
  return launch_status(launch(a, q_map, q_map, q_map, ctas, stream), "attention");
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t sv_attention_workspace_size(const sv_cache* c, int q_heads) {
  if (check_cache(c) != SV_OK) return 0;
  if (q_heads < 1 || q_heads % c->kv_heads != 0 || q_heads / c->kv_heads > kTile) {
    set_error(SV_ERR_INVALID_ARG, "q_heads=%d: 1 to %d times kv_heads=%d are needed", q_heads, kTile, c->kv_heads);
    return 0;
  }
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
  if (q_heads < 1 || q_heads % c->kv_heads != 0 || q_heads / c->kv_heads > kTile)
    return set_error(SV_ERR_INVALID_ARG, "q_heads=%d: 1 to %d times kv_heads=%d are needed", q_heads, kTile, c->kv_heads);
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
  // two heads at a time where they lie side by side and all nodes' rows of both fit into a tile (else a tile would be
  // read once for each of their row tiles; 64 contexts of 8192, 16 heads of 64, one node: 322 us against 504 one by one; the window's 33 trees 41 against 50)
  const int group = q_heads / c->kv_heads;
  const bool pair = c->head_dim == 64 && c->head_stride == 64 && c->kv_heads % 2 == 0 && 2 * Nmax * group <= kTile;
  const int tile_nodes = std::min(kTile / group, Nmax);
  // the line of work is counted in 32 bits
  const int64_t tiles = ((static_cast<int64_t>(table_width) * c->page_size + kTile - 1) / kTile + 1 + kExtra) *
                        ((Nmax + tile_nodes - 1) / tile_nodes);
  if (tiles > INT_MAX || tiles * c->kv_heads > INT_MAX || tiles * c->kv_heads * B > INT_MAX)
    return set_error(SV_ERR_INVALID_ARG, "B=%d requests of up to %lld tiles a head are too many for one call", B, (long long)tiles);
  const size_t offset = static_cast<size_t>(layer) * c->layer_stride * 2;
  CUtensorMap q_map, k_map, v_map;
  if (!encode_queries(&q_map, q, q_row_stride, q_head_stride, c->head_dim, q_heads, n_rows, group, tile_nodes))
    return set_error(SV_ERR_CUDA, "the query rows' strides or sizes cannot be described to the copy engine");
  if (!encode_pool(&k_map, c, static_cast<const unsigned char*>(c->k) + offset) ||
      !encode_pool(&v_map, c, static_cast<const unsigned char*>(c->v) + offset))
    return set_error(SV_ERR_CUDA, "the cache's strides or sizes cannot be described to the copy engine");
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return launch_status(e, "device");
  const int ctas = std::min(sms, kMaxCtas);
  const Layout L = layout_of(kMaxCtas, c->head_dim);
  unsigned char* w = static_cast<unsigned char*>(ws);
  AttendParams a = {};
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
  a.units = pair ? c->kv_heads / 2 : c->kv_heads;
  a.group = group;
  a.tile_nodes = tile_nodes;
  a.tile_rows = tile_nodes * group;
  a.over_group = (65536 + group - 1) / group;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale;
  a.v_scale = 1.0f;
  // as many copies of a row tile as its height leaves room for (window's 33 trees, 32 rows: 41 us with four, 43 with two, 45
  // with one; 64 trees of 64 rows: 114 with two, 121 with one; 64 contexts of 1000, 4 rows: 57, 58, 60)
  const int tile_rows = tile_nodes * group * (pair ? 2 : 1), copies = tile_rows <= 32 ? 4 : tile_rows <= 64 ? 2 : 1;
  a.half_rows = kTile / copies / (pair ? 2 : 1);
  a.extra = kExtra;
  const auto launch = pair                 ? (copies == 4   ? launch_attention<64, true, 4, false>
                                              : copies == 2 ? launch_attention<64, true, 2, false>
                                                            : launch_attention<64, true, 1, false>)
                      : c->head_dim == 128 ? (copies == 4   ? launch_attention<128, false, 4, false>
                                              : copies == 2 ? launch_attention<128, false, 2, false>
                                                            : launch_attention<128, false, 1, false>)
                                           : (copies == 4   ? launch_attention<64, false, 4, false>
                                              : copies == 2 ? launch_attention<64, false, 2, false>
                                                            : launch_attention<64, false, 1, false>);
  return launch_status(launch(a, q_map, k_map, v_map, ctas, stream), "attention");
}

}  // extern "C"
