// Internal declarations shared by the round's operators (sampling, paged cache, tree attention):
// host-side checks and small device helpers.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>
#include <mutex>

#include "sv_internal.h"

namespace sv {

// ---- host checks -----------------------------------------------------------------------------
inline sv_status check_workspace(const void* ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr) return set_error(SV_ERR_WORKSPACE, "workspace is NULL");
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return set_error(SV_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (ws_bytes < need) return set_error(SV_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  return SV_OK;
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The pool's description (sv_cache.cu).
sv_status check_cache(const sv_cache* c);
sv_status check_cache4(const sv_cache4* c);  // (sv_cache4.cu)
sv_status check_table(const int32_t* page_table, int table_width, const int32_t* seq_len, int B);

// sv_tree_attention4 by tiles of 128 rows (sv_attention.cu): arguments as in sv.h, checked by the caller.
size_t attention4_tiles_workspace(int head_dim);
sv_status attention4_tiles(const sv_cache4* c, int layer, const void* q, int64_t q_row_stride, int64_t q_head_stride, int q_heads,
                           const int32_t* page_table, int table_width, const int32_t* seq_len, const int32_t* node_offsets,
                           int64_t n_rows, const int32_t* parent, int B, int Nmax, float scale, int window, int sinks, void* out,
                           int64_t out_row_stride, int64_t out_head_stride, float* out_lse, void* ws, void* stream);

inline sv_status launch_status(cudaError_t e, const char* what) {
  return e == cudaSuccess ? SV_OK : set_error(SV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Dynamic shared memory of a kernel, raised once per device (and again only for more).  Setting the limit and noting it are
// one step for all host threads: set by one and noted by another in between, the note could stay above the limit, and
// every launch of that size would fail from then on.
constexpr int kMaxDevices = 64;
template <auto kKernel>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<size_t> allowed[kMaxDevices];
  static std::mutex raising;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices && allowed[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
  const std::lock_guard<std::mutex> lock(raising);
  if (dev < kMaxDevices && allowed[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess && dev < kMaxDevices) allowed[dev].store(bytes, std::memory_order_release);
  return e;
}

// Multiprocessors of the current device, looked up once per device.
inline cudaError_t sm_count(int* out) {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  *out = dev < kMaxDevices ? known[dev].load(std::memory_order_relaxed) : 0;
  if (*out > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < kMaxDevices) known[dev].store(*out, std::memory_order_relaxed);
  return e;
}

// Launch behind the stream's previous kernel with programmatic dependent launch: the launch
// overlaps that kernel's tail, and the kernel waits in pdl_wait() before it touches memory.  Left
// out while instrumentation puts events between kernels.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, void* stream, int prof_id,
                             int cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (!prof_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  prof_before(prof_id, stream);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
  prof_after(prof_id, stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

#ifdef __CUDACC__
// The request whose rows hold `row`: the last i with offsets[i] <= row, by one whole warp (32
// probes a step, so 4096 requests take three dependent loads).
__device__ __forceinline__ int request_of_row(const int32_t* offsets, int B, int64_t row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lane * step;
    const unsigned le = __ballot_sync(0xFFFFFFFFu, at < n && offsets[lo + at] <= row);
    const int c = max(__popc(le) - 1, 0) * step;
    lo += c;
    n = min(step, n - c);
  }
  return lo;
}
#endif

}  // namespace sv
