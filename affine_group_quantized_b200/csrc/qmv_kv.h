// qmv_kv.h -- what the key-value cache sources share: the device view of a
// paged cache, and the host interface of the attention kernels
// (qmv_kv_attn.cuh), used by the entry points in qmv_kv.cu.  Internal to the
// library.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <mutex>

#include "qmv.h"

namespace qmvc {

// Rows (page, kv head, slot) of the cache and the block table that names a
// sequence's pages; passed by value to every kernel.
struct CacheView {
  uint8_t *k, *v;                                          // code rows (or bf16 rows)
  uint16_t *k_scales, *k_biases, *v_scales, *v_biases;     // null for bf16 rows
  const int *table;                                        // [batch][width]
  int num_pages, H, S, D, bits, G;                         // G: groups of a row
  int width;                                               // pages per sequence
  int row_bytes;                                           // of one K or V row
  int *status;                                             // or null
};

#ifdef __CUDACC__
// A page's number if it lies in the cache, else -1 (and the caller's status
// word is told).
__device__ __forceinline__ int checked_page(const CacheView &c, int page) {
  if (static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages)) return page;
  if (c.status) atomicOr(c.status, 1);
  return -1;
}

// Row number of slot `at` of page `page`, head `h` (fewer than 2^31 rows).
__device__ __forceinline__ uint32_t cache_row(const CacheView &c, int page, int h, int at) {
  return (static_cast<uint32_t>(page) * c.H + h) * c.S + at;
}

// Programmatic dependent launch: the kernels are scheduled as the previous one of
// the stream ends, and wait here for it before their first global access.  None
// lets its successor start earlier: resident blocks that wait slowed the kernel
// they waited for (attention's second kernel by up to 1.5 us, eviction of one slot
// from 9.6 to 10.4 us).
__device__ __forceinline__ void wait_for_previous_grid() {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
}
#endif

struct AttnArgs {
  CacheView cache;
  const void *q;
  long long q_stride;
  const int *lens;
  void *out;
  int batch, num_q_heads;
  float scale;
  float *weights;       // or null
  int state_width;
  void *workspace;
  cudaStream_t stream;
};

// What the launches ask of a device, once.
constexpr int kMaxDevices = 64;
struct Device {
  int id = 0, sms = 0;
};

// Allows a kernel `bytes` of dynamic shared memory on a device, and once allowed
// does not ask again (one `granted` per kernel).  The attribute is the kernel's, not
// the launch's, and calls of other sizes may ask at the same time: look, set and
// note are one step, and the limit is only ever raised.
struct Granted {
  std::mutex mutex;
  std::atomic<int> bytes[kMaxDevices];
};
template <typename... KArgs>
cudaError_t allow_smem(void (*kern)(KArgs...), Granted &granted, const Device &dev, int bytes) {
  std::atomic<int> &allowed = granted.bytes[dev.id];
  if (bytes <= allowed.load(std::memory_order_acquire)) return cudaSuccess;
  std::lock_guard<std::mutex> hold(granted.mutex);
  if (bytes <= allowed.load(std::memory_order_relaxed)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)  // as many blocks of an SM as the rest allows
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess) allowed.store(bytes, std::memory_order_release);
  else cudaGetLastError();  // clear it
  return e;
}

// Bytes of workspace a call needs, and the launches themselves, by width
// (qmv_kv_attn4.cu, 8 and 16).
size_t attn_workspace_4(const CacheView &c, int batch, int num_q_heads, bool weights, int sms);
size_t attn_workspace_8(const CacheView &c, int batch, int num_q_heads, bool weights, int sms);
size_t attn_workspace_16(const CacheView &c, int batch, int num_q_heads, bool weights, int sms);
cudaError_t attn_launch_4(const AttnArgs &a, const Device &dev);
cudaError_t attn_launch_8(const AttnArgs &a, const Device &dev);
cudaError_t attn_launch_16(const AttnArgs &a, const Device &dev);

// A launch that may be scheduled while the previous kernel of the stream
// finishes: the kernels hold their first global access until then
// (wait_for_previous_grid).  cluster: CTAs of a thread-block cluster, or 1.
template <typename... KArgs, typename... Args>
cudaError_t launch_overlapped(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem,
                              int cluster, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) cudaGetLastError();  // clear it
  return e;
}

}  // namespace qmvc
