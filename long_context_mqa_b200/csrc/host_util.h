// Host-side helpers shared by the hs2 launchers: TMA descriptor encoding (driver entry point
// fetched through the runtime, so the library needs no libcuda link), device checks, and the
// bounded-wait limit.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>

#include <utility>

#include "../../include/hs2.h"

namespace hs2 {

// Encodes a 3D tensor map of bf16 (elem_bytes 2) or bytes (1): dims (inner, rows, batch) with
// strides in elements, box (box_inner, box_rows, 1), 128-byte swizzle, out-of-range elements
// read as zero.
bool make_tmap_3d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t batch,
                  uint64_t row_stride_el, uint64_t batch_stride_el, uint32_t box_inner, uint32_t box_rows,
                  bool swizzle128 = true, int elem_bytes = 2);

// 2D variant: dims (inner, rows), row stride in elements.
bool make_tmap_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t row_stride_el,
                  uint32_t box_inner, uint32_t box_rows);

// 4D tensor map of a page pool [n_pages, page, Hk, d], bf16 or bytes (e4m3 codes), strides in elements:
// dims (d, page, Hk, n_pages), box (128 bytes of d, box_rows, 1, 1), 128-byte swizzle, zeros past the pool.
bool make_tmap_pool(CUtensorMap* m, const void* base, int d, int page, int Hk, int n_pages, long long page_stride,
                    long long row_stride, long long head_stride, int box_rows, bool f8);

long long wait_limit_ns();
int num_sms();
bool device_is_sm100();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Strides (page, row, head, in elements) that a page pool may have: whole 16-byte units.
inline bool pool_strides_ok(const long long* s, int e4m3) {
  const int unit = e4m3 ? 16 : 8;
  for (int i = 0; i < 3; ++i)
    if (s[i] <= 0 || s[i] % unit != 0) return false;
  return true;
}

// Scale of an e4m3 cache: positive, finite, and so is its reciprocal.
inline bool cache_scale_ok(float s) { return s > 0.f && s < HUGE_VALF && 1.f / s < HUGE_VALF; }

// Launches `kernel` on `stream`; with pdl = true the launch may begin while the previous
// kernel on the stream is still running (the kernel must call griddep_wait() before it reads
// anything that kernel wrote, and not by __ldg, whose data may not change from the kernel's start).
// With cluster > 1 the grid's x dimension is cut into clusters of that many blocks.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters_k(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool pdl,
                              int cluster, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = n ? attr : nullptr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}
template <typename... KArgs, typename... Args>
cudaError_t launch_k(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool pdl,
                     Args&&... args) {
  return launch_clusters_k(kernel, grid, block, smem, stream, pdl, 1, std::forward<Args>(args)...);
}

// Launch accounting: every kernel launch site wraps its launch in a LaunchScope, which counts
// the launch and, when per-kernel timing is on for `name`, records CUDA events around it.
class LaunchScope {
 public:
  LaunchScope(const char* name, cudaStream_t stream);
  ~LaunchScope();

 private:
  int slot_;
  cudaStream_t stream_;
  const char* name_;
};

}  // namespace hs2
