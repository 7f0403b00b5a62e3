// dsa3d_host.cuh -- host helpers of the transformer block's entry points: alignment, overlap and
// launch-size rules shared by dsa3d_block.cu and dsa3d_ffn.cu.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstddef>
#include <cstdint>

#include "dsa3d.h"
#include "dsa3d_timing.cuh"

namespace dsa3d {
namespace host {

inline bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1u)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }
inline size_t elem_size(dsa3d_dtype_t t) { return t == DSA3D_F32 ? 4 : 2; }
inline bool known(dsa3d_dtype_t t) { return t == DSA3D_F32 || t == DSA3D_BF16; }
// Alignment of a tensor whose rows have n elements: 16 bytes, or where rows are no multiple of them what every
// row of a 16-byte aligned tensor keeps, so that a shard may start at any row.  The kernels load such rows by
// pieces of that size at most.
inline unsigned row_alignment(int64_t n, dsa3d_dtype_t t) {
  const uint64_t bytes = (uint64_t)n * elem_size(t);
  return (unsigned)std::min<uint64_t>(16, bytes & (~bytes + 1));
}

struct Range {
  uintptr_t lo, hi;
};
inline Range range_of(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, p ? a + bytes : a};
}
inline bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

// Devices this process has asked about; further ones are looked up on every call.
constexpr int kKnownDevices = 64;

// SMs of the current device (a property that does not change, looked up once per device).
inline int sm_count() {
  static std::atomic<int> known[kKnownDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev < kKnownDevices && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return 1;
  if (dev < kKnownDevices) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// One launch inside the optional per-kernel timer.
template <typename F>
dsa3d_status_t launch(int kernel_id, cudaStream_t st, F&& f) {
  TimedLaunch tl(kernel_id, st);
  f();
  const bool launched = cudaGetLastError() == cudaSuccess;
  return (tl.finish() && launched) ? DSA3D_OK : DSA3D_ERR_CUDA;
}

// A launch whose blocks may start while the stream's previous kernel is still running; the kernel calls
// prior_kernel_done() before it touches what that kernel writes.
template <typename... P, typename... A>
dsa3d_status_t launch_early(int kernel_id, cudaStream_t st, void (*kern)(P...), dim3 grid, dim3 block, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return launch(kernel_id, st, [&] { cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...); });
}

}  // namespace host
}  // namespace dsa3d
