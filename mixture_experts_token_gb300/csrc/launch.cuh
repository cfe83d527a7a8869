// Host-side launch helpers shared by the block norms and the 4-bit products:
// device properties and kernel occupancy, asked for once and kept (they
// belong to the device and the kernel, not to a call's data), and a launch
// that may begin while the kernel before it drains.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace moe {
namespace launch {

constexpr int kMaxDevices = 64;

struct Device {
  int id = 0, sms = 0;
  int smem_sm = 0;   // shared memory of an SM
  int smem_cta = 0;  // the most that one CTA may have
};

inline cudaError_t device(Device* d) {
  static std::atomic<uint64_t> known[kMaxDevices];
  cudaError_t e = cudaGetDevice(&d->id);
  if (e != cudaSuccess) return e;
  if (d->id < 0 || d->id >= kMaxDevices) return cudaErrorInvalidDevice;
  uint64_t v = known[d->id].load(std::memory_order_relaxed);
  if (v == 0) {
    int sms = 0, sm = 0, cta = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount,
                                    d->id)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(
             &sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, d->id)) !=
            cudaSuccess ||
        (e = cudaDeviceGetAttribute(
             &cta, cudaDevAttrMaxSharedMemoryPerBlockOptin, d->id)) !=
            cudaSuccess)
      return e;
    v = static_cast<uint64_t>(sms) << 48 | static_cast<uint64_t>(sm) << 24 |
        static_cast<uint64_t>(cta);
    known[d->id].store(v, std::memory_order_relaxed);
  }
  d->sms = static_cast<int>(v >> 48);
  d->smem_sm = static_cast<int>(v >> 24 & 0xffffff);
  d->smem_cta = static_cast<int>(v & 0xffffff);
  return cudaSuccess;
}

// Lets the kernel have as much dynamic shared memory as the device gives.
// Every call of a kernel sets the same limit, so calls of other threads with
// other sizes cannot get in between.
template <auto Kernel>
cudaError_t allow_shared(const Device& d) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = 1ull << d.id;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, Kernel);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(
        Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        d.smem_cta - static_cast<int>(at.sharedSizeBytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// CTAs of the kernel that fit on an SM (at least 1).  The last answer is
// kept: calls repeat with the same shape.
template <auto Kernel>
cudaError_t ctas_per_sm(const Device& d, int threads, int bytes, int* n) {
  static std::atomic<uint64_t> last{0};
  const uint64_t key = static_cast<uint64_t>(d.id + 1) << 48 |
                       static_cast<uint64_t>(threads) << 32 |
                       static_cast<uint64_t>(bytes) << 8;
  const uint64_t v = last.load(std::memory_order_relaxed);
  if (v >> 8 == key >> 8) {
    *n = static_cast<int>(v & 255);
    return cudaSuccess;
  }
  int fit = 0;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
      &fit, Kernel, threads, bytes);
  if (e != cudaSuccess) return e;
  *n = fit < 1 ? 1 : fit;
  last.store(key | static_cast<uint64_t>(*n), std::memory_order_relaxed);
  return cudaSuccess;
}

// Launches a kernel whose CTAs may start while those of the kernel before it
// on the stream finish; the kernel calls wait_for_previous() before it reads
// or writes anything of that kernel's.
template <typename... P, typename... A>
cudaError_t overlapping(void (*kernel)(P...), dim3 grid, dim3 block,
                        int bytes, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = static_cast<size_t>(bytes);
  c.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// All of the kernels before this one have ended and their writes are seen.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// The next kernel on the stream may begin to start.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace launch
}  // namespace moe
