// launch.cuh -- launches that are set up while the kernel before them in the stream
// ends (programmatic stream serialisation), and kernels' shared memory.
//
// Such a kernel's CTAs start as the last ones of the kernel before leave, instead of
// after all it wrote has been made visible: 2.5 us a call between other kernels on one
// stream (one row for each of 256 users 44.5 -> 41.9 us, reads of 1024 candidates
// 32.8 -> 30.2, a cut history's three launches 91.9 -> 84.5).  The kernel before does nothing
// for it.  (Its asking for them early, as soon as its own CTAs had all begun, measured
// slower where all SMs were full: 88.2 for 86.3.)
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace ikbo {

// Every thread of a kernel launched by launch_behind calls this before it touches global
// memory, and before it returns: it comes back once all before it in the stream has ended
// and can be seen, and what follows in the stream waits for this kernel alone.  Ahead of it,
// at most barriers and shared memory are set up (and what no kernel just before may
// write is read); tensor memory is not taken, which a kernel that still runs may be waiting for.
// Loads behind it are ordinary ones or from L2, not __ldg's: what the kernel before wrote
// has not been read-only for as long as this one runs.
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// An ordinary load, by way of L1, for what many warps read (from L2 alone the reads of 1024 candidates
// took 30.5 us for 29.3; the scans' few, two long histories', 83.9 from L2 and 85.5 so).
template <typename T>
__device__ __forceinline__ T fresh(const T* p) {
  return *p;
}

// Lets a kernel use `bytes` of dynamic shared memory, once on each device (asking each
// time took half a microsecond of a call).  `done` is the kernel's own.
template <typename F>
cudaError_t allow_smem(F* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <typename... Params, typename... Args>
inline cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) cudaGetLastError();  // (reported here, not by the next call)
  return e;
}

}  // namespace ikbo
