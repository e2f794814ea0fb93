// Launching kernels that take one argument block.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>

namespace twell {

// kernel(a) on a stream.  One call of the runtime: <<<>>> makes three, which take
// the host 0.2 to 0.3 us longer, of some 3.5, and a call of small kernels is as long
// as the host takes for it.
template <class Args>
hipError_t launch(void (*kernel)(Args), dim3 grid, unsigned threads, size_t lds, hipStream_t s, Args a) {
  void* args[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), args, lds, s);
}

// The same for a kernel that is handed LDS at launch, kMost bytes at the most.  More
// than 64 KB together with what the kernel declares itself has to be asked for, which
// the first launch does (a process drives one GPU).  A refusal goes to the caller, and
// the next call asks again.
template <auto kKernel, size_t kMost, class Args>
hipError_t launch_lds(dim3 grid, unsigned threads, size_t lds, hipStream_t s, const Args& a) {
  static std::atomic<bool> allowed{false};
  if (!allowed.load(std::memory_order_relaxed)) {
    const void* kernel = reinterpret_cast<const void*>(kKernel);
    hipFuncAttributes f{};
    hipError_t e = hipFuncGetAttributes(&f, kernel);
    if (e == hipSuccess && f.sharedSizeBytes + kMost > 64 * 1024)
      e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMost));
    if (e != hipSuccess) return e;
    allowed.store(true, std::memory_order_relaxed);
  }
  return launch(kKernel, grid, threads, lds, s, a);
}

}  // namespace twell
