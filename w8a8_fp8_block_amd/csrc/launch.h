// Host side of a kernel launch, shared by the kernel sources.
#pragma once

#include <atomic>

#include <hip/hip_runtime.h>

namespace fp8q {
namespace {

// Dynamic LDS beyond the default, allowed once a kernel.
template <auto kernel, int BYTES>
hipError_t allow_lds() {
  static std::atomic<bool> done{false};  // idempotent: racing threads repeat it
  if (done.load(std::memory_order_acquire)) return hipSuccess;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, BYTES);
  if (e == hipSuccess) done.store(true, std::memory_order_release);
  return e;
}

}  // namespace
}  // namespace fp8q
