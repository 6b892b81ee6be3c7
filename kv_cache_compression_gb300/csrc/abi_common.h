// Host-side helpers shared by the C ABI files (abi.cu, cache_abi.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

namespace snapkv {

constexpr int64_t kMaxPrompt = (int64_t)1 << 30;

inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + bn && b0 < a0 + an;
}

// An NVTX range around an entry point's host work (validation and enqueueing), so that a profiler's
// timeline shows which library call enqueued which kernels; without a tool attached it costs a few
// nanoseconds.
struct HostRange {
  explicit HostRange(const char* name) { nvtxRangePushA(name); }
  ~HostRange() { nvtxRangePop(); }
  HostRange(const HostRange&) = delete;
  HostRange& operator=(const HostRange&) = delete;
};

}  // namespace snapkv
