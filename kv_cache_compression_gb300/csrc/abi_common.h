// Host-side helpers shared by the C ABI files (abi.cu, cache_abi.cu, draft_abi.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

#include "../../include/snapkv.h"

namespace snapkv {

constexpr int64_t kMaxPrompt = (int64_t)1 << 30;

inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + bn && b0 < a0 + an;
}

inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

struct Span {
  const void* at;
  size_t bytes;
  bool written;
};

// Whether no array that a call writes overlaps another of its arrays (NULL ones are skipped).
template <int N> bool disjoint(const Span (&s)[N]) {
  for (int i = 0; i < N; ++i)
    for (int k = i + 1; k < N; ++k)
      if (s[i].at && s[k].at && (s[i].written || s[k].written) && overlaps(s[i].at, s[i].bytes, s[k].at, s[k].bytes))
        return false;
  return true;
}

// The sizes that every operator on a cache takes.
inline snapkv_status check_sizes(int32_t batch, int32_t heads, int32_t head_dim, int64_t cap) {
  if (batch < 1 || heads < 1 || head_dim < 1 || cap < 1 || cap > kMaxPrompt) return SNAPKV_ERR_INVALID_ARG;
  if ((int64_t)batch * heads > 65535) return SNAPKV_ERR_INVALID_ARG;  // grid.y limit
  if (head_dim != 64 && head_dim != 128) return SNAPKV_ERR_UNSUPPORTED;
  return SNAPKV_OK;
}

inline bool known_dtype(int32_t dtype) { return dtype == SNAPKV_F32 || dtype == SNAPKV_BF16; }

inline size_t elem_bytes(int32_t dtype) { return dtype == SNAPKV_BF16 ? 2 : 4; }

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
