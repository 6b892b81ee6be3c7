// Internal launcher interface between cache_abi.cu and the kernels behind include/snapkv_cache.h.
#pragma once

#include <atomic>

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace snapkv {

// Lets `kernel` take `bytes` of dynamic shared memory on the current device (the attribute belongs to
// the kernel's instance on a device; it is set on the first launch there).
template <auto* Kernel> cudaError_t allow_dynamic_smem(int bytes) {
  static std::atomic<uint64_t> done{0};   // one bit per device
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  err = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return err;
}

constexpr int kMaxQueryTile = 16;   // query heads of one KV head that one pass over its rows serves, at most

// One scored decode attention, dense (k_meta null: k, v of `dtype`) or over a 4-bit cache.
struct AttendJob {
  int batch, q_heads, heads, head_dim, dtype;
  int64_t cap;
  const void* q;
  const void* k;        // rows, or codes
  const void* v;
  const void* k_meta;
  const void* v_meta;
  const int32_t* len;
  float* score;         // may be null
  float decay;
  void* out;
  void* workspace;      // attend_workspace_bytes(...)
  int32_t* dev_status;
  cudaStream_t stream;
};

// Workspace layout of an attention call (byte offsets, each 256-aligned), and how its queries are cut.
struct AttendLayout {
  size_t parts, stats, upto, logits, total;
  int64_t logit_stride;
  int tile_q, passes, max_ctas;
  bool direct;          // a CTA per head in one launch, without workspace
};

// Caches of up to this many rows leave a head to one CTA, in one launch: 4 heads of 83 fp32 rows take 5.7 us so
// and 9.0 in two launches, 4 heads of 1000 4-bit rows 12.0 and 8.0.
constexpr int kDirectRows = 256;

constexpr int kMaxAttendCtas = 1024;   // bounds the workspace, not tied to a device's SM count

// The layout for passes of at most `most_q` queries, and the workspace that a call of a type needs.
AttendLayout attend_layout(int batch, int q_heads, int heads, int head_dim, int64_t cap, bool scored, int most_q);
size_t attend_workspace_bytes(int batch, int q_heads, int heads, int head_dim, int64_t cap, bool scored, int dtype);
cudaError_t launch_attend(const AttendJob& job);

struct Q4Job {
  int batch, heads, head_dim, dtype;
  int64_t cap, rows;
  void* codes[2];       // K, V
  void* meta[2];
  const void* in[2];    // append: rows [B, H, rows, d]
  void* out[2];         // read: rows [B, H, rows, d]
  const int32_t* n_new; // append; may be null
  const int32_t* len;   // append: len_in; read: start, may be null
  int32_t* len_out;
  int32_t* dev_status;
  cudaStream_t stream;
};

cudaError_t launch_q4_append(const Q4Job& job);
cudaError_t launch_q4_read(const Q4Job& job);

struct EvictJob {
  int batch, heads, row_bytes, meta_bytes;   // of one row of K or of V (meta_bytes 0: none)
  int64_t cap;
  void* rows[2];        // K, V (or their codes)
  void* meta[2];
  float* score;
  const int32_t* len;
  int32_t* len_out;
  int64_t keep, recent;
  int32_t* idx;         // may be null
  int32_t* slots;       // workspace [B*H][cap]
  int32_t* dev_status;
  cudaStream_t stream;
};

// Bytes of slot lists that an eviction needs: none for caches whose heads each get one CTA and whose moves
// always fit its shared-memory list.
constexpr int64_t kEvictNoListCap = 2048;
inline size_t evict_slots_bytes(int batch, int heads, int64_t cap) {
  return cap <= kEvictNoListCap ? 0 : (size_t)batch * heads * (size_t)cap * sizeof(int32_t);
}

cudaError_t launch_evict(const EvictJob& job);

}  // namespace snapkv
