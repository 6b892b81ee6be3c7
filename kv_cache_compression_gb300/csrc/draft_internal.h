// Internal launcher interface between draft_abi.cu and the kernels behind include/snapkv_draft.h.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace snapkv {

// One attention of several tokens a sequence, over a dense cache (k_step null: rows of `dtype`) or one in 8 bits.
struct TreeJob {
  int batch, q_heads, heads, head_dim, tokens, dtype;
  int64_t cap;
  const void* q;
  const void* k;          // rows, or codes
  const void* v;
  const void* k_step;
  const void* v_step;
  const int32_t* len;
  const void* k_new;      // may be null (with v_new)
  const void* v_new;
  const int32_t* n_new;   // may be null
  const void* mask;       // may be null
  int64_t mask_stride;
  void* out;
  float* lse;             // may be null
  void* workspace;        // tree_workspace_bytes(...)
  int32_t* dev_status;
  cudaStream_t stream;
};

size_t tree_workspace_bytes(int batch, int q_heads, int heads, int head_dim, int tokens, int64_t cap);
cudaError_t launch_tree(const TreeJob& job);

// Rows appended to a cache, dense (step[0] null: rows of `dtype`) or in 8 bits, or read out of one in 8 bits.
struct RowJob {
  int batch, heads, head_dim, dtype;
  int64_t cap, rows;      // rows of in (append) or out (read) per head
  int64_t count;          // append: rows of a sequence at most (picks, or rows)
  void* held[2];          // K, V: rows, or codes
  void* step[2];
  const void* in[2];
  void* out[2];
  const int32_t* pick;    // may be null
  const int32_t* n_new;   // may be null
  const int32_t* len;     // append: len_in; read: start, may be null
  int32_t* len_out;
  int32_t* dev_status;
  cudaStream_t stream;
};

cudaError_t launch_append_rows(const RowJob& job);
cudaError_t launch_q8_read(const RowJob& job);

}  // namespace snapkv
