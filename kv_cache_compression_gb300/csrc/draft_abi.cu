// C ABI of include/snapkv_draft.h: argument validation and launches. Every argument error is found
// here, on the host, before anything is enqueued.
#include "../../include/snapkv_draft.h"

#include "abi_common.h"
#include "draft_internal.h"

namespace snapkv {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 22;   // B * Hq * T of an attention call (32-bit schedules)

snapkv_status check_cache(const snapkv_q8_cache* c) {
  if (!c || !c->k_codes || !c->k_step || !c->v_codes || !c->v_step) return SNAPKV_ERR_INVALID_ARG;
  const snapkv_status st = check_sizes(c->batch, c->heads, c->head_dim, c->cap);
  if (st != SNAPKV_OK) return st;
  if (!aligned16(c->k_codes) || !aligned4(c->k_step) || !aligned16(c->v_codes) || !aligned4(c->v_step))
    return SNAPKV_ERR_INVALID_ARG;
  return SNAPKV_OK;
}

size_t step_bytes(const snapkv_q8_cache* c) { return (size_t)c->batch * c->heads * (size_t)c->cap * sizeof(float); }
size_t codes_bytes(const snapkv_q8_cache* c) { return (size_t)c->batch * c->heads * (size_t)c->cap * c->head_dim; }

bool known_rows(int32_t batch, int32_t q_heads, int32_t heads, int32_t tokens) {
  if (q_heads < heads || q_heads % heads != 0 || tokens < 1) return false;
  return q_heads <= kMaxRows && (int64_t)batch * q_heads <= kMaxRows && (int64_t)batch * q_heads * tokens <= kMaxRows;
}

// The part of an attention call that the two formats share.
snapkv_status run_tree(const TreeJob& job, size_t kv_bytes, size_t kv_step_bytes, size_t workspace_bytes) {
  if (!job.q || !job.k || !job.v || !job.len || !job.out) return SNAPKV_ERR_INVALID_ARG;
  if (!known_rows(job.batch, job.q_heads, job.heads, job.tokens) || !known_dtype(job.dtype)) return SNAPKV_ERR_INVALID_ARG;
  if (!job.k_new != !job.v_new || (job.mask && !job.k_new)) return SNAPKV_ERR_INVALID_ARG;
  const int64_t square = (int64_t)job.tokens * job.tokens;
  if (job.mask && job.mask_stride != 0 && job.mask_stride != square) return SNAPKV_ERR_INVALID_ARG;
  if (!aligned16(job.q) || !aligned16(job.k) || !aligned16(job.v) || !aligned16(job.k_new) || !aligned16(job.v_new) ||
      !aligned16(job.out) || !aligned4(job.len) || !aligned4(job.n_new) || !aligned4(job.lse) || !aligned4(job.dev_status))
    return SNAPKV_ERR_INVALID_ARG;
  const size_t need = tree_workspace_bytes(job.batch, job.q_heads, job.heads, job.head_dim, job.tokens, job.cap);
  if (need && (!job.workspace || workspace_bytes < need || ((uintptr_t)job.workspace & 255u))) return SNAPKV_ERR_WORKSPACE;
  const size_t rows = (size_t)job.batch * job.q_heads * job.tokens;
  const size_t q_bytes = rows * job.head_dim * elem_bytes(job.dtype);
  const size_t new_bytes = (size_t)job.batch * job.heads * job.tokens * job.head_dim * elem_bytes(job.dtype);
  const Span spans[] = {{job.q, q_bytes, false},
                        {job.k, kv_bytes, false},
                        {job.v, kv_bytes, false},
                        {job.k_step, kv_step_bytes, false},
                        {job.v_step, kv_step_bytes, false},
                        {job.len, (size_t)job.batch * 4, false},
                        {job.k_new, new_bytes, false},
                        {job.v_new, new_bytes, false},
                        {job.n_new, (size_t)job.batch * 4, false},
                        {job.mask, (size_t)(job.mask_stride ? job.batch : 1) * (size_t)square, false},
                        {job.out, q_bytes, true},
                        {job.lse, rows * 4, true},
                        {need ? job.workspace : nullptr, need, true},
                        {job.dev_status, 4, true}};
  if (!disjoint(spans)) return SNAPKV_ERR_INVALID_ARG;
  return launch_tree(job) == cudaSuccess ? SNAPKV_OK : SNAPKV_ERR_CUDA;
}

// The part of an append that the two formats share.
snapkv_status run_append(RowJob& job, int64_t picks, size_t held_bytes, size_t held_step_bytes) {
  if (!job.held[0] || !job.held[1] || !job.in[0] || !job.in[1] || !job.len || !job.len_out) return SNAPKV_ERR_INVALID_ARG;
  if (job.rows < 1 || job.rows > kMaxPrompt || !known_dtype(job.dtype)) return SNAPKV_ERR_INVALID_ARG;
  if (job.pick && (picks < 1 || picks > kMaxPrompt)) return SNAPKV_ERR_INVALID_ARG;
  if (!aligned16(job.held[0]) || !aligned16(job.held[1]) || !aligned16(job.in[0]) || !aligned16(job.in[1]) ||
      !aligned4(job.pick) || !aligned4(job.n_new) || !aligned4(job.len) || !aligned4(job.len_out) ||
      !aligned4(job.dev_status))
    return SNAPKV_ERR_INVALID_ARG;
  job.count = job.pick ? picks : job.rows;
  const size_t in_bytes = (size_t)job.batch * job.heads * (size_t)job.rows * job.head_dim * elem_bytes(job.dtype);
  const size_t seq_bytes = (size_t)job.batch * 4;
  const Span spans[] = {{job.in[0], in_bytes, false},
                        {job.in[1], in_bytes, false},
                        {job.pick, seq_bytes * (size_t)picks, false},
                        {job.n_new, seq_bytes, false},
                        {job.len, seq_bytes, false},
                        {job.len_out, seq_bytes, true},
                        {job.held[0], held_bytes, true},
                        {job.held[1], held_bytes, true},
                        {job.step[0], held_step_bytes, true},
                        {job.step[1], held_step_bytes, true},
                        {job.dev_status, 4, true}};
  if (!disjoint(spans)) return SNAPKV_ERR_INVALID_ARG;
  return launch_append_rows(job) == cudaSuccess ? SNAPKV_OK : SNAPKV_ERR_CUDA;
}

}  // namespace
}  // namespace snapkv

using namespace snapkv;

extern "C" {

size_t snapkv_tree_workspace_size(int32_t batch, int32_t q_heads, int32_t heads, int32_t head_dim, int32_t tokens,
                                  int64_t cap) {
  if (check_sizes(batch, heads, head_dim, cap) != SNAPKV_OK || !known_rows(batch, q_heads, heads, tokens)) return 0;
  return tree_workspace_bytes(batch, q_heads, heads, head_dim, tokens, cap);
}

snapkv_status snapkv_tree_attend(const void* q, const void* k_cache, const void* v_cache, int64_t cap, const int32_t* len,
                                 const void* k_new, const void* v_new, const int32_t* n_new, const void* mask,
                                 int64_t mask_stride, void* out, float* lse, int32_t batch, int32_t q_heads,
                                 int32_t heads, int32_t head_dim, int32_t tokens, int32_t dtype, void* workspace,
                                 size_t workspace_bytes, int32_t* dev_status, snapkv_stream_t stream) {
  HostRange nvtx_range("snapkv_tree_attend");
  const snapkv_status st = check_sizes(batch, heads, head_dim, cap);
  if (st != SNAPKV_OK) return st;
  TreeJob job = {};
  job.batch = batch;
  job.q_heads = q_heads;
  job.heads = heads;
  job.head_dim = head_dim;
  job.tokens = tokens;
  job.dtype = dtype;
  job.cap = cap;
  job.q = q;
  job.k = k_cache;
  job.v = v_cache;
  job.len = len;
  job.k_new = k_new;
  job.v_new = v_new;
  job.n_new = n_new;
  job.mask = mask;
  job.mask_stride = mask_stride;
  job.out = out;
  job.lse = lse;
  job.workspace = workspace;
  job.dev_status = dev_status;
  job.stream = reinterpret_cast<cudaStream_t>(stream);
  return run_tree(job, (size_t)batch * heads * (size_t)cap * head_dim * elem_bytes(dtype), 0, workspace_bytes);
}

snapkv_status snapkv_q8_tree_attend(const void* q, const snapkv_q8_cache* cache, const int32_t* len, const void* k_new,
                                    const void* v_new, const int32_t* n_new, const void* mask, int64_t mask_stride,
                                    void* out, float* lse, int32_t q_heads, int32_t tokens, int32_t dtype,
                                    void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                    snapkv_stream_t stream) {
  HostRange nvtx_range("snapkv_q8_tree_attend");
  const snapkv_status st = check_cache(cache);
  if (st != SNAPKV_OK) return st;
  TreeJob job = {};
  job.batch = cache->batch;
  job.q_heads = q_heads;
  job.heads = cache->heads;
  job.head_dim = cache->head_dim;
  job.tokens = tokens;
  job.dtype = dtype;
  job.cap = cache->cap;
  job.q = q;
  job.k = cache->k_codes;
  job.v = cache->v_codes;
  job.k_step = cache->k_step;
  job.v_step = cache->v_step;
  job.len = len;
  job.k_new = k_new;
  job.v_new = v_new;
  job.n_new = n_new;
  job.mask = mask;
  job.mask_stride = mask_stride;
  job.out = out;
  job.lse = lse;
  job.workspace = workspace;
  job.dev_status = dev_status;
  job.stream = reinterpret_cast<cudaStream_t>(stream);
  return run_tree(job, codes_bytes(cache), step_bytes(cache), workspace_bytes);
}

snapkv_status snapkv_append_rows(void* k_cache, void* v_cache, int64_t cap, const void* k_new, const void* v_new,
                                 int64_t rows, const int32_t* pick, int64_t picks, const int32_t* n_new,
                                 const int32_t* len_in, int32_t* len_out, int32_t batch, int32_t heads,
                                 int32_t head_dim, int32_t dtype, int32_t* dev_status, snapkv_stream_t stream) {
  HostRange nvtx_range("snapkv_append_rows");
  const snapkv_status st = check_sizes(batch, heads, head_dim, cap);
  if (st != SNAPKV_OK) return st;
  RowJob job = {};
  job.batch = batch;
  job.heads = heads;
  job.head_dim = head_dim;
  job.dtype = dtype;
  job.cap = cap;
  job.rows = rows;
  job.held[0] = k_cache;
  job.held[1] = v_cache;
  job.in[0] = k_new;
  job.in[1] = v_new;
  job.pick = pick;
  job.n_new = n_new;
  job.len = len_in;
  job.len_out = len_out;
  job.dev_status = dev_status;
  job.stream = reinterpret_cast<cudaStream_t>(stream);
  return run_append(job, picks, (size_t)batch * heads * (size_t)cap * head_dim * elem_bytes(dtype), 0);
}

snapkv_status snapkv_q8_append(const snapkv_q8_cache* cache, const void* k_new, const void* v_new, int64_t rows,
                               const int32_t* pick, int64_t picks, const int32_t* n_new, const int32_t* len_in,
                               int32_t* len_out, int32_t dtype, int32_t* dev_status, snapkv_stream_t stream) {
  HostRange nvtx_range("snapkv_q8_append");
  const snapkv_status st = check_cache(cache);
  if (st != SNAPKV_OK) return st;
  RowJob job = {};
  job.batch = cache->batch;
  job.heads = cache->heads;
  job.head_dim = cache->head_dim;
  job.dtype = dtype;
  job.cap = cache->cap;
  job.rows = rows;
  job.held[0] = cache->k_codes;
  job.held[1] = cache->v_codes;
  job.step[0] = cache->k_step;
  job.step[1] = cache->v_step;
  job.in[0] = k_new;
  job.in[1] = v_new;
  job.pick = pick;
  job.n_new = n_new;
  job.len = len_in;
  job.len_out = len_out;
  job.dev_status = dev_status;
  job.stream = reinterpret_cast<cudaStream_t>(stream);
  return run_append(job, picks, codes_bytes(cache), step_bytes(cache));
}

snapkv_status snapkv_q8_read(const snapkv_q8_cache* cache, const int32_t* start, int64_t rows, void* k_out, void* v_out,
                             int32_t dtype, snapkv_stream_t stream) {
  HostRange nvtx_range("snapkv_q8_read");
  const snapkv_status st = check_cache(cache);
  if (st != SNAPKV_OK) return st;
  if (!k_out || !v_out || rows < 1 || rows > kMaxPrompt || !known_dtype(dtype)) return SNAPKV_ERR_INVALID_ARG;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned4(start)) return SNAPKV_ERR_INVALID_ARG;
  const size_t out_bytes = (size_t)cache->batch * cache->heads * (size_t)rows * cache->head_dim * elem_bytes(dtype);
  const Span spans[] = {{cache->k_codes, codes_bytes(cache), false},
                        {cache->k_step, step_bytes(cache), false},
                        {cache->v_codes, codes_bytes(cache), false},
                        {cache->v_step, step_bytes(cache), false},
                        {start, (size_t)cache->batch * 4, false},
                        {k_out, out_bytes, true},
                        {v_out, out_bytes, true}};
  if (!disjoint(spans)) return SNAPKV_ERR_INVALID_ARG;
  RowJob job = {};
  job.batch = cache->batch;
  job.heads = cache->heads;
  job.head_dim = cache->head_dim;
  job.dtype = dtype;
  job.cap = cache->cap;
  job.rows = rows;
  job.held[0] = cache->k_codes;
  job.held[1] = cache->v_codes;
  job.step[0] = cache->k_step;
  job.step[1] = cache->v_step;
  job.out[0] = k_out;
  job.out[1] = v_out;
  job.len = start;
  job.stream = reinterpret_cast<cudaStream_t>(stream);
  return launch_q8_read(job) == cudaSuccess ? SNAPKV_OK : SNAPKV_ERR_CUDA;
}

}  // extern "C"
