// C ABI of include/snapkv_cache.h: argument validation and launches. Every argument error is found
// here, on the host, before anything is enqueued.
#include "../../include/snapkv_cache.h"

#include "abi_common.h"
#include "cache_internal.h"

namespace snapkv {
namespace {

constexpr int64_t kMaxQueries = (int64_t)1 << 22;   // B * Hq of an attention call (32-bit schedules)

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

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

snapkv_status check_sizes(int32_t batch, int32_t heads, int32_t head_dim, int64_t cap) {
  if (batch < 1 || heads < 1 || head_dim < 1 || cap < 1 || cap > kMaxPrompt) return SNAPKV_ERR_INVALID_ARG;
  if ((int64_t)batch * heads > 65535) return SNAPKV_ERR_INVALID_ARG;  // grid.y limit
  if (head_dim != 64 && head_dim != 128) return SNAPKV_ERR_UNSUPPORTED;
  return SNAPKV_OK;
}

bool known_dtype(int32_t dtype) { return dtype == SNAPKV_F32 || dtype == SNAPKV_BF16; }

size_t elem_bytes(int32_t dtype) { return dtype == SNAPKV_BF16 ? 2 : 4; }

snapkv_status check_cache(const snapkv_q4_cache* c) {
  if (!c || !c->k_codes || !c->k_meta || !c->v_codes || !c->v_meta) return SNAPKV_ERR_INVALID_ARG;
  const snapkv_status st = check_sizes(c->batch, c->heads, c->head_dim, c->cap);
  if (st != SNAPKV_OK) return st;
  if (!aligned16(c->k_codes) || !aligned16(c->k_meta) || !aligned16(c->v_codes) || !aligned16(c->v_meta))
    return SNAPKV_ERR_INVALID_ARG;
  return SNAPKV_OK;
}

size_t cache_rows(const snapkv_q4_cache* c) { return (size_t)c->batch * c->heads * (size_t)c->cap; }
size_t codes_bytes(const snapkv_q4_cache* c) { return cache_rows(c) * (c->head_dim / 2); }
size_t meta_bytes(const snapkv_q4_cache* c) { return cache_rows(c) * (c->head_dim / 16); }

// The part of an attention call that the two formats share.
snapkv_status run_attend(AttendJob& job, size_t kv_bytes, size_t kv_meta_bytes, void* workspace,
                         size_t workspace_bytes) {
  if (!job.q || !job.k || !job.v || !job.len || !job.out) return SNAPKV_ERR_INVALID_ARG;
  if (job.q_heads < job.heads || job.q_heads % job.heads != 0) return SNAPKV_ERR_INVALID_ARG;
  if ((int64_t)job.batch * job.q_heads > kMaxQueries) return SNAPKV_ERR_INVALID_ARG;
  if (!known_dtype(job.dtype) || !(job.decay >= 0.f && job.decay <= 1.f)) return SNAPKV_ERR_INVALID_ARG;
  if (!aligned16(job.q) || !aligned16(job.k) || !aligned16(job.v) || !aligned16(job.out) || !aligned16(job.score) ||
      !aligned4(job.len) || !aligned4(job.dev_status))
    return SNAPKV_ERR_INVALID_ARG;
  const size_t need =
      attend_workspace_bytes(job.batch, job.q_heads, job.heads, job.head_dim, job.cap, job.score != nullptr, job.dtype);
  if (need && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))) return SNAPKV_ERR_WORKSPACE;
  const size_t q_bytes = (size_t)job.batch * job.q_heads * job.head_dim * elem_bytes(job.dtype);
  const Span spans[] = {{job.q, q_bytes, false},
                        {job.k, kv_bytes, false},
                        {job.v, kv_bytes, false},
                        {job.k_meta, kv_meta_bytes, false},
                        {job.v_meta, kv_meta_bytes, false},
                        {job.len, (size_t)job.batch * 4, false},
                        {job.score, (size_t)job.batch * job.heads * (size_t)job.cap * 4, true},
                        {job.out, q_bytes, true},
                        {need ? workspace : nullptr, need, true},
                        {job.dev_status, 4, true}};
  if (!disjoint(spans)) return SNAPKV_ERR_INVALID_ARG;
  job.workspace = workspace;
  return launch_attend(job) == cudaSuccess ? SNAPKV_OK : SNAPKV_ERR_CUDA;
}

// The part of an eviction that the two formats share.
snapkv_status run_evict(EvictJob& job, void* workspace, size_t workspace_bytes) {
  if (!job.rows[0] || !job.rows[1] || !job.score || !job.len || !job.len_out) return SNAPKV_ERR_INVALID_ARG;
  if (job.keep < 0 || job.recent < 0 || job.keep > job.cap || job.recent > job.cap || job.keep + job.recent < 1 ||
      job.keep + job.recent > job.cap)
    return SNAPKV_ERR_INVALID_ARG;
  if (!aligned16(job.rows[0]) || !aligned16(job.rows[1]) || !aligned16(job.score) || !aligned4(job.len) ||
      !aligned4(job.len_out) || !aligned4(job.idx) || !aligned4(job.dev_status))
    return SNAPKV_ERR_INVALID_ARG;
  const size_t slots = (size_t)job.batch * job.heads * (size_t)job.cap;
  const size_t need = evict_slots_bytes(job.batch, job.heads, job.cap);
  if (need && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u))) return SNAPKV_ERR_WORKSPACE;
  const Span spans[] = {{job.rows[0], slots * job.row_bytes, true},
                        {job.rows[1], slots * job.row_bytes, true},
                        {job.meta[0], slots * job.meta_bytes, true},
                        {job.meta[1], slots * job.meta_bytes, true},
                        {job.score, slots * 4, true},
                        {job.len, (size_t)job.batch * 4, false},
                        {job.len_out, (size_t)job.batch * 4, true},
                        {job.idx, (size_t)job.batch * job.heads * (size_t)(job.keep + job.recent) * 4, true},
                        {need ? workspace : nullptr, need, true},
                        {job.dev_status, 4, true}};
  if (!disjoint(spans)) return SNAPKV_ERR_INVALID_ARG;
  job.slots = static_cast<int32_t*>(workspace);
  return launch_evict(job) == cudaSuccess ? SNAPKV_OK : SNAPKV_ERR_CUDA;
}

}  // namespace
}  // namespace snapkv

using namespace snapkv;

extern "C" {

size_t snapkv_scored_workspace_size(int32_t batch, int32_t q_heads, int32_t heads, int32_t head_dim, int64_t cap,
                                    int32_t scored) {
  if (check_sizes(batch, heads, head_dim, cap) != SNAPKV_OK) return 0;
  if (q_heads < heads || q_heads % heads != 0 || (int64_t)batch * q_heads > kMaxQueries) return 0;
  const size_t f32 = attend_workspace_bytes(batch, q_heads, heads, head_dim, cap, scored != 0, SNAPKV_F32);
  const size_t bf16 = attend_workspace_bytes(batch, q_heads, heads, head_dim, cap, scored != 0, SNAPKV_BF16);
  return f32 > bf16 ? f32 : bf16;
}

snapkv_status snapkv_decode_attend_scored(const void* q, const void* k_cache, const void* v_cache, int64_t cap,
                                          const int32_t* len, float* score, float decay, void* out, int32_t batch,
                                          int32_t q_heads, int32_t heads, int32_t head_dim, int32_t dtype,
                                          void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                          snapkv_stream_t stream) {
  HostRange nvtx_range("snapkv_decode_attend_scored");
  const snapkv_status st = check_sizes(batch, heads, head_dim, cap);
  if (st != SNAPKV_OK) return st;
  AttendJob job = {};
  job.batch = batch;
  job.q_heads = q_heads;
  job.heads = heads;
  job.head_dim = head_dim;
  job.dtype = dtype;
  job.cap = cap;
  job.q = q;
  job.k = k_cache;
  job.v = v_cache;
  job.len = len;
  job.score = score;
  job.decay = decay;
  job.out = out;
  job.dev_status = dev_status;
  job.stream = reinterpret_cast<cudaStream_t>(stream);
  const size_t kv_bytes = (size_t)batch * heads * (size_t)cap * head_dim * elem_bytes(dtype);
  return run_attend(job, kv_bytes, 0, workspace, workspace_bytes);
}

snapkv_status snapkv_q4_decode_attend(const void* q, const snapkv_q4_cache* cache, const int32_t* len, float* score,
                                      float decay, void* out, int32_t q_heads, int32_t dtype, void* workspace,
                                      size_t workspace_bytes, int32_t* dev_status, snapkv_stream_t stream) {
  HostRange nvtx_range("snapkv_q4_decode_attend");
  const snapkv_status st = check_cache(cache);
  if (st != SNAPKV_OK) return st;
  AttendJob job = {};
  job.batch = cache->batch;
  job.q_heads = q_heads;
  job.heads = cache->heads;
  job.head_dim = cache->head_dim;
  job.dtype = dtype;
  job.cap = cache->cap;
  job.q = q;
  job.k = cache->k_codes;
  job.v = cache->v_codes;
  job.k_meta = cache->k_meta;
  job.v_meta = cache->v_meta;
  job.len = len;
  job.score = score;
  job.decay = decay;
  job.out = out;
  job.dev_status = dev_status;
  job.stream = reinterpret_cast<cudaStream_t>(stream);
  return run_attend(job, codes_bytes(cache), meta_bytes(cache), workspace, workspace_bytes);
}

snapkv_status snapkv_q4_append(const snapkv_q4_cache* cache, const void* k_new, const void* v_new, int64_t rows,
                               const int32_t* n_new, const int32_t* len_in, int32_t* len_out, int32_t dtype,
                               int32_t* dev_status, snapkv_stream_t stream) {
  HostRange nvtx_range("snapkv_q4_append");
  const snapkv_status st = check_cache(cache);
  if (st != SNAPKV_OK) return st;
  if (!k_new || !v_new || !len_in || !len_out || rows < 1 || rows > kMaxPrompt || !known_dtype(dtype))
    return SNAPKV_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned4(n_new) || !aligned4(len_in) || !aligned4(len_out) ||
      !aligned4(dev_status))
    return SNAPKV_ERR_INVALID_ARG;
  const size_t in_bytes = (size_t)cache->batch * cache->heads * (size_t)rows * cache->head_dim * elem_bytes(dtype);
  const Span spans[] = {{k_new, in_bytes, false},
                        {v_new, in_bytes, false},
                        {n_new, (size_t)cache->batch * 4, false},
                        {len_in, (size_t)cache->batch * 4, false},
                        {len_out, (size_t)cache->batch * 4, true},
                        {cache->k_codes, codes_bytes(cache), true},
                        {cache->v_codes, codes_bytes(cache), true},
                        {cache->k_meta, meta_bytes(cache), true},
                        {cache->v_meta, meta_bytes(cache), true},
                        {dev_status, 4, true}};
  if (!disjoint(spans)) return SNAPKV_ERR_INVALID_ARG;
  Q4Job job = {};
  job.batch = cache->batch;
  job.heads = cache->heads;
  job.head_dim = cache->head_dim;
  job.dtype = dtype;
  job.cap = cache->cap;
  job.rows = rows;
  job.codes[0] = cache->k_codes;
  job.codes[1] = cache->v_codes;
  job.meta[0] = cache->k_meta;
  job.meta[1] = cache->v_meta;
  job.in[0] = k_new;
  job.in[1] = v_new;
  job.n_new = n_new;
  job.len = len_in;
  job.len_out = len_out;
  job.dev_status = dev_status;
  job.stream = reinterpret_cast<cudaStream_t>(stream);
  return launch_q4_append(job) == cudaSuccess ? SNAPKV_OK : SNAPKV_ERR_CUDA;
}

snapkv_status snapkv_q4_read(const snapkv_q4_cache* cache, const int32_t* start, int64_t rows, void* k_out,
                             void* v_out, int32_t dtype, snapkv_stream_t stream) {
  HostRange nvtx_range("snapkv_q4_read");
  const snapkv_status st = check_cache(cache);
  if (st != SNAPKV_OK) return st;
  if (!k_out || !v_out || rows < 1 || rows > kMaxPrompt || !known_dtype(dtype)) return SNAPKV_ERR_INVALID_ARG;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned4(start)) return SNAPKV_ERR_INVALID_ARG;
  const size_t out_bytes = (size_t)cache->batch * cache->heads * (size_t)rows * cache->head_dim * elem_bytes(dtype);
  const Span spans[] = {{cache->k_codes, codes_bytes(cache), false},
                        {cache->v_codes, codes_bytes(cache), false},
                        {cache->k_meta, meta_bytes(cache), false},
                        {cache->v_meta, meta_bytes(cache), false},
                        {start, (size_t)cache->batch * 4, false},
                        {k_out, out_bytes, true},
                        {v_out, out_bytes, true}};
  if (!disjoint(spans)) return SNAPKV_ERR_INVALID_ARG;
  Q4Job job = {};
  job.batch = cache->batch;
  job.heads = cache->heads;
  job.head_dim = cache->head_dim;
  job.dtype = dtype;
  job.cap = cache->cap;
  job.rows = rows;
  job.codes[0] = cache->k_codes;
  job.codes[1] = cache->v_codes;
  job.meta[0] = cache->k_meta;
  job.meta[1] = cache->v_meta;
  job.out[0] = k_out;
  job.out[1] = v_out;
  job.len = start;
  job.stream = reinterpret_cast<cudaStream_t>(stream);
  return launch_q4_read(job) == cudaSuccess ? SNAPKV_OK : SNAPKV_ERR_CUDA;
}

size_t snapkv_evict_workspace_size(int32_t batch, int32_t heads, int64_t cap) {
  if (check_sizes(batch, heads, 64, cap) != SNAPKV_OK) return 0;
  return up256(evict_slots_bytes(batch, heads, cap));
}

snapkv_status snapkv_evict(void* k_cache, void* v_cache, int64_t cap, float* score, const int32_t* len_in,
                           int32_t* len_out, int64_t keep, int64_t recent, int32_t* idx_out, int32_t batch,
                           int32_t heads, int32_t head_dim, int32_t dtype, void* workspace, size_t workspace_bytes,
                           int32_t* dev_status, snapkv_stream_t stream) {
  HostRange nvtx_range("snapkv_evict");
  const snapkv_status st = check_sizes(batch, heads, head_dim, cap);
  if (st != SNAPKV_OK) return st;
  if (!known_dtype(dtype)) return SNAPKV_ERR_INVALID_ARG;
  EvictJob job = {};
  job.batch = batch;
  job.heads = heads;
  job.row_bytes = head_dim * (int)elem_bytes(dtype);
  job.cap = cap;
  job.rows[0] = k_cache;
  job.rows[1] = v_cache;
  job.score = score;
  job.len = len_in;
  job.len_out = len_out;
  job.keep = keep;
  job.recent = recent;
  job.idx = idx_out;
  job.dev_status = dev_status;
  job.stream = reinterpret_cast<cudaStream_t>(stream);
  return run_evict(job, workspace, workspace_bytes);
}

snapkv_status snapkv_q4_evict(const snapkv_q4_cache* cache, float* score, const int32_t* len_in, int32_t* len_out,
                              int64_t keep, int64_t recent, int32_t* idx_out, void* workspace,
                              size_t workspace_bytes, int32_t* dev_status, snapkv_stream_t stream) {
  HostRange nvtx_range("snapkv_q4_evict");
  const snapkv_status st = check_cache(cache);
  if (st != SNAPKV_OK) return st;
  EvictJob job = {};
  job.batch = cache->batch;
  job.heads = cache->heads;
  job.row_bytes = cache->head_dim / 2;
  job.meta_bytes = cache->head_dim / 16;
  job.cap = cache->cap;
  job.rows[0] = cache->k_codes;
  job.rows[1] = cache->v_codes;
  job.meta[0] = cache->k_meta;
  job.meta[1] = cache->v_meta;
  job.score = score;
  job.len = len_in;
  job.len_out = len_out;
  job.keep = keep;
  job.recent = recent;
  job.idx = idx_out;
  job.dev_status = dev_status;
  job.stream = reinterpret_cast<cudaStream_t>(stream);
  return run_evict(job, workspace, workspace_bytes);
}

}  // extern "C"
