/*
 * snapkv_draft.h — C ABI of the SnapKV library's operators for several tokens at a time over a cache: attention of
 * a tree of drafted tokens (and of tokens that read cached states alone), a cache held in 8 bits, and the rows of
 * accepted tokens appended to a cache. They stand beside snapkv_cache.h, whose calls take one token per sequence.
 *
 * A step of speculative decoding: draft T tokens per sequence; in every layer run snapkv_tree_attend with the
 * tokens' own K and V rows (nothing is written to the cache); pick the path that the model accepts; append that
 * path's rows with snapkv_append_rows or snapkv_q8_append.
 *
 * Conventions, status codes and types are those of snapkv.h: device pointers of the current device, dense row-major
 * tensors, 16-byte aligned (lengths, indices, steps and status words: 4; masks: 1), work enqueued on `stream`,
 * nothing allocated, kept or synchronised, argument errors found on the host before anything is enqueued. All sizes
 * are B = batch, H = heads (KV heads), Hq = q_heads (a multiple of H; query heads h*G .. h*G + G - 1, G = Hq / H, share
 * KV head h), d = head_dim (64 or 128), T = tokens; B * H <= 65535, B * Hq * T <= 2^22. An array of a call must not
 * overlap one that the call writes.
 *
 * Every call may be captured into a CUDA graph. Calls that share a workspace (also as nodes of two graphs) must not
 * overlap on the GPU.
 */
#ifndef SNAPKV_DRAFT_H
#define SNAPKV_DRAFT_H

#include "snapkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * snapkv_tree_attend — attention of T tokens per sequence over the cached rows and the tokens' own:
 *   s_r = q[b,i,t] . K_r / sqrt(d),  p = softmax of s over the rows that token t sees,  out[b,i,t] = sum_r p_r V_r
 *   lse[b,i,t] = log of the sum of exp(s_r) over those rows
 * Token t < n_new[b] sees the cached rows r < len[b], and of the drafted rows j < n_new[b] those with mask[b,t,j] != 0
 * (without a mask: j <= t). Without drafted rows it sees the cached rows alone: cross attention to an encoder's
 * states, or a decode step whose row is in the cache already.
 *
 * q        device [B, Hq, T, d]
 * k_cache, v_cache  device [B, H, cap, d]; rows at or past len[b] are not used, whatever they hold
 * len      device int32 [B]; len[b] > cap is clamped to cap and reported as SNAPKV_ERR_CAPACITY; len[b] <= 0: no
 *          cached rows
 * k_new, v_new  device [B, H, T, d], or both NULL: no drafted rows. Rows at or past n_new[b] are not used
 * n_new    device int32 [B], 0 <= n_new[b] <= T (NULL: T everywhere): the tokens that sequence b has. Values outside are
 *          clamped and reported as SNAPKV_ERR_INVALID_ARG
 * mask     device bytes, [B, T, T] with mask_stride = T * T or one [T, T] for all sequences with mask_stride = 0 (NULL:
 *          causal). Needs k_new
 * out      device [B, Hq, T, d]; tokens at or past n_new[b] and tokens that see no row (or whose logits are all -inf)
 *          get zeros
 * lse      device fp32 [B, Hq, T] (NULL: not returned); -inf where out is zeros for one of these reasons
 * dtype    snapkv_dtype of q, k_cache, v_cache, k_new, v_new and out. Products and sums are of fp32 accuracy. In bf16 calls
 *          weights enter the second product rounded: to two bf16 parts (16 bits) in calls of up to 16 query rows (G * T) a KV head
 *          (over 8-bit caches 32), to one (8 bits) in calls of more, which moves an output by 2^-8 sum_r p_r |V_r| at
 *          most. Values that a token sees must be finite, and so must be, in fp32, the sum over the channels of |q_c K_r,c| for
 *          each row and 2^8 times the sum over the rows of |V_r| for each channel (weights times V are summed up before they are
 *          divided by the weights' sum; values of V below 2^89 are small enough for any cache). A NaN or infinity in a drafted row
 *          reaches none of the tokens that do not see the row (of those that do, it makes all outputs NaN where it lies in V of a
 *          bf16 call)
 * workspace device, >= snapkv_tree_workspace_size(...) bytes, 256-byte aligned (contents on entry do not matter); the size
 *          serves calls of either type and format. Where it is 0 (caches of up to 256 rows with up to 16 query rows, G * T,
 *          a KV head; also the answer for invalid sizes) the workspace is not used and may be NULL
 * Sums run in a fixed order: the same call on the same device gives the same bits.
 */
SNAPKV_API size_t snapkv_tree_workspace_size(int32_t batch, int32_t q_heads, int32_t heads, int32_t head_dim,
                                             int32_t tokens, int64_t cap);
SNAPKV_API snapkv_status snapkv_tree_attend(const void* q, const void* k_cache, const void* v_cache, int64_t cap,
                                            const int32_t* len, const void* k_new, const void* v_new,
                                            const int32_t* n_new, const void* mask, int64_t mask_stride, void* out,
                                            float* lse, int32_t batch, int32_t q_heads, int32_t heads,
                                            int32_t head_dim, int32_t tokens, int32_t dtype, void* workspace,
                                            size_t workspace_bytes, int32_t* dev_status, snapkv_stream_t stream);

/*
 * A cache held in 8 bits. A row (of K or of V, d channels) has a step h (fp32) and one byte per channel, its sign in
 * bit 7 and a magnitude u in bits 0 .. 6, and stands for +-u h:
 *   h = fp32(max |x| / 127) of the row (0 where that is below 2^-80), u = rint(|x| / h), ties to even (0 where h = 0)
 * Values must be finite and below 2^48 in size; a row that holds an infinity or NaN reads back as NaN (h is NaN then).
 *
 * k_codes, v_codes  device [B, H, cap, d] bytes
 * k_step, v_step    device fp32 [B, H, cap]
 * (A row costs d + 4 bytes: 132 for d = 128, against 256 in bf16 and 72 in the 4 bits of snapkv_cache.h.)
 */
typedef struct {
  void* k_codes;
  void* k_step;
  void* v_codes;
  void* v_step;
  int64_t cap;        /* rows per head                                                              */
  int32_t batch;
  int32_t heads;
  int32_t head_dim;
} snapkv_q8_cache;

/*
 * snapkv_q8_tree_attend — snapkv_tree_attend over an 8-bit cache: K_cache[r] and V_cache[r] are the values that the
 * rows stand for. dtype is that of q, k_new, v_new and out; arguments and workspace as there. In bf16 calls queries must be
 * below 2^48 in size and the sum over the channels of |q_c k_c| below 2^62 for a drafted row, as queries are scaled on their way
 * to the tensor cores, and outputs on their way back: of a drafted row's weight what is below 2^-81 is lost, and of what a row
 * adds to an output what is below 2^-96.
 */
SNAPKV_API snapkv_status snapkv_q8_tree_attend(const void* q, const snapkv_q8_cache* cache, const int32_t* len,
                                               const void* k_new, const void* v_new, const int32_t* n_new,
                                               const void* mask, int64_t mask_stride, void* out, float* lse,
                                               int32_t q_heads, int32_t tokens, int32_t dtype, void* workspace,
                                               size_t workspace_bytes, int32_t* dev_status, snapkv_stream_t stream);

/*
 * snapkv_append_rows — appends rows to a dense cache: for every sequence b and i < n_b, row pick[b,i] of k_new / v_new (row
 * i without a pick) goes to row len_in[b] + i, and len_out[b] = len_in[b] + n_b. Rows go in as they are.
 *
 * k_new, v_new  device [B, H, rows, d], rows >= 1
 * pick     device int32 [B, picks], picks >= 1 (NULL: rows 0 .. n_b - 1; picks is then not used). A row may be picked
 *          more than once. Every block that writes rows of a sequence reads all of its picks first, which counts where they are
 *          many (16384 picked rows of 32 heads take 95 us, all rows without a pick 85; quantised 101 and 71)
 * n_new    device int32 [B], 0 <= n_new[b] <= picks (rows without a pick) (NULL: n_b = picks, or rows)
 * len_in   device int32 [B]; len_out device int32 [B], must not overlap len_in
 * A sequence whose rows do not fit (or with len_in[b] < 0, n_new[b] out of range, or one of its picks out of 0 ..
 * rows - 1) is left as it was, len_out[b] = len_in[b], and SNAPKV_ERR_CAPACITY (SNAPKV_ERR_INVALID_ARG for n_new and
 * pick) is reported in *dev_status.
 */
SNAPKV_API snapkv_status snapkv_append_rows(void* k_cache, void* v_cache, int64_t cap, const void* k_new,
                                            const void* v_new, int64_t rows, const int32_t* pick, int64_t picks,
                                            const int32_t* n_new, const int32_t* len_in, int32_t* len_out,
                                            int32_t batch, int32_t heads, int32_t head_dim, int32_t dtype,
                                            int32_t* dev_status, snapkv_stream_t stream);

/* snapkv_q8_append — snapkv_append_rows for an 8-bit cache: the rows (of dtype) are quantised as they are written. */
SNAPKV_API snapkv_status snapkv_q8_append(const snapkv_q8_cache* cache, const void* k_new, const void* v_new,
                                          int64_t rows, const int32_t* pick, int64_t picks, const int32_t* n_new,
                                          const int32_t* len_in, int32_t* len_out, int32_t dtype,
                                          int32_t* dev_status, snapkv_stream_t stream);

/*
 * snapkv_q8_read — the values that rows start[b] .. start[b] + rows - 1 of the cache stand for (start NULL: row 0),
 * rounded once to dtype. Rows outside 0 .. cap - 1 are returned as zeros.
 *
 * k_out, v_out  device [B, H, rows, d]
 */
SNAPKV_API snapkv_status snapkv_q8_read(const snapkv_q8_cache* cache, const int32_t* start, int64_t rows, void* k_out,
                                        void* v_out, int32_t dtype, snapkv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SNAPKV_DRAFT_H */
