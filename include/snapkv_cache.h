/*
 * snapkv_cache.h — C ABI of the SnapKV library's operators on a cache that is being decoded over:
 * attention that keeps a running score of every cached row, eviction by that score, and a cache
 * held in 4 bits. They go on where snapkv.h ends: snapkv_compress leaves a compressed cache, decoding
 * makes it grow again, and these keep it small.
 *
 * Conventions, status codes and types are those of snapkv.h: device pointers of the current device,
 * dense row-major tensors, 16-byte aligned (lengths, indices and status words: 4), work enqueued on `stream`, nothing allocated, kept or
 * synchronised, argument errors found on the host before anything is enqueued. All sizes are
 * B = batch, H = heads (KV heads), Hq = q_heads (a multiple of H; query heads h*G .. h*G + G - 1,
 * G = Hq / H, share KV head h), d = head_dim (64 or 128); B * H <= 65535, B * Hq <= 2^22. An array of a call
 * must not overlap one that the call writes.
 *
 * Every call may be captured into a CUDA graph. Calls that share a workspace (also as nodes of two
 * graphs) must not overlap on the GPU.
 */
#ifndef SNAPKV_CACHE_H
#define SNAPKV_CACHE_H

#include "snapkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * snapkv_decode_attend_scored — decode attention over a dense cache with grouped queries, which
 * also accumulates how much attention every cached row receives:
 *   s_gr = q_g . K_cache[r] / sqrt(d),  p_gr = softmax over r < len[b],  o_g = sum_r p_gr V_cache[r]
 *   score[b,h,r] = decay * score[b,h,r] + sum over the G queries of head h of p_gr,   r < len[b]
 * With G = 1 and no score it computes what snapkv_decode_attend computes. That one is the faster for the caches of
 * one layer of one sequence (32 heads of 1057 bf16 rows: 8 us, 12 here) and for short ones, this one for lengths that
 * differ much and long caches (64 heads of 8192 to 16384 rows: 65 us, 81 there); the rest are within 2 %.
 *
 * q        device [B, Hq, d]
 * k_cache, v_cache  device [B, H, cap, d]; rows at or past len[b] are not used, whatever they hold
 * len      device int32 [B]; len[b] > cap is clamped to cap and reported as SNAPKV_ERR_CAPACITY;
 *          len[b] <= 0 gives o = 0 and leaves the scores as they were (a query whose logits are all -inf
 *          gives o = 0 too, and adds nothing)
 * score    device fp32 [B, H, cap] (NULL: not accumulated). Entries at or past len[b] are left as
 *          they were, so a caller clears the array once; snapkv_evict keeps them cleared.
 * decay    in [0, 1]: 1 accumulates plain sums; 0 stores this step's weights alone (the old entries
 *          are then not read)
 * out      device [B, Hq, d]
 * dtype    snapkv_dtype of q, k_cache, v_cache and out. Products and sums are of fp32 accuracy: bf16
 *          weights enter the second product as two bf16 parts, fp32 values as three. Visible values must
 *          be finite, fp32 ones below 2^127 in size: as the parts of an infinity are not all infinite, an
 *          output or score that it reaches may be NaN.
 *          A NaN reaches, whatever the lengths, all of a query's outputs (if it is in the query or in a
 *          visible row of K) and the scores of all visible rows of the KV head.
 * workspace device, >= snapkv_scored_workspace_size(...) bytes, 256-byte aligned (contents on entry
 *          do not matter); `scored` says whether a score is given (its logits then need most of the room).
 *          Where the size is 0 (short caches; also the answer for invalid sizes) it is not used and may be NULL. The
 *          size serves calls of either dtype; bf16 calls of 9 to 16 queries a KV head use none, and take NULL, over
 *          caches for which calls of up to 8 use none.
 * Sums run in a fixed order: the same call on the same device gives the same bits.
 */
SNAPKV_API size_t snapkv_scored_workspace_size(int32_t batch, int32_t q_heads, int32_t heads, int32_t head_dim,
                                               int64_t cap, int32_t scored);
SNAPKV_API snapkv_status snapkv_decode_attend_scored(const void* q, const void* k_cache, const void* v_cache,
                                                     int64_t cap, const int32_t* len, float* score, float decay,
                                                     void* out, int32_t batch, int32_t q_heads, int32_t heads,
                                                     int32_t head_dim, int32_t dtype, void* workspace,
                                                     size_t workspace_bytes, int32_t* dev_status,
                                                     snapkv_stream_t stream);

/*
 * A cache held in 4 bits. Each row is split into groups of 64 channels; a group is a step h and a
 * centre z (bf16) and one level t = 2u - 15, u = 0 .. 15, per channel, and stands for z + h t:
 *   h = bf16((max - min) / 30) of the group (0 where that is below 2^-126), z = bf16((max + min) / 2)
 *   u = clamp(rint((x - z) / (2h) + 7.5), 0, 15), ties to even (u = 8 where h = 0)
 * Values must be finite and below 2^48 in size; a group that holds an infinity or NaN reads back as
 * NaN (z and h are NaN then).
 *
 * k_codes, v_codes  device [B, H, cap, d / 2] bytes, 16-byte aligned: d / 8 little-endian 32-bit words
 *          per row, word (d / 64) * ((c % 64) / 8) + c / 64 holding channel c with seven others. Channel
 *          e = c % 8 sits in the low (e even) or high (e odd) 16 bits, pair j = e / 2: the level's sign
 *          (1: negative) at bit {15, 14, 7, 6}[j] and (|t| - 1) / 2 at bits {3, 0, 11, 8}[j] and the two
 *          above.
 * k_meta, v_meta  device [B, H, cap, d / 64, 2] bf16, 16-byte aligned: h, then z
 * (A row costs d / 2 + d / 16 bytes: 72 for d = 128, against 256 in bf16.)
 */
typedef struct {
  void* k_codes;
  void* k_meta;
  void* v_codes;
  void* v_meta;
  int64_t cap;        /* rows per head                                                              */
  int32_t batch;
  int32_t heads;
  int32_t head_dim;
} snapkv_q4_cache;

/*
 * snapkv_q4_append — quantises new rows into the cache: for every sequence b, rows 0 .. n_b - 1 of
 * k_new / v_new go to rows len_in[b] .. len_in[b] + n_b - 1, and len_out[b] = len_in[b] + n_b. One row
 * per sequence is a decode step; a compressed or whole prompt is written at len_in[b] = 0.
 *
 * k_new, v_new  device [B, H, rows, d], rows >= 1
 * n_new    device int32 [B], 0 <= n_new[b] <= rows (NULL: n_b = rows for every sequence)
 * len_in   device int32 [B]; len_out device int32 [B], must not overlap len_in
 * dtype    snapkv_dtype of k_new and v_new
 * A sequence whose rows do not fit (or with len_in[b] < 0, or n_new[b] out of range) is left as it
 * was, len_out[b] = len_in[b], and SNAPKV_ERR_CAPACITY (SNAPKV_ERR_INVALID_ARG for n_new) is reported
 * in *dev_status.
 */
SNAPKV_API snapkv_status snapkv_q4_append(const snapkv_q4_cache* cache, const void* k_new, const void* v_new,
                                          int64_t rows, const int32_t* n_new, const int32_t* len_in,
                                          int32_t* len_out, int32_t dtype, int32_t* dev_status,
                                          snapkv_stream_t stream);

/*
 * snapkv_q4_read — the values that rows start[b] .. start[b] + rows - 1 of the cache stand for
 * (start NULL: row 0), rounded once to dtype. Rows outside 0 .. cap - 1 are returned as zeros.
 *
 * k_out, v_out  device [B, H, rows, d]
 */
SNAPKV_API snapkv_status snapkv_q4_read(const snapkv_q4_cache* cache, const int32_t* start, int64_t rows,
                                        void* k_out, void* v_out, int32_t dtype, snapkv_stream_t stream);

/*
 * snapkv_q4_decode_attend — snapkv_decode_attend_scored over a 4-bit cache: K_cache[r] and V_cache[r]
 * are the values that the rows stand for. Arguments as there; dtype is that of q and out; q must be below
 * 2^56 in size (it is scaled on its way to the tensor cores); the workspace size is
 * snapkv_scored_workspace_size(...) of the cache's sizes.
 */
SNAPKV_API snapkv_status snapkv_q4_decode_attend(const void* q, const snapkv_q4_cache* cache, const int32_t* len,
                                                 float* score, float decay, void* out, int32_t q_heads,
                                                 int32_t dtype, void* workspace, size_t workspace_bytes,
                                                 int32_t* dev_status, snapkv_stream_t stream);

/*
 * snapkv_evict — drops the rows with the least accumulated attention, in place and per head. A
 * sequence with len_in[b] > keep + recent comes down to keep + recent rows; others stay as they are.
 * With n = len_in[b] - recent, for every head:
 *   - of slots 0 .. n - 1 the `keep` of largest score stay (equal scores: the lower slot; NaN counts as
 *     the lowest);
 *   - staying slots below `keep` do not move; the freed slots below `keep`, in ascending order, take
 *     the staying rows from slots keep .. n - 1, in ascending order;
 *   - the last `recent` rows follow in their order, at slots keep .. keep + recent - 1.
 * (Attention does not depend on the order of the rows, so only rows whose slot must change are moved,
 * and the newest rows stay last, in order, for the next call.) Scores move with their rows; the scores
 * of the freed slots keep + recent .. len_in[b] - 1 become 0.
 *
 * k_cache, v_cache  device [B, H, cap, d], changed in place (rows at or past keep + recent keep their bytes)
 * score    device fp32 [B, H, cap], changed in place
 * len_in   device int32 [B] (clamped to cap, reported as SNAPKV_ERR_CAPACITY); len_out device int32 [B],
 *          must not overlap len_in
 * keep, recent  >= 0, 1 <= keep + recent <= cap
 * idx_out  device int32 [B, H, keep + recent] (NULL: not returned): the slot that each slot's row came
 *          from (a sequence that stays as it is gets the identity)
 * workspace device, >= snapkv_evict_workspace_size(...) bytes, 256-byte aligned (contents on entry do not
 *          matter); not used, and may be NULL, where that is 0 (short caches; also the answer for invalid sizes)
 */
SNAPKV_API size_t snapkv_evict_workspace_size(int32_t batch, int32_t heads, int64_t cap);
SNAPKV_API snapkv_status snapkv_evict(void* k_cache, void* v_cache, int64_t cap, float* score,
                                      const int32_t* len_in, int32_t* len_out, int64_t keep, int64_t recent,
                                      int32_t* idx_out, int32_t batch, int32_t heads, int32_t head_dim,
                                      int32_t dtype, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                      snapkv_stream_t stream);

/* snapkv_q4_evict — snapkv_evict of a 4-bit cache (codes and (h, z) pairs are moved as they are). */
SNAPKV_API snapkv_status snapkv_q4_evict(const snapkv_q4_cache* cache, float* score, const int32_t* len_in,
                                         int32_t* len_out, int64_t keep, int64_t recent, int32_t* idx_out,
                                         void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                         snapkv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SNAPKV_CACHE_H */
