// Host side of the tree attention (see tree_schedule.cuh): workspace, the cut of a call, and which kernel takes it.
#include <math.h>

#include "tc_common.cuh"
#include "tree_launch.h"
#include "tree_maps.h"
#include "tree_schedule.cuh"

namespace snapkv {
namespace {

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

// Tiles of a call that are possible, all passes apart.
int64_t most_tiles(int batch, int heads, int64_t passes, int tokens, int64_t cap, int tile, int fresh) {
  return (int64_t)batch * heads * passes * ((cap + tile - 1) / tile + (tokens + fresh - 1) / fresh);
}

size_t upto_bytes(int batch) { return up(((size_t)batch + 1) * sizeof(int64_t)); }
// Short caches of few rows leave a head to one CTA, in one launch and without workspace. One limit for both types, as a call's
// workspace does not depend on its type. bf16 calls gain on both sides of it (128 channels, one query, 32 heads: 256 rows 8.3 us,
// 12.9 with a list and a joining launch; 512 rows 11.3 and 14.0; 1024 rows 17.1 and 15.8; over 8 bits 7.8 and 14.6, 10.6 and 15.9, 14.7
// and 17.3). fp32 calls gain up to 64 rows (8.2 us, 11.2) and, where heads are many, up to 256 (512 heads 48 and 52); few heads of 256
// rows lose by it (one query of 32 heads 16.7 and 14.1, sixteen 27.6 and 17.1).
bool is_direct(int64_t rows, int64_t cap) { return rows <= 16 && cap <= 256; }

// Query rows a KV head up to which bf16 calls take mma.sync. Dense caches: a pass of it, which memory bounds (sixteen rows over
// 131072 keys of eight heads 92 us, where 32 rows on tcgen05 take 94; two passes would read everything twice). 8-bit caches: two
// passes, of which the second reads from L2, against tcgen05's unpacking into shared memory: 64 x 32 heads of 20 rows over
// 2140 keys 550 us against 577, 8 x 8 heads of 32 rows over 16384 keys of 64 channels 77 against 91 (32 rows over 131072 keys 108
// against 102); but 64 rows 199 against 105.
constexpr int kMmaRows = 16, kMmaRowsQ8 = 32;
constexpr size_t kCutBytes = (size_t)kMaxTreeCtas * 2 * sizeof(int4);
static_assert(kCutBytes % 256 == 0, "parts follow");

// A CTA's two parts.
size_t part_bytes(int tile_q, int head_dim) { return (size_t)2 * tile_q * (head_dim + 2) * sizeof(float); }
size_t parts_bytes(int64_t ctas, int tile_q, int head_dim) { return up((size_t)ctas * part_bytes(tile_q, head_dim)); }

int64_t bounded(int64_t tiles, int64_t most) { return tiles < most ? tiles : most; }

}  // namespace

size_t tree_workspace_bytes(int batch, int q_heads, int heads, int head_dim, int tokens, int64_t cap) {
  const int64_t rows = (int64_t)(q_heads / heads) * tokens;
  if (is_direct(rows, cap)) return 0;
  const int simt = rows <= 8 ? 8 : kSimtRows;
  size_t parts = parts_bytes(bounded(most_tiles(batch, heads, (rows + simt - 1) / simt, tokens, cap, 16, 16), kMaxTreeCtas), simt, head_dim);
  if (rows > kMmaRows) {
    const int wide = rows <= 128 ? 128 : 256;   // (where more rows go in passes of 128, there are at most twice as many of half the parts)
    const size_t tc = parts_bytes(bounded(most_tiles(batch, heads, (rows + wide - 1) / wide, tokens, cap, 128, 128), kMaxTcCtas), wide, head_dim);
    parts = tc > parts ? tc : parts;
  }
  return upto_bytes(batch) + kCutBytes + parts;
}

tree::Args tree_args(const TreeJob& job, int tile_q) {
  tree::Args a = {};
  a.q = job.q;
  a.k = job.k;
  a.v = job.v;
  a.k_step = static_cast<const float*>(job.k_step);
  a.v_step = static_cast<const float*>(job.v_step);
  a.len = job.len;
  a.k_new = job.k_new;
  a.v_new = job.v_new;
  a.n_new = job.n_new;
  a.mask = static_cast<const uint8_t*>(job.mask);
  a.mask_stride = job.mask_stride;
  a.out = job.out;
  a.lse = job.lse;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)job.head_dim));
  a.cap = job.cap;
  a.batch = job.batch;
  a.heads = job.heads;
  a.group = job.q_heads / job.heads;
  a.tokens = job.tokens;
  a.tile_q = tile_q;
  a.siblings = 1;
  a.least = 1;
  a.direct = is_direct((int64_t)a.group * a.tokens, a.cap);
  a.dev_status = job.dev_status;
  return a;
}

cudaError_t tree_fill(tree::Args& a, const TreeJob& job, int tile, int fresh, int64_t ctas) {
  if (a.direct) {
    a.ctas = a.batch * a.heads;
    return cudaSuccess;
  }
  const int64_t rows = (int64_t)a.group * a.tokens, passes = (rows + a.tile_q - 1) / a.tile_q;
  // No more CTAs than there are parts and notes for in the workspace, whatever a launcher asks for.
  const size_t room = tree_workspace_bytes(job.batch, job.q_heads, job.heads, job.head_dim, job.tokens, job.cap) - upto_bytes(a.batch) - kCutBytes;
  const int64_t fit = bounded((int64_t)(room / part_bytes(a.tile_q, job.head_dim)), kMaxTreeCtas);
  a.ctas = (int)bounded(bounded(ctas, fit), most_tiles(a.batch, a.heads, passes, a.tokens, a.cap, tile, fresh));
  a.ctas -= a.ctas % a.siblings;
  char* ws = static_cast<char*>(job.workspace);
  a.upto = reinterpret_cast<int64_t*>(ws);
  a.cuts = reinterpret_cast<int4*>(ws + upto_bytes(a.batch));
  a.parts = reinterpret_cast<float*>(ws + upto_bytes(a.batch) + kCutBytes);
  return cudaSuccess;
}

namespace {

bool code_map(CUtensorMap* map, const void* codes, const TreeJob& job, int tile) {
  auto enc = tc::encode_fn();
  if (!enc) return false;
  const int d = job.head_dim;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)job.cap, (cuuint64_t)job.batch * job.heads};
  const cuuint64_t strides[2] = {(cuuint64_t)d, (cuuint64_t)job.cap * d};
  const cuuint32_t box[3] = {(cuuint32_t)d, (cuuint32_t)tile, 1}, one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool tree_maps(TreeMaps* maps, const TreeJob& job, int tile, int fresh) {
  const int64_t bh = (int64_t)job.batch * job.heads;
  if (job.k_step) {
    if (!code_map(&maps->k, job.k, job, tile) || !code_map(&maps->v, job.v, job, tile)) return false;
  } else if (!tc::make_map(&maps->k, job.k, job.head_dim, job.cap, bh, tile) ||
             !tc::make_map(&maps->v, job.v, job.head_dim, job.cap, bh, tile)) {
    return false;
  }
  if (!tc::make_map(&maps->q, job.q, job.head_dim, (int64_t)job.batch * job.q_heads * job.tokens, 1, tile)) return false;
  if (!job.k_new) {
    maps->k_new = maps->k;
    maps->v_new = maps->v;
    return true;
  }
  return tc::make_map(&maps->k_new, job.k_new, job.head_dim, job.tokens, bh, fresh) &&
         tc::make_map(&maps->v_new, job.v_new, job.head_dim, job.tokens, bh, fresh);
}

cudaError_t launch_tree(const TreeJob& job) {
  if (job.dtype == SNAPKV_F32) return launch_tree_simt(job);
  const int64_t rows = (int64_t)(job.q_heads / job.heads) * job.tokens;
  return rows <= (job.k_step ? kMmaRowsQ8 : kMmaRows) ? launch_tree_mma(job) : launch_tree_tc(job);
}

}  // namespace snapkv
