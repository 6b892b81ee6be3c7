// Kernels that take rows into and out of a cache, 4-bit, 8-bit or dense: which rows a thread has, and the grid.
#pragma once

#include "snapkv_common.cuh"
#include "snapkv_internal.h"

namespace snapkv {

constexpr int kRowThreads = 128;   // (writing a bf16 prompt of 16384 rows and 32 heads in 4 bits: 73 us, 77 with 256, 81 with 512)

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 two = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&two);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// The rows of a launch. Long calls have a head per blockIdx.y, whose blocks take turns; calls of few rows
// (FLAT) are one list of `flat_rows` rows over all heads, as a head's rows would leave most of a block idle.

// Calls f(head, row, mine, seq(sequence)) for this thread's rows, the whole warp at once (mine false: some other
// row that exists). seq, what a row needs to know of its sequence, is asked once per head where it can be.
template <bool FLAT, int TPR, typename Seq, typename F>
__device__ __forceinline__ void for_rows(unsigned flat_rows, int heads, int64_t rows, Seq seq, F f) {
  constexpr int kRows = kRowThreads / TPR;
  if constexpr (FLAT) {
    const unsigned at = blockIdx.x * kRows + threadIdx.x / TPR;
    const bool mine = at < flat_rows;
    const unsigned bh = mine ? at / (unsigned)rows : 0u;
    f(bh, (int)(mine ? at - bh * (unsigned)rows : 0u), mine, seq((int)(bh / (unsigned)heads)));
  } else {
    const unsigned bh = blockIdx.y;
    const auto known = seq((int)(bh / (unsigned)heads));
    for (int r0 = (int)blockIdx.x * kRows; r0 < (int)rows; r0 += (int)gridDim.x * kRows) {
      const int row = r0 + (int)threadIdx.x / TPR;
      f(bh, row < (int)rows ? row : 0, row < (int)rows, known);
    }
  }
}

constexpr int64_t kFlatRows = 32;   // calls of fewer rows a head are one list

// Blocks and threads: a flat list of few rows; else all blocks together are about `waves` waves of sixteen per
// SM, so that a long prompt amortises a block's set-up over several turns. Writing a bf16 prompt of 16384 rows
// and 32 heads (K and V: 344 MB of traffic, 51 us at 6.79 TB/s) takes 74 us in 2 waves, 77 in 1 and (in
// blocks of 256 threads) 82 in 8; reading it back 79 in 2, 58 in 8 and 61 in 24. One row of 2048 heads: 3.0
// and 2.3 us, 9.5 with a block per head.
inline dim3 row_grid(int batch, int heads, int64_t rows, int threads_per_row, int waves) {
  const int per_turn = kRowThreads / threads_per_row;
  const int64_t bh = (int64_t)batch * heads;
  if (rows < kFlatRows) return dim3((unsigned)((bh * rows + per_turn - 1) / per_turn), 1, 2);
  const int64_t turns = (rows + per_turn - 1) / per_turn;
  int64_t blocks = ((int64_t)device_sm_count() * 16 * waves + 2 * bh - 1) / (2 * bh);
  if (blocks > turns) blocks = turns;
  return dim3((unsigned)(blocks < 1 ? 1 : blocks), (unsigned)bh, 2);
}

}  // namespace snapkv
