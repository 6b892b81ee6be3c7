// What the kernels of the tree attention share: a call's arguments, how its work is cut, and the parts that are joined.
//
// The query rows of a KV head are (g, t), g < G query heads, t < n tokens that the sequence has: r = g n + t of M = G n.
// A pass serves QT of them. The keys of a head are cut into tiles of TILE cached rows and, after those, NEW drafted rows.
// All tiles of all heads (and passes) are one flat list, of which every share takes an equal, contiguous piece, whatever
// the sequences' lengths: the end of one head, whole heads, the start of another. A head that lies in one share is
// finished there; of others the shares leave parts (outputs not yet normalised, maxima, sums), and a second launch joins
// them. Fixed order, no atomics: repeats give the same bits.
//
// With `siblings` = P > 1 the list has each head once, not once a pass, and a share belongs to P CTAs, a pass each, that
// walk the same tiles side by side, so that all but the first read them from L2.
#pragma once

#include "draft_internal.h"
#include "snapkv_common.cuh"

namespace snapkv {
namespace tree {

struct Args {
  const void* q;
  const void* k;
  const void* v;
  const float* k_step;
  const float* v_step;
  const int32_t* len;
  const void* k_new;
  const void* v_new;
  const int32_t* n_new;
  const uint8_t* mask;
  int64_t mask_stride;
  void* out;
  float* lse;
  float scale_log2;     // log2(e) / sqrt(d)
  int64_t cap;
  int batch, heads, group, tokens;
  int tile_q;           // query rows of a pass (of a part)
  int ctas, siblings;   // of the first launch; shares = ctas / siblings
  int least;            // tiles that a share has at least, where there are as many
  bool direct;          // a CTA per head, which finishes it: no list, workspace or joining launch
  // workspace
  int64_t* upto;        // [batch + 1]: tiles in the sequences before, and in all
  int4* cuts;           // [shares][2]: (sequence, head, pass, tile), (tiles, tokens, -, -) where a share is the first to begin
                        // inside a head; else tile 0
  float* parts;         // [ctas][2] of (o [tile_q][D] or [D][tile_q], m [tile_q] (log2 domain), l [tile_q])
  int32_t* dev_status;
};

constexpr float kNoMax = -3.402823466e38f;   // the lowest finite value, so that differences to it are no NaN

// 8-bit codes as operands of bf16 products are subnormal: sign and magnitude stand for u 2^-133. Queries and weights carry the powers
// of two that bring products back; with drafted rows, whose values are as they are, others do.
constexpr float kQ8Q = 0x1p64f;                         // queries
constexpr float kQ8Dot = 0x1p69f;                       // undoes 2^64 2^-133
constexpr float kQ8P = 0x1p80f;                         // weights
constexpr float kQ8Out = 0x1p53f;                       // undoes 2^80 2^-133
constexpr float kNewDot = 0x1p-64f, kNewP = 0x1p-53f;   // drafted rows'

__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 two = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&two);
}

__device__ __forceinline__ int cached_rows(const Args& a, int b) {
  const int n = a.len[b];
  return n < 0 ? 0 : (int64_t)n > a.cap ? (int)a.cap : n;
}
__device__ __forceinline__ int tokens_of(const Args& a, int b) {
  const int n = a.n_new ? a.n_new[b] : a.tokens;
  return n < 0 ? 0 : n > a.tokens ? a.tokens : n;
}

// A sequence: its cached rows, tokens, passes in the list and tiles of a pass.
struct Seq {
  int rows, n, passes, cache_tiles, tiles;
  __device__ __forceinline__ int64_t units(int heads) const { return (int64_t)heads * passes * tiles; }
};
template <int TILE, int NEW> __device__ __forceinline__ Seq seq_of(const Args& a, int b) {
  Seq s;
  s.rows = cached_rows(a, b);
  s.n = tokens_of(a, b);
  s.passes = a.siblings > 1 ? 1 : (a.group * s.n + a.tile_q - 1) / a.tile_q;
  s.cache_tiles = (s.rows + TILE - 1) / TILE;
  s.tiles = s.n == 0 ? 0 : s.cache_tiles + (a.k_new ? (s.n + NEW - 1) / NEW : 0);
  return s;
}

__device__ __forceinline__ int working_shares(const Args& a, int64_t total) {
  const int64_t shares = a.ctas / a.siblings, most = (total + a.least - 1) / a.least;
  return (int)(most < shares ? most : shares);
}
// (c <= shares <= 320 and total <= 2^52: no product overflows; short lists, where the latency counts, get by with a
// 32-bit division)
__device__ __forceinline__ int64_t share_start(int64_t total, int shares, int c) {
  if (total < (1 << 23)) return (uint32_t)total * (uint32_t)c / (uint32_t)shares;
  return total * c / shares;
}
// The share that holds flat tile t: the last one that starts at or before it.
__device__ __forceinline__ int share_of(int64_t total, int shares, int64_t t) {
  int c = total < (1 << 23) ? (int)((uint32_t)t * (uint32_t)shares / (uint32_t)total) : (int)(t * shares / total);
  while (c + 1 < shares && share_start(total, shares, c + 1) <= t) ++c;   // (the quotient's share starts at or before t)
  return c;
}

// A place in the list: a tile of a head's pass, and what its sequence is.
struct Place {
  int seq, head, pass, tile;
  Seq s;
};
// The place of tile `in` of the sequence p.seq (with p.s).
__device__ __forceinline__ void place_at(Place& p, int64_t in) {
  const int64_t unit = in < ((int64_t)1 << 31) ? (int64_t)((uint32_t)in / (uint32_t)p.s.tiles) : in / p.s.tiles;
  p.tile = (int)(in - unit * p.s.tiles);
  const uint32_t u = (uint32_t)unit;   // (heads and passes: 65535 by 2^22 at most, and fewer than 2^31 together)
  p.head = (int)(u / (uint32_t)p.s.passes);
  p.pass = (int)(u - (uint32_t)p.head * (uint32_t)p.s.passes);
}
// Where a CTA's share lies: tiles at .. end - 1 of the list.
struct Share {
  int64_t at, end;
  int64_t previous;   // where the share before begins (the first one's: its own)
  Place first;        // of tile `at`
};

// All threads of a block of THREADS find their CTA's share (at == end: none). Sequence lengths are summed up by every
// CTA for itself, of up to 32 sequences by every warp (with a block's
// exchanges, and each role of tree_tc.cu looking for the first place by itself, 64 rows over 16384 keys of 64 heads took 85 us, 80 so); CTA 0 leaves the sums for the joining launch and reports what is
// out of range.
template <int THREADS> struct ShareScratch {   // shared memory
  int64_t warp_sums[THREADS / 32];
  Share found;
};
template <int TILE, int NEW, int THREADS> __device__ __forceinline__ Share find_share(const Args& a, ShareScratch<THREADS>& scratch) {
  const int tid = threadIdx.x, lane = tid % 32;
  auto note = [&](int b, int64_t sum) {   // (CTA 0)
    a.upto[b] = sum;
    if ((int64_t)a.len[b] > a.cap) report(a.dev_status, SNAPKV_ERR_CAPACITY);
    if (a.n_new && (a.n_new[b] < 0 || a.n_new[b] > a.tokens)) report(a.dev_status, SNAPKV_ERR_INVALID_ARG);
  };
  if (a.batch <= 32) {
    Seq s = {};
    if (lane < a.batch) s = seq_of<TILE, NEW>(a, lane);
    const int64_t mine = s.units(a.heads);
    int64_t x = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    const int64_t total = __shfl_sync(0xffffffffu, x, 31), upto = x - mine;
    if (blockIdx.x == 0 && tid < 32) {
      if (lane < a.batch) note(lane, upto);
      if (lane == 0) a.upto[a.batch] = total;
    }
    Share share = {};
    const int shares = working_shares(a, total), c = (int)blockIdx.x / a.siblings;
    if (c < shares) {
      share.at = share_start(total, shares, c);
      share.end = share_start(total, shares, c + 1);
      share.previous = share_start(total, shares, c > 0 ? c - 1 : 0);
      const int b = __ffs(__ballot_sync(0xffffffffu, share.at >= upto && share.at < x)) - 1;
      Place& p = share.first;
      p.seq = b;
      p.s.rows = __shfl_sync(0xffffffffu, s.rows, b);
      p.s.n = __shfl_sync(0xffffffffu, s.n, b);
      p.s.passes = __shfl_sync(0xffffffffu, s.passes, b);
      p.s.cache_tiles = __shfl_sync(0xffffffffu, s.cache_tiles, b);
      p.s.tiles = __shfl_sync(0xffffffffu, s.tiles, b);
      place_at(p, share.at - __shfl_sync(0xffffffffu, upto, b));
    }
    __syncthreads();   // (what the block initialised before can be seen, as below)
    return share;
  }
  int64_t (&warp_sums)[THREADS / 32] = scratch.warp_sums;
  Share& found = scratch.found;
  const int chunk = (a.batch + THREADS - 1) / THREADS;
  const int b0 = min(a.batch, tid * chunk), b1 = min(a.batch, b0 + chunk);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += seq_of<TILE, NEW>(a, b).units(a.heads);
  int64_t x = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_sums[tid / 32] = x;
  if (tid == 0) found.at = found.end = 0;
  __syncthreads();
  int64_t total = 0, upto = x - mine;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < tid / 32) upto += warp_sums[w];
    total += warp_sums[w];
  }
  if (blockIdx.x == 0) {
    int64_t sum = upto;
    for (int b = b0; b < b1; ++b) {
      note(b, sum);
      sum += seq_of<TILE, NEW>(a, b).units(a.heads);
    }
    if (tid == 0) a.upto[a.batch] = total;
  }
  const int shares = working_shares(a, total), c = (int)blockIdx.x / a.siblings;
  if (c < shares) {
    const int64_t at = share_start(total, shares, c);
    if (at >= upto && at < upto + mine) {
      int b = b0;
      for (int64_t u; at >= upto + (u = seq_of<TILE, NEW>(a, b).units(a.heads)); ++b) upto += u;
      found.at = at;
      found.end = share_start(total, shares, c + 1);
      found.previous = share_start(total, shares, c > 0 ? c - 1 : 0);
      found.first.seq = b;
      found.first.s = seq_of<TILE, NEW>(a, b);
      place_at(found.first, at - upto);
    }
  }
  __syncthreads();
  return found;
}

// Leaves a share's note for the joining launch (one thread of every CTA): whether it is the first to begin inside a head.
__device__ __forceinline__ void leave_note(const Args& a, const Share& share) {
  const int c = (int)blockIdx.x / a.siblings;
  if (blockIdx.x % a.siblings != 0) return;
  int tile = 0;
  if (share.at < share.end && c > 0) {
    const Place& p = share.first;
    const bool first = p.tile > 0 && share.previous <= share.at - p.tile;
    a.cuts[2 * c + 1] = make_int4(p.s.tiles, p.s.n, 0, 0);
    tile = first ? p.tile : 0;
    a.cuts[2 * c] = make_int4(p.seq, p.head, p.pass, tile);
  } else {
    a.cuts[2 * c] = make_int4(0, 0, 0, 0);
  }
}
// The next head's (or pass's) first tile, which exists.
template <int TILE, int NEW> __device__ __forceinline__ void next_head(const Args& a, Place& p) {
  p.tile = 0;
  if (++p.pass < p.s.passes) return;
  p.pass = 0;
  if (++p.head < a.heads) return;
  p.head = 0;
  do p.s = seq_of<TILE, NEW>(a, ++p.seq);
  while (p.s.tiles == 0);
}

// This CTA's pass of the place's head, and its query rows q0 .. q0 + count - 1 (count <= 0: none of this pass).
__device__ __forceinline__ int pass_of(const Args& a, const Place& p) {
  return a.siblings > 1 ? (int)blockIdx.x % a.siblings : p.pass;
}

template <int D> __device__ __forceinline__ float* part_at(const Args& a, int cta, int slot) {
  return a.parts + ((int64_t)cta * 2 + slot) * a.tile_q * (D + 2);
}

// A query head's tokens `first` and later: zeros, and lse -inf (all threads of a block).
template <typename IO, int D, int THREADS> __device__ __forceinline__ void write_zeros(const Args& a, int64_t q_head, int first) {
  const int64_t at = q_head * a.tokens + first;
  const int none = a.tokens - first;
  uint4* const out = reinterpret_cast<uint4*>(static_cast<IO*>(a.out) + at * D);
  for (int u = threadIdx.x; u < none * (D * (int)sizeof(IO) / 16); u += THREADS) out[u] = make_uint4(0u, 0u, 0u, 0u);
  if (a.lse)
    for (int u = threadIdx.x; u < none; u += THREADS) a.lse[at + u] = -INFINITY;
}

// A direct call: this CTA's head as a share of its own, at its first tile in `p`; what is out of range is reported and what
// nobody computes is written. False: nothing is left to do.
template <typename IO, int D, int TILE, int NEW, int THREADS> __device__ __forceinline__ bool direct_share(const Args& a, Share& share, Place& p) {
  p.seq = (int)blockIdx.x / a.heads;
  p.head = (int)blockIdx.x - p.seq * a.heads;
  p.pass = p.tile = 0;
  p.s = seq_of<TILE, NEW>(a, p.seq);
  share = Share{0, p.s.tiles, 0, p};
  if (p.head == 0 && threadIdx.x == 0) {
    if ((int64_t)a.len[p.seq] > a.cap) report(a.dev_status, SNAPKV_ERR_CAPACITY);
    if (a.n_new && (a.n_new[p.seq] < 0 || a.n_new[p.seq] > a.tokens)) report(a.dev_status, SNAPKV_ERR_INVALID_ARG);
  }
  const int first = p.s.tiles == 0 ? 0 : p.s.n;
  if (first < a.tokens)
    for (int g = 0; g < a.group; ++g) write_zeros<IO, D, THREADS>(a, (int64_t)blockIdx.x * a.group + g, first);
  return p.s.tiles > 0;
}

// What sums that belong to maximum m are multiplied by under the maximum `top` (of at least m).
__device__ __forceinline__ float rescale(float m, float top) { return ex2(m - top); }

template <typename T> __device__ __forceinline__ void store1(T* p, float x);
template <> __device__ __forceinline__ void store1<float>(float* p, float x) { *p = x; }
template <> __device__ __forceinline__ void store1<__nv_bfloat16>(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// log of sum exp from the maximum (log2 domain) and the sum under it.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace tree

// The joining launch: out and lse of the rows whose heads were cut, and of those that see nothing.
template <typename IO, int D, int TILE, int NEW> cudaError_t launch_tree_join(const tree::Args& a, cudaStream_t stream);
// The same for bf16 calls of passes of 128 or 256 rows, whose parts hold o as [D][tile_q].
template <int D, int TILE> cudaError_t launch_tree_join_wide(const tree::Args& a, cudaStream_t stream);

}  // namespace snapkv
