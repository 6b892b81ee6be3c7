// Tree attention in fp32 instructions: fp32 calls, over a dense cache or one in 8 bits (tree_schedule.cuh has the schedule).
//
//   s_rk = q_r . k_k / sqrt(d) over the keys k that row r sees,  p = softmax,  o_r = sum p_rk v_k
//
// A CTA walks its share of the 64-key tiles with an online softmax: products of QT query rows with a tile's keys (each
// thread some rows by some keys, channels in steps of four), weights through shared memory, and products with the
// tile's values (each thread four rows by four channels of a KS-th of the keys). Products and sums are fp32 FMAs that
// round to nearest. K's and V's tiles have a buffer each: V's rows are under way while the logits are computed, the next
// K's while the outputs are, and a second CTA per SM fills the rest.
//
// Measured (128 channels): 8 x 8 KV heads of 28 rows over 8192 keys, half of the sequences shorter, 190 us, 2.1 TB/s: loads from
// shared memory take 61 % of its clocks, FMAs and the rest of the instructions 50 % of the schedulers', and the barriers between a
// tile's steps keep them apart; eight rows 127 us, 4.2 TB/s. Three bf16 parts an operand on mma.sync (six products, as accurate)
// took 7 % more for the 28 rows and for eight, blocks of 4 x 4 logits and 8 x 4 outputs a thread 5 % more and 4 % less.
#include "tree_schedule.cuh"

#include <atomic>

#include "cache_internal.h"
#include "q4.cuh"
#include "sm100_ptx.cuh"
#include "snapkv_internal.h"
#include "tree_launch.h"

namespace snapkv {
namespace {

using namespace tree;

constexpr int kThreads = 256;
constexpr int kTile = 64;   // keys

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A tile: where its rows lie, and how many it has.
struct Rows {
  const void* k;
  const void* v;
  const float* k_step;   // null: rows of the call's type
  const float* v_step;
  int count;             // rows of the tile that may be seen (the rest of kTile is zeros)
  int draft0;            // the first one's number among the drafted rows; -1: cached rows
};

template <bool Q8, int D> __device__ __forceinline__ Rows rows_of(const Args& a, const Place& p) {
  Rows r;
  const int64_t bh = (int64_t)p.seq * a.heads + p.head;
  if (p.tile < p.s.cache_tiles) {
    const int64_t row = bh * a.cap + (int64_t)p.tile * kTile;
    const int64_t bytes = Q8 ? D : D * (int)sizeof(float);
    r.k = static_cast<const uint8_t*>(a.k) + row * bytes;
    r.v = static_cast<const uint8_t*>(a.v) + row * bytes;
    r.k_step = Q8 ? a.k_step + row : nullptr;
    r.v_step = Q8 ? a.v_step + row : nullptr;
    r.count = min(kTile, p.s.rows - p.tile * kTile);
    r.draft0 = -1;
    if (!in_bounds(row >= 0 && row + r.count <= (int64_t)a.batch * a.heads * a.cap, a.dev_status)) r.count = 0;
  } else {
    r.draft0 = (p.tile - p.s.cache_tiles) * kTile;
    const int64_t row = bh * a.tokens + r.draft0;
    r.k = static_cast<const float*>(a.k_new) + row * D;
    r.v = static_cast<const float*>(a.v_new) + row * D;
    r.k_step = r.v_step = nullptr;
    r.count = min(kTile, p.s.n - r.draft0);
    if (!in_bounds(row >= 0 && row + r.count <= (int64_t)a.batch * a.heads * a.tokens, a.dev_status)) r.count = 0;
  }
  return r;
}

// The values of four codes of a row with step h: u h rounded once (2^23 + u less 2^23, times h, in one FMA), with the code's sign.
__device__ __forceinline__ float4 values4(uint32_t codes, float h) {
  const uint32_t u = codes & 0x7F7F7F7Fu;
  const float less = -8388608.0f * h;
  const float x = fmaf(__uint_as_float(prmt(u, 0x4B000000u, 0x7650)), h, less), y = fmaf(__uint_as_float(prmt(u, 0x4B000000u, 0x7651)), h, less),
              z = fmaf(__uint_as_float(prmt(u, 0x4B000000u, 0x7652)), h, less), w = fmaf(__uint_as_float(prmt(u, 0x4B000000u, 0x7653)), h, less);
  return make_float4(__uint_as_float(__float_as_uint(x) ^ (codes << 24 & 0x80000000u)), __uint_as_float(__float_as_uint(y) ^ (codes << 16 & 0x80000000u)),
                     __uint_as_float(__float_as_uint(z) ^ (codes << 8 & 0x80000000u)), __uint_as_float(__float_as_uint(w) ^ (codes & 0x80000000u)));
}

// A tile's rows on their way to `to`, a row's 16-byte pieces XORed with hash(row); rows past `count` become zeros. fp32 rows go
// by cp.async; codes wait in registers, sixteen a vector, until put() writes their values (which takes the latency of their loads
// off the tile: 8 x 8 heads of 8192 rows, 28 query rows each, 455 us -> 275; seven rows, 333 -> 141).
template <bool Q8, int D> struct Loader {
  static constexpr int kN = Q8 ? kTile * D / 16 / kThreads : 1;   // vectors of a thread
  uint4 codes[kN];
  float h[kN];
  bool coded;

  template <typename Hash> __device__ __forceinline__ void load(float* to, const void* from, const float* step, int count, Hash hash) {
    coded = Q8 && step;
    if (coded) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int u = threadIdx.x + i * kThreads, row = u / (D / 16);
        codes[i] = make_uint4(0u, 0u, 0u, 0u);
        h[i] = 0.f;
        if (row < count) {
          codes[i] = __ldg(static_cast<const uint4*>(from) + u);
          h[i] = __ldg(step + row);
        }
      }
      return;
    }
    constexpr int kPieces = D / 4;
#pragma unroll 4
    for (int u = threadIdx.x; u < kTile * kPieces; u += kThreads) {
      const int row = u / kPieces, c = u % kPieces;
      const bool there = row < count;
      cp_async16(to + row * D + 4 * (c ^ hash(row)), static_cast<const float*>(from) + (there ? (int64_t)u * 4 : 0), there);
    }
  }
  template <typename Hash> __device__ __forceinline__ void put(float* to, Hash hash) const {
    if constexpr (!Q8) return;
    if (!coded) return;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int u = threadIdx.x + i * kThreads, row = u / (D / 16), c = u % (D / 16);
      const int turn = c / 2 % 4;   // (four codes at a time, from another of a vector's words in every other lane: eight lanes, eight pieces)
      uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
      if (turn & 1) {
        const uint32_t x = w[0];
        w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = x;
      }
      if (turn & 2) {
        const uint32_t x = w[0], y = w[1];
        w[0] = w[2], w[1] = w[3], w[2] = x, w[3] = y;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(to + row * D + 4 * ((4 * c + (j + turn) % 4) ^ hash(row))) = values4(w[j], h[i]);
    }
  }
};

template <int D, int QT> struct Shape {
  static constexpr int kRq = QT == 32 ? 4 : 2, kRk = QT == 32 ? 2 : 1;      // logits of a thread: rows by keys
  static_assert(QT / kRq * (kTile / kRk) == kThreads, "a thread for every block of logits");
  static constexpr int kKs = kThreads * 16 / (QT * D);                      // key groups of the second product
  static constexpr int kPs = QT + 4;                                        // floats between two keys' weights
  static constexpr int smem() { return 4 * (QT * D + 2 * kTile * D + kTile * kPs + 3 * QT); }
};

template <bool Q8, int D, int QT>
__global__ void __launch_bounds__(kThreads, 2) tree_simt_kernel(Args a) {
  using S = Shape<D, QT>;
  constexpr int kRq = S::kRq, kRk = S::kRk, kKs = S::kKs, kPs = S::kPs;
  extern __shared__ __align__(16) float smem[];
  float* const qs = smem;                  // [QT][D], pieces XORed
  float* const ks = qs + QT * D;           // [kTile][D], pieces XORed
  float* const vs = ks + kTile * D;        // [kTile][D]
  float* const ps = vs + kTile * D;        // [kTile][kPs]: logits, then weights
  float* const ms = ps + kTile * kPs;      // [QT]: running maxima, sums, and this tile's factors
  float* const ls = ms + QT;
  float* const fs = ls + QT;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  auto q_hash = [](int row) { return (row / kRq) & 7; };
  auto k_hash = [](int row) { return (row / kRk) & 7; };
  auto v_hash = [](int) { return 0; };
  __shared__ ShareScratch<kThreads> scratch;
  Share share;
  Place here;
  if (a.direct) {
    if (!direct_share<float, D, kTile, kTile, kThreads>(a, share, here)) return;
  } else {
    share = find_share<kTile, kTile, kThreads>(a, scratch);
    if (share.at >= share.end) return;
    here = share.first;
  }
  // first product: rows kRq qg .. by keys kRk kg .. (a warp has eight rows, so that where there are fewer rows some rest)
  constexpr int kWarpQg = 8 / kRq, kWarpKg = 32 / kWarpQg;   // of a warp's lanes
  constexpr int kRowWarps = QT / 8;                          // warps along the rows
  const int qg = warp % kRowWarps * kWarpQg + lane % kWarpQg, kg = warp / kRowWarps * kWarpKg + lane / kWarpQg;
  // second product: rows 4 og .. by channels 4 cg .. of the keys of group kh
  const int kh = tid / (kThreads / kKs), in = tid % (kThreads / kKs);
  constexpr int kOg = QT / 4;
  constexpr int kOw = kOg < 4 ? kOg : 4;   // of a warp's lanes along the rows
  const int cg = (in / kOw) % (D / 4), og = in % kOw + kOw * (in / (kOw * (D / 4)));

  int64_t at = share.at;
  while (at < share.end) {
    const int64_t left = share.end - at;
    const int seg = left < here.s.tiles - here.tile ? (int)left : here.s.tiles - here.tile;   // tiles of this head in this share
    const bool whole = seg == here.s.tiles;
    const int pass = pass_of(a, here), r0 = pass * a.tile_q, n = here.s.n;
    const int count = min(a.tile_q, a.group * n - r0);   // (at least one: passes follow from the rows there are)
    const int64_t bh = (int64_t)here.seq * a.heads + here.head;
    auto row_at = [&](int i) {   // the query row in [B, Hq, T]
      const int r = r0 + i, g = r / n;
      return (bh * a.group + g) * a.tokens + (r - g * n);
    };
    // ---- queries, and the first tile's keys
    Rows tile = rows_of<Q8, D>(a, here);
    Loader<Q8, D> k_rows, v_rows;
    k_rows.load(ks, tile.k, tile.k_step, tile.count, k_hash);
    cp_commit();
    for (int u = tid; u < QT * (D / 4); u += kThreads) {
      const int i = u / (D / 4), c = u % (D / 4);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < count) x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + row_at(i) * D + 4 * c));
      *reinterpret_cast<float4*>(qs + i * D + 4 * (c ^ q_hash(i))) = x;
    }
    for (int i = tid; i < QT; i += kThreads) {
      ms[i] = kNoMax;
      ls[i] = 0.f;
    }
    float2 o[4][2];   // rows by pairs of channels
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r][0] = o[r][1] = make_float2(0.f, 0.f);

    k_rows.put(ks, k_hash);

    for (int j = 0; j < seg; ++j, ++here.tile) {
      v_rows.load(vs, tile.v, tile.v_step, tile.count, v_hash);
      cp_commit();
      cp_wait<1>();
      __syncthreads();   // K and Q are there
      // ---- logits
      if (qg / kWarpQg * 8 < count) {
        float2 s[kRq][kRk];
#pragma unroll
        for (int x = 0; x < kRq; ++x)
#pragma unroll
          for (int y = 0; y < kRk; ++y) s[x][y] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int c = 0; c < D / 4; ++c) {
          float4 qv[kRq], kv[kRk];
#pragma unroll
          for (int x = 0; x < kRq; ++x) qv[x] = *reinterpret_cast<const float4*>(qs + (kRq * qg + x) * D + 4 * (c ^ (qg & 7)));
#pragma unroll
          for (int y = 0; y < kRk; ++y) kv[y] = *reinterpret_cast<const float4*>(ks + (kRk * kg + y) * D + 4 * (c ^ (kg & 7)));
#pragma unroll
          for (int x = 0; x < kRq; ++x)
#pragma unroll
            for (int y = 0; y < kRk; ++y) {
              s[x][y] = fma2(make_float2(qv[x].x, qv[x].y), make_float2(kv[y].x, kv[y].y), s[x][y]);
              s[x][y] = fma2(make_float2(qv[x].z, qv[x].w), make_float2(kv[y].z, kv[y].w), s[x][y]);
            }
        }
#pragma unroll
        for (int y = 0; y < kRk; ++y) {
          const int key = kRk * kg + y;
          float l[kRq];
#pragma unroll
          for (int x = 0; x < kRq; ++x) {
            l[x] = (s[x][y].x + s[x][y].y) * a.scale_log2;
            bool seen = key < tile.count;
            if (tile.draft0 >= 0 && seen) {
              const int i = kRq * qg + x;
              const int t = (r0 + i) % n, k = tile.draft0 + key;
              seen = i < count && (a.mask ? a.mask[here.seq * a.mask_stride + (int64_t)t * a.tokens + k] != 0 : k <= t);
            }
            if (!seen) l[x] = -INFINITY;
          }
          if constexpr (kRq == 4)
            *reinterpret_cast<float4*>(ps + key * kPs + 4 * qg) = make_float4(l[0], l[1], l[2], l[3]);
          else
            *reinterpret_cast<float2*>(ps + key * kPs + 2 * qg) = make_float2(l[0], l[1]);
        }
      }
      v_rows.put(vs, v_hash);
      __syncthreads();   // the logits are there, and K's buffer is free
      const Rows now = tile;
      if (j + 1 < seg) {
        Place next = here;
        ++next.tile;
        tile = rows_of<Q8, D>(a, next);
        k_rows.load(ks, tile.k, tile.k_step, tile.count, k_hash);
      }
      cp_commit();
      // ---- weights: eight lanes a row
      for (int r = warp * 4 + lane % 4; r < QT && warp * 4 < count; r += 32) {
        float* p = ps + (lane / 4) * kPs + r;
        float x[kTile / 8], top = kNoMax;
#pragma unroll
        for (int e = 0; e < kTile / 8; ++e) {
          x[e] = p[8 * e * kPs];
          top = fmaxf(top, x[e]);
        }
        const unsigned lanes = __activemask();
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(lanes, top, off));
        const float old = ms[r], m = fmaxf(old, top);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < kTile / 8; ++e) {
          x[e] = ex2(x[e] - m);
          sum += x[e];
          p[8 * e * kPs] = x[e];
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(lanes, sum, off);
        __syncwarp(lanes);
        if (lane / 4 == 0) {
          const float f = rescale(old, m);
          fs[r] = f;
          ms[r] = m;
          ls[r] = fmaf(ls[r], f, sum);
        }
      }
      cp_wait<1>();
      __syncthreads();   // the weights and V are there
      // ---- outputs
      if (kOw * 4 * (in / (kOw * (D / 4))) < count) {   // (a warp has 4 kOw rows)
        const float4 f = *reinterpret_cast<const float4*>(fs + 4 * og);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float fr = r == 0 ? f.x : r == 1 ? f.y : r == 2 ? f.z : f.w;
#pragma unroll
          for (int c = 0; c < 2; ++c) o[r][c] = mul2(o[r][c], make_float2(fr, fr));
        }
        // A row that nobody may see (or that is masked) has weight zero, but its values may be anything: a drafted
        // row's infinity or NaN must not reach the rows that do not see it.
        const bool careful = now.draft0 >= 0;
#pragma unroll 4
        for (int e = 0; e < kTile / kKs; ++e) {
          const int key = kh + e * kKs;
          const float4 w = *reinterpret_cast<const float4*>(ps + key * kPs + 4 * og);
          const float4 v = *reinterpret_cast<const float4*>(vs + key * D + 4 * cg);
          const float wr[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float2 ww = make_float2(wr[r], wr[r]);
            if (!careful || wr[r] != 0.f) {
              o[r][0] = fma2(ww, make_float2(v.x, v.y), o[r][0]);
              o[r][1] = fma2(ww, make_float2(v.z, v.w), o[r][1]);
            }
          }
        }
      }
      if (j + 1 < seg) k_rows.put(ks, k_hash);
      __syncthreads();   // V's buffer and the weights are free
    }

    // ---- the head's end in this share: the key groups meet, in the keys' buffer
    float* const meet = ks;   // [kKs][QT][D]
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *reinterpret_cast<float4*>(meet + (kh * QT + 4 * og + r) * D + 4 * cg) = make_float4(o[r][0].x, o[r][0].y, o[r][1].x, o[r][1].y);
    __syncthreads();
    float* const part = part_at<D>(a, (int)blockIdx.x, at > share.at ? 1 : 0);
    for (int u = tid; u < count * D; u += kThreads) {
      const int i = u / D, c = u % D;
      float x = meet[u];
#pragma unroll
      for (int g = 1; g < kKs; ++g) x += meet[g * QT * D + u];
      if (whole)
        static_cast<float*>(a.out)[row_at(i) * D + c] = x * (ls[i] == 0.f ? 0.f : 1.0f / ls[i]);
      else
        part[u] = x;
    }
    for (int i = tid; i < count; i += kThreads) {
      if (!whole) {
        part[a.tile_q * D + i] = ms[i];
        part[a.tile_q * (D + 1) + i] = ls[i];
      } else if (a.lse) {
        a.lse[row_at(i)] = lse_of(ms[i], ls[i]);
      }
    }
    __syncthreads();
    at += seg;
    if (at < share.end) next_head<kTile, kTile>(a, here);
  }
  cp_wait<0>();
}

template <bool Q8, int D, int QT> cudaError_t launch_typed(const TreeJob& job) {
  using S = Shape<D, QT>;
  Args a = tree_args(job, QT);
  cudaError_t err = allow_dynamic_smem<tree_simt_kernel<Q8, D, QT>>(S::smem());
  if (err != cudaSuccess) return err;
  int64_t ctas = 2 * (int64_t)device_sm_count();
  err = tree_fill(a, job, kTile, kTile, ctas);
  if (err != cudaSuccess) return err;
  tree_simt_kernel<Q8, D, QT><<<a.ctas, kThreads, S::smem(), job.stream>>>(a);
  err = cudaGetLastError();
  return err != cudaSuccess || a.direct ? err : launch_tree_join<float, D, kTile, kTile>(a, job.stream);
}

// Passes of eight rows where there are no more: 64 KV heads of 8192 fp32 rows took 145 us with them, 192 with 32 (127 now).
template <bool Q8, int D> cudaError_t launch_dim(const TreeJob& job) {
  const int rows = job.q_heads / job.heads * job.tokens;
  return rows <= 8 ? launch_typed<Q8, D, 8>(job) : launch_typed<Q8, D, 32>(job);
}

template <bool Q8> cudaError_t launch_format(const TreeJob& job) {
  return job.head_dim == 64 ? launch_dim<Q8, 64>(job) : launch_dim<Q8, 128>(job);
}

}  // namespace

cudaError_t launch_tree_simt(const TreeJob& job) {
  return job.k_step ? launch_format<true>(job) : launch_format<false>(job);
}

}  // namespace snapkv
