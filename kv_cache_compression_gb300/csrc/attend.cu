// Scored decode attention with grouped queries, over a dense cache or one held in 4 bits.
//
//   s_gr = q_g . k_r / sqrt(d),  p_gr = softmax over r < len,  o_g = sum_r p_gr v_r
//   score_r = decay * score_r + sum_g p_gr
//
// One thread-block cluster per (sequence, KV head); its CTAs take equal spans of the head's rows,
// the warps of a CTA every kWarps-th tile of the span. A warp runs an online softmax (running
// maximum m and sum l per query, output o not yet normalised, logits in the log2 domain) over its
// tiles; warps meet in shared memory, CTAs through distributed shared memory, and the last step
// normalises. A score needs the final maximum and sum, so the logits of a span wait in shared memory
// (or, where they do not fit, in the workspace) and are turned into weights after that meeting:
// rows are read once, in one launch.
//
// Both products run on the tensor cores as m16n8k16 with eight queries: q K^T has the queries as
// rows 0 .. 7 of A and eight cached rows as the columns of B; P V has the weights as A, which the
// first product's accumulators already are, lane for lane. Rows 8 .. 15 of A are not wasted: they hold
// the same queries' second bf16 part, so that a weight enters the second product with 16 bits of
// mantissa. fp32 calls split q, p and the cached values into three bf16 parts (24 bits); a product
// drops nothing above 2^-24 of its factors.
//
// With a decode step's few queries the kernel is bound by the cache's bytes. Legacy mma.sync is fast
// enough for that (128 cached values per instruction, against about 50 per clock and SM that HBM
// delivers at 4 bits), and unlike tcgen05.mma it takes levels and weights from registers, where
// unpacking and the softmax leave them.
//
// Each warp moves its own tiles with cp.async through a ring of its own, so warps never wait for
// one another inside the row loop.
#include "cache_internal.h"
#include "q4.cuh"
#include "sm100_ptx.cuh"
#include "snapkv_internal.h"

namespace snapkv {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kLogitsSmem = 64 * 1024;   // a span's logits stay in shared memory up to this size

struct AttendArgs {
  const void* q;
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* km;
  const uint8_t* vm;
  const int32_t* len;
  float* score;
  float* logits;      // null: in shared memory
  void* out;
  float decay, scale_log2;
  int64_t cap;
  int heads, group;
  int32_t* dev_status;
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
template <int N> __device__ __forceinline__ void cp_async_small(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(ptx::smem_u32(dst)), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two fp32 values as a bf16 pair (x in the low half), and what that leaves of them.
__device__ __forceinline__ uint32_t split2(float& x, float& y) {
  const __nv_bfloat162 two = __floats2bfloat162_rn(x, y);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&two);
  x -= __uint_as_float(w << 16);
  y -= __uint_as_float(w & 0xFFFF0000u);
  return w;
}

template <typename T> __device__ __forceinline__ void store1(T* p, float x);
template <> __device__ __forceinline__ void store1<float>(float* p, float x) { *p = x; }
template <> __device__ __forceinline__ void store1<__nv_bfloat16>(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Powers of two around the subnormal operands of a 4-bit cache. Pairs 1 and 3 of a word are worth
// 2^-133 a level, pairs 0 and 2 2^-131: queries are multiplied by 2^64 and 2^62 against them, so that
// both give 2^-69, and weights by 2^80, which keeps p h t normal in fp32 for h from 2^-70 to 2^46.
constexpr float kQ4QEven = 0x1p62f, kQ4QOdd = 0x1p64f, kQ4Dot = 0x1p69f;
constexpr float kQ4P = 0x1p80f, kQ4OutEven = 0x1p51f, kQ4OutOdd = 0x1p53f;

// Format Q4 (codes and pairs) or dense rows of IO; IO is the type of q and out.
template <bool Q4, typename IO, int D> struct Shape {
  static constexpr bool kWide = sizeof(IO) == 4;                    // fp32: three bf16 parts
  static constexpr int kNg = D / kQ4Group;
  static constexpr int kRow = Q4 ? D / 2 : D * (int)sizeof(IO);     // bytes of a row of K (and of V)
  static constexpr int kMeta = Q4 ? 4 * kNg : 0;
  // Rows of a tile: 4 to 9 KB of K and V together.
  static constexpr int kTile = Q4 ? 32 : (kRow >= 256 ? 16 : 32);
  static constexpr int kStage = 2 * kTile * (kRow + kMeta);
  static constexpr int kStages = Q4 ? 4 : (kRow >= 512 ? 2 : 3);
  static constexpr int kWarps = 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRing = kWarps * kStages * kStage;
  // After the row loop the ring holds the warps' partial outputs, then the CTA's.
  static constexpr int kMerge = (kWarps + 1) * kQueryTile * D * 4;
  static constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
};

// 16-byte pieces of a row are stored XORed with the row's low three bits where rows are a multiple of
// 128 bytes: the eight rows (first product) or four rows (second) that a warp reads at a time then
// fall into different banks. 4-bit rows are shorter and need none.
template <int ROW> __device__ __forceinline__ uint32_t piece_at(int row, int piece) {
  if constexpr (ROW >= 128) return row * ROW + ((piece ^ (row & 7)) << 4);
  return row * ROW + (piece << 4);
}

template <bool Q4, typename IO, int D>
__global__ void __launch_bounds__(Shape<Q4, IO, D>::kThreads) attend_kernel(AttendArgs a) {
  using S = Shape<Q4, IO, D>;
  constexpr int kSteps = D / 16;          // 16-channel steps of the first product
  constexpr int kCols = D / 8;            // 8-channel column tiles of the second
  constexpr int kSub = S::kTile / 16;     // 16-row parts of a tile
  constexpr int kNg = S::kNg;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float warp_m[S::kWarps][kQueryTile], warp_l[S::kWarps][kQueryTile];
  __shared__ float cta_m[kQueryTile], cta_l[kQueryTile];   // read by the whole cluster
  __shared__ float head_m[kQueryTile], head_r[kQueryTile]; // the head's maximum, and 1 / its sum

  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int qi = lane / 4, li = lane % 4;   // this lane's query (or column), and its place among four
  const uint32_t rank = ptx::cluster_rank(), csize = ptx::cluster_size();
  const int64_t bh = blockIdx.x / csize;
  const int b = (int)(bh / a.heads);
  int n = a.len[b];
  if ((int64_t)n > a.cap) {
    if (rank == 0 && tid == 0 && bh % a.heads == 0) report(a.dev_status, SNAPKV_ERR_CAPACITY);
    n = (int)a.cap;
  }
  if (n < 0) n = 0;
  // Spans are whole tiles; r1 - r0 is 0 for CTAs past the end.
  const int per = ((n + (int)csize - 1) / (int)csize + S::kTile - 1) / S::kTile * S::kTile;
  const int r0 = min((int64_t)n, (int64_t)rank * per), r1 = min((int64_t)n, (int64_t)r0 + per);
  const int tiles = (r1 - r0 + S::kTile - 1) / S::kTile;
  const uint8_t* kc = a.k + bh * a.cap * S::kRow;
  const uint8_t* vc = a.v + bh * a.cap * S::kRow;
  const uint8_t* kmc = Q4 ? a.km + bh * a.cap * S::kMeta : nullptr;
  const uint8_t* vmc = Q4 ? a.vm + bh * a.cap * S::kMeta : nullptr;
  uint8_t* ring = smem + warp * (S::kStages * S::kStage);

  // Copies tile t of the span into ring slot `slot`; rows at or past r1 become zeros, whatever the
  // cache holds there.
  auto fetch = [&](int t, int slot) {
    uint8_t* dst = ring + slot * S::kStage;
    const int base = r0 + t * S::kTile;
    constexpr int kPieces = S::kRow / 16, kAll = S::kTile * kPieces;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint8_t* src = kv ? vc : kc;
      uint8_t* to = dst + kv * (S::kTile * S::kRow);
#pragma unroll
      for (int j = 0; j < kAll / 32; ++j) {
        const int u = lane + 32 * j, row = u / kPieces, piece = u % kPieces;
        const bool in = base + row < r1;
        cp_async16(to + piece_at<S::kRow>(row, piece), src + (int64_t)(in ? base + row : r0) * S::kRow + piece * 16, in ? 16 : 0);
      }
      if constexpr (Q4) {
        const uint8_t* msrc = kv ? vmc : kmc;
        uint8_t* mto = dst + 2 * (S::kTile * S::kRow) + kv * (S::kTile * S::kMeta);
#pragma unroll
        for (int j = 0; j < (S::kTile + 31) / 32; ++j) {
          const int row = lane + 32 * j;
          const bool in = base + row < r1;
          cp_async_small<S::kMeta>(mto + row * S::kMeta, msrc + (int64_t)(in ? base + row : r0) * S::kMeta, in ? S::kMeta : 0);
        }
      }
    }
  };

  const int passes = (a.group + kQueryTile - 1) / kQueryTile;
  for (int pass = 0; pass < passes; ++pass) {
    const int tile_q = min(kQueryTile, a.group - pass * kQueryTile);   // queries of this pass
    const int64_t q0 = bh * a.group + pass * kQueryTile;
    const bool live = qi < tile_q;
    float* logits = a.logits ? a.logits + (bh * a.cap + r0) * min(kQueryTile, a.group)
                             : reinterpret_cast<float*>(smem + S::kSmem);

    // The ring starts filling before the queries are looked at.
#pragma unroll
    for (int s = 0; s < S::kStages - 1; ++s) {
      if (warp + s * S::kWarps < tiles) fetch(warp + s * S::kWarps, s);
      cp_commit();
    }

    // A operands of the first product: channels c .. c + 3 of query qi for each step, as the lane's
    // share of the row is laid out (see `first product` below).
    uint32_t qa[kSteps][S::kWide ? 6 : 2];
    float qsum[Q4 ? kNg : 1];
    if constexpr (Q4) {
#pragma unroll
      for (int g = 0; g < kNg; ++g) qsum[g] = 0.f;
    }
    const IO* qp = static_cast<const IO*>(a.q) + (q0 + (live ? qi : 0)) * D;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      int c;
      if constexpr (Q4)
        c = 64 * (s / 4) + 16 * li + 8 * ((s % 4) / 2) + 4 * (s % 2);
      else
        c = S::kWide ? 16 * s + 4 * li : 32 * (s / 2) + 8 * li + 4 * (s % 2);
      float x[4];
      if constexpr (S::kWide) {
        const float4 f = *reinterpret_cast<const float4*>(qp + c);
        x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
      } else {
        const uint2 f = *reinterpret_cast<const uint2*>(qp + c);
        x[0] = __uint_as_float(f.x << 16); x[1] = __uint_as_float(f.x & 0xFFFF0000u);
        x[2] = __uint_as_float(f.y << 16); x[3] = __uint_as_float(f.y & 0xFFFF0000u);
      }
      if (!live) x[0] = x[1] = x[2] = x[3] = 0.f;
      if constexpr (Q4) {
        qsum[s / 4] += (x[0] + x[1]) + (x[2] + x[3]);
        x[0] *= kQ4QEven; x[1] *= kQ4QEven; x[2] *= kQ4QOdd; x[3] *= kQ4QOdd;
      }
#pragma unroll
      for (int part = 0; part < (S::kWide ? 3 : 1); ++part) {
        qa[s][2 * part] = split2(x[0], x[1]);
        qa[s][2 * part + 1] = split2(x[2], x[3]);
      }
    }
    if constexpr (Q4) {
#pragma unroll
      for (int g = 0; g < kNg; ++g) {
        qsum[g] += __shfl_xor_sync(0xffffffffu, qsum[g], 1);
        qsum[g] += __shfl_xor_sync(0xffffffffu, qsum[g], 2);
        qsum[g] *= a.scale_log2;
      }
    }
    const float dot_scale = Q4 ? a.scale_log2 * kQ4Dot : a.scale_log2;

    float m = -INFINITY, l = 0.f;
    float o[kCols][4];
#pragma unroll
    for (int t = 0; t < kCols; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    float oz[Q4 ? kNg : 1];
    if constexpr (Q4) {
#pragma unroll
      for (int g = 0; g < kNg; ++g) oz[g] = 0.f;
    }

    // A product of A (two or three parts) with one B pair of words whose values need no split.
    auto mma_parts = [&](float* c, const uint32_t* w, uint32_t b0, uint32_t b1) {
      if constexpr (S::kWide) {
        mma16816(c, w[0], w[2], w[1], w[3], b0, b1);
        mma16816(c, w[4], 0u, w[5], 0u, b0, b1);
      } else {
        mma16816(c, w[0], 0u, w[1], 0u, b0, b1);
      }
    };

    int slot = 0;
    for (int t = warp; t < tiles; t += S::kWarps) {
      cp_wait<S::kStages - 2>();
      __syncwarp();   // every lane's copies of this tile have landed; the slot before it is free
      {
        const int ahead = t + (S::kStages - 1) * S::kWarps;
        const int into = slot == 0 ? S::kStages - 1 : slot - 1;
        if (ahead < tiles) fetch(ahead, into);
        cp_commit();
      }
      const uint8_t* kt = ring + slot * S::kStage;
      const uint8_t* vt = kt + S::kTile * S::kRow;
      const uint8_t* kmt = kt + 2 * (S::kTile * S::kRow);
      const uint8_t* vmt = kmt + S::kTile * S::kMeta;
      slot = slot + 1 == S::kStages ? 0 : slot + 1;
      const int base = r0 + t * S::kTile;

      // ---- first product: logits of kSub x 16 rows. Column 2i of an 8-row tile is row i, column 2i + 1
      // row i + 4, so that the rows a lane reads in the second product are neighbours of other lanes' rows.
      float sv[kSub][4];   // rows li, 4 + li, 8 + li, 12 + li of a part, for query qi
      const int krow = (qi >> 1) + 4 * (qi & 1);
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int row = 16 * sub + 8 * half + krow;
          if constexpr (Q4) {
            uint32_t w[2 * kNg];   // words (o = 0, 1; g) of this lane's 16 channels a group
            if constexpr (kNg == 2) {
              const uint4 x = *reinterpret_cast<const uint4*>(kt + row * S::kRow + 16 * li);
              w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(kt + row * S::kRow + 8 * li);
              w[0] = x.x; w[1] = x.y;
            }
            float dot[kNg][4];
#pragma unroll
            for (int g = 0; g < kNg; ++g) {
              dot[g][0] = dot[g][1] = dot[g][2] = dot[g][3] = 0.f;
#pragma unroll
              for (int o2 = 0; o2 < 2; ++o2) {
                const uint32_t word = w[q4_word<kNg>(g, o2)];
                uint32_t e[4];
                q4_operands(word, prmt(word, word, 0x2301), e);
                mma_parts(dot[g], qa[4 * g + 2 * o2], e[0], e[1]);
                mma_parts(dot[g], qa[4 * g + 2 * o2 + 1], e[2], e[3]);
              }
            }
#pragma unroll
            for (int col = 0; col < 2; ++col) {
              const int r = 16 * sub + 8 * half + 4 * col + li;
              float d = 0.f, zq = 0.f;
#pragma unroll
              for (int g = 0; g < kNg; ++g) {
                const uint32_t hz = *reinterpret_cast<const uint32_t*>(kmt + r * S::kMeta + 4 * g);
                const float x = S::kWide ? dot[g][col] + dot[g][col + 2] : dot[g][col];
                d = fmaf(__uint_as_float(hz << 16), x, d);
                zq = fmaf(__uint_as_float(hz & 0xFFFF0000u), qsum[g], zq);
              }
              sv[sub][2 * half + col] = fmaf(d, dot_scale, zq);
            }
          } else {
            float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s4 = 0; s4 < S::kRow / 64; ++s4) {
              const uint4 x = *reinterpret_cast<const uint4*>(kt + piece_at<S::kRow>(row, 4 * s4 + li));
              if constexpr (S::kWide) {
                float f[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)};
                const uint32_t* w = qa[s4];
#pragma unroll
                for (int part = 0; part < 3; ++part) {
                  const uint32_t b0 = split2(f[0], f[1]), b1 = split2(f[2], f[3]);
                  mma16816(dot, w[0], w[2], w[1], w[3], b0, b1);
                  if (part == 0) mma16816(dot, w[4], 0u, w[5], 0u, b0, b1);
                }
              } else {
                mma16816(dot, qa[2 * s4][0], 0u, qa[2 * s4][1], 0u, x.x, x.y);
                mma16816(dot, qa[2 * s4 + 1][0], 0u, qa[2 * s4 + 1][1], 0u, x.z, x.w);
              }
            }
#pragma unroll
            for (int col = 0; col < 2; ++col)
              sv[sub][2 * half + col] = (S::kWide ? dot[col] + dot[col + 2] : dot[col]) * dot_scale;
          }
        }
      }

      // ---- masks, the running maximum, and the logits that the scores will need
      const bool whole = base + S::kTile <= r1;
      float top = -INFINITY;
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = base + 16 * sub + 4 * e + li;
          if (!whole && r >= r1) sv[sub][e] = -INFINITY;
          if (a.score && live && (whole || r < r1)) logits[(int64_t)(r - r0) * tile_q + qi] = sv[sub][e];
          top = fmaxf(top, sv[sub][e]);
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float m_new = fmaxf(m, top);
      if (__any_sync(0xffffffffu, m_new > m)) {
        const float corr = m == -INFINITY ? 0.f : ex2(m - m_new);
        l *= corr;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          o[c][0] *= corr; o[c][1] *= corr; o[c][2] *= corr; o[c][3] *= corr;
        }
        if constexpr (Q4) {
#pragma unroll
          for (int g = 0; g < kNg; ++g) oz[g] *= corr;
        }
        m = m_new;
      }
      const float shift = m == -INFINITY ? 0.f : m;

      // ---- second product
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = ex2(sv[sub][e] - shift);
          l += p[e];
        }
        const int c0 = krow;   // this lane's column tile channels: 8 c0 .. + 7 (and 64 on)
        if constexpr (Q4) {
          uint32_t hz[4][kNg];
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int g = 0; g < kNg; ++g)
              hz[e][g] = *reinterpret_cast<const uint32_t*>(vmt + (16 * sub + 4 * e + li) * S::kMeta + 4 * g);
          uint32_t w[4][kNg];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint8_t* at = vt + (16 * sub + 4 * e + li) * S::kRow + 4 * kNg * c0;
            if constexpr (kNg == 2) {
              const uint2 x = *reinterpret_cast<const uint2*>(at);
              w[e][0] = x.x; w[e][1] = x.y;
            } else {
              w[e][0] = *reinterpret_cast<const uint32_t*>(at);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int g = 0; g < kNg; ++g) oz[g] = fmaf(p[e], __uint_as_float(hz[e][g] & 0xFFFF0000u), oz[g]);
            p[e] *= kQ4P;
          }
#pragma unroll
          for (int g = 0; g < kNg; ++g) {
            float ph[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) ph[e] = p[e] * __uint_as_float(hz[e][g] << 16);
            uint32_t pa[S::kWide ? 6 : 4];
#pragma unroll
            for (int part = 0; part < (S::kWide ? 3 : 2); ++part) {
              pa[2 * part] = split2(ph[0], ph[1]);
              pa[2 * part + 1] = split2(ph[2], ph[3]);
            }
            uint32_t lo[2][4], hi[2][4];   // [even, odd channels][pair]: rows (li, 4 + li), rows (8 + li, 12 + li)
#pragma unroll
            for (int odd = 0; odd < 2; ++odd) {
              const uint32_t sel = odd ? 0x7632 : 0x5410, swap = odd ? 0x6723 : 0x4501;
              q4_operands(prmt(w[0][g], w[1][g], sel), prmt(w[0][g], w[1][g], swap), lo[odd]);
              q4_operands(prmt(w[2][g], w[3][g], sel), prmt(w[2][g], w[3][g], swap), hi[odd]);
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              mma16816(o[8 * g + c], pa[0], pa[2], pa[1], pa[3], lo[c & 1][c >> 1], hi[c & 1][c >> 1]);
              if constexpr (S::kWide) mma16816(o[8 * g + c], pa[4], 0u, pa[5], 0u, lo[c & 1][c >> 1], hi[c & 1][c >> 1]);
            }
          }
        } else {
          uint32_t pa[S::kWide ? 6 : 4];
#pragma unroll
          for (int part = 0; part < (S::kWide ? 3 : 2); ++part) {
            pa[2 * part] = split2(p[0], p[1]);
            pa[2 * part + 1] = split2(p[2], p[3]);
          }
#pragma unroll
          for (int g = 0; g < kNg; ++g) {
            if constexpr (S::kWide) {
#pragma unroll
              for (int h2 = 0; h2 < 2; ++h2) {
                float f[4][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float4 x = *reinterpret_cast<const float4*>(
                      vt + piece_at<S::kRow>(16 * sub + 4 * e + li, 16 * g + 2 * c0 + h2));
                  f[e][0] = x.x; f[e][1] = x.y; f[e][2] = x.z; f[e][3] = x.w;
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  float* acc = o[8 * g + 4 * h2 + c];
#pragma unroll
                  for (int part = 0; part < 3; ++part) {
                    const uint32_t b0 = split2(f[0][c], f[1][c]), b1 = split2(f[2][c], f[3][c]);
                    mma16816(acc, pa[0], pa[2], pa[1], pa[3], b0, b1);
                    if (part == 0) mma16816(acc, pa[4], 0u, pa[5], 0u, b0, b1);
                  }
                }
              }
            } else {
              uint32_t w[4][4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint4 x = *reinterpret_cast<const uint4*>(vt + piece_at<S::kRow>(16 * sub + 4 * e + li, 8 * g + c0));
                w[e][0] = x.x; w[e][1] = x.y; w[e][2] = x.z; w[e][3] = x.w;
              }
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const uint32_t sel = c & 1 ? 0x7632 : 0x5410;
                mma16816(o[8 * g + c], pa[0], pa[2], pa[1], pa[3], prmt(w[0][c >> 1], w[1][c >> 1], sel),
                         prmt(w[2][c >> 1], w[3][c >> 1], sel));
              }
            }
          }
        }
      }
    }
    cp_wait<0>();

    // ---- the warps of the CTA meet. Lane (qi, li) holds, of query qi, channels 8 li + c (column 0) and
    // 32 + 8 li + c (column 1) of each 64-channel group; rows 8 .. 15 of the accumulators add to them.
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if constexpr (Q4) {
#pragma unroll
      for (int g = 0; g < kNg; ++g) {
        oz[g] += __shfl_xor_sync(0xffffffffu, oz[g], 1);
        oz[g] += __shfl_xor_sync(0xffffffffu, oz[g], 2);
      }
    }
    __syncthreads();   // every warp is done with its ring
    float* part = reinterpret_cast<float*>(smem);
    if (li == 0) {
      warp_m[warp][qi] = m;
      warp_l[warp][qi] = l;
    }
#pragma unroll
    for (int g = 0; g < kNg; ++g)
#pragma unroll
      for (int col = 0; col < 2; ++col) {
        float* to = part + (warp * kQueryTile + qi) * D + 64 * g + 32 * col + 8 * li;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float x = o[8 * g + c][col] + o[8 * g + c][col + 2];
          if constexpr (Q4) x = fmaf(x, (c >> 1) & 1 ? kQ4OutOdd : kQ4OutEven, oz[g]);
          to[c] = x;
        }
      }
    __syncthreads();
    float* cta_o = part + S::kWarps * kQueryTile * D;
    for (int u = tid; u < tile_q * D; u += S::kThreads) {
      const int qq = u / D, c = u % D;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < S::kWarps; ++w) top = fmaxf(top, warp_m[w][qq]);
      float x = 0.f, sum = 0.f;
#pragma unroll
      for (int w = 0; w < S::kWarps; ++w) {
        const float f = warp_m[w][qq] == -INFINITY ? 0.f : ex2(warp_m[w][qq] - top);
        x = fmaf(part[(w * kQueryTile + qq) * D + c], f, x);
        sum = fmaf(warp_l[w][qq], f, sum);
      }
      cta_o[u] = x;
      if (c == 0) {
        cta_m[qq] = top;
        cta_l[qq] = sum;
      }
    }

    // ---- the CTAs of the head meet
    ptx::cluster_sync();
    if (tid < tile_q) {
      float top = -INFINITY;
      for (uint32_t r = 0; r < csize; ++r)
        top = fmaxf(top, __uint_as_float(ptx::dsmem_ld_u32(ptx::map_rank(&cta_m[tid], r))));
      float sum = 0.f;
      for (uint32_t r = 0; r < csize; ++r) {
        const float mr = __uint_as_float(ptx::dsmem_ld_u32(ptx::map_rank(&cta_m[tid], r)));
        if (mr != -INFINITY) sum = fmaf(__uint_as_float(ptx::dsmem_ld_u32(ptx::map_rank(&cta_l[tid], r))), ex2(mr - top), sum);
      }
      head_m[tid] = top == -INFINITY ? 0.f : top;
      head_r[tid] = sum == 0.f ? 0.f : 1.0f / sum;   // no row: zeros; a NaN stays one
    }
    __syncthreads();
    IO* out = static_cast<IO*>(a.out) + q0 * D;
    for (int u = (int)rank * S::kThreads + tid; u < tile_q * D; u += (int)csize * S::kThreads) {
      const int qq = u / D;
      float x = 0.f;
      for (uint32_t r = 0; r < csize; ++r) {
        const float mr = __uint_as_float(ptx::dsmem_ld_u32(ptx::map_rank(&cta_m[qq], r)));
        if (mr != -INFINITY) x = fmaf(__uint_as_float(ptx::dsmem_ld_u32(ptx::map_rank(&cta_o[u], r))), ex2(mr - head_m[qq]), x);
      }
      store1<IO>(out + u, x * head_r[qq]);
    }
    if (a.score) {
      float* sc = a.score + bh * a.cap + r0;
      const float decay = pass == 0 ? a.decay : 1.0f;
      for (int r = tid; r < r1 - r0; r += S::kThreads) {
        float w = 0.f;
        for (int qq = 0; qq < tile_q; ++qq) w = fmaf(ex2(logits[(int64_t)r * tile_q + qq] - head_m[qq]), head_r[qq], w);
        sc[r] = decay != 0.f ? fmaf(decay, sc[r], w) : w;
      }
    }
    ptx::cluster_sync();   // no CTA leaves, or reuses its memory, while its partial may still be read
  }
}

template <bool Q4, typename IO, int D>
cudaError_t launch_typed(const AttendJob& job) {
  using S = Shape<Q4, IO, D>;
  const int64_t bh = (int64_t)job.batch * job.heads;
  const int group = job.q_heads / job.heads, tile_q = group < kQueryTile ? group : kQueryTile;
  // CTAs per head: enough for two per SM, with at least a tile per warp each.
  int64_t csize = 2 * (int64_t)device_sm_count() / bh;
  const int64_t most = (job.cap + S::kTile * S::kWarps - 1) / (S::kTile * S::kWarps);
  if (csize > most) csize = most;
  if (csize > kMaxCluster) csize = kMaxCluster;
  if (csize < 1) csize = 1;
  const int64_t per = ((job.cap + csize - 1) / csize + S::kTile - 1) / S::kTile * S::kTile;
  const int64_t logits = job.score ? per * tile_q * 4 : 0;
  AttendArgs a;
  a.q = job.q;
  a.k = static_cast<const uint8_t*>(job.k);
  a.v = static_cast<const uint8_t*>(job.v);
  a.km = static_cast<const uint8_t*>(job.k_meta);
  a.vm = static_cast<const uint8_t*>(job.v_meta);
  a.len = job.len;
  a.score = job.score;
  a.logits = logits <= kLogitsSmem ? nullptr : job.logits;
  a.out = job.out;
  a.decay = job.decay;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
  a.cap = job.cap;
  a.heads = job.heads;
  a.group = group;
  a.dev_status = job.dev_status;
  const cudaError_t err = allow_dynamic_smem<attend_kernel<Q4, IO, D>>(S::kSmem + kLogitsSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(bh * csize));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem + (a.logits ? 0 : (size_t)logits);
  cfg.stream = job.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)csize;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_kernel<Q4, IO, D>, a);
}

template <bool Q4> cudaError_t launch_format(const AttendJob& job) {
  if (job.dtype == SNAPKV_BF16)
    return job.head_dim == 64 ? launch_typed<Q4, __nv_bfloat16, 64>(job) : launch_typed<Q4, __nv_bfloat16, 128>(job);
  return job.head_dim == 64 ? launch_typed<Q4, float, 64>(job) : launch_typed<Q4, float, 128>(job);
}

}  // namespace

size_t attend_logits_bytes(int batch, int q_heads, int heads, int head_dim, int64_t cap) {
  (void)head_dim;
  const int group = q_heads / heads;
  return (size_t)batch * heads * (size_t)cap * (group < kQueryTile ? group : kQueryTile) * sizeof(float);
}

cudaError_t launch_attend(const AttendJob& job) {
  return job.k_meta ? launch_format<true>(job) : launch_format<false>(job);
}

}  // namespace snapkv
