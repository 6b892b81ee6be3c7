// Tree attention of few query rows a KV head, bf16, over a dense cache (up to sixteen) or one in 8 bits (up to 32, in passes
// of sixteen): one token, or a few drafted ones (tree_schedule.cuh has the schedule).
//
//   S = Q K^T,  P = exp2(S - m),  O = sum P V,  running m and sum per row
//
// So few rows are bound by the cache's bytes, and mma.sync (1024 products a clock and SM, as measured) is fast enough:
// sixteen rows take 768 clocks of it per 128 keys of 128 channels, in which HBM delivers 32 keys' bf16 rows or 63 in 8
// bits (6787 GB/s over 152 SMs at 2.07 GHz: 21.6 bytes a clock and SM). Unlike tcgen05.mma it takes codes and weights from registers, where unpacking and the softmax leave them.
// Every warp walks tiles of its own (TMA into a ring of its own) with its own m, sum and O; at the end of a head the four
// warps meet in shared memory. Two CTAs an SM: with 225 to 255 registers a thread there is room for no third.
//
// Weights enter the second product in two bf16 parts (16 bits): of up to eight rows (HALF) the second parts are the other
// eight rows of the same product, so that they cost nothing (a token over 131072 8-bit rows 178 -> 173 us). 8-bit codes
// become operands by one byte permute and one AND per two values, as *subnormal* bf16: sign and seven magnitude bits are
// u 2^-133, which mma.sync multiplies exactly. The powers of two are made up for where it costs nothing: queries are
// scaled by 2^64, weights by 2^80. A step multiplies its key's logits and weights.
//
// Measured (128 channels): one token over 32 heads of 131072 8-bit rows 170 us, 6.5 TB/s; 64 x 32 heads of 2208 8-bit rows, up
// to six tokens each, 215 us, 5.4 TB/s (its joining launch and uneven ends); 64 x 32 heads of 2140 bf16 rows, four tokens,
// 350 us, 6.4 TB/s; 32 heads of 1057 bf16 rows, eight tokens, 16 us, which is latency of two launches. Bytes bound it, and
// over 8-bit rows the permutes come next (ALU 39 %).
#include "tree_schedule.cuh"

#include <type_traits>

#include "cache_internal.h"
#include "q4.cuh"
#include "sm100_ptx.cuh"
#include "snapkv_internal.h"
#include "tc_common.cuh"
#include "tree_launch.h"
#include "tree_maps.h"

namespace snapkv {
namespace {

using namespace tree;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr long long kWaitLimit = 4000000000LL;   // about two seconds

// HALF: up to eight rows, the lower half of sixteen.
template <bool Q8, int D, bool HALF> struct Shape {
  static constexpr int kRows = HALF ? 8 : 16;
  static constexpr int kTile = Q8 ? 32 : 2048 / D;                   // cached keys of a tile
  static constexpr int kNew = 16;                                    // drafted ones
  static constexpr int kStage = 2 * kTile * D * (Q8 ? 1 : 2);        // K, V
  static constexpr int kStages = HALF ? 3 : 2;                       // (two CTAs share an SM's 227 KB)
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kSteps = Q8 ? kWarps * kStages * 2 * kTile * 4 : 0;
  static constexpr int kMeet = kWarps / 2 * kRows * D * 4;
  static constexpr int smem() { return 1024 + kRing + kSteps + kMeet; }
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool TRANS> __device__ __forceinline__ void load_matrices(uint32_t at, uint32_t (&x)[4]) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts128_zero(uint32_t at) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0) : "memory");
}
// The pair as bf16, and in x, y what that leaves.
__device__ __forceinline__ uint32_t split2(float& x, float& y) {
  const uint32_t w = pack2(x, y);
  x -= __uint_as_float(w << 16);
  y -= __uint_as_float(w & 0xFFFF0000u);
  return w;
}
// Bytes lo and hi (0 .. 3 of a, 4 .. 7 of b) as a pair of operands.
template <int LO, int HI> __device__ __forceinline__ uint32_t operand(uint32_t a, uint32_t b) {
  return prmt(a, b, LO | (LO << 4) | (HI << 8) | (HI << 12)) & 0x807F807Fu;
}

// Shared memory of a tile: bf16 rows in blocks of 64 channels (128 bytes), 8-bit rows as they are; 16-byte pieces XORed as
// TMA's swizzles do.
template <int ROWS> __device__ __forceinline__ uint32_t bf16_at(int row, int piece) {   // piece: of eight channels
  return (piece / 8) * (ROWS * 128) + row * 128 + (((piece % 8) ^ (row & 7)) << 4);
}
template <int D> __device__ __forceinline__ uint32_t code_at(int row, int piece) {      // of sixteen channels
  if constexpr (D == 128) return row * 128 + ((piece ^ (row & 7)) << 4);
  return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}

template <bool Q8, int D, bool HALF>
__global__ void __launch_bounds__(kThreads, 2) tree_mma_kernel(const Args a, const __grid_constant__ TreeMaps maps) {
  using S = Shape<Q8, D, HALF>;
  constexpr int kTile = S::kTile, kNew = S::kNew, kRows = S::kRows, kStages = S::kStages;
  constexpr int kK = D / 16;      // steps of the first product
  constexpr int kN = D / 8;       // channel tiles of the second
  constexpr int kH = HALF ? 1 : 2;   // row halves in use
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ float warp_m[kWarps][kRows], warp_l[kWarps][kRows];
  __shared__ int abort;
  uint8_t* const smem = raw + ((1024 - (ptx::smem_u32(raw) & 1023)) & 1023);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, j = lane / 4, i = lane % 4;
  if (tid == 0) {
    abort = 0;
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < kStages; ++s) ptx::mbar_init(&full[w][s], Q8 ? 33 : 1);
    ptx::fence_mbar_init();
  }
  __shared__ ShareScratch<kThreads> scratch;
  Share share;
  Place here;
  if (a.direct) {
    if (!direct_share<__nv_bfloat16, D, kTile, kNew, kThreads>(a, share, here)) return;
    __syncthreads();   // the barriers are initialised
  } else {
    share = find_share<kTile, kNew, kThreads>(a, scratch);   // (with barriers)
    if (share.at >= share.end) return;
    here = share.first;
  }
  Place ahead = here;              // the next tile to load
  int64_t ahead_at = share.at + warp;
  uint8_t* const ring = smem + warp * (kStages * S::kStage);
  float* const steps = reinterpret_cast<float*>(smem + S::kRing) + warp * (kStages * 2 * kTile);
  float* const meet = reinterpret_cast<float*>(smem + S::kRing + S::kSteps);

  // Moves p on by `by` tiles, to the head that holds them (which exists).
  auto advance = [&](Place& p, int by) {
    by += p.tile;
    while (by >= p.s.tiles) {
      by -= p.s.tiles;
      next_head<kTile, kNew>(a, p);
    }
    p.tile = by;
  };
  // Sends for the tile `ahead` into a stage (the whole warp; the stage has been read).
  auto send = [&](int stage) {
    uint8_t* const k = ring + stage * S::kStage;
    const int bh = ahead.seq * a.heads + ahead.head;
    if (ahead.tile == 0) {   // a new head: its queries come into L2
      const int r = (a.siblings > 1 ? (int)blockIdx.x % a.siblings : ahead.pass) * kRows + lane / (D / 64), g = r / ahead.s.n;
      if (lane / (D / 64) < kRows && r < a.group * ahead.s.n)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const __nv_bfloat16*>(a.q) +
                                                      (((int64_t)bh * a.group + g) * a.tokens + (r - g * ahead.s.n)) * D + lane % (D / 64) * 64));
    }
    uint64_t* const bar = &full[warp][stage];
    if (ahead.tile < ahead.s.cache_tiles) {
      const int row0 = ahead.tile * kTile;
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(bar, S::kStage);
#pragma unroll
        for (int c = 0; c < (Q8 ? 1 : D / 64); ++c) {
          ptx::tma_load_3d(k + c * kTile * 128, &maps.k, 64 * c, row0, bh, bar);
          ptx::tma_load_3d(k + S::kStage / 2 + c * kTile * 128, &maps.v, 64 * c, row0, bh, bar);
        }
      }
      if constexpr (Q8) {
        float* const to = steps + stage * 2 * kTile + lane;
        const int64_t from = (int64_t)bh * a.cap + row0 + lane;
        const int bytes = row0 + lane < ahead.s.rows ? 4 : 0;
        if (in_bounds(bytes == 0 || from < (int64_t)a.batch * a.heads * a.cap, a.dev_status)) {
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ptx::smem_u32(to)), "l"(a.k_step + (bytes ? from : 0)), "r"(bytes) : "memory");
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ptx::smem_u32(to + kTile)), "l"(a.v_step + (bytes ? from : 0)), "r"(bytes) : "memory");
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
      }
    } else {
      const int row0 = (ahead.tile - ahead.s.cache_tiles) * kNew;
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(bar, 2 * kNew * D * 2);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          ptx::tma_load_3d(k + c * kNew * 128, &maps.k_new, 64 * c, row0, bh, bar);
          ptx::tma_load_3d(k + kNew * D * 2 + c * kNew * 128, &maps.v_new, 64 * c, row0, bh, bar);
        }
      }
      if constexpr (Q8) ptx::mbar_arrive(bar);
    }
  };
  auto send_next = [&](int stage) {
    if (ahead_at >= share.end) return;
    send(stage);
    ahead_at += kWarps;
    if (ahead_at < share.end) advance(ahead, kWarps);
  };
  if (ahead_at < share.end) advance(ahead, warp);
#pragma unroll
  for (int s = 0; s < kStages; ++s) send_next(s);

  int stage = 0;
  uint32_t parity = 0;
  int64_t at = share.at;
  while (at < share.end) {
    const int64_t left = share.end - at;
    const int seg = left < here.s.tiles - here.tile ? (int)left : here.s.tiles - here.tile;
    const bool whole = seg == here.s.tiles;
    const int n = here.s.n, pass = a.siblings > 1 ? (int)blockIdx.x % a.siblings : here.pass;
    const int first_row = pass * kRows, count = min(kRows, a.group * n - first_row);   // query rows of this pass
    const int64_t bh = (int64_t)here.seq * a.heads + here.head;
    auto row_at = [&](int i) {
      const int r = first_row + i, g = r / n;
      return (bh * a.group + g) * a.tokens + (r - g * n);
    };
    // ---- queries, as A operands: rows j and j + 8; dense: channels 16 s + 2 i, + 1, + 8, + 9; 8 bits: the four at
    // 4 s of this lane's run (D / 4 channels from D / 4 i)
    uint32_t q[kK][2 * kH];
#pragma unroll
    for (int e = 0; e < kH; ++e) {
      const int r = j + 8 * e;
      const bool there = r < count;
      const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(a.q) + (there ? row_at(r) : 0) * D;
#pragma unroll
      for (int s = 0; s < kK; ++s) {
        uint2 w = make_uint2(0u, 0u);
        if (there) {
          if constexpr (Q8) {
            w = __ldg(reinterpret_cast<const uint2*>(from + (D / 4) * i + 4 * s));
          } else {
            w.x = __ldg(reinterpret_cast<const uint32_t*>(from + 16 * s + 2 * i));
            w.y = __ldg(reinterpret_cast<const uint32_t*>(from + 16 * s + 2 * i + 8));
          }
        }
        if constexpr (Q8) {
          w.x = pack2(__uint_as_float(w.x << 16) * kQ8Q, __uint_as_float(w.x & 0xFFFF0000u) * kQ8Q);
          w.y = pack2(__uint_as_float(w.y << 16) * kQ8Q, __uint_as_float(w.y & 0xFFFF0000u) * kQ8Q);
        }
        q[s][2 * e] = w.x;
        q[s][2 * e + 1] = w.y;
      }
    }
    float m[kH], l[kH], o[kN][4];
#pragma unroll
    for (int e = 0; e < kH; ++e) {
      m[e] = kNoMax;
      l[e] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < kN; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
    auto mma_q = [&](float (&c)[4], int s, uint32_t b0, uint32_t b1) {
      if constexpr (HALF)
        mma(c, q[s][0], 0u, q[s][1], 0u, b0, b1);
      else
        mma(c, q[s][0], q[s][2 % (2 * kH)], q[s][1], q[s][3 % (2 * kH)], b0, b1);
    };
    // The online softmax of NT tiles of eight keys: c becomes weights. Keys of a lane: 2 i and 2 i + 1 of each.
    auto softmax = [&](auto& c, auto nt) {
      constexpr int NT = decltype(nt)::value;
#pragma unroll
      for (int e = 0; e < kH; ++e) {
        float top = m[e];
#pragma unroll
        for (int t = 0; t < NT; ++t) top = fmaxf(top, fmaxf(c[t][2 * e], c[t][2 * e + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const bool grew = top > m[e];
        if (__any_sync(0xffffffffu, grew)) {
          const float f = rescale(m[e], top);
          m[e] = top;
          l[e] *= f;
#pragma unroll
          for (int t = 0; t < kN; ++t)
#pragma unroll
            for (int x = HALF ? 0 : 2 * e; x < (HALF ? 4 : 2 * e + 2); ++x) o[t][x] *= f;
        }
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int x = 2 * e; x < 2 * e + 2; ++x) {
            c[t][x] = ex2(c[t][x] - m[e]);
            sum += c[t][x];
          }
        l[e] += sum;
      }
    };
    // Two key tiles' weights as the A operands of the second product, part by part. Of up to eight rows the second parts are
    // rows eight and on, so that one product takes both and O's upper half is what they add.
    auto operands = [&](float (&x)[4], float (&y)[4], uint32_t (&p)[2][4]) {
      p[0][0] = split2(x[0], x[1]);
      p[0][2] = split2(y[0], y[1]);
      p[HALF ? 0 : 1][HALF ? 1 : 0] = pack2(x[0], x[1]);
      p[HALF ? 0 : 1][HALF ? 3 : 2] = pack2(y[0], y[1]);
      if constexpr (!HALF) {
        p[0][1] = split2(x[2], x[3]);
        p[0][3] = split2(y[2], y[3]);
        p[1][1] = pack2(x[2], x[3]);
        p[1][3] = pack2(y[2], y[3]);
      }
    };
    auto mma_p = [&](float (&c)[4], const uint32_t (&p)[2][4], uint32_t b0, uint32_t b1) {
      mma(c, p[0][0], p[0][1], p[0][2], p[0][3], b0, b1);
      if constexpr (!HALF) mma(c, p[1][0], p[1][1], p[1][2], p[1][3], b0, b1);
    };

    // this warp's first tile of the segment: tiles of the share go to the warps in turn
    const int turn = (int)((at - share.at) % kWarps);
    for (int f = (warp - turn + kWarps) % kWarps; f < seg; f += kWarps) {
      const int tile = here.tile + f;
      const uint32_t kt = ptx::smem_u32(ring + stage * S::kStage);
      if (!ptx::mbar_wait(&full[warp][stage], parity, &abort, kWaitLimit)) {
        *reinterpret_cast<volatile int*>(&abort) = 1;
        report(a.dev_status, SNAPKV_ERR_TIMEOUT);
      }
      __syncwarp();
      bool dirty = false;
      const bool cached = tile < here.s.cache_tiles;
      if (Q8 && cached) {
        // ---- 32 keys in 8 bits
        const int valid = here.s.rows - tile * kTile;
        const float* const ks = steps + stage * 2 * kTile;
        float c[kTile / 8][4];
#pragma unroll
        for (int t = 0; t < kTile / 8; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) c[t][e] = 0.f;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            const uint4 w = lds128(kt + code_at<D>(8 * t + j, (D / 64) * i + h));
            const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int s = 0; s < 4; ++s) mma_q(c[t], 4 * h + s, operand<0, 1>(word[s], word[s]), operand<2, 3>(word[s], word[s]));
          }
          const float2 h2 = *reinterpret_cast<const float2*>(ks + 8 * t + 2 * i);
          const float f0 = h2.x * (a.scale_log2 * kQ8Dot), f1 = h2.y * (a.scale_log2 * kQ8Dot);
          const bool s0 = 8 * t + 2 * i < valid, s1 = 8 * t + 2 * i + 1 < valid;
#pragma unroll
          for (int e = 0; e < kH; ++e) {
            c[t][2 * e] = s0 ? c[t][2 * e] * f0 : -INFINITY;
            c[t][2 * e + 1] = s1 ? c[t][2 * e + 1] * f1 : -INFINITY;
          }
        }
        softmax(c, std::integral_constant<int, kTile / 8>());
        const uint32_t vt = kt + S::kStage / 2;
#pragma unroll
        for (int g = 0; g < kTile / 16; ++g) {
#pragma unroll
          for (int t = 2 * g; t < 2 * g + 2; ++t) {
            float2 h2 = *reinterpret_cast<const float2*>(ks + kTile + 8 * t + 2 * i);
            h2.x = 8 * t + 2 * i < valid ? h2.x * kQ8P : 0.f;   // (what lies behind the rows may be anything)
            h2.y = 8 * t + 2 * i + 1 < valid ? h2.y * kQ8P : 0.f;
#pragma unroll
            for (int e = 0; e < kH; ++e) {
              c[t][2 * e] *= h2.x;
              c[t][2 * e + 1] *= h2.y;
            }
          }
          uint32_t p[2][4];
          operands(c[2 * g], c[2 * g + 1], p);
          const int r = 16 * g + 2 * i;
          if constexpr (D == 128) {
            const uint4 r0 = lds128(vt + code_at<D>(r, j)), r1 = lds128(vt + code_at<D>(r + 1, j)),
                        r8 = lds128(vt + code_at<D>(r + 8, j)), r9 = lds128(vt + code_at<D>(r + 9, j));
            const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w}, w8[4] = {r8.x, r8.y, r8.z, r8.w},
                           w9[4] = {r9.x, r9.y, r9.z, r9.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              mma_p(o[4 * w], p, operand<0, 4>(w0[w], w1[w]), operand<0, 4>(w8[w], w9[w]));
              mma_p(o[4 * w + 1], p, operand<1, 5>(w0[w], w1[w]), operand<1, 5>(w8[w], w9[w]));
              mma_p(o[4 * w + 2], p, operand<2, 6>(w0[w], w1[w]), operand<2, 6>(w8[w], w9[w]));
              mma_p(o[4 * w + 3], p, operand<3, 7>(w0[w], w1[w]), operand<3, 7>(w8[w], w9[w]));
            }
          } else {
            auto at8 = [&](int row) { return vt + code_at<D>(row, j / 2) + 8 * (j % 2); };
            const uint2 r0 = lds64(at8(r)), r1 = lds64(at8(r + 1)), r8 = lds64(at8(r + 8)), r9 = lds64(at8(r + 9));
            const uint32_t w0[2] = {r0.x, r0.y}, w1[2] = {r1.x, r1.y}, w8[2] = {r8.x, r8.y}, w9[2] = {r9.x, r9.y};
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              mma_p(o[4 * w], p, operand<0, 4>(w0[w], w1[w]), operand<0, 4>(w8[w], w9[w]));
              mma_p(o[4 * w + 1], p, operand<1, 5>(w0[w], w1[w]), operand<1, 5>(w8[w], w9[w]));
              mma_p(o[4 * w + 2], p, operand<2, 6>(w0[w], w1[w]), operand<2, 6>(w8[w], w9[w]));
              mma_p(o[4 * w + 3], p, operand<3, 7>(w0[w], w1[w]), operand<3, 7>(w8[w], w9[w]));
            }
          }
        }
      } else {
        // ---- bf16 keys: cached ones of a dense cache, or 16 drafted ones
        auto rows = [&](auto size, bool drafted) {
          constexpr int R = decltype(size)::value;
          const int first = drafted ? (tile - here.s.cache_tiles) * kNew : tile * kTile;
          const int valid = min(R, (drafted ? n : here.s.rows) - first);
          const uint32_t vt = kt + R * D * 2;
          // V's rows that nobody sees become zeros, as do drafted ones with an infinity or NaN, which the rows that see
          // them get as a NaN weight: 0 times it must not reach the others.
          uint32_t bad = 0;
          if (drafted) {
            bool mine = false;
            const int row = lane / 2;
            if (row < valid)
              for (int c = lane % 2; c < D / 8; c += 2) {
                const uint4 w = lds128(vt + bf16_at<R>(row, c));
                for (uint32_t x : {w.x, w.y, w.z, w.w}) mine |= (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
              }
            const uint32_t votes = __ballot_sync(0xffffffffu, mine);
            bad = (votes | (votes >> 1)) & 0x55555555u;   // bit 2 row
          }
          if (valid < R || bad) {
            for (int u = lane; u < R * (D / 8); u += 32) {
              const int row = u / (D / 8);
              if (row >= valid || (drafted && (bad >> (2 * (row & 15)) & 1))) sts128_zero(vt + bf16_at<R>(row, u % (D / 8)));
            }
            dirty = true;
            __syncwarp();
          }
          float c[R / 8][4];
#pragma unroll
          for (int t = 0; t < R / 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[t][e] = 0.f;
#pragma unroll
          for (int t = 0; t < R / 8; ++t) {
            if constexpr (Q8) {   // (the queries' channels lie as 8-bit rows want them)
#pragma unroll
              for (int s = 0; s < kK; ++s) {
                const int ch = (D / 4) * i + 4 * s;
                const uint2 w = lds64(kt + bf16_at<R>(8 * t + j, ch / 8) + 2 * (ch % 8));
                mma_q(c[t], s, w.x, w.y);
              }
            } else {
#pragma unroll
              for (int s = 0; s < kK; s += 2) {
                uint32_t x[4];
                load_matrices<false>(kt + bf16_at<R>(8 * t + lane % 8, 2 * s + lane / 8), x);
                mma_q(c[t], s, x[0], x[1]);
                mma_q(c[t], s + 1, x[2], x[3]);
              }
            }
          }
          const float f = Q8 ? a.scale_log2 * kNewDot : a.scale_log2;
#pragma unroll
          for (int t = 0; t < R / 8; ++t)
#pragma unroll
            for (int e = 0; e < 2 * kH; ++e) c[t][e] *= f;
          if (drafted) {
#pragma unroll
            for (int e = 0; e < kH; ++e) {
              const int r = j + 8 * e, token = (first_row + r) % n;
              const uint8_t* see = a.mask ? a.mask + here.seq * a.mask_stride + (int64_t)token * a.tokens : nullptr;
#pragma unroll
              for (int t = 0; t < R / 8; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const int k = 8 * t + 2 * i + x, key = first + k;
                  const bool seen = k < valid && r < count && (see ? see[key] != 0 : key <= token);
                  if (!seen)
                    c[t][2 * e + x] = -INFINITY;
                  else if (bad >> (2 * (k & 15)) & 1)
                    c[t][2 * e + x] = __uint_as_float(0x7FC00000u);
                }
            }
          } else if (valid < R) {
#pragma unroll
            for (int t = 0; t < R / 8; ++t)
#pragma unroll
              for (int e = 0; e < 2 * kH; ++e)
                if (8 * t + 2 * i + e % 2 >= valid) c[t][e] = -INFINITY;
          }
          softmax(c, std::integral_constant<int, R / 8>());
#pragma unroll
          for (int g = 0; g < R / 16; ++g) {
            if constexpr (Q8)
#pragma unroll
              for (int t = 2 * g; t < 2 * g + 2; ++t)
#pragma unroll
                for (int e = 0; e < 2 * kH; ++e) c[t][e] *= kNewP;
            uint32_t p[2][4];
            operands(c[2 * g], c[2 * g + 1], p);
            if constexpr (Q8) {
#pragma unroll
              for (int t = 0; t < kN; ++t) {   // channel tile t has channels kN n + t
                const int ch = kN * j + t;
                auto pair = [&](int row) {
                  return lds16(vt + bf16_at<R>(row, ch / 8) + 2 * (ch % 8)) | lds16(vt + bf16_at<R>(row + 1, ch / 8) + 2 * (ch % 8)) << 16;
                };
                mma_p(o[t], p, pair(16 * g + 2 * i), pair(16 * g + 2 * i + 8));
              }
            } else {
#pragma unroll
              for (int t = 0; t < kN; t += 2) {
                uint32_t x[4];
                load_matrices<true>(vt + bf16_at<R>(16 * g + lane % 16, t + lane / 16), x);
                mma_p(o[t], p, x[0], x[1]);
                mma_p(o[t + 1], p, x[2], x[3]);
              }
            }
          }
        };
        if constexpr (!Q8 && kTile != kNew) {
          if (cached)
            rows(std::integral_constant<int, kTile>(), false);
          else
            rows(std::integral_constant<int, kNew>(), true);
        } else {
          rows(std::integral_constant<int, kNew>(), !cached);
        }
      }
      // ---- the stage has been read
      if (dirty) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      send_next(stage);
      if (++stage == kStages) {
        stage = 0;
        parity ^= 1;
      }
    }

    // ---- the warps meet: two leave their parts, two add theirs
#pragma unroll
    for (int e = 0; e < kH; ++e) {
      const int r = j + 8 * e;
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      if (i == 0) {
        warp_m[warp][r] = m[e];
        warp_l[warp][r] = l[e];
      }
    }
    __syncthreads();
    auto leave = [&](bool add) {
#pragma unroll
      for (int e = 0; e < kH; ++e) {
        const int r = j + 8 * e;
        float f = rescale(m[e], fmaxf(fmaxf(warp_m[0][r], warp_m[1][r]), fmaxf(warp_m[2][r], warp_m[3][r])));
        if (Q8) f *= kQ8Out;
        float* const to = meet + (warp % 2 * kRows + r) * D;
#pragma unroll
        for (int t = 0; t < kN; ++t) {
          const float x = (HALF ? o[t][0] + o[t][2] : o[t][2 * e]) * f, y = (HALF ? o[t][1] + o[t][3] : o[t][2 * e + 1]) * f;
          if constexpr (Q8) {
            float* const u = to + kN * 2 * i + t;
            u[0] = add ? u[0] + x : x;
            u[kN] = add ? u[kN] + y : y;
          } else {
            float2* const u = reinterpret_cast<float2*>(to + 8 * t + 2 * i);
            *u = add ? make_float2(u->x + x, u->y + y) : make_float2(x, y);
          }
        }
      }
    };
    if (warp < 2) leave(false);
    __syncthreads();
    if (warp >= 2) leave(true);
    __syncthreads();
    float* const part = part_at<D>(a, (int)blockIdx.x, at > share.at ? 1 : 0);
    for (int u = tid; u < count * (D / 2); u += kThreads) {
      const int r = u / (D / 2), c = 2 * (u % (D / 2));
      const float top = fmaxf(fmaxf(warp_m[0][r], warp_m[1][r]), fmaxf(warp_m[2][r], warp_m[3][r]));
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum = fmaf(warp_l[w][r], rescale(warp_m[w][r], top), sum);
      const float2 x = *reinterpret_cast<const float2*>(meet + r * D + c), y = *reinterpret_cast<const float2*>(meet + (kRows + r) * D + c);
      if (whole) {
        const float scale = sum == 0.f ? 0.f : 1.0f / sum;
        const int64_t row = row_at(r);
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row * D + c) = pack2((x.x + y.x) * scale, (x.y + y.y) * scale);
        if (a.lse && c == 0) a.lse[row] = lse_of(top, sum);
      } else {
        *reinterpret_cast<float2*>(part + r * D + c) = make_float2(x.x + y.x, x.y + y.y);
        if (c == 0) {
          part[a.tile_q * D + r] = top;
          part[a.tile_q * (D + 1) + r] = sum;
        }
      }
    }
    __syncthreads();   // the meeting area is free
    at += seg;
    here.tile += seg;
    if (at < share.end) next_head<kTile, kNew>(a, here);
  }
}

template <bool Q8, int D, bool HALF> cudaError_t launch_typed(const TreeJob& job) {
  using S = Shape<Q8, D, HALF>;
  Args a = tree_args(job, S::kRows);
  a.least = kWarps;
  TreeMaps maps;
  if (!tree_maps(&maps, job, S::kTile, S::kNew)) return cudaErrorInvalidValue;
  cudaError_t err = allow_dynamic_smem<tree_mma_kernel<Q8, D, HALF>>(S::smem());
  if (err != cudaSuccess) return err;
  // Passes over the same rows side by side (where tokens differ, some siblings would have nothing to do).
  const int64_t passes = ((int64_t)a.group * a.tokens + S::kRows - 1) / S::kRows, ctas = 2 * (int64_t)device_sm_count();
  if (!job.n_new && passes > 1 && 4 * passes <= ctas) a.siblings = (int)passes;
  err = tree_fill(a, job, S::kTile, S::kNew, ctas - ctas % a.siblings);
  if (err != cudaSuccess) return err;
  tree_mma_kernel<Q8, D, HALF><<<a.ctas, kThreads, S::smem(), job.stream>>>(a, maps);
  err = cudaGetLastError();
  return err != cudaSuccess || a.direct ? err : launch_tree_join<__nv_bfloat16, D, S::kTile, S::kNew>(a, job.stream);
}

template <bool Q8, int D> cudaError_t launch_dim(const TreeJob& job) {
  return job.q_heads / job.heads * job.tokens <= 8 ? launch_typed<Q8, D, true>(job) : launch_typed<Q8, D, false>(job);
}

}  // namespace

cudaError_t launch_tree_mma(const TreeJob& job) {
  if (job.k_step) return job.head_dim == 64 ? launch_dim<true, 64>(job) : launch_dim<true, 128>(job);
  return job.head_dim == 64 ? launch_dim<false, 64>(job) : launch_dim<false, 128>(job);
}

}  // namespace snapkv
