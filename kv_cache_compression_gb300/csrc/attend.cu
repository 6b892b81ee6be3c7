// Scored decode attention with grouped queries, over a dense cache or one held in 4 bits.
//
//   s_gr = q_g . k_r / sqrt(d),  p_gr = softmax over r < len,  o_g = sum_r p_gr v_r
//   score_r = decay * score_r + sum_g p_gr
//
// Two launches. The first walks all tiles (a few dozen rows of one head) of all heads as one flat list,
// of which every CTA of one wave takes an equal, contiguous share, whatever the sequences' lengths: a
// CTA's share covers the end of one head, whole heads, and the start of another. A warp takes every
// kWarps-th tile of the share with an online softmax (running maximum m and sum l per query, output o
// not yet normalised, logits in the log2 domain); at the end of a head the CTA's warps meet in shared
// memory. A head that lies in one share is finished there; the parts of others, and the logits that a
// score will need, go to the workspace. The second launch joins the parts and turns logits into
// weights. It is released early (programmatic dependent launch) and waits on the device for the first.
// Rows are read once per pass of up to sixteen queries (fp32: eight) a KV head. (One cluster per head with
// the logits in shared memory, and everything in one launch, was measured first: 222 us where this takes 131
// on 2048 4-bit heads of 2208 rows, and 115 us where this takes 76 on 64 bf16 heads of 8192 to 16384 rows
// with four queries each.)
//
// Both products run on the tensor cores as m16n8k16 with eight queries as the columns: K Q^T has sixteen
// cached rows by sixteen channels as A, V^T P^T sixteen channels by sixteen cached rows. Weights cross
// from one's accumulators to the other's B operand by an 8 x 8 transpose in registers (movmatrix). They
// enter the second product in two bf16 parts (16 bits of mantissa: 0.1 to 0.3 % of the bf16 outputs are the
// neighbours of the exact ones, and 0.05 to 0.25 % with fp32 operations throughout); fp32 calls split q, p and the cached
// values into three (24 bits) and drop nothing above 2^-24 of a product's factors. (With the queries as
// rows of A in the first product no transpose is needed, but half of A is zeros, which cost twice the
// instructions and, as A takes four neighbouring registers, moves around each: 475 instructions per
// 16 rows of 4-bit K and V against 427, and 318 with the constants and tiles of today.)
//
// With a decode step's few queries the kernel is bound by the cache's bytes. Legacy mma.sync is fast
// enough for that (128 cached values per instruction, against about 50 per clock and SM that HBM
// delivers at 4 bits), and unlike tcgen05.mma it takes levels and weights from registers, where
// unpacking and the softmax leave them.
//
// Each warp moves its own tiles with cp.async through a ring of its own, which runs ahead across the
// ends of heads; at the end of a head a warp leaves its part and goes on.
//
// Measured (GB300, first launch and join; HBM floor at 6.79 TB/s in brackets): bf16, 2048 heads of about 2140
// rows 322 us without scores [331] and 368 with [336]; 64 heads of 8192 to 16384 rows, four queries, with scores
// 77 us [60]; 32 heads of 1057 rows 12 us without scores [2.6]; fp32, 64 heads of 8192 rows, four queries, with
// scores 100 us [80]. 4 bits: the 2048 heads 131 us without scores [93] and 157 with [98], the grouped ones with
// scores 38 us [18], 32 heads of 131072 rows without 115 us [89].
// Dense rows are read at the rate of a copy; scores add their logits' traffic and the second launch (8 to 10 us
// on the grouped heads). 4-bit rows are bound by instructions: 318 per 16 rows, 140 of them on the logic pipe,
// which is 70 of the 137 cycles that an SM takes (98 would be HBM's); copying the same tiles and computing
// nothing takes 103 and 98 us where this takes 131 and 115.
#include <type_traits>

#include "cache_internal.h"
#include "q4.cuh"
#include "sm100_ptx.cuh"
#include "snapkv_internal.h"

namespace snapkv {
namespace {

struct AttendArgs {
  const void* q;
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* km;
  const uint8_t* vm;
  const int32_t* len;
  float* score;
  void* out;
  float decay, scale_log2;
  int64_t cap;
  int batch, heads, group;
  int passes, tile_q;   // queries are served tile_q at a time (the last of `passes` passes may have fewer)
  int ctas;             // of the first launch
  bool direct;          // a CTA per head, which finishes it (no second launch)
  // workspace: a head is (sequence, KV head, pass) here
  float* logits;        // [heads][tile_q][logit_stride] (scores only)
  int64_t logit_stride; // cap, rounded up to whole 32-byte sectors
  float* stats;         // [heads][2][tile_q]: maximum and sum of a head that one CTA finished
  int64_t* upto;        // [batch + 1]: tiles of a head in the sequences before, and of all (more than kWarpBatch)
  float* parts;         // [ctas][2] of (o [tile_q][D], m [tile_q], l [tile_q])
  int32_t* dev_status;
  Q4Ones ones;
};

// The CTAs of the first launch that get a share: no more than give every warp a tile.
constexpr int kWarps = 4;
__device__ __forceinline__ int working_ctas(int64_t total, int ctas) {
  const int64_t most = (total + kWarps - 1) / kWarps;
  return most < ctas ? (int)most : ctas;
}

// CTA c's share of `total` tiles starts here. (c <= ctas <= 1024 and total <= 2^45: no product overflows;
// short lists, where the latency counts, get by with a 32-bit division.)
__device__ __forceinline__ int64_t share_start(int64_t total, int ctas, int c) {
  if (total < (1 << 22)) return (uint32_t)total * (uint32_t)c / (uint32_t)ctas;
  return total * c / ctas;
}

// The CTA whose share holds flat tile t: the last one that starts at or before it.
__device__ __forceinline__ int share_of(int64_t total, int ctas, int64_t t) {
  int c = total < (1 << 22) ? (int)((uint32_t)t * (uint32_t)ctas / (uint32_t)total) : (int)(t * ctas / total);
  while (c + 1 < ctas && share_start(total, ctas, c + 1) <= t) ++c;   // (the quotient's share starts at or before t)
  return c;
}

__device__ __forceinline__ int visible_rows(const AttendArgs& a, int b) {
  const int n = a.len[b];
  return n < 0 ? 0 : (int64_t)n > a.cap ? (int)a.cap : n;
}

// Flat tile index = (tiles of the sequences before, times heads per sequence) + (head within the sequence) *
// tiles + tile.
template <int TILE> __device__ __forceinline__ int tiles_of(const AttendArgs& a, int b) {
  return (visible_rows(a, b) + TILE - 1) / TILE;
}

// Sums over the sequences: a thread takes sequences b0 .. b1 - 1, with `mine` tiles after `upto`, of `total`.
// Up to kWarpBatch sequences every warp asks for itself, lane by lane, and the joining kernel asks again. More are
// summed up by all threads of a CTA of the first launch, whose CTAs also leave `upto` of every sequence and the
// total for the joining kernel: bf16, scores, 500 to 1000 rows of 64 channels, 1024 sequences of 8 heads take 310 us
// [239 at 6.79 TB/s], 4096 of one head 168 [120]. With every warp of both kernels summing up they took 532 and 666.
constexpr int kWarpBatch = 32;
struct SeqScan {
  int b0, b1;
  int64_t upto, mine, total;
};

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ int64_t warp_scan(int64_t x) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
    if ((int)threadIdx.x % 32 >= off) x += y;
  }
  return x;
}

template <int TILE> __device__ __forceinline__ SeqScan scan_by_warp(const AttendArgs& a) {
  SeqScan s;
  s.b0 = min(a.batch, (int)threadIdx.x % 32);
  s.b1 = min(a.batch, s.b0 + 1);
  s.mine = s.b0 < s.b1 ? tiles_of<TILE>(a, s.b0) : 0;
  const int64_t x = warp_scan(s.mine);
  s.total = __shfl_sync(0xffffffffu, x, 31);
  s.upto = x - s.mine;
  return s;
}

template <int TILE> __device__ __forceinline__ SeqScan scan_by_block(const AttendArgs& a, int64_t (&sums)[kWarps]) {
  const int tid = threadIdx.x, chunk = (a.batch + 32 * kWarps - 1) / (32 * kWarps);
  SeqScan s;
  s.b0 = min(a.batch, tid * chunk);
  s.b1 = min(a.batch, s.b0 + chunk);
  s.mine = 0;
#pragma unroll 8
  for (int b = s.b0; b < s.b1; ++b) s.mine += tiles_of<TILE>(a, b);
  const int64_t x = warp_scan(s.mine);
  if (tid % 32 == 31) sums[tid / 32] = x;
  __syncthreads();
  s.total = 0;
  s.upto = x - s.mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < tid / 32) s.upto += sums[w];
    s.total += sums[w];
  }
  return s;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src) : "memory");
}
template <int N> __device__ __forceinline__ void cp_async_small(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(ptx::smem_u32(dst)), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit elements that the warp holds a row per four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Four 8 x 8 matrices of 16-bit elements, their 16-byte rows at the addresses of lanes 0 .. 7, 8 .. 15, ...
template <bool TRANS> __device__ __forceinline__ void load_matrices(const void* row, uint32_t (&x)[4]) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(ptx::smem_u32(row)) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(ptx::smem_u32(row)) : "memory");
}

// Two fp32 values as a bf16 pair (x in the low half).
__device__ __forceinline__ uint32_t pack2(float2 v) {
  const __nv_bfloat162 two = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&two);
}
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// The pair, and in v what `share` times it leaves of the values.
__device__ __forceinline__ uint32_t split2(float2& v, float share = 1.0f) {
  const uint32_t w = pack2(v);
  v = fma2(unpack2(w), make_float2(-share, -share), v);
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

// Format Q4 (codes and pairs) or dense rows of IO; IO is the type of q and out; QT: tiles of eight queries.
template <bool Q4, typename IO, int D, int QT> struct Shape {
  static constexpr bool kWide = sizeof(IO) == 4;                    // fp32: three bf16 parts
  static constexpr int kParts = kWide ? 3 : 2;                      // of a weight
  static constexpr int kNg = D / kQ4Group;
  static constexpr int kRow = Q4 ? D / 2 : D * (int)sizeof(IO);     // bytes of a row of K (and of V)
  static constexpr int kMeta = Q4 ? 4 * kNg : 0;
  static constexpr int kTile = Q4 ? (QT == 1 ? 64 : 32) : (kRow >= 256 ? 16 : 32);   // rows
  static constexpr int kStage = 2 * kTile * (kRow + kMeta);         // 4 to 16 KB of K and V together
  static constexpr int kStages = Q4 ? 2 : 3;
  static constexpr int kWarps = snapkv::kWarps;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRing = kWarps * kStages * kStage;
  // What the ring, the meeting area and the registers leave room for. Sixteen queries over dense rows of 128 channels: 96 KB
  // of ring and 18 to 32 of meeting, one CTA. Its four warps then wait for one another's latency more than for anything else
  // (64 heads of 8192 rows: an instruction in 24 % of a scheduler's cycles, DRAM at 60 %).
  static constexpr int kCtasPerSm = Q4 ? (kWide || QT > 1 ? 2 : 3) : kRow * QT >= 512 ? 1 : 2;
  static constexpr int smem(int tile_q, bool direct) {   // and a direct head's logits
    return kRing + kWarps * tile_q * D * 4 + (direct ? tile_q * kDirectRows * 4 : 0);
  }
};

// 16-byte pieces of a row are stored XORed with the row's low three bits where rows are a multiple of
// 128 bytes: the eight rows (first product) or four rows (second) that a warp reads at a time then
// fall into different banks. 4-bit rows are shorter and need none.
template <int ROW> __device__ __forceinline__ uint32_t piece_at(int row, int piece) {
  if constexpr (ROW >= 128) return row * ROW + ((piece ^ (row & 7)) << 4);
  return row * ROW + (piece << 4);
}

// NG 32-bit words of shared memory (the second is 0 where there is one).
template <int NG> __device__ __forceinline__ uint2 load_words(const uint8_t* at) {
  if constexpr (NG == 2) return *reinterpret_cast<const uint2*>(at);
  return make_uint2(*reinterpret_cast<const uint32_t*>(at), 0u);
}

// Row j of an 8-row tile. Where the second product gathers its rows by hand, they are mixed so that the
// rows 2 i and 2 i + 1 of the four lanes that read together lie in different banks.
template <bool MIXED> __device__ __forceinline__ int row_of(int j) { return MIXED ? (j >> 1) + 4 * (j & 1) : j; }

// Counts this warp in, after what all its lanes wrote to shared memory; returns how many came before (and
// what those wrote can then be read).
__device__ __forceinline__ int arrive(int* count) {
  __syncwarp();
  int before = 0;
  if (threadIdx.x % 32 == 0)
    asm volatile("atom.acq_rel.cta.shared::cta.add.s32 %0, [%1], 1;" : "=r"(before) : "r"(ptx::smem_u32(count)) : "memory");
  before = __shfl_sync(0xffffffffu, before, 0);
  __syncwarp();
  return before;
}

__device__ __forceinline__ void publish(int* value, int x) {
  asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(ptx::smem_u32(value)), "r"(x) : "memory");
}

// Waits (about two seconds at most; false then) until *value >= x was published.
__device__ __forceinline__ bool wait_for(int* value, int x) {
  int seen;
  const long long t0 = clock64();
  do {
    asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(seen) : "r"(ptx::smem_u32(value)) : "memory");
  } while (seen < x && clock64() - t0 < 4000000000LL);
  __syncwarp();
  return seen >= x;
}

// FOUR (bf16, at most four queries a pass): the second product's columns 4 .. 7 are the second parts of
// the weights in columns 0 .. 3, and one instruction does for both. The first product then has every
// query twice.
// QT = 2 (bf16): sixteen queries a pass share the work on each row's operands.
template <bool Q4, typename IO, int D, int QT, bool FOUR>
__global__ void __launch_bounds__(Shape<Q4, IO, D, QT>::kThreads, Shape<Q4, IO, D, QT>::kCtasPerSm) attend_kernel(AttendArgs a) {
  using S = Shape<Q4, IO, D, QT>;
  static_assert(!FOUR || (!S::kWide && QT == 1), "two parts of four queries");
  static_assert(QT == 1 || !S::kWide, "registers");
  constexpr int kParts = FOUR ? 1 : S::kParts;
  constexpr int kSteps = D / 16;          // 16-channel steps of the first product
  constexpr int kPairs = D / 16;          // 16-channel tiles of the second: two of a lane's D / 8 channels
  constexpr int kSub = S::kTile / 16;     // 16-row parts of a tile
  constexpr int kNg = S::kNg;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float warp_m[S::kWarps][8 * QT], warp_l[S::kWarps][8 * QT];
  __shared__ float head_m[8 * QT], head_r[8 * QT];
  __shared__ int64_t sums[kWarps], shared_before;   // (more than kWarpBatch sequences)
  __shared__ int shared_seq;
  __shared__ int arrived, merged;   // warps whose part of this head is in `meet`; heads merged

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  // In accumulators a lane holds row (K Q^T) or channel (V^T P^T) j and j + 8 of 16 for queries qa and qa + 1; in
  // operands it holds column j, or rows j and j + 8, at places 2 i, 2 i + 1, 2 i + 8 and 2 i + 9 along k.
  const int j = lane / 4, i = lane % 4;
  const int qa = FOUR ? 2 * i % 4 : 2 * i;
  const float part2 = FOUR && i >= 2 ? 1.0f : 0.0f;   // this lane's columns are second parts
  const int jrow = row_of<Q4 || S::kWide>(j);         // row j of an 8-row tile, as it lies in the cache
  const int per_seq = a.heads * a.passes;   // heads of a sequence
  const Q4Ones ones = a.ones;
  if (tid == 0) arrived = merged = 0;
  __syncthreads();

  // ---- this CTA's share of the tiles, and the sequence it starts in (every warp finds them for itself)
  int64_t at, end, before;
  int first_seq;
  if (a.direct) {
    const int vh = (int)blockIdx.x;
    first_seq = vh / per_seq;
    const int tiles = tiles_of<S::kTile>(a, first_seq);
    before = 0;   // (a list of this sequence alone)
    at = (int64_t)(vh - first_seq * per_seq) * tiles;
    end = at + tiles;
    if (vh % per_seq == 0 && tid == 0 && (int64_t)a.len[first_seq] > a.cap) report(a.dev_status, SNAPKV_ERR_CAPACITY);
    if (tiles == 0) {
      const int pass = vh % a.passes, bh = vh / a.passes;
      IO* out = static_cast<IO*>(a.out) + ((int64_t)bh * a.group + pass * a.tile_q) * D;
      for (int u = tid; u < min(a.tile_q, a.group - pass * a.tile_q) * D; u += S::kThreads) store1<IO>(out + u, 0.f);
      return;
    }
  } else {
    const bool by_warp = a.batch <= kWarpBatch;
    const SeqScan scan = by_warp ? scan_by_warp<S::kTile>(a) : scan_by_block<S::kTile>(a, sums);
    // Each thread's sequences are looked after by one CTA.
    if (by_warp ? blockIdx.x == 0 && warp == 0 : tid % gridDim.x == blockIdx.x) {
      int64_t upto = scan.upto;
      for (int b = scan.b0; b < scan.b1; ++b) {
        if ((int64_t)a.len[b] > a.cap) report(a.dev_status, SNAPKV_ERR_CAPACITY);
        if (!by_warp) {
          a.upto[b] = upto;
          upto += tiles_of<S::kTile>(a, b);
        }
      }
      if (!by_warp && tid == 0) a.upto[a.batch] = scan.total;
    }
    const int64_t total = scan.total * per_seq;
    const int ctas = working_ctas(total, a.ctas);
    if ((int)blockIdx.x >= ctas) return;
    at = share_start(total, ctas, (int)blockIdx.x);
    end = share_start(total, ctas, (int)blockIdx.x + 1);   // > at
    int seq = -1;
    int64_t upto = scan.upto;
    if (at >= upto * per_seq && at < (upto + scan.mine) * per_seq) {
      seq = scan.b0;
      for (int t; at >= (upto + (t = tiles_of<S::kTile>(a, seq))) * per_seq; ++seq) upto += t;
    }
    if (by_warp) {
      const int owner = __ffs(__ballot_sync(0xffffffffu, seq >= 0)) - 1;
      first_seq = __shfl_sync(0xffffffffu, seq, owner);
      before = __shfl_sync(0xffffffffu, upto, owner);
    } else {
      if (seq >= 0) {
        shared_seq = seq;
        shared_before = upto;
      }
      __syncthreads();
      first_seq = shared_seq;
      before = shared_before;
    }
  }

  // A place in the list: a tile of a head, and what its addresses need.
  struct Place {
    int seq, head, rows, tiles, tile;   // head: within the sequence, over passes
    int64_t row0;                       // the KV head's first row in the cache
  };
  auto first_row = [&](const Place& p) {
    return ((int64_t)p.seq * a.heads + (a.passes == 1 ? p.head : p.head / a.passes)) * a.cap;
  };
  Place here;
  here.seq = first_seq;
  here.rows = visible_rows(a, here.seq);
  here.tiles = (here.rows + S::kTile - 1) / S::kTile;
  {
    const int64_t in_seq = at - before * per_seq;
    here.head = in_seq < ((int64_t)1 << 32) ? (int)((uint32_t)in_seq / (uint32_t)here.tiles) : (int)(in_seq / here.tiles);
    here.tile = (int)(in_seq - (int64_t)here.head * here.tiles);
    here.row0 = first_row(here);
  }
  // Moves p, whose tile may have run past its head, to the head that holds it (which exists).
  auto settle = [&](Place& p) {
    while (p.tile >= p.tiles) {
      p.tile -= p.tiles;
      if (++p.head == per_seq) {
        p.head = 0;
        do {
          p.rows = visible_rows(a, ++p.seq);
          p.tiles = (p.rows + S::kTile - 1) / S::kTile;
        } while (p.tiles == 0);
      }
      p.row0 = first_row(p);
    }
  };

  uint8_t* ring = smem + warp * (S::kStages * S::kStage);
  float* meet = reinterpret_cast<float*>(smem + S::kRing);   // [kWarps][tile_q][D]

  // Copies a tile into ring slot `slot`; rows past the head's end become zeros, whatever the cache holds.
  auto fetch = [&](const Place& p, int slot) {
    constexpr int kPieces = S::kRow / 16, kAll = S::kTile * kPieces;
    uint8_t* dst = ring + slot * S::kStage;
    const int64_t row0 = p.row0 + (int64_t)p.tile * S::kTile;
    const int left = p.rows - p.tile * S::kTile;   // > 0
    auto copy = [&](auto whole) {   // whole tiles, all but a head's last, need no look at each row
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint8_t* src = (kv ? a.v : a.k) + row0 * S::kRow + lane * 16;
        uint8_t* to = dst + kv * (S::kTile * S::kRow);
#pragma unroll
        for (int j = 0; j < kAll / 32; ++j) {
          const int u = lane + 32 * j, row = u / kPieces, piece = u % kPieces;
          if constexpr (decltype(whole)::value) {
            cp_async16(to + piece_at<S::kRow>(row, piece), src + j * 512);
          } else {
            const bool in = row < left;
            cp_async16(to + piece_at<S::kRow>(row, piece), in ? src + j * 512 : src - lane * 16, in ? 16 : 0);
          }
        }
        if constexpr (Q4) {
          const uint8_t* msrc = (kv ? a.vm : a.km) + row0 * S::kMeta + lane * S::kMeta;
          uint8_t* mto = dst + 2 * (S::kTile * S::kRow) + kv * (S::kTile * S::kMeta) + lane * S::kMeta;
          static_assert(S::kTile % 32 == 0, "a pair of each row per lane and turn");
#pragma unroll
          for (int row = 0; row < S::kTile; row += 32) {
            if constexpr (decltype(whole)::value) {
              cp_async_small<S::kMeta>(mto + row * S::kMeta, msrc + row * S::kMeta, S::kMeta);
            } else {
              const bool in = lane + row < left;
              cp_async_small<S::kMeta>(mto + row * S::kMeta, in ? msrc + row * S::kMeta : msrc - lane * S::kMeta, in ? S::kMeta : 0);
            }
          }
        }
      }
    };
    if (!in_bounds(p.seq < a.batch && p.head < per_seq && left > 0 && p.rows <= a.cap, a.dev_status)) return;
    if (left >= S::kTile)
      copy(std::true_type{});
    else
      copy(std::false_type{});
  };

  // The ring starts filling: tiles at + warp, + kWarps, ...
  Place ahead = here;
  int64_t ahead_at = at + warp;
  ahead.tile += warp;
  auto fetch_next = [&](int slot) {
    if (ahead_at < end) {
      settle(ahead);
      fetch(ahead, slot);
      ahead.tile += S::kWarps;
      ahead_at += S::kWarps;
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) fetch_next(s);
  int slot = 0;
  int64_t mine_at = at + warp;            // this warp's next tile
  const int64_t share0 = at;

  for (int segment = 0; at < end; ++segment) {   // one head, or the part of it that lies in the share
    const int pass = a.passes == 1 ? 0 : here.head % a.passes;
    const int tile_q = min(a.tile_q, a.group - pass * a.tile_q);
    const int64_t bh = (int64_t)here.seq * a.heads + (a.passes == 1 ? here.head : here.head / a.passes);
    const int64_t vh = (int64_t)here.seq * per_seq + here.head;
    const int64_t q0 = bh * a.group + (int64_t)pass * a.tile_q;
    const int64_t seg_end = min(end, at + (here.tiles - here.tile));
    const int n = here.rows;
    float* logits = !a.score ? nullptr : a.direct ? meet + S::kWarps * a.tile_q * D : a.logits + vh * a.tile_q * a.logit_stride;
    // (Every address of the segment follows from these; the whole CTA agrees.)
    if (!in_bounds(here.seq < a.batch && here.head < per_seq && tile_q >= 1 && tile_q <= 8 * QT && n <= a.cap &&
                       n <= a.logit_stride && here.tile + (seg_end - at) <= here.tiles && (a.direct || (int)blockIdx.x < a.ctas),
                   a.dev_status))
      break;

    // B operands of the first product: channels c .. c + 3 of the query of column j for each step, as the
    // lane's share of the rows is laid out (see `first product` below).
    uint32_t qb[QT][kSteps][S::kWide ? 6 : 2];
    float qsum[QT][Q4 ? kNg : 1][2];   // per group, of queries qa and qa + 1
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const int qcol = 8 * t + (FOUR ? j % 4 : j);
      const IO* qp = static_cast<const IO*>(a.q) + (q0 + (qcol < tile_q ? qcol : 0)) * D;
      float sum[Q4 ? kNg : 1] = {};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        int c;
        if constexpr (Q4)
          c = 64 * (s / 4) + 16 * i + 8 * ((s % 4) / 2) + 4 * (s % 2);
        else
          c = 16 * s + (S::kWide ? 4 * i : 2 * i);
        float2 x, y;
        if constexpr (S::kWide) {
          const float4 f = *reinterpret_cast<const float4*>(qp + c);
          x = make_float2(f.x, f.y);
          y = make_float2(f.z, f.w);
        } else {
          const uint32_t* f = reinterpret_cast<const uint32_t*>(qp + c);
          x = unpack2(f[0]);
          y = unpack2(f[Q4 ? 1 : 4]);
        }
        if (qcol >= tile_q) x = y = make_float2(0.f, 0.f);
        if constexpr (Q4) {
          sum[s / 4] += (x.x + x.y) + (y.x + y.y);
          x = mul2(x, make_float2(kQ4QEven, kQ4QEven));
          y = mul2(y, make_float2(kQ4QOdd, kQ4QOdd));
        }
#pragma unroll
        for (int part = 0; part < (S::kWide ? 3 : 1); ++part) {
          qb[t][s][2 * part] = split2(x);
          qb[t][s][2 * part + 1] = split2(y);
        }
      }
      if constexpr (Q4) {
#pragma unroll
        for (int g = 0; g < kNg; ++g) {
          sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
          sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
          sum[g] *= a.scale_log2;
          qsum[t][g][0] = __shfl_sync(0xffffffffu, sum[g], 4 * qa);
          qsum[t][g][1] = __shfl_sync(0xffffffffu, sum[g], 4 * qa + 4);
        }
      }
    }
    const float dot_scale = Q4 ? a.scale_log2 * kQ4Dot : a.scale_log2;

    // Per query qa, qa + 1 of each tile of queries:
    float m[QT][2], l[QT][2];
    // Channel pair t of the lane: [0], [1] its first channel for queries qa, qa + 1; [2], [3] its second.
    float o[QT][kPairs][4];
    float oz[QT][Q4 ? kNg : 1][2];   // sum of p z over this lane's rows
#pragma unroll
    for (int q = 0; q < QT; ++q) {
      m[q][0] = m[q][1] = -INFINITY;
      l[q][0] = l[q][1] = 0.f;
#pragma unroll
      for (int t = 0; t < kPairs; ++t) o[q][t][0] = o[q][t][1] = o[q][t][2] = o[q][t][3] = 0.f;
#pragma unroll
      for (int g = 0; g < (Q4 ? kNg : 1); ++g) oz[q][g][0] = oz[q][g][1] = 0.f;
    }

    // First product: B in one part (bf16), or three (fp32: the small parts' products have an accumulator of
    // their own, as a tensor-core addition truncates at its accumulator's magnitude).
    auto mma_q = [&](float* c, float* small, const uint32_t* w, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
      mma16816(c, a0, a1, a2, a3, w[0], w[1]);
      if constexpr (S::kWide) {
        mma16816(small, a0, a1, a2, a3, w[2], w[3]);
        mma16816(small, a0, a1, a2, a3, w[4], w[5]);
      }
    };

    // Weights of rows j (x[0]) and j + 8 (x[1]), for queries qa and qa + 1, as B operands in parts.
    auto weight_parts = [&](float2 (&x)[2], uint32_t (&w)[S::kParts][2]) {
#pragma unroll
      for (int part = 0; part < kParts; ++part)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if constexpr (FOUR) {
            split2(x[half], part2);
            w[0][half] = transpose8(pack2(x[half]));
          } else {
            w[part][half] = transpose8(split2(x[half]));
          }
        }
    };

    for (; mine_at < seg_end; mine_at += S::kWarps) {
      cp_wait<S::kStages - 2>();
      __syncwarp();   // every lane's copies of this tile have landed; the slot before it is free
      fetch_next(slot == 0 ? S::kStages - 1 : slot - 1);
      const uint8_t* kt = ring + slot * S::kStage;
      const uint8_t* vt = kt + S::kTile * S::kRow;
      const uint8_t* kmt = kt + 2 * (S::kTile * S::kRow);
      const uint8_t* vmt = kmt + S::kTile * S::kMeta;
      slot = slot + 1 == S::kStages ? 0 : slot + 1;
      const int base = (here.tile + (int)(mine_at - at)) * S::kTile;

      // ---- first product: logits of kSub x 16 rows
      float sv[QT][kSub][4];   // row j of a part for queries qa, qa + 1, then row j + 8
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
        if constexpr (Q4) {
          uint32_t w[2][2 * kNg];   // words (o = 0, 1; g) of this lane's 16 channels a group, of rows j, j + 8
          float2 hz[2][kNg];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int row = 16 * sub + 8 * half + jrow;
            const uint2 kz = load_words<kNg>(kmt + row * S::kMeta);
            hz[half][0] = unpack2(kz.x);
            if constexpr (kNg == 2) {
              hz[half][1] = unpack2(kz.y);
              const uint4 x = *reinterpret_cast<const uint4*>(kt + row * S::kRow + 16 * i);
              w[half][0] = x.x; w[half][1] = x.y; w[half][2] = x.z; w[half][3] = x.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(kt + row * S::kRow + 8 * i);
              w[half][0] = x.x; w[half][1] = x.y;
            }
          }
          float d[QT][4] = {}, zq[QT][4] = {};
#pragma unroll
          for (int g = 0; g < kNg; ++g) {
            float dot[QT][4] = {}, small[QT][4] = {};
#pragma unroll
            for (int o2 = 0; o2 < 2; ++o2) {
              uint32_t e[2][4];
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t word = w[half][q4_word<kNg>(g, o2)];
                q4_operands(ones, word, prmt(word, word, 0x2301), e[half]);
              }
#pragma unroll
              for (int q = 0; q < QT; ++q) {
                mma_q(dot[q], small[q], qb[q][4 * g + 2 * o2], e[0][0], e[1][0], e[0][1], e[1][1]);
                mma_q(dot[q], small[q], qb[q][4 * g + 2 * o2 + 1], e[0][2], e[1][2], e[0][3], e[1][3]);
              }
            }
#pragma unroll
            for (int q = 0; q < QT; ++q)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                d[q][e] = fmaf(hz[e / 2][g].x, S::kWide ? dot[q][e] + small[q][e] : dot[q][e], d[q][e]);
                zq[q][e] = fmaf(hz[e / 2][g].y, qsum[q][g][e % 2], zq[q][e]);
              }
          }
#pragma unroll
          for (int q = 0; q < QT; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) sv[q][sub][e] = fmaf(d[q][e], dot_scale, zq[q][e]);
        } else if constexpr (S::kWide) {
          float dot[4] = {}, small[4] = {};
#pragma unroll
          for (int s4 = 0; s4 < kSteps; ++s4) {
            float2 f[2][2];   // [rows j, j + 8][channels 4 i, + 1 and 4 i + 2, + 3 of the step's 16]
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const float4 x = *reinterpret_cast<const float4*>(kt + piece_at<S::kRow>(16 * sub + 8 * half + jrow, 4 * s4 + i));
              f[half][0] = make_float2(x.x, x.y);
              f[half][1] = make_float2(x.z, x.w);
            }
#pragma unroll
            for (int kp = 0; kp < 3; ++kp) {   // parts of the keys; those of the queries with them
              const uint32_t a0 = split2(f[0][0]), a1 = split2(f[1][0]), a2 = split2(f[0][1]), a3 = split2(f[1][1]);
#pragma unroll
              for (int part = 0; part < 3 - kp; ++part)
                mma16816(kp + part ? small : dot, a0, a1, a2, a3, qb[0][s4][2 * part], qb[0][s4][2 * part + 1]);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sv[0][sub][e] = (dot[e] + small[e]) * dot_scale;
        } else {
          float dot[QT][4] = {};
#pragma unroll
          for (int s4 = 0; s4 < kSteps; ++s4) {
            // matrices: rows 0 .. 7 and 8 .. 15 of the step's first eight channels, then of the others
            uint32_t x[4];
            load_matrices<false>(kt + piece_at<S::kRow>(16 * sub + lane % 16, 2 * s4 + lane / 16), x);
#pragma unroll
            for (int q = 0; q < QT; ++q) mma_q(dot[q], dot[q], qb[q][s4], x[0], x[1], x[2], x[3]);
          }
#pragma unroll
          for (int q = 0; q < QT; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) sv[q][sub][e] = dot[q][e] * dot_scale;
        }
      }

      // ---- masks, the running maximum, and the logits that the scores will need
      const int left = n - base - jrow;   // rows 16 sub + 8 half of the tile below this are visible
      float2 shift[QT];
#pragma unroll
      for (int q = 0; q < QT; ++q) {
        if (base + S::kTile > n) {
#pragma unroll
          for (int sub = 0; sub < kSub; ++sub)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (16 * sub + 8 * (e / 2) >= left) sv[q][sub][e] = -INFINITY;
        }
        if (logits && !(FOUR && i >= 2)) {
#pragma unroll
          for (int e2 = 0; e2 < 2; ++e2) {
            const int qq = 8 * q + qa + e2;
            float* to = logits + qq * a.logit_stride + base + jrow;
            if (qq < tile_q) {
#pragma unroll
              for (int sub = 0; sub < kSub; ++sub)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                  if (16 * sub + 8 * half < left && in_bounds(base + jrow + 16 * sub + 8 * half < n, a.dev_status))
                    to[16 * sub + 8 * half] = sv[q][sub][2 * half + e2];
            }
          }
        }
        float top[2] = {m[q][0], m[q][1]};
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
          top[0] = fmaxf(top[0], fmaxf(sv[q][sub][0], sv[q][sub][2]));
          top[1] = fmaxf(top[1], fmaxf(sv[q][sub][1], sv[q][sub][3]));
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], off));
          top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], off));
        }
        if (__any_sync(0xffffffffu, top[0] > m[q][0] || top[1] > m[q][1])) {
          const float c0 = m[q][0] == -INFINITY ? 0.f : ex2(m[q][0] - top[0]);
          const float c1 = m[q][1] == -INFINITY ? 0.f : ex2(m[q][1] - top[1]);
          l[q][0] *= c0;
          l[q][1] *= c1;
#pragma unroll
          for (int t = 0; t < kPairs; ++t) {
            o[q][t][0] *= c0; o[q][t][1] *= c1; o[q][t][2] *= c0; o[q][t][3] *= c1;
          }
          if constexpr (Q4) {
#pragma unroll
            for (int g = 0; g < kNg; ++g) {
              oz[q][g][0] *= c0;
              oz[q][g][1] *= c1;
            }
          }
          m[q][0] = top[0];
          m[q][1] = top[1];
        }
        shift[q] = make_float2(m[q][0] == -INFINITY ? 0.f : -m[q][0], m[q][1] == -INFINITY ? 0.f : -m[q][1]);
      }

      // ---- second product
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
        float2 p[QT][2];   // rows j, j + 8
#pragma unroll
        for (int q = 0; q < QT; ++q)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float2 x = add2(make_float2(sv[q][sub][2 * half], sv[q][sub][2 * half + 1]), shift[q]);
            p[q][half] = make_float2(ex2(x.x), ex2(x.y));
            l[q][0] += p[q][half].x;
            l[q][1] += p[q][half].y;
          }
        if constexpr (Q4) {
          float2 hz[2][kNg];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint2 vz = load_words<kNg>(vmt + (16 * sub + 8 * half + jrow) * S::kMeta);
            hz[half][0] = unpack2(vz.x);
            if constexpr (kNg == 2) hz[half][1] = unpack2(vz.y);
          }
          uint32_t w[4][kNg];   // rows 2 i, 2 i + 1, 2 i + 8, 2 i + 9: i, 4 + i, 8 + i, 12 + i of the cache
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint2 x = load_words<kNg>(vt + (16 * sub + 4 * e + i) * S::kRow + 4 * kNg * j);
            w[e][0] = x.x;
            if constexpr (kNg == 2) w[e][1] = x.y;
          }
#pragma unroll
          for (int q = 0; q < QT; ++q)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
              for (int g = 0; g < kNg; ++g) {
                oz[q][g][0] = fmaf(p[q][half].x, hz[half][g].y, oz[q][g][0]);
                oz[q][g][1] = fmaf(p[q][half].y, hz[half][g].y, oz[q][g][1]);
              }
              p[q][half] = mul2(p[q][half], make_float2(kQ4P, kQ4P));
            }
#pragma unroll
          for (int g = 0; g < kNg; ++g) {
            uint32_t pb[QT][S::kParts][2];
#pragma unroll
            for (int q = 0; q < QT; ++q) {
              float2 ph[2] = {mul2(p[q][0], make_float2(hz[0][g].x, hz[0][g].x)), mul2(p[q][1], make_float2(hz[1][g].x, hz[1][g].x))};
              weight_parts(ph, pb[q]);
            }
            // channels 2 c (odd = 0) and 2 c + 1 of rows 2 i, 2 i + 1 and of rows 2 i + 8, 2 i + 9
            uint32_t lo[2][4], hi[2][4];
#pragma unroll
            for (int odd = 0; odd < 2; ++odd) {
              const uint32_t sel = odd ? 0x7632 : 0x5410, swap = odd ? 0x6723 : 0x4501;
              q4_operands(ones, prmt(w[0][g], w[1][g], sel), prmt(w[0][g], w[1][g], swap), lo[odd]);
              q4_operands(ones, prmt(w[2][g], w[3][g], sel), prmt(w[2][g], w[3][g], swap), hi[odd]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int q = 0; q < QT; ++q) {
                float t[4] = {};   // fp32: these rows' sum, from the smallest part, then added with rounding
                float* acc = S::kWide ? t : o[q][4 * g + c];
#pragma unroll
                for (int part = kParts - 1; part >= 0; --part)
                  mma16816(acc, lo[0][c], lo[1][c], hi[0][c], hi[1][c], pb[q][part][0], pb[q][part][1]);
                if constexpr (S::kWide) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[q][4 * g + c][e] += t[e];
                }
              }
          }
        } else if constexpr (S::kWide) {
          uint32_t pb[S::kParts][2];
          weight_parts(p[0], pb);
#pragma unroll
          for (int c4 = 0; c4 < kPairs / 2; ++c4) {   // channels 4 of 32 c4 + 4 j on
            float f[4][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 x = *reinterpret_cast<const float4*>(vt + piece_at<S::kRow>(16 * sub + 4 * e + i, 8 * c4 + j));
              f[e][0] = x.x; f[e][1] = x.y; f[e][2] = x.z; f[e][3] = x.w;
            }
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
              float2 v0 = make_float2(f[0][c], f[1][c]), v2 = make_float2(f[2][c], f[3][c]);
              float2 v1 = make_float2(f[0][c + 1], f[1][c + 1]), v3 = make_float2(f[2][c + 1], f[3][c + 1]);
              uint32_t va[3][4];
#pragma unroll
              for (int vp = 0; vp < 3; ++vp) {
                va[vp][0] = split2(v0);
                va[vp][1] = split2(v1);
                va[vp][2] = split2(v2);
                va[vp][3] = split2(v3);
              }
              float t[4] = {};   // these rows' sum, from the smallest products, then added with rounding
#pragma unroll
              for (int order = 2; order >= 0; --order)
#pragma unroll
                for (int vp = 0; vp <= order; ++vp)
                  mma16816(t, va[vp][0], va[vp][1], va[vp][2], va[vp][3], pb[order - vp][0], pb[order - vp][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[0][2 * c4 + c / 2][e] += t[e];
            }
          }
        } else {
          uint32_t pb[QT][S::kParts][2];
#pragma unroll
          for (int q = 0; q < QT; ++q) weight_parts(p[q], pb[q]);
#pragma unroll
          for (int t = 0; t < kPairs; ++t) {
            // transposed matrices: the first and the second eight channels by rows 0 .. 7, then by rows 8 .. 15
            uint32_t x[4];
            load_matrices<true>(vt + piece_at<S::kRow>(16 * sub + lane % 8 + 8 * (lane / 16), 2 * t + (lane / 8) % 2), x);
#pragma unroll
            for (int q = 0; q < QT; ++q)
#pragma unroll
              for (int part = 0; part < kParts; ++part)
                mma16816(o[q][t], x[0], x[1], x[2], x[3], pb[q][part][0], pb[q][part][1]);
          }
        }
      }
    }

    // ---- the warps meet: each leaves its part, the last to arrive merges them, and the others go on with the
    // next head (at whose end they wait, in case, until this one is merged)
#pragma unroll
    for (int q = 0; q < QT; ++q)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[q][e] += __shfl_xor_sync(0xffffffffu, l[q][e], off);
          if constexpr (Q4) {
#pragma unroll
            for (int g = 0; g < kNg; ++g) oz[q][g][e] += __shfl_xor_sync(0xffffffffu, oz[q][g][e], off);
          }
        }
    if constexpr (FOUR) {   // columns 4 .. 7 onto columns 0 .. 3
#pragma unroll
      for (int t = 0; t < kPairs; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[0][t][e] += __shfl_xor_sync(0xffffffffu, o[0][t][e], 2);
    }
    if (!wait_for(&merged, segment) && lane == 0) report(a.dev_status, SNAPKV_ERR_TIMEOUT);
#pragma unroll
    for (int q = 0; q < QT; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int qq = 8 * q + qa + e;
        if (qq < tile_q && !(FOUR && i >= 2)) {
          if (j == 0) {
            warp_m[warp][qq] = m[q][e];
            warp_l[warp][qq] = l[q][e];
          }
          float* to = meet + (warp * a.tile_q + qq) * D;
#pragma unroll
          for (int t = 0; t < kPairs; ++t) {
            float x = o[q][t][e], y = o[q][t][e + 2];
            int c;   // the pair's first channel
            if constexpr (Q4) {
              const int g = t / 4, pair = t % 4;
              c = 64 * g + 8 * j + 2 * pair;
              x = fmaf(x, pair & 1 ? kQ4OutOdd : kQ4OutEven, oz[q][g][e]);
              y = fmaf(y, pair & 1 ? kQ4OutOdd : kQ4OutEven, oz[q][g][e]);
            } else {
              c = S::kWide ? 32 * (t / 2) + 4 * j + 2 * (t % 2) : 16 * t + j;
            }
            to[c] = x;
            to[c + (Q4 || S::kWide ? 1 : 8)] = y;
          }
        }
      }
    const bool last = arrive(&arrived) == S::kWarps - 1;
    if (last) {
      const bool whole = here.tile == 0 && seg_end == at + here.tiles;   // the head lies in this share
      float* part = a.parts + ((int64_t)blockIdx.x * 2 + (at > share0 ? 1 : 0)) * a.tile_q * (D + 2);
      for (int qq = 0; qq < tile_q; ++qq) {
        float top = -INFINITY, sum = 0.f, f[S::kWarps];
#pragma unroll
        for (int w = 0; w < S::kWarps; ++w) top = fmaxf(top, warp_m[w][qq]);
#pragma unroll
        for (int w = 0; w < S::kWarps; ++w) {
          f[w] = warp_m[w][qq] == -INFINITY ? 0.f : ex2(warp_m[w][qq] - top);
          sum = fmaf(warp_l[w][qq], f[w], sum);
        }
        const float scale = sum == 0.f ? 0.f : 1.0f / sum;   // a NaN stays one
#pragma unroll
        for (int c = lane; c < D; c += 32) {
          float x = 0.f;
#pragma unroll
          for (int w = 0; w < S::kWarps; ++w) x = fmaf(meet[(w * a.tile_q + qq) * D + c], f[w], x);
          if (whole)
            store1<IO>(static_cast<IO*>(a.out) + (q0 + qq) * D + c, x * scale);
          else
            part[qq * D + c] = x;
        }
        if (lane == 0) {
          if (!whole) {
            part[a.tile_q * D + qq] = top;
            part[a.tile_q * (D + 1) + qq] = sum;
          } else if (a.direct) {
            head_m[qq] = top == -INFINITY ? 0.f : top;
            head_r[qq] = scale;
          } else if (a.score) {
            a.stats[vh * 2 * a.tile_q + qq] = top;
            a.stats[(vh * 2 + 1) * a.tile_q + qq] = sum;
          }
        }
      }
      __syncwarp();
      if (lane == 0) {
        arrived = 0;
        publish(&merged, segment + 1);
      }
    }
    if (a.direct && a.score) {   // (one pass: the launcher saw to it)
      __syncthreads();
      float* sc = a.score + bh * a.cap;
      for (int r = tid; r < n; r += S::kThreads) {
        float w = 0.f;
        for (int qq = 0; qq < tile_q; ++qq) w = fmaf(ex2(logits[qq * a.logit_stride + r] - head_m[qq]), head_r[qq], w);
        sc[r] = a.decay != 0.f ? fmaf(a.decay, sc[r], w) : w;
      }
    }
    // the next head
    here.tile += (int)(seg_end - at);
    at = seg_end;
    if (at < end) settle(here);
  }
  cp_wait<0>();
}

// The second launch. The warps of its first blocks each join 64 channels of an output row whose head was
// cut (or is empty); the other blocks each add the weights of PER rows a thread to a head's scores, or of every
// `chunks`-th such run of its rows. Where a head's parts lie follows from the schedule. The kernel is all
// latency: loads are issued together and early, and registers are kept to what lets four blocks share an SM.
constexpr int kJoinThreads = 256;

// A head's parts: the last segment of one CTA (its slot 1, unless the share starts with the head) and the
// first of `more` others after it.
struct Parts {
  const float* first;
  const float* rest;
  int64_t stride;   // from one of the rest to the next
  int more;
  bool inside = true;   // of the parts that there are (checked build)
  __device__ __forceinline__ const float* operator[](int i) const { return i ? rest + (i - 1) * stride : first; }
};

template <int D> __device__ __forceinline__ Parts find_parts(const AttendArgs& a, int64_t total, int64_t f0, int tiles) {
  const int ctas = working_ctas(total, a.ctas);
  const int64_t size = (int64_t)a.tile_q * (D + 2);
  const int c0 = share_of(total, ctas, f0);
  Parts p;
  p.more = share_of(total, ctas, f0 + tiles - 1) - c0;
  p.inside = in_bounds(f0 >= 0 && f0 + tiles <= total && c0 >= 0 && p.more >= 0 && c0 + p.more < a.ctas, a.dev_status);
  p.first = a.parts + ((int64_t)c0 * 2 + (share_start(total, ctas, c0) < f0 ? 1 : 0)) * size;
  p.rest = a.parts + ((int64_t)c0 + 1) * 2 * size;
  p.stride = 2 * size;
  return p;
}

// What sums that belong to maximum m are multiplied by under the maximum `top` (of at least m). Sums under -inf are
// zero, or NaN where a logit is (maxima pass NaN over): multiplied, not left out, they keep it.
__device__ __forceinline__ float rescale(float m, float top) { return m == -INFINITY ? 0.f : ex2(m - top); }

// Adds a part's maximum and sum to a running pair.
__device__ __forceinline__ void join(float& top, float& sum, float m, float l) {
  const float next = fmaxf(top, m);
  sum = fmaf(l, rescale(m, next), sum * rescale(top, next));
  top = next;
}

template <typename IO, int D, int TILE, int PER>
__global__ void __launch_bounds__(kJoinThreads, 4) attend_join_kernel(AttendArgs a, int out_blocks, int chunks) {
  constexpr int kRows = PER * kJoinThreads;
  __shared__ float head_m[kMaxQueryTile], head_r[kMaxQueryTile];
  const int tid = threadIdx.x, lane = tid % 32;
  const int per_seq = a.heads * a.passes;
  const bool scores = (int)blockIdx.x >= out_blocks;
  // This block's head, or this warp's output row and 64 of its channels.
  constexpr int kSlices = D / 64;
  const int64_t slice = (int64_t)blockIdx.x * (kJoinThreads / 32) + tid / 32;
  const int block = (int)blockIdx.x - out_blocks;
  const int64_t out_row = slice / kSlices;
  if (!scores && out_row >= (int64_t)a.batch * a.heads * a.group) return;
  const int bh = scores ? block / chunks : (int)(out_row / a.group);
  const int b = bh / a.heads, h = bh - b * a.heads;
  const int n = visible_rows(a, b), tiles = tiles_of<TILE>(a, b);
  const int r0 = scores ? (block - bh * chunks) * kRows : 0;
  if (scores && r0 >= n) return;
  int64_t total, f0;   // tiles in all, and before this head's first pass
  Parts parts = {};   // of the first pass, or of the output row's
  auto find = [&](int64_t upto) {
    f0 = upto * per_seq + (int64_t)h * a.passes * tiles;
    const int pass = scores ? 0 : (int)(out_row - (int64_t)bh * a.group) / a.tile_q;
    if (tiles > 0) parts = find_parts<D>(a, total, f0 + (int64_t)pass * tiles, tiles);
  };
  if (a.batch <= kWarpBatch) {
    const SeqScan scan = scan_by_warp<TILE>(a);
    total = scan.total * per_seq;
    find(__shfl_sync(0xffffffffu, scan.upto, b));
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (a.batch > kWarpBatch) {
    total = __ldcg(a.upto + a.batch) * per_seq;
    find(__ldcg(a.upto + b));
  }

  if (!scores) {
    const int g = (int)(out_row - (int64_t)bh * a.group), pass = g / a.tile_q, q = g - pass * a.tile_q;
    const int c = (int)(slice % kSlices) * 64 + 2 * lane;
    float x = 0.f, y = 0.f, sum = 0.f;
    if (tiles > 0) {
      if (parts.more == 0 || !parts.inside) return;   // finished in the first launch
      const int at_m = a.tile_q * D + q, at_l = a.tile_q * (D + 1) + q;
      float top = -INFINITY;
      for (int i0 = 0; i0 <= parts.more; i0 += 32) {   // a part per lane, and eight parts' channels at a time
        const bool in = i0 + lane <= parts.more;
        const int here = min(32, parts.more + 1 - i0);
        float2 v[8];
        auto load = [&](int i) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = i + e < here ? __ldcg(reinterpret_cast<const float2*>(parts[i0 + i + e] + q * D + c)) : make_float2(0.f, 0.f);
        };
        const float m = in ? __ldcg(parts[i0 + lane] + at_m) : -INFINITY, l = in ? __ldcg(parts[i0 + lane] + at_l) : 0.f;
        load(0);
        const float next = fmaxf(top, warp_max(m));
        const float f = rescale(m, next), old = rescale(top, next);
        top = next;
        x *= old;
        y *= old;
        sum = fmaf(sum, old, warp_sum(l * f));
#pragma unroll 1
        for (int i = 0; i < here; i += 8) {
          if (i > 0) load(i);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float w = __shfl_sync(0xffffffffu, f, (i + e) & 31);
            x = fmaf(v[e].x, w, x);
            y = fmaf(v[e].y, w, y);
          }
        }
      }
    }
    const float scale = sum == 0.f ? 0.f : 1.0f / sum;   // a NaN stays one
    IO* out = static_cast<IO*>(a.out) + out_row * D + c;
    store1<IO>(out, x * scale);
    store1<IO>(out + 1, y * scale);
    return;
  }

  constexpr int kAtOnce = 16 / PER;   // sixteen loads a thread
  for (int64_t row0 = r0; row0 < n; row0 += (int64_t)chunks * kRows) {
    const int row = (int)row0 + tid;   // + kJoinThreads, ...
    if (!in_bounds(bh < a.batch * a.heads && row0 >= 0 && n <= a.cap && n <= a.logit_stride, a.dev_status)) break;
    float* sc = a.score + (int64_t)bh * a.cap + row;
    float w[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) w[i] = a.decay != 0.f && row + i * kJoinThreads < n ? a.decay * sc[i * kJoinThreads] : 0.f;
    for (int pass = 0; pass < a.passes; ++pass) {
      const int tile_q = min(a.tile_q, a.group - pass * a.tile_q);
      const int64_t vh = (int64_t)bh * a.passes + pass;
      const float* logits = a.logits + vh * a.tile_q * a.logit_stride + row;
      auto load = [&](int q, float (&x)[PER]) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          x[i] = row + i * kJoinThreads < n ? __ldcg(logits + q * a.logit_stride + i * kJoinThreads) : -INFINITY;
      };
      float x[kAtOnce][PER];   // some queries' logits are under way while the maxima are found
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q)
        if (q < tile_q) load(q, x[q]);
      if (a.passes > 1 || row0 == r0) {
        if (a.passes > 1) parts = find_parts<D>(a, total, f0 + (int64_t)pass * tiles, tiles);
        if (!parts.inside) return;   // (the whole block)
        for (int q = tid / 32; q < tile_q; q += kJoinThreads / 32) {   // a warp per query
          float top = -INFINITY, sum = 0.f;
          if (parts.more == 0) {
            top = __ldcg(a.stats + vh * 2 * a.tile_q + q);
            sum = __ldcg(a.stats + (vh * 2 + 1) * a.tile_q + q);
          } else {
            for (int i = lane; i <= parts.more; i += 32) {
              const float* p = parts[i] + a.tile_q * D + q;
              join(top, sum, __ldcg(p), __ldcg(p + a.tile_q));
            }
            const float all = warp_max(top);
            sum = warp_sum(sum * rescale(top, all));
            top = all;
          }
          if (lane == 0) {
            head_m[q] = top == -INFINITY ? 0.f : top;
            head_r[q] = sum == 0.f ? 0.f : 1.0f / sum;
          }
        }
        __syncthreads();
      }
      for (int q0 = 0; q0 < tile_q; q0 += kAtOnce) {
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
          if (q0 + e < tile_q) {
            const float m = head_m[q0 + e], r = head_r[q0 + e];
#pragma unroll
            for (int i = 0; i < PER; ++i) w[i] = fmaf(ex2(x[e][i] - m), r, w[i]);
            if (q0 + e + kAtOnce < tile_q) load(q0 + e + kAtOnce, x[e]);
          }
      }
      if (a.passes > 1) __syncthreads();   // the maxima have been used
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (row + i * kJoinThreads < n) sc[i * kJoinThreads] = w[i];
  }
}

template <bool Q4, typename IO, int D, int QT, bool FOUR>
cudaError_t launch_typed(const AttendJob& job) {
  using S = Shape<Q4, IO, D, QT>;
  const AttendLayout L = attend_layout(job.batch, job.q_heads, job.heads, D, job.cap, job.score != nullptr, 8 * QT);
  char* ws = static_cast<char*>(job.workspace);
  AttendArgs a;
  a.q = job.q;
  a.k = static_cast<const uint8_t*>(job.k);
  a.v = static_cast<const uint8_t*>(job.v);
  a.km = static_cast<const uint8_t*>(job.k_meta);
  a.vm = static_cast<const uint8_t*>(job.v_meta);
  a.len = job.len;
  a.score = job.score;
  a.out = job.out;
  a.decay = job.decay;
  a.scale_log2 = (float)(1.4426950408889634 / sqrt((double)D));
  a.cap = job.cap;
  a.batch = job.batch;
  a.heads = job.heads;
  a.group = job.q_heads / job.heads;
  a.passes = L.passes;
  a.tile_q = L.tile_q;
  a.upto = reinterpret_cast<int64_t*>(ws + L.upto);
  a.parts = reinterpret_cast<float*>(ws + L.parts);   // (no workspace, and none of these, for a direct call)
  a.stats = reinterpret_cast<float*>(ws + L.stats);
  a.logits = reinterpret_cast<float*>(ws + L.logits);
  a.logit_stride = L.logit_stride;
  a.dev_status = job.dev_status;
  // One wave of CTAs, or fewer where their warps would have no tile each.
  a.direct = L.direct;
  const int smem = S::smem(L.tile_q, L.direct);
  cudaError_t err = allow_dynamic_smem<attend_kernel<Q4, IO, D, QT, FOUR>>(S::smem(8 * QT, true));
  if (err != cudaSuccess) return err;
  // CTAs per SM by device and tile_q (0: not asked yet), as the shares, and with them a result's bits, follow from it.
  constexpr int kMaxDev = 64;
  static std::atomic<int> occupancy[kMaxDev][8 * QT + 1];
  int resident = 1;
  if (!L.direct) {
    int dev = 0;
    err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    std::atomic<int>* known = dev < kMaxDev ? &occupancy[dev][L.tile_q] : nullptr;
    resident = known ? known->load(std::memory_order_relaxed) : 0;
    if (resident < 1) {
      err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, attend_kernel<Q4, IO, D, QT, FOUR>, S::kThreads, smem);
      if (err != cudaSuccess) return err;
      if (resident < 1) return cudaErrorInvalidConfiguration;
      if (known) known->store(resident, std::memory_order_relaxed);
    }
  }
  const int64_t heads = (int64_t)job.batch * job.heads * L.passes;
  const int64_t tiles = heads * ((job.cap + S::kTile - 1) / S::kTile);
  int64_t ctas = (int64_t)device_sm_count() * resident;
  if (ctas > (tiles + kWarps - 1) / kWarps) ctas = (tiles + kWarps - 1) / kWarps;
  if (ctas > L.max_ctas) ctas = L.max_ctas;
  if (a.direct) ctas = heads;
  a.ctas = (int)ctas;
  attend_kernel<Q4, IO, D, QT, FOUR><<<(unsigned)ctas, S::kThreads, smem, job.stream>>>(a);
  err = cudaGetLastError();
  if (err != cudaSuccess || a.direct) return err;
  const int64_t slices = (int64_t)job.batch * job.q_heads * (D / 64);
  const int64_t out_blocks = (slices + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  // Rows a thread: as few as let all blocks run at once (four per SM), so that the loads of more queries are
  // under way at a time. A second wave costs its blocks' set-up: 64 heads of 8192 4-bit rows, four queries,
  // take 29.1 us in one wave of four rows a thread, 30.6 with eight and 33.4 in two waves with two. (Several
  // passes have work enough for their blocks: 32 heads of 16384 bf16 rows, 64 queries, take 229, 236, 247 us
  // with two, four and eight.)
  const int64_t kv_heads = (int64_t)job.batch * job.heads;
  int per = 2;
  int64_t chunks = 0;
  if (job.score)
    for (;; per *= 2) {
      chunks = (job.cap + per * kJoinThreads - 1) / (per * kJoinThreads);
      if (per == 8 || L.passes > 1 || out_blocks + kv_heads * chunks <= 4 * (int64_t)device_sm_count()) break;
    }
  // No more than two waves of blocks, which then take turns: caches are often longer than what they hold (512 heads
  // of 1000 bf16 rows, 64 channels, in caches of 65536 rows: 37 us, 49 with a block for each run of rows).
  const int64_t turns = (kv_heads * chunks + 8 * (int64_t)device_sm_count() - 1) / (8 * (int64_t)device_sm_count());
  if (turns > 1) chunks = (chunks + turns - 1) / turns;
  const int64_t blocks = out_blocks + kv_heads * chunks;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = job.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto* join = per == 2 ? attend_join_kernel<IO, D, S::kTile, 2>
               : per == 4 ? attend_join_kernel<IO, D, S::kTile, 4> : attend_join_kernel<IO, D, S::kTile, 8>;
  return cudaLaunchKernelEx(&cfg, join, a, (int)out_blocks, (int)chunks);
}

template <bool Q4, int D> cudaError_t launch_dim(const AttendJob& job) {
  const int group = job.q_heads / job.heads;
  if (job.dtype == SNAPKV_F32) return launch_typed<Q4, float, D, 1, false>(job);
  // 8 sequences of 8192 bf16 rows and 4 KV heads with scores: 16 queries a head take 49 us in one pass of
  // sixteen, where two of eight take 56.
  if (group > 8) return launch_typed<Q4, __nv_bfloat16, D, 2, false>(job);
  return group <= 4 ? launch_typed<Q4, __nv_bfloat16, D, 1, true>(job) : launch_typed<Q4, __nv_bfloat16, D, 1, false>(job);
}

template <bool Q4> cudaError_t launch_format(const AttendJob& job) {
  return job.head_dim == 64 ? launch_dim<Q4, 64>(job) : launch_dim<Q4, 128>(job);
}

}  // namespace

AttendLayout attend_layout(int batch, int q_heads, int heads, int head_dim, int64_t cap, bool scored, int most_q) {
  AttendLayout L;
  const int group = q_heads / heads;
  L.passes = (group + most_q - 1) / most_q;
  L.tile_q = (group + L.passes - 1) / L.passes;   // passes of about equal size
  L.direct = cap <= kDirectRows && L.passes == 1;
  const size_t vh = (size_t)batch * heads * L.passes;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  // No more CTAs than there can be tiles for their warps (the smallest tile has 16 rows).
  const int64_t tiles = (int64_t)vh * ((cap + 15) / 16);
  L.max_ctas = (int)(tiles < kMaxAttendCtas ? tiles : kMaxAttendCtas);
  L.parts = 0;
  L.stats = L.parts + up((size_t)L.max_ctas * 2 * L.tile_q * (head_dim + 2) * sizeof(float));
  L.upto = L.stats + up(vh * 2 * L.tile_q * sizeof(float));
  L.logits = L.upto + up(batch > kWarpBatch ? ((size_t)batch + 1) * sizeof(int64_t) : 0);
  L.logit_stride = L.direct ? kDirectRows : (cap + 7) / 8 * 8;
  if (L.direct)   // shared memory holds everything
    L.total = 0;
  else
    L.total = L.logits + (scored ? up(vh * (size_t)L.logit_stride * L.tile_q * sizeof(float)) : 0);
  return L;
}

size_t attend_workspace_bytes(int batch, int q_heads, int heads, int head_dim, int64_t cap, bool scored, int dtype) {
  return attend_layout(batch, q_heads, heads, head_dim, cap, scored, dtype == SNAPKV_F32 ? 8 : kMaxQueryTile).total;
}

cudaError_t launch_attend(const AttendJob& job) {
  return job.k_meta ? launch_format<true>(job) : launch_format<false>(job);
}

}  // namespace snapkv
