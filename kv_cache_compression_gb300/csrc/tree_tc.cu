// Tree attention of many query rows a KV head, bf16, over a dense cache or one in 8 bits (tree_schedule.cuh has the
// schedule): wide trees, grouped queries, prompts that read an encoder's states.
//
//   S = Q K^T,  P = exp2(S - m),  O = sum P V,  running m and sum per row
//
// tcgen05 with 128 query rows by 128 keys: S (fp32) and O stand in TMEM, P goes back over S as the second product's A
// operand, K and V are B operands in shared memory. Two slots, each an S, an O and its softmax warps, keep the tensor
// cores busy while the other slot's weights are computed. In passes of 128 rows (TWO false) both slots serve the same
// rows and take the key tiles in turn, each from a ring of its own, and their halves of O meet at the head's end; in passes of
// 256 a slot has 128 rows each and every key tile serves both, so that the cache is read once. Passes go side by side where all
// sequences have as many. A slot issues P V of a tile and Q K^T of its next as one block (S is overwritten when
// P V has read P: the tensor core takes them one after the other), and passes the turn on.
//
// Weights enter the second product as one bf16 value, rounded by half a step (2^-8); they are summed up as they were. That is a
// choice: outputs are off by 0.0022 to 0.0024 of their norm so, and by 0.0017, their own rounding, with a second part for what the
// first leaves. With both P V takes twice as long: 4 x 8 KV heads of 256 rows over 32768 keys 119 us, 153 with two parts; up to 440
// tokens over 1500 keys of 256 heads of 64 channels 72 and 89; 64 x 32 heads of 20 rows over 2140 keys 376 and 438; 8 x 8 heads of
// 128 rows over 8 bits 101 and 114; where memory binds most, 64 rows over 16384 keys, 79 and 85. Calls in fp32, over 8 bits too, round
// no weight. A row's maximum is only raised, and its O rescaled, when it would grow by more than 2^8 (over 8 bits 2^6); sums and
// outputs stay under the same maximum, so that nothing is lost.
//
// Measured (128 channels): 4 x 8 KV heads of 256 rows over 32768 keys 119 us, 1100 TFLOP/s; 8 x 8 heads of 64 rows over 16384
// keys, half of the sequences shorter, 80 us, 5.0 TB/s. With up to 128 rows a KV head memory bounds it; with more, a slot's
// way from S to P (1100 clocks), to the other warps and back (300), and through both products (1100 with 64 channels, 1400 with 128,
// where the tensor cores need 512 and 1024), during which the other slot's is hidden but for its own products: 3400 clocks for
// 256 rows by 128 keys, 3100 with 64 channels.
//
// 8-bit rows arrive as they are; eight more warps unpack them into the tiles that TMA writes for bf16 rows (8 x 8 KV heads of
// 128 rows over 16384 keys, half of the sequences shorter: 101 us; four warps took 16 more, sixteen 13 more). As operands they
// are *subnormal* bf16 (sign and seven magnitude bits, u 2^-133: a byte permute and an AND per two values), for which queries
// are scaled by 2^64 and weights by 2^80; a step multiplies its key's logits and weights. The way of a tile through the
// unpacking warps bounds it (two waits, loads, stores and a fence, 1400 clocks for K and for V each of the 3500 that a tile takes).
#include "tree_schedule.cuh"

#include <type_traits>

#include "cache_internal.h"
#include "q4.cuh"
#include "sm100_ptx.cuh"
#include "snapkv_internal.h"
#include "tree_launch.h"
#include "tree_maps.h"

namespace snapkv {
namespace {

using namespace tree;

constexpr int kTile = 128;                       // keys; also a slot's query rows
constexpr long long kWaitLimit = 4000000000LL;   // about two seconds

// What is small in shared memory. (All of it is laid out here: with 192 KB of tiles 160 bytes are left.)
struct Bars {
  uint64_t kv_full[12], kv_empty[12], raw_full[8], raw_empty[8];
  uint64_t q_full, q_empty, s_full[2], p_ready[2];
  uint64_t o_full, o_free, drain[2], turn[2];   // (turn: the slot may issue its next products)
};
template <int THREADS> struct Small {
  Bars bars;
  uint32_t tmem;
  int abort;
  uint32_t bad_keys[2][4];
  uint8_t pending[12];   // of a stage's last load, if any: 1 + its phase's parity
  ShareScratch<THREADS> share;
};

template <bool Q8, int D, bool TWO> struct Shape {
  static constexpr int kRows = TWO ? 256 : 128;                // query rows of a pass
  // Softmax warps: two for 32 rows of a slot, half of the keys each. Beside an 8-bit cache one has time enough for all of
  // them, and eight more unpack.
  static constexpr int kHalves = Q8 ? 1 : 2;
  static constexpr int kSoft = 8 * kHalves;
  static constexpr int kUnpack = Q8 ? 8 : 0;
  static constexpr int kWarps = 4 + kSoft + kUnpack;
  static constexpr int kThreads = 32 * kWarps;
  // Registers go from the warps that move data to those of the softmax (both sum up to no more than the block is launched with):
  // 2 % less time for 4 x 8 KV heads of 256 rows over 32768 keys; beside an 8-bit cache they let 32 keys be computed on at a time,
  // 8 % less for 8 x 8 heads of 128 rows over 16384.
  static constexpr int kLaunchRegs = 96, kSoftRegs = Q8 ? 120 : 104, kMoveRegs = Q8 ? 80 : 64;
  static_assert(32 * kSoft * kSoftRegs + (kThreads - 32 * kSoft) * kMoveRegs <= kThreads * kLaunchRegs, "registers");
  // log2 of what weights may exceed 1 by. Over 8 bits a weight is multiplied by its key's step, up to 2^48 / 127 < 2^41.02, and by
  // kQ8P = 2^80: with 2^6 that stays below 2^127.02, with 2^8 it would be infinite for values of V above 2^47.
  static constexpr float kSlack = Q8 ? 6.0f : 8.0f;
  static constexpr int kSlotQ = kTile * D * 2;                 // bytes of 128 rows of queries
  static constexpr int kStage = kTile * D * 2;                 // of a tile of K or V
  static constexpr int kStages = (Q8 ? (TWO ? 3 : 4) : TWO ? 4 : 6) * (128 / D);   // (TWO: of one ring; else of two, a slot's each)
  static constexpr int kTurn = TWO ? kStages : kStages / 2;
  static constexpr int kRaw = kTile * D;                       // of a tile of codes
  static constexpr int kRaws = Q8 ? 3 * (128 / D) : 0;
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + (TWO ? 2 : 1) * kSlotQ;
  static constexpr int kRawRing = kRing + kStages * kStage;
  static constexpr int kSwap = kRawRing + kRaws * kRaw;        // [2 slots][2 halves][128] floats
  static constexpr int kFactors = kSwap + 4 * kTile * 4;       // [2 slots][2][K, V][128] floats (8 bits)
  static constexpr int kSmall = kFactors + (Q8 ? 2 * 2 * 2 * kTile * 4 : 0);
  static constexpr int smem() { return kSmall + (int)sizeof(Small<kThreads>); }
  // The stage of a ring's tile `at`: of a slot's tile i, K is 2 i and V 2 i + 1.
  __device__ __forceinline__ static uint32_t stage(int slot, uint32_t at) { return (TWO ? 0 : slot * kTurn) + at % kTurn; }
  static constexpr int kS(int slot) { return slot * 128; }     // TMEM columns
  static constexpr int kO(int slot) { return 256 + slot * D; }
  static constexpr int kColumns = 512;
};

__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
      "%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at), "r"(r[0]), "r"(r[1]),
      "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
      "r"(r[14]), "r"(r[15])
      : "memory");
}
// Whether x is true in any thread of the two warps that meet at a named barrier.
__device__ __forceinline__ bool any_of_pair(int barrier, bool x) {
  uint32_t any;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(any) : "r"((uint32_t)x), "r"(barrier) : "memory");
  return any != 0;
}

// The MMA warp runs as a whole, so that descriptors stay in uniform registers (computed by one thread, each product took 90
// clocks to issue, of which it executes in 64); its first thread alone issues. A value of which the compiler cannot see that it
// is the same in all threads goes through a reduction, whose result is.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }

// D (+)= A B^T, bf16 operands, fp32 sums; A in shared memory (ss) or TMEM (ts). lo: the low words of descriptors.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 e, %0, 0;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 x, {%2, %4};\n\tmov.b64 y, {%3, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%1], x, y, %5, p;\n\t}" ::"r"(leader),
      "r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 y;\n\tsetp.ne.b32 e, %0, 0;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 y, {%3, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], y, %5, p;\n\t}" ::"r"(leader),
      "r"(d), "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %0, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(leader), "r"(ptx::smem_u32(bar))
      : "memory");
}

// Descriptors, low and high words. Queries and K: rows of 128 bytes (64 channels, the products' k), 128-byte swizzle, eight rows
// 1024 bytes apart. V as B: keys (the product's k) are rows of 128 bytes of 64 channels (its n), eight keys 1024 bytes
// apart, 64 channels a block of kTile rows.
__device__ __forceinline__ constexpr uint32_t k_desc(uint32_t at) { return ((at >> 4) & 0x3FFFu) | 1u << 16; }
__device__ __forceinline__ constexpr uint32_t v_desc(uint32_t at) { return ((at >> 4) & 0x3FFFu) | (uint32_t)((kTile * 128) >> 4) << 16; }
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;   // stride, version, swizzle

// A piece (eight channels) of a row of a tile in shared memory.
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
  return (piece / 8) * (kTile * 128) + row * 128 + (((piece % 8) ^ (row & 7)) << 4);
}

// The segments of a share: runs of tiles of one head (and pass). Every role walks them for itself.
struct Segments {
  Place p;
  int64_t at, end;
  int tiles;       // of this segment
  int index;
  __device__ __forceinline__ Segments(const Args& a, const Share& s) : p(s.first), at(s.at), end(s.end), index(0) { cut(); }
  __device__ __forceinline__ void cut() {
    const int64_t left = end - at;
    const int more = p.s.tiles - p.tile;
    tiles = left < more ? (int)left : more;
  }
  __device__ __forceinline__ bool next(const Args& a) {
    at += tiles;
    if (at >= end) return false;
    next_head<kTile, kTile>(a, p);
    ++index;
    cut();
    return true;
  }
  __device__ __forceinline__ bool whole() const { return tiles == p.s.tiles; }
};

template <bool Q8, int D, bool TWO>
__global__ void __launch_bounds__(Shape<Q8, D, TWO>::kThreads, 1) tree_tc_kernel(const Args a, const __grid_constant__ TreeMaps maps) {
  using S = Shape<Q8, D, TWO>;
  constexpr int kStages = S::kStages, kRaws = S::kRaws > 0 ? S::kRaws : 1;
  static_assert(kStages <= 12 && kRaws <= 8, "barriers");
  extern __shared__ __align__(1024) uint8_t smem[];   // (swizzled tiles: 1024 bytes)
  Small<S::kThreads>& small = *reinterpret_cast<Small<S::kThreads>*>(smem + S::kSmall);
  Bars& bars = small.bars;
  int& abort = small.abort;
  if ((ptx::smem_u32(smem) & 1023) != 0) {
    report(a.dev_status, SNAPKV_ERR_INTERNAL);
    return;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid % 32, warp = __shfl_sync(0xffffffffu, tid / 32, 0);
  if (tid == 0) {
    abort = 0;
    for (int i = 0; i < 12; ++i) small.pending[i] = 0;
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&bars.kv_full[i], Q8 ? S::kUnpack : 1);
      ptx::mbar_init(&bars.kv_empty[i], TWO ? 2 : 1);   // (slots)
    }
    if constexpr (Q8) {
      for (int i = 0; i < kRaws; ++i) {
        ptx::mbar_init(&bars.raw_full[i], 1);
        ptx::mbar_init(&bars.raw_empty[i], S::kUnpack);
      }
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars.s_full[i], 1);
      ptx::mbar_init(&bars.p_ready[i], S::kSoft / 2);
    }
    ptx::mbar_init(&bars.q_full, 1);
    ptx::mbar_init(&bars.q_empty, 2);
    ptx::mbar_init(&bars.o_full, 2);
    ptx::mbar_init(&bars.o_free, S::kSoft);
    ptx::mbar_init(&bars.drain[0], 1);
    ptx::mbar_init(&bars.drain[1], 1);
    ptx::mbar_init(&bars.turn[0], 1);
    ptx::mbar_init(&bars.turn[1], 1);
    ptx::fence_mbar_init();
  }
  {
    const Share mine = find_share<kTile, kTile, S::kThreads>(a, small.share);   // (with barriers)
    if (tid == 64) {
      leave_note(a, mine);
      small.share.found = mine;
    }
    if (mine.at >= mine.end) return;
  }
  if (warp == 1) {
    ptx::tmem_alloc(&small.tmem, S::kColumns);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = small.tmem;
  const Share& share = small.share.found;
  const uint32_t ring = ptx::smem_u32(smem + S::kRing), q_smem = ptx::smem_u32(smem + S::kQ);
  const int pass0 = a.siblings > 1 ? (int)blockIdx.x % a.siblings : 0;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ptx::mbar_wait(bar, parity & 1, &abort, kWaitLimit)) return true;
    *reinterpret_cast<volatile int*>(&abort) = 1;
    report(a.dev_status, SNAPKV_ERR_TIMEOUT);
    return false;
  };
  auto aborted = [&] { return *reinterpret_cast<volatile int*>(&abort) != 0; };
  // The query rows r0 .. r0 + rows - 1 of a segment.
  auto r0_of = [&](const Segments& s) { return (a.siblings > 1 ? pass0 : s.p.pass) * a.tile_q; };
  auto rows_of = [&](const Segments& s) { return min(a.tile_q, a.group * s.p.s.n - r0_of(s)); };
  const uint32_t total = (uint32_t)(share.end - share.at);   // tiles
  constexpr uint32_t kPair = TWO ? 1 : 2;                    // they are loaded, K before V

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kMoveRegs));
    if (warp == 0) {
      // ---- loads, in the order in which the products take them
      if (lane == 0) {
        Segments ks(a, share), vs(a, share);
        int kf = 0, vf = 0;   // tiles of the segments so far
        uint32_t sent = 0;    // raw ones (8 bits)
        auto send = [&](Segments& s, int& f, uint32_t t, bool key) {   // K or V of the share's tile t
          const int tile = s.p.tile + f, bh = s.p.seq * a.heads + s.p.head;
          const bool cached = tile < s.p.s.cache_tiles;
          if (!Q8 || cached) {   // (drafted rows beside an 8-bit cache are copied by the warps that unpack)
            const uint32_t at = 2 * (TWO ? t : t / 2) + (key ? 0 : 1);
            const uint32_t slot = Q8 ? sent % kRaws : S::stage(t & 1, at), turn = Q8 ? sent / kRaws : at / S::kTurn;
            if (turn > 0 && !wait(Q8 ? &bars.raw_empty[slot] : &bars.kv_empty[slot], turn - 1)) return false;
            uint64_t* const bar = Q8 ? &bars.raw_full[slot] : &bars.kv_full[slot];
            uint8_t* const to = smem + (Q8 ? S::kRawRing + slot * S::kRaw : S::kRing + slot * S::kStage);
            const CUtensorMap* const map = cached ? (key ? &maps.k : &maps.v) : (key ? &maps.k_new : &maps.v_new);
            const int row0 = (cached ? tile : tile - s.p.s.cache_tiles) * kTile;
            ptx::mbar_arrive_expect_tx(bar, Q8 ? S::kRaw : S::kStage);
#pragma unroll
            for (int c = 0; c < (Q8 ? 1 : D / 64); ++c) ptx::tma_load_3d(to + c * kTile * 128, map, 64 * c, row0, bh, bar);
            small.pending[slot] = (uint8_t)(1 + (turn & 1));
            ++sent;
          }
          if (++f == s.tiles) {
            f = 0;
            s.next(a);
          }
          return true;
        };
        bool ok = true;
        for (uint32_t t = 0; ok && t < total; t += kPair)
          for (int key = 1; ok && key >= 0; --key)
            for (uint32_t u = t; ok && u < t + kPair && u < total; ++u) ok = key ? send(ks, kf, u, true) : send(vs, vf, u, false);
        // Copies in flight land before the block ends, also after a wait ran out.
        const int none = 0;
        for (int i = 0; i < (Q8 ? kRaws : kStages); ++i)
          if (small.pending[i]) ptx::mbar_wait(Q8 ? &bars.raw_full[i] : &bars.kv_full[i], small.pending[i] - 1, &none, kWaitLimit);
      }
    } else if (warp < 3) {
      // ---- products of a slot. (One warp for both slots left the tensor core idle for 2000 of a tile's 5200 clocks, while it
      // waited on barriers that had long been reached and counted: a product is issued no more than a few ahead.)
      const int slot = warp - 1;
      constexpr uint32_t kIdescQk = ptx::idesc_bf16_f32(128, kTile), kIdescPv = ptx::idesc_bf16_f32(128, D) | 1u << 16;   // (V: n-major)
      const uint32_t leader = lane == 0;
      const uint32_t s_at = uniform(tmem + S::kS(slot)), o_at = uniform(tmem + S::kO(slot));
      auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };   // (the warp stays together)
      // The slots issue in turn: P V of a tile and Q K^T of the slot's next as a block, all that they wait for before. (Left to
      // themselves both slots' products mix, and then both softmaxes run, and both products wait, at the same time; and a wait
      // between products, even for a barrier long reached, leaves the tensor core idle.)
      uint32_t steps = 0, turns = 0;   // P V of this slot, and turns, so far
      auto my_turn = [&] {
        const bool mine = slot == 0 && turns == 0 ? true : wait_all(&bars.turn[slot], slot == 0 ? turns - 1 : turns);
        ++turns;
        ptx::tc_fence_after();
        return mine;
      };
      auto pass_on = [&] {
        if (leader) ptx::mbar_arrive(&bars.turn[1 - slot]);
        __syncwarp();
      };
      auto full = [&](uint32_t at) { return wait_all(&bars.kv_full[S::stage(slot, at)], at / S::kTurn); };
      // S = Q K^T of the ring's tile `at`.
      const uint32_t q_lo = uniform(k_desc(q_smem + (TWO ? slot : 0) * S::kSlotQ));
      auto qk = [&](uint32_t at) {
        const uint32_t k_lo = uniform(k_desc(ring + S::stage(slot, at) * S::kStage));
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t off = ((s / 4) * (kTile * 128) + (s % 4) * 32) >> 4;
          mma_ss(leader, s_at, q_lo + off, k_lo + off, kDescHigh, kIdescQk, s > 0);
        }
      };
      // O += P V of the ring's tile `at`; `fresh`: O =.
      auto pv = [&](uint32_t at, bool fresh) {
        const uint32_t v_lo = uniform(v_desc(ring + S::stage(slot, at) * S::kStage));
        constexpr int kHalf = kTile / S::kHalves / 16;   // (weights begin where their half's logits did)
#pragma unroll
        for (int s = 0; s < kTile / 16; ++s)
          mma_ts(leader, o_at, s_at + s / kHalf * (kTile / S::kHalves) + s % kHalf * 8, v_lo + s * (2048 >> 4), kDescHigh, kIdescPv, !(fresh && s == 0));
      };
      // Walks of the Q K^T and of the P V, the first a tile of the slot's ahead. A slot waits for every segment's queries and outputs
      // and counts in on q_empty and o_full at its end, whether it had tiles of it or not: barriers know a phase by its parity
      // alone, so that none may be passed over. Up to 128 rows the slot's tiles are every second of the share; of more, all tiles,
      // but of segments in whose rows it has no part it only lets the loads go on.
      constexpr int kBy = TWO ? 1 : 2;
      Segments qs(a, share), ps(a, share);
      int qf = TWO ? 0 : slot, pf = qf;        // within the segments
      uint32_t q_t = 0, p_t = 0;               // the slot's tiles so far
      bool q_end = false, p_end = false, ok = true;
      auto takes_part = [&](const Segments& s) { return !TWO || slot == 0 || rows_of(s) > kTile; };
      bool q_mine = takes_part(qs), p_mine = q_mine;
      auto queries = [&] { return wait_all(&bars.q_full, qs.index); };
      auto outputs = [&] { return ps.index == 0 || wait_all(&bars.o_free, ps.index - 1); };
      auto q_next = [&] {
        qf -= qs.tiles;
        commit(leader, &bars.q_empty);
        q_end = !qs.next(a);
        if (!q_end) q_mine = takes_part(qs);
      };
      auto p_next = [&] {
        pf -= ps.tiles;
        commit(leader, &bars.o_full);
        p_end = !ps.next(a);
        if (!p_end) p_mine = takes_part(ps);
      };
      for (bool begin = true; ok; begin = false) {
        // what this turn's products need
        if (!begin) {
          while (ok && !p_end && pf >= ps.tiles) {   // a segment without tiles of the slot's
            ok = outputs();
            if (ok) p_next();
          }
          if (!ok || p_end) break;
          ok = (pf >= kBy || outputs()) && full(2 * p_t + 1);   // (a segment's first tiles are its slots' first)
          if (ok && p_mine) ok = wait_all(&bars.p_ready[slot], steps);
        }
        while (ok && !q_end && qf >= qs.tiles) {
          ok = queries();
          if (ok) q_next();
        }
        const bool more = !q_end;
        if (ok && more) ok = (qf >= kBy || queries()) && full(2 * q_t);
        if (!ok || !my_turn()) break;
        if (!begin && p_mine) pv(2 * p_t + 1, pf < kBy);
        if (more && q_mine) qk(2 * q_t);
        pass_on();
        // what waits for them
        if (more && q_mine) commit(leader, &bars.s_full[slot]);
        if (!begin) {
          commit(leader, &bars.kv_empty[S::stage(slot, 2 * p_t + 1)]);
          if (p_mine) ++steps;
          ++p_t;
          pf += kBy;
          if (pf >= ps.tiles) p_next();
        }
        if (more) {
          commit(leader, &bars.kv_empty[S::stage(slot, 2 * q_t)]);
          ++q_t;
          qf += kBy;
          if (qf >= qs.tiles) q_next();
        }
      }
      // Products in flight end before the block does.
      commit(leader, &bars.drain[slot]);
      const int none = 0;
      ptx::mbar_wait(&bars.drain[slot], 0, &none, kWaitLimit);
    } else {
      // ---- queries into shared memory
      const int at = lane;
      Segments seg(a, share);
      do {
        if (seg.index > 0) wait(&bars.q_empty, seg.index - 1);
        const int r0 = r0_of(seg), rows = rows_of(seg), n = seg.p.s.n;
        const int64_t bh = (int64_t)seg.p.seq * a.heads + seg.p.head;
        const int slots = TWO && rows > 128 ? 2 : 1;
        if (!Q8 && (a.group == 1 || n == a.tokens)) {   // the rows follow one another: whole tiles, whatever lies behind the head's
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(&bars.q_full, slots * S::kSlotQ);
            const int row0 = (int)(bh * a.group * a.tokens) + r0;
            for (int x = 0; x < slots; ++x)
              for (int c = 0; c < D / 64; ++c) ptx::tma_load_3d(smem + S::kQ + x * S::kSlotQ + c * kTile * 128, &maps.q, 64 * c, row0 + x * kTile, 0, &bars.q_full);
          }
          continue;
        }
        // A thread has every (32 / kPieces)-th row's piece c, all of them under way at a time. Rows follow one another in memory but for
        // the tokens that a sequence does not have. (A warp alone: what it computes for a piece is what the load takes.)
        constexpr int kPieces = D / 8, kStep = 32 / kPieces;
        const int c = at % kPieces, first = at / kPieces;
        int t = (r0 + first) % n;
        const int64_t gap = (int64_t)(a.tokens - n) * D;
        const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(a.q) + (bh * a.group + (r0 + first) / n) * a.tokens * D + (int64_t)t * D + 8 * c;
        uint32_t place[8 / kStep];   // of rows first + e kStep, and of those 8, 16, ... further on but for a multiple of 1024
#pragma unroll
        for (int e = 0; e < 8 / kStep; ++e) place[e] = q_smem + piece_at(first + e * kStep, c);
#pragma unroll 1
        for (int x = 0; x < slots * kTile; x += 8) {
          const uint32_t base = (x / kTile) * S::kSlotQ + (x % kTile) * 128;
#pragma unroll
          for (int e = 0; e < 8 / kStep; ++e) {
            const bool there = x + first + e * kStep < rows;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(place[e] + base), "l"(there ? from : static_cast<const __nv_bfloat16*>(a.q)), "r"(there ? 16 : 0) : "memory");
            from += kStep * D;
            for (t += kStep; t >= n; t -= n) from += gap;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if constexpr (Q8) {
#pragma unroll 4
          for (int r = first; r < min(rows, slots * kTile); r += kStep) {
            uint4* const u = reinterpret_cast<uint4*>(smem + S::kQ + (r / kTile) * S::kSlotQ + piece_at(r % kTile, c));
            uint4 v = *u;
            uint32_t* const w = &v.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack2(__uint_as_float(w[i] << 16) * kQ8Q, __uint_as_float(w[i] & 0xFFFF0000u) * kQ8Q);
            *u = v;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars.q_full);
      } while (seg.next(a) && !__any_sync(0xffffffffu, aborted()));
      if (lane == 0) {   // (a copy in flight lands before the block ends)
        const int none = 0;
        ptx::mbar_wait(&bars.q_full, seg.index & 1, &none, kWaitLimit);
      }
    }
  } else if (warp < 4 + S::kSoft) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kSoftRegs));
    // ---- softmax: kHalves threads per row of a slot, a share of the keys each
    constexpr int kHalves = S::kHalves, kKeys = kTile / kHalves, kWords = kKeys / 32;
    constexpr int kChunk = Q8 ? 32 : 16, kChunks = kKeys / kChunk, kE = kChunk / 2;   // keys that are computed on at a time, and their pairs
    const int slot = (warp - 4) / (4 * kHalves), half = (warp - 4) / 4 % kHalves, quarter = warp % 4, row = quarter * 32 + lane;
    const uint32_t o_lane = tmem + ((uint32_t)(quarter * 32) << 16), s_at = o_lane + S::kS(slot);
    float* const swap = reinterpret_cast<float*>(smem + S::kSwap) + slot * 2 * kTile;   // [half][row]
    float* const factors = reinterpret_cast<float*>(smem + S::kFactors) + slot * 4 * kTile;
    const int pair = 4 + slot * 4 + quarter;   // the named barrier of the warps that share rows
    constexpr int kSlotThreads = 32 * S::kSoft / 2;
    uint32_t steps = 0;                // of this slot
    uint32_t done = 0;                 // tiles of the share in the segments so far
    Segments seg(a, share);
    do {
      const int r0 = r0_of(seg) + (TWO ? slot * kTile : 0), n = seg.p.s.n;
      const int rows = min(kTile, rows_of(seg) - (TWO ? slot * kTile : 0));   // this slot's (none or less: it rests)
      const bool mine = quarter * 32 < rows;                                  // this warp has rows
      float m = kNoMax, l = 0.f;       // l: of this thread's keys
      bool first = true;
      for (int f = TWO ? 0 : (int)((done ^ slot) & 1); rows > 0 && f < seg.tiles; f += TWO ? 1 : 2) {
        const int tile = seg.p.tile + f;
        const bool drafted = tile >= seg.p.s.cache_tiles;
        const int key0 = (drafted ? tile - seg.p.s.cache_tiles : tile) * kTile;
        const int valid = min(kTile, (drafted ? n : seg.p.s.rows) - key0);
        const bool edge = drafted || valid < kTile;
        // This row's bits of the thread's keys: those that it sees, and (below) those that make it NaN.
        uint32_t see[kWords], bad[kWords];
#pragma unroll
        for (int w = 0; w < kWords; ++w) see[w] = ~0u, bad[w] = 0u;
        if (edge) {
          const int token = (r0 + row) % n;
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            const int k0 = kKeys * half + 32 * w;
            see[w] = valid >= k0 + 32 ? ~0u : valid > k0 ? (1u << (valid - k0)) - 1u : 0u;
          }
          if (drafted && a.mask) {
            // lane e looks at key k0 + e for one row after the other (rows that are not there have a token, too)
            const uint8_t* const mask = a.mask + seg.p.seq * a.mask_stride + key0;
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
              const int k0 = kKeys * half + 32 * w;
              if (valid <= k0) break;
              const uint8_t* const from = mask + min(k0 + lane, valid - 1);
              uint32_t word = 0;
              if (mine)
#pragma unroll 1
                for (int x = 0; x < 32; x += 16) {
                  uint8_t bit[16];
#pragma unroll
                  for (int e = 0; e < 16; ++e) bit[e] = __ldg(from + (int64_t)__shfl_sync(0xffffffffu, token, x + e) * a.tokens);
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    const uint32_t votes = __ballot_sync(0xffffffffu, bit[e] != 0);
                    if (lane == x + e) word = votes;
                  }
                }
              see[w] &= word;
            }
          } else if (drafted) {   // causal
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
              const int upto = token - key0 + 1 - (kKeys * half + 32 * w);
              see[w] &= upto >= 32 ? ~0u : upto > 0 ? (1u << upto) - 1u : 0u;
            }
          }
        }
        float* const fk = factors + (steps & 1) * 2 * kTile;   // this tile's factors of logits and weights (8 bits)
        if constexpr (Q8) {
          float x = 0.f, y = 0.f;
          if (drafted) {
            x = kNewDot;
            y = kNewP;
          } else if (row < valid) {
            const int64_t at = ((int64_t)seg.p.seq * a.heads + seg.p.head) * a.cap + key0 + row;
            if (in_bounds(at < (int64_t)a.batch * a.heads * a.cap, a.dev_status)) {
              x = __ldg(a.k_step + at) * kQ8Dot;
              y = __ldg(a.v_step + at) * kQ8P;
            }
          }
          fk[row] = x * a.scale_log2;
          fk[kTile + row] = y;
          ptx::named_barrier(1 + slot, kSlotThreads);
        }
        wait(&bars.s_full[slot], steps);
        ptx::tc_fence_after();
        if (edge && (!Q8 || drafted)) {
          // V's rows that nobody sees become zeros, as do drafted ones with an infinity or NaN, which the rows that see
          // them get as a NaN weight: 0 times it must not reach the others. A thread looks after a key. (S is there, so the slot's
          // last P V is done, and the stage's phase before V's has passed.)
          if (half == kHalves - 1 && (!TWO || slot == 0)) {
            const uint32_t at = 2 * (TWO ? done + f : steps) + 1, stage = S::stage(slot, at);   // V's place in the ring
            wait(&bars.kv_full[stage], at / S::kTurn);
            uint8_t* const v = smem + S::kRing + stage * S::kStage;
            bool fix = row >= valid;
            if (drafted) {
              bool inf = false;
              if (!fix)
                for (int c = 0; c < D / 8; ++c) {
                  const uint4 w = *reinterpret_cast<const uint4*>(v + piece_at(row, c));
                  for (uint32_t x : {w.x, w.y, w.z, w.w}) inf |= (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
                }
              const uint32_t votes = __ballot_sync(0xffffffffu, inf);
              if (lane == 0) small.bad_keys[slot][quarter] = votes;
              fix |= inf;
            }
            if (fix)
              for (int c = 0; c < D / 8; ++c) *reinterpret_cast<uint4*>(v + piece_at(row, c)) = make_uint4(0u, 0u, 0u, 0u);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          const bool both = TWO && rows_of(seg) > kTile;
          if (drafted || both) ptx::named_barrier(both ? 3 : 1 + slot, both ? 2 * kSlotThreads : kSlotThreads);   // (the other slot's products read V, too)
          if (drafted) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) bad[w] = small.bad_keys[TWO ? 0 : slot][kWords * half + w] & see[w];
            ptx::named_barrier(both ? 3 : 1 + slot, both ? 2 * kSlotThreads : kSlotThreads);   // (before the next tile's are written)
          }
        }
        if (mine) {
          const float2 by = make_float2(a.scale_log2, a.scale_log2);
          // Logits of chunk c less `low`, in the log2 domain.
          auto load = [&](float2 (&y)[kE], int c, float low) {
            const int k0 = kKeys * half + kChunk * c;
            uint32_t x[kChunk];
            tmem_ld(s_at + k0, x);
            ptx::tmem_wait_ld();
            const float2 down = make_float2(-low, -low);
#pragma unroll
            for (int e = 0; e < kE; e += 2) {
              float4 k = make_float4(by.x, by.y, by.x, by.y);
              if constexpr (Q8) k = *reinterpret_cast<const float4*>(fk + k0 + 2 * e);
              y[e] = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), make_float2(k.x, k.y), down);
              y[e + 1] = fma2(make_float2(__uint_as_float(x[2 * e + 2]), __uint_as_float(x[2 * e + 3])), make_float2(k.z, k.w), down);
            }
          };
          auto highest = [](const float2 (&y)[kE], float top) {
            float other = -INFINITY;
#pragma unroll
            for (int e = 0; e < kE; e += 2) {
              top = fmaxf(fmaxf(top, y[e].x), y[e].y);
              other = fmaxf(fmaxf(other, y[e + 1].x), y[e + 1].y);
            }
            return fmaxf(top, other);
          };
          // Weights of chunk c, rounded to bf16; they are summed up as they were.
          float2 sum = make_float2(0.f, 0.f);
          auto pack = [&](float2 (&y)[kE], int c, uint32_t* p) {
            float2 other = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < kE; e += 2) {
              sum = add2(sum, y[e]);
              other = add2(other, y[e + 1]);
              if constexpr (Q8) {
                const float4 v = *reinterpret_cast<const float4*>(fk + kTile + kKeys * half + kChunk * c + 2 * e);
                y[e] = mul2(y[e], make_float2(v.x, v.y));
                y[e + 1] = mul2(y[e + 1], make_float2(v.z, v.w));
              }
              p[e] = pack2(y[e].x, y[e].y);
              p[e + 1] = pack2(y[e + 1].x, y[e + 1].y);
            }
            sum = add2(sum, other);
          };
          // Most tiles: the maximum as it is, and the weights in registers until both threads of a row know that none is too large.
          // (Straight code, and little of it: sixteen warps out of step fetch it, and what all of the tile's cases take together
          // in one piece cost 2800 clocks a tile, most of them without an instruction.)
          bool left = true;
          if (!Q8 && !first && !edge) {
            uint32_t p[kKeys / 2];
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              float2 y[kE];
              load(y, c, m);
              top = highest(y, top);
#pragma unroll
              for (int e = 0; e < kE; ++e) y[e] = make_float2(ex2(y[e].x), ex2(y[e].y));
              pack(y, c, p + kE * c);
            }
            left = any_of_pair(pair, top > S::kSlack);
            if constexpr (!Q8)
              if (!left) tmem_st(s_at + kKeys * half, p);
          }
          if (left) {
            // ---- a head's first tile, its last ones, and where the maximum grows: chunk by chunk
            auto mask = [&](float2 (&y)[kE], int c, bool nan) {
              if (!edge) return;
              uint32_t keep = see[0], not_a = bad[0];
#pragma unroll
              for (int w = 1; w < kWords; ++w)
                if (kChunk * c / 32 == w) keep = see[w], not_a = bad[w];
              keep >>= kChunk * c % 32;
              not_a >>= kChunk * c % 32;
#pragma unroll
              for (int e = 0; e < kE; ++e) {
                if (!(keep >> (2 * e) & 1)) y[e].x = -INFINITY;
                if (!(keep >> (2 * e + 1) & 1)) y[e].y = -INFINITY;
                if (nan && (not_a >> (2 * e) & 1)) y[e].x = __uint_as_float(0x7FC00000u);
                if (nan && (not_a >> (2 * e + 1) & 1)) y[e].y = __uint_as_float(0x7FC00000u);
              }
            };
            float top = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
              float2 y[kE];
              load(y, c, 0.f);
              mask(y, c, false);
              top = highest(y, top);
            }
            if constexpr (kHalves == 2) {
              swap[half * kTile + row] = top;
              ptx::named_barrier(pair, 64);
              top = fmaxf(top, swap[(half ^ 1) * kTile + row]);
            }
            const float next = first ? fmaxf(m, top) : top - m > S::kSlack ? top : m;
            if (!first && __any_sync(0xffffffffu, next != m)) {   // (the same for both threads of a row)
              const float fall = rescale(m, next);
              l *= fall;
#pragma unroll 1
              for (int c = half * (D / kHalves); c < (half + 1) * (D / kHalves); c += 16) {
                uint32_t x[16];
                tmem_ld(o_lane + S::kO(slot) + c, x);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * fall);
                tmem_st(o_lane + S::kO(slot) + c, x);
              }
            }
            m = next;
            sum = make_float2(0.f, 0.f);
            uint32_t p[kE];
            // The maximum is a logit as it was rounded. An FMA's difference to it is that of the logit before its rounding, off by
            // half a unit of the logit, which from 2^30 on is a weight of 2^+-64 and more. So for a row whose maximum is large logits
            // are rounded alike before the difference: an FMA less zero, and an addition (row by row, as what one row does must not hang
            // on its neighbours; with a zero that the compiler can see it makes one FMA of both). Over 8 bits, where every tile comes this
            // way, in a loop of its own (for all rows 3 % more time); the few tiles of dense caches that do have the one loop.
            auto weigh = [&](auto rounded) {
              const bool large = fabsf(m) > 0x1p20f;
#pragma unroll 1
              for (int c = 0; c < kChunks; ++c) {   // (a chunk's weights stand where logits of the first chunks stood)
                float2 y[kE];
                if constexpr (decltype(rounded)::value) {
                  load(y, c, large ? 0.f : m);
                  const float rest = large ? -m : -0.f;
#pragma unroll
                  for (int e = 0; e < kE; ++e) y[e] = add2(y[e], make_float2(rest, rest));
                } else {
                  load(y, c, m);
                }
                mask(y, c, true);
#pragma unroll
                for (int e = 0; e < kE; ++e) y[e] = make_float2(ex2(y[e].x), ex2(y[e].y));
                pack(y, c, p);
                tmem_st(s_at + kKeys * half + kE * c, p);
              }
            };
            if constexpr (!Q8)
              weigh(std::true_type());
            else if (__any_sync(0xffffffffu, fabsf(m) > 0x1p20f))
              weigh(std::true_type());
            else
              weigh(std::false_type());
          }
          l += sum.x + sum.y;
          ptx::tmem_wait_st();
        }
        first = false;
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars.p_ready[slot]);
        ++steps;
      }

      // ---- the head's end in this share: the halves' sums meet, and up to 128 rows the slots' m, sums and O
      const bool whole = seg.whole();
      if (half == 1) swap[row] = l;   // (the other half has read what stood there: its own l is from after the last swap)
      wait(&bars.o_full, seg.index);
      ptx::tc_fence_after();
      float* const part = part_at<D>(a, (int)blockIdx.x, seg.at > share.at ? 1 : 0);
      const int pr = row + (TWO ? slot * kTile : 0);   // the row in a part
      const int r = r0 + row, g = r / n;
      const int64_t to = (((int64_t)seg.p.seq * a.heads + seg.p.head) * a.group + g) * a.tokens + (r - g * n);
      auto finish = [&](float top, float sum) {        // what is written beside the row; returns the output's factor
        if (row < rows) {
          if (!whole) {
            part[a.tile_q * D + pr] = top;
            part[a.tile_q * (D + 1) + pr] = sum;
          } else if (a.lse) {
            a.lse[to] = lse_of(top, sum);
          }
        }
        return (Q8 ? kQ8Out : 1.0f) * (!whole ? 1.0f : sum == 0.f ? 0.f : 1.0f / sum);
      };
      auto write = [&](int c, const uint32_t (&x)[16]) {   // channels c .. c + 15 of this thread's row
        if (row >= rows) return;
        if (whole) {
          uint4* const u = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + to * D + c);
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = pack2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
          u[0] = make_uint4(w[0], w[1], w[2], w[3]);
          u[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
          float* const u = part + c * S::kRows + pr;   // (a warp's rows lie side by side)
#pragma unroll
          for (int e = 0; e < 16; ++e) u[e * S::kRows] = __uint_as_float(x[e]);
        }
      };
      if constexpr (kHalves == 2) {
        ptx::named_barrier(pair, 64);
        if (half == 0) l += swap[row];
      }
      if constexpr (TWO) {
        if (half == 0) {
          const float scale = finish(m, l);
          swap[kTile + row] = scale;
        }
        if constexpr (kHalves == 2) ptx::named_barrier(pair, 64);
        if (mine) {
          const float scale = swap[kTile + row];
#pragma unroll 1
          for (int c = half * (D / kHalves); c < (half + 1) * (D / kHalves); c += 16) {
            uint32_t x[16];
            tmem_ld(o_lane + S::kO(slot) + c, x);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * scale);
            write(c, x);
          }
        }
      } else {
        // each slot and half writes its share of the channels
        const bool other = seg.tiles > 1;   // (of one tile, one slot has none)
        const int only = (int)(done & 1);   // the first tile's slot
        float* const factor = reinterpret_cast<float*>(smem + S::kSwap);   // slot 0's: the two factors of a row, in the end
        if (half == 0 && slot == 1) {
          swap[row] = l;
          swap[kTile + row] = m;
        }
        ptx::named_barrier(3, 2 * kSlotThreads);
        if (half == 0 && slot == 0) {
          const float l1 = swap[2 * kTile + row], m1 = swap[3 * kTile + row];   // slot 1's
          const float top = fmaxf(m, m1), f0 = rescale(m, top), f1 = rescale(m1, top);
          const float scale = finish(top, fmaf(l, f0, l1 * f1));
          factor[row] = f0 * scale;
          factor[kTile + row] = f1 * scale;
        }
        ptx::named_barrier(3, 2 * kSlotThreads);
        if (mine) {
          const float f0 = factor[row], f1 = factor[kTile + row];
          const float fx = other || only == 0 ? f0 : f1;
          constexpr int kMine = D / (2 * kHalves);
#pragma unroll 1
          for (int c = (kHalves * slot + half) * kMine; c < (kHalves * slot + half + 1) * kMine; c += 16) {
            uint32_t x[16], y[16];
            tmem_ld(o_lane + S::kO(other ? 0 : only) + c, x);
            if (other) tmem_ld(o_lane + S::kO(1) + c, y);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float z = __uint_as_float(x[e]) * fx;
              x[e] = __float_as_uint(other ? fmaf(__uint_as_float(y[e]), f1, z) : z);
            }
            write(c, x);
          }
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars.o_free);
      ptx::named_barrier(3, 2 * kSlotThreads);   // (the swap area is free)
      done += (uint32_t)seg.tiles;
    } while (seg.next(a));
  } else if constexpr (Q8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kMoveRegs));
    // ---- codes into bf16 tiles: two threads per key, half of the channels each
    const int key = tid % kTile, part = (tid - 32 * (4 + S::kSoft)) / kTile;
    Segments ks(a, share), vs(a, share);
    int kf = 0, vf = 0;
    uint32_t used = 0;                 // raw tiles
    auto make = [&](Segments& s, int& f, uint32_t t, bool is_key) {
      const uint32_t place = 2 * (TWO ? t : t / 2) + (is_key ? 0 : 1), slot = S::stage(t & 1, place), turn = place / S::kTurn;
      const int tile = s.p.tile + f;
      const int64_t bh = (int64_t)s.p.seq * a.heads + s.p.head;
      const bool cached = tile < s.p.s.cache_tiles;
      uint8_t* const to = smem + S::kRing + slot * S::kStage;
      if (cached) {
        const uint32_t at = used % kRaws;
        wait(&bars.raw_full[at], used / kRaws);
        const uint8_t* const from = smem + S::kRawRing + at * S::kRaw;
        const bool there = key < s.p.s.rows - tile * kTile;
        constexpr int kMine = D / 32;   // pieces of sixteen codes
        uint4 w[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int c = part * kMine + i;
          const uint32_t off = D == 128 ? key * 128 + ((c ^ (key & 7)) << 4) : key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
          w[i] = there ? *reinterpret_cast<const uint4*>(from + off) : make_uint4(0u, 0u, 0u, 0u);
        }
        if (turn > 0) wait(&bars.kv_empty[slot], turn - 1);
        auto low = [](uint32_t x) { return prmt(x, x, 0x1100) & 0x807F807Fu; };
        auto high = [](uint32_t x) { return prmt(x, x, 0x3322) & 0x807F807Fu; };
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int c = part * kMine + i;
          *reinterpret_cast<uint4*>(to + piece_at(key, 2 * c)) = make_uint4(low(w[i].x), high(w[i].x), low(w[i].y), high(w[i].y));
          *reinterpret_cast<uint4*>(to + piece_at(key, 2 * c + 1)) = make_uint4(low(w[i].z), high(w[i].z), low(w[i].w), high(w[i].w));
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars.raw_empty[at]);
        ++used;
      } else {
        const int row = (tile - s.p.s.cache_tiles) * kTile + key;
        const bool there = row < s.p.s.n;
        const __nv_bfloat16* const from = static_cast<const __nv_bfloat16*>(is_key ? a.k_new : a.v_new) + (bh * a.tokens + (there ? row : 0)) * D;
        if (turn > 0) wait(&bars.kv_empty[slot], turn - 1);
#pragma unroll 8
        for (int c = part * (D / 16); c < (part + 1) * (D / 16); ++c)
          *reinterpret_cast<uint4*>(to + piece_at(key, c)) = there ? ld_nc_v4(from + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars.kv_full[slot]);
      if (++f == s.tiles) {
        f = 0;
        s.next(a);
      }
    };
    for (uint32_t t = 0; t < total && !__any_sync(0xffffffffu, aborted()); t += kPair) {   // (all of a warp leave together)
      for (uint32_t u = t; u < t + kPair && u < total; ++u) make(ks, kf, u, true);
      for (uint32_t u = t; u < t + kPair && u < total; ++u) make(vs, vf, u, false);
    }
  }

  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, S::kColumns);
  }
}

template <bool Q8, int D, bool TWO> cudaError_t launch_typed(const TreeJob& job) {
  using S = Shape<Q8, D, TWO>;
  Args a = tree_args(job, S::kRows);
  a.least = 2;
  const int64_t rows = (int64_t)a.group * a.tokens, passes = (rows + S::kRows - 1) / S::kRows;
  int64_t ctas = device_sm_count() < kMaxTcCtas ? device_sm_count() : kMaxTcCtas;
  if (!job.n_new && passes > 1 && 4 * passes <= ctas) {   // (where tokens differ, some siblings would have nothing to do)
    a.siblings = (int)passes;
    ctas -= ctas % passes;
  }
  TreeMaps maps;
  if (!tree_maps(&maps, job, kTile, kTile)) return cudaErrorInvalidValue;
  cudaError_t err = allow_dynamic_smem<tree_tc_kernel<Q8, D, TWO>>(S::smem());
  if (err != cudaSuccess) return err;
  err = tree_fill(a, job, kTile, kTile, ctas);
  if (err != cudaSuccess) return err;
  tree_tc_kernel<Q8, D, TWO><<<a.ctas, S::kThreads, S::smem(), job.stream>>>(a, maps);
  err = cudaGetLastError();
  return err != cudaSuccess ? err : launch_tree_join_wide<D, kTile>(a, job.stream);
}

// Passes of 128 rows or of 256, which read the cache half as often. Where all sequences have as many tokens, an odd number of
// halves leaves one empty: 384 rows over 1500 keys of 64 channels take 79 us in passes of 128 (93 of 256), 280 over 16384 of 128
// channels 94 (114), and nine halves (1100 rows) over 1500 keys of 256 heads of 64 channels 203 (210), over 2000 keys of 32 heads 39 (53).
// Of eleven (1400) 257 (247) and 54 (60), so that nine are the last. Even numbers differ little where heads are few (900 rows over
// 8192 keys of 16 heads 56 us either way) and are better in passes of 256 where they are many (over 1500 keys of 256 heads 182 (171)).
// Where sequences have fewer tokens, most have an odd number of halves or one, and passes come one after the other, so that what
// a wave of heads holds has to stay in L2: with 128 channels passes of 128 are as good or better up to 1 MB a head (128 heads, up to
// 600 rows each: 0.9 MB 77 us (85), 1 MB 82 (85), 2 MB 136 (124), 8 MB 451 (361); up to 256 rows 54 (59), 52 (61), 83 (83), 264 (215)). With
// 64 channels the way from logits to weights counts more than reading (0.5 MB 59 (64), 1 MB 85 (94), 8 MB 465 (523)), and over 8 bits
// unpacking does (up to 256 rows over 16384 keys 136 us (159), up to 440 192 (215)).
template <bool Q8, int D> bool narrow_passes(const TreeJob& job) {
  const int64_t rows = (int64_t)(job.q_heads / job.heads) * job.tokens, halves = (rows + 127) / 128;
  if (halves > 9) return false;
  if (!job.n_new || halves == 1) return halves % 2 != 0;
  return Q8 || D == 64 || job.cap * D * 4 <= 1024 * 1024;
}

template <bool Q8, int D> cudaError_t launch_dim(const TreeJob& job) {
  return narrow_passes<Q8, D>(job) ? launch_typed<Q8, D, false>(job) : launch_typed<Q8, D, true>(job);
}

}  // namespace

cudaError_t launch_tree_tc(const TreeJob& job) {
  if (job.k_step) return job.head_dim == 64 ? launch_dim<true, 64>(job) : launch_dim<true, 128>(job);
  return job.head_dim == 64 ? launch_dim<false, 64>(job) : launch_dim<false, 128>(job);
}

}  // namespace snapkv
