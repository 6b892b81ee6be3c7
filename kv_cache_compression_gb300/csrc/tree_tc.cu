// Tree attention of many query rows a KV head, bf16, over a dense cache or one in 8 bits (tree_schedule.cuh has the
// schedule): wide trees, grouped queries, prompts that read an encoder's states.
//
//   S = Q K^T,  P = exp2(S - m),  O = sum P V,  running m and sum per row
//
// tcgen05 with 128 query rows by 128 keys: S (fp32) and O stand in TMEM, P goes back over S as the second product's A
// operand, K and V are B operands in shared memory. Two slots, each an S, an O and four softmax warps (a thread per row),
// keep the tensor cores busy while the other slot's weights are computed. Up to 128 rows (TWO false) both slots serve the
// same rows and take the key tiles in turn, and their halves of O meet at the head's end; up to 256 a slot has 128 rows
// each and every key tile serves both, so that the cache is read once. MMAs are issued in the order P V of a tile, then
// Q K^T of the slot's next, which overwrites what P V has read: the tensor core takes them one after the other.
//
// Weights enter the second product in two bf16 parts (16 bits), P V twice as long as Q K^T: 1536 clocks for a tile of 128
// channels, in which HBM delivers 70 keys' bf16 rows. A row's maximum is only raised, and its O rescaled, when it would
// grow by more than 2^8; sums and outputs stay under the same maximum, so that nothing is lost.
//
// 8-bit rows arrive as they are; four more warps unpack them into the tiles that TMA writes for bf16 rows. As operands
// they are *subnormal* bf16 (sign and seven magnitude bits, u 2^-133: a byte permute and an AND per two values), for
// which queries are scaled by 2^64 and weights by 2^80; a step multiplies its key's logits and weights.
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
constexpr float kSlack = 8.0f;                   // log2 of what weights may exceed 1 by

constexpr float kQ8Q = 0x1p64f, kQ8Dot = 0x1p69f, kQ8P = 0x1p80f, kQ8Out = 0x1p53f;
constexpr float kNewDot = 0x1p-64f, kNewP = 0x1p-53f;   // for drafted rows, whose values are as they are

template <bool Q8, int D, bool TWO> struct Shape {
  static constexpr int kRows = TWO ? 256 : 128;                // query rows of a pass
  static constexpr int kWarps = Q8 ? 16 : 12;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kSlotQ = kTile * D * 2;                 // bytes of 128 rows of queries
  static constexpr int kQBufs = TWO || Q8 ? 1 : 2;
  static constexpr int kStage = kTile * D * 2;                 // of a tile of K or V
  static constexpr int kStages = (Q8 ? (TWO ? 3 : 4) : 5) * (128 / D);
  static constexpr int kRaw = kTile * D;                       // of a tile of codes
  static constexpr int kRaws = Q8 ? 3 * (128 / D) : 0;
  static constexpr int kQ = 0;
  static constexpr int kRing = kQ + (TWO ? 2 : kQBufs) * kSlotQ;
  static constexpr int kRawRing = kRing + kStages * kStage;
  static constexpr int kMeet = kRawRing + kRaws * kRaw;        // [128] float2
  static constexpr int kFactors = kMeet + kTile * 8;           // [2 slots][2][K, V][128] floats (8 bits)
  static constexpr int kBytes = kFactors + (Q8 ? 2 * 2 * 2 * kTile * 4 : 0);
  static constexpr int smem() { return 1024 + kBytes; }
  static constexpr int kS(int slot) { return slot * 128; }     // TMEM columns
  static constexpr int kO(int slot) { return 256 + slot * D; }
  static constexpr int kColumns = 512;
};

struct Bars {
  uint64_t kv_full[12], kv_empty[12], raw_full[8], raw_empty[8];
  uint64_t q_full[2], q_empty[2], s_full[2], p_ready[2];
  uint64_t o_full, o_free, drain;
};

__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
      "%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}

// D (+)= A[tmem] B[smem], bf16 operands, fp32 sums.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a),
      "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor of V as B: keys (the product's k) are rows of 128 bytes of 64 channels (its n), 128-byte swizzle; eight keys
// are 1024 bytes apart, 64 channels a block of kTile rows.
__device__ __forceinline__ uint64_t v_desc(uint32_t at) {
  return (uint64_t)((at >> 4) & 0x3FFFu) | (uint64_t)((kTile * 128) >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}

__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 two = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&two);
}

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
  __device__ __forceinline__ Segments(const Args& a, const Share& s) : p(first_place<kTile, kTile>(a, s)), at(s.at), end(s.end), index(0) { cut(); }
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
  extern __shared__ uint8_t raw_smem[];
  __shared__ Bars bars;
  __shared__ uint32_t tmem_at;
  __shared__ int abort;
  __shared__ uint32_t bad_keys[2][4];
  uint8_t* const smem = raw_smem + ((1024 - (ptx::smem_u32(raw_smem) & 1023)) & 1023);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid % 32, warp = __shfl_sync(0xffffffffu, tid / 32, 0);
  if (tid == 0) {
    abort = 0;
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&bars.kv_full[i], Q8 ? 4 : 1);   // (four unpacking warps)
      ptx::mbar_init(&bars.kv_empty[i], 1);
    }
    for (int i = 0; i < kRaws; ++i) {
      ptx::mbar_init(&bars.raw_full[i], 1);
      ptx::mbar_init(&bars.raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars.q_full[i], 64);
      ptx::mbar_init(&bars.q_empty[i], 1);
      ptx::mbar_init(&bars.s_full[i], 1);
      ptx::mbar_init(&bars.p_ready[i], 4);
    }
    ptx::mbar_init(&bars.o_full, 1);
    ptx::mbar_init(&bars.o_free, 8);
    ptx::mbar_init(&bars.drain, 1);
    ptx::fence_mbar_init();
  }
  const Share share = find_share<kTile, kTile, S::kThreads>(a);   // (with barriers)
  if (share.at >= share.end) return;
  if (warp == 1) {
    ptx::tmem_alloc(&tmem_at, S::kColumns);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_at;
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
  const int64_t total = share.end - share.at;   // tiles

  if (warp == 0) {
    // ---- loads, in the order in which the products take them. Up to 128 rows: K0 K1 V0 K2 V1 K3 ..; more: K0 V0 K1 V1 ..
    if (lane == 0) {
      Segments ks(a, share), vs(a, share);
      int kf = 0, vf = 0;   // tiles of the segments so far
      uint32_t sent = 0;
      auto send = [&](Segments& s, int& f, bool key) {
        constexpr int kSlots = Q8 ? kRaws : kStages;
        const uint32_t slot = sent % kSlots, turn = sent / kSlots;
        const int tile = s.p.tile + f, bh = s.p.seq * a.heads + s.p.head;
        const bool cached = tile < s.p.s.cache_tiles;
        if (!Q8 || cached) {   // (drafted rows beside an 8-bit cache are copied by the warps that unpack)
          if (turn > 0 && !wait(Q8 ? &bars.raw_empty[slot] : &bars.kv_empty[slot], turn - 1)) return false;
          uint64_t* const bar = Q8 ? &bars.raw_full[slot] : &bars.kv_full[slot];
          uint8_t* const to = smem + (Q8 ? S::kRawRing + slot * S::kRaw : S::kRing + slot * S::kStage);
          const CUtensorMap* const map = cached ? (key ? &maps.k : &maps.v) : (key ? &maps.k_new : &maps.v_new);
          const int row0 = (cached ? tile : tile - s.p.s.cache_tiles) * kTile;
          ptx::mbar_arrive_expect_tx(bar, Q8 ? S::kRaw : S::kStage);
#pragma unroll
          for (int c = 0; c < (Q8 ? 1 : D / 64); ++c) ptx::tma_load_3d(to + c * kTile * 128, map, 64 * c, row0, bh, bar);
          ++sent;
        }
        if (++f == s.tiles) {
          f = 0;
          s.next(a);
        }
        return true;
      };
      bool ok = send(ks, kf, true);
      if (ok && !TWO && total > 1) ok = send(ks, kf, true);
      for (int64_t t = 0; ok && t < total; ++t) {
        ok = send(vs, vf, false);
        if (ok && t + (TWO ? 1 : 2) < total) ok = send(ks, kf, true);
      }
      // Copies in flight land before the block ends, also after a wait ran out.
      constexpr uint32_t kSlots = Q8 ? kRaws : kStages;
      const int none = 0;
      for (uint32_t i = sent > kSlots ? sent - kSlots : 0; i < sent; ++i)
        ptx::mbar_wait(Q8 ? &bars.raw_full[i % kSlots] : &bars.kv_full[i % kSlots], (i / kSlots) & 1, &none, kWaitLimit);
    }
  } else if (warp == 1) {
    // ---- products
    if (lane == 0) {
      constexpr uint32_t kIdescQk = ptx::idesc_bf16_f32(128, kTile), kIdescPv = ptx::idesc_bf16_f32(128, D) | 1u << 16;   // (V: n-major)
      Segments qs(a, share), ps(a, share);
      int qf = 0, pf = 0;
      uint32_t taken = 0;              // ring tiles so far, in order
      uint32_t s_steps[2] = {0, 0}, p_steps[2] = {0, 0};
      uint32_t k_slot = 0, v_slot = 0;
      auto take = [&](uint32_t& slot) {
        slot = taken % kStages;
        const bool ok = wait(&bars.kv_full[slot], taken / kStages);
        ++taken;
        ptx::tc_fence_after();
        return ok;
      };
      // S of a slot = Q K^T of the tile in k_slot.
      auto qk = [&](int slot) {
        const uint32_t q_at = q_smem + (TWO ? slot : qs.index % S::kQBufs) * S::kSlotQ, k_at = ring + k_slot * S::kStage;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t off = (s / 4) * (kTile * 128) + (s % 4) * 32;
          ptx::mma_bf16(tmem + S::kS(slot), ptx::smem_desc_k_sw128(q_at + off), ptx::smem_desc_k_sw128(k_at + off), kIdescQk, s > 0);
        }
        ptx::mma_commit(&bars.s_full[slot]);
        ++s_steps[slot];
      };
      // O of a slot += P V of the tile in v_slot, `fresh`: O =.
      auto pv = [&](int slot, bool fresh) {
        const uint32_t v_at = ring + v_slot * S::kStage;
#pragma unroll
        for (int s = 0; s < kTile / 16; ++s)
#pragma unroll
          for (int part = 0; part < 2; ++part)
            mma_ts(tmem + S::kO(slot), tmem + S::kS(slot) + (s / 2) * 32 + part * 16 + (s % 2) * 8, v_desc(v_at + s * 2048), kIdescPv,
                   !(fresh && s == 0 && part == 0));
      };
      auto weights = [&](int slot) {
        const bool ok = wait(&bars.p_ready[slot], p_steps[slot]);
        ++p_steps[slot];
        ptx::tc_fence_after();
        return ok;
      };
      auto queries = [&] { return qf > 0 || wait(&bars.q_full[qs.index % S::kQBufs], qs.index / S::kQBufs); };
      auto outputs = [&] { return pf > 0 || ps.index == 0 || wait(&bars.o_free, ps.index - 1); };
      auto qk_done = [&] {             // of the tile, by all slots
        ptx::mma_commit(&bars.kv_empty[k_slot]);
        if (++qf == qs.tiles) {
          ptx::mma_commit(&bars.q_empty[qs.index % S::kQBufs]);
          qf = 0;
          qs.next(a);
        }
      };
      auto pv_done = [&] {
        ptx::mma_commit(&bars.kv_empty[v_slot]);
        if (++pf == ps.tiles) {
          ptx::mma_commit(&bars.o_full);
          pf = 0;
          ps.next(a);
        }
      };
      bool ok = true;
      if constexpr (!TWO) {
        uint32_t step = 0;
        auto next_qk = [&](int slot) {
          if (!queries() || !take(k_slot)) return false;
          qk(slot);
          qk_done();
          return true;
        };
        ok = next_qk(0) && (total < 2 || next_qk(1));
        for (int64_t t = 0; ok && t < total; ++t, ++step) {
          const int slot = (int)(step & 1);
          ok = weights(slot) && take(v_slot) && outputs();
          if (!ok) break;
          pv(slot, pf < 2);            // (a segment's first two tiles are its slots' first)
          pv_done();
          if (t + 2 < total) ok = next_qk(slot);
        }
      } else {
        bool two = rows_of(qs) > 128;  // the second slot has rows of the segment qs
        ok = queries() && take(k_slot);
        if (ok) {
          qk(0);
          if (two) qk(1);
          qk_done();
        }
        for (int64_t t = 0; ok && t < total; ++t) {
          const bool second = rows_of(ps) > 128, more = t + 1 < total;
          ok = weights(0) && take(v_slot) && outputs();
          if (!ok) break;
          const bool fresh = pf == 0;
          pv(0, fresh);
          if (more) {
            two = rows_of(qs) > 128;
            ok = queries() && take(k_slot);
            if (!ok) break;
            qk(0);
          }
          if (second) {
            ok = weights(1);
            if (!ok) break;
            pv(1, fresh);
          }
          pv_done();
          if (more) {
            if (two) qk(1);
            qk_done();
          }
        }
      }
      // Products in flight end before the block does.
      ptx::mma_commit(&bars.drain);
      const int none = 0;
      ptx::mbar_wait(&bars.drain, 0, &none, kWaitLimit);
    }
  } else if (warp < 4) {
    // ---- queries into shared memory
    const int at = tid - 64;
    Segments seg(a, share);
    do {
      const int buf = seg.index % S::kQBufs, turn = seg.index / S::kQBufs;
      if (turn > 0) wait(&bars.q_empty[buf], turn - 1);
      const int r0 = r0_of(seg), rows = rows_of(seg), n = seg.p.s.n;
      const int64_t bh = (int64_t)seg.p.seq * a.heads + seg.p.head;
      const int slots = TWO && rows > 128 ? 2 : 1;
      // A thread has every (64 / kPieces)-th row's piece c, eight of them under way at a time.
      constexpr int kPieces = D / 8, kStep = 64 / kPieces;
      const int c = at % kPieces;
#pragma unroll 1
      for (int x = at / kPieces; x < slots * kTile; x += 8 * kStep) {
        uint4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = x + e * kStep, row = r0 + r, g = row / n;
          v[e] = make_uint4(0u, 0u, 0u, 0u);
          if (r < rows) v[e] = ld_nc_v4(static_cast<const __nv_bfloat16*>(a.q) + ((bh * a.group + g) * a.tokens + (row - g * n)) * D + 8 * c);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = x + e * kStep;
          if constexpr (Q8) {
            uint32_t* const w = &v[e].x;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack2(__uint_as_float(w[i] << 16) * kQ8Q, __uint_as_float(w[i] & 0xFFFF0000u) * kQ8Q);
          }
          *reinterpret_cast<uint4*>(smem + S::kQ + (TWO ? r / kTile : buf) * S::kSlotQ + piece_at(r % kTile, c)) = v[e];
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      ptx::mbar_arrive(&bars.q_full[buf]);
    } while (seg.next(a) && !aborted());
  } else if (warp < 12) {
    // ---- softmax: a thread per row of a slot
    const int slot = (warp - 4) / 4, quarter = warp % 4, row = quarter * 32 + lane;
    const uint32_t s_at = tmem + ((uint32_t)(quarter * 32) << 16) + S::kS(slot);
    const uint32_t o_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    float2* const meet = reinterpret_cast<float2*>(smem + S::kMeet);
    float* const factors = reinterpret_cast<float*>(smem + S::kFactors) + slot * 4 * kTile;
    uint32_t steps = 0;                // of this slot
    uint32_t done = 0;                 // tiles of the share in the segments so far
    Segments seg(a, share);
    do {
      const int r0 = r0_of(seg) + (TWO ? slot * kTile : 0), n = seg.p.s.n;
      const int rows = min(kTile, rows_of(seg) - (TWO ? slot * kTile : 0));   // this slot's (none or less: it rests)
      const bool mine = quarter * 32 < rows;                                  // this warp has rows
      const int64_t bh = (int64_t)seg.p.seq * a.heads + seg.p.head;
      const int r = r0 + row, g = r / n, token = r - g * n;
      float m = kNoMax, l = 0.f;
      bool first = true;
      for (int f = TWO ? 0 : (int)((done ^ slot) & 1); rows > 0 && f < seg.tiles; f += TWO ? 1 : 2) {
        const int tile = seg.p.tile + f;
        const bool drafted = tile >= seg.p.s.cache_tiles;
        const int key0 = (drafted ? tile - seg.p.s.cache_tiles : tile) * kTile;
        const int valid = min(kTile, (drafted ? n : seg.p.s.rows) - key0);
        const bool edge = drafted || valid < kTile;
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
        if (edge) {
#pragma unroll
          for (int w = 0; w < 4; ++w) see[w] = valid >= 32 * w + 32 ? ~0u : valid > 32 * w ? (1u << (valid - 32 * w)) - 1u : 0u;
          if (drafted && a.mask) {
            // lane e looks at key 32 w + e for one row after the other (rows that are not there have a token, too)
            const uint8_t* const mask = a.mask + seg.p.seq * a.mask_stride + key0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              if (valid <= 32 * w) break;
              const uint8_t* const from = mask + min(32 * w + lane, valid - 1);
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
            const int upto = token - key0 + 1;
#pragma unroll
            for (int w = 0; w < 4; ++w) see[w] &= upto >= 32 * w + 32 ? ~0u : upto > 32 * w ? (1u << (upto - 32 * w)) - 1u : 0u;
          }
        }
        float* const fk = factors + (steps & 1) * 2 * kTile;   // this tile's factors of logits and weights (8 bits)
        if constexpr (Q8) {
          float k = 0.f, v = 0.f;
          if (drafted) {
            k = kNewDot;
            v = kNewP;
          } else if (row < valid) {
            const int64_t at = bh * a.cap + key0 + row;
            if (in_bounds(at < (int64_t)a.batch * a.heads * a.cap, a.dev_status)) {
              k = __ldg(a.k_step + at) * kQ8Dot;
              v = __ldg(a.v_step + at) * kQ8P;
            }
          }
          fk[row] = k * a.scale_log2;
          fk[kTile + row] = v;
          ptx::named_barrier(1 + slot, 128);
        }
        uint32_t bad[4] = {0u, 0u, 0u, 0u};
        if (edge && (!Q8 || drafted)) {
          // V's rows that nobody sees become zeros, as do drafted ones with an infinity or NaN, which the rows that see
          // them get as a NaN weight: 0 times it must not reach the others. A thread looks after a key.
          if (!TWO || slot == 0) {
            const uint32_t t = done + f;
            const uint32_t at = TWO ? 2 * t + 1 : (int64_t)t + 1 == total ? 2 * t + 1 : 2 * t + 2;   // V's place in the ring's order
            wait(&bars.kv_full[at % kStages], at / kStages);
            uint8_t* const v = smem + S::kRing + (at % kStages) * S::kStage;
            bool fix = row >= valid;
            if (drafted) {
              bool inf = false;
              if (!fix)
                for (int c = 0; c < D / 8; ++c) {
                  const uint4 w = *reinterpret_cast<const uint4*>(v + piece_at(row, c));
                  for (uint32_t x : {w.x, w.y, w.z, w.w}) inf |= (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
                }
              const uint32_t votes = __ballot_sync(0xffffffffu, inf);
              if (lane == 0) bad_keys[slot][quarter] = votes;
              fix |= inf;
            }
            if (fix)
              for (int c = 0; c < D / 8; ++c) *reinterpret_cast<uint4*>(v + piece_at(row, c)) = make_uint4(0u, 0u, 0u, 0u);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          if (drafted) {
            const bool both = TWO && rows_of(seg) > 128;
            ptx::named_barrier(both ? 3 : 1 + slot, both ? 256 : 128);
#pragma unroll
            for (int w = 0; w < 4; ++w) bad[w] = bad_keys[TWO ? 0 : slot][w] & see[w];
            ptx::named_barrier(both ? 3 : 1 + slot, both ? 256 : 128);   // (before the next tile's are written)
          }
        }
        wait(&bars.s_full[slot], steps);
        ptx::tc_fence_after();
        // Logits of chunk c (32 keys) as they are compared: 8-bit keys' steps are in.
        auto scaled = [&](uint32_t (&x)[32], int c) {
          if constexpr (Q8) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 k = *reinterpret_cast<const float4*>(fk + 32 * c + e);
              const float2 y = mul2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), make_float2(k.x, k.y));
              const float2 z = mul2(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), make_float2(k.z, k.w));
              x[e] = __float_as_uint(y.x), x[e + 1] = __float_as_uint(y.y), x[e + 2] = __float_as_uint(z.x), x[e + 3] = __float_as_uint(z.y);
            }
          }
        };
        auto raise = [&](float top) {   // the row's maximum, and what stands under it
          if constexpr (!Q8) top *= a.scale_log2;
          if (first) {
            m = fmaxf(m, top);
          } else if (__any_sync(0xffffffffu, top > m + kSlack)) {
            const float next = top > m + kSlack ? top : m, fall = rescale(m, next);
            m = next;
            l *= fall;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t x[32];
              tmem_ld32(o_lane + S::kO(slot) + c, x);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * fall);
              tmem_st32(o_lane + S::kO(slot) + c, x);
            }
            ptx::tmem_wait_st();
          }
        };
        // Weights of chunk c from its (scaled) logits; `keep` and `nan` are this row's bits of its keys.
        float2 sum = make_float2(0.f, 0.f);
        auto weigh = [&](const uint32_t (&x)[32], int c, auto masked, uint32_t keep, uint32_t nan) {
          const float2 down = make_float2(-m, -m), by = make_float2(a.scale_log2, a.scale_log2);
          uint32_t p[32];   // first parts, then second parts
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float2 y = make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
            y = Q8 ? add2(y, down) : fma2(y, by, down);
            y = make_float2(ex2(y.x), ex2(y.y));
            if constexpr (decltype(masked)::value) {
              if (!(keep >> e & 1)) y.x = 0.f;
              if (!(keep >> (e + 1) & 1)) y.y = 0.f;
              if (nan >> e & 1) y.x = __uint_as_float(0x7FC00000u);
              if (nan >> (e + 1) & 1) y.y = __uint_as_float(0x7FC00000u);
            }
            sum = add2(sum, y);
            if constexpr (Q8) y = mul2(y, *reinterpret_cast<const float2*>(fk + kTile + 32 * c + e));
            const uint32_t w = pack2(y.x, y.y);
            p[e / 2] = w;
            p[16 + e / 2] = pack2(y.x - __uint_as_float(w << 16), y.y - __uint_as_float(w & 0xFFFF0000u));
          }
          tmem_st32(s_at + 32 * c, p);
        };
        auto highest = [](const uint32_t (&x)[32], float top) {
          float other = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            top = fmaxf(fmaxf(top, __uint_as_float(x[e])), __uint_as_float(x[e + 1]));
            other = fmaxf(fmaxf(other, __uint_as_float(x[e + 2])), __uint_as_float(x[e + 3]));
          }
          return fmaxf(top, other);
        };
        if (mine && !edge) {
          // Chunks 0 and 1, then 2 and 3 for the maximum; weights from 2 and 3 while they are there, then 0 and 1 again.
          uint32_t x[32], y[32];
          float top = -INFINITY;
          tmem_ld32(s_at, x);
          ptx::tmem_wait_ld();
          tmem_ld32(s_at + 32, y);
          scaled(x, 0);
          top = highest(x, top);
          ptx::tmem_wait_ld();
          tmem_ld32(s_at + 64, x);
          scaled(y, 1);
          top = highest(y, top);
          ptx::tmem_wait_ld();
          tmem_ld32(s_at + 96, y);
          scaled(x, 2);
          top = highest(x, top);
          ptx::tmem_wait_ld();
          scaled(y, 3);
          raise(highest(y, top));
          weigh(x, 2, std::false_type(), 0u, 0u);
          tmem_ld32(s_at, x);
          weigh(y, 3, std::false_type(), 0u, 0u);
          ptx::tmem_wait_ld();
          tmem_ld32(s_at + 32, y);
          scaled(x, 0);
          weigh(x, 0, std::false_type(), 0u, 0u);
          ptx::tmem_wait_ld();
          scaled(y, 1);
          weigh(y, 1, std::false_type(), 0u, 0u);
        } else if (mine) {
          auto word = [](const uint32_t (&w)[4], int c) { return c == 0 ? w[0] : c == 1 ? w[1] : c == 2 ? w[2] : w[3]; };
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32];
            tmem_ld32(s_at + 32 * c, x);
            ptx::tmem_wait_ld();
            scaled(x, c);
            const uint32_t keep = word(see, c);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (keep >> e & 1) top = fmaxf(top, __uint_as_float(x[e]));
          }
          raise(top);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32];
            tmem_ld32(s_at + 32 * c, x);
            ptx::tmem_wait_ld();
            scaled(x, c);
            weigh(x, c, std::true_type(), word(see, c), word(bad, c));
          }
        }
        if (mine) {
          l += sum.x + sum.y;
          ptx::tmem_wait_st();
        }
        first = false;
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars.p_ready[slot]);
        ++steps;
      }

      // ---- the head's end in this share
      const bool whole = seg.whole();
      wait(&bars.o_full, seg.index);
      ptx::tc_fence_after();
      float* const part = part_at<D>(a, (int)blockIdx.x, seg.at > share.at ? 1 : 0);
      const int pr = row + (TWO ? slot * kTile : 0);   // the row in a part
      const int64_t to = (bh * a.group + g) * a.tokens + token;
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
      auto write = [&](int c, const float (&x)[32]) {   // channels c .. c + 31 of this thread's row
        if (row >= rows) return;
        if (whole) {
          uint4* const u = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + to * D + c);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            u[e] = make_uint4(pack2(x[8 * e], x[8 * e + 1]), pack2(x[8 * e + 2], x[8 * e + 3]), pack2(x[8 * e + 4], x[8 * e + 5]), pack2(x[8 * e + 6], x[8 * e + 7]));
        } else {
          float4* const u = reinterpret_cast<float4*>(part + (int64_t)pr * D + c);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
        }
      };
      if constexpr (TWO) {
        if (mine) {
          const float scale = finish(m, l);
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t x[32];
            float y[32];
            tmem_ld32(o_lane + S::kO(slot) + c, x);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(x[e]) * scale;
            write(c, y);
          }
        }
      } else {
        // the two slots' halves of the keys meet; each slot writes half of the channels
        const bool other = seg.tiles > 1;   // (of one tile, one slot has none)
        const int only = (int)(done & 1);   // the first tile's slot
        if (slot == 1) meet[row] = make_float2(m, l);
        ptx::named_barrier(3, 256);
        float2 f;
        if (slot == 0) {
          const float2 y = meet[row];
          const float top = fmaxf(m, y.x), f0 = rescale(m, top), f1 = rescale(y.x, top);
          const float scale = finish(top, fmaf(l, f0, y.y * f1));
          f = make_float2(f0 * scale, f1 * scale);
          meet[row] = f;
        }
        ptx::named_barrier(3, 256);
        if (slot == 1) f = meet[row];
        if (mine) {
#pragma unroll
          for (int c = slot * (D / 2); c < (slot + 1) * (D / 2); c += 32) {
            uint32_t x[32];
            float y[32];
            tmem_ld32(o_lane + S::kO(other ? 0 : only) + c, x);
            ptx::tmem_wait_ld();
            const float fx = other || only == 0 ? f.x : f.y;
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(x[e]) * fx;
            if (other) {
              tmem_ld32(o_lane + S::kO(1) + c, x);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = fmaf(__uint_as_float(x[e]), f.y, y[e]);
            }
            write(c, y);
          }
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars.o_free);
      done += (uint32_t)seg.tiles;
    } while (seg.next(a));
  } else if constexpr (Q8) {
    // ---- codes into bf16 tiles: a thread per key
    const int key = tid - 12 * 32;
    Segments ks(a, share), vs(a, share);
    int kf = 0, vf = 0;
    uint32_t made = 0, used = 0;       // tiles made, and raw ones used
    auto make = [&](Segments& s, int& f, bool is_key) {
      const uint32_t slot = made % kStages, turn = made / kStages;
      const int tile = s.p.tile + f;
      const int64_t bh = (int64_t)s.p.seq * a.heads + s.p.head;
      const bool cached = tile < s.p.s.cache_tiles;
      uint8_t* const to = smem + S::kRing + slot * S::kStage;
      if (cached) {
        const uint32_t at = used % kRaws;
        wait(&bars.raw_full[at], used / kRaws);
        const uint8_t* const from = smem + S::kRawRing + at * S::kRaw;
        const bool there = key < s.p.s.rows - tile * kTile;
        uint4 w[D / 16];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint32_t off = D == 128 ? key * 128 + ((c ^ (key & 7)) << 4) : key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
          w[c] = there ? *reinterpret_cast<const uint4*>(from + off) : make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars.raw_empty[at]);
        ++used;
        if (turn > 0) wait(&bars.kv_empty[slot], turn - 1);
        auto low = [](uint32_t x) { return prmt(x, x, 0x1100) & 0x807F807Fu; };
        auto high = [](uint32_t x) { return prmt(x, x, 0x3322) & 0x807F807Fu; };
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          *reinterpret_cast<uint4*>(to + piece_at(key, 2 * c)) = make_uint4(low(w[c].x), high(w[c].x), low(w[c].y), high(w[c].y));
          *reinterpret_cast<uint4*>(to + piece_at(key, 2 * c + 1)) = make_uint4(low(w[c].z), high(w[c].z), low(w[c].w), high(w[c].w));
        }
      } else {
        const int row = (tile - s.p.s.cache_tiles) * kTile + key;
        const bool there = row < s.p.s.n;
        const __nv_bfloat16* const from = static_cast<const __nv_bfloat16*>(is_key ? a.k_new : a.v_new) + (bh * a.tokens + (there ? row : 0)) * D;
        if (turn > 0) wait(&bars.kv_empty[slot], turn - 1);
#pragma unroll 8
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<uint4*>(to + piece_at(key, c)) = there ? ld_nc_v4(from + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars.kv_full[slot]);
      ++made;
      if (++f == s.tiles) {
        f = 0;
        s.next(a);
      }
    };
    make(ks, kf, true);
    if (!TWO && total > 1) make(ks, kf, true);
    for (int64_t t = 0; t < total && !__any_sync(0xffffffffu, aborted()); ++t) {   // (all of a warp leave together)
      make(vs, vf, false);
      if (t + (TWO ? 1 : 2) < total) make(ks, kf, true);
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
  return err != cudaSuccess ? err : launch_tree_join<__nv_bfloat16, D, kTile, kTile>(a, job.stream);
}

template <bool Q8, int D> cudaError_t launch_dim(const TreeJob& job) {
  return job.q_heads / job.heads * job.tokens <= 128 ? launch_typed<Q8, D, false>(job) : launch_typed<Q8, D, true>(job);
}

}  // namespace

cudaError_t launch_tree_tc(const TreeJob& job) {
  if (job.k_step) return job.head_dim == 64 ? launch_dim<true, 64>(job) : launch_dim<true, 128>(job);
  return job.head_dim == 64 ? launch_dim<false, 64>(job) : launch_dim<false, 128>(job);
}

}  // namespace snapkv
