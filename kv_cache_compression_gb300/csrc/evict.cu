// In-place eviction by accumulated attention: the heaviest rows and the newest ones stay.
//
// One thread-block cluster per (sequence, head). The candidates' scores (slots below n = len - recent)
// become 32-bit keys whose unsigned order is the scores' order; each CTA keeps its span's keys in
// shared memory where they fit. A radix select (four 8-bit digits, histograms added up through
// distributed shared memory) finds the key of rank `keep`; ties at it go to the lower slots. A scan in
// slot order then lists the freed slots below `keep` and the staying rows above it, and the i-th of
// the one takes the i-th of the other.
//
// In-place order of moves. Freed slots are nobody's source and the rows they take lie at or above
// `keep`, so those moves need no order among themselves. The newest rows then come down by
// E = n - keep slots, which may overlap their old place: every CTA of the cluster has its own 16-byte
// columns of the rows (columns never meet), loads a batch of rows, waits for its threads, stores it, and
// goes on upwards; a batch's stores land below every later load.
//
// The bytes are few (4 per candidate's score, and the rows that change their slot), so the kernel is
// bound by HBM only for many heads; otherwise by the latency of its steps.
#include "cache_internal.h"
#include "sm100_ptx.cuh"
#include "snapkv_common.cuh"
#include "snapkv_internal.h"

namespace snapkv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kKeysSmem = 64 * 1024;   // a span's keys stay in shared memory up to this size
constexpr int kMaxIndex = kThreads;    // pairs resolved at a time

struct EvictArgs {
  EvictJob j;
  int keys_in_smem;
};

// Unsigned order = order of the scores; NaN lowest, -0 = +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sum over the block's threads of v, in thread order; *total is the block's sum. `sums` holds
// kWarps + 1 values; the caller syncs between two uses of the same one.
__device__ __forceinline__ int block_scan(int v, int* sums, int* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = lane < kWarps ? sums[lane] : 0;
#pragma unroll
    for (int off = 1; off < kWarps; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += y;
    }
    if (lane < kWarps) sums[lane] = s;
  }
  __syncthreads();
  *total = sums[kWarps - 1];
  return x - v + (warp ? sums[warp - 1] : 0);
}

template <int ROW, int META>
__global__ void __launch_bounds__(kThreads) evict_kernel(EvictArgs args) {
  const EvictJob& j = args.j;
  constexpr int kPieces = ROW / 16;       // 16-byte pieces of a row of K (and of V)
  extern __shared__ uint32_t key_smem[];
  __shared__ uint32_t hist[4][256];       // one per digit, read by the whole cluster
  __shared__ uint32_t all[256];
  __shared__ uint32_t pick_digit, pick_left;
  __shared__ int counts[3];               // ties, freed slots, staying rows of this CTA's span
  __shared__ int sums_a[kWarps + 1], sums_b[kWarps + 1];
  __shared__ int first_free[kMaxCluster + 1], first_stay[kMaxCluster + 1];
  __shared__ int pair_to[kMaxIndex], pair_from[kMaxIndex];

  const int tid = threadIdx.x;
  const uint32_t rank = ptx::cluster_rank(), csize = ptx::cluster_size();
  const int64_t bh = blockIdx.x / csize;
  const int b = (int)(bh / j.heads);
  const bool first = bh % j.heads == 0 && rank == 0 && tid == 0;
  int len = j.len[b];
  if ((int64_t)len > j.cap) {
    if (first) report(j.dev_status, SNAPKV_ERR_CAPACITY);
    len = (int)j.cap;
  }
  if (len < 0) len = 0;
  const int keep = (int)j.keep, recent = (int)j.recent, left = keep + recent;
  if (first) j.len_out[b] = len > left ? left : len;
  int32_t* idx = j.idx ? j.idx + bh * left : nullptr;
  if (len <= left) {   // the whole cluster agrees
    if (idx)
      for (int s = (int)rank * kThreads + tid; s < left; s += (int)csize * kThreads) idx[s] = s;
    return;
  }
  const int n = len - recent;
  float* score = j.score + bh * j.cap;
  int32_t* slots = j.slots + bh * j.cap;
  const int per = (n + (int)csize - 1) / (int)csize;
  const int s0 = min((int64_t)n, (int64_t)rank * per), s1 = min((int64_t)n, (int64_t)s0 + per);

  for (int i = tid; i < 4 * 256; i += kThreads) (&hist[0][0])[i] = 0;
  if (tid < 3) counts[tid] = 0;
  if (args.keys_in_smem)
    for (int s = s0 + tid; s < s1; s += kThreads) key_smem[s - s0] = order_key(score[s]);
  __syncthreads();
  auto key_of = [&](int s) { return args.keys_in_smem ? key_smem[s - s0] : order_key(score[s]); };

  // ---- the key of rank `keep` from the top, digit by digit; `want` of the keys that share the digits
  // found so far are kept. (keep = 0: nothing is, whatever the digits.)
  uint32_t prefix = 0, want = (uint32_t)keep;
  for (int d = 3; d >= 0; --d) {
    const int shift = 8 * d;
    for (int s = s0 + tid; s < s1; s += kThreads) {
      const uint32_t key = key_of(s);
      if (d == 3 || key >> (shift + 8) == prefix) atomicAdd(&hist[d][(key >> shift) & 255u], 1u);
    }
    ptx::cluster_sync();
    if (tid < 256) {
      uint32_t x = 0;
      for (uint32_t r = 0; r < csize; ++r) x += ptx::dsmem_ld_u32(ptx::map_rank(&hist[d][tid], r));
      all[tid] = x;
    }
    __syncthreads();
    if (tid < 32) {   // eight bins a lane, from the top
      uint32_t mine = 0;
      for (int i = 0; i < 8; ++i) mine += all[255 - (8 * tid + i)];
      uint32_t upto = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, upto, off);
        if (tid >= off) upto += y;
      }
      uint32_t above = upto - mine;
      if (want > above && want <= upto)
        for (int i = 0; i < 8; ++i) {
          const uint32_t bin = 255 - (8 * tid + i);
          if (want <= above + all[bin]) {
            pick_digit = bin;
            pick_left = want - above;
            break;
          }
          above += all[bin];
        }
      if (keep == 0 && tid == 0) {
        pick_digit = 255;
        pick_left = 0;
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | pick_digit;
    want = pick_left;
  }

  // ---- ties before this span
  {
    int mine = 0;
    for (int s = s0 + tid; s < s1; s += kThreads) mine += key_of(s) == prefix;
    if (mine) atomicAdd(&counts[0], mine);
  }
  ptx::cluster_sync();
  int ties = 0;
  for (uint32_t r = 0; r < rank; ++r) ties += (int)ptx::dsmem_ld_u32(ptx::map_rank(&counts[0], r));

  // ---- in slot order: freed slots below `keep` are listed from the front of the span's part of
  // `slots`, staying rows at or above it from its back.
  int n_free = 0, n_stay = 0;
  for (int base = s0; base < s1; base += kThreads) {
    const int s = base + tid;
    const uint32_t key = s < s1 ? key_of(s) : 0u;
    const bool tie = s < s1 && key == prefix;
    int tie_total, total;
    const int tie_rank = ties + block_scan(tie, sums_a, &tie_total);
    const bool stays = s < s1 && (key > prefix ? keep > 0 : tie && tie_rank < (int)want);
    const bool frees = s < s1 && !stays && s < keep, above = stays && s >= keep;
    // two counts in one scan: both are at most kThreads
    const int at = block_scan((int)frees | ((int)above << 16), sums_b, &total);
    if (frees) slots[s0 + n_free + (at & 0xFFFF)] = s;
    if (above) slots[s1 - 1 - (n_stay + (at >> 16))] = s;
    if (idx && stays && s < keep) idx[s] = s;
    ties += tie_total;
    n_free += total & 0xFFFF;
    n_stay += total >> 16;
  }
  if (tid == 0) {
    counts[1] = n_free;
    counts[2] = n_stay;
  }
  ptx::cluster_sync();   // also makes the lists of the other CTAs visible
  if (tid <= (int)csize) {
    int f = 0, t = 0;
    for (int r = 0; r < tid; ++r) {
      f += (int)ptx::dsmem_ld_u32(ptx::map_rank(&counts[1], (uint32_t)r));
      t += (int)ptx::dsmem_ld_u32(ptx::map_rank(&counts[2], (uint32_t)r));
    }
    first_free[tid] = f;
    first_stay[tid] = t;
  }
  __syncthreads();

  // ---- the i-th freed slot takes the i-th staying row; pairs are shared out evenly over the CTAs
  const int pairs = min(first_free[csize], first_stay[csize]);   // (equal)
  const int p_per = (pairs + (int)csize - 1) / (int)csize;
  const int p0 = min(pairs, (int)rank * p_per), p1 = min(pairs, p0 + p_per);
  for (int base = p0; base < p1; base += kMaxIndex) {
    const int count = min(kMaxIndex, p1 - base);
    if (tid < count) {
      const int p = base + tid;
      int rf = 0, rs = 0;
      while (p >= first_free[rf + 1]) ++rf;
      while (p >= first_stay[rs + 1]) ++rs;
      const int e1 = min((int64_t)n, (int64_t)(rs + 1) * per);   // end of that CTA's span
      const int to = __ldcg(slots + (int64_t)rf * per + (p - first_free[rf]));
      const int from = __ldcg(slots + e1 - 1 - (p - first_stay[rs]));
      const bool ok = in_bounds(to >= 0 && to < keep && from >= keep && from < n, j.dev_status);
      pair_to[tid] = ok ? to : 0;
      pair_from[tid] = ok ? from : 0;
      score[pair_to[tid]] = score[pair_from[tid]];
      if (idx) idx[pair_to[tid]] = pair_from[tid];
      if constexpr (META > 0) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          uint8_t* meta = static_cast<uint8_t*>(j.meta[kv]) + bh * j.cap * META;
          if constexpr (META == 8)
            reinterpret_cast<uint2*>(meta)[pair_to[tid]] = reinterpret_cast<const uint2*>(meta)[pair_from[tid]];
          else
            reinterpret_cast<uint32_t*>(meta)[pair_to[tid]] = reinterpret_cast<const uint32_t*>(meta)[pair_from[tid]];
        }
      }
    }
    __syncthreads();
    constexpr int kUnroll = 4;
    const int items = count * 2 * kPieces;
    for (int u0 = tid; u0 < items; u0 += kUnroll * kThreads) {
      uint4 x[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int u = u0 + i * kThreads;
        if (u < items) {
          const int p = u / (2 * kPieces), kv = (u / kPieces) & 1, c = u % kPieces;
          x[i] = static_cast<const uint4*>(j.rows[kv])[(bh * j.cap + pair_from[p]) * kPieces + c];
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int u = u0 + i * kThreads;
        if (u < items) {
          const int p = u / (2 * kPieces), kv = (u / kPieces) & 1, c = u % kPieces;
          static_cast<uint4*>(j.rows[kv])[(bh * j.cap + pair_to[p]) * kPieces + c] = x[i];
        }
      }
    }
    __syncthreads();
  }
  ptx::cluster_sync();   // every staying row has left its old place

  // ---- the newest rows: slots n .. len - 1 come down to keep .. left - 1
  {
    // This CTA's columns: pieces rank, rank + csize, ... of the 2 * kPieces of a row's K and V.
    const int mine = (2 * kPieces - (int)rank + (int)csize - 1) / (int)csize;
    if (mine > 0) {
      constexpr int kUnroll = 4;
      const int batch = kThreads / mine * kUnroll;   // rows at a time (2 * kPieces <= 64 < kThreads)
      const int lane_row = tid / mine, lane_col = (int)rank + (int)csize * (tid % mine);
      const int kv = lane_col / kPieces, c = lane_col % kPieces;
      const bool active = lane_row < kThreads / mine;
      uint4* rows = static_cast<uint4*>(j.rows[active ? kv : 0]) + bh * j.cap * kPieces + c;
      for (int base = 0; base < recent; base += batch) {
        uint4 x[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          const int r = base + lane_row + i * (kThreads / mine);
          if (active && r < recent) x[i] = rows[(int64_t)(n + r) * kPieces];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          const int r = base + lane_row + i * (kThreads / mine);
          if (active && r < recent) rows[(int64_t)(keep + r) * kPieces] = x[i];
        }
      }
    }
  }
  if (rank == csize - 1) {   // scores, (h, z) pairs and indices are small: one CTA
    for (int base = 0; base < recent; base += kThreads) {
      const int r = base + tid;
      float x = 0.f;
      uint2 m[2] = {};
      if (r < recent) {
        x = score[n + r];
        if (idx) idx[keep + r] = n + r;
        if constexpr (META > 0) {
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint8_t* meta = static_cast<const uint8_t*>(j.meta[kv]) + bh * j.cap * META;
            if constexpr (META == 8)
              m[kv] = reinterpret_cast<const uint2*>(meta)[n + r];
            else
              m[kv].x = reinterpret_cast<const uint32_t*>(meta)[n + r];
          }
        }
      }
      __syncthreads();
      if (r < recent) {
        score[keep + r] = x;
        if constexpr (META > 0) {
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            uint8_t* meta = static_cast<uint8_t*>(j.meta[kv]) + bh * j.cap * META;
            if constexpr (META == 8)
              reinterpret_cast<uint2*>(meta)[keep + r] = m[kv];
            else
              reinterpret_cast<uint32_t*>(meta)[keep + r] = m[kv].x;
          }
        }
      }
    }
    __syncthreads();
    for (int s = left + tid; s < len; s += kThreads) score[s] = 0.f;
  }
  ptx::cluster_sync();   // no CTA leaves while its counts may still be read
}

template <int ROW, int META> cudaError_t launch_typed(const EvictJob& job) {
  const int64_t bh = (int64_t)job.batch * job.heads;
  // CTAs per head: up to one per 2048 candidates, while all heads together fill two per SM.
  int64_t csize = 2 * (int64_t)device_sm_count() / bh;
  const int64_t most = (job.cap + 2047) / 2048;
  if (csize > most) csize = most;
  if (csize > kMaxCluster) csize = kMaxCluster;
  if (csize < 1) csize = 1;
  const int64_t key_bytes = (job.cap + csize - 1) / csize * 4;
  EvictArgs a;
  a.j = job;
  a.keys_in_smem = key_bytes <= kKeysSmem;
  const cudaError_t err = allow_dynamic_smem<evict_kernel<ROW, META>>(kKeysSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(bh * csize));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = a.keys_in_smem ? (size_t)key_bytes : 0;
  cfg.stream = job.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)csize;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel<ROW, META>, a);
}

}  // namespace

cudaError_t launch_evict(const EvictJob& job) {
  switch (job.row_bytes) {   // d = 64 or 128 in 4 bits, bf16 or fp32
    case 32: return launch_typed<32, 4>(job);
    case 64: return launch_typed<64, 8>(job);
    case 128: return launch_typed<128, 0>(job);
    case 256: return launch_typed<256, 0>(job);
    case 512: return launch_typed<512, 0>(job);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace snapkv
