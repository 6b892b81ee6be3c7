// In-place eviction by accumulated attention: the heaviest rows and the newest ones stay.
//
// A CTA per (sequence, head), or a thread-block cluster for long caches of few heads. The candidates'
// scores (slots below n = len - recent) become 32-bit keys whose unsigned order is the scores' order;
// each CTA keeps its span's keys in shared memory where they fit. A radix select (four 8-bit digits,
// histograms added up through distributed shared memory in a cluster) finds the key of rank `keep`; ties
// at it go to the lower slots. A scan in slot order then lists the freed slots below `keep` and the staying
// rows above it, and the i-th of the one takes the i-th of the other.
//
// In-place order of moves. Freed slots are nobody's source and the rows they take lie at or above
// `keep`, so those moves need no order among themselves. The newest rows then come down by
// E = n - keep slots, which may overlap their old place: every CTA of the cluster has its own 16-byte
// columns of the rows (columns never meet), loads a batch of rows, waits for its threads, stores it, and
// goes on upwards; a batch's stores land below every later load.
//
// The bytes are few: 4 per candidate's score, and the rows that change their slot. Selection (with the newest rows) and the
// other moves, measured apart by shuffling heavy scores below slot `keep` and light ones above it (GB300; in brackets the
// floor of both at 6.79 TB/s):
//   2048 heads of 2208 bf16 rows of 128 channels, 128 leave:   33 us, and  40 for 250 MB  [52]
//   32 heads of 131072 such rows, an eighth leaves:            30 us, and  90 for 470 MB  [75]
//   512 heads of 65536 rows of 64 channels, 1504 leave:       132 us, and 115 for 385 MB  [93]
// The selection's instructions and the latency of its steps show, with six CTAs per SM to hide them in the batch and
// clusters of eight over the long caches. The moves run at 6.2, 5.2 and 3.3 TB/s: rows of 256 or 128 bytes that lie far
// apart. (Over the 32 long caches, clusters of sixteen or blocks of 1024 threads no longer fit the GPU at once and take
// 200 us.) 4-bit rows: 2048 heads of 2208 58 us [19]; 4 heads of 97 6.9 us.
#include "cache_internal.h"
#include "sm100_ptx.cuh"
#include "snapkv_common.cuh"
#include "snapkv_internal.h"

namespace snapkv {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kKeysSmem = 96 * 1024;   // a span's keys stay in shared memory up to this size (two CTAs per SM)
constexpr int kMaxIndex = 1024;        // pairs resolved at a time
static_assert(kEvictNoListCap <= 2 * kMaxIndex, "min(keep, n - keep) pairs at most");
constexpr int kRun = 15;               // keys a thread looks at between two scans, at most (odd: no bank conflicts)

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

// Exclusive sum over the block's threads of v, in thread order; *total is the block's sum. The caller
// syncs between two uses of `sums`.
template <int WARPS> __device__ __forceinline__ int block_scan(int v, int* sums, int* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const int y = sums[w];
    if (w < warp) before += y;
    all += y;
  }
  *total = all;
  return before + x - v;
}

template <int ROW, int META, int THREADS>
__global__ void __launch_bounds__(THREADS) evict_kernel(EvictArgs args) {
  const EvictJob& j = args.j;
  constexpr int kPieces = ROW / 16;       // 16-byte pieces of a row of K (and of V)
  constexpr int kWarps = THREADS / 32;
  extern __shared__ uint32_t key_smem[];
  __shared__ __align__(16) uint32_t hist[4][256];       // one per digit, read by the whole cluster
  __shared__ __align__(16) uint32_t all[256];
  __shared__ uint32_t found[3];           // a digit, how many keys of it are kept, and of how many
  __shared__ int listed;
  __shared__ int counts[3];               // ties, freed slots, staying rows of this CTA's span
  __shared__ int sums_a[kWarps], sums_b[kWarps];
  __shared__ int first_free[kMaxCluster + 1], first_stay[kMaxCluster + 1];
  __shared__ int pair_to[kMaxIndex], pair_from[kMaxIndex];

  const int tid = threadIdx.x, lane = tid % 32;
  const uint32_t rank = ptx::cluster_rank(), csize = ptx::cluster_size();
  const bool alone = csize == 1;
  auto sync_head = [&] {   // all CTAs of the head
    if (alone)
      __syncthreads();
    else
      ptx::cluster_sync();
  };
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
      for (int s = (int)rank * THREADS + tid; s < left; s += (int)csize * THREADS) idx[s] = s;
    return;
  }
  const int n = len - recent;
  float* score = j.score + bh * j.cap;
  int32_t* slots = j.slots + bh * j.cap;
  const int per = (n + (int)csize - 1) / (int)csize;
  const int s0 = min((int64_t)n, (int64_t)rank * per), s1 = min((int64_t)n, (int64_t)s0 + per);

  int* list = pair_to;        // (free until the pairs are)
  uint32_t among_16 = 0;
  // The keys arrive while the histograms are cleared; the first digit is counted from them on the way.
  if (tid < 3) counts[tid] = 0;
  if (tid == 0) listed = 0;
  for (int i = tid; i < 4 * 256; i += THREADS) (&hist[0][0])[i] = 0;
  __syncthreads();
  auto key_of = [&](int s) { return args.keys_in_smem ? key_smem[s - s0] : order_key(score[s]); };
#pragma unroll 8
  for (int s = s0 + tid; s < s1; s += THREADS) {
    const uint32_t key = order_key(score[s]);
    if (args.keys_in_smem) key_smem[s - s0] = key;
    atomicAdd(&hist[3][key >> 24], 1u);
  }

  // ---- the key of rank `keep` from the top, digit by digit; `want` of the keys that share the digits
  // found so far are kept, of `among`. (keep = 0: none, and the search runs to the largest key.)
  uint32_t prefix = 0, want = (uint32_t)keep, among = (uint32_t)n;
  for (int d = 3; d >= 0; --d) {
    const int shift = 8 * d;
    auto count = [&](uint32_t key) { atomicAdd(&hist[d][(key >> shift) & 255u], 1u); };
    if (d == 0 && among_16 <= (uint32_t)kMaxIndex) {
      for (int i = tid; i < listed; i += THREADS)
        if ((uint32_t)list[i] >> 8 == prefix) count((uint32_t)list[i]);
    } else if (d < 3) {
      if (d == 1) among_16 = among;   // few keys share two digits: they are listed for the last one
      const bool keep_list = d == 1 && among <= (uint32_t)kMaxIndex;
      for (int s = s0 + tid; s < s1; s += THREADS) {
        const uint32_t key = key_of(s);
        if (key >> (shift + 8) == prefix) {
          count(key);
          if (keep_list) {
            const int at = atomicAdd(&listed, 1);
            if (in_bounds(at < kMaxIndex, j.dev_status)) list[at] = (int)key;
          }
        }
      }
    }
    sync_head();
    if (!alone) {
      for (int i = tid; i < 256; i += THREADS) {
        uint32_t x = 0;
        for (uint32_t r = 0; r < csize; ++r) x += ptx::dsmem_ld_u32(ptx::map_rank(&hist[d][i], r));
        all[i] = x;
      }
      __syncthreads();
    }
    if (tid < 32) {   // one warp finds the digit, eight bins a lane from the top
      const uint32_t* sum = alone ? hist[d] : all;
      const uint4 hi = *reinterpret_cast<const uint4*>(&sum[252 - 8 * lane]), lo = *reinterpret_cast<const uint4*>(&sum[248 - 8 * lane]);
      const uint32_t bins[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += bins[i];
      uint32_t above = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, above, off);
        if (lane >= off) above += y;
      }
      above -= mine;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (want > above && want <= above + bins[i]) {
          found[0] = 255 - (8 * lane + i);
          found[1] = want - above;
          found[2] = bins[i];
        }
        above += bins[i];
      }
      if (keep == 0 && lane == 0) {
        found[0] = 255;
        found[1] = found[2] = 0;
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | found[0];
    want = found[1];
    among = found[2];
    // (`found` and `all` are written again behind the next digit's first barrier)
  }

  // ---- ties before this span, where not all of them stay
  const bool rank_ties = want < among;
  int ties = 0;
  if (!alone && rank_ties) {
    int mine = 0;
    for (int s = s0 + tid; s < s1; s += THREADS) mine += key_of(s) == prefix;
    if (mine) atomicAdd(&counts[0], mine);
    ptx::cluster_sync();
    for (uint32_t r = 0; r < rank; ++r) ties += (int)ptx::dsmem_ld_u32(ptx::map_rank(&counts[0], r));
  }

  // ---- in slot order: freed slots below `keep` are listed from the front, staying rows at or above it
  // from the back of the span's part of `slots` (or, few pairs of one CTA, in shared memory).
  const bool in_smem = alone && min(keep, n - keep) <= kMaxIndex;
  if (idx)   // slots that keep their row; the pairs below overwrite the others
    for (int s = s0 + tid; s < min(s1, keep); s += THREADS) idx[s] = s;
  const int run = min(kRun, (s1 - s0 + THREADS - 1) / THREADS | 1);   // neighbouring slots of a thread
  int n_free = 0, n_stay = 0;
  for (int base = s0; base < s1; base += run * THREADS) {
    const int t0 = min((int64_t)s1, (int64_t)base + tid * run), t1 = min((int64_t)s1, (int64_t)t0 + run);
    int tie_rank = 0;
    if (rank_ties) {
      int mine = 0, tie_total;
      for (int s = t0; s < t1; ++s) mine += key_of(s) == prefix;
      tie_rank = ties + block_scan<kWarps>(mine, sums_a, &tie_total);
      ties += tie_total;
    }
    uint32_t marks = 0;   // slots of the run to list: freed below `keep`, staying above
    int mine = 0, total;
    for (int s = t0; s < t1; ++s) {
      const uint32_t key = key_of(s);
      bool stay = key > prefix;
      if (key == prefix) {
        stay = want > 0 && (!rank_ties || tie_rank < (int)want);
        ++tie_rank;
      }
      if (stay != (s < keep)) {
        marks |= 1u << (s - t0);
        mine += stay ? 1 << 16 : 1;   // two counts of at most run * THREADS < 2^15
      }
    }
    int at = block_scan<kWarps>(mine, sums_b, &total);
    for (; marks; marks &= marks - 1) {
      const int s = t0 + __ffs(marks) - 1;
      if (s < keep) {
        const int p = n_free + (at & 0xFFFF);
        if (!in_bounds(p < (in_smem ? kMaxIndex : s1 - s0), j.dev_status)) break;
        if (in_smem)
          pair_to[p] = s;
        else
          slots[s0 + p] = s;
        at += 1;
      } else {
        const int p = n_stay + (at >> 16);
        if (!in_bounds(p < (in_smem ? kMaxIndex : s1 - s0), j.dev_status)) break;
        if (in_smem)
          pair_from[p] = s;
        else
          slots[s1 - 1 - p] = s;
        at += 1 << 16;
      }
    }
    n_free += total & 0xFFFF;
    n_stay += total >> 16;
    __syncthreads();   // the scans' sums are free again
  }
  if (alone) {
    if (tid == 0) {
      first_free[0] = first_stay[0] = 0;
      first_free[1] = n_free;
      first_stay[1] = n_stay;
    }
    __syncthreads();
  } else {
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
  }

  // ---- the i-th freed slot takes the i-th staying row; pairs are shared out evenly over the CTAs
  const int pairs = min(first_free[csize], first_stay[csize]);   // (equal)
  const int p_per = (pairs + (int)csize - 1) / (int)csize;
  const int p0 = min(pairs, (int)rank * p_per), p1 = min(pairs, p0 + p_per);
  for (int base = p0; base < p1; base += kMaxIndex) {
    const int count = min(kMaxIndex, p1 - base);
    for (int t = tid; t < count; t += THREADS) {
      int to, from;
      if (in_smem) {
        to = pair_to[t];
        from = pair_from[t];
      } else {
        const int p = base + t;
        int rf = 0, rs = 0;
        while (p >= first_free[rf + 1]) ++rf;
        while (p >= first_stay[rs + 1]) ++rs;
        const int e1 = min((int64_t)n, (int64_t)(rs + 1) * per);   // end of that CTA's span
        to = __ldcg(slots + (int64_t)rf * per + (p - first_free[rf]));
        from = __ldcg(slots + e1 - 1 - (p - first_stay[rs]));
      }
      const bool ok = in_bounds(to >= 0 && to < keep && from >= keep && from < n, j.dev_status);
      pair_to[t] = ok ? to : 0;
      pair_from[t] = ok ? from : 0;
      score[pair_to[t]] = score[pair_from[t]];
      if (idx) idx[pair_to[t]] = pair_from[t];
      if constexpr (META > 0) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          uint8_t* meta = static_cast<uint8_t*>(j.meta[kv]) + bh * j.cap * META;
          if constexpr (META == 8)
            reinterpret_cast<uint2*>(meta)[pair_to[t]] = reinterpret_cast<const uint2*>(meta)[pair_from[t]];
          else
            reinterpret_cast<uint32_t*>(meta)[pair_to[t]] = reinterpret_cast<const uint32_t*>(meta)[pair_from[t]];
        }
      }
    }
    __syncthreads();
    // A thread has one 16-byte column of K or V (two where a row of both has 64), and every kStep-th pair.
    constexpr int kCols = 2 * kPieces < 64 ? 2 * kPieces : 32;
    constexpr int kStep = THREADS / kCols, kUnroll = 4;
    const int first_pair = tid / kCols;
#pragma unroll
    for (int half = 0; half < 2 * kPieces / kCols; ++half) {
      const int col = half * kCols + tid % kCols, kv = col / kPieces;
      uint4* rows = static_cast<uint4*>(kv ? j.rows[1] : j.rows[0]) + bh * j.cap * kPieces + col % kPieces;
      for (int p = first_pair; p < count; p += kUnroll * kStep) {
        uint4 x[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
          if (p + i * kStep < count) x[i] = rows[(int64_t)pair_from[p + i * kStep] * kPieces];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
          if (p + i * kStep < count) rows[(int64_t)pair_to[p + i * kStep] * kPieces] = x[i];
      }
    }
    __syncthreads();
  }
  sync_head();   // every staying row has left its old place

  // ---- the newest rows: slots n .. len - 1 come down to keep .. left - 1
  {
    // This CTA's columns: pieces rank, rank + csize, ... of the 2 * kPieces of a row's K and V.
    const int mine = (2 * kPieces - (int)rank + (int)csize - 1) / (int)csize;
    if (mine > 0) {
      constexpr int kUnroll = 4;
      const int batch = THREADS / mine * kUnroll;   // rows at a time (2 * kPieces <= 64 < THREADS)
      const int lane_row = tid / mine, lane_col = (int)rank + (int)csize * (tid % mine);
      const int kv = lane_col / kPieces, c = lane_col % kPieces;
      const bool active = lane_row < THREADS / mine;
      uint4* rows = static_cast<uint4*>(j.rows[active ? kv : 0]) + bh * j.cap * kPieces + c;
      for (int base = 0; base < recent; base += batch) {
        uint4 x[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          const int r = base + lane_row + i * (THREADS / mine);
          if (active && r < recent) x[i] = rows[(int64_t)(n + r) * kPieces];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
          const int r = base + lane_row + i * (THREADS / mine);
          if (active && r < recent) rows[(int64_t)(keep + r) * kPieces] = x[i];
        }
      }
    }
  }
  if (rank == csize - 1) {   // scores, (h, z) pairs and indices are small: one CTA
    for (int base = 0; base < recent; base += THREADS) {
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
    for (int s = left + tid; s < len; s += THREADS) score[s] = 0.f;
  }
  if (!alone) ptx::cluster_sync();   // no CTA leaves while its counts may still be read
}

template <int ROW, int META, int THREADS> cudaError_t launch_sized(const EvictJob& job, int64_t csize) {
  const int64_t bh = (int64_t)job.batch * job.heads;
  const int64_t key_bytes = (job.cap + csize - 1) / csize * 4;
  EvictArgs a;
  a.j = job;
  a.keys_in_smem = key_bytes <= kKeysSmem;
  const cudaError_t err = allow_dynamic_smem<evict_kernel<ROW, META, THREADS>>(kKeysSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(bh * csize));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = a.keys_in_smem ? (size_t)key_bytes : 0;
  cfg.stream = job.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)csize;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel<ROW, META, THREADS>, a);
}

template <int ROW, int META> cudaError_t launch_typed(const EvictJob& job) {
  const int64_t bh = (int64_t)job.batch * job.heads;
  // CTAs per head: up to one per 2048 candidates, while all heads together fill two per SM; and, up to about 600
  // heads, as many as hold all keys in shared memory, although they do not all run at once then: full caches of
  // 65536 bf16 rows of 64 channels, 512 heads, 244 us (291 with one CTA, which reads the scores six times),
  // 131072 rows, 256 heads, 275 (325). Beyond, heads in plenty hide the reads better: 2048 heads of 32768 rows
  // 434 us (502 with clusters), 1024 heads 236 (258).
  int64_t csize = 2 * (int64_t)device_sm_count() / bh;
  const int64_t most = (job.cap + kEvictNoListCap - 1) / kEvictNoListCap;
  if (csize > most) csize = most;
  const int64_t fit = (job.cap * 4 + kKeysSmem - 1) / kKeysSmem;
  if (bh <= 4 * (int64_t)device_sm_count() && csize < fit) csize = fit;
  if (csize > kMaxCluster) csize = kMaxCluster;
  if (csize < 1) csize = 1;
  return (job.cap + csize - 1) / csize <= 4096 ? launch_sized<ROW, META, 256>(job, csize)
                                               : launch_sized<ROW, META, 512>(job, csize);
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
