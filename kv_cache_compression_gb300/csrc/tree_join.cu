// The second launch of the tree attention: joins the parts of the heads that the first launch cut, and writes the
// rows that see nothing.
//
// Heads are cut where a share begins inside one. The first launch leaves a note for each of its shares; every warp reads the notes
// of all (320 at most) and takes its part of what there is to do. (A look at every query row, most of them finished, took longer than
// the joining: 37 us for 256 heads of two passes, 16 us for 2048 heads of six rows.) All latency: loads of several parts are
// under way at a time.
#include "tree_schedule.cuh"

#include "snapkv_internal.h"
#include "tree_launch.h"

namespace snapkv {
namespace {

using namespace tree;
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

// The shares that are the first to begin inside a head, as bits.
struct Notes {
  uint32_t word[kMaxTreeCtas / 32];
  int count;
  __device__ __forceinline__ Notes(const Args& a) : count(0) {
    const int lane = threadIdx.x % 32, shares = a.ctas / a.siblings;
    int tile[kMaxTreeCtas / 32];
#pragma unroll
    for (int w = 0; w < kMaxTreeCtas / 32; ++w) tile[w] = 32 * w + lane < shares ? __ldcg(&a.cuts[2 * (32 * w + lane)].w) : 0;
#pragma unroll
    for (int w = 0; w < kMaxTreeCtas / 32; ++w) {
      word[w] = __ballot_sync(0xffffffffu, tile[w] > 0);
      count += __popc(word[w]);
    }
  }
  __device__ __forceinline__ int share(int k) const {   // the k-th of them (the whole warp)
    uint32_t in = 0;
    int base = 0;
#pragma unroll
    for (int w = 0; w < kMaxTreeCtas / 32; ++w) {
      const int here = __popc(word[w]);
      if (k >= 0 && k < here) {
        in = word[w];
        base = 32 * w;
        break;
      }
      k -= here;
    }
    const int lane = threadIdx.x % 32;
    const uint32_t hit = __ballot_sync(0xffffffffu, (in >> lane & 1) && __popc(in & ((1u << lane) - 1u)) == k);
    return base + __ffs(hit) - 1;
  }
};

// A head (and pass) that was cut.
struct Cut {
  int seq, head, pass, n;
  int first, more;   // its first share, and how many others have parts of it
  int slot;          // of the first one's part
};
__device__ __forceinline__ bool cut_at(const Args& a, int64_t total, int shares, int c, Cut& cut) {
  const int4 note = __ldcg(a.cuts + 2 * c), rest = __ldcg(a.cuts + 2 * c + 1);
  cut.seq = note.x;
  cut.head = note.y;
  cut.pass = note.z;
  cut.n = rest.y;
  const int64_t f0 = share_start(total, shares, c) - note.w;
  cut.first = c - 1;
  cut.slot = share_start(total, shares, c - 1) < f0 ? 1 : 0;
  cut.more = share_of(total, shares, f0 + rest.x - 1) - (c - 1);
  return in_bounds(c > 0 && note.y < a.heads && cut.more >= 1 && c - 1 + cut.more < shares, a.dev_status);
}

// Tokens that are not there, and all of sequences without rows to see.
template <typename IO, int D, int TILE, int NEW> __device__ __forceinline__ void write_all_zeros(const Args& a) {
  const int q_heads = a.heads * a.group;
  for (int64_t v = blockIdx.x; v < (int64_t)a.batch * q_heads; v += gridDim.x) {
    const Seq s = seq_of<TILE, NEW>(a, (int)((uint32_t)v / (uint32_t)q_heads));
    write_zeros<IO, D, kJoinThreads>(a, v, s.tiles == 0 ? 0 : s.n);
  }
}

template <int D> struct Vec;
template <> struct Vec<64> { using T = float2; };
template <> struct Vec<128> { using T = float4; };

// Few rows a pass: a warp per row of the call, which finds the row's parts from the schedule (the notes would be one more load to wait
// for: 32 heads of 1057 rows take 16.4 us so, 20.1 with them); a part's maximum per lane, and eight parts' channels at a time.
template <typename IO, int D, int TILE, int NEW>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(Args a) {
  constexpr int kPer = D / 32;   // channels of a lane
  const int lane = threadIdx.x % 32;
  const uint32_t rows = (uint32_t)a.batch * a.heads * a.group * a.tokens;   // (2^22 at most)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t total = __ldcg(a.upto + a.batch);
  const int shares = working_shares(a, total);
  for (uint32_t at = blockIdx.x * kJoinWarps + threadIdx.x / 32; at < rows; at += gridDim.x * kJoinWarps) {
    const uint32_t hq = at / (uint32_t)a.tokens, bh = hq / (uint32_t)a.group, b = bh / (uint32_t)a.heads;
    const int t = (int)(at - hq * a.tokens), g = (int)(hq - bh * a.group), h = (int)(bh - b * a.heads);
    const Seq s = seq_of<TILE, NEW>(a, (int)b);
    if (t >= s.n || s.tiles == 0) continue;
    const int r = g * s.n + t, pass = r / a.tile_q, i = r - pass * a.tile_q;
    const int64_t f0 = __ldcg(a.upto + b) + ((int64_t)h * s.passes + (a.siblings > 1 ? 0 : pass)) * s.tiles;
    const int sib = a.siblings > 1 ? pass : 0;
    Cut cut;
    cut.first = share_of(total, shares, f0);
    cut.more = share_of(total, shares, f0 + s.tiles - 1) - cut.first;
    cut.slot = share_start(total, shares, cut.first) < f0 ? 1 : 0;
    if (cut.more == 0) continue;   // finished in the first launch
    if (!in_bounds(cut.first >= 0 && cut.first + cut.more < shares && i < a.tile_q, a.dev_status)) continue;
    auto part = [&](int k) { return part_at<D>(a, (cut.first + k) * a.siblings + sib, k == 0 ? cut.slot : 0); };
    float x[kPer] = {}, top = kNoMax, sum = 0.f;
    for (int k0 = 0; k0 <= cut.more; k0 += 32) {
      const int here = min(32, cut.more + 1 - k0);
      float m = kNoMax, l = 0.f;
      if (lane < here) {
        const float* p = part(k0 + lane) + (int64_t)a.tile_q * D + i;
        m = __ldcg(p);
        l = __ldcg(p + a.tile_q);
      }
      const float next = fmaxf(top, warp_max(m));
      const float f = rescale(m, next), old = rescale(top, next);
      top = next;
      sum = fmaf(sum, old, warp_sum(l * f));
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[e] *= old;
      for (int k = 0; k < here; k += 8) {
        typename Vec<D>::T v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (k + e < here) v[e] = __ldcg(reinterpret_cast<const typename Vec<D>::T*>(part(k0 + k + e) + (int64_t)i * D) + lane);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = __shfl_sync(0xffffffffu, f, (k + e) & 31);
          if (k + e < here) {
            const float* y = reinterpret_cast<const float*>(&v[e]);
#pragma unroll
            for (int q = 0; q < kPer; ++q) x[q] = fmaf(y[q], w, x[q]);
          }
        }
      }
    }
    const float scale = sum == 0.f ? 0.f : 1.0f / sum;   // a NaN stays one
    IO* out = static_cast<IO*>(a.out) + (int64_t)at * D + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; ++e) store1<IO>(out + e, x[e] * scale);
    if (a.lse && lane == 0) a.lse[at] = lse_of(top, sum);
  }
  write_all_zeros<IO, D, TILE, NEW>(a);
}

// Passes of many rows: a warp joins 32 rows (a lane each) and eight channels, four parts at a time.
template <int D, int TILE>
__global__ void __launch_bounds__(kJoinThreads) tree_join_wide_kernel(Args a) {
  constexpr int kC = 8, kAtOnce = 4;
  const int lane = threadIdx.x % 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t total = __ldcg(a.upto + a.batch);
  const int shares = working_shares(a, total);
  const Notes notes(a);
  const int per_head = (a.tile_q / 32) * (D / kC), units = notes.count * a.siblings * per_head;
  for (int u = (int)blockIdx.x * kJoinWarps + threadIdx.x / 32; u < units; u += (int)gridDim.x * kJoinWarps) {
    const int v = u / per_head, w = u - v * per_head, k = v / a.siblings, sib = v - k * a.siblings;
    const int c0 = w % (D / kC) * kC, i = w / (D / kC) * 32 + lane;
    Cut cut;
    if (!cut_at(a, total, shares, notes.share(k), cut)) continue;
    const int r = (a.siblings > 1 ? sib : cut.pass) * a.tile_q + i;
    if (r >= a.group * cut.n) continue;   // (the parts' other rows were not written)
    float x[kC] = {}, top = kNoMax, sum = 0.f;
    for (int k0 = 0; k0 <= cut.more; k0 += kAtOnce) {
      float y[kAtOnce][kC], m[kAtOnce], l[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const bool in = k0 + j <= cut.more;
        const float* const p = part_at<D>(a, (cut.first + (in ? k0 + j : cut.more)) * a.siblings + sib, k0 + j == 0 ? cut.slot : 0);
        m[j] = in ? __ldcg(p + (int64_t)a.tile_q * D + i) : kNoMax;
        l[j] = in ? __ldcg(p + (int64_t)a.tile_q * (D + 1) + i) : 0.f;
#pragma unroll
        for (int e = 0; e < kC; ++e) y[j][e] = in ? __ldcg(p + (int64_t)(c0 + e) * a.tile_q + i) : 0.f;
      }
      float next = top;
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) next = fmaxf(next, m[j]);
      const float old = rescale(top, next);
      top = next;
      sum *= old;
#pragma unroll
      for (int e = 0; e < kC; ++e) x[e] *= old;
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const float f = rescale(m[j], next);
        sum = fmaf(l[j], f, sum);
#pragma unroll
        for (int e = 0; e < kC; ++e) x[e] = fmaf(y[j][e], f, x[e]);
      }
    }
    const int g = r / cut.n, t = r - g * cut.n;
    const int64_t at = (((int64_t)cut.seq * a.heads + cut.head) * a.group + g) * a.tokens + t;
    const float scale = sum == 0.f ? 0.f : 1.0f / sum;   // a NaN stays one
    __nv_bfloat162 y[kC / 2];
#pragma unroll
    for (int e = 0; e < kC / 2; ++e) y[e] = __floats2bfloat162_rn(x[2 * e] * scale, x[2 * e + 1] * scale);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at * D + c0) = *reinterpret_cast<const uint4*>(y);
    if (a.lse && c0 == 0) a.lse[at] = lse_of(top, sum);
  }
  write_all_zeros<__nv_bfloat16, D, TILE, TILE>(a);
}

// Blocks for the units of work that there may be and for the heads that may have zeros, `per_sm` an SM at most.
cudaError_t launch_join(void (*kernel)(Args), const Args& a, int64_t units, int per_sm, cudaStream_t stream) {
  int64_t blocks = (units + kJoinWarps - 1) / kJoinWarps;
  const int64_t heads = (int64_t)a.batch * a.heads * a.group, most = per_sm * (int64_t)device_sm_count();
  if (blocks < heads && (a.n_new || blocks == 0)) blocks = heads;
  if (blocks < 1) blocks = 1;
  if (blocks > most) blocks = most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

template <typename IO, int D, int TILE, int NEW> cudaError_t launch_tree_join(const Args& a, cudaStream_t stream) {
  return launch_join(tree_join_kernel<IO, D, TILE, NEW>, a, (int64_t)a.batch * a.heads * a.group * a.tokens, 8, stream);
}

template <int D, int TILE> cudaError_t launch_tree_join_wide(const Args& a, cudaStream_t stream) {
  return launch_join(tree_join_wide_kernel<D, TILE>, a, (int64_t)(a.ctas - 1) * (a.tile_q / 32) * (D / 8), 2, stream);
}

#define INSTANCE(IO, D, TILE, NEW) template cudaError_t launch_tree_join<IO, D, TILE, NEW>(const Args&, cudaStream_t);
INSTANCE(float, 64, 64, 64)
INSTANCE(float, 128, 64, 64)
INSTANCE(__nv_bfloat16, 64, 32, 16)
INSTANCE(__nv_bfloat16, 128, 32, 16)
INSTANCE(__nv_bfloat16, 128, 16, 16)
#undef INSTANCE
template cudaError_t launch_tree_join_wide<64, 128>(const Args&, cudaStream_t);
template cudaError_t launch_tree_join_wide<128, 128>(const Args&, cudaStream_t);

}  // namespace snapkv
