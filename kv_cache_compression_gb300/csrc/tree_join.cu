// The second launch of the tree attention: joins the parts of the heads that the first launch cut, and writes the
// rows that see nothing. All latency: a warp takes a query row, finds its parts from the schedule, and has a part's
// maximum per lane and eight parts' channels under way at a time.
#include "tree_schedule.cuh"

#include "snapkv_internal.h"

namespace snapkv {
namespace {

using namespace tree;
constexpr int kJoinThreads = 256;

template <int D> struct Vec;
template <> struct Vec<64> { using T = float2; };
template <> struct Vec<128> { using T = float4; };

template <typename IO, int D, int TILE, int NEW>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(Args a) {
  constexpr int kPer = D / 32;   // channels of a lane
  const int lane = threadIdx.x % 32;
  const int64_t rows = (int64_t)a.batch * a.heads * a.group * a.tokens;
  const int64_t warps = (int64_t)gridDim.x * (kJoinThreads / 32);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t total = __ldcg(a.upto + a.batch);
  const int shares = working_shares(a, total);
  for (int64_t at = (int64_t)blockIdx.x * (kJoinThreads / 32) + threadIdx.x / 32; at < rows; at += warps) {
    const int64_t hq = at / a.tokens;
    const int t = (int)(at - hq * a.tokens);
    const int bh = (int)(hq / a.group), g = (int)(hq - (int64_t)bh * a.group);
    const int b = bh / a.heads, h = bh - b * a.heads;
    const Seq s = seq_of<TILE, NEW>(a, b);
    float x[kPer] = {}, top = kNoMax, sum = 0.f;
    if (t < s.n && s.tiles > 0) {
      const int r = g * s.n + t, pass = r / a.tile_q, i = r - pass * a.tile_q;
      const int64_t f0 = __ldcg(a.upto + b) + ((int64_t)h * s.passes + (a.siblings > 1 ? 0 : pass)) * s.tiles;
      const int c0 = share_of(total, shares, f0), more = share_of(total, shares, f0 + s.tiles - 1) - c0;
      if (more == 0) continue;   // finished in the first launch
      if (!in_bounds(c0 >= 0 && c0 + more < shares && i < a.tile_q, a.dev_status)) continue;
      const int slot0 = share_start(total, shares, c0) < f0 ? 1 : 0;
      const int sib = a.siblings > 1 ? pass : 0;
      auto part = [&](int k) { return part_at<D>(a, (c0 + k) * a.siblings + sib, k == 0 ? slot0 : 0); };
      for (int k0 = 0; k0 <= more; k0 += 32) {
        const int here = min(32, more + 1 - k0);
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
              for (int c = 0; c < kPer; ++c) x[c] = fmaf(y[c], w, x[c]);
            }
          }
        }
      }
    }
    const float scale = sum == 0.f ? 0.f : 1.0f / sum;   // a NaN stays one
    IO* out = static_cast<IO*>(a.out) + at * D + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; ++e) store1<IO>(out + e, x[e] * scale);
    if (a.lse && lane == 0) a.lse[at] = lse_of(top, sum);
  }
}

// Passes of many rows: a warp joins 32 rows (a lane each) and eight channels of a head that was cut, and has four parts under way.
template <int D, int TILE>
__global__ void __launch_bounds__(kJoinThreads) tree_join_wide_kernel(Args a) {
  constexpr int kC = 8, kBlocks = D / kC, kAtOnce = 4;
  const int lane = threadIdx.x % 32;
  const int64_t warps = (int64_t)gridDim.x * (kJoinThreads / 32);
  const int blocks = a.tile_q / 32;                                               // of a pass's rows
  const int passes = (int)(((int64_t)a.group * a.tokens + a.tile_q - 1) / a.tile_q);   // of a head, at most
  const int64_t units = (int64_t)a.batch * a.heads * passes * blocks * kBlocks;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t total = __ldcg(a.upto + a.batch);
  const int shares = working_shares(a, total);
  for (int64_t u = (int64_t)blockIdx.x * (kJoinThreads / 32) + threadIdx.x / 32; u < units; u += warps) {
    const int cb = (int)(u % kBlocks);
    const int64_t v = u / kBlocks, hp = v / blocks;
    const int block = (int)(v - hp * blocks), pass = (int)(hp % passes);
    const int bh = (int)(hp / passes), b = bh / a.heads, h = bh - b * a.heads;
    const Seq s = seq_of<TILE, TILE>(a, b);
    const int r0 = pass * a.tile_q + 32 * block, i = 32 * block + lane;
    if (s.tiles == 0 || r0 >= a.group * s.n) continue;
    const int64_t f0 = __ldcg(a.upto + b) + ((int64_t)h * s.passes + (a.siblings > 1 ? 0 : pass)) * s.tiles;
    const int c0 = share_of(total, shares, f0), more = share_of(total, shares, f0 + s.tiles - 1) - c0;
    if (more == 0) continue;   // finished in the first launch
    if (!in_bounds(c0 >= 0 && c0 + more < shares && i < a.tile_q, a.dev_status)) continue;
    const int slot0 = share_start(total, shares, c0) < f0 ? 1 : 0, sib = a.siblings > 1 ? pass : 0;
    const bool mine = r0 + lane < a.group * s.n;   // (the parts' other rows were not written)
    float x[kC], top = kNoMax, sum = 0.f;
#pragma unroll
    for (int e = 0; e < kC; ++e) x[e] = 0.f;
    if (!mine) continue;
    for (int k0 = 0; k0 <= more; k0 += kAtOnce) {
      float y[kAtOnce][kC], m[kAtOnce], l[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const bool in = k0 + k <= more;
        const float* const p = part_at<D>(a, (c0 + (in ? k0 + k : more)) * a.siblings + sib, k0 + k == 0 ? slot0 : 0);
        m[k] = in ? __ldcg(p + (int64_t)a.tile_q * D + i) : kNoMax;
        l[k] = in ? __ldcg(p + (int64_t)a.tile_q * (D + 1) + i) : 0.f;
#pragma unroll
        for (int e = 0; e < kC; ++e) y[k][e] = in ? __ldcg(p + (int64_t)(kC * cb + e) * a.tile_q + i) : 0.f;
      }
      float next = top;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) next = fmaxf(next, m[k]);
      const float old = rescale(top, next);
      top = next;
      sum *= old;
#pragma unroll
      for (int e = 0; e < kC; ++e) x[e] *= old;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const float f = rescale(m[k], next);
        sum = fmaf(l[k], f, sum);
#pragma unroll
        for (int e = 0; e < kC; ++e) x[e] = fmaf(y[k][e], f, x[e]);
      }
    }
    const int r = r0 + lane, g = r / s.n, t = r - g * s.n;
    const int64_t at = ((int64_t)bh * a.group + g) * a.tokens + t;
    const float scale = sum == 0.f ? 0.f : 1.0f / sum;   // a NaN stays one
    __nv_bfloat162 y[kC / 2];
#pragma unroll
    for (int e = 0; e < kC / 2; ++e) y[e] = __floats2bfloat162_rn(x[2 * e] * scale, x[2 * e + 1] * scale);
    uint4* const to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at * D + kC * cb);
#pragma unroll
    for (int e = 0; e < kC / 8; ++e) to[e] = reinterpret_cast<const uint4*>(y)[e];
    if (a.lse && cb == 0) a.lse[at] = lse_of(top, sum);
  }
  // ---- tokens that are not there, and those of sequences without rows to see
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    const Seq s = seq_of<TILE, TILE>(a, b);
    const int first = s.tiles == 0 ? 0 : s.n, none = a.tokens - first;
    const int64_t rows = (int64_t)a.heads * a.group * none;
    for (int64_t u = threadIdx.x; u < rows * (D / 8); u += kJoinThreads) {
      const int64_t row = u / (D / 8), hq = row / none;
      const int64_t at = ((int64_t)b * a.heads * a.group + hq) * a.tokens + first + (row - hq * none);
      const int c = (int)(u % (D / 8));
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at * D)[c] = make_uint4(0u, 0u, 0u, 0u);
      if (a.lse && c == 0) a.lse[at] = -INFINITY;
    }
  }
}

// One wave of blocks at most, but for the last few.
cudaError_t launch_join(void (*kernel)(Args), const Args& a, int64_t blocks, cudaStream_t stream) {
  const int64_t most = 8 * (int64_t)device_sm_count();
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
  const int64_t rows = (int64_t)a.batch * a.heads * a.group * a.tokens;
  return launch_join(tree_join_kernel<IO, D, TILE, NEW>, a, (rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32), stream);
}

template <int D, int TILE> cudaError_t launch_tree_join_wide(const Args& a, cudaStream_t stream) {
  const int64_t passes = ((int64_t)a.group * a.tokens + a.tile_q - 1) / a.tile_q;
  const int64_t units = (int64_t)a.batch * a.heads * passes * (a.tile_q / 32) * (D / 8);
  return launch_join(tree_join_wide_kernel<D, TILE>, a, (units + kJoinThreads / 32 - 1) / (kJoinThreads / 32), stream);
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
