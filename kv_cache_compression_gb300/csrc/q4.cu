// Rows into and out of a cache held in 4 bits (the format of include/snapkv_cache.h).
//
// One thread holds eight channels of a row, eight neighbouring threads a group of 64: the group's
// largest and smallest value are three shuffles away, and a thread's eight levels are one word of
// the row. Both kernels read and write every byte once and are bound by HBM.
#include "cache_internal.h"
#include "q4.cuh"
#include "snapkv_internal.h"

namespace snapkv {
namespace {

constexpr int kQ4Threads = 256;

// max.NaN / min.NaN: a NaN in the group must reach its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T> __device__ __forceinline__ void load8(const T* p, float* x);
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float* x) {
  Elem<__nv_bfloat16>::widen(ld_stream_v4(p), x);
}
template <> __device__ __forceinline__ void load8<float>(const float* p, float* x) {
  Elem<float>::widen(ld_stream_v4(p), x);
  Elem<float>::widen(ld_stream_v4(p + 4), x + 4);
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 two = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&two);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// The level numbers of eight values as nibbles, in q4_pack's order. (x - z) / (2h) + 7.5 has to be
// rounded as if computed exactly: ties are common (0.7 % of normal bf16 values lie half-way between
// two levels). So no quotient is trusted: a product with r = 1 / (2h) only finds the nearest border
// between levels, z + 2h k, and the sign of x - z - 2h k, exact in fp32 up to the difference's own
// rounding error (which kExact puts back; bf16 values leave none that a border is near to), says on
// which side x lies. The border's error of one does not matter where it can occur, half-way between two
// borders. On the border itself the even level wins: level numbers there are k + 7 and k + 8.
// kClamp is for groups whose rounded h and z leave a value more than a step outside the levels.
template <bool kExact, bool kClamp> __device__ __forceinline__ uint32_t levels(const float* x, float h, float z, float r) {
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: adding it rounds to a whole number, in the low bits
  const float nz = 0.0f - z;              // (not -z: x + nz is never -0)
  const float2 nz2 = make_float2(nz, nz), r2 = make_float2(r, r), magic = make_float2(kMagic, kMagic),
               unmagic = make_float2(-kMagic, -kMagic), step = make_float2(-2.0f * h, -2.0f * h);
  float whole[8], side[8];
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 v = make_float2(x[e], x[e + 1]);
    const float2 d = add2(v, nz2);
    float2 w = fma2(d, r2, magic);
    if (kClamp) {
      w.x = fminf(fmaxf(w.x, kMagic - 7.0f), kMagic + 7.0f);
      w.y = fminf(fmaxf(w.y, kMagic - 7.0f), kMagic + 7.0f);
    }
    float2 s = fma2(add2(w, unmagic), step, d);
    if (kExact) {
      const float bx = d.x - v.x, by = d.y - v.y;
      s.x += (v.x - (d.x - bx)) + (nz - bx);
      s.y += (v.y - (d.y - by)) + (nz - by);
    }
    whole[e] = w.x;
    whole[e + 1] = w.y;
    side[e] = s.x;
    side[e + 1] = s.y;
  }
  // k + 8, less one below the border, or on it if that is odd: (bits of s) - (k & 1) is negative just then.
  constexpr int kOrder[8] = {5, 7, 1, 3, 4, 6, 0, 2};   // from the top nibble down
  uint32_t u = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t k = __float_as_uint(whole[kOrder[i]]);
    const int below = (__float_as_int(side[kOrder[i]]) - (int)(k & 1u)) >> 31;
    u = u * 16u + k + (uint32_t)below;
  }
  // each k came with the bits of 1.5 * 2^23, and 8 is still missing: whole nibbles again, mod 2^32
  constexpr uint32_t kBits = 0x4B400000u;
  constexpr uint32_t kAll = kBits * 0x11111111u;
  return u - kAll + 0x88888888u;
}

template <typename T, int D>
__global__ void __launch_bounds__(kQ4Threads) q4_append_kernel(Q4Job a) {
  constexpr int kTpr = D / 8;               // threads per row
  constexpr int kNg = D / kQ4Group;
  const int64_t bh = blockIdx.y;
  const int b = (int)(bh / a.heads);
  const int which = blockIdx.z;             // K or V
  int64_t n = a.rows;
  const int len = a.len[b];
  bool fits = len >= 0;
  if (a.n_new) {
    n = a.n_new[b];
    if (n < 0 || n > a.rows) {
      if (blockIdx.x == 0 && which == 0 && bh % a.heads == 0 && threadIdx.x == 0)
        report(a.dev_status, SNAPKV_ERR_INVALID_ARG);
      fits = false;
      n = 0;
    }
  }
  if (!fits || (int64_t)len + n > a.cap) {
    if (len < 0 || (int64_t)len + n > a.cap)
      if (blockIdx.x == 0 && which == 0 && bh % a.heads == 0 && threadIdx.x == 0)
        report(a.dev_status, SNAPKV_ERR_CAPACITY);
    n = 0;
  }
  if (blockIdx.x == 0 && which == 0 && bh % a.heads == 0 && threadIdx.x == 0) a.len_out[b] = (int)(len + n);
  const T* in = static_cast<const T*>(which ? a.in[1] : a.in[0]) + bh * a.rows * D;
  uint32_t* codes = static_cast<uint32_t*>(which ? a.codes[1] : a.codes[0]) + (bh * a.cap + len) * (D / 8);
  uint32_t* meta = static_cast<uint32_t*>(which ? a.meta[1] : a.meta[0]) + (bh * a.cap + len) * kNg;
  const int c = threadIdx.x % kTpr, g = c / 8, o = c % 8;   // group, and which eight of its channels
  // Every lane of a warp takes the same number of turns (the shuffles below need them all).
  for (int64_t r0 = (int64_t)blockIdx.x * (kQ4Threads / kTpr); r0 < n; r0 += (int64_t)gridDim.x * (kQ4Threads / kTpr)) {
    const int64_t row = r0 + threadIdx.x / kTpr;
    const bool mine = row < n;
    float x[8];
    if (mine) {
      load8<T>(in + row * D + 8 * c, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
    }
    float hi = x[0], lo = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      hi = max_nan(hi, x[e]);
      lo = min_nan(lo, x[e]);
    }
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    }
    // (hi - lo) / 30 rounded once: the difference's and the quotient's rounding errors are put back.
    const float diff = hi - lo;
    const float back = hi - diff;
    const float err = (hi - (diff + back)) + (back - lo);
    float q = diff * (1.0f / 30.0f);
    q = fmaf(fmaf(-q, 30.0f, diff) + err, 1.0f / 30.0f, q);
    __nv_bfloat16 hb = __float2bfloat16_rn(q), zb = __float2bfloat16_rn(0.5f * (hi + lo));
    float h = __bfloat162float(hb), z = __bfloat162float(zb);
    if (h < 0x1p-126f) h = 0.f;
    uint32_t u = 0x88888888u;
    if (!(h < INFINITY) || !(fabsf(z) < INFINITY)) {
      h = z = __uint_as_float(0x7FC00000u);
    } else if (h > 0.f) {
      const float r = __fdividef(1.0f, 2.0f * h);
      constexpr bool kExact = sizeof(T) == 4;
      u = fmaxf(hi - z, z - lo) < 15.9f * h ? levels<kExact, false>(x, h, z, r) : levels<kExact, true>(x, h, z, r);
    }
    if (mine) {
      codes[row * (D / 8) + q4_word<kNg>(g, o)] = q4_pack(u);
      if (o == 0) meta[row * kNg + g] = (__float_as_uint(h) >> 16) | (__float_as_uint(z) & 0xFFFF0000u);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kQ4Threads) q4_read_kernel(Q4Job a) {
  constexpr int kTpr = D / 8;
  constexpr int kNg = D / kQ4Group;
  const int64_t bh = blockIdx.y;
  const int b = (int)(bh / a.heads);
  const int which = blockIdx.z;
  const int64_t start = a.len ? a.len[b] : 0;
  const uint32_t* codes = static_cast<const uint32_t*>(which ? a.codes[1] : a.codes[0]) + bh * a.cap * (D / 8);
  const uint32_t* meta = static_cast<const uint32_t*>(which ? a.meta[1] : a.meta[0]) + bh * a.cap * kNg;
  T* out = static_cast<T*>(which ? a.out[1] : a.out[0]) + bh * a.rows * D;
  const int c = threadIdx.x % kTpr, g = c / 8, o = c % 8;
  for (int64_t r0 = (int64_t)blockIdx.x * (kQ4Threads / kTpr); r0 < a.rows;
       r0 += (int64_t)gridDim.x * (kQ4Threads / kTpr)) {
    const int64_t row = r0 + threadIdx.x / kTpr, src = start + row;
    if (row >= a.rows) break;
    float x[8];
    if (src >= 0 && src < a.cap) {
      const uint32_t w = __ldg(codes + src * (D / 8) + q4_word<kNg>(g, o));
      const uint32_t m = __ldg(meta + src * kNg + g);
      const float h = __uint_as_float(m << 16), z = __uint_as_float(m & 0xFFFF0000u);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(h, (float)q4_level(w, e), z);   // h t is exact in fp32
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
    }
    store8(out + row * D + 8 * c, x);
  }
}

// A block takes 256 / (d / 8) rows at a turn. All blocks together are about eight waves, so that a
// long prompt amortises the head's set-up over several turns.
dim3 q4_grid(const Q4Job& job) {
  const int per_turn = kQ4Threads / (job.head_dim / 8);
  const int64_t turns = (job.rows + per_turn - 1) / per_turn;
  const int64_t bh = (int64_t)job.batch * job.heads;
  int64_t blocks = ((int64_t)device_sm_count() * 8 * 8 + 2 * bh - 1) / (2 * bh);
  if (blocks > turns) blocks = turns;
  return dim3((unsigned)(blocks < 1 ? 1 : blocks), (unsigned)bh, 2);
}

}  // namespace

cudaError_t launch_q4_append(const Q4Job& job) {
  const dim3 grid = q4_grid(job);
  if (job.dtype == SNAPKV_BF16) {
    if (job.head_dim == 64)
      q4_append_kernel<__nv_bfloat16, 64><<<grid, kQ4Threads, 0, job.stream>>>(job);
    else
      q4_append_kernel<__nv_bfloat16, 128><<<grid, kQ4Threads, 0, job.stream>>>(job);
  } else {
    if (job.head_dim == 64)
      q4_append_kernel<float, 64><<<grid, kQ4Threads, 0, job.stream>>>(job);
    else
      q4_append_kernel<float, 128><<<grid, kQ4Threads, 0, job.stream>>>(job);
  }
  return cudaGetLastError();
}

cudaError_t launch_q4_read(const Q4Job& job) {
  const dim3 grid = q4_grid(job);
  if (job.dtype == SNAPKV_BF16) {
    if (job.head_dim == 64)
      q4_read_kernel<__nv_bfloat16, 64><<<grid, kQ4Threads, 0, job.stream>>>(job);
    else
      q4_read_kernel<__nv_bfloat16, 128><<<grid, kQ4Threads, 0, job.stream>>>(job);
  } else {
    if (job.head_dim == 64)
      q4_read_kernel<float, 64><<<grid, kQ4Threads, 0, job.stream>>>(job);
    else
      q4_read_kernel<float, 128><<<grid, kQ4Threads, 0, job.stream>>>(job);
  }
  return cudaGetLastError();
}

}  // namespace snapkv
