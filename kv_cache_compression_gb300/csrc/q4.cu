// Rows into and out of a cache held in 4 bits (the format of include/snapkv_cache.h).
//
// A thread holds two or four words' channels of a group of 64 (every fourth or second of its eight words, so
// that neighbouring threads load neighbouring 16 bytes), and the group's largest and smallest value are one
// or two shuffles away. Both kernels read and write every byte once. Writing 16-bit rows costs 2.6 bytes of
// HBM traffic a value, which is too little to hide the arithmetic behind: at 435 instructions per warp and
// 1024 values the kernel issues in two thirds of all cycles and moves 4.7 TB/s. It took 3.0 ms with a 64-bit
// division wherever a value lies close to half-way between two levels, as 0.7 % of normal bf16 values do.
#include "cache_internal.h"
#include "q4.cuh"
#include "row_list.cuh"
#include "snapkv_internal.h"

namespace snapkv {
namespace {

// Words (of eight channels of one group) of a thread. Four share more of the work on a group, where there are
// rows enough: writing 16384 rows of 32 heads takes 77 us with four words, 88 with two and 108 with all
// eight (in blocks of 256 threads); one row of 2048 heads 3.4, 3.0 and 5.2 us. Reading has little to share: 70, 59 and 65 us with one, two
// and four, and 2.2, 2.3 and 2.6.
template <bool FLAT> constexpr int kAppendWords = FLAT ? 2 : 4;
constexpr int kReadWords = 2;

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

// W words' values in pairs, `step` values from one word to the next, and the largest and smallest of them.
template <int W> __device__ __forceinline__ void load_values(const __nv_bfloat16* p, int step, float2* x, float* hi, float* lo) {
  uint32_t w[4 * W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const uint4 v = ld_stream_v4(p + i * step);
    w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
  }
  uint32_t top = w[0], low = w[0];   // two at a time
#pragma unroll
  for (int i = 1; i < 4 * W; ++i) {
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(w[i]));
    asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(low) : "r"(w[i]));
  }
#pragma unroll
  for (int i = 0; i < 4 * W; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  *hi = max_nan(__uint_as_float(top << 16), __uint_as_float(top & 0xFFFF0000u));
  *lo = min_nan(__uint_as_float(low << 16), __uint_as_float(low & 0xFFFF0000u));
}
template <int W> __device__ __forceinline__ void load_values(const float* p, int step, float2* x, float* hi, float* lo) {
#pragma unroll
  for (int i = 0; i < 2 * W; ++i) {
    const uint4 w = ld_stream_v4(p + (i / 2) * step + 4 * (i % 2));
    x[2 * i] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    x[2 * i + 1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
  *hi = max_nan(x[0].x, x[0].y);
  *lo = min_nan(x[0].x, x[0].y);
#pragma unroll
  for (int e = 1; e < 4 * W; ++e) {
    *hi = max_nan(*hi, max_nan(x[e].x, x[e].y));
    *lo = min_nan(*lo, min_nan(x[e].x, x[e].y));
  }
}

// The level numbers of eight values as nibbles, in q4_pack's order. (x - z) / (2h) + 7.5 has to be
// rounded as if computed exactly: ties are common (0.7 % of normal bf16 values lie half-way between
// two levels). So no quotient is trusted: a product with r = 1 / (2h) only finds the nearest border
// between levels, z + 2h k, and the sign of s = x - (z + 2h k) says on which side x lies. For bf16 rows the
// border is exact in fp32 (z is zero or a multiple of 2^-9 of the group's largest value), so the sign is;
// for fp32 rows (kExact) s is (x - z) - 2h k, exact but for the rounding error of x - z, which is put back.
// An error of one in k does not matter where it can occur, half-way between two borders. s then becomes 0,
// 1/2 or 1 (anything but zero, times 2^127, saturates), and k + 7 plus that is rounded to the even level
// where x lies on the border. (fp32 instructions of two values each do most of it, as the logic pipe is what
// this kernel runs out of.)
// kClamp is for groups whose rounded h and z leave a value more than a step outside the levels.
template <bool kExact, bool kClamp>
__device__ __forceinline__ uint32_t levels(const float2* x, float h, float z, float r) {
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: adding it rounds to a whole number, in the low bits
  const float nz = 0.0f - z;              // (not -z: x + nz is never -0)
  const float2 nz2 = make_float2(nz, nz), r2 = make_float2(r, r), magic = make_float2(kMagic, kMagic),
               unmagic = make_float2(-kMagic, -kMagic), step = make_float2(-2.0f * h, -2.0f * h),
               magic7 = make_float2(kMagic + 7.0f, kMagic + 7.0f);
  float2 level[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 d = add2(x[e], nz2);
    float2 k = add2(fma2(d, r2, magic), unmagic);
    if (kClamp) {
      k.x = fminf(fmaxf(k.x, -7.0f), 7.0f);
      k.y = fminf(fmaxf(k.y, -7.0f), 7.0f);
    }
    float2 s;
    if (!kExact) {
      s = add2(x[e], fma2(k, step, nz2));
    } else {
      s = fma2(k, step, d);
      const float bx = d.x - x[e].x, by = d.y - x[e].y;
      s.x += (x[e].x - (d.x - bx)) + (nz - bx);
      s.y += (x[e].y - (d.y - by)) + (nz - by);
    }
    const float2 side = make_float2(__saturatef(fmaf(s.x, 0x1p127f, 0.5f)), __saturatef(fmaf(s.y, 0x1p127f, 0.5f)));
    level[e] = add2(add2(add2(k, side), magic7), unmagic);
  }
  // The halves' nibbles, both at once in fp32 (16 bits are exact): pairs 2, 3, 0, 1 from the top.
  const float2 up = make_float2(16.0f, 16.0f);
  const float2 half = add2(fma2(fma2(fma2(level[2], up, level[3]), up, level[0]), up, level[1]), make_float2(8388608.0f, 8388608.0f));
  return prmt(__float_as_uint(half.x), __float_as_uint(half.y), 0x5410);
}

struct AppendSeq {
  int b, len, n;     // rows held, rows to write
  bool counts, fits; // n_new is in range; the rows fit
};

template <typename T, int D, bool FLAT>
__global__ void __launch_bounds__(kRowThreads) q4_append_kernel(Q4Job a, unsigned flat_rows) {
  constexpr int W = kAppendWords<FLAT>;
  constexpr int kTpr = D / (8 * W), kTpg = 8 / W;   // threads per row, and per group
  constexpr int kNg = D / kQ4Group;
  const int which = blockIdx.z;                     // K or V
  const int c = threadIdx.x % kTpr, g = c / kTpg, o = c % kTpg;   // group, and the first of this thread's eights
  auto seq = [&](int b) {
    AppendSeq s;
    s.b = b;
    s.len = a.len[b];
    s.n = a.n_new ? a.n_new[b] : (int)a.rows;
    s.counts = s.n >= 0 && s.n <= (int)a.rows;
    s.fits = s.len >= 0 && s.counts && (int64_t)s.len + s.n <= a.cap;
    return s;
  };
  for_rows<FLAT, kTpr>(flat_rows, a.heads, a.rows, seq, [&](unsigned bh, int row, bool mine, const AppendSeq& s) {
    if (mine && row == 0 && c == 0 && which == 0 && bh == (unsigned)s.b * a.heads) {   // once per sequence
      a.len_out[s.b] = s.fits ? s.len + s.n : s.len;
      if (!s.counts) report(a.dev_status, SNAPKV_ERR_INVALID_ARG);
      if (s.len < 0 || (s.counts && (int64_t)s.len + s.n > a.cap)) report(a.dev_status, SNAPKV_ERR_CAPACITY);
    }
    mine = mine && s.fits && row < s.n;
    if (!__any_sync(0xffffffffu, mine)) return;
    float2 x[4 * W];
    float hi = 0.f, lo = 0.f;
    if (mine) {
      load_values<W>(static_cast<const T*>(which ? a.in[1] : a.in[0]) + ((int64_t)bh * a.rows + row) * D + kQ4Group * g + 8 * o,
                     8 * kTpg, x, &hi, &lo);
    } else {
#pragma unroll
      for (int e = 0; e < 4 * W; ++e) x[e] = make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int off = 1; off < kTpg; off <<= 1) {
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    }
    // (hi - lo) / 30 rounded once: the difference's and the quotient's rounding errors are put back.
    const float diff = hi - lo;
    const float back = hi - diff;
    const float err = (hi - (diff + back)) + (back - lo);
    float q = diff * (1.0f / 30.0f);
    q = fmaf(fmaf(-q, 30.0f, diff) + err, 1.0f / 30.0f, q);
    float h = __bfloat162float(__float2bfloat16_rn(q)), z = __bfloat162float(__float2bfloat16_rn(0.5f * (hi + lo)));
    if (h < 0x1p-126f) h = 0.f;
    uint32_t u[W];
#pragma unroll
    for (int w = 0; w < W; ++w) u[w] = 0x88888888u;
    if (!(h < INFINITY) || !(fabsf(z) < INFINITY)) {
      h = z = __uint_as_float(0x7FC00000u);
    } else if (h > 0.f) {
      const float r = __fdividef(1.0f, 2.0f * h);
      constexpr bool kExact = sizeof(T) == 4;
      const bool near = fmaxf(hi - z, z - lo) < 15.9f * h;
#pragma unroll
      for (int w = 0; w < W; ++w)
        u[w] = near ? levels<kExact, false>(x + 4 * w, h, z, r) : levels<kExact, true>(x + 4 * w, h, z, r);
    }
    if (mine && in_bounds((int64_t)s.len + row < a.cap, a.dev_status)) {
      const int64_t at = bh * a.cap + (s.len + row);
      uint32_t* codes = static_cast<uint32_t*>(which ? a.codes[1] : a.codes[0]) + at * (D / 8);
#pragma unroll
      for (int w = 0; w < W; ++w) codes[q4_word<kNg>(g, o + kTpg * w)] = q4_pack(u[w]);
      if (o == 0)
        static_cast<uint32_t*>(which ? a.meta[1] : a.meta[0])[at * kNg + g] =
            (__float_as_uint(h) >> 16) | (__float_as_uint(z) & 0xFFFF0000u);
    }
  });
}

// The values of a word's eight channels: its operands (levels in units of 2^-131 and 2^-133) as fp32.
__device__ __forceinline__ void q4_values(const Q4Ones& one, uint32_t w, float h, float z, float* x) {
  uint32_t e[4];
  q4_operands(one, w, prmt(w, w, 0x2301), e);
  const float2 up = make_float2(0x1p127f, 0x1p127f), zz = make_float2(z, z);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float s = j & 1 ? h * 64.0f : h * 16.0f;
    // h t is exact in fp32, so that the value is rounded once
    const float2 t = mul2(make_float2(__uint_as_float(e[j] << 16), __uint_as_float(e[j] & 0xFFFF0000u)), up);
    const float2 v = fma2(t, make_float2(s, s), zz);
    x[2 * j] = v.x;
    x[2 * j + 1] = v.y;
  }
}

template <typename T, int D, bool FLAT>
__global__ void __launch_bounds__(kRowThreads) q4_read_kernel(Q4Job a, unsigned flat_rows, Q4Ones one) {
  constexpr int W = kReadWords;
  constexpr int kTpr = D / (8 * W), kTpg = 8 / W;
  constexpr int kNg = D / kQ4Group;
  const int which = blockIdx.z;
  const int c = threadIdx.x % kTpr, g = c / kTpg, o = c % kTpg;
  auto seq = [&](int b) { return a.len ? a.len[b] : 0; };
  for_rows<FLAT, kTpr>(flat_rows, a.heads, a.rows, seq, [&](unsigned bh, int row, bool mine, int start) {
    if (!mine) return;
    const int64_t src = (int64_t)start + row;
    float x[8 * W];
    if (src >= 0 && src < a.cap) {
      const int64_t at = bh * a.cap + src;
      const uint32_t* codes = static_cast<const uint32_t*>(which ? a.codes[1] : a.codes[0]) + at * (D / 8);
      const uint32_t m = __ldg(static_cast<const uint32_t*>(which ? a.meta[1] : a.meta[0]) + at * kNg + g);
      const float h = __uint_as_float(m << 16), z = __uint_as_float(m & 0xFFFF0000u);
#pragma unroll
      for (int w = 0; w < W; ++w) q4_values(one, __ldg(codes + q4_word<kNg>(g, o + kTpg * w)), h, z, x + 8 * w);
    } else {
#pragma unroll
      for (int e = 0; e < 8 * W; ++e) x[e] = 0.f;
    }
    T* out = static_cast<T*>(which ? a.out[1] : a.out[0]) + ((int64_t)bh * a.rows + row) * D + kQ4Group * g + 8 * o;
#pragma unroll
    for (int w = 0; w < W; ++w) store8(out + 8 * kTpg * w, x + 8 * w);
  });
}

template <typename T, int D, bool FLAT> cudaError_t q4_append_typed(const Q4Job& job) {
  q4_append_kernel<T, D, FLAT><<<row_grid(job.batch, job.heads, job.rows, job.head_dim / (8 * kAppendWords<FLAT>), 2), kRowThreads, 0, job.stream>>>(
      job, FLAT ? (unsigned)(job.batch * job.heads * job.rows) : 0u);
  return cudaGetLastError();
}

template <typename T, int D, bool FLAT> cudaError_t q4_read_typed(const Q4Job& job) {
  q4_read_kernel<T, D, FLAT><<<row_grid(job.batch, job.heads, job.rows, job.head_dim / (8 * kReadWords), 8), kRowThreads, 0, job.stream>>>(
      job, FLAT ? (unsigned)(job.batch * job.heads * job.rows) : 0u, Q4Ones());
  return cudaGetLastError();
}

template <typename T, int D> cudaError_t q4_append_rows(const Q4Job& job) {
  return job.rows < kFlatRows ? q4_append_typed<T, D, true>(job) : q4_append_typed<T, D, false>(job);
}

template <typename T, int D> cudaError_t q4_read_rows(const Q4Job& job) {
  return job.rows < kFlatRows ? q4_read_typed<T, D, true>(job) : q4_read_typed<T, D, false>(job);
}

}  // namespace

cudaError_t launch_q4_append(const Q4Job& job) {
  if (job.dtype == SNAPKV_BF16)
    return job.head_dim == 64 ? q4_append_rows<__nv_bfloat16, 64>(job) : q4_append_rows<__nv_bfloat16, 128>(job);
  return job.head_dim == 64 ? q4_append_rows<float, 64>(job) : q4_append_rows<float, 128>(job);
}

cudaError_t launch_q4_read(const Q4Job& job) {
  if (job.dtype == SNAPKV_BF16)
    return job.head_dim == 64 ? q4_read_rows<__nv_bfloat16, 64>(job) : q4_read_rows<__nv_bfloat16, 128>(job);
  return job.head_dim == 64 ? q4_read_rows<float, 64>(job) : q4_read_rows<float, 128>(job);
}

}  // namespace snapkv
