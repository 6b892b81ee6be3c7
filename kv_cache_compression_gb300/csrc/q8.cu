// Rows appended to a cache, as they are or quantised to 8 bits, and read out of 8 bits (include/snapkv_draft.h).
//
// A row's lanes are a power of two, so that the largest |x| of a row is a few shuffles away; each lane has every
// kTpr-th run of eight channels, so that neighbouring lanes load neighbouring 16 bytes (bf16). Every byte is read and
// written once: 32 heads of 16384 bf16 rows of 128 channels, K and V, quantised and read back in 142 us (5.7 TB/s; bytes bound
// the reading, while quantising has the schedulers busy for 74 %); 64 x 32 heads, up to six picked rows each, 7.6 us, the
// latency of a launch. Picks are made for accepted tokens: every block checks all of its sequence's before it writes, so that a sequence
// with a bad one is left as it was without a launch more. 33 picks cost nothing so, 16384 of 32 heads 10 us of 95 (dense) or 30 of 101.
#include "draft_internal.h"
#include "q4.cuh"
#include "row_list.cuh"

namespace snapkv {
namespace {

// Runs of eight channels of a thread.
constexpr int kRuns = 2;

__device__ __forceinline__ float max_nan(float a, float b) {   // a NaN stays one
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A thread's values as they lie in memory: kRuns runs of eight.
template <typename T> struct Raw {
  static constexpr int kVec = (int)sizeof(T) / 2;   // 16-byte vectors per run
  uint4 w[kRuns * kVec];
  __device__ __forceinline__ void load(const T* p, int step) {
#pragma unroll
    for (int i = 0; i < kRuns * kVec; ++i) w[i] = ld_stream_v4(p + (i / kVec) * step + (16 / (int)sizeof(T)) * (i % kVec));
  }
  __device__ __forceinline__ void store(T* p, int step) const {
#pragma unroll
    for (int i = 0; i < kRuns * kVec; ++i)
      *reinterpret_cast<uint4*>(p + (i / kVec) * step + (16 / (int)sizeof(T)) * (i % kVec)) = w[i];
  }
  __device__ __forceinline__ void widen(float* x) const {
#pragma unroll
    for (int i = 0; i < kRuns * kVec; ++i) Elem<T>::widen(w[i], x + i * Elem<T>::kVec);
  }
};

// max |x| / 127 rounded once. r = RN(1 / 127) and q = RN(a r) are within one unit of a / 127, a - 127 q is exact, and
// a quotient corrected so by a correctly rounded reciprocal is the rounded one (Markstein).
__device__ __forceinline__ float step_of(float a) {
  constexpr float r = 1.0f / 127.0f;
  const float q = a * r;
  const float h = fmaf(fmaf(-127.0f, q, a), r, q);
  return h < 0x1p-80f ? 0.f : h;   // (a NaN stays one; an infinity has become one)
}

// The codes of four values. |x| / h has to be rounded as if computed exactly: its ties are common where h has few bits
// (rows of 16-bit values whose largest is 127 times a power of two). The product with r = 1 / h only finds the nearest
// border f + 1/2 between two magnitudes; the sign of s = |x| - (f + 1/2) h, one FMA, is exact. s then becomes 0,
// 1/2 or 1 (anything but zero, times 2^127, saturates: |s| is zero or above 2^-106, as h is 2^-80 at least), and f plus
// that is rounded to the even number where |x| lies on the border.
__device__ __forceinline__ uint32_t codes4(const float* x, float h, float r) {
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: adding it rounds to a whole number, in the low bits
  const float2 magic = make_float2(kMagic, kMagic), unmagic = make_float2(-kMagic, -kMagic), half = make_float2(-0.5f, -0.5f),
               r2 = make_float2(r, r), nh = make_float2(-h, -h);
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const float2 a = make_float2(fabsf(x[e]), fabsf(x[e + 1]));
    const float2 f = add2(add2(fma2(a, r2, half), magic), unmagic);

    const float2 s = fma2(add2(f, make_float2(0.5f, 0.5f)), nh, a);
    const float2 side = make_float2(__saturatef(fmaf(s.x, 0x1p127f, 0.5f)), __saturatef(fmaf(s.y, 0x1p127f, 0.5f)));
    const float2 m = add2(add2(f, side), magic);
    u[e] = __float_as_uint(m.x);
    u[e + 1] = __float_as_uint(m.y);
  }
  const uint32_t mag = prmt(prmt(u[0], u[1], 0x0040), prmt(u[2], u[3], 0x0040), 0x5410);
  const uint32_t sign = prmt(prmt(__float_as_uint(x[0]), __float_as_uint(x[1]), 0x0073),
                             prmt(__float_as_uint(x[2]), __float_as_uint(x[3]), 0x0073), 0x5410);
  return (mag & 0x7F7F7F7Fu) | (sign & 0x80808080u);
}

struct AppendSeq {
  int b, len, n;          // rows held, rows to write
  bool valid, fits;       // n_new and the picks are in range; the rows fit
};

template <typename T, int D, bool FLAT, bool Q8>
__global__ void __launch_bounds__(kRowThreads) append_rows_kernel(RowJob a, unsigned flat_rows) {
  constexpr int kTpr = D / (8 * kRuns);             // threads per row
  const int which = blockIdx.z;                     // K or V
  const int c = threadIdx.x % kTpr;
  auto seq = [&](int b) {                           // (called by whole warps; by the whole block where not FLAT)
    AppendSeq s;
    s.b = b;
    s.len = a.len[b];
    s.n = a.n_new ? a.n_new[b] : (int)a.count;
    s.valid = s.n >= 0 && s.n <= (int)a.count;
    if (a.pick) {
      const int32_t* pick = a.pick + (int64_t)b * a.count;
      const int n = s.valid ? s.n : 0;
      bool bad = false;
      for (int i = FLAT ? c : (int)threadIdx.x; i < n; i += FLAT ? kTpr : kRowThreads) {
        const int p = __ldg(pick + i);
        bad |= p < 0 || p >= (int)a.rows;
      }
      if constexpr (FLAT) {
#pragma unroll
        for (int off = 1; off < kTpr; off <<= 1) bad |= __shfl_xor_sync(0xffffffffu, (int)bad, off) != 0;
      } else {
        bad = __syncthreads_or(bad);
      }
      s.valid = s.valid && !bad;
    }
    s.fits = s.len >= 0 && s.valid && (int64_t)s.len + s.n <= a.cap;
    return s;
  };
  for_rows<FLAT, kTpr>(flat_rows, a.heads, a.count, seq, [&](unsigned bh, int row, bool mine, const AppendSeq& s) {
    if (mine && row == 0 && c == 0 && which == 0 && bh == (unsigned)s.b * a.heads) {   // once per sequence
      a.len_out[s.b] = s.fits ? s.len + s.n : s.len;
      if (!s.valid) report(a.dev_status, SNAPKV_ERR_INVALID_ARG);
      if (s.len < 0 || (s.valid && (int64_t)s.len + s.n > a.cap)) report(a.dev_status, SNAPKV_ERR_CAPACITY);
    }
    mine = mine && s.fits && row < s.n;
    if (!__any_sync(0xffffffffu, mine)) return;
    Raw<T> raw;
    if (mine) {
      const int64_t from = (int64_t)bh * a.rows + (a.pick ? __ldg(a.pick + (int64_t)s.b * a.count + row) : row);
      raw.load(static_cast<const T*>(which ? a.in[1] : a.in[0]) + from * D + 8 * c, 8 * kTpr);
    } else {
#pragma unroll
      for (int i = 0; i < kRuns * Raw<T>::kVec; ++i) raw.w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    mine = mine && in_bounds((int64_t)s.len + row < a.cap, a.dev_status);
    const int64_t at = (int64_t)bh * a.cap + s.len + row;
    if constexpr (!Q8) {
      if (mine) raw.store(static_cast<T*>(which ? a.held[1] : a.held[0]) + at * D + 8 * c, 8 * kTpr);
    } else {
      float x[8 * kRuns];
      raw.widen(x);
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 8 * kRuns; ++e) top = max_nan(top, fabsf(x[e]));
#pragma unroll
      for (int off = 1; off < kTpr; off <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
      float h = step_of(top);
      uint32_t u[2 * kRuns];
#pragma unroll
      for (int i = 0; i < 2 * kRuns; ++i) u[i] = 0u;
      if (!(h < INFINITY)) {
        h = __uint_as_float(0x7FC00000u);
      } else if (h > 0.f) {
        const float r = __fdividef(1.0f, h);
#pragma unroll
        for (int i = 0; i < 2 * kRuns; ++i) u[i] = codes4(x + 4 * i, h, r);
      }
      if (mine) {
        uint8_t* codes = static_cast<uint8_t*>(which ? a.held[1] : a.held[0]) + at * D + 8 * c;
#pragma unroll
        for (int i = 0; i < kRuns; ++i) *reinterpret_cast<uint2*>(codes + i * 8 * kTpr) = make_uint2(u[2 * i], u[2 * i + 1]);
        if (c == 0) static_cast<float*>(which ? a.step[1] : a.step[0])[at] = h;
      }
    }
  });
}

// u h rounded once to T, with x's sign. For bf16 the product is first cut to fp32 with its last bit set where anything
// was cut off, after which rounding to fewer bits is as if from the whole product.
template <typename T> __device__ __forceinline__ float product(float u, float h) {
  if constexpr (sizeof(T) == 4) return u * h;
  const float p = __fmul_rz(u, h);
  return __uint_as_float(__float_as_uint(p) | (fmaf(u, h, -p) != 0.f ? 1u : 0u));
}

template <typename T, int D, bool FLAT>
__global__ void __launch_bounds__(kRowThreads) q8_read_kernel(RowJob a, unsigned flat_rows) {
  constexpr int kTpr = D / (8 * kRuns);
  const int which = blockIdx.z;
  const int c = threadIdx.x % kTpr;
  auto seq = [&](int b) { return a.len ? a.len[b] : 0; };
  for_rows<FLAT, kTpr>(flat_rows, a.heads, a.rows, seq, [&](unsigned bh, int row, bool mine, int start) {
    if (!mine) return;
    const int64_t src = (int64_t)start + row;
    T* out = static_cast<T*>(which ? a.out[1] : a.out[0]) + ((int64_t)bh * a.rows + row) * D + 8 * c;
    uint2 code[kRuns];
    float h = 0.f;
#pragma unroll
    for (int i = 0; i < kRuns; ++i) code[i] = make_uint2(0u, 0u);
    if (src >= 0 && src < a.cap) {
      const int64_t at = (int64_t)bh * a.cap + src;
      const uint8_t* codes = static_cast<const uint8_t*>(which ? a.held[1] : a.held[0]) + at * D + 8 * c;
#pragma unroll
      for (int i = 0; i < kRuns; ++i) code[i] = __ldg(reinterpret_cast<const uint2*>(codes + i * 8 * kTpr));
      h = __ldg(static_cast<const float*>(which ? a.step[1] : a.step[0]) + at);
    }
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t byte = ((e < 4 ? code[i].x : code[i].y) >> (8 * (e % 4))) & 0xFFu;
        const float v = product<T>(__uint_as_float(0x4B000000u | (byte & 0x7Fu)) - 8388608.0f, h);
        x[e] = __uint_as_float(__float_as_uint(v) ^ ((byte & 0x80u) << 24));
      }
      store8(out + i * 8 * kTpr, x);
    }
  });
}

template <typename T, int D, bool FLAT> cudaError_t append_typed(const RowJob& job) {
  const dim3 grid = row_grid(job.batch, job.heads, job.count, D / (8 * kRuns), 2);
  const unsigned flat = FLAT ? (unsigned)(job.batch * job.heads * job.count) : 0u;
  if (job.step[0])
    append_rows_kernel<T, D, FLAT, true><<<grid, kRowThreads, 0, job.stream>>>(job, flat);
  else
    append_rows_kernel<T, D, FLAT, false><<<grid, kRowThreads, 0, job.stream>>>(job, flat);
  return cudaGetLastError();
}

template <typename T, int D> cudaError_t append_dim(const RowJob& job) {
  return job.count < kFlatRows ? append_typed<T, D, true>(job) : append_typed<T, D, false>(job);
}

template <typename T, int D> cudaError_t read_dim(const RowJob& job) {
  const dim3 grid = row_grid(job.batch, job.heads, job.rows, D / (8 * kRuns), 8);
  if (job.rows < kFlatRows)
    q8_read_kernel<T, D, true><<<grid, kRowThreads, 0, job.stream>>>(job, (unsigned)(job.batch * job.heads * job.rows));
  else
    q8_read_kernel<T, D, false><<<grid, kRowThreads, 0, job.stream>>>(job, 0u);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_rows(const RowJob& job) {
  if (job.dtype == SNAPKV_BF16)
    return job.head_dim == 64 ? append_dim<__nv_bfloat16, 64>(job) : append_dim<__nv_bfloat16, 128>(job);
  return job.head_dim == 64 ? append_dim<float, 64>(job) : append_dim<float, 128>(job);
}

cudaError_t launch_q8_read(const RowJob& job) {
  if (job.dtype == SNAPKV_BF16) return job.head_dim == 64 ? read_dim<__nv_bfloat16, 64>(job) : read_dim<__nv_bfloat16, 128>(job);
  return job.head_dim == 64 ? read_dim<float, 64>(job) : read_dim<float, 128>(job);
}

}  // namespace snapkv
