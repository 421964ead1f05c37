// Rows of bf16 or fp32 values and of 8-bit checkpoints, 16 columns a thread: what
// the passes over activations share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace muon {

constexpr int kBlock = 32;   // columns that share a scale of a checkpoint
constexpr double kCodeBytes = 1.0 + 1.0 / kBlock;   // of a value of a checkpoint

// Quotient by a fixed divisor of numbers below 2^31: with l = ceil(log2 d) and
// m = ceil(2^(31+l) / d), m*d exceeds 2^(31+l) by less than 2^l, so the
// product's error stays below one part in n for n < 2^31.
struct Divider {
  uint32_t mul, shift, d;
};

inline Divider divider(uint32_t d) {
  uint32_t l = 0;
  while ((uint64_t{1} << l) < d) ++l;
  const uint64_t two = uint64_t{1} << (31 + l);
  return {static_cast<uint32_t>((two + d - 1) / d), 31 + l, d};
}

__device__ __forceinline__ uint32_t quotient(uint32_t n, const Divider& v) {
  return static_cast<uint32_t>((static_cast<uint64_t>(n) * v.mul) >> v.shift);
}

struct Plane {          // one operand: base of the first row, row stride in elements
  void* p;
  int64_t stride;
};

struct Packed {
  int8_t* codes;
  int64_t code_stride;
  uint8_t* exps;
  int64_t exp_stride;
};

// ---- 16 values of a row ------------------------------------------------------
// Columns col .. col + N - 1 of a row, of which n are in the row (the others are
// 0).  WHOLE: rows start on 32-byte boundaries (N = 16).
template <typename T, bool WHOLE, int N>
__device__ __forceinline__ void load_values(const Plane& pl, int64_t row, int col, int n,
                                            float (&x)[N]) {
  static_assert(!WHOLE || N == kCols);
  constexpr int kWords = kCols * sizeof(T) / 4;
  const T* p = static_cast<const T*>(pl.p) + row * pl.stride + col;
  if constexpr (WHOLE) {
    if (n >= kCols) {
      uint32_t w[kWords];
#pragma unroll
      for (int q = 0; q < kWords; q += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + q);
        w[q] = u.x; w[q + 1] = u.y; w[q + 2] = u.z; w[q + 3] = u.w;
      }
      to_floats<T>(w, x);
    } else {
#pragma unroll
      for (int k = 0; k < kCols; ++k) x[k] = k < n ? static_cast<float>(p[k]) : 0.f;
    }
  } else {
    load_shifted(p, n, x);
  }
}

// The reverse; the whole warp calls it (n <= 0: nothing of this thread's is in the row).
template <typename T, bool WHOLE, int N>
__device__ __forceinline__ void store_values(const Plane& pl, int64_t row, int col, int n,
                                             const float (&x)[N]) {
  constexpr int kWords = kCols * sizeof(T) / 4;
  T* p = static_cast<T*>(pl.p) + row * pl.stride + col;
  if constexpr (WHOLE) {
    if (n >= kCols) {
      uint32_t w[kWords];
      to_words<T>(x, w);
#pragma unroll
      for (int q = 0; q < kWords; q += 8)
        st_global_v8(reinterpret_cast<uint32_t*>(p) + q, make_uint4(w[q], w[q + 1], w[q + 2], w[q + 3]),
                     make_uint4(w[q + 4], w[q + 5], w[q + 6], w[q + 7]));
    } else {
#pragma unroll
      for (int k = 0; k < kCols; ++k)
        if (k < n) store_one(p + k, x[k]);
    }
  } else {
    const int lane = threadIdx.x & 31;
    store_shifted(p, n, lane > 0 && col > 0, lane < 31 ? min(max(n - N, 0), N) : 0, x);
  }
}

// The same as load_values in two steps, for rows in flight together: fetch issues
// the loads, values_of waits for them (turning bf16 into floats where they are
// loaded makes the next row's loads wait: 596 us for 8 rows of 7168 bf16 a token,
// 16384 tokens, where fp32 of the same bytes took 299).
template <typename T, bool WHOLE, int N>
struct Fetched {
  static constexpr int kWords = N * sizeof(T) / 4;
  uint32_t w[WHOLE ? kWords : kWords + 4];
  uint32_t by;   // bytes before the first column
};

// Where rows start on 32-byte boundaries the sectors that hold one of the n columns
// are read whole.
template <typename T, bool WHOLE, int N>
__device__ __forceinline__ void fetch(const Plane& pl, int64_t row, int col, int n,
                                      Fetched<T, WHOLE, N>& f) {
  constexpr int kWords = Fetched<T, WHOLE, N>::kWords;
  const T* p = static_cast<const T*>(pl.p) + row * pl.stride + col;
  if constexpr (WHOLE) {
#pragma unroll
    for (int q = 0; q < kWords; q += 8) {
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (n * static_cast<int>(sizeof(T)) > 4 * q) ld_global_v8(reinterpret_cast<const uint32_t*>(p) + q, a, b);
      f.w[q] = a.x; f.w[q + 1] = a.y; f.w[q + 2] = a.z; f.w[q + 3] = a.w;
      f.w[q + 4] = b.x; f.w[q + 5] = b.y; f.w[q + 6] = b.z; f.w[q + 7] = b.w;
    }
  } else {
    f.by = reinterpret_cast<uintptr_t>(p) & 15u;
    const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - f.by);
#pragma unroll
    for (int c = 0; c <= kWords / 4; ++c) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (n > 0 && 16 * c < static_cast<int>(f.by) + min(n, N) * static_cast<int>(sizeof(T))) u = q[c];
      f.w[4 * c] = u.x; f.w[4 * c + 1] = u.y; f.w[4 * c + 2] = u.z; f.w[4 * c + 3] = u.w;
    }
  }
}

// Columns from n on are 0.
template <typename T, bool WHOLE, int N>
__device__ __forceinline__ void values_of(Fetched<T, WHOLE, N>& f, int n, float (&x)[N]) {
  if constexpr (!WHOLE) shift_words<T, Fetched<T, WHOLE, N>::kWords>(f.w, f.by);
  to_floats<T>(f.w, x);
  if (n < N) {
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = k < n ? x[k] : 0.f;
  }
}

// ---- the code --------------------------------------------------------------
// Biased exponent of the scale of a block with largest magnitude amax
// (0 <= amax, or NaN / infinity): with amax = m * 2^k, 1 <= m < 2, and
// 127 * 2^e = (127/64) 2^(e+6), e is k - 6, and one more where m > 127/64
// (mantissa bits above 0x7E0000), at least -126.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int b = static_cast<int>((bits + 0x1FFFFu) >> 23) - 6;
  return bits >= 0x7F800000u ? 255 : max(b, 1);
}

__device__ __forceinline__ float exponent_value(int b) {   // 2^(b - 127); infinity for 255
  return __uint_as_float(static_cast<uint32_t>(b) << 23);
}

// max(|a|, |b|), with a sign that the caller drops; NaN if either is.
__device__ __forceinline__ float max_magnitude(float a, float b) {
  float m;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// Largest magnitude of a block from the values of its 32 / N threads; NaN if one is.
template <int N>
__device__ __forceinline__ float block_amax(const float (&x)[N]) {
  float m = x[0];
#pragma unroll
  for (int k = 1; k < N; ++k) m = max_magnitude(m, x[k]);
#pragma unroll
  for (int o = 1; o < kBlock / N; o *= 2) m = max_magnitude(m, __shfl_xor_sync(0xffffffffu, m, o));
  return fabsf(m);
}

// Codes and biased exponent of this thread's values; the whole warp calls it.
// x / 2^e is exact, and adding 1.5 * 2^23 rounds it to the nearest integer, ties
// to even, whose two's complement is the sum's low byte.
template <int N>
struct Codes {
  uint32_t w[N / 4];
  int b;
};

template <int N>
__device__ __forceinline__ Codes<N> encode(const float (&x)[N]) {
  Codes<N> out;
  out.b = scale_exponent(block_amax(x));
  // 2^-e: the biased exponent of the reciprocal is 254 - b, in [5, 253]
  const float inv = out.b == 255 ? 0.f : exponent_value(254 - out.b);
  uint32_t c[N];
#pragma unroll
  for (int k = 0; k < N; ++k) c[k] = __float_as_uint(fmaf(x[k], inv, 12582912.f));
  if (out.b == 249) {   // 64 * 2^122 would overflow
#pragma unroll
    for (int k = 0; k < N; ++k)
      c[k] = __float_as_uint(fminf(fmaxf(x[k] * inv, -63.f), 63.f) + 12582912.f);
  }
#pragma unroll
  for (int k = 0; k < N / 4; ++k)
    out.w[k] = __byte_perm(__byte_perm(c[4 * k], c[4 * k + 1], 0x0040),
                           __byte_perm(c[4 * k + 2], c[4 * k + 3], 0x0040), 0x5410);
  return out;
}

template <int N>
__device__ __forceinline__ void store_codes(const Packed& out, int64_t row, int col, const Codes<N>& c) {
  int8_t* p = out.codes + row * out.code_stride + col;
  if constexpr (N == 16)
    *reinterpret_cast<uint4*>(p) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
  else if constexpr (N == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(c.w[0], c.w[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = c.w[0];
  if (col % kBlock == 0) out.exps[row * out.exp_stride + col / kBlock] = static_cast<uint8_t>(c.b);
}

// Quantises the values of this thread; the whole warp calls it.
__device__ __forceinline__ void write_codes(const Packed& out, int64_t row, int col,
                                            const float (&x)[kCols], bool on) {
  const Codes<kCols> c = encode(x);
  if (on) store_codes(out, row, col, c);
}

// ---- host ------------------------------------------------------------------
inline int64_t blocks_of(int cols) { return (static_cast<int64_t>(cols) + kBlock - 1) / kBlock; }

inline muon_status_t check_act8(const muon_act8_t* a) {
  if (a == nullptr || a->rows < 0 || a->cols < 1) return MUON_ERR_INVALID_ARG;
  if (a->cols > (1 << 26)) return MUON_ERR_UNSUPPORTED;
  if (a->code_stride < a->cols || a->exp_stride < blocks_of(a->cols)) return MUON_ERR_INVALID_ARG;
  if (a->rows > 0 && (a->codes == nullptr || a->exps == nullptr)) return MUON_ERR_INVALID_ARG;
  if (a->code_stride % kBlock != 0 || a->exp_stride % 16 != 0 || !at_multiple(a->codes, 16) ||
      !at_multiple(a->exps, 16))
    return MUON_ERR_MISALIGNED;
  return MUON_OK;
}

inline Packed packed(const muon_act8_t* a) { return {a->codes, a->code_stride, a->exps, a->exp_stride}; }

inline bool rows_aligned(const Plane& p, int dtype) {
  return p.p == nullptr || (at_multiple(p.p, 32) && p.stride * esize(dtype) % 32 == 0);
}

inline Plane plane(const void* p, int64_t stride) { return {const_cast<void*>(p), stride}; }

}  // namespace muon
