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
// Columns col .. col + 15 of a row, of which n are in the row (the others are
// 0).  WHOLE: rows start on 32-byte boundaries.
template <typename T, bool WHOLE>
__device__ __forceinline__ void load_values(const Plane& pl, int64_t row, int col, int n,
                                            float (&x)[kCols]) {
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
template <typename T, bool WHOLE>
__device__ __forceinline__ void store_values(const Plane& pl, int64_t row, int col, int n,
                                             const float (&x)[kCols]) {
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
    store_shifted(p, n, lane > 0 && col > 0, lane < 31 ? min(max(n - kCols, 0), kCols) : 0, x);
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

// Largest magnitude of a block from its two threads' values; NaN if one is.
__device__ __forceinline__ float block_amax(const float (&x)[kCols]) {
  float m = x[0];
#pragma unroll
  for (int k = 1; k < kCols; ++k) m = max_magnitude(m, x[k]);
  return fabsf(max_magnitude(m, __shfl_xor_sync(0xffffffffu, m, 1)));
}

// Codes and biased exponent of this thread's values; the whole warp calls it.
// x / 2^e is exact, and adding 1.5 * 2^23 rounds it to the nearest integer, ties
// to even, whose two's complement is the sum's low byte.
struct Codes {
  uint4 w;
  int b;
};

__device__ __forceinline__ Codes encode(const float (&x)[kCols]) {
  const int b = scale_exponent(block_amax(x));
  // 2^-e: the biased exponent of the reciprocal is 254 - b, in [5, 253]
  const float inv = b == 255 ? 0.f : exponent_value(254 - b);
  uint32_t c[kCols];
#pragma unroll
  for (int k = 0; k < kCols; ++k) c[k] = __float_as_uint(fmaf(x[k], inv, 12582912.f));
  if (b == 249) {   // 64 * 2^122 would overflow
#pragma unroll
    for (int k = 0; k < kCols; ++k)
      c[k] = __float_as_uint(fminf(fmaxf(x[k] * inv, -63.f), 63.f) + 12582912.f);
  }
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = __byte_perm(__byte_perm(c[4 * k], c[4 * k + 1], 0x0040),
                       __byte_perm(c[4 * k + 2], c[4 * k + 3], 0x0040), 0x5410);
  return {make_uint4(w[0], w[1], w[2], w[3]), b};
}

__device__ __forceinline__ void store_codes(const Packed& out, int64_t row, int col, const Codes& c) {
  *reinterpret_cast<uint4*>(out.codes + row * out.code_stride + col) = c.w;
  if (col % kBlock == 0) out.exps[row * out.exp_stride + col / kBlock] = static_cast<uint8_t>(c.b);
}

// Quantises the values of this thread; the whole warp calls it.
__device__ __forceinline__ void write_codes(const Packed& out, int64_t row, int col,
                                            const float (&x)[kCols], bool on) {
  const Codes c = encode(x);
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
