// Consecutive columns of a row of bf16 or fp32 (16, or fewer: N) as a thread's values,
// read and written in 16-byte pieces wherever the row starts.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace muon {

constexpr int kCols = 16;   // a thread's columns, where nothing else is said

template <typename T, int N>
__device__ __forceinline__ void to_floats(const uint32_t* w, float (&x)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if constexpr (sizeof(T) == 4)
      x[k] = __uint_as_float(w[k]);
    else   // a bf16 is the upper half of an fp32
      x[k] = __uint_as_float(k % 2 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
  }
}

template <typename T, int N>
__device__ __forceinline__ void to_words(const float (&x)[N], uint32_t* w) {
#pragma unroll
  for (int k = 0; k < N; k += 4 / sizeof(T)) {
    if constexpr (sizeof(T) == 4) {
      w[k] = __float_as_uint(x[k]);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[k], x[k + 1]);
      w[k / 2] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}

__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Words from byte `by` of w on (by < 16, a multiple of sizeof(T)); 4 words more
// than N come in.
template <typename T, int N>
__device__ __forceinline__ void shift_words(uint32_t (&w)[N + 4], uint32_t by) {
#pragma unroll
  for (int k = 0; k < N + 2; ++k) w[k] = by & 8 ? w[k + 2] : w[k];
#pragma unroll
  for (int k = 0; k < N + 1; ++k) w[k] = by & 4 ? w[k + 1] : w[k];
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = by & 2 ? __byte_perm(w[k], w[k + 1], 0x5432) : w[k];
  }
}

// Columns p[0 .. N-1], of which the first n are in the row (the others are 0):
// the 16-byte pieces that hold a byte of them.  A piece may begin before the
// row or end after it; those bytes are shifted out or cleared.
template <typename T, int N>
__device__ __forceinline__ void load_shifted(const T* p, int n, float (&x)[N]) {
  constexpr int kWords = N * sizeof(T) / 4;
  const uint32_t by = reinterpret_cast<uintptr_t>(p) & 15u;
  const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) - by);
  uint32_t w[kWords + 4];
#pragma unroll
  for (int c = 0; c <= kWords / 4; ++c) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (16 * c < static_cast<int>(by) + min(n, N) * static_cast<int>(sizeof(T)) && n > 0) u = q[c];
    w[4 * c] = u.x; w[4 * c + 1] = u.y; w[4 * c + 2] = u.z; w[4 * c + 3] = u.w;
  }
  shift_words<T, kWords>(w, by);
  to_floats<T>(w, x);
  if (n < N) {
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = k < n ? x[k] : 0.f;
  }
}

// The reverse; the whole warp calls it.  A chain of lanes holds consecutive
// columns of a row: `before` says that the lane before this one holds the N
// columns before these, `next` how many columns the lane after it goes on with
// (0 to N; it counts where n >= N).  n <= 0: nothing of this thread's is in the
// row.  A thread writes the 16-byte pieces that begin in its columns, with the
// next lane's first values in the last; a chain's first and last bytes, which
// fill no piece, go out in 8, 4 and 2 bytes.
template <typename T, int N>
__device__ __forceinline__ void store_shifted(T* p, int n, bool before, int next, const float (&x)[N]) {
  constexpr int kWords = N * sizeof(T) / 4;
  constexpr int kSize = sizeof(T);
  uint32_t w[kWords + 4];
  {
    uint32_t mine[kWords];
    to_words<T>(x, mine);
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = mine[k];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) w[kWords + k] = __shfl_down_sync(0xffffffffu, w[k], 1);
  const int head = static_cast<int>(-reinterpret_cast<uintptr_t>(p) & 15u);   // bytes before the first piece
  const int own = min(n, N) * kSize;
  const int all = n >= N ? own + next * kSize : own;
  char* at = reinterpret_cast<char*>(p);
  if (head != 0 && !before && own > 0) {
    if (own < head) {   // a row of a few columns
#pragma unroll
      for (int k = 0; k < 16 / kSize; ++k)
        if (k * kSize < own) store_one(p + k, x[k]);
    } else {
      if (kSize == 2 && head & 2) *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(w[0]);
      const uint32_t a = kSize == 2 && head & 2 ? __byte_perm(w[0], w[1], 0x5432) : w[0];
      const uint32_t b = kSize == 2 && head & 2 ? __byte_perm(w[1], w[2], 0x5432) : w[1];
      const uint32_t c = kSize == 2 && head & 2 ? __byte_perm(w[2], w[3], 0x5432) : w[2];
      if (head & 4) *reinterpret_cast<uint32_t*>(at + (head & 2)) = a;
      if (head & 8)
        *reinterpret_cast<uint2*>(at + (head & 6)) = head & 4 ? make_uint2(b, c) : make_uint2(a, b);
    }
  }
  shift_words<T, kWords>(w, head);
  at += head;
  uint4 last = make_uint4(0, 0, 0, 0);
  int left = 0;   // bytes of the last piece, if not all
#pragma unroll
  for (int c = 0; c < kWords / 4; ++c) {
    const uint4 piece = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    if (head + 16 * c < own) {
      if (head + 16 * c + 16 <= all) {
        *reinterpret_cast<uint4*>(at + 16 * c) = piece;
      } else {
        last = piece;
        left = all - head - 16 * c;
        at += 16 * c;
      }
    }
  }
  if (left > 0) {
    if (left & 8) *reinterpret_cast<uint2*>(at) = make_uint2(last.x, last.y);
    const uint32_t a = left & 8 ? last.z : last.x, b = left & 8 ? last.w : last.y;
    if (left & 4) *reinterpret_cast<uint32_t*>(at + (left & 8)) = a;
    if (kSize == 2 && left & 2)
      *reinterpret_cast<uint16_t*>(at + (left & 12)) = static_cast<uint16_t>(left & 4 ? b : a);
  }
}

}  // namespace muon
