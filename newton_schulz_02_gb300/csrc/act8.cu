// Activations held in 8 bits between the forward and the backward pass, and
// the gated feed-forward activation on them (muon_act8_pack, _unpack,
// _swiglu_forward, _swiglu_backward).
//
// A block of 32 columns of a row shares a power-of-two scale 2^e, so both
// directions are exact but for the one rounding of x / 2^e to an integer, and
// a code's value (7 significant bits) is exact in bf16.  A power of two costs
// up to one of the eight bits against a free scale; in return the code's
// value needs no rounding where the tensor cores read it.
//
// All four passes are bound by HBM: each value is read once and written once.
// A thread takes 16 consecutive columns; two threads share a block's maximum by
// one shuffle.  Where every row starts on a 32-byte boundary a thread writes
// whole 32-byte sectors.  Elsewhere (an odd width, a shifted view) it reads the
// 16-byte pieces that hold its columns and shifts them into place, and writes
// the 16-byte pieces that begin in its columns, with the next thread's first
// values in the last.  One column a thread coalesces at any alignment too, and
// took 3 to 6 times as long.  Measured at 16384 rows, in us (and the share of
// the copy rate):
//                       pack        unpack      forward     backward with h8
//   7168 bf16           56 (94%)    54 (98%)    153 (91%)   164 (96%)
//   7001 bf16           62 (83%)    66 (78%)    177 (77%)   201 (76%)
//   7168 fp32           84 (103%)   88 (99%)    234 (104%)  254 (103%)
//   7001 fp32           86 (99%)    117 (73%)   248 (96%)   294 (87%)
// The shifted rows are not bound by HBM (42 to 59% busy where 7168 columns have it
// 60 to 74%, 8192 rows bf16): shifting is half as many instructions again (issue 65 to
// 77% busy), and a sector goes out in two pieces (10.7 against 5.5 million sector
// writes at L2 for unpack, L1 78% busy).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 32;   // columns that share a scale

// Quotient by a fixed divisor of numbers below 2^31: with l = ceil(log2 d) and
// m = ceil(2^(31+l) / d), m*d exceeds 2^(31+l) by less than 2^l, so the
// product's error stays below one part in n for n < 2^31.
struct Divider {
  uint32_t mul, shift, d;
};

Divider divider(uint32_t d) {
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

struct Act8Args {
  uint32_t items;       // threads' work items: rows x items of a row
  int cols;
  Divider per_row;      // items of a row
  Plane x, y, z;        // roles by kernel
  Packed a, b, c;
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

// Quantises the values of this thread; the whole warp calls it.  x / 2^e is
// exact, and adding 1.5 * 2^23 rounds it to the nearest integer, ties to even,
// whose two's complement is the sum's low byte.
__device__ __forceinline__ void write_codes(const Packed& out, int64_t row, int col,
                                            const float (&x)[kCols], bool on) {
  const int b = scale_exponent(block_amax(x));
  // 2^-e: the biased exponent of the reciprocal is 254 - b, in [5, 253]
  const float inv = b == 255 ? 0.f : exponent_value(254 - b);
  if (!on) return;
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
  *reinterpret_cast<uint4*>(out.codes + row * out.code_stride + col) = make_uint4(w[0], w[1], w[2], w[3]);
  if (col % kBlock == 0) out.exps[row * out.exp_stride + col / kBlock] = static_cast<uint8_t>(b);
}

// Values of 16 codes.  Biased by 128 a code is the low byte of 2^23 + 128 +
// code, so a byte permute and a subtraction make the float (the conversion
// unit is needed for the exponentials), and times 2^e is exact.
__device__ __forceinline__ void read_codes(const Packed& in, int64_t row, int col, float (&x)[kCols]) {
  const int b = in.exps[row * in.exp_stride + col / kBlock];
  const float s = b == 255 ? __uint_as_float(0x7FC00000u) : exponent_value(b);
  const uint4 u = *reinterpret_cast<const uint4*>(in.codes + row * in.code_stride + col);
  const uint32_t w[4] = {u.x ^ 0x80808080u, u.y ^ 0x80808080u, u.z ^ 0x80808080u, u.w ^ 0x80808080u};
#pragma unroll
  for (int k = 0; k < kCols; ++k)
    x[k] = (__uint_as_float(__byte_perm(w[k / 4], 0x4B000000u, 0x7440 + k % 4)) - 8388736.f) * s;
}

struct Place {
  int64_t row;
  int col, n;    // n: columns of this item inside the row (<= 0: padding of the last block)
  bool on;
};

__device__ __forceinline__ Place place(const Act8Args& a) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  Place p;
  p.on = i < a.items;
  const uint32_t at = p.on ? i : a.items - 1;
  const uint32_t row = quotient(at, a.per_row);
  p.row = row;
  p.col = static_cast<int>(at - row * a.per_row.d) * kCols;
  p.n = p.on ? a.cols - p.col : 0;
  return p;
}

template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kThreads) k_act8_pack(const __grid_constant__ Act8Args a) {
  const Place p = place(a);
  float x[kCols];
  load_values<T, WHOLE>(a.x, p.row, p.col, p.n, x);
  write_codes(a.a, p.row, p.col, x, p.on);
}

template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kThreads) k_act8_unpack(const __grid_constant__ Act8Args a) {
  const Place p = place(a);
  float x[kCols];
  read_codes(a.a, p.row, p.col, x);
  store_values<T, WHOLE>(a.x, p.row, p.col, p.n, x);
}

// 1 / (1 + e^-g) with the fast exponential and reciprocal: an error of a few
// units plus (1 - sigma) |g| units in the last place.  (With expf and a division
// fp32 rows of 7001 columns take 266 us forward and 333 backward instead of 248 and 294.)
__device__ __forceinline__ float sigma(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

// x = gate, y = up, z = h; a, b = the checkpoints of gate and up.
template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kThreads) k_act8_swiglu_forward(const __grid_constant__ Act8Args a) {
  const Place p = place(a);
  float g[kCols], u[kCols], h[kCols];
  load_values<T, WHOLE>(a.x, p.row, p.col, p.n, g);
  load_values<T, WHOLE>(a.y, p.row, p.col, p.n, u);
  write_codes(a.a, p.row, p.col, g, p.on);
  write_codes(a.b, p.row, p.col, u, p.on);
#pragma unroll
  for (int k = 0; k < kCols; ++k) h[k] = g[k] * sigma(g[k]) * u[k];
  store_values<T, WHOLE>(a.z, p.row, p.col, p.n, h);
}

// x = dh, y = dgate, z = dup; a, b = the checkpoints of gate and up, c = h8.
// Four blocks an SM (64 registers) and the codes read first: 165 us at 16384 x
// 7168 bf16, 179 without the bound, 186 with dh read first.
template <typename T, bool WHOLE, bool H8>
__global__ void __launch_bounds__(kThreads, 4) k_act8_swiglu_backward(const __grid_constant__ Act8Args a) {
  const Place p = place(a);
  float g[kCols], u[kCols], d[kCols], h[H8 ? kCols : 1];
  read_codes(a.a, p.row, p.col, g);
  read_codes(a.b, p.row, p.col, u);
  load_values<T, WHOLE>(a.x, p.row, p.col, p.n, d);
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
    const float s = sigma(g[k]);
    const float act = g[k] * s;
    if (H8) h[k] = k < p.n ? act * u[k] : 0.f;
    const float dg = d[k] * u[k] * fmaf(act, 1.f - s, s);
    u[k] = d[k] * act;
    g[k] = dg;
  }
  if constexpr (!WHOLE) __syncwarp();   // dh may be dgate or dup: the warp's reads are over
  if (!WHOLE || p.on) {   // the others exchange their ends: the whole warp
    store_values<T, WHOLE>(a.y, p.row, p.col, p.n, g);
    store_values<T, WHOLE>(a.z, p.row, p.col, p.n, u);
  }
  if constexpr (H8) write_codes(a.c, p.row, p.col, h, p.on);
}

// ---- host ------------------------------------------------------------------
int64_t blocks_of(int cols) { return (static_cast<int64_t>(cols) + kBlock - 1) / kBlock; }

muon_status_t check_act8(const muon_act8_t* a) {
  if (a == nullptr || a->rows < 0 || a->cols < 1) return MUON_ERR_INVALID_ARG;
  if (a->cols > (1 << 26)) return MUON_ERR_UNSUPPORTED;
  if (a->code_stride < a->cols || a->exp_stride < blocks_of(a->cols)) return MUON_ERR_INVALID_ARG;
  if (a->rows > 0 && (a->codes == nullptr || a->exps == nullptr)) return MUON_ERR_INVALID_ARG;
  if (a->code_stride % kBlock != 0 || a->exp_stride % 16 != 0 || !at_multiple(a->codes, 16) ||
      !at_multiple(a->exps, 16))
    return MUON_ERR_MISALIGNED;
  return MUON_OK;
}

muon_status_t check_plane(const void* p, int64_t stride, int dtype, const muon_act8_t* like) {
  if (dtype != MUON_BF16 && dtype != MUON_F32) return MUON_ERR_INVALID_ARG;
  if (stride < like->cols || (like->rows > 0 && p == nullptr)) return MUON_ERR_INVALID_ARG;
  return at_multiple(p, esize(dtype)) ? MUON_OK : MUON_ERR_MISALIGNED;
}

bool same_size(const muon_act8_t* a, const muon_act8_t* b) {
  return a->rows == b->rows && a->cols == b->cols;
}

Packed packed(const muon_act8_t* a) { return {a->codes, a->code_stride, a->exps, a->exp_stride}; }

bool rows_aligned(const Plane& p, int dtype) {
  return p.p == nullptr || (at_multiple(p.p, 32) && p.stride * esize(dtype) % 32 == 0);
}

enum Pass { kPack, kUnpack, kForward, kBackward, kBackwardH8 };

template <typename T, bool WHOLE>
void launch_pass(Pass pass, unsigned grid, cudaStream_t st, const Act8Args& a) {
  switch (pass) {
    case kPack: k_act8_pack<T, WHOLE><<<grid, kThreads, 0, st>>>(a); break;
    case kUnpack: k_act8_unpack<T, WHOLE><<<grid, kThreads, 0, st>>>(a); break;
    case kForward: k_act8_swiglu_forward<T, WHOLE><<<grid, kThreads, 0, st>>>(a); break;
    case kBackward: k_act8_swiglu_backward<T, WHOLE, false><<<grid, kThreads, 0, st>>>(a); break;
    case kBackwardH8: k_act8_swiglu_backward<T, WHOLE, true><<<grid, kThreads, 0, st>>>(a); break;
  }
}

// Every row's items in one launch, or in several of fewer than 2^30 items.
muon_status_t run_pass(Pass pass, int dtype, int64_t rows, int cols, Act8Args a, double bytes,
                       cudaStream_t st) {
  if (rows == 0) return MUON_OK;
  const bool whole = rows_aligned(a.x, dtype) && rows_aligned(a.y, dtype) && rows_aligned(a.z, dtype);
  const int64_t per_row = blocks_of(cols) * (kBlock / kCols);
  a.cols = cols;
  a.per_row = divider(static_cast<uint32_t>(per_row));
  int64_t most = (int64_t{1} << 30) / per_row;
  if (most < 1) most = 1;
  const KernelKind kind = pass == kPack || pass == kUnpack ? kKindAct8 : kKindSwiglu;
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    const int64_t n = rows - r0 < most ? rows - r0 : most;
    Act8Args b = a;
    b.items = static_cast<uint32_t>(n * per_row);
    for (Plane* p : {&b.x, &b.y, &b.z})
      if (p->p != nullptr) p->p = static_cast<char*>(p->p) + r0 * p->stride * esize(dtype);
    for (Packed* p : {&b.a, &b.b, &b.c})
      if (p->codes != nullptr) {
        p->codes += r0 * p->code_stride;
        p->exps += r0 * p->exp_stride;
      }
    const unsigned grid = (b.items + kThreads - 1) / kThreads;
    prof_begin(kind, st);
    if (dtype == MUON_F32) {
      if (whole) launch_pass<float, true>(pass, grid, st, b);
      else launch_pass<float, false>(pass, grid, st, b);
    } else {
      if (whole) launch_pass<__nv_bfloat16, true>(pass, grid, st, b);
      else launch_pass<__nv_bfloat16, false>(pass, grid, st, b);
    }
    prof_end(kind, st, 0.0, bytes * static_cast<double>(n) * cols);
    if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
  }
  return MUON_OK;
}

constexpr double kCodeBytes = 1.0 + 1.0 / kBlock;

Plane plane(const void* p, int64_t stride) { return {const_cast<void*>(p), stride}; }

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status_t muon_act8_pack(const void* x, muon_dtype_t xdt, int64_t x_stride,
                             const muon_act8_t* out, muon_stream_t stream) {
  muon_status_t s = check_act8(out);
  if (s == MUON_OK) s = check_plane(x, x_stride, xdt, out);
  if (s != MUON_OK) return s;
  Act8Args a{};
  a.x = plane(x, x_stride);
  a.a = packed(out);
  return run_pass(kPack, xdt, out->rows, out->cols, a, esize(xdt) + kCodeBytes,
                  reinterpret_cast<cudaStream_t>(stream));
}

muon_status_t muon_act8_unpack(const muon_act8_t* in, void* x, muon_dtype_t xdt, int64_t x_stride,
                               muon_stream_t stream) {
  muon_status_t s = check_act8(in);
  if (s == MUON_OK) s = check_plane(x, x_stride, xdt, in);
  if (s != MUON_OK) return s;
  Act8Args a{};
  a.x = plane(x, x_stride);
  a.a = packed(in);
  return run_pass(kUnpack, xdt, in->rows, in->cols, a, esize(xdt) + kCodeBytes,
                  reinterpret_cast<cudaStream_t>(stream));
}

muon_status_t muon_act8_swiglu_forward(const void* gate, int64_t gate_stride, const void* up,
                                       int64_t up_stride, muon_dtype_t dt, void* h,
                                       int64_t h_stride, const muon_act8_t* gate8,
                                       const muon_act8_t* up8, muon_stream_t stream) {
  muon_status_t s = check_act8(gate8);
  if (s == MUON_OK) s = check_act8(up8);
  if (s == MUON_OK) s = check_plane(gate, gate_stride, dt, gate8);
  if (s == MUON_OK) s = check_plane(up, up_stride, dt, gate8);
  if (s == MUON_OK) s = check_plane(h, h_stride, dt, gate8);
  if (s != MUON_OK) return s;
  if (!same_size(gate8, up8)) return MUON_ERR_INVALID_ARG;
  Act8Args a{};
  a.x = plane(gate, gate_stride);
  a.y = plane(up, up_stride);
  a.z = plane(h, h_stride);
  a.a = packed(gate8);
  a.b = packed(up8);
  return run_pass(kForward, dt, gate8->rows, gate8->cols, a, 3.0 * esize(dt) + 2 * kCodeBytes,
                  reinterpret_cast<cudaStream_t>(stream));
}

muon_status_t muon_act8_swiglu_backward(const void* dh, int64_t dh_stride, muon_dtype_t dt,
                                        const muon_act8_t* gate8, const muon_act8_t* up8,
                                        void* dgate, int64_t dgate_stride, void* dup,
                                        int64_t dup_stride, const muon_act8_t* h8,
                                        muon_stream_t stream) {
  muon_status_t s = check_act8(gate8);
  if (s == MUON_OK) s = check_act8(up8);
  if (s == MUON_OK && h8 != nullptr) s = check_act8(h8);
  if (s == MUON_OK) s = check_plane(dh, dh_stride, dt, gate8);
  if (s == MUON_OK) s = check_plane(dgate, dgate_stride, dt, gate8);
  if (s == MUON_OK) s = check_plane(dup, dup_stride, dt, gate8);
  if (s != MUON_OK) return s;
  if (!same_size(gate8, up8) || (h8 != nullptr && !same_size(gate8, h8)))
    return MUON_ERR_INVALID_ARG;
  Act8Args a{};
  a.x = plane(dh, dh_stride);
  a.y = plane(dgate, dgate_stride);
  a.z = plane(dup, dup_stride);
  a.a = packed(gate8);
  a.b = packed(up8);
  if (h8 != nullptr) a.c = packed(h8);
  return run_pass(h8 != nullptr ? kBackwardH8 : kBackward, dt, gate8->rows, gate8->cols, a,
                  3.0 * esize(dt) + (h8 != nullptr ? 3 : 2) * kCodeBytes,
                  reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
