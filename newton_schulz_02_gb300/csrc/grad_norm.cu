// Norm of all gradients of a model together and the factor that clips it
// (muon_grad_norm).
//
//   n = sqrt(sum over all tensors of g^2),  scale = min(1, max_norm / (n + 1e-6))
//
// One pass: every gradient is read once, and nothing else of size is moved (the
// optimizer steps multiply by the scale where they read the gradient), so HBM's
// read rate is the bound.  Tensors of any number and size share a launch: a
// persistent grid strides over fixed pieces of every tensor.
//
// A thread adds the squares of 32 values (64 of bf16) in fp32, which leaves at most 11
// roundings in a chain (11 x 2^-24 of the sum, half of that of the norm; 1.1e-8 of the sum
// was seen for Gaussian bf16, whose squares end in few bits and round down more often than
// up).  Those sums are added in a pair of fp32 (the rounding error of each addition is kept in
// the second), which costs 7 additions for 32 values and holds 48 bits; an fp64 addition
// for each value would take five times as long as the reads.  Squares outside fp32's
// comfortable range (that sum below 2^-96 or above 2^80, infinite or NaN)
// are added up in fp64 instead, value by value.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "internal.h"
#include "planes.cuh"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;                                       // values of a vector
// Vectors of a thread in a piece, 128 bytes of either type (0.54 G values of bf16: 154 us,
// with 64 bytes 159).
constexpr int kUnrollBf16 = 8, kUnrollF32 = 4;
int64_t piece_values(int dtype) {
  return int64_t{kThreads} * kVec * (dtype == MUON_BF16 ? kUnrollBf16 : kUnrollF32);
}
constexpr int kMaxGroups = 64;                                // groups of a launch
constexpr int kFinThreads = 256;
constexpr int kBlocksPerSm = 3;
constexpr size_t kHeader = 256;

struct NormGroup {
  const void* const* ptrs;
  int64_t vecs;              // whole vectors of a tensor
  int64_t pieces;            // pieces of a tensor
  int64_t stride;            // vectors between rows; 0: one run of values
  Divider per_row;           // vectors of a row
  int tail;                  // values after the last whole vector
  int dtype;
};

struct NormArgs {
  int groups;
  int64_t begin[kMaxGroups + 1];   // first piece of a group
  NormGroup g[kMaxGroups];
  float2* sums;                    // [blocks] of this launch: the pairs,
  double* wide;                    // [blocks] what is not in them,
  uint32_t* flags;                 // [blocks] and conditions
};

constexpr uint32_t kFlagWide = 1u << 31;   // of a block: there is something in its `wide`

struct Sum {
  float hi, lo;    // hi + lo
  double wide;     // what does not fit there
};

// (hi, lo) += (h, l); |lo| stays within a rounding of hi.
__device__ __forceinline__ void add_pair(Sum& s, float h, float l) {
  const float t = s.hi + h, b = t - s.hi;
  const float e = (s.hi - (t - b)) + (h - b) + (s.lo + l);
  s.hi = t + e;
  s.lo = e - (s.hi - t);
}

// Value k of a vector as it was loaded.
__device__ __forceinline__ float value(const uint4 (&u)[1], int k) {   // bf16
  const uint32_t w = k < 2 ? u[0].x : k < 4 ? u[0].y : k < 6 ? u[0].z : u[0].w;
  return __uint_as_float(k % 2 ? w & 0xFFFF0000u : w << 16);
}
__device__ __forceinline__ float value(const uint4 (&u)[2], int k) {   // fp32
  const uint4& v = u[k / 4];
  return __uint_as_float(k % 4 == 0 ? v.x : k % 4 == 1 ? v.y : k % 4 == 2 ? v.z : v.w);
}

// Adds the squares of a thread's values of a piece, WORDS 16-byte words a vector.
template <int WORDS, int N>
__device__ __forceinline__ void add_squares(Sum& s, const uint4 (&u)[N][WORDS]) {
  float part[N];
#pragma unroll
  for (int r = 0; r < N; ++r) {
    part[r] = value(u[r], 0) * value(u[r], 0);
#pragma unroll
    for (int k = 1; k < kVec; ++k) part[r] = fmaf(value(u[r], k), value(u[r], k), part[r]);
  }
#pragma unroll
  for (int half = N / 2; half >= 1; half /= 2)
#pragma unroll
    for (int r = 0; r < half; ++r) part[r] += part[r + half];
  const float sq = part[0];
  if (sq >= 0x1p-96f && sq <= 0x1p80f) {
    const float t = s.hi + sq, b = t - s.hi;
    s.lo += (s.hi - (t - b)) + (sq - b);
    s.hi = t;
    return;
  }
  if (sq == 0.f) {   // nearly always nothing but zeros: an expert without tokens
    uint32_t any = 0;
#pragma unroll
    for (int r = 0; r < N; ++r)
#pragma unroll
      for (int w = 0; w < WORDS; ++w) any |= u[r][w].x | u[r][w].y | u[r][w].z | u[r][w].w;
    if ((any & 0x7FFF7FFFu) == 0 && (WORDS == 1 || (any & 0x7FFFFFFFu) == 0)) return;
  }
#pragma unroll
  for (int r = 0; r < N; ++r)
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const double v = value(u[r], k);
      s.wide = fma(v, v, s.wide);
    }
}

// Loads a thread's vectors of a piece, which begins at vector v0 of the tensor at p (0
// where there is none), and adds their squares.
template <int WORDS, int N>
__device__ __forceinline__ void add_piece(Sum& s, const NormGroup& G, const char* p, int64_t v0, int tid) {
  int64_t at[N];   // vectors from the tensor's start; -1: none
  if (G.stride == 0) {
#pragma unroll
    for (int r = 0; r < N; ++r) {
      const int64_t v = v0 + r * kThreads + tid;
      at[r] = v < G.vecs ? v : -1;
    }
  } else {
    const int64_t row0 = v0 / G.per_row.d;
    const uint32_t col0 = static_cast<uint32_t>(v0 - row0 * G.per_row.d);
#pragma unroll
    for (int r = 0; r < N; ++r) {
      const uint32_t c = col0 + r * kThreads + tid;
      const uint32_t down = quotient(c, G.per_row);
      at[r] = v0 + r * kThreads + tid < G.vecs ? (row0 + down) * G.stride + (c - down * G.per_row.d) : -1;
    }
  }
  uint4 u[N][WORDS];
#pragma unroll
  for (int r = 0; r < N; ++r)
#pragma unroll
    for (int w = 0; w < WORDS; ++w) {
      u[r][w] = make_uint4(0, 0, 0, 0);
      if (at[r] >= 0) u[r][w] = reinterpret_cast<const uint4*>(p)[WORDS * at[r] + w];
    }
  add_squares(s, u);
}

// Pieces first, first + step, ... of all tensors, thread tid of the kThreads that
// take a piece; sets *flags.
__device__ __forceinline__ Sum sum_pieces(const NormArgs& a, int64_t first, int64_t step, int tid,
                                          uint32_t* flags) {
  const int64_t total = a.begin[a.groups];
  Sum s{0.f, 0.f, 0.0};
  int gi = 0;
  for (int64_t item = first; item < total; item += step) {
    while (item >= a.begin[gi + 1]) ++gi;
    const NormGroup& G = a.g[gi];
    const int64_t local = item - a.begin[gi];
    const int64_t tensor = local / G.pieces;
    const int64_t piece = local - tensor * G.pieces;
    const char* p = static_cast<const char*>(G.ptrs[tensor]);
    if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0) {
      *flags |= MUON_FLAG_MISALIGNED;
      continue;   // the tensor is left out
    }
    if (G.dtype == MUON_BF16)
      add_piece<1, kUnrollBf16>(s, G, p, piece * kThreads * kUnrollBf16, tid);
    else
      add_piece<2, kUnrollF32>(s, G, p, piece * kThreads * kUnrollF32, tid);
    if (G.tail > 0 && piece == G.pieces - 1 && tid < G.tail) {   // fewer than 8 values
      const int64_t i = G.vecs * kVec + tid;
      const float v = G.dtype == MUON_BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i])
                                           : reinterpret_cast<const float*>(p)[i];
      s.wide = fma(static_cast<double>(v), static_cast<double>(v), s.wide);
    }
  }
  return s;
}

// The sum over a block of THREADS, in a fixed order, in thread 0; *all: the flags of
// all threads.  In fp32 pairs: an fp64 addition of every thread of a warp takes 16
// clocks of an SM, and made 1.9 us of a small call.
template <int THREADS>
__device__ __forceinline__ Sum block_sum(Sum s, uint32_t flags, uint32_t* all) {
  constexpr int kWarps = THREADS / 32;
  __shared__ float2 red[kWarps];
  __shared__ double red_wide[kWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    add_pair(s, __shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o));
  if (lane == 0) red[w] = make_float2(s.hi, s.lo);
  const int bad = __syncthreads_or(flags & MUON_FLAG_MISALIGNED);
  const int wide = __syncthreads_or(!(s.wide == 0.0));   // or NaN
  *all = (bad ? MUON_FLAG_MISALIGNED : 0u) | (wide ? kFlagWide : 0u);
  if (wide) {   // rare: the same for all threads
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s.wide += __shfl_xor_sync(0xffffffffu, s.wide, o);
    if (lane == 0) red_wide[w] = s.wide;
    __syncthreads();
  }
  if (w == 0) {
    const float2 v = lane < kWarps ? red[lane] : make_float2(0.f, 0.f);
    s.hi = v.x;
    s.lo = v.y;
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1)
      add_pair(s, __shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o));
    s.wide = 0.0;
    if (wide)
      for (int k = 0; k < kWarps; ++k) s.wide += red_wide[k];
  }
  return s;
}

// Three blocks an SM: without the bound the fp64 path takes 124 registers and two fit
// (0.54 G bf16 169 us); four spill (353).
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) k_grad_norm(const __grid_constant__ NormArgs a) {
  griddep_launch_dependents();
  uint32_t flags = 0;
  const Sum mine = sum_pieces(a, blockIdx.x, gridDim.x, threadIdx.x, &flags);
  const Sum s = block_sum<kThreads>(mine, flags, &flags);
  if (threadIdx.x == 0) {
    a.sums[blockIdx.x] = make_float2(s.hi, s.lo);
    a.wide[blockIdx.x] = s.wide;
    a.flags[blockIdx.x] = flags;
  }
}

struct FinishArgs {
  const float2* sums;
  const double* wide;
  const uint32_t* flags;
  int blocks;
  float max_norm;
  float* norm;
  float* scale;
  uint32_t* status;
};

// The norm and the factor.  From the pair alone in fp32 pairs, too: a root and a quotient
// with what their first values leave over: in fp64 they take 0.7 us of a call's 4.
__device__ __forceinline__ void write_norm(const FinishArgs& a, const Sum& s, uint32_t flags) {
  uint32_t status = flags & MUON_FLAG_MISALIGNED;
  if (flags & kFlagWide) {
    const double n = sqrt((static_cast<double>(s.hi) + static_cast<double>(s.lo)) + s.wide);
    const bool finite = isfinite(n);
    if (!finite) status |= MUON_FLAG_NONFINITE;
    *a.norm = static_cast<float>(n);
    *a.scale = finite ? static_cast<float>(fmin(1.0, static_cast<double>(a.max_norm) / (n + 1e-6)))
                      : __uint_as_float(0x7FC00000u);
  } else {
    const float n = sqrtf(s.hi);
    const float rest = s.hi > 0.f ? (fmaf(-n, n, s.hi) + s.lo) / (2.f * n) : 0.f;   // n + rest is the norm
    const float d = n + 1e-6f, big = fmaxf(n, 1e-6f);
    const float low = rest + (fminf(n, 1e-6f) - (d - big));                         // d + low divides
    const float q = a.max_norm / d;
    *a.norm = n + rest;
    *a.scale = q >= 1.f + 0x1p-20f ? 1.f : fminf(1.f, q + (fmaf(-q, d, a.max_norm) - q * low) / d);
  }
  *a.status = status;
}

__global__ void __launch_bounds__(kFinThreads) k_grad_norm_finish(FinishArgs a) {
  griddep_wait();
  Sum s{0.f, 0.f, 0.0};
  uint32_t flags = 0;
  for (int i = threadIdx.x; i < a.blocks; i += kFinThreads) {
    const float2 v = a.sums[i];
    add_pair(s, v.x, v.y);
    const uint32_t f = a.flags[i];
    if (f & kFlagWide) s.wide += a.wide[i];
    flags |= f;
  }
  s = block_sum<kFinThreads>(s, flags, &flags);
  if (threadIdx.x == 0) write_norm(a, s, flags);
}

// Blocks of a launch: as many as run at once on the current device, at most one a piece.
cudaError_t resident_blocks(int* out) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  *out = sms * kBlocksPerSm;
  return e;
}

constexpr int kMaxBlocks = 2048;    // of a launch
constexpr size_t kBlockBytes = 20;  // a pair, a double and the conditions

bool empty(const muon_grads_t& g) { return g.count == 0 || g.rows == 0 || g.cols == 0; }

muon_status_t check_grads(const muon_grads_t* g, int n_groups, int* used) {
  if (n_groups < 0 || (n_groups > 0 && g == nullptr)) return MUON_ERR_INVALID_ARG;
  *used = 0;
  for (int i = 0; i < n_groups; ++i) {
    if (g[i].count < 0 || g[i].rows < 0 || g[i].cols < 0) return MUON_ERR_INVALID_ARG;
    if (g[i].dtype != MUON_BF16 && g[i].dtype != MUON_F32) return MUON_ERR_INVALID_ARG;
    if (empty(g[i])) continue;
    if (g[i].ptrs == nullptr) return MUON_ERR_INVALID_ARG;
    if (!at_multiple(g[i].ptrs, 8)) return MUON_ERR_MISALIGNED;
    if (g[i].rows > 1) {
      if (g[i].row_stride < g[i].cols) return MUON_ERR_INVALID_ARG;
      if (g[i].row_stride > g[i].cols) {
        if (g[i].cols % kVec != 0 || g[i].cols > (int64_t{1} << 32)) return MUON_ERR_UNSUPPORTED;
        if (g[i].row_stride % kVec != 0) return MUON_ERR_MISALIGNED;
      }
      if (g[i].rows > (int64_t{1} << 62) / g[i].row_stride) return MUON_ERR_UNSUPPORTED;
    }
    ++*used;
  }
  return MUON_OK;
}

int launches_of(int used) { return (used + kMaxGroups - 1) / kMaxGroups; }

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status_t muon_grad_norm_workspace_size(const muon_grads_t* groups, int n_groups, size_t* bytes) {
  if (bytes == nullptr) return MUON_ERR_INVALID_ARG;
  int used = 0;
  const muon_status_t s = check_grads(groups, n_groups, &used);
  if (s != MUON_OK) return s;
  *bytes = kHeader + static_cast<size_t>(launches_of(used)) * kMaxBlocks * kBlockBytes;
  return MUON_OK;
}

muon_status_t muon_grad_norm(const muon_grads_t* groups, int n_groups, float max_norm, float* norm,
                             float* scale, void* workspace, size_t workspace_bytes,
                             muon_stream_t stream) {
  int used = 0;
  muon_status_t s = check_grads(groups, n_groups, &used);
  if (s != MUON_OK) return s;
  if (!(max_norm >= 0.f) || norm == nullptr || scale == nullptr || workspace == nullptr)
    return MUON_ERR_INVALID_ARG;
  if (!at_multiple(norm, 4) || !at_multiple(scale, 4) || !at_multiple(workspace, 256))
    return MUON_ERR_MISALIGNED;
  size_t need = 0;
  s = muon_grad_norm_workspace_size(groups, n_groups, &need);
  if (s != MUON_OK) return s;
  if (workspace_bytes < need) return MUON_ERR_WORKSPACE_TOO_SMALL;

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const size_t most = static_cast<size_t>(launches_of(used)) * kMaxBlocks;
  double* wide = reinterpret_cast<double*>(ws + kHeader);
  float2* sums = reinterpret_cast<float2*>(wide + most);
  uint32_t* flags = reinterpret_cast<uint32_t*>(sums + most);
  FinishArgs f{sums, wide, flags, 0, max_norm, norm, scale, reinterpret_cast<uint32_t*>(ws)};
  int resident = 0;
  if (resident_blocks(&resident) != cudaSuccess) return MUON_ERR_CUDA;
  if (resident > kMaxBlocks) resident = kMaxBlocks;
  for (int next = 0; next < n_groups;) {
    NormArgs a{};
    double bytes = 0.0;
    for (; next < n_groups && a.groups < kMaxGroups; ++next) {
      const muon_grads_t& src = groups[next];
      if (empty(src)) continue;
      NormGroup& g = a.g[a.groups];
      const int64_t values = src.rows * src.cols;
      const bool strided = src.rows > 1 && src.row_stride > src.cols;
      g.ptrs = src.ptrs;
      g.vecs = values / kVec;
      g.tail = static_cast<int>(values % kVec);
      g.pieces = (values + piece_values(src.dtype) - 1) / piece_values(src.dtype);
      g.stride = strided ? src.row_stride / kVec : 0;
      g.per_row = divider(strided ? static_cast<uint32_t>(src.cols / kVec) : 1);
      g.dtype = src.dtype;
      a.begin[a.groups + 1] = a.begin[a.groups] + g.pieces * src.count;
      bytes += static_cast<double>(values) * src.count * esize(src.dtype);
      ++a.groups;
    }
    const int64_t items = a.begin[a.groups];
    if (items == 0) break;
    const int grid = static_cast<int>(items < resident ? items : resident);
    a.sums = sums + f.blocks;
    a.wide = wide + f.blocks;
    a.flags = flags + f.blocks;
    f.blocks += grid;
    prof_begin(kKindGradNorm, st);
    k_grad_norm<<<grid, kThreads, 0, st>>>(a);
    prof_end(kKindGradNorm, st, 0.0, bytes);
    if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
  }
  // a programmatic dependent of the last kernel before (it waits for the sums)
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kFinThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = f.blocks > 0 ? 1 : 0;
  prof_begin(kKindGradNorm, st);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_grad_norm_finish, f);
  prof_end(kKindGradNorm, st, 0.0, 12.0 * f.blocks);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

}  // extern "C"
