// Weight gradients of a set of experts from 8-bit activation checkpoints
// (muon_act8_weight_grad):
//
//   G_e[o][i] = sum_{t in expert e} dy[t][o] * code[t][i] * 2^(e[t][i/32])
//
// A block computes a 64 x 64 tile of one expert's G: 16 tokens at a time of
// dy and of the decoded x go through shared memory, each thread accumulates
// 4 x 4 sums in fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64, kTok = 16;
constexpr size_t kHeader = 256;

struct WgradArgs {
  int rows, out, in, experts;
  const void* dy;
  int dy_dtype;
  int64_t dy_stride;
  const int8_t* codes;
  int64_t code_stride;
  const uint8_t* exps;
  int64_t exp_stride;
  const int32_t* offsets;
  void* const* g_ptrs;
  void* g_base;
  int64_t g_batch_stride, g_stride;
  int g_dtype, accumulate;
  int tiles_o, tiles_i;
  uint32_t* status;
};

__device__ __forceinline__ void span_of(const WgradArgs& a, int e, int& b, int& n) {
  if (a.offsets == nullptr) {
    b = 0;
    n = a.rows;
    return;
  }
  b = min(max(a.offsets[e], 0), a.rows);
  n = min(max(a.offsets[e + 1], b), a.rows) - b;
}

__global__ void __launch_bounds__(kThreads) k_act8_wgrad(const __grid_constant__ WgradArgs a) {
  __shared__ float sy[kTok][kTile + 4], sx[kTok][kTile + 4];
  const int e = blockIdx.z;
  int begin, n;
  span_of(a, e, begin, n);
  if (a.offsets != nullptr && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) {
    const int b = a.offsets[e], c = a.offsets[e + 1];
    if (b < 0 || c < b || c > a.rows) atomicOr(a.status, MUON_FLAG_INDEX);
  }
  const int o0 = blockIdx.y * kTile, i0 = blockIdx.x * kTile;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int t0 = 0; t0 < n; t0 += kTok) {
    for (int v = threadIdx.x; v < kTok * kTile; v += kThreads) {
      const int r = v / kTile, c = v % kTile;
      const int64_t t = begin + t0 + r;
      float y = 0.f, x = 0.f;
      if (t0 + r < n) {
        if (o0 + c < a.out)
          y = a.dy_dtype == MUON_F32
                  ? static_cast<const float*>(a.dy)[t * a.dy_stride + o0 + c]
                  : __bfloat162float(static_cast<const __nv_bfloat16*>(a.dy)[t * a.dy_stride + o0 + c]);
        if (i0 + c < a.in) {
          const float s = __uint_as_float(
              static_cast<uint32_t>(a.exps[t * a.exp_stride + (i0 + c) / 32]) << 23);
          x = fmaf(static_cast<float>(a.codes[t * a.code_stride + i0 + c]), s, s - s);
        }
      }
      sy[r][c] = y;
      sx[r][c] = x;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kTok; ++r) {
      float y[4], x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        y[k] = sy[r][ty * 4 + k];
        x[k] = sx[r][tx * 4 + k];
      }
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[p][q] = fmaf(y[p], x[q], acc[p][q]);
    }
    __syncthreads();
  }
  void* g = a.g_ptrs != nullptr ? a.g_ptrs[e]
                                : static_cast<char*>(a.g_base) +
                                      e * a.g_batch_stride * (a.g_dtype == MUON_F32 ? 4 : 2);
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int o = o0 + ty * 4 + p, i = i0 + tx * 4 + q;
      if (o >= a.out || i >= a.in) continue;
      const int64_t at = o * a.g_stride + i;
      if (a.g_dtype == MUON_F32) {
        float* w = static_cast<float*>(g) + at;
        *w = a.accumulate ? *w + acc[p][q] : acc[p][q];
      } else {
        __nv_bfloat16* w = static_cast<__nv_bfloat16*>(g) + at;
        *w = __float2bfloat16_rn(a.accumulate ? __bfloat162float(*w) + acc[p][q] : acc[p][q]);
      }
    }
}

int esize(int dtype) { return dtype == MUON_BF16 ? 2 : 4; }

bool at_multiple(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

muon_status_t check_sizes(const muon_weight_grad_t* d) {
  if (d == nullptr || d->rows < 0 || d->out < 1 || d->experts < 1 || d->x.cols < 1)
    return MUON_ERR_INVALID_ARG;
  if (d->dy_dtype != MUON_BF16 && d->dy_dtype != MUON_F32) return MUON_ERR_INVALID_ARG;
  if (d->g_dtype != MUON_BF16 && d->g_dtype != MUON_F32) return MUON_ERR_INVALID_ARG;
  if (d->rows >= (int64_t{1} << 31) - (1 << 20) || d->out > (1 << 22) || d->x.cols > (1 << 22) ||
      d->experts > 65535)
    return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status_t muon_act8_weight_grad_workspace_size(const muon_weight_grad_t* d, size_t* bytes) {
  if (bytes == nullptr) return MUON_ERR_INVALID_ARG;
  const muon_status_t s = check_sizes(d);
  if (s != MUON_OK) return s;
  *bytes = kHeader;
  return MUON_OK;
}

muon_status_t muon_act8_weight_grad(const muon_weight_grad_t* d, void* workspace,
                                    size_t workspace_bytes, muon_stream_t stream) {
  size_t need = 0;
  muon_status_t s = muon_act8_weight_grad_workspace_size(d, &need);
  if (s != MUON_OK) return s;
  const muon_act8_t& x = d->x;
  if (x.rows != d->rows || x.code_stride < x.cols || x.exp_stride * 32 < x.cols)
    return MUON_ERR_INVALID_ARG;
  if (d->rows > 0 && (d->dy == nullptr || x.codes == nullptr || x.exps == nullptr))
    return MUON_ERR_INVALID_ARG;
  if (d->dy_stride < d->out || d->g_stride < x.cols) return MUON_ERR_INVALID_ARG;
  if (d->accumulate != 0 && d->accumulate != 1) return MUON_ERR_INVALID_ARG;
  if (d->offsets == nullptr && d->experts != 1) return MUON_ERR_INVALID_ARG;
  if (d->g_ptrs == nullptr && d->g_base == nullptr) return MUON_ERR_INVALID_ARG;
  if (workspace == nullptr) return MUON_ERR_INVALID_ARG;
  if (x.code_stride % 32 != 0 || x.exp_stride % 16 != 0 || !at_multiple(x.codes, 16) ||
      !at_multiple(x.exps, 16) || !at_multiple(d->dy, esize(d->dy_dtype)) ||
      !at_multiple(d->offsets, 4) || !at_multiple(d->g_ptrs, 8) ||
      !at_multiple(d->g_base, esize(d->g_dtype)) || !at_multiple(workspace, 256))
    return MUON_ERR_MISALIGNED;
  if (workspace_bytes < need) return MUON_ERR_WORKSPACE_TOO_SMALL;

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, kHeader, st) != cudaSuccess) return MUON_ERR_CUDA;
  WgradArgs a{};
  a.rows = static_cast<int>(d->rows);
  a.out = d->out;
  a.in = x.cols;
  a.experts = d->experts;
  a.dy = d->dy;
  a.dy_dtype = d->dy_dtype;
  a.dy_stride = d->dy_stride;
  a.codes = x.codes;
  a.code_stride = x.code_stride;
  a.exps = x.exps;
  a.exp_stride = x.exp_stride;
  a.offsets = d->offsets;
  a.g_ptrs = d->g_ptrs;
  a.g_base = d->g_base;
  a.g_batch_stride = d->g_batch_stride;
  a.g_stride = d->g_stride;
  a.g_dtype = d->g_dtype;
  a.accumulate = d->accumulate;
  a.status = static_cast<uint32_t*>(workspace);
  const dim3 grid((x.cols + kTile - 1) / kTile, (d->out + kTile - 1) / kTile, d->experts);
  if (grid.y > 65535) return MUON_ERR_UNSUPPORTED;
  const double rows = static_cast<double>(d->rows);
  prof_begin(kKindWeightGrad, st);
  k_act8_wgrad<<<grid, kThreads, 0, st>>>(a);
  prof_end(kKindWeightGrad, st, 2.0 * rows * d->out * x.cols,
           rows * (d->out * esize(d->dy_dtype) + x.cols * (1.0 + 1.0 / 32)) +
               static_cast<double>(d->experts) * d->out * x.cols * esize(d->g_dtype) *
                   (d->accumulate ? 2 : 1));
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

}  // extern "C"
