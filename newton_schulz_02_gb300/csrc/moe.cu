// Tokens sorted by expert, and the layer's activations on their way to the
// experts and back (muon_moe_sort, _dispatch, _dispatch_backward, _combine,
// _combine_backward).
//
//   sort      copy i = t K + k of token t has the key chosen[t][k];
//             order: the copies with a key by (key, i);  place[order[r]] = r
//   dispatch  xs[place[t][k]] = x[t]          dx[t] = sum_k dxs[place[t][k]]
//   combine   out[t] = sum_k w[t][k] ys[place[t][k]]
//             dys[place[t][k]] = w[t][k] dout[t],  dw[t][k] = <ys[place[t][k]], dout[t]>
//
// Every pass over activations goes by token, not by row: a token's values are
// read (or written) once and its K rows are whole rows wherever they are, so
// the traffic is what the definition has, and a token's sum is a loop over k
// in one thread, in that order, with no atomics.  Going by row would read a
// token's values once for each expert, from HBM where they do not fit in L2.
// A copy without a row has place -1; a place outside [0, rows) is taken as that.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "planes.cuh"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;

// ---- sort -------------------------------------------------------------------
constexpr int kMaxExperts = 1024;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxPer = 8;       // copies a thread holds at a time
constexpr int kSortBlocks = 152;
constexpr size_t kHeader = 256;

struct SortPlan {
  int per;      // copies of a thread in a round
  int rounds;   // rounds of a block
  int blocks;
};

// One block where it holds all copies at once, else up to a wave of blocks with
// as few copies each as that allows, in several rounds when 8 a thread are not
// enough.  The order does not depend on it.
SortPlan sort_plan(int64_t copies) {
  SortPlan p{1, 1, 1};
  while (p.per < kMaxPer && copies > static_cast<int64_t>(p.per) * kSortThreads) p.per *= 2;
  if (copies <= static_cast<int64_t>(p.per) * kSortThreads) return p;
  p.per = 1;
  while (p.per < kMaxPer && copies > static_cast<int64_t>(p.per) * kSortThreads * kSortBlocks) p.per *= 2;
  const int64_t round = static_cast<int64_t>(p.per) * kSortThreads;
  p.rounds = static_cast<int>((copies + round * kSortBlocks - 1) / (round * kSortBlocks));
  p.blocks = static_cast<int>((copies + round * p.rounds - 1) / (round * p.rounds));
  return p;
}

struct SortArgs {
  uint32_t copies, rows;
  int experts, per, rounds, blocks;
  int group_bits;            // log2 of the threads that hold one row of counts
  Divider topk;
  const void* chosen;
  int chosen_bytes;
  int64_t chosen_stride;
  const uint8_t* mask;
  int32_t* offsets;
  int32_t* order;
  int32_t* place;
  int* counts;               // [blocks][experts]
  uint32_t* flags;           // [blocks]
  uint32_t* status;
};

// Expert of copy i, or -1; a number that is neither sets *bad.
__device__ __forceinline__ int key_of(const SortArgs& a, uint32_t i, bool* bad) {
  if (i >= a.copies) return -1;
  const uint32_t t = quotient(i, a.topk);
  if (a.mask != nullptr && a.mask[t] == 0) return -1;
  const int64_t at = static_cast<int64_t>(t) * a.chosen_stride + (i - t * a.topk.d);
  const int64_t e = a.chosen_bytes == 8 ? static_cast<const int64_t*>(a.chosen)[at]
                                        : static_cast<const int32_t*>(a.chosen)[at];
  if (e >= 0 && e < a.experts) return static_cast<int>(e);
  if (e != -1) *bad = true;
  return -1;
}

// First copy of a block; a block's copies are consecutive.
__device__ __forceinline__ uint64_t block_begin(const SortArgs& a, int block) {
  return static_cast<uint64_t>(block) * a.rounds * a.per * kSortThreads;
}

__global__ void __launch_bounds__(kSortThreads) k_moe_count(const __grid_constant__ SortArgs a) {
  extern __shared__ int sm[];
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) sm[e] = 0;
  griddep_launch_dependents();
  __syncthreads();
  bool bad = false;
  const uint64_t begin = block_begin(a, blockIdx.x);
  for (int j = 0; j < a.rounds * a.per; ++j) {
    const uint64_t i = begin + static_cast<uint64_t>(j) * kSortThreads + threadIdx.x;
    if (i >= a.copies) break;
    const int e = key_of(a, static_cast<uint32_t>(i), &bad);
    if (e >= 0) atomicAdd(&sm[e], 1);
  }
  const int any = __syncthreads_or(bad);
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads)
    a.counts[static_cast<int64_t>(blockIdx.x) * a.experts + e] = sm[e];
  if (threadIdx.x == 0) a.flags[blockIdx.x] = any ? MUON_FLAG_INDEX : 0u;
}

// Exclusive sum over the block's threads, in thread order; *all gets the total.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* all) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[w] = s;
  __syncthreads();
  if (w == 0) {
    int t = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    warp_sums[lane] = t;
  }
  __syncthreads();
  *all = warp_sums[31];
  return s - v + (w > 0 ? warp_sums[w - 1] : 0);
}

// Places the copies of one block.  A warp owns consecutive copies, counts them by
// expert in its own row of `hist`, and after the rows are summed up over the
// warps walks them once more: a lane's row is its warp's next one of that expert
// plus the number of lower lanes with the same expert.
__global__ void __launch_bounds__(kSortThreads) k_moe_place(const __grid_constant__ SortArgs a) {
  extern __shared__ int sm[];
  int* hist = sm;                              // [warps][experts], before that two of [threads]
  int* base = sm + max(kSortWarps * a.experts, 2 * kSortThreads);   // [experts]: next row of this block
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  bool bad = false;
  if (a.blocks > 1) {
    griddep_wait();
    // the experts' totals, and what the blocks before this one have of them
    const int e = tid & ((1 << a.group_bits) - 1), g = tid >> a.group_bits;
    const int groups = kSortThreads >> a.group_bits;
    int before = 0, total = 0;
    if (e < a.experts) {
#pragma unroll 8
      for (int b = g; b < a.blocks; b += groups) {
        const int c = a.counts[b * a.experts + e];
        total += c;
        before += b < static_cast<int>(blockIdx.x) ? c : 0;
      }
    }
    hist[tid] = total;
    hist[kSortThreads + tid] = before;
    __syncthreads();
    total = before = 0;
    if (tid < a.experts) {
      for (int k = 0; k < groups; ++k) {
        total += hist[(k << a.group_bits) + tid];
        before += hist[kSortThreads + (k << a.group_bits) + tid];
      }
    }
    int all;
    const int first = block_scan(total, warp_sums, &all);
    if (tid < a.experts) base[tid] = first + before;
    if (blockIdx.x == 0) {
      if (tid < a.experts) a.offsets[tid] = min(static_cast<uint32_t>(first), a.rows);
      uint32_t f = tid < a.blocks ? a.flags[tid] : 0u;
      if (static_cast<uint32_t>(all) > a.rows) f |= MUON_FLAG_INDEX;
      const int any = __syncthreads_or(f != 0);
      if (tid == 0) {
        a.offsets[a.experts] = min(static_cast<uint32_t>(all), a.rows);
        *a.status = any ? MUON_FLAG_INDEX : 0u;
      }
    }
  }
  uint64_t begin = block_begin(a, blockIdx.x) + static_cast<uint64_t>(w) * a.per * 32 + lane;
  for (int round = 0; round < a.rounds; ++round, begin += static_cast<uint64_t>(a.per) * kSortThreads) {
    __syncthreads();
    for (int i = tid; i < kSortWarps * a.experts; i += kSortThreads) hist[i] = 0;
    int key[kMaxPer];
#pragma unroll
    for (int j = 0; j < kMaxPer; ++j) {
      const uint64_t i = begin + j * 32;
      key[j] = j < a.per && i < a.copies ? key_of(a, static_cast<uint32_t>(i), &bad) : -1;
    }
    __syncthreads();
    int* mine = hist + w * a.experts;
#pragma unroll
    for (int j = 0; j < kMaxPer; ++j)
      if (key[j] >= 0) atomicAdd(&mine[key[j]], 1);
    __syncthreads();
    if (a.blocks == 1) {   // the only round: the totals are these counts'
      int total = 0;
      if (tid < a.experts)
        for (int k = 0; k < kSortWarps; ++k) total += hist[k * a.experts + tid];
      int all;
      const int first = block_scan(total, warp_sums, &all);
      if (tid < a.experts) {
        base[tid] = first;
        a.offsets[tid] = min(static_cast<uint32_t>(first), a.rows);
      }
      const int any = __syncthreads_or(bad || static_cast<uint32_t>(all) > a.rows);
      if (tid == 0) {
        a.offsets[a.experts] = min(static_cast<uint32_t>(all), a.rows);
        *a.status = any ? MUON_FLAG_INDEX : 0u;
      }
    }
    if (tid < a.experts) {
      int next = base[tid];
#pragma unroll 8
      for (int k = 0; k < kSortWarps; ++k) {
        const int c = hist[k * a.experts + tid];
        hist[k * a.experts + tid] = next;
        next += c;
      }
      base[tid] = next;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMaxPer; ++j) {
      if (j >= a.per) break;   // the same for all threads
      const uint32_t same = __match_any_sync(0xffffffffu, key[j]);
      const int rank = __popc(same & ((1u << lane) - 1));
      const int first = key[j] >= 0 ? mine[key[j]] : 0;
      __syncwarp();
      if (key[j] >= 0 && rank == 0) mine[key[j]] = first + __popc(same);
      __syncwarp();
      const uint64_t i = begin + j * 32;
      const uint32_t row = static_cast<uint32_t>(first + rank);
      const bool on = key[j] >= 0 && row < a.rows;
      if (i < a.copies) a.place[i] = on ? static_cast<int32_t>(row) : -1;
      if (on) a.order[row] = static_cast<int32_t>(i);
    }
  }
}

size_t sort_smem(int experts) {
  const int words = kSortWarps * experts > 2 * kSortThreads ? kSortWarps * experts : 2 * kSortThreads;
  return static_cast<size_t>(words + experts) * 4;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// ---- rows of a token --------------------------------------------------------
struct RowArgs {
  uint32_t tokens, items;   // items: tokens x items of a row
  int cols, topk, accumulate;
  uint32_t rows;            // of the rows' buffers
  Divider per_row;          // items of a row
  const int32_t* place;     // [tokens][topk]
  const void* w;            // weights [tokens][topk], or nullptr
  int64_t w_stride;
  void* dw;
  int64_t dw_stride;
  int wdt;
  Plane x, y, z;            // x: by token; y, z: by row
  Packed codes;             // by row
};

struct Item {
  uint32_t token;
  int col, n;    // n: columns of this item inside the row (<= 0: padding of the last block)
  bool on;
};

__device__ __forceinline__ Item item_of(const RowArgs& a) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  Item p;
  p.on = i < a.items;
  const uint32_t at = p.on ? i : a.items - 1;
  p.token = quotient(at, a.per_row);
  p.col = static_cast<int>(at - p.token * a.per_row.d) * kCols;
  p.n = p.on ? a.cols - p.col : 0;
  return p;
}

__device__ __forceinline__ float weight_at(const void* w, int wdt, int64_t i) {
  return wdt == MUON_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i])
                          : static_cast<const float*>(w)[i];
}

// A token's values to all of its rows, and their codes to the checkpoint's.
template <typename TX, typename TY, bool WHOLE, bool CODES>
__global__ void __launch_bounds__(kThreads) k_moe_dispatch(const __grid_constant__ RowArgs a) {
  const Item p = item_of(a);
  float x[kCols];
  load_values<TX, WHOLE>(a.x, p.token, p.col, p.n, x);
  Codes c;
  if constexpr (CODES) c = encode(x);
  const int32_t* at = a.place + static_cast<int64_t>(p.token) * a.topk;
  for (int k = 0; k < a.topk; ++k) {
    const uint32_t row = static_cast<uint32_t>(at[k]);
    const bool in = p.on && row < a.rows;
    store_values<TY, WHOLE>(a.y, in ? row : 0, p.col, in ? p.n : 0, x);
    if constexpr (CODES) {
      if (in) store_codes(a.codes, row, p.col, c);
    }
  }
}

// out = sum_k w_k y_k (w_k = 1 without weights), added to what it holds if asked.
template <typename TY, typename TO, bool WHOLE, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads) k_moe_combine(const __grid_constant__ RowArgs a) {
  constexpr int kAhead = sizeof(TY) == 2 ? 4 : 2;   // rows in flight
  const Item p = item_of(a);
  float acc[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
  const int32_t* at = a.place + static_cast<int64_t>(p.token) * a.topk;
  for (int k0 = 0; k0 < a.topk; k0 += kAhead) {
    float y[kAhead][kCols], w[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint32_t row = p.on && k0 + j < a.topk ? static_cast<uint32_t>(at[k0 + j]) : a.rows;
      const bool in = row < a.rows;
      load_values<TY, WHOLE>(a.y, in ? row : 0, p.col, in ? p.n : 0, y[j]);
      w[j] = !in ? 0.f : WEIGHTS ? weight_at(a.w, a.wdt, p.token * a.w_stride + k0 + j) : 1.f;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = fmaf(w[j], y[j][c], acc[c]);
  }
  if (a.accumulate) {
    float old[kCols];
    load_values<TO, WHOLE>(a.x, p.token, p.col, p.n, old);
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[c] += old[c];
    if constexpr (!WHOLE) __syncwarp();   // the warp's reads are over
  }
  store_values<TO, WHOLE>(a.x, p.token, p.col, p.n, acc);
}

constexpr int kDots = 8;   // choices of a token that a pass over its columns takes

// The sums over the warp's lanes of v[0 .. 7]; lane l gets that of v[l / 4].
__device__ __forceinline__ float warp_sums8(float (&v)[kDots], int lane) {
#pragma unroll
  for (int half = 4, bit = 16; half >= 1; half >>= 1, bit >>= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int j = 0; j < half; ++j) {
      const float send = up ? v[j] : v[j + half];
      const float keep = up ? v[j + half] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
  }
  float s = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 2);
  return s + __shfl_xor_sync(0xffffffffu, s, 1);
}

// x = dout, y = ys, z = dys.  `blockDim.x` threads (whole warps) take one token and
// blockDim.y tokens share a block.
template <typename TX, typename TY, bool WHOLE>
__global__ void __launch_bounds__(512) k_moe_combine_backward(const __grid_constant__ RowArgs a) {
  constexpr int kAhead = sizeof(TY) == 2 ? 4 : 2;   // rows in flight
  __shared__ float red[16][kDots];
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int first_warp = threadIdx.y * warps, warp = first_warp + (threadIdx.x >> 5);
  const uint32_t t = blockIdx.x * blockDim.y + threadIdx.y;
  const bool on = t < a.tokens;
  const uint32_t token = on ? t : a.tokens - 1;
  const int32_t* at = a.place + static_cast<int64_t>(token) * a.topk;
  const int span = blockDim.x * kCols, width = a.per_row.d * kCols;
  for (int k0 = 0; k0 < a.topk; k0 += kDots) {
    float dot[kDots];
#pragma unroll
    for (int j = 0; j < kDots; ++j) dot[j] = 0.f;
    for (int c0 = 0; c0 < width; c0 += span) {   // the same number of times for all threads
      const int col = c0 + threadIdx.x * kCols;
      const int n = on ? a.cols - col : 0;
      float d[kCols];
      load_values<TX, WHOLE>(a.x, token, col, n, d);
#pragma unroll
      for (int j0 = 0; j0 < kDots; j0 += kAhead) {
        if (k0 + j0 >= a.topk) break;   // the same for all threads
        float y[kAhead][kCols], w[kAhead];
        uint32_t row[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int k = k0 + j0 + j;
          row[j] = on && k < a.topk ? static_cast<uint32_t>(at[k]) : a.rows;
          const bool in = row[j] < a.rows;
          load_values<TY, WHOLE>(a.y, in ? row[j] : 0, col, in ? n : 0, y[j]);
          w[j] = in ? weight_at(a.w, a.wdt, token * a.w_stride + k) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
          for (int c = 0; c < kCols; ++c) dot[j0 + j] = fmaf(d[c], y[j][c], dot[j0 + j]);
        if constexpr (!WHOLE) __syncwarp();   // dys may be ys: the warp's reads are over
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const bool in = row[j] < a.rows;
          float g[kCols];
#pragma unroll
          for (int c = 0; c < kCols; ++c) g[c] = w[j] * d[c];
          store_values<TY, WHOLE>(a.z, in ? row[j] : 0, col, in ? n : 0, g);
        }
      }
    }
    float s = warp_sums8(dot, lane);
    if (warps > 1) {
      if ((lane & 3) == 0) red[warp][lane >> 2] = s;
      __syncthreads();
      s = 0.f;
      for (int v = 0; v < warps; ++v) s += red[first_warp + v][lane >> 2];
      __syncthreads();
    }
    const int k = k0 + (lane >> 2);
    if (on && threadIdx.x < 32 && (lane & 3) == 0 && k < a.topk) {
      const bool in = static_cast<uint32_t>(at[k]) < a.rows;
      const int64_t i = token * a.dw_stride + k;
      if (a.wdt == MUON_BF16)
        static_cast<__nv_bfloat16*>(a.dw)[i] = __float2bfloat16_rn(in ? s : 0.f);
      else
        static_cast<float*>(a.dw)[i] = in ? s : 0.f;
    }
  }
}

// ---- host ------------------------------------------------------------------
constexpr int64_t kMaxCopies = (int64_t{1} << 31) - 1;

muon_status_t check_sort_sizes(int64_t tokens, int experts, int topk) {
  if (tokens < 0 || experts < 1 || topk < 1) return MUON_ERR_INVALID_ARG;
  if (experts > kMaxExperts || topk > kMaxExperts || tokens > kMaxCopies / topk) return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

muon_status_t check_routing(const muon_routing_t* r) {
  if (r == nullptr) return MUON_ERR_INVALID_ARG;
  const muon_status_t s = check_sort_sizes(r->tokens, r->experts, r->topk);
  if (s != MUON_OK) return s;
  if (r->rows < 0) return MUON_ERR_INVALID_ARG;
  if (r->rows > kMaxCopies) return MUON_ERR_UNSUPPORTED;
  if (r->tokens > 0 && r->place == nullptr) return MUON_ERR_INVALID_ARG;
  return at_multiple(r->place, 4) ? MUON_OK : MUON_ERR_MISALIGNED;
}

muon_status_t check_rows(const void* p, int64_t rows, int dtype, int64_t stride, int width) {
  if (dtype != MUON_BF16 && dtype != MUON_F32) return MUON_ERR_INVALID_ARG;
  if (stride < width || (rows > 0 && p == nullptr)) return MUON_ERR_INVALID_ARG;
  return at_multiple(p, esize(dtype)) ? MUON_OK : MUON_ERR_MISALIGNED;
}

// What all passes over activations check, and their common arguments.
muon_status_t row_args(const muon_routing_t* r, int width, RowArgs* a) {
  const muon_status_t s = check_routing(r);
  if (s != MUON_OK) return s;
  if (width < 1) return MUON_ERR_INVALID_ARG;
  if (width > (1 << 26)) return MUON_ERR_UNSUPPORTED;
  a->cols = width;
  a->topk = r->topk;
  a->rows = static_cast<uint32_t>(r->rows);
  a->place = r->place;
  a->per_row = divider(static_cast<uint32_t>(blocks_of(width) * (kBlock / kCols)));
  return MUON_OK;
}

// `launch(args, first token)` for every token, in pieces of fewer than 2^30 items.
template <class F>
muon_status_t by_tokens(RowArgs a, int64_t tokens, int xdt, F launch) {
  int64_t most = (int64_t{1} << 30) / a.per_row.d;
  if (most < 1) most = 1;
  for (int64_t t0 = 0; t0 < tokens; t0 += most) {
    const int64_t n = tokens - t0 < most ? tokens - t0 : most;
    RowArgs b = a;
    b.tokens = static_cast<uint32_t>(n);
    b.items = static_cast<uint32_t>(n * a.per_row.d);
    b.place += t0 * a.topk;
    b.x.p = static_cast<char*>(a.x.p) + t0 * a.x.stride * esize(xdt);
    if (b.w != nullptr) b.w = static_cast<const char*>(b.w) + t0 * b.w_stride * esize(b.wdt);
    if (b.dw != nullptr) b.dw = static_cast<char*>(b.dw) + t0 * b.dw_stride * esize(b.wdt);
    launch(b);
    if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
  }
  return MUON_OK;
}

unsigned grid_of(const RowArgs& a) { return (a.items + kThreads - 1) / kThreads; }

template <typename TX, typename TY>
void launch_dispatch(const RowArgs& a, bool whole, bool codes, cudaStream_t st) {
  const unsigned grid = grid_of(a);
  if (whole && codes) k_moe_dispatch<TX, TY, true, true><<<grid, kThreads, 0, st>>>(a);
  else if (whole) k_moe_dispatch<TX, TY, true, false><<<grid, kThreads, 0, st>>>(a);
  else if (codes) k_moe_dispatch<TX, TY, false, true><<<grid, kThreads, 0, st>>>(a);
  else k_moe_dispatch<TX, TY, false, false><<<grid, kThreads, 0, st>>>(a);
}

template <typename TY, typename TO>
void launch_combine(const RowArgs& a, bool whole, cudaStream_t st) {
  const unsigned grid = grid_of(a);
  const bool weights = a.w != nullptr;
  if (whole && weights) k_moe_combine<TY, TO, true, true><<<grid, kThreads, 0, st>>>(a);
  else if (whole) k_moe_combine<TY, TO, true, false><<<grid, kThreads, 0, st>>>(a);
  else if (weights) k_moe_combine<TY, TO, false, true><<<grid, kThreads, 0, st>>>(a);
  else k_moe_combine<TY, TO, false, false><<<grid, kThreads, 0, st>>>(a);
}

// Threads of a token: enough for its columns at once, up to 512; narrow tokens
// share a block of up to 256 threads.
template <typename TX, typename TY>
void launch_combine_backward(const RowArgs& a, bool whole, cudaStream_t st) {
  const unsigned items = a.per_row.d;
  const unsigned threads = items >= 512 ? 512 : (items + 31) / 32 * 32;
  const unsigned tokens = threads >= 256 ? 1 : 256 / threads;
  const dim3 block(threads, tokens);
  const unsigned grid = (a.tokens + tokens - 1) / tokens;
  if (whole) k_moe_combine_backward<TX, TY, true><<<grid, block, 0, st>>>(a);
  else k_moe_combine_backward<TX, TY, false><<<grid, block, 0, st>>>(a);
}

// F<first type, second type> for a pair of types.
template <class F>
void by_types(int first, int second, F f) {
  if (first == MUON_F32 && second == MUON_F32) f(float{}, float{});
  else if (first == MUON_F32) f(float{}, __nv_bfloat16{});
  else if (second == MUON_F32) f(__nv_bfloat16{}, float{});
  else f(__nv_bfloat16{}, __nv_bfloat16{});
}

muon_status_t combine(const void* ys, muon_dtype_t ydt, int64_t y_stride, const muon_routing_t* r,
                      const void* weights, muon_dtype_t wdt, int64_t w_stride, int width, void* out,
                      muon_dtype_t odt, int64_t out_stride, int accumulate, cudaStream_t st) {
  RowArgs a{};
  muon_status_t s = row_args(r, width, &a);
  if (s == MUON_OK) s = check_rows(ys, r->rows, ydt, y_stride, width);
  if (s == MUON_OK) s = check_rows(out, r->tokens, odt, out_stride, width);
  if (s == MUON_OK && weights != nullptr) s = check_rows(weights, r->tokens, wdt, w_stride, r->topk);
  if (s != MUON_OK) return s;
  if (accumulate != 0 && accumulate != 1) return MUON_ERR_INVALID_ARG;
  a.x = plane(out, out_stride);
  a.y = plane(ys, y_stride);
  a.w = weights;
  a.wdt = wdt;
  a.w_stride = w_stride;
  a.accumulate = accumulate;
  const bool whole = rows_aligned(a.x, odt) && rows_aligned(a.y, ydt);
  return by_tokens(a, r->tokens, odt, [&](const RowArgs& b) {
    prof_begin(kKindMoe, st);
    by_types(ydt, odt, [&](auto ty, auto to) { launch_combine<decltype(ty), decltype(to)>(b, whole, st); });
    prof_end(kKindMoe, st, 0.0, static_cast<double>(b.tokens) * width *
                                    (r->topk * esize(ydt) + esize(odt) * (accumulate ? 2 : 1)));
  });
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status_t muon_moe_sort_workspace_size(int64_t tokens, int experts, int topk, size_t* bytes) {
  if (bytes == nullptr) return MUON_ERR_INVALID_ARG;
  const muon_status_t s = check_sort_sizes(tokens, experts, topk);
  if (s != MUON_OK) return s;
  const SortPlan p = sort_plan(tokens * topk);
  *bytes = kHeader + align256(static_cast<size_t>(p.blocks) * 4) +
           static_cast<size_t>(p.blocks) * experts * 4;
  return MUON_OK;
}

muon_status_t muon_moe_sort(const void* chosen, int chosen_bytes, int64_t chosen_stride,
                            const uint8_t* token_mask, const muon_routing_t* r, void* workspace,
                            size_t workspace_bytes, muon_stream_t stream) {
  muon_status_t s = check_routing(r);
  if (s != MUON_OK) return s;
  if (chosen_bytes != 4 && chosen_bytes != 8) return MUON_ERR_INVALID_ARG;
  if (chosen_stride < r->topk || (r->tokens > 0 && chosen == nullptr)) return MUON_ERR_INVALID_ARG;
  if (r->offsets == nullptr || (r->rows > 0 && r->order == nullptr) || workspace == nullptr)
    return MUON_ERR_INVALID_ARG;
  if (!at_multiple(chosen, chosen_bytes) || !at_multiple(r->offsets, 4) || !at_multiple(r->order, 4) ||
      !at_multiple(workspace, 256))
    return MUON_ERR_MISALIGNED;
  size_t need = 0;
  s = muon_moe_sort_workspace_size(r->tokens, r->experts, r->topk, &need);
  if (s != MUON_OK) return s;
  if (workspace_bytes < need) return MUON_ERR_WORKSPACE_TOO_SMALL;

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const SortPlan plan = sort_plan(r->tokens * r->topk);
  char* ws = static_cast<char*>(workspace);
  SortArgs a{};
  a.copies = static_cast<uint32_t>(r->tokens * r->topk);
  a.rows = static_cast<uint32_t>(r->rows);
  a.experts = r->experts;
  a.per = plan.per;
  a.rounds = plan.rounds;
  a.blocks = plan.blocks;
  a.group_bits = 5;
  while ((1 << a.group_bits) < r->experts) ++a.group_bits;
  a.topk = divider(static_cast<uint32_t>(r->topk));
  a.chosen = chosen;
  a.chosen_bytes = chosen_bytes;
  a.chosen_stride = chosen_stride;
  a.mask = token_mask;
  a.offsets = r->offsets;
  a.order = r->order;
  a.place = r->place;
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.flags = reinterpret_cast<uint32_t*>(ws + kHeader);
  a.counts = reinterpret_cast<int*>(ws + kHeader + align256(static_cast<size_t>(plan.blocks) * 4));
  const double bytes = static_cast<double>(a.copies) * (chosen_bytes + 8);
  const size_t smem = sort_smem(r->experts);
  // per device, and cheap: the attribute is set with every call that needs it
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(k_moe_place, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(sort_smem(kMaxExperts))) != cudaSuccess)
    return MUON_ERR_CUDA;
  if (plan.blocks > 1) {
    prof_begin(kKindMoe, st);
    k_moe_count<<<plan.blocks, kSortThreads, r->experts * 4, st>>>(a);
    prof_end(kKindMoe, st, 0.0, 0.0);
    if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(plan.blocks);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = plan.blocks > 1 ? 1 : 0;   // alone it depends on what was enqueued before the call
  prof_begin(kKindMoe, st);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_moe_place, a);
  prof_end(kKindMoe, st, 0.0, bytes);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

muon_status_t muon_moe_dispatch(const void* x, muon_dtype_t xdt, int64_t x_stride,
                                const muon_routing_t* r, int width, void* xs, muon_dtype_t xsdt,
                                int64_t xs_stride, const muon_act8_t* x8, muon_stream_t stream) {
  RowArgs a{};
  muon_status_t s = row_args(r, width, &a);
  if (s == MUON_OK) s = check_rows(x, r->tokens, xdt, x_stride, width);
  if (s == MUON_OK) s = check_rows(xs, r->rows, xsdt, xs_stride, width);
  if (s == MUON_OK && x8 != nullptr) s = check_act8(x8);
  if (s != MUON_OK) return s;
  if (x8 != nullptr && (x8->rows != r->rows || x8->cols != width)) return MUON_ERR_INVALID_ARG;
  a.x = plane(x, x_stride);
  a.y = plane(xs, xs_stride);
  if (x8 != nullptr) a.codes = packed(x8);
  const bool whole = rows_aligned(a.x, xdt) && rows_aligned(a.y, xsdt);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return by_tokens(a, r->tokens, xdt, [&](const RowArgs& b) {
    prof_begin(kKindMoe, st);
    by_types(xdt, xsdt, [&](auto tx, auto ty) {
      launch_dispatch<decltype(tx), decltype(ty)>(b, whole, x8 != nullptr, st);
    });
    prof_end(kKindMoe, st, 0.0, static_cast<double>(b.tokens) * width *
                                    (esize(xdt) + r->topk * (esize(xsdt) + (x8 != nullptr ? kCodeBytes : 0.0))));
  });
}

muon_status_t muon_moe_dispatch_backward(const void* dxs, muon_dtype_t dxsdt, int64_t dxs_stride,
                                         const muon_routing_t* r, int width, void* dx,
                                         muon_dtype_t dxdt, int64_t dx_stride, int accumulate,
                                         muon_stream_t stream) {
  return combine(dxs, dxsdt, dxs_stride, r, nullptr, MUON_F32, 0, width, dx, dxdt, dx_stride, accumulate,
                 reinterpret_cast<cudaStream_t>(stream));
}

muon_status_t muon_moe_combine(const void* ys, muon_dtype_t ydt, int64_t y_stride,
                               const muon_routing_t* r, const void* weights, muon_dtype_t wdt,
                               int64_t w_stride, int width, void* out, muon_dtype_t odt,
                               int64_t out_stride, int accumulate, muon_stream_t stream) {
  if (r != nullptr && r->tokens > 0 && weights == nullptr) return MUON_ERR_INVALID_ARG;
  return combine(ys, ydt, y_stride, r, weights, wdt, w_stride, width, out, odt, out_stride, accumulate,
                 reinterpret_cast<cudaStream_t>(stream));
}

muon_status_t muon_moe_combine_backward(const void* dout, muon_dtype_t ddt, int64_t dout_stride,
                                        const void* ys, muon_dtype_t ydt, int64_t y_stride,
                                        const muon_routing_t* r, const void* weights,
                                        muon_dtype_t wdt, int64_t w_stride, int width, void* dys,
                                        int64_t dys_stride, void* dweights, int64_t dw_stride,
                                        muon_stream_t stream) {
  RowArgs a{};
  muon_status_t s = row_args(r, width, &a);
  if (s == MUON_OK) s = check_rows(dout, r->tokens, ddt, dout_stride, width);
  if (s == MUON_OK) s = check_rows(ys, r->rows, ydt, y_stride, width);
  if (s == MUON_OK) s = check_rows(dys, r->rows, ydt, dys_stride, width);
  if (s == MUON_OK) s = check_rows(weights, r->tokens, wdt, w_stride, r->topk);
  if (s == MUON_OK) s = check_rows(dweights, r->tokens, wdt, dw_stride, r->topk);
  if (s != MUON_OK) return s;
  a.x = plane(dout, dout_stride);
  a.y = plane(ys, y_stride);
  a.z = plane(dys, dys_stride);
  a.w = weights;
  a.wdt = wdt;
  a.w_stride = w_stride;
  a.dw = dweights;
  a.dw_stride = dw_stride;
  const bool whole = rows_aligned(a.x, ddt) && rows_aligned(a.y, ydt) && rows_aligned(a.z, ydt);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return by_tokens(a, r->tokens, ddt, [&](const RowArgs& b) {
    prof_begin(kKindMoe, st);
    by_types(ddt, ydt, [&](auto tx, auto ty) {
      launch_combine_backward<decltype(tx), decltype(ty)>(b, whole, st);
    });
    prof_end(kKindMoe, st, 0.0,
             static_cast<double>(b.tokens) * width * (esize(ddt) + 2.0 * r->topk * esize(ydt)));
  });
}

}  // extern "C"
