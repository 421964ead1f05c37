// Router balance loss: per-expert counts, the loss and the gradient of the
// logits (muon_balance_forward, muon_balance_backward).
//
//   p_t  = softmax(l_t)  or  sigma(l_t) / sum sigma(l_t)
//   f_se = E / (K n_s) c_se,   loss = coef/N sum_s sum_{t in s} sum_e f_se p_te
//   dl   = coef/N p (f - sum_j f_j p_j)  [* (1 - sigma(l))]
//
// Both passes are bound by the logits' bytes: the forward pass reads them
// once, the backward pass reads them once and writes the gradient.  A row of
// logits lives in the registers of LANES lanes (VPT values each), so its
// maximum, sum and dot product are shuffles and the probabilities are
// recomputed in the backward pass instead of being stored.  The expert sums
// over tokens (sum_t p_te and c_se) stay in registers and shared memory over a
// chunk of tokens of one sequence; each chunk leaves one row of partial sums,
// which the second kernel adds in index order, so no float atomics are used.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxExperts = 1024;
constexpr int kFinWide = 1024, kFinNarrow = 256;   // threads of a finalize block
constexpr int kTotalThreads = 1024;
constexpr int kTotalItems = 4096;   // more chunks than these are counted once, not by every block
constexpr size_t kHeader = 256;     // status word, ticket of the finalize blocks, counts of the batch

// Blocks of the forward pass that an SM holds at once.  Up to 512 experts five, by
// 48 registers: with four, 100 experts and more take 7 to 36% longer (131072 x 256
// bf16 48.8 us for 35.9), also at the widths whose bound checks then cost a few
// spilled registers (131072 x 200 bf16 49.1 for 40.8), and fewer experts as long or
// longer.  More than 512 experts need the registers, and two fit.
constexpr int blocks_per_sm(int experts) { return experts <= 512 ? 5 : 2; }

// Tokens of a chunk.  Chunks and the cuts at sequence bounds together make up
// to one wave of blocks on 152 SMs (65536 x 1024 fp32 63 us, in two waves 65, in two and a
// half 74); with many sequences there are up to half a wave beside their cuts.  A
// function of the sizes alone, as the order of the sums follows it.
int chunk_tokens(int64_t tokens, int experts, int sequences) {
  const int wave = 152 * blocks_per_sm(experts);
  const int64_t most = wave - std::min(sequences, wave / 2);
  const int64_t c = tokens / most + 1;
  return static_cast<int>(c < 32 ? 32 : c);
}

// Chunks are cut at absolute multiples of the chunk length and at sequence
// bounds.  Sequence s that starts at token b owns the chunks b/C + s ...
// (e-1)/C + s: one number for each (chunk, sequence) pair, ascending, without
// knowing the bounds on the host.
int64_t chunk_items(int64_t tokens, int experts, int sequences) {
  return tokens / chunk_tokens(tokens, experts, sequences) + sequences;
}

struct BalanceArgs {
  int tokens, experts, topk, sequences, chunk, items;
  const void* logits;
  int dtype;
  int64_t logits_stride;
  const void* chosen;
  int chosen_bytes;
  int64_t chosen_stride;
  const int32_t* seq_begin;   // nullptr: one sequence
  const uint8_t* mask;        // nullptr: all valid
  int sigmoid;
  float coef;
  int vec, lvec;              // rows of logits, of load, may be read four values at a time
  // forward
  float* psum;                // [items][experts]
  int* pcnt;                  // [items][experts]
  int* pval;                  // [items]: valid tokens
  int* pflag;                 // [items]: device conditions seen
  float* lossp;               // [sequences * expert blocks]
  uint32_t* status;
  int* ticket;
  int* bounds;                // whether the sequence bounds were out of order
  int* total;                 // valid tokens of the batch, conditions seen; nullptr: finalize adds pval
  float* loss;
  int32_t* counts;
  float* load;
  // backward
  const float* dloss;
  void* dlogits;
  int ddt;
  int64_t dlogits_stride;
  int dvec;
  int accumulate;
  int row_steps;              // rows a group of lanes walks
  int levels;                 // look for sequences whose experts share one load
};

__device__ __forceinline__ int clamp_token(int v, int tokens) { return min(max(v, 0), tokens); }

__device__ __forceinline__ int seq_at(const BalanceArgs& a, int s) {
  return a.seq_begin == nullptr ? (s == 0 ? 0 : a.tokens)
                                : clamp_token(__ldg(a.seq_begin + s), a.tokens);
}

// Largest s whose first chunk is at most `item` (0 if none).
__device__ int seq_of_item(const BalanceArgs& a, int item) {
  int lo = 0, hi = a.sequences - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_at(a, mid) / a.chunk + mid <= item)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Largest s with seq_begin[s] <= t, or -1.
__device__ int seq_of_token(const BalanceArgs& a, int t) {
  int lo = -1, hi = a.sequences - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_at(a, mid) <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Value j of lane `sub` is column (j / 4) * 4 LANES + 4 sub + j % 4: four
// consecutive columns a lane, LANES lanes side by side.
template <int LANES>
__device__ __forceinline__ int column(int sub, int j) {
  return (j >> 2) * (4 * LANES) + 4 * sub + (j & 3);
}

// Columns column(sub, 0..VPT-1) of a row of n values; columns from n on are
// `fill`.  FULL: n = LANES * VPT.
template <int LANES, int VPT, bool FULL>
__device__ __forceinline__ void load_row(const void* base, int64_t off, int dtype, int n, int vec,
                                         int sub, float fill, float (&x)[VPT]) {
  if (vec && dtype == MUON_F32) {
    const float* p = static_cast<const float*>(base) + off;
#pragma unroll
    for (int q = 0; q < VPT / 4; ++q) {
      const int c = column<LANES>(sub, 4 * q);
      float4 v = make_float4(fill, fill, fill, fill);
      if (FULL || c < n) v = *reinterpret_cast<const float4*>(p + c);
      x[4 * q] = v.x; x[4 * q + 1] = v.y; x[4 * q + 2] = v.z; x[4 * q + 3] = v.w;
    }
  } else if (vec) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + off;
    uint2 w[VPT / 4];
#pragma unroll
    for (int q = 0; q < VPT / 4; ++q) {
      const int c = column<LANES>(sub, 4 * q);
      if (FULL || c < n) w[q] = *reinterpret_cast<const uint2*>(p + c);
    }
#pragma unroll
    for (int q = 0; q < VPT / 4; ++q) {
      const bool in = FULL || column<LANES>(sub, 4 * q) < n;
      x[4 * q] = in ? __uint_as_float(w[q].x << 16) : fill;
      x[4 * q + 1] = in ? __uint_as_float(w[q].x & 0xFFFF0000u) : fill;
      x[4 * q + 2] = in ? __uint_as_float(w[q].y << 16) : fill;
      x[4 * q + 3] = in ? __uint_as_float(w[q].y & 0xFFFF0000u) : fill;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = column<LANES>(sub, j);
      x[j] = fill;
      if (c < n)
        x[j] = dtype == MUON_F32 ? static_cast<const float*>(base)[off + c]
                                 : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[off + c]);
    }
  }
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = LANES / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int d = LANES / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

// 2^y, flushed to 0 below the normal range.
__device__ __forceinline__ float exp2_fast(float y) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  return r;
}

constexpr float kLog2e = 1.44269504f;

// Scores of a row in place of its logits, up to the factor that makes them
// probabilities, which is returned: softmax exp(l - max); sigmoid 1 / (1 + t),
// or with KEEP_T the t = exp(-l) itself.  A row whose scores sum to 0 (every
// expert disabled) gets the factor 0; NaN stays NaN.
template <int LANES, int VPT, bool SIGMOID, bool KEEP_T>
__device__ __forceinline__ float row_scores(float (&x)[VPT]) {
  float z = 0.f;
  if constexpr (SIGMOID) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const float t = exp2_fast(-kLog2e * x[j]);
      const float s = __fdividef(1.f, 1.f + t);
      x[j] = KEEP_T ? t : s;
      z += s;
    }
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPT; ++j) m = fmaxf(m, x[j]);
    m = group_max<LANES>(m);
    if (m == -INFINITY) m = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      x[j] = exp2_fast(kLog2e * (x[j] - m));
      z += x[j];
    }
  }
  z = group_sum<LANES>(z);
  return z == 0.f ? 0.f : 1.f / z;
}

// Whether a row's sigmoids are all so small (their sum's reciprocal is inv) that
// they, or those of its other experts, are lost below the normal range.
__device__ __forceinline__ bool is_low(float inv) { return inv == 0.f || inv > 0x1p32f; }

// Such a row (low; the whole warp calls it) is multiplied by exp(-m), m its
// largest logit, which gives exp(l - m): sigma(l) and exp(l) agree in every bit there.
// Its lanes read it again, value by value, as it is rare and a row's registers are all
// in use.  Below -700 (nothing in 64 bits either; a mask's lowest value) it has no
// scores.  SIGMOID is a parameter of the kernels so that softmax does without this:
// 131072 x 200 bf16, backward, 42.4 us in one kernel for both, 39.0 so.
template <int LANES, int VPT>
struct LowRow {
  float m, z;
  const BalanceArgs& a;
  int64_t off;
  int sub;

  __device__ __forceinline__ LowRow(const BalanceArgs& args, int t, int lane, bool low)
      : m(-INFINITY), z(0.f), a(args), off(static_cast<int64_t>(t) * args.logits_stride), sub(lane) {
#pragma unroll 1
    for (int j = 0; j < VPT; ++j) m = fmaxf(m, low ? logit(j) : -INFINITY);
    m = group_max<LANES>(m);
#pragma unroll 1
    for (int j = 0; j < VPT; ++j) z += score(j);
    z = group_sum<LANES>(z);
  }
  __device__ __forceinline__ float logit(int j) const {
    const int c = column<LANES>(sub, j);
    if (c >= a.experts) return -INFINITY;
    return a.dtype == MUON_F32 ? static_cast<const float*>(a.logits)[off + c]
                               : __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[off + c]);
  }
  __device__ __forceinline__ bool any() const { return m > -700.f; }
  __device__ __forceinline__ float score(int j) const { return any() ? exp2_fast(kLog2e * (logit(j) - m)) : 0.f; }
  __device__ __forceinline__ float inverse() const { return any() ? 1.f / z : 0.f; }
};

// One chunk of tokens of one sequence per block: sum_t p_te, c_e and the
// number of valid tokens.
template <int LANES, int VPT, bool FULL, bool SIGMOID>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(LANES * VPT))
    k_balance_forward(const __grid_constant__ BalanceArgs a) {
  constexpr int kGroups = kThreads / LANES;
  constexpr int kCols = LANES * VPT;
  __shared__ float s_sum[kGroups * kCols];
  __shared__ int s_cnt[kCols];
  __shared__ int s_val, s_flag;
  griddep_launch_dependents();
  const int item = blockIdx.x;
  const int s = seq_of_item(a, item);
  const int64_t c0 = static_cast<int64_t>(item - s) * a.chunk;
  const int b = seq_at(a, s), e = seq_at(a, s + 1);
  const int t0 = static_cast<int>(max(static_cast<int64_t>(b), c0));
  const int t1 = static_cast<int>(min(static_cast<int64_t>(e), c0 + a.chunk));
  if (item == 0) {
    for (int i = threadIdx.x; i < a.experts; i += kThreads) a.counts[i] = 0;
    if (threadIdx.x == 0) *a.ticket = 0;
  }
  if (c0 < 0 || t0 >= t1) {   // no sequence has this chunk
    if (threadIdx.x == 0) a.pval[item] = a.pflag[item] = 0;
    return;
  }
  for (int i = threadIdx.x; i < kCols; i += kThreads) s_cnt[i] = 0;
  if (threadIdx.x == 0) s_val = s_flag = 0;
  __syncthreads();

  const int group = threadIdx.x / LANES, sub = threadIdx.x % LANES;
  float acc[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) acc[j] = 0.f;
  int valid = 0, bad = 0;
  const auto is_on = [&](int t) { return t < t1 && (a.mask == nullptr || a.mask[t] != 0); };
  const auto choice = [&](int t, int k) {
    const int64_t at = static_cast<int64_t>(t) * a.chosen_stride + k;
    return a.chosen_bytes == 4 ? static_cast<int64_t>(static_cast<const int32_t*>(a.chosen)[at])
                               : static_cast<const int64_t*>(a.chosen)[at];
  };
  // A row's loads depend on its mask, which is fetched a row ahead; the choices
  // are fetched beside the logits.
  bool next_on = is_on(t0 + group);
  for (int tb = t0; tb < t1; tb += kGroups) {   // uniform trip count: shuffles need every lane
    const int t = tb + group;
    const bool on = next_on;
    next_on = is_on(t + kGroups);
    int64_t id = -1;
    float x[VPT];
    if (on) {
      load_row<LANES, VPT, FULL>(a.logits, static_cast<int64_t>(t) * a.logits_stride, a.dtype,
                                 a.experts, a.vec, sub, -INFINITY, x);
      if (sub < a.topk) id = choice(t, sub);
    } else {
#pragma unroll
      for (int j = 0; j < VPT; ++j) x[j] = -INFINITY;
    }
    float inv = row_scores<LANES, VPT, SIGMOID, false>(x);
    const bool low = SIGMOID && on && is_low(inv);
    if (low) inv = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) acc[j] = fmaf(x[j], inv, acc[j]);
    if (SIGMOID && __any_sync(0xffffffffu, low)) {
      const LowRow<LANES, VPT> row(a, t, sub, low);
      inv = row.inverse();
#pragma unroll
      for (int j = 0; j < VPT; ++j) acc[j] = fmaf(row.score(j), inv, acc[j]);
    }
    if (on) {
      valid += sub == 0;
      for (int k = sub; k < a.topk;) {
        if (id >= 0 && id < a.experts)
          atomicAdd(&s_cnt[id], 1);
        else if (id != -1)
          bad = 1;
        k += LANES;
        if (k < a.topk) id = choice(t, k);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) s_sum[group * kCols + column<LANES>(sub, j)] = acc[j];
  if (valid) atomicAdd(&s_val, valid);
  if (bad) s_flag = 1;
  __syncthreads();
  for (int i = threadIdx.x; i < a.experts; i += kThreads) {
    float v = 0.f;
#pragma unroll 8
    for (int g = 0; g < kGroups; ++g) v += s_sum[g * kCols + i];
    a.psum[static_cast<int64_t>(item) * a.experts + i] = v;
    a.pcnt[static_cast<int64_t>(item) * a.experts + i] = s_cnt[i];
  }
  if (threadIdx.x == 0) {
    a.pval[item] = s_val;
    a.pflag[item] = s_flag;
  }
}

// Valid tokens of the batch and the conditions seen, from every chunk's: with
// 65536 sequences the pass as a whole takes 0.9 ms, 5.1 where every block of the
// next kernel adds them up.
__global__ void __launch_bounds__(kTotalThreads) k_balance_total(const __grid_constant__ BalanceArgs a) {
  __shared__ int s_n[kTotalThreads / 32], s_bad[kTotalThreads / 32];
  int n = 0, bad = 0;
#pragma unroll 8
  for (int i = threadIdx.x; i < a.items; i += kTotalThreads) {
    n += a.pval[i];
    bad |= a.pflag[i];
  }
  n = __reduce_add_sync(0xffffffffu, n);
  bad = __any_sync(0xffffffffu, bad);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) {
    s_n[warp] = n;
    s_bad[warp] = bad;
  }
  __syncthreads();
  if (warp == 0) {
    n = __reduce_add_sync(0xffffffffu, s_n[lane]);
    bad = __any_sync(0xffffffffu, s_bad[lane]);
    if (lane == 0) {
      a.total[0] = n;
      a.total[1] = bad;
    }
  }
}

// One block per (sequence, 32 experts): adds the chunks' partial rows, writes
// the load, adds the counts; the last block to finish adds the loss.  Its time
// is that of a few dependent trips to L2.
__global__ void __launch_bounds__(kFinWide) k_balance_finalize(const __grid_constant__ BalanceArgs a) {
  __shared__ float s_f[kFinWide / 32][32];
  __shared__ int s_i[kFinWide / 32][32];
  __shared__ int s_all[kFinWide / 32], s_mine[kFinWide / 32], s_bad[kFinWide / 32];
  __shared__ int s_last;
  const int threads = blockDim.x, warps = threads / 32;
  const int eblocks = (a.experts + 31) / 32;
  const int s = blockIdx.x / eblocks, eb = blockIdx.x % eblocks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = seq_at(a, s), end = seq_at(a, s + 1);
  const int i0 = b / a.chunk + s, i1 = b < end ? min((end - 1) / a.chunk + s, a.items - 1) : i0 - 1;
  int misplaced = 0;   // bounds that do not ascend within [0, tokens]
  if (blockIdx.x == 0 && a.seq_begin != nullptr)
    for (int i = threadIdx.x; i <= a.sequences; i += threads) {
      const int at = a.seq_begin[i];
      if (at < 0 || at > a.tokens || (i > 0 && at < a.seq_begin[i - 1])) misplaced = 1;
    }
  griddep_wait();
  // Partial rows: warp w takes every `warps`th, a lane one expert.  Where bounds are
  // out of order a sequence may span chunks that no sequence had in the first pass:
  // they have no valid token, and their rows were not written.
  float p = 0.f;
  int c = 0;
  if (eb * 32 + lane < a.experts) {
    const int64_t at = static_cast<int64_t>(eb) * 32 + lane;
#pragma unroll 4
    for (int i = i0 + warp; i <= i1; i += warps) {
      const bool written = a.pval[i] != 0;
      const float pi = a.psum[i * static_cast<int64_t>(a.experts) + at];
      const int ci = a.pcnt[i * static_cast<int64_t>(a.experts) + at];
      p += written ? pi : 0.f;
      c += written ? ci : 0;
    }
  }
  // valid tokens of the batch and of this sequence, device conditions
  int all = 0, mine = 0, bad = 0;
#pragma unroll 4
  for (int i = a.total == nullptr ? threadIdx.x : a.items; i < a.items; i += threads) {
    all += a.pval[i];
    bad |= a.pflag[i];
  }
  for (int i = i0 + threadIdx.x; i <= i1; i += threads) mine += a.pval[i];
  all = __reduce_add_sync(0xffffffffu, all);
  mine = __reduce_add_sync(0xffffffffu, mine);
  bad = __any_sync(0xffffffffu, bad);
  s_f[warp][lane] = p;
  s_i[warp][lane] = c;
  if (lane == 0) {
    s_all[warp] = all;
    s_mine[warp] = mine;
    s_bad[warp] = bad;
  }
  misplaced = __syncthreads_or(misplaced);
  if (warp == 0) {
    p = 0.f;
    c = 0;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {
      p += s_f[w][lane];
      c += s_i[w][lane];
    }
    all = __reduce_add_sync(0xffffffffu, lane < warps ? s_all[lane] : 0);
    mine = __reduce_add_sync(0xffffffffu, lane < warps ? s_mine[lane] : 0);
    bad = __any_sync(0xffffffffu, lane < warps ? s_bad[lane] : 0);
    if (a.total != nullptr) {
      all = a.total[0];
      bad = a.total[1];
    }
    const int e = eb * 32 + lane;
    float contrib = 0.f;
    if (e < a.experts) {
      const float scale = mine == 0 ? 0.f
                                    : a.coef / static_cast<float>(all) *
                                          (static_cast<float>(a.experts) /
                                           (static_cast<float>(a.topk) * static_cast<float>(mine)));
      const float f = scale * static_cast<float>(c);
      contrib = f * p;
      a.load[static_cast<int64_t>(s) * a.experts + e] = f;
      if (c) atomicAdd(a.counts + e, c);
    }
    contrib = group_sum<32>(contrib);
    if (lane == 0 && gridDim.x == 1) {
      *a.loss = contrib;
      *a.status = bad || misplaced ? MUON_FLAG_INDEX : 0u;
    } else if (lane == 0) {
      a.lossp[blockIdx.x] = contrib;
      if (blockIdx.x == 0) *a.bounds = misplaced;
      __threadfence();
      s_last = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
    }
  }
  if (gridDim.x == 1) return;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  float v = 0.f;
  for (unsigned i = threadIdx.x; i < gridDim.x; i += threads) v += __ldcg(a.lossp + i);
  v = group_sum<32>(v);
  if (lane == 0) s_f[0][warp] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = 0.f;
    for (int w = 0; w < warps; ++w) v += s_f[0][w];
    *a.loss = v;
    *a.status = bad || __ldcg(a.bounds) ? MUON_FLAG_INDEX : 0u;
  }
}

template <int LANES, int VPT, bool FULL>
__device__ __forceinline__ void store_row(const BalanceArgs& a, int64_t off, int sub,
                                          const float (&d)[VPT]) {
#pragma unroll
  for (int q = 0; q < VPT / 4; ++q) {
    const int c = column<LANES>(sub, 4 * q);
    if (a.dvec) {
      if (!FULL && c >= a.experts) continue;
      if (a.ddt == MUON_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.dlogits) + off + c);
        float4 v = make_float4(d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]);
        if (a.accumulate) {
          const float4 o = *p;
          v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
        }
        *p = v;
      } else {
        uint2* p = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.dlogits) + off + c);
        float v[4] = {d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]};
        if (a.accumulate) {
          const uint2 o = *p;
          const float2 f0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&o.x));
          const float2 f1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&o.y));
          v[0] += f0.x; v[1] += f0.y; v[2] += f1.x; v[3] += f1.y;
        }
        const __nv_bfloat162 h0 = __floats2bfloat162_rn(v[0], v[1]);
        const __nv_bfloat162 h1 = __floats2bfloat162_rn(v[2], v[3]);
        *p = make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (c + k >= a.experts) continue;
        if (a.ddt == MUON_F32) {
          float* p = static_cast<float*>(a.dlogits) + off + c + k;
          *p = a.accumulate ? *p + d[4 * q + k] : d[4 * q + k];
        } else {
          __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.dlogits) + off + c + k;
          *p = __float2bfloat16_rn(a.accumulate ? __bfloat162float(*p) + d[4 * q + k] : d[4 * q + k]);
        }
      }
    }
  }
}

// Where every expert of a sequence has the load `level` or none and a token's
// probability is mostly on the former, f - sum f p of those is level times the
// probability of the others: `rest`, which does not cancel.  (It is 0 where every
// token takes every expert that is enabled, and so is the gradient.)  The whole
// warp calls it; true: use rest where f is not 0.
template <int LANES, int VPT, typename Score>
__device__ __forceinline__ bool near_level(float level, float dot, float inv, const float (&f)[VPT],
                                           const Score& score, float& rest) {
  const bool near = dot > 0.5f * level && level > 0.f;
  if (__any_sync(0xffffffffu, near)) {
    float others = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) others += f[j] == 0.f ? score(j) : 0.f;
    rest = group_sum<LANES>(others) * inv * level;
  }
  return near;
}

// The gradient of a low row (1 - sigma is 1), from its sequence's row of load, value by
// value; dlogits may be the logits: a value is read before its own is written.
template <int LANES, int VPT>
__device__ __forceinline__ void low_gradient(const BalanceArgs& a, int t, int s, float scale, int sub, bool low) {
  const LowRow<LANES, VPT> row(a, t, sub, low);
  const float inv = row.inverse();
  const float* load = a.load + static_cast<int64_t>(low ? s : 0) * a.experts;
  float dot = 0.f;
#pragma unroll 1
  for (int j = 0; j < VPT; ++j) {
    const int c = column<LANES>(sub, j);
    if (c < a.experts) dot = fmaf(load[c], row.score(j), dot);
  }
  dot = group_sum<LANES>(dot) * inv;
  if (!low) return;
#pragma unroll 1
  for (int j = 0; j < VPT; ++j) {
    const int c = column<LANES>(sub, j);
    if (c >= a.experts) continue;
    const float d = scale * inv * row.score(j) * (load[c] - dot);
    const int64_t at = static_cast<int64_t>(t) * a.dlogits_stride + c;
    if (a.ddt == MUON_F32) {
      float* p = static_cast<float*>(a.dlogits) + at;
      *p = a.accumulate ? *p + d : d;
    } else {
      __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.dlogits) + at;
      *p = __float2bfloat16_rn(a.accumulate ? __bfloat162float(*p) + d : d);
    }
  }
}

// LEVELS: with near_level.
template <int LANES, int VPT, bool FULL, bool SIGMOID, bool LEVELS>
__global__ void __launch_bounds__(kThreads, VPT <= 16 ? 4 : 2)
    k_balance_backward(const __grid_constant__ BalanceArgs a) {
  constexpr int kGroups = kThreads / LANES;
  const int group = threadIdx.x / LANES, sub = threadIdx.x % LANES;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kGroups * a.row_steps);
  const int64_t last = first + static_cast<int64_t>(a.row_steps) * kGroups;
  const int stop = static_cast<int>(last < a.tokens ? last : a.tokens);
  const float scale = a.dloss == nullptr ? 1.f : *a.dloss;
  int s = -2, s_end = 0;
  float level = 0.f;   // the one load of a sequence whose experts have that or none; else 0
  float f[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) f[j] = 0.f;
  const auto is_on = [&](int t) { return t < stop && (a.mask == nullptr || a.mask[t] != 0); };
  bool next_on = is_on(static_cast<int>(first) + group);   // fetched a row ahead, as in the forward pass
  for (int tb = static_cast<int>(first); tb < stop; tb += kGroups) {   // the whole block together
    const bool in = tb + group < stop;
    const int t = in ? tb + group : stop - 1;
    const bool fresh = s == -2 || t >= s_end;
    if (fresh) {
      s = seq_of_token(a, t);
      s_end = s + 1 <= a.sequences ? seq_at(a, s + 1) : a.tokens;
      const bool inside = s >= 0 && t < s_end;
      if (!inside) s_end = t;   // between sequences: look again at the next token
      load_row<LANES, VPT, FULL>(a.load, static_cast<int64_t>(inside ? s : 0) * a.experts, MUON_F32,
                                 a.experts, a.lvec, sub, 0.f, f);
      if (!inside) s = -2;
    }
    if (LEVELS && __any_sync(0xffffffffu, fresh)) {   // the reductions take the whole warp
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < VPT; ++j) top = fmaxf(top, f[j]);
      top = group_max<LANES>(top);
      int other = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) other |= f[j] != 0.f && f[j] != top;
      level = group_sum<LANES>(static_cast<float>(other)) == 0.f ? top : 0.f;
    }
    const bool on = next_on && s >= 0;
    next_on = is_on(tb + group + kGroups);
    float x[VPT];
    if (on) {
      load_row<LANES, VPT, FULL>(a.logits, static_cast<int64_t>(t) * a.logits_stride, a.dtype,
                                 a.experts, a.vec, sub, -INFINITY, x);
    } else {
#pragma unroll
      for (int j = 0; j < VPT; ++j) x[j] = -INFINITY;
    }
    const float inv = row_scores<LANES, VPT, SIGMOID, true>(x);
    const bool low = SIGMOID && on && is_low(inv);
    const float by = scale * inv;
    float dot = 0.f, rest = 0.f;
    if constexpr (SIGMOID) {
      // x holds t = exp(-l): the score is s = 1 / (1 + t), its slope s (1 - s) with
      // 1 - s = t s where s is near 1 (no cancellation)
#pragma unroll
      for (int j = 0; j < VPT; ++j) dot = fmaf(f[j], __fdividef(1.f, 1.f + x[j]), dot);
      dot = group_sum<LANES>(dot) * inv;
      const auto score = [&](int j) { return __fdividef(1.f, 1.f + x[j]); };
      const bool near = LEVELS && near_level<LANES, VPT>(level, dot, inv, f, score, rest);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const float r = __fdividef(1.f, 1.f + x[j]);
        const float slope = x[j] < 1.f ? x[j] * r : 1.f - r;
        x[j] = by * r * slope * (near && f[j] != 0.f ? rest : f[j] - dot);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPT; ++j) dot = fmaf(f[j], x[j], dot);
      dot = group_sum<LANES>(dot) * inv;
      const auto score = [&](int j) { return x[j]; };
      const bool near = LEVELS && near_level<LANES, VPT>(level, dot, inv, f, score, rest);
#pragma unroll
      for (int j = 0; j < VPT; ++j) x[j] = by * x[j] * (near && f[j] != 0.f ? rest : f[j] - dot);
    }
    if (!on) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) x[j] = 0.f;
    }
    if (in && (on || !a.accumulate) && !low)
      store_row<LANES, VPT, FULL>(a, static_cast<int64_t>(t) * a.dlogits_stride, sub, x);
    if (SIGMOID && __any_sync(0xffffffffu, low)) low_gradient<LANES, VPT>(a, t, s, scale, sub, low);
  }
}

// Lanes and values a row takes: the narrowest that holds it, with up to 16
// values a lane before more lanes (a value costs its share of the row's three
// reductions, which take log2(lanes) shuffles each).
template <template <int, int, bool> class F, int LANES, int VPT>
cudaError_t full_or_not(const BalanceArgs& a, cudaStream_t st) {
  return a.experts == LANES * VPT ? F<LANES, VPT, true>::run(a, st) : F<LANES, VPT, false>::run(a, st);
}

template <template <int, int, bool> class F>
cudaError_t by_width(const BalanceArgs& a, cudaStream_t st) {
  if (a.experts <= 32) return full_or_not<F, 8, 4>(a, st);
  if (a.experts <= 64) return full_or_not<F, 8, 8>(a, st);
  if (a.experts <= 128) return full_or_not<F, 8, 16>(a, st);
  if (a.experts <= 256) return full_or_not<F, 16, 16>(a, st);
  if (a.experts <= 384) return full_or_not<F, 32, 12>(a, st);
  if (a.experts <= 512) return full_or_not<F, 32, 16>(a, st);
  return F<32, 32, false>::run(a, st);
}

template <int LANES, int VPT, bool FULL>
struct Forward {
  static cudaError_t run(const BalanceArgs& a, cudaStream_t st) {
    if (a.sigmoid)
      k_balance_forward<LANES, VPT, FULL, true><<<a.items, kThreads, 0, st>>>(a);
    else
      k_balance_forward<LANES, VPT, FULL, false><<<a.items, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
};

template <int LANES, int VPT, bool FULL>
struct Backward {
  static cudaError_t run(const BalanceArgs& a, cudaStream_t st) {
    // a group keeps its sequence's load over up to 8 rows, fewer where the
    // tokens would not fill 152 SMs eight times over
    constexpr int kGroups = kThreads / LANES;
    BalanceArgs b = a;
    const int steps = a.tokens / (kGroups * 152 * 8);
    b.row_steps = steps < 1 ? 1 : steps > 8 ? 8 : steps;
    const int64_t rows = static_cast<int64_t>(kGroups) * b.row_steps;
    const unsigned blocks = static_cast<unsigned>((a.tokens + rows - 1) / rows);
    if (a.sigmoid)
      run_scored<true>(b, blocks, st);
    else
      run_scored<false>(b, blocks, st);
    return cudaGetLastError();
  }

  template <bool SIGMOID>
  static void run_scored(const BalanceArgs& a, unsigned blocks, cudaStream_t st) {
    if constexpr (LANES * VPT <= 64) {
      if (a.levels) {
        k_balance_backward<LANES, VPT, FULL, SIGMOID, true><<<blocks, kThreads, 0, st>>>(a);
        return;
      }
    }
    k_balance_backward<LANES, VPT, FULL, SIGMOID, false><<<blocks, kThreads, 0, st>>>(a);
  }
};

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct Layout {
  size_t psum, pcnt, pval, pflag, lossp, total;
};

Layout layout(int64_t tokens, int experts, int sequences) {
  const size_t items = static_cast<size_t>(chunk_items(tokens, experts, sequences));
  Layout l;
  l.psum = kHeader;
  l.pcnt = l.psum + align256(items * experts * 4);
  l.pval = l.pcnt + align256(items * experts * 4);
  l.pflag = l.pval + align256(items * 4);
  l.lossp = l.pflag + align256(items * 4);
  l.total = l.lossp + align256(static_cast<size_t>(sequences) * ((experts + 31) / 32) * 4);
  return l;
}

// Rows that may be read (or written) four values at a time.
int vectorised(const void* p, int dtype, int64_t stride, int n) {
  return n % 4 == 0 && stride % 4 == 0 && at_multiple(p, 4 * esize(dtype));
}

muon_status_t check_sizes(int64_t tokens, int experts, int sequences) {
  if (tokens < 0 || experts < 1 || sequences < 1) return MUON_ERR_INVALID_ARG;
  if (experts > kMaxExperts || tokens >= (int64_t{1} << 31) - (1 << 20) || sequences > (1 << 20))
    return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

muon_status_t check_balance(const muon_balance_t* b) {
  if (b == nullptr) return MUON_ERR_INVALID_ARG;
  const muon_status_t s = check_sizes(b->tokens, b->experts, b->sequences);
  if (s != MUON_OK) return s;
  if (b->dtype != MUON_BF16 && b->dtype != MUON_F32) return MUON_ERR_INVALID_ARG;
  if (b->score != MUON_SCORE_SOFTMAX && b->score != MUON_SCORE_SIGMOID) return MUON_ERR_INVALID_ARG;
  if (b->logits_stride < b->experts) return MUON_ERR_INVALID_ARG;
  if (b->tokens > 0 && b->logits == nullptr) return MUON_ERR_INVALID_ARG;
  if (b->seq_begin == nullptr && b->sequences != 1) return MUON_ERR_INVALID_ARG;
  if (!at_multiple(b->logits, esize(b->dtype)) || !at_multiple(b->seq_begin, 4))
    return MUON_ERR_MISALIGNED;
  return MUON_OK;
}

BalanceArgs base_args(const muon_balance_t* b) {
  BalanceArgs a{};
  a.tokens = static_cast<int>(b->tokens);
  a.experts = b->experts;
  a.topk = b->topk;
  a.sequences = b->sequences;
  a.chunk = chunk_tokens(b->tokens, b->experts, b->sequences);
  a.items = static_cast<int>(chunk_items(b->tokens, b->experts, b->sequences));
  a.logits = b->logits;
  a.dtype = b->dtype;
  a.logits_stride = b->logits_stride;
  a.chosen = b->chosen;
  a.chosen_bytes = b->chosen_bytes;
  a.chosen_stride = b->chosen_stride;
  a.seq_begin = b->seq_begin;
  a.mask = b->token_mask;
  a.sigmoid = b->score == MUON_SCORE_SIGMOID;
  a.coef = b->coef;
  a.vec = vectorised(b->logits, b->dtype, b->logits_stride, b->experts);
  return a;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status_t muon_balance_workspace_size(int64_t tokens, int experts, int sequences,
                                          size_t* bytes) {
  if (bytes == nullptr) return MUON_ERR_INVALID_ARG;
  const muon_status_t s = check_sizes(tokens, experts, sequences);
  if (s != MUON_OK) return s;
  *bytes = layout(tokens, experts, sequences).total;
  return MUON_OK;
}

muon_status_t muon_balance_forward(const muon_balance_t* b, float* loss, int32_t* counts,
                                   float* load, void* workspace, size_t workspace_bytes,
                                   muon_stream_t stream) {
  muon_status_t s = check_balance(b);
  if (s != MUON_OK) return s;
  if (b->topk < 1 || b->topk > b->experts || !std::isfinite(b->coef)) return MUON_ERR_INVALID_ARG;
  if (b->chosen_bytes != 4 && b->chosen_bytes != 8) return MUON_ERR_INVALID_ARG;
  if (b->chosen_stride < b->topk || (b->tokens > 0 && b->chosen == nullptr))
    return MUON_ERR_INVALID_ARG;
  if (loss == nullptr || counts == nullptr || load == nullptr || workspace == nullptr)
    return MUON_ERR_INVALID_ARG;
  if (!at_multiple(b->chosen, b->chosen_bytes) || !at_multiple(loss, 4) ||
      !at_multiple(counts, 4) || !at_multiple(load, 4) || !at_multiple(workspace, 256))
    return MUON_ERR_MISALIGNED;
  const Layout l = layout(b->tokens, b->experts, b->sequences);
  if (workspace_bytes < l.total) return MUON_ERR_WORKSPACE_TOO_SMALL;

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  BalanceArgs a = base_args(b);
  a.psum = reinterpret_cast<float*>(ws + l.psum);
  a.pcnt = reinterpret_cast<int*>(ws + l.pcnt);
  a.pval = reinterpret_cast<int*>(ws + l.pval);
  a.pflag = reinterpret_cast<int*>(ws + l.pflag);
  a.lossp = reinterpret_cast<float*>(ws + l.lossp);
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.ticket = reinterpret_cast<int*>(ws) + 1;
  a.bounds = reinterpret_cast<int*>(ws) + 2;
  a.total = a.items > kTotalItems ? reinterpret_cast<int*>(ws) + 3 : nullptr;
  a.loss = loss;
  a.counts = counts;
  a.load = load;
  const double rows = static_cast<double>(b->tokens);
  prof_begin(kKindBalance, st);
  cudaError_t e = by_width<Forward>(a, st);
  prof_end(kKindBalance, st, 0.0,
           rows * (b->experts * esize(b->dtype) + b->topk * b->chosen_bytes));
  if (e != cudaSuccess) return MUON_ERR_CUDA;
  if (a.total != nullptr) {
    prof_begin(kKindBalance, st);
    k_balance_total<<<1, kTotalThreads, 0, st>>>(a);
    prof_end(kKindBalance, st, 0.0, 0.0);
    if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
  }
  // a programmatic dependent of the kernel before (it waits for the partial rows)
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(b->sequences) * ((b->experts + 31) / 32));
  // A block with few partial rows is small, so that more of them run beside each
  // other: 131072 x 64 in 1000 sequences 74 -> 44 us, in 32 sequences 44 -> 42.  A
  // sequence of many rows wants a warp for each of them: one sequence takes 27 us,
  // 35 with the small block.
  cfg.blockDim = dim3(a.items > 64 * b->sequences ? kFinWide : kFinNarrow);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  prof_begin(kKindBalance, st);
  e = cudaLaunchKernelEx(&cfg, k_balance_finalize, a);
  prof_end(kKindBalance, st, 0.0, 4.0 * b->sequences * b->experts);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

muon_status_t muon_balance_backward(const muon_balance_t* b, const float* load,
                                    const float* dloss, void* dlogits, muon_dtype_t ddt,
                                    int64_t dlogits_stride, int accumulate,
                                    muon_stream_t stream) {
  const muon_status_t s = check_balance(b);
  if (s != MUON_OK) return s;
  if (ddt != MUON_BF16 && ddt != MUON_F32) return MUON_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return MUON_ERR_INVALID_ARG;
  if (dlogits_stride < b->experts || load == nullptr || (b->tokens > 0 && dlogits == nullptr))
    return MUON_ERR_INVALID_ARG;
  if (!at_multiple(load, 4) || !at_multiple(dloss, 4) || !at_multiple(dlogits, esize(ddt)))
    return MUON_ERR_MISALIGNED;
  if (b->tokens == 0) return MUON_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  BalanceArgs a = base_args(b);
  a.load = const_cast<float*>(load);
  a.dloss = dloss;
  a.dlogits = dlogits;
  a.ddt = ddt;
  a.dlogits_stride = dlogits_stride;
  a.lvec = vectorised(load, MUON_F32, b->experts, b->experts);
  a.dvec = vectorised(dlogits, ddt, dlogits_stride, b->experts);
  a.accumulate = accumulate;
  // Tokens that take a good part of a few experts may take all that are enabled, and
  // get their exact 0.  Elsewhere the search is left out, and a rounding remainder
  // left: looking for such sequences at every width, by the loads themselves, costs
  // every batch (131072 x 256: fp32 47.8 -> 49.8 us, bf16 36.9 -> 40.9; 200 experts
  // bf16 39.3 -> 45.2).
  a.levels = 4 * static_cast<int64_t>(b->topk) >= b->experts;
  prof_begin(kKindBalance, st);
  const cudaError_t e = by_width<Backward>(a, st);
  prof_end(kKindBalance, st, 0.0,
           static_cast<double>(b->tokens) * b->experts *
               (esize(b->dtype) + esize(ddt) * (accumulate ? 2 : 1)));
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

}  // extern "C"
