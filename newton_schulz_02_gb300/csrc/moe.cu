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
// the traffic is what the definition has (but for dout in combine's gradient, which is
// read once for every 8 choices, and once more where two kernels take it), and a
// token's sum is a loop over k in one thread, in that order, with no atomics.  Going by row would read a
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
// Copies a thread, up to which one block does it: 2048 copies take it 4.6 us in a graph, one
// launch less; 4096 took it 7.0, the two kernels 5.1.
constexpr int64_t kAlonePer = 2;
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
  if (copies <= kAlonePer * kSortThreads) {
    const int64_t per = (copies + kSortThreads - 1) / kSortThreads;
    return {per < 1 ? 1 : static_cast<int>(per), 1, 1};
  }
  const int64_t wave = int64_t{kSortThreads} * kSortBlocks;
  SortPlan p{kMaxPer, 1, 1};
  if (copies <= kMaxPer * wave) p.per = static_cast<int>((copies + wave - 1) / wave);
  else p.rounds = static_cast<int>((copies + kMaxPer * wave - 1) / (kMaxPer * wave));
  const int64_t block = int64_t{kSortThreads} * p.per * p.rounds;
  p.blocks = static_cast<int>((copies + block - 1) / block);
  return p;
}

struct SortArgs {
  uint32_t copies, rows;
  int experts, per, rounds, blocks;
  int dense;                 // copy i's choice is chosen[i]
  int quad_bits;             // log2 of the threads that read one row of counts
  int stride;                // of the rows of counts, a multiple of 4
  Divider topk;
  const void* chosen;
  int chosen_bytes;
  int64_t chosen_stride;
  const uint8_t* mask;
  int32_t* offsets;
  int32_t* order;
  int32_t* place;
  int* counts;               // [blocks][stride]
  uint32_t* flags;           // [blocks]
  uint32_t* status;
};

// Copy j of a thread's, or one that is there: loads from it need no branch between them, so
// that all are on their way before one is looked at (131072 x 8 of 256 13.7 -> 12.5 us).
__device__ __forceinline__ uint32_t some_copy(const SortArgs& a, uint32_t begin, int j) {
  return min(begin + (j < a.per ? 32 * j : 0), a.copies - 1);
}

// Choices of copies begin, begin + 32, ... as they are.  PER is a.per up to 2, which is
// loads fewer (16384 x 8 8.6 -> 7.2 us), else 8 (a form for 4 took 65536 x 8 11.8 us, this
// 10.5).  There are copies.
template <int PER>
__device__ __forceinline__ void load_choices(const SortArgs& a, uint32_t begin, int64_t (&e)[PER]) {
  int64_t at[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) at[j] = some_copy(a, begin, j);
  if (!a.dense) {   // rows apart from each other
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const uint32_t i = static_cast<uint32_t>(at[j]), t = quotient(i, a.topk);
      at[j] = t * a.chosen_stride + (i - t * a.topk.d);
    }
  }
  if (a.chosen_bytes == 8) {
#pragma unroll
    for (int j = 0; j < PER; ++j) e[j] = static_cast<const int64_t*>(a.chosen)[at[j]];
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) e[j] = static_cast<const int32_t*>(a.chosen)[at[j]];
  }
}

// Their experts, -1 where there is none; a number that is neither sets *bad.
template <int PER>
__device__ __forceinline__ void load_keys(const SortArgs& a, uint32_t begin, int (&key)[PER], bool* bad) {
#pragma unroll
  for (int j = 0; j < PER; ++j) key[j] = -1;
  if (a.copies == 0) return;
  int64_t e[PER];
  uint32_t valid[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) valid[j] = 1;
  load_choices(a, begin, e);
  if (a.mask != nullptr) {
#pragma unroll
    for (int j = 0; j < PER; ++j) valid[j] = a.mask[quotient(some_copy(a, begin, j), a.topk)];
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const bool on = j < a.per && begin + 32 * j < a.copies && valid[j] != 0;
    const bool known = static_cast<uint64_t>(e[j]) < static_cast<uint64_t>(a.experts);
    if (on && known) key[j] = static_cast<int>(e[j]);
    if (on && !known && e[j] != -1) *bad = true;
  }
}

// Ranks that k_moe_rank left, -1 for a copy without an expert; key gets the choice of the
// others.
template <int PER>
__device__ __forceinline__ void load_ranks(const SortArgs& a, uint32_t begin, const int64_t (&e)[PER],
                                           int (&key)[PER], int (&rank)[PER]) {
#pragma unroll
  for (int j = 0; j < PER; ++j) rank[j] = a.place[some_copy(a, begin, j)];
#pragma unroll
  for (int j = 0; j < PER; ++j)
    key[j] = j < a.per && begin + 32 * j < a.copies && rank[j] >= 0 ? static_cast<int>(e[j]) : -1;
}

// First of a lane's copies in a round: a block's copies are consecutive, and so
// are a warp's in each round.  (Below 2^32: copies are fewer than 2^31, and a
// block's rounds reach at most one block's length past them.)
__device__ __forceinline__ uint32_t lane_begin(const SortArgs& a, int round) {
  return ((blockIdx.x * a.rounds + round) * kSortWarps + (threadIdx.x >> 5)) * 32 * a.per + (threadIdx.x & 31);
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
  if (lane == 31) warp_sums[w] = s;
  __syncthreads();
  int t = warp_sums[lane];   // every warp sums the warps' totals up for itself
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += u;
  }
  *all = __shfl_sync(0xffffffffu, t, 31);
  const int before = __shfl_sync(0xffffffffu, t, w > 0 ? w - 1 : 0);
  return s - v + (w > 0 ? before : 0);
}

// offsets[e] of this thread's expert, the end, and the status word.
__device__ __forceinline__ void write_offsets(const SortArgs& a, int first, int all, bool bad) {
  if (static_cast<int>(threadIdx.x) < a.experts)
    a.offsets[threadIdx.x] = static_cast<int32_t>(min(static_cast<uint32_t>(first), a.rows));
  const int any = __syncthreads_or(bad || static_cast<uint32_t>(all) > a.rows);
  if (threadIdx.x == 0) {
    a.offsets[a.experts] = static_cast<int32_t>(min(static_cast<uint32_t>(all), a.rows));
    *a.status = any ? MUON_FLAG_INDEX : 0u;
  }
}

__device__ __forceinline__ void write_copy(const SortArgs& a, uint32_t i, bool keyed, uint32_t row) {
  const bool on = keyed && row < a.rows;
  if (i < a.copies) a.place[i] = on ? static_cast<int32_t>(row) : -1;
  if (on) a.order[row] = static_cast<int32_t>(i);
}

// Ranks the copies of a block among those of the same expert.  A warp owns consecutive
// copies and counts them by itself, 32 at a time: every lane sets its bit in its
// expert's word of `lanes`, and its rank is the count so far plus the bits below its
// own; the lowest lane clears the word and moves the count on.  Then the counts are
// summed up over the warps.  Both kernels for
// 131072 x 8 of 256 take 12.5 us; finding the lanes of one expert with a match over the
// warp took 6.3 us more, with a vote for each bit of its number 3.7.  Half of each
// kernel is its first loads: choices in the one; ranks and counts, 147 KB that
// every SM reads, in the other.
// ALONE: the block holds all copies, and its ranks become rows at once; else they
// are left in `place` for k_moe_place, with the block's counts.
template <bool ALONE, int PER>
__global__ void __launch_bounds__(kSortThreads) k_moe_rank(const __grid_constant__ SortArgs a) {
  extern __shared__ int sm[];
  int* base = sm;                                              // [experts]: ALONE: first row
  uint32_t* lanes = reinterpret_cast<uint32_t*>(sm + a.experts);   // [warps][experts]
  uint16_t* hist = reinterpret_cast<uint16_t*>(lanes + kSortWarps * a.experts);   // [warps][experts]
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x, lane = tid & 31;
  uint32_t* my_lanes = lanes + (tid >> 5) * a.experts;
  uint16_t* mine = hist + (tid >> 5) * a.experts;
  if (!ALONE) griddep_launch_dependents();
  bool bad = false;
  int total = 0;                               // of this thread's expert, over the rounds
  for (int round = 0; round < a.rounds; ++round) {
    const uint32_t begin = lane_begin(a, round);
    int key[PER], rank[PER];
    load_keys(a, begin, key, &bad);
    for (int e = lane; e < a.experts; e += 32) {
      mine[e] = 0;
      my_lanes[e] = 0;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (j >= a.per) break;   // the same for all threads
      const bool on = key[j] >= 0;
      if (on) atomicOr(&my_lanes[key[j]], 1u << lane);
      __syncwarp();
      const uint32_t same = on ? my_lanes[key[j]] : 0u;
      const uint32_t lower = same & ((1u << lane) - 1);
      rank[j] = (on ? mine[key[j]] : 0) + __popc(lower);
      __syncwarp();
      if (on && lower == 0) {
        mine[key[j]] = static_cast<uint16_t>(rank[j] + __popc(same));
        my_lanes[key[j]] = 0;
      }
      __syncwarp();
    }
    __syncthreads();
    const int rounds_before = total;
    if (tid < a.experts) {
      int next = 0;            // at most 8192 in a round
#pragma unroll 8
      for (int k = 0; k < kSortWarps; ++k) {
        const int c = hist[k * a.experts + tid];
        hist[k * a.experts + tid] = static_cast<uint16_t>(next);
        next += c;
      }
      total += next;
    }
    int first = 0, all = 0;
    if constexpr (ALONE) {
      first = block_scan(total, warp_sums, &all);
    }
    if (tid < a.experts) base[tid] = ALONE ? first : rounds_before;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (j >= a.per) break;
      const uint32_t i = begin + 32 * j;
      int r = key[j] >= 0 ? mine[key[j]] + rank[j] : -1;
      if (key[j] >= 0 && (ALONE || a.rounds > 1)) r += base[key[j]];
      if constexpr (ALONE)
        write_copy(a, i, key[j] >= 0, static_cast<uint32_t>(r));
      else if (i < a.copies)
        a.place[i] = r;
    }
    if constexpr (ALONE) write_offsets(a, first, all, bad);
    else if (round + 1 < a.rounds) __syncthreads();   // base and hist have been read
  }
  if constexpr (!ALONE) {
    if (tid < a.experts) a.counts[static_cast<int64_t>(blockIdx.x) * a.stride + tid] = total;
    const int any = __syncthreads_or(bad);
    if (tid == 0) a.flags[blockIdx.x] = any ? MUON_FLAG_INDEX : 0u;
  }
}

// Ranks to rows: the block's first row of each expert is the expert's plus what the
// blocks before this one have of it.  The copies of a block that has one round go out
// sorted, so that runs of `order` are written together: 131072 x 8 of 256 17.2 -> 13.7 us.
template <int PER>
__global__ void __launch_bounds__(kSortThreads) k_moe_place(const __grid_constant__ SortArgs a) {
  extern __shared__ int sm[];                  // [8 threads]: sums by thread, then the sorted copies
  int4* part = reinterpret_cast<int4*>(sm);    // totals, then counts of the blocks before
  int* base = sm + 8 * kSortThreads;           // [experts]
  int* local = base + a.experts;               // [experts]: first of the expert among the sorted copies
  __shared__ int warp_sums[32];
  const int tid = threadIdx.x;
  const bool sorted = a.rounds == 1;
  int64_t choice[PER];
  int key[PER], rank[PER];
  load_choices(a, lane_begin(a, 0), choice);   // before the wait
  griddep_wait();
  load_ranks(a, lane_begin(a, 0), choice, key, rank);
  const bool bad_choice = blockIdx.x == 0 && tid < a.blocks && a.flags[tid] != 0;
  const int own = tid < a.experts ? a.counts[blockIdx.x * a.stride + tid] : 0;
  const int quads = 1 << a.quad_bits;          // threads of a row of counts, four experts each
  const int q = tid & (quads - 1), groups = min(kSortThreads >> a.quad_bits, 32);   // 32: more are slower to join
  int4 total = make_int4(0, 0, 0, 0), before = total;
  if (4 * q < a.experts) {
#pragma unroll 8
    for (int b = tid >> a.quad_bits; b < a.blocks && (tid >> a.quad_bits) < groups; b += groups) {
      const int4 c = *reinterpret_cast<const int4*>(a.counts + b * a.stride + 4 * q);
      const int on = b < static_cast<int>(blockIdx.x) ? -1 : 0;
      total.x += c.x; total.y += c.y; total.z += c.z; total.w += c.w;
      before.x += c.x & on; before.y += c.y & on; before.z += c.z & on; before.w += c.w & on;
    }
  }
  part[tid] = total;
  part[kSortThreads + tid] = before;
  int held, all;
  const int first_local = block_scan(own, warp_sums, &held);   // and a barrier
  int sum = 0, mine = 0;
  if (tid < a.experts) {
#pragma unroll 4
    for (int g = 0; g < groups; ++g) {
      sum += sm[4 * (g << a.quad_bits) + tid];
      mine += sm[4 * (kSortThreads + (g << a.quad_bits)) + tid];
    }
  }
  __syncthreads();
  const int first = block_scan(sum, warp_sums, &all);
  if (tid < a.experts) {
    base[tid] = first + mine - (sorted ? first_local : 0);
    local[tid] = first_local;
  }
  __syncthreads();
  if (sorted) {
    const uint32_t block_first = blockIdx.x * a.per * kSortThreads;
    uint32_t* stage = reinterpret_cast<uint32_t*>(sm);   // expert and copy of the block
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (key[j] < 0) continue;
      const uint32_t i = lane_begin(a, 0) + 32 * j;
      const int at = local[key[j]] + rank[j];
      const uint32_t row = static_cast<uint32_t>(base[key[j]] + at);
      a.place[i] = row < a.rows ? static_cast<int32_t>(row) : -1;
      stage[at] = static_cast<uint32_t>(key[j]) << 16 | (i - block_first);
    }
    __syncthreads();
    for (int at = tid; at < held; at += kSortThreads) {
      const uint32_t v = stage[at];
      const uint32_t row = static_cast<uint32_t>(base[v >> 16] + at);
      if (row < a.rows) a.order[row] = static_cast<int32_t>(block_first + (v & 0xFFFFu));
    }
  } else {
    for (int round = 0; round < a.rounds; ++round) {
      const uint32_t begin = lane_begin(a, round);
      if (round > 0) {
        load_choices(a, begin, choice);
        load_ranks(a, begin, choice, key, rank);
      }
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (key[j] >= 0)
          write_copy(a, begin + 32 * j, true, static_cast<uint32_t>(base[key[j]] + rank[j]));
    }
  }
  if (blockIdx.x == 0)
    write_offsets(a, first, all, bad_choice);
}

size_t rank_smem(int experts) { return static_cast<size_t>(6 * kSortWarps + 4) * experts; }
size_t place_smem(int experts) { return static_cast<size_t>(8 * kSortThreads + 2 * experts) * 4; }
static_assert(kMaxPer <= 8 && kMaxPer * kSortThreads <= 1 << 16 && kMaxExperts <= kSortThreads);

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

template <int N>
__device__ __forceinline__ Item item_of(const RowArgs& a) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  Item p;
  p.on = i < a.items;
  const uint32_t at = p.on ? i : a.items - 1;
  p.token = quotient(at, a.per_row);
  p.col = static_cast<int>(at - p.token * a.per_row.d) * N;
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
  const Item p = item_of<kCols>(a);
  const int32_t* at = a.place + static_cast<int64_t>(p.token) * a.topk;
  uint32_t next = static_cast<uint32_t>(at[0]);   // a row ahead
  float x[kCols];
  load_values<TX, WHOLE>(a.x, p.token, p.col, p.n, x);
  Codes<kCols> c;
  if constexpr (CODES) c = encode(x);
  for (int k = 0; k < a.topk; ++k) {
    const uint32_t row = next;
    if (k + 1 < a.topk) next = static_cast<uint32_t>(at[k + 1]);
    const bool in = p.on && row < a.rows;
    store_values<TY, WHOLE>(a.y, in ? row : 0, p.col, in ? p.n : 0, x);
    if constexpr (CODES) {
      if (in) store_codes(a.codes, row, p.col, c);
    }
  }
}

// The same for rows that start anywhere, and are wide enough for a warp: a warp takes
// 32 x kPieces pieces of 16 bytes of a token, side by side.  All of a warp's
// pieces are off a row's 16-byte boundaries by the same amount, so a shift is a choice
// of registers in a branch that all lanes take together, with the next lane's first words
// behind the own ones; what is before the first boundary and after the last goes out one
// value a lane.  8 rows of 7001 columns a token take 313 us (8192 tokens, fp32) and 312
// (16384, bf16), 97% of the copy rate; with 16 columns a thread, whose sectors go out in
// two halves, 661 and 467.
// Words Q .. Q + 3 of a lane's four and the next lane's (HALF: from the middle of word
// Q on); lane 31's next is lane 0 of `after`.
template <int Q, bool HALF>
__device__ __forceinline__ uint4 piece_from(const uint32_t (&w)[4], const uint32_t (&after)[4], int lane) {
  constexpr int kNext = Q + (HALF ? 1 : 0);
  uint32_t all[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) all[k] = w[k];
#pragma unroll
  for (int k = 0; k < kNext; ++k)
    all[4 + k] = __shfl_sync(0xffffffffu, lane == 0 ? after[k] : w[k], (lane + 1) & 31);
  uint32_t out[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    out[k] = HALF ? __byte_perm(all[Q + k], all[Q + k + (HALF ? 1 : 0)], 0x5432) : all[Q + k];
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// The 16 bytes from byte `by` (even, below 16, the same for all lanes) of the lane's
// words on.
__device__ __forceinline__ uint4 shifted_piece(const uint32_t (&w)[4], const uint32_t (&after)[4], int by,
                                               int lane) {
  switch (by >> 1) {
    case 0: return piece_from<0, false>(w, after, lane);
    case 2: return piece_from<1, false>(w, after, lane);
    case 4: return piece_from<2, false>(w, after, lane);
    case 6: return piece_from<3, false>(w, after, lane);
    case 1: return piece_from<0, true>(w, after, lane);
    case 3: return piece_from<1, true>(w, after, lane);
    case 5: return piece_from<2, true>(w, after, lane);
    default: return piece_from<3, true>(w, after, lane);
  }
}

// Writes a warp's n columns, PIECES x 32 pieces side by side in w, from p on, wherever
// that is.  `end`: in lane l < 8 the column l, in lane 8 + m the last column but m
// (their numbers in `edge`).
template <typename T, int PIECES>
__device__ __forceinline__ void store_pieces(T* p, int n, const uint32_t (&w)[PIECES + 1][4], int edge,
                                             float end, int lane) {
  constexpr int N = 16 / sizeof(T);
  const int by = static_cast<int>(-reinterpret_cast<uintptr_t>(p) & 15u);   // bytes before the boundary
  const int head = by / static_cast<int>(sizeof(T));
  const int tail = n > head ? (n - head) % N : 0;
  if (lane < 8 ? lane < min(head, n) : lane < 8 + tail) store_one(p + edge, end);
  const int full = (n - head) / N;   // whole pieces (none if negative)
  uint4* q = reinterpret_cast<uint4*>(p + head);
#pragma unroll
  for (int j = 0; j < PIECES; ++j) {
    if (j * 32 >= full) break;   // the same for all lanes
    const uint4 u = shifted_piece(w[j], w[j + 1], by, lane);
    if (j * 32 + lane < full) q[j * 32 + lane] = u;
  }
}

// Column of a warp's n that lane `lane` holds for store_pieces; -1: none.
__device__ __forceinline__ int edge_column(int n, int lane) {
  const int e = lane < 8 ? lane : n - 1 - (lane - 8);
  return lane < 16 && e >= 0 && e < n ? e : -1;
}

// Piece j of a warp's n columns from p on, of any type: N columns a lane, 0 behind n.
template <typename T, int N>
__device__ __forceinline__ void load_piece(const T* p, int n, int j, int lane, float (&x)[N]) {
  const int first = (j * 32 + lane) * N;
  if constexpr (N * sizeof(T) >= 16) {
    load_shifted(p + first, n - first, x);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = first + k < n ? static_cast<float>(p[first + k]) : 0.f;
  }
}

// WEIGHTS: a row gets w times the values (the rows' gradient in combine's).
template <typename TX, typename TY, bool CODES, bool WEIGHTS, int kPieces>
__global__ void __launch_bounds__(kThreads, sizeof(TY) == 4 || kPieces == 2 ? 4 : 3)
    k_moe_dispatch_wide(const __grid_constant__ RowArgs a) {
  constexpr int N = 16 / sizeof(TY);        // columns of a piece
  constexpr int kSpan = 32 * kPieces * N;   // columns of a warp
  const int lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (item >= a.items) return;   // whole warps
  const uint32_t token = quotient(item, a.per_row);
  const int col = static_cast<int>(item - token * a.per_row.d) * kSpan;
  const int n = min(a.cols - col, kSpan);   // columns of this warp
  const int32_t* at = a.place + static_cast<int64_t>(token) * a.topk;
  uint32_t next = static_cast<uint32_t>(at[0]);   // a row ahead, and its weight
  float next_w = WEIGHTS ? weight_at(a.w, a.wdt, token * a.w_stride) : 1.f;
  const TX* x = static_cast<const TX*>(a.x.p) + token * a.x.stride + col;
  float v[kPieces][N];
  uint32_t w[kPieces + 1][4];
  Codes<N> c[CODES ? kPieces : 1];
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    load_piece(x, n, j, lane, v[j]);
    if constexpr (CODES) c[j] = encode(v[j]);
    if constexpr (!WEIGHTS) to_words<TY>(v[j], w[j]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) w[kPieces][k] = 0;   // behind the last: never written
  const int edge = edge_column(n, lane);
  const float end = edge >= 0 ? static_cast<float>(x[edge]) : 0.f;
  for (int k = 0; k < a.topk; ++k) {
    const uint32_t row = next;
    const float by = next_w;
    if (k + 1 < a.topk) {
      next = static_cast<uint32_t>(at[k + 1]);
      if constexpr (WEIGHTS) next_w = weight_at(a.w, a.wdt, token * a.w_stride + k + 1);
    }
    if (row >= a.rows) continue;   // the same for all lanes
    if constexpr (WEIGHTS) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        float g[N];
#pragma unroll
        for (int e = 0; e < N; ++e) g[e] = by * v[j][e];
        to_words<TY>(g, w[j]);
      }
    }
    store_pieces<TY, kPieces>(static_cast<TY*>(a.y.p) + row * a.y.stride + col, n, w, edge, by * end, lane);
    if constexpr (CODES) {
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int first = col + (j * 32 + lane) * N;
        if (first / kBlock * kBlock < a.cols) store_codes(a.codes, row, first, c[j]);
      }
    }
  }
}

// out = sum_k w_k y_k (w_k = 1 without weights), added to what it holds if asked.
template <typename TY, typename TO, bool WHOLE, bool WEIGHTS, int kAhead>
__global__ void __launch_bounds__(kThreads) k_moe_combine(const __grid_constant__ RowArgs a) {
  constexpr int N = kCols;
  const Item p = item_of<N>(a);
  float acc[N];
#pragma unroll
  for (int c = 0; c < N; ++c) acc[c] = 0.f;
  const int32_t* at = a.place + static_cast<int64_t>(p.token) * a.topk;
  for (int k0 = 0; k0 < a.topk; k0 += kAhead) {
    Fetched<TY, WHOLE, N> y[kAhead];
    float w[kAhead];
    int n[kAhead];
    // before the rows: behind them they came last (16384 tokens to fp32 369 us, 336 here)
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      w[j] = !WEIGHTS ? 1.f : k0 + j < a.topk ? weight_at(a.w, a.wdt, p.token * a.w_stride + k0 + j) : 0.f;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint32_t row = p.on && k0 + j < a.topk ? static_cast<uint32_t>(at[k0 + j]) : a.rows;
      const bool in = row < a.rows;
      n[j] = in ? p.n : 0;
      fetch(a.y, in ? row : 0, p.col, n[j], y[j]);
      w[j] = in ? w[j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      float v[N];
      values_of(y[j], n[j], v);
#pragma unroll
      for (int c = 0; c < N; ++c) acc[c] = fmaf(w[j], v[c], acc[c]);
    }
  }
  if (a.accumulate) {
    float old[N];
    load_values<TO, WHOLE>(a.x, p.token, p.col, p.n, old);
#pragma unroll
    for (int c = 0; c < N; ++c) acc[c] += old[c];
    if constexpr (!WHOLE) __syncwarp();   // the warp's reads are over
  }
  store_values<TO, WHOLE>(a.x, p.token, p.col, p.n, acc);
}

// The sums over the warp's lanes of v[0 .. N-1]; lane l gets that of v[l / (32 / N)].
// Each step halves the values a lane holds: N + 1 shuffles or so instead of 5 N.
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N], int lane) {
  int bit = 16;
#pragma unroll
  for (int half = N / 2; half >= 1; half >>= 1, bit >>= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int j = 0; j < half; ++j) {
      const float send = up ? v[j] : v[j + half];
      const float keep = up ? v[j + half] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
    }
  }
  float s = v[0];
#pragma unroll
  for (; bit >= 1; bit >>= 1) s += __shfl_xor_sync(0xffffffffu, s, bit);
  return s;
}

// x = dout, y = ys, z = dys.  blockDim.x threads take one token (whole warps, or a
// part of one: SUB) and blockDim.y tokens share a block.  kDots choices are taken in
// a pass over the columns.  Without ROWS only the weights' gradient is formed.
template <typename TY, bool ROWS, int kDots>
constexpr int kBackwardThreads = ROWS ? (kDots > 2 ? 512 : 768) : sizeof(TY) == 2 ? 1024 : 768;   // of an SM

template <typename TX, typename TY, bool WHOLE, bool SUB, bool ROWS, int kDots>
__global__ void __maxnreg__((65536 / kBackwardThreads<TY, ROWS, kDots> / 8 * 8))
    k_moe_combine_backward(const __grid_constant__ RowArgs a) {
  constexpr int kAhead = kDots > 2 && ROWS && sizeof(TY) == 2 ? 4 : 2;   // rows in flight
  constexpr int N = kCols;
  constexpr int kEach = 32 / kDots;                              // lanes that hold one sum
  __shared__ float red[kThreads / 32][kDots];
  const int lane = (threadIdx.y * blockDim.x + threadIdx.x) & 31, warps = blockDim.x >> 5;
  const int first_warp = threadIdx.y * warps, warp = first_warp + (threadIdx.x >> 5);
  const uint32_t t = blockIdx.x * blockDim.y + threadIdx.y;
  const bool on = t < a.tokens;
  const uint32_t token = on ? t : a.tokens - 1;
  const int32_t* at = a.place + static_cast<int64_t>(token) * a.topk;
  const int span = blockDim.x * N, width = a.per_row.d * N;
  for (int k0 = 0; k0 < a.topk; k0 += kDots) {
    float dot[kDots];
#pragma unroll
    for (int j = 0; j < kDots; ++j) dot[j] = 0.f;
    for (int c0 = 0; c0 < width; c0 += span) {   // the same number of times for all threads
      const int col = c0 + threadIdx.x * N;
      const int n = on ? a.cols - col : 0;
      float d[N];
      Fetched<TX, WHOLE, N> d_raw;
      if constexpr (ROWS) fetch(a.x, token, col, n, d_raw);   // on its way beside the rows
      else load_values<TX, WHOLE>(a.x, token, col, n, d);     // (too many registers)
#pragma unroll
      for (int j0 = 0; j0 < kDots; j0 += kAhead) {
        if (k0 + j0 >= a.topk) break;   // the same for all threads
        Fetched<TY, WHOLE, N> y[kAhead];
        uint32_t row[kAhead];
        float w[kAhead];
        if constexpr (ROWS) {   // all that is read is asked for before any of it is looked at:
                                // 16384 tokens, 8 rows of 7168 bf16 639 -> 602 us
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            w[j] = k0 + j0 + j < a.topk ? weight_at(a.w, a.wdt, token * a.w_stride + k0 + j0 + j) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int k = k0 + j0 + j;
          row[j] = on && k < a.topk ? static_cast<uint32_t>(at[k]) : a.rows;
          const bool in = row[j] < a.rows;
          fetch(a.y, in ? row[j] : 0, col, in ? n : 0, y[j]);
        }
        if constexpr (ROWS) {
          if (j0 == 0) values_of(d_raw, n, d);
        }
        if constexpr (ROWS) {
          // dys needs nothing of ys: written while that is on its way.  It may be ys, so the
          // reads come first: the warp's, or (WHOLE) the thread's own, which the compiler
          // must not move a plain store in front of (fetch does not tell it what it reads)
          if constexpr (!WHOLE) __syncwarp();
          else asm volatile("" ::: "memory");
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            const bool in = row[j] < a.rows;
            float g[N];
#pragma unroll
            for (int c = 0; c < N; ++c) g[c] = w[j] * d[c];
            store_values<TY, WHOLE>(a.z, in ? row[j] : 0, col, in ? n : 0, g);
          }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          float v[N];
          values_of(y[j], n, v);   // all 0 for a copy without a row
#pragma unroll
          for (int c = 0; c < N; ++c) dot[j0 + j] = fmaf(d[c], v[c], dot[j0 + j]);
        }
      }
    }
    const auto write = [&](int k, float s) {
      if (!on || k >= a.topk) return;
      const float v = static_cast<uint32_t>(at[k]) < a.rows ? s : 0.f;
      const int64_t i = token * a.dw_stride + k;
      if (a.wdt == MUON_BF16)
        static_cast<__nv_bfloat16*>(a.dw)[i] = __float2bfloat16_rn(v);
      else
        static_cast<float*>(a.dw)[i] = v;
    };
    if constexpr (SUB) {
      for (int bit = blockDim.x >> 1; bit > 0; bit >>= 1)
#pragma unroll
        for (int j = 0; j < kDots; ++j) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], bit);
      if (threadIdx.x == 0) {
#pragma unroll
        for (int j = 0; j < kDots; ++j) write(k0 + j, dot[j]);
      }
    } else {
      float s = warp_sums(dot, lane);
      if (warps > 1) {
        if (lane % kEach == 0) red[warp][lane / kEach] = s;
        __syncthreads();
        s = 0.f;
        for (int v = 0; v < warps; ++v) s += red[first_warp + v][lane / kEach];
        if (k0 + kDots < a.topk) __syncthreads();
      }
      if (threadIdx.x < 32 && lane % kEach == 0) write(k0 + lane / kEach, s);
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

// Whether one of `runs` runs of `bytes` bytes, each `step` (>= bytes) behind the one before,
// holds a byte of [q, q + size).
bool runs_overlap(const void* p, int64_t runs, uint64_t bytes, uint64_t step, const void* q, uint64_t size) {
  const uint64_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  if (runs <= 0 || size == 0 || a >= b + size) return false;
  uint64_t last = (b + size - 1 - a) / step;   // of the runs that begin in front of the end
  if (last >= static_cast<uint64_t>(runs)) last = static_cast<uint64_t>(runs) - 1;
  return a + last * step + bytes > b;
}

// Whether the choices or the mask share memory with what the sort writes: its second kernel
// reads the choices again while other blocks write, and so does the first the mask.
bool sort_overlaps(const void* chosen, int bytes, int64_t stride, const uint8_t* mask, const muon_routing_t& r) {
  const uint64_t apart = static_cast<uint64_t>(stride < (int64_t{1} << 48) ? stride : int64_t{1} << 48) * bytes;
  const uint64_t row = static_cast<uint64_t>(r.topk) * bytes;
  const auto with = [&](const void* q, int64_t n) {
    const uint64_t size = static_cast<uint64_t>(n) * 4;
    return runs_overlap(chosen, r.tokens, row, apart, q, size) ||
           (mask != nullptr && runs_overlap(mask, r.tokens, 1, 1, q, size));
  };
  return with(r.offsets, r.experts + 1) || with(r.order, r.rows) || with(r.place, r.tokens * r.topk);
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
  return MUON_OK;
}

template <bool ALONE, int PER>
cudaError_t run_sort(const SortArgs& a, double bytes, cudaStream_t st) {
  const size_t smem = rank_smem(a.experts);
  if (smem > 48 * 1024) {   // per device, so with every call that needs it
    const cudaError_t e =
        cudaFuncSetAttribute(k_moe_rank<ALONE, PER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(rank_smem(kMaxExperts)));
    if (e != cudaSuccess) return e;
  }
  prof_begin(kKindMoe, st);
  k_moe_rank<ALONE, PER><<<a.blocks, kSortThreads, smem, st>>>(a);
  prof_end(kKindMoe, st, 0.0, bytes);
  const cudaError_t e = cudaGetLastError();
  if (ALONE || e != cudaSuccess) return e;
  // a programmatic dependent of the kernel before (it waits for the ranks)
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(a.blocks);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = place_smem(a.experts);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  prof_begin(kKindMoe, st);
  const cudaError_t p = cudaLaunchKernelEx(&cfg, k_moe_place<PER>, a);
  prof_end(kKindMoe, st, 0.0, 0.0);
  return p;
}

// `launch` for every token, `cols` columns an item, in pieces of fewer than 2^30 items.
template <class F>
muon_status_t by_tokens(RowArgs a, int64_t tokens, int xdt, int cols, F launch) {
  // (whole blocks of a checkpoint: 16 columns divide 32, and 32 a warp's)
  const int64_t padded = blocks_of(a.cols) * kBlock;
  a.per_row = divider(static_cast<uint32_t>((padded + cols - 1) / cols));
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

// Columns of an item of the dispatch: a warp's where rows start anywhere and hold a warp's
// pieces, else a thread's.  (65536 tokens, 8 rows each: 257 columns of bf16 80 us by
// warps, 97 by threads; 801 155 and 236; 129 of fp32 64 and 128.)  A lane takes two
// pieces where that is the whole row, else four (257 columns of bf16 62 us with two, 77
// with four; 257 of fp32, a column more than two hold, 120 and 101).
int dispatch_cols(int xsdt, bool whole, int width) {
  const int warp = 32 * 16 / esize(xsdt);
  return whole || width < warp ? kCols : width <= 2 * warp ? 2 * warp : 4 * warp;
}

template <typename TX, typename TY, bool CODES, bool WEIGHTS>
void launch_dispatch_wide(const RowArgs& a, int cols, cudaStream_t st) {
  const unsigned grid = (a.items + kThreads / 32 - 1) / (kThreads / 32);
  if (cols == 2 * 32 * 16 / static_cast<int>(sizeof(TY)))
    k_moe_dispatch_wide<TX, TY, CODES, WEIGHTS, 2><<<grid, kThreads, 0, st>>>(a);
  else
    k_moe_dispatch_wide<TX, TY, CODES, WEIGHTS, 4><<<grid, kThreads, 0, st>>>(a);
}

template <typename TX, typename TY>
void launch_dispatch(const RowArgs& a, bool whole, bool codes, int cols, cudaStream_t st) {
  if (cols > kCols) {
    if (codes) launch_dispatch_wide<TX, TY, true, false>(a, cols, st);
    else launch_dispatch_wide<TX, TY, false, false>(a, cols, st);
    return;
  }
  const unsigned grid = grid_of(a);
  if (whole && codes) k_moe_dispatch<TX, TY, true, true><<<grid, kThreads, 0, st>>>(a);
  else if (whole) k_moe_dispatch<TX, TY, true, false><<<grid, kThreads, 0, st>>>(a);
  else if (codes) k_moe_dispatch<TX, TY, false, true><<<grid, kThreads, 0, st>>>(a);
  else k_moe_dispatch<TX, TY, false, false><<<grid, kThreads, 0, st>>>(a);
}

// Rows in flight: four of bf16 on 32-byte boundaries, else two, so that more blocks fit
// (8 rows of 7001 bf16, 16384 tokens: 343 us with two, 430 with four; 2 rows of 4096 68
// and 84).
template <typename TY, typename TO, int AHEAD>
void launch_combine_ahead(const RowArgs& a, bool whole, cudaStream_t st) {
  const unsigned grid = grid_of(a);
  const bool weights = a.w != nullptr;
  if (whole && weights) k_moe_combine<TY, TO, true, true, AHEAD><<<grid, kThreads, 0, st>>>(a);
  else if (whole) k_moe_combine<TY, TO, true, false, AHEAD><<<grid, kThreads, 0, st>>>(a);
  else if (weights) k_moe_combine<TY, TO, false, true, 2><<<grid, kThreads, 0, st>>>(a);
  else k_moe_combine<TY, TO, false, false, 2><<<grid, kThreads, 0, st>>>(a);
}

template <typename TY, typename TO>
void launch_combine(const RowArgs& a, bool whole, cudaStream_t st) {
  if constexpr (sizeof(TY) == 2) {
    if (a.topk > 2 && whole) return launch_combine_ahead<TY, TO, 4>(a, whole, st);
  }
  launch_combine_ahead<TY, TO, 2>(a, whole, st);
}

// Threads of a token: up to 256, as many as make the passes over its columns
// equally long; narrow tokens share a block and, below a warp's columns, a warp.
template <typename TX, typename TY, int DOTS>
void launch_combine_backward_of(const RowArgs& a, bool whole, bool rows, cudaStream_t st) {
  const unsigned items = a.per_row.d;
  unsigned threads = 2;
  while (threads < items && threads < 32) threads *= 2;
  if (items > 32) {
    const unsigned passes = (items + kThreads - 1) / kThreads;
    threads = ((items + passes - 1) / passes + 31) / 32 * 32;
  }
  // as many tokens a block as fill an SM's threads best (6 rows of 1472 bf16, 96 threads a
  // token, in a graph: 4752 tokens 40 us with one a block, 45 with two; 19008 142 and 166)
  const unsigned most = rows ? kBackwardThreads<TY, true, DOTS> : kBackwardThreads<TY, false, DOTS>;
  unsigned tokens = kThreads / threads;
  for (unsigned n = tokens; n > 0; --n)
    if (most / (n * threads) * n > most / (tokens * threads) * tokens) tokens = n;
  const dim3 block(threads, tokens);   // a token's threads are lanes side by side
  const unsigned grid = (a.tokens + tokens - 1) / tokens;
  const bool sub = threads < 32;
  if (whole && sub) k_moe_combine_backward<TX, TY, true, true, true, DOTS><<<grid, block, 0, st>>>(a);
  else if (whole) k_moe_combine_backward<TX, TY, true, false, true, DOTS><<<grid, block, 0, st>>>(a);
  else if (rows && sub) k_moe_combine_backward<TX, TY, false, true, true, DOTS><<<grid, block, 0, st>>>(a);
  else if (rows) k_moe_combine_backward<TX, TY, false, false, true, DOTS><<<grid, block, 0, st>>>(a);
  else if (sub) k_moe_combine_backward<TX, TY, false, true, false, DOTS><<<grid, block, 0, st>>>(a);
  else k_moe_combine_backward<TX, TY, false, false, false, DOTS><<<grid, block, 0, st>>>(a);
}

// Rows that start anywhere and hold a warp's pieces are written by the dispatch, after
// the weights' gradient has read ys (which may be dys): one more read of dout, and 8
// rows of 7001 bf16 columns, 16384 tokens, take 682 us
// for 889 (8192 tokens, fp32: 662 for 748).  Up to kOneKernelBytes of rows the second launch
// costs more than that: 64 tokens, 6 rows of 1111 fp32 12.4 us in two, 7.5 in one, 1023
// tokens, 6 of 1111 bf16 (14 MB) 16.5 and 14.5; 27 MB 20.7 and 20.9, 43 MB 26.8 and 33.7.
// In a graph, in two and in one, at 8, 16, 32 and 64 MB of rows:
//   2 rows of 1111 bf16   9.1  8.8   18.0 16.4   30.6 30.2   59.1 56.2
//   2 of 4099 bf16        8.9  8.4   16.6 16.0   25.8 27.3   47.8 48.6
//   2 of 1111 fp32        7.8  8.2   15.3 17.4   23.4 27.4   43.5 51.4
//   8 of 257 bf16        10.6  9.5   18.6 18.0   30.0 32.9   51.7 59.4
//   8 of 1111 fp32       10.7  8.2   14.5  9.9   20.4 21.9   36.3 34.7
// so the border is about the same however few the choices are; fp32 with one or two would
// take two kernels from 8 MB on.
constexpr double kOneKernelBytes = 16e6;

template <typename TX, typename TY>
void launch_combine_backward(const RowArgs& a, bool whole, cudaStream_t st) {
  const int cols = dispatch_cols(sizeof(TY) == 2 ? MUON_BF16 : MUON_F32, whole, a.cols);
  const double tokens = static_cast<double>(a.tokens) * a.cols, row = sizeof(TY) * static_cast<double>(a.topk);
  const bool rows = whole || cols == kCols || tokens * row <= kOneKernelBytes;   // by the same kernel
  prof_begin(kKindMoe, st);
  if (a.topk <= 2) launch_combine_backward_of<TX, TY, 2>(a, whole, rows, st);
  else launch_combine_backward_of<TX, TY, 8>(a, whole, rows, st);
  prof_end(kKindMoe, st, 0.0, tokens * (sizeof(TX) + (rows ? 2 : 1) * row));
  if (rows) return;
  prof_begin(kKindMoe, st);
  RowArgs b = a;
  b.y = a.z;
  b.per_row = divider(static_cast<uint32_t>((a.cols + cols - 1) / cols));
  b.items = a.tokens * b.per_row.d;
  launch_dispatch_wide<TX, TY, false, true>(b, cols, st);
  prof_end(kKindMoe, st, 0.0, tokens * row);
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
  return by_tokens(a, r->tokens, odt, kCols, [&](const RowArgs& b) {
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
           static_cast<size_t>(p.blocks) * round_up(experts, 4) * 4;
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
  if (sort_overlaps(chosen, chosen_bytes, chosen_stride, token_mask, *r)) return MUON_ERR_INVALID_ARG;
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
  while (4 << a.quad_bits < r->experts) ++a.quad_bits;
  a.dense = chosen_stride == r->topk;
  a.stride = static_cast<int>(round_up(r->experts, 4));
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
  const bool alone = plan.blocks == 1;
  cudaError_t e;
  if (plan.per == 1) e = alone ? run_sort<true, 1>(a, bytes, st) : run_sort<false, 1>(a, bytes, st);
  else if (plan.per == 2) e = alone ? run_sort<true, 2>(a, bytes, st) : run_sort<false, 2>(a, bytes, st);
  else e = run_sort<false, 8>(a, bytes, st);
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
  const int cols = dispatch_cols(xsdt, whole, width);
  return by_tokens(a, r->tokens, xdt, cols, [&](const RowArgs& b) {
    prof_begin(kKindMoe, st);
    by_types(xdt, xsdt, [&](auto tx, auto ty) {
      launch_dispatch<decltype(tx), decltype(ty)>(b, whole, x8 != nullptr, cols, st);
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
  if (dys == ys && r->rows > 1 && dys_stride != y_stride) return MUON_ERR_INVALID_ARG;
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
  return by_tokens(a, r->tokens, ddt, kCols, [&](const RowArgs& b) {
    by_types(ddt, ydt, [&](auto tx, auto ty) {
      launch_combine_backward<decltype(tx), decltype(ty)>(b, whole, st);
    });
  });
}

}  // extern "C"
