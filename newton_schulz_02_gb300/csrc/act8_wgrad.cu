// Weight gradients of a set of experts from 8-bit activation checkpoints
// (muon_act8_weight_grad):
//
//   G_e[o][i] = sum_{t in expert e} dy[t][o] * code[t][i] * 2^(e[t][i/32])
//
// A code's value has at most 7 significant bits, so it is exact in bf16 and
// the product runs on the bf16 tensor cores without losing anything of x:
// dy^T (MN-major A) and x (MN-major B), contracted over the tokens, fp32
// accumulators in tensor memory.
//
// k_wgrad: a CTA pair computes 256 x 256 of G (tcgen05 cta_group::2; each CTA
// holds 128 output columns of dy and 128 input columns of x).  Per 64 tokens
// the dy tile, the codes and the exponents come by TMA; groups of four warps
// turn the codes into the swizzled bf16 operand (2.25 operations a code); one
// thread of the pair issues the MMAs; eight warps drain the accumulators, of
// which there are two, while the next tile runs.  The ranges of tokens are
// ragged: rows of the last block that belong to the next expert are zeroed in
// both operands (a zero times their NaN would be NaN).
//
// Where TMA cannot fetch dy (rows off 16-byte boundaries, fp32), k_wgrad_dy
// writes it to the workspace first, on such boundaries.  An fp32 value becomes
// three bf16 of 8 bits each, whose sum it is, and the MMA runs once for each:
// products stay exact.
//
// Few tiles and many tokens: the tokens of a tile are cut into slices that
// leave fp32 partial sums in the workspace, which k_wgrad_join adds in order.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>

#include "internal.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace muon {
namespace {

constexpr size_t kHeader = 256;   // status word

// Where sums go: G itself, or slices of partial sums.
struct Matrices {
  void* const* ptrs;      // device pointers, or nullptr: base + e * batch_stride
  void* base;
  int64_t batch_stride, stride;
  int rows, cols;         // of a matrix
  int dtype, accumulate;
};

struct WgradArgs {
  int rows, out, in, experts;
  const int32_t* offsets;
  Matrices g;
  int tiles_o, tiles_i;   // 256 x 256 tiles of a matrix
  int slices;             // of a tile's tokens; slice s of expert e goes to matrix s * experts + e
  int cut;                // sums are cut into chunks, one after the other, added up in G
  int units;              // tiles x slices of all experts
  uint32_t* status;
  uint64_t timeout_ns;
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

// ---- 256 x 256 tiles on CTA pairs -------------------------------------------
constexpr int kBK = 64;                          // tokens per block of the contraction
constexpr int kConvWarps = 4, kEpiWarps = 8;     // converter warps of one group
constexpr uint32_t kDyBytes = kBK * 128 * 2;     // a plane: two 64-column atoms of 128-byte rows
constexpr uint32_t kCodeBytes = kBK * 128;
constexpr uint32_t kExpBytes = kBK * 16;         // 16 blocks' bytes a row, four of them used
constexpr uint32_t kAtomBytes = kBK * 128;       // 64 columns x kBK rows
constexpr uint32_t kSlotBytes = 2 * kAtomBytes;
constexpr int kUnits = 16;                       // units announced at a time, two batches ahead

// PLANES: of dy.  Six dy stages and four decoded blocks cover the latency of a
// load (about 1 us under load, a block's MMAs take 0.3); with three planes a
// block's MMAs take three times as long, and three and two do.
template <int PLANES>
struct Cfg {
  static constexpr int kDyStages = PLANES == 1 ? 6 : 3;   // dy tiles in flight or in use
  static constexpr int kSlots = PLANES == 1 ? 4 : 2;      // decoded blocks, a converter group each
  static constexpr int kConv0 = 4, kEpi0 = kConv0 + kSlots * kConvWarps;   // first warps
  static constexpr int kThreads = 32 * (kEpi0 + kEpiWarps);
  static constexpr uint32_t kStageBytes = PLANES * kDyBytes;   // 64 columns of every plane, 64 more

  // What the roles of a CTA share besides the operands.  An mbarrier's parity
  // tells only the current phase from the one before, so every role that waits
  // for phase f of a barrier has seen phase f - 1 end: it waited for it itself,
  // or for something that came after.  A converter group waits for every phase
  // of its code stage (as many stages as groups); block c - kDyStages is over
  // when the MMAs of block c - kSlots are (at least as many dy stages as slots).
  struct Shared {
    uint64_t dy_full[kDyStages], dy_empty[kDyStages];     // loads landed; MMAs on the stage done
    uint64_t code_full[kSlots], code_empty[kSlots];       // loads landed; read into registers
    uint64_t ready[kSlots];                               // both operands of a block in place, in both CTAs
    uint64_t unit_full[2], unit_empty[2];                 // a batch of units announced; taken
    uint64_t tfull[2], tempty[2];                         // accumulator summed; drained
    uint64_t drain;
    uint32_t tmem_slot;
    int abort;
    uint32_t notes[kSlots][kConvWarps];                   // what the odd CTA's notices store; not read
    alignas(16) int units[2 * kUnits][8];
  };
  static constexpr size_t kSmem = kDyStages * kStageBytes +
                                  kSlots * (kSlotBytes + kCodeBytes + kExpBytes) +
                                  sizeof(Shared) + 1024;
};
static_assert(Cfg<1>::kThreads == 896, "see the register split");
static_assert(Cfg<1>::kSmem <= 232448 && Cfg<3>::kSmem <= 232448, "");

constexpr uint32_t kTmemCols = 512;              // two accumulators of 256 columns
// D fp32, A and B bf16, both MN-major, M = 256, N = 256
constexpr uint32_t kIdesc = idesc_bf16_f32(256, 256, true) | (1u << 15);
constexpr int kGroupO = 8;                       // tiles walked down before the next column

// Unit u of the walk: expert (-1: no more), the tile's first row and column,
// the expert's tokens.  Within an expert, columns of kGroupO tiles are walked
// side by side, so that the tiles in flight share operands in L2.
struct Unit {
  int e, o0, i0, begin, n;
  int m;     // matrix the sums go to
  int add;   // to what earlier chunks left there
};

__device__ __forceinline__ Unit unit_of(const WgradArgs& a, int u) {
  const int slice = u % a.slices;
  u /= a.slices;
  const int per = a.tiles_o * a.tiles_i;
  Unit t;
  t.e = u / per;
  const int r = u - t.e * per;
  const int band = r / (kGroupO * a.tiles_i);
  const int rows = min(kGroupO, a.tiles_o - band * kGroupO);
  const int q = r - band * kGroupO * a.tiles_i;
  t.o0 = (band * kGroupO + q % rows) * 256;
  t.i0 = (q / rows) * 256;
  span_of(a, t.e, t.begin, t.n);
  t.m = slice * a.experts + t.e;
  t.add = 0;
  if (a.slices > 1) {   // whole blocks, as even as can be
    const int blocks = (t.n + kBK - 1) / kBK;
    const int b0 = static_cast<int>(static_cast<int64_t>(blocks) * slice / a.slices);
    const int b1 = static_cast<int>(static_cast<int64_t>(blocks) * (slice + 1) / a.slices);
    t.n = min(t.n, b1 * kBK) - b0 * kBK;
    t.begin += b0 * kBK;
  }
  return t;
}

// Tokens of a chunk of a unit of n tokens whose sums are kept in fp32.  The tensor
// core's additions truncate, and the error grows with their number (6e-6 of the
// result for 384); so after 32 blocks (128 additions) at most the accumulator is
// drained and added, with rounding, to what G holds, which the same pair finds in
// L2.  The drain runs beside the next chunk.  A matter of each unit's own tokens, as
// one expert may have most of them (16000 of 16384 on one of 64: 1.9e-5 in one
// piece, 2.4e-6 cut).  Units of 17 to 32 blocks are cut in two where the drain does
// run beside the next one (one plane): fp32 sums of so few products are themselves
// good to 5e-7.  (14336 x 4096 over 8192 tokens: 665 us with fp32 G; bf16
// G, in one piece, 640.)
template <int PLANES>
__device__ __forceinline__ int chunk_of(const WgradArgs& a, int n) {
  const int blocks = (n + kBK - 1) / kBK;
  int chunks = 1;
  if (a.cut) chunks = blocks > 32 ? (blocks + 31) / 32 : blocks > 16 && PLANES == 1 ? 2 : 1;
  return max((blocks + chunks - 1) / chunks, 1) * kBK;
}

__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred P1;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 P1, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, P1;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// mbar_wait_bounded for a barrier that the pair's other CTA arrives on too
// (acquire at cluster scope); the timer is read only when the wait is not
// over at once.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort,
                                             uint32_t* status, uint64_t timeout_ns) {
  const uint32_t a = smem_u32(bar);
  if (try_wait_cluster(a, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (try_wait_cluster(a, parity)) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > timeout_ns) {
      *abort = 1;
      atomicOr(status, kFlagTimeout);
      return false;
    }
  }
}

// Waits for what is still in flight when a role ends, whatever became of the others.
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity, uint32_t* status,
                                           uint64_t timeout_ns) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(a, parity))
    if (global_timer_ns() - t0 > timeout_ns) {
      atomicOr(status, kFlagTimeout);
      return;
    }
}

__device__ __forceinline__ void tma_load_2d(void* dst, const void* map, uint64_t* bar, int32_t x,
                                            int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

// Codes 0 and 2 of the four int8 in p as a pair of bf16 (with p >> 8: codes 1
// and 3).  0x4300 is 128 in bf16 and its 7 mantissa bits count units, so
// 0x4300 | (c & 127) is 128 + (c & 127); what is subtracted is 128 for c >= 0
// and 256 for c < 0, which 0x4300 | (c & 128) spells.  Every step is exact.
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t p, __nv_bfloat162 scale) {
  const uint32_t hi = (p & 0x007F007Fu) | 0x43004300u;
  const uint32_t lo = (p & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 v = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&hi),
                                           *reinterpret_cast<const __nv_bfloat162*>(&lo)),
                                   scale);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 16 lanes x 64 fp32 columns: registers 4b .. 4b+3 of lane l hold columns 8b +
// 2 (l % 4) + {0, 1} of tensor-memory lane l / 4, then of lane l / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// The same of 32 columns, 16 registers.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 rows x 64 columns of an accumulator as fp32 bits (two accumulators' sum
// with three planes): registers 4b + 2h + k of lane l are row l / 4 + 8h,
// position 8b + 2 (l % 4) + k.
template <int PLANES>
__device__ __forceinline__ void load_piece(uint32_t at, uint32_t (&raw)[32]) {
  tmem_ld_16x256b_x8(at, raw);
  tmem_ld_wait(raw);
  if constexpr (PLANES > 1) {
#pragma unroll
    for (int b = 0; b < 32; b += 16) {
      uint32_t rest[16];
      tmem_ld_16x256b_x4(at + 256u + 2 * b, rest);
      tmem_ld_wait();
      tmem_ld_tie(rest);
#pragma unroll
      for (int k = 0; k < 16; ++k)
        raw[b + k] = __float_as_uint(__uint_as_float(raw[b + k]) + __uint_as_float(rest[k]));
    }
  }
}

// Register of column c (0..15) of row l / 4 + 8h (see the order of the operand's columns).
__host__ __device__ constexpr int reg_of(int h, int c) {
  return 4 * (2 * (c >> 2) + (c & 1)) + 2 * h + ((c >> 1) & 1);
}

// 32 bytes of G: a whole sector in one access (rows on 32-byte boundaries), or
// two of 16.
template <bool SECTOR>
__device__ __forceinline__ void load32(const char* p, uint4& x, uint4& y) {
  if constexpr (SECTOR) {
    ld_global_v8(p, x, y);
  } else {
    x = reinterpret_cast<const uint4*>(p)[0];
    y = reinterpret_cast<const uint4*>(p)[1];
  }
}

template <bool SECTOR>
__device__ __forceinline__ void store32(char* p, const uint4& x, const uint4& y) {
  if constexpr (SECTOR) {
    st_global_v8(p, x, y);
  } else {
    reinterpret_cast<uint4*>(p)[0] = x;
    reinterpret_cast<uint4*>(p)[1] = y;
  }
}

// 32 rows x 128 columns of G that lie inside the matrix, rows on 16-byte
// boundaries.  p: this lane's 16 columns of row l / 4.  Not unrolled: the roles
// share the instruction caches, and 1510 against 1310 us is what the unrolled
// form costs 256 experts of 16 tokens.
template <int PLANES, bool F32, bool ADD, bool SECTOR>
__device__ __forceinline__ void drain_whole(uint32_t src, char* p, int64_t row_bytes) {
#pragma unroll 1
  for (int dc = 0; dc < 128; dc += 64) {
#pragma unroll 1
    for (int dr = 0; dr < 32; dr += 16) {
      uint32_t raw[32];
      load_piece<PLANES>(src + (static_cast<uint32_t>(dr) << 16) + dc, raw);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        char* at = p + (h * 8 + dr) * row_bytes + dc * (F32 ? 4 : 2);
        if constexpr (F32) {
#pragma unroll
          for (int c = 0; c < 16; c += 8) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = raw[reg_of(h, c + k)];
            if constexpr (ADD) {
              uint4 x, y;
              load32<SECTOR>(at + 4 * c, x, y);
              const uint32_t old[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
              for (int k = 0; k < 8; ++k)
                w[k] = __float_as_uint(__uint_as_float(w[k]) + __uint_as_float(old[k]));
            }
            store32<SECTOR>(at + 4 * c, make_uint4(w[0], w[1], w[2], w[3]),
                            make_uint4(w[4], w[5], w[6], w[7]));
          }
        } else {
          uint32_t w[8];
          uint32_t old[8];
          if constexpr (ADD) {
            uint4 x, y;
            load32<SECTOR>(at, x, y);
            old[0] = x.x; old[1] = x.y; old[2] = x.z; old[3] = x.w;
            old[4] = y.x; old[5] = y.y; old[6] = y.z; old[7] = y.w;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float lo = __uint_as_float(raw[reg_of(h, 2 * k)]);
            float hi = __uint_as_float(raw[reg_of(h, 2 * k + 1)]);
            if constexpr (ADD) {
              lo += __uint_as_float(old[k] << 16);
              hi += __uint_as_float(old[k] & 0xFFFF0000u);
            }
            w[k] = pack2(lo, hi);
          }
          store32<SECTOR>(at, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
        }
      }
    }
  }
}

// The same of an expert without tokens, and the choice among the forms.
template <int PLANES, bool SECTOR>
__device__ __forceinline__ void drain_inside(uint32_t src, const Matrices& g, char* p, int64_t row_bytes,
                                             bool empty, bool add) {
  const bool f32 = g.dtype == MUON_F32;
  if (empty) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 1
    for (int r = 0; r < 32; r += 8, p += 8 * row_bytes)
#pragma unroll 1
      for (int c = 0; c < (f32 ? 512 : 256); c += f32 ? 256 : 128) {
        store32<SECTOR>(p + c, zero, zero);
        if (f32) store32<SECTOR>(p + c + 32, zero, zero);
      }
  } else if (f32) {
    if (add)
      drain_whole<PLANES, true, true, SECTOR>(src, p, row_bytes);
    else
      drain_whole<PLANES, true, false, SECTOR>(src, p, row_bytes);
  } else {
    if (add)
      drain_whole<PLANES, false, true, SECTOR>(src, p, row_bytes);
    else
      drain_whole<PLANES, false, false, SECTOR>(src, p, row_bytes);
  }
}

// The same for any tile: 32 rows x 128 columns of which some may lie outside the
// matrix, rows at any alignment.  g: the first element; rows, cols: of the matrix
// from there on; empty: all zeros.  The four threads of a row write the 16-byte
// pieces of its 64 columns.  (Element by element, 32 consecutive columns of one
// row at a time, 16 experts of 50 tokens, 6755 x 3757, took 990 us.)
template <int PLANES, typename T, bool ADD>
__device__ __forceinline__ void drain_pieces(uint32_t src, T* g, int64_t stride, int rows, int cols,
                                             bool empty) {
  const int lane = threadIdx.x & 31, mine = 16 * (lane & 3);
#pragma unroll 1
  for (int dc = 0; dc < 128 && dc < cols; dc += 64) {   // the whole warp
#pragma unroll 1
    for (int dr = 0; dr < 32 && dr < rows; dr += 16) {
      uint32_t raw[32];
      __syncwarp();   // tcgen05.ld takes the warp together
      if (empty) {
#pragma unroll
        for (int k = 0; k < 32; ++k) raw[k] = 0u;
      } else {
        load_piece<PLANES>(src + (static_cast<uint32_t>(dr) << 16) + dc, raw);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = dr + 8 * h + (lane >> 2);
        const int n = row < rows ? cols - dc - mine : 0;
        T* p = g + row * stride + dc + mine;
        float x[kCols];
#pragma unroll
        for (int k = 0; k < kCols; ++k) x[k] = __uint_as_float(raw[reg_of(h, k)]);
        if constexpr (ADD) {
          float old[kCols];
          load_shifted(p, n, old);
#pragma unroll
          for (int k = 0; k < kCols; ++k) x[k] += old[k];
          __syncwarp();   // a piece holds columns of two threads: reads before writes
        }
        store_shifted(p, n, mine > 0, mine < 48 ? min(max(n - kCols, 0), kCols) : 0, x);
      }
    }
  }
}

template <int PLANES>
__device__ __noinline__ void drain_any(uint32_t src, void* g, int64_t stride, int rows, int cols, bool f32,
                                       bool empty, bool add) {
  if (f32) {
    if (add)
      drain_pieces<PLANES, float, true>(src, static_cast<float*>(g), stride, rows, cols, empty);
    else
      drain_pieces<PLANES, float, false>(src, static_cast<float*>(g), stride, rows, cols, empty);
  } else {
    if (add)
      drain_pieces<PLANES, __nv_bfloat16, true>(src, static_cast<__nv_bfloat16*>(g), stride, rows, cols, empty);
    else
      drain_pieces<PLANES, __nv_bfloat16, false>(src, static_cast<__nv_bfloat16*>(g), stride, rows, cols, empty);
  }
}

__device__ __forceinline__ char* matrix_of(const Matrices& g, int m) {
  return static_cast<char*>(g.ptrs != nullptr
                                ? g.ptrs[m]
                                : static_cast<char*>(g.base) +
                                      m * g.batch_stride * (g.dtype == MUON_F32 ? 4 : 2));
}

// 32 rows from o, 128 columns from i of the matrix at g.  p: this lane's first 16
// columns.  PLANES > 1: both accumulators' sum.
template <int PLANES, bool EDGE>
__device__ __forceinline__ void drain_unit(uint32_t src, const Matrices& m, char* g, char* p, int64_t row_bytes,
                                           int o, int i, bool empty, bool add) {
  const uint64_t bits = reinterpret_cast<uintptr_t>(g) | static_cast<uint64_t>(row_bytes);
  const bool inside = o + 32 <= m.rows && i + 128 <= m.cols;
  const int esz = m.dtype == MUON_F32 ? 4 : 2;
  if (inside && bits % 32 == 0)
    drain_inside<PLANES, true>(src, m, p, row_bytes, empty, add);
  else if (inside && (!EDGE || bits % 16 == 0))
    drain_inside<PLANES, false>(src, m, p, row_bytes, empty, add);
  else if constexpr (EDGE)
    drain_any<PLANES>(src, g + o * row_bytes + static_cast<int64_t>(i) * esz, m.stride, m.rows - o, m.cols - i,
                      m.dtype == MUON_F32, empty, add);
}

// dy [rows][out] as planes of bf16 [rows][pitch] at `to`, `plane` values apart
// (pitch: out rounded up to 16; columns past out are 0).  bf16: one plane, the
// values themselves.  fp32: three, the upper 8 significant bits, the next 8 and
// the last 8, whose sum is the value; an infinity or a NaN is the first alone.
// 16 columns a thread; bound by HBM.  Clears the call's status word too, before
// k_wgrad may start.  (Loading, splitting and shifting dy in k_wgrad instead, by
// eight warps of its own, cost more than this pass: 16384 tokens, 256 x 7168
// fp32 158 us against 127; 8192 tokens, 4097 x 4096 bf16 417 against 215.)
template <typename T>
__global__ void __launch_bounds__(256)
    k_wgrad_dy(const T* dy, int64_t stride, int64_t items, int out, __nv_bfloat16* to, int pitch, int64_t plane,
               uint32_t* status) {
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *status = 0;
    __threadfence();
  }
  griddep_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= items) return;
  const uint32_t per = static_cast<uint32_t>(pitch) / kCols;   // items of a row
  const int64_t row = items >> 32 == 0 ? static_cast<uint32_t>(i) / per : i / per;
  const int col = static_cast<int>(i - row * per) * kCols;
  float x[kCols];
  load_shifted(dy + row * stride + col, out - col, x);
  __nv_bfloat16* p = to + row * pitch + col;
  const auto store = [](__nv_bfloat16* q, const uint32_t (&w)[8]) {
    st_global_v8(q, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
  };
  uint32_t w[8];
  if constexpr (sizeof(T) == 2) {
    to_words<T>(x, w);
    store(p, w);
  } else {
    uint32_t u[3][kCols];
#pragma unroll
    for (int k = 0; k < kCols; ++k) {
      const uint32_t b = __float_as_uint(x[k]);
      const float r = x[k] - __uint_as_float(b & 0xFFFF0000u);
      u[0][k] = b;
      u[1][k] = __float_as_uint(r);
      u[2][k] = __float_as_uint(r - __uint_as_float(u[1][k] & 0xFFFF0000u));
      if ((b & 0x7F800000u) == 0x7F800000u) {
        if ((b & 0x007FFFFFu) != 0) u[0][k] = 0x7FC00000u;
        u[1][k] = u[2][k] = 0u;
      }
    }
#pragma unroll
    for (int z = 0; z < 3; ++z) {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = __byte_perm(u[z][2 * k], u[z][2 * k + 1], 0x7632);
      store(p + z * plane, w);
    }
  }
}

// EDGE: some 32 x 128 piece of G may lie partly outside it, or off 16-byte
// boundaries.  (A kernel of its own, as the call that drains such a piece costs
// the other one registers: 469 against 438 us for 64 experts of 256 tokens.)
template <int PLANES, bool EDGE>
__global__ void __launch_bounds__(Cfg<PLANES>::kThreads, 1)
    k_wgrad(const __grid_constant__ CUtensorMap tm_dy, const __grid_constant__ CUtensorMap tm_codes,
                 const __grid_constant__ CUtensorMap tm_exps, const __grid_constant__ WgradArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  using C = Cfg<PLANES>;
  constexpr int kDyStages = C::kDyStages, kSlots = C::kSlots;
  // Two accumulators take turns.  The tensor core's additions truncate, so with
  // three planes a sum of more than 256 tokens has both: one for the upper parts
  // and one for the rest.  Apart, the long sum is added to a third as often, and
  // the error of 32 blocks against 64 bits falls from 6e-6 to 2e-6.  (Few tokens
  // need that less than the overlap: 16 experts of 50, 6752 x 3760 344 -> 285 us.)
  const auto both = [](const Unit& t) { return PLANES > 1 && t.n > 256; };
  uint8_t* sm_dy = smem;                                    // swizzled: 1024-byte boundaries
  uint8_t* sm_x = sm_dy + kDyStages * C::kStageBytes;       // decoded, swizzled
  uint8_t* sm_codes = sm_x + kSlots * kSlotBytes;           // swizzled
  uint8_t* sm_exps = sm_codes + kSlots * kCodeBytes;
  typename C::Shared& bars = *reinterpret_cast<typename C::Shared*>(sm_exps + kSlots * kExpBytes);
  uint64_t *dy_full = bars.dy_full, *dy_empty = bars.dy_empty, *code_full = bars.code_full,
           *code_empty = bars.code_empty, *ready = bars.ready, *unit_full = bars.unit_full,
           *unit_empty = bars.unit_empty, *tfull = bars.tfull, *tempty = bars.tempty,
           *drain = &bars.drain;
  volatile int* abort_flag = &bars.abort;
  uint32_t* tmem_slot = &bars.tmem_slot;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&unit_full[s], 1);
      // TMA threads, converters, epilogue; the MMA issuer in the even CTA
      mbar_init(&unit_empty[s], 2 + kSlots * kConvWarps + kEpiWarps + (rank == 0 ? 1 : 0));
    }
    for (int s = 0; s < kDyStages; ++s) {
      mbar_init(&dy_full[s], 1);                // this CTA's loads
      mbar_init(&dy_empty[s], 1);               // the pair's MMA commit, multicast
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&code_full[s], 1);
      mbar_init(&code_empty[s], kConvWarps);    // read into registers
      mbar_init(&ready[s], kConvWarps);         // the even CTA's warps, beside the odd CTA's bytes
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  griddep_launch_dependents();   // k_wgrad_join, which waits for this grid's end

  // One warp works out the units, a batch at a time, ahead of the other roles,
  // which take them in the same order and number the blocks of 64 tokens c = 0,
  // 1, ... since the start.
  uint32_t taken = 0;
  const auto take = [&](Unit& t, bool whole_warp) {
    const uint32_t at = taken % (2 * kUnits), batch = at / kUnits;
    if (at % kUnits == 0) {
      bool ok = mbar_wait_bounded(&unit_full[batch], taken / (2 * kUnits) & 1u, abort_flag, a.status,
                                  a.timeout_ns);
      if (whole_warp) ok = __all_sync(0xffffffffu, ok);
      if (!ok) return false;
    }
    const int4 v = *reinterpret_cast<const int4*>(bars.units[at]);
    const int4 w = *reinterpret_cast<const int4*>(bars.units[at] + 4);
    t.e = v.x;
    t.o0 = v.y;
    t.i0 = v.z;
    t.begin = v.w;
    t.n = w.x;
    t.m = w.y;
    t.add = w.z;
    if (at % kUnits == kUnits - 1) {
      if (whole_warp) __syncwarp();
      if (lane == 0) mbar_arrive(&unit_empty[batch]);
    }
    ++taken;
    return t.e >= 0;
  };

  // The single-thread roles hand registers to the epilogue: 7 warpgroups of 72
  // a thread at launch = 40 + 4 x 72 + 2 x 88.  (With three planes there are 5 of
  // 96.)
  if (warp < C::kConv0) {
    if constexpr (PLANES == 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0 || warp == 2) {
      if (lane == 0) {
        // ----------------------------------- TMA: dy (warp 0), codes + exponents
        const bool is_dy = warp == 0;
        uint64_t* full = is_dy ? dy_full : code_full;
        uint64_t* empty = is_dy ? dy_empty : code_empty;
        const uint32_t stages = is_dy ? kDyStages : kSlots;
        if (is_dy) griddep_wait();   // k_wgrad_dy's planes
        uint32_t c = 0, s = 0, phase = 0;
        bool ok = true;
        Unit t;
        while (ok && take(t, false)) {
          const int o = t.o0 + static_cast<int>(rank) * 128, i = t.i0 + static_cast<int>(rank) * 128;
          for (int k0 = 0; k0 < t.n; k0 += kBK, ++c) {
            if (!mbar_wait_bounded(&empty[s], phase ^ 1u, abort_flag, a.status, a.timeout_ns)) {
              ok = false;
              break;
            }
            if (is_dy) {
              mbar_arrive_expect_tx(&full[s], C::kStageBytes);
              uint8_t* d = sm_dy + s * C::kStageBytes;
              tma_load_3d(d, &tm_dy, &full[s], o, t.begin + k0, 0);
              tma_load_3d(d + PLANES * kAtomBytes, &tm_dy, &full[s], o + 64, t.begin + k0, 0);
            } else {
              mbar_arrive_expect_tx(&full[s], kCodeBytes + kExpBytes);
              tma_load_2d(sm_codes + s * kCodeBytes, &tm_codes, &full[s], i, t.begin + k0);
              tma_load_2d(sm_exps + s * kExpBytes, &tm_exps, &full[s], (i / 32) & ~15, t.begin + k0);
            }
            if (++s == stages) {
              s = 0;
              phase ^= 1u;
            }
          }
        }
        // every load has landed before the CTA exits
        for (uint32_t k = c > stages ? c - stages : 0; k < c; ++k)
          wait_drain(&full[k % stages], k / stages & 1u, a.status, a.timeout_ns);
      }
    } else if (warp == 1) {
      if (lane == 0 && rank == 0) {
        // -------------------------------------------------------- MMA issuer
        uint32_t c = 0, s = 0;
        uint32_t turn = 0, phase = 0;   // the next accumulator; whose turn's parity is odd
        bool ok = true;
        Unit t;
        while (ok && take(t, false)) {
          if (t.n == 0) continue;
          const bool two = both(t);
          const uint32_t acc = two ? 0 : turn;
          if (!mbar_wait_bounded(&tempty[acc], (phase >> acc & 1u) ^ 1u, abort_flag, a.status,
                                 a.timeout_ns) ||
              (two && !mbar_wait_bounded(&tempty[1], (phase >> 1 & 1u) ^ 1u, abort_flag, a.status,
                                         a.timeout_ns)))
            break;
          tc_fence_after();
          const uint32_t d = tmem_base + acc * 256u;
          for (int k0 = 0; k0 < t.n; k0 += kBK, ++c) {
            const uint32_t b = c % kSlots;
            if (!wait_cluster(&ready[b], c / kSlots & 1u, abort_flag, a.status, a.timeout_ns)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t b_addr = smem_u32(sm_x + b * kSlotBytes);
#pragma unroll
            for (int p = PLANES - 1; p >= 0; --p) {
              const uint32_t a_addr = smem_u32(sm_dy + s * C::kStageBytes + p * kAtomBytes);
#pragma unroll
              for (int ks = 0; ks < kBK / 16; ++ks)
                tc_mma_bf16_pair(d + (p > 0 && two ? 256u : 0u),
                                 smem_desc_sw128(a_addr + ks * 2048, PLANES * kAtomBytes, 1024),
                                 smem_desc_sw128(b_addr + ks * 2048, kAtomBytes, 1024), kIdesc,
                                 k0 == 0 && ((p == 0 && two) || p == PLANES - 1) && ks == 0 ? 0u : 1u);
            }
            tc_commit_pair_multicast(&dy_empty[s], 0x3);
            if (++s == kDyStages) s = 0;
          }
          if (!ok) break;
          tc_commit_pair_multicast(&tfull[acc], 0x3);
          if (two) tc_commit_pair_multicast(&tfull[1], 0x3);
          phase ^= two ? 3u : 1u << acc;
          turn ^= two ? 0u : 1u;
        }
        tc_commit_pair_multicast(drain, 0x1);
        wait_drain(drain, 0, a.status, a.timeout_ns);
      }
    } else if (warp == 3) {
      // ------------------------------------------------------------- walker
      const int step = static_cast<int>(gridDim.x >> 1);
      // Entry j of a batch (lane j's) is a chunk of one of the next 32 units, found in
      // the running sum of their numbers of chunks; lane kUnits finds where the next
      // batch starts.  Past the last unit there is an entry without an expert.
      int first = 0, chunk0 = 0;   // the pair's next unit, and its next chunk
      for (uint32_t k = 0;; ++k) {
        const int64_t u = (blockIdx.x >> 1) + static_cast<int64_t>(first + lane) * step;
        Unit t{-1, 0, 0, 0, 0, 0, 0};
        if (u < a.units) t = unit_of(a, static_cast<int>(u));
        int per = chunk_of<PLANES>(a, t.n);
        int upto = max((t.n + per - 1) / per, 1) - (lane == 0 ? chunk0 : 0);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += v;
        }
        int from = 0;   // units whose chunks all come before this entry (at most lane of them)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          const int v = __shfl_sync(0xffffffffu, upto, from + d - 1);
          if (v <= lane) from += d;
        }
        const int before = __shfl_sync(0xffffffffu, upto, max(from - 1, 0));
        const int chunk = from == 0 ? lane + chunk0 : lane - before;
        per = __shfl_sync(0xffffffffu, per, from);
        t.e = __shfl_sync(0xffffffffu, t.e, from);
        t.o0 = __shfl_sync(0xffffffffu, t.o0, from);
        t.i0 = __shfl_sync(0xffffffffu, t.i0, from);
        t.m = __shfl_sync(0xffffffffu, t.m, from);
        t.begin = __shfl_sync(0xffffffffu, t.begin, from) + chunk * per;
        t.n = min(__shfl_sync(0xffffffffu, t.n, from) - chunk * per, per);
        t.add = chunk > 0;
        first += __shfl_sync(0xffffffffu, from, kUnits);
        chunk0 = __shfl_sync(0xffffffffu, chunk, kUnits);
        const bool end = __any_sync(0xffffffffu, lane < kUnits && t.e < 0);
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&unit_empty[k % 2], (k / 2 & 1u) ^ 1u, abort_flag,
                                                       a.status, a.timeout_ns)))
          break;
        if (lane < kUnits) {
          int* p = bars.units[k % 2 * kUnits + lane];
          *reinterpret_cast<int4*>(p) = make_int4(t.e, t.o0, t.i0, t.begin);
          *reinterpret_cast<int4*>(p + 4) = make_int4(t.n, t.m, t.add, 0);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&unit_full[k % 2]);
        if (end) break;
      }
    }
  } else if (warp < C::kEpi0) {
    // ---------------------------------------------------------- converters
    // Group g decodes the blocks c = g, g + kSlots, ... into slot g, so that the
    // latencies of one block's chain (wait, read, decode, write, fence, arrive)
    // overlap with the others'; the codes are decoded in registers before the
    // slot is free.  Thread -> row r of the block and 64 columns (two
    // exponents, one swizzled row of the operand).
    //
    // The 64 columns go into the operand in an order of their own: position
    // 8b + 2q + i holds column 16q + 4 (b / 2) + b % 2 + 2i.  Decoding then
    // takes codes 0, 2 and 1, 3 of a word as they lie, and a thread of the
    // epilogue, which reads positions 8b + 2q + {0, 1} of every b, ends up with
    // 16 consecutive columns of G.
    const int g = (warp - C::kConv0) / kConvWarps;
    const int wi = (warp - C::kConv0) % kConvWarps;
    const int r = (wi & 1) * 32 + lane, j = wi >> 1;
    // Where zeros begin in a row.  Eight rows at eight places go out without a
    // conflict: 64 experts of 192 tokens 441 -> 411 us.  But experts of one block
    // leave the whole time to G's stores, and those get slower the closer together
    // they come: 256 experts of 16 tokens 1222 -> 1310 us, so those stay as they are.
    const int turn = PLANES > 1 || a.rows / a.experts > kBK ? r & 7 : 0;
    const uint32_t ready_g = mapa_shared(&ready[g], 0), note = mapa_shared(&bars.notes[g][wi], 0);
    const uint32_t dst = smem_u32(sm_x) + g * kSlotBytes + j * kAtomBytes + r * 128 + ((r & 7) << 4);
    const uint32_t src = smem_u32(sm_codes) + r * 128 + ((j * 4 ^ (r & 7)) << 4);
    uint32_t c0 = 0;   // blocks before this unit
    bool ok = true;
    Unit t;
    while (ok && take(t, true)) {
      const int blk = (t.i0 + static_cast<int>(rank) * 128) / 32;
      const uint32_t blocks = static_cast<uint32_t>((t.n + kBK - 1) / kBK);
      for (uint32_t k = (g - c0) % kSlots; k < blocks; k += kSlots) {
        const uint32_t c = c0 + k, s = c % kSlots;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&code_full[s], c / kSlots & 1u,
                                                       abort_flag, a.status, a.timeout_ns));
        if (!ok) break;
        uint32_t w[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[q][0]), "=r"(w[q][1]), "=r"(w[q][2]), "=r"(w[q][3])
                       : "r"((src ^ (q << 4)) + s * kCodeBytes)
                       : "memory");
        const uint32_t ee = *reinterpret_cast<const uint16_t*>(sm_exps + s * kExpBytes + r * 16 +
                                                               (blk & 15) + 2 * j);
        __syncwarp();
        if (lane == 0) mbar_arrive(&code_empty[s]);
        const bool out = static_cast<int>(k) * kBK + r >= t.n;   // a row of the next expert
        uint32_t sb[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t e = ee >> (8 * h) & 255u;
          // 2^(e - 127); a block that held something not finite (255) gives NaN
          const uint32_t v = e == 255u ? 0x7FC0u : e << 7;
          sb[h] = out ? 0u : v | v << 16;
        }
        uint32_t v[8][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const __nv_bfloat162 scale = *reinterpret_cast<const __nv_bfloat162*>(&sb[q >> 1]);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            v[2 * b][q] = codes_to_bf16(w[q][b], scale);
            v[2 * b + 1][q] = codes_to_bf16(w[q][b] >> 8, scale);
          }
        }
        if (c >= kSlots) {   // the MMAs that read this slot are done
          const uint32_t done = c - kSlots;
          ok = __all_sync(0xffffffffu,
                          mbar_wait_bounded(&dy_empty[done % kDyStages], done / kDyStages & 1u,
                                            abort_flag, a.status, a.timeout_ns));
          if (!ok) break;
        }
#pragma unroll
        for (int b = 0; b < 8; ++b)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst ^ (b << 4)),
                       "r"(v[b][0]), "r"(v[b][1]), "r"(v[b][2]), "r"(v[b][3])
                       : "memory");
        const uint32_t ds = c % kDyStages;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&dy_full[ds], c / kDyStages & 1u, abort_flag,
                                                       a.status, a.timeout_ns));
        if (!ok) break;
        if (out) {   // its dy too, this thread's half of the row
#pragma unroll
          for (int p = 0; p < PLANES; ++p) {
            uint4* y = reinterpret_cast<uint4*>(sm_dy + ds * C::kStageBytes +
                                                (j * PLANES + p) * kAtomBytes + r * 128);
#pragma unroll
            for (int z = 0; z < 8; ++z) y[z ^ turn] = make_uint4(0, 0, 0, 0);
          }
        }
        // The readers are the tensor cores, by MMAs that the even CTA issues: each
        // writer's proxy fence, then an arrival that pairs with the issuer's acquire.
        // From the odd CTA that has to release at cluster scope.  An asynchronous store
        // comes after what its thread did before it, and its completion on the barrier
        // is such a release, for which nobody waits.  (An arrival that releases at
        // cluster scope does make its warp wait: 14336 x 4096 over 8192 tokens 835 us
        // against 641, 64 experts of 256 tokens 595 against 509; one thread that does
        // so for the others, 1305 and 858.)
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (rank != 0)
            st_async_cluster(note, 0u, ready_g);
          else if (wi == 0)
            mbar_arrive_expect_tx(&ready[g], kConvWarps * sizeof(uint32_t));
          else
            mbar_arrive(&ready[g]);
        }
      }
      c0 += blocks;
    }
  } else {
    // ------------------------------------------------------------ epilogue
    if constexpr (PLANES == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
    // A warp drains 32 rows x 128 columns in four pieces of 16 x 64: a thread
    // gets 16 consecutive columns of two rows, four threads 64 columns, so that
    // a store of the warp fills eight whole 128-byte lines.
    const int q = warp & 3;                    // tensor-memory lanes 32 q ..
    const int half = (warp - C::kEpi0) >> 2;      // columns 128 half ..
    const uint32_t tempty0 = mapa_shared(&tempty[0], 0);
    uint32_t turn = 0, phase = 0;
    Unit t;
    while (take(t, true)) {
      const bool two = both(t);
      const bool add = a.g.accumulate || t.add;
      if (t.n == 0 && add) continue;
      const uint32_t acc = two ? 0 : turn;
      if (t.n > 0) {
        bool ok = mbar_wait_bounded(&tfull[acc], phase >> acc & 1u, abort_flag, a.status, a.timeout_ns);
        if (two) ok &= mbar_wait_bounded(&tfull[1], phase >> 1 & 1u, abort_flag, a.status, a.timeout_ns);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
      }
      char* g = matrix_of(a.g, t.m);
      const int esz = a.g.dtype == MUON_F32 ? 4 : 2;
      const int64_t row_bytes = a.g.stride * esz;
      const int o = t.o0 + static_cast<int>(rank) * 128 + q * 32;
      const int i = t.i0 + half * 128;
      const uint32_t src = tmem_base + (static_cast<uint32_t>(q) << 21) + acc * 256u + half * 128u;
      char* p = g + (o + (lane >> 2)) * row_bytes + (i + 16 * (lane & 3)) * esz;
      __syncwarp();   // tcgen05.ld takes the warp together
      if (a.g.ptrs != nullptr && reinterpret_cast<uintptr_t>(g) % 16 != 0) {
        if (lane == 0) atomicOr(a.status, kFlagMisaligned);   // left untouched
      } else if (two) {
        drain_unit<PLANES, EDGE>(src, a.g, g, p, row_bytes, o, i, false, add);
      } else {
        drain_unit<1, EDGE>(src, a.g, g, p, row_bytes, o, i, t.n == 0, add);
      }
      if (t.n == 0) continue;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_cluster(tempty0 + acc * 8u);
        if (two) mbar_arrive_cluster(tempty0 + 8u);
      }
      phase ^= two ? 3u : 1u << acc;
      turn ^= two ? 0u : 1u;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
  // Every notice of the odd CTA has been waited for, unless a role gave up: then one may
  // still be on its way into this CTA's shared memory, and takes about 1 us.
  if (rank == 0 && *abort_flag) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 100000) {
    }
  }
  // offsets that do not ascend within [0, rows]
  if (a.offsets != nullptr && blockIdx.x == 0)
    for (int e = threadIdx.x; e < a.experts; e += C::kThreads)
      if (a.offsets[e] < 0 || a.offsets[e + 1] < a.offsets[e] || a.offsets[e + 1] > a.rows)
        atomicOr(a.status, MUON_FLAG_INDEX);
}

// G (+)= the slices' partial sums, added in order.  parts: [slices][experts]
// [rows][stride] fp32.  Four columns of a row per thread.
__global__ void __launch_bounds__(256)
    k_wgrad_join(const float* parts, int slices, int64_t slice_stride, int64_t matrix_stride,
                 int64_t stride, const __grid_constant__ Matrices g, uint32_t* status) {
  const int i = (blockIdx.x * 256 + threadIdx.x) * 4;
  const int o = blockIdx.y, e = blockIdx.z;
  griddep_wait();   // k_wgrad's end
  char* m = matrix_of(g, e);
  if (g.ptrs != nullptr && reinterpret_cast<uintptr_t>(m) % 16 != 0) {   // left untouched
    if (threadIdx.x == 0) atomicOr(status, kFlagMisaligned);
    return;
  }
  if (i >= g.cols) return;
  const float* p = parts + e * matrix_stride + o * stride + i;
  float v[4] = {};
#pragma unroll 4
  for (int s = 0; s < slices; ++s) {
    const float4 w = *reinterpret_cast<const float4*>(p + s * slice_stride);
    v[0] += w.x; v[1] += w.y; v[2] += w.z; v[3] += w.w;
  }
  const int64_t at = o * g.stride + i;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (i + k >= g.cols) break;
    if (g.dtype == MUON_F32) {
      float* w = reinterpret_cast<float*>(m) + at + k;
      *w = g.accumulate ? *w + v[k] : v[k];
    } else {
      __nv_bfloat16* w = reinterpret_cast<__nv_bfloat16*>(m) + at + k;
      *w = __float2bfloat16_rn(g.accumulate ? __bfloat162float(*w) + v[k] : v[k]);
    }
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// The codes or the exponents of `rows` rows, boxes of kBK rows.  What lies past
// an operand's columns and rows reads as 0.
bool map_bytes(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t stride, int box_cols,
               CUtensorMapSwizzle swizzle) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), kBK};
  const cuuint32_t es[2] = {1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Planes of dy, boxes of 64 columns x kBK rows of all planes.
bool map_dy(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t stride, int planes,
            int64_t plane) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride) * 2,
                                 static_cast<cuuint64_t>(planes == 1 ? stride : plane) * 2};
  const cuuint32_t box[3] = {64, kBK, static_cast<cuuint32_t>(planes)};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTA pairs that fit the current device at once (asked once per device).
template <int PLANES, bool EDGE>
cudaError_t resident_pairs(cudaLaunchConfig_t& cfg, int* out) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kDevices && (*out = known[dev].load()) > 0) return cudaSuccess;
  cfg.gridDim = dim3(2);
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, k_wgrad<PLANES, EDGE>, &cfg);
  if (e != cudaSuccess) return e;
  if (n < 1) return cudaErrorInvalidConfiguration;
  if (dev < kDevices) known[dev].store(n);
  *out = n;
  return cudaSuccess;
}

// dy: planes of bf16, rows on 16-byte boundaries.  staged: k_wgrad_dy, just
// launched, writes them; the kernel's start overlaps it.
struct Planes {
  const void* base;
  int64_t stride, plane;
  bool staged;
};

template <int PLANES, bool EDGE>
cudaError_t launch_edge(const WgradArgs& a, const Planes& y, const muon_act8_t& x, cudaStream_t st) {
  using C = Cfg<PLANES>;
  cudaError_t e = cudaFuncSetAttribute(k_wgrad<PLANES, EDGE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(C::kSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  int pairs = 0;
  e = resident_pairs<PLANES, EDGE>(cfg, &pairs);
  if (e != cudaSuccess) return e;
  CUtensorMap dy{}, codes{}, exps{};
  if (a.rows > 0) {
    if (encode_fn() == nullptr) return cudaErrorNotSupported;
    const int64_t blocks = (static_cast<int64_t>(a.in) + 31) / 32;
    if (!map_dy(&dy, y.base, a.rows, a.out, y.stride, PLANES, y.plane) ||
        !map_bytes(&codes, x.codes, a.rows, a.in, x.code_stride, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !map_bytes(&exps, x.exps, a.rows, blocks, x.exp_stride, 16, CU_TENSOR_MAP_SWIZZLE_NONE))
      return cudaErrorInvalidValue;
  }
  cfg.numAttrs = y.staged ? 2 : 1;
  cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min(a.units, pairs)));
  return cudaLaunchKernelEx(&cfg, k_wgrad<PLANES, EDGE>, dy, codes, exps, a);
}

template <int PLANES>
cudaError_t launch(const WgradArgs& a, const Planes& y, const muon_act8_t& x, cudaStream_t st) {
  // pointers in a device array are on 16-byte boundaries, or their matrix is left alone
  const int esz = a.g.dtype == MUON_F32 ? 4 : 2;
  const uint64_t bits = reinterpret_cast<uintptr_t>(a.g.base) |
                        static_cast<uint64_t>((a.g.ptrs != nullptr ? 0 : a.g.batch_stride) * esz) |
                        static_cast<uint64_t>(a.g.stride * esz);
  const bool edge = a.g.rows % 32 != 0 || a.g.cols % 128 != 0 || bits % 16 != 0;
  return edge ? launch_edge<PLANES, true>(a, y, x, st) : launch_edge<PLANES, false>(a, y, x, st);
}

muon_status_t check_sizes(const muon_weight_grad_t* d) {
  if (d == nullptr || d->rows < 0 || d->out < 1 || d->experts < 1 || d->x.cols < 1)
    return MUON_ERR_INVALID_ARG;
  if (d->dy_dtype != MUON_BF16 && d->dy_dtype != MUON_F32) return MUON_ERR_INVALID_ARG;
  if (d->g_dtype != MUON_BF16 && d->g_dtype != MUON_F32) return MUON_ERR_INVALID_ARG;
  if (d->rows >= (int64_t{1} << 31) - (1 << 20) || d->out > (1 << 22) || d->x.cols > (1 << 22) ||
      d->experts > 65535)
    return MUON_ERR_UNSUPPORTED;
  if (static_cast<int64_t>((d->out + 255) / 256) * ((d->x.cols + 255) / 256) * d->experts >=
      (int64_t{1} << 26))
    return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}

// Slices of a tile's tokens.  With `tiles` tiles on 76 CTA pairs the last wave
// leaves pairs idle; s slices shorten the longest pair's share to
// ceil(tiles * s / 76) / s of a tile.  A slice costs its partial sums (256 KB
// written and read, about two blocks' time), so slices have at least 16 blocks
// of the average expert, and none are made for less than a fifth.
int slices_of(int64_t tiles, int64_t rows, int experts) {
  constexpr int kPairs = 76;
  const int64_t blocks = (rows / experts + kBK - 1) / kBK;
  int best = 1;
  double least = static_cast<double>((tiles + kPairs - 1) / kPairs) * 0.8;
  for (int s = 2; s <= 76 && s * 16 <= blocks; ++s) {
    const double share = static_cast<double>((tiles * s + kPairs - 1) / kPairs) / s +
                         2.0 * s / static_cast<double>(blocks);
    if (share < least) {
      least = share;
      best = s;
    }
  }
  return best;
}

struct Plan {
  int tiles_o, tiles_i, slices;
  bool cut;                // fp32 sums, see chunk_of
  int pitch;               // of dy's planes in the workspace
  size_t part_bytes, plane_bytes;   // partial sums; dy's planes behind them
};

Plan plan_of(const muon_weight_grad_t* d) {
  Plan p;
  p.tiles_o = (d->out + 255) / 256;
  p.tiles_i = (d->x.cols + 255) / 256;
  const int64_t tiles = static_cast<int64_t>(p.tiles_o) * p.tiles_i * d->experts;
  p.slices = slices_of(tiles, d->rows, d->experts);
  p.cut = p.slices > 1 || d->g_dtype == MUON_F32;
  p.pitch = (d->out + kCols - 1) / kCols * kCols;
  p.plane_bytes = static_cast<size_t>(d->rows) * p.pitch * 2 * (d->dy_dtype == MUON_F32 ? 3 : 1);
  p.part_bytes = p.slices > 1 ? static_cast<size_t>(tiles) * p.slices * 256 * 256 * 4 : 0;
  return p;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status_t muon_act8_weight_grad_workspace_size(const muon_weight_grad_t* d, size_t* bytes) {
  if (bytes == nullptr) return MUON_ERR_INVALID_ARG;
  const muon_status_t s = check_sizes(d);
  if (s != MUON_OK) return s;
  const Plan p = plan_of(d);
  *bytes = kHeader + p.part_bytes + p.plane_bytes;
  return MUON_OK;
}

muon_status_t muon_act8_weight_grad(const muon_weight_grad_t* d, void* workspace,
                                    size_t workspace_bytes, muon_stream_t stream) {
  muon_status_t s = check_sizes(d);
  if (s != MUON_OK) return s;
  const muon_act8_t& x = d->x;
  if (x.rows != d->rows || x.code_stride < x.cols ||
      x.exp_stride < (static_cast<int64_t>(x.cols) + 31) / 32)
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
  const Plan p = plan_of(d);
  if (workspace_bytes < kHeader + p.part_bytes + p.plane_bytes) return MUON_ERR_WORKSPACE_TOO_SMALL;

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Matrices g{d->g_ptrs, d->g_base, d->g_batch_stride, d->g_stride, d->out, x.cols, d->g_dtype,
                   d->accumulate};
  WgradArgs a{};
  a.rows = static_cast<int>(d->rows);
  a.out = d->out;
  a.in = x.cols;
  a.experts = d->experts;
  a.offsets = d->offsets;
  a.g = g;
  a.tiles_o = p.tiles_o;
  a.tiles_i = p.tiles_i;
  a.slices = p.slices;
  a.cut = p.cut;
  a.units = p.tiles_o * p.tiles_i * d->experts * p.slices;
  a.status = static_cast<uint32_t*>(workspace);
  a.timeout_ns = wait_timeout_ns();
  const int64_t part_stride = static_cast<int64_t>(p.tiles_i) * 256;
  const int64_t part_matrix = part_stride * p.tiles_o * 256;
  float* parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + kHeader);
  if (p.slices > 1)
    a.g = Matrices{nullptr, parts, part_matrix, part_stride, p.tiles_o * 256, p.tiles_i * 256,
                   MUON_F32, 0};
  const double rows = static_cast<double>(d->rows);
  const bool f32 = d->dy_dtype == MUON_F32;
  Planes y{d->dy, d->dy_stride, 0, d->rows > 0 && (f32 || !at_multiple(d->dy, 16) || d->dy_stride % 8 != 0)};
  if (y.staged) {
    auto* to = reinterpret_cast<__nv_bfloat16*>(static_cast<char*>(workspace) + kHeader + p.part_bytes);
    y.base = to;
    y.stride = p.pitch;
    y.plane = d->rows * p.pitch;
    const int64_t items = d->rows * (p.pitch / kCols);
    if (items > int64_t{0x7FFFFFFF} * 256) return MUON_ERR_UNSUPPORTED;
    const unsigned grid = static_cast<unsigned>((items + 255) / 256);
    prof_begin(kKindWeightGrad, st);
    if (f32)
      k_wgrad_dy<<<grid, 256, 0, st>>>(static_cast<const float*>(d->dy), d->dy_stride, items, d->out, to,
                                       p.pitch, y.plane, a.status);
    else
      k_wgrad_dy<<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(d->dy), d->dy_stride, items, d->out,
                                       to, p.pitch, y.plane, a.status);
    prof_end(kKindWeightGrad, st, 0.0, 0.0);
    if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
  } else if (cudaMemsetAsync(workspace, 0, sizeof(uint32_t), st) != cudaSuccess) {
    return MUON_ERR_CUDA;
  }
  prof_begin(kKindWeightGrad, st);
  const cudaError_t e = f32 ? launch<3>(a, y, x, st) : launch<1>(a, y, x, st);
  prof_end(kKindWeightGrad, st, 2.0 * rows * d->out * x.cols,
           rows * (d->out * esize(d->dy_dtype) + x.cols * (1.0 + 1.0 / 32)) +
               static_cast<double>(d->experts) * d->out * x.cols * esize(d->g_dtype) *
                   (d->accumulate ? 2 : 1));
  if (e != cudaSuccess) return MUON_ERR_CUDA;
  if (p.slices > 1) {
    prof_begin(kKindWeightGrad, st);
    const dim3 grid((x.cols + 1023) / 1024, d->out, d->experts);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_wgrad_join, static_cast<const float*>(parts), p.slices,
                                             part_matrix * d->experts, part_matrix, part_stride, g, a.status);
    prof_end(kKindWeightGrad, st, 0.0, 0.0);
    if (e != cudaSuccess) return MUON_ERR_CUDA;
  }
  return MUON_OK;
}

}  // extern "C"
