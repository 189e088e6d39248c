// Experts' products over expert-major segments, and their gradients.
//
// Three products share one tile kernel.  In each, the columns of the output are
// the rows of MFMA's first operand, so that a lane ends up with four
// consecutive columns of one output row and stores them together:
//   forward   z[r, n]  = sum_k w[e, n, k]  x[r, k]      r in segment e
//   grad_x    dx[r, k] = sum_n w[e, n, k] dz[r, n]
//   grad_w    dw[e, n, k] = sum_r x[r, k] dz[r, n]
// An operand whose summed index is contiguous in memory is "direct", the others
// (w in grad_x, both in grad_w) are "turned": the hardware's transposing LDS
// reads give MFMA the values that lie along the summed index.
//
// A tile of 256 x 256 outputs (small problems: 128 x 128) takes 64 bf16 (128
// E4M3) values of the summed index a step: 32 KiB of each operand, moved from
// memory straight into LDS (no registers), in two buffers of each, so that the
// next step's loads run while this step's 64 MFMAs a wave do.  A step reads
// (256 + 256) x 128 bytes from memory and 192 KiB from LDS for 8.4 MFLOP: LDS at
// 128 bytes a clock needs 75% of the time the matrix cores need, which is why
// the tile is this large.  16-byte units of an LDS row are exchanged by the
// row's low bits (by the source address, as the loads fill LDS lane after lane)
// so that operand reads touch every bank once.
//
// Measured on several cards, 32 experts of 4096 x 7168, top 8: forward of 4096 tokens,
// gated, 1500 to 1635 us (1.18 to 1.28 PFLOP/s; E4M3 960 to 1040 us, 1.85 to 2.0
// PFLOP/s), gradients of 2048 tokens 780 to 820 us (grad_x, 1.2 PFLOP/s) and 1120 to
// 1180 us (grad_w, 0.84 PFLOP/s with 1.9 GB stored).  In the forward the matrix cores
// are busy 70 to 72% of the cycles, at a clock that settles at 1.7 to 1.8 GHz of 2.4;
// E4M3 45% at 2.0 to 2.2 GHz.  grad_w (42%) waits for its stores between short
// products; 16 tokens over 64 experts read the weights at 5.9 TB/s (558 to 571 us).
#include <algorithm>
#include <type_traits>

#include "dev.h"
#include "mep_internal.h"

namespace mep {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

enum Mode { kForward, kGradX, kGradW };

struct TileArgs {
  const unsigned char* a;       // first operand: w (forward, grad_x), x (grad_w)
  const unsigned char* b;       // second operand: x (forward), dz (grad_x, grad_w)
  const float* a_scales;        // E4M3 only
  const float* b_scales;
  const float* bias;
  const uint16_t* residual;
  uint16_t* out;
  uint16_t* z;
  const int32_t* counts;
  const int32_t* offsets;
  int64_t cap;
  int32_t E;
  int32_t cols;                 // output columns: N (forward), K (grad_x, grad_w)
  int32_t depth;                // summed index: K (forward), Nz (grad_x); per segment for grad_w
  int32_t rows;                 // grad_w: output rows Nz
  int32_t Nz;
};

// The lane's number, worked out anew where it stands: kept in registers over the
// products, it and what follows from it would push others out to memory.
__device__ __forceinline__ int fresh_lane() {
  int l;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=&v"(l));
  return l;
}

// Rows of segment e that exist (rows past cap_em are left out).
__device__ __forceinline__ int segment_rows(const TileArgs& a, int e) {
  const int64_t off = a.offsets[e], left = a.cap - off;
  const int c = a.counts[e];
  return off < 0 || left <= 0 || c <= 0 ? 0 : left < c ? (int)left : c;
}

__device__ __forceinline__ u32x4 zero4() { return u32x4{0, 0, 0, 0}; }

__device__ __forceinline__ float silu(float z) { return z / (1.0f + expf(-z)); }
__device__ __forceinline__ float gelu(float z) {
  return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
}

// Row of the weight that row r of column tile n holds: with a gated activation
// every 32 rows are 16 gate rows and the 16 rows they gate, so that both halves
// of an output land in the same lane.
template <bool GLU, int BN>
__device__ __forceinline__ int weight_row(int n, int r, int cols) {
  if (!GLU) return min(n * BN + r, cols - 1);
  const int c = min(n * (BN / 2) + (r >> 5) * 16 + (r & 15), cols - 1);
  return (r & 16) ? cols + c : c;
}

#define MEP_LDS __attribute__((address_space(3)))
#define MEP_GLOBAL __attribute__((address_space(1)))

// BYTES a lane straight from memory (a base for the wave, an offset for the
// lane) into LDS, lane after lane from `lds` on.  The empty statement keeps the
// offset in one register: widened outside the loop it would take two.
template <int BYTES = 16>
__device__ __forceinline__ void load_to_lds(const unsigned char* base, uint32_t off,
                                            unsigned char* lds) {
  asm volatile("" : "+v"(off));
  const auto p = (const MEP_GLOBAL uint32_t*)(base + off);
  static_assert(BYTES == 16 || BYTES == 4, "");
  if constexpr (BYTES == 16)
    __builtin_amdgcn_global_load_lds(p, (MEP_LDS uint32_t*)lds, 16, 0, 0);
  else
    __builtin_amdgcn_global_load_lds(p, (MEP_LDS uint32_t*)lds, 4, 0, 0);
}

// Waits (the counters' fields as the ISA lays them out) and a barrier that
// nothing moves across.
constexpr int kAllLdsReads = 0xC07F;  // lgkmcnt(0)
constexpr int loads_left(int n) { return 0x0F70 | (n & 15) | (n >> 4) << 14; }  // vmcnt(n)

__device__ __forceinline__ void phase_end() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// How the units of row k of a turned tile of ROWS columns are exchanged: the
// four rows that 16 lanes of a transposing read touch, and those of the next 16
// lanes, fall on eight different 32-byte pieces of the 256 bytes of banks (rows
// of 128 bytes already alternate between the two halves).
template <int ROWS>
__device__ __forceinline__ int turned_swizzle(int k) {
  return ROWS >= 128 ? ((k & 3) | ((k >> 1) & 4)) << 1 : (((k >> 1) & 1) | ((k >> 2) & 2)) << 1;
}

template <Mode MODE, bool FP8, int ACT, int WN, int WM, int TN, int TM>
struct Tile {
  static constexpr bool GLU = MODE == kForward && ACT == MEP_ACT_SILU_GLU;
  // Forward: an odd last step runs outside the phases, with what is left of the
  // summed index; as another way into the loops the compiler would add waits
  // for it there.  Its depth is a layer's, most often a multiple of two steps;
  // the gradients' are the rows of a segment.
  static constexpr bool EVEN = MODE == kForward;
  static constexpr bool A_TURNED = MODE != kForward, B_TURNED = MODE == kGradW;
  static constexpr int WAVES = WN * WM, THREADS = WAVES * 64;
  static constexpr int BN = WN * TN * 16, BM = WM * TM * 16;
  static constexpr int VALS = FP8 ? 128 : 64;         // summed values a step
  static constexpr int UNIT = FP8 ? 16 : 8;           // values in 16 bytes
  static constexpr int SIZE = FP8 ? 1 : 2;
  static constexpr int COLS = GLU ? BN / 2 : BN;      // output columns a tile
  // loads of 1 KiB a wave and step: of each half of the columns, of each half
  // of the rows
  static constexpr int RA = BN / 16 / WAVES, RB = BM / 16 / WAVES;
  static constexpr int SCALES = FP8 ? BM + (WAVES - BM / 64) * 64 : 0;
  static_assert(WN == 2 && WAVES == 8 && RA > 0 && RB > 0, "");
  static_assert(!FP8 || BM < 512, "a wave for each load of scales");
};

// Where a lane reads COUNT fragments of 16 rows from row `at` of a tile of ROWS
// rows.  Direct: the two units of a step's halves (E4M3: the two halves of a
// lane's 32 values; which values those are is free as long as both operands
// agree, and lanes read together then meet no bank twice: with two neighbouring
// units a lane, conflicts took a sixth of the cycles, though no time beyond the
// spread of runs), the fragments 2 KiB apart.  Turned: a place for each fragment.
template <int ROWS, bool TURNED, bool FP8, int COUNT>
struct Reader {
  static constexpr int N = TURNED ? COUNT : 2;
  uint32_t off[N];

  __device__ __forceinline__ Reader(int at, int lane) {
    const int g = lane >> 4, r16 = lane & 15;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (TURNED) {
        const int k = g * 8 + (r16 >> 2);
        const int u = ((at + i * 16) >> 3) + ((r16 & 3) >> 1);
        off[i] = k * (ROWS * 2) + ((u ^ turned_swizzle<ROWS>(k)) << 4) + (r16 & 1) * 8;
      } else {
        const int u = 4 * i + g;
        off[i] = (at + r16) * 128 + ((u ^ (r16 & 7)) << 4);
      }
    }
  }

  // Called before a phase's reads: without, the sums of these offsets and every
  // array's address would be kept in registers of their own.
  __device__ __forceinline__ void refresh() {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(off[i]));
  }

  __device__ __forceinline__ u32x4 unit(const unsigned char* lds, int i, int q) const {
    return *reinterpret_cast<const u32x4*>(lds + off[q] + i * 2048);
  }

  // 8 values of the summed index: half s of a step's 64, fragment i.
  __device__ __forceinline__ bf16x8 bf16(const unsigned char* lds, int i, int s) const {
    if (!TURNED) return __builtin_bit_cast(bf16x8, unit(lds, i, s));
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    const unsigned char* p = lds + off[TURNED ? i : 0] + s * 32 * (ROWS * 2);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MEP_LDS s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MEP_LDS s16x4*)(p + 4 * ROWS * 2));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }

  // 32 E4M3 values.
  __device__ __forceinline__ i32x8 e4m3(const unsigned char* lds, int i) const {
    return __builtin_bit_cast(i32x8, __builtin_shufflevector(unit(lds, i, 0), unit(lds, i, 1), 0, 1,
                                                             2, 3, 4, 5, 6, 7));
  }
};

// grad_w is written once and large: it passes L2 by, where the operands stay.
__device__ __forceinline__ void store16(uint16_t* p, u32x4 v, bool stream) {
  if (stream) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
  else *reinterpret_cast<u32x4*>(p) = v;
}

// A tile's place: expert, row and column tile, and the segment it lies in.
struct Place {
  int e, m, n, seg;
  int64_t row0;
};

// Row tiles of `size` rows before each expert, by the block's first wave;
// everyone waits.
__device__ __forceinline__ void count_row_tiles(const TileArgs& a, int size, int32_t* first) {
  const int tid = threadIdx.x;
  if (tid < kWave) {
    int base = 0;
    for (int e0 = 0; e0 < a.E; e0 += kWave) {
      const int e = e0 + tid;
      const int n = e < a.E ? (segment_rows(a, e) + size - 1) / size : 0;
      int s = n;
      for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(s, d);
        if (tid >= d) s += o;
      }
      if (e < a.E) first[e] = base + s - n;
      base += __shfl(s, kWave - 1);
    }
    if (tid == 0) first[a.E] = base;
  }
  __syncthreads();
}

// The tile'th tile: experts in order, an expert's column tiles in order, the row
// tiles that share a column tile next to each other.  From four whole row tiles
// (`size` rows) on, the last one, which has fewer rows, comes behind all of them:
// neighbouring blocks then take equally long and stay close enough together to
// share what they load in L2 (4096 tokens, 8 of 32 experts of 4096 x 7168, about
// 1024 rows each: 1573 -> 1520 us).  With fewer, the columns loaded once more
// cost more (512 rows each, gradient of x: 857 -> 882 us).
__device__ __forceinline__ Place find_tile(const TileArgs& a, const int32_t* first, int size,
                                           int col_tiles, int64_t tile) {
  Place at;
  int lo = 0, hi = a.E;  // the last expert whose tiles start at or before this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)first[mid] * col_tiles <= tile) lo = mid; else hi = mid;
  }
  at.e = first_lane(lo);
  at.seg = segment_rows(a, at.e);
  const int all = first[at.e + 1] - first[at.e], whole = at.seg / size;
  const int together = whole >= 4 ? whole : all;
  const int q = (int)(tile - (int64_t)first[at.e] * col_tiles);
  const int behind = q - together * col_tiles;
  at.m = first_lane(behind >= 0 ? whole : q % together);
  at.n = first_lane(behind >= 0 ? behind : q / together);
  at.row0 = a.offsets[at.e];
  return at;
}

template <int ACT>
__device__ __forceinline__ float activate(float z, float up) {
  return ACT == MEP_ACT_GELU       ? gelu(z)
         : ACT == MEP_ACT_SILU     ? silu(z)
         : ACT == MEP_ACT_SILU_GLU ? silu(z) * up
                                   : z;
}

template <Mode MODE, bool FP8, int ACT, int WN, int WM, int TN, int TM, int PER_CU>
__global__ __launch_bounds__(WN * WM * 64, 2 * PER_CU) void tile_kernel(TileArgs a) {
  using T = Tile<MODE, FP8, ACT, WN, WM, TN, TM>;
  constexpr bool GLU = T::GLU;
  constexpr int BN = T::BN, BM = T::BM, RA = T::RA, RB = T::RB;
  // separate arrays: reads of one wait for none of the loads into another.  A
  // step's columns come in two halves (of each wave's), then its rows, with the
  // scales of both behind them.
  __shared__ __attribute__((aligned(1024))) unsigned char a00[BN * 64], a01[BN * 64];
  __shared__ __attribute__((aligned(1024))) unsigned char a10[BN * 64], a11[BN * 64];
  __shared__ __attribute__((aligned(1024))) unsigned char b0[BM * 128 + T::SCALES * 4];
  __shared__ __attribute__((aligned(1024))) unsigned char b1[BM * 128 + T::SCALES * 4];
  extern __shared__ int32_t first[];         // [E+1]: row tiles before each expert

  const int wave = first_lane(threadIdx.x >> 6);
  const int wn = wave % WN, wm = wave / WN;
  const bool late = wave >= T::WAVES / 2;
  const int col_tiles = (a.cols + T::COLS - 1) / T::COLS;

  if (MODE != kGradW) count_row_tiles(a, BM, first);
  const int grad_w_tiles = (a.rows + BM - 1) / BM;
  const int64_t tiles = MODE == kGradW ? (int64_t)a.E * grad_w_tiles * col_tiles
                                       : (int64_t)first[a.E] * col_tiles;
  // blocks go round the 8 XCDs in turn: give each XCD a run of neighbouring tiles
  const int per = gridDim.x / 8;
  int64_t tile = gridDim.x % 8 == 0 ? (blockIdx.x % 8) * (int64_t)per + blockIdx.x / 8
                                    : blockIdx.x;
  if (tile >= tiles) return;

  Place at;
  auto locate = [&]() __attribute__((always_inline)) {
    if (MODE == kGradW) {
      const int per_e = grad_w_tiles * col_tiles;
      at.e = (int)(tile / per_e);
      const int q = (int)(tile % per_e);
      // bands of 4 row tiles, column after column: the 32 tiles that an XCD works
      // on share 4 tiles of dz and 8 of x (1465 -> 1332 us at 2048 tokens, 32
      // experts, 4096 x 7168)
      const int band = q / (4 * col_tiles), h = min(4, grad_w_tiles - band * 4);
      const int r = q - band * (4 * col_tiles);
      at.m = band * 4 + r % h;
      at.n = r / h;
      at.seg = segment_rows(a, at.e);
      at.row0 = a.offsets[at.e];
    } else {
      at = find_tile(a, first, BM, col_tiles, tile);
    }
  };

  // Where this lane's pieces of the two tiles come from, as offsets from bases
  // that move along: for a direct operand 8 rows of 128 bytes a load, for a
  // turned one 1 KiB of whole rows k.  A tile spans at most 256 rows of 2 MiB,
  // so 32 bits hold the offsets.  Rows and columns past the end repeat the last.
  uint32_t oa[2][RA], ob[2 * RB], os = 0;
  const unsigned char *base_a, *base_b, *base_s = nullptr;
  int64_t stepa, stepb;
  int steps, left;    // whole steps; what is left of the summed index behind them
  constexpr int UA = BN / 16, UB = BM / 8;  // 16-byte units in a row of a turned tile
  auto setup = [&]() __attribute__((always_inline)) {
    const int lane = fresh_lane(), du = (lane & 7) ^ (lane >> 3);
    const int depth = MODE == kGradW ? at.seg : a.depth;
    steps = depth / T::VALS;
    left = depth % T::VALS;
    // grad_w: where the rows behind the segment exist, the last step takes them
    // too and leaves them out of its products
    if (MODE == kGradW && left > 0 && at.row0 + (steps + 1) * T::VALS <= a.cap) {
      ++steps;
      left -= T::VALS;
    }
    const int64_t lda = (int64_t)(T::A_TURNED ? a.cols : depth) * T::SIZE;
    const int64_t ldb = (int64_t)(T::B_TURNED ? a.rows : depth) * T::SIZE;
    stepa = T::A_TURNED ? T::VALS * lda : 128;
    stepb = T::B_TURNED ? T::VALS * ldb : 128;
    // gated: a load's 8 rows are all gate rows or all rows they gate, and the
    // same for all of a wave's loads
    const int64_t a_row = MODE == kGradW
                              ? at.row0
                              : (int64_t)at.e * a.Nz + (GLU && (wave & 2) ? a.cols : 0);
    const int an = T::A_TURNED ? 0 : at.n * T::COLS;  // first weight row of the tile
    base_a = a.a + (a_row + an) * lda + (T::A_TURNED ? at.n * BN * 2 : 0);
    base_b = a.b + (T::B_TURNED ? at.row0 * ldb + at.m * BM * 2 : (at.row0 + at.m * BM) * ldb);
    // column r of half h of the tile's columns
    auto column = [](int h, int r) {
      return (r / (BN / 4)) * (BN / 2) + h * (BN / 4) + r % (BN / 4);
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < RA; ++i) {
        const int c = i * T::WAVES + wave;
        if (T::A_TURNED) {
          const int k = c * (64 / UA) + lane / UA;
          const int col = column(h, ((lane % UA) ^ turned_swizzle<BN / 2>(k)) * 8);
          oa[h][i] = (uint32_t)(k * lda) + min(col, a.cols - 8 - at.n * BN) * 2;
        } else {
          const int r = column(h, c * 8 + (lane >> 3));
          const int col = GLU ? (r >> 5) * 16 + (r & 15) : r;
          oa[h][i] = (uint32_t)(min(col, a.cols - 1 - an) * lda) + du * 16;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2 * RB; ++i) {
      const int c = i * T::WAVES + wave;
      if (T::B_TURNED) {
        const int k = c * (64 / UB) + lane / UB;
        const int u = (lane % UB) ^ turned_swizzle<BM>(k);
        ob[i] = (uint32_t)(k * ldb) + min(u * 8, a.rows - 8 - at.m * BM) * 2;
      } else {
        ob[i] = (uint32_t)(min(c * 8 + (lane >> 3), at.seg - 1 - at.m * BM) * ldb) + du * 16;
      }
    }
    if (FP8) {
      // this wave's scales of a step: 64 rows of x, or every 4th row of the
      // weight's tile (a copy for each wave that has no rows)
      const int blocks = depth / 128;
      if (wave < BM / 64) {
        base_s = (const unsigned char*)(a.b_scales + (at.row0 + at.m * BM) * blocks);
        os = (uint32_t)min(wave * 64 + lane, at.seg - 1 - at.m * BM) * blocks * 4;
      } else {
        const int wr = weight_row<GLU, BN>(at.n, min(lane * 4, BN - 1), a.cols);
        base_s = (const unsigned char*)(a.a_scales + (int64_t)at.e * (a.Nz / 128) * blocks);
        os = (uint32_t)(wr / 128) * blocks * 4;
      }
    }
  };
  auto load_a = [&](unsigned char* la, int h) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RA; ++i)
      load_to_lds(base_a, oa[h][i], la + (i * T::WAVES + wave) * 1024);
    if (h == 1) base_a += stepa;
  };
  auto load_b = [&](unsigned char* lb, int h) __attribute__((always_inline)) {
#pragma unroll
    for (int i = h * RB; i < (h + 1) * RB; ++i)
      load_to_lds(base_b, ob[i], lb + (i * T::WAVES + wave) * 1024);
    if (FP8 && h == 0) {
      load_to_lds<4>(base_s, os, lb + BM * 128 + wave * 256);
      base_s += 4;
    }
    if (h == 1) base_b += stepb;
  };
  constexpr int kRows = 2 * RB + (FP8 ? 1 : 0);  // loads of a step's rows
  // A tile's loads before its first phase.  Steps alternate between the two
  // buffers so that the last one finds the second, the first one therefore
  // either.
  auto prologue = [&] {
    auto both = [&](unsigned char* a_0, unsigned char* a_1, unsigned char* b,
                    unsigned char* nb) __attribute__((always_inline)) {
      load_b(b, 0);
      load_b(b, 1);
      load_a(a_0, 0);
      load_a(a_1, 1);
      if (steps > 1) {
        load_b(nb, 0);
        load_b(nb, 1);
      }
    };
    // the comments keep the compiler from joining the two ways' ends, which
    // would hide from it which arrays the loads fill
    if (!T::EVEN && (steps & 1)) {
      both(a10, a11, b1, b0);
      asm volatile("; second buffer first" ::: "memory");
    } else if (steps > (T::EVEN ? 1 : 0)) {
      both(a00, a01, b0, b1);
      asm volatile("; first buffer first" ::: "memory");
    }
  };
  // a part of a step through registers, zeros past the end of the summed index
  auto load_tail = [&](unsigned char* lds, const unsigned char* base, uint32_t off, int c,
                       bool in) {
    const u32x4 v = in ? *reinterpret_cast<const u32x4*>(base + off) : zero4();
    *reinterpret_cast<u32x4*>(lds + c * 1024 + fresh_lane() * 16) = v;
  };

  // Operands: a step's rows stay in registers for both halves of the columns.
  constexpr int HN = TN / 2;            // column fragments of a half
  constexpr int SUB = FP8 ? 1 : 2;      // MFMAs along a step
  using Frag = std::conditional_t<FP8, i32x8, bf16x8>;
  f32x4 acc[TN][TM];
  Frag av[HN][SUB], bv[TM][SUB];
  // E4M3: a wave's columns lie in one block of 128 weight rows (gated: in one
  // of each half)
  constexpr int BLOCKS = GLU ? 2 : 1;
  float scale[BLOCKS][TM];
  Reader<BN / 2, T::A_TURNED, FP8, HN> reader_a(wn * HN * 16, fresh_lane());
  Reader<BM, T::B_TURNED, FP8, TM> reader_b(wm * TM * 16, fresh_lane());
  uint32_t scale_off = BM * 128 + (wm * TM * 16 + (fresh_lane() & 15)) * 4;
  auto read_b = [&](const unsigned char* lb) __attribute__((always_inline)) {
    reader_b.refresh();
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      if constexpr (FP8) {
        bv[j][0] = reader_b.e4m3(lb, j);
      } else {
#pragma unroll
        for (int s = 0; s < SUB; ++s) bv[j][s] = reader_b.bf16(lb, j, s);
      }
    }
    if constexpr (FP8) {
      asm volatile("" : "+v"(scale_off));
      const float* ls = reinterpret_cast<const float*>(lb + BM * 128);
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int q = 0; q < BLOCKS; ++q)
          scale[q][j] = ls[BM + (wn * TN + q) * 4] *
                        *reinterpret_cast<const float*>(lb + scale_off + j * 64);
    }
  };
  auto read_a = [&](const unsigned char* la) __attribute__((always_inline)) {
    reader_a.refresh();
#pragma unroll
    for (int i = 0; i < HN; ++i) {
      if constexpr (FP8) {
        av[i][0] = reader_a.e4m3(la, i);
      } else {
#pragma unroll
        for (int s = 0; s < SUB; ++s) av[i][s] = reader_a.bf16(la, i, s);
      }
    }
  };
  // zeros for the values from `valid` of the step's 64 on: what lies there may
  // be anything, infinities included
  auto mask_values = [&](auto& frags, int valid) __attribute__((always_inline)) {
    if constexpr (!FP8) {
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        const int v = valid - s * 32 - (fresh_lane() >> 4) * 8;
        u32x4 mask;
#pragma unroll
        for (int d = 0; d < 4; ++d)
          mask[d] = v >= 2 * d + 2 ? 0xffffffffu : v == 2 * d + 1 ? 0xffffu : 0u;
#pragma unroll
        for (auto& f : frags)
          f[s] = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, f[s]) & mask);
      }
    }
  };
  // `meanwhile` is issued behind the first MFMAs, so that the matrix cores do
  // not wait for it
  auto multiply = [&](int half, auto meanwhile) __attribute__((always_inline)) {
    if constexpr (FP8) {
      // a product of 128 is scaled and added while the matrix cores work on
      // the next.  Inside, the instruction adds 8 neighbouring products on a grid
      // of 2^-13 of the largest one's power of two, and those sums in fp32: rows
      // of 128 random values come within 2^-16.7 of the sum of magnitudes (2^-19.5
      // on average), well below the result's rounding to bf16.  Codes turned into
      // bf16 would add without that loss, at half the rate.
      f32x4 p[2];
#pragma unroll
      for (int q = 0; q < HN * TM + 1; ++q) {
        if (q < HN * TM)
          p[q % 2] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              av[q / TM][0], bv[q % TM][0], f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
        if (q == TM) {
          __builtin_amdgcn_sched_barrier(0);
          meanwhile();
          __builtin_amdgcn_sched_barrier(0);
        }
        if (q >= 1) {
          const int i = half * HN + (q - 1) / TM, j = (q - 1) % TM;
          f32x4& c = acc[i][j];
#pragma unroll
          for (int v = 0; v < 4; ++v)
            c[v] = fmaf(p[(q - 1) % 2][v], scale[i % BLOCKS][j], c[v]);
          // here and in this order: more products in flight would not fit
          // the registers
          asm volatile("" : "+v"(c));
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < SUB; ++s)
#pragma unroll
        for (int i = 0; i < HN; ++i) {
#pragma unroll
          for (int j = 0; j < TM; ++j)
            acc[half * HN + i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                av[i][s], bv[j][s], acc[half * HN + i][j], 0, 0, 0);
          if (s == 0 && i == 0) {
            __builtin_amdgcn_sched_barrier(0);
            meanwhile();
            __builtin_amdgcn_sched_barrier(0);
          }
        }
    }
  };

  // Two groups of waves, one of each on every SIMD, take turns: while one
  // multiplies a half of its columns from registers the other reads its next
  // operands from LDS; the second group runs one phase behind.  Rows and the
  // first half of the columns of step k are read in the first phase of four,
  // the other half in the third, so their places are free for step k + 2 two
  // phases later: each phase issues a quarter of a step's loads, which have
  // four to six phases to land.  With t = 4k the time of the first group's
  // first phase of step k, both groups issue (each in its own phase then)
  //   t + 2, t + 3: the rows of step k + 2,  t + 4, t + 5: its columns,
  // and wait at t + 3 for rows and first columns of step k + 1 and at t + 1
  // for the other columns of step k, leaving what was issued later in flight.
  // MORE: how many steps follow, as far as loads for them are concerned (2, or
  // in the last two steps, where the loads drain, 1 and 0).
  auto run = [&](auto late_, auto active_) __attribute__((always_inline)) {
    constexpr bool LATE = late_(), ACTIVE = active_();
    auto step = [&](auto more_, unsigned char* a_0, unsigned char* a_1, unsigned char* b,
                    unsigned char* na_0, unsigned char* na_1) __attribute__((always_inline)) {
      constexpr int MORE = more_();
      const bool mask = MODE == kGradW && MORE == 0 && left < 0;
      auto multiplying = [&](int half, auto meanwhile) __attribute__((always_inline)) {
        __builtin_amdgcn_s_setprio(1);
        if (ACTIVE) multiply(half, meanwhile);
        else meanwhile();
        __builtin_amdgcn_s_setprio(0);
      };
      constexpr int kSecond = MORE >= 1 ? kRows + 2 * RA : 0;
      constexpr int kFirst = MORE >= 2 ? kRows + RA : RA;
      if (ACTIVE) { read_b(b); read_a(a_0); }
      if (MORE >= 1) load_a(LATE ? na_1 : na_0, LATE ? 1 : 0);
      __builtin_amdgcn_s_waitcnt(kAllLdsReads);
      if (ACTIVE && mask) { mask_values(bv, left + T::VALS); mask_values(av, left + T::VALS); }
      if (LATE) __builtin_amdgcn_s_waitcnt(loads_left(kSecond));
      phase_end();
      multiplying(0, [&] {
        if (LATE) { if (MORE >= 2) load_b(b, 0); }
        else if (MORE >= 1) load_a(na_1, 1);
      });
      if (!LATE) __builtin_amdgcn_s_waitcnt(loads_left(kSecond));
      phase_end();
      if (ACTIVE) read_a(a_1);
      if (MORE >= 2) load_b(b, LATE ? 1 : 0);
      __builtin_amdgcn_s_waitcnt(kAllLdsReads);
      if (ACTIVE && mask) mask_values(av, left + T::VALS);
      if (LATE) __builtin_amdgcn_s_waitcnt(loads_left(kFirst));
      phase_end();
      multiplying(1, [&] {
        if (MORE >= 2) { if (LATE) load_a(a_0, 0); else load_b(b, 1); }
      });
      if (!LATE) __builtin_amdgcn_s_waitcnt(loads_left(kFirst));
      phase_end();
    };
    using Two = std::integral_constant<int, 2>;
    using One = std::integral_constant<int, 1>;
    using None = std::integral_constant<int, 0>;
    if (LATE) {
      if (!T::EVEN && (steps & 1)) {
        if (steps > 1) load_a(a00, 0);
        asm volatile("; second buffer first" ::: "memory");
      } else {
        load_a(a10, 0);
        asm volatile("; first buffer first" ::: "memory");
      }
      phase_end();
    }
    if (!T::EVEN && (steps & 1) && steps > 1) step(Two{}, a10, a11, b1, a00, a01);
    for (int k = steps & ~1; k > 2; k -= 2) {
      step(Two{}, a00, a01, b0, a10, a11);
      step(Two{}, a10, a11, b1, a00, a01);
    }
    if (steps > 1) step(One{}, a00, a01, b0, a10, a11);
    step(None{}, a10, a11, b1, a00, a01);
    if (!LATE) phase_end();
    // nothing is left in flight; said here, the compiler knows it on every way
    // that leads to the other groups' loops and inserts no waits of its own
    __builtin_amdgcn_s_waitcnt(loads_left(0));
  };

  // A tile's rows and columns in place: activation and what goes with it, and
  // the stores.  A lane has 4 consecutive columns of row r16 in each fragment;
  // two fragments exchange rows of 16 lanes so that it stores 8 of one.
  auto finish = [&](const Place& at) __attribute__((always_inline)) {
    const int lane = fresh_lane(), g = lane >> 4, r16 = lane & 15;
    const int rows = MODE == kGradW ? a.rows : at.seg;
    const int64_t out0 = MODE == kGradW ? (int64_t)at.e * rows : at.row0;
#pragma unroll
    for (int i = 0; i < TN; i += GLU ? 4 : 2) {
      const int col = at.n * T::COLS + (wn * TN + i) * (GLU ? 8 : 16);
      // bias of the two output fragments (gated: of both halves of each)
      f32x4 bias[2][GLU ? 2 : 1];
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int h = 0; h < (GLU ? 2 : 1); ++h) {
          bias[f][h] = f32x4{0, 0, 0, 0};
          const int c = col + f * 16 + g * 4;
          if (MODE == kForward && a.bias && c < a.cols)
            bias[f][h] = *reinterpret_cast<const f32x4*>(a.bias + (int64_t)at.e * a.Nz +
                                                         h * a.cols + c);
        }
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int r = at.m * BM + (wm * TM + j) * 16 + r16;
        const bool in = r < rows;
        const int64_t row = out0 + r;
        u32x2 y[2], zv[2][GLU ? 2 : 1];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          f32x4 v = acc[i + (GLU ? 2 * f : f)][j];
          if (MODE == kForward) {
            v += bias[f][0];
            f32x4 up = f32x4{0, 0, 0, 0};
            if (GLU) up = acc[i + (GLU ? 2 * f + 1 : 0)][j] + bias[f][GLU ? 1 : 0];
            zv[f][0] = u32x2{pack_bf16_rne(v[0], v[1]), pack_bf16_rne(v[2], v[3])};
            if (GLU) zv[f][GLU ? 1 : 0] = u32x2{pack_bf16_rne(up[0], up[1]), pack_bf16_rne(up[2], up[3])};
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = activate<ACT>(v[q], up[q]);
            const int c = col + f * 16 + g * 4;
            if (a.residual && in && c < a.cols) {
              const u32x2 res = *reinterpret_cast<const u32x2*>(a.residual + row * a.cols + c);
              v[0] += bf16_lo(res[0]); v[1] += bf16_hi(res[0]);
              v[2] += bf16_lo(res[1]); v[3] += bf16_hi(res[1]);
            }
          }
          y[f] = u32x2{pack_bf16_rne(v[0], v[1]), pack_bf16_rne(v[2], v[3])};
        }
        auto put = [&](uint16_t* p, int ld, int at_col, int end, u32x2 x0, u32x2 x1) {
          const auto lo = __builtin_amdgcn_permlane16_swap(x0[0], x1[0], false, false);
          const auto hi = __builtin_amdgcn_permlane16_swap(x0[1], x1[1], false, false);
          const int c = (g & 1) * 16 + (g >> 1) * 8;
          if (in && at_col + c < end)
            store16(p + row * ld + at_col + c, u32x4{lo[0], hi[0], lo[1], hi[1]},
                    MODE == kGradW);
        };
        if (MODE == kForward && a.z) {
          put(a.z, a.Nz, col, a.cols, zv[0][0], zv[1][0]);
          if (GLU) put(a.z, a.Nz, a.cols + col, 2 * a.cols, zv[0][GLU ? 1 : 0], zv[1][GLU ? 1 : 0]);
        }
        put(a.out, a.cols, col, a.cols, y[0], y[1]);
      }
    }
  };

  locate();
  setup();
  prologue();
  while (true) {
    const int rows = MODE == kGradW ? a.rows : at.seg;
    const bool active = at.m * BM + wm * (TM * 16) < rows;
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    __builtin_amdgcn_s_waitcnt(loads_left(0));
    phase_end();
    if (steps > (T::EVEN ? 1 : 0)) {
      using Yes = std::true_type;
      using No = std::false_type;
      if (late) {
        if (active) run(Yes{}, Yes{}); else run(Yes{}, No{});
      } else {
        if (active) run(No{}, Yes{}); else run(No{}, No{});
      }
    }
    // bases stand behind the last step of the phases
    int whole = T::EVEN ? steps & 1 : 0;
    for (int rest = whole + (left > 0 ? 1 : 0); rest > 0; --rest, whole = 0) {
      if (whole) {
        load_b(b0, 0);
        load_b(b0, 1);
        load_a(a00, 0);
        load_a(a01, 1);
        __builtin_amdgcn_s_waitcnt(loads_left(0));
      } else {
        const int lane = fresh_lane(), du = (lane & 7) ^ (lane >> 3);
        const auto in_a = [&](int c) {
          return T::A_TURNED ? c * (64 / UA) + lane / UA < left : du * T::UNIT < left;
        };
#pragma unroll
        for (int i = 0; i < RA; ++i) {
          const int c = i * T::WAVES + wave;
          load_tail(a00, base_a, oa[0][i], c, in_a(c));
          load_tail(a01, base_a, oa[1][i], c, in_a(c));
        }
#pragma unroll
        for (int i = 0; i < 2 * RB; ++i) {
          const int c = i * T::WAVES + wave;
          load_tail(b0, base_b, ob[i], c,
                    T::B_TURNED ? c * (64 / UB) + lane / UB < left : du * T::UNIT < left);
        }
        __builtin_amdgcn_s_waitcnt(kAllLdsReads);  // LDS writes count there too
      }
      phase_end();
      if (active) {
        read_b(b0);
        read_a(a00);
        multiply(0, [] {});
        read_a(a01);
        multiply(1, [] {});
      }
      __builtin_amdgcn_s_waitcnt(kAllLdsReads);
      phase_end();
    }
    // every read of the buffers is done: the next tile's first loads run while
    // this one is stored
    const Place done = at;
    tile += gridDim.x;
    const bool more = tile < tiles;
    if (more) {
      locate();
      setup();
      prologue();
    }
    if (active) finish(done);
    if (!more) break;
  }
}

// ---- few rows -----------------------------------------------------------------

// A block takes 16 rows of a segment and 32 weight rows (gated: 16 and the 16
// they gate) and splits the summed index over its 8 waves; operands go from
// memory straight to registers, 8 loads of 1 KiB of the weight a wave in flight,
// and the waves join in order through LDS.  For single tokens there is nothing
// to share in LDS, and what counts is that every CU reads weights from the first
// moment on: one token, 2 experts of 1024 x 7168, takes 35.5 us in 16 tiles of
// 128 x 128 and 19.4 here (1.5 TB/s of weights).
constexpr int kFewRows = 16, kFewWaves = 8;

template <bool FP8, int ACT>
__global__ __launch_bounds__(kFewWaves * 64) void few_rows_kernel(TileArgs a) {
  constexpr bool GLU = ACT == MEP_ACT_SILU_GLU;
  constexpr int COLS = GLU ? 16 : 32;
  constexpr int STEP = FP8 ? 128 : 32, AHEAD = FP8 ? 2 : 4;
  constexpr int SIZE = FP8 ? 1 : 2;
  __shared__ f32x4 join[kFewWaves][2][kWave];
  extern __shared__ int32_t first[];
  const int lane = threadIdx.x & 63, wave = first_lane(threadIdx.x >> 6);
  const int g = lane >> 4, r16 = lane & 15;
  count_row_tiles(a, kFewRows, first);
  const int col_tiles = (a.cols + COLS - 1) / COLS;
  const int64_t tiles = (int64_t)first[a.E] * col_tiles;
  const int depth = a.depth, blocks = depth / 128;
  const int steps = (depth + STEP - 1) / STEP;
  const int k0 = (int)((int64_t)steps * wave / kFewWaves);
  const int k1 = (int)((int64_t)steps * (wave + 1) / kFewWaves);

  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const Place at = find_tile(a, first, kFewRows, col_tiles, tile);
    const int64_t xr = at.row0 + min(at.m * kFewRows + r16, at.seg - 1);
    const unsigned char* px = a.b + xr * depth * SIZE;
    int wr[2];
    const unsigned char* pw[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int c = min(at.n * COLS + (GLU ? 0 : f * 16) + r16, a.cols - 1);
      wr[f] = GLU && f ? a.cols + c : c;
      pw[f] = a.a + ((int64_t)at.e * a.Nz + wr[f]) * depth * SIZE;
    }
    f32x4 acc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
    for (int k = k0; k < k1; k += AHEAD) {
      if constexpr (FP8) {
        i32x8 x[AHEAD], w[2][AHEAD];
        float sx[AHEAD], sw[2][AHEAD];
        auto get = [&](const unsigned char* p, int kk) {
          const u32x4 lo = *reinterpret_cast<const u32x4*>(p + (int64_t)kk * 128 + g * 32);
          const u32x4 hi = *reinterpret_cast<const u32x4*>(p + (int64_t)kk * 128 + g * 32 + 16);
          return __builtin_bit_cast(i32x8,
                                    __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        };
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          const int kk = min(k + u, k1 - 1);
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            w[f][u] = get(pw[f], kk);
            sw[f][u] = a.a_scales[((int64_t)at.e * (a.Nz / 128) + wr[f] / 128) * blocks + kk];
          }
          x[u] = get(px, kk);
          sx[u] = a.b_scales[xr * blocks + kk];
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                w[f][u], x[u], f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
            // all 16 weight rows lie in one block of 128
            const float sc = k + u < k1 ? sw[f][u] * sx[u] : 0.0f;
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[f][q] = k + u < k1 ? fmaf(p[q], sc, acc[f][q]) : acc[f][q];
          }
        }
      } else {
        u32x4 x[AHEAD], w[2][AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          const int kk = (k + u) * 32 + g * 8;
          const int64_t at_k = (int64_t)min(kk, depth - 8) * 2;
#pragma unroll
          for (int f = 0; f < 2; ++f) w[f][u] = *reinterpret_cast<const u32x4*>(pw[f] + at_k);
          x[u] = *reinterpret_cast<const u32x4*>(px + at_k);
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          const bool in = k + u < k1 && (k + u) * 32 + g * 8 < depth;
          const bf16x8 xv = __builtin_bit_cast(bf16x8, in ? x[u] : zero4());
#pragma unroll
          for (int f = 0; f < 2; ++f)
            acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, in ? w[f][u] : zero4()), xv, acc[f], 0, 0, 0);
        }
      }
    }
    join[wave][0][lane] = acc[0];
    join[wave][1][lane] = acc[1];
    __syncthreads();
    // gated: one wave has both halves; otherwise a wave for each fragment
    if (wave < (GLU ? 1 : 2)) {
      const int f = GLU ? 0 : wave;
      f32x4 z = join[0][f][lane], up = join[0][1][lane];
#pragma unroll
      for (int q = 1; q < kFewWaves; ++q) {
        z += join[q][f][lane];
        if (GLU) up += join[q][1][lane];
      }
      const int r = at.m * kFewRows + r16, col = at.n * COLS + f * 16 + g * 4;
      if (r < at.seg && col < a.cols) {
        const int64_t row = at.row0 + r;
        if (a.bias) {
          const float* b = a.bias + (int64_t)at.e * a.Nz + col;
          z += *reinterpret_cast<const f32x4*>(b);
          if (GLU) up += *reinterpret_cast<const f32x4*>(b + a.cols);
        }
        if (a.z) {
          uint16_t* zp = a.z + row * a.Nz + col;
          *reinterpret_cast<u32x2*>(zp) =
              u32x2{pack_bf16_rne(z[0], z[1]), pack_bf16_rne(z[2], z[3])};
          if (GLU)
            *reinterpret_cast<u32x2*>(zp + a.cols) =
                u32x2{pack_bf16_rne(up[0], up[1]), pack_bf16_rne(up[2], up[3])};
        }
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = activate<ACT>(z[q], up[q]);
        if (a.residual) {
          const u32x2 res = *reinterpret_cast<const u32x2*>(a.residual + row * a.cols + col);
          v[0] += bf16_lo(res[0]); v[1] += bf16_hi(res[0]);
          v[2] += bf16_lo(res[1]); v[3] += bf16_hi(res[1]);
        }
        *reinterpret_cast<u32x2*>(a.out + row * a.cols + col) =
            u32x2{pack_bf16_rne(v[0], v[1]), pack_bf16_rne(v[2], v[3])};
      }
    }
    __syncthreads();
  }
}

// ---- gradient before the activation, and the bias' gradient -----------------

// A block takes rows of a segment and 512 columns of grad_y (8 a lane) at a time:
// grad_z in bf16, and, where the bias wants it, the column sums of the unrounded
// grad_z over those rows, 128 then.  bf16 is the type of the products grad_z goes
// into: their error grows from 0.0017 of the norm, the results' own rounding, to
// 0.0023, and fp32 operands would take twice the products.  Without a bias, 32 rows:
// smaller blocks fill the CUs more evenly (16384 rows of 2 x 2048 gated columns, 335
// MB: 97 us; 64 rows 107, 128 rows 112).  Few rows are bound by the loads that follow
// one another, so 8 waves share them (602 rows of 520 columns 7.8 us; 4 waves 12.3).
constexpr int kGradZWaves = 8;

// Rows a block takes.
__host__ __device__ constexpr int grad_z_rows(bool bias) { return bias ? kSegRows : 32; }

template <int ACT>
__global__ __launch_bounds__(kGradZWaves * 64) void grad_z_kernel(LinearBackwardArgs a) {
  constexpr bool GLU = ACT == MEP_ACT_SILU_GLU;
  __shared__ float part[kGradZWaves][GLU ? 2 : 1][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int rows = grad_z_rows(a.grad_bias), share = rows / kGradZWaves;
  for (int64_t blk = blockIdx.x; blk * rows < a.cap; blk += gridDim.x) {
    const int64_t r0 = blk * rows;
    // the end of the segment that r0 lies in (segments may be in any order): 256
    // experts at a time, so that few loads follow one another (whole backward, 64
    // tokens over 1024 experts of 128 x 128: 43 us, 64 at a time 50)
    constexpr int GROUPS = 4;
    int64_t end = r0;
    for (int e0 = 0; e0 < a.E && end == r0; e0 += GROUPS * kWave) {
      int64_t from[GROUPS], to[GROUPS];
#pragma unroll
      for (int u = 0; u < GROUPS; ++u) {
        const int e = min(e0 + u * kWave + lane, a.E - 1);
        from[u] = a.offsets[e];
        to[u] = from[u] + max(a.counts[e], 0);
      }
#pragma unroll
      for (int u = 0; u < GROUPS; ++u) {
        const uint64_t in = ballot(from[u] >= 0 && from[u] <= r0 && r0 < to[u]);
        if (in != 0) end = r0 + lane_value((int)(min(to[u], a.cap) - r0), __builtin_ctzll(in));
      }
    }
    const int col = (blockIdx.y * 64 + lane) * 8;
    float s0[8], s1[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) s0[q] = s1[q] = 0.0f;
    if (col < a.N) {
      const uint16_t* gy = reinterpret_cast<const uint16_t*>(a.grad_y);
      const uint16_t* z = reinterpret_cast<const uint16_t*>(a.z);
      uint16_t* gz = reinterpret_cast<uint16_t*>(a.grad_z);
      const int64_t stop = min(end, r0 + (wave + 1) * share);
      // AHEAD rows' loads in flight: one at a time, a wave waits 16 times
      constexpr int AHEAD = ACT == MEP_ACT_NONE ? 8 : 4;
      for (int64_t r1 = r0 + wave * share; r1 < stop; r1 += AHEAD) {
        u32x4 gq[AHEAD], zq[AHEAD], uq[AHEAD];
#pragma unroll
        for (int t = 0; t < AHEAD; ++t) {
          const int64_t r = min(r1 + t, stop - 1);
          gq[t] = *reinterpret_cast<const u32x4*>(gy + r * a.N + col);
          zq[t] = uq[t] = zero4();
          if (ACT != MEP_ACT_NONE) zq[t] = *reinterpret_cast<const u32x4*>(z + r * a.Nz + col);
          if (GLU) uq[t] = *reinterpret_cast<const u32x4*>(z + r * a.Nz + a.N + col);
        }
#pragma unroll
        for (int t = 0; t < AHEAD; ++t) {
          const int64_t r = r1 + t;
          if (r >= stop) break;
          float d[8], du[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float g = q & 1 ? bf16_hi(gq[t][q >> 1]) : bf16_lo(gq[t][q >> 1]);
            const float v = q & 1 ? bf16_hi(zq[t][q >> 1]) : bf16_lo(zq[t][q >> 1]);
            const float u = q & 1 ? bf16_hi(uq[t][q >> 1]) : bf16_lo(uq[t][q >> 1]);
            du[q] = 0.0f;
            if (ACT == MEP_ACT_GELU) {
              d[q] = g * (0.5f * (1.0f + erff(v * 0.70710678118654752f)) +
                          v * expf(-0.5f * v * v) * 0.39894228040143268f);
            } else if (ACT == MEP_ACT_SILU || GLU) {
              const float sg = 1.0f / (1.0f + expf(-v));
              const float slope = sg * (1.0f + v * (1.0f - sg));
              d[q] = GLU ? g * u * slope : g * slope;
              if (GLU) du[q] = g * (v * sg);
            } else {
              d[q] = g;
            }
            s0[q] += d[q];
            s1[q] += du[q];
          }
          if (ACT != MEP_ACT_NONE)
            *reinterpret_cast<u32x4*>(gz + r * a.Nz + col) =
                u32x4{pack_bf16_rne(d[0], d[1]), pack_bf16_rne(d[2], d[3]),
                      pack_bf16_rne(d[4], d[5]), pack_bf16_rne(d[6], d[7])};
          if (GLU)
            *reinterpret_cast<u32x4*>(gz + r * a.Nz + a.N + col) =
                u32x4{pack_bf16_rne(du[0], du[1]), pack_bf16_rne(du[2], du[3]),
                      pack_bf16_rne(du[4], du[5]), pack_bf16_rne(du[6], du[7])};
        }
      }
    }
    if (!a.grad_bias) continue;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      part[wave][0][lane * 8 + q] = s0[q];
      if (GLU) part[wave][GLU][lane * 8 + q] = s1[q];
    }
    __syncthreads();
    const int c = threadIdx.x, n = blockIdx.y * 512 + c;
    static_assert(kGradZWaves * 64 == 512, "a thread a column");
    if (n < a.N) {
      float* out = a.part + blk * a.Nz + n;
#pragma unroll
      for (int h = 0; h < (GLU ? 2 : 1); ++h) {
        float s = part[0][h][c];
#pragma unroll
        for (int w = 1; w < kGradZWaves; ++w) s += part[w][h][c];
        out[h * a.N] = s;
      }
    }
    __syncthreads();
  }
}

// The blocks' column sums of one segment, added up in order.
__global__ __launch_bounds__(256) void grad_bias_kernel(LinearBackwardArgs a) {
  const int n = blockIdx.x * 256 + threadIdx.x, e = blockIdx.y;
  if (n >= a.Nz) return;
  const int64_t off = a.offsets[e];
  const int64_t rows = off < 0 ? 0 : min((int64_t)max(a.counts[e], 0), a.cap - off);
  double s = 0.0;
  for (int64_t b = off / kSegRows; b * kSegRows < off + rows; ++b)
    s += (double)a.part[b * a.Nz + n];
  a.grad_bias[(int64_t)e * a.Nz + n] = (float)s;
}

// ---- launches ---------------------------------------------------------------

constexpr int kCus = 256;

// An upper bound of the row tiles that num_rows rows in E segments make.
int64_t row_tiles_bound(int64_t num_rows, int E, int bm) {
  return num_rows / bm + std::min<int64_t>(num_rows, E);
}

// `rows`: rows expected in all segments (forward, grad_x).
template <class T>
int64_t count_tiles(const TileArgs& a, Mode mode, int64_t rows) {
  const int64_t cols = (a.cols + T::COLS - 1) / T::COLS;
  return cols * (mode == kGradW ? (int64_t)a.E * ((a.rows + T::BM - 1) / T::BM)
                                : row_tiles_bound(rows, a.E, T::BM));
}

template <Mode MODE, bool FP8, int ACT, int TN, int TM, int PER_CU>
void run_tiles(const TileArgs& a, int64_t rows, hipStream_t s) {
  using T = Tile<MODE, FP8, ACT, 2, 4, TN, TM>;
  const int64_t tiles = count_tiles<T>(a, MODE, rows);
  const size_t lds = MODE == kGradW ? 0 : (size_t)(a.E + 1) * sizeof(int32_t);
  const unsigned grid =
      (unsigned)std::max<int64_t>(1, std::min<int64_t>(tiles, (int64_t)PER_CU * kCus));
  tile_kernel<MODE, FP8, ACT, 2, 4, TN, TM, PER_CU><<<grid, T::THREADS, lds, s>>>(a);
}

// Tiles of 256 x 256, one block a CU, or of 128 x 128, two, which have twice the
// traffic for a product but four times the tiles, and waste less on short
// segments.  Measured, large / small (us): 2048 -> 7168, one segment, 1000 rows,
// 116 large tiles, 47.3 / 33.0; 1536 rows, 168 tiles, 51.1 / 62.0.  7168 -> 2048
// gated, 64 experts, 2 rows each 586 / 581, 32 rows 654 / 632; 256 experts, 64
// rows 2617 / 2649 (small by the rule, 1% the slower), 128 rows 2854 / 4266.
template <Mode MODE, bool FP8, int ACT>
void run_sized(const TileArgs& a, int64_t rows, hipStream_t s) {
  using Large = Tile<MODE, FP8, ACT, 2, 4, 8, 4>;
  const bool enough = count_tiles<Large>(a, MODE, rows) >= 144;
  const bool long_segments = MODE == kGradW || rows > 64 * std::min<int64_t>(a.E, rows);
  if (enough && long_segments) run_tiles<MODE, FP8, ACT, 8, 4, 1>(a, rows, s);
  else run_tiles<MODE, FP8, ACT, 4, 2, 2>(a, rows, s);
}

// Few rows: up to 16 an expert where small tiles are no more than the CUs.
// Measured (us, tiles / few rows): one token over 8 experts of 4096 x 7168, 256
// tiles, 97 and 94 (E4M3 36.9 and 41.1, where the rule, made for both types, takes
// the slower), 2 experts of 1024 x 7168 35.5 and 19.4 (27.0 and 12.2), one of 7168 x
// 2048 13.3 and 8.4 (11.0 and 5.7); 16 tokens over 64 experts of 4096 x 7168, 2048
// tiles, 584 and 658; 33 rows of one expert 15.5 and 15.6.
template <bool FP8, int ACT>
void run_forward(const TileArgs& a, int64_t rows, hipStream_t s) {
  using Small = Tile<kForward, FP8, ACT, 2, 4, 4, 2>;
  if (rows <= kFewRows * std::min<int64_t>(a.E, rows) &&
      count_tiles<Small>(a, kForward, rows) <= kCus) {
    constexpr int COLS = ACT == MEP_ACT_SILU_GLU ? 16 : 32;
    const int64_t tiles =
        (a.cols + COLS - 1) / COLS * row_tiles_bound(rows, a.E, kFewRows);
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(tiles, 4 * kCus));
    few_rows_kernel<FP8, ACT>
        <<<grid, kFewWaves * 64, (size_t)(a.E + 1) * sizeof(int32_t), s>>>(a);
  } else {
    run_sized<kForward, FP8, ACT>(a, rows, s);
  }
}

template <bool FP8>
void run_forward(const TileArgs& t, int act, int64_t rows, hipStream_t s) {
  switch (act) {
    case MEP_ACT_NONE: run_forward<FP8, MEP_ACT_NONE>(t, rows, s); break;
    case MEP_ACT_GELU: run_forward<FP8, MEP_ACT_GELU>(t, rows, s); break;
    case MEP_ACT_SILU: run_forward<FP8, MEP_ACT_SILU>(t, rows, s); break;
    default: run_forward<FP8, MEP_ACT_SILU_GLU>(t, rows, s);
  }
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
  if (a.cap == 0) return hipSuccess;
  TileArgs t{};
  t.a = (const unsigned char*)a.w;
  t.b = (const unsigned char*)a.x;
  t.a_scales = a.w_scales;
  t.b_scales = a.x_scales;
  t.bias = a.bias;
  t.residual = (const uint16_t*)a.residual;
  t.out = (uint16_t*)a.y;
  t.z = (uint16_t*)a.z;
  t.counts = a.counts;
  t.offsets = a.offsets;
  t.cap = a.cap;
  t.E = a.E;
  t.cols = a.N;
  t.depth = a.K;
  t.Nz = a.Nz;
  const int64_t rows = std::min(a.num_rows, a.cap);
  if (a.quant != MEP_QUANT_NONE) run_forward<true>(t, a.act, rows, s);
  else run_forward<false>(t, a.act, rows, s);
  return hipGetLastError();
}

hipError_t launch_linear_backward(const LinearBackwardArgs& a, hipStream_t s) {
  if (a.cap > 0 && (a.act != MEP_ACT_NONE || a.grad_bias)) {
    const int rows = grad_z_rows(a.grad_bias);
    const int64_t blocks = (a.cap + rows - 1) / rows;
    const dim3 grid((unsigned)std::min<int64_t>(blocks, 1 << 16), (unsigned)((a.N + 511) / 512));
    switch (a.act) {
      case MEP_ACT_NONE: grad_z_kernel<MEP_ACT_NONE><<<grid, kGradZWaves * 64, 0, s>>>(a); break;
      case MEP_ACT_GELU: grad_z_kernel<MEP_ACT_GELU><<<grid, kGradZWaves * 64, 0, s>>>(a); break;
      case MEP_ACT_SILU: grad_z_kernel<MEP_ACT_SILU><<<grid, kGradZWaves * 64, 0, s>>>(a); break;
      default: grad_z_kernel<MEP_ACT_SILU_GLU><<<grid, kGradZWaves * 64, 0, s>>>(a);
    }
  }
  if (a.grad_bias)
    grad_bias_kernel<<<dim3((unsigned)((a.Nz + 255) / 256), (unsigned)a.E), 256, 0, s>>>(a);
  TileArgs t{};
  t.counts = a.counts;
  t.offsets = a.offsets;
  t.cap = a.cap;
  t.E = a.E;
  t.Nz = a.Nz;
  t.b = (const unsigned char*)a.grad_z;
  t.cols = a.K;
  if (a.grad_x && a.cap > 0) {
    t.a = (const unsigned char*)a.w;
    t.out = (uint16_t*)a.grad_x;
    t.depth = a.Nz;
    run_sized<kGradX, false, MEP_ACT_NONE>(t, std::min(a.num_rows, a.cap), s);
  }
  if (a.grad_w) {
    t.a = (const unsigned char*)a.x;
    t.out = (uint16_t*)a.grad_w;
    t.rows = a.Nz;
    run_sized<kGradW, false, MEP_ACT_NONE>(t, 0, s);
  }
  return hipGetLastError();
}

}  // namespace mep
