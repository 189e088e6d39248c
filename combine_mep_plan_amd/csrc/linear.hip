// Experts' products over expert-major segments, and their gradients.
//
// Three products share one tile kernel.  In each, the columns of the output are
// the rows of MFMA's first operand, so that a lane ends up with four
// consecutive columns of one output row and stores them together:
//   forward   z[r, n]  = sum_k w[e, n, k]  x[r, k]      r in segment e
//   grad_x    dx[r, k] = sum_n w[e, n, k] dz[r, n]
//   grad_w    dw[e, n, k] = sum_r x[r, k] dz[r, n]
// An operand whose summed index is contiguous in memory is "direct", the others
// (w in grad_x, both in grad_w) are turned around on their way into LDS.
//
// LDS holds tiles of 128 rows by 64 values of the summed index, 128 bytes a
// row, its eight 16-byte units exchanged by the low bits of the row so that the
// MFMA operand reads (16 rows, one unit each) touch every bank once.
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

constexpr int kTile = 128;      // rows and columns of an output tile
constexpr int kThreads = 256;

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

// Rows of segment e that exist (rows past cap_em are left out).
__device__ __forceinline__ int segment_rows(const TileArgs& a, int e) {
  const int64_t off = a.offsets[e], left = a.cap - off;
  const int c = a.counts[e];
  return off < 0 || left <= 0 || c <= 0 ? 0 : left < c ? (int)left : c;
}

__device__ __forceinline__ u32x4 zero4() { return u32x4{0, 0, 0, 0}; }

__device__ __forceinline__ int swizzle(int row, int unit) { return unit ^ (row & 7); }

__device__ __forceinline__ float silu(float z) { return z / (1.0f + expf(-z)); }
__device__ __forceinline__ float gelu(float z) {
  return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
}

// Columns of the weight that LDS row r of the tile at column tile n holds: with a
// gated activation every 32 rows are 16 gate rows and the 16 rows they gate.
template <bool GLU>
__device__ __forceinline__ int weight_row(int n, int r, int cols) {
  if (!GLU) return min(n * kTile + r, cols - 1);
  const int c = min(n * (kTile / 2) + (r >> 5) * 16 + (r & 15), cols - 1);
  return (r & 16) ? cols + c : c;
}

template <Mode MODE, bool FP8, int ACT>
__global__ __launch_bounds__(kThreads) void tile_kernel(TileArgs a) {
  constexpr bool GLU = MODE == kForward && ACT == MEP_ACT_SILU_GLU;
  constexpr int kVals = FP8 ? 128 : 64;      // summed values a step
  constexpr int kUnit = FP8 ? 16 : 8;        // values in 16 bytes
  constexpr int kSize = FP8 ? 1 : 2;
  constexpr int kCols = GLU ? kTile / 2 : kTile;  // output columns a tile
  __shared__ u32x4 la[kTile * 8], lb[kTile * 8];
  extern __shared__ int32_t first[];         // [E+1]: row tiles before each expert

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn = wave & 1, wm = wave >> 1;   // the wave's 64 x 64 quarter
  const int col_tiles = (a.cols + kCols - 1) / kCols;

  // row tiles before each expert: the tiles of a launch follow the counts
  if (MODE != kGradW) {
    if (tid < kWave) {
      int base = 0;
      for (int e0 = 0; e0 < a.E; e0 += kWave) {
        const int e = e0 + tid;
        const int n = e < a.E ? (segment_rows(a, e) + kTile - 1) / kTile : 0;
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
  const int row_tiles = MODE == kGradW ? (a.rows + kTile - 1) / kTile : 0;
  const int64_t tiles = MODE == kGradW ? (int64_t)a.E * row_tiles * col_tiles
                                       : (int64_t)first[a.E] * col_tiles;

  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int n = (int)(tile % col_tiles);
    int e, m;
    if (MODE == kGradW) {
      const int64_t q = tile / col_tiles;
      e = (int)(q / row_tiles);
      m = (int)(q % row_tiles);
    } else {
      const int q = (int)(tile / col_tiles);
      int lo = 0, hi = a.E;  // the last expert with first[e] <= q
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= q) lo = mid; else hi = mid;
      }
      e = lo;
      m = q - first[e];
    }
    const int seg = segment_rows(a, e);
    const int64_t row0 = a.offsets[e];
    const int depth = MODE == kGradW ? seg : a.depth;

    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    for (int k0 = 0; k0 < depth; k0 += kVals) {
      __syncthreads();
      // 128 rows x 8 units of each operand
      if (MODE == kForward) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = tid + i * kThreads, r = c >> 3, u = c & 7;
          const int k = k0 + u * kUnit;
          const int wr = weight_row<GLU>(n, r, a.cols);
          la[r * 8 + swizzle(r, u)] =
              k < depth ? *reinterpret_cast<const u32x4*>(
                              a.a + (((int64_t)e * a.Nz + wr) * depth + k) * kSize)
                        : zero4();
        }
      } else {
        // 64 summed values x 16 units of 8 columns, turned around
        const int ld = a.cols;
        const int64_t r0 = MODE == kGradX ? (int64_t)e * a.Nz : row0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = tid + i * kThreads, k = c >> 4, u = c & 15;
          const int col = n * kTile + u * 8;
          u32x4 v = zero4();
          if (k0 + k < depth && col < a.cols)
            v = *reinterpret_cast<const u32x4*>(a.a + ((r0 + k0 + k) * ld + col) * 2);
          uint16_t* l16 = reinterpret_cast<uint16_t*>(la);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int r = u * 8 + q;
            l16[(r * 8 + swizzle(r, k >> 3)) * 8 + (k & 7)] =
                (uint16_t)(v[q >> 1] >> ((q & 1) * 16));
          }
        }
      }
      if (MODE != kGradW) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = tid + i * kThreads, r = c >> 3, u = c & 7;
          const int k = k0 + u * kUnit;
          const int64_t xr = row0 + min(m * kTile + r, seg - 1);
          lb[r * 8 + swizzle(r, u)] =
              k < depth ? *reinterpret_cast<const u32x4*>(a.b + (xr * depth + k) * kSize)
                        : zero4();
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = tid + i * kThreads, k = c >> 4, u = c & 15;
          const int col = m * kTile + u * 8;
          u32x4 v = zero4();
          if (k0 + k < depth && col < a.rows)
            v = *reinterpret_cast<const u32x4*>(a.b + ((row0 + k0 + k) * a.rows + col) * 2);
          uint16_t* l16 = reinterpret_cast<uint16_t*>(lb);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const int r = u * 8 + q;
            l16[(r * 8 + swizzle(r, k >> 3)) * 8 + (k & 7)] =
                (uint16_t)(v[q >> 1] >> ((q & 1) * 16));
          }
        }
      }
      __syncthreads();

      const int g = lane >> 4, r16 = lane & 15;
      if (FP8) {
        // one MFMA sums a whole scale block; the blocks join in fp32
        i32x8 av[4], bv[4];
        float sb[4];
        const int kb = k0 / 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ra = wn * 64 + i * 16 + r16, rb = wm * 64 + i * 16 + r16;
          const u32x4 a0 = la[ra * 8 + swizzle(ra, 2 * g)], a1 = la[ra * 8 + swizzle(ra, 2 * g + 1)];
          const u32x4 b0 = lb[rb * 8 + swizzle(rb, 2 * g)], b1 = lb[rb * 8 + swizzle(rb, 2 * g + 1)];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            av[i][q] = (int)a0[q]; av[i][q + 4] = (int)a1[q];
            bv[i][q] = (int)b0[q]; bv[i][q + 4] = (int)b1[q];
          }
          const int64_t xr = row0 + min(m * kTile + rb, seg - 1);
          sb[i] = a.b_scales[xr * (depth / 128) + kb];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // 16 columns of a tile lie in one block of 128 weight rows
          const int wr = weight_row<GLU>(n, wn * 64 + i * 16, a.cols);
          const float sa =
              a.a_scales[((int64_t)e * (a.Nz / 128) + wr / 128) * (depth / 128) + kb];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                av[i], bv[j], f32x4{0, 0, 0, 0}, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[i][j][q] = fmaf(p[q], sa * sb[j], acc[i][j][q]);
          }
        }
      } else {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          bf16x8 av[4], bv[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int ra = wn * 64 + i * 16 + r16, rb = wm * 64 + i * 16 + r16;
            av[i] = __builtin_bit_cast(bf16x8, la[ra * 8 + swizzle(ra, s * 4 + g)]);
            bv[i] = __builtin_bit_cast(bf16x8, lb[rb * 8 + swizzle(rb, s * 4 + g)]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[i], bv[j], acc[i][j], 0, 0, 0);
        }
      }
    }

    // a lane has 4 consecutive columns (4 * (lane / 16) of 16) of row lane % 16
    const int c4 = (lane >> 4) * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = m * kTile + wm * 64 + j * 16 + (lane & 15);
      if (r >= (MODE == kGradW ? a.rows : seg)) continue;
      const int64_t orow = MODE == kGradW ? (int64_t)e * a.rows + r : row0 + r;
#pragma unroll
      for (int i = 0; i < 4; i += GLU ? 2 : 1) {
        const int col = GLU ? n * kCols + (wn * 4 + i) * 8 + c4 : n * kCols + wn * 64 + i * 16 + c4;
        if (col >= a.cols) continue;
        float v[4];
        if (MODE == kForward) {
          f32x4 z = acc[i][j], up = f32x4{0, 0, 0, 0};
          if (GLU) up = acc[i + (GLU ? 1 : 0)][j];
          if (a.bias) {
            const float* b = a.bias + (int64_t)e * a.Nz + col;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              z[q] += b[q];
              if (GLU) up[q] += b[a.cols + q];
            }
          }
          if (a.z) {
            uint16_t* zp = a.z + orow * a.Nz + col;
            *reinterpret_cast<u32x2*>(zp) =
                u32x2{pack_bf16_rne(z[0], z[1]), pack_bf16_rne(z[2], z[3])};
            if (GLU)
              *reinterpret_cast<u32x2*>(zp + a.cols) =
                  u32x2{pack_bf16_rne(up[0], up[1]), pack_bf16_rne(up[2], up[3])};
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            v[q] = ACT == MEP_ACT_GELU   ? gelu(z[q])
                   : ACT == MEP_ACT_SILU ? silu(z[q])
                   : GLU                 ? silu(z[q]) * up[q]
                                         : z[q];
          if (a.residual) {
            const u32x2 res = *reinterpret_cast<const u32x2*>(a.residual + orow * a.cols + col);
            v[0] += bf16_lo(res[0]); v[1] += bf16_hi(res[0]);
            v[2] += bf16_lo(res[1]); v[3] += bf16_hi(res[1]);
          }
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = acc[i][j][q];
        }
        *reinterpret_cast<u32x2*>(a.out + orow * a.cols + col) =
            u32x2{pack_bf16_rne(v[0], v[1]), pack_bf16_rne(v[2], v[3])};
      }
    }
  }
}

// ---- gradient before the activation, and the bias' gradient -----------------

// A block takes 128 rows of a segment and 512 columns of grad_y (8 a lane, 32
// rows a wave) at a time: grad_z in bf16, and, where the bias wants it, the
// column sums of the unrounded grad_z over those rows.
template <int ACT>
__global__ __launch_bounds__(256) void grad_z_kernel(LinearBackwardArgs a) {
  constexpr bool GLU = ACT == MEP_ACT_SILU_GLU;
  __shared__ float part[4][2][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int turn = 0; (blockIdx.x + (int64_t)turn * gridDim.x) * kSegRows < a.cap; ++turn) {
    const int64_t blk = blockIdx.x + (int64_t)turn * gridDim.x, r0 = blk * kSegRows;
    int lo = 0, hi = a.E;  // the last segment that starts at or before r0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.offsets[mid] <= r0) lo = mid; else hi = mid;
    }
    int64_t end = min((int64_t)a.offsets[lo] + max(a.counts[lo], 0), a.cap);
    if (a.offsets[lo] > r0) end = 0;
    const int col = (blockIdx.y * 64 + lane) * 8;
    float s0[8], s1[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) s0[q] = s1[q] = 0.0f;
    if (col < a.N) {
      const uint16_t* gy = reinterpret_cast<const uint16_t*>(a.grad_y);
      const uint16_t* z = reinterpret_cast<const uint16_t*>(a.z);
      uint16_t* gz = reinterpret_cast<uint16_t*>(a.grad_z);
      const int64_t stop = min(end, r0 + wave * 32 + 32);
      for (int64_t r = r0 + wave * 32; r < stop; ++r) {
        const u32x4 gq = *reinterpret_cast<const u32x4*>(gy + r * a.N + col);
        u32x4 zq = zero4(), uq = zero4();
        if (ACT != MEP_ACT_NONE) zq = *reinterpret_cast<const u32x4*>(z + r * a.Nz + col);
        if (GLU) uq = *reinterpret_cast<const u32x4*>(z + r * a.Nz + a.N + col);
        float d[8], du[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float g = q & 1 ? bf16_hi(gq[q >> 1]) : bf16_lo(gq[q >> 1]);
          const float v = q & 1 ? bf16_hi(zq[q >> 1]) : bf16_lo(zq[q >> 1]);
          const float u = q & 1 ? bf16_hi(uq[q >> 1]) : bf16_lo(uq[q >> 1]);
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
              u32x4{pack_bf16_rne(d[0], d[1]), pack_bf16_rne(d[2], d[3]), pack_bf16_rne(d[4], d[5]),
                    pack_bf16_rne(d[6], d[7])};
        if (GLU)
          *reinterpret_cast<u32x4*>(gz + r * a.Nz + a.N + col) =
              u32x4{pack_bf16_rne(du[0], du[1]), pack_bf16_rne(du[2], du[3]),
                    pack_bf16_rne(du[4], du[5]), pack_bf16_rne(du[6], du[7])};
      }
    }
    if (!a.grad_bias) continue;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      part[wave][0][lane * 8 + q] = s0[q];
      part[wave][1][lane * 8 + q] = s1[q];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 512; c += 256) {
      const int n = blockIdx.y * 512 + c;
      if (n >= a.N) continue;
      float* out = a.part + blk * a.Nz + n;
      out[0] = part[0][0][c] + part[1][0][c] + part[2][0][c] + part[3][0][c];
      if (GLU) out[a.N] = part[0][1][c] + part[1][1][c] + part[2][1][c] + part[3][1][c];
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

constexpr int kBlocks = 1024;  // resident blocks of the tile kernel: 4 on each of 256 CUs

unsigned grid_for(int64_t tiles) {
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>(tiles, kBlocks));
}

// An upper bound of the row tiles that num_rows rows in E segments make.
int64_t row_tiles_bound(int64_t num_rows, int E) {
  return num_rows / kTile + std::min<int64_t>(num_rows, E) + 1;
}

template <Mode MODE, bool FP8, int ACT>
void run_tiles(const TileArgs& a, int64_t tiles, hipStream_t s) {
  const size_t lds = MODE == kGradW ? 0 : (size_t)(a.E + 1) * sizeof(int32_t);
  tile_kernel<MODE, FP8, ACT><<<grid_for(tiles), kThreads, lds, s>>>(a);
}

template <bool FP8>
void run_forward(const TileArgs& t, int act, int64_t row_tiles, hipStream_t s) {
  const int64_t full = row_tiles * ((t.cols + kTile - 1) / kTile);
  switch (act) {
    case MEP_ACT_NONE: run_tiles<kForward, FP8, MEP_ACT_NONE>(t, full, s); break;
    case MEP_ACT_GELU: run_tiles<kForward, FP8, MEP_ACT_GELU>(t, full, s); break;
    case MEP_ACT_SILU: run_tiles<kForward, FP8, MEP_ACT_SILU>(t, full, s); break;
    default: run_tiles<kForward, FP8, MEP_ACT_SILU_GLU>(t, 2 * full, s);
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
  const int64_t row_tiles = row_tiles_bound(std::min(a.num_rows, a.cap), a.E);
  if (a.quant != MEP_QUANT_NONE) run_forward<true>(t, a.act, row_tiles, s);
  else run_forward<false>(t, a.act, row_tiles, s);
  return hipGetLastError();
}

hipError_t launch_linear_backward(const LinearBackwardArgs& a, hipStream_t s) {
  if (a.cap > 0 && (a.act != MEP_ACT_NONE || a.grad_bias)) {
    const int64_t blocks = (a.cap + kSegRows - 1) / kSegRows;
    const dim3 grid((unsigned)std::min<int64_t>(blocks, 1 << 16), (unsigned)((a.N + 511) / 512));
    switch (a.act) {
      case MEP_ACT_NONE: grad_z_kernel<MEP_ACT_NONE><<<grid, 256, 0, s>>>(a); break;
      case MEP_ACT_GELU: grad_z_kernel<MEP_ACT_GELU><<<grid, 256, 0, s>>>(a); break;
      case MEP_ACT_SILU: grad_z_kernel<MEP_ACT_SILU><<<grid, 256, 0, s>>>(a); break;
      default: grad_z_kernel<MEP_ACT_SILU_GLU><<<grid, 256, 0, s>>>(a);
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
  const int64_t col_tiles = (a.K + kTile - 1) / kTile;
  if (a.grad_x && a.cap > 0) {
    t.a = (const unsigned char*)a.w;
    t.out = (uint16_t*)a.grad_x;
    t.depth = a.Nz;
    const int64_t row_tiles = row_tiles_bound(std::min(a.num_rows, a.cap), a.E);
    run_tiles<kGradX, false, MEP_ACT_NONE>(t, row_tiles * col_tiles, s);
  }
  if (a.grad_w) {
    t.a = (const unsigned char*)a.x;
    t.out = (uint16_t*)a.grad_w;
    t.rows = a.Nz;
    const int64_t row_tiles = (a.Nz + kTile - 1) / kTile;
    run_tiles<kGradW, false, MEP_ACT_NONE>(t, (int64_t)a.E * row_tiles * col_tiles, s);
  }
  return hipGetLastError();
}

}  // namespace mep
