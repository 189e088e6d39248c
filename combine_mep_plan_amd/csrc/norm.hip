// The norms before and after a block, fused with the block's gate and the scaled
// residual, and their gradients.
//
//   hat(u) = u,  u / sqrt(mean u^2 + eps),  or  (u - mean u) / sqrt(var u + eps)
//   v = hat_post(y) (o + w_post) + b_post
//   s = residual_scale x + block_scale g v
//   n = hat_pre(s) (o + w_pre) + b_pre
//
// A row stays in registers from its first load to its last store: 8 neighbouring
// values a thread (a unit; UPT units for long rows), so every byte moves once.  Rows of
// up to 1024 values belong to one wave, longer ones to a block of just as many waves as
// they fill; a block works on several rows and keeps the weights in registers.
#include <algorithm>
#include <type_traits>

#include "dev.h"
#include "mep_internal.h"

namespace mep {

namespace {

constexpr int kUnit = 8;           // values of a unit
constexpr int kMaxWaves = 16;      // of a block
constexpr int kCodeBlock = 128;    // columns that share an E4M3 scale

// ---- sums over a row --------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  const int u = __float_as_int(v);
  return v + __int_as_float(__builtin_amdgcn_update_dpp(u, u, CTRL, 0xf, 0xf, false));
}

// Over 16 lanes, in every lane: exchanges within 2 and 4 lanes, then the mirrored lane
// of 8 and of 16 (all lanes of a part agree by then, so a mirror is an exchange).
__device__ __forceinline__ float sum16(float v) {
  v = dpp_add<0xB1>(v);
  v = dpp_add<0x4E>(v);
  v = dpp_add<0x141>(v);
  return dpp_add<0x140>(v);
}

__device__ __forceinline__ float wave_sum(float v) {
  v = sum16(v);
  uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  u = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Sums over the lanes of a row, in a fixed order and the same in every lane.  Waves
// meet in LDS once a call: two buffers in turn, as the next call's barrier stands
// between a buffer's readers and its next writers.
template <bool WAVE>
struct RowSum {
  float4 (*lds)[kMaxWaves];
  int turn, waves;

  template <int N>
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    static_assert(N <= 4, "");
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (!WAVE) {
      float4 mine = make_float4(v[0], N > 1 ? v[N > 1 ? 1 : 0] : 0.0f,
                                N > 2 ? v[N > 2 ? 2 : 0] : 0.0f, N > 3 ? v[N > 3 ? 3 : 0] : 0.0f);
      if (lane_id() == 0) lds[turn][threadIdx.x / kWave] = mine;
      __syncthreads();
      const int w = lane_id() & (kMaxWaves - 1);
      float4 q = lds[turn][w];
      if (w >= waves) q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      v[0] = sum16(q.x);
      if (N > 1) v[N > 1 ? 1 : 0] = sum16(q.y);
      if (N > 2) v[N > 2 ? 2 : 0] = sum16(q.z);
      if (N > 3) v[N > 3 ? 3 : 0] = sum16(q.w);
      turn ^= 1;
    }
  }
};

// ---- units ------------------------------------------------------------------

template <class TL>
struct Raw;
template <>
struct Raw<uint16_t> {
  u32x4 q;
  __device__ __forceinline__ void load(const void* p, int64_t unit) {
    q = reinterpret_cast<const u32x4*>(p)[unit];
  }
  __device__ __forceinline__ float at(int i) const { return i & 1 ? bf16_hi(q[i / 2]) : bf16_lo(q[i / 2]); }
};
template <>
struct Raw<float> {
  u32x4 q[2];
  __device__ __forceinline__ void load(const void* p, int64_t unit) {
    q[0] = reinterpret_cast<const u32x4*>(p)[2 * unit];
    q[1] = reinterpret_cast<const u32x4*>(p)[2 * unit + 1];
  }
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(q[i / 4][i % 4]); }
};

__device__ __forceinline__ void store_unit(uint16_t*, void* p, int64_t unit, const float (&v)[kUnit]) {
  u32x4 q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = pack_bf16_rne(v[2 * i], v[2 * i + 1]);
  reinterpret_cast<u32x4*>(p)[unit] = q;
}
__device__ __forceinline__ void store_unit(float*, void* p, int64_t unit, const float (&v)[kUnit]) {
  float4* to = reinterpret_cast<float4*>(p) + 2 * unit;
  to[0] = make_float4(v[0], v[1], v[2], v[3]);
  to[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A vector's values at a unit; `none` where there is no vector, else plus `offset`.
__device__ __forceinline__ void load_vector(const float* p, int unit, float none, float offset,
                                            float (&v)[kUnit]) {
  if (p) {
    const float4* q = reinterpret_cast<const float4*>(p) + 2 * unit;
    const float4 a = q[0], b = q[1];
    v[0] = offset + a.x; v[1] = offset + a.y; v[2] = offset + a.z; v[3] = offset + a.w;
    v[4] = offset + b.x; v[5] = offset + b.y; v[6] = offset + b.z; v[7] = offset + b.w;
  } else {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) v[i] = none;
  }
}

// The gate's factor and its slope.
__device__ __forceinline__ float open_gate(float g, int sigmoid, float& slope) {
  if (!sigmoid) {
    slope = 1.0f;
    return g;
  }
  const float e = expf(-fabsf(g)), r = 1.0f / (1.0f + e);
  slope = e * r * r;
  return g < 0.0f ? e * r : r;
}

// A row's values as the norm of `kind` leaves them, in place, and the factor that does
// it.  Units that are not `on` hold 0 and stay so.
template <int UPT, bool WAVE>
__device__ __forceinline__ void norm_row(int kind, float (&v)[UPT][kUnit], const bool (&on)[UPT],
                                         float inv_h, float eps, RowSum<WAVE>& sum) {
  if (kind == MEP_NORM_NONE) return;
  float t[1] = {0.0f};
  if (kind == MEP_NORM_LAYER) {
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
      for (int i = 0; i < kUnit; ++i) t[0] += v[u][i];
    sum(t);
    const float mean = t[0] * inv_h;
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
      for (int i = 0; i < kUnit; ++i) v[u][i] = on[u] ? v[u][i] - mean : 0.0f;
    t[0] = 0.0f;
  }
#pragma unroll
  for (int u = 0; u < UPT; ++u)
#pragma unroll
    for (int i = 0; i < kUnit; ++i) t[0] = fmaf(v[u][i], v[u][i], t[0]);
  sum(t);
  const float r = 1.0f / sqrtf(fmaf(t[0], inv_h, eps));
#pragma unroll
  for (int u = 0; u < UPT; ++u)
#pragma unroll
    for (int i = 0; i < kUnit; ++i) v[u][i] *= r;
}

// ---- forward ----------------------------------------------------------------

// E4M3 codes of a block of 128 columns, which 16 lanes hold: scale = amax / 448, codes of
// the correctly rounded quotients.  The maximum is taken on the bits, where NaN is above
// everything, so a block with a NaN or an infinity in it is NaN throughout.
__device__ __forceinline__ u32x2 encode_unit(const float (&v)[kUnit], float& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kUnit; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  auto step = [&](auto ctrl) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, ctrl(), 0xf, 0xf, false));
  };
  step(std::integral_constant<int, 0xB1>{});
  step(std::integral_constant<int, 0x4E>{});
  step(std::integral_constant<int, 0x141>{});
  step(std::integral_constant<int, 0x140>{});
  scale = __uint_as_float(m) / 448.0f;
  float q[kUnit];
#pragma unroll
  for (int i = 0; i < kUnit; ++i) q[i] = scale == 0.0f ? 0.0f : v[i] / scale;
  return u32x2{pack_e4m3x4(q[0], q[1], q[2], q[3]), pack_e4m3x4(q[4], q[5], q[6], q[7])};
}

template <class TL, int UPT, bool WAVE>
__global__ __launch_bounds__(kMaxWaves * kWave) void norm_kernel(NormArgs a) {
  __shared__ float4 lds[2][kMaxWaves];
  const int lanes = WAVE ? kWave : blockDim.x, l = WAVE ? lane_id() : threadIdx.x;
  const int rows_here = WAVE ? blockDim.x / kWave : 1;
  const int units = a.H / kUnit;
  const float inv_h = 1.0f / (float)a.H;
  RowSum<WAVE> sum{lds, 0, (int)blockDim.x / kWave};
  bool on[UPT];
  int at[UPT];
  float wp[UPT][kUnit], bp[UPT][kUnit], wn[UPT][kUnit], bn[UPT][kUnit];
#pragma unroll
  for (int u = 0; u < UPT; ++u) {
    on[u] = u * lanes + l < units;
    at[u] = min(u * lanes + l, units - 1);
    load_vector(a.post_weight, at[u], 1.0f, a.offset, wp[u]);
    load_vector(a.post_bias, at[u], 0.0f, 0.0f, bp[u]);
    load_vector(a.pre_weight, at[u], 1.0f, a.offset, wn[u]);
    load_vector(a.pre_bias, at[u], 0.0f, 0.0f, bn[u]);
  }
  const int64_t step = (int64_t)gridDim.x * rows_here;
  for (int64_t t = (int64_t)blockIdx.x * rows_here + (WAVE ? threadIdx.x / kWave : 0); t < a.T;
       t += step) {
    const int64_t row = t * units;
    float v[UPT][kUnit];
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
      for (int i = 0; i < kUnit; ++i) v[u][i] = 0.0f;
    Raw<TL> x[UPT];
    if (a.x) {
#pragma unroll
      for (int u = 0; u < UPT; ++u) x[u].load(a.x, row + at[u]);
    }
    if (a.y) {
      Raw<TL> g[UPT];
#pragma unroll
      for (int u = 0; u < UPT; ++u) {
        Raw<TL> y;
        y.load(a.y, row + at[u]);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) v[u][i] = on[u] ? y.at(i) : 0.0f;
      }
      float g_row = 1.0f, slope;
      if (a.gate_kind == MEP_BLOCK_GATE_TOKEN)
        g_row = open_gate(reinterpret_cast<const float*>(a.gate)[t], a.sigmoid, slope);
      if (a.gate_kind == MEP_BLOCK_GATE_ELEMENT) {
#pragma unroll
        for (int u = 0; u < UPT; ++u) g[u].load(a.gate, row + at[u]);
      }
      norm_row<UPT, WAVE>(a.post, v, on, inv_h, a.eps, sum);
#pragma unroll
      for (int u = 0; u < UPT; ++u)
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          float f = fmaf(v[u][i], wp[u][i], bp[u][i]) * g_row;
          if (a.gate_kind == MEP_BLOCK_GATE_ELEMENT) f *= open_gate(g[u].at(i), a.sigmoid, slope);
          v[u][i] = f * a.block_scale;
        }
    }
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        if (a.x) v[u][i] = fmaf(a.residual_scale, x[u].at(i), v[u][i]);
        if (!on[u]) v[u][i] = 0.0f;
      }
      if (a.s && on[u]) store_unit((TL*)nullptr, a.s, row + at[u], v[u]);
    }
    if (!a.n && !a.codes) continue;
    norm_row<UPT, WAVE>(a.pre, v, on, inv_h, a.eps, sum);
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
#pragma unroll
      for (int i = 0; i < kUnit; ++i) v[u][i] = fmaf(v[u][i], wn[u][i], bn[u][i]);
      if (a.n && on[u]) store_unit((TL*)nullptr, a.n, row + at[u], v[u]);
      if (a.codes) {
        float scale;
        const u32x2 c = encode_unit(v[u], scale);
        if (on[u]) {
          reinterpret_cast<u32x2*>(a.codes)[row + at[u]] = c;
          if (at[u] % (kCodeBlock / kUnit) == 0) a.scales[(row + at[u]) / (kCodeBlock / kUnit)] = scale;
        }
      }
    }
  }
}

// ---- gradients --------------------------------------------------------------

// Adds to `grad` what a norm hands back of `g`, the gradient of its result times the
// weight, and leaves the normed row in v.  With h = hat(u) and r the factor,
//   d/du = r (g - mean(g) [layer norms] - h mean(g h)).
template <int UPT, bool WAVE>
__device__ __forceinline__ void norm_row_backward(int kind, float (&v)[UPT][kUnit],
                                                  const float (&g)[UPT][kUnit],
                                                  const bool (&on)[UPT], float inv_h, float eps,
                                                  RowSum<WAVE>& sum, float (&grad)[UPT][kUnit]) {
  if (kind == MEP_NORM_NONE) {
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
      for (int i = 0; i < kUnit; ++i) grad[u][i] += g[u][i];
    return;
  }
  float mean_g = 0.0f;
  if (kind == MEP_NORM_LAYER) {
    float t[2] = {0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        t[0] += v[u][i];
        t[1] += g[u][i];
      }
    sum(t);
    const float mean = t[0] * inv_h;
    mean_g = t[1] * inv_h;
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
      for (int i = 0; i < kUnit; ++i) v[u][i] = on[u] ? v[u][i] - mean : 0.0f;
  }
  float t[2] = {0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < UPT; ++u)
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      t[0] = fmaf(v[u][i], v[u][i], t[0]);
      t[1] = fmaf(v[u][i], g[u][i], t[1]);
    }
  sum(t);
  const float r = 1.0f / sqrtf(fmaf(t[0], inv_h, eps));
  const float along = t[1] * inv_h * r;
#pragma unroll
  for (int u = 0; u < UPT; ++u)
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      v[u][i] *= r;
      grad[u][i] = fmaf(r, g[u][i] - mean_g - v[u][i] * along, grad[u][i]);
    }
}

// Each block adds up its rows' share of the column sums in registers and leaves them in
// a row of `part`; norm_columns_kernel adds those up, in order, so that a result does
// not depend on timing.  BIAS: the biases' sums are wanted too.
template <class TL, int UPT, bool WAVE, bool BIAS>
__global__ __launch_bounds__(kMaxWaves * kWave) void norm_backward_kernel(NormBackwardArgs a) {
  __shared__ float4 lds[2][kMaxWaves];
  const int lanes = WAVE ? kWave : blockDim.x, l = WAVE ? lane_id() : threadIdx.x;
  const int rows_here = WAVE ? blockDim.x / kWave : 1;
  const int units = a.H / kUnit;
  const float inv_h = 1.0f / (float)a.H;
  RowSum<WAVE> sum{lds, 0, (int)blockDim.x / kWave};
  bool on[UPT];
  int at[UPT];
  float wp[UPT][kUnit], bp[UPT][kUnit], wn[UPT][kUnit];
  float acc[BIAS ? 4 : 2][UPT][kUnit];  // post weight, pre weight, their biases
#pragma unroll
  for (int u = 0; u < UPT; ++u) {
    on[u] = u * lanes + l < units;
    at[u] = min(u * lanes + l, units - 1);
    load_vector(a.post_weight, at[u], 1.0f, a.offset, wp[u]);
    load_vector(a.post_bias, at[u], 0.0f, 0.0f, bp[u]);
    load_vector(a.pre_weight, at[u], 1.0f, a.offset, wn[u]);
#pragma unroll
    for (int c = 0; c < (BIAS ? 4 : 2); ++c)
#pragma unroll
      for (int i = 0; i < kUnit; ++i) acc[c][u][i] = 0.0f;
  }
  const int64_t first = (int64_t)blockIdx.x * rows_here + (WAVE ? threadIdx.x / kWave : 0);
  const int64_t step = (int64_t)gridDim.x * rows_here;
  for (int64_t t = first; t < a.T; t += step) {
    const int64_t row = t * units;
    float grad[UPT][kUnit];  // of the stream
    float v[UPT][kUnit], g[UPT][kUnit];
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
      for (int i = 0; i < kUnit; ++i) grad[u][i] = 0.0f;
    if (a.grad_s) {
#pragma unroll
      for (int u = 0; u < UPT; ++u) {
        Raw<TL> q;
        q.load(a.grad_s, row + at[u]);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) grad[u][i] = on[u] ? q.at(i) : 0.0f;
      }
    }
    if (a.grad_n) {
      Raw<TL> gn[UPT];
#pragma unroll
      for (int u = 0; u < UPT; ++u) {
        Raw<TL> q;
        q.load(a.s, row + at[u]);
        gn[u].load(a.grad_n, row + at[u]);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          v[u][i] = on[u] ? q.at(i) : 0.0f;
          g[u][i] = on[u] ? gn[u].at(i) * wn[u][i] : 0.0f;
        }
      }
      norm_row_backward<UPT, WAVE>(a.pre, v, g, on, inv_h, a.eps, sum, grad);
#pragma unroll
      for (int u = 0; u < UPT; ++u)
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          acc[1][u][i] = fmaf(gn[u].at(i), v[u][i], acc[1][u][i]);
          if constexpr (BIAS) acc[3][u][i] += gn[u].at(i);
        }
    }
    if (a.grad_x) {
#pragma unroll
      for (int u = 0; u < UPT; ++u) {
        float f[kUnit];
#pragma unroll
        for (int i = 0; i < kUnit; ++i) f[i] = a.residual_scale * grad[u][i];
        if (on[u]) store_unit((TL*)nullptr, a.grad_x, row + at[u], f);
      }
    }
    if (!a.y) continue;
    // the block's part: gv, the gradient of v, takes the stream's place step by step
    Raw<TL> gate[UPT];
    float g_row = 1.0f, slope_row = 1.0f;
    if (a.gate_kind == MEP_BLOCK_GATE_TOKEN)
      g_row = open_gate(reinterpret_cast<const float*>(a.gate)[t], a.sigmoid, slope_row);
    if (a.gate_kind == MEP_BLOCK_GATE_ELEMENT) {
#pragma unroll
      for (int u = 0; u < UPT; ++u) gate[u].load(a.gate, row + at[u]);
    }
    const float c_row = a.block_scale * g_row;
    float gv[UPT][kUnit], back[UPT][kUnit];
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      Raw<TL> q;
      q.load(a.y, row + at[u]);
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        float slope, f = c_row;
        if (a.gate_kind == MEP_BLOCK_GATE_ELEMENT) f *= open_gate(gate[u].at(i), a.sigmoid, slope);
        v[u][i] = on[u] ? q.at(i) : 0.0f;
        gv[u][i] = f * grad[u][i];
        g[u][i] = on[u] ? gv[u][i] * wp[u][i] : 0.0f;
        back[u][i] = 0.0f;
      }
    }
    norm_row_backward<UPT, WAVE>(a.post, v, g, on, inv_h, a.eps, sum, back);
    float of_gate[1] = {0.0f};
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      float f[kUnit];
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        acc[0][u][i] = fmaf(gv[u][i], v[u][i], acc[0][u][i]);
        if constexpr (BIAS) acc[2][u][i] += gv[u][i];
        // the gradient of the gate's factor
        f[i] = a.block_scale * grad[u][i] * fmaf(v[u][i], wp[u][i], bp[u][i]);
        of_gate[0] += on[u] ? f[i] : 0.0f;
      }
      if (a.grad_y && on[u]) store_unit((TL*)nullptr, a.grad_y, row + at[u], back[u]);
      if (a.grad_gate && a.gate_kind == MEP_BLOCK_GATE_ELEMENT) {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          float slope;
          open_gate(gate[u].at(i), a.sigmoid, slope);
          f[i] *= slope;
        }
        if (on[u]) store_unit((TL*)nullptr, a.grad_gate, row + at[u], f);
      }
    }
    if (a.grad_gate && a.gate_kind == MEP_BLOCK_GATE_TOKEN) {
      sum(of_gate);
      if (l == 0) reinterpret_cast<float*>(a.grad_gate)[t] = of_gate[0] * slope_row;
    }
  }
  // this block's (or wave's) partial sums: wanted columns one after the other
  float* part = a.part + first * a.H;
  const int64_t next = (int64_t)step * a.H;
  constexpr int kOf[4] = {0, 2, 1, 3};  // columns[] in the order of acc
#pragma unroll
  for (int c = 0; c < (BIAS ? 4 : 2); ++c) {
    if (!a.columns[kOf[c]]) continue;
#pragma unroll
    for (int u = 0; u < UPT; ++u)
      if (on[u]) store_unit((float*)nullptr, part, at[u], acc[c][u]);
    part += next;
  }
}

constexpr int kColumns = 64, kSlices = 8;

// The wanted columns' sums: 64 columns a block, 8 threads a column, each every eighth
// partial row, joined in order.
__global__ __launch_bounds__(kColumns * kSlices) void norm_columns_kernel(const float* part, int rows,
                                                                          int H, float* c0, float* c1,
                                                                          float* c2, float* c3) {
  __shared__ double join[kSlices][kColumns];
  const int c = threadIdx.x % kColumns, slice = threadIdx.x / kColumns;
  const int h = blockIdx.x * kColumns + c;
  const float* p = part + (int64_t)blockIdx.y * rows * H;
  double s = 0.0;
  if (h < H) {
#pragma unroll 8
    for (int r = slice; r < rows; r += kSlices) s += (double)p[(int64_t)r * H + h];
  }
  join[slice][c] = s;
  __syncthreads();
  if (slice == 0 && h < H) {
#pragma unroll
    for (int i = 1; i < kSlices; ++i) s += join[i][c];
    float* out = blockIdx.y == 0 ? c0 : blockIdx.y == 1 ? c1 : blockIdx.y == 2 ? c2 : c3;
    out[h] = (float)s;
  }
}

// ---- launches -----------------------------------------------------------------

// How a row of H values is held: by a wave or a block, with so many units a thread.
struct RowShape {
  bool wave;
  int upt, threads, rows;  // rows: a block works on at once
};

RowShape row_shape(int H) {
  const int units = H / kUnit;
  if (units <= 2 * kWave) return {true, units <= kWave ? 1 : 2, 4 * kWave, 4};
  const int upt = units <= kMaxWaves * kWave ? 1 : 2;
  const int lanes = (units + upt - 1) / upt;
  return {false, upt, (lanes + kWave - 1) / kWave * kWave, 1};
}

// Calls f(units a thread, whether a wave holds a row).
template <class F>
void by_shape(const RowShape& r, F f) {
  using std::integral_constant;
  if (r.wave) {
    if (r.upt == 1) f(integral_constant<int, 1>{}, std::true_type{});
    else f(integral_constant<int, 2>{}, std::true_type{});
  } else {
    if (r.upt == 1) f(integral_constant<int, 1>{}, std::false_type{});
    else f(integral_constant<int, 2>{}, std::false_type{});
  }
}

int blocks_for(const RowShape& r, int32_t T, int most) {
  return (int)std::min<int64_t>(((int64_t)T + r.rows - 1) / r.rows, most);
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  const RowShape r = row_shape(a.H);
  const int blocks = blocks_for(r, a.T, 1024);
  by_shape(r, [&](auto upt, auto wave) {
    if (a.dtype == MEP_BF16)
      norm_kernel<uint16_t, upt(), wave()><<<blocks, r.threads, 0, s>>>(a);
    else
      norm_kernel<float, upt(), wave()><<<blocks, r.threads, 0, s>>>(a);
  });
  return hipGetLastError();
}

int norm_backward_blocks(int32_t H, int32_t T) {
  const RowShape r = row_shape(H);
  return blocks_for(r, T, 256) * r.rows;
}

hipError_t launch_block_norm_backward(const NormBackwardArgs& a, hipStream_t s) {
  const RowShape r = row_shape(a.H);
  const int blocks = blocks_for(r, a.T, 256);
  if (blocks > 0) {
    by_shape(r, [&](auto upt, auto wave) {
      auto launch = [&](auto type, auto bias) {
        norm_backward_kernel<decltype(type), upt(), wave(), bias()><<<blocks, r.threads, 0, s>>>(a);
      };
      const bool bias = a.columns[1] || a.columns[3];
      if (a.dtype == MEP_BF16) {
        if (bias) launch(uint16_t{}, std::true_type{}); else launch(uint16_t{}, std::false_type{});
      } else {
        if (bias) launch(float{}, std::true_type{}); else launch(float{}, std::false_type{});
      }
    });
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  float* out[4] = {};
  int n = 0;
  for (const int c : {0, 2, 1, 3})
    if (a.columns[c]) out[n++] = a.columns[c];
  if (n > 0)
    norm_columns_kernel<<<dim3((a.H + kColumns - 1) / kColumns, n), kColumns * kSlices, 0, s>>>(
        a.part, blocks * r.rows, a.H, out[0], out[1], out[2], out[3]);
  return hipGetLastError();
}

}  // namespace mep
