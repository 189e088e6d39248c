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
//
// Bound by memory for many rows: 4096 x 7168 in bf16, both norms, a gate a row, rows and E4M3
// codes out, 49.2 us (265 MB, 5.4 TB/s; a copy reaches 5.1), its gradients 70.6 (352 MB, 5.0
// TB/s).  What stood in the way was instructions as much as loads: a wave's takes 4 cycles,
// and 30 a value would be half of that time.  So a norm that subtracts no mean, has no bias
// and no gate for every value has kernels of its own, its factors are joined before they
// meet the values, and the vector units are 57% (61%) busy; with layer norms 73% (72%).  By
// the launch for few rows: one row of 7168 values 2.9 us, 128 rows 4.1.
#include <algorithm>
#include <type_traits>

#include "dev.h"
#include "mep_internal.h"

namespace mep {

namespace {

constexpr int kUnit = 8;           // values of a unit
constexpr int kMaxWaves = 16;      // of a block
constexpr int kCodeBlock = 128;    // columns that share an E4M3 scale
constexpr int kShare = kCodeBlock / kUnit;  // units that do

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

// The largest of 16 lanes, in every lane; values >= 0.
__device__ __forceinline__ float max16(float v) {
  auto step = [&](auto ctrl) {
    const int u = __float_as_int(v);
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(u, u, ctrl(), 0xf, 0xf, false)));
  };
  step(std::integral_constant<int, 0xB1>{});
  step(std::integral_constant<int, 0x4E>{});
  step(std::integral_constant<int, 0x141>{});
  step(std::integral_constant<int, 0x140>{});
  return v;
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

// One row of a tensor as a buffer: what lies outside (the units past a row's end, and
// everything where there is no such tensor or row) reads as 0 and is not written.
struct RowBuffer {
  __amdgpu_buffer_rsrc_t r;

  __device__ __forceinline__ RowBuffer(const void* p, int64_t t, int64_t T, int bytes) {
    constexpr int kRaw = 0x00027000;  // untyped, offsets in bytes
    const bool on = p != nullptr && t < T;
    r = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<unsigned char*>(reinterpret_cast<const unsigned char*>(p)) + t * bytes, 0,
        on ? bytes : 0, kRaw);
  }
};

constexpr int kPast = 2;  // cache policy of loads and stores: rows are passed once (nt)

template <class TL>
struct Raw;
template <>
struct Raw<uint16_t> {
  u32x4 q;
  __device__ __forceinline__ void load(const RowBuffer& b, int unit) {
    q = __builtin_amdgcn_raw_buffer_load_b128(b.r, unit * 16, 0, kPast);
  }
  __device__ __forceinline__ float at(int i) const { return i & 1 ? bf16_hi(q[i / 2]) : bf16_lo(q[i / 2]); }
  __device__ __forceinline__ void widen(float (&v)[kUnit]) const {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) v[i] = at(i);
  }
  // The compiler forgets what it has made of the values so far, and widens them again
  // where they are needed next instead of keeping them in twice the registers.
  __device__ __forceinline__ void hold() { asm volatile("" : "+v"(q)); }
};
template <>
struct Raw<float> {
  u32x4 q[2];
  __device__ __forceinline__ void load(const RowBuffer& b, int unit) {
    q[0] = __builtin_amdgcn_raw_buffer_load_b128(b.r, unit * 32, 0, kPast);
    q[1] = __builtin_amdgcn_raw_buffer_load_b128(b.r, unit * 32 + 16, 0, kPast);
  }
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(q[i / 4][i % 4]); }
  __device__ __forceinline__ void widen(float (&v)[kUnit]) const {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) v[i] = at(i);
  }
  __device__ __forceinline__ void hold() { asm volatile("" : "+v"(q[0]), "+v"(q[1])); }
};

__device__ __forceinline__ void store_unit(uint16_t*, const RowBuffer& b, int unit,
                                           const float (&v)[kUnit]) {
  u32x4 q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = pack_bf16_pair(v[2 * i], v[2 * i + 1]);
  __builtin_amdgcn_raw_buffer_store_b128(q, b.r, unit * 16, 0, kPast);
}
__device__ __forceinline__ void store_unit(float*, const RowBuffer& b, int unit,
                                           const float (&v)[kUnit]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const u32x4 q = {__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                     __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])};
    __builtin_amdgcn_raw_buffer_store_b128(q, b.r, unit * 32 + 16 * h, 0, kPast);
  }
}

// A vector's values at a unit, read through the caches: every row needs them.
struct RawVector {
  u32x4 q[2];
  __device__ __forceinline__ void load(const float* p, int H, int unit) {
    const RowBuffer b(p, 0, 1, H * 4);
    q[0] = __builtin_amdgcn_raw_buffer_load_b128(b.r, unit * 32, 0, 0);
    q[1] = __builtin_amdgcn_raw_buffer_load_b128(b.r, unit * 32 + 16, 0, 0);
  }
  // Plus `base`: a vector that is not there reads as 0.
  __device__ __forceinline__ void widen(float base, float (&v)[kUnit]) const {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) v[i] = base + __uint_as_float(q[i / 4][i % 4]);
  }
};

// One value of a tensor for the whole row, the same in every lane.
__device__ __forceinline__ float load_token(const void* p, int64_t t, int64_t T) {
  const RowBuffer b(p, t, T, 4);
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b.r, 0, 0, 0));
}

// A gate's factors and their slopes, N of them; sigmoids within 8 half-steps.
template <int N>
__device__ __forceinline__ void open_gate(const float (&g)[N], int sigmoid, float (&f)[N],
                                          float (&slope)[N]) {
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float e = exp_f32(-fabsf(g[i])), r = __builtin_amdgcn_rcpf(1.0f + e);
      slope[i] = e * r * r;
      f[i] = g[i] < 0.0f ? e * r : r;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      slope[i] = 1.0f;
      f[i] = g[i];
    }
  }
}

// Within 2 half-steps of fp32, as the root's error and the quotient's together would be.
__device__ __forceinline__ float inv_root(float mean_square, float eps) {
  return rsqrtf(mean_square + eps);
}

// Which of a row's units a thread holds, and how rows go over blocks.
template <int UPT, bool WAVE>
struct Place {
  int at[UPT];    // units, past the row's end for threads that hold none
  int units, lane;  // of a row; among the row's lanes
  int64_t first, step;

  __device__ __forceinline__ explicit Place(int H) {
    const int lanes = WAVE ? kWave : blockDim.x;
    lane = WAVE ? lane_id() : threadIdx.x;
    units = H / kUnit;
#pragma unroll
    for (int u = 0; u < UPT; ++u) at[u] = u * lanes + lane;
    const int rows = WAVE ? blockDim.x / kWave : 1;
    first = (int64_t)blockIdx.x * rows + (WAVE ? first_lane(threadIdx.x / kWave) : 0);
    step = (int64_t)gridDim.x * rows;
  }
  __device__ __forceinline__ bool on(int u) const { return at[u] < units; }
};

// What a kernel has registers and instructions for: norms without a mean and one factor a
// row; layer norms too; biases, their gradients and a gate for every element too.  Layer
// norms in kernels of their own and in those for everything, with one factor a row (us):
// 4096 x 7168 bf16 forward 44.9 and 51.5, gradients 88.8 and 108.9, in fp32 165 and 249,
// gradients of 4096 x 16384 bf16 239 and 690.  RMS norms take 43.1, 70.5, 153 and 184.
constexpr int kPlain = 0, kMeans = 1, kAll = 2;

// Threads that kernels are built for: four rows of a wave each, or one row of up to 512
// or 1024 threads (which leave a thread 256 or 128 registers).
constexpr int kWaveRows = 0, kHalfBlock = 512, kBlock = 1024;
constexpr int most_threads(int rows) { return rows == kWaveRows ? 4 * kWave : rows; }

// ---- forward ----------------------------------------------------------------

// E4M3 codes of a block of 128 columns, which 16 lanes hold: scale = amax / 448, codes of
// the values times 1 / scale (one rounding; a quotient's five instructions a value were a
// fifth of the kernel's).  A NaN is left out of the maximum and stays a NaN; an infinity
// makes the scale infinite and its whole block NaN.
__device__ __forceinline__ u32x2 encode_unit(const float (&v)[kUnit], float& scale) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < kUnit; ++i) m = fmaxf(m, fabsf(v[i]));
  m = max16(m);
  scale = m / 448.0f;
  // Below 2^-125 the reciprocal may leave fp32, so both factors are lifted by 2^64.  A scale
  // of so few bits may also lie so far below amax / 448 that products pass the largest code
  // (amax = 600 * 2^-149: scale 2^-149), so values are held within 448 scales; the comparison
  // leaves a NaN as it is.  (With quotients held within 448 there the kernels that spill
  // registers took up to 8% longer, 4096 x 16384 bf16 with everything 168 us for 157.)
  float q[kUnit];
  const bool few = scale < 0x1p-125f && scale != 0.0f;
  const float inv = scale == 0.0f ? 0.0f : 1.0f / (few ? scale * 0x1p64f : scale);
  const float most = few ? 448.0f * scale : __builtin_inff();
#pragma unroll
  for (int i = 0; i < kUnit; ++i) q[i] = v[i] * inv;
  if (few) {
#pragma unroll
    for (int i = 0; i < kUnit; ++i)
      q[i] = (fabsf(v[i]) > most ? copysignf(most, v[i]) : v[i]) * 0x1p64f * inv;
  }
  return u32x2{pack_e4m3x4(q[0], q[1], q[2], q[3]), pack_e4m3x4(q[4], q[5], q[6], q[7])};
}

// Waves a SIMD that a forward kernel of bf16 rows is kept to.  8 for whole blocks without
// biases or a gate for every element, so that two blocks of 14 waves (7168 columns) share a
// CU, whose first SIMD then holds 8 waves: 4096 rows with E4M3 codes too take 49.4 us (5.4
// TB/s), an earlier state of the kernel 58 where one block had the CU 64 to 70; with layer
// norms 44.9 us without codes, 51.8 where one has it (few enough vector registers alone do
// not do it).  6 for half blocks with everything: 4096 x 2056 20.6 us, 25.6 with 5; not for
// whole blocks, of which one has the CU either way (4096 x 7168 55.0, 56.6).
constexpr int forward_waves(int rows, int upt, int what, bool bf16) {
  if (rows == kWaveRows || upt > 1 || !bf16) return 1;
  if (what == kAll) return rows == kHalfBlock ? 6 : 1;
  return rows == kBlock ? 8 : 1;
}

template <class TL, int UPT, int ROWS, int WHAT>
__global__ __launch_bounds__(most_threads(ROWS), forward_waves(ROWS, UPT, WHAT, sizeof(TL) == 2))
void norm_kernel(NormArgs a) {
  constexpr bool WAVE = ROWS == kWaveRows, MEANS = WHAT != kPlain, ALL = WHAT == kAll;
  __shared__ float4 lds[2][kMaxWaves];
  const Place<UPT, WAVE> p(a.H);
  const float inv_h = 1.0f / (float)a.H;
  RowSum<WAVE> sum{lds, 0, (int)blockDim.x / kWave};
  const bool by_element = ALL && a.gate_kind == MEP_BLOCK_GATE_ELEMENT;
  const bool by_token = a.gate_kind == MEP_BLOCK_GATE_TOKEN;
  const bool post_layer = MEANS && a.post == MEP_NORM_LAYER;
  const bool pre_layer = MEANS && a.pre == MEP_NORM_LAYER;
  // A row as it lies in memory; the next one's loads run while this one is worked on.
  struct Row {
    Raw<TL> x[UPT], y[UPT], gate[ALL ? UPT : 1];
    float g;
  };
  const int bytes = a.H * (int)sizeof(TL);
  auto load = [&](int64_t t, Row& r) __attribute__((always_inline)) {
    const RowBuffer x(a.x, t, a.T, bytes), y(a.y, t, a.T, bytes), gate(a.gate, t, a.T, bytes);
    if (a.y) {
#pragma unroll
      for (int u = 0; u < UPT; ++u) r.y[u].load(y, p.at[u]);
    }
    if (a.x) {
#pragma unroll
      for (int u = 0; u < UPT; ++u) r.x[u].load(x, p.at[u]);
    }
    if constexpr (ALL)
      if (by_element) {
#pragma unroll
        for (int u = 0; u < UPT; ++u) r.gate[u].load(gate, p.at[u]);
      }
    r.g = 0.0f;
    if (by_token) r.g = reinterpret_cast<const float*>(a.gate)[t];
  };
  Row now;
  int64_t t = p.first;
  if (t >= a.T) return;
  load(t, now);
  float wp[UPT][kUnit], wn[UPT][kUnit];
  float bp[ALL ? UPT : 1][kUnit], bn[ALL ? UPT : 1][kUnit];
  {
    RawVector post_w[UPT], pre_w[UPT], post_b[ALL ? UPT : 1], pre_b[ALL ? UPT : 1];
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      post_w[u].load(a.post_weight, a.H, p.at[u]);
      pre_w[u].load(a.pre_weight, a.H, p.at[u]);
      if constexpr (ALL) {
        post_b[u].load(a.post_bias, a.H, p.at[u]);
        pre_b[u].load(a.pre_bias, a.H, p.at[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      post_w[u].widen(a.post_weight ? a.offset : 1.0f, wp[u]);
      pre_w[u].widen(a.pre_weight ? a.offset : 1.0f, wn[u]);
      if constexpr (ALL) {
        post_b[u].widen(0.0f, bp[u]);
        pre_b[u].widen(0.0f, bn[u]);
      }
    }
  }
  for (; t < a.T; t += p.step) {
    Row next;
    if (t + p.step < a.T) load(t + p.step, next);
    float v[UPT][kUnit];
    if (a.y) {
      float mean = 0.0f, r = 1.0f;
      if (post_layer) {
        float q[1] = {0.0f};
#pragma unroll
        for (int u = 0; u < UPT; ++u)
#pragma unroll
          for (int i = 0; i < kUnit; ++i) q[0] += now.y[u].at(i);  // 0 past the row's end
        sum(q);
        mean = q[0] * inv_h;
      }
      if (a.post != MEP_NORM_NONE) {
        float q[1] = {0.0f};
#pragma unroll
        for (int u = 0; u < UPT; ++u)
          if (!MEANS || p.on(u))
#pragma unroll
            for (int i = 0; i < kUnit; ++i) {
              const float d = MEANS ? now.y[u].at(i) - mean : now.y[u].at(i);
              q[0] = fmaf(d, d, q[0]);
            }
        sum(q);
        r = inv_root(q[0] * inv_h, a.eps);
      }
      float c = a.block_scale;
      if (by_token) {
        float f[1], slope[1];
        open_gate({now.g}, a.sigmoid, f, slope);
        c *= f[0];
      }
#pragma unroll
      for (int u = 0; u < UPT; ++u)
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          if constexpr (ALL) v[u][i] = fmaf((now.y[u].at(i) - mean) * r, wp[u][i], bp[u][i]) * c;
          else if constexpr (MEANS) v[u][i] = (now.y[u].at(i) - mean) * (r * c) * wp[u][i];
          else v[u][i] = now.y[u].at(i) * (r * c) * wp[u][i];
        }
      if (by_element) {
#pragma unroll
        for (int u = 0; u < UPT; ++u) {
          float g[kUnit], f[kUnit], slope[kUnit];
          now.gate[ALL ? u : 0].widen(g);
          open_gate(g, a.sigmoid, f, slope);
#pragma unroll
          for (int i = 0; i < kUnit; ++i) v[u][i] *= f[i];
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < UPT; ++u)
#pragma unroll
        for (int i = 0; i < kUnit; ++i) v[u][i] = 0.0f;
    }
    if (a.x) {
#pragma unroll
      for (int u = 0; u < UPT; ++u)
#pragma unroll
        for (int i = 0; i < kUnit; ++i) v[u][i] = fmaf(a.residual_scale, now.x[u].at(i), v[u][i]);
    }
    if (a.s) {
      const RowBuffer s(a.s, t, a.T, bytes);
#pragma unroll
      for (int u = 0; u < UPT; ++u) store_unit((TL*)nullptr, s, p.at[u], v[u]);
    }
    if (a.n || a.codes) {
      float mean = 0.0f, r = 1.0f;
      if (pre_layer) {
        float q[1] = {0.0f};
#pragma unroll
        for (int u = 0; u < UPT; ++u)
          if (p.on(u))
#pragma unroll
            for (int i = 0; i < kUnit; ++i) q[0] += v[u][i];
        sum(q);
        mean = q[0] * inv_h;
      }
      if (a.pre != MEP_NORM_NONE) {
        float q[1] = {0.0f};
#pragma unroll
        for (int u = 0; u < UPT; ++u)
          if (!MEANS || p.on(u))
#pragma unroll
            for (int i = 0; i < kUnit; ++i) {
              const float d = MEANS ? v[u][i] - mean : v[u][i];
              q[0] = fmaf(d, d, q[0]);
            }
        sum(q);
        r = inv_root(q[0] * inv_h, a.eps);
      }
#pragma unroll
      for (int u = 0; u < UPT; ++u)
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          if constexpr (ALL) v[u][i] = fmaf((v[u][i] - mean) * r, wn[u][i], bn[u][i]);
          else if constexpr (MEANS) v[u][i] = (v[u][i] - mean) * r * wn[u][i];
          else v[u][i] = v[u][i] * r * wn[u][i];
        }
      if (a.n) {
        const RowBuffer n(a.n, t, a.T, bytes);
#pragma unroll
        for (int u = 0; u < UPT; ++u) store_unit((TL*)nullptr, n, p.at[u], v[u]);
      }
      if (a.codes) {
        const RowBuffer codes(a.codes, t, a.T, a.H), scales(a.scales, t, a.T, a.H / kCodeBlock * 4);
#pragma unroll
        for (int u = 0; u < UPT; ++u) {
          float scale;
          const u32x2 c = encode_unit(v[u], scale);
          __builtin_amdgcn_raw_buffer_store_b64(c, codes.r, p.at[u] * kUnit, 0, kPast);
          // one lane of 16 has a block's scale; the others' offsets lie past the row
          const int block = p.at[u] % kShare == 0 ? p.at[u] / kShare : p.units;
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(scale), scales.r, block * 4, 0, 0);
        }
      }
    }
    now = next;
  }
}

// ---- gradients --------------------------------------------------------------

// With h = hat(u), r its factor and g the gradient of the normed row times the weight,
//   d/du = r (g - mean(g) [layer norms] - h mean(g h)).
// A row stays as it lies in memory (raw) while its sums are taken, each value widened
// where it is needed: sums of both norms that do not wait for each other share a round.
// The weights have registers, or lie in LDS where those would not do: 1024 threads leave
// 128 a thread, and what spills costs as much as the rows (4096 x 7168 with layer norms,
// biases and a gate for every element 131 us, with all in registers 248; 4096 x 16384
// without any of these 184 and 345).
//   Each block adds up its rows' share of the column sums in registers and leaves them in
// a row of `part`; norm_columns_kernel adds those up, in order, so that a result does
// not depend on timing.
constexpr bool weights_in_lds(int rows, int upt, bool all, bool bf16) {
  return rows == kBlock ? all || upt > 1 : rows == kHalfBlock && all && bf16;
}
// Half blocks kept to 128 registers, so that 4 waves a SIMD fit whatever the block's
// waves: all but those of fp32 rows with everything, which would spill too much (4096 x 2056
// 88 us, in 128 registers 115).  In bf16 that kernel spills 40 bytes a thread and
// gains by it all the same: 60 us, without the bound 68.
constexpr bool packed_halves(int rows, bool all, bool bf16) {
  return rows == kHalfBlock && (!all || bf16);
}
constexpr int kLdsRow = 8192;  // values of a row of which three vectors fit LDS, else two
__host__ __device__ constexpr int vectors_in_lds(bool all, int H) {
  return all && H <= kLdsRow ? 3 : 2;
}

template <class TL, int UPT, int ROWS, int WHAT>
__global__ __launch_bounds__(most_threads(ROWS), packed_halves(ROWS, WHAT == kAll, sizeof(TL) == 2) ? 4 : 1)
void norm_backward_kernel(NormBackwardArgs a) {
  constexpr bool WAVE = ROWS == kWaveRows, MEANS = WHAT != kPlain, ALL = WHAT == kAll;
  __shared__ float4 lds[2][kMaxWaves];
  constexpr int COLS = ALL ? 4 : 2;  // post weight, pre weight, their biases
  // Rows whose loads have registers, and whether the weights have (else they lie in LDS,
  // as far as that holds them).
  constexpr bool IN_LDS = weights_in_lds(ROWS, UPT, ALL, sizeof(TL) == 2);
  constexpr int AHEAD = sizeof(TL) == 2 && !IN_LDS ? 2 : 1;
  const Place<UPT, WAVE> p(a.H);
  const float inv_h = 1.0f / (float)a.H;
  RowSum<WAVE> sum{lds, 0, (int)blockDim.x / kWave};
  float acc[COLS][UPT][kUnit];
#pragma unroll
  for (int c = 0; c < COLS; ++c)
#pragma unroll
    for (int u = 0; u < UPT; ++u)
#pragma unroll
      for (int i = 0; i < kUnit; ++i) acc[c][u][i] = 0.0f;
  const bool by_element = ALL && a.gate_kind == MEP_BLOCK_GATE_ELEMENT;
  const bool by_token = a.gate_kind == MEP_BLOCK_GATE_TOKEN;
  const int pre = a.grad_n ? a.pre : MEP_NORM_NONE, post = a.y ? a.post : MEP_NORM_NONE;
  struct Row {
    Raw<TL> gs[UPT], gn[UPT], s[UPT], y[UPT], gate[ALL ? UPT : 1];
    float g;
  };
  const int bytes = a.H * (int)sizeof(TL);
  auto load_stream = [&](int64_t t, Row& r) __attribute__((always_inline)) {
    const RowBuffer s(a.grad_n ? a.s : nullptr, t, a.T, bytes), gn(a.grad_n, t, a.T, bytes);
    const RowBuffer gs(a.grad_s, t, a.T, bytes);
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      r.s[u].load(s, p.at[u]);
      r.gn[u].load(gn, p.at[u]);
      r.gs[u].load(gs, p.at[u]);
    }
  };
  auto load_block = [&](int64_t t, Row& r) __attribute__((always_inline)) {
    const RowBuffer y(a.y, t, a.T, bytes), gate(by_element ? a.gate : nullptr, t, a.T, bytes);
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      r.y[u].load(y, p.at[u]);
      if constexpr (ALL) r.gate[u].load(gate, p.at[u]);
    }
    r.g = load_token(by_token ? a.gate : nullptr, t, a.T);
  };
  Row rows[AHEAD];
  int64_t t = p.first;
  load_stream(t, rows[0]);
  load_block(t, rows[0]);
  extern __shared__ float4 weights[];  // IN_LDS: pre weight, post weight, post bias
  const int slots = UPT * blockDim.x;  // units of each
  float kept[IN_LDS ? 1 : ALL ? 3 : 2][UPT][kUnit];
  if constexpr (IN_LDS) {
    for (int v = 0; v < vectors_in_lds(ALL, a.H); ++v) {
      const float* from = v == 0 ? a.pre_weight : v == 1 ? a.post_weight : a.post_bias;
#pragma unroll
      for (int u = 0; u < UPT; ++u) {
        RawVector raw;
        raw.load(from, a.H, p.at[u]);
        float w[kUnit];
        raw.widen(v == 2 ? 0.0f : from ? a.offset : 1.0f, w);
        float4* to = weights + (v * slots + p.at[u]) * 2;
        to[0] = make_float4(w[0], w[1], w[2], w[3]);
        to[1] = make_float4(w[4], w[5], w[6], w[7]);
      }
    }  // read by the thread that wrote them, threads past the row's end with numbers too
  } else {
    RawVector raw[ALL ? 3 : 2][UPT];
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      raw[0][u].load(a.pre_weight, a.H, p.at[u]);
      raw[1][u].load(a.post_weight, a.H, p.at[u]);
      if constexpr (ALL) raw[2][u].load(a.post_bias, a.H, p.at[u]);
    }
    if constexpr (AHEAD == 2) {
      load_stream(t + p.step, rows[1]);
      load_block(t + p.step, rows[1]);
    }
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      raw[0][u].widen(a.pre_weight ? a.offset : 1.0f, kept[0][u]);
      raw[1][u].widen(a.post_weight ? a.offset : 1.0f, kept[1][u]);
      if constexpr (ALL) raw[2][u].widen(0.0f, kept[2][u]);
    }
  }
  // a vector's values at a unit, in the order above
  auto vector = [&](int v, int u, float(&w)[kUnit]) __attribute__((always_inline)) {
    if constexpr (!IN_LDS) {
#pragma unroll
      for (int i = 0; i < kUnit; ++i) w[i] = kept[v][u][i];
    } else if (v < vectors_in_lds(ALL, a.H)) {
      const float4* from = weights + (v * slots + p.at[u]) * 2;
      const float4 lo = from[0], hi = from[1];
      w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w;
      w[4] = hi.x; w[5] = hi.y; w[6] = hi.z; w[7] = hi.w;
    } else {  // the bias of a long row
      RawVector raw;
      raw.load(a.post_bias, a.H, p.at[u]);
      raw.widen(0.0f, w);
    }
  };
  auto hold = [&](Row& r) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      r.s[u].hold();
      r.gn[u].hold();
      r.y[u].hold();
    }
  };
  // one row; its place takes the loads of the row AHEAD steps on as parts of it are done
  auto work = [&](int64_t t, Row& now) __attribute__((always_inline)) {
    const int64_t then = t + AHEAD * p.step;
    // the means of both norms' rows, and of the next norm's gradient
    float mean_s = 0.0f, r_s = 1.0f, mean_n = 0.0f, along_n = 0.0f, mean_y = 0.0f, r_y = 1.0f;
    if (MEANS && (pre == MEP_NORM_LAYER || post == MEP_NORM_LAYER)) {
      float q[3] = {0.0f, 0.0f, 0.0f};  // what lies past the row's end is 0
#pragma unroll
      for (int u = 0; u < UPT; ++u) {
        float wn[kUnit];
        vector(0, u, wn);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
          q[0] += now.s[u].at(i);
          q[1] = fmaf(now.gn[u].at(i), wn[i], q[1]);
          q[2] += now.y[u].at(i);
        }
      }
      sum(q);
      if (pre == MEP_NORM_LAYER) {
        mean_s = q[0] * inv_h;
        mean_n = q[1] * inv_h;
      }
      if (post == MEP_NORM_LAYER) mean_y = q[2] * inv_h;
      hold(now);
    }
    // their factors, and what of the gradient lies along the row
    if (pre != MEP_NORM_NONE || post != MEP_NORM_NONE) {
      float q[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < UPT; ++u) {
        float wn[kUnit];
        vector(0, u, wn);
        if (!MEANS || p.on(u))
#pragma unroll
          for (int i = 0; i < kUnit; ++i) {
            const float s = MEANS ? now.s[u].at(i) - mean_s : now.s[u].at(i);
            const float y = MEANS ? now.y[u].at(i) - mean_y : now.y[u].at(i);
            q[0] = fmaf(s, s, q[0]);
            q[1] = fmaf(s, now.gn[u].at(i) * wn[i], q[1]);
            q[2] = fmaf(y, y, q[2]);
          }
      }
      sum(q);
      if (pre != MEP_NORM_NONE) {
        r_s = inv_root(q[0] * inv_h, a.eps);
        along_n = q[1] * inv_h * r_s;
      }
      if (post != MEP_NORM_NONE) r_y = inv_root(q[2] * inv_h, a.eps);
      hold(now);
    }
    // the stream's gradient
    float grad[UPT][kUnit];
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      float wn[kUnit];
      vector(0, u, wn);
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        float g = now.gs[u].at(i);  // 0 without grad_s; without grad_n, s and gn are 0
        const float gn = now.gn[u].at(i);
        const float h = MEANS ? (now.s[u].at(i) - mean_s) * r_s : now.s[u].at(i) * r_s;
        const float off = MEANS ? fmaf(h, along_n, mean_n) : h * along_n;
        g = fmaf(r_s, fmaf(gn, wn[i], -off), g);
        acc[1][u][i] = fmaf(gn, h, acc[1][u][i]);
        if constexpr (ALL) acc[3][u][i] += gn;
        grad[u][i] = g;
      }
    }
    load_stream(then, now);
    const RowBuffer grad_x(a.grad_x, t, a.T, bytes);
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      float f[kUnit];
#pragma unroll
      for (int i = 0; i < kUnit; ++i) f[i] = a.residual_scale * grad[u][i];
      store_unit((TL*)nullptr, grad_x, p.at[u], f);
    }
    // the block's part (without a block y is 0, and nothing of this is stored)
    float f_row[1] = {1.0f}, slope_row[1] = {1.0f};
    if (by_token) open_gate({now.g}, a.sigmoid, f_row, slope_row);
    const float c = a.block_scale * f_row[0];
    // a unit's gate factors without c, and their slopes
    auto factors = [&](int u, float(&f)[kUnit], float(&slope)[kUnit]) __attribute__((always_inline)) {
      if (by_element) {
        float g[kUnit];
        now.gate[ALL ? u : 0].widen(g);
        open_gate(g, a.sigmoid, f, slope);
      } else {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) f[i] = slope[i] = 1.0f;
      }
    };
    const bool token_grad = by_token && a.grad_gate;
    float mean_v = 0.0f, along_y = 0.0f, of_row = 0.0f;
    if (post != MEP_NORM_NONE || token_grad) {
      float q[ALL ? 3 : MEANS ? 2 : 1] = {0.0f};
#pragma unroll
      for (int u = 0; u < UPT; ++u) {
        float wp[kUnit], bp[kUnit], f[kUnit], slope[kUnit];
        vector(1, u, wp);
        if constexpr (ALL) {
          vector(2, u, bp);
          factors(u, f, slope);
        }
        if (!MEANS || p.on(u))
#pragma unroll
          for (int i = 0; i < kUnit; ++i) {
            if constexpr (ALL) {
              const float h = (now.y[u].at(i) - mean_y) * r_y;
              const float g = f[i] * grad[u][i] * wp[i];
              q[0] = fmaf(g, h, q[0]);
              q[1] += g;
              q[2] = fmaf(grad[u][i], bp[i], q[2]);
            } else if constexpr (MEANS) {
              const float g = grad[u][i] * wp[i];
              q[0] = fmaf(g, (now.y[u].at(i) - mean_y) * r_y, q[0]);
              q[1] += g;
            } else {
              q[0] = fmaf(grad[u][i] * wp[i], now.y[u].at(i), q[0]);
            }
          }
      }
      sum(q);
      if constexpr (!MEANS) q[0] *= r_y;
      if (post != MEP_NORM_NONE) along_y = c * q[0] * inv_h;
      if constexpr (MEANS)
        if (post == MEP_NORM_LAYER) mean_v = c * q[1] * inv_h;
      if constexpr (ALL) q[0] += q[2];
      of_row = a.block_scale * q[0] * slope_row[0];  // a gate a row: sum of grad v
#pragma unroll
      for (int u = 0; u < UPT; ++u) now.y[u].hold();
    }
    const RowBuffer grad_y(a.grad_y, t, a.T, bytes);
    const RowBuffer grad_gate(by_element ? a.grad_gate : nullptr, t, a.T, bytes);
#pragma unroll
    for (int u = 0; u < UPT; ++u) {
      float back[kUnit], of_gate[kUnit], wp[kUnit], bp[kUnit], f[kUnit], slope[kUnit];
      vector(1, u, wp);
      if constexpr (ALL) {
        vector(2, u, bp);
        factors(u, f, slope);
      }
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        if constexpr (ALL) {
          const float h = (now.y[u].at(i) - mean_y) * r_y;
          const float gv = c * f[i] * grad[u][i];
          acc[0][u][i] = fmaf(gv, h, acc[0][u][i]);
          acc[2][u][i] += gv;
          back[i] = r_y * fmaf(gv, wp[i], -fmaf(h, along_y, mean_v));
          of_gate[i] = a.block_scale * slope[i] * grad[u][i] * fmaf(h, wp[i], bp[i]);
        } else {
          const float h = MEANS ? (now.y[u].at(i) - mean_y) * r_y : now.y[u].at(i) * r_y;
          const float gv = c * grad[u][i];
          acc[0][u][i] = fmaf(gv, h, acc[0][u][i]);
          back[i] = r_y * fmaf(gv, wp[i], -(MEANS ? fmaf(h, along_y, mean_v) : h * along_y));
        }
      }
      store_unit((TL*)nullptr, grad_y, p.at[u], back);
      if constexpr (ALL) store_unit((TL*)nullptr, grad_gate, p.at[u], of_gate);
    }
    const RowBuffer row_gate(token_grad ? a.grad_gate : nullptr, t, a.T, 4);
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(of_row), row_gate.r, p.lane * 4, 0, 0);
    load_block(then, now);
  };
  if (t < a.T) {
    while (true) {
      work(t, rows[0]);
      if ((t += p.step) >= a.T) break;
      if constexpr (AHEAD == 2) {
        work(t, rows[1]);
        if ((t += p.step) >= a.T) break;
      }
    }
  }
  // this block's partial sums: wanted columns one after the other
  float* part = a.part + (int64_t)blockIdx.x * a.H;
  constexpr int kOf[4] = {0, 2, 1, 3};  // columns[] in the order of acc
#pragma unroll
  for (int c = 0; c < COLS; ++c) {
    if (!a.columns[kOf[c]]) continue;
    if constexpr (WAVE) {  // four waves' sums first
      __shared__ float4 join[4][UPT * 2 * kWave];
#pragma unroll
      for (int u = 0; u < UPT; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          join[threadIdx.x / kWave][(u * 2 + h) * kWave + p.lane] =
              make_float4(acc[c][u][4 * h], acc[c][u][4 * h + 1], acc[c][u][4 * h + 2], acc[c][u][4 * h + 3]);
      __syncthreads();
      for (int i = threadIdx.x; i < UPT * 2 * kWave; i += 4 * kWave) {
        float4 v = join[0][i];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
          v.x += join[w][i].x; v.y += join[w][i].y; v.z += join[w][i].z; v.w += join[w][i].w;
        }
        const int unit = i / (2 * kWave) * kWave + i % kWave, h = i / kWave % 2;
        if (unit < p.units) reinterpret_cast<float4*>(part)[2 * unit + h] = v;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int u = 0; u < UPT; ++u)
        if (p.on(u)) {  // read again at once: through the caches
          float4* to = reinterpret_cast<float4*>(part) + 2 * p.at[u];
          to[0] = make_float4(acc[c][u][0], acc[c][u][1], acc[c][u][2], acc[c][u][3]);
          to[1] = make_float4(acc[c][u][4], acc[c][u][5], acc[c][u][6], acc[c][u][7]);
        }
    }
    part += (int64_t)gridDim.x * a.H;
  }
}

constexpr int kColumns = 32, kSlices = 16;

// The wanted columns' sums: 32 columns a block, 16 threads a column, each every 16th
// partial row, joined in order in fp64.  (64 columns and 8 threads: 301 rows of 1048
// columns, four vectors, 14.5 us with the gradients for 13.0.)
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
  int kind;                // kWaveRows, kHalfBlock or kBlock
  int upt, threads, rows;  // rows: a block works on at once
};

RowShape row_shape(int H) {
  const int units = H / kUnit;
  if (units <= 2 * kWave) return {kWaveRows, units <= kWave ? 1 : 2, 4 * kWave, 4};
  const int upt = units <= kBlock ? 1 : 2;
  const int lanes = ((units + upt - 1) / upt + kWave - 1) / kWave * kWave;
  return {lanes <= kHalfBlock ? kHalfBlock : kBlock, upt, lanes, 1};
}

// Calls f(units a thread, kind).
template <class F>
void by_shape(const RowShape& r, F f) {
  using std::integral_constant;
  const integral_constant<int, 1> one;
  const integral_constant<int, 2> two;
  if (r.kind == kWaveRows) {
    const integral_constant<int, kWaveRows> kind;
    if (r.upt == 1) f(one, kind); else f(two, kind);
  } else if (r.kind == kHalfBlock) {
    f(one, integral_constant<int, kHalfBlock>{});
  } else {
    const integral_constant<int, kBlock> kind;
    if (r.upt == 1) f(one, kind); else f(two, kind);
  }
}

// Calls f(a value of the rows' type, what).
template <class F>
void by_type(int dtype, int what, F f) {
  using std::integral_constant;
  auto of = [&](auto type) {
    if (what == kPlain) f(type, integral_constant<int, kPlain>{});
    else if (what == kMeans) f(type, integral_constant<int, kMeans>{});
    else f(type, integral_constant<int, kAll>{});
  };
  if (dtype == MEP_BF16) of(uint16_t{});
  else of(float{});
}

int what_of(bool all, int post, int pre) {
  return all ? kAll : post == MEP_NORM_LAYER || pre == MEP_NORM_LAYER ? kMeans : kPlain;
}

int blocks_for(const RowShape& r, int32_t T, int most) {
  return (int)std::min<int64_t>(((int64_t)T + r.rows - 1) / r.rows, most);
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  const RowShape r = row_shape(a.H);
  const bool all = a.post_bias || a.pre_bias || a.gate_kind == MEP_BLOCK_GATE_ELEMENT;
  const bool bf16 = a.dtype == MEP_BF16;
  // Blocks that the CUs hold at once and no more, as each loads the weights.  4096 rows
  // with 256, 512, 1024 blocks (us): 7168 bf16 columns 40.9, 42.8, 46.9, with codes 49.4, 49.2,
  // 55.5, between layer norms 49.4, 44.4, 53.9, with biases and a gate for every element too
  // 54.2, 58.2, 64.9, in fp32 113, 117, 120; 2056 columns 20.4, 16.3, 15.2, in fp32 30.4, 29.8,
  // 30.8, with everything 41.7, 38.7, 46.2; 512 by wave 5.3, 4.7, 4.6 (768: 4.5).
  const int most = r.kind == kWaveRows ? 768
                   : r.kind == kBlock && (all || !bf16 || r.upt > 1) ? 256
                   : bf16 && r.threads <= 384 ? 1024 : 512;
  const int blocks = blocks_for(r, a.T, most);
  by_shape(r, [&](auto upt, auto kind) {
    by_type(a.dtype, what_of(all, a.post, a.pre), [&](auto type, auto what) {
      norm_kernel<decltype(type), upt(), kind(), what()><<<blocks, r.threads, 0, s>>>(a);
    });
  });
  return hipGetLastError();
}

// Blocks of the gradients' launch, each of which leaves a row of partial sums: one a CU,
// two where they fit.  4096 rows with 256 and 512 blocks (us): 2056 bf16 columns 38.2 and
// 31.1, between layer norms 54.2 and 41.3, with everything 75.8 and 59.7, in fp32 88 and 93,
// 7168 bf16 columns 71 and 80, 512 columns by wave 11.2 and 11.4.
static int backward_blocks(const RowShape& r, int32_t T, bool all, bool bf16) {
  return blocks_for(r, T, packed_halves(r.kind, all, bf16) ? 512 : 256);
}

int norm_backward_blocks(int32_t H, int32_t T) {  // the most of all
  return backward_blocks(row_shape(H), T, false, true);
}

hipError_t launch_block_norm_backward(const NormBackwardArgs& a, hipStream_t s) {
  const RowShape r = row_shape(a.H);
  const bool all = a.columns[1] || a.columns[3] || a.post_bias ||
                   a.gate_kind == MEP_BLOCK_GATE_ELEMENT;
  const int blocks = backward_blocks(r, a.T, all, a.dtype == MEP_BF16);
  if (blocks > 0) {
    const size_t lds = weights_in_lds(r.kind, r.upt, all, a.dtype == MEP_BF16)
                           ? (size_t)vectors_in_lds(all, a.H) * r.upt * r.threads * kUnit * sizeof(float)
                           : 0;
    by_shape(r, [&](auto upt, auto kind) {
      by_type(a.dtype, what_of(all, a.post, a.pre), [&](auto type, auto what) {
        norm_backward_kernel<decltype(type), upt(), kind(), what()><<<blocks, r.threads, lds, s>>>(a);
      });
    });
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  float* out[4] = {};
  int n = 0;
  for (const int c : {0, 2, 1, 3})
    if (a.columns[c]) out[n++] = a.columns[c];
  if (n > 0)
    norm_columns_kernel<<<dim3((a.H + kColumns - 1) / kColumns, n), kColumns * kSlices, 0, s>>>(
        a.part, blocks, a.H, out[0], out[1], out[2], out[3]);
  return hipGetLastError();
}

}  // namespace mep
