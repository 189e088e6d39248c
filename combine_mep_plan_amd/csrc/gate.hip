// Router: top-k selection with its weights, the load-balance loss, and their
// gradient with respect to the logits.
//
// A token's E logits sit in the registers of a group of LPT lanes (8 lanes up
// to 64 experts, 16 up to 512, the whole wave beyond), EPL values a lane, so a
// wave works on 64 / LPT tokens at once and reduces over 8 or 16 lanes with
// DPP moves that cost one instruction a step.  Lane l of a group holds, for
// c = 0.., the V consecutive experts (c*LPT + l)*V.. (V: one 16-byte load when
// every row starts on a 16-byte boundary, else single loads of the same
// experts).  Values past E stay out of every maximum and sum.
#include <algorithm>
#include <type_traits>

#include "dev.h"
#include "mep_internal.h"

namespace mep {

namespace {

// ---- reductions over a group of LPT consecutive lanes, result in every lane --

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xf, 0xf, false);
}

// DPP controls: exchanges within 2 and 4 lanes (quad permutations), with the
// mirrored lane of 8 (row_half_mirror) and of 16 (row_mirror).  After the quad
// steps all 4 lanes agree, so a mirror is as good as an exchange.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

template <int LPT, class F>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, F f) {
  v = f(v, dpp<kXor1>(v));
  v = f(v, dpp<kXor2>(v));
  v = f(v, dpp<kHalfMirror>(v));
  if (LPT >= 16) v = f(v, dpp<kMirror>(v));
  if (LPT == 64) {
    v = f(v, (uint32_t)__shfl_xor((int)v, 16));
    v = f(v, (uint32_t)__shfl_xor((int)v, 32));
  }
  return v;
}

template <int LPT>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<LPT>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

template <int LPT>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return group_reduce<LPT>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

template <int LPT>
__device__ __forceinline__ uint32_t group_add(uint32_t v) {
  return group_reduce<LPT>(v, [](uint32_t a, uint32_t b) { return a + b; });
}

// Every lane adds the same pairs (a + b and b + a round alike), so all agree.
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
  return __uint_as_float(group_reduce<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

template <int LPT>
__device__ __forceinline__ float group_fmax(float v) {
  return __uint_as_float(group_reduce<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}

// The largest key of the lanes, the lowest expert among equals.
template <int LPT>
__device__ __forceinline__ void group_best(uint64_t& key, int& e) {
  for (int d = 1; d < LPT; d <<= 1) {
    const uint64_t ok = __shfl_xor((unsigned long long)key, d);
    const int oe = __shfl_xor(e, d);
    if (ok > key || (ok == key && oe < e)) {
      key = ok;
      e = oe;
    }
  }
}

// ---- values ---------------------------------------------------------------

// Unsigned keys in the order of the values: -inf < ... < -0 = +0 < ... < +inf
// are keys above 1, NaN is 1 (ranks last), 0 is below every value (absent).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 + 0 is +0
  const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return v != v ? 1u : k;
}

__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  const uint64_t k = u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
  return v != v ? 1ull : k;
}

// A packed key's value part as the value's own key.
__device__ __forceinline__ uint32_t unpack_key(uint32_t k) {
  const uint32_t v = k & 0xffff0000u;
  return v == 0u ? 1u : v & 0x80000000u ? v : v | 0xffffu;
}

__device__ __forceinline__ float key_value(uint32_t k) {
  if (k == 1u) return __uint_as_float(0x7fc00000u);
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

constexpr float kLog2E = 1.44269504088896341f;

// exp(x) in two instructions: the hardware's power of two of the rounded x log2 e,
// so within 2 + 1.5 |x| half-steps of fp32 (relative).  For the selection's keys,
// whose absolute error counts, and for probabilities of all experts, of which those
// far below the largest add next to nothing to anything (exp_f32 there cost the
// balance loss of 4096 x 256 16.0 -> 17.0 us, the gradient 6.6 -> 6.9).
__device__ __forceinline__ float fast_exp(float x) {
  return __builtin_amdgcn_exp2f(x * kLog2E);
}

// For the weights, which may all be small: exp(x) of x <= 0 within 4 half-steps.
// exp(x) = 2^t exp(x - t ln 2), where t is the rounded x log2 e; the rest, below
// 2^-17, is worked out with ln 2 in two parts and enters to first order.  Where t is
// -inf the rest is NaN (its parts are infinities of both signs), which the maximum
// turns into a number that the power, 0, makes nothing of; NaN stays NaN by the
// power.
__device__ __forceinline__ float exp_f32(float x) {
  constexpr float kLn2 = 0.693147180559945309f;
  constexpr float kLn2Low = (float)(0.693147180559945309 - (double)kLn2);
  const float t = x * kLog2E, y = __builtin_amdgcn_exp2f(t);
  const float rest = fmaxf(fmaf(-t, kLn2Low, fmaf(-t, kLn2, x)), -1.0f);
  return fmaf(y, rest, y);
}

template <bool EXACT>
__device__ __forceinline__ float exp_of(float x) {
  return EXACT ? exp_f32(x) : fast_exp(x);
}

// The sigmoid and its slope s (1 - s), neither with a cancellation; EXACT: by
// exp_f32, so within 8 half-steps.
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float x, float& slope) {
  const float e = exp_of<EXACT>(-fabsf(x)), r = __builtin_amdgcn_rcpf(1.0f + e);
  slope = e * r * r;
  return x < 0.0f ? e * r : r;
}

__device__ __forceinline__ float fast_sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + fast_exp(-x));
}

// Quotients of scores are taken of exponentials relative to the largest logit among
// those that count: always for softmax, and for sigmoids where that logit is below
// -20, where 1 + e^x rounds to 1 and the sigmoid is e^x (further down fp32 has no
// number for it, while the quotients are ordinary ones).
__device__ __forceinline__ bool relative(int score, float largest) {
  return score == MEP_SCORE_SOFTMAX || largest < -20.0f;
}

// What to take off the logits then.  Where no score is left the exponentials of the
// logits as they are, all 0: every logit -inf, or for sigmoids below -708, where
// they leave the range of 64 bits too (masks of the type's lowest value).
__device__ __forceinline__ float shift_of(int score, float largest) {
  return largest > (score == MEP_SCORE_SOFTMAX ? -__builtin_inff() : -708.0f) ? largest : 0.0f;
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}

template <class TL>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void load(const float* p, float* v) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
  static __device__ __forceinline__ void store1(float* p, float v) { *p = v; }
};
template <>
struct Vec<uint16_t> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void load(const uint16_t* p, float* v) {
    const u32x4 q = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(q[i]);
      v[2 * i + 1] = bf16_hi(q[i]);
    }
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float* v) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = pack_bf16_rne(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<u32x4*>(p) = q;
  }
  static __device__ __forceinline__ void store1(uint16_t* p, float v) {
    *p = (uint16_t)pack_bf16_rne(v, 0.0f);
  }
};

// The expert of lane l's register i.
template <class TL, int LPT>
__device__ __forceinline__ int expert_of(int i, int l) {
  constexpr int V = Vec<TL>::V;
  return ((i / V) * LPT + l) * V + i % V;
}

// A row p of E values, T as stored; registers past E get `none`.  `wide`: E is a
// multiple of the logits' V (so of 4), rows are whole 16-byte units and a load
// never straddles E.  Without, single loads, past the end of the last value
// again: no load hides behind a branch, so all of them are in flight together.
template <class TL, int LPT, int EPL>
__device__ __forceinline__ void load_row(const TL* p, int E, int l, bool wide, float none,
                                         float (&x)[EPL]) {
  constexpr int V = Vec<TL>::V;
  if (wide) {
#pragma unroll
    for (int c = 0; c < EPL / V; ++c)
      Vec<TL>::load(p + min((c * LPT + l) * V, E - V), &x[c * V]);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = load_logit(p + min(expert_of<TL, LPT>(i, l), E - 1));
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (expert_of<TL, LPT>(i, l) >= E) x[i] = none;
}

// The same registers of a row of E 32-bit values per expert (a bias, counts).
template <class TL, int LPT, int EPL, class U>
__device__ __forceinline__ void load_per_expert(const U* p, int E, int l, bool wide, U (&x)[EPL]) {
  static_assert(sizeof(U) == 4, "");
  if (wide) {
#pragma unroll
    for (int c = 0; c < EPL / 4; ++c) {
      const int e = min(expert_of<TL, LPT>(c * 4, l), E - 4);
      const u32x4 q = *reinterpret_cast<const u32x4*>(p + e);
#pragma unroll
      for (int v = 0; v < 4; ++v) x[c * 4 + v] = __builtin_bit_cast(U, (uint32_t)q[v]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = p[min(expert_of<TL, LPT>(i, l), E - 1)];
  }
}

// ---- the router -----------------------------------------------------------

constexpr int kGateThreads = 256;

// How far apart two fp32 scores sigmoid(x) + b must be for their order to be
// the order of the exact scores.  The sigmoid's error: s (1 - s) <= 1/4 of the
// exponential's relative one, which is at most 2 + 1.5 |x| half-steps, in all
// below a half-step and a half, 2 for the reciprocal; the sum rounds once more.
// So each score is within 2^-22 (1 + |score|), and two within twice that.
__device__ __forceinline__ bool scores_apart(float hi, float lo) {
  return hi - lo > 4.76837158203125e-07f * (1.0f + fabsf(hi));
}

// k rounds of "largest first, the lowest expert among equals".  The rounds and
// not the one pass over the logits bound the kernel for many experts, so they
// are cut down to one subtraction and half a minimum a value: with all keys of
// a token different, the next key below the last one is last - 1 minus the
// smallest of last - 1 - key, where keys already taken wrap around to large
// numbers and need no removal.
//   bf16 logits: value and expert together fill the 32 bits, and that is all.
//   fp32 values: the low bits are given up for the register's number; the lane
// that has the key is found by a vote.  Where two lanes have it, or neighbours
// among the first k + 1 are equal but for those bits (about 1 token in 300 at
// 256 experts), the token's rounds are run again on the whole values, with
// removal.
//   Biased scores: the same in place of "equal" with neighbours too close for
// fp32 to order sigmoid(x) + b (about 1 token in 150), and the second time in
// fp64 over those that may be among the first k.
//   Measured, 256 experts, top 8: one token 5.2 to 5.9 us, hardly more than a
// launch; 16384 tokens, biased sigmoid scores of bf16 logits, 15.4 us (9.4 MB, which
// alone would take 2), 1156 vector instructions a wave with four waves a SIMD, 8 us
// of issue.  All scores equal, so that every token goes the 64-bit way: 29.2 us.
// Without a bias 5.9 us, of fp32 logits 9.5.
template <class TL, int LPT, int EPL, bool BIAS>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(GateArgs a) {
  constexpr int SLOTS = (kMaxTopk + LPT - 1) / LPT;  // results a lane may hold
  constexpr bool PACKED = !BIAS && sizeof(TL) == 2;
  const int l = threadIdx.x % LPT;
  const int64_t t = ((int64_t)blockIdx.x * kGateThreads + threadIdx.x) / LPT;
  const bool live = t < a.T;
  const int E = a.E, k = a.k;
  const TL* row = reinterpret_cast<const TL*>(a.logits) + (live ? t : a.T - 1) * (int64_t)E;

  float x[EPL], bias[BIAS ? EPL : 1];
  load_row<TL, LPT, EPL>(row, E, l, a.wide, -__builtin_inff(), x);
  if constexpr (BIAS) load_per_expert<TL, LPT, EPL>(a.bias, E, l, a.wide, bias);
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = expert_of<TL, LPT>(i, l);
    float s = x[i];
    if constexpr (BIAS) s = fast_sigmoid(s) + bias[i];
    key[i] = e < E ? order_key(s) : 0u;
    if (PACKED && e < E) key[i] = (key[i] & 0xffff0000u) | (uint32_t)(0xffff - e);
  }

  uint32_t got_key[SLOTS];
  int got[SLOTS];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) { got_key[s] = 1u; got[s] = 0; }
  bool again = false;  // the short keys did not decide
  [[maybe_unused]] uint32_t kth = 0;  // biased: the short key that the k-th round found
  if constexpr (PACKED) {
    uint32_t last = 0xffffffffu;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      for (int jj = 0; jj < LPT; ++jj) {
        const int j = s * LPT + jj;
        if (j >= k) break;
        uint32_t d = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < EPL; ++i) d = min(d, last - 1u - key[i]);
        last = last - 1u - group_min<LPT>(d);
        if (l == jj) {
          got_key[s] = last;
          got[s] = 0xffff - (int)(last & 0xffffu);
        }
      }
    }
    // the values back: a bf16's low half of the order's bits is all ones below
    // zero and all zeros from there on; NaN's key is 1 with the expert over it
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) got_key[s] = unpack_key(got_key[s]);
  } else {
    constexpr uint32_t LOW = EPL - 1;
    static_assert((EPL & (EPL - 1)) == 0, "");
    uint32_t last = 0xffffffffu;
    // one round more than k: the border has to be decided too
#pragma unroll
    for (int s = 0; s < SLOTS + 1; ++s) {
      for (int jj = 0; jj < LPT; ++jj) {
        const int j = s * LPT + jj;
        if (j > k || j >= E) break;
        uint32_t d = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          d = min(d, last - 1u - ((key[i] & ~LOW) | (LOW - i)));
        const uint32_t m = group_min<LPT>(d);
        const uint32_t now = last - 1u - m;
        uint64_t vote = ballot(d == m);
        if (LPT < 64) vote = vote >> (lane_id() & (64 - LPT)) & ((1ull << (LPT & 63)) - 1);
        again |= (vote & (vote - 1)) != 0 || now <= LOW;  // NaN and absent alike
        if (j > 0) {
          if (BIAS) {
            // what the low bits may hide is less than LOW + 1 units of the larger
            const float hi = key_value(last & ~LOW), lo = key_value(now | LOW);
            again |= !scores_apart(hi, lo);
          } else {
            again |= (last & ~LOW) == (now & ~LOW);
          }
        }
        last = now;
        if (BIAS && j == k - 1) kth = now;
        if (s < SLOTS && j < k && l == jj)
          got[s < SLOTS ? s : 0] =
              expert_of<TL, LPT>(LOW - (int)(now & LOW), __builtin_ctzll(vote));
      }
    }
  }
  if constexpr (BIAS) {
    // Where the order needs 64 bits: every expert whose score may be among the
    // first k goes into a list, a lane works out its entries' scores in fp64, and
    // the rounds run over those.  A list that overflows (very many equal scores)
    // is replaced by all experts.
    constexpr int CAP = 64, HAVE = CAP / LPT;
    __shared__ uint16_t lists[kGateThreads / LPT][CAP];
    if (again) {
      // Below the border nobody is among the first k.  Equal short keys leave the
      // rounds together, so all of them may have left before the k-th round, which
      // then found the largest again: fewer than k reach what it found.  The border
      // is 0 in that case, and where the k-th is -inf or NaN.
      constexpr uint32_t LOW = EPL - 1;
      uint32_t reach = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) reach += ((key[i] & ~LOW) | (LOW - i)) >= kth;
      reach = group_add<LPT>(reach);
      const float lo = key_value(kth & ~LOW);
      const uint32_t border =
          reach >= (uint32_t)k && lo > -__builtin_inff()
              ? order_key(lo - 1.9073486328125e-06f * (1.0f + fabsf(lo)))
              : 0u;
      uint16_t* list = lists[threadIdx.x / LPT];
      int n = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = expert_of<TL, LPT>(i, l);
        const bool in = e < E && key[i] >= border;
        uint64_t vote = ballot(in) >> (lane_id() & (64 - LPT));
        if (LPT < 64) vote &= (1ull << (LPT & 63)) - 1;
        const int at = n + __popcll(vote & ((1ull << l) - 1));
        if (in && at < CAP) list[at] = (uint16_t)e;
        n += __popcll(vote);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (n <= CAP) {
        uint64_t sk[HAVE];
        int se[HAVE];
#pragma unroll
        for (int h = 0; h < HAVE; ++h) {
          const int c = h * LPT + l;
          sk[h] = 0;
          se[h] = 0xffff;
          if (c < n) {
            const int e = list[c];
            se[h] = e;
            sk[h] = order_key(1.0 / (1.0 + exp(-(double)load_logit(row + e))) + (double)a.bias[e]);
          }
        }
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
          for (int jj = 0; jj < LPT; ++jj) {
            const int j = s * LPT + jj;
            if (j >= k) break;
            uint64_t best = 0;
            int be = 0xffff;
#pragma unroll
            for (int h = 0; h < HAVE; ++h) {
              if (sk[h] > best || (sk[h] == best && se[h] < be)) {
                best = sk[h];
                be = se[h];
              }
            }
            group_best<LPT>(best, be);
#pragma unroll
            for (int h = 0; h < HAVE; ++h)
              if (se[h] == be) sk[h] = 0;
            if (l == jj) got[s] = be;
          }
        }
      } else {
        uint64_t out = 0;  // this lane's registers already taken
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
          for (int jj = 0; jj < LPT; ++jj) {
            const int j = s * LPT + jj;
            if (j >= k) break;
            uint64_t best = 0;
            int be = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
              const int e = expert_of<TL, LPT>(i, l);
              if (e < E && !((out >> i) & 1)) {
                const uint64_t q =
                    order_key(1.0 / (1.0 + exp(-(double)x[i])) + (double)bias[i]);
                if (q > best) {  // registers hold ascending experts: the lowest wins
                  best = q;
                  be = e;
                }
              }
            }
            group_best<LPT>(best, be);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
              if (expert_of<TL, LPT>(i, l) == be) out |= 1ull << i;
            if (l == jj) got[s] = be;
          }
        }
      }
    }
  } else if (!PACKED && again) {
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      for (int jj = 0; jj < LPT; ++jj) {
        const int j = s * LPT + jj;
        if (j >= k) break;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) m = key[i] > m ? key[i] : m;
        m = group_max<LPT>(m);
        uint32_t e = 0xffffffffu;
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i) {
          if (key[i] == m) e = (uint32_t)expert_of<TL, LPT>(i, l);
        }
        e = group_min<LPT>(e);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if ((uint32_t)expert_of<TL, LPT>(i, l) == e) key[i] = 0u;
        if (l == jj) got[s] = (int)e;
      }
    }
  }

  // weights: lane l holds positions l, l + LPT, ...
  const bool softmax = a.score == MEP_SCORE_SOFTMAX;
  float w[SLOTS];
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    w[s] = -__builtin_inff();
    if (s * LPT + l < k) {
      if constexpr (PACKED) w[s] = key_value(got_key[s]);
      else w[s] = load_logit(row + got[s]);  // a cache hit
    }
  }
  // the largest logit that counts: the first position's, unless a bias chose it
  float m = w[0];
  if constexpr (BIAS) {
#pragma unroll
    for (int s = 1; s < SLOTS; ++s) m = fmaxf(m, w[s]);
    if (a.normalize) m = group_fmax<LPT>(m);
  } else {
    m = __shfl(m, 0, LPT);
  }
  const bool rel = softmax || (a.normalize && relative(a.score, m));
  const float shift = shift_of(a.score, m);
  float sum = 0.0f;
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    [[maybe_unused]] float slope;
    w[s] = s * LPT + l >= k ? 0.0f : rel ? exp_f32(w[s] - shift) : sigmoid<true>(w[s], slope);
    sum += w[s];
  }
  const float scale = a.scale;
  if (a.normalize || softmax) {
    if (!a.normalize) {  // softmax over all experts
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (expert_of<TL, LPT>(i, l) < E) sum += fast_exp(x[i] - shift);
    }
    sum = group_sum<LPT>(sum);
    if (sum == 0.0f) sum = 1.0f;  // no score left: all weights are 0
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) w[s] = w[s] / sum;
  }
  if (!live) return;
#pragma unroll
  for (int s = 0; s < SLOTS; ++s) {
    const int j = s * LPT + l;
    if (j < k) {
      a.indices[t * k + j] = got[s];
      a.weights[t * k + j] = w[s] * scale;
    }
  }
}

// ---- scores as probabilities ----------------------------------------------

// A token's probabilities over the experts in registers: softmax(x), or the
// sigmoids over their sum: p[i] * inv.  A row of -inf has probability 0
// everywhere.  SLOPE: sigmoid scores leave their slopes, on the scale of p, in x.
template <int LPT, int EPL, bool SLOPE>
__device__ __forceinline__ void probabilities(float (&x)[EPL], int score, float (&p)[EPL], float& m,
                                              float& inv) {
  float sum = 0.0f;
  m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < EPL; ++i) m = fmaxf(m, x[i]);
  m = group_fmax<LPT>(m);
  if (relative(score, m)) {
    const float shift = shift_of(score, m);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {  // registers past E hold -inf: exp gives 0
      p[i] = fast_exp(x[i] - shift);
      sum += p[i];
      if (SLOPE && score == MEP_SCORE_SIGMOID) x[i] = p[i];  // s (1 - s) is s down there
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      p[i] = SLOPE ? sigmoid<false>(x[i], x[i]) : fast_sigmoid(x[i]);
      sum += p[i];
    }
  }
  sum = group_sum<LPT>(sum);
  inv = sum == 0.0f ? 0.0f : 1.0f / sum;
}

// ---- balance loss ---------------------------------------------------------

// Groups of lanes sum their tokens' probabilities in registers (a lane keeps its
// experts); a wave's groups join by exchanges, a block's waves through LDS, all
// in a fixed order; named experts are counted with LDS integer atomics.  Each
// block writes a row of partial sums and counts, and the one that finishes last
// adds the rows up in order, so the result does not depend on timing.  What
// bounds it at 4096 x 256 is latency: a pass of loads, the rows' way to memory
// and back (a second launch would cost more), and the last block's loads, which
// 512 threads keep in flight 16 rows each.  16.0 us there, 8.3 for one token, 41
// for 65536 (67 MB, 1.6 TB/s).
constexpr int kBalanceThreads = 512;
constexpr int kRowsAhead = 16;  // partial rows a thread of the last block has in flight

// Threads of the last block that share a column.
__host__ __device__ constexpr int column_share(int E) {
  return E <= 64 ? 8 : E <= 128 ? 4 : E <= 256 ? 2 : 1;
}

template <class TL, int LPT, int EPL, bool WIDE>
__global__ __launch_bounds__(kBalanceThreads) void balance_kernel(BalanceArgs a) {
  constexpr int GROUPS = kBalanceThreads / LPT;
  __shared__ __attribute__((aligned(16)))
  float sums[kBalanceThreads / kWave * LPT * (LPT == 64 ? 16 : EPL)];
  extern __shared__ int cnt[];  // [E] counts and the valid tokens
  const int E = a.E, l = threadIdx.x % LPT, g = threadIdx.x / LPT;
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  for (int e = threadIdx.x; e <= E; e += kBalanceThreads) cnt[e] = 0;
  __syncthreads();

  float acc[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) acc[i] = 0.0f;
  const TL* logits = reinterpret_cast<const TL*>(a.logits);
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  // Two rows in turn: one is worked on while the other's loads run.  They are
  // taken as they lie in memory, without a branch, and looked at only when it is
  // their turn: anything else would wait for them at once.
  constexpr int V = Vec<TL>::V;
  struct Row {
    std::conditional_t<WIDE, u32x4, TL> raw[WIDE ? EPL / V : EPL];
    int32_t e;  // the lane's named expert
    uint8_t valid;
  };
  const uint8_t* mask = a.mask ? a.mask : reinterpret_cast<const uint8_t*>(a.indices);
  auto load = [&](int64_t t, Row& r) __attribute__((always_inline)) {
    const int64_t at = min(t, (int64_t)a.T - 1);
    const TL* p = logits + at * E;
    if constexpr (WIDE) {
#pragma unroll
      for (int c = 0; c < EPL / V; ++c)
        r.raw[c] = *reinterpret_cast<const u32x4*>(p + min((c * LPT + l) * V, E - V));
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) r.raw[i] = p[min(expert_of<TL, LPT>(i, l), E - 1)];
    }
    r.e = a.indices[at * a.k + min(l, a.k - 1)];
    r.valid = mask[a.mask ? at : 0];
  };
  auto work = [&](int64_t t, const Row& r) __attribute__((always_inline)) {
    if (a.mask && r.valid == 0) return;  // the same for all lanes of the group
    float x[EPL], p[EPL], m, inv;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if constexpr (!WIDE) x[i] = load_logit(&r.raw[i]);
      else if constexpr (V == 4) x[i] = __uint_as_float(r.raw[i / V][i % V]);
      else x[i] = i & 1 ? bf16_hi(r.raw[i / V][i % V / 2]) : bf16_lo(r.raw[i / V][i % V / 2]);
      if (expert_of<TL, LPT>(i, l) >= E) x[i] = -__builtin_inff();
    }
    if (l < a.k && r.e >= 0 && r.e < E) atomicAdd(&cnt[r.e], 1);
    for (int j = l + LPT; j < a.k; j += LPT) {
      const int e = a.indices[t * a.k + j];
      if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
    }
    if (l == 0) atomicAdd(&cnt[E], 1);
    probabilities<LPT, EPL, false>(x, a.score, p, m, inv);
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] += p[i] * inv;
  };
  int64_t t = (int64_t)blockIdx.x * GROUPS + g;
  if constexpr (EPL == 64) {  // two would not fit the registers
    for (; t < a.T; t += step) {
      Row row;
      load(t, row);
      work(t, row);
    }
  } else if (t < a.T) {
    Row even, odd;
    load(t, even);
    while (true) {
      load(t + step, odd);
      work(t, even);
      if ((t += step) >= a.T) break;
      load(t + step, even);
      work(t, odd);
      if ((t += step) >= a.T) break;
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
#pragma unroll
    for (int d = LPT; d < kWave; d <<= 1) acc[i] += __shfl_xor(acc[i], d);
  }
  // waves: CHUNK registers of each at a time, which hold WIDTH neighbouring experts
  constexpr int WAVES = kBalanceThreads / kWave;
  constexpr int CHUNK = LPT == 64 ? 16 : EPL, WIDTH = CHUNK * LPT;
  float* part = a.part_sum + (size_t)blockIdx.x * E;
#pragma unroll
  for (int c = 0; c < EPL; c += CHUNK) {
    const int e0 = c * LPT;
    if (e0 >= E) break;
    if (c > 0) __syncthreads();
    if (lane < LPT) {
#pragma unroll
      for (int i = 0; i < CHUNK; i += 4)
        *reinterpret_cast<float4*>(sums + wave * WIDTH + expert_of<TL, LPT>(c + i, l) - e0) =
            make_float4(acc[c + i], acc[c + i + 1], acc[c + i + 2], acc[c + i + 3]);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < WIDTH && e0 + e < E; e += kBalanceThreads) {
      float s = sums[e];
#pragma unroll
      for (int q = 1; q < WAVES; ++q) s += sums[q * WIDTH + e];
      part[e0 + e] = s;
    }
  }
  int32_t* pcnt = a.part_cnt + (size_t)blockIdx.x * (E + 1);
  for (int e = threadIdx.x; e <= E; e += kBalanceThreads) pcnt[e] = cnt[e];

  // the last block to arrive joins the partial rows
  __shared__ int is_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) is_last = atomicAdd(a.done, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  __shared__ double join[kBalanceThreads];
  __shared__ int32_t join_cnt[kBalanceThreads];
  const int rows = (int)gridDim.x;
  // valid tokens: needed at the end, loaded now
  int32_t n = 0;
  for (int r = lane; r < rows; r += kWave) n += a.part_cnt[(size_t)r * (E + 1) + E];
  // `share` threads a column, each every share-th row
  const int share = column_share(E);
  const int width = kBalanceThreads / share;
  const int c = threadIdx.x % width, part_of = threadIdx.x / width;
  double mine = 0.0;
  for (int e0 = 0; e0 < E; e0 += width) {
    const int e = e0 + c;
    double s = 0.0;
    int32_t q = 0;
    if (e < E) {
      for (int r0 = part_of; r0 < rows; r0 += kRowsAhead * share) {
        float v[kRowsAhead];
        int32_t w[kRowsAhead];
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
          const int r = min(r0 + u * share, rows - 1);
          v[u] = a.part_sum[(size_t)r * E + e];
          w[u] = a.part_cnt[(size_t)r * (E + 1) + e];
        }
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
          if (r0 + u * share < rows) {
            s += (double)v[u];
            q += w[u];
          }
        }
      }
    }
    if (e0 == 0)
      for (int d = 1; d < kWave; d <<= 1) n += __shfl_xor(n, d);
    const double inv_n = n > 0 ? 1.0 / (double)n : 0.0;
    __syncthreads();
    join[threadIdx.x] = s;
    join_cnt[threadIdx.x] = q;
    __syncthreads();
    if (part_of == 0 && e < E) {
      for (int u = 1; u < share; ++u) {
        s += join[u * width + c];
        q += join_cnt[u * width + c];
      }
      const double mean = s * inv_n;
      a.counts[e] = q;
      a.prob_mean[e] = (float)mean;
      mine += (double)q * mean;
    }
  }
  __syncthreads();
  for (int d = 1; d < kWave; d <<= 1) mine += __shfl_xor(mine, d);
  if (lane == 0) join[wave] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int i = 0; i < kBalanceThreads / kWave; ++i) s += join[i];
    a.counts[E] = n;
    const double inv_n = n > 0 ? 1.0 / (double)n : 0.0;
    a.loss[0] = (float)(s * inv_n * (double)a.coef * (double)E / (double)a.k);
    *a.done = 0u;  // ready for the next call on this workspace
  }
}

// ---- gradient -------------------------------------------------------------

// One pass over the logits gives both gradients.  The loss: with
// u_e = dL/dp_e = grad_loss coef E c_e / (k n^2),
//   softmax:  dx = p (u - sum u p),   sigmoid:  dx = s (1 - s) / S (u - sum u p).
// The weights: only selected experts receive a gradient of their own; lane j
// works out position j's and adds it through the group's row in LDS, a
// repeated expert's positions added up in order first.  Bound by the launch and
// one trip to memory: 6.6 to 7.0 us at 4096 tokens of 256 fp32 logits (8.7 MB), 8.6
// at 30011 of 60 bf16 logits, whose rows do not start on 16 bytes and are loaded and
// stored value by value.
constexpr int kGradThreads = 256;

template <class TL, int LPT, int EPL>
__global__ __launch_bounds__(kGradThreads) void gate_backward_kernel(GateBackwardArgs a) {
  constexpr int SLOTS = (kMaxTopk + LPT - 1) / LPT;
  extern __shared__ float lds[];  // [groups][E]: what the weights' gradient adds
  const int l = threadIdx.x % LPT, g = threadIdx.x / LPT;
  const int E = a.E, k = a.k;
  const int64_t t = (int64_t)blockIdx.x * (kGradThreads / LPT) + g;
  const bool live = t < a.T;
  const int64_t tt = live ? t : a.T - 1;
  const bool valid = !a.mask || a.mask[tt] != 0;
  const TL* row = reinterpret_cast<const TL*>(a.logits) + tt * E;
  float* extra = lds + (size_t)g * E;

  float x[EPL], p[EPL], m, inv;
  load_row<TL, LPT, EPL>(row, E, l, a.wide, -__builtin_inff(), x);
  probabilities<LPT, EPL, true>(x, a.score, p, m, inv);
  const bool softmax = a.score == MEP_SCORE_SOFTMAX;

  // the loss' gradient for each expert's probability
  float u[EPL], dot = 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) u[i] = 0.0f;
  if (a.counts) {
    int32_t cnt[EPL];
    load_per_expert<TL, LPT, EPL>(a.counts, E, l, a.wide, cnt);
    const double n = (double)a.counts[E];
    const float coef =
        n > 0 ? (float)((double)a.grad_loss[0] * (double)a.coef * E / (k * n * n)) : 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      u[i] = coef * (float)cnt[i];
      dot += u[i] * (p[i] * inv);  // p is 0 past E
    }
    dot = group_sum<LPT>(dot);
  }

  // the weights' gradient for each position
  float shift = 0.0f;  // unnormalised softmax: sum over positions of g p, taken off every expert
  if (a.grad_weights) {
    for (int e = l; e < E; e += LPT) extra[e] = 0.0f;
    int id[SLOTS];
    float v[SLOTS], d[SLOTS], gw[SLOTS];
    float total = 0.0f, gsum = 0.0f, top = -__builtin_inff();
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int j = s * LPT + l;
      id[s] = -1;
      v[s] = -__builtin_inff();
      gw[s] = 0.0f;
      if (j < k) {
        const int e = a.indices[tt * k + j];
        if (e >= 0 && e < E) {
          id[s] = e;
          gw[s] = a.scale * a.grad_weights[tt * k + j];
          v[s] = load_logit(row + e);
        }
      }
      top = fmaxf(top, v[s]);
    }
    // the named experts may lie far below the largest logit (an earlier routing's)
    if (a.normalize) top = group_fmax<LPT>(top); else top = m;
    const bool rel = softmax || (a.normalize && relative(a.score, top));
    const float from = shift_of(a.score, top);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      if (id[s] < 0) v[s] = d[s] = 0.0f;
      else if (rel) v[s] = d[s] = exp_f32(v[s] - from);  // of a sigmoid the slope too
      else v[s] = sigmoid<true>(v[s], d[s]);
      total += v[s];
      gsum += gw[s] * v[s];
    }
    total = group_sum<LPT>(total);
    gsum = group_sum<LPT>(gsum);
    const float tinv = total == 0.0f ? 0.0f : 1.0f / total;
    float add[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      if (softmax)
        add[s] = a.normalize ? v[s] * tinv * (gw[s] - gsum * tinv) : v[s] * inv * gw[s];
      else
        add[s] = a.normalize ? d[s] * tinv * (gw[s] - gsum * tinv) : d[s] * gw[s];
    }
    if (softmax && !a.normalize) shift = gsum * inv;
    __syncthreads();
    // a repeated expert: its first position adds up all of them
    float sum[SLOTS];
    bool mine[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) { sum[s] = 0.0f; mine[s] = id[s] >= 0; }
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      for (int jj = 0; jj < LPT; ++jj) {
        const int j = s * LPT + jj;
        if (j >= k) break;
        const int oe = __shfl(id[s], jj, LPT);
        const float oa = __shfl(add[s], jj, LPT);
#pragma unroll
        for (int q = 0; q < SLOTS; ++q) {
          if (oe == id[q]) {
            sum[q] += oa;
            if (j < q * LPT + l) mine[q] = false;
          }
        }
      }
    }
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
      if (mine[s]) extra[id[s]] = sum[s];
    __syncthreads();
  }

  if (!live) return;
  TL* out = reinterpret_cast<TL*>(a.grad_logits) + t * E;
  float r[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = expert_of<TL, LPT>(i, l);
    float v;
    if (softmax)
      v = p[i] * inv * (u[i] - dot - shift);
    else
      v = x[i] * inv * (u[i] - dot);
    if (a.grad_weights && e < E) v += extra[e];
    r[i] = valid ? v : 0.0f;
  }
  constexpr int V = Vec<TL>::V;
  if (a.wide) {
#pragma unroll
    for (int c = 0; c < EPL / V; ++c) {
      const int e = (c * LPT + l) * V;
      if (e < E) Vec<TL>::store(out + e, &r[c * V]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = expert_of<TL, LPT>(i, l);
      if (e < E) Vec<TL>::store1(out + e, r[i]);
    }
  }
}

// ---- launches -------------------------------------------------------------

// Calls f with the (lanes, values a lane) that hold E experts.
template <class F>
void by_experts(int E, F f) {
  using std::integral_constant;
  if (E <= 64) f(integral_constant<int, 8>{}, integral_constant<int, 8>{});
  else if (E <= 128) f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  else if (E <= 256) f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  else if (E <= 512) f(integral_constant<int, 16>{}, integral_constant<int, 32>{});
  else if (E <= 1024) f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
  else f(integral_constant<int, 64>{}, integral_constant<int, 64>{});
}

int lanes_of(int E) { return E <= 64 ? 8 : E <= 512 ? 16 : 64; }

template <class TL>
void gate_typed(const GateArgs& a, hipStream_t s) {
  const int64_t threads = (int64_t)a.T * lanes_of(a.E);
  const unsigned blocks = (unsigned)((threads + kGateThreads - 1) / kGateThreads);
  by_experts(a.E, [&](auto lpt, auto epl) {
    if (a.bias)
      gate_kernel<TL, lpt(), epl(), true><<<blocks, kGateThreads, 0, s>>>(a);
    else
      gate_kernel<TL, lpt(), epl(), false><<<blocks, kGateThreads, 0, s>>>(a);
  });
}

}  // namespace

static bool is_wide(int E, int dtype) { return E % (dtype == MEP_BF16 ? 8 : 4) == 0; }

// A launch has fewer than 2^32 threads, and a token up to 64 of them: larger
// batches go in parts.
constexpr int32_t kTokensALaunch = 1 << 25;

// Calls f(first token, tokens) for each part.
template <class F>
static hipError_t in_parts(int32_t T, F f) {
  for (int64_t t = 0; t < T; t += kTokensALaunch) {
    f(t, (int32_t)std::min<int64_t>(kTokensALaunch, T - t));
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

static const void* logits_at(const void* logits, int64_t values, int dtype) {
  return (const unsigned char*)logits + values * (dtype == MEP_BF16 ? 2 : 4);
}

hipError_t launch_gate(const GateArgs& a0, hipStream_t s) {
  return in_parts(a0.T, [&](int64_t t, int32_t n) {
    GateArgs a = a0;
    a.T = n;
    a.logits = logits_at(a0.logits, t * a.E, a.dtype);
    a.indices += t * a.k;
    a.weights += t * a.k;
    a.wide = is_wide(a.E, a.dtype);
    if (a.dtype == MEP_BF16) gate_typed<uint16_t>(a, s);
    else gate_typed<float>(a, s);
  });
}

// Blocks: a pass over one token a group takes about 0.6 us, and each block's
// arrival at the counter, which they reach one by one, about 0.08, so the square
// root of 7.5 passes.  Measured with the square root of 4, of 7.5 and of 10 (us):
// 4096 tokens over 256 experts 16.2, 15.9 and 17.6, 65536 tokens 39.9, 41.5 and
// 43.6, 1024 tokens over 512 experts 16.0, 15.2 and 16.6.
int balance_blocks(int E, int64_t T) {
  const int64_t groups = kBalanceThreads / lanes_of(E);
  const int64_t passes = std::max<int64_t>(1, (T + groups - 1) / groups);
  int64_t b = 1;
  while (b < 256 && 2 * b * b < 15 * passes) ++b;
  return (int)std::min(passes, b);
}

hipError_t launch_balance(const BalanceArgs& a, hipStream_t s) {
  const unsigned blocks = (unsigned)balance_blocks(a.E, a.T);
  by_experts(a.E, [&](auto lpt, auto epl) {
    const size_t lds = (size_t)(a.E + 1) * 4;
    auto launch = [&](auto type, auto wide) {
      balance_kernel<decltype(type), lpt(), epl(), wide()>
          <<<blocks, kBalanceThreads, lds, s>>>(a);
    };
    const bool wide = is_wide(a.E, a.dtype);
    using Yes = std::true_type;
    using No = std::false_type;
    if (a.dtype == MEP_BF16) {
      if (wide) launch(uint16_t{}, Yes{}); else launch(uint16_t{}, No{});
    } else {
      if (wide) launch(float{}, Yes{}); else launch(float{}, No{});
    }
  });
  return hipGetLastError();
}

hipError_t launch_gate_backward(const GateBackwardArgs& a0, hipStream_t s) {
  return in_parts(a0.T, [&](int64_t t, int32_t n) {
    GateBackwardArgs a = a0;
    a.T = n;
    a.logits = logits_at(a0.logits, t * a.E, a.dtype);
    a.grad_logits = const_cast<void*>(logits_at(a0.grad_logits, t * a.E, a.dtype));
    a.indices += t * a.k;
    if (a.mask) a.mask += t;
    if (a.grad_weights) a.grad_weights += t * a.k;
    a.wide = is_wide(a.E, a.dtype);
    by_experts(a.E, [&](auto lpt, auto epl) {
      const int groups = kGradThreads / lpt();
      const unsigned blocks = (unsigned)((a.T + groups - 1) / groups);
      const size_t lds = a.grad_weights ? (size_t)groups * a.E * 4 : 0;
      if (a.dtype == MEP_BF16)
        gate_backward_kernel<uint16_t, lpt(), epl()><<<blocks, kGradThreads, lds, s>>>(a);
      else
        gate_backward_kernel<float, lpt(), epl()><<<blocks, kGradThreads, lds, s>>>(a);
    });
  });
}

}  // namespace mep
