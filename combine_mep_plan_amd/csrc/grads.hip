// The global norm of many gradients, and their clipping by it.
//
// The tensors are cut into chunks of 32 KiB; a table of the tensors and of each one's
// first chunk goes along in the launch's arguments (128 tensors a launch), so that a
// list of any sizes is one grid of equal pieces of work and needs no memory of its own.
//
// Bound by memory: 2.8 GB of gradients (1.4 billion values, nearly all bf16) have their norm
// in 458 us (6.2 TB/s, loads alone) and are clipped into buffers of their own in 1050 (5.4
// TB/s).  59 tensors of 1.1 MB together take 8.5 us in three launches, of which calls one by
// one need 15 on the host.
#include <algorithm>

#include "dev.h"
#include "mep_internal.h"

namespace mep {

namespace {

constexpr int kGradThreads = 256;
constexpr int kChunkBytes = 32768;  // 16 KiB: 2.8 GB clipped 0.6% slower
constexpr uint32_t kGradBlocks = 2048;  // blocks of the norm's launches at most: one sum each
constexpr uint32_t kClipBlocks = 8192;  // of the clipping's: 1% faster than 4096, 2% than 2048
constexpr int kPieces = kChunkBytes / 16 / kGradThreads;  // 16-byte pieces a thread

// The tensor that holds a chunk: the last one that starts at or before it.
__device__ __forceinline__ int tensor_of(const GradTable& t, uint32_t chunk) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

struct Chunk {
  const void* data;
  void* out;
  int64_t at;   // first value
  int count;    // values
  bool bf16;
};

__device__ __forceinline__ Chunk chunk_of(const GradTable& t, uint32_t chunk) {
  const int i = tensor_of(t, chunk);
  const int64_t nt = t.numel_type[i];
  const bool bf16 = nt & 1;
  const int per = bf16 ? kChunkBytes / 2 : kChunkBytes / 4;
  const int64_t at = (int64_t)(chunk - t.first[i]) * per;
  return {t.data[i], t.out[i], at, (int)min((int64_t)per, (nt >> 1) - at), bf16};
}

// 16 bytes of a gradient: 8 bf16 or 4 fp32 values.
template <bool BF16>
struct Piece {
  static constexpr int N = BF16 ? 8 : 4;
  u32x4 q;

  __device__ __forceinline__ float at(int i) const {
    if (!BF16) return __uint_as_float(q[i & 3]);
    return i & 1 ? bf16_hi(q[i / 2]) : bf16_lo(q[i / 2]);
  }
  __device__ __forceinline__ void scale(float f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = BF16 ? pack_bf16_pair(bf16_lo(q[i]) * f, bf16_hi(q[i]) * f)
                  : __float_as_uint(__uint_as_float(q[i]) * f);
  }
};

// Calls whole(piece number, pieces) once for the thread's pieces of a chunk, all of them
// loaded before the first is looked at, and single(value's number) for values behind
// the last whole piece.
template <bool BF16, class Whole, class Single>
__device__ __forceinline__ void over_chunk(const Chunk& k, Whole whole, Single single) {
  using P = Piece<BF16>;
  const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const unsigned char*>(k.data) +
                                                  k.at * (BF16 ? 2 : 4));
  const int pieces = k.count / P::N;
  P v[kPieces];
  if (pieces == kPieces * kGradThreads) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) v[i].q = p[i * kGradThreads + threadIdx.x];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) whole(i * kGradThreads + (int)threadIdx.x, v[i]);
    return;
  }
  for (int q = threadIdx.x; q < pieces; q += kGradThreads) {
    v[0].q = p[q];
    whole(q, v[0]);
  }
  const int rest = pieces * P::N + threadIdx.x;
  if (rest < k.count) single(rest);
}

__device__ __forceinline__ double block_sum(double v, double* join) {
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
  if (lane_id() == 0) join[threadIdx.x / kWave] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kGradThreads / kWave; ++i) s += join[i];
  return s;
}

// Squares are added up in fp64: they neither overflow nor vanish, whatever the
// gradients, and the sum of billions of them is as good as its inputs.
template <bool BF16>
__device__ __forceinline__ double chunk_squares(const Chunk& k) {
  double s = 0.0;
  auto add = [&](float v) { s = fma((double)v, (double)v, s); };
  over_chunk<BF16>(
      k,
      [&](int, const Piece<BF16>& v) {
#pragma unroll
        for (int j = 0; j < Piece<BF16>::N; ++j) add(v.at(j));
      },
      [&](int i) {
        if (BF16) add(bf16_lo(reinterpret_cast<const uint16_t*>(k.data)[k.at + i]));
        else add(reinterpret_cast<const float*>(k.data)[k.at + i]);
      });
  return s;
}

__global__ __launch_bounds__(kGradThreads) void grad_norm_kernel(GradTable t, double* part) {
  __shared__ double join[kGradThreads / kWave];
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) {
    const Chunk k = chunk_of(t, c);
    s += k.bf16 ? chunk_squares<true>(k) : chunk_squares<false>(k);
  }
  s = block_sum(s, join);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// All blocks' sums, in order.  A launch of its own: a counter that every block of the
// first one passes costs 0.08 us a block, 160 us at 2048 blocks.
__global__ __launch_bounds__(kGradThreads) void grad_join_kernel(const double* part, int n,
                                                                 float* norm) {
  __shared__ double join[kGradThreads / kWave];
  double s = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < n; i += kGradThreads) s += part[i];
  s = block_sum(s, join);
  if (threadIdx.x == 0) norm[0] = (float)sqrt(s);
}

// Stores go past the caches: nothing here reads them again (0.4% at 2.8 GB).
template <bool BF16>
__device__ __forceinline__ void clip_chunk(const Chunk& k, float f) {
  over_chunk<BF16>(
      k,
      [&](int q, Piece<BF16>& v) {
        v.scale(f);
        store_nt(reinterpret_cast<u32x4*>(reinterpret_cast<unsigned char*>(k.out) +
                                          k.at * (BF16 ? 2 : 4)) + q, v.q);
      },
      [&](int i) {
        if (BF16)
          reinterpret_cast<uint16_t*>(k.out)[k.at + i] = (uint16_t)pack_bf16_pair(
              bf16_lo(reinterpret_cast<const uint16_t*>(k.data)[k.at + i]) * f, 0.0f);
        else
          reinterpret_cast<float*>(k.out)[k.at + i] =
              reinterpret_cast<const float*>(k.data)[k.at + i] * f;
      });
}

__global__ __launch_bounds__(kGradThreads) void grad_clip_kernel(GradTable t, const float* norm,
                                                                 float max_norm, bool in_place) {
  const float f = max_norm / (norm[0] + 1e-6f);
  // Not for NaN; without a limit nothing is over it, an infinite norm neither.
  const bool keep = f >= 1.0f || (max_norm == __builtin_inff() && norm[0] == __builtin_inff());
  if (keep && in_place) return;
  const float factor = keep ? 1.0f : f;
  const uint32_t chunks = t.first[t.n];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Chunk k = chunk_of(t, c);
    if (keep && k.data == k.out) continue;
    if (k.bf16) clip_chunk<true>(k, factor);
    else clip_chunk<false>(k, factor);
  }
}

}  // namespace

uint32_t grad_chunks(int64_t numel, bool bf16) {
  const int64_t per = bf16 ? kChunkBytes / 2 : kChunkBytes / 4;
  return (uint32_t)((numel + per - 1) / per);
}

int32_t grad_norm_blocks(const GradTable& t) {
  return (int32_t)std::max<uint32_t>(1, std::min<uint32_t>(t.first[t.n], kGradBlocks));
}

hipError_t launch_grad_norm(const GradTable& t, double* part, hipStream_t s) {
  grad_norm_kernel<<<grad_norm_blocks(t), kGradThreads, 0, s>>>(t, part);
  return hipGetLastError();
}

hipError_t launch_grad_join(const double* part, int32_t n, float* norm, hipStream_t s) {
  grad_join_kernel<<<1, kGradThreads, 0, s>>>(part, n, norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradTable& t, const float* norm, float max_norm, hipStream_t s) {
  const unsigned blocks = std::min<uint32_t>(t.first[t.n], kClipBlocks);
  if (blocks == 0) return hipSuccess;
  bool in_place = true;
  for (int i = 0; i < t.n; ++i) in_place &= t.data[i] == t.out[i];
  grad_clip_kernel<<<blocks, kGradThreads, 0, s>>>(t, norm, max_norm, in_place);
  return hipGetLastError();
}

}  // namespace mep
