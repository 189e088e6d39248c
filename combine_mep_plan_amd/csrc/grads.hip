// The global norm of many gradients, and their clipping by it.
//
// The tensors are cut into chunks of 32 KiB; a table of the tensors and of each one's
// first chunk goes along in the launch's arguments (128 tensors a launch), so that a
// list of any sizes is one grid of equal pieces of work and needs no memory of its own.
#include <algorithm>

#include "dev.h"
#include "mep_internal.h"

namespace mep {

namespace {

constexpr int kGradThreads = 256;
constexpr int kChunkBytes = 32768;
constexpr uint32_t kGradBlocks = 2048;  // blocks a launch has at most
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

// Squares are added up in fp64: they neither overflow nor vanish, whatever the
// gradients, and the sum of billions of them is as good as its inputs.
__device__ __forceinline__ void add_square(double& s, float v) { s = fma((double)v, (double)v, s); }

__device__ __forceinline__ double block_sum(double v, double* join) {
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if (lane_id() == 0) join[threadIdx.x / kWave] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kGradThreads / kWave; ++i) s += join[i];
  return s;
}

__global__ __launch_bounds__(kGradThreads) void grad_norm_kernel(GradTable t, GradNormArgs a) {
  __shared__ double join[kGradThreads / kWave];
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < t.first[t.n]; c += gridDim.x) {
    const Chunk k = chunk_of(t, c);
    if (k.bf16) {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(k.data) + k.at;
      const int pieces = k.count / 8;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int q = i * kGradThreads + threadIdx.x;
        if (q < pieces) {
          const u32x4 v = reinterpret_cast<const u32x4*>(p)[q];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            add_square(s, bf16_lo(v[j]));
            add_square(s, bf16_hi(v[j]));
          }
        }
      }
      const int rest = pieces * 8 + threadIdx.x;
      if (rest < k.count) add_square(s, bf16_lo(p[rest]));
    } else {
      const float* p = reinterpret_cast<const float*>(k.data) + k.at;
      const int pieces = k.count / 4;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int q = i * kGradThreads + threadIdx.x;
        if (q < pieces) {
          const float4 v = reinterpret_cast<const float4*>(p)[q];
          add_square(s, v.x);
          add_square(s, v.y);
          add_square(s, v.z);
          add_square(s, v.w);
        }
      }
      const int rest = pieces * 4 + threadIdx.x;
      if (rest < k.count) add_square(s, p[rest]);
    }
  }
  s = block_sum(s, join);
  if (threadIdx.x == 0) a.part[a.first_part + blockIdx.x] = s;
  if (a.parts == 0) return;  // another launch follows
  // the last block to arrive adds up all blocks' sums, in order
  __shared__ int is_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) is_last = atomicAdd(a.done, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  s = 0.0;
  for (int i = threadIdx.x; i < a.parts; i += kGradThreads) s += a.part[i];
  s = block_sum(s, join);
  if (threadIdx.x == 0) {
    a.norm[0] = (float)sqrt(s);
    *a.done = 0u;  // ready for the next call on this workspace
  }
}

__global__ __launch_bounds__(kGradThreads) void grad_clip_kernel(GradTable t, const float* norm,
                                                                 float max_norm) {
  const float f = max_norm / (norm[0] + 1e-6f);
  const bool keep = f >= 1.0f;  // not for NaN
  const float factor = keep ? 1.0f : f;
  const uint32_t chunks = t.first[t.n];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Chunk k = chunk_of(t, c);
    if (keep && k.data == k.out) continue;
    if (k.bf16) {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(k.data) + k.at;
      uint16_t* o = reinterpret_cast<uint16_t*>(k.out) + k.at;
      const int pieces = k.count / 8;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int q = i * kGradThreads + threadIdx.x;
        if (q < pieces) {
          u32x4 v = reinterpret_cast<const u32x4*>(p)[q];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = pack_bf16_rne(bf16_lo(v[j]) * factor, bf16_hi(v[j]) * factor);
          reinterpret_cast<u32x4*>(o)[q] = v;
        }
      }
      const int rest = pieces * 8 + threadIdx.x;
      if (rest < k.count) o[rest] = (uint16_t)pack_bf16_rne(bf16_lo(p[rest]) * factor, 0.0f);
    } else {
      const float* p = reinterpret_cast<const float*>(k.data) + k.at;
      float* o = reinterpret_cast<float*>(k.out) + k.at;
      const int pieces = k.count / 4;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int q = i * kGradThreads + threadIdx.x;
        if (q < pieces) {
          float4 v = reinterpret_cast<const float4*>(p)[q];
          v.x *= factor; v.y *= factor; v.z *= factor; v.w *= factor;
          reinterpret_cast<float4*>(o)[q] = v;
        }
      }
      const int rest = pieces * 4 + threadIdx.x;
      if (rest < k.count) o[rest] = p[rest] * factor;
    }
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

hipError_t launch_grad_norm(const GradTable& t, const GradNormArgs& a, hipStream_t s) {
  grad_norm_kernel<<<grad_norm_blocks(t), kGradThreads, 0, s>>>(t, a);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradTable& t, const float* norm, float max_norm, hipStream_t s) {
  const unsigned blocks = std::min<uint32_t>(t.first[t.n], kGradBlocks);
  if (blocks == 0) return hipSuccess;
  grad_clip_kernel<<<blocks, kGradThreads, 0, s>>>(t, norm, max_norm);
  return hipGetLastError();
}

}  // namespace mep
