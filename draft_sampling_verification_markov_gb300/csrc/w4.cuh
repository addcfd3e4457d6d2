// w4.cuh -- what the kernels of grouped 4-bit weights share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "row_pieces.cuh"

namespace spec {
namespace w4 {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kBlock = 128;     // codes of a row that a warp takes at once

__host__ __device__ constexpr int padded(int K) { return (K + kBlock - 1) / kBlock * kBlock; }

// Eight consecutive bf16 elements of a row, zeros past K.
__device__ __forceinline__ uint4 load8_bf16(const void* p, size_t row, int k, int K) {
  const uint16_t* at = static_cast<const uint16_t*>(p) + row + k;
  if (k + 8 <= K && (reinterpret_cast<uintptr_t>(at) & 15) == 0) return ld_coherent16(at);
  uint32_t w[4] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < K) w[i / 2] |= (uint32_t)at[i] << (i & 1 ? 16 : 0);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight consecutive elements of a row as fp32, zeros past K.
__device__ __forceinline__ void load8(const void* p, int dt, size_t row, int k, int K,
                                      float (&v)[8]) {
  if (dt == SPEC_BF16) {
    const uint4 q = load8_bf16(p, row, k, K);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float* at = static_cast<const float*>(p) + row + k;
    if (k + 8 <= K && (reinterpret_cast<uintptr_t>(at) & 15) == 0) {
      const uint4 a = ld_coherent16(at), b = ld_coherent16(at + 4);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = k + i < K ? at[i] : 0.0f;
    }
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ void store8_bf16(void* p, size_t row, int k, int K,
                                            const uint32_t (&w)[4]) {
  uint16_t* at = static_cast<uint16_t*>(p) + row + k;
  if (k + 8 <= K && (reinterpret_cast<uintptr_t>(at) & 15) == 0) {
    *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < K) at[i] = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
  }
}

__device__ __forceinline__ void store8(void* p, int dt, size_t row, int k, int K,
                                       const float (&v)[8]) {
  if (dt == SPEC_BF16) {
    const uint32_t w[4] = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                           bf16_pair(v[6], v[7])};
    store8_bf16(p, row, k, K, w);
  } else {
    float* at = static_cast<float*>(p) + row + k;
    if (k + 8 <= K && (reinterpret_cast<uintptr_t>(at) & 15) == 0) {
      *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(at + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < K) at[i] = v[i];
    }
  }
}

// Four consecutive elements of a row, of which `left` have a place.
__device__ __forceinline__ void store4(float* at, int left, const float (&v)[4]) {
  if (left >= 4 && (reinterpret_cast<uintptr_t>(at) & 15) == 0) {
    *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) at[i] = v[i];
  }
}

__device__ __forceinline__ float load_scale(const void* p, int dt, size_t at) {
  return dt == SPEC_BF16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[at])
                         : static_cast<const float*>(p)[at];
}

// Largest number of columns of a chunk, shared memory of its rows, threads of the product's CTAs.
constexpr int kColumns = 40;
constexpr size_t kRowsMost = 144 * 1024;
constexpr size_t kSmemMost = 225 * 1024;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
// Shared memory of a CTA beside its rings, and of one tile of every ring with its barrier.
__host__ __device__ constexpr int red_stride(int rows) { return rows | 1; }
__host__ __device__ constexpr int pieces_of(int K) { return (padded(K) / 8 + 31) / 32; }
inline size_t rest_bytes(int K, int rows, int parts, int R) {
  return (size_t)padded(K) * 2 * rows * parts + 1024 +
         sizeof(float) * ((size_t)kWarps * 16 * R * red_stride(rows) + rows * (2 + 2 * pieces_of(K)));
}
// Tiles of a warp, of KT that kw warps share: whole multiples of `whole`.
__host__ __device__ constexpr int tiles_of(int KT, int kw, int whole) {
  const int n = (KT + kw - 1) / kw, q = whole > 1 ? whole : 1;
  return (n + q - 1) / q * q;
}
inline size_t stage_bytes(int R, int W) { return (size_t)kWarps * (16 * R * 64 * W + 8); }
// A form of the product: tiles of 16 R matrix rows and W blocks, 8 T columns.
struct Form {
  int R, T, W;
};
// The product for one group size (w4_g32.cu, w4_g64.cu, w4_g128.cu).
cudaError_t launch_g32(const W4Args& a, const CUtensorMap& codes, Form form, cudaStream_t s);
cudaError_t launch_g64(const W4Args& a, const CUtensorMap& codes, Form form, cudaStream_t s);
cudaError_t launch_g128(const W4Args& a, const CUtensorMap& codes, Form form, cudaStream_t s);

}  // namespace w4
}  // namespace spec
