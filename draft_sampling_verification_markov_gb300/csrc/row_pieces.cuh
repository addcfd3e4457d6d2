// row_pieces.cuh -- a logit row as 16-byte pieces, and the order of its tokens as integer keys.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace spec {

// Ordered bits: larger floats have larger bits, zeros of both signs are equal. 0 stands for
// "no place" (NaN and -inf).
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (!(x > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
__device__ __forceinline__ unsigned long long make_key(uint32_t bits, int id) {
  return ((unsigned long long)bits << 32) | (0xffffffffu - (uint32_t)id);
}

// ------------------------------------------------------------------------------ a row's pieces

// A row as 16-byte pieces at 16-byte aligned addresses: piece j holds ids j * N - head ...; the
// first and the last piece may be partly outside the row.
template <int DT>
struct Row {
  static constexpr int N = DT == SPEC_BF16 ? 8 : 4;
  const char* base;  // address of piece 0
  int head, V;

  __device__ Row(const void* x, size_t off, int V_) : V(V_) {
    const char* p = static_cast<const char*>(x) + off * (16 / N);
    const int mis = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    base = p - mis;
    head = mis / (16 / N);
  }
  __device__ int pieces() const { return (head + V + N - 1) / N; }

  // Pieces jb + thread + b * THREADS, b < B.
  template <int B, int THREADS>
  __device__ __forceinline__ void load_batch(uint4 (&q)[B], int jb, int end) const;

  static constexpr uint32_t kNone = DT == SPEC_BF16 ? 0xff80ff80u : 0xff800000u;  // -inf

  // Piece j, with -inf outside the row and past `end`. A row has at most two pieces that are
  // partly outside; they go through a call of their own, so that the loads of whole ones stay in
  // flight together.
  __device__ __forceinline__ uint4 load(int j, int end) const {
    uint4 q = make_uint4(kNone, kNone, kNone, kNone);
    if (j < end) {
      const int v = j * N - head;
      if (v >= 0 && v + N <= V) q = ld_coherent16(base + (size_t)j * 16);
    }
    return q;
  }
  __device__ __forceinline__ bool partial(int j, int end) const {
    const int v = j * N - head;
    return j < end && (v < 0 || v + N > V);
  }
  __device__ __noinline__ uint4 load_partial(int j) const {
    uint32_t w[4] = {kNone, kNone, kNone, kNone};
    const int v = j * N - head;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (v + i < 0 || v + i >= V) continue;
      if constexpr (DT == SPEC_BF16) {
        const uint32_t b = reinterpret_cast<const uint16_t*>(base + (size_t)j * 16)[i];
        w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | b << 16 : (w[i / 2] & 0xffff0000u) | b;
      } else {
        w[i] = reinterpret_cast<const uint32_t*>(base + (size_t)j * 16)[i];
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // Either kind.
  __device__ __forceinline__ uint4 load_any(int j, int end) const {
    return partial(j, end) ? load_partial(j) : load(j, end);
  }
};

template <int DT>
template <int B, int THREADS>
__device__ __forceinline__ void Row<DT>::load_batch(uint4 (&q)[B], int jb, int end) const {
  const int j = jb + threadIdx.x;
  // whole batches inside the row: one address, no tests of single pieces
  if (jb * N >= head && jb + B * THREADS <= end && (jb + B * THREADS) * N - head <= V) {
    const char* p = base + (size_t)j * 16;
#pragma unroll
    for (int b = 0; b < B; ++b) q[b] = ld_coherent16(p + b * THREADS * 16);
  } else {
#pragma unroll
    for (int b = 0; b < B; ++b) q[b] = load(j + b * THREADS, end);
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (partial(j + b * THREADS, end)) q[b] = load_partial(j + b * THREADS);
  }
}

template <int DT>
__device__ __forceinline__ void unpack(const uint4& q, float (&x)[Row<DT>::N]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == SPEC_BF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      x[i] = __uint_as_float(w[i]);
    }
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t w) {
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}
__device__ __forceinline__ uint32_t as_word(__nv_bfloat162 v) {
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
  return fmaxf(a, fmaxf(b, c));
}

}  // namespace spec
