// mx.cu -- block-scaled matrices: quantisation, reading back, and the residual RMS norm that
// writes its output block-scaled. Streaming kernels; every element is read and written once.
//
// Work split. Sixteen consecutive lanes hold a 128-element group of one row, eight elements each:
// four lanes are a block, whose largest magnitude is two shuffles away, and the group's four
// scales are one 32-bit store. A warp's loads and code stores are contiguous.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"

namespace spec {
namespace mx {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kFull = 0xffffffffu;

// Streaming 16-byte load from memory that the same kernel may also write (the coherent path).
__device__ __forceinline__ uint4 ld_coherent16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

template <bool RO>
__device__ __forceinline__ uint4 ld16(const void* p) {
  return RO ? ld_stream16(p) : ld_coherent16(p);
}

template <int DT, bool RO>
__device__ __forceinline__ float ld1(const void* p, size_t i) {
  if constexpr (RO) return ld_elem<DT>(p, i);
  if constexpr (DT == SPEC_BF16)
    return bf16_to_f32(*(reinterpret_cast<const volatile uint16_t*>(p) + i));
  else
    return *(reinterpret_cast<const volatile float*>(p) + i);
}

// Elements v .. v + 7 of a row of K (zero past K); 16-byte loads when `vec`. RO: the memory is
// not written while the kernel runs (the read-only path may serve it).
template <int DT, bool RO>
__device__ __forceinline__ void load8(const void* base, size_t off, int v, int K, bool vec,
                                      float (&x)[8]) {
  if (vec && v + 8 <= K) {
    if constexpr (DT == SPEC_BF16) {
      const uint4 q = ld16<RO>(reinterpret_cast<const uint16_t*>(base) + off + v);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
      const float* p = reinterpret_cast<const float*>(base) + off + v;
      const uint4 a = ld16<RO>(p), b = ld16<RO>(p + 4);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v + i < K ? ld1<DT, RO>(base, off + v + i) : 0.0f;
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int DT>
__device__ __forceinline__ void store8(void* base, size_t off, int v, int K, bool vec,
                                       const float (&x)[8]) {
  if (vec && v + 8 <= K) {
    if constexpr (DT == SPEC_BF16) {
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + off + v) =
          make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                     pack_bf16(x[6], x[7]));
    } else {
      float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + off + v);
      p[0] = make_float4(x[0], x[1], x[2], x[3]);
      p[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (v + i >= K) break;
      if constexpr (DT == SPEC_BF16)
        reinterpret_cast<uint16_t*>(base)[off + v + i] = (uint16_t)pack_bf16(x[i], 0.0f);
      else
        reinterpret_cast<float*>(base)[off + v + i] = x[i];
    }
  }
}

// Quantises this lane's eight elements (element 8 * (lane % 16) of group g of row `row`) and
// stores codes and, from the group's first lane, the scale word. All 32 lanes call it; `live`
// masks the stores. Returns whether the block was finite.
template <int FMT>
__device__ __forceinline__ bool quantize8(const float (&x)[8], int row, int g, int G, bool live,
                                          uint8_t* codes, uint8_t* scales) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
    amax = b > amax ? b : amax;
  }
  amax = max(amax, __shfl_xor_sync(kFull, amax, 1));
  amax = max(amax, __shfl_xor_sync(kFull, amax, 2));
  const int sb = scale_byte<FMT>(amax);
  const bool finite = sb != kNanScale;
  // four block bytes -> one word in the group's first lane
  uint32_t word = (uint32_t)sb << (8 * ((threadIdx.x >> 2) & 3));
  word |= __shfl_xor_sync(kFull, word, 4);
  word |= __shfl_xor_sync(kFull, word, 8);
  if (!live) return true;
  const float f = finite ? unscale(sb) : 0.0f;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = finite ? x[i] * f : 0.0f;
  const int l = threadIdx.x & 15;
  if constexpr (FMT == SPEC_MX_E2M1) {
    const uint32_t c = to_e2m1x2(y[0], y[1]) | to_e2m1x2(y[2], y[3]) << 8 |
                       to_e2m1x2(y[4], y[5]) << 16 | to_e2m1x2(y[6], y[7]) << 24;
    *reinterpret_cast<uint32_t*>(codes + (size_t)row * G * (kGroup / 2) + g * (kGroup / 2) + 4 * l) = c;
  } else {
    const uint2 c = make_uint2(to_e4m3x2(y[0], y[1]) | to_e4m3x2(y[2], y[3]) << 16,
                               to_e4m3x2(y[4], y[5]) | to_e4m3x2(y[6], y[7]) << 16);
    *reinterpret_cast<uint2*>(codes + (size_t)row * G * kGroup + g * kGroup + 8 * l) = c;
  }
  if (l == 0) *reinterpret_cast<uint32_t*>(scales + scale_word(row, g, G)) = word;
  return finite;
}

// ------------------------------------------------------------------------------ quantise

// Groups of all rows, the last tile's missing rows among them (their scales are 0).
template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const void* x, long long ldx, int rows,
                                                            int K, bool vec, uint8_t* codes,
                                                            uint8_t* scales, uint32_t* status) {
  const int G = groups(K);
  const long long units = (long long)((rows + kTileRows - 1) / kTileRows) * kTileRows * G;
  const long long step = (long long)gridDim.x * (kThreads / 16);
  bool finite = true;
  for (long long u0 = (long long)blockIdx.x * (kThreads / 16); u0 < units; u0 += step) {
    const long long u = u0 + threadIdx.x / 16;
    const int row = u < units ? (int)(u / G) : rows, g = (int)(u - (u / G) * G);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const int k = g * kGroup + 8 * (threadIdx.x & 15);
    if (row < rows) load8<DT, true>(x, (size_t)row * ldx, k, K, vec, v);
    finite &= quantize8<FMT>(v, row, g, G, row < rows, codes, scales);
    if (u < units && row >= rows && (threadIdx.x & 15) == 0)
      *reinterpret_cast<uint32_t*>(scales + scale_word(row, g, G)) = 0;
  }
  if (!finite) atomicOr(status, SPEC_DEV_NONFINITE);
}

// ------------------------------------------------------------------------------ read back

template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t* codes,
                                                              const uint8_t* scales, int rows,
                                                              int K, bool vec, void* out,
                                                              long long ldo) {
  const int G = groups(K);
  const long long units = (long long)rows * G;
  const long long step = (long long)gridDim.x * (kThreads / 16);
  const int l = threadIdx.x & 15;
  for (long long u = (long long)blockIdx.x * (kThreads / 16) + threadIdx.x / 16; u < units;
       u += step) {
    const int row = (int)(u / G), g = (int)(u - (long long)row * G);
    const int k = g * kGroup + 8 * l;
    if (k >= K) continue;
    const float s = scale_value(__ldg(scales + scale_word(row, g, G) + (l >> 2)));
    float y[8];
    if constexpr (FMT == SPEC_MX_E2M1) {
      const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(
          codes + (size_t)row * G * (kGroup / 2) + g * (kGroup / 2) + 4 * l));
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = from_e2m1(c >> (4 * i)) * s;
    } else {
      const uint2 c = __ldg(reinterpret_cast<const uint2*>(codes + (size_t)row * G * kGroup +
                                                           g * kGroup + 8 * l));
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = from_e4m3((i < 4 ? c.x : c.y) >> (8 * (i & 3))) * s;
    }
    store8<DT>(out, (size_t)row * ldo, k, K, vec, y);
  }
}

// ------------------------------------------------------------------------------ RMS norm

struct NormArgs {
  const void* x;
  const void* res;
  void* res_out;
  const void* weight;
  long long ldx, ldr, ldo;
  int rows, K, wdt;
  float eps;
  bool vec, wvec;
  uint8_t* codes;
  uint8_t* scales;
  uint32_t* status;
};

__device__ __forceinline__ float round_to(float x, int dt) {
  return dt == SPEC_BF16 ? bf16_to_f32((uint16_t)pack_bf16(x, 0.0f)) : x;
}

// h of one eight-element piece: x, plus the residual and the rounding of its stored form.
template <int DT>
__device__ __forceinline__ void load_h(const NormArgs& a, int row, int k, float (&h)[8]) {
  load8<DT, false>(a.x, (size_t)row * a.ldx, k, a.K, a.vec, h);
  if (a.res) {
    float r[8];
    load8<DT, false>(a.res, (size_t)row * a.ldr, k, a.K, a.vec, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = round_to(h[i] + r[i], DT);
  }
}

__device__ __forceinline__ void load_w(const NormArgs& a, int k, float (&w)[8]) {
  if (a.wdt == SPEC_BF16)
    load8<SPEC_BF16, true>(a.weight, 0, k, a.K, a.wvec, w);
  else
    load8<SPEC_F32, true>(a.weight, 0, k, a.K, a.wvec, w);
}

// One block a row; the last block of the grid clears the scales of the last tile's missing rows.
// The row is read twice (the second time from cache): first its sum of squares, then its codes.
template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) rmsnorm_kernel(NormArgs a) {
  const int G = groups(a.K);
  const int row = blockIdx.x;
  if (row == a.rows) {
    const int last = (a.rows + kTileRows - 1) / kTileRows * kTileRows;
    for (int u = threadIdx.x; u < (last - a.rows) * G; u += kThreads)
      *reinterpret_cast<uint32_t*>(a.scales + scale_word(a.rows + u / G, u % G, G)) = 0;
    return;
  }
  float ss = 0.0f;
  for (int k = 8 * threadIdx.x; k < a.K; k += 8 * kThreads) {
    float h[8];
    load_h<DT>(a, row, k, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(h[i], h[i], ss);
  }
  ss = block_sum(ss);
  // a sum that is not finite makes the whole row NaN
  const float rstd = ss < INFINITY ? 1.0f / sqrtf(ss / (float)a.K + a.eps) : NAN;
  bool finite = true;
  const int Kp = G * kGroup;
  for (int k0 = 0; k0 < Kp; k0 += 8 * kThreads) {
    const int k = k0 + 8 * threadIdx.x;
    float h[8] = {0, 0, 0, 0, 0, 0, 0, 0}, w[8];
    if (k < a.K) {
      load_h<DT>(a, row, k, h);
      if (a.res) store8<DT>(a.res_out, (size_t)row * a.ldo, k, a.K, a.vec, h);
      load_w(a, k, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = h[i] * rstd * w[i];
    }
    finite &= quantize8<FMT>(h, row, k / kGroup, G, k < Kp, a.codes, a.scales);
  }
  if (!finite) atomicOr(a.status, SPEC_DEV_NONFINITE);
}

int grid_for(long long units) {
  const long long blocks = (units + kThreads / 16 - 1) / (kThreads / 16);
  const long long cap = (long long)num_sms() * 8;
  return (int)(blocks < cap ? blocks : cap);
}

bool vec_ok(const void* p, long long ld, int dt) {
  const size_t es = dt == SPEC_BF16 ? 2 : 4;
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * es) % 16 == 0);
}

}  // namespace

}  // namespace mx

void launch_mx_quantize(const void* x, int dt, long long ldx, int rows, int K, int fmt,
                        uint8_t* codes, uint8_t* scales, uint32_t* status, cudaStream_t s) {
  using namespace mx;
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  const bool vec = vec_ok(x, ldx, dt);
  const int grid = grid_for((long long)((rows + 127) / 128) * 128 * groups(K));
  auto k = dt == SPEC_BF16
               ? (fmt == SPEC_MX_E2M1 ? quantize_kernel<SPEC_BF16, SPEC_MX_E2M1>
                                      : quantize_kernel<SPEC_BF16, SPEC_MX_E4M3>)
               : (fmt == SPEC_MX_E2M1 ? quantize_kernel<SPEC_F32, SPEC_MX_E2M1>
                                      : quantize_kernel<SPEC_F32, SPEC_MX_E4M3>);
  k<<<grid, kThreads, 0, s>>>(x, ldx, rows, K, vec, codes, scales, status);
}

void launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int fmt, int rows, int K,
                          void* out, int dt, long long ldo, cudaStream_t s) {
  using namespace mx;
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  const bool vec = vec_ok(out, ldo, dt);
  const int grid = grid_for((long long)rows * groups(K));
  auto k = dt == SPEC_BF16
               ? (fmt == SPEC_MX_E2M1 ? dequantize_kernel<SPEC_BF16, SPEC_MX_E2M1>
                                      : dequantize_kernel<SPEC_BF16, SPEC_MX_E4M3>)
               : (fmt == SPEC_MX_E2M1 ? dequantize_kernel<SPEC_F32, SPEC_MX_E2M1>
                                      : dequantize_kernel<SPEC_F32, SPEC_MX_E4M3>);
  k<<<grid, kThreads, 0, s>>>(codes, scales, rows, K, vec, out, ldo);
}

void launch_rmsnorm_mx(const void* x, long long ldx, const void* res, long long ldr, int dt,
                       const void* weight, int wdt, float eps, int rows, int K, void* res_out,
                       long long ldo, int fmt, uint8_t* codes, uint8_t* scales, uint32_t* status,
                       cudaStream_t s) {
  using namespace mx;
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  NormArgs a{x, res, res_out, weight, ldx, ldr, ldo, rows, K, wdt, eps, false, false, codes,
             scales, status};
  a.vec = vec_ok(x, ldx, dt) && (!res || (vec_ok(res, ldr, dt) && vec_ok(res_out, ldo, dt)));
  a.wvec = vec_ok(weight, 0, wdt);
  auto k = dt == SPEC_BF16 ? (fmt == SPEC_MX_E2M1 ? rmsnorm_kernel<SPEC_BF16, SPEC_MX_E2M1>
                                                  : rmsnorm_kernel<SPEC_BF16, SPEC_MX_E4M3>)
                           : (fmt == SPEC_MX_E2M1 ? rmsnorm_kernel<SPEC_F32, SPEC_MX_E2M1>
                                                  : rmsnorm_kernel<SPEC_F32, SPEC_MX_E4M3>);
  k<<<rows + 1, kThreads, 0, s>>>(a);
}

}  // namespace spec
