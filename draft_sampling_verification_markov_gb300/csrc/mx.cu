// mx.cu -- block-scaled matrices: quantisation, reading back, and the residual RMS norm that
// writes its output block-scaled. Streaming kernels; every element is read and written once.
//
// Work split. Sixteen consecutive lanes hold a 128-element group of one row, eight elements each:
// four lanes are a block, whose largest magnitude is two shuffles away, and the group's four
// scales are one 32-bit store. A warp's loads and code stores are contiguous. A thread has kUnroll
// such pieces in flight: with one, the kernels waited on memory.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"

namespace spec {
namespace mx {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = kThreads / 16;  // groups a block takes at once
constexpr int kUnroll = 4;
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

// Row and group of unit u0 + t (t < 2^16) for a block-uniform u0.
struct Unit {
  int row, g;
  __device__ __forceinline__ Unit(int row0, int g0, int t, int G) {
    const uint32_t x = (uint32_t)(g0 + t), q = x / (uint32_t)G;
    row = row0 + (int)q;
    g = (int)(x - q * (uint32_t)G);
  }
};

// ------------------------------------------------------------------------------ quantise

// Groups of all rows, the last tile's missing rows among them (their scales are 0).
template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const void* x, long long ldx, int rows,
                                                            int K, bool vec, uint8_t* codes,
                                                            uint8_t* scales, uint32_t* status) {
  const int G = groups(K), l = threadIdx.x & 15;
  const int tiled = (rows + kTileRows - 1) / kTileRows * kTileRows;
  const long long units = (long long)tiled * G;
  const long long step = (long long)gridDim.x * kUnits * kUnroll;
  bool finite = true;
  for (long long u0 = (long long)blockIdx.x * kUnits * kUnroll; u0 < units; u0 += step) {
    const int row0 = (int)(u0 / G), g0 = (int)(u0 - (long long)row0 * G);
    float v[kUnroll][8];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const Unit u(row0, g0, i * kUnits + threadIdx.x / 16, G);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
      if (u.row < rows)
        load8<DT, true>(x, (size_t)u.row * ldx, u.g * kGroup + 8 * l, K, vec, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const Unit u(row0, g0, i * kUnits + threadIdx.x / 16, G);
      finite &= quantize8<FMT>(v[i], u.row, u.g, G, u.row < rows, codes, scales);
      if (u.row >= rows && u.row < tiled && l == 0)
        *reinterpret_cast<uint32_t*>(scales + scale_word(u.row, u.g, G)) = 0;
    }
  }
  if (!finite) atomicOr(status, SPEC_DEV_NONFINITE);
}

// ------------------------------------------------------------------------------ read back

template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t* codes,
                                                              const uint8_t* scales, int rows,
                                                              int K, bool vec, void* out,
                                                              long long ldo) {
  const int G = groups(K), l = threadIdx.x & 15;
  const long long units = (long long)rows * G;
  const long long step = (long long)gridDim.x * kUnits * kUnroll;
  for (long long u0 = (long long)blockIdx.x * kUnits * kUnroll; u0 < units; u0 += step) {
    const int row0 = (int)(u0 / G), g0 = (int)(u0 - (long long)row0 * G);
    uint2 c[kUnroll];
    uint32_t sb[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const Unit u(row0, g0, i * kUnits + threadIdx.x / 16, G);
      c[i] = make_uint2(0, 0);
      sb[i] = 0;
      if (u.row >= rows) continue;
      if constexpr (FMT == SPEC_MX_E2M1)
        c[i].x = __ldg(reinterpret_cast<const uint32_t*>(
            codes + ((size_t)u.row * G + u.g) * (kGroup / 2) + 4 * l));
      else
        c[i] = __ldg(reinterpret_cast<const uint2*>(codes + ((size_t)u.row * G + u.g) * kGroup +
                                                    8 * l));
      sb[i] = __ldg(scales + scale_word(u.row, u.g, G) + (l >> 2));
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const Unit u(row0, g0, i * kUnits + threadIdx.x / 16, G);
      const int k = u.g * kGroup + 8 * l;
      if (u.row >= rows || k >= K) continue;
      const float s = scale_value((int)sb[i]);
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        if constexpr (FMT == SPEC_MX_E2M1)
          from_e2m1x2(c[i].x >> (4 * e), y[e], y[e + 1]);
        else
          from_e4m3x2((e < 4 ? c[i].x : c[i].y) >> (8 * (e & 3)), y[e], y[e + 1]);
        y[e] *= s;
        y[e + 1] *= s;
      }
      store8<DT>(out, (size_t)u.row * ldo, k, K, vec, y);
    }
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

// 1 / sqrt(sum / K + eps) as an unevaluated pair, from a sum known as a pair: the quotient with
// its remainder, the exact sum with eps, and one Newton step from the hardware's reciprocal root
// whose residual is formed with fused products. Everything in a row is scaled by this one number,
// so its rounding would move every code of the row the same way. A sum that is not finite gives
// NaN for the whole row.
__device__ __forceinline__ DF inverse_rms(DF sum, float K, float eps) {
  if (!(sum.hi < INFINITY)) return {NAN, 0.0f};
  const float q = __fdiv_rn(sum.hi, K);
  const float ql = (fmaf(-q, K, sum.hi) + sum.lo) / K;
  DF v = two_sum(q, eps);
  v = fast_two_sum(v.hi, v.lo + ql);
  const float y = rsqrtf(v.hi);
  const float t = v.hi * y, te = fmaf(v.hi, y, -t);
  const float r = fmaf(-t, y, 1.0f) - (te + v.lo * y) * y;  // 1 - v y^2
  return fast_two_sum(y, 0.5f * y * r);
}

// h * rstd * w with one rounding: the product with rstd as a pair, then the weight.
__device__ __forceinline__ float scaled(float h, DF rstd, float w) {
  const float q = h * rstd.hi, e = fmaf(h, rstd.hi, -q) + h * rstd.lo;
  return fmaf(q, w, e * w);
}

// Sum over the block of one number a thread, as a pair: fp32 within a warp, exact additions over
// the warps. blockDim.x is a multiple of 32.
__device__ __forceinline__ DF block_sum_pair(float x) {
  __shared__ float part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = warp_sum(x);
  if (lane == 0) part[warp] = x;
  __syncthreads();
  DF s = {part[0], 0.0f};
  for (int w = 1; w < (int)(blockDim.x >> 5); ++w) s = df_add(s, part[w]);
  return s;
}

// The last block of a norm's grid clears the scales of the last tile's missing rows.
__device__ __forceinline__ void clear_missing(const NormArgs& a, int G) {
  const int last = (a.rows + kTileRows - 1) / kTileRows * kTileRows;
  for (int u = threadIdx.x; u < (last - a.rows) * G; u += blockDim.x)
    *reinterpret_cast<uint32_t*>(a.scales + scale_word(a.rows + u / G, u % G, G)) = 0;
}

// One block a row, the row in registers: P pieces of eight elements a thread.
template <int DT, int FMT, int P>
__global__ void __launch_bounds__(1024 / P) rmsnorm_kernel(NormArgs a) {
  const int G = groups(a.K), Kp = G * kGroup, row = blockIdx.x;
  if (row == a.rows) {
    clear_missing(a, G);
    return;
  }
  float h[P][8], ss = 0.0f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int k = 8 * (threadIdx.x + p * blockDim.x);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[p][i] = 0.0f;
    if (k < a.K) load_h<DT>(a, row, k, h[p]);
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      s0 = fmaf(h[p][i], h[p][i], s0);
      s1 = fmaf(h[p][i + 1], h[p][i + 1], s1);
    }
    ss += s0 + s1;
    const int k = 8 * (threadIdx.x + p * blockDim.x);
    if (a.res && k < a.K) store8<DT>(a.res_out, (size_t)row * a.ldo, k, a.K, a.vec, h[p]);
  }
  const DF rstd = inverse_rms(block_sum_pair(ss), (float)a.K, a.eps);
  bool finite = true;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int k = 8 * (threadIdx.x + p * blockDim.x);
    float w[8];
    if (k < a.K) {
      load_w(a, k, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[p][i] = scaled(h[p][i], rstd, w[i]);
    }
    if (k - 8 * (threadIdx.x & 31) < Kp)  // uniform in a warp
      finite &= quantize8<FMT>(h[p], row, k / kGroup, G, k < Kp, a.codes, a.scales);
  }
  if (!finite) atomicOr(a.status, SPEC_DEV_NONFINITE);
}

// Rows too long for registers: read twice (the second time from cache).
template <int DT, int FMT>
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(NormArgs a) {
  const int G = groups(a.K), Kp = G * kGroup, row = blockIdx.x, step = 8 * blockDim.x;
  if (row == a.rows) {
    clear_missing(a, G);
    return;
  }
  DF sum = df_zero();  // a chain of K / 8192 pieces: exact additions
  for (int k = 8 * threadIdx.x; k < a.K; k += step) {
    float h[8], s = 0.0f;
    load_h<DT>(a, row, k, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(h[i], h[i], s);
    sum = df_add(sum, s);
  }
  const DF rstd = inverse_rms(block_sum_pair(df_float(sum)), (float)a.K, a.eps);
  bool finite = true;
  for (int k0 = 0; k0 < Kp; k0 += step) {
    const int k = k0 + 8 * threadIdx.x;
    float h[8] = {0, 0, 0, 0, 0, 0, 0, 0}, w[8];
    if (k < a.K) {
      load_h<DT>(a, row, k, h);
      if (a.res) store8<DT>(a.res_out, (size_t)row * a.ldo, k, a.K, a.vec, h);
      load_w(a, k, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = scaled(h[i], rstd, w[i]);
    }
    finite &= quantize8<FMT>(h, row, k / kGroup, G, k < Kp, a.codes, a.scales);
  }
  if (!finite) atomicOr(a.status, SPEC_DEV_NONFINITE);
}

template <int DT, int FMT>
void launch_norm_t(const NormArgs& a, cudaStream_t s) {
  const int pieces = groups(a.K) * (kGroup / 8), grid = a.rows + 1;
  // one piece a thread while rows are few and latency counts (1 row of 4096: 512 threads), more
  // pieces and smaller blocks, of which an SM holds several rows, once they are many
  const int most = a.rows <= 2 * num_sms() ? 1024 : 256;
  auto threads = [&](int p) { return (pieces + p * 32 - 1) / (p * 32) * 32; };
  if (threads(1) <= most) rmsnorm_kernel<DT, FMT, 1><<<grid, threads(1), 0, s>>>(a);
  else if (threads(2) <= (most < 512 ? most : 512)) rmsnorm_kernel<DT, FMT, 2><<<grid, threads(2), 0, s>>>(a);
  else if (threads(4) <= 256) rmsnorm_kernel<DT, FMT, 4><<<grid, threads(4), 0, s>>>(a);
  else rmsnorm_long_kernel<DT, FMT><<<grid, 1024, 0, s>>>(a);
}

int grid_for(long long units) {
  const long long blocks = (units + kUnits * kUnroll - 1) / (kUnits * kUnroll);
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
  if (dt == SPEC_BF16)
    fmt == SPEC_MX_E2M1 ? launch_norm_t<SPEC_BF16, SPEC_MX_E2M1>(a, s)
                        : launch_norm_t<SPEC_BF16, SPEC_MX_E4M3>(a, s);
  else
    fmt == SPEC_MX_E2M1 ? launch_norm_t<SPEC_F32, SPEC_MX_E2M1>(a, s)
                        : launch_norm_t<SPEC_F32, SPEC_MX_E4M3>(a, s);
}

}  // namespace spec
