// mx.cu -- block-scaled matrices: quantisation, reading back, and the residual RMS norm that
// writes its output block-scaled. Streaming kernels; every element is read and written once.
//
// Work split. Consecutive lanes hold a 128-element group of one row, eight elements each (sixteen
// in the quantiser): four (two) lanes are a block, whose largest magnitude is two (one) shuffles
// away, and the group's four scales are one 32-bit store. A warp's loads and code stores are
// contiguous. A thread has 64 bytes in flight: with 16 the kernels waited on memory. Loads go
// through the coherent path (common.cuh says why).
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"

namespace spec {
namespace mx {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = kThreads / 16;  // groups a block takes at once, eight elements a thread
constexpr int kWide = kThreads / 8;    // ... sixteen elements a thread
// Pieces in flight.
template <int DT>
constexpr int kUnroll = DT == SPEC_BF16 ? 2 : 1;
constexpr int kUnrollBack = 4;
constexpr uint32_t kFull = 0xffffffffu;

// ld_coherent16 of 32 bytes.
__device__ __forceinline__ void ld_coherent32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z),
                 "=r"(b.w)
               : "l"(p)
               : "memory");
}

// Eight consecutive elements as they are stored.
template <int DT>
struct Piece {
  uint4 q[DT == SPEC_BF16 ? 1 : 2];
};

template <int DT>
__device__ __forceinline__ void clear(Piece<DT>& p) {
#pragma unroll
  for (uint4& q : p.q) q = make_uint4(0, 0, 0, 0);
}

// Elements v .. v + 7 of a row of K (zero past K); 16-byte loads when `vec`, kept in L1 when SHARED
// (other blocks of the SM read them too).
template <int DT, bool SHARED = false>
__device__ __forceinline__ void load8(const void* base, size_t off, int v, int K, bool vec,
                                      Piece<DT>& p) {
  constexpr size_t es = DT == SPEC_BF16 ? 2 : 4;
  const char* at = static_cast<const char*>(base) + (off + v) * es;
  if (vec && v + 8 <= K) {
#pragma unroll
    for (int i = 0; i < (int)es / 2; ++i) {
      if constexpr (SHARED)
        p.q[i] = *reinterpret_cast<const uint4*>(at + 16 * i);
      else
        p.q[i] = ld_coherent16(at + 16 * i);
    }
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = v + i < K ? __float_as_uint(ld_elem_coherent<DT>(base, off + v + i)) : 0u;
    if constexpr (DT == SPEC_BF16) {  // an element's bits are the upper half of its fp32's
      p.q[0] = make_uint4(w[0] >> 16 | w[1], w[2] >> 16 | w[3], w[4] >> 16 | w[5],
                          w[6] >> 16 | w[7]);
    } else {
      p.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
      p.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

template <int DT>
__device__ __forceinline__ void unpack(const Piece<DT>& p, float (&x)[8]) {
  if constexpr (DT == SPEC_BF16) {
    const uint32_t w[4] = {p.q[0].x, p.q[0].y, p.q[0].z, p.q[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const uint32_t w[8] = {p.q[0].x, p.q[0].y, p.q[0].z, p.q[0].w,
                           p.q[1].x, p.q[1].y, p.q[1].z, p.q[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight values as they are stored, rounded to the type.
template <int DT>
__device__ __forceinline__ void pack(const float (&x)[8], Piece<DT>& p) {
  if constexpr (DT == SPEC_BF16) {
    p.q[0] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                        pack_bf16(x[6], x[7]));
  } else {
    p.q[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                        __float_as_uint(x[3]));
    p.q[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]),
                        __float_as_uint(x[7]));
  }
}

template <int DT>
__device__ __forceinline__ void store8(void* base, size_t off, int v, int K, bool vec,
                                       const Piece<DT>& p) {
  constexpr size_t es = DT == SPEC_BF16 ? 2 : 4;
  char* at = static_cast<char*>(base) + (off + v) * es;
  if (vec && v + 8 <= K) {
#pragma unroll
    for (int i = 0; i < (int)es / 2; ++i) *reinterpret_cast<uint4*>(at + 16 * i) = p.q[i];
  } else {
    float x[8];
    unpack<DT>(p, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (v + i >= K) break;
      if constexpr (DT == SPEC_BF16)
        reinterpret_cast<uint16_t*>(at)[i] = (uint16_t)(__float_as_uint(x[i]) >> 16);
      else
        reinterpret_cast<float*>(at)[i] = x[i];
    }
  }
}

__device__ __forceinline__ float max_abs_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)));
  return d;
}

// Largest magnitude, NaN if there is one.
__device__ __forceinline__ float max_abs8(const float (&x)[8]) {
  return max_abs_nan(max_abs_nan(max_abs_nan(x[0], x[1]), max_abs_nan(x[2], x[3])),
                     max_abs_nan(max_abs_nan(x[4], x[5]), max_abs_nan(x[6], x[7])));
}

// Quantises this lane's eight products of the norm (element 8 * (lane % 16) of a group): stores its codes at
// `codes` and, from the group's first lane, the scale word at `scale`. All 32 lanes call it;
// `live` masks the stores. Returns whether the block was finite.
template <int FMT>
__device__ __forceinline__ bool quantize8(const float (&x)[8], bool live, uint8_t* codes,
                                          uint8_t* scale) {
  // as integers NaN is above infinity
  uint32_t amax = __float_as_uint(max_abs8(x)) & 0x7fffffffu;
  amax = max(amax, __shfl_xor_sync(kFull, amax, 1));
  amax = max(amax, __shfl_xor_sync(kFull, amax, 2));
  // a product that passes fp32 was truncated to its largest number
  const int sb = amax == 0x7f7fffffu ? kNanScale : scale_byte<FMT>(amax);
  const bool finite = sb != kNanScale;
  // four block bytes -> one word in the group's first lane
  uint32_t word = (uint32_t)sb << (8 * ((threadIdx.x >> 2) & 3));
  word |= __shfl_xor_sync(kFull, word, 4);
  word |= __shfl_xor_sync(kFull, word, 8);
  if (!live) return true;
  const float f = unscale(finite ? sb : 0);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i] * f;
  if constexpr (FMT == SPEC_MX_E2M1) {
    const uint32_t c = to_e2m1x8(y);
    *reinterpret_cast<uint32_t*>(codes) = finite ? c : 0;
  } else {
    const uint2 c = to_e4m3x8(y);
    *reinterpret_cast<uint2*>(codes) = finite ? c : make_uint2(0, 0);
  }
  if ((threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t*>(scale) = word;
  return finite;
}

// Bytes of a group's codes, and of a lane's part of them.
template <int FMT>
constexpr int kGroupCode = FMT == SPEC_MX_E2M1 ? kGroup / 2 : kGroup;
template <int FMT>
constexpr int kLaneCode = kGroupCode<FMT> / 16;

// Row and group of unit u0 + t, t < 64, for a block-uniform u0 at (row0, g0). A row of 64 groups
// or more ends at most once within; a shorter one's quotient comes from its reciprocal (both
// factors are below 128, so ceil(2^32 / G) is exact enough).
struct Unit {
  int row, g;
  __device__ __forceinline__ Unit(int row0, int g0, int t, int G, uint32_t recip) {
    const uint32_t x = (uint32_t)(g0 + t);
    const uint32_t q = G >= 64 ? (x >= (uint32_t)G ? 1u : 0u)
                               : (G == 1 ? x : __umulhi(x, recip));
    row = row0 + (int)q;
    g = (int)(x - q * (uint32_t)G);
  }
};
__device__ __forceinline__ uint32_t reciprocal(int G) { return 0xffffffffu / (uint32_t)G + 1u; }

// ------------------------------------------------------------------------------ quantise

// Sixteen elements from v of a row of K (zero past K): 32-byte loads (vec 2), 16-byte ones (1) or
// single elements.
template <int DT>
__device__ __forceinline__ void load16(const void* base, size_t off, int v, int K, int vec,
                                       Piece<DT> (&p)[2]) {
  constexpr size_t es = DT == SPEC_BF16 ? 2 : 4;
  if (vec == 2 && v + 16 <= K) {
    const char* at = static_cast<const char*>(base) + (off + v) * es;
    if constexpr (DT == SPEC_BF16) {
      ld_coherent32(at, p[0].q[0], p[1].q[0]);
    } else {
      ld_coherent32(at, p[0].q[0], p[0].q[1]);
      ld_coherent32(at + 32, p[1].q[0], p[1].q[1]);
    }
  } else {
    load8<DT>(base, off, v, K, vec > 0, p[0]);
    load8<DT>(base, off, v + 8, K, vec > 0, p[1]);
  }
}

// As quantize8 with sixteen elements a lane (element 16 * (lane % 8) of a group).
template <int FMT>
__device__ __forceinline__ bool quantize16(const float (&x)[2][8], bool live, uint8_t* codes,
                                           uint8_t* scale) {
  const float m = max_abs_nan(max_abs8(x[0]), max_abs8(x[1]));
  uint32_t amax = __float_as_uint(m) & 0x7fffffffu;
  amax = max(amax, __shfl_xor_sync(kFull, amax, 1));
  const int sb = scale_byte<FMT>(amax);
  const bool finite = sb != kNanScale;
  uint32_t word = (uint32_t)sb << (8 * ((threadIdx.x >> 1) & 3));
  word |= __shfl_xor_sync(kFull, word, 2);
  word |= __shfl_xor_sync(kFull, word, 4);
  if (!live) return true;
  const float f = unscale(finite ? sb : 0);
  float y[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) y[h][i] = x[h][i] * f;
  if constexpr (FMT == SPEC_MX_E2M1) {
    const uint2 c = make_uint2(to_e2m1x8(y[0]), to_e2m1x8(y[1]));
    *reinterpret_cast<uint2*>(codes) = finite ? c : make_uint2(0, 0);
  } else {
    const uint2 c = to_e4m3x8(y[0]), d = to_e4m3x8(y[1]);
    *reinterpret_cast<uint4*>(codes) =
        finite ? make_uint4(c.x, c.y, d.x, d.y) : make_uint4(0, 0, 0, 0);
  }
  if ((threadIdx.x & 7) == 0) *reinterpret_cast<uint32_t*>(scale) = word;
  return finite;
}

// Groups of all rows, the last tile's missing rows among them (their scales are 0). 129280 x 4096
// bf16 to E2M1: 212 us, 6.3 TB/s of values read and codes written; with eight elements a lane the
// kernel was bound by issue, at 272 us.
template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const void* x, long long ldx, int rows, int K, int vec, uint8_t* codes,
                    uint8_t* scales, uint32_t* status) {
  const int G = groups(K), l = threadIdx.x & 7;
  const int tiled = (rows + kTileRows - 1) / kTileRows * kTileRows;
  const uint32_t recip = reciprocal(G);
  constexpr int U = kUnroll<DT>;
  bool finite = true;
  grid_dep_wait();
  const long long u0 = (long long)blockIdx.x * kWide * U;
  const int row0 = (int)(u0 / G), g0 = (int)(u0 - (long long)row0 * G);
  Piece<DT> v[U][2];
  int row[U];
  uint8_t* scale[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const Unit u(row0, g0, i * kWide + threadIdx.x / 8, G, recip);
    row[i] = u.row;
    scale[i] = scales + scale_word(u.row, u.g, G);
    clear<DT>(v[i][0]);
    clear<DT>(v[i][1]);
    if (u.row < rows)
      load16<DT>(x, (size_t)u.row * ldx, u.g * kGroup + 16 * l, K, vec, v[i]);
  }
  uint8_t* c = codes + (size_t)(u0 + threadIdx.x / 8) * kGroupCode<FMT> + 2 * kLaneCode<FMT> * l;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float y[2][8];
    unpack<DT>(v[i][0], y[0]);
    unpack<DT>(v[i][1], y[1]);
    finite &= quantize16<FMT>(y, row[i] < rows, c + (size_t)i * kWide * kGroupCode<FMT>, scale[i]);
    if (row[i] >= rows && row[i] < tiled && l == 0) *reinterpret_cast<uint32_t*>(scale[i]) = 0;
  }
  if (!finite) atomicOr(status, SPEC_DEV_NONFINITE);
}

// ------------------------------------------------------------------------------ read back

// 129280 x 4096 E2M1 to bf16: 202 us, 6.6 TB/s of codes read and values written (213 us with loads
// through the read-only path).
template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t* codes,
                                                              const uint8_t* scales, int rows,
                                                              int K, bool vec, void* out,
                                                              long long ldo) {
  const int G = groups(K), l = threadIdx.x & 15;
  const uint32_t recip = reciprocal(G);
  constexpr int U = kUnrollBack;
  grid_dep_wait();
  const long long u0 = (long long)blockIdx.x * kUnits * U;
  const int row0 = (int)(u0 / G), g0 = (int)(u0 - (long long)row0 * G);
  uint2 c[U];
  uint32_t sb[U];
  int row[U], k[U];
  const uint8_t* p = codes + (size_t)(u0 + threadIdx.x / 16) * kGroupCode<FMT> +
                     kLaneCode<FMT> * l;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const Unit u(row0, g0, i * kUnits + threadIdx.x / 16, G, recip);
    row[i] = u.row;
    k[i] = u.g * kGroup + 8 * l;
    c[i] = make_uint2(0, 0);
    sb[i] = 0;
    if (u.row >= rows) continue;
    const uint8_t* at = p + (size_t)i * kUnits * kGroupCode<FMT>;
    if constexpr (FMT == SPEC_MX_E2M1)
      c[i].x = *reinterpret_cast<const uint32_t*>(at);
    else
      c[i] = *reinterpret_cast<const uint2*>(at);
    sb[i] = scales[scale_word(u.row, u.g, G) + (l >> 2)];
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (row[i] >= rows || k[i] >= K) continue;
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
    Piece<DT> o;
    pack<DT>(y, o);
    store8<DT>(out, (size_t)row[i] * ldo, k[i], K, vec, o);
  }
}

// ------------------------------------------------------------------------------ RMS norm

struct NormArgs {
  const void* x;
  const void* res;
  void* res_out;
  const void* weight;
  long long ldx, ldr, ldo;
  int rows, K;
  float eps, inv_K;
  bool vec, wvec;
  uint8_t* codes;
  uint8_t* scales;
  uint32_t* status;
};

// A row's piece of x and of the residual, as loaded.
template <int DT>
struct Pair {
  Piece<DT> x, r;
};

template <int DT>
__device__ __forceinline__ void load_pair(const NormArgs& a, int row, int k, Pair<DT>& p) {
  load8<DT>(a.x, (size_t)row * a.ldx, k, a.K, a.vec, p.x);
  if (a.res) load8<DT>(a.res, (size_t)row * a.ldr, k, a.K, a.vec, p.r);
}

// h of one piece, as it is stored: x, or x + residual rounded to the type (and stored).
template <int DT>
__device__ __forceinline__ Piece<DT> add_pair(const NormArgs& a, int row, int k,
                                              const Pair<DT>& p) {
  if (!a.res) return p.x;
  float h[8], r[8];
  unpack<DT>(p.x, h);
  unpack<DT>(p.r, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] += r[i];
  Piece<DT> o;
  pack<DT>(h, o);
  if (a.res_out) store8<DT>(a.res_out, (size_t)row * a.ldo, k, a.K, a.vec, o);
  return o;
}

// Sum of the squares of one piece times `pre`, a power of two.
template <int DT>
__device__ __forceinline__ float sum_squares(const Piece<DT>& p, float pre) {
  float h[8], s0 = 0.0f, s1 = 0.0f;
  unpack<DT>(p, h);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] *= pre;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    s0 = fmaf(h[i], h[i], s0);
    s1 = fmaf(h[i + 1], h[i + 1], s1);
  }
  return s0 + s1;
}

// sum / K + eps as an unevaluated pair, from a sum known as a pair: the quotient with its
// remainder and the exact sum with eps.
__device__ __forceinline__ DF mean_square(DF sum, float K, float inv_K, float eps) {
  const float q = sum.hi * inv_K;
  const float ql = (fmaf(-q, K, sum.hi) + sum.lo) * inv_K;
  const DF v = two_sum(q, eps);
  return fast_two_sum(v.hi, v.lo + ql);
}

// Squares leave fp32's range before their row does. Where v = mean(h^2) + eps overflows, or is so
// small (below kLeast) that its squares may have lost bits, the sum is taken again over h times a
// power of two, which then scales eps twice and the row's elements once. Shrunk, 2^24 squares
// of at most 2^48 are finite, and a v that overflowed is 2^-80 at least. Grown, a v that was below
// kLeast is below 2^97 and its sum below 2^121; the square of the least subnormal is 2^-102.
constexpr float kShrink = 0x1p-80f, kGrow = 0x1p98f, kLeast = 0x1p-100f;

// 1 / sqrt(v) as an unevaluated pair: one Newton step from the hardware's reciprocal root whose
// residual is formed with fused products. Everything in a row is scaled by this one number, so its
// rounding would move every code of the row the same way. NaN for a v that is not finite.
__device__ __forceinline__ DF inverse_root(DF v) {
  if (!(v.hi < INFINITY)) return {NAN, 0.0f};
  const float y = rsqrtf(v.hi);
  const float t = v.hi * y, te = fmaf(v.hi, y, -t);
  const float r = fmaf(-t, y, 1.0f) - (te + v.lo * y) * y;  // 1 - v y^2
  return fast_two_sum(y, 0.5f * y * r);
}

// Sum of one non-negative number a lane as a pair, exact to 2^-42 of the largest: under the
// largest one's exponent the numbers are two whole numbers of 24 bits each, which the warp's
// integer reduction adds (five rounds of pair additions were most of a row's latency).
__device__ __forceinline__ DF warp_sum_exact(float x) {
  const int e = (int)(__reduce_max_sync(kFull, __float_as_uint(x)) >> 23);
  if (e == 255 || e < 24) return {warp_sum(x), 0.0f};  // not finite, or below 2^-103
  const float f = __uint_as_float((uint32_t)(277 - e) << 23);    // 2^(150 - e): x * f < 2^24
  const float back = __uint_as_float((uint32_t)(e - 23) << 23);  // 2^(e - 150)
  const float t = x * f;
  const uint32_t hi = (uint32_t)t, lo = (uint32_t)((t - (float)hi) * 0x1p24f);
  const uint32_t sh = __reduce_add_sync(kFull, hi), sl = __reduce_add_sync(kFull, lo);
  // sums below 2^29: the upper 23 bits convert exactly
  const DF s = fast_two_sum((float)(sh & ~0x3fu),
                            (float)(sh & 0x3fu) + (float)sl * 0x1p-24f);
  return {s.hi * back, s.lo * back};
}

// The scale of a row: 1 / rms = (hi + lo) * two with `two` a power of two and hi in [1, 2), or a
// factor `pre` other than 1 to take the row's squares with instead (lo is 0 then, too).
// lo is 0 exactly where the root is a fraction with a power of two below: then
// rms^2 = sum / K + eps = 4^j / m^2 with m odd, so m^2 divides K and m has 12 bits at most; a pair
// that is such a number up to its own error (2^-45) is taken to be it.
struct alignas(16) RowScale {
  float hi, lo, two, pre;
  RowScale() = default;
  __device__ __forceinline__ explicit RowScale(DF r) {
    const int e = (int)(__float_as_uint(r.hi) >> 23) - 127;  // a normal number, or NaN
    two = __uint_as_float((uint32_t)(e + 127) << 23);
    const float back = __uint_as_float((uint32_t)(127 - e) << 23);
    hi = r.hi * back;
    lo = r.lo * back;
    if (fabsf(lo) < 0x1p-42f && !(__float_as_uint(hi) & 0xfffu)) lo = 0.0f;
    if (!(r.hi < INFINITY)) hi = NAN, two = 1.0f;
    pre = 1.0f;
  }
};

// h * rstd * w, truncated, with the last bit set where something was cut off (rounding to odd).
// Rounding that to the format rounds the product itself, and a block's scale is the least that fits
// the product; rounding to the nearest fp32 in between meets a midpoint of the format about once
// in 2^20 elements and may then go the wrong way. The power of two comes first: h * two is exact,
// and of the size of the result. EXACT: the product with the weight has no rounding error (two
// bf16 numbers). REST: the product may have no rest, which takes its own look; where lo is not 0
// (the root is no fraction with a power of two below) it always has one.
template <bool EXACT, bool REST>
__device__ __forceinline__ float scaled(float h, const RowScale& r, float w) {
  const float g = h * r.two, p = g * w;
  float low = p * r.lo;
  if (!EXACT) low = fmaf(fmaf(g, w, -p), r.hi, low);
  const float y = __fmaf_rz(p, r.hi, low);
  const bool rest = !REST || r.lo != 0.0f || fmaf(p, r.hi, -y) + low != 0.0f;
  return __uint_as_float(__float_as_uint(y) | (rest ? 1u : 0u));
}

// The products of eight elements from k of a row of K, 0 past K.
template <bool EXACT, bool REST>
__device__ __forceinline__ void scale8(float (&h)[8], const RowScale& r, const float (&w)[8], int k,
                                       int K) {
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = k + i < K ? scaled<EXACT, REST>(h[i], r, w[i]) : 0.0f;
}

// The scale of a row from each thread's sum of squares (of elements times `pre`): fp32 within a
// warp (10 roundings, which put 1 to 3 of the 35.7 million codes of 17408 x 2048 random elements a
// step off those of the exact root), exact over the warps. One warp does what is the same for all
// (done by every thread it was most of the kernel's instructions). blockDim.x is a multiple of 32.
__device__ __forceinline__ RowScale row_scale(float x, const NormArgs& a, float pre) {
  __shared__ float part[32];
  __shared__ RowScale scale;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = warp_sum(x);
  if (lane == 0) part[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const DF sum = warp_sum_exact(lane < (int)(blockDim.x >> 5) ? part[lane] : 0.0f);
    const DF v = mean_square(sum, (float)a.K, a.inv_K, a.eps * pre * pre);
    RowScale rs(inverse_root(v));
    if (pre == 1.0f && !(v.hi >= kLeast && v.hi < INFINITY)) {
      rs.pre = v.hi < kLeast ? kGrow : kShrink;
      rs.lo = 0.0f;
    }
    if (lane == 0) scale = rs;
  }
  __syncthreads();  // after it a next call may write `part`, but not yet `scale`
  return scale;
}

// The last block of a norm's grid clears the scales of the last tile's missing rows.
__device__ __forceinline__ void clear_missing(const NormArgs& a, int G) {
  const int last = (a.rows + kTileRows - 1) / kTileRows * kTileRows;
  for (int u = threadIdx.x; u < (last - a.rows) * G; u += blockDim.x)
    *reinterpret_cast<uint32_t*>(a.scales + scale_word(a.rows + u / G, u % G, G)) = 0;
}

// A block takes rows in turn, each in registers (eight elements a thread), and loads the next one
// while it works on a row: the block's sum and what follows it would leave the memory idle
// otherwise. The weight stays in registers. The last block clears the missing rows' scales. With a
// residual: 17408 x 2048 fp32 73 us (6.4 TB/s), 2048 x 4096 bf16 13.4 us (4.4 TB/s: two block
// barriers and a root each row), one row of 4096 3.2 us.
template <int DT, int WDT, int FMT>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(NormArgs a) {
  constexpr bool kExact = DT == SPEC_BF16 && WDT == SPEC_BF16;
  const int G = groups(a.K), Kp = G * kGroup, blocks = gridDim.x - 1;
  grid_dep_wait();
  if ((int)blockIdx.x == blocks) {
    clear_missing(a, G);
    return;
  }
  const int k = 8 * threadIdx.x;
  Pair<DT> next;
  Piece<WDT> w;
  clear<DT>(next.x);
  clear<DT>(next.r);
  clear<WDT>(w);
  if (k < a.K) {
    load_pair<DT>(a, blockIdx.x, k, next);
    load8<WDT, true>(a.weight, 0, k, a.K, a.wvec, w);
  }
  bool finite = true;
  for (int row = blockIdx.x; row < a.rows; row += blocks) {
    Piece<DT> h;
    clear<DT>(h);
    if (k < a.K) {
      h = add_pair<DT>(a, row, k, next);
      if (row + blocks < a.rows) load_pair<DT>(a, row + blocks, k, next);
    }
    RowScale rs = row_scale(sum_squares<DT>(h, 1.0f), a, 1.0f);
    float y[8], v[8];
    unpack<DT>(h, y);
    unpack<WDT>(w, v);
    if (rs.lo != 0.0f) {  // the same in all threads
      scale8<kExact, false>(y, rs, v, k, a.K);
    } else {
      if (const float pre = rs.pre; pre != 1.0f) {
        rs = row_scale(sum_squares<DT>(h, pre), a, pre);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= pre;
      }
      scale8<kExact, true>(y, rs, v, k, a.K);
    }
    finite &= quantize8<FMT>(y, k < Kp,
                             a.codes + ((size_t)row * G * kGroup + k) / 8 * kLaneCode<FMT>,
                             a.scales + scale_word(row, k / kGroup, G));
  }
  if (!finite) atomicOr(a.status, SPEC_DEV_NONFINITE);
}

// Rows too long for registers, one block each: read twice (the second time from cache), which with
// one row at a time bounds it: 1024 x 16384 bf16 with a residual 35.2 us (3.4 TB/s; with one block an
// SM, above 32 registers a thread, 44), 512 x 16384 fp32 34.0 us, one row 9.4 us.
template <int DT, int WDT, int FMT>
__global__ void __launch_bounds__(1024, 2) rmsnorm_long_kernel(NormArgs a) {
  constexpr bool kExact = DT == SPEC_BF16 && WDT == SPEC_BF16;
  const int G = groups(a.K), Kp = G * kGroup, row = blockIdx.x, step = 8 * blockDim.x;
  grid_dep_wait();
  if (row == a.rows) {
    clear_missing(a, G);
    return;
  }
  NormArgs sum_only = a;
  sum_only.res_out = nullptr;
  auto scale_of = [&](float pre) {
    DF sum = df_zero();  // a chain of K / 8192 pieces: exact additions
    for (int k = 8 * threadIdx.x; k < a.K; k += step) {
      Pair<DT> p;
      load_pair<DT>(a, row, k, p);
      sum = df_add(sum, sum_squares<DT>(add_pair<DT>(sum_only, row, k, p), pre));
    }
    return row_scale(df_float(sum), a, pre);
  };
  RowScale rs = scale_of(1.0f);
  const float pre = rs.pre;
  if (pre != 1.0f) rs = scale_of(pre);  // the same in all threads
  uint8_t* codes = a.codes + (size_t)row * G * kGroupCode<FMT>;
  bool finite = true;
  for (int k0 = 0; k0 < Kp; k0 += step) {
    const int k = k0 + 8 * threadIdx.x;
    float h[8] = {0, 0, 0, 0, 0, 0, 0, 0}, v[8];
    if (k < a.K) {
      Pair<DT> p;
      Piece<WDT> w;
      load_pair<DT>(a, row, k, p);
      load8<WDT, true>(a.weight, 0, k, a.K, a.wvec, w);  // before the sum's store: no wait between
      unpack<DT>(add_pair<DT>(a, row, k, p), h);
      if (pre != 1.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] *= pre;
      }
      unpack<WDT>(w, v);
      if (rs.lo != 0.0f)
        scale8<kExact, false>(h, rs, v, k, a.K);
      else
        scale8<kExact, true>(h, rs, v, k, a.K);
    }
    finite &= quantize8<FMT>(h, k < Kp, codes + k / 8 * kLaneCode<FMT>,
                             a.scales + scale_word(row, k / kGroup, G));
  }
  if (!finite) atomicOr(a.status, SPEC_DEV_NONFINITE);
}

// Blocks of a kernel that an SM holds at once.
template <typename K>
int blocks_per_sm(K k, int threads) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k, threads, 0) != cudaSuccess || n < 1)
    n = 1;
  return n;
}

// Blocks of a streaming kernel: one for each of its units. Loops over fewer, resident blocks were
// slower (129280 x 4096: 237 against 213 us to read back): a new block's loads overlap the end of
// those beside it.
int grid_for(long long units, int per_block) {
  return (int)((units + per_block - 1) / per_block);
}

template <int DT, int FMT>
void launch_quantize_t(const void* x, long long ldx, int rows, int K, int vec, uint8_t* codes,
                       uint8_t* scales, uint32_t* status, cudaStream_t s) {
  const long long units = (long long)((rows + kTileRows - 1) / kTileRows) * kTileRows * groups(K);
  launch_kernel(quantize_kernel<DT, FMT>, grid_for(units, kWide * kUnroll<DT>), kThreads, 0, s,
                true, x, ldx, rows, K, vec, codes, scales, status);
}

template <int DT, int FMT>
void launch_dequantize_t(const uint8_t* codes, const uint8_t* scales, int rows, int K, bool vec,
                         void* out, long long ldo, cudaStream_t s) {
  const int grid = grid_for((long long)rows * groups(K), kUnits * kUnrollBack);
  launch_kernel(dequantize_kernel<DT, FMT>, grid, kThreads, 0, s, true, codes, scales, rows, K, vec,
                out, ldo);
}

template <int DT, int WDT, int FMT>
void launch_norm_t(const NormArgs& a, cudaStream_t s) {
  const int pieces = groups(a.K) * (kGroup / 8), threads = (pieces + 31) / 32 * 32;
  if (threads > 1024) {
    launch_kernel(rmsnorm_long_kernel<DT, WDT, FMT>, a.rows + 1, 1024, 0, s, true, a);
    return;
  }
  auto k = rmsnorm_kernel<DT, WDT, FMT>;
  // by warps of a block; devices differ in their number of SMs
  static int per_sm[33] = {};
  int n = __atomic_load_n(&per_sm[threads / 32], __ATOMIC_RELAXED);
  if (!n) __atomic_store_n(&per_sm[threads / 32], n = blocks_per_sm(k, threads), __ATOMIC_RELAXED);
  n *= num_sms();  // they loop over the rest of the rows
  const int blocks = a.rows < n ? a.rows : n;
  launch_kernel(k, blocks + 1, threads, 0, s, true, a);
}

template <int DT, int WDT>
void launch_norm_w(const NormArgs& a, int fmt, cudaStream_t s) {
  fmt == SPEC_MX_E2M1 ? launch_norm_t<DT, WDT, SPEC_MX_E2M1>(a, s)
                      : launch_norm_t<DT, WDT, SPEC_MX_E4M3>(a, s);
}

// Rows at multiples of `bytes`.
bool vec_ok(const void* p, long long ld, int dt, int bytes = 16) {
  const size_t es = dt == SPEC_BF16 ? 2 : 4;
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % bytes == 0 && (ld * es) % bytes == 0);
}

}  // namespace

}  // namespace mx

void launch_mx_quantize(const void* x, int dt, long long ldx, int rows, int K, int fmt,
                        uint8_t* codes, uint8_t* scales, uint32_t* status, cudaStream_t s) {
  using namespace mx;
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  const int vec = vec_ok(x, ldx, dt, 32) ? 2 : vec_ok(x, ldx, dt) ? 1 : 0;
  auto launch = dt == SPEC_BF16
                    ? (fmt == SPEC_MX_E2M1 ? launch_quantize_t<SPEC_BF16, SPEC_MX_E2M1>
                                           : launch_quantize_t<SPEC_BF16, SPEC_MX_E4M3>)
                    : (fmt == SPEC_MX_E2M1 ? launch_quantize_t<SPEC_F32, SPEC_MX_E2M1>
                                           : launch_quantize_t<SPEC_F32, SPEC_MX_E4M3>);
  launch(x, ldx, rows, K, vec, codes, scales, status, s);
}

void launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int fmt, int rows, int K,
                          void* out, int dt, long long ldo, cudaStream_t s) {
  using namespace mx;
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  const bool vec = vec_ok(out, ldo, dt);
  auto launch = dt == SPEC_BF16
                    ? (fmt == SPEC_MX_E2M1 ? launch_dequantize_t<SPEC_BF16, SPEC_MX_E2M1>
                                           : launch_dequantize_t<SPEC_BF16, SPEC_MX_E4M3>)
                    : (fmt == SPEC_MX_E2M1 ? launch_dequantize_t<SPEC_F32, SPEC_MX_E2M1>
                                           : launch_dequantize_t<SPEC_F32, SPEC_MX_E4M3>);
  launch(codes, scales, rows, K, vec, out, ldo, s);
}

void launch_rmsnorm_mx(const void* x, long long ldx, const void* res, long long ldr, int dt,
                       const void* weight, int wdt, float eps, int rows, int K, void* res_out,
                       long long ldo, int fmt, uint8_t* codes, uint8_t* scales, uint32_t* status,
                       cudaStream_t s) {
  using namespace mx;
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  NormArgs a{x, res, res_out, weight, ldx, ldr, ldo, rows, K, eps, 1.0f / (float)K, false, false,
             codes,
             scales, status};
  a.vec = vec_ok(x, ldx, dt) && (!res || (vec_ok(res, ldr, dt) && vec_ok(res_out, ldo, dt)));
  a.wvec = vec_ok(weight, 0, wdt);
  if (dt == SPEC_BF16)
    wdt == SPEC_BF16 ? launch_norm_w<SPEC_BF16, SPEC_BF16>(a, fmt, s)
                     : launch_norm_w<SPEC_BF16, SPEC_F32>(a, fmt, s);
  else
    wdt == SPEC_BF16 ? launch_norm_w<SPEC_F32, SPEC_BF16>(a, fmt, s)
                     : launch_norm_w<SPEC_F32, SPEC_F32>(a, fmt, s);
}

}  // namespace spec
