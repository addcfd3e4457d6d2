// mx.cuh -- block-scaled (microscaled) floating point: formats, scale rule and layout, shared by
// the kernels that write such matrices (mx.cu) and the product that reads them (mx_logits.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace spec {
namespace mx {

constexpr int kBlock = SPEC_MX_BLOCK;  // elements that share a scale
constexpr int kGroup = SPEC_MX_GROUP;  // elements whose four scales share a 32-bit word
constexpr int kTileRows = 128;         // rows of a scale tile
constexpr int kTileBytes = 512;        // bytes of a scale tile: 128 rows x 4 scales
constexpr int kNanScale = 255;

__host__ __device__ inline int padded(int K) { return (K + kGroup - 1) / kGroup * kGroup; }
__host__ __device__ inline int groups(int K) { return (K + kGroup - 1) / kGroup; }

// Bytes of a padded row's codes.
__host__ __device__ inline size_t code_row(int fmt, int Kp) {
  return fmt == SPEC_MX_E2M1 ? (size_t)Kp / 2 : (size_t)Kp;
}

// Byte offset of the scale word (four scales, 128 elements) of row r and group g. The tile is
// what tcgen05.cp spreads over tensor memory: lane r % 32, column r % 128 / 32.
__host__ __device__ inline size_t scale_word(int r, int g, int G) {
  return ((size_t)(r >> 7) * G + g) * kTileBytes + (size_t)((r & 31) * 16 + ((r >> 5) & 3) * 4);
}

// Stored scale byte of a block whose largest magnitude has the fp32 bits `amax`: the smallest
// power of two 2^(byte - 127) with amax <= top * 2^(byte - 127). top = 1.5 * 2^2 (E2M1) or
// 1.75 * 2^8 (E4M3), so the exponent is amax's less 2 (less 8), plus one if amax's significand
// passes top's. 255 for a block that is not finite (integer order: NaN above infinity).
template <int FMT>
__device__ __forceinline__ int scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return kNanScale;
  const int ex = (int)(amax >> 23), man = (int)(amax & 0x7fffffu);
  const int b = FMT == SPEC_MX_E2M1 ? ex - 2 + (man > 0x400000) : ex - 8 + (man > 0x600000);
  return b < 0 ? 0 : b;
}

// 2^(127 - byte), the factor that brings a block into the format's range (a normal fp32 number
// for every byte a finite block has: 0 .. 253).
__device__ __forceinline__ float unscale(int byte) {
  return __uint_as_float((uint32_t)(254 - byte) << 23);
}

// 2^(byte - 127); byte 0 is a subnormal, 255 a NaN.
__device__ __forceinline__ float scale_value(int byte) {
  return __uint_as_float(byte == kNanScale ? 0x7fc00000u
                                           : (byte == 0 ? 0x00400000u : (uint32_t)byte << 23));
}

// Eight values to the format, nearest with ties to even; the first in the lowest bits.
__device__ __forceinline__ uint2 to_e4m3x8(const float (&y)[8]) {
  uint2 c;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(c.x)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(c.y)
      : "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return c;
}

__device__ __forceinline__ uint32_t to_e2m1x8(const float (&y)[8]) {
  uint32_t c;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(c)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return c;
}

// Values of two codes (exact in fp16, the instruction's result type); the upper bits of c are
// ignored.
__device__ __forceinline__ void half2_to_float(uint32_t h, float& lo, float& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.f32.f16 %0, a;\n\t"
      "cvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

__device__ __forceinline__ void from_e4m3x2(uint32_t c, float& lo, float& hi) {
  uint32_t h;
  asm("{\n\t.reg .b16 a;\n\t"
      "cvt.u16.u32 a, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(h)
      : "r"(c));
  half2_to_float(h, lo, hi);
}

__device__ __forceinline__ void from_e2m1x2(uint32_t c, float& lo, float& hi) {
  uint32_t h;
  asm("{\n\t.reg .b8 a;\n\t"
      "cvt.u8.u32 a, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
      : "=r"(h)
      : "r"(c));
  half2_to_float(h, lo, hi);
}

}  // namespace mx
}  // namespace spec
