// w4.cu -- matrices of 4-bit weights with a scale per group: packing, reading back, and their
// product with a few rows, which are residual-added and RMS-normalised on the way where asked.
//
//   w[n, k] = (code[n, k] - zero[n, k / G]) * scale[n, k / G];   y[m, n] = sum_k a[m, k] w[n, k].
//
// The product reads the packed matrix once: N K / 2 bytes and its scales bound it (129280 x 4096 at
// groups of 128: 273 MB, 40 us at the copy bandwidth), so it has to keep the memory busy and to spend
// little on a weight. A warp's mma.sync m16n8k16 takes 16 matrix rows against 8 columns: the codes
// become bf16 numbers 128 + code with one shift and one logical operation a pair, code - zero with
// one subtraction, both exact; the scale is applied to a group's fp32 sum. tcgen05 would want the
// unpacked matrix in shared memory, four times the bytes, for a multiplication that is not the bound.
//
// Columns. A number of the rows is two or three bf16 numbers that add up to it exactly, each a
// column of its own, so nothing is rounded to 8 bits: one column a row for bf16 rows as they are,
// two where a bf16 norm weight is multiplied in (16 bits), three for 32-bit numbers (24 bits). The
// norm's 1 / rms is applied to the sums.
//
// Order. A code's position in k is free as long as the rows' columns are permuted alike. A lane holds
// words of eight codes; pair s of a word is (code s, code s + 4). With groups of 128 a lane's four
// words of a 128-code block are consecutive, with 64 (32) pairs of (single) words are dealt to a
// quad's lanes, so that an mma never straddles two groups.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace spec {
namespace w4 {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kBlock = 128;     // codes of a row that a warp takes at once
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

__host__ __device__ constexpr int padded(int K) { return (K + kBlock - 1) / kBlock * kBlock; }

// Eight consecutive elements of a row as fp32, zeros past K.
__device__ __forceinline__ void load8(const void* p, int dt, size_t row, int k, int K,
                                      float (&v)[8]) {
  if (dt == SPEC_BF16) {
    const uint16_t* at = static_cast<const uint16_t*>(p) + row + k;
    if (k + 8 <= K && (reinterpret_cast<uintptr_t>(at) & 15) == 0) {
      const uint4 q = ld_coherent16(at);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = k + i < K ? bf16_to_f32(at[i]) : 0.0f;
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

__device__ __forceinline__ void store8(void* p, int dt, size_t row, int k, int K,
                                       const float (&v)[8]) {
  if (dt == SPEC_BF16) {
    uint16_t* at = static_cast<uint16_t*>(p) + row + k;
    const uint32_t w[4] = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                           bf16_pair(v[6], v[7])};
    if (k + 8 <= K && (reinterpret_cast<uintptr_t>(at) & 15) == 0) {
      *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < K) at[i] = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
    }
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

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float load_scale(const void* p, int dt, size_t at) {
  return dt == SPEC_BF16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[at])
                         : static_cast<const float*>(p)[at];
}

// ------------------------------------------------------------------------------ packing

constexpr int kPackThreads = 256;

// A lane takes eight consecutive elements, G / 8 lanes a group. The scale is the least s of its type
// with 7 s >= the group's largest magnitude: the quotient, cut or rounded, is at most one step
// below it, and 7 s against that magnitude is exact in one fused operation. A code is w / s rounded
// to the nearest, ties to even: w * (1 / s) is within one of it, and w - code * s is exact.
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const void* x, int dt, long long ldx,
                                                            int rows, int K, int G,
                                                            uint8_t* codes, void* scales, int sdt,
                                                            uint32_t* status) {
  grid_dep_wait();
  const int Kp = padded(K), per = Kp / 8;
  const long long n = (long long)rows * per;
  for (long long base = (long long)blockIdx.x * kPackThreads; base < n;
       base += (long long)gridDim.x * kPackThreads) {
    const long long at = base + threadIdx.x;
    const bool in = at < n;
    const int row = in ? (int)(at / per) : 0, k = in ? (int)(at % per) * 8 : 0;
    float v[8];
    load8(x, dt, (size_t)row * ldx, k, in ? K : 0, v);
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max_nan(a, fabsf(v[i]));
    for (int o = 1; o < G / 8; o *= 2) a = max_nan(a, __shfl_xor_sync(kFull, a, o));
    const bool bad = !(a < INFINITY);
    float s = __fdiv_rn(a, 7.0f);
    if (sdt == SPEC_BF16) s = __uint_as_float(__float_as_uint(s) & 0xffff0000u);
    if (fmaf(7.0f, s, -a) < 0.0f)
      s = __uint_as_float(__float_as_uint(s) + (sdt == SPEC_BF16 ? 0x10000u : 1u));
    if (bad) s = NAN;
    uint32_t w = 0;
    const bool plain = s > 0x1p-100f;  // 1 / s is finite and normal
    const float r = __fdiv_rn(1.0f, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float c = rintf(plain ? v[i] * r : __fdiv_rn(v[i], s));
      const float e = fmaf(-c, s, v[i]), half = 0.5f * s;
      if (plain) {
        const bool odd = ((int)c) & 1;
        if (e > half || (e == half && odd)) c += 1.0f;
        if (e < -half || (e == -half && odd)) c -= 1.0f;
      }
      const int q = s > 0.0f ? (int)c + 8 : 8;  // zeros, and what has no scale
      w |= (uint32_t)(q & 15) << (4 * i);
    }
    if (!in) continue;
    *reinterpret_cast<uint32_t*>(codes + at * 4) = w;
    if ((k & (G - 1)) == 0) {
      const size_t g = (size_t)row * (Kp / G) + k / G;
      if (sdt == SPEC_BF16)
        static_cast<uint16_t*>(scales)[g] = bad ? 0x7fffu : (uint16_t)(__float_as_uint(s) >> 16);
      else
        static_cast<float*>(scales)[g] = s;
      if (bad) atomicOr(status, SPEC_DEV_NONFINITE);
    }
  }
}

__global__ void __launch_bounds__(kPackThreads) unpack_kernel(const uint8_t* codes,
                                                              const void* scales, int sdt,
                                                              const uint8_t* zeros, int rows, int K,
                                                              int G, void* out, int odt,
                                                              long long ldo) {
  grid_dep_wait();
  const int Kp = padded(K), per = Kp / 8;
  const long long n = (long long)rows * per;
  for (long long at = (long long)blockIdx.x * kPackThreads + threadIdx.x; at < n;
       at += (long long)gridDim.x * kPackThreads) {
    const int row = (int)(at / per), k = (int)(at % per) * 8;
    if (k >= K) continue;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + at * 4);
    const size_t g = (size_t)row * (Kp / G) + k / G;
    const float s = load_scale(scales, sdt, g);
    const int z = zeros ? zeros[g] & 127 : 8;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = (float)((int)(w >> (4 * i) & 15) - z);
      v[i] = __fmul_rn(c, s);
      // towards the odd neighbour where fp32 does not hold the product, so that bf16 rounds it once
      const float rest = fmaf(c, s, -v[i]);
      if (odt == SPEC_BF16 && rest != 0.0f) {
        uint32_t b = __float_as_uint(v[i]);
        if ((rest < 0.0f) != (v[i] < 0.0f)) --b;
        v[i] = __uint_as_float(b | 1u);
      }
    }
    store8(out, odt, (size_t)row * ldo, k, K, v);
  }
}

// ------------------------------------------------------------------------------ product

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes s and s + 4 of a word less the zero point; zz is the pair 128 + zero.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int s, uint32_t zz) {
  const uint32_t q = ((w >> (4 * s)) & 0x000f000fu) | 0x43004300u;  // bf16 128 + code
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&q),
                                   *reinterpret_cast<const __nv_bfloat162*>(&zz));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// What a lane holds of two matrix rows (16 f + lane / 4, and 8 below) of a block.
template <int G>
struct Codes {
  static constexpr int kGroups = kBlock / G;
  uint32_t w[2][4];
  float s[2][kGroups];
  uint32_t z[2];  // zero points, a byte a group
};

struct Frame {
  uint4* x;      // the rows' columns: [block][word][column][lane % 4]
  float* red;    // [warp][16 R][stride]
  float* rstd;   // [rows]
  float* stat;   // [2][rows][kWarps]
};

// The chunk's rows into shared memory as bf16 columns, with their 1 / rms; h goes out, a share from
// each CTA of the chunk.
__device__ __forceinline__ void stage_rows(const W4Args& a, const Frame& f, int m0, int rows,
                                           int cols, int share, int shares) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Kp = padded(a.K), pieces = Kp / 8;
  const bool norm = a.weight != nullptr;
  auto pass = [&](int m, float scale) {
    float most = 0.0f, sum = 0.0f;
    for (int p = tid; p < pieces; p += kThreads) {
      const int k = p * 8;
      float v[8];
      load8(a.x, a.dtype, (size_t)(m0 + m) * a.ldx, k, a.K, v);
      if (a.residual) {
        float r[8];
        load8(a.residual, a.dtype, (size_t)(m0 + m) * a.ldr, k, a.K, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = __fadd_rn(v[i], r[i]);
          if (a.dtype == SPEC_BF16) v[i] = __bfloat162float(__float2bfloat16_rn(v[i]));
        }
        if (p % shares == share) store8(a.h, a.dtype, (size_t)(m0 + m) * a.ldh, k, a.K, v);
      }
      float g[8];
      if (norm) load8(a.weight, a.w_dtype, 0, k, a.K, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        most = max_nan(most, fabsf(v[i]));
        v[i] *= scale;
        sum = fmaf(v[i], v[i], sum);
        if (norm) v[i] *= g[i];
      }
      // piece of the block -> (word, lane of the quad)
      const int pi = p & 15;
      int w, t;
      if (a.group == 128) {
        t = pi >> 2;
        w = pi & 3;
      } else if (a.group == 64) {
        t = (pi & 7) >> 1;
        w = (pi >> 3) * 2 + (pi & 1);
      } else {
        t = pi & 3;
        w = pi >> 2;
      }
      uint4* to = f.x + (size_t)((p >> 4) * 4 + w) * cols * 4 + t;
      for (int q = 0; q < a.parts; ++q) {
        uint32_t top[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // cut, not rounded: nothing overflows, the rest is exact
          top[i] = __float_as_uint(v[i]) & 0xffff0000u;
          v[i] = __fsub_rn(v[i], __uint_as_float(top[i]));
        }
        to[(m * a.parts + q) * 4] =
            make_uint4(top[0] >> 16 | top[4], top[1] >> 16 | top[5], top[2] >> 16 | top[6],
                       top[3] >> 16 | top[7]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      most = max_nan(most, __shfl_xor_sync(kFull, most, o));
      sum += __shfl_xor_sync(kFull, sum, o);
    }
    if (lane == 0) {
      f.stat[m * kWarps + warp] = most;
      f.stat[(rows + m) * kWarps + warp] = sum;
    }
  };
  for (int m = 0; m < rows; ++m) pass(m, 1.0f);
  __syncthreads();
  for (int m = 0; m < rows; ++m) {
    float most = 0.0f, sum = 0.0f;
    for (int w = 0; w < kWarps; ++w) {
      most = max_nan(most, f.stat[m * kWarps + w]);
      sum += f.stat[(rows + m) * kWarps + w];
    }
    float scale = 1.0f;
    if (!(most < INFINITY) && share == 0 && tid == 0) atomicOr(a.status, SPEC_DEV_NONFINITE);
    if (norm && most < INFINITY && most > 0.0f && (most > 0x1p50f || most < 0x1p-40f)) {
      // squares that leave fp32's range: the row once more, by a power of two (no smaller one than
      // eps times its square allows)
      int e = (int)(__float_as_uint(most) >> 23) - 127;
      const int least = a.eps == 0.0f ? -126 : a.eps >= 1.0f ? 0 : -60;
      e = e > least ? e : least;
      scale = __uint_as_float((uint32_t)(127 - (e < 126 ? e : 126)) << 23);
      __syncthreads();
      pass(m, scale);
      __syncthreads();
      sum = 0.0f;
      for (int w = 0; w < kWarps; ++w) sum += f.stat[(rows + m) * kWarps + w];
    }
    if (tid == 0)
      f.rstd[m] = norm ? 1.0f / sqrtf(sum / (float)a.K + a.eps * scale * scale) : 1.0f;
  }
  __syncthreads();
}

template <int G, int R, int T>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const W4Args a) {
  extern __shared__ uint4 smem[];
  constexpr int kGroups = kBlock / G;
  constexpr int D = G == 128 ? 3 : 2;       // blocks in flight a warp
  constexpr int kStride = 8 * T + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int Kp = padded(a.K), KB = Kp / kBlock, groups = Kp / G;
  const int real_groups = (a.K + G - 1) / G;
  const int chunk = blockIdx.x % a.chunks, share = blockIdx.x / a.chunks;
  const int shares = gridDim.x / a.chunks;
  const int m0 = chunk * a.chunk_rows, rows = min(a.chunk_rows, a.M - m0);
  const int cols = rows * a.parts;
  Frame f;
  f.x = smem;
  f.red = reinterpret_cast<float*>(smem + (size_t)KB * 16 * a.chunk_rows * a.parts);
  f.rstd = f.red + kWarps * 16 * R * kStride;
  f.stat = f.rstd + a.chunk_rows;

  const int kw = a.k_warps, wk = warp % kw, wr = warp / kw;
  const int unit_rows = kWarps / kw * 16 * R;
  const int units = (a.N + unit_rows - 1) / unit_rows;
  const int nk = (KB + kw - 1) / kw;
  const int mine = share < units ? (units - share - 1) / shares + 1 : 0;

  grid_dep_wait();
  Codes<G> ring[D][R];
  int pu = share, pk = 0;  // unit and block of the next load
  auto load = [&](Codes<G> (&c)[R]) {
    const int kb = wk * nk + pk;
    if (pu < units && kb < KB) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = min(a.N - 1, pu * unit_rows + wr * 16 * R + r * 16 + h * 8 + g);
          const uint8_t* p = a.codes + (size_t)n * (Kp / 2) + kb * 64;
          if constexpr (G == 128) {
            const uint4 q = ld_coherent16(p + t * 16);
            c[r].w[h][0] = q.x;
            c[r].w[h][1] = q.y;
            c[r].w[h][2] = q.z;
            c[r].w[h][3] = q.w;
          } else if constexpr (G == 64) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint2 q = *reinterpret_cast<const uint2*>(p + i * 32 + t * 8);
              c[r].w[h][2 * i] = q.x;
              c[r].w[h][2 * i + 1] = q.y;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              c[r].w[h][i] = *reinterpret_cast<const uint32_t*>(p + i * 16 + t * 4);
          }
          const size_t at = (size_t)n * groups + kb * kGroups;
          c[r].z[h] = 0x08080808u;
#pragma unroll
          for (int i = 0; i < kGroups; ++i)
            c[r].s[h][i] = kb * kGroups + i < real_groups ? load_scale(a.scales, a.scale_dtype, at + i)
                                                          : 0.0f;
          if (a.zeros) {
            c[r].z[h] = 0;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) c[r].z[h] |= (uint32_t)a.zeros[at + i] << (8 * i);
          }
        }
    }
    if (++pk == nk) {
      pk = 0;
      pu += shares;
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(ring[d]);
  stage_rows(a, f, m0, rows, cols, share, shares);

  float acc[R][T][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < T; ++j) acc[r][j][0] = acc[r][j][1] = acc[r][j][2] = acc[r][j][3] = 0.0f;
  int col[T];  // columns past the last one repeat it and are not used
#pragma unroll
  for (int j = 0; j < T; ++j) col[j] = min(cols - 1, j * 8 + g) * 4 + t;
  int unit = share, ik = 0;
  const int total = mine * nk;
  for (int it = 0; it < total; it += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (it + d >= total) break;
      const int kb = wk * nk + ik;
      if (kb < KB) {
        const uint4* xb = f.x + (size_t)kb * 16 * cols;
        float part[R][T][4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          constexpr int kPer = 4 / kGroups;  // words of a group
          if (w % kPer == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int j = 0; j < T; ++j)
                part[r][j][0] = part[r][j][1] = part[r][j][2] = part[r][j][3] = 0.0f;
          }
          uint4 b[T];
#pragma unroll
          for (int j = 0; j < T; ++j) b[j] = xb[w * cols * 4 + col[j]];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const Codes<G>& c = ring[d][r];
            const uint32_t z0 = c.z[0] >> (8 * (w / kPer)) & 127u;
            const uint32_t z1 = c.z[1] >> (8 * (w / kPer)) & 127u;
            const uint32_t zz0 = 0x43004300u + z0 * 0x10001u, zz1 = 0x43004300u + z1 * 0x10001u;
#pragma unroll
            for (int s = 0; s < 4; s += 2) {
              const uint32_t q[4] = {code_pair(c.w[0][w], s, zz0), code_pair(c.w[1][w], s, zz1),
                                     code_pair(c.w[0][w], s + 1, zz0),
                                     code_pair(c.w[1][w], s + 1, zz1)};
#pragma unroll
              for (int j = 0; j < T; ++j)
                mma(part[r][j], q, s ? b[j].z : b[j].x, s ? b[j].w : b[j].y);
            }
            if (w % kPer == kPer - 1) {
              const float s0 = c.s[0][w / kPer], s1 = c.s[1][w / kPer];
#pragma unroll
              for (int j = 0; j < T; ++j) {
                acc[r][j][0] = fmaf(s0, part[r][j][0], acc[r][j][0]);
                acc[r][j][1] = fmaf(s0, part[r][j][1], acc[r][j][1]);
                acc[r][j][2] = fmaf(s1, part[r][j][2], acc[r][j][2]);
                acc[r][j][3] = fmaf(s1, part[r][j][3], acc[r][j][3]);
              }
            }
          }
        }
      }
      load(ring[d]);
      if (++ik < nk) continue;
      // the unit's sums, over the warps that share its rows
      ik = 0;
      float* red = f.red + warp * 16 * R * kStride;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < T; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            red[(r * 16 + (i >> 1) * 8 + g) * kStride + j * 8 + t * 2 + (i & 1)] = acc[r][j][i];
            acc[r][j][i] = 0.0f;
          }
      __syncthreads();
      for (int e = tid; e < rows * unit_rows; e += kThreads) {
        const int m = e / unit_rows, r = e % unit_rows, n = unit * unit_rows + r;
        if (n >= a.N) continue;
        const float* at = f.red + (size_t)(r / (16 * R)) * kw * 16 * R * kStride +
                          (r % (16 * R)) * kStride + m * a.parts;
        float y = 0.0f;
        for (int w = 0; w < kw; ++w)
          for (int q = 0; q < a.parts; ++q) y += at[(size_t)w * 16 * R * kStride + q];
        y *= f.rstd[m];
        const size_t to = (size_t)(m0 + m) * a.ldo + n;
        if (a.out_dtype == SPEC_BF16)
          static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16_rn(y);
        else
          static_cast<float*>(a.out)[to] = y;
      }
      __syncthreads();
      unit += shares;
    }
  }
}

template <int G, int R, int T>
cudaError_t launch_t(const W4Args& a, cudaStream_t s) {
  const size_t smem = (size_t)padded(a.K) * 2 * a.chunk_rows * a.parts +
                      sizeof(float) * ((size_t)kWarps * 16 * R * (8 * T + 1) +
                                       a.chunk_rows * (1 + 2 * kWarps));
  auto k = product_kernel<G, R, T>;
  const cudaError_t e =
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int unit_rows = kWarps / a.k_warps * 16 * R, units = (a.N + unit_rows - 1) / unit_rows;
  int shares = num_sms() / a.chunks;
  shares = shares < 1 ? 1 : shares < units ? shares : units;
  return launch_kernel(k, dim3((unsigned)(shares * a.chunks)), dim3(kThreads), smem, s, true, a);
}

template <int G>
cudaError_t launch_g(const W4Args& a, int R, int T, cudaStream_t s) {
  if (R == 2) return T == 1 ? launch_t<G, 2, 1>(a, s) : launch_t<G, 2, 2>(a, s);
  return T == 1 ? launch_t<G, 1, 1>(a, s)
                : T == 2 ? launch_t<G, 1, 2>(a, s) : launch_t<G, 1, 4>(a, s);
}

}  // namespace

size_t row_bytes(int parts, int K) { return (size_t)padded(K) * 2 * parts; }
// Shared memory of the largest set of rows.
size_t rows_most() { return 160 * 1024; }

}  // namespace w4

bool w4_fits(int parts, int K) { return w4::row_bytes(parts, K) <= w4::rows_most(); }

cudaError_t launch_w4_logits(W4Args a, cudaStream_t s) {
  using namespace w4;
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  const int KB = padded(a.K) / kBlock;
  const int most = (int)(rows_most() / row_bytes(a.parts, a.K));
  a.chunk_rows = 32 / a.parts;
  if (a.chunk_rows > most) a.chunk_rows = most;
  a.chunks = (a.M + a.chunk_rows - 1) / a.chunk_rows;
  a.chunk_rows = (a.M + a.chunks - 1) / a.chunks;
  const int cols = a.chunk_rows * a.parts, T = cols <= 8 ? 1 : cols <= 16 ? 2 : 4;
  a.k_warps = 1;
  while (a.k_warps < 8 && a.k_warps * 2 <= KB) a.k_warps *= 2;
  // two 16-row tiles a warp where there are units enough for every SM
  int R = T <= 2 ? 2 : 1;
  if (R == 2 && (long long)a.N < (long long)num_sms() * (kWarps / a.k_warps) * 32) R = 1;
  switch (a.group) {
    case 128:
      return launch_g<128>(a, R, T, s);
    case 64:
      return launch_g<64>(a, R, T, s);
    default:
      return launch_g<32>(a, R, T, s);
  }
}

void launch_w4_quantize(const void* x, int dt, long long ldx, int rows, int K, int group,
                        uint8_t* codes, void* scales, int sdt, uint32_t* status, cudaStream_t s) {
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  const long long n = ((long long)rows * (w4::padded(K) / 8) + w4::kPackThreads - 1) /
                      w4::kPackThreads;
  const int most = num_sms() * 8;
  launch_kernel(w4::pack_kernel, dim3((unsigned)(n < most ? n : most)), dim3(w4::kPackThreads), 0, s,
                true, x, dt, ldx, rows, K, group, codes, scales, sdt, status);
}

void launch_w4_dequantize(const uint8_t* codes, const void* scales, int sdt, const uint8_t* zeros,
                          int rows, int K, int group, void* out, int odt, long long ldo,
                          cudaStream_t s) {
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  const long long n = ((long long)rows * (w4::padded(K) / 8) + w4::kPackThreads - 1) /
                      w4::kPackThreads;
  const int most = num_sms() * 8;
  launch_kernel(w4::unpack_kernel, dim3((unsigned)(n < most ? n : most)), dim3(w4::kPackThreads), 0,
                s, true, codes, scales, sdt, zeros, rows, K, group, out, odt, ldo);
}

}  // namespace spec
