// w4_product.cuh -- the product of a few rows with a matrix of grouped 4-bit weights; residual
// addition and RMS norm on the way where asked.
//
//   w[n, k] = (code[n, k] - zero[n, k / G]) * scale[n, k / G];   y[m, n] = sum_k a[m, k] w[n, k].
//
// The product reads the packed matrix once: N K / 2 bytes and its scales bound it (129280 x 4096 at
// groups of 128: 273 MB, 40 us at the copy bandwidth), so it has to keep the memory busy and to spend
// little on a weight. Every warp has a ring of tiles of its own, 16 or 32 matrix rows of 128 codes,
// that its first lane fills by TMA: nothing but the tile's two coordinates is computed for them, and no
// register waits for them. (With the tiles loaded into registers, two to three blocks ahead, one row
// took 104 us.) A warp's mma.sync m16n8k16 takes 16 matrix rows against 8 columns: the codes
// become fp16 numbers 1024 + code, or 1024 + 16 code, with one logical operation a pair (and a shift
// for every second one), code - zero with one more, all exact; the scale is applied to a group's fp32
// sum. Two to sixteen warps that share a tile's rows, each a range of K, add their sums through
// shared memory; such teams go through the matrix by themselves. tcgen05 would want the unpacked
// matrix in shared memory, four times the bytes, for a multiplication that is not the bound (20 to 32 %
// of the tensor pipe's cycles). No unit is full: half the issue slots are used, and memory for one row
// to three quarters; what a warp waits for is the chain from its tile to its sums.
//
// Measured, 129280 x 4096: one row at groups of 128 53 us with its norm (75 % of the copy bandwidth),
// eight rows 88, 59 without the norm; one row at groups of 32 69; 16 rows at groups of 64 171, 111
// without the norm. 4 x 4096 x 8192 with zero points 14 us; 17 rows fp32 of 32000 x 2048, 40 columns,
// 47.
//
// Columns. A number of the rows is one or two fp16 numbers, each a column of its own. One is exact for
// bf16 rows as they are (from 2^-18 of the largest on: fp16's numbers end at 2^-24). 32-bit rows, and
// those with a norm weight multiplied in, take two, the second 2^12 times what the first leaves, so
// that it ends at 2^-36: together off by 2^-23, or by 2^-38 of the largest. That goes for bf16
// products too: with one, of 11 bits, one bf16 output in ten was a step from the 64-bit product's
// rounding, and eight rows of 129280 x 4096 took 65 us with their norm where they take 88 (one row 53
// in both). Rows are scaled by powers of two into fp16's range; that and the norm's 1 / rms are
// applied to the sums.
//
// Order. A code's position in k is free as long as the rows' columns are permuted alike. A lane holds
// words of eight codes; pair s of a word is (code s, code s + 4). With groups of 128 a lane's four
// words of a 128-code block are consecutive, with 64 (32) pairs of (single) words are dealt to a
// quad's lanes, so that an mma never straddles two groups.
#pragma once

#include "tc_ptx.cuh"
#include "w4.cuh"

namespace spec {
namespace w4 {
namespace {

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// c = a b (ZERO), or c += a b.
template <bool ZERO>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (ZERO)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
  else
    mma(c, a, b0, b1);
}

__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma2h(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t masked(uint32_t w, uint32_t mask) {  // (w & mask) | 1024, 1024
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(mask), "r"(0x64006400u));
  return d;
}
// Zero points of a group as fp16 pairs: 1024 + zero, and -(64 + zero).
struct Zero {
  uint32_t a = 0x64086408u, b = 0xd480d480u;  // of 8
  __device__ __forceinline__ Zero() {}
  __device__ __forceinline__ explicit Zero(uint32_t z)
      : a(0x64006400u + z * 0x10001u), b(sub2(0x63806380u, a)) {}  // 960 - (1024 + zero)
};

// Codes s and s + 4 of a word less the zero point, for s = 0 and 1 (of the word's upper bytes: 2 and
// 3). An fp16 number from 1024 to 2047 holds a code in its last bits, or 16 times one four bits up: the
// conversion of unsigned codes that Kim, Henry, Fahim and Awadalla published ("Who Says Elephants
// Can't Run", 2022), from whose arithmetic the constants follow; zero points are subtracted with it.
__device__ __forceinline__ uint32_t codes_even(uint32_t w, const Zero& z) {
  return sub2(masked(w, 0x000f000fu), z.a);
}
__device__ __forceinline__ uint32_t codes_odd(uint32_t w, const Zero& z) {
  return fma2h(masked(w, 0x00f000f0u), 0x2c002c00u, z.b);  // / 16
}

struct Frame {
  uint8_t* ring;  // [warp][stage][16 R rows][64 W bytes], swizzled over that width
  uint4* x;       // the rows' columns: [block][word][column][lane % 4]
  float* red;     // sums: [warp][16 R][stride]
  float* factor;  // [rows]: what a row's sums are multiplied with,
  float* power;   // [rows]: and then with this
  float* stat;    // [2][rows][pieces]
  uint64_t* full; // [warp][stage]
};

// Eight elements of h; x + residual goes out with `write`.
__device__ __forceinline__ void load_h(const W4Args& a, int m, int k, bool write, float (&v)[8]) {
  load8(a.x, a.dtype, (size_t)m * a.ldx, k, a.K, v);
  if (!a.residual) return;
  float r[8];
  load8(a.residual, a.dtype, (size_t)m * a.ldr, k, a.K, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = __fadd_rn(v[i], r[i]);
    if (a.dtype == SPEC_BF16) v[i] = __bfloat162float(__float2bfloat16_rn(v[i]));
  }
  if (write) store8(a.h, a.dtype, (size_t)m * a.ldh, k, a.K, v);
}

// Exponent e with 2^e <= x < 2^(e + 1), x positive and finite (-126 for smaller ones).
__device__ __forceinline__ int exponent(float x) {
  const int e = (int)(__float_as_uint(x) >> 23) - 127;
  return e > -126 ? e : -126;
}
__device__ __forceinline__ float power(int e) {  // 2^e, cut to the normal numbers
  e = e < -126 ? -126 : e > 127 ? 127 : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// A second column is kRest times what the first leaves: at most 2^15, as the numbers are.
constexpr float kRest = 0x1p12f;

// 32 pieces (of eight elements) of row m as fp16 columns, the numbers times hs and `scale`; the largest
// of these and the sum of (h hs)^2.
__device__ __forceinline__ void stage_pieces(const W4Args& a, const Frame& f, int m0, int m, int p,
                                             int cols, float hs, float scale, bool write,
                                             float& most, float& sum) {
  most = sum = 0.0f;
  if (p >= padded(a.K) / 8) return;
  float v[8];
  load_h(a, m0 + m, p * 8, write, v);
  if (a.weight) {
    float g[8];
    load8(a.weight, a.w_dtype, 0, p * 8, a.K, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] *= hs;
      sum = fmaf(v[i], v[i], sum);
      v[i] = v[i] * scale * g[i];  // in this order: the weights may be small
      most = max_nan(most, fabsf(v[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = v[i] * hs * scale;
      most = max_nan(most, fabsf(v[i]));
    }
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
  to += (size_t)m * a.parts * 4;
  __half2 pair[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) pair[i] = __floats2half2_rn(v[i], v[i + 4]);
  *to = *reinterpret_cast<const uint4*>(pair);
  if (a.parts == 1) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 back = __half22float2(pair[i]);
    pair[i] = __floats2half2_rn(__fsub_rn(v[i], back.x) * kRest, __fsub_rn(v[i + 4], back.y) * kRest);
  }
  to[4] = *reinterpret_cast<const uint4*>(pair);
}

// The chunk's rows into shared memory as fp16 columns, with the factors that their sums take; h goes
// out, a share from each CTA of the chunk. fp16 ends at 2^16 and its numbers are 2^-24 apart at the
// least: rows are multiplied by 2^4, which serves if the largest number, |h| |weight|, is then between
// 2 and 2^15; others are staged once more, by the power of two that brings theirs to 2^13 .. 2^14. The
// pieces are dealt to the warps by 32, whatever row they are of.
constexpr float kScale = 16.0f, kScaledLeast = 2.0f, kScaledMost = 0x1p15f;
template <typename F>
__device__ __forceinline__ void stage_rows(const W4Args& a, const Frame& f, int m0, int rows,
                                           int cols, int share, int shares, F&& loaded) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_row = pieces_of(a.K), all = rows * per_row;
  const bool norm = a.weight != nullptr;
  auto pass = [&](int c, float hs, float scale, bool write) {
    const int m = c / per_row, at = c % per_row;
    float most, sum;
    stage_pieces(a, f, m0, m, at * 32 + lane, cols, hs, scale, write, most, sum);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      most = max_nan(most, __shfl_xor_sync(kFull, most, o));
      sum += __shfl_xor_sync(kFull, sum, o);
    }
    if (lane == 0) {
      f.stat[c] = most;
      f.stat[all + c] = sum;
    }
  };
  // every CTA begins elsewhere, or all would ask for the same lines at once
  const int turn = (int)((long long)all * share / shares);
#pragma unroll 4
  for (int i = warp; i < all; i += kWarps) {
    const int c = i + turn < all ? i + turn : i + turn - all;
    pass(c, 1.0f, kScale, c % shares == share);
  }
  loaded();
  __syncthreads();
  // the largest number and the sum of a row, in one warp
  auto row = [&](int m, float& most, float& sum) {
    most = sum = 0.0f;
    for (int i = lane; i < per_row; i += 32) {
      most = max_nan(most, f.stat[m * per_row + i]);
      sum += f.stat[all + m * per_row + i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      most = max_nan(most, __shfl_xor_sync(kFull, most, o));
      sum += __shfl_xor_sync(kFull, sum, o);
    }
  };
  bool again = false;
  for (int m = warp; m < rows; m += kWarps) {
    float most, sum;
    row(m, most, sum);
    const float factor = norm ? 1.0f / sqrtf(sum / (float)a.K + a.eps) : 1.0f;
    const bool serves = most >= kScaledLeast && most < kScaledMost &&
                        (!norm || (sum > 0x1p-60f && sum < INFINITY));
    const bool once = serves || (!norm && most == 0.0f);  // without a norm zeros need no scale
    again |= !once;
    if (lane == 0) {
      f.factor[m] = factor * (1.0f / kScale);
      f.power[m] = once ? 1.0f : 0.0f;
    }
  }
  if (!__syncthreads_or(again)) return;
  // Rows again whose numbers, or their squares, leave the range: h 2^-eh is below 4 (2, but for the
  // largest numbers: 2^-eh has to be one, too), times the weight it is scaled by its own largest.
  // Every warp finds both powers for itself.
  for (int m = 0; m < rows; ++m) {
    if (f.power[m] != 0.0f) continue;
    float most_h = 0.0f, most = 0.0f;
    for (int p = lane; p < per_row * 32; p += 32) {
      if (p * 8 >= a.K) break;
      float v[8];
      load_h(a, m0 + m, p * 8, false, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) most_h = max_nan(most_h, fabsf(v[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      most_h = max_nan(most_h, __shfl_xor_sync(kFull, most_h, o));
    if (!(most_h < INFINITY) && share == 0 && threadIdx.x == 0)
      atomicOr(a.status, SPEC_DEV_NONFINITE);
    const int eh = most_h > 0.0f && most_h < INFINITY ? min(exponent(most_h), 126) : 0;
    if (norm) {
      for (int p = lane; p < per_row * 32; p += 32) {
        if (p * 8 >= a.K) break;
        float v[8], g[8];
        load_h(a, m0 + m, p * 8, false, v);
        load8(a.weight, a.w_dtype, 0, p * 8, a.K, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) most = max_nan(most, fabsf(v[i] * power(-eh) * g[i]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(kFull, most, o));
    } else {
      most = most_h * power(-eh);
    }
    const int e = most > 0.0f && most < INFINITY ? max(exponent(most), -113) : 0;
    __syncthreads();  // the factors and the columns of before have been read
    for (int c = m * per_row + warp; c < (m + 1) * per_row; c += kWarps)
      pass(c, power(-eh), power(13 - e), false);
    __syncthreads();
    if (warp == 0) {
      float sum;
      row(m, most, sum);
      sum /= (float)a.K;
      // beside eps in the scale in which neither passes fp32's range
      const bool small = eh < 0 && a.eps > 0.0f;
      const float q = !norm   ? 1.0f
                      : small ? 1.0f / sqrtf(a.eps + sum * power(eh) * power(eh))
                              : 1.0f / sqrtf(sum + a.eps * power(-eh) * power(-eh));
      // times 2^by, in halves: one number may not hold it
      const int by = (!norm || small ? eh : 0) + e - 13;
      if (lane == 0) {
        f.factor[m] = q * power(by / 2);
        f.power[m] = power(by - by / 2);
      }
    }
  }
  __syncthreads();
}

// What a lane needs of four groups beside the codes: scales (as they are stored) and zero points of
// its matrix rows (16 r + lane / 4, and 8 below). The next block's groups come first.
template <int G, int R, bool ZEROS, bool NARROW>
struct Side {
  static constexpr int kWords = NARROW ? 2 : 4;
  uint32_t s[R][2][kWords];
  uint32_t z[ZEROS ? R : 1][2];  // a byte a group

  // Scale n of the next block, n < 128 / G.
  __device__ __forceinline__ float scale(int r, int h, int n) const {
    if constexpr (NARROW) {
      const uint32_t w = s[r][h][n / 2];
      return __uint_as_float(n & 1 ? w & 0xffff0000u : w << 16);
    } else {
      return __uint_as_float(s[r][h][n]);
    }
  }
  __device__ __forceinline__ void next_block() {
    constexpr int kGroups = kBlock / G;
    if constexpr (kGroups == 4) return;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t(&w)[kWords] = s[r][h];
        if constexpr (NARROW) {
          w[0] = kGroups == 2 ? w[1] : __funnelshift_r(w[0], w[1], 16);
          w[1] >>= 16;
        } else if constexpr (kGroups == 2) {
          w[0] = w[2];
          w[1] = w[3];
        } else {
          w[0] = w[1];
          w[1] = w[2];
          w[2] = w[3];
        }
        if constexpr (ZEROS) z[r][h] >>= 8 * kGroups;
      }
  }
};

// A tile is 16 R matrix rows of W blocks. kw warps (a.k_warps) share its rows, each takes a range of
// the tiles along K; kWarps / kw such teams a CTA go through the matrix by themselves.
template <int G, int R, int T, int W, bool ZEROS, bool NARROW>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const W4Args a, const __grid_constant__ CUtensorMap codes) {
  extern __shared__ __align__(1024) uint8_t smem[];
  typedef Side<G, R, ZEROS, NARROW> SideT;
  constexpr int kGroups = kBlock / G, kChunk = 4 / kGroups;  // blocks of a Side
  constexpr int kRow = 64 * W;                               // bytes of a tile's row
  constexpr int kTile = 16 * R * kRow;
  constexpr int kSize = NARROW ? 2 : 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int Kp = padded(a.K), KB = Kp / kBlock, KT = (KB + W - 1) / W;
  const int real_groups = (a.K + G - 1) / G;
  const int chunk = blockIdx.x % a.chunks, share = blockIdx.x / a.chunks;
  const int shares = gridDim.x / a.chunks;
  const int m0 = chunk * a.chunk_rows, rows = min(a.chunk_rows, a.M - m0);
  const int cols = rows * a.parts, stages = a.stages, stride = red_stride(a.chunk_rows);
  Frame f;
  f.ring = smem + (1024 - (tc::smem_u32(smem) & 1023)) % 1024;
  f.x = reinterpret_cast<uint4*>(f.ring + (size_t)kWarps * stages * kTile);
  f.red = reinterpret_cast<float*>(f.x + (size_t)KB * 16 * a.chunk_rows * a.parts);
  f.full = reinterpret_cast<uint64_t*>(f.red + kWarps * 16 * R * stride);
  f.factor = reinterpret_cast<float*>(f.full + kWarps * stages);
  f.power = f.factor + a.chunk_rows;
  f.stat = f.power + a.chunk_rows;
  __shared__ int abort;
  __shared__ uint64_t sums_there[kWarps / 2], sums_read[kWarps / 2];  // of a team

  const int kw = a.k_warps, wk = warp & (kw - 1), team = warp / kw;
  const int teams = shares * (kWarps / kw), first = share * (kWarps / kw) + team;
  const int units = (a.N + 16 * R - 1) / (16 * R);
  const int nk = tiles_of(KT, kw, kChunk / W);
  const int mine = first < units ? (units - first - 1) / teams + 1 : 0;
  const int my_nk = max(0, min(nk, KT - wk * nk));  // the last warps may have fewer tiles, or none
  const size_t row_groups = Kp / G;
  uint8_t* ring = f.ring + (size_t)warp * stages * kTile;
  uint64_t* full = f.full + warp * stages;

  if (lane == 0)
    for (int i = 0; i < stages; ++i) tc::mbar_init(&full[i], 1);
  if (threadIdx.x < kWarps / kw) {
    tc::mbar_init(&sums_there[threadIdx.x], kw);
    tc::mbar_init(&sums_read[threadIdx.x], kw);
  }
  if (threadIdx.x == 0) abort = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncthreads();
  grid_dep_wait();
  // the copies are of another proxy than the stores of whoever packed the matrix just now
  asm volatile("fence.proxy.async.global;" ::: "memory");

  // tiles, by the first lane: coordinates of the next one
  const uint64_t policy = tc::policy_evict_first();
  const int tiles = mine * my_nk, x_end = (wk * nk + my_nk) * kRow;
  int px = wk * nk * kRow, py = first * 16 * R, issued = 0;
  auto issue = [&](int stage) {
    const bool skip = a.stall && blockIdx.x == 0 && warp == 0 && issued == 0;
    if (issued < tiles && lane == 0 && !skip) {
      tc::mbar_arrive_expect_tx(&full[stage], kTile);
      tc::tma_load_2d(ring + stage * kTile, &codes, px, py, &full[stage], policy);
    }
    ++issued;
    px += kRow;
    if (px == x_end) {
      px = wk * nk * kRow;
      py += teams * 16 * R;
    }
  };

  // scales and zero points, four groups at a time (with the next four loaded ahead the kernels ran out
  // of registers: a row of 129280 x 4096 54 -> 57 us)
  const bool aligned = row_groups % 4 == 0 && (reinterpret_cast<uintptr_t>(a.zeros) & 3) == 0;
  const int first_group = wk * nk * W * kGroups;
  const int end_group = min((int)row_groups, first_group + my_nk * W * kGroups);
  int su = first, sg = first_group;  // of the next load
  const uint8_t *ps = nullptr, *pz = nullptr;
  auto start_unit = [&]() {
    const size_t at = (size_t)(su * 16 * R + g) * row_groups + first_group;
    ps = static_cast<const uint8_t*>(a.scales) + at * kSize;
    if (ZEROS) pz = a.zeros + at;
  };
  auto load_side = [&](SideT& to) {
    if (su >= units) return;
    const uint8_t* p = ps;
    const uint8_t* zp = pz;
    const bool whole = (su + 1) * 16 * R <= a.N;
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) {
      uint32_t(&w)[SideT::kWords] = to.s[i / 2][i % 2];
      if (whole || su * 16 * R + i * 8 + g < a.N) {
        if (aligned) {
          if constexpr (NARROW) {
            const uint2 q = *reinterpret_cast<const uint2*>(p);
            w[0] = q.x;
            w[1] = q.y;
          } else {
            const uint4 q = *reinterpret_cast<const uint4*>(p);
            w[0] = q.x;
            w[1] = q.y;
            w[2] = q.z;
            w[3] = q.w;
          }
          if constexpr (ZEROS) to.z[i / 2][i % 2] = *reinterpret_cast<const uint32_t*>(zp);
        } else {
          uint32_t z = 0;
#pragma unroll
          for (int q = 0; q < SideT::kWords; ++q) w[q] = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (sg + q >= (int)row_groups) continue;
            if constexpr (NARROW)
              w[q / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[q] << (q & 1 ? 16 : 0);
            else
              w[q] = reinterpret_cast<const uint32_t*>(p)[q];
            if (ZEROS) z |= (uint32_t)zp[q] << (8 * q);
          }
          if constexpr (ZEROS) to.z[i / 2][i % 2] = z;
        }
      }
      p += row_groups * (8 * kSize);  // eight rows on
      if (ZEROS) zp += row_groups * 8;
    }
    sg += 4;
    ps += 4 * kSize;
    if (ZEROS) pz += 4;
    if (sg >= end_group) {
      sg = first_group;
      su += teams;
      start_unit();
    }
  };
  SideT side;

  // the rows first: behind the rings' 60 to 190 KB an SM their loads would wait
  stage_rows(a, f, m0, rows, cols, share, shares, [&]() {
    if (my_nk == 0) return;
    for (int i = 0; i < stages; ++i) issue(i);
    start_unit();
    load_side(side);
  });

  float acc[R][T][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < T; ++j) acc[r][j][0] = acc[r][j][1] = acc[r][j][2] = acc[r][j][3] = 0.0f;
  int col[T];  // columns past the last one repeat it and are not used
#pragma unroll
  for (int j = 0; j < T; ++j) col[j] = min(cols - 1, j * 8 + g) * 4 + t;
  // 16-byte chunks of a tile's row are stored at chunk ^ (row / 2 % 4), or ^ (row % 8)
  const int turn = W == 1 ? (g >> 1) & 3 : g & 7;
  int stage = 0, parity = 0, ik = 0, done = 0, in_chunk = 0;
  bool ok = true;

  auto block = [&](const uint8_t* tile, int kb, int i) {
    uint32_t c[R][2][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* p = tile + (r * 16 + h * 8) * kRow;
        if constexpr (G == 128) {
          const uint4 q = *reinterpret_cast<const uint4*>(p + ((4 * i + t) ^ turn) * 16);
          c[r][h][0] = q.x;
          c[r][h][1] = q.y;
          c[r][h][2] = q.z;
          c[r][h][3] = q.w;
        } else if constexpr (G == 64) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint2 q = *reinterpret_cast<const uint2*>(
                p + ((4 * i + 2 * w + (t >> 1)) ^ turn) * 16 + (t & 1) * 8);
            c[r][h][2 * w] = q.x;
            c[r][h][2 * w + 1] = q.y;
          }
        } else {
#pragma unroll
          for (int w = 0; w < 4; ++w)
            c[r][h][w] =
                *reinterpret_cast<const uint32_t*>(p + ((4 * i + w) ^ turn) * 16 + t * 4);
        }
      }
    const uint4* xb = f.x + (size_t)kb * 16 * cols;
    float part[R][T][4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      constexpr int kPer = 4 / kGroups;  // words of a group
      uint4 b[T];
#pragma unroll
      for (int j = 0; j < T; ++j) b[j] = xb[w * cols * 4 + col[j]];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        Zero z0, z1;
        if constexpr (ZEROS) {
          z0 = Zero(side.z[r][0] >> (8 * (w / kPer)) & 127u);
          z1 = Zero(side.z[r][1] >> (8 * (w / kPer)) & 127u);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t w0 = s ? c[r][0][w] >> 8 : c[r][0][w];
          const uint32_t w1 = s ? c[r][1][w] >> 8 : c[r][1][w];
          const uint32_t q[4] = {codes_even(w0, z0), codes_even(w1, z1), codes_odd(w0, z0),
                                 codes_odd(w1, z1)};
#pragma unroll
          for (int j = 0; j < T; ++j) {
            if (s == 0 && w % kPer == 0)
              mma<true>(part[r][j], q, b[j].x, b[j].y);
            else
              mma<false>(part[r][j], q, s ? b[j].z : b[j].x, s ? b[j].w : b[j].y);
          }
        }
        if (w % kPer == kPer - 1) {
          const int n = w / kPer;
          float s0 = side.scale(r, 0, n), s1 = side.scale(r, 1, n);
          if (kGroups > 1 && kb * kGroups + n >= real_groups) s0 = s1 = 0.0f;  // of the padding
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
    side.next_block();
    // a unit may end within four groups
    if (++in_chunk == kChunk || (ik + 1 == my_nk && (i == W - 1 || kb + 1 == KB))) {
      in_chunk = 0;
      load_side(side);
    }
  };
  // A unit's sums go to the other warps that share its rows (a row's columns added first) when they
  // are done, and are added up a tile later: no warp waits for its team in between.
  int unit = first, given = 0, taken = 0;
  float* red = f.red + warp * 16 * R * stride;
  auto give = [&]() {
    if (given) tc::mbar_wait(&sums_read[team], (given - 1) & 1, &abort, a.status);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < T; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float* to = red + (r * 16 + h * 8 + g) * stride;
          const float y0 = acc[r][j][2 * h], y1 = acc[r][j][2 * h + 1];
          acc[r][j][2 * h] = acc[r][j][2 * h + 1] = 0.0f;
          if (a.parts == 2) {
            if (j * 4 + t < rows) to[j * 4 + t] = fmaf(y1, 1.0f / kRest, y0);
          } else {
            if (j * 8 + t * 2 < rows) to[j * 8 + t * 2] = y0;
            if (j * 8 + t * 2 + 1 < rows) to[j * 8 + t * 2 + 1] = y1;
          }
        }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sums_there[team]);
    ++given;
  };
  auto take = [&]() {
    tc::mbar_wait(&sums_there[team], taken & 1, &abort, a.status);
    const float* from = f.red + team * kw * 16 * R * stride;
    for (int e = wk * 32 + lane; e < rows * 16 * R; e += 32 * kw) {
      const int m = e / (16 * R), r = e % (16 * R), n = unit * 16 * R + r;
      if (n >= a.N) continue;
      float y = 0.0f;
      for (int w = 0; w < kw; ++w) y += from[(w * 16 * R + r) * stride + m];
      y = y * f.factor[m] * f.power[m];
      const size_t to = (size_t)(m0 + m) * a.ldo + n;
      if (a.out_dtype == SPEC_BF16)
        static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16_rn(y);
      else
        static_cast<float*>(a.out)[to] = y;
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sums_read[team]);
    ++taken;
    unit += teams;
  };

  if (my_nk == 0) {
    for (int i = 0; i < mine; ++i) {
      give();
      take();
    }
    return;
  }
  for (int it = 0; it < tiles; ++it) {
    if (ok && !tc::mbar_wait(&full[stage], parity, &abort, a.status)) {
      // copies in flight land before the CTA's memory is another's; from here on the warp goes on
      // without waiting or copying
      ok = false;
      const int in_flight = min(issued, tiles) - done;
      for (int i = 0; i < in_flight; ++i) {
        const int at = stage + i < stages ? stage + i : stage + i - stages;
        tc::mbar_drain(&full[at], stage + i < stages ? parity : parity ^ 1);
      }
    }
    ++done;
    const uint8_t* tile = ring + stage * kTile + g * kRow;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int kb = (wk * nk + ik) * W + i;
      if (i == 0 || kb < KB) block(tile, kb, i);
    }
    __syncwarp();  // every lane has read the tile
    if (ok) issue(stage);
    if (++stage == stages) {
      stage = 0;
      parity ^= 1;
    }
    if (taken < given) take();
    if (++ik == my_nk) {
      ik = 0;
      give();
    }
  }
  if (taken < given) take();
}

template <int G, int R, int T, int W, bool ZEROS, bool NARROW>
cudaError_t launch_t(W4Args a, const CUtensorMap& codes, cudaStream_t s) {
  const int units = (a.N + 16 * R - 1) / (16 * R), teams = kWarps / a.k_warps;
  const size_t rest = rest_bytes(a.K, a.chunk_rows, a.parts, R), kStage = stage_bytes(R, W);
  a.stages = 4;
  while (a.stages > 2 && rest + a.stages * kStage > kSmemMost) --a.stages;
  const size_t smem = rest + a.stages * kStage;
  auto k = product_kernel<G, R, T, W, ZEROS, NARROW>;
  // the same for every call: another thread's may come between this and the launch
  const cudaError_t e =
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMost);
  if (e != cudaSuccess) return e;
  int shares = num_sms() / a.chunks;
  const int most = (units + teams - 1) / teams;
  shares = shares < 1 ? 1 : shares < most ? shares : most;
  return launch_kernel(k, dim3((unsigned)(shares * a.chunks)), dim3(kThreads), smem, s, true, a,
                       codes);
}

template <int G, int R, int T, int W>
cudaError_t launch_form(const W4Args& a, const CUtensorMap& codes, cudaStream_t s) {
  const bool narrow = a.scale_dtype == SPEC_BF16;
  if (a.zeros)
    return narrow ? launch_t<G, R, T, W, true, true>(a, codes, s)
                  : launch_t<G, R, T, W, true, false>(a, codes, s);
  return narrow ? launch_t<G, R, T, W, false, true>(a, codes, s)
                : launch_t<G, R, T, W, false, false>(a, codes, s);
}

template <int G>
cudaError_t launch_group(const W4Args& a, const CUtensorMap& codes, Form form, cudaStream_t s) {
  if (form.R == 2)
    return form.T == 1 ? form.W == 2 ? launch_form<G, 2, 1, 2>(a, codes, s)
                                     : launch_form<G, 2, 1, 1>(a, codes, s)
                       : launch_form<G, 2, 2, 1>(a, codes, s);
  return form.T == 1   ? launch_form<G, 1, 1, 1>(a, codes, s)
         : form.T == 2 ? launch_form<G, 1, 2, 1>(a, codes, s)
         : form.T == 3 ? launch_form<G, 1, 3, 1>(a, codes, s)
                       : launch_form<G, 1, 5, 1>(a, codes, s);
}

}  // namespace
}  // namespace w4
}  // namespace spec
