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
// sum. Four warps that share a tile's rows, each a quarter of K, add their sums through shared
// memory; such teams go through the matrix by themselves. tcgen05 would want the unpacked matrix in shared memory, four times the bytes, for a
// multiplication that is not the bound.
//
// Columns. A number of the rows is one or two fp16 numbers, each a column of its own: one for bf16
// rows as they are (exact), two where a bf16 norm weight is multiplied in (16 bits, exact) or for
// 32-bit numbers (off by 2^-24, as the rounding of fp32 is). Rows are scaled by powers of two into
// fp16's range; that and the norm's 1 / rms are applied to the sums.
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
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Zero points of a group as fp16 pairs: 1024 + zero, and -(64 + zero).
struct Zero {
  uint32_t a = 0x64086408u, b = 0xd480d480u;  // of 8
  __device__ __forceinline__ Zero() {}
  __device__ __forceinline__ explicit Zero(uint32_t z)
      : a(0x64006400u + z * 0x10001u), b(sub2(0x63806380u, a)) {}  // 960 - (1024 + zero)
};

// Codes s and s + 4 of a word less the zero point, for s = 0 and 1 (of the word's upper bytes: 2 and
// 3). An fp16 number from 1024 to 2047 holds a code in its last bits, or 16 times one four bits up.
__device__ __forceinline__ uint32_t codes_even(uint32_t w, const Zero& z) {
  return sub2(masked(w, 0x000f000fu), z.a);
}
__device__ __forceinline__ uint32_t codes_odd(uint32_t w, const Zero& z) {
  return fma2h(masked(w, 0x00f000f0u), 0x2c002c00u, z.b);  // / 16
}

struct Frame {
  uint8_t* ring;  // [warp][stage][16 R rows][64 bytes], 64-byte swizzled
  uint4* x;       // the rows' columns: [block][word][column][lane % 4]
  float* red;     // [warp][16 R][stride]
  float* factor;  // [rows]
  float* stat;    // [3][rows][kWarps]
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

// The chunk's rows into shared memory as fp16 columns, with the factors that their sums take; h goes
// out, a share from each CTA of the chunk. A row is scaled by powers of two so that the bound max |h|
// max |weight| of its numbers is between 2^13 and 2^15: fp16 goes down to 2^-24, 2^-37 of that.
__device__ __forceinline__ void stage_rows(const W4Args& a, const Frame& f, int m0, int rows,
                                           int cols, int share, int shares) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pieces = padded(a.K) / 8;
  const bool norm = a.weight != nullptr;
  for (int m = 0; m < rows; ++m) {
    float most = 0.0f, sum = 0.0f, gain = norm ? 0.0f : 1.0f;
    for (int p = tid; p < pieces; p += kThreads) {
      float v[8];
      load_h(a, m0 + m, p * 8, p % shares == share, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        most = max_nan(most, fabsf(v[i]));
        sum = fmaf(v[i], v[i], sum);
      }
      if (norm) {
        load8(a.weight, a.w_dtype, 0, p * 8, a.K, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) gain = max_nan(gain, fabsf(v[i]));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      most = max_nan(most, __shfl_xor_sync(kFull, most, o));
      gain = max_nan(gain, __shfl_xor_sync(kFull, gain, o));
      sum += __shfl_xor_sync(kFull, sum, o);
    }
    if (lane == 0) {
      f.stat[m * kWarps + warp] = most;
      f.stat[(rows + m) * kWarps + warp] = sum;
      f.stat[(2 * rows + m) * kWarps + warp] = gain;
    }
  }
  __syncthreads();
  for (int m = 0; m < rows; ++m) {
    float most = 0.0f, sum = 0.0f, gain = 0.0f;
    for (int w = 0; w < kWarps; ++w) {
      most = max_nan(most, f.stat[m * kWarps + w]);
      sum += f.stat[(rows + m) * kWarps + w];
      gain = max_nan(gain, f.stat[(2 * rows + m) * kWarps + w]);
    }
    if (!(most < INFINITY) && share == 0 && tid == 0) atomicOr(a.status, SPEC_DEV_NONFINITE);
    // h 2^-eh is below 2, times the weight 2^-eg below 4
    const int eh = most > 0.0f && most < INFINITY ? exponent(most) : 0;
    const int eg = gain > 0.0f && gain < INFINITY ? exponent(gain) : 0;
    if (norm && most > 0.0f && most < INFINITY && (most > 0x1p50f || most < 0x1p-40f)) {
      // squares that leave fp32's range: those of h 2^-eh
      __syncthreads();
      sum = 0.0f;
      for (int p = tid; p < pieces; p += kThreads) {
        float v[8];
        load_h(a, m0 + m, p * 8, false, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] *= power(-eh);
          sum = fmaf(v[i], v[i], sum);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      if (lane == 0) f.stat[(rows + m) * kWarps + warp] = sum;
      __syncthreads();
      sum = 0.0f;
      for (int w = 0; w < kWarps; ++w) sum += f.stat[(rows + m) * kWarps + w];
      sum /= (float)a.K;
      // beside eps in the scale in which neither passes fp32's range
      const float q = eh < 0 && a.eps > 0.0f
                          ? power(eh) / sqrtf(a.eps + sum * power(eh) * power(eh))
                          : 1.0f / sqrtf(sum + a.eps * power(-eh) * power(-eh));
      if (tid == 0) f.factor[m] = q * power(eg) * 0x1p-13f;
    } else if (tid == 0) {
      f.factor[m] = norm ? power(eh) / sqrtf(sum / (float)a.K + a.eps) * power(eg) * 0x1p-13f
                         : power(eh) * 0x1p-13f;
    }
    for (int p = tid; p < pieces; p += kThreads) {
      float v[8], g[8];
      load_h(a, m0 + m, p * 8, false, v);
      if (norm) load8(a.weight, a.w_dtype, 0, p * 8, a.K, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] *= power(-eh);
        if (norm) v[i] *= g[i] * power(-eg);
        v[i] *= 0x1p13f;
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
        __half2 c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          c[i] = __floats2half2_rn(v[i], v[i + 4]);
          const float2 back = __half22float2(c[i]);
          v[i] = __fsub_rn(v[i], back.x);
          v[i + 4] = __fsub_rn(v[i + 4], back.y);
        }
        to[(m * a.parts + q) * 4] = *reinterpret_cast<const uint4*>(c);
      }
    }
  }
  __syncthreads();
}

// Scales of the block's groups for one matrix row, as they are stored.
template <int G, bool NARROW>
struct Scales {
  static constexpr int kGroups = kBlock / G;
  static constexpr int kWords = NARROW ? (kGroups + 1) / 2 : kGroups;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (NARROW && kGroups == 1) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (kWords == 1) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kWords == 2) {
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
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (NARROW)
      return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    else
      return __uint_as_float(w[i]);
  }
};

// What a lane needs of a block beside the codes: scales and zero points of its matrix rows (16 r +
// lane / 4, and 8 below).
template <int G, int R, bool ZEROS, bool NARROW>
struct Side {
  Scales<G, NARROW> s[R][2];
  uint32_t z[ZEROS ? R : 1][2];  // a byte a group
};

// kw warps (a.k_warps) share 16 R matrix rows, each takes a range of the blocks; kWarps / kw such
// teams a CTA go through the matrix by themselves.
template <int G, int R, int T, bool ZEROS, bool NARROW>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const W4Args a, const __grid_constant__ CUtensorMap codes) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int kGroups = kBlock / G;
  constexpr int kStride = 8 * T + 1;
  constexpr int kTile = 16 * R * 64;  // bytes
  constexpr int kSize = NARROW ? 2 : 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int Kp = padded(a.K), KB = Kp / kBlock;
  const int real_groups = (a.K + G - 1) / G;
  const int chunk = blockIdx.x % a.chunks, share = blockIdx.x / a.chunks;
  const int shares = gridDim.x / a.chunks;
  const int m0 = chunk * a.chunk_rows, rows = min(a.chunk_rows, a.M - m0);
  const int cols = rows * a.parts, stages = a.stages;
  Frame f;
  f.ring = smem + (1024 - (tc::smem_u32(smem) & 1023)) % 1024;
  f.x = reinterpret_cast<uint4*>(f.ring + (size_t)kWarps * stages * kTile);
  f.red = reinterpret_cast<float*>(f.x + (size_t)KB * 16 * a.chunk_rows * a.parts);
  f.full = reinterpret_cast<uint64_t*>(f.red + kWarps * 16 * R * kStride);
  f.factor = reinterpret_cast<float*>(f.full + kWarps * stages);
  f.stat = f.factor + a.chunk_rows;
  __shared__ int abort;

  const int kw = a.k_warps, wk = warp & (kw - 1), team = warp / kw;
  const int teams = shares * (kWarps / kw), first = share * (kWarps / kw) + team;
  const int units = (a.N + 16 * R - 1) / (16 * R), nk = (KB + kw - 1) / kw;
  const int mine = first < units ? (units - first - 1) / teams + 1 : 0;
  const int my_nk = max(0, min(nk, KB - wk * nk));  // the last warps may have fewer blocks, or none
  const size_t row_groups = Kp / G;
  uint8_t* ring = f.ring + (size_t)warp * stages * kTile;
  uint64_t* full = f.full + warp * stages;

  if (lane == 0)
    for (int i = 0; i < stages; ++i) tc::mbar_init(&full[i], 1);
  if (threadIdx.x == 0) abort = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncthreads();
  grid_dep_wait();

  // tiles, by the first lane: unit and block of the next one
  const uint64_t policy = tc::policy_evict_first();
  const int tiles = mine * my_nk;
  int pu = first, pk = 0, issued = 0;
  auto issue = [&](int stage) {
    if (issued < tiles && lane == 0) {
      tc::mbar_arrive_expect_tx(&full[stage], kTile);
      tc::tma_load_2d(ring + stage * kTile, &codes, (wk * nk + pk) * 64, pu * 16 * R, &full[stage],
                      policy);
    }
    ++issued;
    if (++pk == my_nk) {
      pk = 0;
      pu += teams;
    }
  };
  if (my_nk)
    for (int i = 0; i < stages; ++i) issue(i);

  // scales and zero points, two blocks ahead
  Side<G, R, ZEROS, NARROW> side[2];
  int su = first, sk = 0;
  const uint8_t *ps = nullptr, *pz = nullptr;
  int srow = 0;
  auto load_side = [&](Side<G, R, ZEROS, NARROW>& to) {
    if (su >= units) return;
    if (sk == 0) {
      srow = su * 16 * R + g;
      const size_t at = (size_t)srow * row_groups + (size_t)wk * nk * kGroups;
      ps = static_cast<const uint8_t*>(a.scales) + at * kSize;
      if (ZEROS) pz = a.zeros + at;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int below = r * 16 + h * 8;
        if (srow + below >= a.N) continue;
        to.s[r][h].load(ps + below * (row_groups * kSize));
        if constexpr (ZEROS) {
          const uint8_t* zp = pz + below * row_groups;
          uint32_t z = zp[0];
#pragma unroll
          for (int i = 1; i < kGroups; ++i) z |= (uint32_t)zp[i] << (8 * i);
          to.z[r][h] = z;
        }
      }
    ps += kGroups * kSize;
    if (ZEROS) pz += kGroups;
    if (++sk == my_nk) {
      sk = 0;
      su += teams;
    }
  };
  if (my_nk) {
    load_side(side[0]);
    load_side(side[1]);
  }
  stage_rows(a, f, m0, rows, cols, share, shares);

  float acc[R][T][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < T; ++j) acc[r][j][0] = acc[r][j][1] = acc[r][j][2] = acc[r][j][3] = 0.0f;
  int col[T];  // columns past the last one repeat it and are not used
#pragma unroll
  for (int j = 0; j < T; ++j) col[j] = min(cols - 1, j * 8 + g) * 4 + t;
  // the lane's 16-byte chunks of matrix rows g and g + 8 (mod 16): chunk ^ (row / 2 % 4)
  const int turn = (g >> 1) & 3;
  int stage = 0, parity = 0, unit = first, ik = 0, done = 0;
  bool ok = true;

  auto block = [&](const Side<G, R, ZEROS, NARROW>& sd) {
    if (ok && !tc::mbar_wait(&full[stage], parity, &abort, a.status)) {
      // copies in flight land before the CTA's memory is another's; from here on the warp goes on
      // without waiting or copying, so that its team's barriers are met
      ok = false;
      const int in_flight = min(issued, tiles) - done;
      for (int i = 0; i < in_flight; ++i) {
        const int at = stage + i < stages ? stage + i : stage + i - stages;
        tc::mbar_drain(&full[at], stage + i < stages ? parity : parity ^ 1);
      }
    }
    ++done;
    const uint8_t* tile = ring + stage * kTile + g * 64;
    uint32_t c[R][2][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* p = tile + (r * 16 + h * 8) * 64;
        if constexpr (G == 128) {
          const uint4 q = *reinterpret_cast<const uint4*>(p + (t ^ turn) * 16);
          c[r][h][0] = q.x;
          c[r][h][1] = q.y;
          c[r][h][2] = q.z;
          c[r][h][3] = q.w;
        } else if constexpr (G == 64) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint2 q = *reinterpret_cast<const uint2*>(p + ((2 * i + (t >> 1)) ^ turn) * 16 +
                                                            (t & 1) * 8);
            c[r][h][2 * i] = q.x;
            c[r][h][2 * i + 1] = q.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            c[r][h][i] = *reinterpret_cast<const uint32_t*>(p + (i ^ turn) * 16 + t * 4);
        }
      }
    const int kb = wk * nk + ik;
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
        Zero z0, z1;
        if constexpr (ZEROS) {
          z0 = Zero(sd.z[r][0] >> (8 * (w / kPer)) & 127u);
          z1 = Zero(sd.z[r][1] >> (8 * (w / kPer)) & 127u);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t w0 = s ? c[r][0][w] >> 8 : c[r][0][w];
          const uint32_t w1 = s ? c[r][1][w] >> 8 : c[r][1][w];
          const uint32_t q[4] = {codes_even(w0, z0), codes_even(w1, z1), codes_odd(w0, z0),
                                 codes_odd(w1, z1)};
#pragma unroll
          for (int j = 0; j < T; ++j) mma(part[r][j], q, s ? b[j].z : b[j].x, s ? b[j].w : b[j].y);
        }
        if (w % kPer == kPer - 1) {
          const int i = w / kPer;
          float s0 = sd.s[r][0][i], s1 = sd.s[r][1][i];
          if (kb * kGroups + i >= real_groups) s0 = s1 = 0.0f;  // of the padding
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
    __syncwarp();  // every lane has read the tile
    if (ok) issue(stage);
    if (++stage == stages) {
      stage = 0;
      parity ^= 1;
    }
  };
  // the unit's sums, over the warps that share its rows
  auto finish = [&]() {
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
    bar_sync(1 + team, 32 * kw);
    for (int e = wk * 32 + lane; e < rows * 16 * R; e += 32 * kw) {
      const int m = e / (16 * R), r = e % (16 * R), n = unit * 16 * R + r;
      if (n >= a.N) continue;
      const float* at = f.red + (size_t)team * kw * 16 * R * kStride + r * kStride + m * a.parts;
      float y = 0.0f;
      for (int w = 0; w < kw; ++w)
        for (int q = 0; q < a.parts; ++q) y += at[w * 16 * R * kStride + q];
      y *= f.factor[m];
      const size_t to = (size_t)(m0 + m) * a.ldo + n;
      if (a.out_dtype == SPEC_BF16)
        static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16_rn(y);
      else
        static_cast<float*>(a.out)[to] = y;
    }
    bar_sync(1 + team, 32 * kw);
    unit += teams;
  };

  if (my_nk == 0) {
    for (int i = 0; i < mine; ++i) finish();
  } else {
    for (int it = 0; it < tiles; it += 2) {
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        if (it + d >= tiles) break;
        block(side[d]);
        load_side(side[d]);
        if (++ik == my_nk) {
          ik = 0;
          finish();
        }
      }
    }
  }
}

template <int G, int R, int T, bool ZEROS, bool NARROW>
cudaError_t launch_t(W4Args a, const CUtensorMap& codes, cudaStream_t s) {
  const int units = (a.N + 16 * R - 1) / (16 * R), teams = kWarps / a.k_warps;
  const size_t rest = rest_bytes(a.K, a.chunk_rows, a.parts, R, T), kStage = stage_bytes(R);
  a.stages = 4;
  while (a.stages > 2 && rest + a.stages * kStage > kSmemMost) --a.stages;
  const size_t smem = rest + a.stages * kStage;
  auto k = product_kernel<G, R, T, ZEROS, NARROW>;
  const cudaError_t e =
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  int shares = num_sms() / a.chunks;
  const int most = (units + teams - 1) / teams;
  shares = shares < 1 ? 1 : shares < most ? shares : most;
  return launch_kernel(k, dim3((unsigned)(shares * a.chunks)), dim3(kThreads), smem, s, true, a,
                       codes);
}

template <int G, int R, int T>
cudaError_t launch_form(const W4Args& a, const CUtensorMap& codes, cudaStream_t s) {
  const bool narrow = a.scale_dtype == SPEC_BF16;
  if (a.zeros)
    return narrow ? launch_t<G, R, T, true, true>(a, codes, s)
                  : launch_t<G, R, T, true, false>(a, codes, s);
  return narrow ? launch_t<G, R, T, false, true>(a, codes, s)
                : launch_t<G, R, T, false, false>(a, codes, s);
}

template <int G>
cudaError_t launch_group(const W4Args& a, const CUtensorMap& codes, int R, int T, cudaStream_t s) {
  if (R == 2)
    return T == 1 ? launch_form<G, 2, 1>(a, codes, s) : launch_form<G, 2, 2>(a, codes, s);
  return T == 1   ? launch_form<G, 1, 1>(a, codes, s)
         : T == 2 ? launch_form<G, 1, 2>(a, codes, s)
         : T == 3 ? launch_form<G, 1, 3>(a, codes, s)
                  : launch_form<G, 1, 5>(a, codes, s);
}

}  // namespace
}  // namespace w4
}  // namespace spec
