// w4.cu -- matrices of 4-bit weights with a scale per group: packing, reading back, and the choice of
// a product's form (w4_product.cuh).
#include "w4.cuh"

namespace spec {
namespace w4 {
namespace {

// ------------------------------------------------------------------------------ packing

constexpr int kPackThreads = 256;
constexpr int kPackWarps = kPackThreads / 32;

// A warp takes 1024 consecutive elements of a row at a time, a lane eight of each 256, so that four
// loads are in flight and a row's address is found once for 32 elements of a lane. Groups are powers
// of two: their numbers are shifts (`by`), and the walk over rows and spans has no division.
constexpr int kPieces = 4;
struct Span {
  int row, at, per_row, rows, row_step, at_step;
  __device__ __forceinline__ Span(int rows_, int K) : rows(rows_) {
    per_row = (padded(K) + 1023) / 1024;
    const int first = (int)blockIdx.x * kPackWarps + (int)(threadIdx.x >> 5);
    const int step = (int)gridDim.x * kPackWarps;
    row = first / per_row;
    at = first - row * per_row;
    row_step = step / per_row;
    at_step = step - row_step * per_row;
  }
  __device__ __forceinline__ bool more() const { return row < rows; }
  __device__ __forceinline__ int k0() const { return at * 1024 + (int)(threadIdx.x & 31) * 8; }
  __device__ __forceinline__ void next() {
    at += at_step;
    row += row_step;
    if (at >= per_row) {
      at -= per_row;
      ++row;
    }
  }
};

// The least s of the scales' type with 7 s >= a; 7 s against a is exact in one fused operation. For
// bf16 a seventh of a, rounded up twice, is at most 2^-22 too large, which moves it past one number at
// most; for fp32 a seventh, rounded, is within a step.
template <int SDT>
__device__ __forceinline__ float least_scale(float a) {
  constexpr uint32_t step = SDT == SPEC_BF16 ? 0x10000u : 1u;
  if constexpr (SDT == SPEC_BF16) {
    constexpr float kSeventh = 0x1.24924ap-3f;  // above 1 / 7
    const uint32_t b = (__float_as_uint(__fmul_ru(a, kSeventh)) + 0xffffu) & 0xffff0000u;
    const float less = __uint_as_float(b - step);  // NaN if b is 0
    return fmaf(7.0f, less, -a) >= 0.0f ? less : __uint_as_float(b);
  }
  uint32_t b = __float_as_uint(a * (1.0f / 7.0f));
  if (b && fmaf(7.0f, __uint_as_float(b - step), -a) >= 0.0f) b -= step;
  if (fmaf(7.0f, __uint_as_float(b), -a) < 0.0f) b += step;
  if (fmaf(7.0f, __uint_as_float(b), -a) < 0.0f) b += step;  // a subnormal quotient
  return __uint_as_float(b);
}

// 1 / s to 2^-23, for s above 2^-100 only.
__device__ __forceinline__ float about_inverse(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// Eight elements' codes: w / s rounded to the nearest, ties to even, plus 8. w (1 / s) + 1.5 * 2^23 + 8,
// rounded once, has it in its last bits unless w / s is within 2^-19 of the middle between two codes
// (1 / s is off by 2^-23); then w - code * s, which is exact, decides.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float s) {
  if (!(s > 0.0f)) return 0x88888888u;  // zeros, and what has no scale
  uint32_t w = 0;
  if (s > 0x1p-100f) {
    const float r = about_inverse(s), half = 0.5f * s, near = 0.499997f * s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = fmaf(v[i], r, 12582920.0f), c = t - 12582920.0f;
      const float e = fmaf(-c, s, v[i]);
      uint32_t q = __float_as_uint(t) & 15u;
      if (fabsf(e) > near && (fabsf(e) > half || (fabsf(e) == half && (q & 1u))))
        q += e > 0.0f ? 1u : ~0u;
      w |= q << (4 * i);
    }
    return w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // a quotient may be rounded to the middle: here, too, the remainder decides
    const float c = rintf(__fdiv_rn(v[i], s)), e = 2.0f * fmaf(-c, s, v[i]);
    int q = (int)c + 8;
    if (fabsf(e) > s || (fabsf(e) == s && (q & 1))) q += e > 0.0f ? 1 : -1;
    w |= (uint32_t)(q & 15) << (4 * i);
  }
  return w;
}

// The same where elements and scales are bf16, s > 2^-100. With w = W 2^b and s = S 2^a, 128 <= S, W <
// 256, w / s is the middle between two codes or at least 2^-9 from it: |2 w - (2 c + 1) s| is a
// multiple of 2^a where w >= 128 * 2^(a - 1), and below that w is at most 255 * 2^(a - 2), which is
// s / 2 less s / 512 or more. So w (1 / s) to the nearest multiple of 2^-10 (ulp of 1.5 * 2^13) is on
// the right side, a middle among them exactly, and one more addition rounds it to even: three
// instructions an element, 1.5 * 2^23 + 8 + c times 16^i summed into the word. (With the remainder as
// above, one element in a hundred had to branch: 129280 x 4096 took 656 us, 1039 with a branch for
// eight, 717 without one.)
__device__ __forceinline__ uint32_t codes8_bf16(const uint32_t (&v)[4], float s) {
  const float r = about_inverse(s);
  uint32_t w = 0, m = 1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
    const float t = __fadd_rn(fmaf(x, r, 12288.0f), 12582920.0f - 12288.0f);
    w += __float_as_uint(t) * m;
    m *= 16;
  }
  return w - 0x4b400000u * 0x11111111u;
}

template <int DT, int SDT>
__global__ void __launch_bounds__(kPackThreads)
    pack_kernel(const void* x, long long ldx, int rows, int K, int by, uint8_t* codes, void* scales,
                uint32_t* status) {
  grid_dep_wait();
  const int Kp = padded(K), G = 1 << by, lane = threadIdx.x & 31;
  for (Span at(rows, K); at.more(); at.next()) {
    const int row = at.row, k0 = at.k0();
    const size_t xr = (size_t)row * ldx;
    float v[DT == SPEC_BF16 ? 1 : kPieces][8], a[kPieces];
    uint32_t u[DT == SPEC_BF16 ? kPieces : 1][4];
    if constexpr (DT == SPEC_BF16) {
      const uint16_t* px = static_cast<const uint16_t*>(x) + xr + k0;
      uint4 q[kPieces];
      if (k0 + (kPieces - 1) * 256 + 8 <= K && (reinterpret_cast<uintptr_t>(px) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) q[i] = ld_coherent16(px + i * 256);
      } else {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) q[i] = load8_bf16(x, xr, k0 + i * 256, K);
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        u[i][0] = q[i].x;
        u[i][1] = q[i].y;
        u[i][2] = q[i].z;
        u[i][3] = q[i].w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) load8(x, DT, xr, k0 + i * 256, K, v[i]);
    }
    // the groups' largest magnitudes, NaN if there is one
    if constexpr (DT == SPEC_BF16) {
#pragma unroll
      for (int i = 0; i < kPieces; i += 2) {
        __nv_bfloat162 m[2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
          m[q] = __hmax2_nan(
              __hmax2_nan(__habs2(as_bf2(u[i + q][0])), __habs2(as_bf2(u[i + q][1]))),
              __hmax2_nan(__habs2(as_bf2(u[i + q][2])), __habs2(as_bf2(u[i + q][3]))));
        // two groups' in one word
        __nv_bfloat162 both = __hmax2_nan(as_bf2(__byte_perm(as_word(m[0]), as_word(m[1]), 0x5410)),
                                          as_bf2(__byte_perm(as_word(m[0]), as_word(m[1]), 0x7632)));
        for (int o = 1; o < G / 8; o *= 2)
          both = __hmax2_nan(both, as_bf2(__shfl_xor_sync(kFull, as_word(both), o)));
        a[i] = __uint_as_float(as_word(both) << 16);
        a[i + 1] = __uint_as_float(as_word(both) & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        a[i] = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) a[i] = max_nan(a[i], fabsf(v[i][q]));
        for (int o = 1; o < G / 8; o *= 2) a[i] = max_nan(a[i], __shfl_xor_sync(kFull, a[i], o));
      }
    }
    uint32_t* words = reinterpret_cast<uint32_t*>(codes) + ((size_t)row * Kp + k0) / 8;
    const size_t first = (size_t)row * (Kp >> by) + (k0 >> by);
    const bool leads = (k0 & (G - 1)) == 0;  // its group, in every piece
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if (k0 + i * 256 >= Kp) break;
      const bool bad = !(a[i] < INFINITY);
      const float s = bad ? NAN : least_scale<SDT>(a[i]);
      uint32_t w;
      if constexpr (DT == SPEC_BF16) {
        if (SDT == SPEC_BF16 && s > 0x1p-100f) {
          w = codes8_bf16(u[i], s);
        } else {
          float f[8];
#pragma unroll
          for (int q = 0; q < 8; ++q)
            f[q] = __uint_as_float(q & 1 ? u[i][q / 2] & 0xffff0000u : u[i][q / 2] << 16);
          w = codes8(f, s);
        }
      } else {
        w = codes8(v[i], s);
      }
      words[i * 32] = w;
      if (leads) {
        const size_t g = first + (i * 256 >> by);
        if constexpr (SDT == SPEC_BF16)
          static_cast<uint16_t*>(scales)[g] = bad ? 0x7fffu : (uint16_t)(__float_as_uint(s) >> 16);
        else
          static_cast<float*>(scales)[g] = s;
        if (bad) atomicOr(status, SPEC_DEV_NONFINITE);
      }
    }
  }
}

// The codes of a word as numbers, less the zero point, times the scale. A lane writes 16 bytes at a
// time, eight bf16 or four fp32 elements. With bf16 on both sides two at a time: 128 + code and 128 +
// zero point are bf16, so is their difference, and its product with the scale is rounded once.
template <int DT, int SDT>
__global__ void __launch_bounds__(kPackThreads)
    unpack_kernel(const uint8_t* codes, const void* scales, const uint8_t* zeros, int rows, int K,
                  int by, void* out, long long ldo) {
  grid_dep_wait();
  constexpr int N = DT == SPEC_BF16 ? 8 : 4, kTakes = 32 / N;
  const int Kp = padded(K), lane = threadIdx.x & 31;
  for (Span at(rows, K); at.more(); at.next()) {
    const int row = at.row, k0 = at.at * 1024 + lane * N;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(codes) + (size_t)row * Kp / 8;
    const size_t groups = (size_t)row * (Kp >> by);
    uint32_t w[kTakes];
    float s[kTakes];
    int z[kTakes];
#pragma unroll
    for (int i = 0; i < kTakes; ++i) {
      const int k = k0 + i * 32 * N;
      w[i] = 0;
      s[i] = 0.0f;
      z[i] = 8;
      if (k >= K) continue;
      const size_t g = groups + (k >> by);
      w[i] = words[k / 8];
      s[i] = load_scale(scales, SDT, g);
      if (zeros) z[i] = zeros[g] & 127;
    }
#pragma unroll
    for (int i = 0; i < kTakes; ++i) {
      const int k = k0 + i * 32 * N;
      if (k >= K) break;
      if constexpr (DT == SPEC_BF16 && SDT == SPEC_BF16) {
        const __nv_bfloat162 base = as_bf2((0x4300u | z[i]) * 0x10001u),
                             scale = as_bf2((__float_as_uint(s[i]) >> 16) * 0x10001u);
        uint32_t p[4];  // elements q and q + 4
#pragma unroll
        for (int q = 0; q < 4; ++q)
          p[q] = as_word(__hmul2_rn(
              __hsub2_rn(as_bf2((w[i] >> (4 * q) & 0x000f000fu) | 0x43004300u), base), scale));
        const uint32_t o[4] = {__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                               __byte_perm(p[0], p[1], 0x7632), __byte_perm(p[2], p[3], 0x7632)};
        store8_bf16(out, (size_t)row * ldo, k, K, o);
      } else {
        const float base = 8388608.0f + (float)z[i];
        const uint32_t own = N == 4 ? w[i] >> (lane & 1) * 16 : w[i];
        float v[N];
#pragma unroll
        for (int q = 0; q < N; ++q) {
          const float c = __uint_as_float(0x4b000000u | (own >> (4 * q) & 15u)) - base;
          v[q] = __fmul_rn(c, s[i]);
          if constexpr (DT == SPEC_BF16) {
            // towards the odd neighbour where fp32 does not hold the product, so that bf16 rounds it
            // once
            const float rest = fmaf(c, s[i], -v[q]);
            uint32_t b = __float_as_uint(v[q]);
            if (rest != 0.0f) {
              if ((rest < 0.0f) != (v[q] < 0.0f)) --b;
              v[q] = __uint_as_float(b | 1u);
            }
          }
        }
        if constexpr (DT == SPEC_BF16)
          store8(out, DT, (size_t)row * ldo, k, K, v);
        else
          store4(static_cast<float*>(out) + (size_t)row * ldo + k, K - k, v);
      }
    }
  }
}

}  // namespace
}  // namespace w4

static size_t row_bytes(int parts, int K) { return (size_t)w4::padded(K) * 2 * parts; }

bool w4_fits(int parts, int K) { return row_bytes(parts, K) <= w4::kRowsMost; }

cudaError_t launch_w4_logits(W4Args a, cudaStream_t s) {
  using namespace w4;
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  const int KB = padded(a.K) / kBlock;
  const int most = (int)(kRowsMost / row_bytes(a.parts, a.K));
  a.chunk_rows = kColumns / a.parts;
  if (a.chunk_rows > most) a.chunk_rows = most;
  a.chunks = (a.M + a.chunk_rows - 1) / a.chunk_rows;
  a.chunk_rows = (a.M + a.chunks - 1) / a.chunks;
  const int cols = a.chunk_rows * a.parts, T = cols <= 8 ? 1 : cols <= 16 ? 2 : cols <= 24 ? 3 : 5;
  // Tiles of 32 rows halve what a warp reads of the columns, more warps on a tile leave more tiles
  // for everyone: the form with the fewest blocks behind one another, each new unit counted as one
  // more for its sums. Two blocks a tile, where two such tiles fit a ring, save a little more (a row
  // of 129280 x 4096 took 57 us instead of 61 when this was chosen; it takes 53).
  auto fits = [&](int r, int w) {
    return rest_bytes(a.K, a.chunk_rows, a.parts, r) + 2 * stage_bytes(r, w) <= kSmemMost;
  };
  const int sms = num_sms() / a.chunks > 0 ? num_sms() / a.chunks : 1;
  const int chunk = a.group / 32;  // blocks of four groups
  long long best = 1LL << 60;
  Form form{1, T, 1};
  for (int r = T <= 2 && fits(2, 1) ? 2 : 1; r >= 1; --r) {
    const int wide = r == 2 && T == 1 && KB > 1 && fits(r, 2) ? 2 : 1;
    const int tiles = (KB + wide - 1) / wide;
    for (int kw = 2; kw <= kWarps; kw *= 2) {
      const long long units = (a.N + 16 * r - 1) / (16 * r), teams = (long long)sms * (kWarps / kw);
      const long long cost = ((units + teams - 1) / teams) *
                             (tiles_of(tiles, kw, chunk / wide) * r * wide + 1);
      if (cost < best) {
        best = cost;
        a.k_warps = kw;
        form = Form{r, T, wide};
      }
    }
  }
  a.stall = take_stall_request();
  CUtensorMap codes;
  if (!tc::encode_fn()) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)padded(a.K) / 2, (cuuint64_t)a.N}, stride = dims[0];
  const cuuint32_t box[2] = {64u * form.W, 16u * form.R}, one[2] = {1, 1};
  const CUtensorMapSwizzle swizzle =
      form.W == 1 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (tc::encode_fn()(&codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.codes), dims,
                      &stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return a.group == 128  ? launch_g128(a, codes, form, s)
         : a.group == 64 ? launch_g64(a, codes, form, s)
                         : launch_g32(a, codes, form, s);
}

// CTAs for `rows` rows of K: four times what is resident, so that they drift apart between reading and
// writing (129280 x 4096 bf16 packed in 249 us, 244 since, and read back in 202; with once 267 and
// 243, with one span a warp 273 and 208).
static dim3 pack_grid(int rows, int K) {
  const long long warps = (long long)rows * ((w4::padded(K) + 1023) / 1024);
  const long long n = (warps + w4::kPackWarps - 1) / w4::kPackWarps, most = num_sms() * 32;
  return dim3((unsigned)(n < most ? n : most));
}

static int log2_of(int group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }

template <int DT, int SDT>
static void launch_pack(const void* x, long long ldx, int rows, int K, int group, uint8_t* codes,
                        void* scales, uint32_t* status, cudaStream_t s) {
  launch_kernel(w4::pack_kernel<DT, SDT>, pack_grid(rows, K), dim3(w4::kPackThreads), 0, s, true, x,
                ldx, rows, K, log2_of(group), codes, scales, status);
}

void launch_w4_quantize(const void* x, int dt, long long ldx, int rows, int K, int group,
                        uint8_t* codes, void* scales, int sdt, uint32_t* status, cudaStream_t s) {
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  const bool sb = sdt == SPEC_BF16;
  if (dt == SPEC_BF16)
    (sb ? launch_pack<SPEC_BF16, SPEC_BF16> : launch_pack<SPEC_BF16, SPEC_F32>)(
        x, ldx, rows, K, group, codes, scales, status, s);
  else
    (sb ? launch_pack<SPEC_F32, SPEC_BF16> : launch_pack<SPEC_F32, SPEC_F32>)(
        x, ldx, rows, K, group, codes, scales, status, s);
}

template <int DT, int SDT>
static void launch_unpack(const uint8_t* codes, const void* scales, const uint8_t* zeros, int rows,
                          int K, int group, void* out, long long ldo, cudaStream_t s) {
  launch_kernel(w4::unpack_kernel<DT, SDT>, pack_grid(rows, K), dim3(w4::kPackThreads), 0, s, true,
                codes, scales, zeros, rows, K, log2_of(group), out, ldo);
}

void launch_w4_dequantize(const uint8_t* codes, const void* scales, int sdt, const uint8_t* zeros,
                          int rows, int K, int group, void* out, int odt, long long ldo,
                          cudaStream_t s) {
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  const bool sb = sdt == SPEC_BF16;
  if (odt == SPEC_BF16)
    (sb ? launch_unpack<SPEC_BF16, SPEC_BF16> : launch_unpack<SPEC_BF16, SPEC_F32>)(
        codes, scales, zeros, rows, K, group, out, ldo, s);
  else
    (sb ? launch_unpack<SPEC_F32, SPEC_BF16> : launch_unpack<SPEC_F32, SPEC_F32>)(
        codes, scales, zeros, rows, K, group, out, ldo, s);
}

}  // namespace spec
