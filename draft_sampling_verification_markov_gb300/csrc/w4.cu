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
// loads are in flight and a row's address is found once for 32 elements of a lane.
constexpr int kPieces = 4;

// Eight elements as they are loaded, G / 8 lanes a group. The scale is the least s of its type with
// 7 s >= the group's largest magnitude: a seventh of that, cut, is within a step of it, and 7 s
// against the magnitude is exact in one fused operation. A code is w / s rounded to the
// nearest, ties to even. w (1 / s) + 1.5 * 2^23 + 8, rounded once, has it in its last bits unless w / s
// is within 2^-19 of the middle between two codes (1 / s is off by 2^-23); then w - code * s, which is
// exact, decides.
__device__ __forceinline__ uint32_t pack8(const float (&v)[8], int G, int sdt, float& s, bool& bad) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max_nan(a, fabsf(v[i]));
  for (int o = 1; o < G / 8; o *= 2) a = max_nan(a, __shfl_xor_sync(kFull, a, o));
  bad = !(a < INFINITY);
  const uint32_t step = sdt == SPEC_BF16 ? 0x10000u : 1u;
  uint32_t b = __float_as_uint(a * (1.0f / 7.0f)) & ~(step - 1u);
  if (b && fmaf(7.0f, __uint_as_float(b - step), -a) >= 0.0f) b -= step;
  if (fmaf(7.0f, __uint_as_float(b), -a) < 0.0f) b += step;
  if (fmaf(7.0f, __uint_as_float(b), -a) < 0.0f) b += step;  // a subnormal quotient
  s = bad ? NAN : __uint_as_float(b);
  if (!(s > 0.0f)) return 0x88888888u;  // zeros, and what has no scale
  uint32_t w = 0;
  if (s > 0x1p-100f) {  // 1 / s is finite and normal
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    const float half = 0.5f * s, near = 0.499997f * s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = fmaf(v[i], r, 12582920.0f), c = t - 12582920.0f;
      const float e = fmaf(-c, s, v[i]);
      uint32_t q = __float_as_uint(t) & 15u;
      // one element in a hundred of bf16 matrices: a branch for each took 656 us for 129280 x 4096,
      // one for a lane's eight 1039, none 717
      if (fabsf(e) > near && (fabsf(e) > half || (fabsf(e) == half && (q & 1u))))
        q += e > 0.0f ? 1u : ~0u;
      w |= q << (4 * i);
    }
    return w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w |= (uint32_t)(((int)rintf(__fdiv_rn(v[i], s)) + 8) & 15) << (4 * i);
  return w;
}

template <int DT>
__global__ void __launch_bounds__(kPackThreads)
    pack_kernel(const void* x, long long ldx, int rows, int K, int G, uint8_t* codes, void* scales,
                int sdt, uint32_t* status) {
  grid_dep_wait();
  const int Kp = padded(K), per_row = (Kp + 1023) / 1024, lane = threadIdx.x & 31;
  const long long all = (long long)rows * per_row, step = (long long)gridDim.x * kPackWarps;
  for (long long at = (long long)blockIdx.x * kPackWarps + (threadIdx.x >> 5); at < all; at += step) {
    const int row = (int)(at / per_row), k0 = (int)(at - (long long)row * per_row) * 1024 + lane * 8;
    float v[kPieces][8];
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      load8(x, DT, (size_t)row * ldx, k0 + i * 256, K, v[i]);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int k = k0 + i * 256;
      if (k - lane * 8 >= Kp) break;  // the warp's last pieces are behind the row
      float s;
      bool bad;
      const uint32_t w = pack8(v[i], G, sdt, s, bad);
      if (k >= Kp) continue;  // shuffles stay within groups, which end with the row
      *reinterpret_cast<uint32_t*>(codes + ((size_t)row * Kp + k) / 2) = w;
      if ((k & (G - 1)) == 0) {
        const size_t g = (size_t)row * (Kp / G) + k / G;
        if (sdt == SPEC_BF16)
          static_cast<uint16_t*>(scales)[g] =
              bad ? 0x7fffu : (uint16_t)(__float_as_uint(s) >> 16);
        else
          static_cast<float*>(scales)[g] = s;
        if (bad) atomicOr(status, SPEC_DEV_NONFINITE);
      }
    }
  }
}

// The codes of a word as numbers, less the zero point.
template <int DT>
__global__ void __launch_bounds__(kPackThreads)
    unpack_kernel(const uint8_t* codes, const void* scales, int sdt, const uint8_t* zeros, int rows,
                  int K, int G, void* out, long long ldo) {
  grid_dep_wait();
  const int Kp = padded(K), per_row = (Kp + 1023) / 1024, lane = threadIdx.x & 31;
  const long long all = (long long)rows * per_row, step = (long long)gridDim.x * kPackWarps;
  for (long long at = (long long)blockIdx.x * kPackWarps + (threadIdx.x >> 5); at < all; at += step) {
    const int row = (int)(at / per_row), k0 = (int)(at - (long long)row * per_row) * 1024 + lane * 8;
    uint32_t w[kPieces];
    float s[kPieces];
    int z[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int k = k0 + i * 256;
      w[i] = 0;
      s[i] = 0.0f;
      z[i] = 8;
      if (k >= K) continue;
      const size_t g = (size_t)row * (Kp / G) + k / G;
      w[i] = *reinterpret_cast<const uint32_t*>(codes + ((size_t)row * Kp + k) / 2);
      s[i] = load_scale(scales, sdt, g);
      if (zeros) z[i] = zeros[g] & 127;
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int k = k0 + i * 256;
      if (k >= K) break;
      const float base = 8388608.0f + (float)z[i];
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float c = __uint_as_float(0x4b000000u | (w[i] >> (4 * q) & 15u)) - base;
        v[q] = __fmul_rn(c, s[i]);
        if (DT == SPEC_BF16 && sdt == SPEC_F32) {
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
      store8(out, DT, (size_t)row * ldo, k, K, v);
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
  // of 129280 x 4096 61 -> 57 us).
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
  if (tc::encode_fn()(&codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.codes), dims,
                      &stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, form.W == 1 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return a.group == 128  ? launch_g128(a, codes, form, s)
         : a.group == 64 ? launch_g64(a, codes, form, s)
                         : launch_g32(a, codes, form, s);
}

// CTAs for `rows` rows of K.
static dim3 pack_grid(int rows, int K) {
  const long long warps = (long long)rows * ((w4::padded(K) + 1023) / 1024);
  const long long n = (warps + w4::kPackWarps - 1) / w4::kPackWarps, most = num_sms() * 8;
  return dim3((unsigned)(n < most ? n : most));
}

void launch_w4_quantize(const void* x, int dt, long long ldx, int rows, int K, int group,
                        uint8_t* codes, void* scales, int sdt, uint32_t* status, cudaStream_t s) {
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  launch_kernel(dt == SPEC_BF16 ? w4::pack_kernel<SPEC_BF16> : w4::pack_kernel<SPEC_F32>,
                pack_grid(rows, K), dim3(w4::kPackThreads), 0, s, true, x, ldx, rows, K, group, codes,
                scales, sdt, status);
}

void launch_w4_dequantize(const uint8_t* codes, const void* scales, int sdt, const uint8_t* zeros,
                          int rows, int K, int group, void* out, int odt, long long ldo,
                          cudaStream_t s) {
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  launch_kernel(odt == SPEC_BF16 ? w4::unpack_kernel<SPEC_BF16> : w4::unpack_kernel<SPEC_F32>,
                pack_grid(rows, K), dim3(w4::kPackThreads), 0, s, true, codes, scales, sdt, zeros,
                rows, K, group, out, ldo);
}

}  // namespace spec
