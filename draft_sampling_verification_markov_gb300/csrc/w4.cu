// w4.cu -- matrices of 4-bit weights with a scale per group: packing, reading back, and the choice of
// a product's form (w4_product.cuh).
#include "w4.cuh"

namespace spec {
namespace w4 {
namespace {

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
  // for everyone. The one with the fewest blocks behind one another, each new unit counted as one
  // more for its sums. Two blocks a tile, where both fit three times, halve the rest of its cost.
  auto fits = [&](int r, int w, int stages) {
    return rest_bytes(a.K, a.chunk_rows, a.parts, T) + stages * stage_bytes(r, w) <= kSmemMost;
  };
  const int sms = num_sms() / a.chunks > 0 ? num_sms() / a.chunks : 1;
  long long best = 1LL << 60;
  Form form{1, T, 1};
  for (int r = T <= 2 && fits(2, 1, 2) ? 2 : 1; r >= 1; --r) {
    const int wide = r == 2 && T == 1 && KB > 1 && fits(r, 2, 3) ? 2 : 1;
    const int tiles = (KB + wide - 1) / wide;
    for (int kw = 2; kw <= kWarps; kw *= 2) {
      const long long units = (a.N + 16 * r - 1) / (16 * r), teams = (long long)sms * (kWarps / kw);
      const long long cost = ((units + teams - 1) / teams) * ((tiles + kw - 1) / kw * r * wide + 1);
      if (cost < best) {
        best = cost;
        a.k_warps = kw;
        form = Form{r, T, wide};
      }
    }
  }
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
