// mx_logits.cu -- logits of block-scaled hidden rows against a block-scaled vocabulary matrix.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"

namespace spec {
namespace mx {
namespace {

constexpr int kTile = 32;  // rows of each operand a block takes

template <int FMT>
__device__ __forceinline__ float value(const uint8_t* codes, const uint8_t* scales, int row, int k,
                                       int G) {
  const size_t at = (size_t)row * G * kGroup + k;
  const float s = scale_value(__ldg(scales + scale_word(row, k / kGroup, G) + (k / kBlock & 3)));
  if constexpr (FMT == SPEC_MX_E2M1)
    return from_e2m1(__ldg(codes + at / 2) >> (4 * (k & 1))) * s;
  else
    return from_e4m3(__ldg(codes + at)) * s;
}

// A 32 x 32 tile of the output, 16 x 16 threads with four sums each, 32 elements of K at a time.
template <int AF, int WF>
__global__ void __launch_bounds__(256) logits_kernel(const uint8_t* ac, const uint8_t* as,
                                                     const uint8_t* wc, const uint8_t* wsc, int M,
                                                     int V, int K, void* out, int odt,
                                                     long long ldo) {
  __shared__ float sa[kTile][kTile + 1], sw[kTile][kTile + 1];
  const int G = groups(K), Kp = G * kGroup;
  const int v0 = blockIdx.x * kTile, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int m0 = blockIdx.y * kTile; m0 < M; m0 += gridDim.y * kTile) {
    float acc[2][2] = {};
    for (int k0 = 0; k0 < Kp; k0 += kTile) {
      __syncthreads();
      for (int e = threadIdx.x; e < kTile * kTile; e += 256) {
        const int r = e / kTile, k = k0 + e % kTile;
        sa[r][e % kTile] = m0 + r < M ? value<AF>(ac, as, m0 + r, k, G) : 0.0f;
        sw[r][e % kTile] = v0 + r < V ? value<WF>(wc, wsc, v0 + r, k, G) : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kTile; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = fmaf(sa[ty + 16 * i][k], sw[tx + 16 * j][k], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int m = m0 + ty + 16 * i, v = v0 + tx + 16 * j;
        if (m >= M || v >= V) continue;
        if (odt == SPEC_BF16) {
          uint16_t b;
          asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(acc[i][j]));
          reinterpret_cast<uint16_t*>(out)[(size_t)m * ldo + v] = b;
        } else {
          reinterpret_cast<float*>(out)[(size_t)m * ldo + v] = acc[i][j];
        }
      }
  }
}

}  // namespace
}  // namespace mx

cudaError_t launch_mx_logits(const uint8_t* ac, const uint8_t* as, int af, const uint8_t* wc,
                             const uint8_t* wsc, int wf, int M, int V, int K, void* out, int odt,
                             long long ldo, uint32_t* status, cudaStream_t s) {
  using namespace mx;
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  const int my = (M + kTile - 1) / kTile;
  const dim3 grid((V + kTile - 1) / kTile, my < 65535 ? my : 65535);
  auto k = af == SPEC_MX_E2M1 ? (wf == SPEC_MX_E2M1 ? logits_kernel<SPEC_MX_E2M1, SPEC_MX_E2M1>
                                                    : logits_kernel<SPEC_MX_E2M1, SPEC_MX_E4M3>)
                              : (wf == SPEC_MX_E2M1 ? logits_kernel<SPEC_MX_E4M3, SPEC_MX_E2M1>
                                                    : logits_kernel<SPEC_MX_E4M3, SPEC_MX_E4M3>);
  k<<<grid, 256, 0, s>>>(ac, as, wc, wsc, M, V, K, out, odt, ldo);
  return cudaGetLastError();
}

}  // namespace spec
