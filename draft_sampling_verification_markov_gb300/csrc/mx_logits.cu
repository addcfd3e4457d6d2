// mx_logits.cu -- logits of block-scaled hidden rows against a block-scaled vocabulary matrix on
// the tcgen05 tensor cores (kind::mxf8f6f4: products of 8- and 4-bit elements, one power-of-two
// scale per 32 of them applied by the tensor core, fp32 accumulation).
//
// out[m, v] = sum over blocks b of 2^(ea[m, b] + ew[v, b]) sum_{k in b} a[m, k] w[v, k].
//
// The vocabulary is the M side of the instruction (128 rows, always full) and the hidden rows its
// N side (16 .. 192 of them), so that one request costs no more tensor-core rows than it must and
// the vocabulary matrix, which is the traffic at small batches, is read once for all of them.
// Each CTA (one per SM) walks output tiles of 128 tokens x NT rows; a tile's K runs through a
// ring of stages of 128 elements:
//   warp 0   TMA: vocabulary codes [128 x 128] (4-bit codes are spread to bytes by the copy
//            engine), hidden codes [NT x 128], both with the 128-byte swizzle, and the scale
//            tiles of both (512 bytes for 128 rows);
//   warp 1   copies the stage's scales to tensor memory and issues four MMAs of 32 elements;
//   warps 4-7 read the finished fp32 tile from tensor memory (two accumulators, so that the next
//            tile's MMAs run meanwhile), round and store it: lanes are tokens, so a warp stores
//            32 consecutive tokens of one row at a time.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"
#include "tc_ptx.cuh"

namespace spec {
namespace mx {
namespace {

using namespace tc;

constexpr int kThreads = 256;
constexpr int kTileV = 128;                     // vocabulary rows of a tile
constexpr int kMaxNT = 192;                     // hidden rows of a tile at most
constexpr int kWBytes = kTileV * kGroup;        // a stage's vocabulary codes, spread to bytes
constexpr int kScaleBytes = 3 * kTileBytes;     // one tile of vocabulary scales, two of hidden
constexpr int kMaxStages = 12;
constexpr int kScaleCols = 12;                  // tensor-memory columns of a stage's scales
constexpr int kTmemCols = 512;
constexpr size_t kSmemMax = 232448;
constexpr size_t kSmemFixed = 1024 + 512;       // alignment of the ring, barriers

struct LogitArgs {
  const uint8_t* as;
  const uint8_t* ws;
  void* out;
  long long ldo;
  int M, V, G;
  int NT, n_tok;        // hidden rows of a tile, tiles of them
  long long units;
  int stages;
  uint32_t w_bytes, a_bytes;  // code bytes a copy reports (the gaps of 4-bit codes not counted)
  uint32_t idesc;       // without N
  int odt;
  bool pairs;           // two tokens in one store
  int stall;            // test request: never load the first tile
  uint32_t* status;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__global__ void __launch_bounds__(kThreads, 1)
    logits_kernel(const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ CUtensorMap map_a, const LogitArgs p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring =
      smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int S = p.stages, b_bytes = p.NT * kGroup;
  unsigned char* sA = ring;                          // [S][kWBytes]
  unsigned char* sB = sA + (size_t)S * kWBytes;      // [S][b_bytes]
  unsigned char* sS = sB + (size_t)S * b_bytes;      // [S][kScaleBytes]
  uint64_t* full = reinterpret_cast<uint64_t*>(sS + (size_t)S * kScaleBytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 3);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(done, 1);
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t sf_col0 = 2 * p.NT;  // scales after the two accumulators

  if (warp == 0 || warp == 2 || warp == 3) {
    // ------------------------------------------------------------------ copies
    // one warp each for the vocabulary codes, the hidden codes and the scales
    const uint32_t lead = elect_lane();
    const uint64_t keep = policy_evict_last();
    const uint64_t w_pol = p.n_tok > 1 ? keep : policy_evict_first();
    int s = 0;
    uint32_t ph = 0;
    bool ok = true, skip = p.stall;
    for (long long u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
      const int vt = (int)(u / p.n_tok), tt = (int)(u - (long long)vt * p.n_tok);
      const int m0 = tt * p.NT, rows = min(p.NT, p.M - m0);
      const int st0 = m0 / kTileRows, st1 = (m0 + rows - 1) / kTileRows;
      const uint8_t* wsp = p.ws + (size_t)vt * p.G * kTileBytes;
      const uint8_t* asp = p.as + (size_t)st0 * p.G * kTileBytes;
      for (int g = 0; g < p.G; ++g) {
        ok = mbar_wait_warp(&empty[s], ph ^ 1, abort, p.status);
        if (!ok) break;
        if (warp == 0) {
          expect_tx_if(lead, &full[s], p.w_bytes);
          tma_load_2d_if(skip ? 0 : lead, sA + (size_t)s * kWBytes, &map_w, g * kGroup,
                         vt * kTileV, &full[s], w_pol);
          skip = false;
        } else if (warp == 2) {
          expect_tx_if(lead, &full[s], p.a_bytes);
          tma_load_2d_if(lead, sB + (size_t)s * b_bytes, &map_a, g * kGroup, m0, &full[s], keep);
        } else {
          unsigned char* sc = sS + (size_t)s * kScaleBytes;
          expect_tx_if(lead, &full[s], kTileBytes * (2 + st1 - st0));
          bulk_load_if(lead, sc, wsp + (size_t)g * kTileBytes, kTileBytes, &full[s], w_pol);
          bulk_load_if(lead, sc + kTileBytes, asp + (size_t)g * kTileBytes, kTileBytes, &full[s],
                       keep);
          if (st1 > st0)
            bulk_load_if(lead, sc + 2 * kTileBytes, asp + (size_t)(p.G + g) * kTileBytes,
                         kTileBytes, &full[s], keep);
        }
        if (++s == S) { s = 0; ph ^= 1; }
      }
    }
    // copies in flight land before the CTA's shared memory goes away
    for (int i = 0; i < S; ++i) mbar_drain(&full[i], i < s ? ph : (ph ^ 1));
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    const uint32_t lead = elect_lane();
    int s = 0, as = 0;
    uint32_t ph = 0, aph = 0;
    bool ok = true;
    for (long long u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
      const int tt = (int)(u % p.n_tok), m0 = tt * p.NT, rows = min(p.NT, p.M - m0);
      const int n = (rows + 15) & ~15;
      const uint32_t idesc = p.idesc | ((uint32_t)(n >> 3) << 17);
      const bool two = m0 / kTileRows != (m0 + rows - 1) / kTileRows;
      ok = mbar_wait_warp(&acc_empty[as], aph ^ 1, abort, p.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + as * p.NT;
      for (int g = 0; g < p.G; ++g) {
        ok = mbar_wait_warp(&full[s], ph, abort, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sc = smem_u32(sS + (size_t)s * kScaleBytes);
        const uint32_t sa = tmem + sf_col0 + s * kScaleCols, sb = sa + 4;
        copy_scales(lead, sa, scale_desc(sc));
        copy_scales(lead, sb, scale_desc(sc + kTileBytes));
        if (two) copy_scales(lead, sb + 4, scale_desc(sc + 2 * kTileBytes));
        const uint64_t da = sw128_desc(smem_u32(sA + (size_t)s * kWBytes));
        const uint64_t db = sw128_desc(smem_u32(sB + (size_t)s * b_bytes));
#pragma unroll
        for (int b = 0; b < 4; ++b)  // 32 bytes of a row a step
          mma_mx(lead, d, da + 2 * b, db + 2 * b, idesc | block_scale_ids(b), sa,
                 sb + (m0 % kTileRows) / 32, (g | b) != 0);
        mma_commit_if(lead, &empty[s]);
        if (++s == S) { s = 0; ph ^= 1; }
      }
      if (!ok) break;
      mma_commit_if(lead, &acc_full[as]);
      as ^= 1;
      if (as == 0) aph ^= 1;
    }
    // every MMA issued here completes before tensor memory is released
    mma_commit_if(lead, done);
    mbar_drain(done, 0);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;  // the lane quarter this warp may read
    int as = 0;
    uint32_t aph[2] = {0, 0};
    for (long long u = blockIdx.x; u < p.units; u += gridDim.x) {
      const int vt = (int)(u / p.n_tok), tt = (int)(u - (long long)vt * p.n_tok);
      const int m0 = tt * p.NT, rows = min(p.NT, p.M - m0);
      if (!mbar_wait(&acc_full[as], aph[as], abort, p.status)) break;
      tc_fence_after();
      const int v = vt * kTileV + q * 32 + lane;
      for (int c = 0; c < rows; c += 32) {
        float x[32];
        tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + as * p.NT + c, x);
        if (c + 32 >= rows) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[as]);
        }
        const int n = rows - c;
        const size_t at = (size_t)(m0 + c) * p.ldo + v;
        if (p.odt == SPEC_F32) {
          float* o = reinterpret_cast<float*>(p.out) + at;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < n && v < p.V) o[(size_t)j * p.ldo] = x[j];
        } else if (p.pairs) {
          // neighbouring lanes trade halves: the even lane stores both tokens of row j, the odd
          // one those of row j + 1
          const bool odd = lane & 1;
          uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + at - odd;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float other = __shfl_xor_sync(0xffffffffu, odd ? x[j] : x[j + 1], 1);
            const uint32_t w = odd ? pack_bf16(other, x[j + 1]) : pack_bf16(x[j], other);
            if (j + odd < n && v < p.V)
              *reinterpret_cast<uint32_t*>(o + (size_t)(j + odd) * p.ldo) = w;
          }
        } else {
          uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + at;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < n && v < p.V) o[(size_t)j * p.ldo] = (uint16_t)pack_bf16(x[j], 0.0f);
        }
      }
      aph[as] ^= 1;
      as ^= 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

}  // namespace
}  // namespace mx

cudaError_t launch_mx_logits(const uint8_t* ac, const uint8_t* as, int af, const uint8_t* wc,
                             const uint8_t* wsc, int wf, int M, int V, int K, void* out, int odt,
                             long long ldo, uint32_t* status, cudaStream_t s) {
  using namespace mx;
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  LogitArgs p;
  p.as = as;
  p.ws = wsc;
  p.out = out;
  p.ldo = ldo;
  p.M = M;
  p.V = V;
  p.G = groups(K);
  // tiles of equal height, a multiple of 64 rows where there are several (a scale tile's columns
  // of tensor memory hold 32 rows each, and a tile starts at an even one)
  p.n_tok = (M + kMaxNT - 1) / kMaxNT;
  p.NT = p.n_tok == 1 ? (M + 15) / 16 * 16 : ((M + p.n_tok - 1) / p.n_tok + 63) / 64 * 64;
  p.n_tok = (M + p.NT - 1) / p.NT;
  p.units = (long long)((V + kTileV - 1) / kTileV) * p.n_tok;
  const size_t stage = kWBytes + (size_t)p.NT * kGroup + kScaleBytes;
  int S = (int)((kSmemMax - kSmemFixed) / stage);
  const int cols = (kTmemCols - 2 * p.NT) / kScaleCols;
  S = S < kMaxStages ? S : kMaxStages;
  p.stages = S < cols ? S : cols;
  p.w_bytes = (uint32_t)(kTileV * code_row(wf, kGroup));
  p.a_bytes = (uint32_t)(p.NT * code_row(af, kGroup));
  const int e2m1 = 5, e4m3 = 0;  // the instruction's format codes
  p.idesc = tc::idesc_mx(kTileV, 0, wf == SPEC_MX_E2M1 ? e2m1 : e4m3,
                         af == SPEC_MX_E2M1 ? e2m1 : e4m3);
  p.odt = odt;
  p.pairs = V % 2 == 0 && ldo % 2 == 0 && (reinterpret_cast<uintptr_t>(out) & 3) == 0;
  p.stall = take_stall_request();
  p.status = status;
  CUtensorMap mw, ma;
  if (!make_tensor_map_codes(&mw, wc, wf, padded(K), V, kTileV) ||
      !make_tensor_map_codes(&ma, ac, af, padded(K), M, p.NT))
    return cudaErrorInvalidValue;
  const size_t smem = kSmemFixed + p.stages * stage;
  static_assert(kSmemFixed - 1024 >= (2 * kMaxStages + 5) * 8 + 8, "room for the barriers");
  // the opt-in to large shared memory holds for the life of the device's context
  static bool opted[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !__atomic_load_n(&opted[dev], __ATOMIC_RELAXED)) {
    e = cudaFuncSetAttribute(logits_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kSmemMax);
    if (e != cudaSuccess) return e;
    if (dev < 64) __atomic_store_n(&opted[dev], true, __ATOMIC_RELAXED);
  }
  const int grid = (int)(p.units < num_sms() ? p.units : num_sms());
  logits_kernel<<<grid, kThreads, smem, s>>>(mw, ma, p);
  return cudaGetLastError();
}

}  // namespace spec
