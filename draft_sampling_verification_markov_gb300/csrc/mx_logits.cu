// mx_logits.cu -- logits of block-scaled hidden rows against a block-scaled vocabulary matrix on
// the tcgen05 tensor cores (kind::mxf8f6f4: products of 8- and 4-bit elements, one power-of-two
// scale per 32 of them applied by the tensor core, fp32 accumulation).
//
// out[m, v] = sum over blocks b of 2^(ea[m, b] + ew[v, b]) sum_{k in b} a[m, k] w[v, k].
//
// The vocabulary is the M side of the instruction (always full) and the hidden rows its N side (32
// .. 256 of them), so that one request costs no more tensor-core rows than it must and the
// vocabulary matrix, which is the traffic at small batches, is read once for all of them. CTAs work
// in pairs (cta_group::2) on tiles of 256 tokens x NT rows: each holds 128 tokens' codes and half
// of the hidden rows' codes. A single CTA on 128 tokens x 192 rows was bound by its shared memory
// (4-bit codes are spread to bytes on the way in: 40 KB written and read for 384 tensor-core
// cycles); a pair writes and reads 28 KB an SM for the same products, and 32 KB for the 512 cycles
// of 256 rows. A tile's K runs through a ring of stages of 128 elements:
//   warps 0, 2, 3  TMA: vocabulary codes [128 x 128], hidden codes [NT / 2 x 128], both with the
//                  128-byte swizzle, and the scale tiles of both (512 bytes for 128 rows). One
//                  warp each, in uniform control flow: a single thread that issued all of them
//                  took longer than the copies;
//   warp 1         of the even CTA copies a stage's scales to tensor memory and issues four MMAs
//                  of 32 elements for the pair;
//   warps 4-11     read the finished fp32 tile from tensor memory, round and store it: lanes are
//                  tokens, so a warp stores 32 consecutive tokens of one row at a time. Up to 192
//                  rows two accumulators alternate; above, tensor memory holds one beside the
//                  scales.
//
// Measured (V = 129280, K = 4096, 4-bit vocabulary, 8-bit rows, bf16 out, back to back in a graph,
// two vocabulary matrices in turn so that none of one stays in L2): 64 rows 50.7 us (5.9 TB/s; the
// 298 MB alone are 44 us), 128 rows 55.7, 256 rows 87 us (tensor pipe active 79 %), 1792 rows 517
// us (3.7 PFLOP/s, tensor pipe active 87 %); in a loop of a second the power limit brings the last
// to 600 us. At 256 rows the reading of the accumulator between tiles costs some 14 us, the scale
// copies 5, the stores 10. With an 8-bit vocabulary (546 MB: 81 us at the measured copy rate) one
// row takes 84 us, 64 rows 85.5, 256 rows 110, 1792 rows 555 to 620. Polling the barriers without
// suspending is 1 to 2 % slower, and so is fetching the tensor maps ahead.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "common.cuh"
#include "kernels.h"
#include "mx.cuh"
#include "tc_pair.cuh"

namespace spec {
namespace mx {
namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kTileV = 128;                     // vocabulary rows of a CTA's tile
constexpr int kMaxNT = 256;                     // hidden rows of a tile at most
constexpr int kTwoNT = 192;                     // ... with two accumulators
constexpr int kChunks = kMaxNT / 32 / 2;        // 32-row chunks of an epilogue warp
constexpr int kWBytes = kTileV * kGroup;        // a stage's vocabulary codes, spread to bytes
constexpr int kScaleBytes = 3 * kTileBytes;     // one tile of vocabulary scales, two of hidden
constexpr int kMaxStages = 10;
constexpr int kScaleCols = 12;                  // tensor-memory columns of a stage's scales
constexpr int kTmemCols = 512;
constexpr size_t kSmemMax = 232448;
constexpr int kOutRows = 16;                    // rows of a staged piece of bf16 output
constexpr int kOutBytes = kOutRows * kTileV * 2;
constexpr size_t kSmemFixed = 1024 + 512 + 4 * kOutBytes;  // alignment, barriers, staged output
static_assert(2 * kTwoNT + kMaxStages * kScaleCols <= kTmemCols &&
                  kMaxNT + kMaxStages * kScaleCols <= kTmemCols,
              "tensor memory");
static_assert((2 * kMaxStages + 5) * 8 + 8 <= 512, "room for the barriers");

struct LogitArgs {
  void* out;
  long long ldo;
  int M, V, G;
  int NT, n_tok;        // hidden rows of a tile, tiles of them
  int n_acc;            // accumulators
  int n_voc;            // 128-row tiles of the vocabulary
  long long units;      // pairs of vocabulary tiles x hidden tiles
  int stages;
  uint32_t w_bytes, a_bytes;  // code bytes a copy reports (the gaps of 4-bit codes not counted)
  uint32_t idesc;       // without N
  int odt;
  bool staged;          // bf16 output through shared memory and bulk stores
  bool pairs;           // ... else two tokens in one store
  int stall;            // test request: never load the first tile
  uint32_t* status;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// One unit of work: two vocabulary tiles against one tile of hidden rows.
struct Work {
  int vt;       // this CTA's vocabulary tile
  int m0, rows; // hidden rows
  int n;        // N of the instruction
  int st0, st1; // tiles of their scales, first and last
  __device__ __forceinline__ Work(const LogitArgs& p, long long u, int rank) {
    const int vp = (int)(u / p.n_tok), tt = (int)(u - (long long)vp * p.n_tok);
    vt = 2 * vp + rank;
    m0 = tt * p.NT;
    rows = min(p.NT, p.M - m0);
    n = (rows + 31) & ~31;
    st0 = m0 / kTileRows;
    st1 = (m0 + rows - 1) / kTileRows;
  }
};

// Rows m .. m + min(32, n) - 1 of token v (this lane's), from their fp32 sums.
__device__ __forceinline__ void store_chunk(const LogitArgs& p, const uint32_t (&x)[32], int m,
                                            int n, int v) {
  const size_t at = (size_t)m * p.ldo + v;
  const bool live = v < p.V;
  if (p.odt == SPEC_F32) {
    uint32_t* o = reinterpret_cast<uint32_t*>(p.out) + at;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n && live) o[(size_t)j * p.ldo] = x[j];
  } else if (p.pairs) {
    // neighbouring lanes trade halves: the even lane stores both tokens of row j, the odd one
    // those of row j + 1
    const bool odd = threadIdx.x & 1;
    uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + at - odd + (odd ? p.ldo : 0);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const uint32_t both = pack_bf16(__uint_as_float(x[j]), __uint_as_float(x[j + 1]));
      const uint32_t other = __shfl_xor_sync(0xffffffffu, both, 1);
      const uint32_t b = odd ? __byte_perm(other, both, 0x7632) : __byte_perm(both, other, 0x5410);
      if (j + odd < n && live) *reinterpret_cast<uint32_t*>(o + (size_t)j * p.ldo) = b;
    }
  } else {
    uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + at;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n && live) o[(size_t)j * p.ldo] = (uint16_t)pack_bf16(__uint_as_float(x[j]), 0.0f);
  }
}

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    logits_kernel(const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ CUtensorMap map_ws,
                  const __grid_constant__ CUtensorMap map_as,
                  const __grid_constant__ CUtensorMap map_out, const LogitArgs p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int S = p.stages, b_bytes = p.NT / 2 * kGroup;
  unsigned char* sA = ring;                          // [S][kWBytes]
  unsigned char* sB = sA + (size_t)S * kWBytes;      // [S][b_bytes]
  unsigned char* sO = sB + (size_t)S * b_bytes;      // [2 halves][2][kOutBytes]
  unsigned char* sS = sO + 4 * kOutBytes;            // [S][kScaleBytes]
  uint64_t* full = reinterpret_cast<uint64_t*>(sS + (size_t)S * kScaleBytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1;  // in the pair; 0 issues the MMAs
  const long long u_first = blockIdx.x >> 1, u_step = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 3);   // the even CTA's: its copy warps; bytes of both CTAs
      mbar_init(&empty[s], 1);  // each CTA's own
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);   // each CTA's own
      mbar_init(&acc_empty[i], 16);  // the even CTA's: both CTAs' epilogue warps
    }
    mbar_init(done, 1);
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers are ready
  tc_fence_after();
  grid_dep_wait();
  // what the kernel before wrote with plain stores is read by the copy engine
  asm volatile("fence.proxy.async.global;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  const uint32_t sf_col0 = p.n_acc * p.NT;  // scales after the accumulators

  if (warp == 0 || warp == 2 || warp == 3) {
    // ------------------------------------------------------------------ copies
    // Vocabulary codes, hidden codes and scales. All report to the even CTA's barrier, whose copy
    // warps expect the bytes of both CTAs.
    const uint32_t lead = elect_lane();
    const uint64_t keep = policy_evict_last();
    const uint64_t w_pol = p.n_tok > 1 ? keep : policy_evict_first();
    int s = 0;
    uint32_t ph = 0;
    bool ok = true, skip = p.stall;
    for (long long u = u_first; u < p.units && ok; u += u_step) {
      const Work w(p, u, rank);
      const int ws_row = min(w.vt, p.n_voc - 1) * p.G;  // a pair's second tile may be past the end
      for (int g = 0; g < p.G; ++g) {
        ok = mbar_wait_warp(&empty[s], ph ^ 1, abort, p.status);
        if (!ok) break;
        const uint32_t bar = in_cta(&full[s], 0);
        if (warp == 0) {
          expect_tx_if(rank == 0 ? lead : 0, &full[s], 2 * p.w_bytes);
          tma_load_2d_pair(skip ? 0 : lead, sA + (size_t)s * kWBytes, &map_w, g * kGroup,
                           w.vt * kTileV, bar, w_pol);
          skip = false;
        } else if (warp == 2) {
          expect_tx_if(rank == 0 ? lead : 0, &full[s], 2 * p.a_bytes);
          tma_load_2d_pair(lead, sB + (size_t)s * b_bytes, &map_a, g * kGroup,
                           w.m0 + rank * (w.n / 2), bar, keep);
        } else {
          unsigned char* sc = sS + (size_t)s * kScaleBytes;
          expect_tx_if(rank == 0 ? lead : 0, &full[s], 2 * kTileBytes * (2 + w.st1 - w.st0));
          tma_load_2d_pair(lead, sc, &map_ws, 0, ws_row + g, bar, w_pol);
          tma_load_2d_pair(lead, sc + kTileBytes, &map_as, 0, w.st0 * p.G + g, bar, keep);
          if (w.st1 > w.st0)
            tma_load_2d_pair(lead, sc + 2 * kTileBytes, &map_as, 0, w.st1 * p.G + g, bar, keep);
        }
        if (++s == S) { s = 0; ph ^= 1; }
      }
    }
    // copies in flight (the other CTA's too) land before shared memory goes away
    if (rank == 0)
      for (int i = 0; i < S; ++i) mbar_drain(&full[i], i < s ? ph : (ph ^ 1));
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------------ MMA
    // At small N this warp's own instructions are part of the bound (one more branch a stage cost
    // 8 % at 64 rows): a stage's descriptors are additions to the last one's, and whether the next
    // stage is full is asked before this stage's instructions are issued (64 rows of one
    // matrix: 49.6 -> 47.6 us).
    const uint32_t lead = elect_lane();
    const uint64_t da0 = sw128_desc(smem_u32(sA)), db0 = sw128_desc(smem_u32(sB));
    const uint64_t ds0 = scale_desc(smem_u32(sS));
    uint64_t da = da0, db = db0, ds = ds0;  // of stage s
    uint32_t sf = tmem + sf_col0;
    int s = 0, as = 0;
    uint32_t ph = 0, aph = 0;
    bool ok = true, ready = false;
    for (long long u = u_first; u < p.units && ok; u += u_step) {
      const Work w(p, u, 0);
      const uint32_t idesc = p.idesc | ((uint32_t)(w.n >> 3) << 17);
      const uint32_t sb_col = 4 + (w.m0 % kTileRows) / 32;
      const bool two = w.st1 > w.st0;
      ok = mbar_wait_warp(&acc_empty[as], aph ^ 1, abort, p.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + as * p.NT;
      for (int g = 0; g < p.G; ++g) {
        if (!__all_sync(0xffffffffu, ready)) {
          ok = mbar_wait_warp(&full[s], ph, abort, p.status);
          if (!ok) break;
        }
        tc_fence_after();
        const int next = s + 1 == S ? 0 : s + 1;
        const uint32_t next_ph = s + 1 == S ? ph ^ 1 : ph;
        ready = mbar_test(&full[next], next_ph);
        copy_scales_pair(lead, sf, ds);
        copy_scales_pair(lead, sf + 4, ds + kTileBytes / 16);
        if (two) copy_scales_pair(lead, sf + 8, ds + 2 * kTileBytes / 16);
#pragma unroll
        for (int b = 0; b < 4; ++b)  // 32 bytes of a row a step
          mma_mx_pair(lead, d, da + 2 * b, db + 2 * b, idesc | block_scale_ids(b), sf, sf + sb_col,
                      (g | b) != 0);
        commit_pair(lead, &empty[s]);
        s = next;
        ph = next_ph;
        da = s ? da + kWBytes / 16 : da0;
        db = s ? db + b_bytes / 16 : db0;
        ds = s ? ds + kScaleBytes / 16 : ds0;
        sf = s ? sf + kScaleCols : tmem + sf_col0;
      }
      if (!ok) break;
      commit_pair(lead, &acc_full[as]);
      if (++as == p.n_acc) { as = 0; aph ^= 1; }
    }
    // every MMA issued here completes before tensor memory is released
    commit_pair(lead, done, 1);
    mbar_drain(done, 0);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ epilogue
    // Two warps a lane quarter share its 32-row chunks. A warp takes all of its chunks into
    // registers first, so that a single accumulator is free again after some hundred cycles and
    // the stores run beside the next tile's MMAs. (At the 168 registers that leaves a thread, 48 bytes
    // are spilled.)
    const int q = warp & 3;            // the lane quarter this warp may read
    const int half = (warp - 4) >> 2;
    const int issuer = 128 * (1 + half);  // the half's thread that hands pieces over
    int as = 0;
    uint32_t aph = 0;
    for (long long u = u_first; u < p.units; u += u_step) {
      const Work w(p, u, rank);
      // the four warps of a half meet at barriers below: they go on together or not at all
      if (!all_of(1 + half, 128, mbar_wait_warp(&acc_full[as], aph, abort, p.status))) break;
      tc_fence_after();
      uint32_t x[kChunks][32];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = 32 * (2 * i + half);
        if (c < w.rows)
          tmem_ld32_async(tmem + ((uint32_t)(q * 32) << 16) + as * p.NT + c, x[i]);
      }
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(in_cta(&acc_empty[as], 0));
      const int v = w.vt * kTileV + q * 32 + lane;
      if (p.staged) {
        // pieces of 16 rows x 128 tokens, two buffers a half: the half's four warps write their
        // tokens, one thread hands the piece to the copy engine, which clips it to the output.
        // A piece's buffer must have been read by the copy of the piece before the last. A tile
        // starts with the first buffer whichever the last tile ended with (an odd number of
        // pieces ends with the first, too), so its first piece waits for every copy before it.
#pragma unroll
        for (int i = 0; i < 2 * kChunks; ++i) {
          const int c = 32 * (i - i % 2 + half) + kOutRows * (i % 2);
          if (c >= w.rows) break;
          const uint32_t buf = smem_u32(sO + (2 * half + i % 2) * kOutBytes);
          if (threadIdx.x == issuer) {
            if (i == 0)
              asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            else
              asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          }
          asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
          const uint32_t at = buf + (q * 32 + lane) * 2;
#pragma unroll
          for (int j = 0; j < kOutRows; ++j)
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(at + j * kTileV * 2),
                         "h"((uint16_t)pack_bf16(
                             __uint_as_float(x[i / 2][kOutRows * (i % 2) + j]), 0.0f))
                         : "memory");
          fence_async_smem();
          asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
          if (threadIdx.x == issuer) {
            asm volatile(
                "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                    reinterpret_cast<uint64_t>(&map_out)),
                "r"(w.vt * kTileV), "r"(w.m0 + c), "r"(buf)
                : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int c = 32 * (2 * i + half);
          if (c >= w.rows) break;
          store_chunk(p, x[i], w.m0 + c, w.rows - c, v);
        }
      }
      if (++as == p.n_acc) { as = 0; aph ^= 1; }
    }
    // staged pieces are read before shared memory goes away
    if (threadIdx.x == issuer) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other's copies or MMAs may touch it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

// ------------------------------------------------------------------------------ host side

// A 2-D map of cols x rows elements in boxes of box_cols x box_rows.
bool make_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, long long cols,
              long long rows, long long row_bytes, int box_cols, int box_rows,
              CUtensorMapSwizzle swizzle) {
  if (!tc::encode_fn()) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, estr[2] = {1, 1};
  return tc::encode_fn()(m, type, 2, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of codes in boxes of one group. 4-bit codes land in shared memory spread over 16-byte
// units: sixteen codes, then eight bytes of gap.
bool map_codes(CUtensorMap* m, const void* codes, int fmt, int Kp, int rows, int box_rows) {
  return make_map(m,
                  fmt == SPEC_MX_E2M1 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B
                                      : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                  codes, Kp, rows, (long long)code_row(fmt, Kp), kGroup, box_rows,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scale tiles, one a box.
bool map_scales(CUtensorMap* m, const void* scales, long long tiles) {
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, scales, kTileBytes / 4, tiles, kTileBytes,
                  kTileBytes / 4, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Pairs of CTAs the device holds at once (of the current device; 0 if it cannot be found out).
int max_pairs() {
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && __atomic_load_n(&cached[dev], __ATOMIC_RELAXED)) return cached[dev];
  // the opt-in to large shared memory holds for the life of the device's context
  if (cudaFuncSetAttribute(logits_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kSmemMax) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3(num_sms() / 2 * 2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemMax;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, logits_kernel, &cfg) != cudaSuccess || n < 1) return 0;
  if (dev < 64) __atomic_store_n(&cached[dev], n, __ATOMIC_RELAXED);
  return n;
}

}  // namespace
}  // namespace mx

cudaError_t launch_mx_logits(const uint8_t* ac, const uint8_t* as, int af, const uint8_t* wc,
                             const uint8_t* wsc, int wf, int M, int V, int K, void* out, int odt,
                             long long ldo, uint32_t* status, cudaStream_t s) {
  using namespace mx;
  const int pairs = max_pairs();
  if (pairs < 1) return cudaErrorInvalidConfiguration;
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  LogitArgs p;
  p.out = out;
  p.ldo = ldo;
  p.M = M;
  p.V = V;
  p.G = groups(K);
  // tiles of equal height, a multiple of 64 rows where there are several (a scale tile's columns
  // of tensor memory hold 32 rows each, and a tile starts at an even one)
  p.n_tok = (M + kMaxNT - 1) / kMaxNT;
  p.NT = p.n_tok == 1 ? (M + 31) / 32 * 32 : ((M + p.n_tok - 1) / p.n_tok + 63) / 64 * 64;
  p.n_tok = (M + p.NT - 1) / p.NT;
  p.n_acc = p.NT <= kTwoNT ? 2 : 1;
  p.n_voc = (V + kTileV - 1) / kTileV;
  p.units = (long long)((p.n_voc + 1) / 2) * p.n_tok;
  const size_t stage = kWBytes + (size_t)p.NT / 2 * kGroup + kScaleBytes;
  const int S = (int)((kSmemMax - kSmemFixed) / stage);
  p.stages = S < kMaxStages ? S : kMaxStages;
  const int e2m1 = 5, e4m3 = 0;  // the instruction's format codes
  p.w_bytes = (uint32_t)(kTileV * code_row(wf, kGroup));
  p.a_bytes = (uint32_t)(p.NT / 2 * code_row(af, kGroup));
  p.idesc = tc::idesc_mx(2 * kTileV, 0, wf == SPEC_MX_E2M1 ? e2m1 : e4m3,
                         af == SPEC_MX_E2M1 ? e2m1 : e4m3);
  p.odt = odt;
  p.staged = odt == SPEC_BF16 && (ldo * 2) % 16 == 0 &&
             (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  p.pairs = V % 2 == 0 && ldo % 2 == 0 && (reinterpret_cast<uintptr_t>(out) & 3) == 0;
  p.stall = take_stall_request();
  p.status = status;
  CUtensorMap mw, ma, mws, mas, mo;
  memset(&mo, 0, sizeof mo);
  if (p.staged && !make_map(&mo, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, out, V, M, ldo * 2, kTileV,
                            kOutRows, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  if (!map_codes(&mw, wc, wf, padded(K), V, kTileV) ||
      !map_codes(&ma, ac, af, padded(K), M, p.NT / 2) ||
      !map_scales(&mws, wsc, (long long)p.n_voc * p.G) ||
      !map_scales(&mas, as, (long long)((M + kTileRows - 1) / kTileRows) * p.G))
    return cudaErrorInvalidValue;
  const int grid = 2 * (int)(p.units < pairs ? p.units : pairs);
  return launch_kernel(logits_kernel, grid, kThreads, kSmemFixed + p.stages * stage, s, true, mw, ma,
                       mws, mas, mo, p);
}

}  // namespace spec
