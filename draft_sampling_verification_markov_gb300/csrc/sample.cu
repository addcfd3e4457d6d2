// sample.cu -- truncated sampling: top-k, top-p and min-p over softmax(x / T), one draw a row from a
// given uniform, or the row itself with -inf outside what is left.
//
// Tokens are ordered by key: larger logits first, then lower ids. Each of the three rules leaves a
// prefix of that order, so a row's truncation is one key: a token stays iff its key is at least it.
//   top-k   the k-th key;
//   top-p   the last key before which less than p of the mass (of what top-k left) has been reached;
//   min-p   the last key of a logit >= max x + T log(min_p).
// The draw walks what is left in order of the ids: the first token whose cumulative mass passes u.
//
// A border between two tokens, in the order or in the draw, is decided by the last bits of a sum
// over the vocabulary: a fp32 sum, or an approximate exponential, moves the borders of unlikely
// tokens by more than their own mass. So masses are whole numbers (Weigher): exp((x - max) / T)
// in units of 2^-(S + 1), off by one of them and by about 2^-31 of themselves, summed without
// rounding in 64 bits.
// Sums do not depend on their order, the draw is the same however the row is split, and p and u
// are compared exactly.
//
// The first pass over a row keeps the largest key of every thread's batch (64 bytes; more where a
// row has more than 4096 batches) in shared memory. What comes next is the cheapest that decides:
//   - the first token alone, top-k up to 1024, min-p: the k-th largest of the batches' bounds the k-th
//     largest logit from below, only the batches that reach the bound are read again, from L2, and the
//     rules and the draw are decided on a list of up to 2048 tokens;
//   - top-p of a row: an approximate pass fills bins of 1/32 octave, which tell to within a few hundred
//     tokens where the nucleus ends. A list of all before that decides it, or, where they are more, an
//     exact pass that sums what is above the window and lists the window;
//   - a larger top-k: the k-th logit by its leading bits, 10 at a time, then as before;
//   - thousands of equal logits at the border, as bf16 has them far from zero: the logit by halving,
//     beginning at the window, a pass a step, then the token by counting the equal ones (logits of mean
//     40: 2048 rows at p 0.95 2.6 ms, 14.4 with ids halved too and no window);
//   - a temperature alone: one exact pass.
// An exact pass is bound by its instructions, 23 a token; the others by memory and by the latency of
// a row's steps. 2048 rows of 129280 bf16 logits (529 MB, 78 us at the copy bandwidth): first token 102
// us, top-k 50 144, top-k 200 and p 0.9 185, top-k 1000 285, min-p 0.05 127 to 177, a temperature alone
// 312, p 0.95 464 (64 tokens stand out) to 753 (normal logits); mixed by request 256 to 311, and
// written out instead of drawn from 398 to 447.
//
// Three CTAs of 256 threads an SM, a CTA a row. Few rows are split over a cluster of up to 8 CTAs,
// which merge through distributed shared memory: twice as many as long as there are no more than SMs,
// whatever the rules. Measured beside that: 64 rows on 512 CTAs, more than have a place, instead of 256
// (top-k 50 25 -> 44 us); up to three CTAs for two SMs (180 rows: a temperature alone 56 -> 49, top-k
// 21 -> 28; 64 rows of the former 29 -> 39); 2048 rows on two CTAs each (top-k 50 150 -> 285). A list's
// steps do not get shorter with a row's part; a pass over the whole row may, and the best division
// goes by the rule, which this one does not.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "row_pieces.cuh"
#include "tc_ptx.cuh"

namespace spec {
namespace {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kCtas = 3;                        // of an SM
constexpr int kWarps = kThreads / 32;
static_assert((kWarps & (kWarps - 1)) == 0, "lanes wrap around the warps");
constexpr int kBatch = 4;                       // 16-byte pieces of a thread's batch
constexpr int kWarpStep = 32 * kBatch;          // consecutive pieces of a warp: a segment
constexpr int kStep = kThreads * kBatch;        // ... of a CTA
constexpr int kGroupsMost = 16;                 // index entries of a thread
constexpr int kEntries = kGroupsMost * kThreads;
constexpr int kList = 2048;                     // tokens listed at most
constexpr int kHits = kList;                    // index entries listed at most
constexpr int kTopsMost = 64;                   // largest k bounded by the threads' largest logits
constexpr int kListTop = 1024;                  // largest k that goes through the list
constexpr int kListMost = kList - 256;          // tokens that a guess may put there
constexpr int kBins = 1536;                     // 1/32 octave each
constexpr int kBinsThread = kBins / kThreads;
constexpr int kMaxSplit = 8;
constexpr int kBuckets = kThreads;
constexpr uint32_t kFull = 0xffffffffu;

// Segments of the largest row.
constexpr int kSegs = SPEC_SAMPLE_MAX_VOCAB / 4 / kWarpStep + kWarps;

struct Shared {
  union {
    uint32_t index[kEntries];  // largest order_bits of a thread's batches
    u64 seg[kSegs];            // masses of a part's segments, once the index is not needed
    u64 bucket[kBuckets];
  };
  union {
    u64 keys[kList];           // listed tokens
    struct {                   // while the bins are filled: where in its bin a token lies, of some
      uint32_t off[kBins], offs[kBins];
    };
    struct {                   // then: masses of the bins, and of a share of the cluster's
      float weight[kBins], shares[kBins / 2];
    };
  };
  uint32_t bins[kBins];      // tokens by their mass
  union {
    uint16_t hits[kHits];      // index entries that reach a bound
    u64 picked[2][kBuckets];   // masses of ranges, keys of one
    uint32_t slice[kBins / 2]; // of the cluster's bins, this part's share
  };
  int n_list, n_hits;
  u64 pub[2][2];             // what a CTA shows its cluster
  u64 red[3][kWarps];
  uint32_t best[kWarps];
  float fred[kWarps];
  // the row's parameters
  float scale, ch, cl;
  int k;
  float p;
  bool by_m;
  double below;              // log(min_p) T
  uint32_t tm;               // order_bits of the least logit that min-p leaves
  // decided by one thread or CTA for the others
  u64 limit, total, rest;
  int kept, done, hit;
  int edge[4], before[4], in;
  float cum[2];
  float guess;               // the share of the mass before bin_lo, as the bins have it
  uint32_t lo_bits, hi_bits;
  int n_above, n_window;
};

// ------------------------------------------------------------------------------ whole-number masses

// 2^(30 + j / 32), rounded.
__constant__ uint32_t kPowers[32] = {
    0x40000000u, 0x4166c34cu, 0x42d561b4u, 0x444c0740u, 0x45cae0f2u, 0x47521cc6u, 0x48e1e9bau, 0x4a7a77d4u,
    0x4c1bf829u, 0x4dc69cddu, 0x4f7a9930u, 0x51382182u, 0x52ff6b55u, 0x54d0ad5au, 0x56ac1f75u, 0x5891fac1u,
    0x5a82799au, 0x5c7dd7a4u, 0x5e8451d0u, 0x60962665u, 0x62b39509u, 0x64dcdec3u, 0x6712460bu, 0x69540ec9u,
    0x6ba27e65u, 0x6dfddbccu, 0x70666f76u, 0x72dc8374u, 0x75606374u, 0x77f25cceu, 0x7a92be8bu, 0x7d41d96eu,
};

// exp((x - m) / T) in units of 2^-(S + 1). With c = log2(e) / T as a pair of fp32 numbers,
// y = (x - m) c as a pair, 32 y = i + 32 r with a whole i and |r| <= 1/64:
//   2^y = 2^(i >> 5) 2^((i & 31) / 32) (1 + (2^r - 1)).
// Lane j of a warp holds 2^(j / 32) in 31 bits, 2^r - 1 is its Taylor polynomial of degree 4 (the
// next term is 2^-39), one 64-bit product-sum joins them. The last bit is set instead of rounded:
// the error is between -1 and 1 units with mean 0, so that a hundred thousand small masses are not
// all rounded the same way. Every lane of the warp has to call it. Two at a time share the packed
// fp32 instructions; one alone goes through the same operations.
constexpr float kMagic = 393216.0f;  // 1.5 * 2^18: ulp 1/32
constexpr int kMagicBits = 0x48c00000;
// ln2^j / j! in units of 2^-32; the first with what its fp32 form leaves
constexpr float kUnit = 4294967296.0f;
constexpr float kC4 = 9.618129107e-3f * kUnit, kC3 = 5.550410867e-2f * kUnit,
                kC2 = 2.402265070e-1f * kUnit, kC1 = 6.931471825e-1f * kUnit,
                kC1Rest = -1.904654e-9f * kUnit;

struct Weigher {
  float m, ch, cl, most;   // most: -y above it has no mass
  uint32_t table;          // kPowers[lane]
  int shift;               // 61 - S

  // The mass is 2 half() + 1 where there is one.
  __device__ __forceinline__ u64 half(float t, float q) const {
    const int bits = __float_as_int(t);
    const int tab = (int)__shfl_sync(kFull, table, bits);
    const long long w = ((long long)tab << 32) + (long long)tab * __float2int_rn(q);
    const int by = shift + 1 + (kMagicBits >> 5) - (bits >> 5);
    return (u64)w >> (by & 63);
  }
  __device__ __forceinline__ u64 join(float y, float t, float q) const {  // y: -(x - m) c
    const u64 v = 2 * half(t, q) + 1;
    return y <= most ? v : 0;  // also for NaN
  }

  template <int DT>
  __device__ __forceinline__ u64 operator()(float x) const {
    const float d = __fsub_rn(m, x);
    const float y = __fmul_rn(d, ch);
    float b = fmaf(d, -cl, fmaf(d, -ch, y));
    // A difference of bf16 numbers is exact, unless one is below 2^-16 of the other: it is then off by
    // 2^-24 of itself. Such logits are rare (one in ten thousand of normal ones beside 20), and
    // three more instructions for every pair would cost all rows.
    if constexpr (DT == SPEC_F32) b = fmaf(two_sum(m, -x).lo, -ch, b);
    const float t = __fsub_rn(kMagic, y);
    const float r = __fsub_rn(b, __fadd_rn(__fsub_rn(t, kMagic), y));
    float q = fmaf(r, kC4, kC3);
    q = fmaf(r, q, kC2);
    q = fmaf(r, q, kC1Rest);
    q = fmaf(r, kC1, __fmul_rn(r, q));
    return join(y, t, q);
  }

  template <int DT>
  __device__ __forceinline__ void terms(float x0, float x1, u64& y, u64& t, u64& q) const {
    using namespace tc;
    const u64 x = pack2(x0, x1), m2 = pack2(m, m), n1 = pack2(-1.0f, -1.0f);
    const u64 ch2 = pack2(ch, ch), nch2 = pack2(-ch, -ch), ncl2 = pack2(-cl, -cl);
    const u64 d = fma2(x, n1, m2);
    y = mul2(d, ch2);
    u64 b = fma2(d, ncl2, fma2(d, nch2, y));
    if constexpr (DT == SPEC_F32) {
      const u64 bb = add2(d, pack2(-m, -m));
      const u64 e = fma2(add2(x, bb), n1, fma2(fma2(bb, n1, d), n1, m2));
      b = fma2(e, nch2, b);
    }
    t = fma2(y, n1, pack2(kMagic, kMagic));
    const u64 r = fma2(add2(add2(t, pack2(-kMagic, -kMagic)), y), n1, b);
    q = fma2(r, pack2(kC4, kC4), pack2(kC3, kC3));
    q = fma2(r, q, pack2(kC2, kC2));
    q = fma2(r, q, pack2(kC1Rest, kC1Rest));
    q = fma2(r, pack2(kC1, kC1), mul2(r, q));
  }
  template <int DT>
  __device__ __forceinline__ void pair(float x0, float x1, u64& v0, u64& v1) const {
    u64 y, t, q;
    terms<DT>(x0, x1, y, t, q);
    float y0, y1, t0, t1, q0, q1;
    tc::unpack2(y, y0, y1);
    tc::unpack2(t, t0, t1);
    tc::unpack2(q, q0, q1);
    v0 = join(y0, t0, q0);
    v1 = join(y1, t1, q1);
  }
  // half() of two logits that both have a mass.
  template <int DT>
  __device__ __forceinline__ void halves(float x0, float x1, u64& h0, u64& h1) const {
    u64 y, t, q;
    terms<DT>(x0, x1, y, t, q);
    float t0, t1, q0, q1;
    tc::unpack2(t, t0, t1);
    tc::unpack2(q, q0, q1);
    h0 = half(t0, q0);
    h1 = half(t1, q1);
  }
  // A finite logit from which on every one has a mass: rounded up, for where logits are far apart
  // beside T (100 and its neighbours at T = 1e-5), and no farther below m than fp32's largest number,
  // or m - x would be infinite.
  __device__ __forceinline__ float surely() const {
    constexpr float kMost = 3.402823466e38f;
    return fmaxf(__fsub_ru(m, (most - 0.125f) / ch), __fsub_ru(m, kMost));
  }
  // Bin of a mass, of t = kMagic + y: -32 y rounded; the last one, and what has none, share a bin.
  __device__ __forceinline__ static uint32_t bin(float t) {
    return min((uint32_t)(kMagicBits - __float_as_int(t)), (uint32_t)kBins - 1);
  }
};

// u * z for a u in [0, 1) of whole z: the product exactly, rounded down (or up).
__device__ __forceinline__ u64 exact_share(float u, u64 z, bool up) {
  const uint32_t b = __float_as_uint(u);
  const int e = (int)(b >> 23);                          // u >= 0
  const u64 man = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int sh = 150 - (e ? e : 1);                      // u = man * 2^-sh, sh >= 24
  const u64 hi = __umul64hi(man, z), lo = man * z;       // below 2^88
  u64 v, rest;
  if (sh >= 128) {
    v = 0;
    rest = hi | lo;
  } else if (sh >= 64) {
    v = sh == 64 ? hi : hi >> (sh - 64);
    rest = lo | (sh == 64 ? 0 : hi & ((1ull << (sh - 64)) - 1));
  } else {
    v = lo >> sh | hi << (64 - sh);
    rest = lo & ((1ull << sh) - 1);
  }
  return v + (up && rest ? 1 : 0);
}

// What a key asks for: x > cut, or x == cut with an id up to last.
struct Cut {
  float x;
  uint32_t id;
  __device__ __forceinline__ explicit Cut(u64 key)
      : x(key >> 32 ? order_value((uint32_t)(key >> 32)) : -INFINITY),
        id(key >> 32 ? 0xffffffffu - (uint32_t)key : 0u) {}
  __device__ __forceinline__ bool leaves(float v, int at) const {
    // key 0 leaves everything above -inf
    return v > x || (v == x && (uint32_t)at <= id && v > -INFINITY);
  }
};

// ------------------------------------------------------------------------------ a CTA or cluster

template <bool SPLIT>
struct Team {
  Shared& sh;
  cg::cluster_group cluster;
  int parts, part, turn;

  __device__ Team(Shared& s, int n)
      : sh(s), cluster(cg::this_cluster()), parts(SPLIT ? n : 1),
        part(SPLIT ? (int)(blockIdx.x % n) : 0), turn(0) {}
  __device__ __forceinline__ void sync() {
    if constexpr (SPLIT)
      cluster.sync();
    else
      __syncthreads();
  }
  __device__ __forceinline__ Shared* leader() {
    if constexpr (SPLIT) return cluster.map_shared_rank(&sh, 0);
    return &sh;
  }

  // Sums of two numbers over the team's threads, and the first one's over the parts before. The
  // slots alternate, so a part may be a call ahead of one that still reads.
  struct Sum {
    u64 a, b, before, own;
  };
  __device__ __noinline__ Sum sum(u64 a, u64 b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(kFull, a, o);
      b += __shfl_xor_sync(kFull, b, o);
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) {
      sh.red[0][warp] = a;
      sh.red[1][warp] = b;
    }
    __syncthreads();
    Sum s{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      s.a += sh.red[0][w];
      s.b += sh.red[1][w];
    }
    s.own = s.a;
    if constexpr (SPLIT) {
      if (threadIdx.x == 0) {
        sh.pub[turn][0] = s.a;
        sh.pub[turn][1] = s.b;
      }
      cluster.sync();
      // lane q: part q
      const Shared* o = cluster.map_shared_rank(&sh, lane < parts ? lane : 0);
      u64 x = lane < parts ? o->pub[turn][0] : 0, y = lane < parts ? o->pub[turn][1] : 0;
#pragma unroll
      for (int d = 1; d < kMaxSplit; d <<= 1) {
        const u64 z = __shfl_up_sync(kFull, x, d);
        if (lane >= d) x += z;
        y += __shfl_xor_sync(kFull, y, d);
      }
      s.a = __shfl_sync(kFull, x, kMaxSplit - 1);
      s.b = __shfl_sync(kFull, y, 0);
      s.before = __shfl_sync(kFull, x, part) - s.own;
      turn ^= 1;
    } else {
      __syncthreads();
    }
    return s;
  }
  __device__ __noinline__ uint32_t max(uint32_t a) {
    const int lane = threadIdx.x & 31;
    a = __reduce_max_sync(kFull, a);
    if (lane == 0) sh.best[threadIdx.x >> 5] = a;
    __syncthreads();
    a = __reduce_max_sync(kFull, sh.best[lane & (kWarps - 1)]);
    if constexpr (SPLIT) {
      if (threadIdx.x == 0) sh.pub[turn][0] = a;
      cluster.sync();
      a = __reduce_max_sync(
          kFull, (uint32_t)cluster.map_shared_rank(&sh, lane < parts ? lane : 0)->pub[turn][0]);
      turn ^= 1;
    } else {
      __syncthreads();
    }
    return a;
  }
};

// A part of a row.
template <int DT>
struct Part {
  Row<DT> row;
  int j0, j1;  // its pieces
  __device__ __forceinline__ int steps() const { return (j1 - j0 + kStep - 1) / kStep; }
  // First piece of this thread's batch in step `it`; its pieces are 32 apart.
  __device__ __forceinline__ int first(int it) const {
    return j0 + it * kStep + (int)(threadIdx.x >> 5) * kWarpStep + (int)(threadIdx.x & 31);
  }
  __device__ __forceinline__ void load(uint4 (&q)[kBatch], int it) const {
    const int jw = j0 + it * kStep + (int)(threadIdx.x >> 5) * kWarpStep;
    const int j = jw + (int)(threadIdx.x & 31);
    if (jw * Row<DT>::N >= row.head && jw + kWarpStep <= j1 &&
        (jw + kWarpStep) * Row<DT>::N - row.head <= row.V) {
      const char* p = row.base + (size_t)j * 16;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) q[b] = ld_coherent16(p + b * 512);
    } else {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) q[b] = row.load(j + b * 32, j1);
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (row.partial(j + b * 32, j1)) q[b] = row.load_partial(j + b * 32);
    }
  }
};

// Largest logit of a batch, NaN if there is one.
template <int DT>
__device__ __forceinline__ float batch_max_nan(const uint4 (&q)[kBatch]) {
  if constexpr (DT == SPEC_BF16) {
    __nv_bfloat162 m[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      m[b] = __hmax2_nan(__hmax2_nan(as_bf2(q[b].x), as_bf2(q[b].y)),
                         __hmax2_nan(as_bf2(q[b].z), as_bf2(q[b].w)));
#pragma unroll
    for (int b = 1; b < kBatch; ++b) m[0] = __hmax2_nan(m[0], m[b]);
    const uint32_t w = as_word(m[0]);
    return max_nan(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      m = max_nan(m, max_nan(__uint_as_float(q[b].x), __uint_as_float(q[b].y)));
      m = max_nan(m, max_nan(__uint_as_float(q[b].z), __uint_as_float(q[b].w)));
    }
    return m;
  }
}

// Smallest logit of a batch (NaN ignored).
template <int DT>
__device__ __forceinline__ float batch_min(const uint4 (&q)[kBatch]) {
  float low;
  if constexpr (DT == SPEC_BF16) {
    __nv_bfloat162 m = as_bf2(q[0].x);
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      m = __hmin2(__hmin2(__hmin2(m, as_bf2(q[b].x)), __hmin2(as_bf2(q[b].y), as_bf2(q[b].z))),
                  as_bf2(q[b].w));
    const uint32_t w = as_word(m);
    low = fminf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  } else {
    low = INFINITY;
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      low = fminf(fminf(low, fminf(__uint_as_float(q[b].x), __uint_as_float(q[b].y))),
                  fminf(__uint_as_float(q[b].z), __uint_as_float(q[b].w)));
  }
  return low;
}

// Tokens of a batch above -inf.
template <int DT>
__device__ __forceinline__ uint32_t count_finite(const uint4 (&q)[kBatch]) {
  constexpr int N = Row<DT>::N;
  if (batch_min<DT>(q) > -INFINITY) return kBatch * N;
  uint32_t n = 0;
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    float x[N];
    unpack<DT>(q[b], x);
#pragma unroll
    for (int i = 0; i < N; ++i) n += x[i] > -INFINITY;
  }
  return n;
}

// ------------------------------------------------------------------------------ passes over a row

// Mass of a warp's step into its segment, if SEG.
template <bool SEG>
__device__ __forceinline__ void add_segment(Shared& sh, int it, u64 s) {
  if constexpr (SEG) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    if ((threadIdx.x & 31) == 0) sh.seg[it * kWarps + (threadIdx.x >> 5)] = s;
  }
}

// Mass of the whole part; with SEG those of its segments.
template <int DT, bool SEG>
__device__ __noinline__ u64 pass_all(Shared& sh, const Part<DT> part, const Weigher wt) {
  constexpr int N = Row<DT>::N;
  const int n = part.steps();
  const float least = wt.surely();
  u64 mass = 0;
  uint4 q[kBatch];
  part.load(q, 0);
  for (int it = 0; it < n; ++it) {
    uint4 now[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) now[b] = q[b];
    if (it + 1 < n) part.load(q, it + 1);
    u64 s = 0;
    if (__all_sync(kFull, batch_min<DT>(now) >= least)) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        float x[N];
        unpack<DT>(now[b], x);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          u64 h0, h1;
          wt.template halves<DT>(x[i], x[i + 1], h0, h1);
          s += h0;
          s += h1;
        }
      }
      s = 2 * s + kBatch * N;
    } else {
#pragma unroll 1
      for (int b = 0; b < kBatch; ++b) {
        float x[N];
        uint4 w = now[0];
#pragma unroll
        for (int i = 1; i < kBatch; ++i)
          if (b == i) w = now[i];
        unpack<DT>(w, x);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          u64 v0, v1;
          wt.template pair<DT>(x[i], x[i + 1], v0, v1);
          s += v0;
          s += v1;
        }
      }
    }
    add_segment<SEG>(sh, it, s);
    mass += s;
  }
  return mass;
}

// About the mass of the whole part, in units of 2^-40, and its tokens by their mass. fp32 sums of 16
// approximate exponentials: off by at most kSlack, of which (x - m) c in one product is 2^-18 (its
// error is 3 * 2^-24 ln2 of y, whose mean over the mass is at most log2 V).
constexpr float kSlack = 0x1p-17f;
template <int DT>
__device__ __noinline__ u64 pass_guess(Shared& sh, const Part<DT> part, const Weigher wt) {
  using namespace tc;
  constexpr int N = Row<DT>::N;
  const u64 m2 = pack2(wt.m, wt.m), n1 = pack2(-1.0f, -1.0f), ch2 = pack2(wt.ch, wt.ch);
  const int n = part.steps();
  u64 mass = 0;
  uint4 q[kBatch];
  part.load(q, 0);
  for (int it = 0; it < n; ++it) {
    uint4 now[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) now[b] = q[b];
    if (it + 1 < n) part.load(q, it + 1);
    u64 s = pack2(0.0f, 0.0f);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      float x[N];
      unpack<DT>(now[b], x);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const u64 y = mul2(fma2(pack2(x[i], x[i + 1]), n1, m2), ch2);
        float y0, y1, t0, t1;
        unpack2(y, y0, y1);
        unpack2(fma2(y, n1, pack2(kMagic, kMagic)), t0, t1);
        s = add2(s, pack2(fast_exp2(-y0), fast_exp2(-y1)));
        const uint32_t b0 = Weigher::bin(t0), b1 = Weigher::bin(t1);
        atomicAdd(&sh.bins[b0], 1u);
        atomicAdd(&sh.bins[b1], 1u);
        if (b == 0 && i == 0) {
          // 32 y less the bin, in 1/128, from 0 on: a logit in eight tells where a bin's tokens lie
          const float r = __fadd_rn(__fsub_rn(t0, kMagic), y0);
          atomicAdd(&sh.off[b0], (uint32_t)(__float2int_rn(r * 4096.0f) + 64));
          atomicAdd(&sh.offs[b0], 1u);
        }
      }
    }
    float s0, s1;
    unpack2(s, s0, s1);
    mass += __float2ull_rn((s0 + s1) * 0x1p40f);
  }
  return mass;
}

// Mass (MASS) and number of the part's tokens that a cut leaves; with SEG the masses of its
// segments, too.
template <int DT, bool MASS, bool SEG>
__device__ __noinline__ void pass(Shared& sh, const Part<DT> part, const Weigher wt, u64 key,
                                  u64& mass, u64& count) {
  constexpr int N = Row<DT>::N;
  const Cut cut(key);
  const int n = part.steps();
  mass = 0;
  uint32_t c = 0;
  uint4 q[kBatch];
  part.load(q, 0);
  for (int it = 0; it < n; ++it) {
    const int j = part.first(it);
    uint4 now[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) now[b] = q[b];
    if (it + 1 < n) part.load(q, it + 1);
    u64 s = 0;
    if (__any_sync(kFull, batch_max_nan<DT>(now) >= cut.x)) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        float x[N];
        unpack<DT>(now[b], x);
        const int v = (j + b * 32) * N - part.row.head;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          const bool in0 = cut.leaves(x[i], v + i), in1 = cut.leaves(x[i + 1], v + i + 1);
          c += in0 + in1;
          if constexpr (MASS) {
            u64 v0, v1;
            wt.template pair<DT>(in0 ? x[i] : -INFINITY, in1 ? x[i + 1] : -INFINITY, v0, v1);
            s += v0;
            s += v1;
          }
        }
      }
    }
    add_segment<SEG>(sh, it, s);
    mass += s;
  }
  count = c;
}

// Mass and number of the part's tokens of logits >= hi, the masses of its segments of these, and the
// part's whole mass; tokens from lo to hi go on the list.
template <int DT>
__device__ __noinline__ void pass_window(Shared& sh, const Part<DT> part, const Weigher wt, float lo,
                                         float hi, u64& mass, u64& count, u64& all) {
  constexpr int N = Row<DT>::N;
  const int n = part.steps();
  const float least = wt.surely();
  mass = all = 0;
  uint32_t c = 0;
  uint4 q[kBatch];
  part.load(q, 0);
  for (int it = 0; it < n; ++it) {
    const int j = part.first(it);
    uint4 now[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) now[b] = q[b];
    if (it + 1 < n) part.load(q, it + 1);
    u64 s = 0, z = 0;
    const bool fast = __all_sync(kFull, batch_min<DT>(now) >= least);
    uint32_t in = 0;  // of this batch
    // a piece at a time: the instructions of four do not stay near the issue (2048 flat rows at p 0.95
    // 829 us against 753)
#pragma unroll 1
    for (int b = 0; b < kBatch; ++b) {
      float x[N], below = -INFINITY;  // the largest logit below hi
      uint4 w = now[0];
#pragma unroll
      for (int i = 1; i < kBatch; ++i)
        if (b == i) w = now[i];
      unpack<DT>(w, x);
      if (fast) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          u64 h0, h1;
          wt.template halves<DT>(x[i], x[i + 1], h0, h1);
          z += h0;
          z += h1;
          const bool in0 = x[i] >= hi, in1 = x[i + 1] >= hi;
          if (in0) {
            s += h0;
            ++in;
          }
          if (in1) {
            s += h1;
            ++in;
          }
          below = max3f(below, in0 ? -INFINITY : x[i], in1 ? -INFINITY : x[i + 1]);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < N; ++i) {
          float one = x[0];
#pragma unroll
          for (int q = 1; q < N; ++q)
            if (q == i) one = x[q];
          const u64 v = wt.template operator()<DT>(one);
          z += v;
          if (one >= hi) {
            s += v;
            ++in;
          } else {
            below = fmaxf(below, one);
          }
        }
      }
      if (below >= lo) {
        uint32_t win = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) win |= (uint32_t)(x[i] < hi && x[i] >= lo) << i;
        int at = atomicAdd(&sh.n_list, __popc(win));
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (win >> i & 1) {
            if (at < kList)
              sh.keys[at] = make_key(order_bits(x[i]), (j + b * 32) * N - part.row.head + i);
            ++at;
          }
      }
    }
    c += in;
    if (fast) {
      s = 2 * s + in;
      z = 2 * z + kBatch * N;
    }
    all += z;
    add_segment<true>(sh, it, s);
    mass += s;
  }
  count = c;
}

// ------------------------------------------------------------------------------ the list

// A bound that at least k of this CTA's tokens reach, and not many more where it can be had: the k-th
// largest of its threads' largest logits, or, for a larger k, about that of the index entries.
__device__ __noinline__ uint32_t index_bound(Shared& sh, int groups, int k, uint32_t top) {
  const int tid = threadIdx.x;
  uint32_t e[kGroupsMost], mine = 0;
#pragma unroll
  for (int g = 0; g < kGroupsMost; ++g) {
    e[g] = g < groups ? sh.index[g * kThreads + tid] : 0;
    mine = e[g] > mine ? e[g] : mine;
  }
  if (k <= kTopsMost) {
    uint32_t lo = 1, hi = top;  // lo is enough, or all there are
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2 + 1;
      const int n = __syncthreads_count(mine >= mid);
      if (n < k) {
        hi = mid - 1;
      } else {
        lo = mid;
        if (n <= k + k / 8) break;
      }
    }
    return lo;
  }
  // three pivots a step
  uint32_t lo = 1, hi = top;  // hi + 1 is more than every entry; lo is enough, or all there are
  uint32_t* part = reinterpret_cast<uint32_t*>(sh.red);
  for (int turn = 0; lo < hi; turn ^= 1) {
    const uint32_t q = (hi - lo) / 4 + 1;
    const uint32_t p1 = lo + q, p2 = p1 + q < hi ? p1 + q : hi, p3 = p2 + q < hi ? p2 + q : hi;
    uint32_t n = 0;
#pragma unroll
    for (int g = 0; g < kGroupsMost; ++g)
      n += (uint32_t)(e[g] >= p1) + ((uint32_t)(e[g] >= p2) << 10) +
           ((uint32_t)(e[g] >= p3) << 20);
    const uint32_t n1 = __reduce_add_sync(kFull, n & 1023u),
                   n2 = __reduce_add_sync(kFull, n >> 10 & 1023u),
                   n3 = __reduce_add_sync(kFull, n >> 20);
    if ((tid & 31) < 3)
      part[(turn * 3 + (tid & 31)) * kWarps + (tid >> 5)] =
          (tid & 31) == 0 ? n1 : (tid & 31) == 1 ? n2 : n3;
    __syncthreads();
    int c1 = 0, c2 = 0, c3 = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      c1 += (int)part[(turn * 3 + 0) * kWarps + w];
      c2 += (int)part[(turn * 3 + 1) * kWarps + w];
      c3 += (int)part[(turn * 3 + 2) * kWarps + w];
    }
    int got;
    if (c3 >= k) {
      lo = p3;
      got = c3;
    } else if (c2 >= k) {
      lo = p2;
      hi = p3 - 1;
      got = c2;
    } else if (c1 >= k) {
      lo = p1;
      hi = p2 - 1;
      got = c1;
    } else {
      hi = p1 - 1;
      continue;
    }
    if (got <= k + k / 8) break;
  }
  __syncthreads();
  return lo;
}

template <bool SPLIT>
__device__ __noinline__ int gather(Team<SPLIT>& team);

// Tokens of bits >= bound of the whole row in the leader's list. Returns how many there are; more
// than kList means that they are not all there. The batches that reach the bound are listed, then
// their pieces dealt to the lanes.
template <int DT, bool SPLIT>
__device__ __noinline__ int collect(Team<SPLIT>& team, const Part<DT>& part, int per_group,
                                    uint32_t bound) {
  constexpr int N = Row<DT>::N;
  constexpr int kAtOnce = 4;  // pieces in flight
  Shared& sh = team.sh;
  const int tid = threadIdx.x;
  if (tid == 0) sh.n_list = sh.n_hits = 0;
  __syncthreads();
  const int n = part.steps(), groups = (n + per_group - 1) / per_group;
  // few reach it: a counter update each
#pragma unroll 4
  for (int g = 0; g < groups; ++g)
    if (sh.index[g * kThreads + tid] >= bound) {
      const int at = atomicAdd(&sh.n_hits, 1);
      if (at < kHits) sh.hits[at] = (uint16_t)(g * kThreads + tid);
    }
  __syncthreads();
  const int hits = sh.n_hits;
  if (hits <= kHits) {
    const float least = order_value(bound > 0x00800000u ? bound : 0x00800000u);
    const int pieces = hits * per_group * kBatch;
    for (int base = tid; base < pieces; base += kThreads * kAtOnce) {
      uint4 q[kAtOnce];
      int j[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int at = base + i * kThreads;
        if (i && at >= pieces) break;
        const int batch = at / kBatch, entry = sh.hits[per_group == 1 ? batch : batch / per_group];
        const int t = entry % kThreads;
        const int it = per_group == 1 ? entry / kThreads
                                      : entry / kThreads * per_group + batch % per_group;
        j[i] = part.j0 + it * kStep + (t >> 5) * kWarpStep + (t & 31) + at % kBatch * 32;
        q[i] = part.row.load(j[i], part.j1);
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (i && base + i * kThreads >= pieces) break;
        if (part.row.partial(j[i], part.j1)) q[i] = part.row.load_partial(j[i]);
        float x[N];
        unpack<DT>(q[i], x);
        uint32_t in = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) in |= (uint32_t)(x[e] >= least) << e;
        if (!in) continue;
        int at = atomicAdd(&sh.n_list, __popc(in));
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (in >> e & 1) {
            if (at < kList) sh.keys[at] = make_key(order_bits(x[e]), j[i] * N - part.row.head + e);
            ++at;
          }
      }
    }
  } else if (tid == 0) {
    sh.n_list = kList + 1;
  }
  __syncthreads();
  return gather<SPLIT>(team);
}

// The parts' lists behind one another in the leader's. Returns the number of keys, as collect does.
template <bool SPLIT>
__device__ int gather(Team<SPLIT>& team) {
  Shared& sh = team.sh;
  if constexpr (SPLIT) {
    team.cluster.sync();
    const int lane = threadIdx.x & 31;
    int before = team.cluster.map_shared_rank(&sh, lane < team.parts ? lane : 0)->n_list;
    const int total = __reduce_add_sync(kFull, lane < team.parts ? before : 0);
    before = __reduce_add_sync(kFull, lane < team.part ? before : 0);
    if (total <= kList && team.part) {
      u64* to = team.leader()->keys + before;
      for (int i = threadIdx.x; i < sh.n_list; i += kThreads) to[i] = sh.keys[i];
    }
    team.cluster.sync();
    return total;
  }
  return sh.n_list;
}

// Descending order of sh.keys[0 .. n), n <= kThreads, by counting the larger ones.
__device__ __noinline__ void sort_keys(Shared& sh, int n) {
  const int tid = threadIdx.x;
  const u64 key = tid < n ? sh.keys[tid] : 0;
  int place = 0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) place += sh.keys[i] > key;
  __syncthreads();
  if (tid < n) sh.keys[place] = key;
  __syncthreads();
}

// Exclusive prefix over the CTA's threads, and the sum.
__device__ __noinline__ u64 scan(Shared& sh, u64 v, u64& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh.red[0][warp] = x;
  __syncthreads();
  u64 before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh.red[0][w];
    total += sh.red[0][w];
  }
  __syncthreads();
  return before + x - v;
}

// The key of the c-th token, in order of the ids, whose order_bits are `bits`: its segment by a pass
// that counts, then its place in there. There are at least c.
template <int DT, bool SPLIT>
__device__ __noinline__ u64 nth_equal(Team<SPLIT>& team, const Part<DT>& part, uint32_t bits, u64 c) {
  constexpr int N = Row<DT>::N;
  Shared& sh = team.sh;
  const int tid = threadIdx.x, lane = tid & 31, n = part.steps();
  const float value = order_value(bits);
  u64 own = 0;
  __syncthreads();  // the index may have been read until now
  for (int it = 0; it < n; ++it) {
    uint4 q[kBatch];
    part.load(q, it);
    uint32_t in = 0;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      float x[N];
      unpack<DT>(q[b], x);
#pragma unroll
      for (int i = 0; i < N; ++i) in += x[i] == value;
    }
    own += in;
    in = __reduce_add_sync(kFull, in);
    if (lane == 0) sh.seg[it * kWarps + (tid >> 5)] = in;
  }
  const auto all = team.sum(own, 0);
  uint32_t found = 0;
  if (all.before < c && c <= all.before + all.own) {
    const int segs = n * kWarps, per = (segs + kThreads - 1) / kThreads, first = tid * per;
    const u64 at = c - 1 - all.before;
    u64 mine = 0, t;
    for (int i = first; i < min(segs, first + per); ++i) mine += sh.seg[i];
    u64 before = scan(sh, mine, t);
    if (before <= at && at < before + mine) {
      int i = first;
      for (; before + sh.seg[i] <= at; ++i) before += sh.seg[i];
      sh.hit = i;
      sh.rest = at - before;
    }
    __syncthreads();
    if (tid < 32) {
      int rest = (int)sh.rest;
      const int base = part.j0 + sh.hit * kWarpStep;
      for (int b = 0; b < kBatch; ++b) {
        const int j = base + b * 32 + lane;
        float x[N];
        unpack<DT>(part.row.load_any(j, part.j1), x);
        uint32_t in = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) in |= (uint32_t)(x[i] == value) << i;
        const int here = __popc(in);
        int up = here;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kFull, up, o);
          if (lane >= o) up += y;
        }
        int skip = rest - (up - here);  // of this lane's
        if (skip >= 0 && skip < here) {
          for (; skip; --skip) in &= in - 1;
          found = 0xffffffffu - (uint32_t)(j * N - part.row.head + __ffs(in) - 1);
        }
        rest -= __shfl_sync(kFull, up, 31);
        if (rest < 0) break;  // uniform
      }
    }
  }
  return (u64)bits << 32 | team.max(found);
}

// The largest key that leaves a mass of at least `least` among what `limit` leaves: by halving over the
// logits, a pass a step, from a guess (sh.lo_bits .. sh.hi_bits, which may be wrong) where it holds;
// then by counting the equal ones.
template <int DT, bool SPLIT>
__device__ __noinline__ u64 search(Team<SPLIT>& team, const Part<DT>& part, const Weigher& wt,
                                   u64 limit, u64 least, u64 top_key) {
  auto mass = [&](u64 key) {
    u64 m, c;
    pass<DT, true, false>(team.sh, part, wt, key > limit ? key : limit, m, c);
    return team.sum(m, c).a;
  };
  constexpr int kLow = DT == SPEC_BF16 ? 16 : 0;  // order_bits of a bf16 end in 16 zeros or ones
  constexpr uint32_t kLeast = 0x00800000u >> kLow;  // of the lowest finite number
  uint32_t lo = (uint32_t)(limit >> 32) >> kLow, hi = ((uint32_t)(top_key >> 32) >> kLow) + 1;
  lo = lo > kLeast ? lo : kLeast;
  uint32_t guess[2] = {(team.sh.hi_bits >> kLow) + (kLow ? 1u : 0u), team.sh.lo_bits >> kLow};
  for (int i = 0; hi - lo > 1; ++i) {
    uint32_t mid = i < 2 ? guess[i] : lo + (hi - lo) / 2;
    if (i < 2 && !(lo < mid && mid < hi)) continue;
    if (mass((u64)(mid << kLow) << 32) >= least)
      lo = mid;
    else
      hi = mid;
  }
  uint32_t bits = lo << kLow;
  if (DT == SPEC_BF16 && !(bits & 0x80000000u)) bits |= 0xffffu;
  const u64 larger = mass((u64)(bits + 1) << 32);
  const u64 each = wt.template operator()<DT>(order_value(bits));
  const u64 key = nth_equal<DT, SPLIT>(team, part, bits, (least - larger + each - 1) / each);
  return key > limit ? key : limit;
}

__device__ __forceinline__ float key_value(u64 key) { return order_value((uint32_t)(key >> 32)); }
__device__ __forceinline__ int key_id(u64 key) { return (int)(0xffffffffu - (uint32_t)key); }

// The k-th token by ten leading bits of order_bits at a time: sh.lo_bits .. sh.hi_bits - 1, of which
// there are sh.n_window, hold it, behind sh.n_above of larger ones. It ends as soon as they fit the
// list; equal logits that do not are left. False if fewer than k tokens have a place.
template <int DT, bool SPLIT>
__device__ __noinline__ bool find_kth(Team<SPLIT>& team, const Part<DT>& part, uint32_t k) {
  constexpr int N = Row<DT>::N, kDigit = 1024;
  static_assert(kDigit <= kBins && kDigit % kThreads == 0, "a digit's bins");
  Shared& sh = team.sh;
  const int tid = threadIdx.x, n = part.steps();
  uint32_t prefix = 0, above = 0;
  // digits of 10, 10, 10 and 2 bits
  for (int shift = 22, bits = 10;;) {
    for (int i = tid; i < kDigit; i += kThreads) sh.bins[i] = 0;
    __syncthreads();
    for (int it = 0; it < n; ++it) {
      uint4 q[kBatch];
      part.load(q, it);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        float x[N];
        unpack<DT>(q[b], x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t u = order_bits(x[i]);
          if (u && (shift == 22 || u >> (shift + bits) == prefix))
            atomicAdd(&sh.bins[(u >> shift) & ((1u << bits) - 1)], 1u);
        }
      }
    }
    team.sync();
    // thread t has the values kPer t .. kPer t + kPer - 1
    constexpr int kPer = kDigit / kThreads;
    uint32_t c[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c[i] = 0;
      if constexpr (SPLIT) {
        for (int q = 0; q < team.parts; ++q)
          c[i] += team.cluster.map_shared_rank(&sh, q)->bins[tid * kPer + i];
      } else {
        c[i] = sh.bins[tid * kPer + i];
      }
      mine += c[i];
    }
    u64 total;
    const u64 before = scan(sh, mine, total);
    uint32_t larger = above + (uint32_t)(total - before) - mine;  // behind this thread's values
    if (tid == 0) sh.in = -1;
    __syncthreads();
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i) {
      if (larger < k && k <= larger + c[i]) {
        sh.in = (int)c[i];
        sh.hit = tid * kPer + i;
        sh.n_above = (int)larger;
      }
      larger += c[i];
    }
    team.sync();  // every part has been read
    const int in = sh.in;
    if (in < 0) return false;
    above = (uint32_t)sh.n_above;
    prefix = prefix << bits | (uint32_t)sh.hit;
    __syncthreads();
    if (in <= kListMost || shift == 0) {
      if (tid == 0) {
        const uint32_t lo = prefix << shift;
        sh.lo_bits = lo > 0x00800000u ? lo : 0x00800000u;
        sh.hi_bits = (prefix + 1) << shift;
        sh.n_window = in;
      }
      __syncthreads();
      return true;
    }
    bits = shift < 10 ? shift : 10;
    shift -= bits;
  }
}

// order_bits of about the least logit of bin b.
__device__ __forceinline__ uint32_t edge_bits(const Weigher& wt, int b) {
  const float x = wt.m - ((float)b + 0.5f) / 32.0f / wt.ch;
  const uint32_t bits = x > -INFINITY ? order_bits(x) : 1;
  return bits > 0x00800000u ? bits : 0x00800000u;  // of the lowest finite number
}

// The largest key of the list's n that leaves, with the larger ones, a mass (or number) of at least
// `need` among those from `limit` on: by 256 ranges of the keys, then within one.
template <int DT>
__device__ __noinline__ u64 pick(Shared& sh, const Weigher& wt, int n, u64 limit, u64 need,
                                 bool by_mass, u64 lo, u64 hi) {
  const int tid = threadIdx.x;
  u64 *bucket = sh.picked[0], *some = sh.picked[1];
  while (true) {
    const int bits = 64 - __clzll((long long)(hi - lo)), shift = bits > 8 ? bits - 8 : 0;
    const u64 from = lo > limit ? lo : limit;
    bucket[tid] = 0;
    __syncthreads();
    for (int base = 0; base < n; base += kThreads) {
      const u64 key = base + tid < n ? sh.keys[base + tid] : 0;
      const bool in = key >= from && key <= hi && key;
      const u64 w = by_mass ? wt.template operator()<DT>(in ? key_value(key) : -INFINITY) : 1;
      if (in && w) {
        // equal logits have equal masses and one range, until the ids are told apart: one addition
        // for all of a warp's (the few hundred tokens of a bf16 logit met on one counter otherwise)
        const uint32_t same = shift >= 32 ? __match_any_sync(__activemask(), (uint32_t)(key >> 32))
                                          : 1u << (tid & 31);
        if ((tid & 31) == __ffs(same) - 1)
          atomicAdd(&bucket[(key - lo) >> shift], w * (u64)__popc(same));
      }
    }
    __syncthreads();
    const u64 v = bucket[tid];
    u64 total;
    const u64 before = scan(sh, v, total), above = total - before - v;
    if (above < need && need <= above + v) {
      sh.hit = tid;
      sh.rest = need - above;
      sh.done = 0;
    }
    __syncthreads();
    need = sh.rest;
    lo += (u64)sh.hit << shift;
    const u64 end = lo + ((1ull << shift) - 1);
    hi = end < hi ? end : hi;
    if (shift == 0) return lo;
    const u64 first = lo > limit ? lo : limit;
    for (int i = tid; i < n; i += kThreads) {
      const u64 key = sh.keys[i];
      if (key < first || key > hi) continue;
      const int at = atomicAdd(&sh.done, 1);
      if (at < kThreads) some[at] = key;
    }
    __syncthreads();
    const int m = sh.done;
    if (m <= kThreads) {
      const u64 key = tid < m ? some[tid] : 0;
      const u64 w = by_mass ? wt.template operator()<DT>(tid < m ? key_value(key) : -INFINITY) : 1;
      bucket[tid] = w;
      __syncthreads();
      u64 larger = 0;
      for (int i = 0; i < m; ++i)
        if (some[i] > key) larger += bucket[i];
      if (tid < m && larger < need && need <= larger + w) sh.limit = key;
      __syncthreads();
      return sh.limit;
    }
    __syncthreads();
  }
}

// Mass and number of the list's keys from `limit` on.
template <int DT>
__device__ __noinline__ u64 list_mass(Shared& sh, const Weigher& wt, int n, u64 limit, int& count) {
  u64 mine = 0, total;
  int c = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + threadIdx.x;
    const u64 key = i < n ? sh.keys[i] : 0;
    const bool in = key && key >= limit;
    c += in;
    mine += wt.template operator()<DT>(in ? key_value(key) : -INFINITY);
  }
  scan(sh, mine, total);
  c = __reduce_add_sync(kFull, c);
  if ((threadIdx.x & 31) == 0) sh.red[1][threadIdx.x >> 5] = (u64)c;
  __syncthreads();
  count = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) count += (int)sh.red[1][w];
  __syncthreads();
  return total;
}

// The three rules on the n keys of the list, of which top-k leaves nk, in one CTA: sh.kept of them,
// of sh.total mass, stay, those from sh.limit on. `all` is the mass that p refers to where that is
// not the nk tokens' own (0), to within `slack`; the list may begin behind a mass of `above`. kNo if
// the nucleus ends before or behind the list, which holds every token of bits >= bound (and before
// that, unless `above`), kUnsure if the slack decides where, or if min-p leaves none of the list. No
// key is above last_key. Up to kThreads keys are left in descending order.
enum : int { kNo = 0, kYes = 1, kUnsure = 2 };
template <int DT>
__device__ __noinline__ int rules(Shared& sh, const Weigher& wt, int n, int nk, u64 all, u64 slack,
                                  u64 above, uint32_t bound, u64 last_key) {
  const bool by_p = sh.p < 1.0f;
  const int tid = threadIdx.x;
  if (n > kThreads) {
    const u64 lo = (u64)bound << 32;
    // all of the list: not all of the row, which is what 0 leaves
    u64 limit = nk < n ? pick<DT>(sh, wt, n, 0, (u64)nk, false, lo, last_key)
                       : (u64)(bound > 0x00800000u ? bound : 0x00800000u) << 32;
    int kept;
    u64 mass = list_mass<DT>(sh, wt, n, limit, kept);
    const u64 key_m = sh.tm > 1 ? (u64)sh.tm << 32 : 0;
    if (by_p) {
      const u64 base = all ? all : mass;
      u64 need = exact_share(sh.p, base - slack, true), most = exact_share(sh.p, base + slack, true);
      if (above && need <= above) return kNo;
      need -= above;
      most -= above;
      if (mass < most && all && sh.tm < bound) return kNo;
      if (need && need <= mass) {
        const u64 key = pick<DT>(sh, wt, n, limit, need, true, lo, last_key);
        limit = key;
        mass = list_mass<DT>(sh, wt, n, limit, kept);
        // this token also ends the nucleus of a larger need
        if (mass < most && key_m <= key) return kUnsure;
      }
    }
    if (key_m > limit) {
      limit = key_m;
      mass = list_mass<DT>(sh, wt, n, limit, kept);
    }
    if (tid == 0) {
      sh.kept = kept;
      sh.total = mass;
      sh.limit = limit;
    }
    __syncthreads();
    return kept > 0 ? kYes : above ? kUnsure : kNo;
  }
  sort_keys(sh, n);
  const u64 key = tid < n ? sh.keys[tid] : 0;
  const u64 w = wt.template operator()<DT>(tid < nk ? key_value(key) : -INFINITY);
  u64 mass;
  const u64 before = scan(sh, w, mass);
  u64 need = ~0ull, most = ~0ull;
  if (by_p) {
    const u64 base = all ? all : mass;
    need = exact_share(sh.p, base - slack, true);
    most = exact_share(sh.p, base + slack, true);
    if (above && need <= above) return kNo;
    need -= above;
    most -= above;
    if (all && mass < most && sh.tm < bound) return kNo;
  }
  // each rule leaves a prefix; the first token always stays
  const bool other = tid < nk && (uint32_t)(key >> 32) >= sh.tm;
  const int kept = __syncthreads_count(tid == 0 || (other && before < need));
  if (slack && __syncthreads_count(tid == 0 || (other && before < most)) != kept) return kUnsure;
  if (tid == kept - 1) {
    sh.kept = kept;
    sh.total = before + w;
    sh.limit = key;
  }
  __syncthreads();
  return kYes;
}

// Where a share p of the mass of sh.bins (of every part) ends: bins sh.bin_lo .. sh.bin_hi, with
// the number of tokens before and in them. A bin's mass is its tokens' number times that of their mean
// (of those that were looked at; `again`: of the bin's middle), so the place is a guess, to be
// checked: the bins in which a share of p (1 -+ kSure) ends, or p alone where those do not fit the
// list. A token alone in its bin, which was not looked at, is off by up to 2^(1/64), so that a peaked
// row's place may be a token further: the window has at least kAtLeast tokens, larger ones included.
constexpr float kSure = 0.0005f;
constexpr uint32_t kAtLeast = 64;
template <bool SPLIT>
__device__ __noinline__ void find_window(Team<SPLIT>& team, const Weigher& wt, float p, bool again) {
  Shared& sh = team.sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __syncthreads();
  for (int at = tid; at < kBins; at += kThreads) {
    const uint32_t q = again ? 0 : sh.offs[at];
    const float off = q ? (float)sh.off[at] / (float)q * (1.0f / 128.0f) - 0.5f : 0.0f;
    sh.weight[at] = at == kBins - 1 ? 0.0f : (float)sh.bins[at] * fast_exp2((at + off) * -0.03125f);
  }
  // the cluster's bins: each part sums a share of them, then every part reads all shares
  const int share_bins = kBins / team.parts;
  if constexpr (SPLIT) {
    team.sync();
    float w[kBins / 2 / kThreads];
#pragma unroll
    for (int i = 0; i < kBins / 2 / kThreads; ++i) {
      const int at = tid + i * kThreads;
      uint32_t sum = 0;
      w[i] = 0.0f;
      if (at >= share_bins) continue;
      for (int q = 0; q < team.parts; ++q) {
        const Shared* o = team.cluster.map_shared_rank(&sh, q);
        sum += o->bins[team.part * share_bins + at];
        w[i] += o->weight[team.part * share_bins + at];
      }
      sh.slice[at] = sum;
      sh.shares[at] = w[i];
    }
  }
  team.sync();
  uint32_t n[kBinsThread], count = 0;
  float e[kBinsThread], mine = 0.0f;
#pragma unroll
  for (int i = 0; i < kBinsThread; ++i) {
    const int at = tid * kBinsThread + i;
    if constexpr (SPLIT) {
      const Shared* o = team.cluster.map_shared_rank(&sh, at / share_bins);
      n[i] = o->slice[at % share_bins];
      e[i] = o->shares[at % share_bins];
    } else {
      n[i] = sh.bins[at];
      e[i] = sh.weight[at];
    }
    if (at == kBins - 1) n[i] = 0;  // no mass
    mine += e[i];
    count += n[i];
  }
  float up = mine;
  uint32_t cup = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_up_sync(kFull, up, o);
    const uint32_t z = __shfl_up_sync(kFull, cup, o);
    if (lane >= o) {
      up += y;
      cup += z;
    }
  }
  if (lane == 31) {
    sh.fred[warp] = up;
    sh.red[0][warp] = cup;
  }
  if (tid < 4) {
    sh.edge[tid] = kBins - 1;
    sh.before[tid] = 0;
  }
  __syncthreads();
  float c = up - mine, total = 0.0f;
  uint32_t before = cup - count;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      c += sh.fred[w];
      before += (uint32_t)sh.red[0][w];
    }
    total += sh.fred[w];
  }
  // thread ranges follow one another, so the three places are each in one thread's
  const float share[3] = {total * p * (1.0f - kSure), total * p, total * p * (1.0f + kSure)};
#pragma unroll
  for (int i = 0; i < kBinsThread; ++i) {
    const float next = c + e[i];
#pragma unroll
    for (int q = 0; q < 3; ++q)
      if (n[i] && c < share[q] && next >= share[q]) {
        sh.edge[q] = tid * kBinsThread + i;
        sh.before[q] = (int)(q == 2 ? before + n[i] : before);  // up to the bin, or with it
        if (q < 2) sh.cum[q] = c / total;
        if (q == 1) sh.in = (int)n[i];
      }
    if (before < kAtLeast && before + n[i] >= kAtLeast) {
      sh.edge[3] = tid * kBinsThread + i;
      sh.before[3] = (int)(before + n[i]);
    }
    c = next;
    before += n[i];
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t all = 0;
    for (int w = 0; w < kWarps; ++w) all += (uint32_t)sh.red[0][w];
    if (sh.edge[2] == kBins - 1) sh.before[2] = (int)all;
    int lo = sh.edge[0], hi = sh.edge[2];
    sh.guess = sh.cum[0];
    sh.n_above = sh.before[0];
    sh.n_window = sh.before[2] - sh.before[0];
    if (hi < sh.edge[3] && sh.edge[3] < kBins - 1 && sh.before[3] <= kThreads) {
      hi = sh.edge[3];
      sh.n_window = sh.before[3] - sh.before[0];
    }
    if (sh.n_window > kListMost && sh.edge[1] < kBins - 1) {
      lo = hi = sh.edge[1];
      sh.guess = sh.cum[1];
      sh.n_above = sh.before[1];
      sh.n_window = sh.in;
    }
    sh.lo_bits = edge_bits(wt, hi);
    sh.hi_bits = lo ? edge_bits(wt, lo - 1) : 0xff800000u;  // infinity: nothing is above
  }
  team.sync();
}

// ------------------------------------------------------------------------------ outputs

__device__ __forceinline__ float log_mass(u64 mass, const Weigher& wt) {
  // mass / 2^(S + 1) as a pair
  const float hi = __ull2float_rn(mass);
  const long long rest = (long long)(mass - __float2ull_rz(hi));
  const float unit = ldexpf(1.0f, wt.shift - 62);
  return df_log(DF{hi * unit, __ll2float_rn(rest) * unit});
}

__device__ __forceinline__ void write_draw(const SampleArgs& a, int row, int id, float x,
                                           const Weigher& wt, float scale, u64 total, int kept) {
  a.tokens[row] = id;
  if (a.logp) a.logp[row] = (x - wt.m) * scale - log_mass(total, wt);
  if (a.kept) a.kept[row] = kept;
}

__device__ __forceinline__ u64 draw_at(const SampleArgs& a, float u, u64 total) {
  if (!(u >= 0.0f && u < 1.0f)) {
    atomicOr(a.status, SPEC_DEV_BAD_PARAM);
    if (u >= 1.0f) return total - 1;
    u = 0.0f;
  }
  return exact_share(u, total, false);
}

// The draw among the listed keys from sh.limit on: by 256 ranges of ids, then within one.
template <int DT>
__device__ __noinline__ void draw_list(Shared& sh, const SampleArgs& a, int row, float u,
                                       const Weigher& wt, float scale, int listed) {
  u64* bucket = sh.bucket;
  const int tid = threadIdx.x;
  if (listed <= kThreads) {  // every token that stays against every other
    const int n = sh.kept;
    const u64 key = tid < n ? sh.keys[tid] : 0;
    const u64 w = wt.template operator()<DT>(tid < n ? key_value(key) : -INFINITY);
    bucket[tid] = w;
    __syncthreads();
    u64 below = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i)
      if ((uint32_t)sh.keys[i] > (uint32_t)key) below += bucket[i];  // lower ids
    const u64 at = draw_at(a, u, sh.total);
    if (tid < n && below <= at && at < below + w)
      write_draw(a, row, key_id(key), key_value(key), wt, scale, sh.total, n);
    return;
  }
  int by = 0;
  while ((a.V - 1) >> by >= kBuckets) ++by;
  bucket[tid] = 0;
  __syncthreads();
  const u64 limit = sh.limit;
  for (int base = 0; base < listed; base += kThreads) {
    const int i = base + tid;
    const u64 key = i < listed ? sh.keys[i] : 0;
    const u64 w = wt.template operator()<DT>(key && key >= limit ? key_value(key) : -INFINITY);
    if (w) atomicAdd(&bucket[key_id(key) >> by], w);
  }
  __syncthreads();
  const u64 at = draw_at(a, u, sh.total), mine = bucket[tid];
  u64 t;
  const u64 before = scan(sh, mine, t);
  if (before <= at && at < before + mine) {
    sh.hit = tid;
    sh.rest = at - before;
  }
  __syncthreads();
  const int hit = sh.hit;
  const u64 rest = sh.rest;
  // this bucket's tokens, few of them, behind one another in place of the index
  u64* some = sh.seg;
  if (tid == 0) sh.done = 0;
  __syncthreads();
  for (int i = tid; i < listed; i += kThreads)
    if (sh.keys[i] >= limit && key_id(sh.keys[i]) >> by == hit)
      some[atomicAdd(&sh.done, 1)] = sh.keys[i];
  __syncthreads();
  const int m = sh.done;
  for (int base = 0; base < m; base += kThreads) {
    const bool in = base + tid < m;
    const u64 key = in ? some[base + tid] : 0;
    u64 below = 0;
    for (int q = 0; q < m; ++q) {
      const u64 w = wt.template operator()<DT>(key_value(some[q]));
      if (in && key_id(some[q]) < key_id(key)) below += w;
    }
    const u64 w = wt.template operator()<DT>(in ? key_value(key) : -INFINITY);
    if (in && below <= rest && rest < below + w)
      write_draw(a, row, key_id(key), key_value(key), wt, scale, sh.total, sh.kept);
  }
}

// The draw among all tokens that the cut leaves, from the segments' masses; in the CTA whose part
// holds it.
template <int DT>
__device__ __noinline__ void draw_segment(Shared& sh, const SampleArgs& a, int row,
                                          const Part<DT>& part, const Weigher& wt, float scale,
                                          u64 key, u64 at, u64 total, int kept) {
  constexpr int N = Row<DT>::N;
  const int n = part.steps() * kWarps, per = (n + kThreads - 1) / kThreads;
  const int first = threadIdx.x * per, lane = threadIdx.x & 31;
  u64 mine = 0, t;
  for (int i = first; i < min(n, first + per); ++i) mine += sh.seg[i];
  u64 before = scan(sh, mine, t);
  if (before <= at && at < before + mine) {
    int i = first;
    for (; before + sh.seg[i] <= at; ++i) before += sh.seg[i];
    sh.hit = i;
    sh.rest = at - before;
  }
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int base = part.j0 + sh.hit * kWarpStep;
  u64 rest = sh.rest;
  const Cut cut(key);
  uint4 q[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) q[b] = part.row.load(base + b * 32 + lane, part.j1);
#pragma unroll
  for (int b = 0; b < kBatch; ++b)
    if (part.row.partial(base + b * 32 + lane, part.j1))
      q[b] = part.row.load_partial(base + b * 32 + lane);
#pragma unroll 1
  for (int b = 0; b < kBatch; ++b) {
    const int j = base + b * 32 + lane;
    float x[N];
    uint4 now = q[0];
#pragma unroll
    for (int i = 1; i < kBatch; ++i)
      if (i == b) now = q[i];
    unpack<DT>(now, x);
    const int v = j * N - part.row.head;
    u64 w[N], s = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[i] = wt.template operator()<DT>(cut.leaves(x[i], v + i) ? x[i] : -INFINITY);
      s += w[i];
    }
    u64 up = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(kFull, up, o);
      if (lane >= o) up += y;
    }
    u64 c = up - s;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (c <= rest && rest < c + w[i])
        write_draw(a, row, v + i, x[i], wt, scale, total, kept);
      c += w[i];
    }
    const u64 all = __shfl_sync(kFull, up, 31);
    if (rest < all) break;  // uniform
    rest -= all;
  }
}

// The part with -inf where the cut does not leave a token (everything, where `copy`).
template <int DT>
__device__ __noinline__ void write_part(const SampleArgs& a, int row, const Part<DT>& part, u64 key,
                                        bool copy) {
  constexpr int N = Row<DT>::N;
  const Cut cut(key);
  const Row<DT> to(a.out, (size_t)row * a.ldo, a.V);
  char* base = const_cast<char*>(to.base);
  const bool same = to.head == part.row.head;
  const int n = part.steps();
  // what a bf16 above cut.x is above; one that equals it may be cut.x or not
  const __nv_bfloat162 at = __float2bfloat162_rn(__bfloat162float(__float2bfloat16_rd(cut.x)));
  for (int it = 0; it < n; ++it) {
    uint4 q[kBatch];
    part.load(q, it);
    const int j = part.first(it);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int v = (j + b * 32) * N - part.row.head;
      uint32_t w[4] = {q[b].x, q[b].y, q[b].z, q[b].w};
      bool even = !copy;  // whether the logits decide, without the ids
      if constexpr (DT == SPEC_BF16) {
        uint32_t equal = 0, o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t m = __hgt2_mask(as_bf2(w[i]), at);
          equal |= __heq2_mask(as_bf2(w[i]), at);
          o[i] = (w[i] & m) | (0xff80ff80u & ~m);
        }
        even = even && !equal;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (even) w[i] = o[i];
      } else {
        even = false;
      }
      if (!copy && !even) {
        float x[N];
        unpack<DT>(q[b], x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const bool in = cut.leaves(x[i], v + i);
          if constexpr (DT == SPEC_BF16) {
            if (!in) w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | 0xff800000u
                                      : (w[i / 2] & 0xffff0000u) | 0xff80u;
          } else {
            if (!in) w[i] = 0xff800000u;
          }
        }
      }
      if (j + b * 32 >= part.j1) continue;
      if (same && v >= 0 && v + N <= a.V) {
        __stcs(reinterpret_cast<uint4*>(base + (size_t)(j + b * 32) * 16),
               make_uint4(w[0], w[1], w[2], w[3]));
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (v + i < 0 || v + i >= a.V) continue;
          const size_t at = (size_t)(to.head + v + i);
          if constexpr (DT == SPEC_BF16)
            reinterpret_cast<uint16_t*>(base)[at] = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
          else
            reinterpret_cast<uint32_t*>(base)[at] = w[i];
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------ kernel

// The row's parameters, out of range ones replaced and flagged; by one thread.
__device__ __noinline__ void read_params(Shared& sh, const SampleArgs& a, int row) {
  const int at = row / a.rows_per_param;
  float T = a.temperature ? a.temperature[at] : a.temperature_all;
  int k = a.top_k ? a.top_k[at] : a.top_k_all;
  float p = a.top_p ? a.top_p[at] : a.top_p_all;
  float mp = a.min_p ? a.min_p[at] : a.min_p_all;
  bool bad = false;
  if (!(T >= 0.0f) || T == INFINITY) {
    T = 1.0f;
    bad = true;
  }
  if (p != p) {
    p = 1.0f;
    bad = true;
  }
  if (mp != mp) {
    mp = 0.0f;
    bad = true;
  }
  if (bad) atomicOr(a.status, SPEC_DEV_BAD_PARAM);
  const float inv = T > 0.0f ? 1.0f / T : INFINITY;
  const bool greedy = inv == INFINITY || p <= 0.0f || k == 1;
  const float scale = inv == INFINITY ? 1.0f : inv;
  // log2(e) / T in a pair; 1 / T near the largest number is cut so that the product is finite
  constexpr float kHi = 1.44269502162933349609f, kLo = 1.92596303350e-8f;
  const float sc = fminf(scale, 1.5e38f);
  sh.scale = scale;
  sh.ch = sc * kHi;
  sh.cl = fmaf(sc, kLo, fmaf(sc, kHi, -sh.ch));
  sh.k = greedy ? 1 : (k <= 0 || k >= a.V ? 0 : k);
  sh.p = p < 0.0f ? 0.0f : p;
  sh.by_m = mp > 0.0f;
  if (sh.by_m) sh.below = log((double)fminf(mp, 1.0f)) / (double)scale;
}

template <int DT, bool SPLIT, bool WRITE>
__global__ void __launch_bounds__(kThreads, kCtas) sample_kernel(const SampleArgs a, const int parts) {
  __shared__ Shared sh;
  Team<SPLIT> team(sh, parts);
  const int tid = threadIdx.x, lane = tid & 31;
  grid_dep_wait();
  int rows = a.rows;
  if (a.row_count) rows = min(rows, max(0, *a.row_count));
  Weigher wt;
  wt.table = kPowers[lane];
  int bits = 0;
  while ((1 << bits) < a.V) ++bits;
  const int S = min(46, 62 - bits);
  wt.shift = 61 - S;
  wt.most = (float)(S + 1);

  const int row = SPLIT ? blockIdx.x / parts : blockIdx.x;
  if (row >= rows) return;
  const float u = WRITE ? 0.0f : a.u[row];  // on its way while the logits are read
  {
    Part<DT> part{Row<DT>(a.x, (size_t)row * a.ld, a.V), 0, 0};
    {
      const int np = part.row.pieces(), per = (np + team.parts - 1) / team.parts;
      part.j0 = min(np, team.part * per);
      part.j1 = min(np, part.j0 + per);
    }
    const int steps = part.steps(), per_group = max(1, (steps + kGroupsMost - 1) / kGroupsMost);
    const int groups = (steps + per_group - 1) / per_group;

    // the largest logit, and those of the batches
    float m = -INFINITY;
    uint32_t finite = 0;  // tokens above -inf
    {
      uint4 q[2][kBatch];
      part.load(q[0], 0);
      part.load(q[1], 1);
      if (tid == 0) read_params(sh, a, row);
      float e = -INFINITY;
      int in = 0, g = 0;
      auto take = [&](const uint4 (&w)[kBatch]) {
        e = max_nan(e, batch_max_nan<DT>(w));
        finite += count_finite<DT>(w);
        if (++in == per_group) {
          sh.index[g++ * kThreads + tid] = order_bits(e);
          m = max_nan(m, e);
          e = -INFINITY;
          in = 0;
        }
      };
      for (int it = 0; it < steps; it += 2) {
        take(q[0]);
        part.load(q[0], it + 2);
        if (it + 1 < steps) take(q[1]);
        part.load(q[1], it + 3);
      }
      if (in) {
        sh.index[g * kThreads + tid] = order_bits(e);
        m = max_nan(m, e);
      }
    }
    // NaN comes out as the largest
    const uint32_t top = team.max(m != m ? ~0u : order_bits(m));
    if (top == ~0u || top == 0 || order_value(top) == INFINITY) {
      // no distribution: the largest logit's id, or 0
      u64 best = 0;
      for (int it = 0; it < steps; ++it)
        for (int b = 0; b < kBatch; ++b) {
          const int j = part.first(it) + b * 32;
          float x[Row<DT>::N];
          unpack<DT>(part.row.load_any(j, part.j1), x);
          for (int i = 0; i < Row<DT>::N; ++i) {
            const uint32_t o = order_bits(x[i]);
            const u64 key = o ? make_key(o, j * Row<DT>::N - part.row.head + i) : 0;
            best = key > best ? key : best;
          }
        }
      const uint32_t most = team.max((uint32_t)(best >> 32));
      const uint32_t low = team.max((uint32_t)(best >> 32) == most ? (uint32_t)best : 0);
      if (team.part == 0 && tid == 0) {
        atomicOr(a.status, SPEC_DEV_NONFINITE);
        if (a.tokens) a.tokens[row] = most ? (int)(0xffffffffu - low) : 0;
        if (a.logp) a.logp[row] = NAN;
        if (a.kept) a.kept[row] = 0;
        if (a.stats) a.stats[2 * (size_t)row] = a.stats[2 * (size_t)row + 1] = NAN;
      }
      if (WRITE) write_part<DT>(a, row, part, 0, true);
      team.sync();
      return;
    }
    const u64 top_key = (u64)top << 32 | 0xffffffffu;
    wt.m = order_value(top);
    wt.ch = sh.ch;
    wt.cl = sh.cl;
    const float scale = sh.scale;
    int k = sh.k;
    const bool by_p = sh.p < 1.0f;
    uint32_t tm = 1;
    if (sh.by_m) {  // the least fp32 number x with (x - m) / T >= log(min_p)
      float f = __double2float_ru((double)wt.m + sh.below);
      f = f < wt.m ? f : wt.m;
      if (f > -INFINITY) tm = order_bits(f);
      if (tid == 0) sh.tm = tm;
    } else if (tid == 0) {
      sh.tm = 1;
    }
    const bool by_m = tm > 1;

    u64 limit = 0, total = 0;
    int kept = 0;
    if (k == 1) {
      uint32_t best = 0;
      for (int g = 0; g < groups; ++g) {
        if (sh.index[g * kThreads + tid] != top) continue;
        for (int it = g * per_group; it < min(steps, (g + 1) * per_group); ++it)
          for (int b = 0; b < kBatch; ++b) {
            const int j = part.first(it) + b * 32;
            float x[Row<DT>::N];
            unpack<DT>(part.row.load_any(j, part.j1), x);
            for (int i = 0; i < Row<DT>::N; ++i)
              if (x[i] == wt.m)
                best = max(best, 0xffffffffu - (uint32_t)(j * Row<DT>::N - part.row.head + i));
          }
      }
      limit = (u64)top << 32 | team.max(best);
      kept = 1;
      total = 1ull << (S + 1);
      if (!WRITE && team.part == 0 && tid == 0)
        write_draw(a, row, key_id(limit), wt.m, wt, scale, total, 1);
    } else if (k || by_p || by_m) {
      u64 all = 0, slack = 0;  // the mass that p refers to, where that is not the list's
      uint32_t bound = tm;
      bool list = true, window = false, binned = k ? k > kListTop : by_p;
      if (k && !binned) {
        if constexpr (SPLIT) {
          // as many tokens in every part as make k together, or k in one
          bound = ~team.max(~index_bound(sh, groups, (k + team.parts - 1) / team.parts, top));
          if (bound == 1) bound = team.max(index_bound(sh, groups, k, top));
        } else {
          bound = index_bound(sh, groups, k, top);
        }
      }
      while (true) {
        if (k && binned && !find_kth<DT, SPLIT>(team, part, (uint32_t)k)) {
          k = 0;  // every token of the row
          binned = by_p;
          list = by_m;
          bound = tm;
          if (!by_p && !by_m) break;
        }
        if (k && binned) {
          list = sh.n_above + sh.n_window <= kListMost;
          window = !list && sh.n_window <= kListMost;
          bound = sh.lo_bits;
        } else if (binned) {
          for (int i = tid; i < kBins; i += kThreads) sh.bins[i] = sh.off[i] = sh.offs[i] = 0;
          __syncthreads();
          const u64 mass = team.sum(pass_guess<DT>(sh, part, wt), 0).a;
          find_window<SPLIT>(team, wt, sh.p, false);
          all = mass << (S + 1 - 40);
          slack = (u64)((float)all * kSlack);
          list = sh.n_above + sh.n_window <= kListMost;
          window = !list && sh.n_window <= kListMost;
          bound = sh.lo_bits;
          // min-p's last token is enough, and may be before where the nucleus seems to end
          if (tm > bound || !list) bound = tm;
          if (!list) list = by_m && tm >= sh.hi_bits;
        }
        if (list) {
          const int n = collect<DT, SPLIT>(team, part, per_group, bound);
          if (n <= kList) {
            int done = kNo;
            while (true) {
              if (team.part == 0) {
                const int is = k == 0 || k <= n || bound <= 0x00800000u
                                   ? rules<DT>(sh, wt, n, k && k < n ? k : n, all, slack, 0, bound,
                                               top_key)
                                   : kNo;
                if (tid == 0) sh.done = is;
              }
              team.sync();
              done = team.leader()->done;
              if (done != kUnsure) break;
              all = team.sum(pass_all<DT, false>(sh, part, wt), 0).a;
              slack = 0;
            }
            const Shared* lead = team.leader();
            if (done) {
              limit = lead->limit;
              total = lead->total;
              kept = lead->kept;
              if (SPLIT) team.sync();
              if (!WRITE && team.part == 0) draw_list<DT>(sh, a, row, u, wt, scale, n);
            }
          }
          // the guess was wrong: again with the mass that there is
          window = !kept && !k && binned && by_p && n <= kList && sh.n_window <= kListMost;
        }
        if (kept || !k || binned) break;
        binned = true;  // too many tokens of the k-th logit, or near it
      }
      bool of_k = false;  // whether `all` is the mass of top-k's tokens, those from `limit` on
      for (int turn = 0; !kept && window && turn < 3; ++turn) {
        // too many for the list: its piece around the border, the mass before it
        if (tid == 0) sh.n_list = 0;
        const uint32_t lo_bits = sh.lo_bits, hi_bits = sh.hi_bits;
        const u64 last_key = ((u64)hi_bits << 32) - 1;
        __syncthreads();
        u64 mm, cc, zz;
        pass_window<DT>(sh, part, wt, order_value(lo_bits), order_value(hi_bits), mm, cc, zz);
        const auto s = team.sum(mm, cc);
        const u64 whole = team.sum(zz, 0).a;
        if (!k && !of_k) all = whole;
        slack = 0;
        const int n = gather<SPLIT>(team), nk = k ? k - (int)s.b : n;
        window = n <= kList && nk > 0 && nk <= n;
        if (!window) break;
        if (team.part == 0) {
          int is = kNo;
          if (k && by_p) {  // the mass that p refers to comes first
            const u64 key = pick<DT>(sh, wt, n, 0, (u64)nk, false, (u64)lo_bits << 32, last_key);
            if (tid == 0) sh.limit = key;
          } else {
            is = rules<DT>(sh, wt, n, nk, all, 0, s.a, lo_bits, last_key);
            // min-p ends before the window, the other two do not
            if (is == kYes && (uint32_t)(sh.limit >> 32) < tm) is = kUnsure;
          }
          if (tid == 0) sh.done = is;
          // what stays of the list, into the segments
          if (is == kYes && !WRITE)
            for (int base = 0; base < n; base += kThreads) {
              const u64 key = base + tid < n ? sh.keys[base + tid] : 0;
              const bool in = key && key >= sh.limit;
              const u64 w = wt.template operator()<DT>(in ? key_value(key) : -INFINITY);
              if (!in) continue;
              const int j = (key_id(key) + part.row.head) / Row<DT>::N;
              const int per = part.j1 - part.j0, q = SPLIT ? j / per : 0;
              Shared* to = &sh;
              if constexpr (SPLIT) to = team.cluster.map_shared_rank(&sh, q);
              atomicAdd(&to->seg[(j - q * per) / kWarpStep], w);
            }
        }
        team.sync();
        const Shared* lead = team.leader();
        const int done = lead->done;
        if (done == kYes) {
          limit = lead->limit;
          total = s.a + lead->total;
          kept = (int)s.b + lead->kept;
          u64 own = 0;
          if (!WRITE)
            for (int i = tid; i < steps * kWarps; i += kThreads) own += sh.seg[i];
          const auto d = team.sum(own, 0);
          if (!WRITE) {
            const u64 at = draw_at(a, u, total);
            if (d.before <= at && at < d.before + d.own)
              draw_segment<DT>(sh, a, row, part, wt, scale, limit, at - d.before, total, kept);
          }
        } else if (done == kUnsure) {
          limit = (u64)tm << 32;
          break;
        } else if (k && by_p) {
          // the mass of top-k's tokens; its share ends where one of the row's mass does
          limit = lead->limit;
          pass<DT, true, false>(sh, part, wt, limit, mm, cc);
          all = team.sum(mm, cc).a;
          for (int i = tid; i < kBins; i += kThreads) sh.bins[i] = sh.off[i] = sh.offs[i] = 0;
          __syncthreads();
          pass_guess<DT>(sh, part, wt);
          find_window<SPLIT>(team, wt, sh.p * (float)((double)all / (double)whole), false);
          window = sh.n_window <= kListMost;
          of_k = true;
          turn = -1;
          k = 0;
        } else if (k) {
          window = false;
          team.sync();
        } else {
          // once more by the mass that there is before the window
          const float off = (float)((double)s.a / (double)whole) - sh.guess;
          const float share = of_k ? sh.p * (float)((double)all / (double)whole) : sh.p;
          __syncthreads();
          find_window<SPLIT>(team, wt, share - off, true);
          window = sh.n_window <= kListMost;
        }
      }
      const u64 key_m = (u64)tm << 32;
      if (!kept && !(by_m && limit == key_m)) {
        // the k-th token is one of many equal ones
        if (k && !limit)
          limit = nth_equal<DT, SPLIT>(team, part, sh.lo_bits, (u64)(k - sh.n_above));
        if (by_p) {
          if (!k && slack) all = team.sum(pass_all<DT, false>(sh, part, wt), 0).a;
          if (limit && !of_k) {
            u64 mm, cc;
            pass<DT, true, false>(sh, part, wt, limit, mm, cc);
            all = team.sum(mm, cc).a;
          }
          const u64 need = exact_share(sh.p, all, true);
          bool more = true;  // whether the nucleus may end before min-p's last token
          if (by_m) {
            u64 mm, cc;
            pass<DT, true, false>(sh, part, wt, key_m > limit ? key_m : limit, mm, cc);
            more = team.sum(mm, cc).a > need;
          }
          if (more) limit = search<DT, SPLIT>(team, part, wt, limit, need ? need : 1, top_key);
        }
        limit = by_m && key_m > limit ? key_m : limit;
      }
    }
    if (!kept) {
      u64 mm, cc;
      __syncthreads();
      if (limit) {
        pass<DT, true, true>(sh, part, wt, limit, mm, cc);
      } else {
        mm = pass_all<DT, !WRITE>(sh, part, wt);
        cc = finite;
      }
      const auto s = team.sum(mm, cc);
      total = s.a;
      kept = (int)s.b;
      if (!WRITE) {
        const u64 at = draw_at(a, u, total);
        if (s.before <= at && at < s.before + s.own)
          draw_segment<DT>(sh, a, row, part, wt, scale, limit, at - s.before, total, kept);
      }
    }
    if (WRITE) {
      write_part<DT>(a, row, part, limit, false);
      if (team.part == 0 && tid == 0) {
        if (a.kept) a.kept[row] = kept;
        if (a.stats) {
          a.stats[2 * (size_t)row] = wt.m * scale;
          a.stats[2 * (size_t)row + 1] = log_mass(total, wt);
        }
      }
    }
    team.sync();  // no part leaves before it has been read
  }
}

template <int DT, bool SPLIT, bool WRITE>
cudaError_t launch_t(const SampleArgs& a, int split, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = trace_active() ? 0 : 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.rows * split);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<DT, SPLIT, WRITE>, a, split);
}

template <int DT, bool WRITE>
cudaError_t launch_split(const SampleArgs& a, int split, cudaStream_t s) {
  return split > 1 ? launch_t<DT, true, WRITE>(a, split, s) : launch_t<DT, false, WRITE>(a, 1, s);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, int dt, cudaStream_t s) {
  TraceScope ts(SPEC_KCLASS_SELECT, s);
  const int batch = kStep * (dt == SPEC_BF16 ? 8 : 4);
  int split = 1;
  while (split < kMaxSplit && (long long)a.rows * split <= num_sms() && a.V >= 2 * split * batch)
    split *= 2;
  if (dt == SPEC_BF16)
    return a.out ? launch_split<SPEC_BF16, true>(a, split, s)
                 : launch_split<SPEC_BF16, false>(a, split, s);
  return a.out ? launch_split<SPEC_F32, true>(a, split, s)
               : launch_split<SPEC_F32, false>(a, split, s);
}

}  // namespace spec
