// logprobs.cu -- log-probabilities of given tokens with rank, entropy and top alternatives, in
// one pass over the logits.
//
// With z = x / T, m = max z and e = exp(z - m):  S = sum e,  S1 = sum e (z - m);
//   log p(t) = z_t - m - log S,   entropy = log S - S1 / S,   rank = 1 + #{x > x_t}.
// A thread keeps S and S1 of its elements against a reference logit m of its own, in the base-2
// scale (x - m) log2(e) / T, and moves them to another reference (2^d S, 2^d (S1 + d S) for a
// shift d) where a logit is far above; the parts are merged the same way in a fixed order.
//
// The largest k <= 32 logits need no second pass. The maxima of 64 groups of the first batches
// bound the k-th largest logit from below (k groups hold a logit at least as large as the k-th
// group maximum). A thread's batch of 64 bytes then goes on a list when its maximum reaches the
// bound: some two hundred batches of a row of 129280 logits. At the end the same argument on the
// listed maxima gives a bound that few elements reach; those are ranked by counting, larger logits
// first, then lower ids. Rows that defeat the bound (long ascending runs, hundreds of equal
// logits) overflow a list and take a radix selection over the row instead.
//
// Few rows are split over a thread-block cluster of up to 8 CTAs, which merge through distributed
// shared memory: no workspace, one launch.
//
// Measured (V = 129280): 2048 bf16 rows 87 us without alternatives (6.1 TB/s), 105 us with 20 (5.1
// TB/s), 256 rows 21 us, one row 7.7 us; 1024 fp32 rows with 20 95 us (5.6 TB/s). Without
// alternatives memory bounds it. With them each row takes 41 instead of 33 thousand warp
// instructions, and an SM issues in 64 % of its cycles; half of the difference is the lists, half
// the row's end. Prefetching the next row into L2 during that end is slower (107 to 111 us).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace spec {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;             // 16-byte pieces of a thread's batch
constexpr int kMaxTop = SPEC_LOGPROBS_MAX_TOP;
constexpr int kEntries = 512;         // listed batches at most
constexpr int kKeys = 512;            // elements ranked at most
constexpr int kMaxSplit = 8;          // parts of a row at most
constexpr int kGroups = 64;           // maxima behind a bound; at least 2 * kMaxTop
constexpr uint32_t kFull = 0xffffffffu;

constexpr float kOctaves = 4.0f;
constexpr float kLowest2 = -256.0f;   // 2^kLowest2 is 0 in fp32
// The fast sums need log2(e) / T = c in (kFastLeast, kFastScale) and a reference |m| < kFastMax:
// then 2^101 c is finite, and (-2^100 - m) c is below -256.
constexpr float kFastMax = 0x1p99f, kFastScale = 0x1p20f, kFastLeast = 0x1p-90f;

struct Sums {
  float m, s, s1;  // reference logit, S, S1 (in base 2)
};

static_assert(kKeys >= kMaxSplit * kMaxTop && kMaxTop == 32, "the merged lists");
static_assert(kBatch * 8 <= 32, "a lane an element of a listed batch");

struct Shared {
  alignas(16) float group[kGroups];
  float bound, room;                  // entries until the next renewal
  bool full[2];
  int n_entries, n_keys;
  uint4 entry[kEntries][kBatch];      // listed batches: content, first piece, maximum
  uint32_t entry_at[kEntries];
  float entry_max[kEntries];
  unsigned long long keys[kKeys];
  unsigned long long top[kMaxTop];    // this CTA's largest, in order; 0 = none
  Sums sums[kWarps];
  int count[kWarps];
  Sums total;                         // of this part
  int total_count;
  Sums row;                           // (maximum, log S) of a split row
  // radix selection
  int hist[256];
  uint32_t prefix;
  int need, running;
  int scan[kWarps];
};

// Ordered bits: larger floats have larger bits, zeros of both signs are equal. 0 stands for
// "no place" (NaN and -inf).
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (!(x > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
__device__ __forceinline__ unsigned long long make_key(uint32_t bits, int id) {
  return ((unsigned long long)bits << 32) | (0xffffffffu - (uint32_t)id);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The sums of the first n lanes (a power of two) in every one of them: against their largest
// reference, then added.
template <int n>
__device__ __forceinline__ Sums merge_lanes(Sums a, float c) {
  float m = a.m;
#pragma unroll
  for (int o = n / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  if (a.m > -INFINITY) {
    const float d = fmaxf((a.m - m) * c, kLowest2), f = fast_exp2(d);
    a.s1 = f * (a.s1 + d * a.s);
    a.s *= f;
  }  // else 0, or NaN
  a.m = m;
#pragma unroll
  for (int o = n / 2; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(kFull, a.s, o);
    a.s1 += __shfl_xor_sync(kFull, a.s1, o);
  }
  return a;
}

// ------------------------------------------------------------------------------ a row's pieces

// A row as 16-byte pieces at 16-byte aligned addresses: piece j holds ids j * N - head ...; the
// first and the last piece may be partly outside the row.
template <int DT>
struct Row {
  static constexpr int N = DT == SPEC_BF16 ? 8 : 4;
  const char* base;  // address of piece 0
  int head, V;

  __device__ Row(const void* x, size_t off, int V_) : V(V_) {
    const char* p = static_cast<const char*>(x) + off * (16 / N);
    const int mis = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    base = p - mis;
    head = mis / (16 / N);
  }
  __device__ int pieces() const { return (head + V + N - 1) / N; }

  // Pieces jb + thread + b * kThreads, b < B.
  template <int B>
  __device__ __forceinline__ void load_batch(uint4 (&q)[B], int jb, int end) const;

  static constexpr uint32_t kNone = DT == SPEC_BF16 ? 0xff80ff80u : 0xff800000u;  // -inf

  // Piece j, with -inf outside the row and past `end`. A row has at most two pieces that are
  // partly outside; they go through a call of their own, so that the loads of whole ones stay in
  // flight together.
  __device__ __forceinline__ uint4 load(int j, int end) const {
    uint4 q = make_uint4(kNone, kNone, kNone, kNone);
    if (j < end) {
      const int v = j * N - head;
      if (v >= 0 && v + N <= V) q = ld_coherent16(base + (size_t)j * 16);
    }
    return q;
  }
  __device__ __forceinline__ bool partial(int j, int end) const {
    const int v = j * N - head;
    return j < end && (v < 0 || v + N > V);
  }
  __device__ __noinline__ uint4 load_partial(int j) const {
    uint32_t w[4] = {kNone, kNone, kNone, kNone};
    const int v = j * N - head;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (v + i < 0 || v + i >= V) continue;
      if constexpr (DT == SPEC_BF16) {
        const uint32_t b = reinterpret_cast<const uint16_t*>(base + (size_t)j * 16)[i];
        w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | b << 16 : (w[i / 2] & 0xffff0000u) | b;
      } else {
        w[i] = reinterpret_cast<const uint32_t*>(base + (size_t)j * 16)[i];
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // Either kind.
  __device__ __forceinline__ uint4 load_any(int j, int end) const {
    return partial(j, end) ? load_partial(j) : load(j, end);
  }
};

template <int DT>
template <int B>
__device__ __forceinline__ void Row<DT>::load_batch(uint4 (&q)[B], int jb, int end) const {
  const int j = jb + threadIdx.x;
  // whole batches inside the row: one address, no tests of single pieces
  if (jb * N >= head && jb + B * kThreads <= end && (jb + B * kThreads) * N - head <= V) {
    const char* p = base + (size_t)j * 16;
#pragma unroll
    for (int b = 0; b < B; ++b) q[b] = ld_coherent16(p + b * kThreads * 16);
  } else {
#pragma unroll
    for (int b = 0; b < B; ++b) q[b] = load(j + b * kThreads, end);
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (partial(j + b * kThreads, end)) q[b] = load_partial(j + b * kThreads);
  }
}

template <int DT>
__device__ __forceinline__ void unpack(const uint4& q, float (&x)[Row<DT>::N]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == SPEC_BF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      x[i] = __uint_as_float(w[i]);
    }
  }
}

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t w) {
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}
__device__ __forceinline__ uint32_t as_word(__nv_bfloat162 v) {
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
  return fmaxf(a, fmaxf(b, c));
}

// Maximum of a batch (NaN ignored, unless there is nothing else).
template <int DT>
__device__ __forceinline__ float batch_max(const uint4 (&q)[kBatch]) {
  if constexpr (DT == SPEC_BF16) {
    __nv_bfloat162 m[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      m[b] = __hmax2(__hmax2(as_bf2(q[b].x), as_bf2(q[b].y)),
                     __hmax2(as_bf2(q[b].z), as_bf2(q[b].w)));
#pragma unroll
    for (int b = 1; b < kBatch; ++b) m[0] = __hmax2(m[0], m[b]);
    const uint32_t w = as_word(m[0]);
    return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      m = max3f(max3f(m, __uint_as_float(q[b].x), __uint_as_float(q[b].y)),
                __uint_as_float(q[b].z), __uint_as_float(q[b].w));
    return m;
  }
}

// The piece with everything below -2^100 (masked logits) raised to it, NaN kept. Against a
// reference that the fast sums take such a logit still has exp = 0, and (x - m) c stays finite,
// so that its term of S1 is 0 too and needs no comparison of its own.
template <int DT>
__device__ __forceinline__ uint4 raised(const uint4& q) {
  if constexpr (DT == SPEC_BF16) {
    const __nv_bfloat162 low = as_bf2(0xf180f180u);
    return make_uint4(as_word(__hmax2_nan(as_bf2(q.x), low)),
                      as_word(__hmax2_nan(as_bf2(q.y), low)),
                      as_word(__hmax2_nan(as_bf2(q.z), low)),
                      as_word(__hmax2_nan(as_bf2(q.w), low)));
  } else {
    const float low = -0x1p100f;
    return make_uint4(__float_as_uint(max_nan(__uint_as_float(q.x), low)),
                      __float_as_uint(max_nan(__uint_as_float(q.y), low)),
                      __float_as_uint(max_nan(__uint_as_float(q.z), low)),
                      __float_as_uint(max_nan(__uint_as_float(q.w), low)));
  }
}

// Elements of a batch larger than the given token's logit.
template <int DT>
__device__ __forceinline__ int count_larger(const uint4 (&q)[kBatch], float xt) {
  if constexpr (DT == SPEC_BF16) {
    // two comparisons an instruction, each a mask of 16 bits, and integer sums of the masks:
    // 65535 lo + 65535 * 65536 hi, or -lo modulo 2^16 and then 65536 (lo - hi) modulo 2^32
    const __nv_bfloat162 t = __float2bfloat162_rn(xt);
    uint32_t n = 0;
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      n += __hgt2_mask(as_bf2(q[b].x), t) + __hgt2_mask(as_bf2(q[b].y), t) +
           __hgt2_mask(as_bf2(q[b].z), t) + __hgt2_mask(as_bf2(q[b].w), t);
    const int lo = -n & 0xffffu;
    return 2 * lo - ((int)(n + lo) >> 16);
  } else {
    int n = 0;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      float x[4];
      unpack<DT>(q[b], x);
      n += (x[0] > xt) + (x[1] > xt) + (x[2] > xt) + (x[3] > xt);
    }
    return n;
  }
}

// A thread's sums against a reference `m`, one of its logits and at most kOctaves of
// exp((max - m) / T) below its maximum, so that the reference changes in few batches. A term of S1
// is up to kOctaves times one of S, and its roundings count against the entropy: with 32 octaves
// the entropy of peaked rows was off by up to 2e-5. z = (x - m) c is a subtraction and a product:
// the largest logit of a row is exactly 1 in S, so a point mass has log-probability and entropy 0.
struct RunningSums {
  float m, limit;                    // reference, and the logit that calls for another
  float most;                        // maximum
  unsigned long long s, s1;          // S and S1, two partial sums each

  __device__ __forceinline__ void start() {
    m = limit = most = -INFINITY;
    s = s1 = tc::pack2(0.0f, 0.0f);
  }
  // The same sums against another reference.
  __device__ __forceinline__ void rebase(float to, float c) {
    const float d = fmaxf((m - to) * c, kLowest2), f = fast_exp2(d);
    const unsigned long long f2 = tc::pack2(f, f);
    s1 = tc::mul2(f2, tc::fma2(tc::pack2(d, d), s, s1));
    s = tc::mul2(f2, s);
  }
  // Against the maximum, where the log-probabilities of likely tokens cancel least.
  __device__ __forceinline__ Sums sums(float c) {
    Sums o;
    float a, b;
    if (m > -INFINITY) rebase(most, c);
    o.m = most;
    tc::unpack2(s, a, b);
    o.s = a + b;
    tc::unpack2(s1, a, b);
    o.s1 = a + b;
    return o;
  }
};

// One batch into the lists, the sums and the count; j is this thread's first piece.
template <int DT, bool TOP>
__device__ __forceinline__ void take_batch(Shared& sh, const uint4 (&q)[kBatch], int j,
                                           float bound, float xt, float c, bool tame,
                                           RunningSums& run, int& larger) {
  constexpr int N = Row<DT>::N;
  const float bm = batch_max<DT>(q);
  if (TOP && bm >= bound) {
    const int at = atomicAdd(&sh.n_entries, 1);
    if (at < kEntries) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) sh.entry[at][b] = q[b];
      sh.entry_at[at] = j;
      sh.entry_max[at] = bm;
    }
  }
  run.most = fmaxf(run.most, bm);
  if (bm > run.limit) {
    if (run.m > -INFINITY) run.rebase(bm, c);
    run.m = bm;
    run.limit = bm + kOctaves / c;
  }
  if (tame && fabsf(run.m) < kFastMax) {
    const unsigned long long c2 = tc::pack2(c, c), m2 = tc::pack2(-run.m, -run.m);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      float x[N];
      unpack<DT>(raised<DT>(q[b]), x);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const unsigned long long z = tc::mul2(tc::add2(tc::pack2(x[i], x[i + 1]), m2), c2);
        float z0, z1;
        tc::unpack2(z, z0, z1);
        const unsigned long long e = tc::pack2(fast_exp2(z0), fast_exp2(z1));
        run.s = tc::add2(run.s, e);
        run.s1 = tc::fma2(e, z, run.s1);
      }
    }
  } else {
    // extreme maxima, extreme temperatures, or nothing above -inf yet (then measured from 0: the
    // terms are 0, or NaN)
    const float m = run.m > -INFINITY ? run.m : 0.0f;
#pragma unroll 1
    for (int b = 0; b < kBatch; ++b) {
      float x[N];
      uint4 w = q[0];
#pragma unroll
      for (int i = 1; i < kBatch; ++i)
        if (b == i) w = q[i];
      unpack<DT>(w, x);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float z0 = max_nan((x[i] - m) * c, kLowest2);
        const float z1 = max_nan((x[i + 1] - m) * c, kLowest2);
        const unsigned long long e = tc::pack2(fast_exp2(z0), fast_exp2(z1));
        run.s = tc::add2(run.s, e);
        run.s1 = tc::fma2(e, tc::pack2(z0, z1), run.s1);
      }
    }
  }
  if (bm > xt) larger += count_larger<DT>(q, xt);
}

// ------------------------------------------------------------------------------ bounds

// The k-th largest of 64 group maxima (a group: kPer neighbouring threads), a lower bound of the
// k-th largest of the elements behind `local`. Every thread calls it and gets the bound. A
// group's threads rank its maximum, each against its share of the others; equal ones in order of
// their index.
__device__ __forceinline__ float bound_of(Shared& sh, float local, int k) {
  constexpr int kPer = kThreads / kGroups, kShare = kGroups / kPer;
  const int g = threadIdx.x / kPer, part = threadIdx.x % kPer;
#pragma unroll
  for (int o = 1; o < kPer; o *= 2) local = fmaxf(local, __shfl_xor_sync(kFull, local, o));
  if (part == 0) sh.group[g] = local;
  __syncthreads();
  int place = 0;
#pragma unroll
  for (int i = 0; i < kShare; i += 4) {
    const int at = kShare * part + i;
    const float4 o = *reinterpret_cast<const float4*>(&sh.group[at]);
    place += (o.x > local || (o.x == local && at < g)) +
             (o.y > local || (o.y == local && at + 1 < g)) +
             (o.z > local || (o.z == local && at + 2 < g)) +
             (o.w > local || (o.w == local && at + 3 < g));
  }
#pragma unroll
  for (int o = 1; o < kPer; o *= 2) place += __shfl_xor_sync(kFull, place, o);
  if (place == k - 1 && part == 0) sh.bound = local;
  __syncthreads();
  return sh.bound;
}

// This thread's share of the n listed maxima. Neighbours in the list go to different groups of
// bound_of: with consecutive ones in a group, a list of a hundred left most groups empty and the
// bound low (2048 rows of 32000, top 20: 47.0 -> 43.1 us; 256 of 129280: 21.8 -> 21.2).
__device__ __forceinline__ float listed_max(const Shared& sh, int n) {
  constexpr int kPer = kThreads / kGroups;
  float m = -INFINITY;
  for (int i = threadIdx.x / kPer + threadIdx.x % kPer * kGroups; i < n; i += kThreads)
    m = fmaxf(m, sh.entry_max[i]);
  return m;
}

// The bound renewed from the listed batches if there are more than sh.room, which doubles for the
// next call; +inf (list nothing more) once they do not fit. `turn` alternates between two calls.
__device__ __forceinline__ float renewed(Shared& sh, float bound, int k, int turn) {
  if (threadIdx.x == 0) {
    // one thread's count, however many entries others add meanwhile: all go the same way
    sh.full[turn] = *(volatile int*)&sh.n_entries > sh.room;
    sh.room *= 2.0f;
  }
  __syncthreads();
  // a thread may reach the next call, but not the one after it, before another reads this
  if (!sh.full[turn]) return bound;
  const int n = sh.n_entries;
  if (n > kEntries) return INFINITY;
  return fmaxf(bound, bound_of(sh, listed_max(sh, n), k));
}

// ------------------------------------------------------------------------------ radix selection

// The k largest elements of pieces [j0, j1) into sh.keys (sh.n_keys of them), whatever their order
// and however many are equal: the k-th largest value by its leading bytes, then every larger
// element and the first of the equal ones. Two (bf16) or four passes more over the row: 2048 equal
// or ascending rows of 129280 take 0.93 and 1.0 ms in bf16, 2.3 and 2.4 ms in fp32.
template <int DT>
__device__ __noinline__ void select_radix(Shared& sh, const Row<DT>& row, int j0, int j1, int k) {
  constexpr int N = Row<DT>::N;
  constexpr int kBits = DT == SPEC_BF16 ? 16 : 32;  // a bf16's ordered bits are the upper half
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    sh.prefix = 0;
    sh.need = k;
    sh.n_keys = 0;
    sh.running = 0;
  }
  bool all = false;  // fewer than k elements have a place
  for (int shift = kBits - 8; shift >= 0 && !all; shift -= 8) {
    for (int b = tid; b < 256; b += kThreads) sh.hist[b] = 0;
    __syncthreads();
    const uint32_t prefix = sh.prefix;
    for (int j = j0 + tid; j < j1; j += kThreads) {
      float x[N];
      unpack<DT>(row.load_any(j, j1), x);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t u = order_bits(x[i]);
        const uint32_t b = u >> (32 - kBits);
        // shift + 8 may be the whole width, where every element matches
        if (u && (shift + 8 == kBits || (b >> (shift + 8)) == prefix))
          atomicAdd(&sh.hist[(b >> shift) & 255], 1);
      }
    }
    __syncthreads();
    if (tid == 0) {
      int cum = 0, b = 255;
      for (; b >= 0 && cum + sh.hist[b] < sh.need; --b) cum += sh.hist[b];
      if (b < 0) {
        sh.need = -1;
      } else {
        sh.prefix = prefix << 8 | (uint32_t)b;
        sh.need -= cum;
      }
    }
    __syncthreads();
    all = sh.need < 0;
    __syncthreads();
  }
  const uint32_t cut = all ? 0 : sh.prefix;
  const int need = all ? 0 : sh.need;
  for (int j = j0; j < j1; j += kThreads) {  // ascending, a piece a thread
    float x[N];
    unpack<DT>(row.load_any(j + tid, j1), x);
    uint32_t same = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t u = order_bits(x[i]), b = u >> (32 - kBits);
      if (u && (all || b > cut)) sh.keys[atomicAdd(&sh.n_keys, 1)] =
          make_key(u, (j + tid) * N - row.head + i);
      if (u && !all && b == cut) same |= 1u << i;
    }
    if (sh.running >= need) continue;  // uniform: written between the barriers below only
    // place of this thread's equal elements among all of them
    int c = __popc(same), at = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, at, o);
      if (lane >= o) at += y;
    }
    if (lane == 31) sh.scan[warp] = at;
    __syncthreads();
    int before = sh.running + at - c, sum = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.scan[w];
      sum += sh.scan[w];
    }
    for (uint32_t s = same; s && before < need; s &= s - 1, ++before) {
      const int i = __ffs(s) - 1;
      uint32_t u = 0;
#pragma unroll
      for (int q = 0; q < N; ++q)
        if (q == i) u = order_bits(x[q]);
      sh.keys[atomicAdd(&sh.n_keys, 1)] = make_key(u, (j + tid) * N - row.head + i);
    }
    __syncthreads();
    if (tid == 0) sh.running += sum;
    __syncthreads();
  }
  __syncthreads();
}

// ------------------------------------------------------------------------------ kernel

// A row's scalar outputs; returns (maximum, log S) for the alternatives.
__device__ __forceinline__ Sums write_row(const LogprobArgs& a, int row, bool bad, float xt,
                                          Sums sum, int larger) {
  const bool finite = sum.s > 0.0f && sum.s < INFINITY && sum.m > -INFINITY;
  const float ls = finite ? logf(sum.s) : NAN;
  if (!finite) atomicOr(a.status, SPEC_DEV_NONFINITE);
  if (a.tokens && bad) atomicOr(a.status, SPEC_DEV_BAD_TOKEN);
  if (a.logp) a.logp[row] = bad ? NAN : (xt - sum.m) * a.scale - ls;
  if (a.rank) a.rank[row] = bad ? 0 : larger + 1;
  if (a.entropy) a.entropy[row] = ls - sum.s1 / sum.s * kLn2;
  return {sum.m, ls, 0.0f};
}

// The a.top largest elements of pieces [j0, j1) as keys, unordered, sh.n_keys of them or a few
// more: those of the listed pieces that reach the list's bound, or by radix selection.
template <int DT>
__device__ __forceinline__ void collect_keys(Shared& sh, const Row<DT>& r, int j0, int j1,
                                             float bound, int k) {
  constexpr int N = Row<DT>::N;
  const int tid = threadIdx.x, lane = tid & 31, n = sh.n_entries;
  bool fits = n <= kEntries;
  if (fits) {
    // fewer listed batches than places leave the bound they were listed by
    const float cut = fmaxf(bound_of(sh, listed_max(sh, n), k), bound);
    // a warp takes every kWarps-th batch, its lanes the elements of those that reach the cut
    for (int base = tid >> 5; base < n; base += kThreads) {
      const int mine = base + lane * kWarps;
      uint32_t hit = __ballot_sync(kFull, mine < n && sh.entry_max[mine] >= cut);
      while (hit) {
        constexpr int kAtOnce = 2;
        int i[kAtOnce], n_mine = 0;
        float x[kAtOnce];
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
          i[q] = base + (hit ? __ffs(hit) - 1 : 0) * kWarps;
          x[q] = -INFINITY;
          if (hit && lane < kBatch * N) {
            if constexpr (DT == SPEC_BF16)
              x[q] = bf16_to_f32(reinterpret_cast<const uint16_t*>(sh.entry[i[q]])[lane]);
            else
              x[q] = reinterpret_cast<const float*>(sh.entry[i[q]])[lane];
          }
          n_mine += x[q] >= cut;
          hit &= hit - 1;
        }
        if (!n_mine) continue;
        int at = atomicAdd(&sh.n_keys, n_mine);
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q)
          if (x[q] >= cut && at < kKeys)
            sh.keys[at++] =
                make_key(order_bits(x[q]), ((int)sh.entry_at[i[q]] + lane / N * kThreads) * N -
                                               r.head + lane % N);
      }
    }
    __syncthreads();
    fits = sh.n_keys <= kKeys;
  }
  if (!fits) {
    __syncthreads();
    select_radix<DT>(sh, r, j0, j1, k);
  }
}

// Place of a key among the n of sh.keys.
__device__ __forceinline__ int place_of(const Shared& sh, unsigned long long key, int n) {
  int place = 0;
#pragma unroll 8
  for (int q = 0; q < n; ++q) place += sh.keys[q] > key;
  return place;
}

__device__ __forceinline__ void write_top(const LogprobArgs& a, int row, int place,
                                          unsigned long long key, Sums ms) {
  const size_t at = (size_t)row * a.top + place;
  const float x = order_value((uint32_t)(key >> 32));
  if (a.top_ids) a.top_ids[at] = key ? (int)(0xffffffffu - (uint32_t)key) : -1;
  if (a.top_logp) a.top_logp[at] = key ? (x - ms.m) * a.scale - ms.s : -INFINITY;
}

// D batches of a thread in flight: 2, and four CTAs an SM, or for rows that leave an SM two CTAs 4.
// 256 rows of 129280 with 2 / 4, us: bf16 22.7 / 21.7, fp32 32.9 / 28.9 (parts of split rows gain
// nothing). 512 threads a CTA instead: 23.3 and 30.0.
__host__ __device__ constexpr int ctas(int D) { return 8 / D; }

// SPLIT: a cluster takes one row, each CTA a part of it. Else a CTA takes rows in turn and has the
// first batches of the next one on their way before it finishes a row: all CTAs of an SM start
// together and would leave the memory idle together (10 of 56 thousand cycles a row).
template <int DT, bool TOP, bool SPLIT, int D>
__global__ void __launch_bounds__(kThreads, ctas(D)) logprobs_kernel(const LogprobArgs a,
                                                                     const int parts,
                                                                     const float room) {
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int split = SPLIT ? parts : 1;
  const int part = SPLIT ? blockIdx.x % split : 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float c = a.scale * kLog2e;
  const bool tame = c < kFastScale && c > kFastLeast;
  constexpr int kStep = kBatch * kThreads;

  grid_dep_wait();
  int row = SPLIT ? blockIdx.x / split : blockIdx.x;
  Row<DT> r(a.x, (size_t)row * a.ld, a.V);
  // the first logits are on their way while the token is read
  uint4 q[D][kBatch];
  {
    const int np = r.pieces(), per = (np + split - 1) / split;
#pragma unroll
    for (int d = 0; d < D; ++d)
      r.template load_batch<kBatch>(q[d], part * per + d * kStep, min(np, part * per + per));
  }
  int t = a.tokens ? a.tokens[row] : 0;
  while (true) {
    const int next = SPLIT ? a.rows : row + gridDim.x;
    const int t_next = next < a.rows && a.tokens ? a.tokens[next] : 0;
    const bool skip = a.tokens && t == -1;
    if (SPLIT && skip) return;  // the whole cluster
    const int np = r.pieces(), per = (np + split - 1) / split;
    const int j0 = part * per, j1 = min(np, j0 + per);
    if (!skip) {
      const bool bad = t < 0 || t >= a.V;
      const float xt = bad || !a.tokens ? INFINITY : ld_elem_coherent<DT>(a.x, (size_t)row * a.ld + t);
      float bound = INFINITY;
      if (TOP) {
        if (tid == 0) {
          sh.n_entries = 0;
          sh.room = room;
          sh.n_keys = 0;
        }
        float first = -INFINITY;  // a batch of NaN has the maximum NaN
#pragma unroll
        for (int d = 0; d < D; ++d) first = fmaxf(first, batch_max<DT>(q[d]));
        // nothing of -inf has a place
        bound = fmaxf(bound_of(sh, first, a.top), -3.402823466e38f);
      }
      RunningSums run;
      run.start();
      int larger = 0;
      // Whenever the number of batches seen has doubled, the bound is renewed from the list if the
      // list would pass half its room by the row's end at this rate. 2048 bf16 rows of 129280:
      // always renewed 110 us, never 105; uniform on [0, 1), with hundreds of logits equal to the
      // k-th, the list overflows without: 166 us against 465. By this rule 106 and 162.
      int renew = j0 + 2 * D * kStep;
      for (int jb = j0; jb < j1; jb += D * kStep) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          const int j = jb + d * kStep;
          if (d && j >= j1) break;
          take_batch<DT, TOP>(sh, q[d], j + tid, bound, xt, c, tame, run, larger);
          r.template load_batch<kBatch>(q[d], j + D * kStep, j1);
        }
        if (TOP && jb + D * kStep == renew && renew < j1) {
          renew += renew - j0;
          bound = renewed(sh, bound, a.top, __ffs(renew - j0) & 1);
        }
      }
      const Row<DT> done = r;
      if (next < a.rows) {
        r = Row<DT>(a.x, (size_t)next * a.ld, a.V);
#pragma unroll
        for (int d = 0; d < D; ++d) r.template load_batch<kBatch>(q[d], d * kStep, r.pieces());
      }

      // this CTA's sums: lanes against their warp's maximum, then warps against the CTA's
      Sums acc = merge_lanes<32>(run.sums(c), c);
      larger = __reduce_add_sync(kFull, larger);
      if (lane == 0) {
        sh.sums[warp] = acc;
        sh.count[warp] = larger;
      }
      if (TOP && SPLIT && tid < kMaxTop) sh.top[tid] = 0;
      __syncthreads();  // every push, too
      if (warp == kWarps - 1) {
        const bool has = lane < kWarps;
        acc = merge_lanes<kWarps>(has ? sh.sums[lane] : Sums{-INFINITY, 0.0f, 0.0f}, c);
        larger = __reduce_add_sync(kFull, has ? sh.count[lane] : 0);
        if (lane == 0) {
          sh.total = SPLIT ? acc : write_row(a, row, bad, xt, acc, larger);
          sh.total_count = larger;
        }
      }
      if (TOP) {
        collect_keys<DT>(sh, done, j0, j1, bound, a.top);
        const int nk = sh.n_keys;
        for (int i = tid; i < nk; i += kThreads) {
          const unsigned long long key = sh.keys[i];
          const int place = place_of(sh, key, nk);
          if (place >= a.top) continue;
          if (SPLIT)
            sh.top[place] = key;
          else
            write_top(a, row, place, key, sh.total);
        }
        // places that no logit has
        if (!SPLIT && tid < a.top && tid >= nk) write_top(a, row, tid, 0, sh.total);
      }

      if (SPLIT) {  // the cluster's parts, merged by its first CTA
        cluster.sync();
        if (part == 0) {
          if (warp == kWarps - 1) {  // lane p: part p
            const bool has = lane < split;
            const Shared* other = cluster.map_shared_rank(&sh, has ? lane : 0);
            Sums sum = has ? other->total : Sums{-INFINITY, 0.0f, 0.0f};
            const int count = __reduce_add_sync(kFull, has ? other->total_count : 0);
            sum = merge_lanes<kMaxSplit>(sum, c);
            if (lane == 0) sh.row = write_row(a, row, bad, xt, sum, count);
          }
          if (TOP) {
            for (int i = tid; i < split * kMaxTop; i += kThreads)
              sh.keys[i] = *cluster.map_shared_rank(&sh.top[i % kMaxTop], i / kMaxTop);
            __syncthreads();
            // place of each part's entry: its own place in its part's list, plus the larger
            // entries of every other (descending, zeros at the end)
            for (int i = tid; i < split * kMaxTop; i += kThreads) {
              const unsigned long long key = sh.keys[i];
              if (!key) continue;
              int place = i % kMaxTop;
#pragma unroll
              for (int o = 0; o < kMaxSplit; ++o) {
                if (o >= split || o == i / kMaxTop) continue;
                const unsigned long long* list = sh.keys + o * kMaxTop;
                int n = 0;
#pragma unroll
                for (int w = kMaxTop / 2; w > 0; w /= 2) n += list[n + w - 1] > key ? w : 0;
                place += n + (list[n] > key ? 1 : 0);
              }
              if (place < a.top) write_top(a, row, place, key, sh.row);
            }
            if (warp == 0) {  // places that no logit has
              int have = 0;
              for (int o = 0; o < split; ++o)
                have += __popc(__ballot_sync(kFull, sh.keys[o * kMaxTop + lane] != 0));
              if (lane < a.top && lane >= have) write_top(a, row, lane, 0, sh.row);
            }
          }
        }
        cluster.sync();  // no part leaves before it has been read
        return;
      }
      if (next < a.rows) __syncthreads();  // the next row reuses the shared state
    } else if (next < a.rows) {
      r = Row<DT>(a.x, (size_t)next * a.ld, a.V);
#pragma unroll
      for (int d = 0; d < D; ++d) r.template load_batch<kBatch>(q[d], d * kStep, r.pieces());
    }
    if (next >= a.rows) return;
    row = next;
    t = t_next;
  }
}

template <int DT, bool TOP, bool SPLIT, int D>
cudaError_t launch_t(const LogprobArgs& a, int split, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = trace_active() ? 0 : 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  const int most = ctas(D) * num_sms();
  cfg.gridDim = dim3((unsigned)(SPLIT ? a.rows * split : (a.rows < most ? a.rows : most)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  // entries a part may list before its first renewal if it is to fill half the list by its end
  const float room = kEntries / 2 * 2.0f * D * kBatch * kThreads * Row<DT>::N * split / a.V;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, TOP, SPLIT, D>, a, split, room);
}

template <int DT, bool TOP>
cudaError_t launch_split(const LogprobArgs& a, int split, cudaStream_t s) {
  if (split > 1) return launch_t<DT, TOP, true, 2>(a, split, s);
  return a.rows <= ctas(4) * num_sms() ? launch_t<DT, TOP, false, 4>(a, 1, s)
                                       : launch_t<DT, TOP, false, 2>(a, 1, s);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, int dt, cudaStream_t s) {
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  // A CTA has some 5 us of latencies outside its stream of logits, more in a cluster: rows are
  // split while the parts still find SMs of their own and have a batch or more. 129280 bf16
  // logits, top 20, us at splits of 1 / 2 / 4 / 8: 1 row 12.8 / 10.9 / 8.6 / 7.8, 64 rows 15.1 /
  // 13.3 / 11.9 / 14.0, 128 rows 15.8 / 15.7 / 17.2 / 24.9, 256 rows 21.0 / 23.1 / 28.0 / 42.8.
  const int batch = kThreads * kBatch * (dt == SPEC_BF16 ? 8 : 4);
  int split = 1;
  while (split < kMaxSplit && (long long)a.rows * split <= num_sms() &&
         a.V >= 2 * split * batch)
    split *= 2;
  if (dt == SPEC_BF16)
    return a.top ? launch_split<SPEC_BF16, true>(a, split, s)
                 : launch_split<SPEC_BF16, false>(a, split, s);
  return a.top ? launch_split<SPEC_F32, true>(a, split, s)
               : launch_split<SPEC_F32, false>(a, split, s);
}

}  // namespace spec
