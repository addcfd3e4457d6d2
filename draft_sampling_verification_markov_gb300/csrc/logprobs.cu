// logprobs.cu -- log-probabilities of given tokens with rank, entropy and top alternatives.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace spec {
namespace {

constexpr int kThreads = 512;

// One block a row: a pass for the maximum, one for the sums and the rank, one a place of the
// alternatives (the largest logit after the place before it).
template <int DT>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(LogprobArgs a) {
  const int row = blockIdx.x;
  const int t = a.tokens ? a.tokens[row] : -1;
  if (a.tokens && t == -1) return;
  const bool bad = t < 0 || t >= a.V;
  if (a.tokens && bad && threadIdx.x == 0) atomicOr(a.status, SPEC_DEV_BAD_TOKEN);
  const size_t off = (size_t)row * a.ld;
  const float xt = bad ? INFINITY : ld_elem<DT>(a.x, off + t);
  float m = -INFINITY;
  for (int v = threadIdx.x; v < a.V; v += kThreads) m = fmaxf(m, ld_elem<DT>(a.x, off + v));
  m = block_merge({m, 0.0f, 0}).m;
  float s = 0.0f, s1 = 0.0f, rank = 0.0f;
  for (int v = threadIdx.x; v < a.V; v += kThreads) {
    const float x = ld_elem<DT>(a.x, off + v);
    const float z = (x - m) * a.scale, e = expf(z);
    s += e;
    if (!(e == 0.0f)) s1 += e * z;
    rank += x > xt ? 1.0f : 0.0f;
  }
  s = block_sum(s);
  s1 = block_sum(s1);
  rank = block_sum(rank);
  const bool finite = s > 0.0f && s < INFINITY && m > -INFINITY;
  const float ls = finite ? logf(s) : NAN;
  if (threadIdx.x == 0) {
    if (!finite) atomicOr(a.status, SPEC_DEV_NONFINITE);
    if (a.tokens && a.logp) a.logp[row] = bad ? NAN : (xt - m) * a.scale - ls;
    if (a.tokens && a.rank) a.rank[row] = bad ? 0 : (int)rank + 1;
    if (a.entropy) a.entropy[row] = ls - s1 / s;
  }
  float px = INFINITY;
  int pi = -1;
  for (int j = 0; j < a.top; ++j) {
    StatsAcc b = stats_empty();
    for (int v = threadIdx.x; v < a.V; v += kThreads) {
      const float x = ld_elem<DT>(a.x, off + v);
      if ((x < px || (x == px && v > pi)) && x > b.m) b = {x, 0.0f, v};
    }
    b = block_merge(b);
    px = b.m;
    pi = b.idx;
    const bool none = b.m == -INFINITY;
    if (threadIdx.x == 0) {
      const size_t o = (size_t)row * a.top + j;
      if (a.top_ids) a.top_ids[o] = none ? -1 : pi;
      if (a.top_logp) a.top_logp[o] = none ? -INFINITY : (px - m) * a.scale - ls;
    }
  }
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, int dt, cudaStream_t s) {
  TraceScope ts(SPEC_KCLASS_OTHER, s);
  if (dt == SPEC_BF16)
    logprobs_kernel<SPEC_BF16><<<a.rows, kThreads, 0, s>>>(a);
  else
    logprobs_kernel<SPEC_F32><<<a.rows, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace spec
