// w4_g128.cu -- the product's kernels for groups of 128.
#include "w4_product.cuh"

namespace spec {
namespace w4 {

cudaError_t launch_g128(const W4Args& a, const CUtensorMap& codes, int R, int T, cudaStream_t s) {
  return launch_group<128>(a, codes, R, T, s);
}

}  // namespace w4
}  // namespace spec
