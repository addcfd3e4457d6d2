// w4_g32.cu -- the product's kernels for groups of 32.
#include "w4_product.cuh"

namespace spec {
namespace w4 {

cudaError_t launch_g32(const W4Args& a, const CUtensorMap& codes, Form form, cudaStream_t s) {
  return launch_group<32>(a, codes, form, s);
}

}  // namespace w4
}  // namespace spec
