// gmm_mx.cuh's down product, apart from the gate and up product so that they
// compile side by side.
#include "gmm_mx.cuh"

namespace moe {
namespace mx {

template <int BLOCK>
static cudaError_t pick(const GmmArgs& a, const void* codes, cudaStream_t s) {
  return many_rows(a) ? launch_one<false, BLOCK, 192, true>(a, codes, s)
                      : launch_one<false, BLOCK, 64, false>(a, codes, s);
}
cudaError_t launch_gmm_mx_down(const GmmArgs& a, const void* codes,
                               cudaStream_t s) {
  return a.l.block == 16 ? pick<16>(a, codes, s) : pick<32>(a, codes, s);
}

}  // namespace mx
}  // namespace moe
