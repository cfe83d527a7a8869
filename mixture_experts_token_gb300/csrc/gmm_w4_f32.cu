// The 4-bit products over float32 rows (gmm_w4.cuh).
#include "gmm_w4.cuh"

namespace moe {
namespace w4 {

cudaError_t launch_gmm_w4_f32(bool dual, const GmmArgs& a, int tokens,
                              cudaStream_t s) {
  return dual ? launch_rows<float, true>(a, tokens, s)
              : launch_rows<float, false>(a, tokens, s);
}

}  // namespace w4
}  // namespace moe
