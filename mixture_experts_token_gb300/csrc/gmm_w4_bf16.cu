// The 4-bit products over bfloat16 rows (gmm_w4.cuh).
#include "gmm_w4.cuh"

namespace moe {
namespace w4 {

cudaError_t launch_gmm_w4_bf16(bool dual, const GmmArgs& a, int tokens,
                              cudaStream_t s) {
  return dual ? launch_rows<__nv_bfloat16, true>(a, tokens, s)
              : launch_rows<__nv_bfloat16, false>(a, tokens, s);
}

}  // namespace w4
}  // namespace moe
