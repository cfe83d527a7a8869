// Entry points of the products with 4-bit expert weights; the kernels are in
// gmm_w4.cuh.
#include "gmm_w4.cuh"

namespace moe {
namespace {

using namespace w4;

template <bool DUAL>
cudaError_t launch(const moe_config_t& c, const GmmArgs& a, cudaStream_t s) {
  return c.dtype == MOE_F32 ? launch_gmm_w4_f32(DUAL, a, c.T, s)
                            : launch_gmm_w4_bf16(DUAL, a, c.T, s);
}

GmmArgs args_of(const moe_config_t& c, const moe_w4_t& o, const Groups& g,
                const int32_t* offsets, int K, int N, int32_t* status) {
  GmmArgs a = {};
  a.offsets = offsets;
  a.map = g.map;
  a.status = status;
  a.l = layout(o, K, N);
  a.n_experts = c.E;
  a.n_groups = g.n;
  a.rows = c.T * c.k;
  return a;
}

moe_status_t gate_up(const moe_config_t& c, const moe_w4_t& o,
                     const Groups& g, const void* x, const int32_t* offsets,
                     const void* wg, const void* wu, void* h, int32_t* status,
                     cudaStream_t s) {
  GmmArgs a = args_of(c, o, g, offsets, c.H, c.F, status);
  a.x = static_cast<const char*>(x);
  a.w0 = static_cast<const char*>(wg);
  a.w1 = static_cast<const char*>(wu);
  a.out = h;
  return launch<true>(c, a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t down(const moe_config_t& c, const moe_w4_t& o, const Groups& g,
                  const void* h, const int32_t* offsets, const void* wd,
                  void* y, int32_t* status, bool early, cudaStream_t s) {
  GmmArgs a = args_of(c, o, g, offsets, c.F, c.H, status);
  a.early = early;
  a.x = static_cast<const char*>(h);
  a.w0 = static_cast<const char*>(wd);
  a.out = y;
  return launch<false>(c, a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t check(const moe_config_t* cfg, const moe_w4_t* opt,
                   int32_t n_groups, const int32_t* map, Groups* g) {
  const moe_status_t st = validate(cfg);
  if (st != MOE_OK) return st;
  if (!w4::options_ok(opt) || cfg->F < 1 ||
      !groups_of(*cfg, n_groups, map, g))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_gmm_gate_up_w4(const moe_config_t* cfg, const moe_w4_t* opt,
                                int32_t n_groups, const int32_t* group_expert,
                                const void* x_sorted,
                                const int32_t* group_offsets,
                                const void* w_gate, const void* w_up, void* h,
                                int32_t* status_word, moe_stream_t stream) {
  Groups g;
  const moe_status_t st = check(cfg, opt, n_groups, group_expert, &g);
  if (st != MOE_OK || cfg->T == 0) return st;
  if (!ok_ptr(x_sorted, true) || !ok_ptr(group_offsets, false) ||
      !ok_ptr(w_gate, true) || !ok_ptr(w_up, true) || !ok_ptr(h, true))
    return MOE_ERR_INVALID_ARG;
  return gate_up(*cfg, *opt, g, x_sorted, group_offsets, w_gate, w_up, h,
                 status_word, stream);
}

moe_status_t moe_gmm_down_w4(const moe_config_t* cfg, const moe_w4_t* opt,
                             int32_t n_groups, const int32_t* group_expert,
                             const void* h, const int32_t* group_offsets,
                             const void* w_down, void* y_sorted,
                             int32_t* status_word, moe_stream_t stream) {
  Groups g;
  const moe_status_t st = check(cfg, opt, n_groups, group_expert, &g);
  if (st != MOE_OK || cfg->T == 0) return st;
  if (!ok_ptr(h, true) || !ok_ptr(group_offsets, false) ||
      !ok_ptr(w_down, true) || !ok_ptr(y_sorted, true))
    return MOE_ERR_INVALID_ARG;
  return down(*cfg, *opt, g, h, group_offsets, w_down, y_sorted, status_word,
              false, stream);
}

moe_status_t moe_gmm_swiglu_w4(const moe_config_t* cfg, const moe_w4_t* opt,
                               const void* x_sorted,
                               const int32_t* group_offsets,
                               const void* w_gate, const void* w_up,
                               const void* w_down, void* h, void* y_sorted,
                               int32_t* status_word, moe_stream_t stream) {
  Groups g;
  const moe_status_t st = check(cfg, opt, 0, nullptr, &g);
  if (st != MOE_OK || cfg->T == 0) return st;
  if (!ok_ptr(x_sorted, true) || !ok_ptr(group_offsets, false) ||
      !ok_ptr(w_gate, true) || !ok_ptr(w_up, true) ||
      !ok_ptr(w_down, true) || !ok_ptr(h, true) || !ok_ptr(y_sorted, true))
    return MOE_ERR_INVALID_ARG;
  const moe_status_t up = gate_up(*cfg, *opt, g, x_sorted, group_offsets,
                                  w_gate, w_up, h, status_word, stream);
  if (up != MOE_OK) return up;
  // Only gate_up's h is still to come when this one starts early: its
  // weights and offsets were final before gate_up started.
  return down(*cfg, *opt, g, h, group_offsets, w_down, y_sorted, status_word,
              true, stream);
}

}  // extern "C"
