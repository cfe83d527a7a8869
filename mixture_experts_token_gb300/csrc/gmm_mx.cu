// Entry points of the products with microscaled 4-bit experts; the kernels are
// in gmm_mx.cuh.
#include "gmm_mx.cuh"

namespace moe {

cudaError_t launch_mx_rows(int block, int R, int K, moe_dtype_t dtype,
                           const void* x, float scale, uint8_t* codes,
                           uint8_t* scales, cudaStream_t s);

namespace {

using namespace mx;

moe_status_t status_of(cudaError_t e) {
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

GmmArgs args_of(const moe_config_t& c, const moe_mx_t& o, const Groups& g,
                const int32_t* offsets, int K, int N, int32_t* status) {
  GmmArgs a = {};
  a.offsets = offsets;
  a.map = g.map;
  a.status = status;
  a.l = {K, N, o.block};
  a.n_experts = c.E;
  a.n_groups = g.n;
  a.rows = c.T * c.k;
  a.tokens = c.T;
  a.f32 = c.dtype == MOE_F32;
  a.stall_after_fills = tc::g_stall_after_fills.load();
  return a;
}

cudaError_t gate_up(const moe_config_t& c, const moe_mx_t& o, const Groups& g,
                    const uint8_t* x_codes, const uint8_t* x_scales,
                    const int32_t* offsets, const void* wg, const void* wu,
                    const float* sg, const float* su, uint8_t* h_codes,
                    uint8_t* h_scales, int32_t* status, bool early,
                    cudaStream_t s) {
  GmmArgs a = args_of(c, o, g, offsets, c.H, c.F, status);
  a.x_scales = x_scales;
  a.w0 = static_cast<const char*>(wg);
  a.w1 = static_cast<const char*>(wu);
  a.s0 = sg;
  a.s1 = su;
  a.x_scale = o.x_scale;
  a.inv_out = 1.0f / o.h_scale;
  a.h_codes = h_codes;
  a.h_scales = h_scales;
  a.early = early;
  return launch_gmm_mx_gate_up(a, x_codes, s);
}

cudaError_t down(const moe_config_t& c, const moe_mx_t& o, const Groups& g,
                 const uint8_t* h_codes, const uint8_t* h_scales,
                 const int32_t* offsets, const void* wd, const float* sd,
                 void* y, int32_t* status, bool early, cudaStream_t s) {
  GmmArgs a = args_of(c, o, g, offsets, c.F, c.H, status);
  a.x_scales = h_scales;
  a.w0 = static_cast<const char*>(wd);
  a.s0 = sd;
  a.x_scale = o.h_scale;
  a.y = y;
  a.early = early;
  return launch_gmm_mx_down(a, h_codes, s);
}

moe_status_t check(const moe_config_t* cfg, const moe_mx_t* opt,
                   int32_t n_groups, const int32_t* map, Groups* g) {
  const moe_status_t st = validate(cfg);
  if (st != MOE_OK) return st;
  if (!mx::options_ok(opt) || cfg->F < 1 ||
      !groups_of(*cfg, n_groups, map, g))
    return MOE_ERR_INVALID_ARG;
  if (!length_ok(cfg->H) || !length_ok(cfg->F)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
// The scales of the E matrices: absent with blocks of 32.
bool scales_ok(const moe_mx_t& o, const float* s) {
  return s == nullptr || (o.block == 16 && ok_ptr(s, false));
}

struct Workspace {
  uint8_t *x_codes, *x_scales, *h_codes, *h_scales;
};
Workspace carve(void* base, const moe_config_t& c, const moe_mx_t& o,
                size_t* bytes) {
  Carve cv(base);
  Workspace w;
  const size_t rows = static_cast<size_t>(c.T) * c.k;
  w.x_codes = cv.take<uint8_t>(rows * (c.H / 2));
  w.x_scales = cv.take<uint8_t>(row_scale_bytes(o.block, rows, c.H));
  w.h_codes = cv.take<uint8_t>(rows * (c.F / 2));
  w.h_scales = cv.take<uint8_t>(row_scale_bytes(o.block, rows, c.F));
  *bytes = cv.off;
  return w;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_mx_workspace_bytes(const moe_config_t* cfg, const moe_mx_t* opt) {
  Groups g;
  if (check(cfg, opt, 0, nullptr, &g) != MOE_OK) return 0;
  size_t bytes = 0;
  carve(nullptr, *cfg, *opt, &bytes);
  return bytes;
}

moe_status_t moe_gmm_gate_up_mx(
    const moe_config_t* cfg, const moe_mx_t* opt, int32_t n_groups,
    const int32_t* group_expert, const uint8_t* x_codes,
    const uint8_t* x_scales, const int32_t* group_offsets, const void* w_gate,
    const void* w_up, const float* gate_scale, const float* up_scale,
    uint8_t* h_codes, uint8_t* h_scales, int32_t* status_word,
    moe_stream_t stream) {
  Groups g;
  const moe_status_t st = check(cfg, opt, n_groups, group_expert, &g);
  if (st != MOE_OK || cfg->T == 0) return st;
  if (!ok_ptr(x_codes, true) || !ok_ptr(x_scales, true) ||
      !ok_ptr(group_offsets, false) || !ok_ptr(w_gate, true) ||
      !ok_ptr(w_up, true) || !scales_ok(*opt, gate_scale) ||
      !scales_ok(*opt, up_scale) || !ok_ptr(h_codes, true) ||
      !ok_ptr(h_scales, true))
    return MOE_ERR_INVALID_ARG;
  return status_of(gate_up(*cfg, *opt, g, x_codes, x_scales, group_offsets,
                           w_gate, w_up, gate_scale, up_scale, h_codes,
                           h_scales, status_word, false, stream));
}

moe_status_t moe_gmm_down_mx(const moe_config_t* cfg, const moe_mx_t* opt,
                             int32_t n_groups, const int32_t* group_expert,
                             const uint8_t* h_codes, const uint8_t* h_scales,
                             const int32_t* group_offsets, const void* w_down,
                             const float* down_scale, void* y_sorted,
                             int32_t* status_word, moe_stream_t stream) {
  Groups g;
  const moe_status_t st = check(cfg, opt, n_groups, group_expert, &g);
  if (st != MOE_OK || cfg->T == 0) return st;
  if (!ok_ptr(h_codes, true) || !ok_ptr(h_scales, true) ||
      !ok_ptr(group_offsets, false) || !ok_ptr(w_down, true) ||
      !scales_ok(*opt, down_scale) || !ok_ptr(y_sorted, true))
    return MOE_ERR_INVALID_ARG;
  return status_of(down(*cfg, *opt, g, h_codes, h_scales, group_offsets,
                        w_down, down_scale, y_sorted, status_word, false,
                        stream));
}

moe_status_t moe_gmm_swiglu_mx(
    const moe_config_t* cfg, const moe_mx_t* opt, const void* x_sorted,
    const int32_t* group_offsets, const void* w_gate, const void* w_up,
    const void* w_down, const float* gate_scale, const float* up_scale,
    const float* down_scale, void* y_sorted, int32_t* status_word,
    void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  Groups g;
  const moe_status_t st = check(cfg, opt, 0, nullptr, &g);
  if (st != MOE_OK || cfg->T == 0) return st;
  if (!ok_ptr(x_sorted, true) || !ok_ptr(group_offsets, false) ||
      !ok_ptr(w_gate, true) || !ok_ptr(w_up, true) || !ok_ptr(w_down, true) ||
      !scales_ok(*opt, gate_scale) || !scales_ok(*opt, up_scale) ||
      !scales_ok(*opt, down_scale) || !ok_ptr(y_sorted, true))
    return MOE_ERR_INVALID_ARG;
  size_t bytes = 0;
  const Workspace w = carve(workspace, *cfg, *opt, &bytes);
  if (!ok_ptr(workspace, true) || workspace_bytes < bytes)
    return MOE_ERR_WORKSPACE;
  // Each product starts while the kernel before it drains: its weights and
  // offsets were final before the first of the three started.
  cudaError_t e =
      launch_mx_rows(opt->block, cfg->T * cfg->k, cfg->H, cfg->dtype, x_sorted,
                     opt->x_scale, w.x_codes, w.x_scales, stream);
  if (e == cudaSuccess)
    e = gate_up(*cfg, *opt, g, w.x_codes, w.x_scales, group_offsets, w_gate,
                w_up, gate_scale, up_scale, w.h_codes, w.h_scales,
                status_word, true, stream);
  if (e == cudaSuccess)
    e = down(*cfg, *opt, g, w.h_codes, w.h_scales, group_offsets, w_down,
             down_scale, y_sorted, status_word, true, stream);
  return status_of(e);
}

}  // extern "C"
