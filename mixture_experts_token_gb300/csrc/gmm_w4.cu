// Products of the routed rows with 4-bit expert weights (w4.cuh).
//
//   gate_up: h[r] = silu(x[r] Wg) * (x[r] Wu)      down: y[r] = h[r] Wd
//   W[k, n] = (code - zero) * scale, over groups of rows of W
//
// A CTA takes the 16 columns of one record (of both matrices for gate_up)
// of one group with rows, eight rows at a time; its warps split k by tiles
// and their float32 partial sums are added in warp order.  A lane's 32
// codes of a tile belong to two columns, so a scale is applied once per
// column and half tile, to the partial sum over (code - zero) * x.
#include <cuda_bf16.h>

#include "w4.cuh"

namespace moe {
namespace {

using namespace w4;

constexpr int kWarps = 8;
constexpr int kRows = 8;

struct GmmArgs {
  const void* x;
  const int32_t *offsets, *map;
  const char *w0, *w1;
  void* out;
  int32_t* status;
  Layout l;
  int n_experts, n_groups, rows;
};

// x[row, k..k+7] as float32, zero past K.
__device__ __forceinline__ void load_x(const float* x, int k, int K,
                                       float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float4 q = make_float4(0, 0, 0, 0);
    if (k + 4 * i < K) q = __ldg(reinterpret_cast<const float4*>(x + k) + i);
    f[4 * i] = q.x;
    f[4 * i + 1] = q.y;
    f[4 * i + 2] = q.z;
    f[4 * i + 3] = q.w;
  }
}
__device__ __forceinline__ void load_x(const __nv_bfloat16* x, int k, int K,
                                       float* f) {
  int4 q = make_int4(0, 0, 0, 0);
  if (k < K) q = __ldg(reinterpret_cast<const int4*>(x + k));
  const int u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __int_as_float(u[i] << 16);
    f[2 * i + 1] = __int_as_float(u[i] & 0xffff0000);
  }
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16(v);
}

template <typename T, bool DUAL>
__global__ void __launch_bounds__(kWarps * 32) gmm_w4_simt(const GmmArgs a) {
  constexpr int M = DUAL ? 2 : 1;
  __shared__ float part[kWarps][M][kRows][16];
  const int g = blockIdx.y;
  const int r0 = max(0, a.offsets[g]);
  const int r1 = min(a.rows, a.offsets[g + 1]);
  if (r0 >= r1) return;
  const int e = a.map ? a.map[g] : g;
  if (e < 0 || e >= a.n_experts) {
    if (threadIdx.x == 0 && a.status) atomicOr(a.status, MOE_DEV_BAD_INDEX);
    return;
  }
  const Layout l = a.l;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane >> 2, t = lane & 3, Gs = l.stored_groups();
  const long long at = e * l.matrix() + blockIdx.x * l.record();
  const char* rec[2] = {a.w0 + at, DUAL ? a.w1 + at : nullptr};
  const T* x = static_cast<const T*>(a.x);
  for (int r = r0; r < r1; r += kRows) {
    float acc[M][2][kRows] = {};
    for (int kt = warp; kt < l.tiles_k(); kt += kWarps) {
      uint32_t q[M][4];
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(rec[m]) +
                              kt * 32 + lane);
        q[m][0] = v.x, q[m][1] = v.y, q[m][2] = v.z, q[m][3] = v.w;
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int k = kt * kTileK + 32 * half + 8 * t;
        float s[M][2];
        int z[M][2];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int i =
                (c * Gs + (kt * kTileK + 32 * half) / l.group) * 2 + j;
            s[m][j] = __bfloat162float(
                reinterpret_cast<const __nv_bfloat16*>(rec[m] +
                                                       l.scales_at())[i]);
            z[m][j] = l.zeros ? reinterpret_cast<const uint8_t*>(
                                    rec[m] + l.zeros_at())[i]
                              : 8;
          }
#pragma unroll
        for (int b = 0; b < kRows; ++b) {
          if (r + b >= r1) break;
          float f[8];
          load_x(x + static_cast<long long>(r + b) * l.K, k, l.K, f);
#pragma unroll
          for (int m = 0; m < M; ++m)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float sum = 0.0f;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                // k + i: word 2 half + i/4, nibble of (column j, i % 4)
                const int nib = j + (i & 2) + 4 * (i & 1);
                const int code =
                    q[m][2 * half + (i >> 2)] >> (4 * nib) & 15;
                sum = fmaf(static_cast<float>(code - z[m][j]), f[i], sum);
              }
              acc[m][j][b] = fmaf(s[m][j], sum, acc[m][j][b]);
            }
        }
      }
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int b = 0; b < kRows; ++b) {
          float v = acc[m][j][b];
          v += __shfl_xor_sync(0xffffffffu, v, 1);
          v += __shfl_xor_sync(0xffffffffu, v, 2);
          if (t == 0) part[warp][m][b][c + 8 * j] = v;
        }
    __syncthreads();
    const int b = threadIdx.x >> 4, col = threadIdx.x & 15;
    const int n = blockIdx.x * kTileN + col;
    if (b < kRows && r + b < r1 && n < l.N) {
      float v[M] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int m = 0; m < M; ++m) v[m] += part[w][m][b][col];
      if (DUAL) v[0] = v[0] / (1.0f + expf(-v[0])) * v[M - 1];
      put(static_cast<T*>(a.out) + static_cast<long long>(r + b) * l.N + n,
          v[0]);
    }
    __syncthreads();
  }
}

template <bool DUAL>
cudaError_t launch(const moe_config_t& c, const GmmArgs& a, cudaStream_t s) {
  const dim3 grid(a.l.tiles_n(), a.n_groups);
  if (c.dtype == MOE_F32)
    gmm_w4_simt<float, DUAL><<<grid, kWarps * 32, 0, s>>>(a);
  else
    gmm_w4_simt<__nv_bfloat16, DUAL><<<grid, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
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
  a.x = x;
  a.w0 = static_cast<const char*>(wg);
  a.w1 = static_cast<const char*>(wu);
  a.out = h;
  return launch<true>(c, a, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t down(const moe_config_t& c, const moe_w4_t& o, const Groups& g,
                  const void* h, const int32_t* offsets, const void* wd,
                  void* y, int32_t* status, cudaStream_t s) {
  GmmArgs a = args_of(c, o, g, offsets, c.F, c.H, status);
  a.x = h;
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
              stream);
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
  return down(*cfg, *opt, g, h, group_offsets, w_down, y_sorted, status_word,
              stream);
}

}  // extern "C"
