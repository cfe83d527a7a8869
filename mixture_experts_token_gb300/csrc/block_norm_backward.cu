// Backward of the block's norms (forward: block_norm.cu).
//
// With vh = v * rstd and w' = w_offset + w, the norm N(v; w) = vh * w' has
//   dv = rstd * (dN * w' - vh * mean_c(dN * w' * vh)),   dw = sum_t dN * vh.
// The branch's end out = res_scale * x + gate * N(y; w_post) followed by
// h_next = N(out; w_next) then has, with dO the whole gradient of `out`,
//   dO = dout + dN^T(dh_next)        dx = res_scale * dO
//   dn = dO * gate                   dy = rstd_y * (dn w' - yh mean(dn w' yh))
//   dgate = dO * N(y)  summed to the gate's shape.
// Two facts save work.  The row sum of the second norm and a per-token
// gate's gradient are one reduction, sum_c dO * N(y).  And one column sum
// A[c] = sum_t dO yh (times the gate, where it differs by row) gives both
// column gradients of a per-channel gate: dw_post = gate * A, dgate = w' A.
//
// Each CTA walks its rows with the column sums in registers (a thread keeps
// the same columns) and leaves one partial per CTA; a second kernel adds the
// partials in CTA order.  No atomics: the result does not depend on timing.
#include <cuda_bf16.h>

#include <algorithm>

#include "block_norm.cuh"

namespace moe {
namespace {

using namespace block;

struct BwdArgs {
  const int4 *y, *v, *dout, *dh;  // v: the stored row the next norm read
  const float *w_post, *w_next, *rstd_y, *rstd_v;
  const void* gate;
  int4 *dx, *dy;
  void* dgate;   // per token or in full; per channel goes to the partials
  float* parts;  // [grid, 2, H]: sums of dO yh (gate), then of dh vh
  float inv_h, w_offset, res_scale;
  int T, n16, gate_kind;
  bool vec_w;
};

// POST: the branch's end is part of it; else only the norm of v.
template <typename T, int NV, bool WARP, int MAXT, bool POST>
__global__ void __launch_bounds__(MAXT) block_bwd_kernel(const BwdArgs a) {
  using V = Vec<T>;
  constexpr int N = V::N;
  __shared__ float red[2][32];
  __shared__ float cols[WARP ? 32 * NV * N : 1];
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int step = WARP ? 32 : blockDim.x;
  const int first = WARP ? blockIdx.x * kRowWarps + (threadIdx.x >> 5)
                         : blockIdx.x;
  const int rows = WARP ? gridDim.x * kRowWarps : gridDim.x;
  float sum_post[NV][N], sum_next[NV][N];
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int i = 0; i < N; ++i) sum_post[u][i] = sum_next[u][i] = 0.0f;

  for (int t = first; t < a.T; t += rows) {
    const long long base = static_cast<long long>(t) * a.n16;
    int4 v[NV], dh[NV], go[NV], y[NV];
    float d[NV][N];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = tid + u * step;
      v[u] = dh[u] = go[u] = y[u] = make_int4(0, 0, 0, 0);
      if (c < a.n16) {
        if (a.dh) {
          v[u] = load_stream(a.v + base + c);
          dh[u] = load_stream(a.dh + base + c);
        }
        if (a.dout) go[u] = load_stream(a.dout + base + c);
        if (POST) y[u] = load_stream(a.y + base + c);
      }
    }
    // dO = dout + rstd (dh w' - vh mean(dh w' vh))
    if (a.dh) {
      const float r = a.rstd_v[t];
      float s = 0.0f;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int c = tid + u * step;
        float fv[N], w[N];
        V::load(v[u], fv);
        V::load(dh[u], d[u]);
        if (c < a.n16) {
          load_weight<N>(a.w_next, c, a.vec_w, w);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) w[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float vh = fv[i] * r;
          sum_next[u][i] = fmaf(d[u][i], vh, sum_next[u][i]);
          d[u][i] *= a.w_offset + w[i];
          s = fmaf(d[u][i], vh, s);
        }
      }
      s = row_sum<WARP>(s, red[0]) * a.inv_h;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float fv[N], g[N];
        V::load(v[u], fv);
        V::load(go[u], g);
#pragma unroll
        for (int i = 0; i < N; ++i)
          d[u][i] = fmaf(r, d[u][i] - fv[i] * r * s, g[i]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < NV; ++u) V::load(go[u], d[u]);
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = tid + u * step;
      float f[N];
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = a.res_scale * d[u][i];
      if (c < a.n16) store_stream(a.dx + base + c, V::store(f));
    }
    if (!POST) continue;
    // The branch.  A per-token gate multiplies whole rows, so it stays out
    // of the row sum, which is then that gate's gradient.
    const bool post = a.w_post != nullptr;
    const float r = post ? a.rstd_y[t] : 1.0f;
    const bool token = a.gate_kind == MOE_GATE_TOKEN;
    const float gt = token ? static_cast<const float*>(a.gate)[t] : 1.0f;
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = tid + u * step;
      if (c >= a.n16) continue;
      float fy[N], w[N], g[N];
      V::load(y[u], fy);
#pragma unroll
      for (int i = 0; i < N; ++i) fy[i] *= r;
      if (post) {
        load_weight<N>(a.w_post, c, a.vec_w, w);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] += a.w_offset;
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = 1.0f;
      }
      if (a.gate_kind == MOE_GATE_FULL) {
        float dg[N];
        V::load(load_stream(static_cast<const int4*>(a.gate) + base + c), g);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dg[i] = d[u][i] * fy[i] * w[i];
          d[u][i] *= g[i];
        }
        store_stream(static_cast<int4*>(a.dgate) + base + c, V::store(dg));
      }
      // a per-channel gate multiplies this column sum once, at the end
#pragma unroll
      for (int i = 0; i < N; ++i)
        sum_post[u][i] = fmaf(gt * d[u][i], fy[i], sum_post[u][i]);
      if (a.gate_kind == MOE_GATE_CHANNEL) {
        load_weight<N>(static_cast<const float*>(a.gate), c, a.vec_w, g);
#pragma unroll
        for (int i = 0; i < N; ++i) d[u][i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        d[u][i] *= w[i];
        s = fmaf(d[u][i], fy[i], s);
      }
    }
    if (post || token) {
      s = row_sum<WARP>(s, red[1]);
      if (token && tid == 0) static_cast<float*>(a.dgate)[t] = s;
      s = post ? s * a.inv_h : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = tid + u * step;
      if (c >= a.n16) continue;
      float fy[N];
      V::load(y[u], fy);
#pragma unroll
      for (int i = 0; i < N; ++i)
        d[u][i] = gt * r * (d[u][i] - (post ? fy[i] * r * s : 0.0f));
      store_stream(a.dy + base + c, V::store(d[u]));
    }
  }

  // One partial per CTA: this thread's columns, or, where every warp holds
  // whole rows, the warps' columns added in warp order.
  const int H = a.n16 * N;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float* out = a.parts + (static_cast<long long>(blockIdx.x) * 2 + q) * H;
    if (WARP) {
      for (int w = 0; w < kRowWarps; ++w) {
        if (static_cast<int>(threadIdx.x >> 5) == w) {
#pragma unroll
          for (int u = 0; u < NV; ++u)
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const int at = (tid + u * step) * N + i;
              const float add = q == 0 ? sum_post[u][i] : sum_next[u][i];
              cols[at] = w == 0 ? add : cols[at] + add;
            }
        }
        __syncthreads();
      }
      for (int c = threadIdx.x; c < H; c += blockDim.x) out[c] = cols[c];
      __syncthreads();
    } else {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int c = tid + u * step;
        if (c >= a.n16) continue;
#pragma unroll
        for (int i = 0; i < N; i += 4)
          *reinterpret_cast<float4*>(out + c * N + i) =
              q == 0 ? make_float4(sum_post[u][i], sum_post[u][i + 1],
                                   sum_post[u][i + 2], sum_post[u][i + 3])
                     : make_float4(sum_next[u][i], sum_next[u][i + 1],
                                   sum_next[u][i + 2], sum_next[u][i + 3]);
      }
    }
  }
}

struct ColArgs {
  const float *parts, *w_post, *gate;  // gate: per channel, or null
  float *dw_post, *dgate, *dw_next;
  float w_offset;
  int n_parts, H;
  bool accumulate;
};

constexpr int kColThreads = 32;  // columns of a CTA
constexpr int kColRows = 8;      // partials added side by side

// Adds the CTAs' partials: blockIdx.y 0 the branch's column sums, 1 the next
// norm's.
__global__ void __launch_bounds__(kColThreads* kColRows)
    block_bwd_columns(const ColArgs a) {
  __shared__ float part[kColRows][kColThreads];
  const int c = blockIdx.x * kColThreads + threadIdx.x;
  const int q = blockIdx.y;
  float s = 0.0f;
  if (c < a.H) {
    const float* p = a.parts + static_cast<long long>(q) * a.H + c;
#pragma unroll 4
    for (int i = threadIdx.y; i < a.n_parts; i += kColRows)
      s += p[static_cast<long long>(i) * 2 * a.H];
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || c >= a.H) return;
#pragma unroll
  for (int i = 1; i < kColRows; ++i) s += part[i][threadIdx.x];
  const auto put = [&](float* p, float v) {
    if (p) p[c] = a.accumulate ? p[c] + v : v;
  };
  if (q == 1) {
    put(a.dw_next, s);
    return;
  }
  const float w = a.w_post ? a.w_offset + a.w_post[c] : 1.0f;
  put(a.dw_post, a.gate ? a.gate[c] * s : s);
  if (a.gate) put(a.dgate, w * s);
}

// CTAs of the row kernel (and partials): two per SM where the rows allow.
constexpr int kMaxParts = 304;

int parts_of(const moe_config_t& c) {
  const int n = row_words(c) <= 128 ? (c.T + kRowWarps - 1) / kRowWarps : c.T;
  return std::max(1, std::min(n, kMaxParts));
}

template <typename T, int NV, bool WARP, int MAXT>
cudaError_t launch_post(const BwdArgs& a, bool post, int grid, int threads,
                        cudaStream_t s) {
  if (post)
    block_bwd_kernel<T, NV, WARP, MAXT, true><<<grid, threads, 0, s>>>(a);
  else
    block_bwd_kernel<T, NV, WARP, MAXT, false><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rows(const BwdArgs& a, bool post, int grid,
                        cudaStream_t s) {
  constexpr int W = kRowWarps * 32;
  if (a.n16 <= 32) return launch_post<T, 1, true, W>(a, post, grid, W, s);
  if (a.n16 <= 64) return launch_post<T, 2, true, W>(a, post, grid, W, s);
  if (a.n16 <= 128) return launch_post<T, 4, true, W>(a, post, grid, W, s);
  const auto threads = [&](int nv) {
    return ((a.n16 + nv - 1) / nv + 31) / 32 * 32;
  };
  if (a.n16 <= 512)
    return launch_post<T, 1, false, 512>(a, post, grid, threads(1), s);
  if (a.n16 <= 1024)
    return launch_post<T, 2, false, 512>(a, post, grid, threads(2), s);
  if (a.n16 <= 2048)
    return launch_post<T, 4, false, 512>(a, post, grid, threads(4), s);
  return launch_post<T, 4, false, 1024>(a, post, grid, threads(4), s);
}

moe_status_t run(const moe_config_t& c, BwdArgs a, ColArgs ca, bool post,
                 void* workspace, cudaStream_t s) {
  a.T = c.T;
  a.n16 = row_words(c);
  a.inv_h = 1.0f / static_cast<float>(c.H);
  Carve cv(workspace);
  const int grid = parts_of(c);
  a.parts = cv.take<float>(static_cast<size_t>(grid) * 2 * c.H);
  ca.parts = a.parts;
  ca.H = c.H;
  ca.n_parts = grid;
  ca.w_offset = a.w_offset;
  cudaError_t e = c.dtype == MOE_F32
                      ? launch_rows<float>(a, post, grid, s)
                      : launch_rows<__nv_bfloat16>(a, post, grid, s);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  const dim3 cols((c.H + kColThreads - 1) / kColThreads, 2);
  block_bwd_columns<<<cols, dim3(kColThreads, kColRows), 0, s>>>(ca);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t check(const moe_config_t* cfg, const moe_block_norm_t* opt,
                   const void* workspace, size_t workspace_bytes) {
  const moe_status_t st = moe_validate_config(cfg);
  if (st != MOE_OK) return st;
  if (!options_ok(opt)) return MOE_ERR_INVALID_ARG;
  if (row_words(*cfg) > kMaxRowWords) return MOE_ERR_UNSUPPORTED;
  if (workspace == nullptr || workspace_bytes < block_backward_bytes(*cfg) ||
      !ok_ptr(workspace, true))
    return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

}  // namespace

size_t block_backward_bytes(const moe_config_t& c) {
  Carve cv(nullptr);
  cv.take<float>(static_cast<size_t>(parts_of(c)) * 2 * c.H);
  return align_up(cv.off, 256);
}

}  // namespace moe

using namespace moe;
using namespace moe::block;

extern "C" {

moe_status_t moe_norm_backward(const moe_config_t* cfg,
                               const moe_block_norm_t* opt, const void* x,
                               const float* w, const float* rstd,
                               const void* dh, const void* dres, void* dx,
                               float* dw, int32_t accumulate,
                               void* workspace, size_t workspace_bytes,
                               moe_stream_t stream) {
  const moe_status_t st = check(cfg, opt, workspace, workspace_bytes);
  if (st != MOE_OK) return st;
  if (!ok_ptr(w, false) || !ok_ptr(dw, false)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!ok_ptr(x, true) || !ok_ptr(rstd, false) ||
                     !ok_ptr(dh, true) || !opt_ptr(dres, true) ||
                     !ok_ptr(dx, true)))
    return MOE_ERR_INVALID_ARG;
  BwdArgs a = {};
  a.v = static_cast<const int4*>(x);
  a.w_next = w;
  a.rstd_v = rstd;
  a.dh = static_cast<const int4*>(dh);
  a.dout = static_cast<const int4*>(dres);
  a.dx = static_cast<int4*>(dx);
  a.w_offset = opt->w_offset;
  a.res_scale = 1.0f;
  a.vec_w = aligned16(w);
  ColArgs ca = {};
  ca.dw_next = dw;
  ca.accumulate = accumulate != 0;
  return run(*cfg, a, ca, false, workspace, stream);
}

moe_status_t moe_block_out_backward(
    const moe_config_t* cfg, const moe_block_norm_t* opt, const void* y,
    const float* w_post, const void* gate, const float* rstd_y,
    const void* out, const float* w_next, const float* rstd_out,
    const void* dout, const void* dh_next, void* dx, void* dy,
    float* dw_post, void* dgate, float* dw_next, int32_t accumulate,
    void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  const moe_status_t st = check(cfg, opt, workspace, workspace_bytes);
  if (st != MOE_OK) return st;
  const bool next = dh_next != nullptr;
  if (dout == nullptr && !next && cfg->T > 0) return MOE_ERR_INVALID_ARG;
  if (!opt_ptr(w_post, false) || !opt_ptr(w_next, false) ||
      (w_post != nullptr && !ok_ptr(dw_post, false)) ||
      (w_next != nullptr && !ok_ptr(dw_next, false)) ||
      (next && w_next == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (opt->gate_kind == MOE_GATE_CHANNEL &&
      (!ok_ptr(gate, false) || !ok_ptr(dgate, false)))
    return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 &&
      (!ok_ptr(y, true) || !gate_ok(*opt, gate) || !opt_ptr(dout, true) ||
       !opt_ptr(dh_next, true) || !ok_ptr(dx, true) || !ok_ptr(dy, true) ||
       (w_post != nullptr && !ok_ptr(rstd_y, false)) ||
       (next && (!ok_ptr(out, true) || !ok_ptr(rstd_out, false))) ||
       (opt->gate_kind != MOE_GATE_NONE &&
        !ok_ptr(dgate, opt->gate_kind == MOE_GATE_FULL))))
    return MOE_ERR_INVALID_ARG;
  BwdArgs a = {};
  a.y = static_cast<const int4*>(y);
  a.v = static_cast<const int4*>(out);
  a.dout = static_cast<const int4*>(dout);
  a.dh = static_cast<const int4*>(dh_next);
  a.w_post = w_post;
  a.w_next = w_next;
  a.rstd_y = rstd_y;
  a.rstd_v = rstd_out;
  a.gate = gate;
  a.dx = static_cast<int4*>(dx);
  a.dy = static_cast<int4*>(dy);
  a.dgate = dgate;
  a.w_offset = opt->w_offset;
  a.res_scale = opt->res_scale;
  a.gate_kind = opt->gate_kind;
  a.vec_w = columns_aligned(*opt, w_post, w_next, gate);
  ColArgs ca = {};
  ca.w_post = w_post;
  ca.dw_post = w_post ? dw_post : nullptr;
  ca.dw_next = w_next ? dw_next : nullptr;
  if (opt->gate_kind == MOE_GATE_CHANNEL) {
    ca.gate = static_cast<const float*>(gate);
    ca.dgate = static_cast<float*>(dgate);
  }
  ca.accumulate = accumulate != 0;
  return run(*cfg, a, ca, true, workspace, stream);
}

}  // extern "C"
