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
//
// Measured, 8192 x 7168 bf16 with a channel gate: 126 us (705 MB, 5.6 TB/s);
// 2047 x 5120 float32 with a full gate 63 us (335 MB, 5.3 TB/s).  HBM bounds
// the row kernel; what is left is two block-wide reductions a row (16 warps,
// one CTA an SM) and 9 us for the column sums, which overlap its tail.
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

// Rows wider than the streamed form holds (1280 words): one row per CTA, in
// registers, which the column sums of four words a thread take most of.  bf16
// spills: 376 bytes a thread with the branch up to 2048 words, 1756 (732
// without it) above, where a thread has 64 registers.  Measured with a channel
// gate: 2048 x 7168 float32 99 us (3.6 TB/s), 2048 x 16384 bf16 152 us (2.7),
// 1024 x 32768 bf16 364 us (1.1); the norm alone 50, 75 and 159 us.  The
// streamed form at its widest, 2048 x 10240 bf16, takes 88 us (2.9 TB/s; it
// spills up to 196 bytes) and the norm alone 37 us (4.5).
// POST: the branch's end is part of it; else only the norm of v.
template <typename T, int NV, int MAXT, bool POST>
__global__ void __launch_bounds__(MAXT) block_bwd_kernel(const BwdArgs a) {
  using V = Vec<T>;
  constexpr int N = V::N;
  __shared__ float red[2][32];
  const int tid = threadIdx.x, step = blockDim.x;
  float sum_post[NV][N], sum_next[NV][N];
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int i = 0; i < N; ++i) sum_post[u][i] = sum_next[u][i] = 0.0f;

  // Row sums so far: they alternate between two buffers, so that a warp that
  // is a sum ahead does not write what another still reads.
  int sums = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
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
      s = row_sum<false>(s, red[sums++ & 1]) * a.inv_h;
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
      s = row_sum<false>(s, red[sums++ & 1]);
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

  // one partial per CTA
#pragma unroll
  for (int q = POST ? 0 : 1; q < 2; ++q) {
    float* out =
        a.parts + (static_cast<long long>(blockIdx.x) * 2 + q) * a.n16 * N;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = tid + u * step;
      if (c >= a.n16) continue;
      const float(&f)[N] = q == 0 ? sum_post[u] : sum_next[u];
#pragma unroll
      for (int i = 0; i < N; i += 4)
        *reinterpret_cast<float4*>(out + c * N + i) =
            make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    }
  }
}

// ---- rows streamed through shared memory -------------------------------
// S rows ahead.  A row belongs to a group of `threads` threads, of which a
// CTA has one or more: thread tid of a group holds word tid of the row (and
// tid + threads with NV = 2), copies it to shared memory itself and reads it
// back where it is needed, so only the column weights, the column sums and
// dO stay in registers.  A word is copied anew, for the row S on, as soon as
// it has been read for the last time.
template <typename T, int NV, int MAXT, bool POST, int GATE, int S>
__global__ void __launch_bounds__(MAXT)
    block_bwd_stream(const BwdArgs a, int threads) {
  using V = Vec<T>;
  constexpr int N = V::N;
  constexpr bool FULL = GATE == MOE_GATE_FULL;
  constexpr bool TOKEN = GATE == MOE_GATE_TOKEN;
  constexpr int W = 3 + POST + FULL;  // groups of copies of a row
  extern __shared__ __align__(16) char queue[];
  __shared__ float red[2][32];
  // All CTAs of this grid are resident, so the column sums' can only take
  // what they leave.
  launch::let_next_start();
  const int group = threadIdx.x / threads, tid = threadIdx.x % threads;
  const int groups = blockDim.x / threads;
  const int t0 = blockIdx.x * groups + group, t_step = gridDim.x * groups;
  const bool next = a.dh != nullptr;
  const bool post = POST && a.w_post != nullptr;
  const bool in = tid < a.n16;
  const auto held = [&](int u) {
    return NV == 1 ? in : tid + u * threads < a.n16;
  };
  const long long row_step = static_cast<long long>(t_step) * a.n16;
  long long base = static_cast<long long>(t0) * a.n16 + tid;
  // a row's words in shared memory, in this order; absent ones have no room
  const uint32_t word = threads * NV * 16;
  const uint32_t at_v = word, at_go = next ? 2 * word : 0;
  const uint32_t at_y = at_go + (a.dout ? word : 0);
  const uint32_t at_g = at_y + word;
  const uint32_t row_bytes =
      at_y + (POST ? word : 0) + (FULL ? word : 0);
  const uint32_t first =
      shared_address(queue) + group * S * row_bytes + tid * 16;
  const uint32_t last = first + (S - 1) * row_bytes;
  const int4* gate = static_cast<const int4*>(a.gate);
  const auto copy = [&](const int4* p, long long at, uint32_t dst) {
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (held(u)) copy16(dst + u * threads * 16, p + at + u * threads);
  };
  // places past the row's end stay zero
#pragma unroll
  for (int u = 0; u < NV; ++u)
    if (!held(u))
      for (uint32_t p = 0; p < S * row_bytes; p += word)
        zero16(first + p + u * threads * 16);
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const bool on = t0 + static_cast<long long>(i) * t_step < a.T;
    const long long at = base + i * row_step;
    const uint32_t dst = first + i * row_bytes;
    if (on && next) copy(a.dh, at, dst);
    copies_commit();
    if (on && next) copy(a.v, at, dst + at_v);
    copies_commit();
    if (on && a.dout) copy(a.dout, at, dst + at_go);
    copies_commit();
    if (POST) {
      if (on) copy(a.y, at, dst + at_y);
      copies_commit();
    }
    if (FULL) {
      if (on) copy(gate, at, dst + at_g);
      copies_commit();
    }
  }
  // per-row numbers, loaded a row ahead
  const float* gates = static_cast<const float*>(a.gate);
  float rv = 0.0f, ry = 1.0f, gt = 1.0f;
  const auto load_row = [&](long long t) {
    if (t >= a.T) return;
    if (next) rv = a.rstd_v[t];
    if (post) ry = a.rstd_y[t];
    if (TOKEN) gt = gates[t];
  };
  load_row(t0);

  // w' of the next norm, and of the post norm (times a channel's gate)
  float wn[NV][N], wp[NV][N];
  float sum_post[NV][N], sum_next[NV][N];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int c = tid + u * threads;
    columns_or<N>(next ? a.w_next : nullptr, c, c < a.n16, a.vec_w, 0.0f,
                  wn[u]);
    if (POST) {
      columns_or<N>(a.w_post, c, c < a.n16, a.vec_w, 1.0f, wp[u]);
      float g[N];
      columns_or<N>(GATE == MOE_GATE_CHANNEL ? gates : nullptr, c, c < a.n16,
                    a.vec_w, 1.0f, g);
#pragma unroll
      for (int i = 0; i < N; ++i)
        wp[u][i] = g[i] * (post ? wp[u][i] + a.w_offset : 1.0f);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      wn[u][i] += a.w_offset;
      sum_post[u][i] = sum_next[u][i] = 0.0f;
    }
  }
  const auto load = [&](uint32_t p, int u, float (&f)[N]) {
    V::load(read16(p + u * threads * 16), f);
  };
  uint32_t src = first;
  int sums = 0;  // row sums so far: they alternate between two buffers
#pragma unroll 1
  for (int t = t0; t < a.T; t += t_step) {
    const float r_v = rv, r_y = ry, g_t = gt;
    load_row(static_cast<long long>(t) + t_step);
    const bool more = static_cast<long long>(t) + S * t_step < a.T;
    const long long ahead = base + S * row_step;
    float d[NV][N];
    copies_wait<S * W - 2>();  // dh and v
    if (next) {
      // dO = dout + rstd (dh w' - vh mean(dh w' vh))
      float s = 0.0f;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float v[N];
        load(src + at_v, u, v);
        load(src, u, d[u]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float vh = v[i] * r_v;
          sum_next[u][i] = fmaf(d[u][i], vh, sum_next[u][i]);
          d[u][i] *= wn[u][i];
          s = fmaf(d[u][i], vh, s);
        }
      }
      if (more) copy(a.dh, ahead, src);
      copies_commit();
      s = group_sum(s, red[sums++ & 1], group, threads) * a.inv_h * r_v * r_v;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float v[N];
        load(src + at_v, u, v);
#pragma unroll
        for (int i = 0; i < N; ++i)
          d[u][i] = fmaf(r_v, d[u][i], -(v[i] * s));
      }
      if (more) copy(a.v, ahead, src + at_v);
      copies_commit();
    } else {
      copies_commit();
      copies_commit();
    }
    copies_wait<S * W - 1>();  // dout
    if (a.dout) {
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float g[N];
        load(src + at_go, u, g);
#pragma unroll
        for (int i = 0; i < N; ++i) d[u][i] = next ? d[u][i] + g[i] : g[i];
      }
      if (more) copy(a.dout, ahead, src + at_go);
    }
    copies_commit();
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      float f[N];
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = a.res_scale * d[u][i];
      if (held(u)) store_stream(a.dx + base + u * threads, V::store(f));
    }
    if (POST) {
      // The branch.  A per-token gate multiplies whole rows, so it stays
      // out of the row sum, which is then that gate's gradient; a
      // per-channel gate multiplies its column sum once, at the end.
      copies_wait<S * W - (FULL ? 2 : 1)>();  // y (and the gate)
      float s = 0.0f;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float y[N], g[N];
        load(src + at_y, u, y);
        if (FULL) {
          float dg[N];
          load(src + at_g, u, g);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            y[i] *= r_y;
            dg[i] = d[u][i] * y[i] * wp[u][i];
            d[u][i] *= g[i];
            sum_post[u][i] = fmaf(d[u][i], y[i], sum_post[u][i]);
            d[u][i] *= wp[u][i];
            s = fmaf(d[u][i], y[i], s);
          }
          if (held(u))
            store_stream(static_cast<int4*>(a.dgate) + base + u * threads,
                         V::store(dg));
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            y[i] *= r_y;
            sum_post[u][i] = fmaf(TOKEN ? g_t * d[u][i] : d[u][i], y[i],
                                  sum_post[u][i]);
            d[u][i] *= wp[u][i];
            s = fmaf(d[u][i], y[i], s);
          }
        }
      }
      if (post || TOKEN) {
        s = group_sum(s, red[sums++ & 1], group, threads);
        if (TOKEN && tid == 0) static_cast<float*>(a.dgate)[t] = s;
        s = post ? s * a.inv_h * r_y : 0.0f;
      }
      const float scale = g_t * r_y;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float y[N];
        load(src + at_y, u, y);
#pragma unroll
        for (int i = 0; i < N; ++i)
          d[u][i] = scale * (d[u][i] - (post ? y[i] * s : 0.0f));
        if (held(u)) store_stream(a.dy + base + u * threads, V::store(d[u]));
      }
      if (more) copy(a.y, ahead, src + at_y);
      copies_commit();
      if (FULL) {
        if (more) copy(gate, ahead, src + at_g);
        copies_commit();
      }
    }
    src = src == last ? first : src + row_bytes;
    base += row_step;
  }
  copies_wait<0>();

  // One partial per CTA: this thread's columns, or the groups' added in
  // group order.
  float* cols = reinterpret_cast<float*>(queue);
  const int H = a.n16 * N;
#pragma unroll
  for (int q = POST ? 0 : 1; q < 2; ++q) {
    float* out = a.parts + (static_cast<long long>(blockIdx.x) * 2 + q) * H;
    for (int g = 0; g < groups; ++g) {
      if (groups > 1) __syncthreads();
      if (g != group) continue;
      float* to = g == groups - 1 ? out : cols;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const float(&f)[N] = q == 0 ? sum_post[u] : sum_next[u];
        const int c = (tid + u * threads) * N;
        if (!held(u)) continue;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          float4 v = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
          if (g > 0) {
            const float4 w = *reinterpret_cast<const float4*>(cols + c + i);
            v = make_float4(w.x + v.x, w.y + v.y, w.z + v.z, w.w + v.w);
          }
          *reinterpret_cast<float4*>(to + c + i) = v;
        }
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
constexpr int kColRows = 32;     // partials added side by side
static_assert(kColThreads == 32 && kColRows == 32, "summed by warps");

// Adds the CTAs' partials: the next norm's column sums where blockIdx.y is
// the last, else (with two) the branch's.
__global__ void __launch_bounds__(kColThreads* kColRows)
    block_bwd_columns(const ColArgs a) {
  __shared__ float part[kColRows][kColThreads + 1];
  int c = blockIdx.x * kColThreads + threadIdx.x;
  const int q = 2 - gridDim.y + blockIdx.y;
  launch::wait_for_previous();
  float s = 0.0f;
  if (c < a.H) {
    const float* p = a.parts + static_cast<long long>(q) * a.H + c;
#pragma unroll 10
    for (int i = threadIdx.y; i < a.n_parts; i += kColRows)
      s += p[static_cast<long long>(i) * 2 * a.H];
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  // 32 x 32 sums: a warp per column, its lanes' by halving
  s = part[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  c = blockIdx.x * kColThreads + threadIdx.y;
  if (threadIdx.x != 0 || c >= a.H) return;
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
  return std::max(1, std::min(c.T, kMaxParts));
}

template <typename T, int NV, int MAXT>
cudaError_t launch_post(const BwdArgs& a, bool post, int grid, int threads,
                        cudaStream_t s) {
  if (post)
    block_bwd_kernel<T, NV, MAXT, true><<<grid, threads, 0, s>>>(a);
  else
    block_bwd_kernel<T, NV, MAXT, false><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

// CTAs of the streamed form: `groups` groups of `threads` threads, as many
// CTAs as fit and at most `parts`; returns their number in *grid, or 0 where
// the rows do not fit.
template <typename T, int NV, int MAXT, bool POST, int GATE, int S>
cudaError_t launch_stream(const BwdArgs& a, int parts, int threads,
                          int groups, const Device& d, int* grid,
                          cudaStream_t s) {
  const int words = (a.dh ? 2 : 0) + (a.dout ? 1 : 0) + POST +
                    (GATE == MOE_GATE_FULL);
  // the same memory takes the columns that the groups add at the end
  const int bytes =
      std::max(groups * S * words * threads * NV * 16,
               groups > 1 ? a.n16 * Vec<T>::N * static_cast<int>(sizeof(float))
                          : 0);
  *grid = 0;
  if (bytes + 1024 > d.smem_cta) return cudaSuccess;
  constexpr auto kernel = block_bwd_stream<T, NV, MAXT, POST, GATE, S>;
  int per_sm = 0;
  cudaError_t e = launch::allow_shared<kernel>(d);
  if (e == cudaSuccess)
    e = launch::ctas_per_sm<kernel>(d, threads * groups, bytes, &per_sm);
  if (e != cudaSuccess) return e;
  const int rows = (a.T + groups - 1) / groups;
  *grid = std::min({parts, rows, per_sm * d.sms});
  kernel<<<*grid, threads * groups, bytes, s>>>(a, threads);
  return cudaGetLastError();
}

template <typename T, int NV, int MAXT, int S>
cudaError_t launch_stream_post(const BwdArgs& a, bool post, int parts,
                               int* grid, cudaStream_t s) {
  Device d;
  const cudaError_t e = device(&d);
  if (e != cudaSuccess) return e;
  const int threads = ((a.n16 + NV - 1) / NV + 31) / 32 * 32;
  // groups that make a CTA of about 512 threads (a barrier for each)
  const int groups = std::max(1, std::min(8, 512 / threads));
  if (!post)
    return launch_stream<T, NV, MAXT, false, MOE_GATE_NONE, S>(
        a, parts, threads, groups, d, grid, s);
#define MOE_GATE_CASE(GATE)                                                 \
  if (a.gate_kind == GATE)                                                  \
  return launch_stream<T, NV, MAXT, true, GATE, S>(a, parts, threads,       \
                                                   groups, d, grid, s)
  MOE_GATE_CASE(MOE_GATE_NONE);
  MOE_GATE_CASE(MOE_GATE_TOKEN);
  MOE_GATE_CASE(MOE_GATE_CHANNEL);
  MOE_GATE_CASE(MOE_GATE_FULL);
#undef MOE_GATE_CASE
  return cudaErrorInvalidValue;
}

// At most `parts` CTAs; *grid receives how many partials there are.
template <typename T>
cudaError_t launch_rows(const BwdArgs& a, bool post, int parts, int* grid,
                        cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  *grid = 0;
  if (a.n16 <= 512)
    e = launch_stream_post<T, 1, 512, 3>(a, post, parts, grid, s);
  else if (a.n16 <= 1024)
    e = launch_stream_post<T, 2, 512, 3>(a, post, parts, grid, s);
  if (e != cudaSuccess || *grid > 0) return e;
  if (a.n16 <= 1280)
    e = launch_stream_post<T, 2, 640, 2>(a, post, parts, grid, s);
  if (e != cudaSuccess || *grid > 0) return e;
  *grid = parts;
  const int threads = (a.n16 + 127) / 128 * 32;
  if (a.n16 <= 2048)
    return launch_post<T, 4, 512>(a, post, parts, threads, s);
  return launch_post<T, 4, 1024>(a, post, parts, threads, s);
}

moe_status_t run(const moe_config_t& c, BwdArgs a, ColArgs ca, bool post,
                 void* workspace, cudaStream_t s) {
  a.T = c.T;
  a.n16 = row_words(c);
  a.inv_h = 1.0f / static_cast<float>(c.H);
  Carve cv(workspace);
  const int parts = parts_of(c);
  a.parts = cv.take<float>(static_cast<size_t>(parts) * 2 * c.H);
  ca.parts = a.parts;
  ca.H = c.H;
  ca.w_offset = a.w_offset;
  // Without rows there are no partials, and every column sum is zero.
  if (c.T > 0) {
    const cudaError_t e =
        c.dtype == MOE_F32
            ? launch_rows<float>(a, post, parts, &ca.n_parts, s)
            : launch_rows<__nv_bfloat16>(a, post, parts, &ca.n_parts, s);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  const dim3 cols((c.H + kColThreads - 1) / kColThreads, post ? 2 : 1);
  return launch::overlapping(block_bwd_columns, cols,
                             dim3(kColThreads, kColRows), 0, s,
                             ca) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
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
