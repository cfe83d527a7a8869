// The norms before and after a block, with the branch's gate and the
// residual's scale, forward.
//
//   N(v; w)[t, c] = v[t, c] * rstd_t * (w_offset + w[c]),
//   rstd_t = 1 / sqrt(mean_c v[t, c]^2 + eps)
//   out = res_scale * x + gate * N(y; w_post),   h_next = N(out; w_next)
//
// Three entry points: the norm alone (moe_norm), the branch's end
// (moe_block_out) and the branch's end with the weighted combine in front
// (moe_combine_block_out).  HBM bounds all of it, so a row is read once and
// each output written once: a row is kept on chip over both reductions.  `y`
// and `out` are rounded to the layer's type where they are stored and the
// norm that follows reads the rounded value: a backward pass that starts from
// the stored tensors then differentiates what was computed.  Sums of squares
// are float32.
//
// Measured, bf16: 8192 x 7168 with a channel gate 78 us (470 MB, 6.0 TB/s);
// 8192 x 5120 with one expert combined 81 us (420 MB, 5.2 TB/s); the norm
// alone, 8192 x 7168, 44 us (235 MB, 5.4 TB/s); one token of 7168 5.9 us a
// call, of which most is the call.  float32: 2047 x 5120 with a full gate 37 us
// (210 MB, 5.6 TB/s).
#include <cuda_bf16.h>

#include <algorithm>

#include "block_norm.cuh"

namespace moe {
namespace {

using namespace block;

enum Mode { kNormOnly = 0, kOut = 1, kCombineOut = 2 };

// Rows of up to 128 words (WARP: a warp per row, several rows per CTA), which
// leave a scheduler many short rows to choose from, and rows too wide for the
// streamed form below (over 1280 words: more than 640 threads of two words do
// not have registers for the column weights): NV 16-byte words of the row per
// thread, in registers.  One row a CTA at a time: the end of the block with a
// channel gate takes 45 us at 2048 x 7168 float32 (5.3 TB/s), 63 us at
// 2048 x 16384 bf16 (4.3) and 80 us at 1024 x 32768 bf16 (3.3); the streamed
// form 31 us at 2048 x 10240 bf16 (5.4).
template <typename T, int NV, bool WARP, int MAXT, int MODE>
__global__ void __launch_bounds__(MAXT)
    block_fwd_kernel(const FwdArgs a) {
  using V = Vec<T>;
  __shared__ float red[2][32];
  __shared__ int rows[kMaxTopK];
  __shared__ float wts[kMaxTopK];
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int step = WARP ? 32 : blockDim.x;
  const int t = WARP ? blockIdx.x * kRowWarps + (threadIdx.x >> 5)
                     : blockIdx.x;
  if (WARP && t >= a.T) return;
  const long long base = static_cast<long long>(t) * a.n16;
  int4 x[NV], y[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int c = tid + u * step;
    x[u] = y[u] = make_int4(0, 0, 0, 0);
    if (c < a.n16) {
      x[u] = load_stream(a.x + base + c);
      if (MODE == kOut) y[u] = load_stream(a.y + base + c);
    }
  }
  if (MODE == kCombineOut) {
    const long long r0 = static_cast<long long>(t) * a.k;
    if (!WARP) {
      if (tid < a.k) {
        rows[tid] = a.row_of[r0 + tid];
        wts[tid] = a.topk_w[r0 + tid];
      }
      __syncthreads();
    }
    float acc[NV][V::N];
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int i = 0; i < V::N; ++i) acc[u][i] = 0.0f;
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
      const int r = WARP ? a.row_of[r0 + j] : rows[j];
      const float w = WARP ? a.topk_w[r0 + j] : wts[j];
      if (r < 0) continue;
      const int4* src = a.y_sorted + static_cast<long long>(r) * a.n16;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const int c = tid + u * step;
        if (c < a.n16) {
          float f[V::N];
          V::load(load_stream(src + c), f);
#pragma unroll
          for (int i = 0; i < V::N; ++i) acc[u][i] = fmaf(w, f[i], acc[u][i]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = tid + u * step;
      y[u] = V::store(acc[u]);
      if (c < a.n16 && a.y_out) store_stream(a.y_out + base + c, y[u]);
    }
  }
  if (MODE != kNormOnly) {
    float r = 1.0f;
    if (a.w_post) {
      float s = 0.0f;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        float f[V::N];
        V::load(y[u], f);
#pragma unroll
        for (int i = 0; i < V::N; ++i) s = fmaf(f[i], f[i], s);
      }
      s = row_sum<WARP>(s, red[0]);
      r = rsqrtf(s * a.inv_h + a.eps);
      if (tid == 0 && a.rstd_y) a.rstd_y[t] = r;
    }
    const float gt = a.gate_kind == MOE_GATE_TOKEN
                         ? static_cast<const float*>(a.gate)[t]
                         : 1.0f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int c = tid + u * step;
      if (c >= a.n16) continue;
      float fx[V::N], fy[V::N], w[V::N];
      V::load(x[u], fx);
      V::load(y[u], fy);
      if (a.w_post) {
        load_weight<V::N>(a.w_post, c, a.vec_w, w);
#pragma unroll
        for (int i = 0; i < V::N; ++i) fy[i] *= r * (a.w_offset + w[i]);
      }
      if (a.gate_kind == MOE_GATE_CHANNEL) {
        load_weight<V::N>(static_cast<const float*>(a.gate), c, a.vec_w, w);
      } else if (a.gate_kind == MOE_GATE_FULL) {
        V::load(load_stream(static_cast<const int4*>(a.gate) + base + c), w);
      } else {
#pragma unroll
        for (int i = 0; i < V::N; ++i) w[i] = gt;
      }
#pragma unroll
      for (int i = 0; i < V::N; ++i)
        fx[i] = fmaf(w[i], fy[i], a.res_scale * fx[i]);
      x[u] = V::store(fx);
      store_stream(a.out + base + c, x[u]);
    }
  }
  if (a.w_next == nullptr) return;
  float s = 0.0f;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    float f[V::N];
    V::load(x[u], f);
#pragma unroll
    for (int i = 0; i < V::N; ++i) s = fmaf(f[i], f[i], s);
  }
  s = row_sum<WARP>(s, red[1]);
  const float r = rsqrtf(s * a.inv_h + a.eps);
  if (tid == 0 && a.rstd_out) a.rstd_out[t] = r;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int c = tid + u * step;
    if (c >= a.n16) continue;
    float f[V::N], w[V::N];
    V::load(x[u], f);
    load_weight<V::N>(a.w_next, c, a.vec_w, w);
#pragma unroll
    for (int i = 0; i < V::N; ++i) f[i] *= r * (a.w_offset + w[i]);
    store_stream(a.h + base + c, V::store(f));
  }
}

template <typename T, int NV, bool WARP, int MAXT>
cudaError_t launch_mode(const FwdArgs& a, int mode, int threads,
                        cudaStream_t s) {
  const unsigned grid =
      WARP ? (a.T + kRowWarps - 1) / kRowWarps : static_cast<unsigned>(a.T);
  if (mode == kNormOnly)
    block_fwd_kernel<T, NV, WARP, MAXT, kNormOnly><<<grid, threads, 0, s>>>(a);
  else if (mode == kOut)
    block_fwd_kernel<T, NV, WARP, MAXT, kOut><<<grid, threads, 0, s>>>(a);
  else
    block_fwd_kernel<T, NV, WARP, MAXT, kCombineOut><<<grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

// ---- rows streamed through shared memory -------------------------------
// For rows of one CTA.  A persistent CTA walks its rows with the column
// weights in registers (read once) and the rows' words in a queue in shared
// memory that runs kQueue words ahead, across rows: a row's reductions leave
// memory no pause.  A thread holds word tid of the row (and tid + blockDim.x
// with NV = 2, which halves the instructions of the reductions where a row
// has over 512 words: 7168 bf16 columns and one expert 113 -> 81 us).  A row
// is, in queue order, y (or its k expert rows), x, and a full gate.
// Words in flight: eight experts' and x, so that one row needs no second
// round trip, or four rows of two.
template <int MODE>
constexpr int kQueueOf = MODE == kCombineOut ? 10 : 8;
// Where the words of the coming rows are, for the combine: a ring of rows
// whose entries are a word's address and its weight.
struct Entry {
  const int4* src;  // null: nothing to copy
  float weight;
};
constexpr int kEntries = 144;  // four rows of 32 experts, x and a gate
constexpr int kMaxAhead = 12;  // rows that the ring runs ahead

template <typename T, int NV, int MAXT, int MODE, bool FULL>
__global__ void __launch_bounds__(MAXT) block_fwd_stream(const FwdArgs a) {
  using V = Vec<T>;
  constexpr int N = V::N;
  constexpr int kQueue = kQueueOf<MODE>;
  extern __shared__ __align__(16) char queue[];
  __shared__ float red[2][32];
  __shared__ Entry table[MODE == kCombineOut ? kEntries : 1];
  const int tid = threadIdx.x, step = blockDim.x;
  const long long row_step = static_cast<long long>(gridDim.x) * a.n16;
  const uint32_t word_bytes = step * NV * 16;
  const uint32_t first = shared_address(queue) + tid * 16;
  const uint32_t last = first + (kQueue - 1) * word_bytes;
  const bool in = NV == 1 ? tid < a.n16 : true;  // NV = 2 tests each word
  const auto held = [&](int u) {
    return NV == 1 ? in : tid + u * step < a.n16;
  };

  constexpr int kTail = 1 + (FULL ? 1 : 0);  // words after y
  const int ys = MODE == kNormOnly ? 0 : MODE == kOut ? 1 : a.k;
  const int words = ys + kTail;
  const int held_rows = min(kMaxAhead + 1, kEntries / words);
  const int ahead = held_rows - 1;
  // entry tid of the i-th row of this CTA
  const auto load_entry = [&](int i) {
    const long long t = blockIdx.x + static_cast<long long>(i) * gridDim.x;
    Entry e = {nullptr, 0.0f};
    if (tid < words && t < a.T) {
      if (tid < ys) {
        const int r = a.row_of[t * a.k + tid];
        e.weight = a.topk_w[t * a.k + tid];
        if (r >= 0) e.src = a.y_sorted + static_cast<long long>(r) * a.n16;
      } else {
        e.src = (tid == ys ? a.x : static_cast<const int4*>(a.gate)) +
                t * a.n16;
      }
    }
    return e;
  };
  const auto keep_entry = [&](int i, const Entry& e) {
    if (tid < words) table[i % held_rows * words + tid] = e;
  };
  Entry entry = {nullptr, 0.0f};  // of row i + ahead, loaded a row ago
  if (MODE == kCombineOut) {
    for (int i = 0; i < ahead; ++i) keep_entry(i, load_entry(i));
    entry = load_entry(ahead);
    __syncthreads();
  }
  const bool token = MODE != kNormOnly && !FULL &&
                     a.gate_kind == MOE_GATE_TOKEN;
  const float* gates = static_cast<const float*>(a.gate);
  float gate = token ? gates[blockIdx.x] : 0.0f;  // of the row, loaded ahead

  // --- the queue's end: the next word to copy
  const long long at0 = static_cast<long long>(blockIdx.x) * a.n16 + tid;
  const int4* xp = a.x + at0;
  const int4* yp = MODE == kOut ? a.y + at0 : nullptr;
  const int4* gp = FULL ? static_cast<const int4*>(a.gate) + at0 : nullptr;
  int copy_row = blockIdx.x, copy_word = 0;  // or the entry in the table
  uint32_t dst = first;
  const auto copy_from = [&](const int4* src) {
#pragma unroll
    for (int u = 0; u < NV; ++u)
      if (held(u)) copy16(dst + u * step * 16, src + u * step);
  };
  const auto copy = [&] {
    if (MODE == kCombineOut) {
      const int4* src = table[copy_word].src;
      if (src != nullptr) copy_from(src + tid);
      if (++copy_word == held_rows * words) copy_word = 0;
    } else if (copy_row < a.T) {
      copy_from(MODE == kOut && copy_word == 0 ? yp
                : !FULL || copy_word == ys     ? xp
                                               : gp);
      if (++copy_word == ys + kTail) {
        copy_word = 0;
        copy_row += gridDim.x;
        xp += row_step;
        if (MODE == kOut) yp += row_step;
        if (FULL) gp += row_step;
      }
    }
    copies_commit();
    dst = dst == last ? first : dst + word_bytes;
  };
  // --- its front: the next word to read, whose place is copied into again
  uint32_t src = first;
  const auto next = [&](int4 (&v)[NV]) {
    copies_wait<kQueue - 1>();
#pragma unroll
    for (int u = 0; u < NV; ++u)
      v[u] = held(u) ? read16(src + u * step * 16) : make_int4(0, 0, 0, 0);
    src = src == last ? first : src + word_bytes;
    copy();
  };
#pragma unroll 1
  for (int i = 0; i < kQueue; ++i) copy();

  // w' of the post norm (times a channel's gate) and of the next norm
  float wp[NV][N], wn[NV][N];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int c = tid + u * step;
    float wg[N];
    if (MODE != kNormOnly) {
      columns_or<N>(a.w_post, c, c < a.n16, a.vec_w, 1.0f, wp[u]);
      columns_or<N>(a.gate_kind == MOE_GATE_CHANNEL ? gates : nullptr, c,
                    c < a.n16, a.vec_w, 1.0f, wg);
    }
    columns_or<N>(a.w_next, c, c < a.n16, a.vec_w, 0.0f, wn[u]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (MODE != kNormOnly)
        wp[u][i] = wg[i] * (a.w_post ? wp[u][i] + a.w_offset : 1.0f);
      wn[u][i] += a.w_offset;
    }
  }

  int sums = 0;  // row sums so far: they alternate between two buffers
  const auto inverse_rms = [&](const float (&f)[NV][N]) {
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) s = fmaf(f[u][i], f[u][i], s);
    return rsqrtf(row_sum<false>(s, red[sums++ & 1]) * a.inv_h + a.eps);
  };
  long long base = at0;
  int at = 0;  // the row's first entry in the table
#pragma unroll 1
  for (int t = blockIdx.x, i = 0; t < a.T; t += gridDim.x, ++i) {
    float f[NV][N];  // the row that is stored, and the next norm reads
    int4 q[NV];
    if (MODE == kNormOnly) {
      next(q);
#pragma unroll
      for (int u = 0; u < NV; ++u) V::load(q[u], f[u]);
    } else {
      float y[NV][N];
      if (MODE == kOut) {
        next(q);
      } else {
#pragma unroll
        for (int u = 0; u < NV; ++u)
#pragma unroll
          for (int n = 0; n < N; ++n) y[u][n] = 0.0f;
#pragma unroll 1
        for (int j = 0; j < a.k; ++j) {
          const Entry e_j = table[at + j];
          next(q);
          if (e_j.src == nullptr) continue;
#pragma unroll
          for (int u = 0; u < NV; ++u) {
            float e[N];
            V::load(q[u], e);
#pragma unroll
            for (int n = 0; n < N; ++n)
              y[u][n] = fmaf(e_j.weight, e[n], y[u][n]);
          }
        }
#pragma unroll
        for (int u = 0; u < NV; ++u) {
          q[u] = V::store(y[u]);
          if (held(u) && a.y_out)
            store_stream(a.y_out + base + u * step, q[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < NV; ++u) V::load(q[u], y[u]);
      float r = 1.0f;
      if (a.w_post) {
        r = inverse_rms(y);
        if (tid == 0 && a.rstd_y) a.rstd_y[t] = r;
      }
      if (token) {
        r *= gate;
        const long long later = static_cast<long long>(t) + gridDim.x;
        if (later < a.T) gate = gates[later];
      }
      next(q);
#pragma unroll
      for (int u = 0; u < NV; ++u) V::load(q[u], f[u]);
      if (FULL) {
        next(q);
#pragma unroll
        for (int u = 0; u < NV; ++u) {
          float g[N];
          V::load(q[u], g);
#pragma unroll
          for (int n = 0; n < N; ++n) y[u][n] *= g[n];
        }
      }
#pragma unroll
      for (int u = 0; u < NV; ++u) {
#pragma unroll
        for (int n = 0; n < N; ++n)
          f[u][n] = fmaf(y[u][n], r * wp[u][n], a.res_scale * f[u][n]);
        const int4 o = V::store(f[u]);
        if (held(u)) store_stream(a.out + base + u * step, o);
        V::load(o, f[u]);
      }
    }
    // the routing that the queue will need; the row sums' barriers lie
    // between a table row's last reader, its writer and its next reader
    if (MODE == kCombineOut) {
      keep_entry(i + ahead, entry);
      entry = load_entry(i + ahead + 1);
      at = at + words == held_rows * words ? 0 : at + words;
    }
    if (a.w_next) {
      const float r = inverse_rms(f);
      if (tid == 0 && a.rstd_out) a.rstd_out[t] = r;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
#pragma unroll
        for (int n = 0; n < N; ++n) f[u][n] *= r * wn[u][n];
        if (held(u)) store_stream(a.h + base + u * step, V::store(f[u]));
      }
    } else if (MODE == kCombineOut && !a.w_post) {
      __syncthreads();
    }
    base += row_step;
  }
  copies_wait<0>();
}

template <typename T, int NV, int MAXT, int MODE, bool FULL>
cudaError_t launch_stream(const FwdArgs& a, cudaStream_t s) {
  Device d;
  cudaError_t e = device(&d);
  if (e != cudaSuccess) return e;
  const int threads = ((a.n16 + NV - 1) / NV + 31) / 32 * 32;
  const int bytes = kQueueOf<MODE> * threads * NV * 16;
  constexpr auto kernel = block_fwd_stream<T, NV, MAXT, MODE, FULL>;
  int per_sm = 0;
  if ((e = launch::allow_shared<kernel>(d)) != cudaSuccess ||
      (e = launch::ctas_per_sm<kernel>(d, threads, bytes, &per_sm)) !=
          cudaSuccess)
    return e;
  kernel<<<std::min(a.T, per_sm * d.sms), threads, bytes, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int NV, int MAXT>
cudaError_t launch_stream_mode(const FwdArgs& a, int mode, cudaStream_t s) {
  if (mode == kNormOnly)
    return launch_stream<T, NV, MAXT, kNormOnly, false>(a, s);
  if (a.gate_kind == MOE_GATE_FULL)
    return mode == kOut ? launch_stream<T, NV, MAXT, kOut, true>(a, s)
                        : launch_stream<T, NV, MAXT, kCombineOut, true>(a, s);
  return mode == kOut ? launch_stream<T, NV, MAXT, kOut, false>(a, s)
                      : launch_stream<T, NV, MAXT, kCombineOut, false>(a, s);
}

template <typename T>
cudaError_t launch_typed(const FwdArgs& a, int mode, cudaStream_t s) {
  constexpr int W = kRowWarps * 32;
  if (a.n16 <= 32) return launch_mode<T, 1, true, W>(a, mode, W, s);
  if (a.n16 <= 64) return launch_mode<T, 2, true, W>(a, mode, W, s);
  if (a.n16 <= 128) return launch_mode<T, 4, true, W>(a, mode, W, s);
  const auto threads = [&](int nv) {
    return ((a.n16 + nv - 1) / nv + 31) / 32 * 32;
  };
  if (a.n16 <= 512) return launch_stream_mode<T, 1, 512>(a, mode, s);
  if (a.n16 <= 1024) return launch_stream_mode<T, 2, 512>(a, mode, s);
  if (a.n16 <= 1280) return launch_stream_mode<T, 2, 640>(a, mode, s);
  if (a.n16 <= 2048)
    return launch_mode<T, 4, false, 512>(a, mode, threads(4), s);
  return launch_mode<T, 4, false, 1024>(a, mode, threads(4), s);
}

}  // namespace

cudaError_t launch_block_fwd(const moe_config_t& c, const block::FwdArgs& a,
                             int mode, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (c.dtype == MOE_F32) return launch_typed<float>(a, mode, s);
  return launch_typed<__nv_bfloat16>(a, mode, s);
}

}  // namespace moe

using namespace moe;

namespace {

// T rows of x, and the float arrays of the columns.
moe_status_t check_common(const moe_config_t* cfg,
                          const moe_block_norm_t* opt) {
  const moe_status_t st = moe_validate_config(cfg);
  if (st != MOE_OK) return st;
  if (!block::options_ok(opt)) return MOE_ERR_INVALID_ARG;
  if (block::row_words(*cfg) > block::kMaxRowWords)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

block::FwdArgs common_args(const moe_config_t& c, const moe_block_norm_t& o) {
  block::FwdArgs a = {};
  a.T = c.T;
  a.n16 = block::row_words(c);
  a.k = c.k;
  a.inv_h = 1.0f / static_cast<float>(c.H);
  a.eps = o.eps;
  a.w_offset = o.w_offset;
  a.res_scale = o.res_scale;
  a.gate_kind = o.gate_kind;
  return a;
}

moe_status_t block_out(const moe_config_t* cfg, const moe_block_norm_t* opt,
                       block::FwdArgs a, int mode, const void* x,
                       const float* w_post, const void* gate,
                       const float* w_next, void* out, void* h_next,
                       float* rstd_y, float* rstd_out, cudaStream_t s) {
  if (!ok_ptr(x, true) || !ok_ptr(out, true) ||
      !block::opt_ptr(w_post, false) || !block::opt_ptr(w_next, false) ||
      !block::gate_ok(*opt, gate) || !block::opt_ptr(rstd_y, false) ||
      !block::opt_ptr(rstd_out, false) ||
      (w_next != nullptr && !ok_ptr(h_next, true)))
    return MOE_ERR_INVALID_ARG;
  a.x = static_cast<const int4*>(x);
  a.w_post = w_post;
  a.w_next = w_next;
  a.gate = gate;
  a.out = static_cast<int4*>(out);
  a.h = static_cast<int4*>(h_next);
  a.rstd_y = rstd_y;
  a.rstd_out = rstd_out;
  a.vec_w = block::columns_aligned(*opt, w_post, w_next, gate);
  return launch_block_fwd(*cfg, a, mode, s) == cudaSuccess ? MOE_OK
                                                           : MOE_ERR_CUDA;
}

}  // namespace

extern "C" {

moe_status_t moe_norm(const moe_config_t* cfg, const moe_block_norm_t* opt,
                      const void* x, const float* w, void* h, float* rstd,
                      moe_stream_t stream) {
  const moe_status_t st = check_common(cfg, opt);
  if (st != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;
  if (!ok_ptr(x, true) || !ok_ptr(w, false) || !ok_ptr(h, true) ||
      !block::opt_ptr(rstd, false))
    return MOE_ERR_INVALID_ARG;
  block::FwdArgs a = common_args(*cfg, *opt);
  a.x = static_cast<const int4*>(x);
  a.w_next = w;
  a.h = static_cast<int4*>(h);
  a.rstd_out = rstd;
  a.vec_w = aligned16(w);
  return launch_block_fwd(*cfg, a, kNormOnly, stream) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status_t moe_block_out(const moe_config_t* cfg,
                           const moe_block_norm_t* opt, const void* x,
                           const void* y, const float* w_post,
                           const void* gate, const float* w_next, void* out,
                           void* h_next, float* rstd_y, float* rstd_out,
                           moe_stream_t stream) {
  const moe_status_t st = check_common(cfg, opt);
  if (st != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;
  if (!ok_ptr(y, true)) return MOE_ERR_INVALID_ARG;
  block::FwdArgs a = common_args(*cfg, *opt);
  a.y = static_cast<const int4*>(y);
  return block_out(cfg, opt, a, kOut, x, w_post, gate, w_next, out, h_next,
                   rstd_y, rstd_out, stream);
}

moe_status_t moe_combine_block_out(
    const moe_config_t* cfg, const moe_block_norm_t* opt,
    const void* y_sorted, const int32_t* row_of, const float* topk_w,
    const void* x, const float* w_post, const void* gate,
    const float* w_next, void* y, void* out, void* h_next, float* rstd_y,
    float* rstd_out, moe_stream_t stream) {
  const moe_status_t st = check_common(cfg, opt);
  if (st != MOE_OK) return st;
  if (cfg->T == 0) return MOE_OK;
  if (!ok_ptr(y_sorted, true) || !ok_ptr(row_of, false) ||
      !ok_ptr(topk_w, false) || !block::opt_ptr(y, true))
    return MOE_ERR_INVALID_ARG;
  block::FwdArgs a = common_args(*cfg, *opt);
  a.y_sorted = static_cast<const int4*>(y_sorted);
  a.row_of = row_of;
  a.topk_w = topk_w;
  a.y_out = static_cast<int4*>(y);
  return block_out(cfg, opt, a, kCombineOut, x, w_post, gate, w_next, out,
                   h_next, rstd_y, rstd_out, stream);
}

}  // extern "C"
