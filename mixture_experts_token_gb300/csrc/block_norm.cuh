// Shared pieces of the block-norm kernels (block_norm.cu, forward;
// block_norm_backward.cu): 16-byte row words, column weights, the sum over
// a row, and the host-side argument checks.
#pragma once

#include <cuda_bf16.h>

#include "internal.h"
#include "launch.cuh"

namespace moe {
namespace block {

// A row is held in the registers of at most 1024 threads, 4 words each.
constexpr int kMaxRowWords = 4096;
// Rows per CTA where a warp holds a row.
constexpr int kRowWarps = 4;

struct FwdArgs {
  const int4 *x, *y, *y_sorted;  // y or (y_sorted, row_of, topk_w)
  const int32_t* row_of;
  const float* topk_w;
  const float *w_post, *w_next;
  const void* gate;
  int4 *y_out, *out, *h;
  float *rstd_y, *rstd_out;
  float inv_h, eps, w_offset, res_scale;
  int T, n16, k, gate_kind;
  bool vec_w;  // the float columns may be read 16 bytes at a time
};

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ static void load(const int4& q, float* f) {
    f[0] = __int_as_float(q.x);
    f[1] = __int_as_float(q.y);
    f[2] = __int_as_float(q.z);
    f[3] = __int_as_float(q.w);
  }
  __device__ static int4 store(const float* f) {
    return make_int4(__float_as_int(f[0]), __float_as_int(f[1]),
                     __float_as_int(f[2]), __float_as_int(f[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void load(const int4& q, float* f) {
    const int u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __int_as_float(u[i] << 16);
      f[2 * i + 1] = __int_as_float(u[i] & 0xffff0000);
    }
  }
  __device__ static int4 store(const float* f) {
    int u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const int*>(&p);
    }
    return make_int4(u[0], u[1], u[2], u[3]);
  }
};

// Rows are read and written once: they pass through without displacing the
// column weights, which every row reads again.
__device__ __forceinline__ int4 load_stream(const int4* p) {
  return __ldcs(p);
}
__device__ __forceinline__ void store_stream(int4* p, const int4& v) {
  __stcs(p, v);
}

// 16 bytes from global to shared memory, asynchronously; a lane reads back
// only what it copied itself, so waiting for its own copies is enough.
__device__ __forceinline__ uint32_t shared_address(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ int4 read16(uint32_t a) {
  int4 v;
  asm volatile("ld.shared.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

__device__ __forceinline__ void zero16(uint32_t a) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0)
               : "memory");
}

// N float column values that belong to the row's word c.
template <int N>
__device__ __forceinline__ void load_weight(const float* p, int c, bool vec,
                                            float* w) {
  p += static_cast<long long>(c) * N;
  if (vec) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(p) + i);
      w[4 * i] = q.x;
      w[4 * i + 1] = q.y;
      w[4 * i + 2] = q.z;
      w[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(p + i);
  }
}

// Sum over the threads that hold a row, in every one of them, in a fixed
// order: within a warp by halving, over warps in warp order.  `red` holds 32
// floats; sums that follow each other take different ones: nothing keeps a
// warp from writing the next sum's place while another still reads this one's.
template <bool WARP>
__device__ __forceinline__ float row_sum(float s, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (WARP) return s;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = lane < warps ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// The N column values of word c, or `other` where there are none.
template <int N>
__device__ __forceinline__ void columns_or(const float* p, int c, bool in,
                                           bool vec, float other, float* w) {
  if (p != nullptr && in) {
    load_weight<N>(p, c, vec, w);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = other;
  }
}

// The same over the `threads` (a multiple of 32) consecutive threads of
// group `group` of the CTA; `red` has a place for each warp of the CTA.
__device__ __forceinline__ float group_sum(float s, float* red, int group,
                                           int threads) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (threads == 32) return s;
  const int lane = threadIdx.x & 31, warps = threads >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = s;
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
  s = lane < warps ? red[group * warps + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// ------------------------------------------------------------- host ------
using launch::Device;
using launch::device;
inline int row_words(const moe_config_t& c) {
  return static_cast<int>(static_cast<int64_t>(c.H) * elem_bytes(c.dtype) /
                          16);
}
inline bool opt_ptr(const void* p, bool need16) {
  return p == nullptr || ok_ptr(p, need16);
}
inline bool options_ok(const moe_block_norm_t* o) {
  return o != nullptr && o->eps > 0.0f && o->eps < 1e30f &&
         o->gate_kind >= MOE_GATE_NONE && o->gate_kind <= MOE_GATE_FULL;
}
inline bool gate_ok(const moe_block_norm_t& o, const void* gate) {
  if (o.gate_kind == MOE_GATE_NONE) return gate == nullptr;
  return ok_ptr(gate, o.gate_kind == MOE_GATE_FULL);
}
// Whether the float columns in use all start on 16 bytes.
inline bool columns_aligned(const moe_block_norm_t& o, const void* w_post,
                            const void* w_next, const void* gate) {
  return aligned16(w_post) && aligned16(w_next) &&
         (o.gate_kind != MOE_GATE_CHANNEL || aligned16(gate));
}

}  // namespace block
}  // namespace moe
